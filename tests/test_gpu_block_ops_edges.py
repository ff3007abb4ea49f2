"""The operators around the routed layer at the ends of their range, on the GPU against the fp64 oracle.

Where a test compares codes or results for equality, the operator's definition leaves no room: codes are the roundings of
the exact numbers, and the sums of the closed forms fit the 24 bits of fp32."""
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from tests.test_gpu_block_ops import (DEV, DTS, MFMA, WORK, check_route, elements, f64, half_step, operand, q, rand,  # noqa: F401
                                      subnormal)

pytestmark = pytest.mark.gpu


# ---- SwiGLU ------------------------------------------------------------------------------------------------------
def swiglu_in_fp32(x):
    """silu(g) u of the fp64 rows x, infinite where fp32 does not hold it."""
    with np.errstate(over="ignore", invalid="ignore"):
        d = O.swiglu(x)
        return np.where(np.isinf(d.astype(np.float32)), np.sign(d) * np.inf, d)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu_overflow_makes_its_block_nan(q, fmt, dtype):
    """Products past fp32's largest number, infinities and NaN in either half; the last row's product stays below."""
    x = torch.ones(8, 256, dtype=dtype)
    x[0, 3], x[0, 131] = 1e20, 1e20
    x[1, 40], x[1, 168] = 1e30, -1e30
    x[2, 70], x[2, 198] = 100.0, 1e38
    x[3, 5] = math.inf
    x[4, 133] = -math.inf
    x[5, 33] = math.nan
    x[6, 100] = -math.inf
    x[7, 0], x[7, 128] = 2.0, 1.5e38
    codes, scales = elements(q.mx_swiglu_quantize(x.to(DEV), fmt))
    want_c, want_s = O.mx_quantize(swiglu_in_fp32(x.double().numpy()), fmt)
    assert [tuple(np.flatnonzero(r == 255)) for r in want_s] == [(0,), (1,), (2,), (0,), (0,), (1,), (3,), ()]
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("dtype", DTS)
def test_swiglu_of_vanishing_gates_and_large_ups(q, fmt, dtype):
    """silu down to 2^-190 and below, times up values of up to 2^120 (fp16: 2^13): also where silu alone is subnormal or 0."""
    g = torch.Generator().manual_seed(1)
    gate = -80 - 60 * torch.rand(256, 2048, generator=g)
    gate[::4] = torch.randn(64, 2048, generator=g) * 2.0 ** -130
    top = 13 if dtype == torch.float16 else 120
    up = torch.randn(256, 2048, generator=g) * torch.exp2(top * torch.rand(256, 64, generator=g)).repeat_interleave(32, 1)
    x = torch.cat((gate, up), 1).to(dtype)
    codes, scales = elements(q.mx_swiglu_quantize(x.to(DEV), fmt))
    want_c, want_s = O.mx_quantize(O.swiglu(x.double().numpy()), fmt)
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu_of_subnormal_products(q, fmt, dtype):
    g = torch.Generator().manual_seed(2)
    gate = torch.randn(128, 4096, generator=g)
    x = torch.cat((gate, torch.randn(128, 4096, generator=g) * 2.0 ** -131), 1).to(dtype)
    codes, scales = elements(q.mx_swiglu_quantize(x.to(DEV), fmt))
    want_c, want_s = O.mx_quantize(O.swiglu(x.double().numpy()), fmt)
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)


@pytest.mark.parametrize("fmt", [1, 2])
def test_swiglu_codes_next_to_borders(q, fmt):
    """Up values that put every product within 2^-22 of a border between two elements, for gates from -200 to 200."""
    g = torch.Generator().manual_seed(9)
    rows, cols = 48, 4096
    gate = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float())
    gate[::3] = 400 * torch.rand(rows // 3, cols, generator=g) - 200
    gate[1::3, ::5] = -78 - 12 * torch.rand(rows // 3, len(range(0, cols, 5)), generator=g)
    gate = torch.where(gate.abs() < 2.0 ** -20, torch.ones(()), gate)
    silu = gate.double() / (1 + torch.exp(-gate.double()))
    # halfway between elements of the two octaves below the largest, which stays clear of borders
    table = torch.from_numpy(O.TABLE[fmt])
    mid = ((table[1:] + table[:-1]) / 2)[-17 if fmt == 2 else -5:-1]
    y = mid[torch.randint(0, len(mid), (rows, cols), generator=g)]
    y[:, ::32] = float(table[-1]) * 0.98
    up = (y / silu).clamp(-3e38, 3e38).float() * (1 + torch.randint(-2, 3, (rows, cols), generator=g) * 2.0 ** -23)
    x = torch.cat((gate, up.float()), 1)
    codes, scales = elements(q.mx_swiglu_quantize(x.to(DEV), fmt))
    want_c, want_s = O.mx_quantize(O.swiglu(x.double().numpy()), fmt)
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)


def test_swiglu_repeats_itself(q):
    x = rand((2048, 4096), 21, torch.float16, 3.0)
    a = q.mx_swiglu_quantize(x, 2)
    codes, scales = a.codes.clone(), a.scales.clone()
    for _ in range(5):
        b = q.mx_swiglu_quantize(x, 2)
        assert torch.equal(b.codes, codes) and torch.equal(b.scales, scales)


# ---- products of 8-bit rows --------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("m", [1, 20, 32, 33, 40, 300, 2100])
def test_gemm_keeps_small_elements_in_every_type(q, m, dtype):
    """8-bit elements of 2^-9 next to 256 and -256, whose products cancel: the sums fit 24 bits, so y is their rounding,
    by either side of the kernels' 32-row border."""
    g = torch.Generator(device=DEV).manual_seed(m)
    k, n = 384, 80
    a = torch.randint(-7, 8, (m, k), generator=g, device=DEV).float() * 2.0 ** -9
    a[:, ::8] = 256.0
    a[:, 8::16] = -256.0
    w = torch.randint(-1, 2, (n, k), generator=g, device=DEV).float()
    w[:, 0::8] = 6.0                               # scales of 1
    qa, qw = q.mx_quantize(a, 2), q.mx_quantize(w, 1)
    assert torch.equal(qa.dequantize(), a) and torch.equal(qw.dequantize(), w)
    want = (a.double() @ w.double().T).float()
    assert torch.equal(q.mx_gemm(qa, qw, out_dtype=dtype), want.to(dtype))


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("m,n,k", [(33, 257, 640), (200, 130, 2048), (600, 1030, 1500), (2050, 2050, 512)])
def test_gemm_of_8_bit_rows_loses_no_product(q, m, n, k, dtype):
    """The bound of an fp32 sum and one rounding, with nothing for cut products; rows with elements twenty times the rest."""
    x = rand((m, k), 3)
    x[:, ::29] *= 20.0
    a, w = q.mx_quantize(x, 2), operand(q, n, k, 1, 4)
    y = q.mx_gemm(a, w, out_dtype=dtype).double()
    A, W = a.dequantize().double(), w.dequantize().double()
    want, size = A @ W.T, A.abs() @ W.abs().T
    err = (y - want).abs()
    assert (err <= half_step(dtype) * want.abs() + MFMA * size * (1 + half_step(dtype)) + subnormal(dtype)).all()


def cornered(m, n, k):
    """Operands of zeros whose blocks have scales of 1, set by a 448 of a and a 6 of w that meet zeros."""
    a, w = torch.zeros(m, k, device=DEV), torch.zeros(n, k, device=DEV)
    a[:, 31::32], w[:, 30::32] = 448.0, 6.0
    return a, w


def assert_exact_product(q, a, w):
    qa, qw = q.mx_quantize(a, 2), q.mx_quantize(w, 1)
    assert torch.equal(qa.dequantize(), a) and torch.equal(qw.dequantize(), w)
    assert torch.equal(q.mx_gemm(qa, qw, out_dtype=torch.float32).double(), a.double() @ w.double().T)


@pytest.mark.parametrize("m", [1, 20, 40, 300])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("large,small,by", [(3.75, 2.0 ** -9, 0.5), (3.75, 3 * 2.0 ** -9, 0.5), (3.75, 13 * 2.0 ** -9, 1.5),
                                            (3.5, 5 * 2.0 ** -9, 0.5), (2.0, 2.0 ** -9, 0.5), (448.0, 4.5, 0.5),
                                            (448.0, 4.5, 1.5), (448.0, 5.0, 0.5), (416.0, 4.5, 0.5)])
def test_gemm_split_keeps_products_whole(q, m, sign, large, small, by):
    """The largest product of either part of an 8-bit operand, times 6 with a carry, next to the smallest of the same part in
    the same eight columns: the sums fit 24 bits, so any cut shows."""
    a, w = cornered(m, 64, 128)
    for b in range(0, 128, 32):
        a[:, b], w[:, b] = sign * large, 6.0
        a[:, b + 1:b + 8] = small * torch.tensor([1, 1, 0, 1, 1, 0, 1.0], device=DEV)
        w[:, b + 1:b + 8] = by
    assert_exact_product(q, a, w)


@pytest.mark.parametrize("m", [4, 30, 64, 1000])
def test_gemm_of_any_four_products_is_exact(q, m):
    """Four elements of one eight, any of either format: their sum fits 24 bits."""
    g = torch.Generator().manual_seed(m)
    a, w = cornered(m, 512, 128)
    sign = lambda *shape: 1 - 2 * torch.randint(0, 2, shape, generator=g)    # noqa: E731
    four = torch.zeros(m, 8).scatter_(1, torch.rand(m, 8, generator=g).argsort(1)[:, :4], 1.0)
    a[:, :8] = (torch.from_numpy(O.E4M3).float()[torch.randint(0, 127, (m, 8), generator=g)] * four * sign(m, 8)).to(DEV)
    w[:, :8] = (torch.from_numpy(O.E2M1).float()[torch.randint(0, 8, (512, 8), generator=g)] * sign(512, 8)).to(DEV)
    assert_exact_product(q, a, w)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("m", [4, 64])
def test_gemm_of_subnormal_results(q, fmt, m):
    a, w = q.mx_quantize(rand((m, 128), 3) * 2.0 ** -68, fmt), q.mx_quantize(rand((64, 128), 4) * 2.0 ** -68, 1)
    y = q.mx_gemm(a, w, out_dtype=torch.float32).double()
    A, W = a.dequantize().double(), w.dequantize().double()
    # each of the two parts' eights may round to 2^-149
    assert ((y - A @ W.T).abs() <= MFMA * (A.abs() @ W.abs().T) + 32 * 2.0 ** -150).all()


@pytest.mark.parametrize("fmt", [1, 2])
def test_gemm_of_more_rows_than_a_launch_takes(q, fmt):
    """2^19 rows and a few: the second launch starts at its own rows of a, add and y."""
    m, n, k = (1 << 19) + 17, 40, 160
    a, w, c = operand(q, m, k, fmt, 1), operand(q, n, k, 1, 2), rand((m, n + 3), 3, torch.float16)[:, 1:1 + n]
    y = q.mx_gemm(a, w, add=c)
    A, W = a.dequantize().double(), w.dequantize().double()
    want, size = A @ W.T + c.double(), A.abs() @ W.abs().T + c.double().abs()
    t = half_step(torch.float16)
    assert ((y.double() - want).abs() <= t * want.abs() + MFMA * size * (1 + t) + subnormal(torch.float16)).all()


def test_gemm_of_interleaved_rows(q):
    """add and y in one buffer whose rows do not meet, of one stride or two: nothing is refused, and nothing else written."""
    rng = np.random.default_rng(3)
    done = 0
    while done < 60:
        m, n = int(rng.integers(1, 50)), int(rng.integers(1, 40))
        sx, sy = (int(v) for v in rng.integers(n, 3 * n + 8, 2))
        sy = sx if rng.random() < 0.6 else sy
        at = int(rng.integers(0, 4 * n + 8))
        x = np.arange(m)[:, None] * sx + np.arange(n)
        y = at + np.arange(m)[:, None] * sy + np.arange(n)
        if np.intersect1d(x, y).size:
            continue
        done += 1
        buf = rand((50 * 130 + 400,), done, torch.float16)
        a, w = operand(q, m, 200, 1 + done % 2, 1), operand(q, n, 200, 1, 2)
        add, out = buf.as_strided((m, n), (sx, 1)), buf.as_strided((m, n), (sy, 1), at)
        want, kept = q.mx_gemm(a, w, add=add.clone()), buf.clone()
        q.mx_gemm(a, w, add=add, out=out)
        kept.as_strided((m, n), (sy, 1), at).copy_(want)
        assert torch.equal(buf, kept), (m, n, sx, sy, at)


def test_norm_of_rows_around_its_outputs(q):
    """Outputs in the gap between the rows of x."""
    buf = rand((2, 4000), 1, torch.float16)
    x, flat = buf[:, :300], buf.view(-1)
    want = q.add_rms_norm(x.clone(), None, residual=x.clone(), mx_fmt=2)
    y, s = flat[300:900].view(2, 300), flat[1000:1600].view(2, 300)
    got = q.add_rms_norm(x, None, residual=x, out=y, sum_out=s, mx_fmt=2)
    assert torch.equal(y, want[0]) and torch.equal(s, want[1]) and torch.equal(got[2].codes, want[2].codes)


# ---- norm --------------------------------------------------------------------------------------------------------
def check_norm(q, x, w, fmt, eps=0.0):
    """y and, with fmt, the codes of the exact numbers; what fp32 does not hold is infinite, and its block NaN."""
    y, _, mx = q.add_rms_norm(x, w, eps=eps, out_dtype=torch.float32, mx_fmt=fmt)
    exact = O.rms_norm(f64(x), f64(w), float(np.float32(eps)))
    with np.errstate(over="ignore"):
        near = exact.astype(np.float32).astype(np.float64)
    held = np.isfinite(near)
    assert np.array_equal(f64(y)[~held], near[~held])
    err = np.abs(f64(y) - exact)[held]
    assert (err <= (half_step(torch.float32) + WORK) * np.abs(exact[held]) + subnormal(torch.float32)).all()
    if fmt:
        want_c, want_s = O.mx_quantize(np.where(held, exact, near), fmt)
        codes, scales = elements(mx)
        assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)
    return held


@pytest.mark.parametrize("fmt", [None, 1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_overflow_makes_its_block_nan(q, fmt, dtype):
    x = rand((6, 96), 1, dtype, 1e-9)
    w = (rand((96,), 2).double() * 1e38).clamp(-3e38, 3e38).float()
    held = check_norm(q, x, w, fmt)
    assert held.any() and not held.all()


@pytest.mark.parametrize("fmt", [None, 1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale,weight,cols", [(1e16, 1e23, 64), (1e16, 1e22, 100), (1e-9, 1e-31, 96), (1e-9, 1e-37, 33),
                                               (1.0, 1e38, 64), (1.0, 3e38, 64), (1.0, 1e-38, 64), (1e10, 1e-38, 520),
                                               (1e18, 1.0, 64), (1e-30, 1.0, 64), (1e-30, 1e30, 64)])
def test_norm_of_extreme_rows_and_weights(q, fmt, dtype, scale, weight, cols):
    """Products of a row and its weights that pass fp32's ends where the result does not, subnormal results, and rows that go
    by 64 bits; zeros among them."""
    x, w = rand((40, cols), 1, dtype, scale), (rand((cols,), 2).double() * weight).clamp(-3e38, 3e38).float()
    x[:, 5], w[7] = 0, 0
    check_norm(q, x, w, fmt)


@pytest.mark.parametrize("fmt", [None, 1, 2])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("rows", [3, 600])
def test_norm_of_weights_extreme_in_places(q, fmt, dtype, rows):
    """Eights of columns that go by 64 bits next to ordinary ones of the same blocks."""
    x, w = rand((rows, 1000), 1, dtype), rand((1000,), 2)
    for first, by in ((8, 1e-37), (40, 1e37), (203, 0.0), (320, 1e-30), (701, 1e-33)):
        w[first:first + 8] *= by
    check_norm(q, x, w, fmt, eps=1e-6)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [4096, 16384])
def test_norm_codes_next_to_borders(q, fmt, dtype, cols):
    """Weights that put every result within 2^-22 of a border between two elements, in rows of one large number and seven small
    ones each eight, whose squares a sum in 32 bits would lose."""
    g = torch.Generator().manual_seed(cols)
    x = torch.rand(cols, generator=g, dtype=torch.float64) * 0.2 + 0.9
    x[::8] = x[::8] * 1.5
    small = torch.ones(cols, dtype=torch.bool)
    small[::8] = False
    x = (torch.where(small, x * 2.0 ** -12.4, x) * (1 - 2 * torch.randint(0, 2, (cols,), generator=g))).to(dtype)
    rms = math.sqrt(float((x.double() ** 2).mean()) + 1e-6)
    # halfway between elements of the two octaves below the largest, which stays clear of borders
    table = torch.from_numpy(O.TABLE[fmt])
    mid = ((table[1:] + table[:-1]) / 2)[-17 if fmt == 2 else -5:-1]
    y = mid[torch.randint(0, len(mid), (cols,), generator=g)]
    y[::32] = float(table[-1]) * 0.98
    w = (y * rms / x.double()).float()
    w = w * (1 + torch.randint(-2, 3, (cols,), generator=g) * 2.0 ** -23)
    _, _, mx = q.add_rms_norm(x[None].to(DEV), w.float().to(DEV), eps=1e-6, mx_fmt=fmt)
    exact = O.rms_norm(x[None].double().numpy(), w.double().numpy(), float(np.float32(1e-6)))
    want_c, want_s = O.mx_quantize(exact, fmt)
    codes, scales = elements(mx)
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)


# ---- routing -----------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_route_of_more_tokens_than_a_grid_takes(q, dtype):
    """2^26 tokens and a few, in several launches: the tokens at their ends are those of a small call."""
    T = (1 << 26) + 11
    lg = torch.randint(-8, 8, (T, 3), dtype=torch.int8, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(dtype)
    idx, w = q.route_scored(lg, 2, score="sigmoid")
    pick = torch.tensor([0, 1, (1 << 22) - 1, 1 << 22, (1 << 25) + 3, (1 << 26) - 1, 1 << 26, T - 1], device=DEV)
    want_i, want_w = q.route_scored(lg[pick], 2, score="sigmoid")
    assert torch.equal(idx[pick], want_i) and torch.equal(w[pick], want_w)
    assert (idx >= 0).all() and (w.sum(1) - 1).abs().max() <= 2.0 ** -22


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("spread", [2.0 ** -14, 2.0 ** -17, 2.0 ** -18, 2.0 ** -19, 2.0 ** -21, 2.0 ** -24])
def test_route_of_sums_within_the_margins(q, score, spread):
    """Biases that bring all sums within `spread` of each other, around the margins that 32 bits are trusted with: the choice is
    that of 64 bits, with groups and without."""
    g = torch.Generator().manual_seed(11)
    for E, G, keep in ((256, 1, 1), (256, 8, 3), (96, 4, 2)):
        for _ in range(6):
            lg = 3 * torch.randn(1, E, generator=g)
            s = torch.softmax(lg.double(), 1) if score == "softmax" else torch.sigmoid(lg.double())
            bias = (1 - s[0] + spread * torch.randn(E, generator=g).double()).float().to(DEV)
            for rule in ("max", "top2"):
                check_route(q, lg.to(DEV), 8, score=score, bias=bias, n_groups=G, keep_groups=keep, group_score=rule)


# ---- the routed layer with slots that have no expert ------------------------------------------------------------
@pytest.fixture(scope="module")
def two_tables(q):
    """The same experts twice; in the second table every number of expert 0 is NaN."""
    from synth import config_seed, gen_matrices
    seed = config_seed(72)
    H, I, E = 2048, 1024, 12
    up = gen_matrices(seed, [(e, m) for e in range(E) for m in (0, 1)], I, H, device=torch.device(DEV))
    down = gen_matrices(seed, [(e, 2) for e in range(E)], H, I, device=torch.device(DEV))
    packed = [(q.pack_matrix(up[2 * e]), q.pack_matrix(up[2 * e + 1]), q.pack_matrix(down[e])) for e in range(E)]
    for m in (up[0], up[1], down[0]):
        m.block_scales.fill_(0x7E00)
    bad = tuple(q.pack_matrix(m) for m in (up[0], up[1], down[0]))
    return H, I, E, q.expert_table(packed), q.expert_table([bad] + packed[1:])


def paths(q, T):
    """Flags of every path of the layer that takes T tokens."""
    flags = [0, q.GALE_PATH_GROUPED]
    return flags + [q.GALE_DECODE_STAGED, q.GALE_PATH_DECODE] if T <= 64 else flags


@pytest.mark.parametrize("T", [1, 3, 64, 100, 700])
@pytest.mark.parametrize("k", [1, 4, 8])
def test_given_slots_without_an_expert_add_nothing(q, two_tables, T, k):
    """No bit of y hangs on expert 0 where no slot names it, even if all its numbers are NaN; tokens without any expert are
    zero, and the weight of an empty slot does not matter."""
    H, I, E, good, bad = two_tables
    g = torch.Generator().manual_seed(100 * T + k)
    idx = 1 + torch.rand(T, E - 1, generator=g).argsort(1)[:, :k].int()
    idx[torch.rand(T, k, generator=g) < 0.4] = -1
    idx[T // 2] = -1 if T > 1 else idx[T // 2]
    w = torch.rand(T, k, generator=g)
    x = rand((T, H), 5, torch.float16)
    for flags in paths(q, T):
        for choice in (idx, torch.full_like(idx, -1)):
            i = choice.to(DEV)
            y = q.moe_layer_fwd_given(good, H, I, i, w.to(DEV), x, flags=flags)
            assert y.isfinite().all() and (y[(i < 0).all(1)] == 0).all()
            assert torch.equal(q.moe_layer_fwd_given(bad, H, I, i, w.to(DEV), x, flags=flags), y)
            odd = torch.where(i < 0, torch.full_like(i, 3).float() * math.nan, w.to(DEV))
            assert torch.equal(q.moe_layer_fwd_given(bad, H, I, i, odd, x, flags=flags), y)


@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_given_empty_slots_are_as_if_absent(q, two_tables, T):
    """With one column of slots empty for every token, y is that of the call without this column."""
    H, I, E, good, _ = two_tables
    idx = torch.rand(T, E, generator=torch.Generator().manual_seed(T)).argsort(1)[:, :4].int().to(DEV)
    w, x = torch.rand(T, 4, device=DEV), rand((T, H), 6, torch.float16)
    for flags in paths(q, T):
        for c in range(4):
            rest = [j for j in range(4) if j != c]
            holed = idx.clone()
            holed[:, c] = -1
            y = q.moe_layer_fwd_given(good, H, I, holed, w, x, flags=flags)
            want = q.moe_layer_fwd_given(good, H, I, idx[:, rest].contiguous(), w[:, rest].contiguous(), x, flags=flags)
            assert torch.equal(y, want), (flags, c)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_masked_tokens_through_router_and_layer(q, two_tables, T):
    """Tokens whose logits leave nothing, or fewer experts than slots, go from the router into the layer: the first are
    zero, and the others' empty slots add nothing."""
    H, I, E, good, bad = two_tables
    lg = rand((T, E), 7)
    lg[:, 0] = -math.inf                           # expert 0, whose numbers are NaN in `bad`, is masked
    lg[0] = -math.inf
    if T > 1:
        lg[1, 2:] = -math.inf                      # one expert
        lg[2, 5:] = math.nan                       # four
    idx, w = q.route_scored(lg, 6, score="sigmoid", n_groups=2, keep_groups=2)
    assert (idx[0] == -1).all()
    x = rand((T, H), 8, torch.float16)
    y = q.moe_layer_fwd_given(good, H, I, idx, w, x)
    assert (y[0] == 0).all() and y.isfinite().all()
    assert torch.equal(q.moe_layer_fwd_given(bad, H, I, idx, w, x), y)
    if T > 1:
        assert (idx[1] == torch.tensor([1, -1, -1, -1, -1, -1], device=DEV)).all() and (y[1] != 0).any()
