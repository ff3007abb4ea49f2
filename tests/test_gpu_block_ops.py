"""The operators around the routed layer on the GPU against the fp64 oracle.

Tolerances, derived from the arithmetic:
  * MX quantisation: exact (codes and scales equal the oracle's).
  * fp32 work (norm, SwiGLU): WORK = 2^-18 relative.  A sum of squares of up to 16,384 terms runs in chains of at most
    32 additions and ten tree levels, each off by at most 2^-24 of a sum of positive terms; the square root halves that;
    the divisions, products and the exponential add a few 2^-24 each, below 2^-18 together.
  * a rounding to type t: half a step, finfo(t).eps / 2 relative, plus half the smallest subnormal.
  * products: the MFMA carries 2^-18 of a 128-column group's sum of |products| (measured for the GEMV's closed forms),
    so the sum over all groups is within 2^-18 of the row's sum of |products|; closed forms whose sums fit 24 bits are
    exact.
    With 8-bit activations and a 16-bit result the instruction cuts the products of each eight consecutive columns to
    multiples of 2^(e - 13), e the exponent of the largest of them (measured with constructed operands; it is never cut
    itself, having four significant bits): at most seven cuts below 2^(e - 13) <= 2^-13 max |a| max |w| each.
  * weights of the router: computed in 64 bits and rounded once, 2^-24 relative, 2^-23 allowed.
"""
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTS = [torch.float16, torch.bfloat16, torch.float32]
WORK = 2.0 ** -18
MFMA = 2.0 ** -18


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_expert_gemv_amd as qq
    qq.lib()
    return qq


def rand(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(t):
    return torch.finfo(t).eps / 2


def subnormal(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def elements(mx):
    return O.mx_elements(mx.codes.cpu().numpy(), mx.fmt), mx.scales.cpu().numpy().astype(np.int64)


def assert_mx_of(mx, exact, work=WORK):
    """mx is the quantisation of numbers within `work` of exact: the scale fits their largest magnitude, the elements
    are within half a step of them, and what lies behind the columns is zero."""
    codes, scales = elements(mx)
    cols = mx.cols
    table = O.TABLE[mx.fmt]
    assert not codes[:, cols:].any() and not scales[:, -(-cols // 32):].any()
    pad = np.pad(exact, ((0, 0), (0, codes.shape[1] - cols))).reshape(len(exact), -1, 32)
    top = np.abs(pad).max(axis=2)
    unit = 2.0 ** (scales - 127.0)
    assert (top <= table[-1] * unit * (1 + work)).all()
    assert ((top >= table[-1] / 2 * unit * (1 - work)) | (scales == 0)).all()
    a = np.minimum(np.abs(pad) / unit[..., None], table[-1])
    i = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    step = table[i] - table[i - 1]
    v = O.mx_values(codes, scales, mx.fmt, codes.shape[1]).reshape(pad.shape)
    # a number next to a border of two step sizes may round with the larger one
    bound = unit[..., None] * step * (0.5 + 2 * work * table[-1]) + work * np.abs(pad)
    assert (np.abs(v - pad) <= bound).all()


# ---- MX numbers --------------------------------------------------------------------------------------------------
def hard_rows(rows, cols, dtype, seed):
    """Numbers of many magnitudes, ties of both formats, blocks of zeros and of one number."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    x *= 2.0 ** torch.randint(-12, 13, (rows, -(-cols // 32)), generator=g).repeat_interleave(32, 1)[:, :cols]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 17.0, 19.0, 6.5, 7.5], dtype=torch.float64)
    x[0] = ties[torch.randint(0, len(ties), (cols,), generator=g)] * (1 - 2 * torch.randint(0, 2, (cols,), generator=g))
    if rows > 1:
        x[1] = 0
        x[1, 0] = -1.5
    if rows > 2:
        x[2] *= 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -130
    return x.to(dtype)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 32), (4, 33), (2, 127), (9, 128), (3, 131), (17, 520), (3, 4096)])
def test_quantize_is_exact(q, fmt, dtype, rows, cols):
    x = hard_rows(rows, cols, dtype, 100 + cols)
    want_c, want_s = O.mx_quantize(x.double().numpy(), fmt)
    mx = q.mx_quantize(x.to(DEV), fmt)
    got_c, got_s = elements(mx)
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(got_c, want_c)
    for t in DTS:
        y = q.mx_dequantize(mx, t)
        want = torch.from_numpy(O.mx_values(want_c, want_s, fmt, cols)).to(t)
        assert torch.equal(y.cpu(), want), t


@pytest.mark.parametrize("fmt", [1, 2])
def test_quantize_special_values(q, fmt):
    """Infinities and NaN make their own block NaN and no other; the ends of the fp32 range scale without overflow."""
    x = torch.ones(4, 160)
    x[0, 3], x[1, 40], x[2, 159] = math.inf, math.nan, -math.inf
    x[3, :32] = torch.finfo(torch.float32).max
    x[3, 32:64] = 2.0 ** -149
    x[3, 64:96] = 2.0 ** -126
    mx = q.mx_quantize(x.to(DEV), fmt)
    codes, scales = elements(mx)
    assert [tuple(np.flatnonzero(r == 255)) for r in scales] == [(0,), (1,), (4,), ()]
    assert not codes[0, :32].any() and not codes[1, 32:64].any()
    y = mx.dequantize().cpu()
    bad = torch.zeros(4, 160, dtype=torch.bool)
    bad[0, :32] = bad[1, 32:64] = bad[2, 128:] = True
    assert torch.equal(y.isnan(), bad)
    want = O.mx_values(*O.mx_quantize(x[3:].double().numpy(), fmt), fmt, 160)
    assert torch.equal(y[3:], torch.from_numpy(want).float())


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("offset,stride", [(0, 200), (1, 200), (3, 133), (0, 136)])
def test_quantize_strided_rows(q, dtype, offset, stride):
    base = rand((7, stride + offset), 5, dtype)
    x = base.as_strided((6, 131), (stride, 1), offset)
    want = q.mx_quantize(x.contiguous().clone(), 1)
    got = q.mx_quantize(x, 1)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    out = torch.full((6, stride), 7.0, dtype=dtype, device=DEV)
    q.mx_dequantize(want, dtype, out=out[:, :131])
    assert torch.equal(out[:, :131], q.mx_dequantize(want, dtype)) and (out[:, 131:] == 7).all()


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 130), (2, 2048)])
def test_swiglu_quantize(q, fmt, dtype, rows, cols):
    x = rand((rows, 2 * cols), 11 + cols, dtype, 4.0)
    x[0, 0] = -90.0          # silu vanishes without overflowing
    mx = q.mx_swiglu_quantize(x, fmt)
    assert_mx_of(mx, O.swiglu(f64(x)))


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("dtype", DTS)
def test_swiglu_codes_are_those_of_64_bits(q, fmt, dtype):
    """400,000 elements: about 25 of them lie within the 32-bit arithmetic's error of a border, and take the 64-bit side."""
    x = rand((200, 4096), 21, dtype, 3.0)
    codes, scales = elements(q.mx_swiglu_quantize(x, fmt))
    want_c, want_s = O.mx_quantize(O.swiglu(f64(x)), fmt)
    assert np.array_equal(scales, want_s) and np.array_equal(codes, want_c)


def test_quantize_past_2_31_elements(q):
    rows, cols = 33000, 65536                      # 2.16e9 fp16 numbers
    x = torch.zeros(rows, cols, dtype=torch.float16, device=DEV)
    tail = rand((2, cols), 3, torch.float16)
    x[-2:] = tail
    mx = q.mx_quantize(x, 1)
    want = q.mx_quantize(tail, 1)
    assert torch.equal(mx.codes[-2:], want.codes) and torch.equal(mx.scales[-2:], want.scales)
    assert not mx.codes[:-2].any()
    y = q.mx_dequantize(mx, torch.float16, out=x)
    assert torch.equal(y[-2:], q.mx_dequantize(want, torch.float16))


def test_no_rows(q):
    e = torch.empty(0, 256, dtype=torch.float16, device=DEV)
    mx = q.mx_quantize(e, 1)
    w = q.mx_quantize(rand((8, 256), 1), 1)
    assert mx.rows == 0 and q.mx_gemm(mx, w).shape == (0, 8)
    y, s, m = q.add_rms_norm(e, None, mx_fmt=2)
    assert y.shape == (0, 256) and m.rows == 0
    idx, wt = q.route_scored(e, 4)
    assert idx.shape == (0, 4) and wt.shape == (0, 4)


# ---- products ----------------------------------------------------------------------------------------------------
def operand(q, rows, cols, fmt, seed):
    return q.mx_quantize(rand((rows, cols), seed, scale=1.0) * torch.exp2(rand((rows, 1), seed + 1).round()), fmt)


def check_product(q, a, w, dtype, add=None, rows=None, out=None):
    """y against fp64 (on the GPU, from the exact numbers), at every row or at `rows`."""
    y = q.mx_gemm(a, w, add=add, out=out, out_dtype=dtype)
    pick = slice(None) if rows is None else rows
    A, W = a.dequantize()[pick].double(), w.dequantize().double()
    want, size = A @ W.T, A.abs() @ W.abs().T
    if add is not None:
        want = want + add[pick].double()
        size = size + add[pick].double().abs()
    cut = 0
    if a.fmt == 2 and dtype != torch.float32:
        top = [torch.nn.functional.pad(t.abs(), (0, -t.shape[1] % 8)).reshape(len(t), -1, 8).amax(2) for t in (A, W)]
        cut = 7 * 2.0 ** -13 * (top[0] @ top[1].T)
    got = y[pick].double()
    bound = half_step(dtype) * want.abs() + (MFMA * size + cut) * (1 + half_step(dtype)) + subnormal(dtype)
    err = (got - want).abs()
    assert (err <= bound).all(), float((err / bound).max())
    return y


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 16, 128), (2, 17, 130), (7, 64, 32), (15, 100, 257), (16, 256, 512),
                                   (17, 33, 1024), (31, 48, 384), (33, 128, 640), (64, 250, 96), (65, 70, 2048),
                                   (128, 128, 128), (129, 257, 260), (256, 512, 1152), (300, 130, 1500), (1, 4096, 4096),
                                   (5, 513, 7168), (513, 300, 300)])
def test_gemm(q, fmt, m, n, k):
    a, w = operand(q, m, k, fmt, 7 * m + n), operand(q, n, k, 1, k + 13)
    for dtype in DTS:
        check_product(q, a, w, dtype)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("m,n,k", [(1, 20, 256), (48, 300, 384), (200, 260, 520), (600, 520, 260)])
@pytest.mark.parametrize("dtype", DTS)
def test_gemm_add_and_strides(q, fmt, m, n, k, dtype):
    a, w = operand(q, m, k, fmt, 1), operand(q, n, k, 1, 2)
    wide = rand((m, n + 13), 3, dtype)
    add = wide[:, 5:5 + n]
    guard = torch.full((m + 2, n + 7), 3.0, dtype=dtype, device=DEV)
    y = check_product(q, a, w, dtype, add=add, out=guard[1:-1, 2:2 + n])
    rim = guard.clone()
    rim[1:-1, 2:2 + n] = 3.0
    assert (rim == 3.0).all()                      # nothing around y was touched
    plain = q.mx_gemm(a, w, add=add.contiguous())
    assert torch.equal(plain, y)
    inplace = add.contiguous()
    q.mx_gemm(a, w, add=inplace, out=inplace)
    assert torch.equal(inplace, y)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("m,n", [(40, 90), (100, 300), (500, 4090), (1020, 4090), (2040, 4090), (4090, 4090), (3000, 5000)])
@pytest.mark.parametrize("k", [128, 900])
def test_gemm_tile_shapes(q, fmt, m, n, k):
    """Sizes for which each tile shape is taken (64 x 64 to 256 x 256), with ragged last tiles and odd column groups."""
    a, w = operand(q, m, k, fmt, m + k), operand(q, n, k, 1, n)
    rows = None if m * n < 10 ** 6 else torch.randint(0, m, (300,), device=DEV, generator=torch.Generator(DEV).manual_seed(m))
    for dtype in DTS:
        check_product(q, a, w, dtype, rows=rows)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("m,n,k", [(1, 48, 640), (33, 65, 512), (300, 270, 384), (520, 516, 256)])
def test_gemm_closed_form(q, fmt, m, n, k):
    """Small whole numbers and scales of 2^-2 .. 2^2: every sum fits 24 bits, so the product is exact and any misplaced
    element or scale shows."""
    g = torch.Generator(device=DEV).manual_seed(k)
    a = torch.randint(-2, 3, (m, k), generator=g, device=DEV).float()
    w = torch.randint(-2, 3, (n, k), generator=g, device=DEV).float()
    a *= torch.exp2(torch.randint(-2, 3, (m, -(-k // 32)), generator=g, device=DEV).float()).repeat_interleave(32, 1)[:, :k]
    w *= torch.exp2(torch.randint(-2, 3, (n, -(-k // 32)), generator=g, device=DEV).float()).repeat_interleave(32, 1)[:, :k]
    qa, qw = q.mx_quantize(a, fmt), q.mx_quantize(w, 1)
    assert torch.equal(qa.dequantize(), a) and torch.equal(qw.dequantize(), w)
    assert torch.equal(q.mx_gemm(qa, qw, out_dtype=torch.float32).double(), a.double() @ w.double().T)


@pytest.mark.parametrize("m", [1, 20, 40, 300])
def test_gemm_keeps_small_elements_next_to_large_ones(q, m):
    """8-bit elements of 2^-9 next to 256 in the same eight columns: an fp32 result has every one of them (the sums fit
    24 bits, so it is exact)."""
    g = torch.Generator(device=DEV).manual_seed(m)
    k, n = 384, 80
    a = torch.randint(-7, 8, (m, k), generator=g, device=DEV).float() * 2.0 ** -9
    a[:, ::8] = 256.0
    a[:, 8::16] = -256.0
    w = torch.randint(-1, 2, (n, k), generator=g, device=DEV).float()
    w[:, 0::32] = 6.0                              # scales of 1
    qa, qw = q.mx_quantize(a, 2), q.mx_quantize(w, 1)
    assert torch.equal(qa.dequantize(), a) and torch.equal(qw.dequantize(), w)
    assert torch.equal(q.mx_gemm(qa, qw, out_dtype=torch.float32).double(), a.double() @ w.double().T)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("m", [1, 24, 300])
def test_gemm_nan_blocks_and_extreme_scales(q, fmt, m):
    a, w = rand((m, 512), 1), rand((64, 512), 2)
    a[m // 2, 200] = math.nan
    w[5, 300] = math.inf
    y = q.mx_gemm(q.mx_quantize(a, fmt), q.mx_quantize(w, 1), out_dtype=torch.float32)
    bad = torch.zeros(m, 64, dtype=torch.bool, device=DEV)
    bad[m // 2] = True
    bad[:, 5] = True
    assert torch.equal(y.isnan(), bad)
    # 2^120 times 2^-120: the scales meet in the product only
    a, w = rand((m, 256), 3) * 2.0 ** 110, rand((64, 256), 4) * 2.0 ** -110
    check_product(q, q.mx_quantize(a, fmt), q.mx_quantize(w, 1), torch.float32)


@pytest.mark.parametrize("m", [2, 20, 70, 300])
@pytest.mark.parametrize("k", [128, 384, 640, 1152])
def test_gemm_nan_elements_stay_in_their_row(q, m, k):
    """An 8-bit element may be NaN by itself: its row is, and the row before it, whose last columns lie next to it in
    memory, is not."""
    a, w = operand(q, m, k, 2, 1), operand(q, 70, k, 1, 2)
    want = q.mx_gemm(a, w)
    a.codes[m - 1] = 0x7F
    y = q.mx_gemm(a, w)
    assert y[m - 1].isnan().all() and torch.equal(y[:-1], want[:-1])


@pytest.mark.parametrize("m", [3, 200])
def test_gemm_rows_hang_on_their_own_row(q, m):
    a, w = operand(q, m, 640, 2, 1), operand(q, 96, 640, 1, 2)
    y = q.mx_gemm(a, w)
    b = operand(q, m, 640, 2, 9)
    b.codes[1], b.scales[1] = a.codes[1], a.scales[1]
    assert torch.equal(q.mx_gemm(b, w)[1], y[1])
    assert torch.equal(q.mx_gemm(a, w), y)


def test_gemm_result_past_2_31_elements(q):
    m, n, k = 300_000, 8192, 128                   # 2.46e9 fp16 results
    a, w = operand(q, m, k, 1, 1), operand(q, n, k, 1, 2)
    check_product(q, a, w, torch.float16, rows=torch.tensor([0, 1, 262_143, 262_144, m - 2, m - 1], device=DEV))


# ---- norm --------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 5), (3, 64), (300, 100), (5, 1000), (2, 4096), (3, 7168), (1, 8200),
                                       (2, 16384), (3, 16383)])
@pytest.mark.parametrize("res", [True, False])
def test_norm(q, dtype, rows, cols, res):
    x, r = rand((rows, cols), 1, dtype, 3.0), rand((rows, cols), 2, dtype) if res else None
    w = rand((cols,), 3, torch.float32 if cols % 3 else dtype)
    s_want = (x.float() + r.float()).to(dtype) if res else x
    exact = O.rms_norm(f64(s_want), f64(w), 1e-5)
    for y_dtype in DTS:
        for fmt in (None, 1, 2):
            y, s, mx = q.add_rms_norm(x, w, residual=r, eps=1e-5, out_dtype=y_dtype, mx_fmt=fmt)
            assert torch.equal(s, s_want)
            err = np.abs(f64(y) - exact)
            assert (err <= (half_step(y_dtype) + WORK) * np.abs(exact) + subnormal(y_dtype)).all()
            assert (mx is None) == (fmt is None)
            if mx is not None and rows * cols <= 40000:
                assert_mx_of(mx, exact)
    y1, _, _ = q.add_rms_norm(x, None, residual=r, eps=1e-5, out_dtype=torch.float32)
    one = O.rms_norm(f64(s_want), None, 1e-5)
    assert (np.abs(f64(y1) - one) <= (half_step(torch.float32) + WORK) * np.abs(one)).all()


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("cols,stride,offset", [(96, 100, 0), (96, 128, 1), (130, 131, 0), (4096, 4104, 8)])
def test_norm_strides_and_in_place(q, dtype, cols, stride, offset):
    x = rand((9, stride + offset), 1, dtype).as_strided((8, cols), (stride, 1), offset)
    r = rand((8, stride + 3), 2, dtype)[:, 3:3 + cols]
    w = rand((cols + 1,), 3, dtype)[1:]
    y, s, mx = q.add_rms_norm(x, w, residual=r, mx_fmt=2)
    yc, sc, mc = q.add_rms_norm(x.contiguous(), w.clone(), residual=r.contiguous(), mx_fmt=2)
    assert torch.equal(y, yc) and torch.equal(s, sc) and torch.equal(mx.codes, mc.codes) and torch.equal(mx.scales, mc.scales)
    xi, ri = x.contiguous().clone(), r.contiguous().clone()
    y2, s2, _ = q.add_rms_norm(xi, w, residual=ri, out=xi, sum_out=ri)
    assert s2 is ri and y2 is xi and torch.equal(xi, y) and torch.equal(ri, s)


def test_norm_special_rows(q):
    """A row of zeros without eps is NaN (0 / 0) as the formula says, with eps zero; rows do not touch each other."""
    x = rand((4, 200), 1)
    x[1] = 0
    x[2, 7] = math.nan
    x[3, 0] = math.inf
    y, _, mx = q.add_rms_norm(x, None, eps=0.0, mx_fmt=1)
    assert y[1].isnan().all() and y[2].isnan().all() and y[3, 0].isnan() and (y[3, 1:] == 0).all()
    codes, scales = elements(mx)
    assert not codes[:, 200:].any() and not scales[:, 7:].any()
    assert (scales[1, :7] == 255).all() and (scales[2, :7] == 255).all() and scales[3, 0] == 255 and scales[3, 1] != 255
    assert_mx_of(q.add_rms_norm(x[:1], None, eps=0.0, mx_fmt=1)[2], O.rms_norm(f64(x[:1]), None, 0.0))
    y, _, _ = q.add_rms_norm(x, None, eps=1e-6)
    assert (y[1] == 0).all()


def test_norm_many_rows(q):
    """More rows than one launch takes."""
    rows = (1 << 20) + 3
    x = rand((rows, 8), 1, torch.float16)
    y, _, mx = q.add_rms_norm(x, None, mx_fmt=2)
    pick = torch.tensor([0, (1 << 20) - 1, 1 << 20, rows - 1], device=DEV)
    yp, _, mp = q.add_rms_norm(x[pick], None, mx_fmt=2)
    assert torch.equal(y[pick], yp) and torch.equal(mx.codes[pick], mp.codes) and torch.equal(mx.scales[pick], mp.scales)


# ---- routing -----------------------------------------------------------------------------------------------------
def check_route(q, logits, k, **kw):
    idx, w = q.route_scored(logits, k, **kw)
    okw = dict(kw)
    if okw.get("bias") is not None:
        okw["bias"] = okw["bias"].cpu().numpy()
    want_i, want_w = O.route_scored(logits.double().cpu().numpy(), k, **okw)
    assert np.array_equal(idx.cpu().numpy(), want_i)
    assert (np.abs(f64(w) - want_w) <= 2.0 ** -23 * np.abs(want_w) + 2.0 ** -149).all()
    return idx, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k,G,keep,rule", [
    (1, 256, 8, 8, 4, "top2"), (5, 1, 1, 1, 1, "max"), (33, 7, 3, 1, 1, "top2"), (64, 64, 8, 1, 1, "max"),
    (130, 384, 8, 8, 4, "top2"), (9, 512, 8, 1, 1, "max"), (17, 512, 8, 64, 3, "top2"), (12, 160, 6, 8, 3, "max"),
    (12, 510, 8, 5, 2, "top2"), (12, 495, 8, 33, 9, "max"), (8, 12, 2, 12, 2, "top2"), (300, 128, 4, 4, 1, "max"),
    (20, 100, 8, 50, 50, "top2")])
@pytest.mark.parametrize("dtype", DTS)
def test_route(q, score, biased, T, E, k, G, keep, rule, dtype):
    lg = rand((T, E), T + E, dtype, 2.0)
    bias = 0.001 * torch.randint(-100, 101, (E,), device=DEV).float() if biased else None
    for renorm in (True, False):
        check_route(q, lg, k, score=score, bias=bias, n_groups=G, keep_groups=keep, group_score=rule, renormalize=renorm,
                    scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,keep", [(1, 1), (4, 2), (3, 1)])
def test_route_masks_ties_and_special_values(q, score, G, keep):
    E, inf = 48, math.inf
    low = torch.finfo(torch.float32).min
    lg = rand((12, E), 4, scale=2.0)
    lg[0] = -inf                                   # nothing to choose
    lg[1] = -inf
    lg[1, 17] = 0.5                                # one expert
    lg[2] = low                                    # masked with the type's lowest value: still candidates
    lg[3] = 0.0                                    # all tied
    lg[3, ::2] = -0.0
    lg[4, 5] = math.nan
    lg[4, 6:20] = -inf
    lg[5, 40] = inf
    lg[5, 41] = inf
    lg[6] = lg[6].round()                          # many ties
    lg[7, :24] = low
    lg[8] = math.nan
    lg[9] = 1000.0 * lg[9]                         # scores that vanish
    bias = torch.zeros(E, device=DEV)
    bias[3], bias[9], bias[20], bias[21] = -inf, math.nan, inf, 0.5
    for b in (None, torch.zeros(E, device=DEV), bias):
        for rule in ("max", "top2"):
            for renorm in (True, False):
                check_route(q, lg, 6, score=score, bias=b, n_groups=G, keep_groups=keep, group_score=rule,
                            renormalize=renorm)
    idx, w = q.route_scored(lg, 6, score=score, n_groups=G, keep_groups=keep)
    assert (idx[0] == -1).all() and (w[0] == 0).all() and (idx[8] == -1).all()
    assert idx[1].tolist() == [17, -1, -1, -1, -1, -1] and w[1].tolist() == [1, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_many_equal_keys(q, score):
    """More equal candidates than a wavefront has lanes, with and without a bias, in one group and in eight."""
    lg = torch.zeros(3, 512, device=DEV)
    lg[1, 300:] = 1.0
    lg[2, ::2] = -2.0
    for b in (None, torch.zeros(512, device=DEV)):
        for G, keep in ((1, 1), (8, 5)):
            check_route(q, lg, 8, score=score, bias=b, n_groups=G, keep_groups=keep)


def test_route_large_batch_of_ties(q):
    """16-bit logits and stepped biases: many margins are not kept, and the choice is the oracle's all the same."""
    lg = rand((1500, 384), 8, torch.bfloat16, 0.02)
    bias = 0.001 * torch.randint(-3, 4, (384,), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).float()
    check_route(q, lg, 8, score="sigmoid", bias=bias, n_groups=8, keep_groups=4)
    check_route(q, lg, 8, score="softmax", bias=bias, n_groups=8, keep_groups=4, renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_biases_that_cancel(q, score):
    """Biases of 10,000 and -10,000 meet in the groups' sums of two: what is left is far below their own rounding in 32 bits."""
    lg = rand((3000, 32), 5)
    bias = torch.full((32,), -10000.0, device=DEV)
    bias[::4] = 10000.0
    check_route(q, lg, 4, score=score, bias=bias, n_groups=8, keep_groups=3)


def test_route_close_scores_keep_their_order(q):
    """Biases that differ by one part in 2^40 of the scores' sum order experts that 32 bits cannot tell apart."""
    lg = torch.zeros(1, 16, device=DEV)
    bias = torch.zeros(16, device=DEV)
    bias[11], bias[4] = 2.0 ** -40, 2.0 ** -41
    idx, _ = check_route(q, lg, 3, score="sigmoid", bias=bias)
    assert idx[0].tolist() == [11, 4, 0]


@pytest.mark.parametrize("dtype", DTS)
def test_route_strided_logits(q, dtype):
    base = rand((40, 77), 3, dtype)
    check_route(q, base[:, 4:68], 4, n_groups=4, keep_groups=2)
    assert torch.equal(q.route_scored(base[:, 4:68], 4)[0], q.route_scored(base[:, 4:68].contiguous(), 4)[0])


# ---- streams, graphs, the whole chain ----------------------------------------------------------------------------
@pytest.fixture(scope="module")
def experts(q):
    from synth import config_seed, gen_matrices
    seed = config_seed(71)
    H, I, E = 2048, 1024, 16
    up = gen_matrices(seed, [(e, m) for e in range(E) for m in (0, 1)], I, H, device=torch.device(DEV))
    down = gen_matrices(seed, [(e, 2) for e in range(E)], H, I, device=torch.device(DEV))
    packed = [(q.pack_matrix(up[2 * e]), q.pack_matrix(up[2 * e + 1]), q.pack_matrix(down[e])) for e in range(E)]
    return H, I, E, q.expert_table(packed)


@pytest.mark.parametrize("T", [1, 5, 100])
@pytest.mark.parametrize("staged", [False, True])
def test_given_layer_is_the_routed_layer(q, experts, T, staged):
    """With the layer's own choice and weights given, the same bits; a slot without an expert adds nothing."""
    H, I, E, tab = experts
    flags = q.GALE_DECODE_STAGED if staged else 0
    x, lg = rand((T, H), 1, torch.float16), rand((T, E), 2)
    y, idx, w = q.moe_layer_fwd(tab, H, I, lg, x, top_k=4, flags=flags)
    assert torch.equal(q.moe_layer_fwd_given(tab, H, I, idx, w, x, flags=flags), y)
    # other weights, through the routed layer's sum
    half = q.moe_layer_fwd_given(tab, H, I, idx, 2 * w, x, flags=flags)
    assert torch.allclose(half.float(), 2 * y.float(), rtol=2 * half_step(torch.float16), atol=2 * 2.0 ** -24)
    none_i, none_w, zero_i = idx.clone(), w.clone(), idx.clone()
    none_i[:, 2], none_w[:, 2], zero_i[:, 2] = -1, 0.0, 0
    a = q.moe_layer_fwd_given(tab, H, I, none_i, none_w, x, flags=flags)
    assert torch.equal(a, q.moe_layer_fwd_given(tab, H, I, zero_i, none_w, x, flags=flags))
    assert not torch.equal(a, y)
    assert (none_i[:, 2] == -1).all()              # the caller's choice is read only


def block(q, experts, st):
    """An MoE block on the residual stream: norm, scored routing, routed experts, and a shared expert in MX numbers."""
    H, I, E, tab = experts
    x, s, mx = q.add_rms_norm(st["x"], st["nw"], residual=st["r"], out_dtype=torch.float16, mx_fmt=q.GALE_MX_E4M3)
    logits = q.mx_gemm(mx, st["router"], out_dtype=torch.float32)
    idx, w = q.route_scored(logits, 4, score="sigmoid", bias=st["bias"], n_groups=4, keep_groups=2, scale=1.5)
    routed = q.moe_layer_fwd_given(tab, H, I, idx, w, x, ws=st["ws"])
    h = q.mx_swiglu_quantize(q.mx_gemm(mx, st["gate_up"]), q.GALE_MX_E4M3)
    y = q.mx_gemm(h, st["down"], add=routed)
    return y, s, idx, w, routed, x, mx, logits, h


def block_state(q, experts, T, seed):
    H, I, E, _ = experts
    shared = 640
    return {"x": rand((T, H), seed, torch.bfloat16), "r": rand((T, H), seed + 1, torch.bfloat16),
            "nw": 1 + rand((H,), 3, torch.bfloat16, 0.1), "bias": rand((E,), 4, scale=0.1),
            "router": q.mx_quantize(rand((E, H), 5, scale=H ** -0.5), 1),
            "gate_up": q.mx_quantize(rand((2 * shared, H), 6, scale=H ** -0.5), 1),
            "down": q.mx_quantize(rand((H, shared), 7, scale=shared ** -0.5), 1),
            "ws": q.moe_workspace(q.moe_workspace_bytes(T, E, 4, H, I), DEV)}


@pytest.mark.parametrize("T", [1, 6, 150])
def test_block_runs_together(q, experts, T):
    """Each step against the oracle on what the step before it gave."""
    st = block_state(q, experts, T, 50 + T)
    y, s, idx, w, routed, x, mx, logits, h = block(q, experts, st)
    assert torch.equal(s, (st["x"].float() + st["r"].float()).bfloat16())
    exact = O.rms_norm(f64(s), f64(st["nw"]), 1e-6)
    assert (np.abs(f64(x) - exact) <= (half_step(torch.float16) + WORK) * np.abs(exact) + subnormal(torch.float16)).all()
    assert_mx_of(mx, exact)
    check_product(q, mx, st["router"], torch.float32)
    want_i, want_w = O.route_scored(f64(logits), 4, score="sigmoid", bias=f64(st["bias"]), n_groups=4, keep_groups=2,
                                    scale=1.5)
    assert np.array_equal(idx.cpu().numpy(), want_i) and (np.abs(f64(w) - want_w) <= 2.0 ** -23 * want_w).all()
    assert_mx_of(h, O.swiglu(f64(q.mx_gemm(mx, st["gate_up"]))))
    assert torch.equal(check_product(q, h, st["down"], torch.float16, add=routed), y)


@pytest.mark.parametrize("T", [1, 6, 150])
def test_block_in_a_graph(q, experts, T):
    """Captured once, replayed on new inputs with eager work in between: each replay equals the eager call."""
    st = block_state(q, experts, T, 10)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block(q, experts, st)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(q, experts, st)[:4]
    for i in range(4):
        new = block_state(q, experts, T, 200 + 10 * i)
        st["x"].copy_(new["x"])
        st["r"].copy_(new["r"])
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = block(q, experts, new)[:4]
        for a, b in zip(kept, want):
            assert torch.equal(a, b)


def test_two_streams_at_once(q):
    """Independent calls on two streams do not meet (no state is shared between calls)."""
    a, w = operand(q, 96, 2048, 2, 1), operand(q, 1024, 2048, 1, 2)
    b = operand(q, 24, 2048, 1, 3)
    want = q.mx_gemm(a, w), q.mx_gemm(b, w)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(one):
            x = q.mx_gemm(a, w)
        with torch.cuda.stream(two):
            y = q.mx_gemm(b, w)
        got.append((x, y))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) and torch.equal(y, want[1]) for x, y in got)
