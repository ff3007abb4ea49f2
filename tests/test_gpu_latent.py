"""Latent attention, its paged cache and its block tables on the GPU against the fp64 oracle.

Tolerances, derived from the arithmetic (w: the weights, v: the values, A = sum_j w_j |v_j|):
  * plans and written cache rows: exact.
  * a score: products of 16-bit numbers are exact and 576 of them (192 expanded) are summed in fp32: off by at most
    2^-18 of scale * sum |a b| (the bound that the library's other MFMA sums keep), plus 2^-21 of |score| for its scaling and
    the exponent's argument.  D: the largest such error of a query.  Every weight is then off by at most 2 D relative (its own
    and the normalisation's) for D << 1.
  * a weight's rounding to the queries' type: half a step, eps / 2 relative; in fp16, whose weights are taken 2^7 times as large,
    at least 2^-32 absolute (half the smallest subnormal over 2^7).
  * 2^-16 relative for exponentials, sums over keys and rescaling (each a few 2^-24, at most a few hundred in a chain).
  so out is off by at most A (2 D + eps / 2 + 2^-16) + 2^-32 sum |v| + half a step of itself, lse by D + 2^-18 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle, latent_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5
T16 = [torch.float16, torch.bfloat16]


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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---- plans -------------------------------------------------------------------------------------------------------
def make_plan(q, rng, R, block_size, past_top, new_top, width, spare, idle=0.2):
    past = [0 if rng.random() < idle else rng.integers(0, past_top + 1) for _ in range(R)]
    new = [0 if rng.random() < idle else rng.integers(0, new_top + 1) for _ in range(R)]
    old = [-(-int(p) // block_size) for p in past]
    need = sum(-(-int(p + n) // block_size) - o for p, n, o in zip(past, new, old))
    ids = rng.permutation(sum(old) + need + 5)
    table = np.full((R, width), -7)
    at = 0
    for r, o in enumerate(old):
        table[r, : min(o, width)] = ids[at: at + o][:width]
        at += o
    return past, new, table, ids[at:], int(need * spare)


def check_plan(q, past, new, table, free, n_free, block_size, n_tok):
    dev = i32(table)
    got = q.paged_plan(i32(past), i32(new), i32(free), i32([n_free]), dev, block_size, n_tok)
    want = O.paged_plan(past, new, free, n_free, table, block_size, n_tok)
    for name, g, w in zip(("slots", "q_starts", "kv_lens", "taken", "table"), (*got, dev), want):
        assert np.array_equal(g.cpu().numpy().reshape(np.shape(w)), w), name


@pytest.mark.parametrize("R", [1, 2, 3, 64, 255, 256, 257, 1023, 1024, 1025, 2500])
@pytest.mark.parametrize("block_size", [1, 16, 64, 1024])
def test_plan(q, R, block_size):
    rng = np.random.default_rng(R * 7 + block_size)
    for new_top, spare in ((1, 1.0), (40, 1.0), (40, 0.5), (3, 0.0)):
        past, new, table, free, n_free = make_plan(q, rng, R, block_size, 300, new_top, 340 // block_size + 1, spare)
        check_plan(q, past, new, table, free, n_free, block_size, sum(map(int, new)) + int(rng.integers(0, 5)))


def test_plan_without_room(q):
    rng = np.random.default_rng(5)
    for trial in range(6):
        past, new, table, free, n_free = make_plan(q, rng, 300, 16, 200, 60, 9, 0.7)     # rows of 9 blocks: some are too long
        total = sum(map(int, new))
        check_plan(q, past, new, table, free, n_free, 16, (total, total - 1, total // 2, 1, 0, total + 300)[trial])
    check_plan(q, [-5, 3], [2, -4], np.array([[1, 2], [3, 4]]), [9], 1, 4, 4)             # negative lengths count as 0
    check_plan(q, [5, 0], [1, 2], np.array([[1, -1], [3, 4]]), [9, 8], 77, 4, 4)           # n_free past the list; a negative id
    check_plan(q, [0], [3], np.array([[5]]), [9, 8], -3, 4, 4)
    check_plan(q, [0], [3], np.zeros((1, 0), dtype=int), [9, 8], 2, 4, 4)                  # a table without columns
    check_plan(q, [], [], np.zeros((0, 3), dtype=int), [9], 1, 4, 3)
    check_plan(q, [2 ** 31 - 1, 1], [5, 1], np.array([[1, 2], [3, 4]]), [9, 8], 2, 1024, 9)  # a length past the table


def test_plan_of_long_prompts_and_strided_table(q):
    past, new, bs = [70000, 0, 5], [60000, 131072, 1], 64
    width = 2100
    table = np.full((3, width), -1)
    rng = np.random.default_rng(6)
    ids = rng.permutation(8000)
    table[0, :1094], table[2, 0] = ids[:1094], ids[1094]
    wide = torch.full((3, width + 13), -9, dtype=torch.int32, device=DEV)
    wide[:, :width] = i32(table)
    n_tok = sum(new) + 700
    got = q.paged_plan(i32(past), i32(new), i32(ids[1095:]), i32([len(ids) - 1095]), wide[:, :width], bs, n_tok)
    want = O.paged_plan(past, new, ids[1095:], len(ids) - 1095, table, bs, n_tok)
    for g, w in zip((*got, wide[:, :width]), want):
        assert np.array_equal(g.cpu().numpy().reshape(np.shape(w)), w)
    assert (wide[:, width:] == -9).all()


# ---- the cache's writer --------------------------------------------------------------------------------------------
def filled(q, n_blocks, block_size, dtype, mx, seed, strided=False, scale=1.0):
    slots = n_blocks * block_size
    rows = rand((slots, 576), seed, dtype, scale)
    if mx:
        return q.LatentCache(q.mx_quantize(rows[:, :512].contiguous(), q.GALE_MX_E2M1), rows[:, 512:].contiguous(), block_size)
    return q.LatentCache(rows[:, :512], rows[:, 512:], block_size) if strided else \
        q.LatentCache(rows[:, :512].contiguous(), rows[:, 512:].contiguous(), block_size)


@pytest.mark.parametrize("dtype", T16)
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 3, 4, 65, 1000])
def test_append(q, dtype, mx, T):
    cache = filled(q, 80, 16, dtype, mx, 1, strided=T % 2 == 1)
    x = rand((T, 576), 2, dtype, 3.0)
    x[0, :32] = 0
    x[T // 2, 5] = math.nan
    x[T - 1, 40] = math.inf
    g = torch.Generator(device=DEV).manual_seed(T)
    slots = torch.randperm(1280, generator=g, device=DEV)[:T]
    if T > 3:
        slots[1], slots[2], slots[3] = -1, 1280, 1 << 40          # skipped
    keep = (slots >= 0) & (slots < 1280)
    parts = [cache.latent.codes, cache.latent.scales, cache.rope] if mx else [cache.latent, cache.rope]
    want = [p.clone() for p in parts]
    if mx:
        m = q.mx_quantize(x[:, :512].contiguous(), q.GALE_MX_E2M1)
        new = [m.codes, m.scales, x[:, 512:]]
    else:
        new = [x[:, :512], x[:, 512:]]
    for w, n in zip(want, new):
        w[slots[keep]] = n[keep]
    q.latent_append(cache, x[:, :512], x[:, 512:], slots)
    for p, w in zip(parts, want):
        assert torch.equal(p.view(torch.uint8), w.contiguous().view(torch.uint8).view_as(p.view(torch.uint8)))


def test_append_of_rows_that_are_not_aligned_and_of_nothing(q):
    cache = filled(q, 4, 16, torch.bfloat16, False, 1)
    x = rand((7, 600), 3, torch.bfloat16)
    slots = torch.arange(7, device=DEV) * 9
    q.latent_append(cache, x[:, 1:513], x[:, 517:581], slots)
    assert torch.equal(cache.latent[slots], x[:, 1:513]) and torch.equal(cache.rope[slots], x[:, 517:581])
    q.latent_append(cache, x[:0, :512], x[:0, :64], slots[:0])


# ---- attention over the cache --------------------------------------------------------------------------------------
def batch(q, lens, news, block_size, seed, spare=3):
    """(table, q_starts, kv_lens, n_blocks): pages in random order."""
    rng = np.random.default_rng(seed)
    need = [-(-n // block_size) for n in lens]
    n_blocks = sum(need) + spare
    ids, at = rng.permutation(n_blocks), 0
    table = np.full((len(lens), max(max(need), 1)), -1)
    for r, n in enumerate(need):
        table[r, :n] = ids[at: at + n]
        at += n
    return table, np.concatenate(([0], np.cumsum(news))), np.array(lens), n_blocks


def cache_values(q, cache):
    """(c, r) in fp64, 4-bit latents as numbers of the queries' type."""
    if isinstance(cache.latent, q.MXTensor):
        m = cache.latent
        c = block_oracle.mx_values(block_oracle.mx_elements(m.codes.cpu().numpy(), 1), m.scales.cpu().numpy().astype(np.int64), 1, 512)
        c = torch.tensor(c).to(cache.dtype).double().numpy()
    else:
        c = f64(cache.latent)
    return c, f64(cache.rope)


def bounds(x, keys, scale, dtype, spread, values, out, lse):
    """(of out, of lse): x [n, d] and keys [m, d] as absolute values, one query."""
    size = abs(scale) * (keys @ x).max() if len(keys) else 0.0
    D = 2.0 ** -18 * size + 2.0 ** -21 * size
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -32 * values + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    return spread * (2 * D + half + 2.0 ** -16) + half * np.abs(out) + tiny, D + 2.0 ** -18 * (1 + np.abs(lse))


def check_latent(q, cache, x, table, starts, lens, causal=True, scale=SCALE, tokens=None, **kw):
    out, l = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), scale, causal, **kw)
    c, r = cache_values(q, cache)
    xs = f64(x)
    bs, n_blocks = cache.block_size, cache.n_blocks
    got, got_l = f64(out), f64(l)
    for i in range(len(lens)):
        a, b = int(starts[i]), int(starts[i + 1])
        for t in range(a, b):
            if tokens is not None and t not in tokens:
                continue
            seen = max(0, int(lens[i]) - (b - a) + (t - a) + 1) if causal else int(lens[i])
            pos = np.arange(seen)
            blk = table[i][pos // bs]
            fine = (blk >= 0) & (blk < n_blocks)
            rows = (blk * bs + pos % bs)[fine]
            k = np.concatenate((c[rows], r[rows]), 1)
            for h in range(x.shape[1]):
                want, wl, spread = O.attend(xs[t, h], k, c[rows], scale)
                bo, bl = bounds(np.abs(xs[t, h]), np.abs(k), scale, x.dtype, spread, np.abs(c[rows]).sum(0), want, wl)
                assert (np.abs(got[t, h] - want) <= bo).all(), (i, t, h, np.abs(got[t, h] - want).max(), bo.min())
                if math.isinf(wl):
                    assert got_l[t, h] == wl
                else:
                    assert abs(got_l[t, h] - wl) <= bl, (i, t, h, got_l[t, h], wl, bl)
    return out, l


LENS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 0, 511, 700]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dtype", T16)
@pytest.mark.parametrize("heads", [1, 5, 16, 32, 33, 64, 128])
def test_decode(q, dtype, mx, heads):
    bs = {1: 1, 5: 2, 16: 16, 32: 64, 33: 8, 64: 128, 128: 32}[heads]
    lens = LENS if heads < 64 else LENS[::2]
    table, starts, lens, n = batch(q, lens, [1] * len(lens), bs, heads)
    cache = filled(q, n, bs, dtype, mx, 3, strided=heads == 5)
    check_latent(q, cache, rand((len(lens), heads, 576), 4, dtype), table, starts, lens)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [1, 3, 16, 40, 128])
def test_drafts(q, mx, causal, heads):
    news = [1, 4, 0, 2, 7, 3, 1, 5]
    lens = [64, 4, 50, 129, 300, 1, 0, 96]              # also fewer keys than queries: rows that see nothing
    table, starts, lens, n = batch(q, lens, news, 16, heads)
    cache = filled(q, n, 16, torch.bfloat16, mx, 5)
    check_latent(q, cache, rand((sum(news), heads, 576), 6, torch.bfloat16), table, starts, lens, causal)


@pytest.mark.parametrize("dtype,heads,mx", [(torch.float16, 16, False), (torch.bfloat16, 128, False), (torch.bfloat16, 8, True),
                                            (torch.float16, 64, True)])
def test_long_contexts(q, dtype, heads, mx):
    """Keys of one request in many workgroups, and workgroups that hold parts of several requests."""
    lens = [9000, 1, 4097, 130, 20000]
    table, starts, lens, n = batch(q, lens, [1] * 5, 64, heads)
    cache = filled(q, n, 64, dtype, mx, 7)
    check_latent(q, cache, rand((5, heads, 576), 8, dtype), table, starts, lens)


def test_a_prompt_in_absorbed_form(q):
    table, starts, lens, n = batch(q, [150, 90], [150, 61], 16, 1)
    cache = filled(q, n, 16, torch.bfloat16, False, 9)
    check_latent(q, cache, rand((211, 6, 576), 10, torch.bfloat16), table, starts, lens,
                 tokens=[0, 1, 31, 32, 63, 64, 100, 149, 150, 151, 200, 210])


def test_many_requests(q):
    rng = np.random.default_rng(11)
    lens, news = rng.integers(0, 60, 1500), rng.integers(0, 3, 1500)
    table, starts, lens, n = batch(q, list(lens), list(news), 4, 2)
    cache = filled(q, n, 4, torch.float16, False, 11)
    check_latent(q, cache, rand((int(starts[-1]), 2, 576), 12, torch.float16), table, starts, lens,
                 tokens=set(range(0, int(starts[-1]), 7)))


@pytest.mark.parametrize("mx", [False, True])
def test_what_is_not_seen_has_no_influence(q, mx):
    news, bs = [3, 1, 2], 16
    table, starts, lens, n = batch(q, [70, 40, 33], news, bs, 3)
    table[1, 1] = -1                                     # a hole, and ids outside the cache
    table[2, 0] = n + 5
    table = np.pad(table, ((0, 0), (0, 2)), constant_values=1 << 28)
    cache = filled(q, n, bs, torch.bfloat16, mx, 13)
    x = rand((6, 20, 576), 14, torch.bfloat16)
    out, l = check_latent(q, cache, x, table, starts, lens)
    # NaN and infinity in every slot that no key is in, and in the keys that only later queries see
    seen = np.concatenate([table[i][np.arange(m) // bs] * bs + np.arange(m) % bs for i, m in enumerate(lens)])
    late = [table[0][p // bs] * bs + p % bs for p in (68, 69)] + [table[2][32 // bs] * bs + 32 % bs]
    bad = torch.ones(n * bs, dtype=torch.bool, device=DEV)
    bad[torch.tensor(seen[(seen >= 0) & (seen < n * bs)], device=DEV)] = False
    bad[torch.tensor(late, device=DEV)] = True
    if mx:
        cache.latent.scales[bad] = 255
    else:
        cache.latent[bad] = math.nan
        cache.latent[bad, 7] = math.inf
    cache.rope[bad] = math.inf
    out2, l2 = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    for t in (0, 3, 4):                                  # token 0 sees 68 keys, token 4 sees 32
        assert torch.equal(l2[t], l[t]) or torch.allclose(l2[t], l[t], rtol=2.0 ** -18, atol=2.0 ** -18)
        assert torch.isfinite(out2[t]).all()
        assert (out2[t].float() - out[t].float()).abs().max() <= 2.0 ** -7 * out[t].float().abs().max()
    for t in (1, 2, 5):
        assert torch.isnan(out2[t]).any() and not torch.isfinite(l2[t]).any()


def test_nan_queries_stay_alone(q):
    table, starts, lens, n = batch(q, [100, 100], [2, 1], 16, 3)
    cache = filled(q, n, 16, torch.float16, False, 15)
    x = rand((3, 16, 576), 16, torch.float16)
    a, la = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    x[1, 3, 9] = math.nan
    b, lb = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    assert torch.isnan(b[1, 3]).all() and torch.isnan(lb[1, 3])
    b[1, 3], lb[1, 3] = a[1, 3], la[1, 3]
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dtype", T16)
def test_scores_of_many_sizes(q, dtype):
    """Rising, falling and far-apart scores: the running maximum moves often, by little and by much."""
    lens = [700, 700, 700, 700]
    table, starts, lens, n = batch(q, lens, [1] * 4, 32, 4)
    cache = filled(q, n, 32, dtype, False, 17)
    x = rand((4, 16, 576), 18, dtype)
    for r, f in enumerate((lambda p: p / 20, lambda p: -p / 20, lambda p: 40 * np.sin(p), lambda p: 100.0 * (p == 650))):
        p = np.arange(700)
        slots = torch.tensor(table[r][p // 32] * 32 + p % 32, device=DEV)
        cache.rope[slots, 0] = torch.tensor(f(p), device=DEV).to(dtype)
    x[:, :, 512] = 8.0
    check_latent(q, cache, x, table, starts, lens)
    check_latent(q, cache, x, table, starts, lens, scale=-0.3)
    check_latent(q, cache, x, table, starts, lens, scale=0.0)


def test_weights_far_below_the_largest_are_summed(q):
    """A key 16 above 60,000 others in score: those hold 0.7 % of the weight, each 1.1e-7 of it."""
    lens = [60001]
    table, starts, lens, n = batch(q, lens, [1], 64, 4)
    cache = filled(q, n, 64, torch.float16, False, 19)
    cache.latent[:] = 1.0
    cache.rope[:] = 0
    first = int(table[0][0]) * 64
    cache.latent[first] = -1.0
    cache.rope[first, 0] = 16.0
    x = torch.zeros(1, 1, 576, dtype=torch.float16, device=DEV)
    x[..., 512] = 1.0
    out, l = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), 1.0)
    rest = 60000 * math.exp(-16.0)
    assert abs(out[0, 0, 0].item() - (rest - 1) / (rest + 1)) < 2.0 ** -11 + 60000 * 2.0 ** -32 * 2
    # the sum, 1 to 1 + rest, takes the others in steps of 32 keys or more: at most 60,001 / 32 additions, each off by half an
    # ulp of 1 to the same side (2^-24), and its logarithm next to 16 is rounded to 2^-20
    assert abs(l[0, 0].item() - (16 + math.log1p(rest))) < 60001 / 32 * 2.0 ** -24 + 2.0 ** -20


def test_tokens_of_no_request_and_strides(q):
    table, starts, lens, n = batch(q, [40, 9], [2, 1], 8, 5)
    cache = filled(q, n, 8, torch.bfloat16, False, 20, strided=True)
    big = rand((6, 3 * 4 * 576), 21, torch.bfloat16)
    x = big.view(6, 3, 4, 576)[:, 1]
    wide = torch.full((6, 4 * 512 + 64), 5.0, dtype=torch.bfloat16, device=DEV)
    out = wide[:, : 4 * 512].view(6, 4, 512) if False else torch.as_strided(wide, (6, 4, 512), (4 * 512 + 64, 512, 1))
    lse = torch.full((6, 4), 7.0, device=DEV)
    check_latent(q, cache, x, table, starts, lens, out=out, lse=lse)
    assert (wide[3:] == 5).all() and (wide[:, 4 * 512:] == 5).all() and (lse[3:] == 7).all()
    a = out.clone()
    odd = torch.empty(6 * 4 * 576 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(6, 4, 576)
    odd.copy_(x)
    b, _ = q.latent_attention(odd, cache, i32(table), i32(starts), i32(lens), SCALE)
    assert torch.equal(a[:3], b[:3])


def test_bad_starts_and_lengths_are_clamped(q):
    table, starts, lens, n = batch(q, [40, 9], [2, 1], 8, 5)
    cache = filled(q, n, 8, torch.bfloat16, False, 20)
    x = rand((3, 4, 576), 21, torch.bfloat16)
    width = table.shape[1] * 8
    a, _ = q.latent_attention(x, cache, i32(table), i32([0, 2, 3]), i32([width, 0]), SCALE)
    b, l = q.latent_attention(x, cache, i32(table), i32([-4, 2, 99]), i32([2 ** 31 - 1, -5]), SCALE)
    assert torch.equal(a, b) and torch.isinf(l[2]).all() and not b[2].any()


def test_offsets_past_32_bits(q):
    """Rows of the cache more than 4 GiB from its start."""
    bs, n = 64, 1 << 17                                  # 8.4 million slots: 8.6 GB of latents, 1 GB of rope
    for mx in (False, True):
        cache = q.LatentCache.empty(n, bs, torch.bfloat16, mx=mx, device=DEV)
        small = filled(q, 4, bs, torch.bfloat16, mx, 22)
        ids = [n - 1, 7, n - 3, n // 2 + 1]
        for i, b in enumerate(ids):
            src, dst = slice(i * bs, (i + 1) * bs), slice(b * bs, (b + 1) * bs)
            if mx:
                cache.latent.codes[dst], cache.latent.scales[dst] = small.latent.codes[src], small.latent.scales[src]
            else:
                cache.latent[dst] = small.latent[src]
            cache.rope[dst] = small.rope[src]
        x = rand((1, 16, 576), 23, torch.bfloat16)
        a = q.latent_attention(x, small, i32([[0, 1, 2, 3]]), i32([0, 1]), i32([250]), SCALE)
        b = q.latent_attention(x, cache, i32([ids]), i32([0, 1]), i32([250]), SCALE)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        # and the writer
        y = rand((2, 576), 24, torch.bfloat16)
        q.latent_append(cache, y[:, :512], y[:, 512:], torch.tensor([n * bs - 1, n * bs - 70], device=DEV))
        if not mx:
            assert torch.equal(cache.latent[n * bs - 1], y[0, :512]) and torch.equal(cache.latent[n * bs - 70], y[1, :512])
        else:
            m = q.mx_quantize(y[:, :512].contiguous(), q.GALE_MX_E2M1)
            assert torch.equal(cache.latent.codes[n * bs - 1], m.codes[0])
        assert torch.equal(cache.rope[n * bs - 70], y[1, 512:])
        del cache


def test_4bit_values_at_the_ends(q):
    """Scales at both ends of what fp16 holds, and a NaN block in the middle of what is seen."""
    table, starts, lens, n = batch(q, [50, 20], [1, 1], 16, 6)
    cache = filled(q, n, 16, torch.float16, True, 25)
    s = cache.latent.scales
    s[:, 3], s[:, 4], s[:, 5] = 127 - 22, 0, 127 + 10    # values among fp16's subnormals, 2^-127 times, up to 6144
    x = rand((2, 4, 576), 26, torch.float16, 0.02)
    check_latent(q, cache, x, table, starts, lens)
    s[int(table[1][0]) * 16 + 3, 9] = 255
    out, l = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all() and torch.isnan(l[1]).all()


# ---- prompts -------------------------------------------------------------------------------------------------------
def check_prompt(q, x, k, kr, v, starts, kstarts, causal=True, scale=SCALE, tokens=None, heads=None, **kw):
    out, l = q.latent_attention_expanded(x, k, kr, v, i32(starts), i32(kstarts), scale, causal, **kw)
    xs, ks, rs, vs, got, got_l = f64(x), f64(k), f64(kr), f64(v), f64(out), f64(l)
    for i in range(len(starts) - 1):
        a, b, s0, s1 = starts[i], starts[i + 1], kstarts[i], kstarts[i + 1]
        for t in range(a, b):
            if tokens is not None and t not in tokens:
                continue
            seen = max(0, (s1 - s0) - (b - a) + (t - a) + 1) if causal else s1 - s0
            for h in heads or range(x.shape[1]):
                keys = np.concatenate((ks[s0: s0 + seen, h], rs[s0: s0 + seen]), 1)
                val = vs[s0: s0 + seen, h]
                want, wl, spread = O.attend(xs[t, h], keys, val, scale)
                bo, bl = bounds(np.abs(xs[t, h]), np.abs(keys), scale, x.dtype, spread, np.abs(val).sum(0), want, wl)
                assert (np.abs(got[t, h] - want) <= bo).all(), (i, t, h, np.abs(got[t, h] - want).max())
                if math.isinf(wl):
                    assert got_l[t, h] == wl
                else:
                    assert abs(got_l[t, h] - wl) <= bl, (i, t, h)
    return out, l


def prompts(lens, keys, heads, dtype, seed, halves=True):
    T, S = sum(lens), sum(keys)
    x, kr = rand((T, heads, 192), seed, dtype), rand((S, 64), seed + 1, dtype)
    kv = rand((S, heads, 256), seed + 2, dtype)
    k, v = (kv[..., :128], kv[..., 128:]) if halves else (kv[..., :128].contiguous(), kv[..., 128:].contiguous())
    return x, k, kr, v, [0, *np.cumsum(lens).tolist()], [0, *np.cumsum(keys).tolist()]


@pytest.mark.parametrize("dtype", T16)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 64, 65, 127, 128, 129, 257, 300])
def test_prompt(q, dtype, causal, n):
    args = prompts([n], [n], 3, dtype, n, halves=n % 2 == 0)
    check_prompt(q, *args, causal=causal, tokens=None if n < 70 else set(range(0, n, 9)) | {n - 1, n - 2, 127, 128, 63, 64})


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [1, 8, 11])
def test_prompts_behind_earlier_text(q, causal, heads):
    lens, keys = [5, 0, 130, 1, 40, 17, 64], [5, 9, 400, 77, 12, 0, 64]         # also fewer keys than queries, and none
    args = prompts(lens, keys, heads, torch.bfloat16, heads)
    check_prompt(q, *args, causal=causal, tokens=set(range(0, sum(lens), 3)) | {4, 5, 134, 135, 136, 175, 176})


def test_long_prompt(q):
    n = 5000
    args = prompts([n], [n], 2, torch.bfloat16, 1)
    check_prompt(q, *args, tokens={0, 1, 63, 64, 1023, 1024, 2500, 4095, 4096, 4998, 4999})


def test_prompts_of_many_requests(q):
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 20, 1300).tolist()
    args = prompts(lens, lens, 2, torch.float16, 2)
    check_prompt(q, *args, tokens=set(range(0, sum(lens), 11)))


def test_prompt_masks_nan(q):
    lens, keys = [200, 70], [200, 90]
    x, k, kr, v, s, ks = prompts(lens, keys, 2, torch.float16, 5)
    out, l = check_prompt(q, x, k, kr, v, s, ks, tokens={0, 149, 150, 199, 200, 269})
    v[150, 1, 3] = math.nan
    v[200 + 60, 0, 5] = math.inf
    k[150, 1, 9] = math.nan
    kr[200 + 60, 1] = math.inf
    out2, l2 = q.latent_attention_expanded(x, k, kr, v, i32(s), i32(ks), SCALE)
    close = lambda a, b: (a.float() - b.float()).abs().max() <= 2.0 ** -10 * (1 + b.float().abs().max())      # noqa: E731
    assert close(out2[:150], out[:150]) and close(out2[:200, 0], out[:200, 0]) and torch.allclose(l2[:150], l[:150], atol=2.0 ** -18)
    assert torch.isnan(out2[150:200, 1]).any(1).all() and torch.isnan(l2[150:200, 1]).all()
    assert close(out2[200:240], out[200:240])           # 70 queries, 90 keys: token 40 is the first to see key 60
    up = x[240:, 0, 129] > 0                             # the key's score is +infinity, for the others -infinity: weight 0
    assert up.any() and not torch.isfinite(out2[240:, 0]).all(1)[up].any()


def test_prompt_strides_lse_and_untouched_rows(q):
    lens = [33, 90]
    x, k, kr, v, s, ks = prompts(lens, lens, 4, torch.bfloat16, 6)
    wide_x = rand((130, 4 * 192 + 8), 7, torch.bfloat16)
    xs = torch.as_strided(wide_x, (130, 4, 192), (4 * 192 + 8, 192, 1))
    xs[:123].copy_(x)
    wide_r = rand((123, 72), 8, torch.bfloat16)
    wide_r[:, 8:].copy_(kr)
    out = torch.full((130, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((130, 4), 7.0, device=DEV)
    a, la = q.latent_attention_expanded(x, k, kr, v, i32(s), i32(ks), SCALE)
    q.latent_attention_expanded(xs, k, wide_r[:, 8:], v.contiguous(), i32(s), i32(ks), SCALE, out=out, lse=lse)
    assert torch.equal(out[:123], a) and torch.equal(lse[:123], la) and (out[123:] == 5).all() and (lse[123:] == 7).all()
    b, _ = q.latent_attention_expanded(x, k, kr, v, i32([-3, 33, 999]), i32([-1, 33, 500]), SCALE)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", T16)
def test_prompt_scores_of_many_sizes(q, dtype):
    n = 260
    x, k, kr, v, s, ks = prompts([n] * 4, [n] * 4, 2, dtype, 9)
    p = np.arange(n)
    for r, f in enumerate((lambda p: p / 8, lambda p: -p / 8, lambda p: 40 * np.sin(p), lambda p: 100.0 * (p == 200))):
        kr[r * n: (r + 1) * n, 0] = torch.tensor(f(p), device=DEV).to(dtype)
    x[:, :, 128] = 8.0
    for scale in (SCALE, -0.3, 0.0):
        check_prompt(q, x, k, kr, v, s, ks, scale=scale, tokens=set(range(0, 4 * n, 37)) | {200, 259, 460, 519, 980, 1039})


# ---- lse may be left out, streams, graphs, equal bits ------------------------------------------------------------------
def test_without_lse(q):
    table, starts, lens, n = batch(q, [40], [1], 8, 5)
    cache = filled(q, n, 8, torch.bfloat16, False, 20)
    x = rand((1, 4, 576), 21, torch.bfloat16)
    a, _ = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    out = torch.empty_like(a)
    tab, st, kl = i32(table), i32(starts), i32(lens)
    ws = torch.empty(q.latent_workspace_bytes(1, 1, 4), dtype=torch.uint8, device=DEV)
    assert q.lib().gale_latent_attention(cache.desc, tab.data_ptr(), tab.shape[1], tab.shape[1], kl.data_ptr(), st.data_ptr(), 1,
                                         x.data_ptr(), 4 * 576, 1, 4, SCALE, 1, out.data_ptr(), 4 * 512, None, ws.data_ptr(),
                                         ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(a, out)
    y, k, kr, v, s, ks = prompts([20], [20], 1, torch.bfloat16, 6)
    a, _ = q.latent_attention_expanded(y, k, kr, v, i32(s), i32(ks), SCALE)
    out, s, ks = torch.empty_like(a), i32(s), i32(ks)
    assert q.lib().gale_latent_attention_expanded(
        y.data_ptr(), 192, k.data_ptr(), 256, 128, kr.data_ptr(), 64, v.data_ptr(), 256, 128, 3, 20, 20, 1, s.data_ptr(),
        ks.data_ptr(), 1, SCALE, 1, out.data_ptr(), 128, None, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(a, out)


def test_a_step_in_a_graph(q):
    """Plan, append and attention of one step, captured once and replayed over changing lengths; two graphs share a workspace."""
    bs, R, H = 16, 5, 16
    width = 40
    for mx in (False, True):
        cache = filled(q, 220, bs, torch.bfloat16, mx, 30)
        table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
        ids = torch.randperm(220, generator=torch.Generator().manual_seed(1)).int().to(DEV)
        for r in range(R):
            table[r, :30] = ids[40 * r: 40 * r + 30]
        free = ids[200:].contiguous()
        past, new, n_free = i32([100, 1, 0, 300, 47]), i32([1, 2, 1, 1, 3]), i32([20])
        new_c, x = rand((8, 576), 31, torch.bfloat16), rand((8, H, 576), 32, torch.bfloat16)
        ws = torch.empty(q.latent_workspace_bytes(8, R, H), dtype=torch.uint8, device=DEV)

        def step(outs, out, lse):
            slots, starts, keys, _ = q.paged_plan(past, new, free, n_free, table, bs, 8, out=outs)
            q.latent_append(cache, new_c[:, :512], new_c[:, 512:], slots)
            q.latent_attention(x, cache, table, starts, keys, SCALE, out=out, lse=lse, ws=ws)

        def buffers():
            return ((torch.empty(8, dtype=torch.int64, device=DEV), i32([0] * (R + 1)), i32([0] * R), i32([0])),
                    torch.zeros(8, H, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(8, H, device=DEV))

        bufs = [buffers() for _ in range(3)]
        step(*bufs[2])
        torch.cuda.synchronize()
        graphs = []
        for b in bufs[:2]:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step(*b)
            graphs.append(g)
        for turn, lens in enumerate(([100, 1, 0, 300, 47], [5, 470, 33, 64, 0], [0, 0, 0, 0, 0], [150, 9, 31, 128, 480])):
            past.copy_(i32(lens))
            new_c.copy_(rand((8, 576), 40 + turn, torch.bfloat16))
            x.copy_(rand((8, H, 576), 50 + turn, torch.bfloat16))
            for g, b in zip(graphs, bufs):
                g.replay()
            torch.cuda.synchronize()
            step(*bufs[2])
            torch.cuda.synchronize()
            for b in bufs[:2]:
                assert torch.equal(b[1], bufs[2][1]) and torch.equal(b[2], bufs[2][2])
                assert all(torch.equal(u, w) for u, w in zip(b[0], bufs[2][0]))


def test_prompt_in_a_graph_and_on_another_stream(q):
    x, k, kr, v, s, ks = prompts([100, 33], [120, 33], 3, torch.float16, 6)
    s, ks = i32(s), i32(ks)
    want, lw = q.latent_attention_expanded(x, k, kr, v, s, ks, SCALE)
    out, lse = torch.zeros_like(want), torch.zeros_like(lw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.latent_attention_expanded(x, k, kr, v, s, ks, SCALE, out=out, lse=lse)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, lw)
        assert torch.equal(q.latent_attention_expanded(x, k, kr, v, s, ks, SCALE)[0], want)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        again, _ = q.latent_attention_expanded(x, k, kr, v, s, ks, SCALE)
    other.synchronize()
    assert torch.equal(again, want)


@pytest.mark.parametrize("heads,mx", [(16, False), (16, True), (64, False), (128, False)])
def test_equal_calls_give_equal_bits(q, heads, mx):
    lens = [3000, 77, 1500, 640]
    table, starts, lens, n = batch(q, lens, [2] * 4, 16, 8)
    cache = filled(q, n, 16, torch.bfloat16, mx, 33)
    x = rand((8, heads, 576), 34, torch.bfloat16)
    a = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    for _ in range(5):
        b = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---- together --------------------------------------------------------------------------------------------------------
def test_a_layer_runs_together(q):
    """A prompt and then single tokens through a 4-bit cache: plan, append, the up-projection of the cached rows (the cache
    is itself an operand of the MX product), prompts in expanded form, and the same queries in absorbed form."""
    H, bs, lens = 4, 16, [37, 64, 1]
    T, R, width = sum(lens), len(lens), 8
    cache = filled(q, 20, bs, torch.bfloat16, True, 40)
    table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(20, generator=torch.Generator().manual_seed(2)).int().to(DEV)
    c, kr = rand((T, 512), 41, torch.bfloat16), rand((T, 64), 42, torch.bfloat16)
    slots, starts, keys, taken = q.paged_plan(i32([0] * R), i32(lens), free, i32([20]), table, bs, T)
    assert taken.item() == 3 + 4 + 1 and keys.tolist() == lens
    q.latent_append(cache, c, kr, slots)
    w = q.mx_quantize(rand((H * 256, 512), 43, torch.float32, 512 ** -0.5), q.GALE_MX_E2M1)
    rows = q.MXTensor(cache.latent.codes[slots], cache.latent.scales[slots], 512, q.GALE_MX_E2M1)
    kv = q.mx_gemm(rows, w, out_dtype=torch.bfloat16).view(T, H, 256)
    x = rand((T, H, 192), 44, torch.bfloat16)
    out, lse = q.latent_attention_expanded(x, kv[..., :128], kr, kv[..., 128:], starts, starts, SCALE)
    up = f64(w.dequantize()).reshape(H, 256, 512)
    cd = f64(rows.dequantize())
    k64, v64 = np.einsum("hdk,sk->shd", up[:, :128], cd), np.einsum("hdk,sk->shd", up[:, 128:], cd)
    s64 = [0, 37, 101, 102]
    want, wl, spread = O.expanded_attention(f64(x), k64, f64(kr), v64, s64, s64, SCALE)
    # kv is rounded to bf16: scores move by 2^-9 of scale sum |a k|, values by 2^-9 of themselves
    size = np.array([[SCALE * (np.abs(np.concatenate((k64[:, h], f64(kr)), 1)) @ np.abs(f64(x)[t, h])).max() for h in range(H)]
                     for t in range(T)])
    D = size * (2.0 ** -9 + 2.0 ** -18)
    tol = spread * (2 * D[..., None] * np.exp(2 * D[..., None]) + 2 * 2.0 ** -9 + 2.0 ** -16) + 2.0 ** -8 * np.abs(want) + 2.0 ** -30
    assert (np.abs(f64(out) - want) <= tol).all() and (np.abs(f64(lse) - wl) <= D + 2.0 ** -17).all()
    # absorbed: the key's up-projection goes into the queries (rounded to bf16 once more)
    xa64 = np.concatenate((np.einsum("thd,hdk->thk", f64(x)[..., :128], up[:, :128]), f64(x)[..., 128:]), 2)
    xa = torch.tensor(xa64, device=DEV).bfloat16()
    lat, lse2 = q.latent_attention(xa, cache, table, starts, keys, SCALE)
    got = np.einsum("thk,hdk->thd", f64(lat), up[:, 128:])
    keys64 = np.concatenate((cd, f64(kr)), 1)
    D2 = np.array([[SCALE * 2.0 ** -9 * 1.01 * (np.abs(keys64) @ np.abs(xa64[t, h])).max() for h in range(H)] for t in range(T)])
    latw, _, lats = O.latent_attention(xa64, *cache_values(q, cache), table.cpu().numpy(), s64, lens, bs, SCALE)
    # each latent output: its weights' errors, its rounding; then the exact up-projection of those errors
    tol = np.einsum("thk,hdk->thd", lats * (2 * D2[..., None] * np.exp(2 * D2[..., None]) + 2.0 ** -9 + 2.0 ** -16) +
                    2.0 ** -9 * np.abs(latw), np.abs(up[:, 128:])) + 2.0 ** -30
    assert (np.abs(got - want) <= tol).all() and (np.abs(f64(lse2) - wl) <= D2 + 2.0 ** -17).all()
    # one more token for each request
    x1, c1, kr1 = rand((R, H, 576), 45, torch.bfloat16), rand((R, 512), 46, torch.bfloat16), rand((R, 64), 47, torch.bfloat16)
    slots, starts, keys, taken = q.paged_plan(i32(lens), i32([1] * R), free[8:].contiguous(), i32([12]), table, bs, R)
    assert taken.item() == 1 and keys.tolist() == [38, 65, 2]
    q.latent_append(cache, c1, kr1, slots)
    check_latent(q, cache, x1, table.cpu().numpy(), [0, 1, 2, 3], [38, 65, 2])


# ---- the largest calls: sizes at which a grid dimension, or a 32-bit place, would pass its range -----------------------------
def room(gib):
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"{gib} GiB of device memory are not free")


@pytest.mark.parametrize("R", [63, 64, 65, 4096, 4097, 20000])
def test_prompts_of_thousands_of_requests(q, R):
    rng = np.random.default_rng(R)
    lens = rng.choice([0, 0, 0, 1, 2, 3, 128, 129] if R < 1000 else [0, 0, 1, 1, 2, 3, 5, 129], R).tolist()
    keys = [n + int(rng.integers(0, 3)) for n in lens]
    args = prompts(lens, keys, 1, torch.bfloat16, R)
    T = args[4][-1]
    check_prompt(q, *args, tokens={0, T - 1, *map(int, rng.integers(0, T, 100))})


def test_prompts_of_more_workgroups_than_a_grid_dimension_holds(q):
    room(40)
    R, H = 16400, 1024                                                   # 2^24 workgroups of 256 threads are 2^32 threads
    x = torch.zeros((R, H, 192), dtype=torch.float16, device=DEV)
    k, v, kr = rand((3, H, 128), 1, torch.float16), rand((3, H, 128), 2, torch.float16), rand((3, 64), 3, torch.float16)
    starts = torch.arange(R + 1, dtype=torch.int32, device=DEV)
    kstarts = torch.zeros(R + 1, dtype=torch.int32, device=DEV)
    kstarts[R // 2 + 1:] = 1                                             # one key for the request in the middle, two for the last
    kstarts[R] = 3
    out, lse = q.latent_attention_expanded(x, k, kr, v, starts, kstarts, SCALE, causal=False)
    some = torch.ones(R, dtype=torch.bool, device=DEV)
    some[R // 2] = some[R - 1] = False
    assert (lse[some] == -math.inf).all() and not out[some].any()
    assert torch.equal(out[R // 2], v[0]) and lse[R // 2].abs().max() <= 2 ** -18
    # equal scores: the mean of two values, rounded once (their sum is exact in fp32)
    assert torch.equal(out[R - 1], (v[1:].float().sum(0) / 2).half()) and torch.allclose(lse[R - 1], torch.tensor(math.log(2.0)).to(DEV))


def test_append_of_more_tokens_than_a_grid_dimension_holds(q):
    room(100)
    n = 2 ** 26 + 5                                                      # a wavefront of 64 each: past 2^32 threads
    cache = filled(q, 2, 16, torch.bfloat16, False, 1)
    x = torch.empty((n, 576), dtype=torch.bfloat16, device=DEV)
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    want = [cache.latent.clone(), cache.rope.clone()]
    for i, (t, slot) in enumerate([(0, 3), (n // 2, 30), (n - 1, 17)]):
        x[t] = rand((576,), 7 + i, torch.bfloat16)
        slots[t] = slot
        want[0][slot], want[1][slot] = x[t, :512], x[t, 512:]
    q.latent_append(cache, x[:, :512], x[:, 512:], slots)
    assert torch.equal(cache.latent, want[0]) and torch.equal(cache.rope, want[1])


def test_plan_of_the_most_places(q):
    room(40)
    n = 2 ** 31 - 1
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    slots, starts, keys, taken = q.paged_plan(i32([0, 5]), i32([3, 70]), i32([9, 4, 6]), i32([3]), table, 64, n)
    assert slots[:3].tolist() == [576, 577, 578] and starts.tolist() == [0, 3, 73] and keys.tolist() == [3, 75]
    assert taken.tolist() == [2] and table.tolist() == [[9, -1, -1], [-1, 4, -1]]
    assert slots.numel() == n and all((slots[a: a + 2 ** 28] == -1).all() for a in range(73, n, 2 ** 28))


def test_the_longest_row_of_a_block_table(q):
    """2^31 - 1024 positions: all in one block of zeros but for the last block, whose last key has score 40."""
    n, bs = q.GALE_MAX_KEYS, 1024
    latent = torch.zeros((2 * bs, 512), dtype=torch.bfloat16, device=DEV)
    rope = torch.zeros((2 * bs, 64), dtype=torch.bfloat16, device=DEV)
    latent[-1] = rand((512,), 1, torch.bfloat16)
    rope[-1, 0] = 5
    cache = q.LatentCache(latent, rope, bs)
    table = torch.zeros((1, n // bs), dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    x = torch.zeros((1, 1, 576), dtype=torch.bfloat16, device=DEV)
    x[0, 0, 512] = 8
    out, lse = q.latent_attention(x, cache, table, i32([0, 1]), i32([n]), 1.0)
    # the others' share is 2^31 exp(-40) < 2^-26 of the sum: below half a step of bf16 and of lse
    assert torch.equal(out[0, 0], latent[-1]) and abs(lse.item() - 40) <= 2 ** -18 * 41
    out, lse = q.latent_attention(x, cache, table, i32([0, 1]), i32([n - 1]), 1.0)
    # a lane adds fours, 2^-8 of them, up to 2^17 times: exact; what joins them and the logarithm: the bound above
    assert not out.any() and abs(lse.item() - math.log(n - 1)) <= 2 ** -18 * (1 + math.log(n - 1))


# ---- every way to cut a batch: a table of many columns counts as long contexts, whatever the lengths are -----------------------------
class WideTables:
    """The library, with block tables widened to 2^19 and more positions (their new entries are no blocks)."""

    def __init__(self, q):
        self.q = q

    def __getattr__(self, name):
        return getattr(self.q, name)

    def latent_attention(self, x, cache, table, *args, **kw):
        more = 64 * 8200 // cache.block_size
        return self.q.latent_attention(x, cache, torch.nn.functional.pad(table, (0, more), value=-1), *args, **kw)


@pytest.fixture(scope="module")
def wide(q):
    return WideTables(q)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dtype", T16)
@pytest.mark.parametrize("heads", [5, 17, 32, 33, 64, 65, 128])
def test_decode_in_every_split(wide, dtype, mx, heads):
    lens, bs = (LENS if heads < 64 else LENS[::2]), 16 if heads % 2 else 4
    table, starts, lens, n = batch(wide, lens, [1] * len(lens), bs, heads)
    cache = filled(wide, n, bs, dtype, mx, 3, strided=heads == 17)
    check_latent(wide, cache, rand((len(lens), heads, 576), 4, dtype), table, starts, lens)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [1, 3, 16, 40, 128])
def test_drafts_in_every_split(wide, mx, causal, heads):
    test_drafts(wide, mx, causal, heads)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("heads", [7, 16, 31, 61])                       # two tokens a request: 14, 32, 62, 122 rows
def test_unseen_nan_in_every_split(wide, heads, mx):
    q, bs = wide, 16
    table, starts, lens, n = batch(q, [70, 40, 33], [3, 1, 2], bs, 3)
    table[1, 1], table[2, 0] = -1, n + 5
    cache = filled(q, n, bs, torch.bfloat16, mx, 13)
    x = rand((6, heads, 576), 14, torch.bfloat16)
    out, l = check_latent(q, cache, x, table, starts, lens)
    bad = torch.ones(n * bs, dtype=torch.bool, device=DEV)
    for i, m in enumerate(lens):
        rows = table[i][np.arange(m) // bs] * bs + np.arange(m) % bs
        bad[torch.tensor(rows[(rows >= 0) & (rows < n * bs)], device=DEV)] = False
    late = [table[0][p // bs] * bs + p % bs for p in (68, 69)] + [table[2][32 // bs] * bs + 32 % bs]
    bad[torch.tensor(late, device=DEV)] = True
    if mx:
        cache.latent.scales[bad] = 255
    else:
        cache.latent[bad] = math.nan
    cache.rope[bad] = math.inf
    out2, l2 = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    # what a query sees is what it was: the same products in the same tiles
    for t in (0, 3, 4):
        assert torch.equal(out2[t], out[t]) and torch.equal(l2[t], l[t])
    for t in (1, 2, 5):
        assert torch.isnan(out2[t]).any() and not torch.isfinite(l2[t]).any()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_unseen_nan_where_a_run_is_one_token(wide, heads, mx):
    """Three requests without tokens take the average to one: a run is a token's heads, and none of them sees the last keys."""
    q, bs = wide, 64
    table, starts, lens, n = batch(q, [70, 64, 200, 9, 9, 9], [3, 1, 2, 0, 0, 0], bs, 5)
    cache = filled(q, n, bs, torch.bfloat16, mx, 15)
    x = rand((6, heads, 576), 16, torch.bfloat16)
    out, l = check_latent(q, cache, x, table, starts, lens)
    late = torch.tensor([int(table[r][p // bs]) * bs + p % bs for r, p in ((0, 68), (0, 69), (2, 199))], device=DEV)
    if mx:
        cache.latent.scales[late] = 255
    else:
        cache.latent[late, 40] = -math.inf
    cache.rope[late, 3] = math.nan
    out2, l2 = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    for t in (0, 3, 4):
        assert torch.equal(out2[t], out[t]) and torch.equal(l2[t], l[t])
    for t in (1, 2, 5):
        assert torch.isnan(out2[t]).any() and not torch.isfinite(l2[t]).any()


@pytest.mark.parametrize("dtype", T16)
def test_scores_of_many_sizes_in_every_split(wide, dtype):
    lens = [700, 700, 700, 700]
    table, starts, lens, n = batch(wide, lens, [1] * 4, 32, 4)
    cache = filled(wide, n, 32, dtype, False, 17)
    for r, f in enumerate((lambda p: p / 20, lambda p: -p / 20, lambda p: 40 * np.sin(p), lambda p: 100.0 * (p == 650))):
        p = np.arange(700)
        slots = torch.tensor(table[r][p // 32] * 32 + p % 32, device=DEV)
        cache.rope[slots, 0] = torch.tensor(f(p), device=DEV).to(dtype)
    for heads in (32, 64, 128):
        x = rand((4, heads, 576), 18, dtype)
        x[:, :, 512] = 8.0
        check_latent(wide, cache, x, table, starts, lens)


@pytest.mark.parametrize("heads,mx", [(16, False), (32, True), (64, False), (128, False), (128, True)])
def test_equal_calls_give_equal_bits_in_every_split(wide, heads, mx):
    test_equal_calls_give_equal_bits(wide, heads, mx)


# ---- scores that are all minus infinity: the formula is 0 / 0, which is not the 0 of a query that sees nothing ------------------------
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("wider", [False, True])
def test_scores_that_are_all_minus_infinity(q, wide, wider, heads, mx):
    """Request 0 sees such keys only, 1 none, 2 (in many parts) such keys and from key 900 on finite ones, 3 nothing but holes, 4 (in many
    parts) such keys only, 5 three of them behind a hole."""
    bs, lens = 16, [3, 0, 5000, 40, 6000, 19]
    table, starts, lens, n = batch(q, lens, [1] * 6, bs, 4)
    table[3, :3], table[5, 0] = -1, n
    cache = filled(q, n, bs, torch.bfloat16, mx, 51)
    for r, m in ((0, 3), (2, 900), (4, 6000), (5, 19)):
        pos = np.arange(16 if r == 5 else 0, m)
        cache.rope[torch.tensor(table[r][pos // bs] * bs + pos % bs, device=DEV), 3] = math.inf
    x = rand((6, heads, 576), 52, torch.bfloat16)
    x[:, :, 515] = -1.0
    out, l = (wide if wider else q).latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    for r in (0, 4, 5):
        assert torch.isnan(out[r]).all() and not torch.isfinite(l[r]).any() and not (l[r] == math.inf).any(), r
    for r in (1, 3):
        assert not out[r].any() and (l[r] == -math.inf).all(), r
    c, kr = cache_values(q, cache)
    pos = np.arange(900, 5000)
    rows = table[2][pos // bs] * bs + pos % bs
    k = np.concatenate((c[rows], kr[rows]), 1)
    for h in range(0, heads, 5):
        want, wl, spread = O.attend(f64(x)[2, h], k, c[rows], SCALE)
        bo, bl = bounds(np.abs(f64(x)[2, h]), np.abs(k), SCALE, x.dtype, spread, np.abs(c[rows]).sum(0), want, wl)
        assert (np.abs(f64(out)[2, h] - want) <= bo).all() and abs(l[2, h].item() - wl) <= bl


@pytest.mark.parametrize("mx", [False, True])
def test_drafts_whose_scores_are_all_minus_infinity(q, wide, mx):
    """The first of three tokens sees no key, the second one of score -infinity, the third a finite one too; 40 heads."""
    table, starts, lens, n = batch(q, [2], [3], 16, 4)
    cache = filled(q, n, 16, torch.float16, mx, 53)
    cache.rope[int(table[0, 0]) * 16, 3] = math.inf
    x = rand((3, 40, 576), 54, torch.float16)
    x[:, :, 515] = -1.0
    for lib in (q, wide):
        out, l = lib.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
        assert not out[0].any() and (l[0] == -math.inf).all()
        assert torch.isnan(out[1]).all() and not torch.isfinite(l[1]).any()
        c, _ = cache_values(q, cache)
        assert (f64(out[2]) == c[int(table[0, 0]) * 16 + 1]).all()        # one weight, exactly 1 after its division by itself


@pytest.mark.parametrize("dtype", T16)
def test_prompt_scores_that_are_all_minus_infinity(q, dtype):
    lens, keys = [150, 2, 3], [150, 0, 1]
    x, k, kr, v, s, ks = prompts(lens, keys, 2, dtype, 55)
    kr[:100, 3] = math.inf
    kr[150, 3] = math.inf
    x[:, :, 128 + 3] = -1.0
    out, l = q.latent_attention_expanded(x, k, kr, v, i32(s), i32(ks), SCALE)
    assert torch.isnan(out[:100]).all() and not torch.isfinite(l[:100]).any()
    assert not out[150:154].any() and (l[150:154] == -math.inf).all()      # no keys; three queries of one key: the last sees it
    assert torch.isnan(out[154]).all() and not torch.isfinite(l[154]).any()
    for t in range(100, 150, 7):
        for h in range(2):
            keys64 = np.concatenate((f64(k)[100: t + 1, h], f64(kr)[100: t + 1]), 1)
            val = f64(v)[100: t + 1, h]
            want, wl, spread = O.attend(f64(x)[t, h], keys64, val, SCALE)
            bo, bl = bounds(np.abs(f64(x)[t, h]), np.abs(keys64), SCALE, dtype, spread, np.abs(val).sum(0), want, wl)
            assert (np.abs(f64(out)[t, h] - want) <= bo).all() and abs(l[t, h].item() - wl) <= bl


# ---- values near the end of bf16: a weighted mean is no larger than the largest value ---------------------------------------------------
def check_large_mean(out, lse, keys):
    """The values were 2^127 in even columns and -2^127 in odd ones, the scores equal: out is those, rounded weights or not."""
    want = torch.full((out.shape[-1],), 2.0 ** 127, device=DEV)
    want[1::2] *= -1
    # a sum over keys in fp32 is off by 2^-16 of itself at most (the file's bound), which is less than half a step of bf16
    assert torch.equal(out.float(), want.expand(out.shape)), out
    assert (lse - math.log(keys)).abs().max() <= 2.0 ** -18 * (1 + math.log(keys))


@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 300, 2000, 70000])
def test_means_of_the_largest_values(q, wide, heads, n):
    table, starts, lens, blocks = batch(q, [n, 5], [1, 1], 64, 3)
    cache = filled(q, blocks, 64, torch.bfloat16, False, 1)
    cache.latent[:, ::2], cache.latent[:, 1::2] = 2.0 ** 127, -2.0 ** 127
    x = rand((2, heads, 576), 2, torch.bfloat16)
    x[..., :512] = 0
    cache.rope[:] = 0
    for lib in (q, wide):
        out, lse = lib.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
        check_large_mean(out[0], lse[0], n)
        check_large_mean(out[1], lse[1], 5)


@pytest.mark.parametrize("n", [1, 300, 2000, 70000])
def test_prompt_means_of_the_largest_values(q, n):
    x, k, kr, v, s, ks = prompts([2, 1], [n, 3], 3, torch.bfloat16, 3)
    x[:] = 0
    v[..., ::2], v[..., 1::2] = 2.0 ** 127, -2.0 ** 127
    out, lse = q.latent_attention_expanded(x, k, kr, v, i32(s), i32(ks), SCALE, causal=False)
    check_large_mean(out[:2], lse[:2], n)
    check_large_mean(out[2], lse[2], 3)


@pytest.mark.parametrize("heads", [16, 128])
def test_means_of_the_largest_values_under_rising_scores(q, heads):
    """Scores that rise by less than what the running maximum may lag behind: 5 in powers of two over 700 keys."""
    table, starts, lens, blocks = batch(q, [700], [1], 64, 3)
    cache = filled(q, blocks, 64, torch.bfloat16, False, 1)
    cache.latent[:] = 1.5 * 2.0 ** 127
    cache.rope[:] = 0
    pos = np.arange(700)
    cache.rope[torch.tensor(table[0][pos // 64] * 64 + pos % 64, device=DEV), 0] = torch.tensor(np.floor(pos / 50) / 4, device=DEV).bfloat16()
    x = torch.zeros(1, heads, 576, dtype=torch.bfloat16, device=DEV)
    x[..., 512] = 1.0
    out, lse = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), 1.0)
    # weights are rounded by 2^-9 relative, then the result: both to either side
    assert ((out.float() / 2.0 ** 127 - 1.5).abs() <= 1.5 * (2.0 ** -9 + 2.0 ** -16) + 2.0 ** -8).all() and torch.isfinite(lse).all()
    x, k, kr, v, s, ks = prompts([200], [700], 2, torch.bfloat16, 4)
    x[:], x[..., 128], v[:], kr[:] = 0, 1.0, 1.5 * 2.0 ** 127, 0
    kr[:, 0] = torch.tensor(np.floor(pos / 50) / 4, device=DEV).bfloat16()
    out, lse = q.latent_attention_expanded(x, k, kr, v, i32(s), i32(ks), 1.0)
    assert ((out.float() / 2.0 ** 127 - 1.5).abs() <= 1.5 * (2.0 ** -9 + 2.0 ** -16) + 2.0 ** -8).all() and torch.isfinite(lse).all()


def test_means_of_the_largest_values_in_4_bits(q):
    """MX codes of 6 times 2^125: 1.5 times 2^127."""
    table, starts, lens, blocks = batch(q, [3000, 5], [1, 1], 64, 3)
    cache = filled(q, blocks, 64, torch.bfloat16, True, 1)
    cache.latent.codes[:], cache.latent.scales[:], cache.rope[:] = 0x77, 127 + 125, 0
    x = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device=DEV)
    out, lse = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    assert (out.float() == 1.5 * 2.0 ** 127).all()


@pytest.mark.parametrize("heads", [16, 128])
def test_the_largest_scale_and_scores(q, heads):
    """Scores of 0 under a scale of 2^127 give the mean; scores of 2^126 and -2^126 the first value."""
    table, starts, lens, n = batch(q, [2], [1], 16, 3)
    cache = filled(q, n, 16, torch.bfloat16, False, 57)
    rows = int(table[0, 0]) * 16 + np.arange(2)
    cache.latent[rows] = rand((2, 512), 58).round().bfloat16()            # whole numbers: their mean is exact in fp32
    x = torch.zeros(1, heads, 576, dtype=torch.bfloat16, device=DEV)
    for scale in (2.0 ** 127, -2.0 ** 127):
        out, lse = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), scale)
        assert torch.equal(out[0], (cache.latent[rows].float().sum(0) / 2).bfloat16().expand(heads, 512))
        assert torch.allclose(lse, torch.full_like(lse, math.log(2.0)), rtol=2.0 ** -18)
    cache.rope[rows, 0] = torch.tensor([2.0 ** 63, -2.0 ** 63], device=DEV).bfloat16()
    x[..., 512] = 2.0 ** 63
    out, lse = q.latent_attention(x, cache, i32(table), i32(starts), i32(lens), 1.0)
    assert torch.equal(out[0], cache.latent[rows[0]].expand(heads, 512)) and ((lse / 2.0 ** 126 - 1).abs() <= 2.0 ** -21).all()
    y, k, kr, v, s, ks = prompts([1], [2], 2, torch.bfloat16, 59)
    y[:] = 0
    v[:] = rand((2, 2, 128), 60).round().bfloat16()
    out, lse = q.latent_attention_expanded(y, k, kr, v, i32(s), i32(ks), 2.0 ** 127, causal=False)
    assert torch.equal(out[0], (v.float().sum(0) / 2).bfloat16()) and torch.allclose(lse, torch.full_like(lse, math.log(2.0)), rtol=2.0 ** -18)
    y[..., 128], kr[:, 0] = 2.0 ** 63, torch.tensor([2.0 ** 63, -2.0 ** 63], device=DEV).bfloat16()
    out, lse = q.latent_attention_expanded(y, k, kr, v, i32(s), i32(ks), 1.0, causal=False)
    assert torch.equal(out[0], v[0]) and ((lse / 2.0 ** 126 - 1).abs() <= 2.0 ** -21).all()


# ---- a request's neighbours ----------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("keys", [1, 15, 16, 17, 33, 49, 63, 64, 65, 100])
@pytest.mark.parametrize("n,causal", [(3, False), (40, False), (1, True)])
def test_rows_of_the_next_request_have_no_influence(q, keys, n, causal):
    """The last tile of a request ends inside its 64 rows: NaN and infinity behind its last key leave every bit as it is."""
    x, k, kr, v, s, ks = prompts([n, 2, 1], [keys, 70, 64], 2, torch.float16, keys)
    a, la = q.latent_attention_expanded(x, k, kr, v, i32(s), i32(ks), SCALE, causal)
    k[keys:], kr[keys:], v[keys:] = math.nan, math.inf, math.nan
    v[keys + 1::3] = math.inf
    b, lb = q.latent_attention_expanded(x, k, kr, v, i32(s), i32(ks), SCALE, causal)
    assert torch.isfinite(a).all() and torch.equal(a[:n], b[:n]) and torch.equal(la[:n], lb[:n])


# ---- more than 256 runs: records by the part that a run begins in --------------------------------------------------------------------------
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dtype", T16)
@pytest.mark.parametrize("heads", [16, 24, 48, 128])                      # runs of 16, 32, 64 and 128 rows under a wide table
def test_more_runs_than_records(wide, dtype, mx, heads):
    rng = np.random.default_rng(heads)
    R = 300
    lens = rng.integers(0, 40, R)
    lens[[3, 150, 297]] = 3000, 5000, 2100                                # these are cut into parts
    news = np.ones(R, dtype=np.int64)
    news[[10, 20, 150]], news[[30, 40, 299]] = 2, 0
    table, starts, lens, n = batch(wide, list(lens), list(news), 16, heads)
    cache = filled(wide, n, 16, dtype, mx, 61)
    T = int(starts[-1])
    x = rand((T, heads, 576), 62, dtype)
    need = wide.latent_workspace_bytes(T, R, heads)
    around = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    tokens = {0, 3, int(starts[150]), int(starts[150]) + 1, int(starts[297]), T - 1, *map(int, rng.integers(0, T, 12))}
    check_latent(wide, cache, x, table, starts, lens, tokens=tokens, ws=around[256: 256 + need])
    assert (around[:256] == 0xA5).all() and (around[256 + need:] == 0xA5).all()


@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_the_workspace_is_all_that_is_written(wide, heads):
    """Few long runs, each in many parts."""
    table, starts, lens, n = batch(wide, [9000, 20000], [1, 1], 64, heads)
    cache = filled(wide, n, 64, torch.bfloat16, False, 63)
    x = rand((2, heads, 576), 64, torch.bfloat16)
    need = wide.latent_workspace_bytes(2, 2, heads)
    around = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    a, la = wide.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE, ws=around[256: 256 + need])
    assert (around[:256] == 0xA5).all() and (around[256 + need:] == 0xA5).all()
    b, lb = wide.latent_attention(x, cache, i32(table), i32(starts), i32(lens), SCALE)
    assert torch.equal(a, b) and torch.equal(la, lb)
