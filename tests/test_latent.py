"""Latent attention and its paged cache on the CPU: pins of their oracle, and every refusal of a bad call before any GPU
work."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_expert_gemv_amd as q
from oracle import latent_oracle as O
from quantized_expert_gemv_amd.binding import gale_latent_cache

F = 1 << 40          # a fake aligned pointer: never dereferenced, every call below is refused
MB = 1 << 30         # apart from each other
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE = -1, -2, -3, -4, -5


# ---- the oracle --------------------------------------------------------------------------------------------------
def test_plan_of_a_small_batch():
    # blocks of 4: a fresh request of 5, one of 4 old and 1 new tokens, an idle one, one that grows inside its block
    table = np.array([[-1, -1, -1], [7, -1, -1], [8, 9, -1], [3, -1, -1]])
    slots, starts, keys, taken, after = O.paged_plan([0, 4, 6, 1], [5, 1, 0, 2], [20, 21, 22, 23], 4, table, 4, 10)
    assert list(starts) == [0, 5, 6, 6, 8] and list(keys) == [5, 5, 6, 3] and taken == 3
    assert list(slots) == [80, 81, 82, 83, 84, 88, 13, 14, -1, -1]
    assert after.tolist() == [[20, 21, -1], [7, 22, -1], [8, 9, -1], [3, -1, -1]]


def test_plan_refuses_requests_without_room():
    table = np.full((4, 2), -1)
    # the second needs more than is free; the third fits no table row; the fourth needs none and has old room
    table[3, 0] = 5
    slots, starts, keys, taken, after = O.paged_plan([0, 0, 0, 1], [4, 8, 12, 1], [1, 2], 2, table, 4, 25)
    assert list(keys) == [4, 0, 0, 2] and taken == 1 and list(starts) == [0, 4, 12, 24, 25]
    assert list(slots[:4]) == [4, 5, 6, 7] and (slots[4:24] == -1).all() and slots[24] == 21
    assert after.tolist() == [[1, -1], [-1, -1], [-1, -1], [5, -1]]
    # the batch ends inside a request
    slots, starts, keys, taken, _ = O.paged_plan([0, 0], [2, 3], [1, 2], 2, np.full((2, 1), -1), 4, 4)
    assert list(keys) == [2, 0] and list(starts) == [0, 2, 4] and list(slots) == [4, 5, -1, -1] and taken == 1


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((5, 3))
    # equal scores: the mean; one score far above: its value
    out, lse, _ = O.attend(np.zeros(2), rng.standard_normal((5, 2)), v, 1.0)
    assert np.allclose(out, v.mean(0)) and np.isclose(lse, np.log(5))
    out, lse, _ = O.attend(np.array([800.0, 0]), np.eye(5, 2), v, 1.0)
    assert np.allclose(out, v[0]) and np.isclose(lse, 800)
    out, lse, _ = O.attend(np.zeros(2), np.zeros((0, 2)), np.zeros((0, 3)), 1.0)
    assert not out.any() and lse == -np.inf


def test_the_two_forms_agree():
    """Absorbing the up-projection into query and output gives the expanded form."""
    rng = np.random.default_rng(2)
    H, n, m, bs = 3, 4, 9, 2
    wk, wv = rng.standard_normal((H, 128, 512)) / 23, rng.standard_normal((H, 128, 512)) / 23
    c, r = rng.standard_normal((20, 512)), rng.standard_normal((20, 64))
    table = np.array([[4, 1, 9, 0, 7]])
    rows = (table[0][np.arange(m) // bs] * bs + np.arange(m) % bs)
    x = rng.standard_normal((n, H, 192))
    k = np.einsum("hdk,sk->shd", wk, c[rows])
    v = np.einsum("hdk,sk->shd", wv, c[rows])
    want, lse, _ = O.expanded_attention(x, k, r[rows], v, [0, n], [0, m], 0.1)
    xa = np.concatenate((np.einsum("thd,hdk->thk", x[..., :128], wk), x[..., 128:]), 2)
    lat, lse2, _ = O.latent_attention(xa, c, r, table, [0, n], [m], bs, 0.1)
    assert np.allclose(lse, lse2) and np.allclose(np.einsum("thk,hdk->thd", lat, wv), want)


def test_oracle_masks():
    rng = np.random.default_rng(3)
    c, r, x = rng.standard_normal((8, 512)), rng.standard_normal((8, 64)), rng.standard_normal((3, 1, 576))
    # three queries, two keys: the first query sees none; tokens behind the last request stay untouched
    out, lse, _ = O.latent_attention(x, c, r, np.array([[0]]), [0, 3], [2], 4, 1.0)
    assert lse[0, 0] == -np.inf and not out[0].any() and np.allclose(out[1, 0], c[0])
    out, _, _ = O.latent_attention(x, c, r, np.array([[0]]), [0, 1], [2], 4, 1.0)
    assert np.isnan(out[1:]).all() and not np.isnan(out[0]).any()
    # a block that does not exist is not seen
    a, _, _ = O.latent_attention(x[:1], c, r, np.array([[0, -1]]), [0, 1], [8], 4, 1.0)
    b, _, _ = O.latent_attention(x[:1], c, r, np.array([[0, 5]]), [0, 1], [4], 4, 1.0)
    assert np.array_equal(a, b)


# ---- refusals ----------------------------------------------------------------------------------------------------
def _refused(name, good, changes):
    f = getattr(q.lib(), name)
    for want, change in changes:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert f(*args) == want, (name, change, q.lib().gale_last_error())
        assert name in q.lib().gale_last_error().decode()


def _cache(**change):
    d = dict(latent=F, scales=None, rope=F + 16 * MB, latent_stride=512, rope_stride=64, dtype=1, fmt=0, n_blocks=100,
             block_size=64)
    d.update(change)
    return gale_latent_cache(**d)


BAD_CACHES = [(DTYPE, dict(dtype=2)), (DTYPE, dict(fmt=2)), (SHAPE, dict(n_blocks=0)), (SHAPE, dict(block_size=0)),
              (SHAPE, dict(block_size=48)), (SHAPE, dict(block_size=2048)), (SHAPE, dict(n_blocks=1 << 25)),
              (SHAPE, dict(latent_stride=511)), (SHAPE, dict(rope_stride=63)), (NULL, dict(latent=None)), (NULL, dict(rope=None)),
              (NULL, dict(fmt=1)), (ALIGN, dict(latent=F + 8)), (ALIGN, dict(rope=F + 2)), (ALIGN, dict(latent_stride=516)),
              (ALIGN, dict(rope_stride=65)), (ALIGN, dict(fmt=1, scales=F + 9 * MB + 4))]


def test_plan_refusals():
    # past, new, R, block, free, cap, n_free, table, stride, max_blocks, n_tok, slots, q_starts, kv_lens, taken, stream
    good = [F, F + MB, 8, 64, F + 2 * MB, 50, F + 3 * MB, F + 4 * MB, 16, 16, 100, F + 5 * MB, F + 6 * MB, F + 7 * MB, F + 8 * MB,
            None]
    _refused("gale_paged_plan", good, [
        (SHAPE, {2: -1}), (SHAPE, {2: 65537}), (SHAPE, {3: 0}), (SHAPE, {3: 24}), (SHAPE, {3: 2048}), (SHAPE, {5: -1}),
        (SHAPE, {9: -1}), (SHAPE, {8: 15}), (SHAPE, {10: -1}),
        (NULL, {0: None}), (NULL, {1: None}), (NULL, {4: None}), (NULL, {6: None}), (NULL, {7: None}), (NULL, {11: None}),
        (NULL, {12: None}), (NULL, {13: None}), (NULL, {14: None}),
        (ALIGN, {0: F + 2}), (ALIGN, {1: F + MB + 1}), (ALIGN, {4: F + 2 * MB + 2}), (ALIGN, {6: F + 3 * MB + 2}),
        (ALIGN, {7: F + 4 * MB + 1}), (ALIGN, {11: F + 5 * MB + 4}), (ALIGN, {12: F + 6 * MB + 2}), (ALIGN, {13: F + 7 * MB + 2}),
        (ALIGN, {14: F + 8 * MB + 2}),
        (SHAPE, {13: F}), (SHAPE, {12: F + MB}), (SHAPE, {14: F + 3 * MB}), (SHAPE, {11: F + 6 * MB}), (SHAPE, {7: F + 2 * MB + 8}),
        (SHAPE, {13: F + 6 * MB + 32})])


def test_append_refusals():
    # cache, latent, stride, rope, stride, slots, n_tok, stream
    good = [_cache(), F + 32 * MB, 512, F + 33 * MB, 64, F + 34 * MB, 4, None]
    _refused("gale_latent_append", good, [(w, {0: _cache(**c)}) for w, c in BAD_CACHES])
    _refused("gale_latent_append", good, [
        (NULL, {0: None}), (SHAPE, {6: -1}), (SHAPE, {2: 511}), (SHAPE, {4: 63}), (NULL, {1: None}), (NULL, {3: None}),
        (NULL, {5: None}), (ALIGN, {1: F + 32 * MB + 8}), (ALIGN, {2: 514}), (ALIGN, {3: F + 33 * MB + 2}), (ALIGN, {4: 66}),
        (ALIGN, {5: F + 34 * MB + 4}), (SHAPE, {1: F + 1024}), (SHAPE, {3: F + 16 * MB}), (SHAPE, {5: F + 16 * MB}),
        (SHAPE, {0: _cache(rope=F + 512 * 2)})])
    # latent and rope parts of one row do not overlap
    one = _cache(latent_stride=576, rope_stride=576, rope=F + 1024)
    good[0], good[6] = one, 0
    assert q.lib().gale_latent_append(*good) == 0


def test_attention_refusals():
    # cache, table, stride, max_blocks, kv_lens, q_starts, R, q, q_stride, T, H, scale, causal, out, out_stride, lse, ws, bytes
    need = q.latent_workspace_bytes(10, 4, 16)
    good = [_cache(), F + 40 * MB, 8, 8, F + 41 * MB, F + 42 * MB, 4, F + 43 * MB, 16 * 576, 10, 16, 0.1, 1, F + 44 * MB, 16 * 512,
            F + 45 * MB, F + 46 * MB, need, None]
    _refused("gale_latent_attention", good, [(w, {0: _cache(**c)}) for w, c in BAD_CACHES])
    _refused("gale_latent_attention", good, [
        (NULL, {0: None}), (SHAPE, {2: 7}), (SHAPE, {3: -1}), (SHAPE, {6: -1}), (SHAPE, {6: 65537}), (SHAPE, {9: -1}), (SHAPE, {10: 0}),
        (SHAPE, {10: 1025}), (SHAPE, {9: 1 << 30}), (SHAPE, {8: 16 * 576 - 1}), (SHAPE, {14: 16 * 512 - 1}),
        (SHAPE, {11: float("inf")}), (SHAPE, {11: float("nan")}),
        (NULL, {1: None}), (NULL, {4: None}), (NULL, {5: None}), (NULL, {7: None}), (NULL, {13: None}),
        (ALIGN, {1: F + 40 * MB + 2}), (ALIGN, {4: F + 41 * MB + 2}), (ALIGN, {5: F + 42 * MB + 1}), (ALIGN, {7: F + 43 * MB + 8}),
        (ALIGN, {8: 16 * 576 + 4}), (ALIGN, {13: F + 44 * MB + 8}), (ALIGN, {14: 16 * 512 + 4}), (ALIGN, {15: F + 45 * MB + 2}),
        (ALIGN, {16: F + 46 * MB + 128}), (WORKSPACE, {17: need - 1}), (WORKSPACE, {16: None}),
        (SHAPE, {13: F + 43 * MB}), (SHAPE, {13: F}), (SHAPE, {15: F + 44 * MB}), (SHAPE, {15: F + 41 * MB}),
        (SHAPE, {16: F + 43 * MB}), (SHAPE, {16: F + 44 * MB})])
    for i in (6, 9):
        args = list(good)
        args[i] = 0
        assert q.lib().gale_latent_attention(*args) == 0


def test_expanded_refusals():
    # q, qs, k, ks, kh, kr, krs, v, vs, vh, dtype, T, S, H, q_starts, kv_starts, R, scale, causal, out, out_stride, lse, stream
    good = [F, 16 * 192, F + MB, 4096, 256, F + 2 * MB, 64, F + MB + 256, 4096, 256, 3, 10, 20, 16, F + 4 * MB, F + 5 * MB, 2, 0.1, 1,
            F + 6 * MB, 16 * 128, F + 7 * MB, None]
    _refused("gale_latent_attention_expanded", good, [
        (DTYPE, {10: 2}), (DTYPE, {10: 0}), (SHAPE, {1: 16 * 192 - 1}), (SHAPE, {3: 15 * 256 + 127}), (SHAPE, {4: 127}),
        (SHAPE, {4: 1 << 31}), (SHAPE, {6: 63}), (SHAPE, {8: 15 * 256 + 127}), (SHAPE, {9: 120}), (SHAPE, {9: 1 << 33}), (SHAPE, {11: -1}),
        (SHAPE, {12: -1}), (SHAPE, {13: 0}), (SHAPE, {13: 1025}), (SHAPE, {11: 1 << 28}), (SHAPE, {16: -1}), (SHAPE, {16: 65537}),
        (SHAPE, {17: float("nan")}), (SHAPE, {20: 16 * 128 - 1}), (SHAPE, {3: 1 << 24}), (SHAPE, {6: 1 << 24}), (SHAPE, {8: 1 << 24}),
        (NULL, {0: None}), (NULL, {2: None}), (NULL, {5: None}), (NULL, {7: None}), (NULL, {14: None}), (NULL, {15: None}),
        (NULL, {19: None}),
        (ALIGN, {0: F + 8}), (ALIGN, {1: 16 * 192 + 4}), (ALIGN, {2: F + MB + 2}), (ALIGN, {3: 4100}), (ALIGN, {4: 257}), (ALIGN, {5: F + 2 * MB + 8}),
        (ALIGN, {6: 68}), (ALIGN, {7: F + MB + 264}), (ALIGN, {8: 4100}), (ALIGN, {9: 260, 8: 4160}), (ALIGN, {14: F + 4 * MB + 2}),
        (ALIGN, {15: F + 5 * MB + 2}), (ALIGN, {19: F + 6 * MB + 4}), (ALIGN, {20: 16 * 128 + 4}), (ALIGN, {21: F + 7 * MB + 2}),
        (SHAPE, {19: F}), (SHAPE, {19: F + MB + 512}), (SHAPE, {21: F + 2 * MB}), (SHAPE, {21: F + 6 * MB + 64}), (SHAPE, {21: F + 4 * MB})])
    for i in (11, 16):
        args = list(good)
        args[i] = 0
        assert q.lib().gale_latent_attention_expanded(*args) == 0


def test_workspace_sizes():
    assert q.latent_workspace_bytes(1, 1, 16) >= 0
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, 0), (1, 1, 1025), (1 << 30, 1, 16), (1, 65537, 1)):
        assert q.latent_workspace_bytes(*bad) == 0


def test_binding_refusals():
    rope = torch.zeros(128, 64, dtype=torch.float16)
    latent = torch.zeros(128, 512, dtype=torch.float16)
    c = q.LatentCache(latent, rope, 64)
    assert c.n_blocks == 2 and c.desc.latent_stride == 512 and c.desc.fmt == 0
    both = torch.zeros(128, 576, dtype=torch.float16)
    assert q.LatentCache(both[:, :512], both[:, 512:], 32).desc.rope_stride == 576
    mx = q.LatentCache.empty(2, 64, torch.bfloat16, mx=True, device="cpu")
    assert mx.desc.fmt == q.GALE_MX_E2M1 and mx.desc.scales and mx.latent.rows == 128
    for bad in (lambda: q.LatentCache(latent, rope[:64], 64), lambda: q.LatentCache(latent.float(), rope, 64),
                lambda: q.LatentCache(latent, rope.float(), 64), lambda: q.LatentCache(latent, rope, 48),
                lambda: q.LatentCache(latent, rope, 256), lambda: q.LatentCache(latent[:, :500], rope, 64),
                lambda: q.LatentCache(q.MXTensor.empty(128, 512, q.GALE_MX_E4M3, "cpu"), rope, 64),
                lambda: q.LatentCache(latent.bfloat16(), rope, 64)):
        with pytest.raises(ValueError):
            bad()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)       # noqa: E731
    x = torch.zeros(3, 2, 576, dtype=torch.float16)
    for bad in (lambda: q.latent_attention(x.float(), c, i32(1, 2), i32(2), i32(1), 1.0),
                lambda: q.latent_attention(x[..., :575], c, i32(1, 2), i32(2), i32(1), 1.0),
                lambda: q.latent_attention(x, c, i32(1, 2), i32(3), i32(1), 1.0),
                lambda: q.latent_attention(x, c, i32(2, 2), i32(2), i32(1), 1.0),
                lambda: q.latent_attention(x, c, i32(1, 2).long(), i32(2), i32(1), 1.0),
                lambda: q.latent_attention(x, c, i32(1, 2), i32(2), i32(1), 1.0, out=torch.zeros(3, 2, 512)),
                lambda: q.latent_attention(x, c, i32(1, 2), i32(2), i32(1), 1.0),                  # not on a GPU
                lambda: q.latent_append(c, latent, rope[:3], torch.zeros(128, dtype=torch.int64)),
                lambda: q.latent_append(c, latent, rope, torch.zeros(128, dtype=torch.int32)),
                lambda: q.paged_plan(i32(2), i32(3), i32(4), i32(1), i32(2, 4), 16, 8),
                lambda: q.paged_plan(i32(2), i32(2), i32(4), i32(1), i32(3, 4), 16, 8),
                lambda: q.latent_attention_expanded(x[..., :192], x[..., :128], rope[:2], x[..., :128], i32(2), i32(2), 1.0),
                lambda: q.latent_attention_expanded(x[..., :192], x[..., :128], rope[:3], x[..., :127], i32(2), i32(2), 1.0)):
        with pytest.raises(ValueError):
            bad()


def test_attention_refuses_tables_past_the_last_position():
    need = q.latent_workspace_bytes(1, 1, 16)
    wide = q.GALE_MAX_KEYS // 64 + 1
    good = [_cache(), F + 40 * MB, 8, 8, F + 41 * MB, F + 42 * MB, 1, F + 43 * MB, 16 * 576, 1, 16, 0.1, 1, F + 44 * MB, 16 * 512,
            None, F + 46 * MB, need, None]
    _refused("gale_latent_attention", good, [(SHAPE, {2: wide, 3: wide})])


def test_scales_without_a_finite_logarithm_base_are_refused():
    """Scores are taken in powers of two: a scale times log2(e) has to be finite."""
    need = q.latent_workspace_bytes(1, 1, 16)
    good = [_cache(), F + 40 * MB, 8, 8, F + 41 * MB, F + 42 * MB, 1, F + 43 * MB, 16 * 576, 1, 16, 0.1, 1, F + 44 * MB, 16 * 512,
            None, F + 46 * MB, need, None]
    _refused("gale_latent_attention", good, [(SHAPE, {11: 2.0 ** 127 * 1.01}), (SHAPE, {11: -3.4e38})])
    good = [F, 16 * 192, F + MB, 4096, 256, F + 2 * MB, 64, F + MB + 256, 4096, 256, 3, 10, 20, 16, F + 4 * MB, F + 5 * MB, 2, 0.1, 1,
            F + 6 * MB, 16 * 128, F + 7 * MB, None]
    _refused("gale_latent_attention_expanded", good, [(SHAPE, {17: 2.0 ** 127 * 1.01}), (SHAPE, {17: -3.4e38})])


def test_workspace_sizes_of_each_shape():
    """Records (256 + 256 of 16 bytes), then two places for each of 256 workgroups: maxima and sums of weights, and 512 sums of 4
    bytes, for each row of a run."""
    for (tokens, requests, heads), rows in {(1, 1, 16): 16, (4, 4, 1): 16, (1, 1, 32): 32, (64, 64, 17): 32, (1, 1, 64): 64,
                                            (2, 1, 32): 64, (1, 1, 33): 64, (1, 1, 128): 128, (8, 8, 128): 128, (300, 300, 128): 128,
                                            (0, 0, 16): 16, (1, 65536, 1024): 16}.items():
        assert q.latent_workspace_bytes(tokens, requests, heads) == 256 + 4096 + 512 * rows * (8 + 4 * 512), (tokens, requests, heads)
