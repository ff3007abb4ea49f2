"""Latent attention, its paged cache and its block tables in fp64, by the definitions (plain numpy, token by token)."""
import numpy as np


def paged_plan(past_lens, new_lens, free_blocks, n_free, table, block_size, n_tok):
    """(slots, q_starts, kv_lens, taken, table) of one batch."""
    table = np.array(table, dtype=np.int64)
    max_blocks = table.shape[1]
    R = len(past_lens)
    slots = np.full(n_tok, -1, dtype=np.int64)
    q_starts, kv_lens = np.zeros(R + 1, dtype=np.int64), np.zeros(R, dtype=np.int64)
    n_free = max(0, min(int(n_free), len(free_blocks)))
    total = asked = taken = 0
    for r in range(R):
        past, new = max(0, int(past_lens[r])), max(0, int(new_lens[r]))
        q_starts[r] = min(total, n_tok)
        begin, total = total, total + new
        have, want = -(-past // block_size), -(-(past + new) // block_size)
        kv_lens[r] = past
        if want > max_blocks or total > n_tok:
            continue
        need = want - have
        asked += need
        if need and asked > n_free:
            continue
        kv_lens[r] = past + new
        for i in range(need):
            table[r, have + i] = free_blocks[taken + i]
        taken += need
        for i in range(new):
            pos = past + i
            block = table[r, pos // block_size]
            if block >= 0:
                slots[begin + i] = block * block_size + pos % block_size
    q_starts[R] = min(total, n_tok)
    return slots, q_starts, kv_lens, taken, table


def attend(x, k, v, scale):
    """(out, lse, spread) of one query x over the keys it sees; spread[d] = sum_j w_j |v_jd|, the size of what is summed."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1])
    s = scale * (k @ x)
    top = s.max()
    e = np.exp(s - top)
    w = e / e.sum()
    return w @ v, top + np.log(e.sum()), w @ np.abs(v)


def latent_attention(q, c, r, table, q_starts, kv_lens, block_size, scale, causal=True):
    """Absorbed form: q [T, H, 576]; c [slots, 512], r [slots, 64]; NaN rows of the outputs for tokens of no request."""
    T, H, _ = q.shape
    out, lse = np.full((T, H, 512), np.nan), np.full((T, H), np.nan)
    spread = np.full((T, H, 512), np.nan)
    n_blocks = len(c) // block_size
    for i in range(len(kv_lens)):
        a, b = int(q_starts[i]), int(q_starts[i + 1])
        n, m = b - a, min(max(int(kv_lens[i]), 0), table.shape[1] * block_size)
        for t in range(a, b):
            seen = max(0, m - n + (t - a) + 1) if causal else m
            pos = np.arange(seen)
            block = table[i][pos // block_size]
            fine = (block >= 0) & (block < n_blocks)
            rows = (block * block_size + pos % block_size)[fine]
            k = np.concatenate((c[rows], r[rows]), 1)
            for h in range(H):
                out[t, h], lse[t, h], spread[t, h] = attend(q[t, h], k, c[rows], scale)
    return out, lse, spread


def expanded_attention(q, k, kr, v, q_starts, kv_starts, scale, causal=True):
    """Expanded form: q [T, H, 192], k [S, H, 128], kr [S, 64], v [S, H, 128]."""
    T, H, _ = q.shape
    out, lse = np.full((T, H, 128), np.nan), np.full((T, H), np.nan)
    spread = np.full((T, H, 128), np.nan)
    for i in range(len(q_starts) - 1):
        a, b, s0, s1 = int(q_starts[i]), int(q_starts[i + 1]), int(kv_starts[i]), int(kv_starts[i + 1])
        n, m = b - a, s1 - s0
        for t in range(a, b):
            seen = max(0, m - n + (t - a) + 1) if causal else m
            for h in range(H):
                keys = np.concatenate((k[s0: s0 + seen, h], kr[s0: s0 + seen]), 1)
                out[t, h], lse[t, h], spread[t, h] = attend(q[t, h], keys, v[s0: s0 + seen, h], scale)
    return out, lse, spread
