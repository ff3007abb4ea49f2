"""Plain fp64 CPU oracle for what surrounds the routed layer: MX numbers, their products, the residual RMS norm and
scored routing.

TEST INFRASTRUCTURE ONLY, like gale_oracle.py: it shares no code with the library.  MX numbers are spelled out as
tables of every element's value, and a value is rounded by looking for the nearest entry.
"""
from __future__ import annotations

import numpy as np

# magnitudes of the 8 (E2M1) or 127 (E4M3; the pattern 127 is NaN) non-negative element codes
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])
TABLE = {1: E2M1, 2: E4M3}       # by format code


def mx_round(a: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Codes of the entries nearest to the magnitudes a <= table[-1], ties to the even code."""
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    below, above = a - table[lo], table[hi] - a
    return np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))


def mx_quantize(x: np.ndarray, fmt: int):
    """x [rows, cols] -> (codes [rows, padded cols] one element per entry, sign in the format's top bit; scale bytes
    [rows, padded cols / 32]), padded with zeros to whole groups of 128 columns."""
    table = TABLE[fmt]
    sign_bit = 8 if fmt == 1 else 128
    rows, cols = x.shape
    pad = -cols % 128
    x = np.pad(np.asarray(x, dtype=np.float64), ((0, 0), (0, pad))).reshape(rows, -1, 32)
    codes = np.zeros(x.shape, dtype=np.int64)
    scales = np.zeros(x.shape[:2], dtype=np.int64)
    for r in range(rows):
        for b in range(x.shape[1]):
            v = x[r, b]
            if not np.all(np.isfinite(v)):
                scales[r, b] = 255
                continue
            top = np.abs(v).max()
            e = -127
            if top > 0:
                e = int(np.floor(np.log2(top))) - 10      # from safely below, up to the smallest that fits
                while top > table[-1] * 2.0 ** e:
                    e += 1
                e = max(e, -127)
            scales[r, b] = e + 127
            codes[r, b] = mx_round(np.abs(v) / 2.0 ** e, table) | np.where(np.signbit(v), sign_bit, 0)
    return codes.reshape(rows, -1), scales


def mx_values(codes: np.ndarray, scales: np.ndarray, fmt: int, cols: int) -> np.ndarray:
    """The numbers of mx_quantize's codes (one element per entry) and scales, [rows, cols]."""
    table = TABLE[fmt]
    sign_bit = 8 if fmt == 1 else 128
    mag = np.concatenate([table, [np.nan]])[np.minimum(codes & (sign_bit - 1), len(table))]
    v = np.where(codes & sign_bit, -mag, mag)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales - 127.0))
    return (v.reshape(len(codes), -1, 32) * s[..., None]).reshape(len(codes), -1)[:, :cols]


def mx_elements(packed: np.ndarray, fmt: int) -> np.ndarray:
    """Stored code bytes [rows, bytes] -> one element per entry."""
    if fmt == 2:
        return packed.astype(np.int64)
    return np.stack((packed & 15, packed >> 4), axis=2).reshape(len(packed), -1).astype(np.int64)


def swiglu(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    g, u = np.split(x, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def rms_norm(s: np.ndarray, weight, eps: float) -> np.ndarray:
    s = np.asarray(s, dtype=np.float64)
    w = 1.0 if weight is None else np.asarray(weight, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        return s / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps) * w


def route_scored(logits, top_k, score="softmax", bias=None, n_groups=1, keep_groups=1, group_score="top2",
                 renormalize=True, scale=1.0):
    """(idx int32 [T, k], w fp64 [T, k]), expert by expert and slot by slot."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    size = E // n_groups
    idx = np.full((T, top_k), -1, dtype=np.int32)
    w = np.zeros((T, top_k))
    for t in range(T):
        l = np.minimum(np.where(np.isnan(logits[t]), -np.inf, logits[t]), np.finfo(np.float32).max)
        ok = l > -np.inf
        if bias is not None:
            b = np.asarray(bias, dtype=np.float64)
            ok &= ~np.isnan(b) & (b > -np.inf)
        if not ok.any():
            continue
        with np.errstate(over="ignore"):
            s = np.where(ok, np.exp(l - l[ok].max()) if score == "softmax" else 1 / (1 + np.exp(-l)), 0.0)
        if score == "softmax":
            s = s / s.sum()
        c = s if bias is None else s + np.where(ok, b, 0.0)
        groups = []
        for g in range(n_groups):
            own = sorted((c[e] for e in range(g * size, (g + 1) * size) if ok[e]), reverse=True)
            if own:
                value = sum(own[:2]) if group_score == "top2" else own[0]
                groups.append((-value, g))
        kept = {g for _, g in sorted(groups)[:keep_groups]}
        order = sorted(((-l[e] if bias is None else -c[e]), e) for e in range(E) if ok[e] and e // size in kept)
        chosen = [e for _, e in order[:top_k]]
        total = sum(s[e] for e in chosen)
        for j, e in enumerate(chosen):
            idx[t, j] = e
            w[t, j] = scale * ((s[e] / total if total > 0 else 0.0) if renormalize else s[e])
    return idx, w
