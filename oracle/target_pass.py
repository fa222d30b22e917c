"""The steps of the target's verification pass, in fp64.  TEST INFRASTRUCTURE ONLY.

Root-mean-square norm with the residual's addition and an e4m3 output, the product of e4m3
operands with a scale for each block of 128, attention of a tree of drafted nodes over a paged
cache, and the commit of accepted nodes into it, each as a direct loop over its definition.

e4m3 (OCP, the "fn" variant): sign, 4 exponent bits with bias 7, 3 mantissa bits; exponent 0 is
subnormal (steps of 2^-9), 0x7f is NaN, the largest finite value is 448.
"""
from __future__ import annotations

import numpy as np

GROUP = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100


def _e4m3_values() -> np.ndarray:
    """The values of codes 0 .. 0x7e, ascending."""
    codes = np.arange(0x7F)
    e, m = codes >> 3, codes & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


E4M3 = _e4m3_values()


def e4m3_decode(codes: np.ndarray) -> np.ndarray:
    """fp64 values of e4m3 codes (uint8)."""
    mag = codes & 0x7F
    v = np.where(mag == 0x7F, np.nan, E4M3[np.minimum(mag, 0x7E)])
    return np.where(codes & 0x80, -v, v)


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """The nearest e4m3 value of each |x| <= 464, ties to the even code; larger magnitudes give NaN."""
    mag = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.clip(np.searchsorted(E4M3, mag), 1, len(E4M3) - 1)
    lo = hi - 1
    up, down = E4M3[hi] - mag, mag - E4M3[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    v = np.where(take_hi, E4M3[hi], E4M3[lo])
    v = np.where(mag > 464.0, np.nan, v)
    return np.copysign(np.where(np.isnan(mag), np.nan, v), x)


def norm_q8(x, weight, residual=None, eps=1e-6):
    """(y [rows, d], scale [groups, rows], v = y / scale before its rounding, s)."""
    s = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    rows, d = s.shape
    y = s / np.sqrt((s * s).sum(axis=1, keepdims=True) / d + eps) * np.asarray(weight, np.float64)
    G = -(-d // GROUP)
    scale = np.empty((G, rows))
    v = np.empty_like(y)
    for g in range(G):
        cols = slice(g * GROUP, min(d, (g + 1) * GROUP))
        scale[g] = np.maximum(np.abs(y[:, cols]).max(axis=1) / E4M3_MAX, SCALE_MIN)
        v[:, cols] = y[:, cols] / scale[g][:, None]
    return y, scale, v, s


def linear_q8(a, a_scale, w, w_scale):
    """(out [rows, N], the same sum over magnitudes) from e4m3 values and scales."""
    a, w = np.asarray(a, np.float64), np.asarray(w, np.float64)
    (rows, K), N = a.shape, w.shape[0]
    out, mag = np.zeros((rows, N)), np.zeros((rows, N))
    for g in range(-(-K // GROUP)):
        k = slice(g * GROUP, min(K, (g + 1) * GROUP))
        f = np.asarray(a_scale, np.float64)[g][:, None] * np.repeat(np.asarray(w_scale, np.float64)[:, g], GROUP)[None, :N]
        out += a[:, k] @ w[:, k].T * f
        mag += np.abs(a[:, k]) @ np.abs(w[:, k]).T * np.abs(f)
    return out, mag


def ancestors(parents):
    """For each node the list of nodes it sees (itself and its ancestors); None for an unused node."""
    T = len(parents)
    used = [-1 <= parents[t] < t for t in range(T)]
    out = []
    for t in range(T):
        if not used[t]:
            out.append(None)
            continue
        seen, a = [], t
        while a >= 0 and used[a]:
            seen.append(a)
            a = parents[a]
        out.append(seen)
    return out


def tree_attention(q, k_new, v_new, parents, k_pages, v_pages, block_table, lens, scale):
    """(out [B, T, Hq, D], sum_j w_j |v_j|, largest sum |q k| scale of a row, keys of a row)."""
    B, T, Hq, D = q.shape
    page, g = k_pages.shape[2], Hq // k_pages.shape[1]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    dots, keys = np.zeros((B, T, Hq)), np.zeros((B, T, Hq))
    for b in range(B):
        sees = ancestors(parents[b])
        pos = np.arange(lens[b])
        pages = block_table[b][pos // page]
        for t in range(T):
            if sees[t] is None:
                continue
            for h in range(Hq):
                kv = h // g
                k = np.concatenate([k_pages[pages, kv, pos % page], k_new[b, sees[t], kv]]).astype(np.float64)
                v = np.concatenate([v_pages[pages, kv, pos % page], v_new[b, sees[t], kv]]).astype(np.float64)
                x = q[b, t, h].astype(np.float64)
                s = k @ x * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[b, t, h], mag[b, t, h] = w @ v, w @ np.abs(v)
                dots[b, t, h], keys[b, t, h] = (np.abs(k) @ np.abs(x)).max() * scale, len(s)
    return out, mag, dots, keys


def cache_commit(k_new, v_new, nodes, counts, k_pages, v_pages, block_table, lens):
    """(k_pages, v_pages, lens) after the accepted nodes went in; the inputs stay as they are."""
    k_pages, v_pages = k_pages.copy(), v_pages.copy()
    B, T = k_new.shape[:2]
    page, width = k_pages.shape[2], block_table.shape[1]
    P = T if nodes is None else nodes.shape[1]
    new = np.array(lens)
    for b in range(B):
        n = min(max(int(counts[b]), 0), P)
        new[b] = max(int(lens[b]), 0) + n
        for i in range(n):
            at = max(int(lens[b]), 0) + i
            node = i if nodes is None else int(nodes[b, i])
            if at // page >= width or not 0 <= node < T or not 0 <= block_table[b, at // page] < len(k_pages):
                continue
            k_pages[block_table[b, at // page], :, at % page] = k_new[b, node]
            v_pages[block_table[b, at // page], :, at % page] = v_new[b, node]
    return k_pages, v_pages, new
