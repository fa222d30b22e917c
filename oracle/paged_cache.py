"""The operators around a paged cache, in fp64.  TEST INFRASTRUCTURE ONLY.

Positions of a drafted tree's nodes, rotary positions and the schedules of their frequencies, the append of
rotated tokens to the cache, and tree attention over a prefix that the batch shares, each as a direct loop over its
definition.
"""
from __future__ import annotations

import numpy as np

from .target_pass import ancestors


def tree_positions(parents, lens, prefix=0):
    out = []
    for row, n in zip(parents, lens):
        before = min(max(int(prefix), 0), 1 << 30) + min(max(int(n), 0), 1 << 30)
        out.append([min(before + (0 if seen is None else len(seen) - 1), 2 ** 31 - 1) for seen in ancestors(row)])
    return np.array(out, dtype=np.int64)


def frequencies(rot, base, scaling=None, factor=1.0, original=0.0, beta_fast=32.0, beta_slow=1.0):
    """(frequencies of the pairs, amplitude)."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2 * i / rot)
    if scaling is None:
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        return (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0
    wave = 2 * np.pi / f  # positions of one turn
    if scaling == "bands":
        out = np.empty_like(f)
        for j in range(len(f)):
            if wave[j] < original / beta_fast:
                out[j] = f[j]
            elif wave[j] > original / beta_slow:
                out[j] = f[j] / factor
            else:
                r = (original / wave[j] - beta_slow) / (beta_fast - beta_slow)
                out[j] = (1 - r) * f[j] / factor + r * f[j]
        return out, 1.0
    # the pair that turns beta times over the original positions: original / wave = beta
    pair = lambda beta: rot * np.log(original / (2 * np.pi * beta)) / (2 * np.log(base))  # noqa: E731
    low = min(max(np.floor(pair(beta_fast)), 0), rot - 1)
    high = min(max(np.ceil(pair(beta_slow)), 0), rot - 1)
    r = np.clip((i - low) / (high - low if high > low else 1e-3), 0, 1)
    return f * (1 - r) + f / factor * r, 0.1 * np.log(factor) + 1 if factor > 1 else 1.0


def rotate(x, positions, freqs, layout="half", amplitude=1.0):
    """(x [rows, heads, D] turned, amplitude (|x1| + |x2|) of each value's pair; zero where nothing is turned)."""
    y, mag = np.array(x, dtype=np.float64), np.zeros(np.shape(x))
    n = len(freqs)
    for r, p in enumerate(positions):
        for i in range(n):
            a = float(p) * float(freqs[i])
            one, two = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
            x1, x2 = x[r, :, one].astype(np.float64), x[r, :, two].astype(np.float64)
            y[r, :, one] = amplitude * (x1 * np.cos(a) - x2 * np.sin(a))
            y[r, :, two] = amplitude * (x2 * np.cos(a) + x1 * np.sin(a))
            mag[r, :, one] = mag[r, :, two] = amplitude * (np.abs(x1) + np.abs(x2))
    return y, mag


def append_slots(starts, rows, table, lens, n_pages, page, prefix=0):
    """For each row (position of its angles, page, row of the page); None for a row that is no token, and page None
    where it is not written."""
    out = [None] * rows
    for b in range(len(lens)):
        n = max(int(lens[b]), 0)
        for r in range(max(int(starts[b]), 0), min(int(starts[b + 1]), rows)):
            at = n + r - int(starts[b])
            there = at // page < table.shape[1] and 0 <= table[b, at // page] < n_pages
            out[r] = (max(int(prefix), 0) + at, int(table[b, at // page]) if there else None, at % page)
    return out


def tree_attention_shared(q, k_new, v_new, parents, k_pages, v_pages, prefix_table, prefix_len, block_table, lens, scale):
    """(out [B, T, Hq, D], sum_j w_j |v_j|, largest sum |q k| scale of a row, keys of a row)."""
    B, T, Hq, D = q.shape
    page, g = k_pages.shape[2], Hq // k_pages.shape[1]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    dots, keys = np.zeros((B, T, Hq)), np.zeros((B, T, Hq))
    far = np.arange(prefix_len)
    for b in range(B):
        sees = ancestors(parents[b])
        pos = np.arange(lens[b])
        for kv in range(Hq // g):
            cached = [np.concatenate([p[prefix_table[far // page], kv, far % page],
                                      p[block_table[b][pos // page], kv, pos % page]]) for p in (k_pages, v_pages)]
            for t in range(T):
                if sees[t] is None:
                    continue
                k = np.concatenate([cached[0], k_new[b, sees[t], kv]]).astype(np.float64)
                v = np.concatenate([cached[1], v_new[b, sees[t], kv]]).astype(np.float64)
                for h in range(kv * g, (kv + 1) * g):
                    x = q[b, t, h].astype(np.float64)
                    s = k @ x * scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[b, t, h], mag[b, t, h] = w @ v, w @ np.abs(v)
                    dots[b, t, h], keys[b, t, h] = (np.abs(k) @ np.abs(x)).max() * scale, len(s)
    return out, mag, dots, keys
