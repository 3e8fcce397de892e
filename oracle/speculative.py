"""Float64 definitions of the speculative step's operators (numpy, CPU): norm +
rotation + cache write, tree attention, path acceptance and the read-back of
FP8 rows.  Test infrastructure only; shares no code with the kernels.
"""

from __future__ import annotations

import numpy as np

from . import e4m3_value


def e4m3_table() -> np.ndarray:
    """Values of the 256 E4M3 codes."""
    return np.array([e4m3_value(c) for c in range(256)])


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """Rows x [T, h, D] normed (weight None: not) and rotated, float64.

    Also returns, per element, |a cos| + |b sin| of its pair (or |n|): the scale
    that rounding errors of the rotation are relative to."""
    n = np.asarray(x, dtype=np.float64)
    if weight is not None:
        n = n / np.sqrt((n * n).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, mag = n.copy(), np.abs(n)
    if cos_sin is not None and cos_sin.shape[1]:
        rows = np.asarray(cos_sin, np.float64)[positions]
        half = rows.shape[1] // 2
        for i in range(half):
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = rows[:, None, i], rows[:, None, half + i]
            a, b = n[..., ia], n[..., ib]
            y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
            mag[..., ia] = np.abs(a * c) + np.abs(b * s)
            mag[..., ib] = np.abs(b * c) + np.abs(a * s)
    return y, mag


def tree_attention(q, k, v, block_tables, seq_lens, query_start, mask, scale, num_kv_heads):
    """Tree attention over caches k, v [NB, bs, Hk, D] of values (float64).

    mask: bool [Tq, nodes].  Returns out [Tq, H, D] and the terms of an error
    bound per element: mean |v| under the weights (A), and per row the largest
    sum |q||k| of a visible score, the visible keys, max |v| and the weight sum
    relative to the largest weight."""
    q = np.asarray(q, np.float64)
    Tq, H, D = q.shape
    G = H // num_kv_heads
    bs = k.shape[1]
    out, A = np.zeros((Tq, H, D)), np.zeros((Tq, H, D))
    smax, sumw = np.zeros((Tq, H, 1)), np.ones((Tq, H, 1))
    vmax, nvis = np.zeros((Tq, H, 1)), np.zeros((Tq, H, 1))
    for i in range(len(seq_lens)):
        L, q0, q1 = int(seq_lens[i]), int(query_start[i]), int(query_start[i + 1])
        Q = q1 - q0
        pos = np.arange(L)
        ids = np.asarray(block_tables[i])[pos // bs].astype(np.int64)
        ok = (ids >= 0) & (ids < k.shape[0])
        for h in range(num_kv_heads):
            kk = np.asarray(k[np.where(ok, ids, 0), pos % bs, h], np.float64)
            vv = np.asarray(v[np.where(ok, ids, 0), pos % bs, h], np.float64)
            for r in range(q0, q1):
                sees = ok.copy()
                sees[L - Q:] &= mask[r, :Q]
                if not sees.any():
                    continue
                K, V = kk[sees], vv[sees]
                for g in range(h * G, (h + 1) * G):
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = (K * q[r, g]).sum(-1) * scale
                        top = s.max()
                        if top == -np.inf:
                            continue
                        w = np.exp(s - top)
                        out[r, g] = (w[:, None] * V).sum(0) / w.sum()
                        A[r, g] = (w[:, None] * np.abs(V)).sum(0) / w.sum()
                        smax[r, g] = (np.abs(K * q[r, g]).sum(-1) * abs(scale)).max()
                        sumw[r, g], vmax[r, g], nvis[r, g] = w.sum(), np.abs(V).max(), len(V)
    return out, dict(A=A, smax=smax, sumw=sumw, vmax=vmax, nvis=nvis)


def tree_tolerance(ref, t, head_dim):
    """Largest |got - ref| of fp32 arithmetic with fp16 weights and outputs.

    Output rounding: half a step, 2^-11 |ref|, or 2^-25 below the normal range.
    Weights rounded to fp16: 2^-11 relative each (A 2^-11), or, when subnormal,
    2^-25 where the row's largest weight is 2^11 or more: 2^-36 of it, and less
    than 2^-35 with the reference's own rounding; against a normaliser of
    unrounded weights.
    Scores: a sum of head_dim products in fp32, (head_dim + 4) 2^-24 of
    sum |q||k|, and 4 2^-24 for the scaling, the subtraction of the maximum and
    the exponential's argument; an error d of a score moves its weight by d
    relative, and the normaliser too.  Exponential 2^-21.  Accumulation of one
    rounding (at most a whole step, 2^-23) per 16 keys and merge.
    """
    d = (head_dim + 8) * 2.0 ** -24 * t["smax"]
    rel = 2.0 ** -11 + 2 * d + 2.0 ** -20 + (t["nvis"] / 16 + 64) * 2.0 ** -23
    return (np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + rel * t["A"] +
            t["nvis"] * 2.0 ** -35 * t["vmax"] / t["sumw"])


def tree_accept(rows, path, ctx_lens, block_tables, block_size):
    """rows [NB * bs, ...] of one cache and layer after the accepted paths moved."""
    old, new = np.asarray(rows), np.array(rows)
    for i, nodes in enumerate(path):
        for depth, node in enumerate(nodes):
            if node < 0:
                break
            a, b = int(ctx_lens[i]) + depth, int(ctx_lens[i]) + int(node)
            dst = int(block_tables[i][a // block_size]) * block_size + a % block_size
            src = int(block_tables[i][b // block_size]) * block_size + b % block_size
            new[dst] = old[src]
    return new


def mask_words(mask, words=None):
    """bool [Tq, nodes] -> int64 [Tq, words]: bit j % 64 of word j // 64."""
    Tq, n = mask.shape
    words = words or max(1, -(-n // 64))
    out = np.zeros((Tq, words), np.uint64)
    for j in range(n):
        out[:, j // 64] |= mask[:, j].astype(np.uint64) << np.uint64(j % 64)
    return out.view(np.int64)


def random_tree(rng, nodes, reach=4):
    """Ancestor mask bool [nodes, nodes] of a random tree numbered root first."""
    mask = np.zeros((nodes, nodes), bool)
    for j in range(nodes):
        if j:
            mask[j] = mask[int(rng.integers(max(0, j - reach * 3), j))]
        mask[j, j] = True
    return mask
