"""Float64 definitions of a serving step's operators (numpy, CPU): block tables and
slot maps from lengths, verification of drafted trees, attention under score
rules.  Test infrastructure only; shares no code with the kernels.
"""

from __future__ import annotations

import numpy as np


def resize(tables, seq_lens, new_lens, free, free_count, block_size, max_tokens, num_blocks):
    """The step sequence by sequence.  Returns (tables, out_lens, free, count,
    query_start, slots, positions); entries of ``free`` from the new count on are
    what the walk leaves there."""
    tables, free = np.array(tables), np.array(free)
    S, MB = tables.shape
    bs, cap = block_size, len(free)
    room = MB * bs
    old = [int(x) for x in seq_lens]
    new = [int(x) if 0 <= int(x) <= room and 0 <= old[i] <= room else old[i]
           for i, x in enumerate(new_lens)]

    def blocks(n):
        return -(-n // bs)

    stack = [int(b) for b in free[:min(max(int(free_count), 0), cap)]]
    given = []
    for i in range(S):
        given += [int(tables[i, k]) for k in range(blocks(new[i]), blocks(old[i]))
                  if new[i] != old[i]]
    given = given[:cap - len(stack)]
    stack += given[::-1]
    free[:len(stack)] = stack
    top, asked, rows = len(stack), 0, 0
    out, start = [], [0]
    slots, positions = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int64)
    for i in range(S):
        L, N = old[i], new[i]
        want = max(blocks(N) - blocks(L), 0) if N > L else 0
        asked += want
        ok = N <= L or (rows + N - L <= max_tokens and (want == 0 or asked <= top))
        if ok:
            for k in range(want):
                tables[i, blocks(L) + k] = stack.pop()
        for pos in range(L, N):
            if rows < max_tokens:
                positions[rows] = pos
                if ok:
                    b = int(tables[i, pos // bs])
                    if 0 <= b < num_blocks:
                        slots[rows] = b * bs + pos % bs
            rows += 1
        start.append(min(rows, max_tokens))
        out.append(N if ok else L)
    return (tables, np.array(out, np.int32), free, len(stack), np.array(start, np.int32), slots,
            positions)


def verify(tokens, parents, query_start, target, draft, accept_u, sample_u, max_depth):
    """Tree verification, the normalised rest of the target carried from rejection to
    rejection.  Also returns the smallest relative distance of a comparison from
    its border, per sequence: a result is certain only where that is above the
    rounding of the implementation compared."""
    S, V = len(query_start) - 1, target.shape[1]
    path = np.full((S, max_depth), -1, np.int32)
    lens, nxt, near = np.zeros(S, np.int32), np.full(S, -1, np.int32), np.full(S, np.inf)

    def clip(u):
        return min(max(float(u), 0.0), 1 - 2.0 ** -24)

    def clean(x):
        x = np.asarray(x, np.float64)
        return np.where(x > 0, x, 0.0)

    for i in range(S):
        r0, r1 = int(query_start[i]), int(query_start[i + 1])
        if r1 == r0:
            continue
        at, depth = 0, 1
        path[i, 0] = 0
        while True:
            p = clean(target[r0 + at])
            rest, step = p, -1
            for k in range(at + 1, r1 - r0) if depth < max_depth else ():
                tok = int(tokens[r0 + k])
                if int(parents[r0 + k]) != at or not 0 <= tok < V:
                    continue
                u = clip(accept_u[r0 + k])
                if draft is None:
                    ask, have = u, rest[tok]
                    left = rest.copy()
                    left[tok] = 0
                    # (the rest is normalised: what is left of it by subtraction)
                    mass = 1.0 - have
                else:
                    q = clean(draft[r0 + at])
                    ask, have = u * q[tok], rest[tok]
                    left = np.maximum(rest - q, 0)
                    mass = left.sum()
                near[i] = min(near[i], abs(ask - have) / max(ask, have, 1e-300))
                if ask < have:
                    step = k
                    break
                if mass <= 0:
                    break
                rest = left / mass
            if step < 0:
                break
            path[i, depth] = step
            depth, at = depth + 1, step
        lens[i] = depth
        total = np.cumsum(rest)
        if total[-1] > 0:
            goal = clip(sample_u[i]) * total[-1]
            nxt[i] = int(np.argmax(total > goal))
            near[i] = min(near[i], np.abs(total - goal).min() / total[-1])
    return path, lens, nxt, near


def scored_attention(q, k, v, block_tables, seq_lens, query_start, scale, num_kv_heads,
                     softcap=0.0, window=0, slopes=None, prefix_lens=None, rows=None):
    """Attention under score rules over caches k, v [NB, bs, Hk, D] of values.

    rows: only these query rows.  Returns out [Tq, H, D] and a bound [Tq, H, D] on what fp32 arithmetic with fp16
    weights and outputs may be off by.  Per key, in units of its weight: 2^-11 for
    the weight's rounding; the score's error in nats -- (D + 8) 2^-24 of
    sum |q||k| scale for the dot product, its scaling and the exponential's
    argument, for the capping 10 2^-24 of the cap up to caps of 355 (1 - 2 / (1 + e^2y):
    2^-23 for the exponential's 2 units in its last place times the largest slope 1/2 of
    tanh in its logarithm, 2^-24 / 2 for its argument, 2^-22 and 2^-23 for the quotient
    and its divisor, which is at most 2, 2^-24 for the difference), for higher ones
    14 2^-24 of the score (the same past the cap, where tanh is above 0.76; less below),
    4 2^-24 of slope * distance for the bias -- and 2^-20 for the exponential and sums of roundings.  A weight's
    error moves the output by its share times (v - out).  Weights below fp16's
    normal range are off by 2^-32 of the largest at most."""
    q = np.asarray(q, np.float64)
    Tq, H, D = q.shape
    G, bs = H // num_kv_heads, k.shape[1]
    out, tol = np.zeros((Tq, H, D)), np.full((Tq, H, D), 2.0 ** -25)
    for i in range(len(seq_lens)):
        L, q0, q1 = int(seq_lens[i]), int(query_start[i]), int(query_start[i + 1])
        pos = np.arange(L)
        ids = np.asarray(block_tables[i])[pos // bs].astype(np.int64)
        ok = (ids >= 0) & (ids < k.shape[0])
        prefix = 0 if prefix_lens is None else int(prefix_lens[i])
        for r in range(q0, q1):
            if rows is not None and r not in rows:
                continue
            a = L - (q1 - r)
            sees = (pos <= a) & ((a - pos < window) if window else True)
            sees = (sees | (pos < prefix)) & ok
            if not sees.any():
                continue
            at = pos[sees]
            for h in range(H):
                K = np.asarray(k[ids[sees], at % bs, h // G], np.float64)
                V = np.asarray(v[ids[sees], at % bs, h // G], np.float64)
                s = (K @ q[r, h]) * scale
                err = (np.abs(K) @ np.abs(q[r, h])) * abs(scale) * (D + 8) * 2.0 ** -24
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                    err = err + (10 * softcap if softcap <= 355 else 14 * np.abs(s)) * 2.0 ** -24
                if slopes is not None:
                    bias = float(slopes[h]) * np.abs(a - at)
                    s = s - bias
                    err = err + np.abs(bias) * 4 * 2.0 ** -24
                err = err + np.abs(s) * 2.0 ** -23
                w = np.exp(s - s.max())
                o = (w @ V) / w.sum()
                rel = 2.0 ** -11 + 2 * err + 2.0 ** -20 + (len(at) / 16 + 64) * 2.0 ** -23
                out[r, h] = o
                tol[r, h] += (np.abs(o) * 2.0 ** -11 +
                              ((w * rel) @ (np.abs(V) + np.abs(o))) / w.sum() +
                              len(at) * 2.0 ** -31 * np.abs(V).max() / w.sum())
    return out, tol
