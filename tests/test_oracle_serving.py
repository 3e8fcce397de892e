"""Pins of the float64 definitions of a serving step's operators."""

import numpy as np
import pytest

from oracle import serving as srv


def test_resize_by_hand():
    tables = np.array([[4, -1, -1], [1, 6, 3], [5, 2, -1]], np.int32)
    free = np.array([7, 0, -1, -1, -1, -1, -1, -1], np.int32)
    # 4 + 3 tokens need a block, 12 shrink to 5 and give one back, 8 get one token
    # and need a block, with blocks of 4
    t, lens, f, n, start, slots, pos = srv.resize(tables, [4, 12, 8], [7, 5, 9], free, 2, 4, 6, 8)
    assert lens.tolist() == [7, 5, 9] and n == 1 and f[0] == 7
    assert t[0].tolist() == [4, 3, -1]     # the block just given back is taken first
    assert t[2].tolist() == [5, 2, 0]      # then the top of the list
    assert start.tolist() == [0, 3, 3, 4]
    assert slots.tolist() == [12, 13, 14, 0, -1, -1]
    assert pos.tolist() == [4, 5, 6, 8, 0, 0]


def test_resize_taken_back():
    rng = np.random.default_rng(1)
    S, MB, NB, bs = 9, 12, 100, 8
    ids = rng.permutation(NB)
    lens = rng.integers(0, 60, S)
    tables = np.full((S, MB), -1, np.int32)
    at = 0
    for i in range(S):
        k = -(-int(lens[i]) // bs)
        tables[i, :k] = ids[at:at + k]
        at += k
    free = np.full(NB, -1, np.int32)
    free[:NB - at] = ids[at:]
    new = lens + rng.integers(1, 30, S)
    t, out, f, n, *_ = srv.resize(tables, lens, new, free, NB - at, bs, 300, NB)
    assert (out == new).all()
    held = [int(t[i, k]) for i in range(S) for k in range(-(-int(new[i]) // bs))]
    assert sorted(held + f[:n].tolist()) == list(range(NB))
    _, out, f, n, *_ = srv.resize(t, new, lens, f, n, bs, 300, NB)
    assert (out == lens).all() and n == NB - at and (f[:n] == free[:n]).all()


def test_resize_grants_in_order_while_they_last():
    tables = np.full((4, 4), -1, np.int32)
    free = np.arange(8, dtype=np.int32)
    # 2 + 3 + 1 blocks of 4 with three there: the second is refused, the third too
    # (it stands behind the second), the fourth needs none
    t, lens, _, n, start, slots, _ = srv.resize(tables, [0, 0, 0, 0], [8, 9, 1, 0], free, 3, 4, 99, 8)
    assert lens.tolist() == [8, 0, 0, 0] and n == 1 and (slots[8:] == -1).all()
    # rows that end past max_tokens
    _, lens, _, n, start, slots, _ = srv.resize(tables, [0] * 4, [4, 5, 1, 0], free, 8, 4, 8, 8)
    assert lens.tolist() == [4, 0, 0, 0] and start.tolist() == [0, 4, 8, 8, 8] and n == 7
    assert (slots[4:] == -1).all()


def simulate(parents, target, draft, n, seed, fixed=None):
    """Next tokens after the root's level: children drawn from the root's drafts."""
    rng = np.random.default_rng(seed)
    Q, V = len(parents), target.shape[1]
    first = np.zeros(V)
    for _ in range(n):
        tokens = np.zeros(Q, int)
        for k in range(1, Q):
            q = draft[parents[k]]
            tokens[k] = rng.choice(V, p=q) if fixed is None else fixed[k]
        path, lens, nxt, _ = srv.verify(tokens, parents, [0, Q], target,
                                        draft if fixed is None else None, rng.random(Q),
                                        rng.random(1), Q)
        first[tokens[path[0, 1]] if lens[0] > 1 else nxt[0]] += 1
    return first / n


@pytest.mark.parametrize("fixed", [None, [0, 2, 0, 1]])
def test_verify_keeps_the_targets_distribution(fixed):
    rng = np.random.default_rng(3)
    V, n = 5, 20000
    target, draft = rng.dirichlet(np.ones(V), 4), rng.dirichlet(np.ones(V), 4)
    got = simulate([-1, 0, 0, 0], target, draft, n, 4, fixed)
    # five standard deviations of a share of n
    assert np.all(np.abs(got - target[0]) <= 5 * np.sqrt(target[0] * (1 - target[0]) / n))


def test_verify_by_hand():
    p = np.array([[0.5, 0.25, 0.25], [0, 1, 0], [0.1, 0.2, 0.7]])
    q = np.array([[0.25, 0.5, 0.25], [1, 0, 0], [0.3, 0.3, 0.4]])

    def run(tokens, au, su, parents=(-1, 0, 1), draft=q, depth=3):
        path, n, nxt, _ = srv.verify(tokens, parents, [0, 3], p, draft, au, [su], depth)
        return path[0].tolist(), int(n[0]), int(nxt[0])

    # token 0 at the root: accepted whatever the number (p > q); then token 1 after
    # it: p = 1, q = 0 -> accepted; the leaf draws from its p
    assert run([0, 0, 1], [0, 0.99, 0.99], 0.29) == ([0, 1, 2], 3, 1)
    assert run([0, 0, 1], [0, 0.99, 0.99], 0.31) == ([0, 1, 2], 3, 2)
    # token 1 at the root is accepted up to 0.5; else the rest is token 0 alone
    assert run([0, 1, 2], [0, 0.49, 0.9], 0.5)[1:] == (2, 1)
    assert run([0, 1, 2], [0, 0.51, 0.9], 0.5) == ([0, -1, -1], 1, 0)
    # a path cut short draws from the node's p
    assert run([0, 0, 1], [0, 0.1, 0.1], 0.8, depth=2) == ([0, 1], 2, 1)
    # fixed guesses: token 1 (0.25) rejected, then token 2 has 0.25 of the 0.75 left
    assert run([0, 1, 2], [0, 0.26, 0.32], 0.0, (-1, 0, 0), None)[:2] == ([0, 2, -1], 2)
    assert run([0, 1, 2], [0, 0.26, 0.34], 0.99, (-1, 0, 0), None) == ([0, -1, -1], 1, 0)


def attention_case(rng, L, Q, H, Hk, D):
    bs = 4
    n = -(-L // bs)
    k, v = (rng.standard_normal((n + 1, bs, Hk, D)) for _ in range(2))
    q = rng.standard_normal((Q, H, D))
    return q, k, v, rng.permutation(n + 1)[None, :n], [L], [0, Q]


def test_scored_attention_closed_forms():
    rng = np.random.default_rng(5)
    L, Q, H, Hk, D = 21, 6, 4, 2, 8
    q, k, v, bt, lens, start = case = attention_case(rng, L, Q, H, Hk, D)
    pos = np.arange(L)
    K, V = k[bt[0][pos // 4], pos % 4], v[bt[0][pos // 4], pos % 4]

    def run(scale=0.3, **rules):
        return srv.scored_attention(*case, scale, Hk, **rules)[0]

    # without rules: causal softmax, written out
    for r, h in ((0, 0), (3, 2), (5, 3)):
        n = L - Q + r + 1
        w = np.exp(0.3 * K[:n, h // 2] @ q[r, h])
        assert np.allclose(run()[r, h], w @ V[:n, h // 2] / w.sum(), atol=1e-12)
    # a window of one: the token's own value; one that reaches everything: no window
    assert np.allclose(run(window=1)[4, 1], V[L - 2, 0], atol=1e-12)
    assert np.allclose(run(window=L), run(), atol=1e-12)
    # equal scores: means over what is seen
    assert np.allclose(run(0.0, window=3)[2, 0], V[L - 6:L - 3, 0].mean(0), atol=1e-12)
    assert np.allclose(run(0.0, window=3, prefix_lens=[2])[2, 3],
                       np.concatenate([V[:2, 1], V[L - 6:L - 3, 1]]).mean(0), atol=1e-12)
    assert np.allclose(run(0.0, prefix_lens=[99])[0, 0], V[:, 0].mean(0), atol=1e-12)
    # a cap far away changes nothing, one of almost nothing makes scores equal
    assert np.allclose(run(softcap=1e6), run(), atol=1e-9)
    assert np.allclose(run(softcap=1e-12), run(0.0), atol=1e-9)
    # the bias alone: weights 2^-distance
    s = np.full(H, np.log(2.0))
    w = 0.5 ** (L - 1 - pos)
    assert np.allclose(run(0.0, slopes=s)[5, 1], w @ V[:, 0] / w.sum(), atol=1e-12)
    # distances count in both directions inside a prefix
    w = 0.5 ** np.abs(L - Q - pos)
    assert np.allclose(run(0.0, slopes=s, prefix_lens=[L])[0, 1], w @ V[:, 0] / w.sum(), atol=1e-12)


def test_scored_attention_equals_the_chunk_oracle(orc):
    rng = np.random.default_rng(6)
    S, H, Hk, D, bs = 3, 4, 2, 64, 16
    lens, qlens = np.array([40, 17, 1], np.int32), [9, 17, 1]
    start = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    k, v = (rng.standard_normal((10, bs, Hk, D)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((int(start[-1]), H, D)).astype(np.float16)
    bt = rng.permutation(10)[:9].reshape(S, 3).astype(np.int32)
    want = orc.chunk_attention(q, k, v, bt, lens, start, 0.125)
    got, _ = srv.scored_attention(q, k, v, bt, lens, start, 0.125, Hk)
    assert np.allclose(got, want, atol=1e-12)
