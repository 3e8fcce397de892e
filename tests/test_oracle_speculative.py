"""Pins of the speculative step's float64 definitions, on the CPU."""

import numpy as np
import pytest

from oracle import speculative as spec


def _rope_table(n, rot, base=10000.0):
    inv = base ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(n)[:, None] * inv[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(interleaved):
    rng = np.random.default_rng(1)
    t = _rope_table(200, 64)
    x = rng.standard_normal((3, 2, 64))
    y, _ = spec.norm_rope(x, None, 0.0, t, np.array([0, 17, 150]), interleaved)
    assert np.array_equal(y[0], x[0])  # position 0 turns nothing
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-6)
    # a dot product depends on the difference of the positions alone
    a, b = rng.standard_normal((2, 1, 1, 64))
    def dot(p, q):
        return (spec.norm_rope(a, None, 0, t, np.array([p]), interleaved)[0] *
                spec.norm_rope(b, None, 0, t, np.array([q]), interleaved)[0]).sum()
    assert dot(5, 25) == pytest.approx(dot(105, 125), abs=1e-4)


def test_the_pairings_differ_and_the_tail_passes():
    t = _rope_table(10, 32)
    x = np.random.default_rng(2).standard_normal((1, 1, 64))
    h, _ = spec.norm_rope(x, None, 0, t, np.array([3]), False)
    i, _ = spec.norm_rope(x, None, 0, t, np.array([3]), True)
    assert np.array_equal(h[..., 32:], x[..., 32:]) and np.array_equal(i[..., 32:], x[..., 32:])
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    h2, _ = spec.norm_rope(x[..., perm], None, 0, t[:, :], np.array([3]), False)
    assert np.allclose(h2, i[..., perm])


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(3).standard_normal((4, 2, 128)) * 7
    y, _ = spec.norm_rope(x, np.ones(128), 0.0, None, None, False)
    assert np.allclose((y * y).mean(-1), 1.0)


def test_causal_mask_is_the_chunk_attention(orc):
    rng = np.random.default_rng(4)
    NB, Hk, H, D, lens, qlens = 12, 2, 4, 64, [37, 20], [5, 20]
    k, v = (rng.standard_normal((NB, 16, Hk, D)).astype(np.float16) for _ in range(2))
    tables = rng.permutation(NB)[:10].reshape(2, 5).astype(np.int32)
    qs = np.array([0, 5, 25], np.int32)
    q = rng.standard_normal((25, H, D)).astype(np.float16)
    mask = np.concatenate([np.tril(np.ones((n, 20), bool))[:n] for n in qlens])
    got, _ = spec.tree_attention(q, k, v, tables, lens, qs, mask, 0.125, Hk)
    ref = orc.chunk_attention(q, k, v, tables, np.array(lens, np.int32), qs, 0.125)
    assert np.abs(got - ref).max() < 1e-12


def test_masked_tokens_do_not_matter_and_empty_rows_are_zero():
    rng = np.random.default_rng(5)
    k, v = (rng.standard_normal((4, 16, 1, 64)) for _ in range(2))
    tables, q = np.array([[2, 0, 3]]), rng.standard_normal((4, 2, 64))
    mask = np.eye(4, dtype=bool)
    mask[3] = False
    args = (tables, [20], [0, 4], mask, 0.1, 1)
    a, _ = spec.tree_attention(q, k, v, *args)
    k2, v2 = k.copy(), v.copy()
    k2[0, 3], v2[0, 3] = np.nan, np.inf  # position 19: drafted token 3, seen by no row
    b, _ = spec.tree_attention(q, k2, v2, *args)
    assert np.array_equal(a, b)
    out, _ = spec.tree_attention(q, k, v, tables, [4], [0, 4], mask, 0.1, 1)
    assert (out[3] == 0).all() and np.allclose(out[0], v[2, 0, 0])


def test_accept_moves_the_path_as_if_at_once():
    rows = np.arange(64).reshape(64, 1)
    tables = np.array([[1, 0, 3], [2, 2, 2]])
    got = spec.tree_accept(rows, [[0, 1, 3, 9, -1, 7], [-1, 0, 0, 0, 0, 0]], [13, 0], tables, 16)
    want = rows.copy()
    # places 13.. of sequence 0 are rows 29, 30, 31, then 0, 1, ...
    want[31], want[0] = rows[0], rows[6]
    assert np.array_equal(got, want)


def test_mask_words_and_trees():
    rng = np.random.default_rng(6)
    m = spec.random_tree(rng, 70)
    assert m.diagonal().all() and m[:, 0].all() and not np.triu(m, 1).any()
    w = spec.mask_words(m).view(np.uint64)
    assert w.shape == (70, 2)
    for i in (0, 5, 64, 69):
        bits = [(int(w[i, j // 64]) >> (j % 64)) & 1 for j in range(70)]
        assert bits == m[i].astype(int).tolist()


def test_e4m3_table_against_torch():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    assert np.array_equal(spec.e4m3_table(), t.numpy(), equal_nan=True)
