"""A step in which the free list does not suffice: the refused sequences are left out of
the write and of the attentions behind it, nothing is recorded, the others are right."""

import numpy as np
import pytest

from oracle import serving as srv
from oracle import speculative as spec

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu
BS, H, Hk, D, MB = 16, 8, 2, 64, 16
i32, i64, f16 = torch.int32, torch.int64, torch.float16
RULES = dict(softcap=8.0, window=40)


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Server:
    def __init__(self, lens, spare, seed):
        rng = self.rng = np.random.default_rng(seed)
        self.S, self.old = len(lens), np.array(lens, np.int32)
        blocks = -(-self.old // BS)
        self.NB = int(blocks.sum()) + spare
        ids = rng.permutation(self.NB).astype(np.int32)
        # entries past the sequences' blocks are stale: other sequences' blocks
        tables, at = ids[rng.integers(0, self.NB, (self.S, MB))], 0
        for i, n in enumerate(blocks):
            tables[i, :n] = ids[at:at + n]
            at += n
        self.tables, self.lens = dev(tables), dev(self.old)
        self.free = dev(np.concatenate([ids[at:], np.zeros(at)]).astype(np.int32))
        self.count = dev(np.array([spare], np.int32))
        self.k, self.v = (dev(rng.standard_normal((self.NB, BS, Hk, D)).astype(np.float16))
                          for _ in range(2))
        self.start = torch.zeros(self.S + 1, dtype=i32, device="cuda")

    def grow(self, new):
        """Blocks, slots and the rows' write; the lengths that the attentions take."""
        T = int(np.maximum(np.array(new) - self.old, 0).sum())
        self.new = dev(np.array(new, np.int32))
        slots, pos = (torch.zeros(T, dtype=i64, device="cuda") for _ in range(2))
        pkv.pkv_resize_sequences(self.tables, self.lens, self.new, self.lens, self.free, self.count,
                                 self.count, self.start, slots, pos, BS, self.NB)
        qkv = dev(self.rng.standard_normal((T, H + 2 * Hk, D)).astype(np.float16))
        self.q = torch.zeros(T, H, D, dtype=f16, device="cuda")
        angle = np.arange(MB * BS)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
        rope = dev(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
        before = [x.cpu().numpy().reshape(-1, Hk, D) for x in (self.k, self.v)]
        pkv.pkv_norm_rope_write(self.q, qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], pos, slots,
                                self.k, self.v, rope)
        # only the granted rows' slots changed
        rest = np.setdiff1d(np.arange(self.NB * BS), slots.cpu().numpy())
        for x, b in zip((self.k, self.v), before):
            assert np.array_equal(x.cpu().numpy().reshape(-1, Hk, D)[rest], b[rest])
        self.out = torch.full_like(self.q, 7.0)
        self.granted = (self.lens == self.new).cpu().numpy()
        return torch.where(self.lens == self.new, self.lens, 0)

    def check(self, lens, tree=None, **rules):
        got, start = self.out.cpu().numpy().astype(float), self.start.cpu().numpy()
        args = (self.q.cpu().numpy(), self.k.cpu().numpy(), self.v.cpu().numpy(),
                self.tables.cpu().numpy(), lens.cpu().numpy(), start)
        if tree is None:
            rows = {r for i in range(self.S) if self.granted[i] for r in range(start[i], start[i + 1])}
            ref, tol = srv.scored_attention(*args, D ** -0.5, Hk, rows=rows, **rules)
            if not rules:
                # (without rules the row's largest weight stands at 1 or above: half a step
                # of fp16's smallest, 2^-25 of it, for each key)
                tol = tol + int(lens.max()) * 2.0 ** -25 * float(self.v.abs().max())
        else:
            keep = np.where(self.granted)[0]
            ref, terms = spec.tree_attention(*args, tree, D ** -0.5, Hk)
            tol = spec.tree_tolerance(ref, terms, D)
            assert len(keep)
        for i in range(self.S):
            rows = slice(start[i], start[i + 1])
            if self.granted[i]:
                assert (np.abs(got[rows] - ref[rows]) <= tol[rows]).all(), i
            else:
                assert (got[rows] == 7).all(), i
        assert pkv.pkv_get_device_error()[0] == 0


STEPS = [
    # lengths, to grow to, spare blocks
    ([40, 0, 17, 0], [41, 70, 90, 30], 6),       # prompts that do not fit, among others that do
    ([40, 0, 0, 33], [41, 70, 30, 35], 3),       # empty ones alone
    ([40, 0, 17, 9], [42, 4, 21, 13], 0),        # short ones (a few tokens each)
    ([40, 30, 100, 5], [44, 130, 104, 40], 2),   # more new tokens than there were
    ([100, 60], [130, 61], 0),                   # fewer
]


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("step", STEPS, ids=["prompts", "empty", "short", "longer", "shorter"])
def test_chunks(step, scored):
    lens, new, spare = step
    s = Server(lens, spare, [len(lens), spare])
    use = s.grow(new)
    assert 0 < s.granted.sum() < s.S
    longest = max(n - o for n, o in zip(new, lens))
    ws = torch.zeros(pkv.pkv_chunk_workspace_bytes(s.S, H, Hk, D, len(s.q), longest, MB * BS),
                     dtype=torch.uint8, device="cuda")
    args = (s.q, s.k, s.v, s.tables, use, s.start, D ** -0.5, H, Hk, D, BS, longest, MB * BS, s.NB, ws)
    rules = RULES if scored else {}
    (pkv.pkv_chunk_attention_scored if scored else pkv.pkv_chunk_attention)(s.out, *args, **rules)
    s.check(use, **rules)
    # a refused prompt of length 0 is left out by its own length too
    if all(o == 0 for o, g in zip(lens, s.granted) if not g):
        s.out.fill_(7.0)
        args = args[:4] + (s.lens,) + args[5:]
        (pkv.pkv_chunk_attention_scored if scored else pkv.pkv_chunk_attention)(s.out, *args, **rules)
        s.check(use, **rules)


@pytest.mark.parametrize("step", [([40, 31, 100], [45, 36, 105], 0), ([0, 40], [6, 46], 0)],
                         ids=["few", "empty"])
def test_trees(step):
    lens, new, spare = step
    s = Server(lens, spare, [7, spare])
    use = s.grow(new)
    assert 0 < s.granted.sum() < s.S
    nodes, T = new[0] - lens[0], len(s.q)
    mask = np.tile(spec.random_tree(np.random.default_rng(3), nodes), (s.S, 1))
    ws = torch.zeros(pkv.pkv_tree_workspace_bytes(s.S, H, Hk, D, T, nodes, MB * BS),
                     dtype=torch.uint8, device="cuda")
    pkv.pkv_tree_attention(s.out, s.q, s.k, s.v, s.tables, use, s.start, dev(spec.mask_words(mask)),
                           D ** -0.5, H, Hk, D, BS, nodes, MB * BS, s.NB, ws)
    # (the definition takes no sequence without tokens: the refused ones' rows count as none)
    full = np.where(s.granted, use.cpu().numpy(), np.array(new)).astype(np.int32)
    s.check(torch.from_numpy(full), tree=mask)
    # an accepted path of none leaves a refused sequence's cache rows alone
    before = [x.cpu().numpy().reshape(-1, Hk, D) for x in (s.k, s.v)]
    path = torch.tensor([[0, 2, 4, -1]] * s.S, dtype=i32, device="cuda")
    path = torch.where((s.lens == s.new)[:, None], path, -1)
    view = pkv.pkv_view(0, 0, BS * Hk * D * 2, Hk * D * 2, 0)
    pkv.pkv_tree_accept([(s.k, view), (s.v, view)], 1, path, dev(s.old), s.tables, BS, s.NB)
    for x, b in zip((s.k, s.v), before):
        want = b.copy()
        for i in np.where(s.granted)[0]:
            at = s.old[i] + np.arange(nodes)
            slot = s.tables.cpu().numpy()[i, at // BS] * BS + at % BS
            want[slot[[1, 2]]] = b[slot[[2, 4]]]
        assert np.array_equal(x.cpu().numpy().reshape(-1, Hk, D), want)
    assert pkv.pkv_get_device_error()[0] == 0


def test_decode():
    lens, new = [40, 16, 32, 9], [41, 17, 33, 10]
    s = Server(lens, 1, 11)
    use = s.grow(new)
    assert s.granted.tolist() == [True, True, False, True]
    ws = torch.zeros(pkv.pkv_decode_workspace_bytes(4, H, Hk, D, MB * BS), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_decode_attention_scored(s.out, s.q, s.k, s.v, s.tables, use, D ** -0.5, H, Hk, D, BS,
                                    MB * BS, s.NB, ws, **RULES)
    assert (s.out[2] == 0).all()  # (a decode's sequence of length 0 gives zeros)
    s.out[2] = 7.0
    s.check(use, **RULES)
