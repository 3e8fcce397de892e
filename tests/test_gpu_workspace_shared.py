"""One workspace, zeroed once, under calls of every kind and of changing shapes: each
result is what the same call gives on a workspace of its own, bit for bit."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu
BS = 16
RULES = dict(window=5000)


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


class Step:
    """Caches and tables of sequences of the given lengths, their last tokens new."""

    def __init__(self, seed, lens, news, H, Hk, D):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.shape, self.S, self.news = (H, Hk, D), len(lens), news
        blocks = [-(-n // BS) for n in lens]
        self.NB, MB = sum(blocks), max(blocks)
        ids = np.random.default_rng(seed).permutation(self.NB).astype(np.int32)
        tables, at = np.zeros((len(lens), MB), np.int32), 0
        for i, n in enumerate(blocks):
            tables[i, :n] = ids[at:at + n]
            at += n
        self.tables = torch.from_numpy(tables).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(news)]).astype(np.int32)).cuda()
        self.T, self.maxq, self.maxl = sum(news), max(news), max(lens)

        def rows(*s):
            return torch.randn(*s, generator=g, device="cuda").half()

        self.q = rows(self.T, H, D)
        self.k, self.v = rows(self.NB, BS, Hk, D), rows(self.NB, BS, Hk, D)
        self.codes = [torch.randint(0, 120, (self.NB, BS, Hk, D), generator=g, device="cuda",
                                    dtype=torch.uint8) for _ in range(2)]
        self.scales = [torch.rand(self.NB, BS, Hk, generator=g, device="cuda") * 0.01
                       for _ in range(2)]

    def bytes(self, kind):
        H, Hk, D = self.shape
        if kind.startswith("chunk"):
            return pkv.pkv_chunk_workspace_bytes(self.S, H, Hk, D, self.T, self.maxq, self.maxl)
        return pkv.pkv_decode_workspace_bytes(self.S, H, Hk, D, self.maxl)

    def call(self, kind, ws):
        H, Hk, D = self.shape
        out = torch.full_like(self.q, 7.0)
        shape = (D ** -0.5, H, Hk, D, BS)
        tables = (self.tables, self.lens)
        if kind.startswith("chunk"):
            fn = pkv.pkv_chunk_attention_scored if kind == "chunk_rules" else pkv.pkv_chunk_attention
            fn(out, self.q, self.k, self.v, *tables, self.start, *shape, self.maxq, self.maxl, self.NB,
               ws, **(RULES if kind == "chunk_rules" else {}))
        elif kind == "fp8":
            pkv.pkv_decode_attention_fp8(out, self.q, *self.codes, *self.scales, *tables, *shape,
                                         self.maxl, self.NB, ws)
        elif kind == "fp8_rules":
            pkv.pkv_decode_attention_scored_fp8(out, self.q, *self.codes, *self.scales, *tables,
                                                *shape, self.maxl, self.NB, ws, **RULES)
        elif kind == "rules":
            pkv.pkv_decode_attention_scored(out, self.q, self.k, self.v, *tables, *shape, self.maxl,
                                            self.NB, ws, **RULES)
        else:
            pkv.pkv_decode_attention(out, self.q, self.k, self.v, *tables, *shape, self.maxl, self.NB,
                                     ws, schedule=pkv.PKV_SCHEDULE_GRID if kind == "grid"
                                     else pkv.PKV_SCHEDULE_AUTO)
        return out


def run(calls):
    """calls: (kind, step) in order; all on one workspace, each against one of its own."""
    n = max(s.bytes(k) for k, s in calls)
    shared = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for i, (kind, s) in enumerate(calls):
        want = s.call(kind, torch.zeros(n, dtype=torch.uint8, device="cuda"))
        got = s.call(kind, shared)
        assert not torch.isnan(want).any()
        assert torch.equal(got, want), f"call {i}, {kind}: {(got != want).any(-1).sum()} rows"
    assert pkv.pkv_get_device_error()[0] == 0


def decodes(counts, H=32, Hk=8, D=64, longest=1200):
    return [Step(S, [max(9, longest - 37 * (i % 20)) for i in range(S)], [1] * S, H, Hk, D)
            for S in counts]


@pytest.mark.parametrize("kind", ["balanced", "rules", "fp8", "fp8_rules", "grid"])
def test_decodes_of_growing_and_shrinking_batches(kind):
    steps = decodes([3, 64, 65, 1, 66, 17])
    run([(kind, s) for s in steps + steps[::-1]])


def test_every_decode_in_turn():
    a, b = decodes([40, 71])
    kinds = ["balanced", "grid", "rules", "fp8", "fp8_rules"]
    run([(k, s) for s in (a, b, a) for k in kinds + kinds[::-1]])


def test_grid_schedule_of_many_sequences():
    """More (sequence, head) pairs than there is room for tickets at the workspace's start."""
    a, b = decodes([600, 601], H=32, Hk=4, longest=700)
    few = decodes([9], H=32, Hk=4)[0]
    run([("grid", few), ("grid", a), ("balanced", few), ("grid", b), ("grid", few), ("grid", a)])


@pytest.mark.parametrize("S,H,Hk,D", [(60, 1, 1, 64), (190, 16, 2, 64), (230, 8, 1, 128),
                                      (620, 8, 2, 128)])
def test_chunks_with_and_without_rules(S, H, Hk, D):
    """Batches that leave the two forms' balanced schedules different grids."""
    lens = [20 + i % 9 for i in range(S)]
    news = [1 + i % 2 for i in range(S)]
    lens[1], news[1] = 9000, 150  # three partitions, two under rules
    lens[S // 2], news[S // 2] = 8200, 70
    s = Step(S, lens, news, H, Hk, D)
    run([(k, s) for k in ("chunk", "chunk_rules", "chunk_rules", "chunk", "chunk_rules", "chunk")])


def test_chunks_of_changing_shapes_between_decodes():
    H, Hk, D = 8, 2, 64
    shapes = [([9000, 300, 4500], [150, 3, 64]), ([700] * 40, [1] * 40), ([9000] * 2, [260, 40]),
              ([800] * 33, [4] * 33), ([12000, 40], [500, 2]), ([500] * 70, [2] * 70)]
    steps = [Step(i, lens, news, H, Hk, D) for i, (lens, news) in enumerate(shapes)]
    few = Step(9, [3000] * 21, [1] * 21, H, Hk, D)
    calls = []
    for s in steps + steps[::-1]:
        calls += [("chunk", s), ("balanced", few), ("chunk_rules", s), ("rules", few), ("grid", few)]
    run(calls)
