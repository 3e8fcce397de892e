"""pkv_resize_sequences against its definition, element by element."""

import numpy as np
import pytest

from oracle import serving as srv

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def pool(rng, S, MB, bs, hi, spare, capacity=None):
    """Tables, lengths and a free list in which every block is held once."""
    lens = rng.integers(0, hi + 1, S).astype(np.int32)
    have = -(-lens // bs)
    NB = int(have.sum()) + spare
    ids = rng.permutation(max(NB, 1)).astype(np.int32)
    tables = rng.integers(-5, 3, (S, MB)).astype(np.int32)  # stale entries past the lengths
    at = 0
    for i in range(S):
        tables[i, :have[i]] = ids[at:at + have[i]]
        at += have[i]
    free = np.full(capacity if capacity is not None else max(NB, 1), -7, np.int32)
    free[:spare] = ids[at:at + spare]
    return tables, lens, free, spare, max(NB, 1)


class Call:
    def __init__(self, tables, lens, new, free, count, bs, T, NB, positions=True):
        S = len(lens)
        self.args = (tables, lens, new, free, count, bs, T, NB)
        self.tables, self.lens, self.new = dev(tables), dev(lens.astype(np.int32)), dev(new.astype(np.int32))
        self.free, self.count = dev(free), dev(np.array([count], np.int32))
        full = lambda n, t: torch.full((n,), 77, dtype=t, device="cuda")  # noqa: E731
        self.out, self.out_count = full(S, torch.int32), full(1, torch.int32)
        self.start = full(S + 1, torch.int32)
        self.slots = full(T, torch.int64)
        self.pos = full(T, torch.int64) if positions else None
        self.bs, self.NB = bs, NB

    def run(self, in_place=False):
        pkv.pkv_resize_sequences(self.tables, self.lens, self.new,
                                 self.lens if in_place else self.out, self.free, self.count,
                                 self.count if in_place else self.out_count, self.start, self.slots,
                                 self.pos, self.bs, self.NB)
        if in_place:
            self.out, self.out_count = self.lens, self.count
        return self

    def check(self):
        tables, lens, new, free, count, bs, T, NB = self.args
        t, out, f, n, start, slots, pos = srv.resize(tables, lens, new, free, count, bs, T, NB)
        got = [x.cpu().numpy() for x in (self.tables, self.out, self.free, self.out_count,
                                         self.start, self.slots)]
        for a, b, what in zip(got, (t, out, f, np.array([n]), start, slots),
                              ("tables", "lens", "free", "count", "start", "slots")):
            assert np.array_equal(a, b), what
        if self.pos is not None:
            assert np.array_equal(self.pos.cpu().numpy(), pos)


CASES = [
    # sequences, blocks a table, block size, longest, spare blocks, rows
    (1, 4, 16, 40, 3, 20), (1, 1, 1, 1, 1, 1), (3, 9, 5, 33, 10, 0), (64, 300, 16, 4000, 400, 64),
    (31, 20, 16, 300, 2, 500), (33, 40, 16, 500, 60, 1025), (1000, 30, 16, 400, 900, 5000),
    (1025, 6, 3, 14, 300, 9000), (2049, 4, 16, 50, 0, 333), (8192, 3, 16, 40, 5000, 20000),
    (2, 9000, 16, 100, 8192, 131072),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[2]}r{c[5]}" for c in CASES])
@pytest.mark.parametrize("in_place", [False, True])
def test_random_steps(case, in_place):
    S, MB, bs, hi, spare, T = case
    rng = np.random.default_rng([S, T])
    tables, lens, free, count, NB = pool(rng, S, MB, bs, hi, spare)
    what = rng.integers(0, 5, S)
    new = np.select([what == 0, what == 1, what == 2, what == 3],
                    [0, np.maximum(lens - rng.integers(0, 40, S), 0), lens + 1, lens],
                    lens + rng.integers(0, 2 * T // S + 2, S))
    new = np.minimum(new, MB * bs)
    Call(tables, lens, new, free, count, bs, T, NB, positions=T % 2 == 0).run(in_place).check()
    assert pkv.pkv_get_device_error()[0] == 0


def test_one_long_prompt_and_back():
    MB, bs, NB = 9000, 16, 9000
    rng = np.random.default_rng(2)
    ids = rng.permutation(NB).astype(np.int32)
    tables, lens = np.full((1, MB), -1, np.int32), np.zeros(1, np.int32)
    new = np.array([131071], np.int32)
    c = Call(tables, lens, new, ids, NB, bs, 131072, NB).run()
    c.check()
    assert int(c.slots[-1]) == -1 and int(c.slots[-2]) >= 0
    back = Call(c.tables.cpu().numpy(), new, lens, c.free.cpu().numpy(), int(c.out_count), bs, 8, NB)
    back.run().check()
    assert np.array_equal(back.free.cpu().numpy(), ids) and int(back.out_count) == NB
    assert pkv.pkv_get_device_error()[0] == 0


def test_same_call_twice_gives_the_same():
    rng = np.random.default_rng(3)
    tables, lens, free, count, NB = pool(rng, 40, 30, 16, 300, 50)
    new = np.minimum(np.maximum(lens + rng.integers(-50, 50, 40), 0), 480)
    c = Call(tables, lens, new, free, count, 16, 2000, NB)
    c.run().check()
    c.run().check()


def test_bad_lengths_leave_their_sequence():
    tables = np.arange(12, dtype=np.int32).reshape(4, 3)
    free = np.full(40, -1, np.int32)
    free[:20] = np.arange(12, 32)
    for lens, new in (([10, 49, 5, 7], [12, 3, 6, 7]), ([10, -1, 5, 7], [12, 3, 6, 7]),
                      ([10, 20, 5, 7], [12, 49, 6, 7]), ([10, 20, 5, 7], [12, -9, 6, 7]),
                      ([10, 2 ** 31 - 1, 5, 7], [12, -2 ** 31, 6, 7])):
        Call(tables, np.array(lens), np.array(new), free, 20, 16, 8, 40).run().check()
        assert pkv.pkv_get_device_error() == (3, 1)


def test_bad_block_ids_get_no_slot():
    tables = np.array([[4, 99], [-3, 5], [1, 2]], np.int32)
    free = np.array([7, 50, 3, -2], np.int32)
    # the first grows in a bad block; the second's last block is fine
    c = Call(tables, np.array([20, 20, 30]), np.array([22, 21, 30]), free, 4, 16, 8, 10)
    c.run().check()
    assert pkv.pkv_get_device_error() == (2, 1)
    # the list's bad top, then 3, then the bad 50
    c = Call(np.array([[4, -1, -1, -1]], np.int32), np.array([16]), np.array([64]), free, 4, 16, 48, 10)
    c.run().check()
    assert pkv.pkv_get_device_error()[0] == 2
    assert c.slots.cpu().numpy()[:16].max() == -1 and c.slots.cpu().numpy()[16] == 48


def test_free_list_counts():
    tables = np.arange(8, dtype=np.int32).reshape(2, 4)
    free = np.arange(8, 14, dtype=np.int32)
    for count in (-3, 7, 2 ** 31 - 1):
        Call(tables, np.array([64, 1]), np.array([64, 30]), free, count, 16, 40, 16).run().check()
        assert pkv.pkv_get_device_error()[0] == 7
    # more given back than the list holds: the last of them are dropped
    Call(tables, np.array([64, 64]), np.array([0, 0]), free, 2, 16, 4, 16).run().check()
    assert pkv.pkv_get_device_error() == (7, 2)
    # nothing there and nothing given back
    Call(tables, np.array([64, 16]), np.array([64, 17]), free[:0], 0, 16, 4, 16).run().check()
    assert pkv.pkv_get_device_error()[0] == 0


def test_captured_with_lengths_that_change_and_on_another_stream():
    rng = np.random.default_rng(9)
    S, MB, bs, T = 20, 10, 16, 64
    tables, lens, free, count, NB = pool(rng, S, MB, bs, 60, 80)
    c = Call(tables, lens, lens, free, count, bs, T, NB)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for seed in range(3):
        r = np.random.default_rng(seed)
        new = np.minimum(np.maximum(lens + r.integers(-20, 20, S), 0), MB * bs).astype(np.int32)
        c.tables.copy_(dev(tables))
        c.free.copy_(dev(free))
        c.new.copy_(dev(new))
        graph.replay()
        c.args = (tables, lens, new, free, count, bs, T, NB)
        c.check()
    assert pkv.pkv_get_device_error()[0] == 0


def test_another_device_or_shape_is_refused():
    c = Call(np.zeros((2, 3), np.int32), np.zeros(2, np.int32), np.ones(2, np.int32),
             np.arange(4, dtype=np.int32), 4, 16, 4, 4)
    c.new = c.new[:1]
    with pytest.raises(ValueError):
        c.run()
    c.new = torch.ones(4, dtype=torch.int32, device="cuda")[::2]
    with pytest.raises(ValueError):
        c.run()
    c.new = torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        c.run()
