"""GPU parity of the tree attention (fp16 and FP8 caches) against its float64
definition, every element, at tolerances derived from the arithmetic."""

import numpy as np
import pytest

from oracle import speculative as spec

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu
BS = 16


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    assert torch.cuda.is_available()
    pkv.pkv_get_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Tree:
    """Sequences of the given lengths and drafted counts over a shuffled pool; slots
    that hold no token are NaN (fp16) or NaN codes and scales (FP8)."""

    def __init__(self, seed, lens, nodes, H, Hk, D, fp8=False, scale=None, spread=1.0, words=None,
                 mask=None, reach=4):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.nodes, self.H, self.Hk, self.D, self.fp8 = lens, nodes, H, Hk, D, fp8
        S = len(lens)
        self.scale = D ** -0.5 if scale is None else scale
        blocks = [-(-n // BS) for n in lens]
        self.MB = max(1, max(blocks)) + 1
        self.NB = sum(blocks) + 4
        ids = rng.permutation(self.NB)
        self.tables = np.full((S, self.MB), self.NB + 77, np.int32)  # unused entries: no block
        at = 0
        for i, b in enumerate(blocks):
            self.tables[i, :b] = ids[at:at + b]
            at += b
        self.qs = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        Tq = int(self.qs[-1])
        self.maxq = max(1, max(nodes))
        self.q = (rng.standard_normal((Tq, H, D)) * spread).astype(np.float16)
        if mask is None:
            mask = np.zeros((Tq, self.maxq), bool)
            for i, n in enumerate(nodes):
                if n:
                    mask[self.qs[i]:self.qs[i] + n, :n] = spec.random_tree(rng, n, reach)
        self.mask = mask
        self.words = words
        live = np.zeros((self.NB, BS), bool)
        for i, n in enumerate(lens):
            p = np.arange(n)
            live[self.tables[i][p // BS], p % BS] = True
        self.k, self.v = [], []
        self.parts = []
        for _ in range(2):
            if fp8:
                codes = rng.integers(0, 256, (self.NB, BS, Hk, D)).astype(np.uint8)
                codes[(codes & 0x7F) == 0x7F] = 0x38
                sc = (rng.uniform(0.5, 1.5, (self.NB, BS, Hk)) / 150).astype(np.float32)
                codes[~live], sc[~live] = 0x7F, np.nan
                self.parts += [codes, sc]
            else:
                x = rng.standard_normal((self.NB, BS, Hk, D)).astype(np.float16)
                x[~live] = np.nan
                self.parts.append(x)

    def slot(self, seq, node):
        p = self.lens[seq] - self.nodes[seq] + node
        return self.tables[seq, p // BS], p % BS

    def values(self):
        if not self.fp8:
            return [x.astype(np.float64) for x in self.parts]
        t = spec.e4m3_table()
        return [t[self.parts[2 * i]] * self.parts[2 * i + 1][..., None].astype(np.float64)
                for i in range(2)]

    def stage(self):
        k = [dev(x) for x in self.parts]
        if self.fp8:
            k = [k[0], k[2], k[1], k[3]]  # codes, then scales
        n = pkv.pkv_tree_workspace_bytes(len(self.lens), self.H, self.Hk, self.D, len(self.q),
                                         self.maxq, max(1, max(self.lens)))
        self.d = dict(caches=k, q=dev(self.q), tables=dev(self.tables),
                      lens=dev(np.array(self.lens, np.int32)), qs=dev(self.qs),
                      mask=dev(spec.mask_words(self.mask, self.words)),
                      out=torch.full(self.q.shape, 7.0, dtype=torch.float16, device="cuda"),
                      # contents of no use to anyone
                      ws=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"))
        return self.d

    def call(self, d=None, out=None, ws=None, stream=None, **kw):
        d = d or self.d
        fn = pkv.pkv_tree_attention_fp8 if self.fp8 else pkv.pkv_tree_attention
        a = dict(maxq=self.maxq, maxL=max(1, max(self.lens)))
        a.update(kw)
        out = d["out"] if out is None else out
        fn(out, d["q"], *d["caches"], d["tables"], d["lens"], d["qs"], d["mask"], self.scale,
           self.H, self.Hk, self.D, BS, a["maxq"], a["maxL"], self.NB, d["ws"] if ws is None else ws,
           stream=stream)
        return out

    def run(self):
        self.stage()
        out = self.call()
        kind = pkv.pkv_get_device_error()
        assert kind == (0, -1), kind
        return out.cpu().numpy().astype(np.float64)

    def want(self):
        k, v = self.values()
        return spec.tree_attention(self.q, k, v, self.tables, self.lens, self.qs, self.mask,
                                   self.scale, self.Hk)

    def check(self, got=None, rows=None):
        got = self.run() if got is None else got
        ref, t = self.want()
        tol = spec.tree_tolerance(ref, t, self.D)
        rows = slice(None) if rows is None else rows
        bad = ~(np.abs(got - ref) <= tol)[rows]
        assert not bad.any(), (f"{bad.sum()} of {bad.size} out of tolerance, worst "
                               f"{np.nanmax(np.abs(got - ref)[rows] / tol[rows]):.2f} of it")


CASES = [
    # seed, lens, drafted, H, Hk, D
    (1, [1], [1], 4, 4, 64),                             # one token alone
    (2, [8], [8], 8, 2, 128),                            # a tree without a context
    (3, [17, 40, 16], [3, 7, 16], 8, 2, 64),
    (4, [130, 128, 127, 129], [2, 1, 8, 4], 8, 8, 128),  # around one step, G 1
    (5, [700, 33, 1], [16, 5, 1], 32, 8, 128),
    (6, [1041], [8], 32, 8, 128),
    (7, [0, 12, 0, 600], [0, 4, 0, 2], 8, 4, 128),       # empty sequences
    (8, [300, 20, 515], [63, 20, 33], 16, 2, 128),       # G 8: 504 rows
    (9, [400, 65], [64, 64], 4, 1, 64),                  # the tree over four steps' edges
    (10, [900, 256, 700], [65, 256, 129], 4, 2, 128),    # more than one mask word
    (11, [2049, 511], [31, 32], 16, 16, 64),
    (12, [5000], [4], 2, 1, 128),                        # one head: split over many CTAs
    (13, [260] * 40, [3] * 40, 8, 4, 64),
    (14, [16, 31, 47, 64, 97, 113], [1, 2, 3, 4, 5, 6], 2, 2, 128),
    (15, [300, 70], [33, 9], 12, 3, 64),                 # three KV heads
    (16, [190, 260], [40, 17], 40, 5, 128),
    (17, [700], [256], 8, 1, 64),                        # sixteen tiles, four mask words
    (18, [100, 400, 90, 390, 80], [3, 40, 70, 1, 20], 16, 2, 128),  # 1, 3, 5, 1, 2 tiles
]


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=[str(c[0]) for c in CASES])
def test_every_element(case, fp8):
    Tree(*case, fp8=fp8).check()


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_large_scores_and_a_negative_scale(fp8):
    # one weight near 1 and the rest tiny; the running maximum moves often
    Tree(31, [900, 77], [20, 9], 8, 2, 128, fp8=fp8, spread=12.0).check()
    Tree(32, [300], [20], 8, 2, 64, fp8=fp8, scale=-0.3).check()
    Tree(33, [300], [20], 8, 2, 64, fp8=fp8, scale=0.0).check()


def test_rising_scores_rescale_every_step():
    # keys grow along the sequence: every step's maximum passes the reference
    t = Tree(34, [1500], [12], 4, 1, 128)
    for p in range(1500):
        t.parts[0][t.tables[0, p // BS], p % BS] = np.float16(0.02 * p) * np.sign(t.q[0, 0])
    t.q[:] = np.abs(t.q) * np.sign(t.q[0, 0])
    t.check()


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_rows_that_see_nothing_are_zero(fp8):
    mask = np.zeros((12, 9), bool)
    mask[0, 0] = mask[7, :4] = True
    t = Tree(41, [3, 9], [3, 9], 8, 2, 64, mask=mask, fp8=fp8)
    got = t.run()
    t.check(got)
    empty = ~mask.any(1)
    empty[:3] |= ~mask[:3, :3].any(1)
    assert (got[empty] == 0).all() and (got[0] != 0).any()


def test_bits_past_the_tree_are_ignored():
    t = Tree(42, [50, 30], [5, 9], 8, 2, 64, words=3)
    ref = t.run()
    w = spec.mask_words(t.mask, 3).view(np.uint64).copy()
    w[:5, 0] |= ~np.uint64(31)
    w[5:, 0] |= ~np.uint64(511)
    w[:, 1:] = ~np.uint64(0)
    t.d["mask"] = dev(w.view(np.int64))
    assert np.array_equal(t.call().cpu().numpy().astype(np.float64), ref)


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_non_finite_drafted_rows_reach_only_those_that_see_them(fp8, value):
    if fp8 and np.isinf(value):
        pytest.skip("E4M3 holds no infinity")
    for seed, lens, nodes in ((51, [40], [20]), (52, [300], [130]), (53, [129, 30], [9, 30])):
        t = Tree(seed, lens, nodes, 8, 2, 128, fp8=fp8)
        Q = nodes[0]
        bad = [Q // 3, Q - 1]
        for j in bad:
            b, o = t.slot(0, j)
            if fp8:
                t.parts[2][b, o, 1, 5::32] = 0x7F
            else:
                t.parts[1][b, o, 1, 5::32] = value
        got = t.run()
        ref, tol = t.want()
        G = t.H // t.Hk
        sees = t.mask[:, bad].any(1)
        sees[Q:] = False
        assert sees.any() and not sees[:Q].all()
        hit = np.zeros(got.shape, bool)
        hit[np.ix_(sees, np.arange(G, 2 * G), np.arange(5, 128, 32))] = True
        assert np.isfinite(got[~hit]).all()
        if np.isnan(value):
            assert np.isnan(got[hit]).all()
        else:
            assert (got[hit] == value).all()
        fin = np.where(np.isfinite(ref), ref, 0)
        lim = spec.tree_tolerance(fin, {k: np.where(np.isfinite(x), x, 8.0) for k, x in tol.items()}, 128)
        assert (np.abs(got[~hit] - ref[~hit]) <= lim[~hit]).all()
    # keys: a masked score is dropped whatever it is
    t = Tree(54, [60], [20], 8, 2, 128, fp8=fp8)
    ref = t.run()
    b, o = t.slot(0, 19)
    if fp8:
        t.parts[0][b, o] = 0x7F
        t.parts[1][b, o] = np.nan
    else:
        t.parts[0][b, o] = value
    got = t.run()
    unseen = ~t.mask[:, 19]
    assert unseen.sum() >= 19 and np.array_equal(got[unseen], ref[unseen])


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_bad_sequences_and_blocks_are_skipped_and_recorded(fp8):
    t = Tree(61, [90, 200, 40], [6, 9, 4], 8, 2, 64, fp8=fp8)
    ref = t.run()
    # a bad block: its keys drop out
    t.tables[1, 3] = t.NB
    t.stage()
    got = t.call().cpu().numpy().astype(np.float64)
    assert pkv.pkv_get_device_error() == (2, t.MB + 3)
    t.check(got)
    t.tables[1, 3] = -1
    t.stage()
    t.check(t.call().cpu().numpy().astype(np.float64))
    assert pkv.pkv_get_device_error() == (2, t.MB + 3)
    # sequences that do not fit their bounds: rows left alone, the others right
    t = Tree(61, [90, 200, 40], [6, 9, 4], 8, 2, 64, fp8=fp8)
    for change in ("short", "long", "negative", "table", "bound"):
        d = t.stage()
        lens = np.array(t.lens, np.int32)
        kw = {}
        if change == "short":
            lens[1] = 8       # fewer tokens than drafted ones
        elif change == "long":
            lens[1] = 201     # past max_seq_len
        elif change == "negative":
            lens[1] = -4
        elif change == "table":
            lens[1], kw = t.MB * BS + 1, dict(maxL=10000)
            d["ws"] = torch.zeros(pkv.pkv_tree_workspace_bytes(3, 8, 2, 64, 19, 9, 10000),
                                  dtype=torch.uint8, device="cuda")
        else:
            kw = dict(maxq=8)
        d["lens"] = dev(lens)
        got = t.call(**kw).cpu().numpy().astype(np.float64)
        assert pkv.pkv_get_device_error() == (3, 1), change
        rows = np.r_[0:6, 15:19]
        assert np.array_equal(got[rows], ref[rows]) and (got[6:15] == 7.0).all()


@pytest.mark.parametrize("start", [(2 ** 31 - 1, -2 ** 31), (-5, 3), (9, 6), (6, 20), (1, -1)])
def test_query_starts_that_do_not_fit_are_skipped_and_recorded(start):
    # the first pair's difference is 1 in 32 bits
    t = Tree(64, [90, 200, 40], [6, 9, 4], 8, 2, 64)
    ref = t.run()
    qs = t.qs.copy()
    qs[1:3] = start  # of sequence 1; its neighbours end and begin there
    t.d["qs"] = dev(qs)
    t.d["out"].fill_(7.0)
    t.call()
    got = t.d["out"].cpu().numpy().astype(np.float64)
    kind, index = pkv.pkv_get_device_error()
    assert kind == 3 and index in (0, 1, 2)
    ok = [i for i in range(3) if 0 <= qs[i] <= qs[i + 1] <= 19
          and int(qs[i + 1]) - int(qs[i]) <= min(9, t.lens[i])]
    rows = np.zeros(19, bool)
    for i in ok:
        rows[qs[i]:qs[i + 1]] = True
    assert (got[~rows] == 7.0).all() and np.isfinite(got[rows]).all()
    if 0 in ok and qs[1] == 6:
        assert np.array_equal(got[:6], ref[:6])


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_in_place_queries(fp8):
    # whole items, items split over many CTAs and several tiles
    t = Tree(65, [90, 6000, 300, 17, 500], [6, 20, 70, 1, 33], 16, 2, 128, fp8=fp8)
    ref = t.run()
    for _ in range(5):
        t.d["q"] = dev(t.q)
        got = t.call(out=t.d["q"]).cpu().numpy().astype(np.float64)
        assert np.array_equal(got, ref)


def test_rows_behind_the_last_sequence_stay():
    t = Tree(62, [90, 50], [6, 5], 8, 2, 64)
    ref = t.run()
    d = t.stage()
    d["q"] = torch.cat([d["q"], torch.full_like(d["q"][:3], float("nan"))])
    d["mask"] = torch.cat([d["mask"], torch.full_like(d["mask"][:3], -1)])
    out = torch.full((14, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    t.call(d, out=out)
    got = out.cpu().numpy().astype(np.float64)
    assert np.array_equal(got[:11], ref) and (got[11:] == 7.0).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_calls_repeat_bit_for_bit_and_stay_in_bounds(fp8):
    t = Tree(63, [3000, 900, 77], [16, 30, 5], 16, 4, 128, fp8=fp8)
    d = t.stage()
    n, pad = d["out"].numel(), 4096
    buf = torch.full((n + 2 * pad,), 0x7BAD, dtype=torch.int16, device="cuda")
    out = buf[pad:pad + n].view(torch.float16).view(d["out"].shape)
    wn = d["ws"].numel()
    ws = torch.full((wn + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    t.call(out=out, ws=ws[:wn])
    a = out.clone()
    ws[:wn] = 0x3C  # nothing is carried from call to call
    for _ in range(5):
        t.call(out=out, ws=ws[:wn])
    assert torch.equal(out, a)
    assert (buf[:pad] == 0x7BAD).all() and (buf[pad + n:] == 0x7BAD).all()
    assert (ws[wn:] == 0xA5).all()
    t.check(a.cpu().numpy().astype(np.float64))


def test_streams_with_their_own_workspaces():
    trees = [Tree(70 + i, [1200 + 311 * i, 90], [12 + i, 4], 16, 4, 128, fp8=i % 2 == 1)
             for i in range(4)]
    refs = [torch.from_numpy(t.run()) for t in trees]
    streams = [torch.cuda.Stream() for _ in trees]
    torch.cuda.synchronize()
    for _ in range(10):
        for t, s in zip(trees, streams):
            with torch.cuda.stream(s):
                t.call()
    torch.cuda.synchronize()
    for t, ref in zip(trees, refs):
        assert torch.equal(t.d["out"].cpu().double(), ref)
    assert pkv.pkv_get_device_error() == (0, -1)


def test_a_long_cache_past_32_bits_of_bytes():
    # block ids at the end of a 4.3 GB cache
    t = Tree(81, [200], [9], 8, 8, 128)
    ref = t.run()
    NB = (1 << 32) // (BS * 8 * 128 * 2) + t.NB
    big = []
    for x in t.parts:
        c = torch.zeros(NB, BS, 8, 128, dtype=torch.float16, device="cuda")
        c[NB - t.NB:] = dev(x)
        big.append(c)
    d = t.stage()
    d["caches"] = big
    d["tables"] = torch.where(d["tables"] < t.NB, d["tables"] + (NB - t.NB), d["tables"])
    t.NB = NB
    assert np.array_equal(t.call().cpu().numpy().astype(np.float64), ref)
    assert pkv.pkv_get_device_error() == (0, -1)


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_more_sequences_than_threads(fp8):
    rng = np.random.default_rng(91)
    nodes = [int(n) for n in rng.integers(0, 4, 700)]
    nodes[13], nodes[600] = 40, 70  # three and five tiles among the many of one
    lens = [n + int(c) for n, c in zip(nodes, rng.integers(0, 60, 700))]
    Tree(92, lens, nodes, 16, 2, 64, fp8=fp8).check()


def test_nothing_to_do_leaves_the_outputs():
    t = Tree(93, [5, 0], [0, 0], 8, 2, 64)
    t.q = np.zeros((3, 8, 64), np.float16)  # rows of no sequence
    t.mask = np.ones((3, 1), bool)
    d = t.stage()
    t.call()
    assert pkv.pkv_get_device_error() == (0, -1) and (d["out"] == 7.0).all()


def test_fp8_scales_over_many_orders():
    # value scales from 1e-7 to 100 and key scales from 1e-5 to 0.1, row by row
    t = Tree(94, [700, 300], [20, 33], 8, 2, 128, fp8=True, spread=3.0)
    rng = np.random.default_rng(95)
    live = np.isfinite(t.parts[1])
    t.parts[1][live] = 10.0 ** rng.uniform(-5, -1, live.sum())
    t.parts[3][live] = 10.0 ** rng.uniform(-7, 2, live.sum())
    t.check()
    # and all of them far out (an output of 1e-12 is nothing in fp16)
    for v in (1e-12, 90.0):
        t.parts[3][live] = v
        t.check()


@pytest.mark.parametrize("value", [1e6, 1e20, 3e38])
def test_fp8_a_masked_rows_large_scale_reaches_only_those_that_see_it(value):
    for seed, lens, nodes in ((101, [300], [20]), (102, [40], [33]), (103, [900, 200], [12, 90])):
        t = Tree(seed, lens, nodes, 8, 2, 128, fp8=True)
        Q = nodes[0]
        b, o = t.slot(0, Q - 1)
        t.parts[3][b, o] = value
        sees = t.mask[:, Q - 1].copy()
        sees[Q:] = False
        assert sees[:Q].sum() < Q
        t.check(rows=~sees)


def test_fp8_a_large_scale_of_a_key_without_weight():
    # a context key that no row gives weight to, with a value scale 1e5 times
    # the others'
    t = Tree(104, [500], [12], 4, 1, 64, fp8=True)
    t.q = np.abs(t.q).astype(np.float16)
    table = spec.e4m3_table()
    for p in (3, 130, 400):
        b, o = t.tables[0, p // BS], p % BS
        t.parts[0][b, o] = 0xF8  # -256 everywhere
        t.parts[1][b, o] = 0.01
        t.parts[3][b, o] = 1000.0
    got = t.run()
    ref, terms = t.want()
    # These keys' scores are 14 or more below their row's largest one, so their
    # weight times 1000 is below e^-14 1000 < 2^-10 of the largest weight, less
    # than that weight times its own scale (0.5/150 > 2^-9).  A product of
    # weight and scale below fp16's normal range is off by 2^-25 of the largest
    # such product, at most (largest weight) 1.5/150, and by 448 times that in
    # O: the bound's max |v| is that of the other rows, 448 * 1.5/150.
    s = -256 * 0.01 * t.q.astype(np.float64).sum(-1) * t.scale
    assert table[0xF8] == -256
    k, v = t.values()
    top = np.array([[(t.q[r, h].astype(np.float64) * k[t.tables[0, np.arange(488) // BS],
                                                       np.arange(488) % BS, 0]).sum(-1).max()
                     for h in range(4)] for r in range(12)]) * t.scale
    assert (s - top < -14).all()
    terms["vmax"] = np.minimum(terms["vmax"], 448 * 1.5 / 150)
    tol = spec.tree_tolerance(ref, terms, 64)
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / tol).max()


@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_fp8_scales_that_are_not_finite(value):
    t = Tree(96, [300], [20], 8, 2, 128, fp8=True)
    ref = t.run()
    b, o = t.slot(0, 7)
    t.parts[3][b, o, 1] = value  # the value scale of drafted token 7, KV head 1
    got = t.run()
    sees = t.mask[:, 7]
    assert sees.any() and not sees.all()
    assert np.array_equal(got[~sees], ref[~sees]) and np.array_equal(got[:, :4], ref[:, :4])
    assert not np.isfinite(got[sees][:, 4:]).any()
    k, v = t.values()
    with np.errstate(invalid="ignore"):
        want = t.want()[0]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    t = Tree(96, [300], [20], 8, 2, 128, fp8=True)
    t.parts[1][b, o, 0] = value  # a key scale: rows that do not see it stay as they were
    got = t.run()
    assert np.array_equal(got[~sees], ref[~sees]) and np.array_equal(got[:, 4:], ref[:, 4:])
    assert np.isnan(got[sees][:, :4]).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_non_finite_context_reaches_every_row(fp8):
    t = Tree(97, [300], [20], 8, 2, 128, fp8=fp8)
    ref = t.run()
    b, o = t.tables[0, 3], 5  # a position of the context, KV head 0
    if fp8:
        t.parts[2][b, o, 0, 9] = 0x7F
    else:
        t.parts[1][b, o, 0, 9] = np.nan
    got = t.run()
    hit = np.zeros(got.shape, bool)
    hit[:, :4, 9] = True
    assert np.isnan(got[hit]).all() and np.array_equal(got[~hit], ref[~hit])


def test_calls_of_other_kinds_follow_on_the_stream():
    # the merge lets the next kernel start early: a decode, a chunk attention
    # and a cache write that follow at once see what they should, and leave the
    # tree's outputs alone
    t = Tree(98, [900, 333, 64], [12, 30, 5], 16, 4, 128)
    d = t.stage()
    S = 3
    q = torch.randn(S, 16, 128, device="cuda").half()
    lens = torch.tensor([880, 300, 59], dtype=torch.int32, device="cuda")
    qs = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    dws = torch.zeros(pkv.pkv_decode_workspace_bytes(S, 16, 4, 128, 1000), dtype=torch.uint8,
                      device="cuda")
    cws = torch.zeros(pkv.pkv_chunk_workspace_bytes(S, 16, 4, 128, S, 1, 1000), dtype=torch.uint8,
                      device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]

    def follow():
        a = (d["tables"], lens)
        pkv.pkv_decode_attention(outs[0], q, *d["caches"], *a, t.scale, 16, 4, 128, BS, 1000, t.NB,
                                 dws)
        t.call()
        pkv.pkv_chunk_attention(outs[1], q, *d["caches"], *a, qs, t.scale, 16, 4, 128, BS, 1, 1000,
                                t.NB, cws)

    t.call()
    torch.cuda.synchronize()
    ref = d["out"].clone()
    follow()
    torch.cuda.synchronize()
    dref = [x.clone() for x in outs]
    for _ in range(30):
        t.call()
        follow()
        t.call()
    torch.cuda.synchronize()
    assert torch.equal(d["out"], ref)
    assert torch.equal(outs[0], dref[0]) and torch.equal(outs[1], dref[1])
    assert pkv.pkv_get_device_error() == (0, -1)
