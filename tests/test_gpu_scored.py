"""Decode and chunk attention under score rules against the float64 definition, each
element within a bound derived from the arithmetic (oracle.serving)."""

import numpy as np
import pytest

from oracle import serving as srv
from oracle import speculative as spec

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu
BS = 16
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def slopes_of(H):
    return (2.0 ** (-8.0 * (np.arange(H) + 1) / H)).astype(np.float32)


class Case:
    """Inputs on the host; every row of the caches that no sequence holds is NaN."""

    def __init__(self, seed, lens, news, H, Hk, D, fp8=False, spread=1.5, extra=3):
        rng = self.rng = np.random.default_rng(seed)
        self.H, self.Hk, self.D, self.fp8 = H, Hk, D, fp8
        self.lens = np.array(lens, np.int32)
        self.news = news
        self.start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        S, blocks = len(lens), -(-self.lens // BS)
        self.NB = int(blocks.sum()) + extra
        ids = rng.permutation(self.NB)
        self.tables = np.full((S, max(1, int(blocks.max()))), -9, np.int32)
        at = 0
        for i in range(S):
            self.tables[i, :blocks[i]] = ids[at:at + blocks[i]]
            at += blocks[i]
        shape = (self.NB, BS, Hk, D)
        self.scale = D ** -0.5
        self.q = (rng.standard_normal((int(self.start[-1]), H, D)) * spread).astype(np.float16)
        self.codes, self.scales, self.values = [], [], []
        table = spec.e4m3_table()
        for _ in range(2):
            if fp8:
                codes = rng.integers(0, 256, shape).astype(np.uint8)
                codes[(codes & 127) == 127] = 0
                # scales of every magnitude, as rows of every magnitude have them
                scale = (rng.uniform(0.004, 0.02, shape[:3])).astype(np.float32)
                self.codes.append(codes)
                self.scales.append(scale)
                self.values.append(None)
            else:
                self.codes.append(rng.standard_normal(shape).astype(np.float16))
        self.table = table
        self.held = np.zeros((self.NB, BS), bool)
        for i in range(S):
            for p in range(int(lens[i])):
                self.held[self.tables[i, p // BS], p % BS] = True
        self.poison(~self.held)

    def poison(self, where, what=np.nan):
        for x in self.codes:
            x[where] = 0x7F if self.fp8 else what
        for x in self.scales:
            x[where] = np.nan

    def at(self, seq, pos):
        m = np.zeros_like(self.held)
        for p in pos:
            m[self.tables[seq, p // BS], p % BS] = True
        return m

    def caches(self):
        if not self.fp8:
            return self.codes
        with np.errstate(invalid="ignore"):
            return [self.table[c] * s[..., None] for c, s in zip(self.codes, self.scales)]

    def want(self, rows=None, **rules):
        k, v = self.caches()
        return srv.scored_attention(self.q, k, v, self.tables, self.lens, self.start, self.scale,
                                    self.Hk, rows=rows, **rules)

    def upload(self, **rules):
        self.d = dict(q=dev(self.q), tables=dev(self.tables), lens=dev(self.lens),
                      start=dev(self.start), codes=[dev(x) for x in self.codes],
                      scales=[dev(x) for x in self.scales])
        self.d["out"] = torch.full_like(self.d["q"], 7.0)
        T, S = len(self.q), len(self.lens)
        self.maxq, self.maxl = max(1, max(self.news)), max(1, int(self.lens.max()))
        n = max(pkv.pkv_decode_workspace_bytes(S, self.H, self.Hk, self.D, self.maxl),
                pkv.pkv_chunk_workspace_bytes(S, self.H, self.Hk, self.D, T, self.maxq, self.maxl))
        self.d["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        self.rules = dict(rules)
        for k in ("slopes", "prefix_lens"):
            if self.rules.get(k) is not None:
                kind = np.float32 if k == "slopes" else np.int32
                self.rules[k] = dev(np.asarray(self.rules[k], kind))
        return self

    def call(self, chunk, out=None, ws=None):
        d = self.d
        out, ws = d["out"] if out is None else out, d["ws"] if ws is None else ws
        shape = (self.scale, self.H, self.Hk, self.D, BS)
        if chunk:
            pkv.pkv_chunk_attention_scored(out, d["q"], *d["codes"], d["tables"], d["lens"],
                                           d["start"], *shape, self.maxq, self.maxl, self.NB, ws,
                                           **self.rules)
        elif self.fp8:
            pkv.pkv_decode_attention_scored_fp8(out, d["q"], *d["codes"], *d["scales"], d["tables"],
                                                d["lens"], *shape, self.maxl, self.NB, ws,
                                                **self.rules)
        else:
            pkv.pkv_decode_attention_scored(out, d["q"], *d["codes"], d["tables"], d["lens"], *shape,
                                            self.maxl, self.NB, ws, **self.rules)
        return out

    def run(self, chunk, **rules):
        return self.upload(**rules).call(chunk).cpu().numpy().astype(np.float64)


def check(got, want, what=""):
    ref, tol = want
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = (np.abs(got - ref) / tol).max()
    assert worst <= 1, f"{what}: {worst} of the bound"


def some_rules(case, seed, H):
    """A handful of rule sets for the lengths of a case, each rule alone and together."""
    rng = np.random.default_rng(seed)
    S, longest = len(case.lens), int(case.lens.max())
    pre = rng.integers(-2, longest + 20, S)
    small = np.full(S, 4)
    s = slopes_of(H)
    w = int(rng.integers(2, max(3, longest)))
    return [dict(softcap=2.0), dict(softcap=30.0), dict(window=1), dict(window=16), dict(window=17),
            dict(window=w), dict(window=INT_MAX), dict(slopes=s), dict(prefix_lens=pre),
            dict(window=w, prefix_lens=small),
            dict(softcap=5.0, window=w // 2 + 1, slopes=s * 0.1, prefix_lens=pre)]


DECODE = [
    # lengths, H, Hk, D
    ([1, 2, 15, 16, 17, 33, 64], 4, 4, 64), ([100, 0, 513, 31], 8, 4, 128),
    ([300, 47], 16, 4, 128), ([129, 1, 290], 16, 2, 64), ([70, 260], 16, 16, 64),
    ([40, 90], 20, 20, 128), ([1500], 2, 1, 128),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", DECODE, ids=[f"{c[1]}h{c[2]}k{c[3]}" for c in DECODE])
def test_decode(case, fp8):
    lens, H, Hk, D = case
    c = Case([len(lens), H, D], lens, [1] * len(lens), H, Hk, D, fp8)
    for rules in some_rules(c, H, H):
        got = c.run(False, **rules)
        assert pkv.pkv_get_device_error()[0] == 0
        empty = [i for i, L in enumerate(lens) if L == 0]
        assert (got[empty] == 0).all()
        check(got, want_of(c, rules), str(rules))
        assert not c.d["ws"][:4 * len(lens) * Hk].any()  # tickets left at zero


def want_of(c, rules, rows=None):
    # (a sequence of length 0 has a query row in a decode, which the definition skips)
    return c.want(rows=rows, **{k: v for k, v in rules.items()})


CHUNK = [
    # lengths, new tokens, H, Hk, D
    ([5, 16, 33, 40, 19], [5, 3, 1, 7, 16], 4, 2, 64),      # short: the columns' policies
    ([1, 17, 50, 2], [1, 1, 1, 1], 32, 8, 128),             # single tokens
    ([30, 200], [2, 1], 16, 2, 64), ([90, 33], [4, 3], 16, 4, 128),
    ([170, 300, 40], [60, 140, 40], 8, 2, 128),             # tiles
    ([150, 213], [133, 97], 4, 4, 128), ([90, 240, 17], [17, 40, 17], 16, 2, 64),
    ([0, 12, 0, 60], [0, 4, 0, 33], 8, 4, 128), ([150, 40, 1, 100], [100, 40, 1, 3], 8, 8, 64),
]


@pytest.mark.parametrize("case", CHUNK, ids=[f"{c[2]}h{c[3]}k{c[4]}q{max(c[1])}" for c in CHUNK])
def test_chunk(case):
    lens, news, H, Hk, D = case
    c = Case([len(lens), H, D, 1], lens, news, H, Hk, D)
    for rules in some_rules(c, H + 1, H):
        got = c.run(True, **rules)
        assert pkv.pkv_get_device_error()[0] == 0
        check(got, want_of(c, rules), str(rules))


@pytest.mark.parametrize("rules", [dict(softcap=20.0), dict(window=5000), dict(window=4096),
                                   dict(window=300, prefix_lens=[4200, 7, 0]),
                                   dict(slopes=1, prefix_lens=[9000, 0, 4500])],
                         ids=["cap", "window5000", "window4096", "prefix", "slopes"])
def test_partitions_of_long_sequences(rules):
    lens, news, H, Hk, D = [9000, 300, 4500], [70, 20, 64], 4, 2, 64
    if rules.get("slopes") is not None:
        rules = dict(rules, slopes=slopes_of(H))
    c = Case(77, lens, news, H, Hk, D)
    rows = {0, 1, 31, 69, 70, 89, 90, 153}
    for _ in range(2):  # (the second call finds the workspace as the first did)
        got = c.run(True, **rules) if not hasattr(c, "d") else c.call(True).cpu().numpy().astype(float)
        ref, tol = want_of(c, rules, rows)
        r = sorted(rows)
        check(got[r], (ref[r], tol[r]))
    assert pkv.pkv_get_device_error()[0] == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_long_decode_split_over_many_ctas(fp8):
    c = Case(78, [20000, 3, 7000], [1] * 3, 8, 2, 128, fp8)
    for rules in (dict(softcap=10.0, slopes=slopes_of(8)), dict(window=6000, prefix_lens=[40, 2, 0]),
                  dict(window=19990, prefix_lens=[5, 5, 5])):
        check(c.run(False, **rules), want_of(c, rules), str(rules))


@pytest.mark.parametrize("fp8", [False, True])
def test_many_small_weights_are_kept(fp8):
    """One key far above 8000 others that together weigh as much as it does."""
    L, D = 8001, 64
    c = Case(79, [L], [1], 1, 1, D, fp8, extra=0)
    c.q[:] = 0
    c.q[0, 0, 0] = 8.0  # scores 8 k_0 / 8 = k_0
    one = 0x38
    for x, s in zip(c.codes, c.scales or [None, None]):
        x[c.held] = 0
        if fp8:
            s[c.held] = 1.0
    first = c.at(0, [0])
    c.codes[0][first] = 0
    if fp8:
        c.codes[0][first, 0, 0], c.scales[0][first, 0] = one, 9.0
        c.codes[1][c.held & ~first] = one
    else:
        c.codes[0][first, 0, 0] = 9.0
        c.codes[1][c.held & ~first] = 1.0
    rules = dict(softcap=60.0)
    got, (ref, tol) = c.run(False, **rules), want_of(c, rules)
    assert 0.3 < ref[0, 0, 0] < 0.7
    check(got, (ref, tol))
    if not fp8:
        c.news = [1]
        check(c.run(True, **rules), (ref, tol))
    # 17 nats down: 8000 e^-17 = 3e-4 of the mass, all of it in weights of 4e-8
    if fp8:
        c.scales[0][first, 0] = 17.0
    else:
        c.codes[0][first, 0, 0] = 17.0
    rules = dict(softcap=1e5)
    check(c.run(False, **rules), want_of(c, rules))


@pytest.mark.parametrize("cap", [1e-3, 0.5, 7.0, 300.0, 1e5, 1e15])
def test_caps_of_every_size(cap):
    c = Case(80, [200, 90], [70, 2], 8, 2, 128, spread=4.0)
    for chunk in (True, False):
        if not chunk:
            c = Case(81, [200, 90], [1, 1], 8, 2, 128, spread=4.0)
        check(c.run(chunk, softcap=cap), c.want(softcap=cap), f"{cap} {chunk}")


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_scales_of_either_sign(scale):
    for news in ([1, 1], [3, 2], [40, 150]):
        c = Case([95, len(news)], [200, 160], news, 8, 2, 64, spread=1.0)
        c.scale = scale
        for rules in (dict(softcap=3.0), dict(softcap=800.0, prefix_lens=[90, 0]), dict(window=30),
                      dict(softcap=2.0, slopes=slopes_of(8), window=90)):
            check(c.run(news != [1, 1], **rules), want_of(c, rules), f"{news} {rules}")


def test_slopes_of_either_sign():
    slopes = (slopes_of(8) * np.where(np.arange(8) % 3 == 1, -0.05, 1.0)).astype(np.float32)
    slopes[4] = 0
    for news in ([1, 1], [3, 2], [40, 150]):
        c = Case([96, len(news)], [300, 160], news, 8, 2, 128)
        for rules in (dict(slopes=slopes), dict(slopes=slopes, softcap=6.0, prefix_lens=[200, 160])):
            check(c.run(news != [1, 1], **rules), want_of(c, rules), f"{news} {rules}")


def test_masked_places_may_hold_anything():
    # decode: positions before the window and behind the prefix, in the same blocks
    for fp8 in (False, True):
        for what in (np.nan, np.inf, -np.inf):
            c = Case(82, [100, 333], [1, 1], 8, 4, 128, fp8)
            rules = dict(window=37, prefix_lens=[3, 20])
            want = want_of(c, rules)
            c.poison(c.at(0, range(3, 63)) | c.at(1, range(20, 296)), what)
            check(c.run(False, **rules), want, f"{fp8} {what}")
    # chunks: positions that no row sees
    for news in ([4, 2], [40, 90]):
        c = Case(83, [150, 333], news, 8, 4, 128)
        rules = dict(window=20, prefix_lens=[3, 0])
        want = want_of(c, rules)
        c.poison(c.at(0, range(3, 150 - news[0] - 19)) | c.at(1, range(0, 333 - news[1] - 19)))
        check(c.run(True, **rules), want, str(news))


@pytest.mark.parametrize("news", [[4], [60]])
@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_values_that_only_some_rows_see(news, what):
    L, Q = 200, news[0]
    c = Case(84, [L], news, 4, 2, 64)
    rules = dict(window=50, prefix_lens=[5])
    ref, tol = want_of(c, rules)
    # an element of the last token's value, one at the edge of the first row's
    # window, and one in the prefix's last block that nobody sees
    places = {L - 1: 3, L - Q - 49: 9, 8: 11, 4: 13}
    for p, d in places.items():
        c.codes[1][c.at(0, [p]), 1, d] = what
    got = c.run(True, **rules)
    for r in range(Q):
        a = L - Q + r
        for h in range(4):
            for d in range(64):
                sees = any(pd == d and h >= 2 and (p < 5 or (p <= a and a - p < 50))
                           for p, pd in places.items())
                if sees:
                    assert not np.isfinite(got[r, h, d]), (r, h, d)
                else:
                    assert abs(got[r, h, d] - ref[r, h, d]) <= tol[r, h, d], (r, h, d)


def test_bad_blocks_are_skipped_and_recorded():
    for news in ([1, 1], [3, 2], [50, 20]):
        c = Case(85, [100, 70], news, 8, 4, 64)
        rules = dict(window=60, prefix_lens=[20, 0], softcap=9.0)
        c.tables[0, 1], c.tables[1, 2] = c.NB, -1
        got = c.run(news != [1, 1], **rules)
        assert pkv.pkv_get_device_error()[0] == 2
        check(got, want_of(c, rules))
    # a block that no rule lets a token see is not looked at
    c = Case(86, [300], [1], 8, 4, 64)
    c.tables[0, 5] = -1
    check(c.run(False, window=40), want_of(c, dict(window=40)))
    assert pkv.pkv_get_device_error()[0] == 0
    # nothing left to see: zeros
    c = Case(87, [10], [1], 8, 4, 64)
    c.tables[0, 0] = -1
    assert (c.run(False, softcap=3.0) == 0).all()
    assert (c.run(True, softcap=3.0) == 0).all()
    assert pkv.pkv_get_device_error()[0] == 2


def test_bad_lengths():
    c = Case(88, [40, 50, 60], [1, 1, 1], 8, 2, 64)
    c.lens[1] = 10 ** 6
    c.upload(window=9)
    c.maxl = 64
    got = c.call(False).cpu().numpy().astype(float)
    assert pkv.pkv_get_device_error() == (3, 1)
    c.lens[1] = c.tables.shape[1] * BS
    ref, tol = c.want(window=9)
    for i in (0, 2):
        check(got[i], (ref[i], tol[i]))
    c = Case(89, [40, 50, 60], [20, 30, 40], 8, 2, 64)
    c.lens[1] = 20  # fewer tokens than new ones
    got = c.run(True, softcap=9.0)
    assert pkv.pkv_get_device_error() == (3, 1)
    ref, tol = c.want(rows=set(range(20)) | set(range(50, 90)), softcap=9.0)
    assert (got[20:50] == 7).all()
    check(np.delete(got, range(20, 50), 0), (np.delete(ref, range(20, 50), 0),
                                             np.delete(tol, range(20, 50), 0)))


@pytest.mark.parametrize("news", [[2, 1, 2], [30, 2, 17]])
def test_bad_query_starts(news):
    """Starts outside the rows, falling, or past the bound that the call was sized for:
    skipped and recorded, the others as they are."""
    lens = [90, 60, 77]
    rules = dict(softcap=4.0, window=33)
    c = Case([97, news[0]], lens, news, 8, 2, 64)
    ref, tol = want_of(c, rules)
    good = c.start.copy()
    for at, value, bad in ((0, -3, {0}), (3, good[3] + 1, {2}), (2, good[1] - 1, {1, 2}),
                           (1, 10 ** 6, {0, 1}), (1, -2 ** 31, {0, 1})):
        c.start = good.copy()
        c.start[at] = value
        got = c.run(True, **rules)
        assert pkv.pkv_get_device_error()[0] == 3
        for i in {0, 1, 2} - bad:
            rows = slice(good[i], good[i + 1])
            check(got[rows], (ref[rows], tol[rows]), f"{at} {value} sequence {i}")
    # more new tokens than max_query_len says (and than the call's kernels hold)
    c.start = good.copy()
    c.upload(**rules)
    if news[0] == 30:
        c.maxq = 2
        got = c.call(True).cpu().numpy().astype(float)
        assert pkv.pkv_get_device_error()[0] == 3
        assert (got[:30] == 7).all() and (got[32:] == 7).all()
        check(got[30:32], (ref[30:32], tol[30:32]))


def test_calls_in_flight_together_and_captured():
    c = Case(90, [500, 90, 1000], [30, 4, 1], 8, 2, 128)
    rules = dict(softcap=11.0, window=200, prefix_lens=[4, 4, 4])
    want = want_of(c, rules)
    c.upload(**rules)
    outs = [torch.zeros_like(c.d["out"]) for _ in range(3)]
    spaces = [torch.zeros_like(c.d["ws"]) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, w in zip(streams, outs, spaces):
            with torch.cuda.stream(s):
                c.call(True, o, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(True)
    c.d["out"].fill_(3.0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    first = outs[0].cpu().numpy()
    for o in outs + [c.d["out"]]:
        check(o.cpu().numpy().astype(float), want)
        assert np.array_equal(o.cpu().numpy(), first)
    assert pkv.pkv_get_device_error()[0] == 0


@pytest.mark.parametrize("H,Hk", [(1, 1), (8, 2)])
def test_many_sequences(H, Hk):
    """Lengths, prefixes and left-out blocks of 2500 sequences in shared memory."""
    S = 2500
    lens = [1 + (7 * i) % 60 for i in range(S)]
    rules = dict(window=9, prefix_lens=np.arange(S) % 5)
    c = Case(93, lens, [1] * S, H, Hk, 64)
    want = want_of(c, rules)
    for chunk in (False, True):
        check(c.run(chunk, **rules), want, str(chunk))
    # chunks of up to 20 tokens: both kernels of the call
    news = [1 + (3 * i) % min(20, n) for i, n in enumerate(lens)]
    c = Case(94, lens, news, H, Hk, 64)
    rows = set(range(0, len(c.q), 97))
    got, (ref, tol) = c.run(True, **rules), want_of(c, rules, rows)
    r = sorted(rows)
    check(got[r], (ref[r], tol[r]))
    assert pkv.pkv_get_device_error()[0] == 0


def test_outputs_stay_inside_their_buffer():
    c = Case(91, [300, 20], [45, 2], 8, 4, 64)
    c.upload(softcap=5.0, slopes=slopes_of(8))
    T = len(c.q)
    big = torch.full((T + 8, 8, 64), 5.0, dtype=torch.float16, device="cuda")
    n = pkv.pkv_chunk_workspace_bytes(2, 8, 4, 64, T, c.maxq, c.maxl)
    ws = torch.zeros(n + 512, dtype=torch.uint8, device="cuda")
    ws[:256], ws[256 + n:] = 0xAB, 0xAB
    for _ in range(2):
        c.call(True, big[4:4 + T], ws[256:256 + n])
    assert (big[:4] == 5).all() and (big[4 + T:] == 5).all()
    assert (ws[:256] == 0xAB).all() and (ws[256 + n:] == 0xAB).all()


def test_refused_tensors():
    c = Case(92, [30, 20], [1, 1], 8, 4, 64).upload(softcap=5.0)
    for rules in (dict(slopes=dev(np.zeros(7, np.float32))), dict(slopes=dev(np.zeros(8))),
                  dict(prefix_lens=dev(np.zeros(3, np.int32))),
                  dict(prefix_lens=torch.zeros(2, dtype=torch.int32))):
        c.rules = rules
        for chunk in (False, True):
            with pytest.raises(ValueError):
                c.call(chunk)
    for rules in (dict(window=-1), dict(window=2 ** 31), dict(window=2 ** 32 + 5)):
        c.rules = rules
        with pytest.raises(ValueError):
            c.call(False)
    c.rules = dict(softcap=-1.0)
    with pytest.raises(pkv.PkvError):
        c.call(False)
    c.rules = {}
    with pytest.raises(pkv.PkvError):
        c.call(True, ws=c.d["ws"][:16])
