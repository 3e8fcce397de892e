"""pkv_tree_verify against its definition: whole numbers, equal wherever no comparison
of the definition is closer to its border than the kernel's rounding."""

import numpy as np
import pytest

from oracle import serving as srv

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu

# An element of the rest is off by 2^-24 of itself (one rounding), its sum by no more,
# and a test or a draw compares a product of two such sums with an element: 2^-22
# covers a chain of rejections up to a few siblings deep, 2^-18 all 255.
BORDER = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def trees(rng, counts, chain=False, wide=False):
    out = []
    for n in counts:
        for j in range(n):
            out.append(-1 if j == 0 else j - 1 if chain else 0 if wide
                       else int(rng.integers(max(0, j // 2 - 2), j)))
    return np.array(out, np.int32)


def make(rng, counts, V, drafted, sharp=3.0, **kw):
    T, S = int(sum(counts)), len(counts)
    parents = trees(rng, counts, **kw)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    logits = rng.standard_normal((T, V)) * sharp

    def softmax(x):
        w = np.exp(x - x.max(1, keepdims=True))
        return (w / w.sum(1, keepdims=True)).astype(np.float32)

    target = softmax(logits)
    noisy = softmax(logits + rng.standard_normal((T, V)) * 0.8)
    tokens = rng.integers(0, V, T).astype(np.int32)
    for i in range(S):
        for k in range(start[i] + 1, start[i + 1]):
            p = noisy[start[i] + parents[k]].astype(np.float64)
            tokens[k] = rng.choice(V, p=p / p.sum())
    return dict(tokens=tokens, parents=parents, start=start, target=target,
                draft=noisy if drafted else None, au=rng.random(T).astype(np.float32),
                su=rng.random(S).astype(np.float32))


def padded(rows, stride, shift):
    """The rows on the device, ``stride`` elements apart, the first at element ``shift``."""
    T, V = rows.shape
    flat = torch.full((shift + T * stride,), float("nan"), device="cuda")
    view = flat[shift:].view(T, stride)[:, :V]
    view.copy_(dev(rows))
    return view


def call(c, depth, target=None, draft=None):
    S = len(c["start"]) - 1
    path = torch.full((S, depth), 77, dtype=torch.int32, device="cuda")
    lens, nxt = (torch.full((S,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    d = None if c["draft"] is None else dev(c["draft"]) if draft is None else draft
    pkv.pkv_tree_verify(path, lens, nxt, dev(c["tokens"]), dev(c["parents"]), dev(c["start"]),
                        dev(c["target"]) if target is None else target, d, dev(c["au"]),
                        dev(c["su"]))
    return [x.cpu().numpy() for x in (path, lens, nxt)]


def check(c, depth, got, certain=0.9):
    path, lens, nxt, near = srv.verify(c["tokens"], c["parents"], c["start"], c["target"],
                                       c["draft"], c["au"], c["su"], depth)
    sure = near > BORDER
    assert sure.mean() >= certain
    for a, b, what in zip(got, (path, lens, nxt), ("path", "lens", "next")):
        assert np.array_equal(a[sure], b[sure]), what
    return lens


CASES = [
    # nodes of the sequences, vocabulary, depth of the path
    ([1], 1, 1), ([5], 3, 4), ([2, 1, 7, 3], 5, 8), ([4] * 9, 127, 4), ([6] * 5, 128, 3),
    ([16] * 20, 1000, 16), ([33, 2, 64, 1], 1025, 8), ([5] * 3, 32000, 5), ([9, 4], 50257, 16),
    ([63] * 2, 4099, 12), ([256, 3], 600, 256), ([8] * 160, 515, 8),
]


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("case", CASES, ids=[f"{len(c[0])}x{c[0][0]}v{c[1]}" for c in CASES])
def test_random_trees(case, drafted):
    counts, V, depth = case
    c = make(np.random.default_rng([len(counts), V]), counts, V, drafted)
    check(c, depth, call(c, depth))
    assert pkv.pkv_get_device_error()[0] == 0


@pytest.mark.parametrize("drafted", [True, False])
def test_chains_and_wide_levels(drafted):
    rng = np.random.default_rng(11)
    lens = []
    for kw in (dict(chain=True), dict(wide=True)):
        c = make(rng, [12] * 40, 300, drafted, sharp=1.0, **kw)
        # numbers near one reject sibling after sibling
        if "wide" in kw:
            c["au"] = (1 - c["au"] * 0.1).astype(np.float32)
        lens.append(check(c, 12, call(c, 12)))
    # (a fixed guess is seldom the target's choice among 300)
    assert (lens[0].max() > 1 or not drafted) and (lens[1] == 1).any()


@pytest.mark.parametrize("stride,shift,dstride,dshift", [(1003, 0, 1003, 0), (1004, 1, 1004, 1),
                                                         (1007, 3, 1010, 2), (1008, 4, 1012, 0)])
def test_rows_apart_and_unaligned(stride, shift, dstride, dshift):
    c = make(np.random.default_rng(12), [5, 9, 2], 1003, True)
    want = call(c, 6)
    got = call(c, 6, padded(c["target"], stride, shift), padded(c["draft"], dstride, dshift))
    for a, b in zip(got, want):
        assert np.array_equal(a, b)
    check(c, 6, got)


def test_borders_of_the_numbers():
    rng = np.random.default_rng(13)
    c = make(rng, [4] * 8, 64, True)
    for a, s in ((0.0, 0.0), (np.nextafter(np.float32(1), np.float32(0)), 0.9999999)):
        c["au"][:], c["su"][:] = a, s
        check(c, 4, call(c, 4), certain=0.0)
    # numbers outside [0, 1) count as the nearest inside
    c["au"][:], c["su"][:] = 0.0, 0.0
    want = call(c, 4)
    c["au"][:], c["su"][:] = -3.0, -1.0
    assert all(np.array_equal(a, b) for a, b in zip(call(c, 4), want))
    c["au"][:], c["su"][:] = 1 - 2.0 ** -24, 1 - 2.0 ** -24
    want = call(c, 4)
    c["au"][:], c["su"][:] = 1.0, 7.0
    assert all(np.array_equal(a, b) for a, b in zip(call(c, 4), want))


def test_zero_probability_is_never_drawn():
    V = 777
    rng = np.random.default_rng(14)
    target = np.zeros((3, V), np.float32)
    target[0, [5, 400, 776]] = [0.25, 0.5, 0.25]
    target[1, 3] = 1
    for su, want in ((0.0, 5), (0.2499, 5), (0.25, 400), (0.7499, 400), (0.75, 776), (0.9999999, 776)):
        c = dict(tokens=np.zeros(3, np.int32), parents=np.full(3, -1, np.int32),
                 start=np.array([0, 1, 2, 3], np.int32), target=target, draft=None,
                 au=rng.random(3).astype(np.float32), su=np.full(3, su, np.float32))
        path, lens, nxt = call(c, 2)
        assert nxt.tolist() == [want, 3, -1]  # (a row without any mass has no next token)
        assert path.tolist() == [[0, -1]] * 3 and lens.tolist() == [1, 1, 1]


def test_an_empty_rest_stands_back():
    # drafts that cover the target whole: a rejected child leaves nothing, and the
    # next token comes from what was there before
    target = np.array([[0.5, 0.5, 0, 0]] * 2, np.float32)
    draft = np.array([[1.0, 1.0, 0, 0]] * 2, np.float32)  # (not a distribution)
    c = dict(tokens=np.array([0, 1], np.int32), parents=np.array([-1, 0], np.int32),
             start=np.array([0, 2], np.int32), target=target, draft=draft,
             au=np.array([0, 0.75], np.float32), su=np.array([0.75], np.float32))
    assert [x.tolist() for x in call(c, 2)] == [[[0, -1]], [1], [1]]
    # the same token guessed twice has nothing left the second time
    c.update(draft=None, tokens=np.array([0, 0, 0], np.int32), start=np.array([0, 3], np.int32),
             parents=np.array([-1, 0, 0], np.int32), target=np.array([[0.5, 0.5, 0, 0]] * 3, np.float32),
             au=np.array([0, 0.6, 0.0], np.float32), su=np.array([0.0], np.float32))
    assert [x.tolist() for x in call(c, 2)] == [[[0, -1]], [1], [1]]


def test_negative_values_and_nan_count_as_zero():
    c = make(np.random.default_rng(15), [6] * 12, 200, True)
    for rows in (c["target"], c["draft"]):
        rows[rows < 1e-4] = np.nan
        rows[(rows < 1e-3) & ~np.isnan(rows)] *= -1
    check(c, 6, call(c, 6))


def test_bad_nodes_are_left_out():
    rng = np.random.default_rng(16)
    c = make(rng, [7] * 6, 90, True)
    clean = dict(c)
    # padding; a token past the vocabulary; a parent that is the node itself
    c["parents"] = c["parents"].copy()
    c["parents"][3] = -1
    got = call(c, 7)
    assert pkv.pkv_get_device_error()[0] == 0
    check(c, 7, got)
    for change in (dict(tokens=90), dict(tokens=-1), dict(parents=4), dict(parents=2 ** 31 - 1)):
        b = dict(clean)
        (name, value), = change.items()
        b[name] = clean[name].copy()
        b[name][4] = value
        got = call(b, 7)
        assert pkv.pkv_get_device_error() == (8, 4)
        b["parents"] = clean["parents"].copy()
        b["tokens"] = clean["tokens"]
        b["parents"][4] = -1
        check(b, 7, got)


def test_sequences_without_nodes_and_bad_starts():
    c = make(np.random.default_rng(17), [3, 0, 4], 50, True)
    got = call(c, 4)
    check(c, 4, got)
    assert got[0][1].tolist() == [-1] * 4 and got[1][1] == 0 and got[2][1] == -1
    assert pkv.pkv_get_device_error()[0] == 0
    for start in ([0, 3, 2, 7], [0, 3, 3, 8], [-1, 3, 3, 7]):
        b = dict(c, start=np.array(start, np.int32))
        got = call(b, 4)
        assert pkv.pkv_get_device_error()[0] == 3
        bad = [i for i in range(3) if start[i] < 0 or start[i + 1] > 7 or start[i] > start[i + 1]]
        for i in bad:
            assert got[0][i].tolist() == [-1] * 4 and got[1][i] == 0 and got[2][i] == -1
    big = make(np.random.default_rng(18), [257], 20, False)
    assert call(big, 4)[1].tolist() == [0] and pkv.pkv_get_device_error() == (3, 0)


def test_captured_and_on_two_streams():
    rng = np.random.default_rng(19)
    cases = [make(rng, [9] * 24, 2000, True) for _ in range(3)]
    buf = {k: dev(v) for k, v in cases[0].items()}
    outs = []
    for _ in range(2):
        outs.append((torch.zeros(24, 9, dtype=torch.int32, device="cuda"),
                     *(torch.zeros(24, dtype=torch.int32, device="cuda") for _ in range(2))))

    def run(o):
        pkv.pkv_tree_verify(*o, buf["tokens"], buf["parents"], buf["start"], buf["target"],
                            buf["draft"], buf["au"], buf["su"])

    run(outs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs[0])
    side = torch.cuda.Stream()
    for c in cases:
        for k, v in c.items():
            buf[k].copy_(dev(v))
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            run(outs[1])
        torch.cuda.current_stream().wait_stream(side)
        for o in outs:
            check(c, 9, [x.cpu().numpy() for x in o])
    assert pkv.pkv_get_device_error()[0] == 0
