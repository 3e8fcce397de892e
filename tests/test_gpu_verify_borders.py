"""pkv_tree_verify against its definition wherever no comparison is closer to its border
than the error that the kernel's arithmetic can have made there, derived rejection by
rejection."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402
from test_gpu_verify import call, make  # noqa: E402

pytestmark = pytest.mark.gpu

# An element of the rest, max(p - C q, 0) with C as a pair of fp32, is two fused
# multiply-adds: each rounds by half a step, 2^-24 of a result that is at most the
# element and C's low part times q (2^-24 of C q).  Four neighbours are added in fp32, two
# more half steps of a partial sum of non-negative numbers, and from there everything is
# a pair, off by 2^-45 of it or so.  SUM is what a sum of the rest is off by, relative to
# itself; what an error of C (a sum of earlier masses) does to it is counted apart.
STEP = 2.0 ** -24
SUM = 4 * STEP + 2.0 ** -40


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


def walk(c, max_depth):
    """The definition in 64 bits, and per sequence the smallest ratio of a comparison's
    distance from its border to the error allowed there."""
    S = len(c["start"]) - 1
    path = np.full((S, max_depth), -1, np.int32)
    lens, nxt, margin = np.zeros(S, np.int32), np.zeros(S, np.int32), np.full(S, np.inf)
    draft, au, su = c["draft"], c["au"].astype(np.float64), c["su"].astype(np.float64)
    for i in range(S):
        r0, r1 = int(c["start"][i]), int(c["start"][i + 1])
        at, depth, path[i, 0] = 0, 1, 0
        while True:
            p = c["target"][r0 + at].astype(np.float64)
            q = None if draft is None else draft[r0 + at].astype(np.float64)
            W, C, eW, eC = 1.0, 0.0, 0.0, 0.0
            rest, step, gone = p, -1, set()
            for k in range(at + 1, r1 - r0) if depth < max_depth else ():
                if int(c["parents"][r0 + k]) != at:
                    continue
                tok, u = int(c["tokens"][r0 + k]), au[r0 + k]
                if q is None:
                    have = 0.0 if tok in gone else p[tok]
                    ask, err = u * W, u * eW + 2.0 ** -44
                else:
                    have = max(p[tok] - C * q[tok], 0.0)
                    ask = u * W * q[tok]
                    err = q[tok] * (u * eW + eC) + 2.0 ** -44 * (p[tok] + C * q[tok])
                margin[i] = min(margin[i], abs(ask - have) / max(err, 1e-300))
                if ask < have:
                    step = k
                    break
                if q is None:
                    gone.add(tok)
                    W, eW = W - have, eW + 2.0 ** -44
                    if W <= 0:
                        raise AssertionError("an empty rest has no border to keep away from")
                else:
                    C, eC = C + W, eC + eW
                    rest = np.maximum(p - C * q, 0.0)
                    W = rest.sum()
                    # (an element within C's error of zero counts with that error)
                    eW = eC * q[p - C * q > -eC * q].sum() + SUM * W + 2.0 ** -24 * STEP * C
                    assert W > 4 * eW
            if step < 0:
                break
            path[i, depth] = step
            depth, at = depth + 1, step
        lens[i] = depth
        if q is None:
            rest = rest.copy()
            rest[list(gone)] = 0
        run = np.cumsum(rest)
        # the running sum before an element and the goal are both sums with their errors
        carried = 0.0 if q is None else eC * np.cumsum(q * (p - C * q > -eC * q))
        err = SUM * run + carried + su[i] * (eW if q is not None and C else SUM * run[-1])
        goal = su[i] * run[-1]
        nxt[i] = int(np.argmax(run > goal))
        border = np.abs(run - goal)
        here = rest > 0  # (a token without mass is never drawn)
        margin[i] = min(margin[i], (border[here] / (err[here] + 2.0 ** -60)).min())
    return path, lens, nxt, margin


CASES = [([2] * 40, 64, 2), ([5] * 30, 1000, 5), ([9] * 30, 4099, 6), ([16] * 16, 32000, 8),
         ([33] * 12, 515, 12), ([3, 1, 6, 2] * 6, 50257, 4)]


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("case", CASES, ids=[f"{len(c[0])}x{c[0][0]}v{c[1]}" for c in CASES])
def test_up_to_the_derived_border(case, drafted):
    counts, V, depth = case
    c = make(np.random.default_rng([21, len(counts), V]), counts, V, drafted, sharp=2.0)
    path, lens, nxt, margin = walk(c, depth)
    sure = margin > 1
    assert sure.mean() > 0.9
    for a, b, what in zip(call(c, depth), (path, lens, nxt), ("path", "lens", "next")):
        assert np.array_equal(a[sure], b[sure]), what
    assert pkv.pkv_get_device_error()[0] == 0


def test_draws_right_beside_a_border():
    """Numbers placed a few derived errors to either side of a running sum."""
    rng = np.random.default_rng(22)
    V, S = 4099, 64
    c = make(rng, [1] * S, V, False, sharp=1.0)
    run = np.cumsum(c["target"].astype(np.float64), 1)
    at = rng.integers(V // 4, V - 1, S)
    side = np.where(np.arange(S) % 2 == 0, -1.0, 1.0)
    goal = run[np.arange(S), at] / run[:, -1]
    # the running sum, the whole sum and the number's own rounding
    c["su"] = (goal * (1 + side * (2 * SUM + 2 * STEP))).astype(np.float32)
    path, lens, nxt, margin = walk(c, 1)
    assert (margin > 1).mean() > 0.9
    got = call(c, 1)[2]
    sure = margin > 1
    assert np.array_equal(got[sure], nxt[sure])
    assert (nxt[side > 0] > at[side > 0])[sure[side > 0]].all()
