"""The tree attention's softmax weights far below a row's largest one: a key of
large weight in front of many alike ones, each of little weight, whose sum
counts.  Rounded to 16 bits for the product with the values, a weight must not
lose more than the bound says, however many keys there are."""

import numpy as np
import pytest

from oracle import speculative as spec
from test_gpu_tree import BS, Tree

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


def bound(ref, t, D):
    """tree_tolerance with weights no further off than 2^-35 of the row's largest.

    A weight stands in fp16 at 2^11 or more for the row's largest score so far
    (or an earlier one's, when that is up to 2^4 times as much): rounding moves
    it by 2^-11 of itself, or by 2^-25 where it is subnormal, 2^-36 of the
    largest.  The reference's own rounding takes less than a factor of two."""
    d = (D + 8) * 2.0 ** -24 * t["smax"]
    rel = 2.0 ** -11 + 2 * d + 2.0 ** -20 + (t["nvis"] / 16 + 64) * 2.0 ** -23
    return (np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + rel * t["A"] +
            t["nvis"] * 2.0 ** -35 * t["vmax"] / t["sumw"])


def sink(lens, nodes, H, Hk, D, fp8, below, at, seed=7):
    """Every row sees key `at` (from the end when negative) with weight 1 and value
    0, and the others e^-below with positive values."""
    t = Tree(seed, lens, nodes, H, Hk, D, fp8=fp8)
    t.mask[:] = True
    t.q[:] = 0
    t.q[..., 0] = 4
    x = below / (4 * t.scale)
    rng = np.random.default_rng(seed + 1)
    slots = [(t.tables[i, (at % n) // BS], (at % n) % BS) for i, n in enumerate(lens)]
    if fp8:
        kc, ks, vc, vs = t.parts
        live = np.isfinite(ks)
        kc[live] = 0
        vc[live] = rng.integers(0x40, 0x7F, vc.shape).astype(np.uint8)[live]  # 2 .. 448
        for b, o in slots:
            kc[b, o, :, 0], ks[b, o] = 0x38, x  # 1.0
            vc[b, o], vs[b, o] = 0, 1.0 / 150
    else:
        k, v = t.parts
        live = np.isfinite(k)
        k[live] = 0
        v[live] = rng.uniform(0.5, 1.5, v.shape).astype(np.float16)[live]
        for b, o in slots:
            k[b, o, :, 0], v[b, o] = x, 0
    return t


def check(t):
    got = t.run()
    ref, terms = t.want()
    tol = bound(ref, terms, t.D)
    assert (ref > 0).all() and np.isfinite(got).all()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"worst {np.max(np.abs(got - ref) / tol):.1f} of the bound, "
                           f"{np.max(np.abs(got / ref - 1)):.3f} relative")


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
@pytest.mark.parametrize("at", [0, 20000, -2], ids=["first", "middle", "drafted"])
@pytest.mark.parametrize("below", [12.0, 16.5, 20.0, 23.0])
def test_many_keys_of_little_weight(below, at, fp8):
    check(sink([40003], [3], 2, 1, 64, fp8, below, at))


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
@pytest.mark.parametrize("at", [0, 1200, -2], ids=["first", "middle", "drafted"])
@pytest.mark.parametrize("below", [12.0, 14.0, 16.5, 18.0, 20.0])
def test_many_keys_of_little_weight_in_a_batch(below, at, fp8):
    # (a single sequence is cut into many pieces, each with a reference of its own)
    check(sink([2500] * 40, [2] * 40, 4, 4, 64, fp8, below, at))


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_a_long_context(fp8):
    check(sink([131072], [2], 1, 1, 128, fp8, 17.4, 0))


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
@pytest.mark.parametrize("at", [0, -1])
def test_items_of_many_sequences(at, fp8):
    # items that one CTA works through from end to end, and ones that are cut
    check(sink([900, 2000, 1500, 700] * 6, [2, 1, 5, 3] * 6, 8, 8, 64, fp8, 16.5, at))


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
@pytest.mark.parametrize("step", [1.3, 2.7, 2.9, 5.5, 11.0])
def test_rising_scores_and_large_values(step, fp8):
    """Every 128 keys' scores are `step` (natural log) above those before: the
    reference follows, or stays just short of it, and the weights stay finite in
    16 bits with values at the type's largest ones."""
    L, D = 128 * 16, 64
    t = Tree(9, [L, 700], [2, 9], 2, 1, D, fp8=fp8)
    t.q[:] = 0
    t.q[..., 0] = 1
    for i, n in enumerate(t.lens):
        p = np.arange(n)
        b, o = t.tables[i, p // BS], p % BS
        score = (p // 128) * step / t.scale
        if fp8:
            t.parts[0][b, o] = 0
            t.parts[0][b, o, :, 0], t.parts[1][b, o, 0] = 0x38, score
            t.parts[2][b, o] = np.where(t.parts[2][b, o] & 0x80, 0xFE, 0x7E)
            t.parts[3][b, o, 0] = 140.0
        else:
            t.parts[0][b, o] = 0
            t.parts[0][b, o, :, 0] = score[:, None]
            t.parts[1][b, o] = np.sign(t.parts[1][b, o]) * 65504
    got = t.run()
    ref, terms = t.want()
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= bound(ref, terms, D)).all()


def test_fp8_value_scales_at_the_types_ends():
    """Scales up to 2^127 and down to 2^-120 on keys of matching scores: the
    products of weight and scale count, each of them finite."""
    t = Tree(10, [500, 260], [4, 9], 2, 1, 64, fp8=True)
    rng = np.random.default_rng(11)
    t.q[:] = 0
    t.q[..., 0] = 1
    for i, n in enumerate(t.lens):
        p = np.arange(n)
        b, o = t.tables[i, p // BS], p % BS
        lg = rng.uniform(-120, 127, n)
        lg[rng.random(n) < 0.3] = 0
        t.parts[0][b, o] = 0
        t.parts[0][b, o, :, 0] = 0x38
        # 2^lg of value for a weight of 2^-lg where it is large, 1 where it is small
        t.parts[1][b, o, 0] = np.where(lg > 0, -lg, 0) * np.log(2) / t.scale
        t.parts[3][b, o, 0] = 2.0 ** lg
        t.parts[2][b, o] = rng.integers(0x30, 0x41, (n, 1, 64))  # 0.5 .. 2.25
    got = t.run()
    ref, terms = t.want()
    assert np.isfinite(got).all() and (ref > 0).all()
    # A product's exponent is a score's and a scale's logarithm, up to 127 each,
    # in 32 bits: each is off by 127 2^-24 and the approximate logarithm by
    # 2^-22 of 127, together below 2^-14 relative; likewise the weight's.  The
    # subnormal term counts products of at most (code 2.25) / (code 0.5) of the
    # row's largest one: 2.25 of it.
    tol = (np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + (2.0 ** -11 + 2.0 ** -13) * terms["A"] +
           terms["nvis"] * 2.0 ** -35 * 2.25 / terms["sumw"] + 2.0 ** -13 * np.abs(ref))
    assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [200, 1000, 2000, 8000, 30000, 60000, -8000])
def test_scores_of_every_size(size, D, fp8):
    """Scores up to 2^36 in units of log2, far apart from each other: the largest
    one a row sees takes all the weight, and its value is the output.

    Keys are multiples c of one +-1 vector, c spread evenly over [-size, size] (in
    fp16, whose step is a tenth of their distance at most): neighbours among n
    keys are 2/n of the largest score apart, 2^-10 and more, where 32-bit sums are
    off by D 2^-24 of it, 2^-17.  The smallest distance is 2^-10 2^19 units: the
    runner-up's weight is nothing."""
    t = Tree(12, [300, 40, 1900], [20, 9, 3], 8, 2, D, fp8=fp8,
             scale=np.sign(size) * D ** -0.5)
    a = abs(size)
    rng = np.random.default_rng(13)
    u = rng.choice([-1, 1], D)
    t.q[:] = a * u * rng.choice([-1, 1], t.q.shape[:2])[..., None]
    for i, n in enumerate(t.lens):
        p = np.arange(n)
        b, o = t.tables[i, p // BS], p % BS
        for h in range(2):
            c = rng.permutation(np.linspace(-a, a, n))
            if fp8:
                t.parts[0][b, o, h] = np.where(u > 0, 0x7E, 0xFE)  # 448, -448
                t.parts[1][b, o, h] = c / 448
            else:
                t.parts[0][b, o, h] = c[:, None] * u
    got = t.run()
    ref, terms = t.want()
    assert (terms["sumw"] < 1 + 1e-6).all()
    tol = np.abs(ref) * 2.0 ** -9 + 2.0 ** -24  # value, weight, quotient, output
    assert (np.abs(got - ref) <= tol).all(), (np.isnan(got).sum(), (got == 0).sum(), got.size)
