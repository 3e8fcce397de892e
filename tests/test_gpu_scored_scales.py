"""FP8 decode under rules with value scales of every magnitude and either sign."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402
from test_gpu_scored import Case, check, slopes_of, want_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


RULES = [dict(softcap=20.0), dict(window=90, prefix_lens=[5, 0, 40]),
         dict(softcap=9.0, slopes=slopes_of(8) * 0.1)]


def scales_of(kind, shape, rng):
    """Value scales; outputs stay below fp16's largest with codes of at most 1 in size."""
    sign = rng.choice([-1.0, 1.0], shape)
    small = rng.uniform(0.004, 0.02, shape)
    if kind == "negative":
        return -small
    if kind == "either_sign":
        return sign * small
    if kind == "negative_among_zeros":
        return np.where(rng.random(shape) < 0.2, -small, 0.0)
    if kind == "zero":
        return np.zeros(shape)
    if kind == "some_zero":
        return np.where(rng.random(shape) < 0.5, small, 0.0)
    if kind == "large":
        return sign * 2.0 ** rng.uniform(8, 15, shape)
    if kind == "tiny":  # (fp32's subnormal numbers among them)
        return sign * 2.0 ** rng.uniform(-149, -30, shape)
    return sign * 2.0 ** rng.uniform(-120, 15, shape)


KINDS = ["negative", "either_sign", "negative_among_zeros", "zero", "some_zero", "large", "tiny",
         "every_magnitude"]


@pytest.mark.parametrize("rules", RULES, ids=["cap", "window_prefix", "cap_bias"])
@pytest.mark.parametrize("kind", KINDS)
def test_value_scales(kind, rules):
    """The bound counts a weight's rounding to fp16, once multiplied by its value's scale
    and brought below 2^15 times the row's largest such product: half a step, 2^-11 of it, or
    for the smallest 2^-25 / 2^15 of the largest; both are in the oracle's bound, whose
    last term holds 2^-31 of the largest value for every key."""
    c = Case([104, KINDS.index(kind)], [300, 47, 1000], [1, 1, 1], 8, 2, 128, True)
    values = np.where((c.codes[1] & 127) > 0x38, c.codes[1] & 0x80 | 0x38, c.codes[1])
    scale = scales_of(kind, c.scales[1].shape, c.rng).astype(np.float32)
    c.codes[1][c.held] = values[c.held]
    c.scales[1][c.held] = scale[c.held]
    with np.errstate(under="ignore"):
        got, want = c.run(False, **rules), want_of(c, rules)
    check(got, want, kind)
    assert pkv.pkv_get_device_error()[0] == 0


def test_a_negated_scale_negates_the_output():
    c = Case(105, [300, 47], [1, 1], 8, 2, 64, True)
    got = c.run(False, softcap=20.0)
    c.scales[1] *= -1
    assert np.array_equal(c.run(False, softcap=20.0), -got)


def test_key_scales_of_either_sign():
    c = Case(106, [300, 47, 90], [1, 1, 1], 8, 2, 64, True)
    c.scales[0][c.held] *= c.rng.choice([-1.0, 1.0], c.scales[0].shape).astype(np.float32)[c.held]
    for rules in RULES:
        check(c.run(False, **rules), want_of(c, rules), str(rules))
