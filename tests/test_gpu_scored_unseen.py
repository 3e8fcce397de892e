"""Under score rules an output does not depend on what a position holds that its token
does not see: equal bits whatever is there."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402
from test_gpu_scored import Case, slopes_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


def fill(c, where, what):
    """what: zeros; the largest finite keys, values and scales; or NaN."""
    for x in c.codes:
        if c.fp8:
            x[where] = {"zeros": 0, "large": 0x7E, "nan": 0x7F}[what]
        else:
            x[where] = {"zeros": 0, "large": 60000, "nan": np.nan}[what]
    for x in c.scales:
        x[where] = {"zeros": 0, "large": 1e30, "nan": np.nan}[what]


def same(got):
    for x in got[1:]:
        assert np.array_equal(got[0], x), f"rows {np.unique(np.where(got[0] != x)[0]).tolist()}"


LENS = [100, 333, 5, 250, 77, 19]
RULES = [dict(softcap=50.0), dict(softcap=50.0, window=37, prefix_lens=[3, 20, 0, 70, 0, 19]),
         dict(softcap=30.0, window=21, slopes=slopes_of(8)), dict(softcap=400.0, window=90)]


def unseen(c, rules):
    """Places that no row of the batch sees: not held, or left out by the rules."""
    window = rules.get("window", 0) or 10 ** 9
    prefix = rules.get("prefix_lens", [0] * len(c.lens))
    sees = np.zeros_like(c.held)
    for i, (L, Q) in enumerate(zip(c.lens, c.news)):
        pos = [p for p in range(L) if p < prefix[i] or p > L - Q - window]
        sees |= c.at(i, pos)
    return ~sees


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rules", RULES, ids=["cap", "window_prefix", "bias", "high_cap"])
def test_decode(rules, fp8):
    c = Case([101, fp8], LENS, [1] * len(LENS), 8, 2, 128, fp8)
    got = []
    for what in ("zeros", "large", "nan"):
        fill(c, unseen(c, rules), what)
        got.append(c.run(False, **rules))
        assert np.isfinite(got[-1]).all()
    same(got)


@pytest.mark.parametrize("news", [[1, 2, 2, 1, 2, 1], [4, 3, 2, 4, 1, 4], [60, 2, 3, 140, 1, 18]],
                         ids=["one_tile", "two_tiles", "long"])
@pytest.mark.parametrize("rules", RULES, ids=["cap", "window_prefix", "bias", "high_cap"])
def test_chunk(rules, news):
    c = Case([102, news[0]], LENS, news, 8, 2, 64)
    got = []
    for what in ("zeros", "large", "nan"):
        fill(c, unseen(c, rules), what)
        got.append(c.run(True, **rules))
        assert np.isfinite(got[-1]).all()
    same(got)


@pytest.mark.parametrize("group", [1, 2, 4])
def test_a_key_that_one_new_token_does_not_see(group):
    """The last new token's key, behind the others' positions: their rows keep their bits."""
    c = Case([103, group], [70, 210], [3, 4], 2 * group, 2, 64)
    rules = dict(softcap=50.0)
    got = []
    for what in ("zeros", "large"):
        fill(c, c.at(0, [69]) | c.at(1, [209]), what)
        got.append(c.run(True, **rules))
    for i, q1 in enumerate(c.start[1:]):
        rows = slice(c.start[i], q1 - 1)
        assert np.array_equal(got[0][rows], got[1][rows]), i
