"""An infinite value that some rows of a chunk see: it is their output, of its own sign,
and no other row's, whichever of the two kernels takes the chunk."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402
from test_gpu_scored import Case, want_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


@pytest.mark.parametrize("L,Q", [(200, 4), (200, 2), (200, 60), (20, 4), (1500, 3)])
@pytest.mark.parametrize("what", [np.inf, -np.inf])
def test_seen_infinities(L, Q, what):
    # places: the last token's value; the oldest key of the first row's window, in
    # the first block of the window; one in the first block of all, in the prefix
    c = Case([107, L, Q], [L], [Q], 4, 2, 64, spread=0.7)
    window = 17
    rules = dict(window=window, prefix_lens=[5], softcap=20.0)
    ref, tol = want_of(c, rules)
    places = {L - 1: 3, max(L - Q - window + 1, 6): 9, 4: 13}
    for p, d in places.items():
        c.codes[1][c.at(0, [p]), 1, d] = what
    got = c.run(True, **rules)
    for r in range(Q):
        a = L - Q + r
        for d in range(64):
            for h in range(4):
                sees = any(pd == d and h >= 2 and (p < 5 or (p <= a and a - p < window))
                           for p, pd in places.items())
                if sees:
                    assert got[r, h, d] == what, (r, h, d, got[r, h, d])
                else:
                    assert abs(got[r, h, d] - ref[r, h, d]) <= tol[r, h, d], (r, h, d)
    assert pkv.pkv_get_device_error()[0] == 0


def test_both_signs_make_nan():
    c = Case(108, [90], [3], 2, 1, 64)
    c.codes[1][c.at(0, [88]), 0, 5] = np.inf
    c.codes[1][c.at(0, [89]), 0, 5] = -np.inf
    got = c.run(True, window=30)
    assert np.isfinite(got[0]).all() and (got[1, :, 5] == np.inf).all()
    assert np.isnan(got[2, :, 5]).all()
