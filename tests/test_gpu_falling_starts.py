"""Query starts that fall: neither the sequence that they fall in nor the one behind it,
which would start inside its neighbour's rows, is computed; the neighbour's rows are its own."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402
from test_gpu_scored import Case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("news,back", [([30, 2, 17], 1), ([30, 2, 17], 12), ([17, 20, 3], 9),
                                       ([2, 1, 1], 1), ([1, 2, 2], 1)])
def test_rows_of_the_sequence_before(news, back, scored):
    c = Case([112, back], [90, 60, 77], news, 8, 2, 64)
    rules = dict(window=33) if scored else {}
    c.upload(**rules)
    rows = set(range(news[0]))
    ref, tol = c.want(rows=rows, **rules)
    # (without rules the row's largest weight stands at 1 or above: half a step of fp16's
    # smallest, 2^-25 of it, for each key)
    tol = tol + 90 * 2.0 ** -25 * 6.0
    bad = c.start.copy()
    bad[2] = bad[1] - back
    bad[3] = bad[2] + min(news)  # (within max_query_len)
    c.d["start"].copy_(torch.from_numpy(bad))
    for _ in range(20):  # (which of two sequences wrote last was a matter of chance)
        c.d["out"].fill_(7.0)
        if scored:
            c.call(True)
        else:
            pkv.pkv_chunk_attention(c.d["out"], c.d["q"], *c.d["codes"], c.d["tables"], c.d["lens"],
                                    c.d["start"], c.scale, 8, 2, 64, 16, c.maxq, c.maxl, c.NB,
                                    c.d["ws"])
        got = c.d["out"].cpu().numpy().astype(float)
        kind, index = pkv.pkv_get_device_error()
        assert kind == 3 and index in (1, 2)
        assert (np.abs(got[:news[0]] - ref[:news[0]]) <= tol[:news[0]]).all()
        assert (got[news[0]:] == 7).all()


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("news", [[30, 2, 17], [2, 1, 2], [4, 0, 3]])
def test_rows_behind_the_last_sequence(news, scored):
    c = Case([113, news[0]], [90, 60, 77], news, 8, 2, 64)
    rules = dict(softcap=6.0) if scored else {}
    T, ref, tol = len(c.q), *c.want(**rules)
    tol = tol + 90 * 2.0 ** -25 * 6.0  # (as above)
    c.q = np.concatenate([c.q, np.full((9, 8, 64), np.nan, np.float16)])
    c.upload(**rules)
    if scored:
        c.call(True)
    else:
        pkv.pkv_chunk_attention(c.d["out"], c.d["q"], *c.d["codes"], c.d["tables"], c.d["lens"],
                                c.d["start"], c.scale, 8, 2, 64, 16, c.maxq, c.maxl, c.NB, c.d["ws"])
    got = c.d["out"].cpu().numpy().astype(float)
    assert pkv.pkv_get_device_error()[0] == 0
    assert (np.abs(got[:T] - ref) <= tol).all() and (got[T:] == 7).all()
