"""Query starts whose difference wraps in 32 bits look like a few rows far outside the
buffers: their sequences are skipped and recorded."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu
LO, HI = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("start", [(HI, LO), (HI, LO + 39), (HI - 20, LO + 19), (HI - 39, LO),
                                   (HI, LO + 3)])
def test_chunk(start, scored):
    # sequences 1 and 2 meet at a start of their own; 40 rows (160 with the group)
    # are the tile kernel's, a few the balanced schedule's
    from test_gpu_scored import Case
    lens, news = [90, 200, 140, 60], [40, 40, 33, 2]
    c = Case([111, scored], lens, news, 8, 2, 64)
    rules = dict(window=50) if scored else {}
    c.upload(**rules)
    last = set(range(int(c.start[3]), int(c.start[4])))
    ref, tol = c.want(rows=last, **rules)
    # (without rules the row's largest weight stands at 1 or above: half a step of fp16's
    # smallest, 2^-25 of it, for each key)
    tol = tol + max(lens) * 2.0 ** -25 * 6.0

    def call():
        c.d["out"].fill_(7.0)
        if scored:
            return c.call(True).cpu().numpy()
        pkv.pkv_chunk_attention(c.d["out"], c.d["q"], *c.d["codes"], c.d["tables"], c.d["lens"],
                                c.d["start"], c.scale, 8, 2, 64, 16, c.maxq, c.maxl, c.NB, c.d["ws"])
        return c.d["out"].cpu().numpy()

    def right(got):
        rows = sorted(last)
        return (np.abs(got[rows].astype(float) - ref[rows]) <= tol[rows]).all()

    got = call()
    assert pkv.pkv_get_device_error()[0] == 0 and np.isfinite(got).all() and right(got)
    bad = c.start.copy()
    bad[1:3] = start
    c.d["start"].copy_(torch.from_numpy(bad))
    got = call()
    kind, index = pkv.pkv_get_device_error()
    assert kind == 3 and index in (0, 1, 2)
    # sequences 0 to 2 end or begin at a bad start
    assert (got[:c.start[3]] == 7).all() and right(got)


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("start", [(HI, LO), (HI, LO + 4), (HI - 3, LO), (HI - 255, LO), (HI, LO + 255)])
def test_verify(start, drafted):
    from test_gpu_verify import call, check, make
    c = make(np.random.default_rng([112, drafted]), [3, 5, 4, 6], 50, drafted)
    check(c, 4, call(c, 4))
    bad = dict(c, start=c["start"].copy())
    bad["start"][1:3] = start
    path, lens, nxt = call(bad, 4)
    kind, index = pkv.pkv_get_device_error()
    assert kind == 3 and index in (0, 1, 2)
    for i in range(3):
        assert path[i].tolist() == [-1] * 4 and lens[i] == 0 and nxt[i] == -1
    want = call(c, 4)
    assert np.array_equal(path[3], want[0][3])
    assert (lens[3], nxt[3]) == (want[1][3], want[2][3])
