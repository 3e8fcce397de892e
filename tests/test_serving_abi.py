"""Refusals of the serving step's entry points: on the host, before any CUDA call."""

import ctypes

import pytest

import paged_kv_cache_131_gb300 as pkv
from paged_kv_cache_131_gb300 import _build

FAKE = 0x100000  # aligned, never dereferenced: every call below fails validation
OK, NULL, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4, -5
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def rules_of(**kw):
    r = dict(softcap=50.0, window=0, slopes=FAKE, prefix_lens=FAKE)
    r.update(kw)
    return pkv.pkv_score_rules(*r.values())


BAD_RULES = [(INVALID, dict(softcap=-1.0)), (INVALID, dict(softcap=float("nan"))),
             (INVALID, dict(softcap=float("inf"))), (INVALID, dict(softcap=3e38)),
             (INVALID, dict(softcap=1e-45, scale=1e6)), (INVALID, dict(window=-1)),
             (ALIGN, dict(slopes=FAKE + 2)), (ALIGN, dict(prefix_lens=FAKE + 1))]


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_scored(lib, fp8):
    def call(rules=True, rule=None, **kw):
        a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, sl=FAKE, scale=0.1,
                 H=32, Hk=8, D=128, bs=16, S=4, MB=8, maxL=100, NB=64, ws=None, wsb=0)
        a.update(kw)
        names = ["out", "q", "k", "v"] + (["ks", "vs"] if fp8 else []) + list(a)[6:]
        fn = lib.pkv_decode_attention_scored_fp8 if fp8 else lib.pkv_decode_attention_scored
        r = rules_of(**(rule or {}))
        return fn(*[a[n] for n in names], ctypes.byref(r) if rules else None, None)

    assert call(S=0) == OK
    assert call(S=-1) == INVALID
    for name in ("out", "q", "k", "v", "bt", "sl") + (("ks", "vs") if fp8 else ()):
        assert call(**{name: None}) == NULL, name
    assert call(rules=False) == NULL
    for kw in (dict(H=30), dict(MB=0), dict(NB=0), dict(scale=float("nan")), dict(maxL=-1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(H=24), dict(D=96), dict(bs=32), dict(S=70000), dict(MB=INT_MAX)):
        assert call(**kw) == UNSUPPORTED, kw
    # the sequences' lengths, prefixes and block counts do not fit shared memory
    assert call(S=20000) == UNSUPPORTED
    for kw in (dict(q=FAKE + 8), dict(sl=FAKE + 2), dict(ws=FAKE + 8)) + (
            (dict(ks=FAKE + 8),) if fp8 else ()):
        assert call(**kw) == ALIGN, kw
    for want, rule in BAD_RULES:
        rule = dict(rule)
        scale = rule.pop("scale", 0.1)
        assert call(rule=rule, scale=scale) == want, rule
    need = lib.pkv_decode_workspace_bytes(4, 32, 8, 128, 100)
    assert call() == WORKSPACE and call(ws=FAKE, wsb=64) == WORKSPACE and need > 64
    assert call(rule=dict(slopes=None, prefix_lens=None, softcap=0.0)) == WORKSPACE


def test_chunk_scored(lib):
    def call(rules=True, rule=None, **kw):
        a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, qs=FAKE, scale=0.1, H=32,
                 Hk=8, D=128, bs=16, S=4, MB=8, Tq=10, maxq=7, maxL=100, NB=64, ws=None, wsb=0)
        a.update(kw)
        r = rules_of(**(rule or {}))
        return lib.pkv_chunk_attention_scored(*a.values(), ctypes.byref(r) if rules else None, None)

    assert call(S=0) == OK and call(Tq=0) == OK
    for name in ("out", "q", "k", "v", "bt", "sl", "qs"):
        assert call(**{name: None}) == NULL, name
    assert call(rules=False) == NULL
    assert call(maxq=0) == INVALID and call(D=96) == UNSUPPORTED and call(qs=FAKE + 2) == ALIGN
    for want, rule in BAD_RULES:
        rule = dict(rule)
        scale = rule.pop("scale", 0.1)
        assert call(rule=rule, scale=scale) == want, rule
    assert call() == WORKSPACE


def test_resize(lib):
    names = ["bt", "sl", "nl", "ol", "fb", "fc", "ofc", "qs", "slots", "pos", "S", "MB", "T", "cap",
             "bs", "NB"]

    def call(**kw):
        a = dict.fromkeys(names[:10], FAKE)
        a.update(S=4, MB=8, T=32, cap=64, bs=16, NB=64)
        a.update(kw)
        return lib.pkv_resize_sequences(*[a[n] for n in names], None)

    assert call(S=0) == OK and call(S=0, bt=None) == OK
    for kw in (dict(S=-1), dict(T=-1), dict(cap=-1), dict(MB=0), dict(bs=0), dict(NB=0)):
        assert call(**kw) == INVALID, kw
    for name in names[:9]:
        assert call(**{name: None}) == NULL, name
    for kw in (dict(S=pkv.PKV_MAX_RESIZE_SEQS + 1), dict(T=2 ** 30), dict(cap=2 ** 30)):
        assert call(**kw) == UNSUPPORTED, kw
    for name in names[:8]:
        assert call(**{name: FAKE + 2}) == ALIGN, name
    assert call(slots=FAKE + 4) == ALIGN and call(pos=FAKE + 4) == ALIGN


def test_verify(lib):
    names = ["path", "depth", "plen", "next", "tok", "par", "qs", "tp", "ts", "dp", "ds", "au", "su",
             "S", "T", "V"]

    def call(**kw):
        a = dict.fromkeys(names, FAKE)
        a.update(depth=4, ts=100, ds=100, S=2, T=9, V=100)
        a.update(kw)
        return lib.pkv_tree_verify(*[a[n] for n in names], None)

    assert call(S=0) == OK
    for kw in (dict(S=-1), dict(T=-1), dict(V=0), dict(depth=0), dict(ts=99), dict(ds=99)):
        assert call(**kw) == INVALID, kw
    for name in ("path", "plen", "next", "tok", "par", "qs", "tp", "au", "su"):
        assert call(**{name: None}) == NULL, name
    assert call(depth=257) == UNSUPPORTED
    assert call(V=2 ** 30 + 1, ts=2 ** 31, ds=2 ** 31) == UNSUPPORTED
    for name in ("path", "plen", "next", "tok", "par", "qs", "tp", "dp", "au", "su"):
        assert call(**{name: FAKE + 2}) == ALIGN, name


def test_the_binding_refuses_what_does_not_fit(lib):
    torch = pytest.importorskip("torch")
    i32 = torch.zeros(2, dtype=torch.int32)
    h = torch.zeros(2, 4, 64, dtype=torch.float16)
    f = torch.zeros(2, 8)
    with pytest.raises(ValueError):  # host tensors
        pkv.pkv_resize_sequences(i32.view(2, 1), i32, i32, i32, i32, i32[:1], i32[:1], i32,
                                 i32.long(), None, 16, 4)
    with pytest.raises(ValueError):
        pkv.pkv_tree_verify(i32.view(2, 1), i32, i32, i32, i32, i32, f, None, f[:, 0], f[:, 0])
    with pytest.raises(ValueError):
        pkv.pkv_decode_attention_scored(h, h, h, h, i32.view(2, 1), i32, 1.0, 4, 4, 64, 16, 16, 1)
    with pytest.raises(ValueError):
        pkv.pkv_chunk_attention_scored(h, h, h, h, i32.view(2, 1), i32, i32, 1.0, 4, 4, 64, 16, 1,
                                       16, 1)
    # elements of a row apart, rows on top of each other
    for bad in (torch.zeros(4, 16)[:, ::2], torch.zeros(16).as_strided((4, 8), (2, 1))):
        with pytest.raises(ValueError):
            pkv._prob_rows(bad, "target_probs", 4, 8, -1)
    assert pkv._prob_rows(torch.zeros(4, 16)[:, :8], "target_probs", 4, 8, -1)[1] == 16
