"""Refusals of the speculative step's entry points: on the host, before any CUDA call."""

import ctypes

import pytest

import paged_kv_cache_131_gb300 as pkv
from paged_kv_cache_131_gb300 import _build

FAKE = 0x100000  # 32-byte aligned, never dereferenced: every call below fails validation
OK, NULL, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_rope_write(lib, fp8):
    def call(nr=None, **kw):
        n = dict(qw=FAKE, kw=FAKE, eps=1e-6, table=FAKE, max_pos=100, rot=64, inter=0)
        n.update(nr or {})
        a = dict(q_out=FAKE, q=FAKE, k=FAKE, v=FAKE, qs=768, ks=768, vs=768, pos=FAKE, slots=FAKE,
                 T=4, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, H=8, Hk=2, D=64, bs=16, NB=4)
        a.update(kw)
        rec = pkv.pkv_norm_rope(*n.values())
        args = [a[x] for x in ("q_out", "q", "k", "v", "qs", "ks", "vs")] + [ctypes.byref(rec)]
        args += [a[x] for x in ("pos", "slots", "T", "kc", "vc")]
        if fp8:
            args += [a["ksc"], a["vsc"]]
        args += [a[x] for x in ("H", "Hk", "D", "bs", "NB")]
        return (lib.pkv_norm_rope_write_fp8 if fp8 else lib.pkv_norm_rope_write)(*args, None)

    assert call(T=0) == OK
    assert call(T=-1) == INVALID
    for name in ("q_out", "q", "k", "v", "pos", "slots", "kc", "vc") + (("ksc", "vsc") if fp8 else ()):
        assert call(**{name: None}) == NULL, name
    assert call(nr=dict(table=None)) == NULL
    for kw in (dict(H=0), dict(Hk=0), dict(bs=0), dict(NB=0), dict(qs=-8), dict(D=0)):
        assert call(**kw) == INVALID, kw
    for nr in (dict(rot=-16), dict(rot=80), dict(eps=-1.0), dict(eps=float("nan")),
               dict(max_pos=0)):
        assert call(nr=nr) == INVALID, nr
    assert call(q_out=FAKE, q=FAKE, qs=768) == INVALID  # in place, but not packed
    other = dict(q_out=FAKE + 4096)
    assert call(**other, D=96) == UNSUPPORTED
    assert call(nr=dict(rot=24), **other) == UNSUPPORTED
    for kw in (dict(q=FAKE + 8), dict(ks=772), dict(slots=FAKE + 4), dict(kc=FAKE + 8),
               dict(pos=FAKE + 4)):
        assert call(**other, **kw) == ALIGN, kw
    assert call(nr=dict(table=FAKE + 8), **other) == ALIGN


def test_cache_read(lib):
    def call(k=FAKE, v=FAKE, slots=FAKE, T=4, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, Hk=2, D=64,
             bs=16, NB=4):
        return lib.pkv_cache_read_fp8(k, v, slots, T, kc, vc, ks, vs, Hk, D, bs, NB, None)

    assert call(T=0) == OK
    assert call(T=-1) == INVALID
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert call(**{name: None}) == NULL, name
    for kw in (dict(Hk=0), dict(bs=0), dict(NB=0), dict(D=-64)):
        assert call(**kw) == INVALID
    assert call(D=32) == UNSUPPORTED
    for kw in (dict(k=FAKE + 16), dict(kc=FAKE + 8), dict(slots=FAKE + 4), dict(ks=FAKE + 2)):
        assert call(**kw) == ALIGN


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention(lib, fp8):
    def call(**kw):
        a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, sl=FAKE, qs=FAKE,
                 mask=FAKE, words=1, scale=0.1, H=32, Hk=8, D=128, bs=16, S=4, MB=8, Tq=10,
                 maxq=7, maxL=100, NB=64, ws=None, wsb=0)
        a.update(kw)
        names = ["out", "q", "k", "v"] + (["ks", "vs"] if fp8 else []) + list(a)[6:]
        fn = lib.pkv_tree_attention_fp8 if fp8 else lib.pkv_tree_attention
        return fn(*[a[n] for n in names], None)

    assert call(S=0) == OK and call(Tq=0) == OK
    assert call(S=-1) == INVALID and call(Tq=-1) == INVALID
    for name in ("out", "q", "k", "v", "bt", "sl", "qs", "mask") + (("ks", "vs") if fp8 else ()):
        assert call(**{name: None}) == NULL, name
    for kw in (dict(H=30), dict(maxq=0), dict(maxL=0), dict(MB=0), dict(NB=0), dict(words=0),
               dict(maxq=65), dict(scale=float("inf")), dict(Hk=0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(H=24), dict(H=128), dict(D=96), dict(bs=32), dict(S=70000),
               dict(maxq=257, words=5)):
        assert call(**kw) == UNSUPPORTED, kw
    # sequences whose last positions do not fit 32 bits; either bound may be large alone
    big = (2 ** 31 - 1) // 16
    assert call(MB=big, maxL=2 ** 31 - 1) == UNSUPPORTED
    assert call(MB=big) == WORKSPACE and call(maxL=2 ** 31 - 1) == WORKSPACE
    for kw in (dict(q=FAKE + 8), dict(qs=FAKE + 2), dict(mask=FAKE + 4), dict(ws=FAKE + 8)):
        assert call(**kw) == ALIGN, kw
    need = lib.pkv_tree_workspace_bytes(4, 32, 8, 128, 10, 7, 100)
    assert need > 0 and call() == WORKSPACE and call(ws=FAKE, wsb=need - 1) == WORKSPACE
    assert lib.pkv_tree_workspace_bytes(4, 30, 8, 128, 10, 7, 100) == 0


def test_tree_accept(lib):
    def call(view=(0, 0, 1024, 64, 0), cache=FAKE, n=1, layers=1, path=FAKE, depth=4, ctx=FAKE,
             bt=FAKE, S=2, MB=4, bs=16, NB=8):
        arr = (pkv.pkv_cache_desc * 33)()
        arr[0] = pkv.pkv_cache_desc(cache, pkv.pkv_view(*view))
        return lib.pkv_tree_accept(arr, n, layers, path, depth, ctx, bt, S, MB, bs, NB, None)

    for kw in (dict(n=0), dict(layers=0), dict(S=0), dict(depth=0)):
        assert call(**kw) == OK
    for kw in (dict(n=-1), dict(layers=-1), dict(S=-1), dict(depth=-1), dict(bs=0), dict(NB=0),
               dict(MB=0), dict(view=(0, 0, 1024, 0, 0)), dict(view=(0, 0, 0, 64, 0)),
               dict(view=(-1, 0, 1024, 64, 0)), dict(layers=2)):
        assert call(**kw) == INVALID, kw
    for name in ("cache", "path", "ctx", "bt"):
        assert call(**{name: None}) == NULL, name
    assert call(n=33) == UNSUPPORTED and call(depth=257) == UNSUPPORTED
    assert call(path=FAKE + 2) == ALIGN


def test_tree_accept_refuses_a_layer_named_twice(lib):
    def call(*descs, layers=1, path=FAKE):
        arr = (pkv.pkv_cache_desc * len(descs))()
        for i, (cache, view) in enumerate(descs):
            arr[i] = pkv.pkv_cache_desc(cache, pkv.pkv_view(*view))
        return lib.pkv_tree_accept(arr, len(descs), layers, path, 4, FAKE, FAKE, 2, 4, 16, 8, None)

    a = (FAKE, (0, 8192, 1024, 64, 0))
    assert call(a, a) == INVALID
    assert call(a, (FAKE, (512, 8192, 1024, 32, 0)), a) == INVALID
    # the same layer by another offset, or inside the other's run of layers
    assert call(a, (FAKE - 8192, (0, 8192, 1024, 64, 1))) == INVALID
    assert call(a, (FAKE, (0, 8192, 1024, 64, 3)), layers=4) == INVALID
    assert call((FAKE, (0, 8192, 1024, 64, 3)), a, layers=4) == INVALID
    # neighbours are fine (the last descriptor's rows are too wide for a launch)
    wide = (FAKE + (1 << 40) + 1, (0, 1 << 40, 1 << 34, 1 << 30, 0))
    assert call(a, (FAKE, (0, 8192, 1024, 64, 1)), wide) == UNSUPPORTED
    assert call(a, (FAKE, (0, 8192, 1024, 64, 4)), (FAKE, (512, 8192, 1024, 64, 2)), wide,
                layers=4) == UNSUPPORTED


def test_the_binding_refuses_what_does_not_fit(lib):
    torch = pytest.importorskip("torch")
    i64 = torch.zeros(4, dtype=torch.int64)
    h = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):  # host tensors
        pkv.pkv_norm_rope_write(h, h, h, h, i64, i64, h, h, num_blocks=1)
    with pytest.raises(ValueError):
        pkv.pkv_cache_read_fp8(h, None, i64, h, None, h, None, 16, 1)
    with pytest.raises(ValueError):
        pkv.pkv_tree_accept([], 1, i64.view(2, 2).int(), i64.int(), i64.view(2, 2).int(), 16, 1)
    with pytest.raises(ValueError):  # heads of a token apart
        pkv._token_rows(torch.zeros(4, 2, 128, dtype=torch.float16)[..., ::2], "q", torch.float16,
                        (4, 2, 64), -1)
