"""GPU parity of the norm + rotation + cache write, the FP8 read-back and the
path acceptance against their float64 definitions."""

import numpy as np
import pytest

from oracle import speculative as spec

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu
BS = 16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    assert torch.cuda.is_available()
    pkv.pkv_get_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def table(n, rot):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    ang = np.arange(n)[:, None] * inv[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


class Case:
    def __init__(self, seed, T, H, Hk, D, rot, norm=True, scale=2.0, max_pos=500, spare=5):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.Hk, self.D, self.rot = T, H, Hk, D, rot
        self.NB = T // BS + spare
        self.qkv = (rng.standard_normal((T, (H + 2 * Hk) * D)) * scale).astype(np.float16)
        self.q, self.k, self.v = (x.reshape(T, -1, D) for x in
                                  np.split(self.qkv, [H * D, (H + Hk) * D], axis=1))
        self.slots = rng.permutation(self.NB * BS)[:T].astype(np.int64)
        self.pos = rng.integers(0, max_pos, T)
        if T:
            self.pos[-1] = max_pos - 1
        self.table = table(max_pos, rot) if rot else None
        self.qw, self.kw = ((1 + 0.3 * rng.standard_normal(D)).astype(np.float16) if norm else None
                            for _ in range(2))
        d = self.d_qkv = dev(self.qkv)
        self.d = dict(q=d[:, :H * D].view(T, H, D), k=d[:, H * D:(H + Hk) * D].view(T, Hk, D),
                      v=d[:, (H + Hk) * D:].view(T, Hk, D))

    def run(self, fp8, interleaved, stream=None, q_out=None, out=None):
        T, H, Hk, D, NB = self.T, self.H, self.Hk, self.D, self.NB
        q_out = torch.full((T, H, D), 7.0, dtype=torch.float16, device="cuda") if q_out is None \
            else q_out
        if fp8:
            c = [torch.full((NB, BS, Hk, D), 0x5A, dtype=torch.uint8, device="cuda")
                 for _ in range(2)]
            c += [torch.full((NB, BS, Hk), 9.0, device="cuda") for _ in range(2)]
            fn = pkv.pkv_norm_rope_write_fp8
        else:
            c = [torch.full((NB, BS, Hk, D), 7.0, dtype=torch.float16, device="cuda")
                 for _ in range(2)]
            fn = pkv.pkv_norm_rope_write
        fn(q_out, self.d["q"], self.d["k"], self.d["v"], dev(self.pos), dev(self.slots), *c,
           None if self.table is None else dev(self.table),
           None if self.qw is None else dev(self.qw), None if self.kw is None else dev(self.kw),
           eps=EPS, interleaved=interleaved, block_size=BS, num_blocks=NB, stream=stream)
        return q_out, c

    def want(self, interleaved):
        q, qm = spec.norm_rope(self.q, self.qw, EPS, self.table, self.pos, interleaved)
        k, km = spec.norm_rope(self.k, self.kw, EPS, self.table, self.pos, interleaved)
        return (q, qm), (k, km), (np.asarray(self.v, np.float64), None)


def fp32_error(mag):
    # fp32: the mean of 128 squares by 8 fma per lane and 4 adds (12 roundings,
    # halved by the square root), rsqrt (2 steps), two products: < 16 half steps;
    # the rotation's two products and one sum: 3 more -- of |a c| + |b s|
    return 20 * 2.0 ** -24 * mag


def check16(got, ref, mag, what):
    got = got.astype(np.float64)
    tol = np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + fp32_error(mag) * (1 + 2.0 ** -10)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(got - ref).max():.3e}"


E4M3 = None


def check8(codes, scale, ref, mag, what):
    """Codes within half a step of y / s (plus the fp32 error of y and s)."""
    global E4M3
    E4M3 = spec.e4m3_table() if E4M3 is None else E4M3
    amax = np.abs(ref).max(-1)
    err = fp32_error(mag).max(-1) if mag is not None else np.zeros_like(amax)
    s = scale.astype(np.float64)
    assert (np.abs(s - amax / 448) <= err / 448 + 2.0 ** -24 * amax / 448 + 1e-44).all(), what
    got = E4M3[codes] * s[..., None]
    # half a step: 2^-4 relative, 2^-10 s below the normal range
    tol = np.abs(ref) * 2.0 ** -4 + s[..., None] * 2.0 ** -10 + 2 * err[..., None] + amax[..., None] * 2.0 ** -21
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}"


CASES = [
    # seed, T, H, Hk, D, rot, norm
    (1, 1, 4, 2, 64, 64, True),
    (2, 1, 32, 8, 128, 128, True),
    (3, 37, 8, 1, 128, 112, True),    # pairs 56 apart
    (4, 64, 1, 1, 64, 16, False),     # fewer rows than a warp's job
    (5, 131, 16, 16, 64, 32, True),
    (6, 700, 32, 8, 128, 64, True),
    (7, 50, 8, 4, 128, 0, True),      # norm alone
    (8, 50, 8, 4, 128, 0, False),     # a plain write with the queries copied
    (9, 2047, 2, 1, 64, 48, False),
    (10, 30, 7, 3, 128, 128, True),   # rows that leave chunks part empty
    (11, 9000, 6, 2, 64, 64, True),   # jobs of several chunks
]


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=[str(c[0]) for c in CASES])
def test_norm_rope_write(case, fp8, interleaved):
    c = Case(*case)
    q_out, caches = c.run(fp8, interleaved)
    (q, qm), (k, km), (v, _) = c.want(interleaved)
    check16(q_out.cpu().numpy(), q, qm, "q")
    rest = np.ones(c.NB * BS, bool)
    rest[c.slots] = False
    for i, (ref, mag, name) in enumerate(((k, km, "k"), (v, None, "v"))):
        rows = caches[i].cpu().numpy().reshape(c.NB * BS, c.Hk, c.D)
        if fp8:
            sc = caches[2 + i].cpu().numpy().reshape(c.NB * BS, c.Hk)
            check8(rows[c.slots], sc[c.slots], ref, mag, name)
            assert (rows[rest] == 0x5A).all() and (sc[rest] == 9.0).all()
        elif name == "v" or (c.qw is None and not c.rot):
            assert np.array_equal(rows[c.slots].view(np.uint16),
                                  (c.k if name == "k" else c.v).view(np.uint16))
        else:
            check16(rows[c.slots], ref, mag, name)
        if not fp8:
            assert (rows[rest] == 7.0).all()
    assert pkv.pkv_get_device_error() == (0, -1)


def test_values_quantise_as_the_plain_write_does():
    c = Case(21, 77, 8, 4, 128, 64)
    _, caches = c.run(True, False)
    ref = [torch.full_like(x, 0x5A if x.dtype == torch.uint8 else 9.0) for x in caches]
    v = c.d["v"].contiguous()
    pkv.pkv_cache_write_fp8(v, v, dev(c.slots), *ref, BS, c.NB)
    assert torch.equal(caches[1], ref[1]) and torch.equal(caches[3], ref[3])


def test_values_of_every_magnitude_quantise_as_the_plain_write_does():
    # the correctly rounded quotient, from fp16's smallest numbers to its largest
    rng = np.random.default_rng(27)
    c = Case(27, 3000, 1, 4, 128, 0, norm=False)
    v = c.d["v"]
    v.copy_(dev((rng.standard_normal(v.shape) * 10.0 ** rng.uniform(-8, 4.6, v.shape[:2] + (1,)))
                .clip(-65504, 65504).astype(np.float16)))
    v[0, 0], v[1, 1] = 0, 2.0 ** -24
    _, caches = c.run(True, False)
    ref = [torch.full_like(x, 0x5A if x.dtype == torch.uint8 else 9.0) for x in caches]
    w = v.contiguous()
    pkv.pkv_cache_write_fp8(w, w, dev(c.slots), *ref, BS, c.NB)
    assert torch.equal(caches[1], ref[1]) and torch.equal(caches[3], ref[3])


def test_tokens_apart():
    # every other token of a wider tensor, and rows of a token reversed in time
    c = Case(28, 40, 8, 2, 64, 64)
    ref, caches = c.run(False, False)
    for n in c.d:
        wide = torch.full((80,) + tuple(c.d[n].shape[1:]), float("nan"), dtype=torch.float16,
                          device="cuda")
        wide[::2] = c.d[n]
        c.d[n] = wide[::2]
    got, again = c.run(False, False)
    assert torch.equal(got, ref) and all(torch.equal(a, b) for a, b in zip(caches, again))


@pytest.mark.parametrize("fp8", [False, True])
def test_padding_and_bad_tokens_are_left_alone(fp8):
    c = Case(22, 20, 8, 2, 64, 64)
    whole_q, whole = c.run(fp8, False)
    slots, pos = c.slots.copy(), c.pos.copy()
    c.slots[3], c.slots[19] = -1, -5
    pos[3] = -99  # of a padding token: not looked at
    c.pos = pos
    q_out, caches = c.run(fp8, False)
    assert pkv.pkv_get_device_error() == (0, -1)
    c.slots[7] = c.NB * BS
    q2, _ = c.run(fp8, False)
    assert pkv.pkv_get_device_error() == (1, 7)
    assert (q2[7] == 7.0).all()
    c.slots[7] = slots[7]
    for bad in (-1, c.table.shape[0], 1 << 40):
        c.pos[11] = bad
        q3, got = c.run(fp8, False)
        assert pkv.pkv_get_device_error() == (5, 11)
        assert (q3[11] == 7.0).all()
    live = [t for t in range(20) if t not in (3, 19)]
    assert torch.equal(q_out[live], whole_q[live]) and (q_out[[3, 19]] == 7.0).all()
    rows = caches[0].flatten(0, 1)
    assert torch.equal(rows[dev(slots[live])], whole[0].flatten(0, 1)[dev(slots[live])])
    assert (rows[dev(slots[[3, 19]])] == (0x5A if fp8 else 7.0)).all()


def test_in_place_queries_and_separate_inputs():
    c = Case(23, 33, 8, 4, 128, 128)
    ref, _ = c.run(False, False)
    for n in c.d:
        c.d[n] = c.d[n].contiguous()
    got, _ = c.run(False, False, q_out=c.d["q"])
    assert torch.equal(got, ref)


def test_one_weight_alone():
    c = Case(24, 9, 4, 2, 64, 32)
    c.kw = None
    q_out, caches = c.run(False, True)
    (q, qm), (k, km), _ = c.want(True)
    check16(q_out.cpu().numpy(), q, qm, "q")
    check16(caches[0].cpu().numpy().reshape(-1, c.Hk, c.D)[c.slots], k, km, "k")


def test_zero_and_non_finite_rows():
    c = Case(25, 6, 4, 2, 64, 64)
    c.d["k"][1] = 0
    c.d["q"][2, 1] = 0
    c.d["v"][3, 0, 5] = float("nan")
    c.d["q"][4, 0, 7] = float("inf")
    q_out, caches = c.run(True, False)
    at = c.slots
    assert (caches[0].flatten(0, 1)[at[1]] == 0).all() and (caches[2].flatten(0, 1)[at[1]] == 0).all()
    assert (q_out[2, 1] == 0).all()
    v = caches[1].flatten(0, 1)[at[3], 0]
    assert (v[5] & 0x7F) == 0x7F and ((v[:5] & 0x7F) != 0x7F).all()
    assert torch.isnan(q_out[4, 0, 7]) and torch.isfinite(q_out[4, 1:]).all()


def test_a_slot_past_32_bits_of_bytes():
    # the last block of a 4.3 GB cache: row offsets above 2^32
    T, Hk, D = 3, 8, 128
    NB = (1 << 32) // (BS * Hk * D * 2) + 9
    c = Case(26, T, 8, Hk, D, 128)
    c.NB = NB
    c.slots = np.array([NB * BS - 1, 5, NB * BS - 40])
    q_out, caches = c.run(False, False)
    _, (k, km), _ = c.want(False)
    got = caches[0].flatten(0, 1)[dev(c.slots)].cpu().numpy()
    check16(got, k, km, "k")
    assert pkv.pkv_get_device_error() == (0, -1)


# ---------------------------------------------------------------- read-back


@pytest.mark.parametrize("T,Hk,D", [(1, 1, 64), (5, 8, 128), (333, 3, 64), (2050, 8, 128),
                                    (40, 1, 128)])
def test_cache_read_fp8(T, Hk, D):
    rng = np.random.default_rng(T)
    NB = T // BS + 3
    codes = [rng.integers(0, 256, (NB, BS, Hk, D)).astype(np.uint8) for _ in range(2)]
    scale = [(10.0 ** rng.uniform(-6, 2, (NB, BS, Hk))).astype(np.float32) for _ in range(2)]
    slots = rng.integers(0, NB * BS, T)  # with repetitions
    slots[T // 2] = -1
    if T > 4:
        slots[4] = NB * BS
    out = [torch.full((T, Hk, D), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    pkv.pkv_cache_read_fp8(out[0], out[1], dev(slots), dev(codes[0]), dev(codes[1]), dev(scale[0]),
                           dev(scale[1]), BS, NB)
    assert pkv.pkv_get_device_error() == ((1, 4) if T > 4 else (0, -1))
    live = (slots >= 0) & (slots < NB * BS)
    tab = spec.e4m3_table().astype(np.float32)
    for i in range(2):
        got = out[i].cpu().numpy()
        with np.errstate(over="ignore"):
            want = (tab[codes[i].reshape(-1, Hk, D)[slots[live]]] *
                    scale[i].reshape(-1, Hk)[slots[live]][..., None]).astype(np.float16)
        assert np.array_equal(got[live], want, equal_nan=True)
        assert (got[~live] == 7.0).all()


def test_cache_read_of_more_units_than_32_bits_count():
    # 2^31 16-code units and more (69 GB of rows), nearly all of them padding
    T, Hk, D = 4098, 65536, 128
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB")
    codes = torch.randint(0, 127, (1, BS, Hk, D), device="cuda", dtype=torch.uint8)
    scale = torch.rand(1, BS, Hk, device="cuda")
    slots = torch.full((T,), -1, device="cuda", dtype=torch.int64)
    slots[3], slots[T - 1], slots[T - 2] = 2, 5, 11
    rows = torch.empty(T, Hk, D, dtype=torch.float16, device="cuda")
    rows[T - 3] = 7.0
    pkv.pkv_cache_read_fp8(rows, None, slots, codes, None, scale, None, BS, 1)
    for t in (3, T - 1, T - 2):
        want = codes[0, slots[t]].view(torch.float8_e4m3fn).float() * scale[0, slots[t]][:, None]
        assert torch.equal(rows[t], want.half())
    assert (rows[T - 3] == 7.0).all()
    del rows
    torch.cuda.empty_cache()


def test_cache_read_keys_alone_and_round_trip():
    T, Hk, D = 100, 4, 128
    x = torch.randn(T, Hk, D, device="cuda").half()
    NB = 9
    slots = torch.randperm(NB * BS, device="cuda")[:T]
    k, v = (torch.zeros(NB, BS, Hk, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(NB, BS, Hk, device="cuda") for _ in range(2))
    pkv.pkv_cache_write_fp8(x, x, slots, k, v, ks, vs, BS, NB)
    got = torch.zeros_like(x)
    pkv.pkv_cache_read_fp8(got, None, slots, k, None, ks, None, BS, NB)
    amax = x.float().abs().amax(-1, keepdim=True)
    tol = x.float().abs() * (2 ** -4 + 2 ** -10) + amax / 448 * 2 ** -10
    assert ((got.float() - x.float()).abs() <= tol).all()


# ------------------------------------------------------------- accepted paths


def _accept_case(seed, S, depth, nodes, bs, NB, MB):
    rng = np.random.default_rng(seed)
    tables = rng.permutation(NB)[:S * MB].reshape(S, MB).astype(np.int32)
    ctx = rng.integers(0, MB * bs - nodes + 1, S).astype(np.int32)
    path = np.full((S, depth), -1, np.int32)
    for i in range(S):
        n = int(rng.integers(0, min(depth, nodes) + 1))
        path[i, :n] = np.sort(rng.choice(nodes, n, replace=False))
    return rng, tables, ctx, path


@pytest.mark.parametrize("seed,S,depth,nodes,bs,width,layers", [
    (1, 1, 1, 1, 16, 2048, 1), (2, 5, 6, 20, 16, 2048, 3), (3, 9, 20, 40, 16, 656, 2),
    (4, 3, 17, 17, 64, 132, 2), (5, 2, 8, 33, 16, 6, 1), (6, 2, 8, 30, 16, 7, 2),
    (7, 1, 256, 256, 16, 4096, 1), (8, 64, 4, 8, 16, 32, 4), (9, 2, 9, 12, 5, 5000, 1),
])
def test_tree_accept(seed, S, depth, nodes, bs, width, layers):
    MB = -(-nodes // bs) + 2
    NB = S * MB + 3
    rng, tables, ctx, path = _accept_case(seed, S, depth, nodes, bs, NB, MB)
    # a layer-outer cache and a block-outer one whose rows are half as wide
    w2 = max(1, width // 2)
    a = rng.integers(0, 256, (layers + 1, NB * bs, width)).astype(np.uint8)
    b = rng.integers(0, 256, (NB, layers, bs, w2)).astype(np.uint8)
    da, db = dev(a), dev(b)
    views = [(da, pkv.pkv_view(0, NB * bs * width, bs * width, width, 1)),
             (db, pkv.pkv_view(0, bs * w2, layers * bs * w2, w2, 0))]
    pkv.pkv_tree_accept(views, layers, dev(path), dev(ctx), dev(tables), bs, NB)
    assert pkv.pkv_get_device_error() == (0, -1)
    for layer in range(layers):
        a[layer + 1] = spec.tree_accept(a[layer + 1], path, ctx, tables, bs)
        rows = np.ascontiguousarray(b[:, layer]).reshape(NB * bs, w2)
        b[:, layer] = spec.tree_accept(rows, path, ctx, tables, bs).reshape(NB, bs, w2)
    assert np.array_equal(da.cpu().numpy(), a) and np.array_equal(db.cpu().numpy(), b)


def test_bad_paths_leave_their_sequence_alone():
    S, MB, NB, bs, W = 6, 3, 20, 16, 64
    rng, tables, ctx, _ = _accept_case(11, S, 3, 4, bs, NB, MB)
    ctx[:] = 10
    good = np.array([[0, 2, 3]] * S, np.int32)
    rows = rng.integers(0, 256, (NB * bs, W)).astype(np.uint8)
    view = pkv.pkv_view(0, 0, bs * W, W, 0)

    def run(path, ctx, tables):
        d = dev(rows)
        pkv.pkv_tree_accept([(d, view)], 1, dev(path), dev(ctx), dev(tables), bs, NB)
        return d.cpu().numpy(), pkv.pkv_get_device_error()

    def check(kind, path=None, ctx_=None, tables_=None):
        got, err = run(good if path is None else path, ctx if ctx_ is None else ctx_,
                       tables if tables_ is None else tables_)
        assert err == (kind, 4)
        keep = np.arange(S) != 4
        want = spec.tree_accept(rows, np.where(keep[:, None], good, -1), ctx, tables, bs)
        assert np.array_equal(got, want)

    p = good.copy()
    p[4] = [0, 3, 3]
    check(6, path=p)
    p[4] = [2, 1, 3]
    check(6, path=p)
    p[4] = [0, 2, MB * bs]
    check(6, path=p)
    p[4] = [0, 2, 2 ** 31 - 1]
    check(6, path=p)
    c = ctx.copy()
    c[4] = -1
    check(6, ctx_=c)
    c[4] = MB * bs - 2
    check(6, ctx_=c)
    t = tables.copy()
    t[4, 0] = NB
    check(2, tables_=t)
    t[4, 0] = -3
    check(2, tables_=t)
