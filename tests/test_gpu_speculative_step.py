"""The speculative step's operators together, as a serving loop runs them: the
drafted tokens' rows normed, rotated and written, the tree verified, a path
accepted, and the next decode over the rows that moved -- eagerly and as a
replayed CUDA graph."""

import numpy as np
import pytest

from oracle import speculative as spec

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu
BS, H, Hk, D, ROT = 16, 8, 2, 128, 128
S, NODES, DEPTH, MB, MAXPOS = 3, 11, 4, 9, 400


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rope_table():
    inv = 10000.0 ** (-np.arange(0, ROT, 2) / ROT)
    ang = np.arange(MAXPOS)[:, None] * inv[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


class Step:
    """Device buffers of one step; ``fill`` brings in a step's inputs."""

    def __init__(self, fp8):
        self.fp8 = fp8
        self.NB = S * MB + 2
        rng = np.random.default_rng(5)
        self.tables = rng.permutation(self.NB)[:S * MB].reshape(S, MB).astype(np.int32)
        self.rope = rope_table()
        self.qw, self.kw = ((1 + 0.2 * rng.standard_normal(D)).astype(np.float16) for _ in range(2))
        T = S * NODES
        z = lambda *s, t=torch.float16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        kind = torch.uint8 if fp8 else torch.float16
        self.caches = [z(self.NB, BS, Hk, D, t=kind) for _ in range(2)]
        self.scales = [z(self.NB, BS, Hk, t=torch.float32) for _ in range(2)] if fp8 else []
        self.qkv = z(T, (H + 2 * Hk) * D)
        self.q_out, self.out = z(T, H, D), z(T, H, D)
        self.dq, self.dout = z(S, H, D), z(S, H, D)
        self.pos, self.slots = z(T, t=torch.int64), z(T, t=torch.int64)
        self.mask = z(T, 1, t=torch.int64)
        self.lens, self.ctx, self.dlens = (z(S, t=torch.int32) for _ in range(3))
        self.path = z(S, DEPTH, t=torch.int32)
        self.qs = torch.arange(0, T + 1, NODES, dtype=torch.int32, device="cuda")
        self.d_tables, self.d_rope = dev(self.tables), dev(self.rope)
        self.d_qw, self.d_kw = dev(self.qw), dev(self.kw)
        self.ws = torch.full((pkv.pkv_tree_workspace_bytes(S, H, Hk, D, T, NODES, MB * BS),), 0xEE,
                             dtype=torch.uint8, device="cuda")
        self.dws = z(pkv.pkv_decode_workspace_bytes(S, H, Hk, D, MB * BS), t=torch.uint8)

    def fill(self, ctx, seed):
        rng = np.random.default_rng(seed)
        T = S * NODES
        trees = [spec.random_tree(rng, NODES) for _ in range(S)]
        depth = np.concatenate([t.sum(1) - 1 for t in trees])
        at = np.repeat(ctx, NODES) + np.tile(np.arange(NODES), S)
        seq = np.repeat(np.arange(S), NODES)
        path = np.full((S, DEPTH), -1, np.int32)
        for i, t in enumerate(trees):
            p = np.flatnonzero(t[int(rng.integers(0, NODES))])[:DEPTH]
            path[i, :len(p)] = p
        host = dict(qkv=rng.standard_normal((T, (H + 2 * Hk) * D)).astype(np.float16),
                    pos=(np.repeat(ctx, NODES) + depth).astype(np.int64),
                    slots=(self.tables[seq, at // BS].astype(np.int64) * BS + at % BS),
                    mask=spec.mask_words(np.concatenate(trees)),
                    lens=(ctx + NODES).astype(np.int32), ctx=ctx.astype(np.int32), path=path,
                    dlens=(ctx + (path >= 0).sum(1)).astype(np.int32),
                    dq=rng.standard_normal((S, H, D)).astype(np.float16))
        for n, a in host.items():
            getattr(self, n).copy_(torch.from_numpy(a))
        self.trees = np.concatenate(trees)
        return host

    def enqueue(self):
        q = self.qkv[:, :H * D].view(-1, H, D)
        k = self.qkv[:, H * D:(H + Hk) * D].view(-1, Hk, D)
        v = self.qkv[:, (H + Hk) * D:].view(-1, Hk, D)
        kw = dict(q_weight=self.d_qw, k_weight=self.d_kw, block_size=BS, num_blocks=self.NB)
        write = pkv.pkv_norm_rope_write_fp8 if self.fp8 else pkv.pkv_norm_rope_write
        write(self.q_out, q, k, v, self.pos, self.slots, *self.caches, *self.scales, self.d_rope,
              **kw)
        tree = pkv.pkv_tree_attention_fp8 if self.fp8 else pkv.pkv_tree_attention
        tree(self.out, self.q_out, *self.caches, *self.scales, self.d_tables, self.lens, self.qs,
             self.mask, D ** -0.5, H, Hk, D, BS, NODES, MB * BS, self.NB, self.ws)
        rows = [(c, c.element_size() * Hk * D) for c in self.caches] + \
            [(c, 4 * Hk) for c in self.scales]
        pkv.pkv_tree_accept([(c, pkv.pkv_view(0, 0, BS * w, w, 0)) for c, w in rows], 1, self.path,
                            self.ctx, self.d_tables, BS, self.NB)
        args = (self.d_tables, self.dlens, D ** -0.5, H, Hk, D, BS, MB * BS, self.NB, self.dws)
        if self.fp8:
            pkv.pkv_decode_attention_fp8(self.dout, self.dq, *self.caches, *self.scales, *args)
        else:
            pkv.pkv_decode_attention(self.dout, self.dq, *self.caches, *args)

    def values(self):
        """The caches' values on the host."""
        if not self.fp8:
            return [c.cpu().numpy().astype(np.float64) for c in self.caches]
        t = spec.e4m3_table()
        return [t[c.cpu().numpy()] * s.cpu().numpy().astype(np.float64)[..., None]
                for c, s in zip(self.caches, self.scales)]

    def check(self, host, before):
        """This step's outputs against the definitions, from the caches before it."""
        T = S * NODES
        q, qm = spec.norm_rope(host["qkv"][:, :H * D].reshape(T, H, D), self.qw, 1e-6, self.rope,
                               host["pos"], False)
        k, _ = spec.norm_rope(host["qkv"][:, H * D:(H + Hk) * D].reshape(T, Hk, D), self.kw, 1e-6,
                              self.rope, host["pos"], False)
        v = host["qkv"][:, (H + Hk) * D:].reshape(T, Hk, D).astype(np.float64)
        q_out = self.q_out.cpu().numpy().astype(np.float64)
        assert (np.abs(q_out - q) <= np.abs(q) * 2.0 ** -11 + 20 * 2.0 ** -24 * qm * 1.01 + 2.0 ** -25).all()
        drafted = []
        for x, c in ((k, before[0]), (v, before[1])):
            c = c.copy().reshape(-1, Hk, D)
            if self.fp8:  # the codes nearest the values
                from oracle import quantize_row
                t = spec.e4m3_table()
                for i, s in enumerate(host["slots"]):
                    for h in range(Hk):
                        codes, sc = quantize_row(x[i, h].astype(np.float16))
                        c[s, h] = t[codes] * float(sc)
            else:
                c[host["slots"]] = x.astype(np.float16)
            drafted.append(c)
        # the rows as drafted, then moved (keys may sit one rounding away)
        now = self.values()
        step = 2.0 ** -4 if self.fp8 else 2.0 ** -11
        for c, n in zip(drafted, now):
            want = spec.tree_accept(c, host["path"], host["ctx"], self.tables, BS)
            amax = np.abs(want).max(-1, keepdims=True)
            assert (np.abs(n.reshape(want.shape) - want) <= 2.1 * step * np.abs(want) +
                    amax * 2.0 ** (-17 if self.fp8 else -20)).all()
        # the decode that follows reads the moved rows
        full = np.ones((S, 1), bool)
        ref, t = spec.tree_attention(host["dq"], now[0], now[1], self.tables, host["dlens"],
                                     np.arange(S + 1), full, D ** -0.5, Hk)
        got = self.dout.cpu().numpy().astype(np.float64)
        assert (np.abs(got - ref) <= 2e-3 + 1e-2 * np.abs(ref)).all()
        return q_out

    def check_tree(self, host, written):
        ref, t = spec.tree_attention(self.q_out.cpu().numpy(), *written, self.tables, host["lens"],
                                     self.qs.cpu().numpy(), self.trees, D ** -0.5, Hk)
        got = self.out.cpu().numpy().astype(np.float64)
        assert (np.abs(got - ref) <= spec.tree_tolerance(ref, t, D)).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_steps_follow_each_other(fp8):
    st = Step(fp8)
    ctx = np.array([0, 15, 40])
    for step in range(4):
        host = st.fill(ctx, 100 + step)
        before = st.values()
        st.enqueue()
        assert pkv.pkv_get_device_error() == (0, -1)
        st.check(host, before)
        # the tree again, over the rows as they were when it ran
        outs = st.out.clone()
        moved = [c.clone() for c in st.caches + st.scales]
        host2 = st.fill(ctx, 100 + step)
        assert all(np.array_equal(host[n], host2[n]) for n in host)
        st.path.fill_(-1)  # nothing accepted: the caches stay as drafted
        st.enqueue()
        assert torch.equal(st.out, outs)  # (context rows are the same; drafted ones written again)
        st.check_tree(host, st.values())
        for c, m in zip(st.caches + st.scales, moved):
            c.copy_(m)
        ctx = host["dlens"].astype(np.int64)


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_a_captured_step_replays_on_new_inputs(fp8):
    st, eager = Step(fp8), Step(fp8)
    ctx = np.array([3, 30, 64])
    st.fill(ctx, 1)
    st.enqueue()  # first calls outside the capture
    torch.cuda.synchronize()
    for c in st.caches + st.scales:
        c.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.enqueue()
    for step in range(5):
        host = st.fill(ctx, 50 + step)
        eager.fill(ctx, 50 + step)
        graph.replay()
        eager.enqueue()
        for a, b in ((st.out, eager.out), (st.dout, eager.dout), (st.q_out, eager.q_out)):
            assert torch.equal(a, b)
        for a, b in zip(st.caches + st.scales, eager.caches + eager.scales):
            assert torch.equal(a, b)
        ctx = host["dlens"].astype(np.int64)
    assert pkv.pkv_get_device_error() == (0, -1)


def test_queries_are_seen_by_the_call_that_follows():
    # norm + rotation straight into a decode and a tree attention, many times
    # over, each time with other queries: no call reads the previous ones
    st = Step(False)
    ctx = np.array([100, 31, 64])
    st.fill(ctx, 9)
    st.enqueue()
    rng = torch.Generator(device="cuda").manual_seed(3)
    rows = [torch.randn(st.qkv.shape, generator=rng, device="cuda").half() for _ in range(40)]
    outs = []
    for r in rows:
        st.qkv.copy_(r)
        st.enqueue()
        outs.append(st.out.clone())
    for r, o in zip(rows, outs):
        st.qkv.copy_(r)
        torch.cuda.synchronize()
        st.enqueue()
        torch.cuda.synchronize()
        assert torch.equal(st.out, o)
