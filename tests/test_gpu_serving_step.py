"""The serving step's operators together, as a loop runs them: blocks and slots from
lengths, rows normed, rotated and written, attention under score rules; then a
drafted tree verified, its path accepted and the rejected blocks given back --
eagerly against the definitions, and as one replayed CUDA graph against that."""

import numpy as np
import pytest

from oracle import serving as srv
from oracle import speculative as spec

torch = pytest.importorskip("torch")
import paged_kv_cache_131_gb300 as pkv  # noqa: E402

pytestmark = pytest.mark.gpu
BS, H, Hk, D, S, MB, NODES, DEPTH, V, MAXPOS = 16, 8, 2, 64, 4, 16, 9, 5, 101, 400
CAPACITY, TOKENS = S * MB, 300
i32, i64, f16 = torch.int32, torch.int64, torch.float16
RULES = dict(softcap=8.0, window=40)


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_131_gb300 import _build
    _build.build()
    pkv.pkv_get_device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Server:
    """The loop's device state: everything that a step reads or writes."""

    def __init__(self):
        rng = np.random.default_rng(1)
        z = lambda *s, t=i32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.k, self.v = z(CAPACITY, BS, Hk, D, t=f16), z(CAPACITY, BS, Hk, D, t=f16)
        self.tables, self.lens, self.new = z(S, MB), z(S), z(S)
        self.free, self.count = dev(rng.permutation(CAPACITY).astype(np.int32)), z(1)
        self.count.fill_(CAPACITY)
        self.start, self.nodes_start = z(S + 1), torch.arange(0, S * NODES + 1, NODES, dtype=i32,
                                                              device="cuda")
        angle = np.arange(MAXPOS)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
        self.rope = dev(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
        self.slopes = dev((2.0 ** -(1.0 + np.arange(H))).astype(np.float32))
        self.prefix = dev(np.array([0, 3, 20, 1], np.int32))
        n = max(pkv.pkv_chunk_workspace_bytes(S, H, Hk, D, TOKENS, TOKENS, MB * BS),
                pkv.pkv_decode_workspace_bytes(S, H, Hk, D, MB * BS))
        self.ws = z(n, t=torch.uint8)
        self.tree_ws = z(pkv.pkv_tree_workspace_bytes(S, H, Hk, D, S * NODES, NODES, MB * BS),
                         t=torch.uint8)
        self.rules = dict(RULES, slopes=self.slopes, prefix_lens=self.prefix)

    def snapshot(self):
        return {n: getattr(self, n).cpu().numpy().copy()
                for n in ("k", "v", "tables", "lens", "free", "count")}

    def resize(self, tokens):
        """Grows or shrinks to self.new, in place; the rows' slots and positions."""
        slots, pos = (torch.empty(tokens, dtype=i64, device="cuda") for _ in range(2))
        pkv.pkv_resize_sequences(self.tables, self.lens, self.new, self.lens, self.free, self.count,
                                 self.count, self.start, slots, pos, BS, CAPACITY)
        return slots, pos

    def write(self, qkv, pos, slots):
        T = qkv.shape[0]
        q = torch.zeros(T, H, D, dtype=f16, device="cuda")
        pkv.pkv_norm_rope_write(q, qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], pos, slots, self.k,
                                self.v, self.rope)
        return q

    def prefill(self, qkv, longest):
        slots, pos = self.resize(qkv.shape[0])
        q = self.write(qkv, pos, slots)
        out = torch.zeros_like(q)
        pkv.pkv_chunk_attention_scored(out, q, self.k, self.v, self.tables, self.lens, self.start,
                                       D ** -0.5, H, Hk, D, BS, longest, MB * BS, CAPACITY, self.ws,
                                       **self.rules)
        return q, out, slots

    def decode(self, qkv):
        torch.add(self.lens, 1, out=self.new)
        slots, pos = self.resize(S)
        q = self.write(qkv, pos, slots)
        out = torch.zeros_like(q)
        pkv.pkv_decode_attention_scored(out, q, self.k, self.v, self.tables, self.lens, D ** -0.5, H,
                                        Hk, D, BS, MB * BS, CAPACITY, self.ws, **self.rules)
        return q, out

    def speculate(self, d):
        """One tree per sequence: its rows, its attention, the accepted path, the rest
        given back."""
        ctx = self.lens.clone()
        torch.add(self.lens, NODES, out=self.new)
        slots, _ = self.resize(S * NODES)
        pos = (ctx.long()[:, None] + d["depth"]).view(-1)
        q = self.write(d["qkv"], pos, slots)
        out = torch.zeros_like(q)
        pkv.pkv_tree_attention(out, q, self.k, self.v, self.tables, self.lens, self.nodes_start,
                               d["mask"], D ** -0.5, H, Hk, D, BS, NODES, MB * BS, CAPACITY,
                               self.tree_ws)
        path = torch.zeros(S, DEPTH, dtype=i32, device="cuda")
        n, nxt = (torch.zeros(S, dtype=i32, device="cuda") for _ in range(2))
        pkv.pkv_tree_verify(path, n, nxt, d["tokens"], d["parents"], self.nodes_start, d["target"],
                            d["draft"], d["au"], d["su"])
        view = pkv.pkv_view(0, 0, BS * Hk * D * 2, Hk * D * 2, 0)
        pkv.pkv_tree_accept([(self.k, view), (self.v, view)], 1, path, ctx, self.tables, BS, CAPACITY)
        torch.add(ctx, n, out=self.new)
        self.resize(0)
        return q, out, path, n, nxt


def drafts(seed):
    """Trees, their rows and the two models' distributions, on the host."""
    rng = np.random.default_rng(seed)
    parents = np.full((S, NODES), -1, np.int32)
    mask = np.zeros((S, NODES, NODES), bool)
    for i in range(S):
        for j in range(NODES):
            if j:
                parents[i, j] = rng.integers(max(0, j - 4), j)
                mask[i, j] = mask[i, parents[i, j]]
            mask[i, j, j] = True
    T = S * NODES
    target = rng.dirichlet(np.full(V, 0.05), T).astype(np.float32)
    draft = (0.7 * target + 0.3 * rng.dirichlet(np.full(V, 0.05), T)).astype(np.float32)
    tokens = rng.integers(0, V, T)
    for i in range(S):
        for j in range(1, NODES):
            p = draft[i * NODES + parents[i, j]].astype(np.float64)
            tokens[i * NODES + j] = rng.choice(V, p=p / p.sum())
    return dict(qkv=rng.standard_normal((T, H + 2 * Hk, D)).astype(np.float16),
                depth=(mask.sum(2) - 1).astype(np.int64), mask=spec.mask_words(mask.reshape(T, NODES)),
                tokens=tokens.astype(np.int32), parents=parents.reshape(-1), target=target,
                draft=draft, au=rng.random(T).astype(np.float32),
                su=rng.random(S).astype(np.float32)), mask.reshape(T, NODES)


def check_attention(server, q, out, start):
    ref, tol = srv.scored_attention(q.cpu().numpy(), server.k.cpu().numpy(), server.v.cpu().numpy(),
                                    server.tables.cpu().numpy(), server.lens.cpu().numpy(), start,
                                    D ** -0.5, Hk, slopes=server.slopes.cpu().numpy(),
                                    prefix_lens=server.prefix.cpu().numpy(), **RULES)
    assert (np.abs(out.cpu().numpy() - ref) <= tol).all()


def check_blocks(server):
    """Every block is held by one sequence or free."""
    s = server.snapshot()
    held = [int(s["tables"][i, k]) for i in range(S) for k in range(-(-int(s["lens"][i]) // BS))]
    assert sorted(held + s["free"][:int(s["count"][0])].tolist()) == list(range(CAPACITY))


def run_prompts(server):
    rng = np.random.default_rng(2)
    prompts = [37, 64, 5, 130]
    server.new.copy_(dev(np.array(prompts, np.int32)))
    qkv = rng.standard_normal((TOKENS, H + 2 * Hk, D)).astype(np.float16)
    return prompts, server.prefill(dev(qkv), max(prompts))


def test_a_loop_against_the_definitions():
    s = Server()
    prompts, (q, out, slots) = run_prompts(s)
    T = sum(prompts)
    assert s.lens.tolist() == prompts and (slots[T:] == -1).all()
    check_attention(s, q[:T], out[:T], np.concatenate([[0], np.cumsum(prompts)]))
    check_blocks(s)
    rng = np.random.default_rng(3)
    lengths = []
    for step in range(4):
        rows = rng.standard_normal((S, H + 2 * Hk, D)).astype(np.float16)
        q, out = s.decode(dev(rows))
        check_attention(s, q, out, np.arange(S + 1))
        before = s.snapshot()
        host, mask = drafts(10 + step)
        q, out, path, n, nxt = s.speculate({k: dev(x) for k, x in host.items()})
        after = s.snapshot()
        want = srv.verify(host["tokens"], host["parents"], s.nodes_start.cpu().numpy(),
                          host["target"], host["draft"], host["au"], host["su"], DEPTH)
        assert (want[3] > 2.0 ** -18).all()
        for got, ref in zip((path, n, nxt), want):
            assert np.array_equal(got.cpu().numpy(), ref)
        lengths += n.tolist()
        # the tables and the free list: grown by the tree, shrunk to the path
        ctx = before["lens"]
        t, lens, free, count, *_ = srv.resize(before["tables"], ctx, ctx + NODES, before["free"],
                                              int(before["count"][0]), BS, S * NODES, CAPACITY)
        grown = t
        t, lens, free, count, *_ = srv.resize(t, lens, ctx + want[1], free, count, BS, 0, CAPACITY)
        assert np.array_equal(after["tables"], t) and np.array_equal(after["lens"], lens)
        assert np.array_equal(after["free"], free) and int(after["count"][0]) == count
        check_blocks(s)
        # the rows that stay: each accepted node's, rotated at its depth, in its place
        for i in range(S):
            for d, node in enumerate(want[0][i, :want[1][i]]):
                row = host["qkv"][i * NODES + node]
                at = ctx[i] + d
                place = after["tables"][i, at // BS], at % BS
                key, _ = spec.norm_rope(row[None, H:H + Hk], None, 0.0, s.rope.cpu().numpy(),
                                        [at], False)
                assert np.abs(after["k"][place] - key[0]).max() <= 2.0 ** -8
                assert np.array_equal(after["v"][place], row[H + Hk:])
        assert grown.shape == t.shape
    assert max(lengths) > 2 and min(lengths) < 3
    assert pkv.pkv_get_device_error()[0] == 0


def test_the_loop_as_a_graph():
    eager, graphed = Server(), Server()
    run_prompts(eager)
    run_prompts(graphed)
    rows = torch.zeros(S, H + 2 * Hk, D, dtype=f16, device="cuda")
    buffers = {k: dev(x) for k, x in drafts(0)[0].items()}
    # a first pass outside the capture, then the state as it was
    saved = {n: getattr(graphed, n).clone() for n in ("k", "v", "tables", "lens", "free", "count")}
    graphed.decode(rows)
    graphed.speculate(buffers)
    for n, x in saved.items():
        getattr(graphed, n).copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = graphed.decode(rows) + graphed.speculate(buffers)
    for step in range(5):
        rng = np.random.default_rng([4, step])
        rows.copy_(dev(rng.standard_normal((S, H + 2 * Hk, D)).astype(np.float16)))
        for k, x in drafts(30 + step)[0].items():
            buffers[k].copy_(dev(x))
        want = eager.decode(rows) + eager.speculate(buffers)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        a, b = graphed.snapshot(), eager.snapshot()
        for n in a:
            if n == "free":  # (entries past the count hold nothing of use)
                c = int(a["count"][0])
                assert np.array_equal(a[n][:c], b[n][:c])
            elif n == "tables":
                for i in range(S):
                    used = -(-int(a["lens"][i]) // BS)
                    assert np.array_equal(a[n][i, :used], b[n][i, :used])
            else:
                assert np.array_equal(a[n], b[n]), n
    assert pkv.pkv_get_device_error()[0] == 0
