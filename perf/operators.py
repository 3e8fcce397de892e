"""Timed cases of the speculative-step operators of libpagedkv.

Four operators around the paged cache, each in a plain form (elementary torch
operations in 32 bits) and through the library's entry points:

* ``norm_rope_write``: per-head RMS norm of queries and keys, rotation by
  position, queries out and keys / values into the paged cache (fp16 or FP8);
* ``cache_read``: rows of an FP8 cache read back as fp16;
* ``tree_attention``: drafted token trees attending to their sequences' paged
  caches (fp16 or FP8);
* ``tree_accept``: the cache rows of an accepted tree path moved to their
  positions, for every layer.

``own`` selects the library's calls; ``prepare`` makes a case's inputs from a
seed, ``run`` is one pass, ``exact`` the definition in 64 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

BS = 16  # block size of the attention caches

# ---------------------------------------------------------------- the cases


def listed():
    return [
        # a decode step of 64 sequences between the QKV product and attention
        dict(name="nrw_decode_64", op="norm_rope_write", tokens=64, heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, norm=True, fp8=False),
        # a prefill step of long prompts
        dict(name="nrw_prefill_16384", op="norm_rope_write", tokens=16384, heads=32, kv_heads=8,
             dim=128, rot=128, interleaved=False, norm=True, fp8=False),
        # an odd token count under a 2048-token budget, partial interleaved
        # rotation, quantised cache
        dict(name="nrw_fp8_2001", op="norm_rope_write", tokens=2001, heads=64, kv_heads=8,
             dim=128, rot=64, interleaved=True, norm=True, fp8=True),
        # one short prompt's rows read back
        dict(name="read_fp8_953", op="cache_read", tokens=953, kv_heads=4, dim=64),
        # four long prompts handed on in 16 bits
        dict(name="read_fp8_131072", op="cache_read", tokens=131072, kv_heads=8, dim=128),
        # one user, a small tree: latency
        dict(name="tree_one", op="tree_attention", seqs=1, lo=1041, hi=1041, nodes=8, heads=32,
             kv_heads=8, dim=128, fp8=False),
        # a serving batch verifying 16 nodes each, ragged lengths
        dict(name="tree_batch", op="tree_attention", seqs=64, lo=256, hi=4096, nodes=16, heads=32,
             kv_heads=8, dim=128, fp8=False),
        # long contexts
        dict(name="tree_long", op="tree_attention", seqs=8, lo=32768, hi=32768, nodes=32, heads=32,
             kv_heads=8, dim=128, fp8=False),
        # wide trees, large head groups: the most arithmetic per cached byte
        dict(name="tree_wide", op="tree_attention", seqs=32, lo=300, hi=4001, nodes=63, heads=64,
             kv_heads=8, dim=128, fp8=False),
        # long contexts in a quantised cache
        dict(name="tree_fp8", op="tree_attention", seqs=16, lo=8000, hi=32768, nodes=16, heads=32,
             kv_heads=8, dim=128, fp8=True),
        # one layer's rows of a few sequences
        dict(name="accept_small", op="tree_accept", seqs=4, path=5, nodes=16, layers=1, kv_heads=8,
             dim=128),
        # a whole model's layers of a serving batch
        dict(name="accept_layers", op="tree_accept", seqs=64, path=7, nodes=63, layers=16,
             kv_heads=8, dim=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope_write", "cache_read", "tree_attention", "tree_attention",
                     "tree_accept"])
    dim = rng.choice([64, 128, 128])
    if op == "norm_rope_write":
        kv = rng.choice([1, 2, 4, 8, 8])
        return dict(op=op, tokens=_log_int(rng, 1, 16000), heads=kv * rng.choice([1, 2, 4]),
                    kv_heads=kv, dim=dim, rot=rng.choice([dim, dim, dim // 2, dim - 16]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8,
                    fp8=rng.random() < 0.5)
    if op == "cache_read":
        return dict(op=op, tokens=_log_int(rng, 1, 130000), kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=dim)
    if op == "tree_accept":
        nodes = rng.randint(3, 64)
        return dict(op=op, seqs=_log_int(rng, 1, 64), path=rng.randint(2, min(8, nodes)),
                    nodes=nodes, layers=_log_int(rng, 1, 16), kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=dim)
    kv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4, 4, 8])
    nodes = rng.randint(1, 64)
    hi = _log_int(rng, nodes + 1, 32768)
    lo = max(nodes, int(hi * rng.uniform(0.1, 1.0)))
    # at most the bytes and operations of the largest listed cases
    most = min(8 * 32768 * 8, 8 * 32768 * 8 * 4 * 32 // (group * nodes))
    seqs = max(1, min(_log_int(rng, 1, 128), most // (hi * kv)))
    return dict(op=op, seqs=seqs, lo=lo, hi=hi, nodes=nodes, heads=kv * group, kv_heads=kv,
                dim=dim, fp8=rng.random() < 0.4)


# ------------------------------------------------------------------- inputs


def _lens(case):
    """Sequence lengths of a tree case: spread over [lo, hi] without order."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int((hi - lo + 1) * ((0.5 + 0.6180339887498949 * i) % 1.0))
            for i in range(case["seqs"])]


def _path_lens(case):
    """Accepted nodes of each sequence: the longest path and shorter ones."""
    P, Q = case["path"], case["nodes"]
    lens = [max(2, P - i % 3) for i in range(case["seqs"])]
    return [min(n, 1 + max(1, Q - n)) for n in lens]


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).half()


def _randn_big(g, *shape):
    """fp16 normals without a 32-bit copy of the whole tensor."""
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float16)


def _tree(nodes, rng):
    """Parents of a token tree whose node 0 is the root, in breadth order."""
    parents = [-1]
    for j in range(1, nodes):
        parents.append(int(rng.integers(max(0, j // 2 - 3), max(1, j * 2 // 3 + 1))))
        parents[-1] = min(parents[-1], j - 1)
    return parents


def _mask_rows(nodes, parents, words):
    """Bit j of row i: node j is node i or an ancestor of it."""
    rows = np.zeros((nodes, words), dtype=np.uint64)
    for i in range(nodes):
        if parents[i] >= 0:
            rows[i] = rows[parents[i]]
        rows[i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return rows.view(np.int64)


def _quantised(g, num_blocks, kv, dim):
    """An FP8 cache as it stands after writes of normal rows: codes, scales."""
    codes = torch.randn(num_blocks, BS, kv, dim, generator=g, device="cuda",
                        dtype=torch.float16).mul_(100.0).clamp_(-448.0, 448.0)
    codes = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.rand(num_blocks, BS, kv, generator=g, device="cuda").mul_(0.006).add_(0.006)
    return codes, scale


def _rope_table(max_pos, rot):
    inv = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    ang = np.arange(max_pos, dtype=np.float64)[:, None] * inv[None, :]
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def _prepare_norm_rope_write(case, seed):
    T, H, Hk, D, rot = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "rot"))
    g = _gen(seed, 1)
    rng = np.random.default_rng([seed, 11])
    # one packed row per token, as the QKV product leaves it
    qkv = _randn(g, T, (H + 2 * Hk) * D, scale=1.7)
    q = qkv[:, :H * D].view(T, H, D)
    k = qkv[:, H * D:(H + Hk) * D].view(T, Hk, D)
    v = qkv[:, (H + Hk) * D:].view(T, Hk, D)
    max_pos = 32768
    nb = T // BS + 9
    slots = rng.permutation(nb * BS)[:T]
    positions = rng.integers(0, max_pos, T)
    state = dict(case=case, q=q, k=k, v=v, num_blocks=nb,
                 positions=torch.from_numpy(positions.astype(np.int64)).cuda(),
                 slots=torch.from_numpy(slots.astype(np.int64)).cuda(),
                 table=_rope_table(max_pos, rot), eps=1e-6,
                 q_out=torch.zeros(T, H, D, device="cuda", dtype=torch.float16),
                 q_weight=None, k_weight=None)
    if case["norm"]:
        state["q_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).half()
        state["k_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).half()
    kind = torch.uint8 if case["fp8"] else torch.float16
    for name in ("k", "v"):
        state[name + "_cache"] = torch.zeros(nb, BS, Hk, D, device="cuda", dtype=kind)
        if case["fp8"]:
            state[name + "_scale"] = torch.zeros(nb, BS, Hk, device="cuda")
    return state


def _prepare_cache_read(case, seed):
    T, Hk, D = case["tokens"], case["kv_heads"], case["dim"]
    g = _gen(seed, 2)
    rng = np.random.default_rng([seed, 12])
    blocks = -(-T // BS)
    nb = blocks + 5
    table = rng.permutation(nb)[:blocks]
    t = np.arange(T)
    state = dict(case=case, num_blocks=nb,
                 slots=torch.from_numpy((table[t // BS] * BS + t % BS).astype(np.int64)).cuda())
    for name in ("k", "v"):
        state[name + "_cache"], state[name + "_scale"] = _quantised(g, nb, Hk, D)
        state[name + "_rows"] = torch.zeros(T, Hk, D, device="cuda", dtype=torch.float16)
    return state


def _prepare_tree_attention(case, seed):
    S, H, Hk, D, Q = (case[k] for k in ("seqs", "heads", "kv_heads", "dim", "nodes"))
    g = _gen(seed, 3)
    rng = np.random.default_rng([seed, 13])
    lens = _lens(case)
    blocks = [-(-n // BS) for n in lens]
    nb = sum(blocks) + 3
    ids = rng.permutation(nb)
    tables = np.zeros((S, max(blocks)), dtype=np.int32)
    at = 0
    for i, b in enumerate(blocks):
        tables[i, :b] = ids[at:at + b]
        at += b
    words = -(-Q // 64)
    mask = np.concatenate([_mask_rows(Q, _tree(Q, rng), words) for _ in range(S)])
    state = dict(case=case, lens=lens, num_blocks=nb, scale=1.0 / math.sqrt(D),
                 q=_randn(g, S * Q, H, D), out=torch.zeros(S * Q, H, D, device="cuda",
                                                           dtype=torch.float16),
                 tables=torch.from_numpy(tables).cuda(),
                 seq_lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                 query_start=torch.arange(0, S * Q + 1, Q, dtype=torch.int32).cuda(),
                 mask=torch.from_numpy(mask).cuda())
    for name in ("k", "v"):
        if case["fp8"]:
            state[name + "_cache"], state[name + "_scale"] = _quantised(g, nb, Hk, D)
        else:
            state[name + "_cache"] = _randn_big(g, nb, BS, Hk, D)
    if own:
        import paged_kv_cache_131_gb300 as pkv
        n = pkv.pkv_tree_workspace_bytes(S, H, Hk, D, S * Q, Q, max(lens))
        state["workspace"] = torch.zeros(n, device="cuda", dtype=torch.uint8)
    return state


def _prepare_tree_accept(case, seed):
    S, P, Q, layers, Hk, D = (case[k] for k in ("seqs", "path", "nodes", "layers", "kv_heads",
                                                "dim"))
    g = _gen(seed, 4)
    rng = np.random.default_rng([seed, 14])
    # node 0 is the root and always accepted; the others come from behind the
    # places that the path fills, so a second pass finds the same rows
    ctx = rng.integers(0, 40, S)
    path = np.full((S, P), -1, dtype=np.int32)
    for i, n in enumerate(_path_lens(case)):
        path[i, 0] = 0
        path[i, 1:n] = np.sort(rng.choice(np.arange(n, Q), n - 1, replace=False))
    mb = (40 + Q) // BS + 1
    nb = S * mb + 2
    tables = rng.permutation(nb)[:S * mb].reshape(S, mb).astype(np.int32)
    return dict(case=case, num_blocks=nb, path=torch.from_numpy(path).cuda(),
                ctx=torch.from_numpy(ctx.astype(np.int32)).cuda(),
                tables=torch.from_numpy(tables).cuda(),
                k_cache=_randn_big(g, layers, nb, BS, Hk, D),
                v_cache=_randn_big(g, layers, nb, BS, Hk, D))


_PREPARE = dict(norm_rope_write=_prepare_norm_rope_write, cache_read=_prepare_cache_read,
                tree_attention=_prepare_tree_attention, tree_accept=_prepare_tree_accept)

# ------------------------------------------------------------------ one pass


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _cache_values(state):
    """The caches as the values they hold: codes as 8-bit floats, and their scales."""
    if state["case"].get("fp8"):
        return (state["k_cache"].view(torch.float8_e4m3fn), state["k_scale"],
                state["v_cache"].view(torch.float8_e4m3fn), state["v_scale"])
    return state["k_cache"], state["v_cache"]


def _own_norm_rope_write(s):
    import paged_kv_cache_131_gb300 as pkv
    kw = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
              interleaved=s["case"]["interleaved"], block_size=BS, num_blocks=s["num_blocks"])
    if s["case"]["fp8"]:
        pkv.pkv_norm_rope_write_fp8(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["slots"],
                                    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                    s["table"], **kw)
    else:
        pkv.pkv_norm_rope_write(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["slots"],
                                s["k_cache"], s["v_cache"], s["table"], **kw)
    return (s["q_out"],) + _cache_values(s)


def _own_cache_read(s):
    import paged_kv_cache_131_gb300 as pkv
    pkv.pkv_cache_read_fp8(s["k_rows"], s["v_rows"], s["slots"], s["k_cache"], s["v_cache"],
                           s["k_scale"], s["v_scale"], BS, s["num_blocks"])
    return s["k_rows"], s["v_rows"]


def _own_tree_attention(s):
    import paged_kv_cache_131_gb300 as pkv
    c = s["case"]
    args = (s["tables"], s["seq_lens"], s["query_start"], s["mask"], s["scale"], c["heads"],
            c["kv_heads"], c["dim"], BS, c["nodes"], max(s["lens"]), s["num_blocks"],
            s["workspace"])
    if c["fp8"]:
        pkv.pkv_tree_attention_fp8(s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"],
                                   s["v_scale"], *args)
    else:
        pkv.pkv_tree_attention(s["out"], s["q"], s["k_cache"], s["v_cache"], *args)
    return s["out"]


def _own_tree_accept(s):
    import paged_kv_cache_131_gb300 as pkv
    c = s["case"]
    row = c["kv_heads"] * c["dim"] * 2
    view = pkv.pkv_view(0, s["num_blocks"] * BS * row, BS * row, row, 0)
    pkv.pkv_tree_accept([(s["k_cache"], view), (s["v_cache"], view)], c["layers"], s["path"],
                        s["ctx"], s["tables"], BS, s["num_blocks"])
    return s["k_cache"], s["v_cache"]


def _plain_rows(x, weight, eps, cos, sin, interleaved):
    """Norm and rotation of rows [T, h, D] in 32 bits; cos, sin [T, rot/2]."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()
    half = cos.shape[1]
    c, n = cos[:, None, :], sin[:, None, :]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = a * c - b * n
        y[..., 1:2 * half:2] = b * c + a * n
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half] = a * c - b * n
        y[..., half:2 * half] = b * c + a * n
    return y


def _plain_norm_rope_write(s):
    rows = s["table"][s["positions"]]
    half = rows.shape[1] // 2
    cos, sin = rows[:, :half], rows[:, half:]
    inter = s["case"]["interleaved"]
    s["q_out"].copy_(_plain_rows(s["q"], s["q_weight"], s["eps"], cos, sin, inter))
    k = _plain_rows(s["k"], s["k_weight"], s["eps"], cos, sin, inter)
    for name, x in (("k", k), ("v", s["v"].float())):
        cache = s[name + "_cache"].flatten(0, 1)
        if s["case"]["fp8"]:
            scale = x.abs().amax(-1) / 448.0
            y = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0)
            cache[s["slots"]] = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_scale"].flatten(0, 1)[s["slots"]] = scale
        else:
            cache[s["slots"]] = x.half()
    return (s["q_out"],) + _cache_values(s)


def _plain_cache_read(s):
    for name in ("k", "v"):
        codes = s[name + "_cache"].flatten(0, 1)[s["slots"]].view(torch.float8_e4m3fn).float()
        s[name + "_rows"].copy_(codes * s[name + "_scale"].flatten(0, 1)[s["slots"]][..., None])
    return s["k_rows"], s["v_rows"]


def _plain_tree_attention(s):
    c = s["case"]
    H, Hk, D, Q = c["heads"], c["kv_heads"], c["dim"], c["nodes"]
    G = H // Hk
    bit = torch.arange(Q, device="cuda")
    for i, L in enumerate(s["lens"]):
        ids = s["tables"][i, :-(-L // BS)].long()
        kv = []
        for name in ("k", "v"):
            x = s[name + "_cache"][ids]
            if c["fp8"]:
                x = x.view(torch.float8_e4m3fn).float() * s[name + "_scale"][ids][..., None]
            kv.append(x.flatten(0, 1)[:L].float().transpose(0, 1))  # [Hk, L, D]
        q = s["q"][i * Q:(i + 1) * Q].float().view(Q, Hk, G, D).transpose(0, 1)
        scores = (q.reshape(Hk, Q * G, D) @ kv[0].transpose(1, 2)).view(Hk, Q, G, L) * s["scale"]
        sees = (s["mask"][i * Q:(i + 1) * Q][:, bit // 64] >> (bit % 64)) & 1
        scores[..., L - Q:].masked_fill_((sees == 0)[None, :, None, :], float("-inf"))
        top = scores.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        w = torch.exp(scores - top)
        den = w.sum(-1, keepdim=True)
        o = (w.view(Hk, Q * G, L) @ kv[1]).view(Hk, Q, G, D)
        o = torch.where(den > 0, o / den, torch.zeros_like(o))
        s["out"][i * Q:(i + 1) * Q] = o.transpose(0, 1).reshape(Q, H, D)
    return s["out"]


def _plain_tree_accept(s):
    path, ctx, tables = s["path"].long(), s["ctx"].long(), s["tables"].long()
    seq, depth = torch.nonzero(path >= 0, as_tuple=True)

    def slot(pos):
        return tables[seq, pos // BS] * BS + pos % BS

    src, dst = slot(ctx[seq] + path[seq, depth]), slot(ctx[seq] + depth)
    for name in ("k_cache", "v_cache"):
        rows = s[name].flatten(1, 2)
        rows[:, dst] = rows[:, src]
    return s["k_cache"], s["v_cache"]


_PLAIN = dict(norm_rope_write=_plain_norm_rope_write, cache_read=_plain_cache_read,
              tree_attention=_plain_tree_attention, tree_accept=_plain_tree_accept)
_OWN = dict(norm_rope_write=_own_norm_rope_write, cache_read=_own_cache_read,
            tree_attention=_own_tree_attention, tree_accept=_own_tree_accept)

# --------------------------------------------------------------------- work


def work(case):
    """Bytes and operations a pass cannot do without."""
    op = case["op"]
    Hk, D = case["kv_heads"], case["dim"]
    if op == "norm_rope_write":
        T, H = case["tokens"], case["heads"]
        kv_out = 2 * Hk * (D + 4) if case["fp8"] else 2 * Hk * D * 2
        # packed rows and positions / slots in, table rows (each at most
        # once), queries and cache rows out
        table = min(T, 32768) * case["rot"] * 4
        return dict(bytes=T * ((H + 2 * Hk) * D * 2 + 16 + H * D * 2 + kv_out) + table,
                    flops=T * (H + Hk) * D * 7)
    if op == "cache_read":
        T = case["tokens"]
        return dict(bytes=T * (2 * Hk * (D + 4) + 2 * Hk * D * 2 + 8), flops=T * 2 * Hk * D)
    if op == "tree_accept":
        # the path's rows but the root's (it stays in place) read and written
        moved = sum(n - 1 for n in _path_lens(case))
        return dict(bytes=case["layers"] * 2 * moved * Hk * D * 2 * 2, flops=0)
    S, H, Q = case["seqs"], case["heads"], case["nodes"]
    tokens = sum(_lens(case))
    row = 2 * Hk * (D + 4) if case["fp8"] else 2 * Hk * D * 2
    return dict(bytes=tokens * row + 2 * S * Q * H * D * 2 + S * Q * 8 + tokens // 4,
                flops=4 * D * H * Q * (tokens - S * Q + S))


# -------------------------------------------------------------------- exact


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_rotated(x, weight, eps, angles, interleaved):
    """Rows as complex pairs turned by cos + i sin, float64."""
    x = x.double()
    if weight is not None:
        rms = torch.linalg.vector_norm(x, dim=-1, keepdim=True).pow(2) / x.shape[-1]
        x = x / torch.sqrt(rms + eps) * weight.double()
    half = angles.shape[1] // 2
    turn = torch.complex(angles[:, :half].double(), angles[:, half:].double())[:, None, :]
    head, tail = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        z = torch.view_as_complex(head.unflatten(-1, (half, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, tail], -1)


def _exact_norm_rope_write(case, s):
    angles = s["table"].index_select(0, s["positions"])
    q = _exact_rotated(s["q"], s["q_weight"], s["eps"], angles, case["interleaved"])
    out = [q]
    rows = dict(k=_exact_rotated(s["k"], s["k_weight"], s["eps"], angles, case["interleaved"]),
                v=s["v"].double())
    for name, x in rows.items():
        shape = s[name + "_cache"].shape
        cache = torch.zeros(shape[0] * BS, shape[2], shape[3], device="cuda", dtype=torch.float64)
        if case["fp8"]:
            # the values before their rounding to a code
            step = x.abs().max(-1).values / 448
            scale = torch.zeros(shape[0] * BS, shape[2], device="cuda", dtype=torch.float64)
            scale.index_copy_(0, s["slots"], step)
            x = torch.where(step[..., None] == 0, torch.zeros_like(x), x / step[..., None])
        cache.index_copy_(0, s["slots"], x)
        out.append(cache.view(shape))
        if case["fp8"]:
            out.append(scale.view(shape[:3]))
    return tuple(out)


def _e4m3_values():
    """The 256 values of the format: sign, four exponent bits (bias 7), three of mantissa."""
    vals = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        vals.append(math.nan if (c & 127) == 127 else (-v if c & 128 else v))
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _exact_cache_read(case, s):
    values = _e4m3_values()
    out = []
    for name in ("k", "v"):
        codes = s[name + "_cache"].flatten(0, 1).index_select(0, s["slots"])
        scale = s[name + "_scale"].flatten(0, 1).index_select(0, s["slots"]).double()
        out.append(values[codes.int()] * scale.unsqueeze(-1))
    return tuple(out)


def _exact_tree_attention(case, s):
    H, Hk, D, Q = case["heads"], case["kv_heads"], case["dim"], case["nodes"]
    G = H // Hk
    values = _e4m3_values() if case["fp8"] else None
    mask = s["mask"].cpu().numpy().view(np.uint64)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, L in enumerate(s["lens"]):
        sees = np.ones((Q, L), dtype=bool)
        for r in range(Q):
            bits = "".join(format(int(w), "064b")[::-1] for w in mask[i * Q + r])
            sees[r, L - Q:] = [b == "1" for b in bits[:Q]]
        sees = torch.from_numpy(sees).cuda()
        pos = torch.arange(L, device="cuda")
        blk, off = s["tables"][i].long()[pos // BS], pos % BS
        for h in range(Hk):
            k, v = (s[n + "_cache"][blk, off, h] for n in ("k", "v"))
            if case["fp8"]:
                k = values[k.int()] * s["k_scale"][blk, off, h].double()[:, None]
                v = values[v.int()] * s["v_scale"][blk, off, h].double()[:, None]
            k, v = k.double(), v.double()
            for j in range(G):
                q = s["q"][i * Q:(i + 1) * Q, h * G + j].double()
                t = torch.where(sees, torch.einsum("qd,ld->ql", q, k) * s["scale"], -math.inf)
                p = torch.softmax(t, dim=1)
                out[i * Q:(i + 1) * Q, h * G + j] = torch.einsum("ql,ld->qd", p, v)
    return out


def _exact_tree_accept(case, s):
    path, ctx = s["path"].tolist(), s["ctx"].tolist()
    tables = s["tables"].tolist()
    caches = [s["k_cache"].clone(), s["v_cache"].clone()]
    for new, old in zip(caches, (s["k_cache"], s["v_cache"])):
        for i, nodes in enumerate(path):
            for depth, node in enumerate(nodes):
                if node >= 0:
                    a, b = ctx[i] + depth, ctx[i] + node
                    new[:, tables[i][a // BS], a % BS] = old[:, tables[i][b // BS], b % BS]
    return tuple(c.double() for c in caches)


_EXACT = dict(norm_rope_write=_exact_norm_rope_write, cache_read=_exact_cache_read,
              tree_attention=_exact_tree_attention, tree_accept=_exact_tree_accept)
