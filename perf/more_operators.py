"""Timed cases of the serving-step operators of libpagedkv.

Three families of operators around the paged cache, each in a plain form
(elementary torch operations) and through the library's entry points:

* ``resize``: block tables, slot maps, positions and the free list of a step,
  from the lengths that the sequences have and are to have;
* ``verify``: drafted trees (or chains) of tokens verified against the target's
  probabilities with given random numbers: accepted path and next token;
* ``decode`` / ``chunk``: attention of one new token, or of several, over the
  paged cache whose scores follow rules: capped by a tanh, a bias that falls
  with the distance, a window, a prefix that every token sees.

``own`` selects the library's calls; ``prepare`` makes a case's inputs from a
seed, ``run`` is one pass, ``exact`` the definition in 64 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

BS = 16  # block size of the caches

# ---------------------------------------------------------------- the cases


def listed():
    return [
        # a decode step's bookkeeping: every sequence gets one token
        dict(name="resize_decode_64", op="resize", seqs=64, lo=256, hi=4096, kind="decode",
             tokens=64, short=False),
        # a mixed step of many requests: finished ones, rejected drafts, decodes, prompts
        dict(name="resize_mixed_1000", op="resize", seqs=1000, lo=1, hi=8000, kind="mixed",
             tokens=16384, short=False),
        # one user's chain of four drafts: latency
        dict(name="verify_chain_one", op="verify", seqs=1, nodes=5, vocab=32000, chain=True,
             drafted=True),
        # a serving batch's trees, drafts drawn from the draft model's distribution
        dict(name="verify_tree_64", op="verify", seqs=64, nodes=16, vocab=128256, chain=False,
             drafted=True),
        # wide trees of a drafter without probabilities, odd vocabulary
        dict(name="verify_fixed_32", op="verify", seqs=32, nodes=63, vocab=50257, chain=False,
             drafted=False),
        # one user, capped scores: latency
        dict(name="decode_cap_one", op="decode", seqs=1, lo=1041, hi=1041, heads=32, kv_heads=8,
             dim=128, cap=50.0, window=0, slopes=False, prefix=0, fp8=False),
        # a serving batch of a windowed layer that keeps its first tokens
        dict(name="decode_window_64", op="decode", seqs=64, lo=256, hi=32768, heads=32,
             kv_heads=8, dim=128, cap=0.0, window=4096, slopes=False, prefix=4, fp8=False),
        # long contexts, bias by distance
        dict(name="decode_bias_long", op="decode", seqs=8, lo=32768, hi=32768, heads=32,
             kv_heads=8, dim=128, cap=0.0, window=0, slopes=True, prefix=0, fp8=False),
        # long contexts in a quantised cache, capped scores
        dict(name="decode_cap_fp8", op="decode", seqs=16, lo=8000, hi=32768, heads=32, kv_heads=8,
             dim=128, cap=30.0, window=0, slopes=False, prefix=0, fp8=True),
        # a few drafted tokens a sequence, capped scores
        dict(name="chunk_draft_64", op="chunk", seqs=64, lo=256, hi=4096, qlo=4, qhi=4, heads=32,
             kv_heads=8, dim=128, cap=50.0, window=0, slopes=False, prefix=0),
        # chunks of long prompts, capped scores: the most arithmetic
        dict(name="chunk_prompt_cap", op="chunk", seqs=4, lo=2048, hi=8192, qlo=2048, qhi=2048,
             heads=32, kv_heads=8, dim=128, cap=50.0, window=0, slopes=False, prefix=0),
        # prompts of odd sizes behind a prefix that sees itself whole (an
        # image's tokens), a window and a bias after it
        dict(name="chunk_prefix_bias", op="chunk", seqs=6, lo=701, hi=5003, qlo=333, qhi=1999,
             heads=16, kv_heads=16, dim=64, cap=0.0, window=1024, slopes=True, prefix=577),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["resize", "verify", "verify", "decode", "decode", "chunk", "chunk"])
    if op == "resize":
        kind = rng.choice(["decode", "mixed", "mixed"])
        seqs = _log_int(rng, 1, 1000)
        hi = _log_int(rng, 40, 8000)
        tokens = seqs if kind == "decode" else max(seqs, _log_int(rng, 32, 16384))
        return dict(op=op, seqs=seqs, lo=_log_int(rng, 1, hi), hi=hi, kind=kind, tokens=tokens,
                    short=rng.random() < 0.3)
    if op == "verify":
        drafted = rng.random() < 0.6
        vocab = rng.choice([_log_int(rng, 500, 131071), 32000, 50257, 128256])
        nodes = rng.randint(1, 64)
        # at most the rows of the largest listed case
        most = 64 * 16 * 128256 // (nodes * vocab)
        return dict(op=op, seqs=max(1, min(_log_int(rng, 1, 128), most)), nodes=nodes, vocab=vocab,
                    chain=rng.random() < 0.3, drafted=drafted)
    kv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4, 4, 8])
    dim = rng.choice([64, 128, 128])
    rules = dict(cap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.4,
                 window=rng.choice([0, 0, _log_int(rng, 1, 8192)]),
                 prefix=rng.choice([0, 0, 4, _log_int(rng, 1, 2000)]))
    hi = _log_int(rng, 2, 32768)
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    if op == "decode":
        seqs = max(1, min(_log_int(rng, 1, 128), 8 * 32768 * 8 // (hi * kv)))
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, heads=kv * group, kv_heads=kv, dim=dim,
                    fp8=rng.random() < 0.4, **rules)
    qhi = _log_int(rng, 1, min(2048, hi))
    qlo = rng.randint(1, qhi)
    # at most the bytes and the operations of the largest listed cases
    most = min(8 * 32768 * 8 // (hi * kv), 4 * 2048 * 5120 * 32 // (hi * qhi * kv * group))
    return dict(op=op, seqs=max(1, min(_log_int(rng, 1, 64), most)), lo=lo, hi=hi, qlo=qlo,
                qhi=qhi, heads=kv * group, kv_heads=kv, dim=dim, **rules)


# ------------------------------------------------------------------- inputs


def _spread(lo, hi, n, phase=0.5):
    """n whole numbers over [lo, hi] without order."""
    return [lo + int((hi - lo + 1) * ((phase + 0.6180339887498949 * i) % 1.0)) for i in range(n)]


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def _cdiv(a, b):
    return -(-a // b)


def _resize_lens(case, rng):
    """Lengths before and after a step: most requests decode, some end, some
    have drafts taken back, some prefill."""
    S, lo, hi, tokens = case["seqs"], case["lo"], case["hi"], case["tokens"]
    old = rng.integers(lo, hi + 1, S)
    if case["kind"] == "decode":
        return old, old + 1
    new = old + 1
    what = rng.random(S)
    new = np.where(what < 0.08, 0, new)
    new = np.where((what >= 0.08) & (what < 0.3), np.maximum(old - rng.integers(0, 15, S), 1), new)
    new = np.where((what >= 0.3) & (what < 0.4), old, new)
    # prompts take the tokens that are left
    left = tokens - int(np.maximum(new - old, 0).sum())
    for i in np.nonzero(what >= 0.94)[0]:
        if left <= 0:
            break
        q = min(left, int(rng.integers(1, 2049)), hi + 2049 - int(old[i]) - 1)
        new[i] = old[i] + 1 + q
        left -= q
    return old, new


def _prepare_resize(case, seed):
    rng = np.random.default_rng([seed, 21])
    S = case["seqs"]
    old, new = _resize_lens(case, rng)
    have, want = _cdiv(old, BS), _cdiv(new, BS)
    mb = _cdiv(case["hi"] + 2049, BS)
    used = int(have.sum())
    need = int(np.maximum(want - have, 0).sum())
    # a pool that holds the step, or one that runs dry in it
    nb = S * (_cdiv(case["hi"], BS) + 1) + case["tokens"] // BS + 1
    spare = need // 2 if case["short"] else nb - used
    ids = rng.permutation(nb).astype(np.int32)
    tables = np.full((S, mb), -1, dtype=np.int32)
    at = np.concatenate([[0], np.cumsum(have)])
    for i in range(S):
        tables[i, :have[i]] = ids[at[i]:at[i + 1]]
    free = np.full(nb, -1, dtype=np.int32)
    free[:spare] = ids[used:used + spare]

    def up(x, kind=torch.int32):
        return torch.from_numpy(np.ascontiguousarray(x)).to(kind).cuda()

    T = case["tokens"]
    return dict(case=case, num_blocks=nb, tables=up(tables), seq_lens=up(old), new_lens=up(new),
                out_lens=torch.zeros(S, device="cuda", dtype=torch.int32), free=up(free),
                free_count=up(np.array([spare])),
                out_free_count=torch.zeros(1, device="cuda", dtype=torch.int32),
                slots=torch.zeros(T, device="cuda", dtype=torch.int64),
                positions=torch.zeros(T, device="cuda", dtype=torch.int64),
                query_start=torch.zeros(S + 1, device="cuda", dtype=torch.int32))


def _tree_parents(case, rng):
    Q = case["nodes"]
    if case["chain"]:
        return np.tile(np.arange(-1, Q - 1), (case["seqs"], 1)).astype(np.int32)
    out = np.full((case["seqs"], Q), -1, dtype=np.int32)
    for j in range(1, Q):
        out[:, j] = rng.integers(max(0, j // 2 - 3), max(1, j * 2 // 3 + 1), case["seqs"])
        out[:, j] = np.minimum(out[:, j], j - 1)
    return out


def _prepare_verify(case, seed):
    S, Q, V = case["seqs"], case["nodes"], case["vocab"]
    g = _gen(seed, 5)
    rng = np.random.default_rng([seed, 22])
    parents = _tree_parents(case, rng)
    T = S * Q
    target = torch.empty(T, V, device="cuda")
    draft = torch.empty(T, V, device="cuda") if case["drafted"] else None
    tokens = torch.zeros(S, Q, device="cuda", dtype=torch.int64)
    tokens[:, 0] = torch.randint(0, V, (S,), generator=g, device="cuda")
    par = torch.from_numpy(parents.astype(np.int64)).cuda()
    for j in range(Q):
        # a language model's distribution: few likely tokens, a long tail; the
        # drafter's is a noisy copy of it
        logits = torch.randn(S, V, generator=g, device="cuda") * 4.0
        rows = torch.arange(S, device="cuda") * Q + j
        target[rows] = torch.softmax(logits, -1)
        if case["drafted"]:
            logits += torch.randn(S, V, generator=g, device="cuda")
            draft[rows] = torch.softmax(logits, -1)
        kids = parents == j
        for i, k in zip(*np.nonzero(kids)):
            row = i * Q + j
            rank = int(kids[i, :k].sum())
            if case["drafted"]:
                # children are drawn independently from the drafter's distribution
                tokens[i, k] = torch.multinomial(draft[row], 1, generator=g)[0]
            else:
                # the likeliest tokens in turn
                tokens[i, k] = torch.topk(logits[i], 1 + rank).indices[rank]
    return dict(case=case, target=target, draft=draft,
                tokens=tokens.reshape(T).to(torch.int32), parents=par.reshape(T).to(torch.int32),
                query_start=torch.arange(0, T + 1, Q, dtype=torch.int32, device="cuda"),
                accept_u=torch.rand(T, generator=g, device="cuda"),
                sample_u=torch.rand(S, generator=g, device="cuda"),
                path=torch.zeros(S, min(Q, 16), device="cuda", dtype=torch.int32),
                path_lens=torch.zeros(S, device="cuda", dtype=torch.int32),
                next_tokens=torch.zeros(S, device="cuda", dtype=torch.int32))


def _lens(case):
    """(lengths, new tokens, prefixes) of an attention case's sequences."""
    S = case["seqs"]
    lens = _spread(case["lo"], case["hi"], S)
    news = [1] * S
    if case["op"] == "chunk":
        news = [min(n, L) for n, L in zip(_spread(case["qlo"], case["qhi"], S, 0.25), lens)]
    prefix = [0] * S
    if case["prefix"]:
        # first tokens that are always kept are as many for everyone; images differ
        p = case["prefix"]
        prefix = [p] * S if p < 16 else _spread(p // 2, p, S, 0.75)
    return lens, news, prefix


def _quantised(g, num_blocks, kv, dim):
    """An FP8 cache as it stands after writes of normal rows: codes, scales."""
    codes = torch.randn(num_blocks, BS, kv, dim, generator=g, device="cuda",
                        dtype=torch.float16).mul_(100.0).clamp_(-448.0, 448.0)
    codes = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.rand(num_blocks, BS, kv, generator=g, device="cuda").mul_(0.006).add_(0.006)
    return codes, scale


def _prepare_attention(case, seed):
    S, H, Hk, D = (case[k] for k in ("seqs", "heads", "kv_heads", "dim"))
    g = _gen(seed, 6)
    rng = np.random.default_rng([seed, 23])
    lens, news, prefix = _lens(case)
    blocks = [_cdiv(n, BS) for n in lens]
    nb = sum(blocks) + 3
    ids = rng.permutation(nb)
    tables = np.zeros((S, max(blocks)), dtype=np.int32)
    at = 0
    for i, b in enumerate(blocks):
        tables[i, :b] = ids[at:at + b]
        at += b
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    T = int(start[-1])
    slopes = None
    if case["slopes"]:
        # a geometric series over the heads, as models with such a bias have it
        slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")
    state = dict(case=case, lens=lens, news=news, prefix=prefix, num_blocks=nb,
                 scale=1.0 / math.sqrt(D),
                 q=(torch.randn(T, H, D, generator=g, device="cuda") * 2.0).half(),
                 out=torch.zeros(T, H, D, device="cuda", dtype=torch.float16),
                 tables=torch.from_numpy(tables).cuda(),
                 seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 query_start=torch.from_numpy(start).cuda(), slopes=slopes,
                 prefix_lens=torch.tensor(prefix, dtype=torch.int32, device="cuda")
                 if case["prefix"] else None)
    for name in ("k", "v"):
        if case.get("fp8"):
            state[name + "_cache"], state[name + "_scale"] = _quantised(g, nb, Hk, D)
        else:
            state[name + "_cache"] = torch.randn(nb, BS, Hk, D, generator=g, device="cuda",
                                                 dtype=torch.float16)
    if own:
        import paged_kv_cache_131_gb300 as pkv
        if case["op"] == "decode":
            n = pkv.pkv_decode_workspace_bytes(S, H, Hk, D, max(lens))
        else:
            n = pkv.pkv_chunk_workspace_bytes(S, H, Hk, D, T, max(news), max(lens))
        state["workspace"] = torch.zeros(n, device="cuda", dtype=torch.uint8)
    return state


_PREPARE = dict(resize=_prepare_resize, verify=_prepare_verify, decode=_prepare_attention,
                chunk=_prepare_attention)

# ------------------------------------------------------------------ one pass


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_resize(s):
    import paged_kv_cache_131_gb300 as pkv
    pkv.pkv_resize_sequences(s["tables"], s["seq_lens"], s["new_lens"], s["out_lens"], s["free"],
                             s["free_count"], s["out_free_count"], s["query_start"], s["slots"],
                             s["positions"], BS, s["num_blocks"])
    return _resized(s)


def _resized(s):
    return (s["tables"], s["out_lens"], s["free"], s["out_free_count"], s["query_start"],
            s["slots"], s["positions"])


def _own_verify(s):
    import paged_kv_cache_131_gb300 as pkv
    pkv.pkv_tree_verify(s["path"], s["path_lens"], s["next_tokens"], s["tokens"], s["parents"],
                        s["query_start"], s["target"], s["draft"], s["accept_u"], s["sample_u"])
    return s["path"], s["path_lens"], s["next_tokens"]


def _rules(s):
    c = s["case"]
    return dict(softcap=c["cap"], window=c["window"], slopes=s["slopes"],
                prefix_lens=s["prefix_lens"])


def _own_decode(s):
    import paged_kv_cache_131_gb300 as pkv
    c = s["case"]
    args = (s["tables"], s["seq_lens"], s["scale"], c["heads"], c["kv_heads"], c["dim"], BS,
            max(s["lens"]), s["num_blocks"], s["workspace"])
    if c["fp8"]:
        pkv.pkv_decode_attention_scored_fp8(s["out"], s["q"], s["k_cache"], s["v_cache"],
                                            s["k_scale"], s["v_scale"], *args, **_rules(s))
    else:
        pkv.pkv_decode_attention_scored(s["out"], s["q"], s["k_cache"], s["v_cache"], *args,
                                        **_rules(s))
    return s["out"]


def _own_chunk(s):
    import paged_kv_cache_131_gb300 as pkv
    c = s["case"]
    pkv.pkv_chunk_attention_scored(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"],
                                   s["seq_lens"], s["query_start"], s["scale"], c["heads"],
                                   c["kv_heads"], c["dim"], BS, max(s["news"]), max(s["lens"]),
                                   s["num_blocks"], s["workspace"], **_rules(s))
    return s["out"]


def _plain_resize(s):
    T, MB = s["slots"].numel(), s["tables"].shape[1]
    old, new = s["seq_lens"].long(), s["new_lens"].long()
    have, want = (old + BS - 1) // BS, (new + BS - 1) // BS
    seq = torch.arange(old.numel(), device="cuda")
    # blocks given back go on the free list, the first of them on top
    back = (have - want).clamp(min=0)
    R = int(back.sum())
    owner = torch.repeat_interleave(seq, back)
    rank = torch.arange(R, device="cuda")
    blk = want[owner] + rank - (back.cumsum(0) - back)[owner]
    count = s["free_count"].long()
    top = count + R
    s["free"][top - 1 - rank] = s["tables"][owner, blk]
    # blocks and tokens are granted in order while they last
    need, tokens = (want - have).clamp(min=0), (new - old).clamp(min=0)
    upto, rows = need.cumsum(0), tokens.cumsum(0)
    grant = (tokens > 0) & (rows <= T) & ((need == 0) | (upto <= top))
    take = torch.where(grant, need, 0)
    P = int(take.sum())
    owner = torch.repeat_interleave(seq, take)
    rank = torch.arange(P, device="cuda")
    blk = have[owner] + rank - (take.cumsum(0) - take)[owner]
    s["tables"][owner, blk] = s["free"][top - 1 - rank]
    s["out_lens"].copy_(torch.where(grant | (tokens == 0), new, old))
    s["out_free_count"].copy_(top - P)
    start = torch.cat([rows.new_zeros(1), rows]).clamp(max=T)
    s["query_start"].copy_(start)
    # one row per new token
    n = int(start[-1])
    owner = torch.repeat_interleave(seq, start[1:] - start[:-1])
    pos = old[owner] + torch.arange(n, device="cuda") - start[owner]
    bid = s["tables"][owner, (pos // BS).clamp(max=MB - 1)].long()
    s["slots"].fill_(-1)
    s["positions"].zero_()
    s["slots"][:n] = torch.where(grant[owner], bid * BS + pos % BS, -1)
    s["positions"][:n] = pos
    return _resized(s)


def _plain_draw(weights, u):
    """Lowest index whose running sum passes u times the sum, in 64 bits."""
    run_ = weights.double().cumsum(0)
    hit = torch.nonzero(run_ > u * run_[-1])[:, 0]
    return int(hit[0])


def _plain_verify(s):
    c = s["case"]
    Q, P = c["nodes"], s["path"].shape[1]
    parents, tokens = s["parents"].tolist(), s["tokens"].tolist()
    au, su = s["accept_u"].double().tolist(), s["sample_u"].double().tolist()
    s["path"].fill_(-1)
    for i in range(c["seqs"]):
        node, path, rest = 0, [0], None
        while len(path) < P:
            p = s["target"][i * Q + node].double()
            rest, mass, step = p, 1.0, None
            for k in range(node + 1, Q):
                if parents[i * Q + k] != node:
                    continue
                tok = tokens[i * Q + k]
                if c["drafted"]:
                    q = s["draft"][i * Q + node].double()
                    take = au[i * Q + k] * mass * float(q[tok]) < float(rest[tok])
                    left = (rest - mass * q).clamp(min=0)
                    left_mass = float(left.sum())
                else:
                    take = au[i * Q + k] * mass < float(rest[tok])
                    left = rest.clone()
                    left[tok] = 0
                    left_mass = mass - float(rest[tok])
                if take:
                    step = k
                    break
                if not left_mass > 0:
                    break
                rest, mass = left, left_mass
            if step is None:
                break
            node = step
            path.append(step)
            rest = None
        if rest is None:
            rest = s["target"][i * Q + node]
        s["path"][i, :len(path)] = torch.tensor(path, dtype=torch.int32)
        s["path_lens"][i] = len(path)
        s["next_tokens"][i] = _plain_draw(rest, su[i])
    return s["path"], s["path_lens"], s["next_tokens"]


def _plain_attention(s):
    c = s["case"]
    H, Hk, D = c["heads"], c["kv_heads"], c["dim"]
    G = H // Hk
    at = 0
    for row, (L, Q, prefix) in enumerate(zip(s["lens"], s["news"], s["prefix"])):
        ids = s["tables"][row, :_cdiv(L, BS)].long()
        kv = []
        for name in ("k", "v"):
            x = s[name + "_cache"][ids]
            if c.get("fp8"):
                x = x.view(torch.float8_e4m3fn).float() * s[name + "_scale"][ids][..., None]
            kv.append(x.flatten(0, 1)[:L].float().transpose(0, 1))  # [Hk, L, D]
        q = s["q"][at:at + Q].float().view(Q, Hk, G, D).transpose(0, 1)
        x = (q.reshape(Hk, Q * G, D) @ kv[0].transpose(1, 2)).view(Hk, Q, G, L) * s["scale"]
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        qpos = torch.arange(L - Q, L, device="cuda")[:, None]
        kpos = torch.arange(L, device="cuda")[None, :]
        sees = kpos <= qpos
        if c["window"]:
            sees = sees & (qpos - kpos < c["window"])
        sees = sees | (kpos < prefix)
        if s["slopes"] is not None:
            far = (qpos - kpos).abs().float()
            x = x - s["slopes"].view(Hk, 1, G, 1) * far[None, :, None, :]
        x = x.masked_fill(~sees[None, :, None, :], float("-inf"))
        w = torch.exp(x - x.amax(-1, keepdim=True))
        o = (w.view(Hk, Q * G, L) @ kv[1]).view(Hk, Q, G, D) / w.sum(-1, keepdim=True)
        s["out"][at:at + Q] = o.transpose(0, 1).reshape(Q, H, D)
        at += Q
    return s["out"]


_PLAIN = dict(resize=_plain_resize, verify=_plain_verify, decode=_plain_attention,
              chunk=_plain_attention)
_OWN = dict(resize=_own_resize, verify=_own_verify, decode=_own_decode, chunk=_own_chunk)

# --------------------------------------------------------------------- work


def work(case):
    """Bytes and operations a pass cannot do without."""
    op = case["op"]
    if op == "resize":
        # lengths in and out, query starts, the free list's count; a slot and a
        # position per row; a table entry read or written per block moved
        S, T = case["seqs"], case["tokens"]
        return dict(bytes=S * 16 + T * 16 + (T // BS + S // 4) * 8, flops=0)
    if op == "verify":
        # one row of the target's probabilities per sequence, and of the
        # drafter's where one was rejected; what the nodes hold
        S, Q, V = case["seqs"], case["nodes"], case["vocab"]
        rows = 2 if case["drafted"] and Q > 1 else 1
        return dict(bytes=S * (rows * V * 4 + Q * 20 + 40), flops=S * V * (2 * rows - 1))
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    W = case["window"]
    tokens = pairs = queries = 0
    for L, Q, p in zip(*_lens(case)):
        p = min(p, L)
        first = np.arange(L - Q, L)
        low = np.maximum(first - W + 1, 0) if W else np.zeros_like(first)
        # positions seen: the window's (or all) up to the token, and the prefix
        pairs += int((first + 1 - low + np.minimum(p, low) + np.maximum(p - first - 1, 0)).sum())
        a = max(L - Q - W + 1, 0) if W else 0
        tokens += L - a + min(p, a)
        queries += Q
    row = 2 * Hk * (D + 4) if case.get("fp8") else 2 * Hk * D * 2
    return dict(bytes=tokens * row + 2 * queries * H * D * 2 + tokens // 4,
                flops=4 * D * H * pairs)


# -------------------------------------------------------------------- exact


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_resize(case, s):
    """The step sequence by sequence, on the host."""
    tables = s["tables"].cpu().numpy().copy()
    free = s["free"].cpu().numpy().copy()
    old, new = s["seq_lens"].tolist(), s["new_lens"].tolist()
    T = case["tokens"]
    stack = [int(b) for b in free[:int(s["free_count"])]]
    given = []
    for i, (a, b) in enumerate(zip(old, new)):
        given += [int(tables[i, k]) for k in range(_cdiv(b, BS), _cdiv(a, BS))]
    stack += given[::-1]
    free[:len(stack)] = stack
    asked = rows = 0
    room = len(stack)
    out, start = [], [0]
    slots, positions = np.full(T, -1, dtype=np.int64), np.zeros(T, dtype=np.int64)
    for i, (a, b) in enumerate(zip(old, new)):
        blocks = max(_cdiv(b, BS) - _cdiv(a, BS), 0)
        asked += blocks
        ok = rows + max(b - a, 0) <= T and (blocks == 0 or asked <= room)
        if ok:
            for k in range(blocks):
                tables[i, _cdiv(a, BS) + k] = stack.pop()
        for pos in range(a, b):
            if rows < T:
                positions[rows] = pos
                if ok:
                    slots[rows] = int(tables[i, pos // BS]) * BS + pos % BS
            rows += 1
        start.append(min(rows, T))
        out.append(b if ok else a)
    return tuple(torch.from_numpy(np.asarray(x)).cuda() for x in (
        tables, np.array(out, np.int32), free, np.array([len(stack)], np.int32),
        np.array(start, np.int32), slots, positions))


def _exact_verify(case, s):
    """Sampling without the running residual: the residual after the siblings'
    rejections is max(p - c q, 0) with c the sum of the masses before them."""
    S, Q, V = case["seqs"], case["nodes"], case["vocab"]
    P = s["path"].shape[1]
    par = s["parents"].view(S, Q).cpu().numpy()
    tok = s["tokens"].view(S, Q).cpu().numpy()
    u = s["accept_u"].view(S, Q).cpu().numpy().astype(np.float64)
    v = s["sample_u"].cpu().numpy().astype(np.float64)
    path = np.full((S, P), -1, dtype=np.int32)
    size, drawn = np.zeros(S, np.int32), np.zeros(S, np.int32)
    for i in range(S):
        at, depth = 0, 1
        path[i, 0] = 0
        while True:
            p = s["target"][i * Q + at].double()
            q = s["draft"][i * Q + at].double() if case["drafted"] else None
            gone = torch.zeros(V, dtype=torch.bool, device="cuda")
            c, mass, onward = 0.0, 1.0, -1
            kids = np.nonzero(par[i] == at)[0] if depth < P else []
            for k in kids:
                t = int(tok[i, k])
                if case["drafted"]:
                    have = max(float(p[t]) - c * float(q[t]), 0.0)
                    if float(u[i, k]) * mass * float(q[t]) < have:
                        onward = int(k)
                        break
                    c_next = c + mass
                    mass_next = float(torch.relu(torch.addcmul(p, q, torch.full_like(q, -c_next)))
                                      .sum())
                    if mass_next <= 0:
                        break
                    c, mass = c_next, mass_next
                else:
                    have = 0.0 if bool(gone[t]) else float(p[t])
                    if float(u[i, k]) * mass < have:
                        onward = int(k)
                        break
                    if mass - have <= 0:
                        break
                    gone[t] = True
                    mass -= have
            if onward < 0:
                left = torch.relu(p - c * q) if case["drafted"] else p.masked_fill(gone, 0.0)
                total = torch.cumsum(left, 0)
                drawn[i] = int(torch.searchsorted(total, float(v[i]) * float(total[-1]),
                                                  right=True))
                break
            path[i, depth] = onward
            depth += 1
            at = onward
        size[i] = depth
    return tuple(torch.from_numpy(x).cuda() for x in (path, size, drawn))


def _e4m3_values():
    """The 256 values of the format: sign, four exponent bits (bias 7), three of mantissa."""
    vals = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        vals.append(math.nan if (c & 127) == 127 else (-v if c & 128 else v))
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _exact_attention(case, s):
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // Hk
    values = _e4m3_values() if case.get("fp8") else None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    start = s["query_start"].tolist()
    for i, L in enumerate(s["lens"]):
        a, b = start[i], start[i + 1]
        pos = torch.arange(L, device="cuda")
        mine = pos[L - (b - a):].unsqueeze(1)
        blk, off = s["tables"][i].long()[pos // BS], pos % BS
        hidden = pos > mine
        if case["window"]:
            hidden |= pos <= mine - case["window"]
        hidden &= pos >= s["prefix"][i]
        for h in range(H):
            k, v = (s[n + "_cache"][blk, off, h // G] for n in ("k", "v"))
            if values is not None:
                k = values[k.int()] * s["k_scale"][blk, off, h // G].double()[:, None]
                v = values[v.int()] * s["v_scale"][blk, off, h // G].double()[:, None]
            t = torch.einsum("qd,ld->ql", s["q"][a:b, h].double(), k.double()) * s["scale"]
            if case["cap"]:
                t = torch.tanh(t / case["cap"]) * case["cap"]
            if s["slopes"] is not None:
                t = t - float(s["slopes"][h]) * torch.abs(mine - pos)
            p = torch.softmax(t.masked_fill_(hidden, -math.inf), dim=1)
            out[a:b, h] = torch.einsum("ql,ld->qd", p, v.double())
    return out


_EXACT = dict(resize=_exact_resize, verify=_exact_verify, decode=_exact_attention,
              chunk=_exact_attention)
