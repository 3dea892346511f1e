"""Cases for the 8-bit latent cache and the verification of drafted tokens.

A serving program whose context outgrows its memory keeps the latent cache in 8
bits: entries are quantised as they are written (``store``), attended where they
lie (``attend``, split over a long context and joined), and read back for the
paths that want bf16 entries (``load``).  The tokens that the layer drafted are
then held against the target's probabilities (``verify``).

An 8-bit entry is 512 latent dims in e4m3 over one power of two a token, and 64
rotary dims in bf16.  ``run`` computes an operator in plain torch (``own`` false)
or through ``head_latent_attention_qkv_gb300.api`` (``own`` true).
"""
from __future__ import annotations

import random

import torch

own = False

DEV = "cuda"
R, DR, DN = 512, 64, 128        # latent dims, rotary dims, query head dims behind the softmax scale
L = R + DR
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
PROB = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _rows(op, name, tokens, page):
    c = {"op": op, "tokens": tokens, "page": page}
    return {**c, "name": name} if name else c


def _attend(name, heads, seqs, ctx_lo, ctx_hi, nodes, page, shape="block", window=0):
    c = {"op": "attend", "heads": heads, "seqs": seqs, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
         "nodes": nodes, "page": page, "shape": shape, "window": window}
    return {**c, "name": name} if name else c


def _verify(name, seqs, nodes, vocab, dtype, shape="chain", draft="drawn"):
    c = {"op": "verify", "seqs": seqs, "nodes": nodes, "vocab": vocab, "dtype": dtype,
         "shape": shape, "draft": draft}
    return {**c, "name": name} if name else c


def listed():
    return [
        # a decode step of 64 sequences writes one entry each
        _rows("store", "store_64", 64, 128),
        # a prefilled batch of contexts, an odd count on small pages
        _rows("store", "store_130k", 130001, 16),
        # one short sequence's entries wanted in bf16
        _rows("load", "load_700", 700, 16),
        # four contexts of 16 k read back for the expanded form
        _rows("load", "load_64k", 65536, 128),
        # one new token of a 16-head layer over a short context: latency alone
        _attend("attend_h16_n1_b1", 16, 1, 300, 300, 1, 128),
        # one new token of 64 sequences of a 32-head layer
        _attend("attend_h32_n1_b64", 32, 64, 1024, 4096, 1, 128),
        # one new token of a 128-head layer, one long context
        _attend("attend_h128_n1_long", 128, 1, 131072, 131072, 1, 64),
        # a padded tree of drafted tokens behind a sliding window, 16-token pages
        _attend("attend_h32_n25_window", 32, 5, 300, 4500, 25, 16, shape="tree", window=512),
        # a block of 16 drafted tokens of a 128-head layer over ragged contexts
        _attend("attend_h128_n16_b4", 128, 4, 7000, 8192, 16, 128),
        # one sequence's chain of five drafted tokens, a small vocabulary
        _verify("verify_chain_b1", 1, 5, 32000, "fp32"),
        # chains of a block's 15 drafted tokens, 64 sequences, a large vocabulary
        _verify("verify_chain_b64", 64, 15, 151936, "fp32"),
        # trees, bf16 probabilities
        _verify("verify_tree_b8", 8, 32, 129280, "bf16", shape="tree"),
    ]


def _logint(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["store", "load", "attend", "attend", "attend", "verify", "verify"])
    if op in ("store", "load"):
        return _rows(op, None, _logint(rng, 1, 130001), rng.choice([16, 32, 64, 128, 256]))
    if op == "attend":
        while True:
            heads = rng.choice([1, 3, 8, 16, 20, 32, 64, 128])
            seqs, hi, nodes = _logint(rng, 1, 64), _logint(rng, 1, 131072), _logint(rng, 1, 40)
            lo = rng.randint(max(1, hi // 4), hi)
            window = rng.choice([0, 0, 0, _logint(rng, 1, 2048)])
            c = _attend(None, heads, seqs, lo, hi, nodes, rng.choice([16, 64, 128, 256]),
                        rng.choice(["block", "block", "tree", "chain"]), window)
            if seqs * nodes * heads * hi <= 4 * 16 * 128 * 8192 and seqs * hi <= 300000:
                return c
    while True:
        c = _verify(None, _logint(rng, 1, 64), _logint(rng, 1, 40), _logint(rng, 100, 152000),
                    rng.choice(["fp32", "fp32", "bf16", "fp16"]), rng.choice(["chain", "tree"]),
                    rng.choice(["drawn", "drawn", "certain"]))
        if c["seqs"] * (c["nodes"] + 1) * c["vocab"] <= 64 * 16 * 151936:
            return c


def _lens(case):
    """Ragged context lengths of a case, the same for every seed."""
    lo, hi, n = case["ctx_lo"], case["ctx_hi"], case["seqs"]
    return [lo + (hi - lo) * ((7 * b + 3) % n) // max(n - 1, 1) for b in range(n)]


def _parents(case):
    """Parents of every sequence's nodes: -1 a child of the context, -2 padding."""
    rng = random.Random(case["nodes"] * 137 + case["seqs"])
    out = []
    for _ in range(case["seqs"]):
        n = case["nodes"]
        if case["shape"] != "tree":
            out.append([i - 1 for i in range(n)])
            continue
        live = rng.randint(max(1, n // 2), n)
        out.append([(-1 if i == 0 else rng.randint(max(-1, i - 5), i - 1)) if i < live else -2
                    for i in range(n)])
    return out


def _depths(par):
    d = []
    for p in par:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _seen(case, par, ctx):
    """Per node the own keys (node indices) and the first context key that it sees."""
    W, dep, out = case["window"], _depths(par), []
    for i in range(case["nodes"]):
        if case["shape"] == "block":
            nodes = [k for k in range(case["nodes"]) if not W or i - k < W]
            out.append((nodes, min(ctx, max(0, ctx + i - W + 1)) if W else 0))
            continue
        nodes, a = [], i
        while a >= 0:
            if not W or dep[i] - dep[a] < W:
                nodes.append(a)
            a = par[a]
        if a < -1:
            out.append(([], ctx))
        else:
            out.append((sorted(nodes), min(ctx, max(0, ctx + dep[i] - W + 1)) if W else 0))
    return out


def work(case):
    entry = R + 2 * DR + 4
    if case["op"] in ("store", "load"):
        return {"bytes": case["tokens"] * (entry + 2 * L + 8), "flops": 0}
    if case["op"] == "attend":
        pairs = keys = 0
        for ctx, par in zip(_lens(case), _parents(case)):
            seen = _seen(case, par, ctx)
            pairs += sum(len(n) + ctx - lo for n, lo in seen)
            keys += ctx - min(lo for _, lo in seen) + len(set().union(*(set(n) for n, _ in seen)))
        rows = case["seqs"] * case["nodes"] * case["heads"]
        return {"bytes": keys * entry + rows * (2 * L + 2 * R + 4),
                "flops": pairs * case["heads"] * 2 * (L + R)}
    e = 4 if case["dtype"] == "fp32" else 2
    rows = 2 if case["draft"] == "drawn" else 1     # the node at which a sequence stops
    return {"bytes": case["seqs"] * (rows * case["vocab"] * e + case["nodes"] * (12 + 2 * e)),
            "flops": 3 * case["seqs"] * case["vocab"]}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _handle(heads, page):
    """The layer handle a serving program keeps (its projections are not used here)."""
    from head_latent_attention_qkv_gb300 import api
    from head_latent_attention_qkv_gb300.workloads import MLADims, weight_shapes
    dims = MLADims(hidden_size=64, num_heads=heads, q_lora_rank=0, kv_lora_rank=R,
                   qk_nope_head_dim=DN, qk_rope_head_dim=DR, v_head_dim=DN, rope_style="neox",
                   rope_theta=1e4, dtype="bf16", max_position=64)
    w = {k: (None if s is None else torch.zeros(s, dtype=torch.bfloat16, device=DEV))
         for k, s in weight_shapes(dims).items()}
    return api.mla_draft_init(dims, w, page)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _entries(n, g):
    """Entries as the layer writes them: a normalised latent under its gains, and rotated
    keys of another size."""
    e = torch.randn(n, L, generator=g, device=DEV)
    e[:, :R] *= 1.0 + 0.3 * torch.randn(R, generator=g, device=DEV)
    e[:, R:] *= 2.5
    return e.bfloat16()


def _quantise(entries):
    """Entries [n, 576] bf16 to (e4m3 [n, 512], bf16 [n, 64], scale [n]): the scale is the
    least power of two that brings the latent's largest element to at most 448."""
    x = entries[:, :R].float()
    m, ex = torch.frexp(x.abs().amax(1))             # amax = m 2^ex, m in [1/2, 1); 448 = (7/8) 2^9
    k = (ex - 9 + (m > 0.875).int()).clamp(min=-64)
    k = torch.where(m > 0, k, torch.full_like(k, -64))
    scale = torch.ldexp(torch.ones_like(m), k)
    return (x / scale[:, None]).to(F8), entries[:, R:], scale


def _empty_cache(pages, page):
    return {"latent": torch.zeros(pages, page, R, dtype=torch.uint8, device=DEV).view(F8),
            "rope": torch.zeros(pages, page, DR, dtype=torch.bfloat16, device=DEV),
            "scale": torch.ones(pages, page, device=DEV)}


def _write(cache, slots, q8, rope, scale):
    cache["latent"].view(torch.uint8).view(-1, R)[slots] = q8.view(torch.uint8)
    cache["rope"].view(-1, DR)[slots] = rope
    cache["scale"].view(-1)[slots] = scale


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = random.Random(seed)
    st = {"case": case}
    if case["op"] in ("store", "load"):
        n, ps = case["tokens"], case["page"]
        pages = (n + ps - 1) // ps + 1
        order = list(range(pages))
        host.shuffle(order)
        t = torch.arange(n, device=DEV)
        st["slots"] = torch.tensor(order, device=DEV)[t // ps] * ps + t % ps
        st["cache"] = _empty_cache(pages, ps)
        st["entries"] = _entries(n, g)
        if case["op"] == "load":
            _write(st["cache"], st["slots"], *_quantise(st["entries"]))
            st["entries"] = torch.zeros_like(st["entries"])
        return st
    par = _parents(case)
    if case["op"] == "attend":
        T, H, ps, n = case["nodes"], case["heads"], case["page"], case["seqs"]
        ctx = _lens(case)
        kv = [c + T for c in ctx]
        per = [(k + ps - 1) // ps for k in kv]
        ids = list(range(sum(per) + 1))
        host.shuffle(ids)
        table, at = [], 0
        for p in per:
            table.append(ids[at:at + p] + [0] * (max(per) - p))
            at += p
        st["kv_host"], st["table_host"], st["width"] = kv, table, max(kv)
        st["table"], st["kv_len"] = _int32(table), _int32(kv)
        st["cache"] = _empty_cache(len(ids), ps)
        for p in range(0, len(ids) * ps, 1 << 18):
            at = torch.arange(p, min(p + (1 << 18), len(ids) * ps), device=DEV)
            _write(st["cache"], at, *_quantise(_entries(len(at), g)))
        block = case["shape"] == "block"
        depth = [list(range(T)) if block else _depths(p) for p in par]
        st["parent"] = None if block else _int32(par).flatten()
        st["positions"] = _int32([[c + d for d in dd] for c, dd in zip(ctx, depth)]).flatten()
        st["window"] = _int32([case["window"]] * n) if case["window"] else None
        st["q"] = torch.randn(n * T * H, L, generator=g, device=DEV).bfloat16()
        st["scale"] = 1.0 / (DN + DR) ** 0.5
        return st
    # verify: the draft's logits follow the target's, from which its tokens are drawn
    n, T, V, dt = case["seqs"], case["nodes"], case["vocab"], PROB[case["dtype"]]
    st["target"] = torch.empty(n, T + 1, V, dtype=dt, device=DEV)
    st["draft"] = torch.empty(n, T, V, dtype=dt, device=DEV) if case["draft"] == "drawn" else None
    st["parent"] = _int32(par)
    tokens = torch.zeros(n, T, dtype=torch.long, device=DEV)
    for b in range(n):
        z = torch.randn(T + 1, V, generator=g, device=DEV) * 2.5
        st["target"][b] = torch.softmax(z, 1).to(dt)
        q = torch.softmax(z[:T] + 0.4 * torch.randn(T, V, generator=g, device=DEV), 1).to(dt)
        if st["draft"] is not None:
            st["draft"][b] = q
        rows = (st["parent"][b].long() + 1).clamp(min=0)
        if case["draft"] == "drawn":
            tokens[b] = torch.multinomial(q.float()[rows], 1, generator=g)[:, 0]
        else:                                        # the draft's likeliest tokens, one a sibling
            rank, count = [], {}
            for p in par[b]:
                rank.append(count.get(p, 0))
                count[p] = rank[-1] + 1
            k = min(V, max(rank) + 1)
            top = q.float()[rows].topk(k, dim=1).indices
            tokens[b] = top.gather(1, torch.tensor(rank, device=DEV).clamp(max=k - 1)[:, None])[:, 0]
    st["tokens"] = tokens.int()
    st["uniforms"] = torch.rand(n, T + 1, generator=g, device=DEV)
    st["first"] = _int32([1000 + 17 * b for b in range(n)])
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from head_latent_attention_qkv_gb300 import api
        st["handle"] = _handle(case.get("heads", 1), case.get("page", 64))
        if "cache" in st:
            st["cache8"] = api.Cache8(**st["cache"])
        if case["op"] == "attend":
            st["desc"] = api.make_desc(st["table"], st["kv_len"], st["window"], None, case["nodes"])
    return st


# --------------------------------------------------------------------------
# plain form
# --------------------------------------------------------------------------
def _visible(st, b):
    """[nodes, keys of sequence b]: which keys each query sees."""
    T, n = st["case"]["nodes"], st["kv_host"][b]
    j = torch.arange(n, device=DEV)
    pos = st["positions"].view(-1, T)[b].long()
    vis = torch.ones(T, n, dtype=torch.bool, device=DEV)
    key_pos = j
    if st["parent"] is not None:
        par = st["parent"].view(-1, T)[b].long()
        anc = (torch.arange(T, device=DEV)[None, :] == par[:, None]).float() + torch.eye(T, device=DEV)
        for _ in range(T.bit_length()):
            anc = ((anc @ anc) > 0).float()
        in_tree = (anc @ (par < -1).float()) == 0
        vis[:, n - T:] = anc > 0
        vis &= in_tree[:, None]
        key_pos = torch.cat([j[:n - T], pos])
    if st["window"] is not None:
        vis &= pos[:, None] - key_pos[None, :] < st["window"][b]
    return vis


def _dequantised(st, b):
    ps, n = st["case"]["page"], st["kv_host"][b]
    j = torch.arange(n, device=DEV)
    slots = st["table"][b].long()[j // ps] * ps + j % ps
    c = st["cache"]
    lat = c["latent"].view(torch.uint8).view(-1, R)[slots].view(F8).float()
    return torch.cat([lat * c["scale"].view(-1)[slots][:, None], c["rope"].view(-1, DR)[slots].float()], 1)


def _plain_attend(st):
    T, H = st["case"]["nodes"], st["case"]["heads"]
    outs, lses = [], []
    for b in range(st["case"]["seqs"]):
        e = _dequantised(st, b)
        q = st["q"][b * T * H:(b + 1) * T * H].float()
        vis = _visible(st, b).repeat_interleave(H, 0)
        s = ((q @ e.T) * st["scale"]).masked_fill(~vis, float("-inf"))
        m = s.amax(1, keepdim=True).clamp(min=-3e38)
        p = (s - m).exp()
        l = p.sum(1, keepdim=True)
        outs.append((p @ e[:, :R]) / l.clamp(min=1e-30))
        lses.append((m + l.log())[:, 0])
    return torch.cat(outs).half(), torch.cat(lses)


def _plain_verify(st):
    """Nodes in their order: a node whose parent is where its sequence stands is taken when
    u s q(x) < w(x), w the target's row there with the mass s that earlier siblings left of it."""
    n, T = st["tokens"].shape
    seq = torch.arange(n, device=DEV)
    cur = torch.full((n,), -1, dtype=torch.long, device=DEV)
    count = torch.zeros(n, dtype=torch.long, device=DEV)
    path = torch.full((n, T), -1, dtype=torch.int32, device=DEV)
    w, s = st["target"][:, 0].double(), torch.ones(n, dtype=torch.float64, device=DEV)
    for i in range(T):
        x, u = st["tokens"][:, i].long(), st["uniforms"][:, i].double()
        here = st["parent"][:, i] == cur
        if st["draft"] is None:
            qx = torch.ones_like(s)
        else:
            q = st["draft"][seq, cur + 1].double()
            qx = q[seq, x]
        take = here & (u * s * qx < w[seq, x])
        drop = here & ~take
        if st["draft"] is None:
            left = s - w[seq, x]
            rest = w.clone()
            rest[seq, x] = 0.0
        else:
            rest = (w - s[:, None] * q).clamp(min=0.0)
            left = rest.sum(1)
        w = torch.where(drop[:, None], rest, w)
        s = torch.where(drop, left, s)
        path[seq, count.clamp(max=T - 1)] = torch.where(
            take, st["first"] + i, path[seq, count.clamp(max=T - 1)])
        count += take
        cur = torch.where(take, torch.full_like(cur, i), cur)
        w = torch.where(take[:, None], st["target"][:, i + 1].double(), w)
        s = torch.where(take, torch.ones_like(s), s)
    row = st["target"][seq, cur + 1].double()
    w = torch.where((w.sum(1) > 0)[:, None], w, row)          # nothing left: the target's own row
    c = w.cumsum(1)
    goal = st["uniforms"][:, T].double() * c[:, -1]
    token = (c <= goal[:, None]).sum(1)
    return path, count.int(), token.int()


def _plain(st):
    op, c = st["case"]["op"], st.get("cache")
    if op == "store":
        _write(c, st["slots"], *_quantise(st["entries"]))
        return c["latent"], c["rope"], c["scale"]
    if op == "load":
        lat = c["latent"].view(torch.uint8).view(-1, R)[st["slots"]].view(F8).float()
        lat = lat * c["scale"].view(-1)[st["slots"]][:, None]
        st["entries"].copy_(torch.cat([lat.bfloat16(), c["rope"].view(-1, DR)[st["slots"]]], 1))
        return st["entries"]
    return _plain_attend(st) if op == "attend" else _plain_verify(st)


def run(st):
    if not own:
        return _plain(st)
    from head_latent_attention_qkv_gb300 import api
    op, h = st["case"]["op"], st["handle"]
    if op == "store":
        api.mla_cache8_store(h, st["entries"], st["slots"], st["cache8"])
        return tuple(st["cache8"])
    if op == "load":
        return api.mla_cache8_load(h, st["cache8"], st["slots"], out=st["entries"])
    if op == "attend":
        lse = torch.empty(st["q"].shape[0], device=DEV)
        o = api.mla_latent_attention8(h, st["q"], st["positions"], st["cache8"], st["desc"],
                                      parent=st["parent"], lse=lse)
        return o, lse
    return api.mla_verify_drafts(h, st["target"], st["draft"], st["tokens"], st["uniforms"],
                                 parent=st["parent"], first=st["first"])


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "verify":
        return None                     # whole numbers
    st = _inputs(case, seed)
    c = st["cache"]
    if case["op"] == "store":
        x, s = st["entries"].double(), st["slots"]
        big = x[:, :R].abs().amax(1)
        k = torch.ceil(torch.log2(big.clamp(min=2.0 ** -64) / F8_MAX)).clamp(min=-64)
        k = k + (big > F8_MAX * 2.0 ** k).double()           # log2's own rounding, either way
        k = k - ((big <= F8_MAX * 2.0 ** (k - 1)) & (k > -64)).double()
        lat, rope = torch.zeros(c["scale"].numel(), R, device=DEV).double(), c["rope"].double().view(-1, DR)
        scale = c["scale"].double().view(-1)
        lat[s], rope[s], scale[s] = x[:, :R] / (2.0 ** k)[:, None], x[:, R:], 2.0 ** k
        return lat.view(c["latent"].shape), rope.view(c["rope"].shape), scale.view(c["scale"].shape)
    if case["op"] == "load":
        lat = c["latent"].double().view(-1, R) * c["scale"].double().view(-1, 1)
        return torch.cat([lat, c["rope"].double().view(-1, DR)], 1)[st["slots"]]
    T, H, ps = case["nodes"], case["heads"], case["page"]
    outs, lses = [], []
    for b, (par, ctx) in enumerate(zip(_parents(case), _lens(case))):
        n = ctx + T
        pages = torch.tensor(st["table_host"][b][:(n + ps - 1) // ps], device=DEV)
        lat = c["latent"].view(torch.uint8)[pages].view(F8).double()
        lat = (lat * c["scale"][pages].double()[:, :, None]).reshape(-1, R)[:n]
        e = torch.cat([lat, c["rope"][pages].reshape(-1, DR)[:n].double()], 1)
        for i, (nodes, lo) in enumerate(_seen(case, par, ctx)):
            at = (b * T + i) * H
            cols = torch.tensor([ctx + k for k in nodes], dtype=torch.long, device=DEV)
            x = st["q"][at:at + H].double()
            z = torch.cat([x @ e[lo:ctx].T, x @ e[cols].T], 1) * st["scale"]
            lse = torch.logsumexp(z, 1)
            p = torch.exp(z - lse[:, None])
            outs.append(p[:, :ctx - lo] @ e[lo:ctx, :R] + p[:, ctx - lo:] @ e[cols, :R])
            lses.append(lse)
    return torch.cat(outs), torch.cat(lses)
