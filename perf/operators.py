"""Cases for the tree-verification and cache-eviction operators.

One serving step of speculative decoding over a bounded latent cache: the
drafted tree attends the paged cache (``tree``), the attention weight each
cached key received is accumulated (``weights``), the keys to keep are chosen
(``select``) and their entries moved together (``compact``).

``run`` computes an operator in plain torch (``own`` false) or through
``head_latent_attention_qkv_gb300.api`` (``own`` true).
"""
from __future__ import annotations

import random

import torch

own = False

DEV = "cuda"
# cache entry: [latent rank | rope], query head dims behind the softmax scale
ENTRY = {"bf16": (512, 64, 128), "fp32": (64, 16, 32)}
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _attn(op, name, dtype, heads, seqs, ctx_lo, ctx_hi, nodes, page, shape="bushy", window=0,
          padded=False):
    c = {"op": op, "dtype": dtype, "heads": heads, "seqs": seqs, "ctx_lo": ctx_lo,
         "ctx_hi": ctx_hi, "nodes": nodes, "page": page, "shape": shape, "window": window,
         "padded": padded}
    if name:
        c["name"] = name
    return c


def _cache(op, name, dtype, seqs, len_lo, len_hi, budget, page, sink=0, recent=0):
    c = {"op": op, "dtype": dtype, "seqs": seqs, "len_lo": len_lo, "len_hi": len_hi,
         "budget": budget, "page": page, "sink": sink, "recent": recent}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the fp32 layer's tree: two short sequences, eight nodes
        _attn("tree", "tree_fp32_tiny", "fp32", 4, 2, 40, 64, 8, 16),
        # a 16-node draft tree of a 32-head layer over eight prefilled sequences
        _attn("tree", "tree_h32_n16_b8", "bf16", 32, 8, 2048, 2048, 16, 128),
        # plain one-token decode of a 128-head layer, one long context (the tree's smallest form)
        _attn("tree", "tree_h128_n1_long", "bf16", 128, 1, 32768, 32768, 1, 64),
        # sliding window, ragged contexts, 16-token pages, trees padded to a common node count
        _attn("tree", "tree_h32_n25_window", "bf16", 32, 5, 300, 4500, 25, 16, window=512, padded=True),
        # a batch of wide trees over long ragged contexts: the verification step that costs most
        _attn("tree", "tree_h128_n64_b4", "bf16", 128, 4, 6001, 8192, 64, 128),
        # the weight each key received in a decode step of 64 sequences
        _attn("weights", "weights_h32_n1_b64", "bf16", 32, 64, 1024, 4096, 1, 128, shape="block"),
        # the same after a block of 16 drafted tokens of a 128-head layer
        _attn("weights", "weights_h128_n16_b4", "bf16", 128, 4, 7000, 8192, 16, 128, shape="block"),
        # weights of a tree's rows, fp32 layer
        _attn("weights", "weights_fp32_tree", "fp32", 4, 3, 50, 700, 12, 16),
        # eviction of a decode batch down to 1024 keys a sequence
        _cache("select", "select_b64_to_1024", "fp32", 64, 1024, 4112, 1024, 128, 4, 64),
        # two very long contexts
        _cache("select", "select_b2_long", "fp32", 2, 120001, 131072, 8192, 64, 16, 512),
        # moving the kept entries of that decode batch into fresh pages
        _cache("compact", "compact_b64_to_1024", "bf16", 64, 1024, 4112, 1024, 128),
        # one long fp32 sequence, odd sizes
        _cache("compact", "compact_fp32_b1", "fp32", 1, 40003, 40003, 9001, 16),
    ]


def _logint(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["tree", "tree", "weights", "select", "compact"])
    if op in ("tree", "weights"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        while True:
            if dtype == "fp32":
                heads, seqs, hi = rng.randint(1, 4), rng.randint(1, 4), _logint(rng, 1, 700)
                nodes = rng.randint(1, 12)
            else:
                heads = rng.choice([1, 3, 8, 16, 20, 32, 64, 128])
                seqs, hi = _logint(rng, 1, 64), _logint(rng, 1, 32768)
                nodes = _logint(rng, 1, 64)
            lo = rng.randint(max(1, hi // 4), hi)
            window = rng.choice([0, 0, _logint(rng, 1, 2048)])
            shape = rng.choice(["bushy", "chain", "stars"] if op == "tree" else
                               ["block", "bushy", "chain"])
            c = _attn(op, None, dtype, heads, seqs, lo, hi, nodes, rng.choice([16, 64, 128]),
                      shape, window, padded=rng.random() < 0.4)
            if seqs * nodes * heads * hi <= 4 * 64 * 128 * 7000 and seqs * hi <= 300000:
                return c
    dtype = rng.choice(["bf16", "fp32"])
    while True:
        seqs, hi = _logint(rng, 1, 64), _logint(rng, 40, 131072)
        lo = rng.randint(hi // 4, hi)
        budget = _logint(rng, 16, hi - 8)
        if seqs * hi <= 300000:
            break
    if op == "select":
        sink = rng.randint(0, min(16, budget // 4))
        recent = rng.randint(0, min(512, budget // 2))
        return _cache(op, None, "fp32", seqs, lo, hi, budget, 64, sink, recent)
    return _cache(op, None, dtype, seqs, lo, hi, budget, rng.choice([16, 64, 128]))


def _lens(lo, hi, n):
    """Ragged lengths of a case, the same for every seed."""
    return [lo + (hi - lo) * ((7 * b + 3) % n) // max(n - 1, 1) for b in range(n)]


def _parents(case):
    """Parents of every sequence's nodes: -1 a child of the context, -2 padding."""
    rng = random.Random(case["nodes"] * 131 + case["seqs"])
    out = []
    for b in range(case["seqs"]):
        n, par = case["nodes"], []
        live = n if not case["padded"] else rng.randint(max(1, n // 2), n)
        for i in range(n):
            if i >= live:
                par.append(-2)
            elif i == 0 or case["shape"] == "stars":
                par.append(-1 if i < 4 else rng.randint(0, 3))
            elif case["shape"] == "chain":
                par.append(i - 1)
            else:
                par.append(rng.randint(max(-1, i - 8), i - 1))
        out.append(par)
    return out


def _depths(par):
    d = []
    for p in par:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _pairs(case):
    """Visible (query, key) pairs of one head, and the cached keys any query sees."""
    pairs = keys = 0
    W, T = case["window"], case["nodes"]
    for ctx, par in zip(_lens(case["ctx_lo"], case["ctx_hi"], case["seqs"]), _parents(case)):
        dep = _depths(par)
        reach, seen = 0, set()
        for i in range(T):
            if case["shape"] == "block":
                vis, nctx = range(T), (ctx if not W else min(ctx, max(0, W - 1 - i)))
            else:
                if par[i] < -1:
                    continue
                vis, a = [], i
                while a >= 0:
                    if not W or dep[i] - dep[a] < W:
                        vis.append(a)
                    a = par[a]
                nctx = ctx if not W else min(ctx, max(0, W - 1 - dep[i]))
            pairs += nctx + len(vis)
            reach = max(reach, nctx)
            seen.update(vis)
        keys += reach + len(seen)
    return pairs, keys


def work(case):
    r, dr, _ = ENTRY[case["dtype"]]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("tree", "weights"):
        rows = case["seqs"] * case["nodes"] * case["heads"]
        pairs, keys = _pairs(case)
        pairs *= case["heads"]
        if case["op"] == "tree":
            return {"bytes": keys * (r + dr) * e + rows * ((r + dr) * e + r * e + 4),
                    "flops": pairs * 2 * (2 * r + dr)}
        return {"bytes": keys * ((r + dr) * e + 8) + rows * ((r + dr) * e + 4),
                "flops": pairs * 2 * (r + dr)}
    lens = _lens(case["len_lo"], case["len_hi"], case["seqs"])
    kept = sum(min(n, case["budget"]) for n in lens)
    if case["op"] == "select":
        return {"bytes": 4 * (sum(lens) + kept), "flops": sum(lens)}
    return {"bytes": kept * (2 * (r + dr) * e + 12), "flops": 0}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _handle(dtype, heads, page):
    """The layer handle a serving program keeps (its projections are not used here)."""
    from head_latent_attention_qkv_gb300 import api
    from head_latent_attention_qkv_gb300.workloads import MLADims, weight_shapes
    r, dr, dn = ENTRY[dtype]
    dims = MLADims(hidden_size=64, num_heads=heads, q_lora_rank=0, kv_lora_rank=r,
                   qk_nope_head_dim=dn, qk_rope_head_dim=dr, v_head_dim=dn, rope_style="neox",
                   rope_theta=1e4, dtype=dtype, max_position=64)
    w = {k: (None if s is None else torch.zeros(s, dtype=DTYPE[dtype], device=DEV))
         for k, s in weight_shapes(dims).items()}
    return api.mla_draft_init(dims, w, page)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = random.Random(seed)
    dt = DTYPE[case["dtype"]]
    r, dr, dn = ENTRY[case["dtype"]]
    ps, n = case["page"], case["seqs"]
    st = {"case": case}
    if case["op"] in ("tree", "weights"):
        T, H = case["nodes"], case["heads"]
        ctx = _lens(case["ctx_lo"], case["ctx_hi"], n)
        par = _parents(case)
        kv = [c + T for c in ctx]
        if case["shape"] == "block":
            st["parent"] = None
            depth = [list(range(T))] * n
        else:
            st["parent"] = _int32(par).flatten()
            depth = [_depths(p) for p in par]
        st["positions"] = _int32([[c + d for d in dd] for c, dd in zip(ctx, depth)]).flatten()
        st["kv_len"] = _int32(kv)
        st["window"] = _int32([case["window"]] * n) if case["window"] else None
    else:
        kv = _lens(case["len_lo"], case["len_hi"], n)
        st["kv_len"] = _int32(kv)
    st["kv_host"] = kv
    width = st["width"] = max(kv)
    mp = (width + ps - 1) // ps
    if case["op"] != "select":
        per = [(k + ps - 1) // ps for k in kv]
        total = sum(per) + (n * ((min(case["budget"], width) + ps - 1) // ps)
                            if case["op"] == "compact" else 0)
        ids = list(range(total + 1))
        host.shuffle(ids)
        table, at = [], 0
        for p in per:
            table.append(ids[at:at + p] + [0] * (mp - p))
            at += p
        st["table"] = _int32(table)
        st["cache"] = torch.randn(total + 1, ps, r + dr, generator=g, device=DEV).to(dt)
    if case["op"] in ("tree", "weights"):
        rows = n * T * H
        st["q"] = torch.randn(rows, r + dr, generator=g, device=DEV).to(dt)
        st["scale"] = 1.0 / (dn + dr) ** 0.5
        if case["op"] == "weights":
            st["prior"] = torch.rand(n, mp * ps, generator=g, device=DEV) * 4
            st["out"] = torch.zeros_like(st["prior"])
            st["lse"] = _softmax(_scores(st)[0])[1]
    else:
        if case["op"] == "select":
            # a few heavy keys, many light ones, a tenth that no query ever looked at
            w = torch.randn(n, width, generator=g, device=DEV).mul_(2).exp_()
            w *= torch.rand(n, width, generator=g, device=DEV) > 0.1
            st["weights"] = w
        else:
            m = min(case["budget"], width)
            mpd = (m + ps - 1) // ps
            st["dst"] = _int32([ids[at + b * mpd:at + (b + 1) * mpd] for b in range(n)])
            keep = torch.zeros(n, m, dtype=torch.int32)
            for b, k in enumerate(kv):
                pick = sorted(host.sample(range(k), min(m, k)))
                keep[b, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
            st["keep"] = keep.to(DEV)
            st["keep_len"] = _int32([min(m, k) for k in kv])
            st["weights"] = torch.rand(n, width, generator=g, device=DEV)
            st["weights_out"] = torch.full((n, width), -1.0, device=DEV)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from head_latent_attention_qkv_gb300 import api
        st["handle"] = _handle(case["dtype"], case.get("heads", 1), case["page"])
        if "q" in st:
            st["desc"] = api.make_desc(st["table"], st["kv_len"], st["window"], None, case["nodes"])
    return st


# --------------------------------------------------------------------------
# plain form
# --------------------------------------------------------------------------
def _slots(st, table, j):
    """Cache rows of logical keys j [seqs, n] through a page table."""
    ps = st["case"]["page"]
    return table.long().gather(1, j // ps) * ps + j % ps


def _visible(st):
    """[seqs, nodes, keys]: which keys each query sees."""
    T, n = st["case"]["nodes"], st["case"]["seqs"]
    j = torch.arange(st["width"], device=DEV)[None, :]
    kv = st["kv_len"].long()[:, None]
    k = j - (kv - T)                                      # node whose own key j is
    node = k.clamp(0, T - 1)[:, None, :].expand(n, T, -1)
    pos = st["positions"].view(n, T)
    vis = (j < kv)[:, None, :].expand(n, T, -1)
    key_pos = j
    if st["parent"] is not None:
        par = st["parent"].view(n, T).long()
        anc = torch.nn.functional.one_hot(par.clamp(min=0), T).float() * (par >= 0)[:, :, None]
        anc = anc + torch.eye(T, device=DEV)
        for _ in range(T.bit_length()):
            anc = ((anc @ anc) > 0).float()
        in_tree = (anc @ (par < -1).float()[:, :, None]) == 0
        vis = vis & in_tree & ((k < 0)[:, None, :] | (anc.gather(2, node) > 0))
        key_pos = torch.where(k < 0, j, pos.long().gather(1, node[:, 0]))
    if st["window"] is not None:
        vis = vis & (pos[:, :, None] - key_pos[:, None, :] < st["window"][:, None, None])
    return vis


def _entries(st):
    j = torch.arange(st["width"], device=DEV)[None, :].expand(st["case"]["seqs"], -1)
    return st["cache"].flatten(0, 1)[_slots(st, st["table"], j)].float()


def _scores(st):
    """[seqs, nodes * heads, keys] scaled scores, -inf where not seen, and the entries."""
    n, H = st["case"]["seqs"], st["case"]["heads"]
    e = _entries(st)
    s = (st["q"].view(n, -1, e.shape[2]).float() @ e.transpose(1, 2)) * st["scale"]
    s = s.masked_fill(~_visible(st).repeat_interleave(H, 1), float("-inf"))
    return s, e


def _softmax(s):
    """Weights of the rows (0 for a row that sees nothing) and their log-sum-exp."""
    m = s.max(2, keepdim=True).values.clamp(min=-3e38)
    p = (s - m).exp()
    l = p.sum(2, keepdim=True)
    return p / l.clamp(min=1e-30), (m + l.log()).flatten()


def _plain(st):
    c = st["case"]
    r = ENTRY[c["dtype"]][0]
    n = c["seqs"]
    if c["op"] == "tree":
        s, e = _scores(st)
        p, lse = _softmax(s)
        o = (p @ e[:, :, :r]).flatten(0, 1)
        return o.to(torch.float16 if c["dtype"] == "bf16" else torch.float32), lse
    j = torch.arange(st["width"], device=DEV)[None, :]
    live = j < st["kv_len"][:, None]
    if c["op"] == "weights":
        lse = st["lse"].view(n, -1, 1)
        p = torch.where(torch.isinf(lse), 0.0, (_scores(st)[0] - lse).exp())
        out = st["out"][:, :st["width"]]
        out.copy_(torch.where(live, 0.5 * st["prior"][:, :st["width"]] + p.sum(1), out))
        return st["out"]
    if c["op"] == "select":
        m = min(c["budget"], st["width"])
        w = st["weights"].masked_fill(~live, float("-inf"))
        w = w.masked_fill((j < c["sink"]) & live, float("inf"))
        w = w.masked_fill((j >= st["kv_len"][:, None] - c["recent"]) & live, float("inf"))
        best = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :m]
        count = st["kv_len"].clamp(max=c["budget"])
        dead = torch.arange(m, device=DEV)[None, :] >= count[:, None]
        best = best.masked_fill(dead, st["width"]).sort(dim=1).values
        keep = torch.full((n, c["budget"]), -1, dtype=torch.int32, device=DEV)
        keep[:, :m] = best.masked_fill(dead, -1)
        return keep, count
    d = torch.arange(st["keep"].shape[1], device=DEV)[None, :].expand(n, -1)
    kept = d < st["keep_len"][:, None]
    src = st["keep"].long()
    flat = st["cache"].flatten(0, 1)
    flat[_slots(st, st["dst"], d)[kept]] = flat[_slots(st, st["table"], src)[kept]]
    w = st["weights_out"]
    w.masked_fill_(live, 0.0)
    w[:, :d.shape[1]] = torch.where(kept, st["weights"].gather(1, src), w[:, :d.shape[1]])
    return st["cache"], w


def run(st):
    if not own:
        return _plain(st)
    from head_latent_attention_qkv_gb300 import api
    c, h = st["case"], st["handle"]
    if c["op"] == "tree":
        lse = torch.empty(st["q"].shape[0], device=DEV)
        o = api.mla_tree_attention(h, st["q"], st["positions"], st["cache"], st["desc"],
                                   st["parent"], lse=lse)
        return o, lse
    if c["op"] == "weights":
        return api.mla_key_weights(h, st["q"], st["positions"], st["cache"], st["desc"], st["lse"],
                                   st["out"], prior=st["prior"], decay=0.5, parent=st["parent"])
    if c["op"] == "select":
        return api.mla_cache_select(h, st["weights"], st["kv_len"], c["budget"], sink=c["sink"],
                                    recent=c["recent"])
    api.mla_cache_compact(h, st["cache"], st["table"], st["kv_len"], st["keep"], st["keep_len"],
                          dst_block_table=st["dst"], weights=st["weights"],
                          weights_out=st["weights_out"])
    return st["cache"], st["weights_out"]


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] in ("select", "compact"):
        return None                     # whole numbers and moved entries: nothing is computed
    T, H, ps = case["nodes"], case["heads"], case["page"]
    r = ENTRY[case["dtype"]][0]
    parents, W = _parents(case), case["window"]
    pos, table = st["positions"].tolist(), st["table"].tolist()
    outs, lses = [], []
    result = st["out"].double() if case["op"] == "weights" else None
    for b, n in enumerate(st["kv_host"]):
        ctx = n - T
        pages = torch.tensor(table[b][:(n + ps - 1) // ps], device=DEV)
        e = st["cache"][pages].reshape(-1, st["cache"].shape[2])[:n].double()
        total = torch.zeros(n, dtype=torch.float64, device=DEV)
        for i in range(T):
            row = b * T + i
            seen, a, ok = [], i, True
            if st["parent"] is None:
                seen = [k for k in range(T) if not W or pos[row] - (ctx + k) < W]
            else:
                while a >= 0:
                    if not W or pos[row] - pos[b * T + a] < W:
                        seen.append(a)
                    a = parents[b][a]
                ok = a == -1
            lo = max(0, pos[row] - W + 1) if W else 0
            cols = torch.cat([torch.arange(min(lo, ctx), ctx, device=DEV),
                              torch.tensor([ctx + k for k in sorted(seen)], dtype=torch.long, device=DEV)])
            cols = cols if ok else cols[:0]
            x = st["q"][row * H:(row + 1) * H].double()
            z = x @ e[cols].T * st["scale"]
            if case["op"] == "weights":
                if len(cols):
                    total[cols] += torch.exp(z - st["lse"][row * H:(row + 1) * H, None].double()).sum(0)
                continue
            lse = torch.logsumexp(z, 1)
            outs.append(torch.exp(z - lse[:, None]) @ e[cols, :r])
            lses.append(lse)
        if result is not None:
            result[b, :n] = 0.5 * st["prior"][b, :n].double() + total
    if result is not None:
        return result
    return torch.cat(outs), torch.cat(lses)
