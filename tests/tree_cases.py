"""Inputs of the tree and eviction tests: a handle, a paged cache, trees."""
import numpy as np
import torch

from head_latent_attention_qkv_gb300 import api, workloads as W

DEV = "cuda"


def dims_for(dtype, heads, **kw):
    base = W.TINY_FP32_MLA if dtype == "fp32" else W.QWEN3_4B_MLA
    return base.replace(num_heads=heads, hidden_size=256, q_lora_rank=0, max_position=8192, **kw)


def make_handle(dtype, heads, page, **kw):
    d = dims_for(dtype, heads, **kw)
    rng = np.random.default_rng(7)
    w = W.make_weights(d, rng)
    dt = api.torch_dtype(d)
    dev = {k: torch.from_numpy(v).to(dt).to(DEV) for k, v in w.items() if v is not None}
    return api.mla_draft_init(d, dev, page), w


def bushy(rng, T, live=None):
    live = T if live is None else live
    return [(-1 if i == 0 else int(rng.integers(max(-1, i - 6), i))) if i < live else -2 for i in range(T)]


def depths(parent):
    d = []
    for p in parent:
        d.append(d[p] + 1 if 0 <= p < len(d) else 0)
    return d


class Paged:
    """Sequences of the given key counts on shuffled pages; unused rows hold NaN."""

    def __init__(self, rng, dims, page, lens, spare=3):
        self.page, self.lens, self.dims = page, list(lens), dims
        per = [-(-n // page) for n in lens]
        ids = rng.permutation(sum(per) + spare)
        self.max_pages = max(max(per), 1)
        table = np.full((len(lens), self.max_pages), -1, dtype=np.int32)
        at = 0
        for b, p in enumerate(per):
            table[b, :p] = ids[at:at + p]
            at += p
        self.table, self.spare = table, ids[at:]
        self.num_pages = sum(per) + spare
        dt = api.torch_dtype(dims)
        flat = torch.full((self.num_pages * page, dims.cache_dim), float("nan"), dtype=dt)
        self.entries = []
        for b, n in enumerate(lens):
            e = torch.from_numpy(rng.normal(size=(n, dims.cache_dim)).astype(np.float32)).to(dt)
            self.entries.append(e.double().numpy())
            flat[self.slots(b, n)] = e
        self.cache = flat.view(self.num_pages, page, dims.cache_dim).to(DEV)

    def slots(self, b, n, table=None):
        j = np.arange(n)
        t = self.table if table is None else table
        return torch.from_numpy(t[b][j // self.page].astype(np.int64) * self.page + j % self.page)

    def set_nan(self, b, keys):
        self.cache.view(-1, self.dims.cache_dim)[self.slots(b, self.lens[b])[keys].to(DEV)] = float("nan")


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV).contiguous()
