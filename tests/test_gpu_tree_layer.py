"""The layer over trees where its attention's key ranges are cut in parts (needs a
GB300): what the call leaves in its workspace against the attention alone, bit
for bit, and the projections behind it from there in fp64.

Bounds: a projection sums K products in fp32, at most (K + 4) 2^-24 of the sum
of their sizes off, and rounds once: o to fp16 (2^-11 of the value, 2^-25 below
its normal range), the output to bf16 (2^-8); fp32 layers round to fp32.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Layer:
    """Sequences of random entries and trees whose own entries the call writes."""

    def __init__(self, dtype, heads, ctx, T, page=128, window=0, masked=False, seed=0):
        from head_latent_attention_qkv_gb300 import api
        from tests.tree_cases import Paged, bushy, depths, i32, make_handle
        rng = np.random.default_rng(seed)
        self.h, self.w = make_handle(dtype, heads, page)
        self.d, self.T, self.n, self.H = self.h.dims, T, len(ctx), heads
        dt = api.torch_dtype(self.d)
        p = self.paged = Paged(rng, self.d, page, [c + T for c in ctx])
        parents = [bushy(rng, T, int(rng.integers(max(1, T // 2), T + 1))) for _ in ctx]
        self.parent = i32(np.concatenate(parents))
        self.positions = i32(np.concatenate([c + np.asarray(depths(x)) for c, x in zip(ctx, parents)]))
        j = [c + np.arange(T) for c in ctx]
        self.slots = torch.from_numpy(np.concatenate([
            p.table[b][x // page].astype(np.int64) * page + x % page for b, x in enumerate(j)])).cuda()
        self.hidden = torch.from_numpy(rng.normal(size=(self.n * T, self.d.hidden_size)).astype(np.float32)).to(dt).cuda()
        qv = np.ones((self.n, T), dtype=np.uint8)
        if masked:
            qv[:, :max(1, T // 3)] = 0
        self.keep = [i32(p.table), i32([c + T for c in ctx]), i32([window] * self.n) if window else None,
                     torch.from_numpy(qv.reshape(-1)).cuda() if masked else None]
        self.desc = api.make_desc(*self.keep, T)
        self.ws = torch.full((api.mla_forward_tree_workspace_bytes(self.h, self.desc),), 0xff, dtype=torch.uint8,
                             device="cuda")

    def part(self, part, cols, dt):
        from head_latent_attention_qkv_gb300 import api
        at, rows = api.mla_forward_workspace_offset(self.h, self.n * self.T, part), self.n * self.T * self.H
        size = rows * cols * torch.empty(0, dtype=dt).element_size()
        assert at + size <= self.ws.numel()
        return self.ws[at:at + size].view(dt).view(rows, cols)

    def forward(self, out=None):
        from head_latent_attention_qkv_gb300 import api
        return api.mla_draft_forward_tree(self.h, self.hidden, self.positions, self.slots, self.paged.cache, self.desc,
                                          self.parent, out=out, workspace=self.ws)

    def parts(self):
        from head_latent_attention_qkv_gb300 import _lib, api
        d, ti = self.d, torch.float16 if self.d.dtype == "bf16" else torch.float32
        return (self.part(_lib.MLA_WS_Q_ABS, d.cache_dim, api.torch_dtype(d)), self.part(_lib.MLA_WS_O_LAT, d.kv_lora_rank, ti),
                self.part(_lib.MLA_WS_O, d.v_head_dim, ti), self.part(_lib.MLA_WS_LSE, 1, torch.float32).view(-1))


CASES = [
    # dtype, heads, contexts, nodes, kernels of the attention, options
    ("fp32", 4, [70, 33], 9, 1, dict(page=16)),
    ("fp32", 2, [300, 0], 5, 1, dict(page=16, window=40, masked=True)),
    ("bf16", 16, [100, 3], 9, 1, dict(page=64)),
    ("bf16", 16, [6000, 4100], 4, 2, {}),                          # parts merged: blocks of one row tile
    ("bf16", 48, [8100], 7, 2, dict(masked=True)),                 # and of pairs of them
    ("bf16", 16, [2000] * 3 + [1700, 900, 2044, 0, 1990], 32, 1, dict(page=16)),   # parts joined in their clusters
    ("bf16", 16, [2000 - 61 * (b % 29) for b in range(40)], 9, 2, dict(page=64)),  # a last wave's launch
    ("bf16", 32, [2500, 1300, 700], 12, 1, dict(page=64, window=300, masked=True)),
    ("bf16", 16, [40 + b % 50 for b in range(110)], 64, 1, dict(page=64)),         # enough tokens for the fused append
]


@pytest.mark.parametrize("dtype,heads,ctx,T,kernels,opt", CASES)
def test_the_layer_against_its_own_steps(dtype, heads, ctx, T, kernels, opt):
    from head_latent_attention_qkv_gb300 import api
    c = Layer(dtype, heads, ctx, T, **opt)
    d, bf16 = c.d, dtype == "bf16"
    out = c.forward()
    torch.cuda.synchronize()
    assert api.mla_get_device_status(c.h) == 0
    q, o_lat, o, lse = c.parts()
    # the attention alone, of the same queries over the entries that the call has written
    want_lse = torch.full_like(lse, float("nan"))
    before = api.mla_kernel_launches(c.h)
    want = api.mla_tree_attention(c.h, q.clone(), c.positions, c.paged.cache, c.desc, c.parent, lse=want_lse)
    assert api.mla_kernel_launches(c.h) == before + kernels
    assert torch.equal(o_lat, want) and torch.equal(lse, want_lse)
    rows = torch.isinf(lse)
    assert rows.any() or T == 1 or not (c.parent == -2).any()
    # what follows it
    H, dn, dv, r = heads, d.qk_nope_head_dim, d.v_head_dim, d.kv_lora_rank
    dt = api.torch_dtype(d)
    wuv = torch.from_numpy(c.w["kv_b_proj"]).to(dt).double().cuda().view(H, dn + dv, r)[:, dn:]
    wo = torch.from_numpy(c.w["o_proj"]).to(dt).double().cuda()
    x = o_lat.double().view(-1, H, r)
    ref = torch.einsum("mhr,hvr->mhv", x, wuv)
    mass = torch.einsum("mhr,hvr->mhv", x.abs(), wuv.abs())
    tol = (r + 4) * 2.0 ** -24 * mass + (2.0 ** -11 if bf16 else 2.0 ** -24) * ref.abs() + (2.0 ** -25 if bf16 else 0)
    got = o.double().view(-1, H, dv)
    assert ((got - ref).abs() <= tol).all(), ((got - ref).abs() - tol).max()
    y = got.reshape(-1, H * dv)
    ref, mass = y @ wo.T, y.abs() @ wo.abs().T
    tol = (H * dv + 4) * 2.0 ** -24 * mass + (2.0 ** -8 if bf16 else 2.0 ** -24) * ref.abs()
    assert ((out.double() - ref).abs() <= tol).all(), ((out.double() - ref).abs() - tol).max()


@pytest.mark.parametrize("dtype,heads,ctx,T,kernels,opt", [CASES[0], CASES[3], CASES[6]])
def test_the_layer_captured_and_replayed(dtype, heads, ctx, T, kernels, opt):
    from head_latent_attention_qkv_gb300 import api
    c = Layer(dtype, heads, ctx, T, **opt)
    out = torch.empty_like(c.hidden)
    c.forward(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward(out)
    want, parts = c.forward().clone(), [x.clone() for x in c.parts()]
    for _ in range(3):
        out.zero_()
        c.ws.fill_(0xff)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(torch.equal(x, y) for x, y in zip(c.parts(), parts))
    assert api.mla_get_device_status(c.h) == 0


@pytest.mark.parametrize("dtype,heads,ctx,T,kernels,opt", CASES)
def test_key_weights_go_on_from_the_layer(dtype, heads, ctx, T, kernels, opt):
    from head_latent_attention_qkv_gb300 import api
    c = Layer(dtype, heads, ctx, T, **opt)
    c.forward()
    q, _, _, lse = c.parts()
    w = torch.zeros(c.n, c.paged.max_pages * c.h.page_size, device="cuda")
    api.mla_key_weights(c.h, q, c.positions, c.paged.cache, c.desc, lse, w, parent=c.parent)
    torch.cuda.synchronize()
    assert api.mla_get_device_status(c.h) == 0
    # every row that sees a key hands out a weight of one in all
    live = torch.isfinite(lse).view(c.n, -1).sum(1).double()
    assert torch.allclose(w.double().sum(1), live, rtol=1e-5, atol=1e-6)
