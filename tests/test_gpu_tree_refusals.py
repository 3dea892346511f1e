"""Arguments that the tree and eviction entry points refuse on the host, before
anything is launched, through the raw entry points (needs a GB300 for a handle).
"""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Layer:
    """A layer, one sequence of `ctx` keys and a tree of `nodes`, and what the
    entry points need beside them; `off` moves the cache by bytes."""

    def __init__(self, dtype, heads, ctx, nodes, page=16):
        from head_latent_attention_qkv_gb300 import api
        from tests.tree_cases import i32, make_handle
        self.h = make_handle(dtype, heads, page)[0]
        d, self.nodes, self.rows = self.h.dims, nodes, nodes * heads
        dt = api.torch_dtype(d)
        mp = -(-(ctx + nodes) // page)
        self.pages = mp
        self.store = torch.zeros(mp * page * d.cache_dim + 16, dtype=dt, device="cuda")
        self.table, self.kv = i32([list(range(mp))]), i32([ctx + nodes])
        self.positions, self.parent = i32([ctx + i for i in range(nodes)]), i32(list(range(-1, nodes - 1)))
        self.hidden = torch.zeros(nodes, d.hidden_size, dtype=dt, device="cuda")
        self.out = torch.zeros_like(self.hidden)
        self.desc = api.make_desc(self.table, self.kv, block_len=nodes)
        self.ref = C.byref(self.desc)

    def forward(self, off=0, ws=None, nws=None):
        from head_latent_attention_qkv_gb300 import api
        from head_latent_attention_qkv_gb300._lib import lib
        need = api.mla_forward_tree_workspace_bytes(self.h, self.desc)
        own = torch.empty(need, dtype=torch.uint8, device="cuda")
        return lib.mla_draft_forward_tree(
            self.h.h, self.hidden.data_ptr(), self.positions.data_ptr(), None, self.store.data_ptr() + off,
            self.pages, self.ref, self.parent.data_ptr(), self.out.data_ptr(),
            own.data_ptr() if ws is None else ws, need if nws is None else nws,
            torch.cuda.current_stream().cuda_stream)

    def launches(self):
        from head_latent_attention_qkv_gb300 import api
        return api.mla_kernel_launches(self.h)


@pytest.mark.parametrize("dtype,heads", [("fp32", 4), ("bf16", 16)])
def test_the_layer_refuses_a_cache_that_is_not_aligned(dtype, heads):
    from head_latent_attention_qkv_gb300 import _lib, api
    c = Layer(dtype, heads, 20, 3)
    before = c.launches()
    for off in (2, 4, 8, 12):
        assert c.forward(off) == _lib.MLA_ERR_INVALID_ARG, off
        assert b"aligned" in _lib.lib.mla_last_error()
    assert c.launches() == before                              # nothing was launched
    assert c.forward(16) == _lib.MLA_OK
    torch.cuda.synchronize()
    assert api.mla_get_device_status(c.h) == 0


@pytest.mark.parametrize("dtype,heads", [("fp32", 4), ("bf16", 16)])
def test_compaction_refuses_a_cache_that_splits_words(dtype, heads):
    from head_latent_attention_qkv_gb300 import _lib, api
    from head_latent_attention_qkv_gb300._lib import lib
    from tests.tree_cases import i32
    c = Layer(dtype, heads, 40, 1)
    keep, num = i32([[1, 3, 7]]), i32([3])
    dst = i32([[0]])
    ws = torch.empty(api.mla_cache_compact_workspace_bytes(c.h, 1, 3), dtype=torch.uint8, device="cuda")

    def run(off, table):
        return lib.mla_cache_compact(c.h.h, c.store.data_ptr() + off, c.pages, c.table.data_ptr(), c.table.shape[1],
                                     c.kv.data_ptr(), 1, keep.data_ptr(), 3, num.data_ptr(), None, table, 1, None,
                                     None, 0, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)

    before = c.launches()
    for off in (1, 2, 6, 15):
        for table in (None, dst.data_ptr()):
            assert run(off, table) == _lib.MLA_ERR_INVALID_ARG, off
            assert b"aligned" in lib.mla_last_error()
    assert c.launches() == before
    # words, but not 16-byte units: rows move by words
    d = c.h.dims.cache_dim
    off = 4 // c.store.element_size()
    rows = c.store[off:off + c.pages * 16 * d].view(-1, d)
    rows.copy_(torch.arange(rows.shape[0], device="cuda")[:, None] + torch.arange(d, device="cuda") / 8)
    want = rows.clone()
    want[:3] = rows[[1, 3, 7]]
    assert run(4, None) == _lib.MLA_OK
    torch.cuda.synchronize()
    assert api.mla_get_device_status(c.h) == 0
    assert torch.equal(rows, want)


# Plans that need a workspace: a long sequence of few rows (parts to be merged), of
# pairs of row tiles, and row parts of the key weights.
WORKSPACES = [("tree", 16, 9000, 4), ("layer", 16, 8000, 4), ("tree", 48, 9000, 7), ("layer", 48, 8000, 7),
              ("weights", 128, 1000, 16)]


@pytest.mark.parametrize("what,heads,ctx,nodes", WORKSPACES)
def test_workspaces_that_are_missing_short_or_not_aligned_are_refused(what, heads, ctx, nodes):
    from head_latent_attention_qkv_gb300 import _lib, api
    from head_latent_attention_qkv_gb300._lib import lib
    c = Layer("bf16", heads, ctx, nodes)
    stream = torch.cuda.current_stream().cuda_stream
    q = torch.zeros(c.rows, c.h.dims.cache_dim, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(c.rows, 512, dtype=torch.float16, device="cuda")
    lse, ldw = torch.zeros(c.rows, device="cuda"), c.pages * 16
    w = torch.zeros(1, ldw, device="cuda")
    if what == "tree":
        need = api.mla_tree_attention_workspace_bytes(c.h, c.desc)

        def run(ws, n):
            return lib.mla_tree_attention(c.h.h, q.data_ptr(), c.positions.data_ptr(), c.store.data_ptr(), c.pages,
                                          c.ref, c.parent.data_ptr(), o.data_ptr(), lse.data_ptr(), ws, n, stream)
    elif what == "layer":
        need = api.mla_forward_tree_workspace_bytes(c.h, c.desc)
        plain = api.mla_tree_attention_workspace_bytes(c.h, c.desc)
        lse_at = api.mla_forward_workspace_offset(c.h, nodes, _lib.MLA_WS_LSE)
        assert plain > 0 and need >= lse_at + 4 * c.rows + plain

        def run(ws, n):
            return lib.mla_draft_forward_tree(c.h.h, c.hidden.data_ptr(), c.positions.data_ptr(), None,
                                              c.store.data_ptr(), c.pages, c.ref, c.parent.data_ptr(),
                                              c.out.data_ptr(), ws, n, stream)
    else:
        need = api.mla_key_weights_workspace_bytes(c.h, c.desc, ldw)

        def run(ws, n):
            return lib.mla_key_weights(c.h.h, q.data_ptr(), c.positions.data_ptr(), c.store.data_ptr(), c.pages, c.ref,
                                       c.parent.data_ptr(), lse.data_ptr(), 1.0, None, w.data_ptr(), ldw, ws, n, stream)
    assert need > 0
    buf = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    at = buf.data_ptr()
    assert at % 256 == 0
    before = c.launches()
    for ws, n in ((None, need), (None, 0), (at, need - 1), (at, 0), (at + 16, need), (at + 128, need + 128)):
        assert run(ws, n) == _lib.MLA_ERR_INVALID_ARG, (ws, n)
        assert b"workspace" in lib.mla_last_error() or ws is None
    assert c.launches() == before                              # nothing was launched
    assert run(at, need) == _lib.MLA_OK
    assert run(at + 256, need) == _lib.MLA_OK
    torch.cuda.synchronize()
    assert api.mla_get_device_status(c.h) == 0 and c.launches() > before
