"""Tree attention and key weights against the fp64 oracle (needs a GB300).

Bounds, from the arithmetic.  A score sums L products in fp32 (in any order):
its error is at most ds = (L + 4) 2^-24 * scale * sum_d |q_d e_d|, here bounded
by its largest value over the seen keys, the rounding of its scaled value
included.  The log-sum-exp moves by at most that and a few roundings of its own
size and of n summands.  The output moves by the weights' relative error, 2 ds
+ 2^-20, times sum_j p_j |v_j|; bf16 layers round each weight to bf16 as it
meets the bf16 values (at most 2^-8 of it), and store fp16 (2^-11 of the value;
below 2^-14 a step of 2^-24).  A key's weight moves by its terms' relative
errors, ds + (|s| + |lse|) 2^-20, and rows 2^-24 of the sum.  Rows that see
nothing: exactly +0 and -inf.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


HANDLES = {}


def handle(dtype, heads, page, **dims):
    from tests.tree_cases import make_handle
    key = (dtype, heads, page, tuple(sorted(dims.items())))
    if key not in HANDLES:
        HANDLES[key] = make_handle(dtype, heads, page, **dims)
    return HANDLES[key][0]


class Case:
    """Queries, cache and descriptor of one batch; entries that nobody sees and
    queries of rows that see nothing are NaN."""

    def __init__(self, dtype, heads, page, ctx, T, seed=0, window=0, padded=False, masked=False,
                 tree=True, parents=None, q_scale=1.0, dims=None, far=0):
        from head_latent_attention_qkv_gb300 import api
        from oracle import tree as O
        from tests.tree_cases import Paged, bushy, depths, i32
        rng = np.random.default_rng(seed)
        self.h = handle(dtype, heads, page, **(dims or {}))
        self.T, self.H, self.d, self.n = T, heads, self.h.dims, len(ctx)
        self.kv = [c + T for c in ctx]
        self.parents = None
        if tree:
            self.parents = parents or [
                bushy(rng, T, int(rng.integers(max(1, T // 2), T + 1)) if padded else None) for _ in ctx]
        dep = [depths(p) for p in self.parents] if tree else [list(range(T))] * self.n
        self.pos = [[c + x for x in dd] for c, dd in zip(ctx, dep)]
        self.windows = [window if b % 2 == 0 else 0 for b in range(self.n)]
        self.qv = np.ones((self.n, T), dtype=np.uint8)
        if masked:
            self.qv[:, : max(1, T // 3)] = 0
        self.paged = Paged(rng, self.d, page, self.kv)
        q = rng.normal(size=(self.n, T, heads, self.d.cache_dim)) * q_scale
        self.vis = [O.visible(self.kv[b], self.pos[b], self.windows[b], self.qv[b],
                              None if self.parents is None else self.parents[b]) for b in range(self.n)]
        for b in range(self.n):
            unseen = np.flatnonzero(~self.vis[b].any(axis=0))
            if len(unseen):
                self.paged.set_nan(b, torch.from_numpy(unseen))
                self.paged.entries[b][unseen] = np.nan
            q[b][~self.vis[b].any(axis=1)] = np.nan
        q = q.reshape(self.n * T * heads, -1)
        self.q = torch.from_numpy(q.astype(np.float32)).to(api.torch_dtype(self.d)).cuda()
        self.q64 = self.q.double().cpu().numpy().reshape(self.n, T, heads, -1)
        if far:                                       # the same pages behind `far` others
            cache = torch.empty(far + self.paged.num_pages, page, self.d.cache_dim,
                                dtype=self.paged.cache.dtype, device="cuda")
            cache[far:] = self.paged.cache
            self.paged.cache, self.paged.num_pages = cache, cache.shape[0]
            self.paged.table = np.where(self.paged.table >= 0, self.paged.table + far, -1).astype(np.int32)
        self.positions = i32(np.concatenate([np.asarray(p).reshape(-1) for p in self.pos]))
        self.parent = None if self.parents is None else i32(np.concatenate(self.parents))
        self.stats = torch.full((self.n * T, 3), -7, dtype=torch.int32, device="cuda")
        self.keep = [i32(self.paged.table), i32(self.kv), i32(self.windows) if window else None,
                     torch.from_numpy(self.qv.reshape(-1)).cuda() if masked else None]
        self.desc = api.make_desc(self.keep[0], self.keep[1], self.keep[2], self.keep[3], T, self.stats)
        self.scale = 1.0 / np.sqrt(self.d.qk_head_dim)

    def score_error(self, b, i):
        """ds of query i's rows [H]."""
        e = np.abs(self.paged.entries[b][self.vis[b][i]])
        if not len(e):
            return np.zeros(self.H)
        mass = self.scale * (np.abs(self.q64[b, i]) @ e.T).max(axis=1)
        return (self.d.cache_dim + 4) * 2.0 ** -24 * mass

    def attention(self, **kw):
        from head_latent_attention_qkv_gb300 import api
        lse = torch.full((self.q.shape[0],), float("nan"), device="cuda")
        o = api.mla_tree_attention(self.h, self.q, self.positions, self.paged.cache, self.desc,
                                   self.parent, lse=lse, **kw)
        return o, lse

    def check_attention(self, o, lse, status=0):
        from head_latent_attention_qkv_gb300 import api
        from oracle import tree as O
        torch.cuda.synchronize()
        assert api.mla_get_device_status(self.h) == status
        r = self.d.kv_lora_rank
        o = o.double().cpu().numpy().reshape(self.n, self.T, self.H, r)
        lse = lse.double().cpu().numpy().reshape(self.n, self.T, self.H)
        stats = self.stats.cpu().numpy().reshape(self.n, self.T, 3)
        bf16 = self.d.dtype == "bf16"
        for b in range(self.n):
            e = self.paged.entries[b]
            ref, l = O.attention(self.q64[b], e, self.vis[b], r, self.scale)
            mass = O.weight_mass(self.q64[b], e, self.vis[b], r, self.scale)
            for i in range(self.T):
                seen = np.flatnonzero(self.vis[b][i])
                want = [len(seen), seen[0], seen[-1]] if len(seen) else [0, -1, -1]
                assert stats[b, i].tolist() == want, (b, i)
                if not len(seen):
                    assert (o[b, i] == 0).all() and not np.signbit(o[b, i]).any()
                    assert np.isneginf(lse[b, i]).all()
                    continue
                ds = self.score_error(b, i)[:, None]
                n = len(seen)
                tol = (2 * ds + (2.0 ** -8 if bf16 else 0.0) + 2.0 ** -20 + n * 2.0 ** -23) * mass[i]
                tol += (2.0 ** -11 if bf16 else 2.0 ** -24) * np.abs(ref[i]) + (2.0 ** -25 if bf16 else 0.0)
                bad = ~(np.abs(o[b, i] - ref[i]) <= tol)
                assert not bad.any(), (b, i, np.abs(o[b, i] - ref[i]).max(), tol[bad].min())
                tl = ds[:, 0] + (np.abs(l[i]) + 1) * 2.0 ** -21 + n * 2.0 ** -24
                assert (np.abs(lse[b, i] - l[i]) <= tl).all(), (b, i, np.abs(lse[b, i] - l[i]).max())

    def weights(self, decay=0.5, with_prior=True, seed=5, pad=3):
        """mla_key_weights into a buffer of `pad` more columns, checked."""
        from head_latent_attention_qkv_gb300 import api
        from oracle import tree as O
        r, width = self.d.kv_lora_rank, max(self.kv) + pad
        rng = np.random.default_rng(seed)
        ref_lse = [O.attention(self.q64[b], self.paged.entries[b], self.vis[b], r, self.scale)[1]
                   for b in range(self.n)]
        lse32 = np.concatenate([x.reshape(-1) for x in ref_lse]).astype(np.float32)
        prior = rng.random((self.n, width)).astype(np.float32)
        out = torch.full((self.n, width), -3.0, device="cuda")
        pd = torch.from_numpy(prior).cuda() if with_prior else None
        api.mla_key_weights(self.h, self.q, self.positions, self.paged.cache, self.desc,
                            torch.from_numpy(lse32).cuda(), out, prior=pd, decay=decay, parent=self.parent)
        torch.cuda.synchronize()
        assert api.mla_get_device_status(self.h) == 0
        got = out.double().cpu().numpy()
        lse64 = lse32.astype(np.float64).reshape(self.n, self.T, self.H)
        for b in range(self.n):
            total, size = O.key_weights(self.q64[b], self.paged.entries[b], self.vis[b], lse64[b], self.scale)
            ds = max((self.score_error(b, i).max() for i in range(self.T)), default=0.0)
            base = decay * prior[b, :self.kv[b]].astype(np.float64) if with_prior else 0.0
            tol = size * (1.01 * ds + 2.0 ** -20 + self.T * self.H * 2.0 ** -24) + 2.0 ** -22 * (base + total) + 1e-30
            err = np.abs(got[b, :self.kv[b]] - base - total)
            assert (err <= tol).all(), (b, err.max(), (err / tol).max())
            assert (got[b, self.kv[b]:] == -3.0).all()          # behind the sequence: left as it was
        return out


SHAPES = [
    # dtype, heads, page, contexts, nodes, options
    ("fp32", 4, 16, [64, 40], 8, {}),
    ("fp32", 3, 16, [0, 1, 33], 5, dict(padded=True)),
    ("fp32", 1, 48, [100], 1, {}),
    ("fp32", 4, 16, [200, 31, 5], 12, dict(window=17, masked=True, padded=True)),
    ("bf16", 32, 128, [300, 128, 127], 16, {}),
    ("bf16", 128, 64, [0, 1, 255, 256, 257], 1, {}),
    ("bf16", 16, 16, [0, 1, 15, 16, 17, 111, 112, 113, 129], 7, dict(padded=True)),
    ("bf16", 1, 32, [700, 2], 1, {}),
    ("bf16", 3, 64, [500, 63, 64], 43, dict(padded=True)),
    ("bf16", 32, 16, [900, 300, 611, 40], 25, dict(window=130, padded=True, masked=True)),
    ("bf16", 8, 256, [1500, 77], 64, dict(window=40)),
    ("bf16", 20, 128, [640, 3], 33, dict(masked=True)),
    ("bf16", 1, 128, [300], 200, {}),
]


@pytest.mark.parametrize("dtype,heads,page,ctx,T,opt", SHAPES)
def test_tree_attention(dtype, heads, page, ctx, T, opt):
    c = Case(dtype, heads, page, ctx, T, **opt)
    c.check_attention(*c.attention())


@pytest.mark.parametrize("dtype,heads,page,ctx,T,opt", SHAPES)
def test_key_weights_of_trees(dtype, heads, page, ctx, T, opt):
    Case(dtype, heads, page, ctx, T, **opt).weights()


@pytest.mark.parametrize("dtype,heads,page,ctx,T,opt", SHAPES[:10])
def test_key_weights_of_blocks(dtype, heads, page, ctx, T, opt):
    Case(dtype, heads, page, ctx, T, **{**opt, "tree": False, "padded": False}).weights(
        decay=0.0, with_prior=False)


@pytest.mark.parametrize("rank,rope", [(48, 6), (16, 2), (64, 18), (512, 512), (208, 40)])
def test_fp32_layers_of_other_widths(rank, rope):
    # entries of 54, 18 and 82 floats (no multiple of 16 bytes), and the widest
    c = Case("fp32", 3, 16, [70, 0, 33], 7, padded=True, window=25,
             dims=dict(kv_lora_rank=rank, qk_rope_head_dim=rope))
    c.check_attention(*c.attention())
    c.weights()


@pytest.mark.parametrize("dtype,heads,T,window", [("bf16", 2, 130, 0), ("bf16", 2, 90, 17), ("bf16", 5, 65, 0),
                                                  ("bf16", 1, 1024, 0), ("fp32", 1, 1024, 100), ("fp32", 2, 90, 17)])
def test_deep_trees(dtype, heads, T, window):
    # more than 64 nodes; chains as deep as the tree in one block, bushy in the other
    from tests.tree_cases import bushy
    rng = np.random.default_rng(T)
    c = Case(dtype, heads, 16, [40, 3], T, parents=[list(range(-1, T - 1)), bushy(rng, T, T - 5)], window=window)
    c.check_attention(*c.attention())
    c.weights()


@pytest.mark.parametrize("dtype,heads,ctx", [("fp32", 4, [60, 20]), ("bf16", 16, [60, 20]), ("bf16", 16, [4000, 20]),
                                             ("bf16", 2, [3000, 20])])
def test_a_nan_that_a_row_sees_reaches_its_output(dtype, heads, ctx):
    from head_latent_attention_qkv_gb300 import api
    c = Case(dtype, heads, 16, ctx, 9)
    c.paged.set_nan(0, torch.tensor([ctx[0] // 2]))
    o, lse = c.attention()
    torch.cuda.synchronize()
    rows = 9 * heads
    assert torch.isnan(o[:rows]).all() and torch.isnan(lse[:rows]).all()
    assert torch.isfinite(o[rows:]).all() and torch.isfinite(lse[rows:]).all()
    w = torch.zeros(2, max(c.kv), device="cuda")
    api.mla_key_weights(c.h, c.q, c.positions, c.paged.cache, c.desc, torch.zeros_like(lse), w, parent=c.parent)
    bad = torch.isnan(w)
    assert bad[0, ctx[0] // 2] and bad.sum() == 1
    assert api.mla_get_device_status(c.h) == 0


@pytest.mark.parametrize("dtype,heads", [("fp32", 4), ("bf16", 8), ("bf16", 48)])
def test_positions_of_rows_that_see_nothing_may_hold_anything(dtype, heads):
    # a window's first key is worked out from the least position: not from those of
    # padding, of nodes under padding, or of queries that are masked
    low = -2 ** 31
    par = [-1, 0, 0, 1, 3, -2, 5]
    for tree in (True, False):
        c = Case(dtype, heads, 16, [700, 650], 7, window=100, masked=True, tree=tree, parents=[par, par])
        dead = torch.from_numpy(np.stack([~v.any(axis=1) for v in c.vis]).reshape(-1)).cuda()
        assert dead.sum() == (8 if tree else 4)
        for junk in (low, low + 50, 2 ** 31 - 1):
            c.positions[dead] = junk
            if tree:
                c.check_attention(*c.attention())
            c.weights()


def test_many_blocks():
    ctx = [(37 * b) % 300 for b in range(75)]
    c = Case("bf16", 4, 16, ctx, 3, padded=True)
    c.check_attention(*c.attention())
    c.weights()


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("heads,T", [(2, 8), (2, 9), (8, 4), (3, 11), (16, 4), (13, 5), (32, 4), (43, 3)])
def test_rows_of_a_block_around_the_sizes_of_its_tile(heads, T, page):
    # up to 32, 64, 128 and more rows; the neighbours' queries in a tile may be NaN
    c = Case("bf16", heads, page, [1900, 3, 700, 0], T, padded=True, masked=T > 8, seed=page + T)
    c.check_attention(*c.attention())
    c.weights()


@pytest.mark.parametrize("rows", [32, 33, 64, 65, 66, 80, 84, 85, 96, 97])
def test_key_weights_around_the_rows_that_share_a_slot(rows):
    # up to 64 rows a block bring three chunks of Q at once, more bring one
    Case("bf16", 1, 64, [700, 255, 0], rows, padded=True).weights()
    Case("bf16", rows, 128, [900], 1, tree=False).weights()


@pytest.mark.parametrize("heads,T,n,window", [(16, 9, 40, 0), (4, 5, 83, 0), (16, 9, 79, 700)])
def test_blocks_of_a_last_wave_cut_in_parts(heads, T, n, window):
    # more clusters than the GPU holds: the last wave's are a launch of their own
    ctx = [2000 - 61 * (b % 29) - (1900 if b % 13 == 5 else 0) for b in range(n)]
    from head_latent_attention_qkv_gb300 import api
    c = Case("bf16", heads, 16, [max(x, 0) for x in ctx], T, padded=True, window=window)
    before = api.mla_kernel_launches(c.h)
    c.check_attention(*c.attention())
    assert api.mla_kernel_launches(c.h) == before + 2
    g = torch.cuda.CUDAGraph()
    want = c.attention()
    with torch.cuda.graph(g):
        got = c.attention()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_pages_behind_four_gigabytes():
    c = Case("bf16", 16, 64, [300, 77], 6, far=61000)           # 4.5 GB of pages before them
    c.check_attention(*c.attention())
    c.weights()
    c = Case("fp32", 4, 64, [100, 30], 5, far=220000)
    c.check_attention(*c.attention())
    c.weights()


def test_weights_rows_shorter_than_the_sequence_are_reported():
    from head_latent_attention_qkv_gb300 import _lib, api
    for dtype, heads in (("fp32", 4), ("bf16", 16)):
        c = Case(dtype, heads, 16, [50, 20], 7)
        full = c.weights(with_prior=False)
        _, lse = c.attention()
        w = torch.full((2, 40), -3.0, device="cuda")
        ref = torch.zeros(2, 64, device="cuda")
        api.mla_key_weights(c.h, c.q, c.positions, c.paged.cache, c.desc, lse, ref, parent=c.parent)
        assert api.mla_get_device_status(c.h) == 0
        api.mla_key_weights(c.h, c.q, c.positions, c.paged.cache, c.desc, lse, w, parent=c.parent)
        assert api.mla_get_device_status(c.h) == _lib.MLA_DEV_BAD_LENGTH
        assert torch.equal(w[0], ref[0, :40]) and torch.equal(w[1, :27], ref[1, :27]) and (w[1, 27:] == -3).all()
        assert full.shape[1] == 60


@pytest.mark.parametrize("dtype,heads", [("fp32", 4), ("bf16", 16)])
def test_chains_and_stars(dtype, heads):
    T = 20
    c = Case(dtype, heads, 16, [70, 9], T, parents=[list(range(-1, T - 1)), [-1] * T])
    c.check_attention(*c.attention())
    c.weights()


def test_long_causal_chain_crosses_tiles():
    T = 300
    c = Case("bf16", 1, 64, [90], T, parents=[list(range(-1, T - 1))])
    c.check_attention(*c.attention())
    c.weights()


@pytest.mark.parametrize("dtype,heads", [("fp32", 4), ("bf16", 32)])
def test_large_scores(dtype, heads):
    # scores of several hundred: the running maximum moves far between tiles
    c = Case(dtype, heads, 16, [900, 260], 6, q_scale=100.0)
    c.check_attention(*c.attention())


def test_long_context_is_split_and_joined():
    c = Case("bf16", 16, 128, [9001], 4)
    c.check_attention(*c.attention())
    c.weights()


def test_lse_may_be_left_out_and_stream_is_taken():
    from head_latent_attention_qkv_gb300 import api
    c = Case("bf16", 32, 128, [300], 4)
    o, lse = c.attention()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2 = api.mla_tree_attention(c.h, c.q, c.positions, c.paged.cache, c.desc, c.parent, stream=s)
    s.synchronize()
    assert torch.equal(o, o2)


@pytest.mark.parametrize("dtype,heads", [("fp32", 4), ("bf16", 32)])
def test_captured_and_replayed(dtype, heads):
    from head_latent_attention_qkv_gb300 import api
    c = Case(dtype, heads, 128, [1500, 90], 6)
    o, lse = c.attention()
    w = torch.zeros(2, 2048, device="cuda")
    api.mla_key_weights(c.h, c.q, c.positions, c.paged.cache, c.desc, lse, w, parent=c.parent)
    o2, lse2, w2 = torch.zeros_like(o), torch.zeros_like(lse), torch.zeros_like(w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.mla_tree_attention(c.h, c.q, c.positions, c.paged.cache, c.desc, c.parent, o_lat=o2, lse=lse2)
        api.mla_key_weights(c.h, c.q, c.positions, c.paged.cache, c.desc, lse2, w2, parent=c.parent)
    for _ in range(2):
        o2.zero_(), lse2.zero_(), w2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(w, w2)


@pytest.mark.parametrize("dtype,heads", [("fp32", 4), ("bf16", 16)])
def test_bad_parents_pages_and_lengths_are_reported(dtype, heads):
    from head_latent_attention_qkv_gb300 import _lib, api
    # a parent that is no earlier node: it and the nodes below it leave the tree
    par = [[-1, 0, 1, 5, 3, 4, -1], [-1, 0, 0, 1, 2, 3, 7]]
    c = Case(dtype, heads, 16, [50, 20], 7, parents=par)
    c.check_attention(*c.attention(), status=_lib.MLA_DEV_BAD_TREE)
    # kv_len shorter than the tree: the block's rows see nothing, the other block is as before
    c = Case(dtype, heads, 16, [50, 20], 7)
    c.keep[1][0] = 6
    c.vis[0][:] = False
    c.check_attention(*c.attention(), status=_lib.MLA_DEV_BAD_LENGTH)
    # kv_len behind the page table
    c = Case(dtype, heads, 16, [50, 20], 7)
    c.keep[1][0] = c.paged.max_pages * 16 + 1
    c.vis[0][:] = False
    c.check_attention(*c.attention(), status=_lib.MLA_DEV_BAD_LENGTH)
    # a page outside the cache is read as zeros by its block alone
    c = Case(dtype, heads, 16, [50, 20], 7)
    c.keep[0][0, 1] = c.paged.num_pages
    c.paged.entries[0][16:32] = 0.0
    c.check_attention(*c.attention(), status=_lib.MLA_DEV_BAD_PAGE)
    w = torch.zeros(2, 64, device="cuda")
    lse = torch.zeros(c.q.shape[0], device="cuda")
    api.mla_key_weights(c.h, c.q, c.positions, c.paged.cache, c.desc, lse, w, parent=c.parent)
    assert api.mla_get_device_status(c.h) & _lib.MLA_DEV_BAD_PAGE
    # a negative window
    c = Case(dtype, heads, 16, [50, 20], 7, window=9)
    c.keep[2][0] = -1
    c.vis[0][:] = False
    c.check_attention(*c.attention(), status=_lib.MLA_DEV_BAD_WINDOW)


def test_equal_calls_give_equal_bits():
    c = Case("bf16", 32, 64, [3000, 700, 64], 9)
    a, b = c.attention(), c.attention()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(c.weights(), c.weights())


@pytest.mark.parametrize("dtype,heads,page", [("fp32", 4, 16), ("bf16", 16, 64)])
def test_forward_over_trees_against_the_layer_oracle(dtype, heads, page):
    """The whole layer over trees: appended contexts, the nodes' own entries
    written by the call, the oracle's expanded form under the tree's mask."""
    from head_latent_attention_qkv_gb300 import api
    from oracle import mla, tree as O
    from tests.parity import compare
    from tests.tree_cases import bushy, depths, i32, make_handle
    h, w = make_handle(dtype, heads, page)
    d, rng, T, ctx = h.dims, np.random.default_rng(11), 9, [70, 33]
    dt = api.torch_dtype(d)
    parents = [bushy(rng, T), bushy(rng, T, 6)]
    mp = -(-(max(ctx) + T) // page)
    table = rng.permutation(2 * mp).reshape(2, mp).astype(np.int32)

    def slot(b, j):
        return int(table[b][j // page]) * page + j % page

    cache = torch.full((2 * mp, page, d.cache_dim), float("nan"), dtype=dt, device="cuda")
    hid = torch.from_numpy(rng.normal(size=(sum(ctx), d.hidden_size)).astype(np.float32)).to(dt)
    pos = np.concatenate([np.arange(c) for c in ctx])
    slots = torch.tensor([slot(b, j) for b, c in enumerate(ctx) for j in range(c)], device="cuda")
    api.mla_latent_cache_append(h, hid.cuda(), i32(pos), slots, cache)
    x = torch.from_numpy(rng.normal(size=(2 * T, d.hidden_size)).astype(np.float32)).to(dt)
    npos = np.concatenate([c + np.asarray(depths(p)) for c, p in zip(ctx, parents)])
    nodes = torch.tensor([slot(b, c + k) for b, c in enumerate(ctx) for k in range(T)], device="cuda")
    bt, kv = i32(table), i32([c + T for c in ctx])
    desc = api.make_desc(bt, kv, block_len=T)
    out = api.mla_draft_forward_tree(h, x.cuda(), i32(npos), nodes, cache, desc, i32(np.concatenate(parents)))
    torch.cuda.synchronize()
    assert api.mla_get_device_status(h) == 0
    got = out.float().cpu().numpy()
    x64, at, refs, live = x.double().numpy(), 0, [], []
    for b, c in enumerate(ctx):
        e = np.concatenate([mla.latent_cache_entries(d, w, hid[at:at + c].double().numpy(), np.arange(c)),
                            mla.latent_cache_entries(d, w, x64[b * T:(b + 1) * T], npos[b * T:(b + 1) * T])])
        at += c
        e = mla.round_to_dtype(d, e)
        p = npos[b * T:(b + 1) * T]
        vis = O.visible(c + T, p.tolist(), 0, None, parents[b])
        ref = mla.block_forward(d, w, x64[b * T:(b + 1) * T], p, [mla.expand_keys(d, w, e)], vis)
        refs.append(mla.round_to_dtype(d, ref))
        live.append(vis.any(axis=1))
    rows = np.concatenate(live)
    compare(got, np.concatenate(refs), d, f"tree {dtype}", rows)
    assert (got[~rows] == 0).all()
    h.close()


def test_refusals():
    """Arguments that the entry points refuse before anything is launched."""
    from head_latent_attention_qkv_gb300 import _lib, api
    c = Case("bf16", 16, 16, [50], 3)
    lse = torch.zeros(48, device="cuda")
    w = torch.zeros(1, 64, device="cuda")
    ok = dict(h=c.h, q_abs=c.q, positions=c.positions, cache=c.paged.cache, desc=c.desc, parent=c.parent)

    def tree(**kw):
        return api.mla_tree_attention(**{**ok, **kw})

    for bad in (dict(q_abs=c.q.float()), dict(q_abs=c.q[:, ::2]), dict(q_abs=c.q[:-1]), dict(q_abs=c.q.cpu()),
                dict(positions=c.positions.long()), dict(positions=c.positions[:2]), dict(parent=c.parent.long()),
                dict(cache=c.paged.cache[:, :8]), dict(cache=c.paged.cache.half()),
                dict(lse=lse[:5]), dict(lse=lse.half()), dict(o_lat=torch.zeros(48, 512, device="cuda"))):
        with pytest.raises(ValueError):
            tree(**bad)
    with pytest.raises(ValueError):
        api.mla_key_weights(c.h, c.q, c.positions, c.paged.cache, c.desc, lse[:4], w)
    with pytest.raises(ValueError):
        api.mla_key_weights(c.h, c.q, c.positions, c.paged.cache, c.desc, lse, w, prior=w[:, :8])
    P = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    o = torch.zeros(48, 512, dtype=torch.float16, device="cuda")

    def raw(desc, q=c.q.data_ptr(), ws=P.data_ptr(), nws=P.numel()):
        return _lib.lib.mla_tree_attention(c.h.h, q, c.positions.data_ptr(), c.paged.cache.data_ptr(),
                                           c.paged.num_pages, desc, c.parent.data_ptr(), o.data_ptr(), None,
                                           ws, nws, None)

    def desc(**kw):
        d = _lib.mla_attn_desc_t()
        for k, _ in d._fields_:
            setattr(d, k, kw.get(k, getattr(c.desc, k)) if k in kw else getattr(c.desc, k))
        return d

    for fields in (dict(block_len=0), dict(num_blocks=-1), dict(max_pages=0), dict(kv_len=None),
                   dict(block_table=None), dict(max_pages=1 << 27)):
        assert raw(desc(**fields)) == _lib.MLA_ERR_INVALID_ARG, fields
    assert raw(c.desc, q=c.q.data_ptr() + 2) == _lib.MLA_ERR_INVALID_ARG
    assert raw(desc(block_len=1025)) == _lib.MLA_ERR_UNSUPPORTED
    assert raw(desc(num_blocks=0)) == _lib.MLA_OK                  # nothing to do
    if api.mla_tree_attention_workspace_bytes(c.h, c.desc):
        assert raw(c.desc, ws=None) == _lib.MLA_ERR_INVALID_ARG
        assert raw(c.desc, nws=16) == _lib.MLA_ERR_INVALID_ARG
    for kw in (dict(budget=0), dict(budget=-1), dict(budget=4, sink=3, recent=2), dict(budget=4, sink=-1)):
        with pytest.raises(_lib.MLAError):
            api.mla_cache_select(c.h, w, c.keep[1], **kw)
    keep, num = api.mla_cache_select(c.h, w, c.keep[1], 8)
    with pytest.raises(_lib.MLAError):                       # weights go to their own place or stay in theirs
        api.mla_cache_compact(c.h, c.paged.cache, c.keep[0], c.keep[1], keep, num, weights=w,
                              weights_out=torch.zeros_like(w))
    with pytest.raises(_lib.MLAError):
        api.mla_cache_compact(c.h, c.paged.cache, c.keep[0], c.keep[1], keep, num,
                              workspace=torch.zeros(2, dtype=torch.uint8, device="cuda"), weights=w)
    torch.cuda.synchronize()
    assert api.mla_get_device_status(c.h) == 0
