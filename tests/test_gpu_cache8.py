"""The 8-bit latent cache against the fp64 oracle (needs a GB300).

Storing and reading back are exact: codes, scales and rotary dims equal the
oracle's, bit for bit.  The attention's bounds, from the arithmetic: the score of
a key sums 576 products of numbers held exactly in fp32 (ds of
``tests/test_gpu_tree.py``, with queries split in two e4m3 numbers that leave at most 2^-10
of a unit in which the row's largest magnitude is 224 or more: 2^-17 of it).  A
softmax weight times its key's scale is held as two e4m3 numbers: off by 2^-8 of itself, and by
2^-20 of the row's largest such product, which meets the key's code |e8| <= 448.  The
output is stored in fp16.  The log-sum-exp takes the weights unrounded.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_tree import Case, handle  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def to_cache8(h, cache, junk=True):
    """The 8-bit cache of a bf16 one, through the library; what holds NaN there holds
    every kind of it here."""
    from head_latent_attention_qkv_gb300 import api
    c = api.make_cache8(h, cache.shape[0])
    flat = cache.view(-1, cache.shape[2])
    api.mla_cache8_store(h, flat, torch.arange(flat.shape[0], device="cuda"), c)
    if junk:
        dead = torch.isnan(c.scale)
        c.latent.view(torch.uint8)[dead] = 0x7F
        c.rope[dead] = float("nan")
    return c


class Case8(Case):
    """A batch over an 8-bit cache; entries that nobody sees hold NaN bytes."""

    def __init__(self, heads, page, ctx, T, **kw):
        from oracle import cache8 as O
        super().__init__("bf16", heads, page, ctx, T, **kw)
        self.c8 = to_cache8(self.h, self.paged.cache)
        del self.paged.cache
        self.codes, self.scales = [], []
        for b, e in enumerate(self.paged.entries):
            q8 = O.quantise(e)
            self.codes.append(np.abs(O.E4M3[q8[0]]))
            self.scales.append(q8[2])
            self.paged.entries[b] = O.dequantise(*q8)

    def score_error(self, b, i):
        e = np.abs(self.paged.entries[b][self.vis[b][i]])
        if not len(e):
            return np.zeros(self.H)
        split = self.scale * 2.0 ** -17 * np.abs(self.q64[b, i]).max(axis=1) * e[:, :512].sum(axis=1).max()
        return super().score_error(b, i) + split

    def attention(self, **kw):
        from head_latent_attention_qkv_gb300 import api
        lse = torch.full((self.q.shape[0],), float("nan"), device="cuda")
        o = api.mla_latent_attention8(self.h, self.q, self.positions, self.c8, self.desc, self.parent, lse=lse, **kw)
        return o, lse

    def check_attention(self, o, lse, status=0):
        from head_latent_attention_qkv_gb300 import api
        from oracle import tree as O
        torch.cuda.synchronize()
        assert api.mla_get_device_status(self.h) == status
        o = o.double().cpu().numpy().reshape(self.n, self.T, self.H, 512)
        lse = lse.double().cpu().numpy().reshape(self.n, self.T, self.H)
        stats = self.stats.cpu().numpy().reshape(self.n, self.T, 3)
        for b in range(self.n):
            e = self.paged.entries[b]
            ref, l = O.attention(self.q64[b], e, self.vis[b], 512, self.scale)
            mass = O.weight_mass(self.q64[b], e, self.vis[b], 512, self.scale)
            for i in range(self.T):
                seen = np.flatnonzero(self.vis[b][i])
                want = [len(seen), seen[0], seen[-1]] if len(seen) else [0, -1, -1]
                assert stats[b, i].tolist() == want, (b, i)
                if not len(seen):
                    assert (o[b, i] == 0).all() and not np.signbit(o[b, i]).any()
                    assert np.isneginf(lse[b, i]).all()
                    continue
                ds, n = self.score_error(b, i)[:, None], len(seen)
                s = self.scale * (self.q64[b, i] @ e[seen].T)
                top = (np.exp(s - l[i][:, None]) * self.scales[b][seen]).max(axis=1)[:, None]
                tol = (2 * ds + 2.0 ** -8 + 2.0 ** -20 + n * 2.0 ** -23) * mass[i]
                tol += 2.0 ** -20 * top * self.codes[b][seen].sum(axis=0) + 2.0 ** -11 * np.abs(ref[i]) + 2.0 ** -25
                bad = ~(np.abs(o[b, i] - ref[i]) <= tol)
                assert not bad.any(), (b, i, np.abs(o[b, i] - ref[i]).max(), tol[bad].min())
                tl = ds[:, 0] + (np.abs(l[i]) + 1) * 2.0 ** -21 + n * 2.0 ** -24
                assert (np.abs(lse[b, i] - l[i]) <= tl).all(), (b, i, np.abs(lse[b, i] - l[i]).max(), tl.min())


# --------------------------------------------------------------------------
# storing and reading back
# --------------------------------------------------------------------------
def bf16_entries(n, seed=0):
    """Ordinary entries, and rows where the scale's rule or a rounding can go wrong."""
    rng = np.random.default_rng(seed)
    e = rng.normal(size=(n, 576)) * np.exp(rng.normal(size=(n, 1)) * 3)
    t = torch.from_numpy(e.astype(np.float32)).bfloat16()
    odd = [0.0, 448.0, 450.0, 449.0, 2.0 ** -133, 2.0 ** -64, 2.0 ** 126, 1.75 * 2.0 ** 100, 1.7578125 * 2.0 ** 100, -3.0]
    for i, v in enumerate(odd):
        if 3 * i < n:
            t[3 * i, :512] *= 0.0 if i % 2 else 1e-30
            t[3 * i, (37 * i) % 512] = v
    for i, (d, v) in enumerate([(5, float("nan")), (511, float("-inf")), (575, float("inf")), (512, float("nan")),
                                (100, 2.0 ** 127)]):
        if 3 * i + 1 < n:
            t[3 * i + 1, d] = v
    return t


@pytest.mark.parametrize("n,page", [(0, 16), (1, 16), (7, 128), (300, 32), (5003, 64)])
def test_store_and_load_are_the_oracles(n, page):
    from head_latent_attention_qkv_gb300 import api
    from oracle import cache8 as O
    h = handle("bf16", 4, page)
    pages = -(-n // page) + 2
    rng = np.random.default_rng(n)
    slots = rng.permutation(pages * page)[:n]
    e = bf16_entries(n)
    c = api.make_cache8(h, pages)
    c.scale.fill_(-5.0)
    dev = torch.from_numpy(slots).cuda()
    api.mla_cache8_store(h, e.cuda(), dev, c)
    back = api.mla_cache8_load(h, c, dev)
    torch.cuda.synchronize()
    assert api.mla_get_device_status(h) == 0
    codes, rope, scale = O.quantise(e.double().numpy())
    got = c.latent.view(torch.uint8).view(-1, 512).cpu().numpy()
    assert (got[slots] == codes).all()
    assert np.array_equal(c.scale.view(-1).cpu().double().numpy()[slots], scale, equal_nan=True)
    assert torch.equal(c.rope.view(-1, 64).cpu()[slots].view(torch.int16), e[:, 512:].contiguous().view(torch.int16))
    want = torch.from_numpy(O.dequantise(codes, rope, scale)).bfloat16()
    assert torch.equal(back.cpu().nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
    rest = np.setdiff1d(np.arange(pages * page), slots)      # the other slots are left as they were
    assert (got[rest] == 0).all() and (c.scale.view(-1).cpu().numpy()[rest] == -5).all()
    again = api.make_cache8(h, pages)
    api.mla_cache8_store(h, back, dev, again)
    assert torch.equal(api.mla_cache8_load(h, again, dev).nan_to_num(7.0, 8.0, 9.0), back.nan_to_num(7.0, 8.0, 9.0))


def test_bad_slots_are_reported_and_skipped():
    from head_latent_attention_qkv_gb300 import _lib, api
    h = handle("bf16", 4, 16)
    e = bf16_entries(40, 3).cuda()
    slots = torch.arange(40, device="cuda")
    c = api.make_cache8(h, 3)
    slots[3], slots[20] = -1, 48
    api.mla_cache8_store(h, e, slots, c)
    assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_SLOT
    assert (c.latent.view(torch.uint8).view(-1, 512)[[3, 20]] == 0).all() and (c.scale.view(-1)[[3, 20]] == 1).all()
    out = torch.full((40, 576), -7.0, dtype=torch.bfloat16, device="cuda")
    api.mla_cache8_load(h, c, slots, out=out)
    assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_SLOT
    assert (out[[3, 20]] == -7).all() and not (out[[4, 21]] == -7).any()


def test_slots_behind_four_gigabytes():
    from head_latent_attention_qkv_gb300 import api
    from oracle import cache8 as O
    h = handle("bf16", 4, 128)
    pages = 2 ** 32 // 512 // 128 + 40
    c = api.Cache8(torch.zeros(pages, 128, 512, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                   torch.zeros(pages, 128, 64, dtype=torch.bfloat16, device="cuda"),
                   torch.ones(pages, 128, device="cuda"))
    e = bf16_entries(300, 9)
    slots = torch.arange(300, device="cuda") * 17 + (pages * 128 - 300 * 17)
    api.mla_cache8_store(h, e.cuda(), slots, c)
    back = api.mla_cache8_load(h, c, slots).cpu()
    want = torch.from_numpy(O.dequantise(*O.quantise(e.double().numpy()))).bfloat16()
    assert torch.equal(back.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------
SHAPES = [
    # heads, page, contexts, nodes, options
    (16, 128, [300], 1, dict(tree=False)),
    (32, 128, [300, 128, 127], 16, {}),
    (32, 128, [1000, 0, 1, 255, 256, 257, 513], 1, dict(tree=False)),
    (128, 64, [0, 1, 255, 256, 257], 1, {}),
    (16, 16, [0, 1, 15, 16, 17, 111, 112, 113, 129], 7, dict(padded=True)),
    (1, 32, [700, 2], 1, {}),
    (3, 64, [500, 63, 64], 43, dict(padded=True)),
    (32, 16, [900, 300, 611, 40], 25, dict(window=130, padded=True, masked=True)),
    (8, 256, [1500, 77], 64, dict(window=40)),
    (20, 128, [640, 3], 33, dict(masked=True, tree=False)),
    (20, 128, [640, 3], 33, dict(window=50, tree=False)),
    (1, 128, [300], 200, {}),
    (2, 16, [40, 3], 130, dict(window=17, padded=True)),
    (5, 384, [1100, 20], 9, dict(tree=False, window=300)),
]


@pytest.mark.parametrize("heads,page,ctx,T,opt", SHAPES)
def test_attention(heads, page, ctx, T, opt):
    c = Case8(heads, page, ctx, T, **opt)
    c.check_attention(*c.attention())


@pytest.mark.parametrize("heads,T", [(1, 1), (1, 15), (1, 16), (1, 17), (1, 31), (1, 32), (1, 33), (3, 21), (5, 13), (64, 1), (96, 1)])
def test_rows_of_a_block_around_the_sizes_of_its_groups(heads, T):
    c = Case8(heads, 64, [1900, 3, 700, 0], T, padded=True, masked=T > 8, seed=T)
    c.check_attention(*c.attention())


def test_many_blocks():
    c = Case8(4, 16, [(37 * b) % 300 for b in range(75)], 3, padded=True)
    c.check_attention(*c.attention())
    c = Case8(2, 128, [(53 * b) % 700 for b in range(600)], 1, tree=False)
    c.check_attention(*c.attention())


@pytest.mark.parametrize("heads,ctx,opt", [
    (32, [(97 * b * b) % 5000 for b in range(40)], dict(tree=False)),       # pieces that start with their unit
    (96, [(331 * b) % 3001 for b in range(50)], dict(tree=False)),          # the same, three units a sequence
    (32, [20000] + [30 * b for b in range(149)], {}),                       # one long sequence among short ones
    (32, [8193] + [40] * 149, dict(tree=False)),                            # the first that needs two segments
    (32, [8191] + [40] * 149, dict(tree=False)),
    (32, [300] * 151 + [9000], dict(tree=False)),                           # as many units as SMs
    (128, [19999, 0], dict(window=15000)),
])
def test_few_units_of_unequal_lengths(heads, ctx, opt):
    c = Case8(heads, 64, ctx, 1, seed=len(ctx), **opt)
    c.check_attention(*c.attention())


@pytest.mark.parametrize("n,heads,wide", [(5500, 2, 0), (700, 33, 600), (4864, 1, 0)])
def test_more_blocks_than_threads_and_more_units_than_a_list(n, heads, wide):
    # (of 152 SMs: a CTA's units beyond its list of 32, blocks in two lots; the last ones whole, 32 a CTA)
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import i32
    c = Case8(heads, 16, [(b * b) % 19 for b in range(n)], 1, tree=False)
    if wide:
        table = np.full((n, wide), -1)
        table[:, :c.paged.max_pages] = c.paged.table
        c.keep[0] = i32(table)
        c.desc = api.make_desc(c.keep[0], c.keep[1], None, None, 1, c.stats)
    c.check_attention(*c.attention())


def test_deep_trees():
    from tests.tree_cases import bushy
    for T, window in ((1024, 0), (90, 17)):
        rng = np.random.default_rng(T)
        c = Case8(1, 16, [40, 3], T, parents=[list(range(-1, T - 1)), bushy(rng, T, T - 5)], window=window)
        c.check_attention(*c.attention())


def test_keys_of_very_different_scales_and_scores():
    # latents from 2^-40 to 2^20 in one sequence, rotary dims as large, sharp and flat rows
    for q_scale in (1e-3, 1.0, 6.0):
        c = Case8(8, 64, [700, 90], 4, seed=3, q_scale=q_scale)
        for b in range(c.n):
            e = c.paged.entries[b]
            size = 2.0 ** np.random.default_rng(b).integers(-40, 1, size=len(e))
            seen = ~np.isnan(e).any(axis=1)
            e[seen, :512] *= size[seen][:, None]
        rebuilt(c)
        c.check_attention(*c.attention())


def rebuilt(c):
    """Case `c` with the 8-bit cache of its (changed) entries, rounded to bf16."""
    from head_latent_attention_qkv_gb300 import api
    from oracle import cache8 as O
    c.c8 = api.make_cache8(c.h, c.paged.num_pages)
    for b, e in enumerate(c.paged.entries):
        t = torch.from_numpy(e).bfloat16()
        api.mla_cache8_store(c.h, t.cuda(), c.paged.slots(b, len(e)).cuda(), c.c8)
        q8 = O.quantise(t.double().numpy())
        c.codes[b], c.scales[b] = np.abs(O.E4M3[q8[0]]), q8[2]
        c.paged.entries[b] = O.dequantise(*q8)


def test_a_sink_and_many_light_keys():
    # one key holds a third of the weight, 20 k others e^-11 of it each: small weights
    # are as many as they are small, and must not round to nothing
    c = Case8(1, 128, [20000], 1, seed=1, tree=False)
    e = c.paged.entries[0]
    q = c.q64[0, 0, 0]
    u = q / np.linalg.norm(q)
    e -= np.outer(e @ u, u)                                    # scores 0 but for rounding
    e[:, :512] += 0.5                                          # (a mean that a bias would show in)
    e -= np.outer(e @ u, u)
    e[77] += u * (11.0 / c.scale / np.linalg.norm(q))
    rebuilt(c)
    c.check_attention(*c.attention())


def test_a_poisoned_entry_reaches_the_rows_that_see_it():
    T = 9
    c = Case8(16, 16, [60, 20], T, parents=[[-1] * T, [-1] * T])
    slot = c.paged.slots(0, c.kv[0])
    from head_latent_attention_qkv_gb300 import api
    e = torch.full((1, 576), float("inf"), dtype=torch.bfloat16, device="cuda")
    api.mla_cache8_store(c.h, e, slot[60 + 4:60 + 5].cuda(), c.c8)      # node 4's own key
    o, lse = c.attention()
    rows = torch.zeros(2 * T * 16, dtype=torch.bool)
    rows[4 * 16:5 * 16] = True
    assert torch.isnan(lse.cpu()[rows]).all() and torch.isnan(o.cpu()[rows]).all()
    assert torch.isfinite(lse.cpu()[~rows]).all() and torch.isfinite(o.cpu()[~rows]).all()
    api.mla_cache8_store(c.h, e, slot[30:31].cuda(), c.c8)              # a key of the context
    o, lse = c.attention()
    assert torch.isnan(lse[:T * 16]).all() and torch.isnan(o[:T * 16]).all()
    assert torch.isfinite(lse[T * 16:]).all() and torch.isfinite(o[T * 16:]).all()


@pytest.mark.parametrize("ctx", [[60, 20], [3000, 700]])
def test_a_query_that_is_no_number_spoils_its_row_only(ctx):
    # (in units that lie in one CTA and in cut ones)
    c = Case8(16, 16, ctx, 3, parents=[[-1] * 3, [-1] * 3])
    want = c.attention()
    c.q[5, 100] = float("nan")
    c.q[21, 570] = float("nan")
    c.q[40, 511] = float("inf")
    c.q[70, 0] = float("-inf")
    got = c.attention()
    rows = torch.ones(len(c.q), dtype=torch.bool, device="cuda")
    rows[[5, 21, 40, 70]] = False
    for x, y in zip(got, want):
        assert torch.equal(x[rows], y[rows])
        assert torch.isnan(x[5]).all() and torch.isnan(x[21]).all()
        assert not torch.isfinite(x[40]).any() and not torch.isfinite(x[70]).any()


def test_device_checks():
    from head_latent_attention_qkv_gb300 import _lib, api
    c = Case8(16, 64, [300, 200, 150], 4)
    want = c.attention()
    table = c.keep[0].clone()
    for bad, bit in ((c.paged.num_pages, _lib.MLA_DEV_BAD_PAGE), (-1, _lib.MLA_DEV_BAD_PAGE)):
        c.keep[0][1, 2] = bad
        o, lse = c.attention()
        assert api.mla_get_device_status(c.h) == bit
        c.keep[0].copy_(table)
        rows = torch.ones(3 * 64, dtype=torch.bool, device="cuda")
        rows[64:128] = False
        assert torch.equal(o[rows], want[0][rows]) and torch.equal(lse[rows], want[1][rows])
    kv = c.keep[1].clone()
    for n in (3, -1, 10 ** 6):
        c.keep[1][1] = n
        o, lse = c.attention()
        assert api.mla_get_device_status(c.h) == _lib.MLA_DEV_BAD_LENGTH
        assert (o[64:128] == 0).all() and torch.isneginf(lse[64:128]).all()
        c.keep[1].copy_(kv)
    c.parent[4 + 2] = 3
    c.attention()
    assert api.mla_get_device_status(c.h) == _lib.MLA_DEV_BAD_TREE
    w = torch.tensor([0, -4, 0], dtype=torch.int32, device="cuda")
    c.desc.window = w.data_ptr()
    c.parent[4 + 2] = 1
    o, lse = c.attention()
    assert api.mla_get_device_status(c.h) == _lib.MLA_DEV_BAD_WINDOW
    assert (o[64:128] == 0).all() and torch.isneginf(lse[64:128]).all()


def test_replays_streams_and_equal_bits():
    c = Case8(32, 64, [3000, 170, 900], 5, padded=True)
    want = c.attention()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = c.attention()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # two calls at once, each on a stream of its own with its own workspace
    d = Case8(32, 64, [2000, 2100], 3, seed=9)
    ref = d.attention()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        x = c.attention(stream=s)
        y = d.attention(stream=t)
    torch.cuda.synchronize()
    assert torch.equal(x[0], want[0]) and torch.equal(y[0], ref[0]) and torch.equal(y[1], ref[1])


def test_a_single_token_over_a_long_context_behind_four_gigabytes():
    from head_latent_attention_qkv_gb300 import api
    c = Case8(16, 128, [3000, 77], 1, tree=False)
    far = 2 ** 32 // 512 // 128 + 5
    big = api.make_cache8(c.h, far + c.paged.num_pages)
    for x, y in zip(big, c.c8):
        x[far:].view(torch.uint8).copy_(y.view(torch.uint8))
    c.c8, table = big, torch.where(c.keep[0] >= 0, c.keep[0] + far, c.keep[0])
    c.keep[0].copy_(table)
    c.check_attention(*c.attention())


# --------------------------------------------------------------------------
# the paths that call them
# --------------------------------------------------------------------------
def test_append_stores_the_bf16_caches_entries():
    from head_latent_attention_qkv_gb300 import api
    h = handle("bf16", 4, 16)
    for n in (1, 5, 200):
        g = torch.Generator(device="cuda").manual_seed(n)
        x = torch.randn(n, h.dims.hidden_size, generator=g, device="cuda").bfloat16()
        pos = torch.arange(n, dtype=torch.int32, device="cuda") * 3
        slots = torch.randperm(256, generator=g, device="cuda")[:n]
        cache = torch.zeros(16, 16, 576, dtype=torch.bfloat16, device="cuda")
        api.mla_latent_cache_append(h, x, pos, slots, cache)
        c, d = api.make_cache8(h, 16), api.make_cache8(h, 16)
        api.mla_latent_cache_append8(h, x, pos, slots, c)
        api.mla_cache8_store(h, cache.view(-1, 576)[slots], slots, d)
        assert api.mla_get_device_status(h) == 0
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c, d))
    bad = slots.clone()
    bad[7], pos[9] = 256, h.dims.max_position
    from head_latent_attention_qkv_gb300 import _lib
    e = api.make_cache8(h, 16)
    api.mla_latent_cache_append8(h, x, pos, bad, e)
    assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_SLOT | _lib.MLA_DEV_BAD_POSITION
    ok = torch.ones(256, dtype=torch.bool, device="cuda")
    ok[slots[[7, 9]]] = False
    assert torch.equal(e.latent.view(torch.uint8).view(256, 512)[ok], c.latent.view(torch.uint8).view(256, 512)[ok])
    assert (e.scale.view(-1)[~ok] == 1).all()


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("heads,T,n", [(32, 1, 3), (16, 6, 2), (4, 40, 4)])
def test_the_layer_is_its_steps(heads, T, n, tree):
    """The layer over the 8-bit cache: its attention is mla_latent_attention8's on the queries
    it leaves, its entries mla_latent_cache_append8's, and over a cache that 8 bits hold
    exactly it is the bf16 layer but for the attention's rounding."""
    from head_latent_attention_qkv_gb300 import _lib, api
    h = handle("bf16", heads, 16)
    ctx = [50 + 33 * b for b in range(n)]
    g = torch.Generator(device="cuda").manual_seed(heads)
    M, pages = n * T, 60
    x = torch.randn(M, h.dims.hidden_size, generator=g, device="cuda").bfloat16()
    parent = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").repeat(n) if tree else None
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[:15 * n].view(n, 15)
    kv = torch.tensor([c + T for c in ctx], dtype=torch.int32, device="cuda")
    pos = torch.tensor([c + i for c in ctx for i in range(T)], dtype=torch.int32, device="cuda")
    slots = torch.tensor([(int(table[b, (c + i) // 16]) * 16 + (c + i) % 16) for b, c in enumerate(ctx)
                          for i in range(T)], device="cuda")
    e = torch.randn(pages * 16, 576, generator=g, device="cuda").bfloat16()
    c8 = api.make_cache8(h, pages)
    every = torch.arange(pages * 16, device="cuda")
    api.mla_cache8_store(h, e, every, c8)
    desc = api.make_desc(table, kv, block_len=T)
    ws = torch.empty(api.mla_forward8_workspace_bytes(h, desc), dtype=torch.uint8, device="cuda")
    out = api.mla_draft_forward8(h, x, pos, slots, c8, desc, parent, workspace=ws)
    torch.cuda.synchronize()
    assert api.mla_get_device_status(h) == 0
    own = api.make_cache8(h, pages)
    api.mla_cache8_store(h, e, every, own)
    api.mla_latent_cache_append8(h, x, pos, slots, own)
    # (another split of the projection's K may round a latent to the neighbouring number)
    a, b = api.mla_cache8_load(h, c8, slots).float(), api.mla_cache8_load(h, own, slots).float()
    assert ((a - b).abs() <= 2.0 ** -3 * b.abs() + 2.0 ** -9).all()
    q = ws[api.mla_forward_workspace_offset(h, M, _lib.MLA_WS_Q_ABS):][:M * heads * 1152].view(torch.bfloat16)
    o = ws[api.mla_forward_workspace_offset(h, M, _lib.MLA_WS_O_LAT):][:M * heads * 1024].view(torch.float16)
    again = api.mla_latent_attention8(h, q.view(-1, 576), pos, c8, desc, parent)
    assert torch.equal(again, o.view(-1, 512))
    bf = api.mla_cache8_load(h, c8, every).view(pages, 16, 576).contiguous()
    want = (api.mla_draft_forward_tree(h, x, pos, None, bf, desc, parent) if tree else
            api.mla_draft_forward(h, x, pos, None, bf, desc))
    rms = want.float().pow(2).mean().sqrt()
    # (both are rounded to bf16, each off by 2^-8 of itself at most, which 2e-2 rms does not
    # hold for outputs of several rms)
    assert ((out.float() - want.float()).abs() <= 2e-2 * rms + 2.0 ** -8 * (out.float().abs() + want.float().abs())).all()
    assert (out.float() - want.float()).abs().mean() <= 2e-3 * rms


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("page,lens,n_keep", [(16, [40, 700, 3], [5, 300, 3]), (128, [1000, 129], [999, 1]),
                                              (64, [5000], [2500]), (32, [64, 64], [0, 64])])
def test_compaction_moves_what_the_entries_stand_for(page, lens, n_keep, in_place):
    # the 8-bit cache compacted and read back is the bf16 cache read back and compacted
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import Paged, i32
    h = handle("bf16", 4, page)
    rng = np.random.default_rng(page)
    p = Paged(rng, h.dims, page, lens, spare=60)
    c8 = to_cache8(h, p.cache, junk=False)
    every = torch.arange(p.num_pages * page, device="cuda")
    bf = api.mla_cache8_load(h, c8, every).view(p.num_pages, page, 576).contiguous()
    firsts = [n // 3 if k < n // 2 else 0 for n, k in zip(lens, n_keep)]
    width = max(max(n_keep), 1)
    keep = np.full((len(lens), width), -1)
    for b, (n, k, f) in enumerate(zip(lens, n_keep, firsts)):
        keep[b, :k] = np.sort(rng.choice(np.arange(f, n), size=k, replace=False))
    dst = None
    if not in_place:
        need = [-(-(f + k) // page) for f, k in zip(firsts, n_keep)]
        d = np.full((len(lens), max(max(need), 1)), -1)
        at = 0
        for b, x in enumerate(need):
            d[b, :x] = p.spare[at:at + x]
            at += x
        dst = i32(d)
    w = torch.from_numpy(rng.random((len(lens), max(lens) + 2)).astype(np.float32)).cuda()
    ws = [w.clone(), w.clone()]
    outs = [None, None] if in_place else [torch.full_like(w, -1.0) for _ in ws]
    args = (i32(p.table), i32(lens), i32(keep), i32(n_keep))
    api.mla_cache8_compact(h, c8, *args, first=i32(firsts), dst_block_table=dst, weights=ws[0], weights_out=outs[0])
    api.mla_cache_compact(h, bf, *args, first=i32(firsts), dst_block_table=dst, weights=ws[1], weights_out=outs[1])
    torch.cuda.synchronize()
    assert api.mla_get_device_status(h) == 0
    got = api.mla_cache8_load(h, c8, every).view_as(bf)
    assert torch.equal(got.nan_to_num(7.0), bf.nan_to_num(7.0))
    pair = ws if in_place else outs
    assert torch.equal(pair[0], pair[1])


def test_compaction_leaves_a_list_that_does_not_ascend_alone():
    from head_latent_attention_qkv_gb300 import _lib, api
    from tests.tree_cases import Paged, i32
    h = handle("bf16", 4, 16)
    p = Paged(np.random.default_rng(1), h.dims, 16, [90, 80])
    c8 = to_cache8(h, p.cache)
    before = [x.clone() for x in c8]
    keep = i32([[3, 9, 9, 20], [1, 2, 30, 40]])
    api.mla_cache8_compact(h, c8, i32(p.table), i32([90, 80]), keep, i32([4, 4]))
    assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_KEEP
    slots, other = p.slots(0, 90).cuda(), p.slots(1, 80).cuda()
    for x, y in zip(c8, before):
        x, y = (t.view(torch.uint8).reshape(p.num_pages * 16, -1) for t in (x, y))
        assert torch.equal(x[slots], y[slots])
        assert torch.equal(x[other[:4]], y[other[[1, 2, 30, 40]]])


@pytest.mark.parametrize("heads,T,kind", [(16, 8, "tree"), (32, 5, "chain")])
def test_serving_steps(heads, T, kind):
    """Three steps as a serving program takes them: the drafted tokens' entries written in 8 bits, their
    attention, verification, the accepted path compacted; then one token over what is left, against
    the oracle on the entries that stayed."""
    from head_latent_attention_qkv_gb300 import api
    from oracle import cache8 as O8, tree as O
    from tests.tree_cases import bushy, depths, i32
    rng = np.random.default_rng(T)
    page, n, V, pages = 16, 3, 5000, 90
    h = handle("bf16", heads, page)
    scale = 1.0 / np.sqrt(h.dims.qk_head_dim)
    table = rng.permutation(pages)[:n * 20].reshape(n, 20)
    c8 = api.make_cache8(h, pages)
    length, kept = [150, 61, 0], [np.zeros((0, 576)) for _ in range(n)]

    def slots(b, keys):
        return torch.from_numpy(table[b][keys // page] * page + keys % page).cuda()

    def store(b, keys):
        e = torch.from_numpy(rng.normal(size=(len(keys), 576)).astype(np.float32)).bfloat16()
        api.mla_cache8_store(h, e.cuda(), slots(b, keys), c8)
        return O8.dequantise(*O8.quantise(e.double().numpy()))

    for b in range(n):
        kept[b] = store(b, np.arange(length[b]))
    for step in range(3):
        parents = [bushy(rng, T) if kind == "tree" else list(range(-1, T - 1)) for _ in range(n)]
        own = [store(b, length[b] + np.arange(T)) for b in range(n)]
        kv, first, par = i32([x + T for x in length]), i32(length), i32(parents)
        pos = i32([x + d for x, q in zip(length, parents) for d in depths(q)])
        q = torch.from_numpy(rng.normal(size=(n * T * heads, 576)).astype(np.float32)).bfloat16().cuda()
        desc = api.make_desc(i32(table), kv, block_len=T)
        o = api.mla_latent_attention8(h, q, pos, c8, desc, parent=par.flatten())
        # (the layers above and the vocabulary's projection would follow)
        z = rng.normal(size=(n, T + 1, V)) * 2
        p = np.exp(z) / np.exp(z).sum(axis=-1, keepdims=True)
        d = 0.7 * p[:, :T] + 0.3 / V
        tokens = np.array([[rng.choice(V, p=d[b, parents[b][i] + 1]) for i in range(T)] for b in range(n)])
        u = rng.random((n, T + 1)).astype(np.float32)
        dev = [torch.from_numpy(x.astype(np.float32)).cuda() for x in (p, d)]
        accepted, count, token = api.mla_verify_drafts(h, *dev, i32(tokens), torch.from_numpy(u).cuda(), parent=par,
                                                       first=first)
        api.mla_cache8_compact(h, c8, i32(table), kv, accepted, count, first=first)
        torch.cuda.synchronize()
        assert api.mla_get_device_status(h) == 0 and torch.isfinite(o).all()
        for b in range(n):
            path, want = O8.verify(dev[0][b].double().cpu().numpy(), dev[1][b].double().cpu().numpy(),
                                   tokens[b].tolist(), u[b], parents[b])
            assert (accepted[b, :count[b]].cpu().numpy() - length[b]).tolist() == path and token[b] == want
            kept[b] = np.concatenate([kept[b], own[b][path]])
            length[b] += len(path)
    q = torch.from_numpy(rng.normal(size=(n * heads, 576)).astype(np.float32)).bfloat16().cuda()
    o = api.mla_latent_attention8(h, q, i32(length), c8, api.make_desc(i32(table), i32(length), block_len=1))
    assert api.mla_get_device_status(h) == 0
    for b in range(n):
        q64 = q.double().cpu().numpy().reshape(n, 1, heads, 576)[b]
        vis = np.ones((1, length[b]), dtype=bool)
        ref = O.attention(q64, kept[b], vis, 512, scale)[0][0]
        mass = O.weight_mass(q64, kept[b], vis, 512, scale)[0]
        got = o.double().cpu().numpy().reshape(n, heads, 512)[b]
        # as above, the scores' error taken at 2^-12 and the least weights at 2^-12 of the mass
        assert (np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -10) * mass + 2.0 ** -11 * np.abs(ref) + 1e-6).all()


def test_short_blocks_whole_and_cut():
    # tables that hold few tiles and wide ones, blocks without a key among them: equal results
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import i32
    for heads, T, ctx in ((16, 3, [0, 5, 200, 90]), (64, 2, [300, 0, 128]), (4, 1, [0])):
        c = Case8(heads, 32, ctx, T, seed=len(ctx), masked=T > 2)
        before = api.mla_kernel_launches(c.h)
        whole = c.attention()
        assert api.mla_kernel_launches(c.h) == before + 2             # no join, and the counts
        c.check_attention(*whole)
        wide = np.full((c.n, 900), -1)
        wide[:, :c.paged.max_pages] = c.paged.table
        c.keep[0] = i32(wide)
        c.desc = api.make_desc(c.keep[0], c.keep[1], None, c.keep[3], T, c.stats)
        c.check_attention(*c.attention())
        assert api.mla_kernel_launches(c.h) == before + 5
        c.keep[1].zero_()                                              # no keys at all
        c.desc.q_visible, c.parent = None, None
        for table in (c.keep[0], i32(c.paged.table)):
            desc = api.make_desc(table, c.keep[1], None, None, T)
            lse = torch.full((c.q.shape[0],), 3.0, device="cuda")
            o = api.mla_latent_attention8(c.h, c.q, c.positions, c.c8, desc, lse=lse)
            assert (o == 0).all() and torch.isneginf(lse).all()


def test_the_workspace_does_not_grow_with_the_rows():
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import i32
    h = handle("bf16", 128, 64)
    sizes = [api.mla_latent_attention8_workspace_bytes(h, api.make_desc(i32(np.zeros((n, 400))), i32([9] * n), block_len=T))
             for n, T in ((2, 1), (50, 16), (50, 700), (3000, 1))]
    assert 0 < sizes[0] <= sizes[-1] <= 21 << 20 and max(sizes) - min(sizes) <= 4 * 3100


def test_pieces_longer_than_what_one_sum_holds():
    # more than 64 tiles in a CTA: its parts are put away and joined (152 SMs, 1.3 M keys)
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import i32
    h = handle("bf16", 32, 128)
    n, kv = 12, 110000
    pages = -(-kv // 128)
    g = torch.Generator(device="cuda").manual_seed(5)
    c = api.make_cache8(h, pages)
    api.mla_cache8_store(h, torch.randn(pages * 128, 576, generator=g, device="cuda").bfloat16(),
                         torch.arange(pages * 128, device="cuda"), c)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(n, 1)
    q = torch.randn(n * 32, 576, generator=g, device="cuda").bfloat16()
    lens = i32([kv - 1000 * b for b in range(n)])
    lse = torch.empty(n * 32, device="cuda")
    o = api.mla_latent_attention8(h, q, lens, c, api.make_desc(table, lens, block_len=1), lse=lse)
    assert api.mla_get_device_status(h) == 0
    e = api.mla_cache8_load(h, c, torch.arange(kv, device="cuda")).double()
    scale = 1.0 / np.sqrt(h.dims.qk_head_dim)
    for b in range(0, n, 5):
        k = kv - 1000 * b
        s = q[32 * b:32 * b + 32].double() @ e[:k].T * scale
        p = torch.softmax(s, 1)
        ref, mass = p @ e[:k, :512], p @ e[:k, :512].abs()
        # a weight is off by 2^-8, and by 2^-20 of the largest; scores (std 1.7) by 2^-16 here
        tol = (2.0 ** -8 + 2.0 ** -14) * mass + 2.0 ** -20 * p.amax(1, keepdim=True) * e[:k, :512].abs().sum(0) + 2.0 ** -11 * ref.abs()
        assert ((o[32 * b:32 * b + 32].double() - ref).abs() <= tol).all()
        assert ((lse[32 * b:32 * b + 32].double() - torch.logsumexp(s, 1)).abs() <= 1e-4).all()


def test_refusals_on_the_host():
    import ctypes as C
    from head_latent_attention_qkv_gb300 import _lib, api
    lib, BAD, NO = _lib.lib, _lib.MLA_ERR_INVALID_ARG, _lib.MLA_ERR_UNSUPPORTED
    c = Case8(16, 16, [60], 4)
    h, ref, s = c.h.h, c.c8._ref, torch.cuda.current_stream().cuda_stream
    before = api.mla_kernel_launches(c.h)
    x = torch.zeros(4 * 16, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    assert lib.mla_cache8_store(h, x.data_ptr() + 2, slots.data_ptr(), 4, ref, 1, s) == BAD
    assert lib.mla_cache8_store(h, x.data_ptr(), None, 4, ref, 1, s) == BAD
    assert lib.mla_cache8_store(h, x.data_ptr(), slots.data_ptr(), -1, ref, 1, s) == BAD
    assert lib.mla_cache8_load(h, ref, 0, slots.data_ptr(), 4, x.data_ptr(), s) == BAD
    assert lib.mla_cache8_load(h, None, 1, slots.data_ptr(), 4, x.data_ptr(), s) == BAD
    for field in ("latent", "rope", "scale"):
        bad = _lib.mla_cache8_t(c.c8._c.latent, c.c8._c.rope, c.c8._c.scale)
        setattr(bad, field, getattr(bad, field) + 8)
        assert lib.mla_cache8_store(h, x.data_ptr(), slots.data_ptr(), 4, C.byref(bad), 1, s) == BAD
        setattr(bad, field, None)
        assert lib.mla_cache8_store(h, x.data_ptr(), slots.data_ptr(), 4, C.byref(bad), 1, s) == BAD
    d, q, pos = C.byref(c.desc), c.q.data_ptr(), c.positions.data_ptr()
    par, n = c.parent.data_ptr(), c.c8.num_pages
    o = torch.zeros(c.q.shape[0], 512, dtype=torch.float16, device="cuda").data_ptr()

    def attend(cache=ref, num_pages=n, desc=d, qp=q, op=o, ws=None, nws=0):
        return lib.mla_latent_attention8(h, qp, pos, cache, num_pages, desc, par, op, None, ws, nws, s)
    assert attend(cache=None) == BAD and attend(num_pages=0) == BAD and attend(num_pages=2 ** 27) == BAD
    assert attend(qp=None) == BAD and attend(qp=q + 2) == BAD and attend(op=o + 2) == BAD and attend(desc=None) == BAD
    wide = api.make_desc(torch.zeros(1, 900, dtype=torch.int32, device="cuda"), c.keep[1], block_len=4)
    need = api.mla_latent_attention8_workspace_bytes(c.h, wide)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    assert need > 0 and attend(desc=C.byref(wide)) == BAD
    assert attend(desc=C.byref(wide), ws=ws.data_ptr(), nws=need - 1) == BAD
    assert attend(desc=C.byref(wide), ws=ws.data_ptr() + 128, nws=need) == BAD
    long = api.make_desc(c.keep[0], c.keep[1], block_len=1025)
    assert attend(desc=C.byref(long)) == NO
    fp32 = handle("fp32", 4, 16)
    assert lib.mla_cache8_store(fp32.h, x.data_ptr(), slots.data_ptr(), 4, ref, 1, s) == NO
    assert lib.mla_latent_attention8(fp32.h, q, pos, ref, n, d, par, o, None, None, 0, s) == NO
    hidden = torch.zeros(4, c.h.dims.hidden_size, dtype=torch.bfloat16, device="cuda")
    need = api.mla_append8_workspace_bytes(c.h, 4)
    assert lib.mla_latent_cache_append8(h, hidden.data_ptr(), pos, slots.data_ptr(), 4, ref, n, ws.data_ptr(), need - 1, s) == BAD
    need = api.mla_forward8_workspace_bytes(c.h, c.desc)
    assert lib.mla_draft_forward8(h, hidden.data_ptr(), pos, None, ref, n, d, par, hidden.data_ptr(), ws.data_ptr(),
                                  min(need - 1, ws.numel()), s) == BAD
    assert api.mla_kernel_launches(c.h) == before
    with pytest.raises(ValueError):
        api.Cache8(c.c8.latent, c.c8.rope, c.c8.scale[:-1])
    with pytest.raises(ValueError):
        api.Cache8(c.c8.latent.view(torch.uint8), c.c8.rope, c.c8.scale)
    with pytest.raises(ValueError):
        api.mla_cache8_load(handle("bf16", 16, 32), c.c8, slots)
