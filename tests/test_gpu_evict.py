"""Key selection, cache compaction and a serving step of all the operators (needs a GB300).

Indices and moved entries are exact.
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


def handle(dtype, page, heads=2):
    from tests.tree_cases import make_handle
    key = (dtype, page, heads)
    if key not in HANDLES:
        HANDLES[key] = make_handle(dtype, heads, page)[0]
    return HANDLES[key]


def check_select(w, lens, budget, sink, recent):
    from head_latent_attention_qkv_gb300 import api
    from oracle import tree as O
    from tests.tree_cases import i32
    h = handle("fp32", 16)
    keep, num = api.mla_cache_select(h, torch.from_numpy(w).cuda(), i32(lens), budget, sink, recent)
    assert api.mla_get_device_status(h) == 0
    keep, num = keep.cpu().numpy(), num.cpu().numpy()
    for b, n in enumerate(lens):
        want = O.select(w[b], n, budget, sink, recent)
        assert num[b] == len(want)
        assert keep[b].tolist() == want + [-1] * (budget - len(want)), b


@pytest.mark.parametrize("width,lens,budget,sink,recent", [
    (40, [40, 0, 1, 17, 39], 16, 2, 5), (1, [1, 0], 1, 0, 0), (33, [33, 32, 31], 32, 0, 32),
    (700, [700, 256, 257, 255], 256, 0, 0), (8192, [8192, 8191, 4097], 100, 4, 64),
    (8193, [8193, 4097, 3], 4096, 4, 64), (20000, [20000, 16383], 16000, 0, 1),
    (50001, [50001], 1, 0, 0), (50001, [50000, 49999, 50], 777, 16, 512), (131072, [131071], 8192, 4, 64),
    (300001, [300001, 17], 5000, 1, 1)])
def test_select_matches_the_oracle(width, lens, budget, sink, recent):
    rng = np.random.default_rng(width)
    w = np.exp(2 * rng.normal(size=(len(lens), width))).astype(np.float32)
    w *= rng.random(w.shape) > 0.2                         # many equal zeros
    check_select(w, lens, budget, sink, recent)


@pytest.mark.parametrize("width", [900, 9000, 70000])
def test_select_orders_ties_zeros_infinities_and_nan(width):
    rng = np.random.default_rng(1)
    vals = np.array([0.0, -0.0, 1.0, 1.0 + 2 ** -23, np.inf, -np.inf, np.nan, -1.0, 1e-42, -1e-42],
                    dtype=np.float32)
    w = vals[rng.integers(0, len(vals), size=(2, width))]
    for budget in (1, width // 10, width // 3, width // 2, width - 7):
        check_select(w, [width, width - 5], budget, 0, 0)
    check_select(np.full((1, width), np.nan, dtype=np.float32), [width], width // 2, 0, 0)
    check_select(np.zeros((1, width), dtype=np.float32), [width], width // 2, 1, 1)


@pytest.mark.parametrize("width", [5, 9000])
def test_select_under_the_largest_budget(width):
    # the list's end is 2^31 - 1: an index that steps over it must not wrap
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import i32
    h = handle("fp32", 16)
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs a list of 8.6 GB")
    keep, num = api.mla_cache_select(h, torch.rand(1, width, device="cuda"), i32([5]), 2 ** 31 - 1, 2, 1)
    torch.cuda.synchronize()
    assert api.mla_get_device_status(h) == 0 and num.tolist() == [5]
    assert keep[0, :5].tolist() == [0, 1, 2, 3, 4]
    for part in keep[0, 5:].split(1 << 28):
        assert (part == -1).all()


def test_select_length_behind_the_row_is_reported():
    from head_latent_attention_qkv_gb300 import _lib, api
    from tests.tree_cases import i32
    h = handle("fp32", 16)
    w = torch.arange(20, dtype=torch.float32, device="cuda").view(2, 10)
    keep, num = api.mla_cache_select(h, w, i32([11, -1]), 4)
    assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_LENGTH
    assert keep.tolist() == [[6, 7, 8, 9], [-1] * 4] and num.tolist() == [4, 0]


def pick(rng, n, k, lo=0):
    return sorted(rng.choice(np.arange(lo, n), size=k, replace=False).tolist())


def run_compact(dtype, page, lens, keeps, firsts=None, in_place=True, weights=True, seed=0, ldk=None):
    from head_latent_attention_qkv_gb300 import api
    from oracle import tree as O
    from tests.tree_cases import Paged, i32
    rng = np.random.default_rng(seed)
    h = handle(dtype, page)
    new = [(firsts[b] if firsts else 0) + len(k) for b, k in enumerate(keeps)]
    dst_pages = 0 if in_place else sum(-(-m // page) for m in new)
    p = Paged(rng, h.dims, page, lens, spare=3 + dst_pages)
    n, width = len(lens), p.max_pages * page
    ldk = max([len(k) for k in keeps] + [1]) if ldk is None else ldk
    keep = np.full((n, ldk), -1, dtype=np.int32)
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = k
    dst = None
    if not in_place:
        dst = np.full((n, max(-(-max(new) // page), 1)), -1, dtype=np.int32)
        at = 0
        for b, m in enumerate(new):
            q = -(-m // page)
            dst[b, :q] = p.spare[at:at + q]
            at += q
    w0 = rng.random((n, width)).astype(np.float32)
    w = torch.from_numpy(w0).cuda() if weights else None
    w_out = None if not weights else (w if in_place else torch.full_like(w, -5.0))
    before = p.cache.clone()
    api.mla_cache_compact(h, p.cache, i32(p.table), i32(lens), i32(keep), i32([len(k) for k in keeps]),
                          first=None if firsts is None else i32(firsts),
                          dst_block_table=None if dst is None else i32(dst), weights=w, weights_out=w_out)
    torch.cuda.synchronize()
    assert api.mla_get_device_status(h) == 0
    want = before.view(-1, h.dims.cache_dim).clone()
    src = before.view(-1, h.dims.cache_dim)
    for b, k in enumerate(keeps):
        f = firsts[b] if firsts else 0
        old = p.slots(b, lens[b]).tolist()
        rows = O.compact(old, f, k)[:f + len(k)]
        to = p.slots(b, f + len(k), dst).tolist()
        if to:
            want[torch.tensor(to, device="cuda")] = src[torch.tensor(rows, device="cuda")]
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(p.cache.view(-1, h.dims.cache_dim).view(bits), want.view(bits))
    if weights:
        got = w_out.cpu().numpy()
        for b, k in enumerate(keeps):
            f = firsts[b] if firsts else 0
            ref = O.compact(w0[b].tolist(), f, k)
            ref = ref[:f + len(k)] + [0.0] * (lens[b] - f - len(k))
            assert got[b, :lens[b]].tolist() == [np.float32(x) for x in ref]
            assert (got[b, lens[b]:] == (w0[b, lens[b]:] if in_place else -5.0)).all()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("bf16", 128), ("fp32", 16), ("fp32", 48)])
def test_compact(dtype, page, in_place):
    rng = np.random.default_rng(page)
    lens = [0, 1, 5, 200, 333, 1000, 700]
    keeps = [[], [0], [1, 4], pick(rng, 200, 120), list(range(333)), pick(rng, 1000, 37), list(range(300, 700))]
    run_compact(dtype, page, lens, keeps, in_place=in_place)
    run_compact(dtype, page, lens, keeps, in_place=in_place, weights=False, ldk=1003)


@pytest.mark.parametrize("dtype,rows", [("bf16", 16), ("fp32", 16)])
def test_compact_of_one_chunk_a_sequence_in_place(dtype, rows):
    # no other chunk to wait for, yet every row stored is the source of the row before it
    n = 608
    for seed in range(4):
        run_compact(dtype, 16, [rows] * n, [list(range(1 + (b + seed) % 3, rows)) for b in range(n)], weights=False,
                    seed=seed)


@pytest.mark.parametrize("in_place", [True, False])
def test_compact_of_an_accepted_path(in_place):
    # the context stays; of 16 drafted nodes the accepted path moves up behind it
    ctx = [0, 100, 257]
    keeps = [[2, 3, 9], [100 + k for k in (0, 4, 5, 15)], []]
    run_compact("bf16", 64, [c + 16 for c in ctx], keeps, firsts=ctx, in_place=in_place)
    run_compact("fp32", 16, [c + 16 for c in ctx], keeps, firsts=ctx, in_place=in_place, weights=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_compact_in_place_of_long_sequences(dtype):
    # many chunks that wait for one another: every second row, all but the first, a far tail
    rng = np.random.default_rng(2)
    lens = [30000, 20011, 20000]
    keeps = [list(range(0, 30000, 2)), list(range(1, 20011)), pick(rng, 20000, 9000, 10500)]
    for seed in range(3):
        run_compact(dtype, 64, lens, keeps, seed=seed)


def test_compact_reports_lists_that_do_not_fit():
    from head_latent_attention_qkv_gb300 import _lib, api
    from tests.tree_cases import Paged, i32
    h = handle("bf16", 16)
    for keep, num, kv, bit in (([3, 2, 5], 3, 40, _lib.MLA_DEV_BAD_KEEP), ([1, 40, 41], 3, 40, _lib.MLA_DEV_BAD_KEEP),
                               ([1, 2, 3], 4, 40, _lib.MLA_DEV_BAD_KEEP), ([1, 2, 3], -1, 40, _lib.MLA_DEV_BAD_KEEP),
                               ([-1, 2, 3], 3, 40, _lib.MLA_DEV_BAD_KEEP), ([1, 2, 3], 3, 100, _lib.MLA_DEV_BAD_LENGTH)):
        p = Paged(np.random.default_rng(0), h.dims, 16, [40, 40])
        before = p.cache.clone()
        api.mla_cache_compact(h, p.cache, i32(p.table), i32([kv, 40]), i32([keep, [5, 6, 7]]), i32([num, 3]))
        assert api.mla_get_device_status(h) == bit
        flat, old = p.cache.view(-1, 576), before.view(-1, 576)
        s = p.slots(1, 40).cuda()
        assert torch.equal(flat[s[:3]], old[s[5:8]]) and torch.equal(flat[s[3:]], old[s[3:]])
        if num != 3:
            s = p.slots(0, 40).cuda()
            assert torch.equal(flat[s], old[s])                 # the sequence is left alone


@pytest.mark.parametrize("kv", [100, -1, 41])
def test_compact_leaves_a_sequence_of_a_bad_length_alone(kv):
    # behind the page table, negative, behind the rows of weights
    from head_latent_attention_qkv_gb300 import _lib, api
    from tests.tree_cases import Paged, i32
    h = handle("bf16", 16)
    p = Paged(np.random.default_rng(0), h.dims, 16, [40, 40])
    before = p.cache.view(torch.int16).clone()
    w = torch.rand(2, 40, device="cuda")
    w0 = w.clone()
    api.mla_cache_compact(h, p.cache, i32(p.table), i32([kv, 40]), i32([[1, 2, 3], [0, 1, 2]]), i32([3, 3]), weights=w)
    assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_LENGTH
    assert torch.equal(p.cache.view(torch.int16), before) and torch.equal(w[0], w0[0])
    assert torch.equal(w[1, :3], w0[1, :3]) and not w[1, 3:].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,at,value", [
    (400, 15, 3), (400, 16, 5), (400, 31, "same"), (400, 100, 400), (400, 199, -1), (400, 0, -5), (400, 150, 2 ** 30),
    (30000, 4095, 0), (30000, 4096, "same"), (30000, 14999, 29000), (12, 5, 2), (12, 0, 12)])
def test_compact_of_a_list_that_does_not_ascend(dtype, n, at, value):
    # in place a row could be the source of a row that no longer waits for it: the
    # whole sequence is left alone.  Into other pages only the row is.
    from head_latent_attention_qkv_gb300 import _lib, api
    from tests.tree_cases import Paged, i32
    h = handle(dtype, 16)
    rng = np.random.default_rng(n + at)
    k = n // 2
    keep = np.stack([np.arange(0, n, 2), np.sort(rng.choice(n, k, replace=False))]).astype(np.int32)
    keep[0, at] = keep[0, at - 1] if value == "same" else value
    pages = -(-k // 16)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    for in_place in (True, False):
        p = Paged(np.random.default_rng(1), h.dims, 16, [n, n], spare=2 * pages)
        dst = None if in_place else p.spare[:2 * pages].reshape(2, pages).astype(np.int32)
        w0 = torch.rand(2, n, device="cuda")
        w = w0.clone()
        w_out = w if in_place else torch.full_like(w, -5.0)
        flat = p.cache.view(-1, h.dims.cache_dim)
        want, want_w = flat.clone(), w_out.clone()
        for b in range(2):
            if in_place and b == 0:
                continue
            rows = np.arange(k)
            if b == 0:                                       # an index above the one before it, inside the sequence
                prev = np.concatenate([[-1], keep[0, :-1]])
                rows = rows[(keep[0] > prev) & (keep[0] < n) & (keep[0] >= rows)]
            old = p.slots(b, n).cuda()
            to = p.slots(b, k, dst).cuda()
            src = torch.from_numpy(keep[b][rows].astype(np.int64)).cuda()
            d = torch.from_numpy(rows).cuda()
            want[to[d]] = flat[old[src]]
            want_w[b, k:] = 0.0
            want_w[b, d] = w0[b, src]
        api.mla_cache_compact(h, p.cache, i32(p.table), i32([n, n]), i32(keep), i32([k, k]),
                              dst_block_table=None if in_place else i32(dst), weights=w, weights_out=w_out)
        assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_KEEP
        assert torch.equal(flat.view(bits), want.view(bits)), in_place
        assert torch.equal(w_out, want_w), in_place
        if in_place:                                         # without weights (12 keys: a single chunk, no flags)
            api.mla_cache_compact(h, p.cache, i32(p.table), i32([n, 0]), i32(keep), i32([k, 0]))
            assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_KEEP
            assert torch.equal(flat.view(bits), want.view(bits))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [-1, "behind"])
def test_compact_leaves_rows_of_a_bad_page_alone(dtype, bad, in_place):
    # neither the entry nor the weight of a row moves when its old or its new page is bad
    from head_latent_attention_qkv_gb300 import _lib, api
    from tests.tree_cases import Paged, i32
    h = handle(dtype, 16)
    p = Paged(np.random.default_rng(1), h.dims, 16, [80, 60], spare=8)
    bad = p.num_pages if bad == "behind" else bad
    keeps = [list(range(0, 80, 2)), list(range(20, 60))]
    table = p.table.copy()
    table[0, 2] = bad
    dst = None
    if not in_place:
        dst = p.spare[:6].reshape(2, 3).astype(np.int32).copy()
        dst[0, 1] = bad
    w0 = torch.rand(2, 80, device="cuda")
    w = w0.clone()
    w_out = w if in_place else torch.full_like(w, -5.0)
    flat = p.cache.view(-1, h.dims.cache_dim)
    want, want_w = flat.clone(), w_out.clone()
    for b, k in enumerate(keeps):
        want_w[b, len(k):p.lens[b]] = 0.0
        for d, s in enumerate(k):
            to = (table if in_place else dst)[b, d // 16]
            if table[b, s // 16] == bad or to == bad:
                continue
            want[int(to) * 16 + d % 16] = flat[int(table[b, s // 16]) * 16 + s % 16]
            want_w[b, d] = w0[b, s]
    api.mla_cache_compact(h, p.cache, i32(table), i32(p.lens), i32([k + [-1] * (40 - len(k)) for k in keeps]),
                          i32([40, 40]), dst_block_table=None if in_place else i32(dst), weights=w, weights_out=w_out)
    assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_PAGE
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(flat.view(bits), want.view(bits))
    assert torch.equal(w_out, want_w)


def test_compact_in_place_of_sequences_that_share_a_prompt():
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import Paged, i32
    h = handle("bf16", 16)
    rng = np.random.default_rng(6)
    p = Paged(rng, h.dims, 16, [100, 120, 64])
    p.table[1:, :4] = p.table[0, :4]                        # 64 keys of a shared prompt
    first = [64, 70, 64]
    keeps = [pick(rng, 100, 9, 64), pick(rng, 120, 20, 70), []]
    keep = np.full((3, 20), -1, dtype=np.int32)
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = k
    want = p.cache.view(-1, 576).clone()
    for b, k in enumerate(keeps):
        s = p.slots(b, p.lens[b])
        want[s[first[b]:first[b] + len(k)].cuda()] = p.cache.view(-1, 576)[s[k].cuda()]
    api.mla_cache_compact(h, p.cache, i32(p.table), i32(p.lens), i32(keep), i32([len(k) for k in keeps]),
                          first=i32(first))
    assert api.mla_get_device_status(h) == 0
    assert torch.equal(p.cache.view(-1, 576).view(torch.int16), want.view(torch.int16))


def test_compact_takes_any_workspace_that_is_large_enough():
    from head_latent_attention_qkv_gb300 import _lib, api
    from tests.tree_cases import Paged, i32
    h = handle("bf16", 16)
    p = Paged(np.random.default_rng(0), h.dims, 16, [400])
    args = (p.cache, i32(p.table), i32([400]), i32([list(range(0, 400, 2))]), i32([200]))
    need = api.mla_cache_compact_workspace_bytes(h, 1, 200)
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            api.mla_cache_compact(h, *args, workspace=bad)
    with pytest.raises(_lib.MLAError):
        api.mla_cache_compact(h, *args, workspace=torch.empty(need // 8 - 1, dtype=torch.int64, device="cuda"))
    want = p.cache.view(-1, 576)[p.slots(0, 400)[::2].cuda()].clone()
    api.mla_cache_compact(h, *args, workspace=torch.empty(need // 8, dtype=torch.int64, device="cuda"))
    assert api.mla_get_device_status(h) == 0
    assert torch.equal(p.cache.view(-1, 576)[p.slots(0, 200).cuda()], want)


def test_compact_behind_four_gigabytes():
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import Paged, i32
    h = handle("bf16", 64)
    rng, far = np.random.default_rng(4), 61000
    p = Paged(rng, h.dims, 64, [500, 200])
    cache = torch.empty(far + p.num_pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    cache[far:] = p.cache
    keep = [pick(rng, 500, 100), list(range(100, 200))]
    args = (i32([500, 200]), i32(keep), i32([100, 100]))
    api.mla_cache_compact(h, p.cache, i32(p.table), *args)
    api.mla_cache_compact(h, cache, i32(np.where(p.table >= 0, p.table + far, -1)), *args)
    assert api.mla_get_device_status(h) == 0
    assert torch.equal(cache[far:].view(torch.int16), p.cache.view(torch.int16))


def test_compact_captured_and_replayed():
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import Paged, i32
    h = handle("bf16", 64)
    rng = np.random.default_rng(3)
    p = Paged(rng, h.dims, 64, [5000])
    args = (i32(p.table), i32([5000]), i32([pick(rng, 5000, 2500)]), i32([2500]))
    start = p.cache.clone()
    api.mla_cache_compact(h, p.cache, *args)
    want = p.cache.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.mla_cache_compact(h, p.cache, *args)
    for _ in range(3):
        p.cache.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.cache.view(torch.int16), want.view(torch.int16))
    assert api.mla_get_device_status(h) == 0


@pytest.mark.parametrize("dtype,heads", [("fp32", 2), ("bf16", 16)])
def test_a_serving_step(dtype, heads):
    """Verify a tree, accept a path, weigh the keys, evict, and decode one token
    over what is left: the last output against the oracle on the kept entries."""
    from head_latent_attention_qkv_gb300 import api
    from oracle import tree as O
    from tests.tree_cases import Paged, bushy, depths, i32
    rng = np.random.default_rng(8)
    page, T, ctx = 16, 8, [150, 61]
    h = handle(dtype, page, heads)
    d = h.dims
    dt, scale = api.torch_dtype(d), 1.0 / np.sqrt(d.qk_head_dim)
    kv = [c + T for c in ctx]
    p = Paged(rng, d, page, kv)
    parents = [bushy(rng, T) for _ in ctx]
    pos = i32([c + x for c, par in zip(ctx, parents) for x in depths(par)])
    table, kvd, par = i32(p.table), i32(kv), i32(np.concatenate(parents))
    q = torch.from_numpy(rng.normal(size=(2 * T * heads, d.cache_dim)).astype(np.float32)).to(dt).cuda()
    desc = api.make_desc(table, kvd, block_len=T)
    lse = torch.empty(q.shape[0], device="cuda")
    api.mla_tree_attention(h, q, pos, p.cache, desc, par, lse=lse)
    w = torch.zeros(2, p.max_pages * page, device="cuda")
    api.mla_key_weights(h, q, pos, p.cache, desc, lse, w, prior=w, decay=0.9, parent=par)
    # each row's weights sum to one
    assert torch.allclose(w.sum(1), torch.full((2,), float(T * heads), device="cuda"), rtol=1e-4)
    # accept the path to the deepest node
    path = [O.paths(x)[int(np.argmax(depths(x)))] for x in parents]
    width = max(len(x) for x in path)
    keep = [[c + k for k in x] + [-1] * (width - len(x)) for c, x in zip(ctx, path)]
    api.mla_cache_compact(h, p.cache, table, kvd, i32(keep), i32([len(x) for x in path]), first=i32(ctx), weights=w)
    kvd = i32([c + len(x) for c, x in zip(ctx, path)])
    # evict to 64 keys
    kept, num = api.mla_cache_select(h, w, kvd, 64, sink=2, recent=8)
    wh = w.cpu().numpy()
    api.mla_cache_compact(h, p.cache, table, kvd, kept, num, weights=w)
    seqs = []
    for b in range(2):
        rows = list(range(ctx[b])) + [ctx[b] + k for k in path[b]]
        stay = O.select(wh[b], len(rows), 64, 2, 8)
        assert kept[b, :num[b]].tolist() == stay
        seqs.append(p.entries[b][[rows[j] for j in stay]])
    # decode one token over the kept keys
    q1 = torch.from_numpy(rng.normal(size=(2 * heads, d.cache_dim)).astype(np.float32)).to(dt).cuda()
    desc1 = api.make_desc(table, num, block_len=1)
    p1 = i32([c + len(x) for c, x in zip(ctx, path)])
    o = api.mla_tree_attention(h, q1, p1, p.cache, desc1, i32([-1, -1]))
    o0 = api.mla_latent_attention(h, q1, p1, p.cache, desc1)
    torch.cuda.synchronize()
    assert api.mla_get_device_status(h) == 0
    q64 = q1.double().cpu().numpy().reshape(2, 1, heads, -1)
    for b in range(2):
        n = len(seqs[b])
        vis = np.ones((1, n), dtype=bool)
        ref, _ = O.attention(q64[b], seqs[b], vis, d.kv_lora_rank, scale)
        mass = O.weight_mass(q64[b], seqs[b], vis, d.kv_lora_rank, scale)[0]
        # as in test_gpu_tree.py, the scores' error taken at 2^-12
        tol = (2.0 ** -11 + (2.0 ** -8 if dtype == "bf16" else 0)) * mass + 2.0 ** -11 * np.abs(ref[0])
        for got in (o, o0):
            g = got.double().cpu().numpy().reshape(2, heads, -1)[b]
            assert (np.abs(g - ref[0]) <= tol + 1e-6).all()
