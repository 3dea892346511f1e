"""Ways of calling the tree and eviction entry points (needs a GB300): two streams
at once, no sequences, a sequence named twice, outputs over their inputs.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def case(*a, **kw):
    from tests.test_gpu_tree import Case
    return Case(*a, **kw)


def step(c, stream=None):
    """Attention and key weights of a case; every output."""
    from head_latent_attention_qkv_gb300 import api
    lse = torch.empty(c.q.shape[0], device="cuda")
    w = torch.zeros(c.n, c.paged.max_pages * c.h.page_size, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    o = api.mla_tree_attention(c.h, c.q, c.positions, c.paged.cache, c.desc, c.parent, lse=lse, stream=stream)
    api.mla_key_weights(c.h, c.q, c.positions, c.paged.cache, c.desc, lse, w, parent=c.parent, stream=stream)
    kept, num = api.mla_cache_select(c.h, w, c.keep[1], 64, 2, 8, stream=stream)
    moved = c.paged.cache.clone()
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    api.mla_cache_compact(c.h, moved, c.keep[0], c.keep[1], kept, num, weights=w, stream=stream)
    return o, lse, w, kept, num, torch.nan_to_num(moved)


def test_two_streams_at_once():
    # one handle, calls that need workspaces of their own, none of which may be shared
    from head_latent_attention_qkv_gb300 import api
    a, b = case("bf16", 16, 64, [9001, 300], 4, seed=1), case("bf16", 16, 64, [7000, 5000], 4, seed=2)
    assert a.h is b.h
    want = [[x.clone() for x in step(c)] for c in (a, b)]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = [step(a, s), step(b, t), step(a, t), step(b, s)]
        torch.cuda.synchronize()
        for g, w in zip(got, want * 2):
            for x, y in zip(g, w):
                x, y = torch.nan_to_num(x), torch.nan_to_num(y)
                assert torch.equal(x, y)
    assert api.mla_get_device_status(a.h) == 0


@pytest.mark.parametrize("dtype,heads", [("fp32", 4), ("bf16", 16)])
def test_no_sequences(dtype, heads):
    from head_latent_attention_qkv_gb300 import api
    from tests.tree_cases import make_handle
    h = make_handle(dtype, heads, 16)[0]
    d, dt = h.dims, api.torch_dtype(h.dims)

    def empty(*shape, t=torch.int32):
        return torch.empty(*shape, dtype=t, device="cuda")

    cache = torch.zeros(4, 16, d.cache_dim, dtype=dt, device="cuda")
    table, kv, one = empty(0, 3), empty(0), empty(0)
    desc = api.make_desc(table, kv, block_len=5)
    before = api.mla_kernel_launches(h)
    assert api.mla_tree_attention(h, empty(0, d.cache_dim, t=dt), one, cache, desc, one).shape == (0, d.kv_lora_rank)
    assert api.mla_draft_forward_tree(h, empty(0, d.hidden_size, t=dt), one, None, cache, desc, one).shape == (0, d.hidden_size)
    w = empty(0, 48, t=torch.float32)
    api.mla_key_weights(h, empty(0, d.cache_dim, t=dt), one, cache, desc, empty(0, t=torch.float32), w, prior=w)
    keep, num = api.mla_cache_select(h, w, kv, 8)
    assert keep.shape == (0, 8) and num.shape == (0,)
    api.mla_cache_compact(h, cache, table, kv, keep, num, weights=w)
    torch.cuda.synchronize()
    assert api.mla_kernel_launches(h) == before and api.mla_get_device_status(h) == 0


@pytest.mark.parametrize("dtype,heads,T", [("fp32", 4, 5), ("bf16", 16, 5), ("bf16", 128, 16)])
def test_a_sequence_named_twice_and_weights_over_their_prior(dtype, heads, T):
    # two blocks read the same pages; the weights go over the prior (row parts, too)
    from head_latent_attention_qkv_gb300 import api
    c = case(dtype, heads, 16, [600], T, seed=4)
    _, lse = c.attention()
    two = lambda x: torch.cat([x, x]).contiguous()
    table, kv, pos, par = two(c.keep[0]), two(c.keep[1]), two(c.positions), two(c.parent)
    desc = api.make_desc(table, kv, block_len=T)
    lse2 = torch.empty(2 * lse.shape[0], device="cuda")
    o2 = api.mla_tree_attention(c.h, two(c.q), pos, c.paged.cache, desc, par, lse=lse2)
    rows = lse.shape[0]
    assert torch.equal(o2[:rows], o2[rows:]) and torch.equal(lse2[:rows], lse2[rows:])
    c.check_attention(o2[:rows], lse2[:rows])              # (two blocks may be cut otherwise than one)
    prior = torch.rand(2, c.paged.max_pages * 16, device="cuda")
    want = torch.full_like(prior, -1.0)
    api.mla_key_weights(c.h, two(c.q), pos, c.paged.cache, desc, lse2, want, prior=prior, decay=0.25, parent=par)
    over = prior.clone()
    api.mla_key_weights(c.h, two(c.q), pos, c.paged.cache, desc, lse2, over, prior=over, decay=0.25, parent=par)
    n = c.kv[0]
    assert torch.equal(over[:, :n], want[:, :n]) and torch.equal(over[:, n:], prior[:, n:])
    assert (want[:, n:] == -1).all()
    # equal blocks, equal sums
    zero = torch.zeros_like(prior)
    api.mla_key_weights(c.h, two(c.q), pos, c.paged.cache, desc, lse2, zero, parent=par)
    assert torch.equal(zero[0], zero[1])
    assert api.mla_get_device_status(c.h) == 0
