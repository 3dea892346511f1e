"""Pages outside an 8-bit cache, and scales that are no powers of two (needs a GB300)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_cache8 import Case8  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def behind(c, pages):
    """Case `c` with its pages behind `pages` others, which are returned."""
    from head_latent_attention_qkv_gb300 import api
    big = api.make_cache8(c.h, pages + c.paged.num_pages)
    for x, y in zip(big, c.c8):
        x[pages:].view(torch.uint8).copy_(y.view(torch.uint8))
    c.c8 = big
    c.keep[0].copy_(torch.where(c.keep[0] >= 0, c.keep[0] + pages, c.keep[0]))
    return [x.view(torch.uint8)[:pages] if x.dtype != torch.float32 else x[:pages] for x in big]


@pytest.mark.parametrize("first", [float("nan"), 0.0, 3.0, 1.0])
@pytest.mark.parametrize("page,ctx", [(16, [300, 200]), (128, [700, 500]), (64, [9000, 70])])
def test_a_page_outside_the_cache_reads_as_zeros(page, ctx, first):
    # whatever the cache's first entry holds: the result is that over a page of zeros
    from head_latent_attention_qkv_gb300 import _lib, api
    c = Case8(16, page, ctx, 4)
    latent, rope, scale = behind(c, 2)
    latent[0], rope[0], scale[0] = 0x7E, 0x7F, first
    table = c.keep[0].clone()
    c.keep[0][0, 1] = 1                              # (zeros, scale 1)
    want = c.attention()
    assert api.mla_get_device_status(c.h) == 0
    for bad in (c.c8.num_pages, -1, 2 ** 31 - 1):
        c.keep[0][0, 1] = bad
        got = c.attention()
        assert api.mla_get_device_status(c.h) == _lib.MLA_DEV_BAD_PAGE
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.keep[0].copy_(table)


@pytest.mark.parametrize("scale", [0.0, 3.0, -1.0, 1.0 + 2.0 ** -23, 2.0 ** -65, 2.0 ** 120, 1e-40, float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx", [[60, 20], [3000, 700]])
def test_a_scale_that_is_no_power_of_two_is_reported(ctx, scale):
    # (in units that lie in one CTA and in cut ones); it counts as NaN: its readers become NaN, others stay
    from head_latent_attention_qkv_gb300 import _lib, api
    T, H = 9, 16
    c = Case8(H, 16, ctx, T, parents=[[-1] * T, [-1] * T])
    want = c.attention()
    slot = c.paged.slots(0, c.kv[0])
    flat = c.c8.scale.view(-1)

    def rows(lo, hi):
        r = torch.zeros(2 * T * H, dtype=torch.bool, device="cuda")
        r[lo * H:hi * H] = True
        return r
    for key, (lo, hi) in ((ctx[0] + 4, (4, 5)), (30, (0, T))):         # a node's own key, one of the context
        was = flat[slot[key]].item()
        flat[slot[key]] = scale
        o, lse = c.attention()
        assert api.mla_get_device_status(c.h) == _lib.MLA_DEV_BAD_SCALE
        bad = rows(lo, hi)
        assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.equal(o[~bad], want[0][~bad]) and torch.equal(lse[~bad], want[1][~bad])
        flat[slot[key]] = was


def test_scales_at_the_ends_of_their_range_and_of_unseen_entries():
    from head_latent_attention_qkv_gb300 import api
    c = Case8(16, 16, [600, 20], 5, padded=True)     # (entries that nobody sees, and pages' ends, hold anything)
    want = c.attention()
    seen = torch.zeros(c.c8.scale.numel(), dtype=torch.bool)
    for b in range(c.n):
        seen[c.paged.slots(b, c.kv[b])[torch.from_numpy(c.vis[b].any(axis=0))]] = True
    for junk in (0.0, 3.0, -2.0, float("inf"), float("nan"), 1e-42):
        c.c8.scale.view(-1)[~seen.cuda()] = junk
        o, lse = c.attention()
        assert api.mla_get_device_status(c.h) == 0
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for k in (-64, 119):                             # zeros of the least scale, and of the largest
        c = Case8(16, 16, [40], 1, tree=False)
        c.c8.latent.view(torch.uint8).zero_()
        c.c8.rope.zero_()
        c.c8.scale.fill_(2.0 ** k)
        o, lse = c.attention()
        assert api.mla_get_device_status(c.h) == 0
        # (the log-sum-exp is the difference of two numbers below 2^7, one of them an fp32 logarithm good to
        # 2^-22 of itself)
        assert (o == 0).all() and ((lse - np.log(41)).abs() <= 2.0 ** -14).all()


def test_latents_of_zeros_keep_their_weight():
    # their scale is the least one, 2^-64, beside others of up to 2^13; every other key has such a latent
    from oracle import tree as O
    from tests.test_gpu_cache8 import rebuilt
    for q_scale, spread in ((1e-6, 21), (0.3, 1), (3.0, 1)):
        c = Case8(8, 64, [700, 90], 3, seed=4, q_scale=q_scale)
        for b, e in enumerate(c.paged.entries):
            e[:, :512] *= 2.0 ** np.random.default_rng(b).integers(1 - spread, spread, size=len(e))[:, None]
            e[::2, :512] = np.where(np.isnan(e[::2, :512]), np.nan, 0.0)
        rebuilt(c)
        o, lse = c.attention()
        # latents of 2^22 leave fp16: what rounds to 65536 or more is infinite there, so that an infinity is right
        # where the exact number, with the weights' 2^-8 and as much again, reaches 65520
        o, count = o.double().view(c.n, c.T, c.H, 512), 0
        for b, e in enumerate(c.paged.entries):
            ref = O.attention(c.q64[b], e, c.vis[b], 512, c.scale)[0]
            mass = O.weight_mass(c.q64[b], e, c.vis[b], 512, c.scale)
            inf = o[b].isinf().cpu().numpy()
            assert (np.abs(ref[inf]) + 2.0 ** -7 * mass[inf] >= 65520).all()
            assert (np.sign(ref[inf]) == np.sign(o[b].cpu().numpy()[inf])).all()
            o[b] = torch.where(o[b].isinf(), torch.from_numpy(ref).cuda(), o[b])
            count += inf.sum()
        assert (count > 0) == (spread > 1)
        c.check_attention(o, lse)
