"""Pages outside an 8-bit cache (needs a GB300)."""
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
