"""Compaction of the 8-bit cache with weights narrower than a sequence (needs a GB300)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_cache8 import to_cache8  # noqa: E402
from tests.test_gpu_tree import handle  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("page,lens,width", [(16, [40, 90, 30], 60), (64, [700, 3000, 650], 2999)])
def test_a_sequence_longer_than_its_weights_is_left_alone(page, lens, width, in_place):
    # every array of it; the others go on
    from head_latent_attention_qkv_gb300 import _lib, api
    from tests.tree_cases import Paged, i32
    h = handle("bf16", 4, page)
    rng = np.random.default_rng(page)
    p = Paged(rng, h.dims, page, lens, spare=200)
    c8 = to_cache8(h, p.cache, junk=False)
    before = [x.clone() for x in c8]
    every = torch.arange(p.num_pages * page, device="cuda")
    bf = api.mla_cache8_load(h, c8, every).view(p.num_pages, page, 576).contiguous()
    n_keep = [n // 2 for n in lens]
    keep = np.full((3, max(n_keep)), -1)
    for b, (n, k) in enumerate(zip(lens, n_keep)):
        keep[b, :k] = np.sort(rng.choice(n, size=k, replace=False))
    dst, target = None, p.table
    if not in_place:
        per = -(-max(n_keep) // page)
        target = p.spare[:3 * per].reshape(3, per)
        dst = i32(target)
    w = torch.from_numpy(rng.random((3, width)).astype(np.float32)).cuda()
    ws = [w.clone(), w.clone()]
    outs = [None, None] if in_place else [torch.full_like(w, -1.0) for _ in ws]
    args = (i32(p.table), i32(lens), i32(keep), i32(n_keep))
    api.mla_cache8_compact(h, c8, *args, dst_block_table=dst, weights=ws[0], weights_out=outs[0])
    assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_LENGTH
    api.mla_cache_compact(h, bf, *args, dst_block_table=dst, weights=ws[1], weights_out=outs[1])
    assert api.mla_get_device_status(h) == _lib.MLA_DEV_BAD_LENGTH
    own = np.concatenate([p.table[1][p.table[1] >= 0]] + ([] if in_place else [target[1]]))
    own = torch.from_numpy(own.astype(np.int64)).cuda()
    for x, y in zip(c8, before):
        assert torch.equal(x.view(torch.uint8)[own], y.view(torch.uint8)[own])
    assert torch.equal(api.mla_cache8_load(h, c8, every).view_as(bf).nan_to_num(7.0), bf.nan_to_num(7.0))
    pair = ws if in_place else outs
    assert torch.equal(pair[0], pair[1])
