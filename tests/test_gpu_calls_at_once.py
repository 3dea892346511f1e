"""Attention over the 8-bit cache and verification, several calls in flight on two streams (needs a
GB300)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_cache8 import Case8  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_attention_calls_at_once():
    # everything is allocated before, nothing waits in between, every call is looked at
    from head_latent_attention_qkv_gb300 import api
    cases = [Case8(32, 64, [3000, 170, 900], 5, padded=True), Case8(32, 64, [2000, 2100], 3, seed=9)]
    want, calls = [c.attention() for c in cases], []
    for c, s in zip(cases, (torch.cuda.Stream(), torch.cuda.Stream())):
        need = api.mla_latent_attention8_workspace_bytes(c.h, c.desc)
        c.desc.vis_stats = None                      # (the same tensor for every call)
        outs = [(torch.full((len(c.q), 512), float("nan"), dtype=torch.float16, device="cuda"),
                 torch.full((len(c.q),), float("nan"), device="cuda")) for _ in range(8)]
        calls.append((c, s, outs, torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for i in range(8):
        for c, s, outs, ws in calls:
            api.mla_latent_attention8(c.h, c.q, c.positions, c.c8, c.desc, c.parent, *outs[i], stream=s, workspace=ws)
    torch.cuda.synchronize()
    for (_, _, outs, _), (o, lse) in zip(calls, want):
        for x, y in outs:
            assert torch.equal(x, o) and torch.equal(y, lse)


def test_verification_calls_at_once():
    from head_latent_attention_qkv_gb300 import api
    from tests.test_gpu_verify import Batch, the_handle
    from tests.tree_cases import i32
    h, calls = the_handle(), []
    for b in (Batch(16, 8, 40000, seed=3, kind="tree", noise=1.0), Batch(9, 5, 30001, seed=6)):
        want = b.run()
        b.check(want)
        args = (b.target.cuda(), b.draft.cuda(), i32(b.tokens), torch.from_numpy(b.u).cuda(), i32(b.parents), i32(b.first))
        calls.append((torch.cuda.Stream(), args, want, []))
    torch.cuda.synchronize()
    for _ in range(8):
        for s, args, _, got in calls:
            got.append(api.mla_verify_drafts(h, *args, stream=s))
    torch.cuda.synchronize()
    for _, _, want, got in calls:
        assert len(got) == 8
        for out in got:
            assert all((x.cpu().numpy() == y).all() for x, y in zip(out, want))
