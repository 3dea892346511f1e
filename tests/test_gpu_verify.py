"""Verification of drafted tokens against the fp64 oracle (needs a GB300): whole
numbers, equal to the oracle's.

The oracle's sums are exact to 2^-53 and the library's to 2^-40; a draw of the tests
would have to fall within 2^-40 of a border to differ, which the oracle is asked
about before the comparison.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def the_handle():
    from tests.test_gpu_tree import handle
    return handle("fp32", 4, 16)


def distributions(rng, n, T, V, dt, noise):
    z = rng.normal(size=(n, T + 1, V)) * 2.5

    def soft(x):
        x = np.exp(x - x.max(axis=-1, keepdims=True))
        return torch.from_numpy((x / x.sum(axis=-1, keepdims=True)).astype(np.float32)).to(dt)
    return soft(z), soft(z[:, :T] + noise * rng.normal(size=(n, T, V)))


def tree(rng, T, kind):
    if kind == "chain":
        return list(range(-1, T - 1))
    if kind == "star":
        return [-1] * T
    live = rng.integers(T // 2, T + 1)
    return [int(rng.integers(max(-1, i - 4), i)) if i < live else -2 for i in range(T)]


class Batch:
    def __init__(self, n, T, V, dtype="fp32", kind="chain", certain=False, noise=0.5, seed=0):
        rng = np.random.default_rng(seed)
        self.n, self.T, self.V = n, T, V
        self.target, self.draft = distributions(rng, n, T, V, TYPES[dtype], noise)
        self.parents = [tree(rng, T, kind) for _ in range(n)]
        self.tokens = np.zeros((n, T), dtype=np.int32)
        for b in range(n):
            used = {}
            for i, p in enumerate(self.parents[b]):
                q = self.draft[b, max(p, -1) + 1].double().numpy()
                if certain:
                    order, k = np.argsort(-q, kind="stable"), used.get(p, 0)
                    used[p] = k + 1
                    self.tokens[b, i] = order[min(k, V - 1)]
                else:
                    self.tokens[b, i] = rng.choice(V, p=q / q.sum())
        if certain:
            self.draft = None
        self.u = rng.random((n, T + 1)).astype(np.float32)
        self.first = rng.integers(0, 1000, n)

    def run(self, parent=True, first=True, **kw):
        from head_latent_attention_qkv_gb300 import api
        i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        out = api.mla_verify_drafts(
            the_handle(), self.target.cuda(), None if self.draft is None else self.draft.cuda(), i32(self.tokens),
            torch.from_numpy(self.u).cuda(), parent=i32(self.parents) if parent else None,
            first=i32(self.first) if first else None, **kw)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in out]

    def oracle(self, b, nudge=0.0, first=True):
        from oracle import cache8 as O
        u = self.u[b].astype(np.float64) * (1 + nudge)
        return O.verify(self.target[b].double().numpy(), None if self.draft is None else self.draft[b].double().numpy(),
                        self.tokens[b].tolist(), u, self.parents[b], int(self.first[b]) if first else 0)

    def check(self, got, status=0, first=True):
        from head_latent_attention_qkv_gb300 import api
        assert api.mla_get_device_status(the_handle()) == status
        path, count, token = got
        for b in range(self.n):
            want = self.oracle(b, first=first)
            for nudge in (2.0 ** -40, -2.0 ** -40):
                assert self.oracle(b, nudge, first) == want, "a draw on a border: take another seed"
            p, t = want
            assert count[b] == len(p) and path[b].tolist() == p + [-1] * (self.T - len(p)) and token[b] == t, b


CASES = [
    # sequences, nodes, vocabulary, options
    (3, 5, 1000, {}), (1, 1, 1, {}), (2, 3, 2, {}), (5, 0, 77, {}), (4, 7, 31, dict(kind="star")),
    (3, 6, 4097, dict(kind="tree")), (2, 4, 32000, {}), (2, 9, 4096, dict(kind="tree", noise=2.0)),
    (1, 12, 50001, dict(kind="star", noise=3.0)), (3, 8, 20011, dict(dtype="bf16", kind="tree", noise=1.5)),
    (2, 5, 151936, dict(dtype="fp16")), (2, 6, 5000, dict(certain=True, kind="star")),
    (4, 9, 333, dict(certain=True, kind="tree")), (2, 4, 9999, dict(certain=True, dtype="bf16")),
    (2, 300, 50, dict(kind="tree", noise=1.0)), (1, 1024, 64, dict(kind="tree", noise=0.1)),
    (1, 1024, 40, dict(certain=True, kind="chain", noise=0.0)), (70, 4, 600, dict(kind="tree")),
    # whole lots of 16-byte loads: each type, refused siblings in them
    (2, 6, 70016, dict(certain=True, kind="star")), (2, 5, 81920, dict(certain=True, kind="star", dtype="bf16")),
    (1, 5, 90112, dict(certain=True, kind="star", dtype="fp16")), (2, 5, 40000, dict(kind="star", noise=3.0, dtype="bf16")),
    (40, 2, 33000, dict(noise=1.0)), (160, 1, 9000, dict(noise=1.0)), (320, 1, 2600, dict(noise=2.0)),
]


@pytest.mark.parametrize("n,T,V,opt", CASES)
def test_verify(n, T, V, opt):
    for seed in range(3):
        b = Batch(n, T, V, seed=seed, **opt)
        b.check(b.run())


def test_many_draws():
    # every kind of end: all kept, refused at each depth, several siblings refused
    b = Batch(500, 4, 97, kind="tree", noise=1.0, seed=5)
    got = b.run()
    b.check(got)
    assert set(got[1]) >= {0, 1, 2}


def test_a_chain_needs_no_parents_and_first_is_optional():
    b = Batch(6, 5, 5003, seed=2)
    for x, y in zip(b.run(), b.run(parent=False)):
        assert (x == y).all()
    got = b.run(parent=False, first=False)
    b.check(got, first=False)


def test_rows_may_be_parts_of_longer_ones():
    b = Batch(3, 4, 5003, seed=4)
    want = b.run()
    pad = torch.full((3, 5, 5100), float("nan"))
    pad[:, :, :5003] = b.target
    dpad = torch.full((3, 4, 6001), 3.0)
    dpad[:, :, 8:5011] = b.draft
    from head_latent_attention_qkv_gb300 import api
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    got = api.mla_verify_drafts(the_handle(), pad.cuda()[:, :, :5003], dpad.cuda()[:, :, 8:5011], i32(b.tokens),
                                torch.from_numpy(b.u).cuda(), parent=i32(b.parents), first=i32(b.first))
    assert all((x.cpu().numpy() == y).all() for x, y in zip(got, want))


@pytest.mark.parametrize("V", [6000, 60000])
def test_masses_at_the_edges(V):
    from head_latent_attention_qkv_gb300 import _lib, api
    b = Batch(6, 3, V, seed=8, kind="star")
    b.target[0, 0] = b.draft[0, 0]                   # the draft's own law: kept for every u < 1
    b.u[0, 0] = 1 - 2.0 ** -24
    b.target[1, 0] = 0.0                             # no mass at all
    b.target[2, 0] = 0.0
    b.target[2, 0, V - 1] = 1.0                      # one token, the last
    b.u[2] = 1 - 2.0 ** -24
    b.target[3, 0, ::7] = float("nan")
    b.target[3, 0, 1::7] = -1.0
    b.target[3, 0, 2::7] = float("inf")
    b.u[4, 3] = 0.0
    b.target[4, 0, :10] = 0.0
    b.target[5, 0] = b.draft[5, 0] * 0.5             # refused, nothing left: the target's row itself
    b.u[5, :3] = 0.75
    got = b.run()
    b.check(got, status=_lib.MLA_DEV_BAD_DRAFT)
    assert got[1][0] == 1 and got[2][1] == -1 and got[2][2] == V - 1 and got[1][5] == 0
    assert api.mla_get_device_status(the_handle()) == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [500, 6000, 60000])
def test_draft_numbers_that_do_not_count(V, dtype):
    # one, two and three refusals at the context: what the draft's bad numbers leave of the
    # target's mass decides about the next sibling and the token
    b = Batch(12, 3, V, dtype=dtype, seed=21, kind="star", noise=3.0)
    rng = np.random.default_rng(3)
    for i, bad in enumerate((float("inf"), float("nan"), -1.0, float("-inf"))):
        at = torch.from_numpy(rng.choice(V, size=V // 6, replace=False))
        b.draft[3 * i:3 * i + 3, 0, at] = bad
    b.draft[0, 0, :] = float("inf")                  # nothing that counts
    b.u[:, :3] = 0.999
    b.tokens[1::2, 0] = b.target[1::2, 0].float().argmin(dim=1).numpy()
    b.check(b.run())


def test_bad_tokens_and_parents_are_reported():
    from head_latent_attention_qkv_gb300 import _lib
    b = Batch(3, 4, 500, seed=1, kind="star")
    b.tokens[0, 0], b.tokens[1, 2] = 500, -1
    b.check(b.run(), status=_lib.MLA_DEV_BAD_DRAFT)
    b = Batch(3, 4, 500, seed=1)
    b.parents[2][1] = 1
    b.check(b.run(), status=_lib.MLA_DEV_BAD_TREE)
    b = Batch(2, 4, 500, seed=1, kind="star")         # (what is not in the tree may hold anything)
    b.parents[0][1], b.tokens[0, 1] = -2, 10 ** 6
    b.check(b.run())


def test_equal_bits_replays_and_streams():
    b = Batch(16, 8, 40000, seed=3, kind="tree", noise=1.0)
    want = b.run()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    c = Batch(9, 5, 30001, seed=6)
    ref = c.run()
    for _ in range(3):
        x, y = b.run(stream=s), c.run(stream=t)
    assert all((p == q).all() for p, q in zip(x, want)) and all((p == q).all() for p, q in zip(y, ref))
    from head_latent_attention_qkv_gb300 import api
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    args = [b.target.cuda(), b.draft.cuda(), i32(b.tokens), torch.from_numpy(b.u).cuda()]
    kw = dict(parent=i32(b.parents), first=i32(b.first))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = api.mla_verify_drafts(the_handle(), *args, **kw)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all((p.cpu().numpy() == q).all() for p, q in zip(got, want))


def test_a_long_run_is_staged_in_parts():
    # one CTA a sequence (many of them): its warps' runs are longer than what is staged at once
    b = Batch(640, 1, 25000, seed=3, noise=0.3)
    b.check(b.run())


def test_refusals():
    from head_latent_attention_qkv_gb300 import _lib, api
    lib, h = _lib.lib, the_handle()
    b = Batch(2, 3, 50)
    t, d = b.target.cuda(), b.draft.cuda()
    tok = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    u, out = torch.zeros(2, 4, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    s, BAD = torch.cuda.current_stream().cuda_stream, _lib.MLA_ERR_INVALID_ARG
    before = api.mla_kernel_launches(h)

    def call(target=t.data_ptr(), ldt=50, draft=d.data_ptr(), ldd=50, dtype=1, tokens=tok.data_ptr(), un=u.data_ptr(),
             n=2, T=3, V=50, acc=out.data_ptr(), cnt=out.data_ptr(), nxt=out.data_ptr()):
        return lib.mla_verify_drafts(h.h, target, ldt, draft, ldd, dtype, tokens, None, un, None, n, T, V, acc, cnt, nxt, s)
    for kw in (dict(target=None), dict(ldt=49), dict(ldd=49), dict(dtype=3), dict(dtype=-1), dict(tokens=None),
               dict(un=None), dict(n=-1), dict(T=-1), dict(V=0), dict(acc=None), dict(cnt=None), dict(nxt=None),
               dict(target=t.data_ptr() + 2), dict(draft=d.data_ptr() + 1)):
        assert call(**kw) == BAD, kw
    assert call(T=1025) == _lib.MLA_ERR_UNSUPPORTED and call(n=0) == _lib.MLA_OK
    assert lib.mla_verify_drafts(None, None, 1, None, 1, 1, None, None, None, None, 1, 1, 1, None, None, None, s) == BAD
    assert api.mla_kernel_launches(h) == before
    for bad in (t[:, :, :49], t[:, :3], t.double(), t.cpu(), t.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            api.mla_verify_drafts(h, bad, d, tok, u)
    with pytest.raises(ValueError):
        api.mla_verify_drafts(h, t, d.half(), tok, u)
