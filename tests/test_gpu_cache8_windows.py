"""Windows of trees over the 8-bit cache whose positions run ahead of the keys' indices (needs a
GB300).  Bounds as in ``tests/test_gpu_cache8.py``."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_cache8 import Case8  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# (of every two blocks the first has the window; nodes that end at a multiple of 128 keys, straddle one,
# begin behind one)
AHEAD = [246, 9, 251, 9, 118, 9, 128, 9, 0, 9, 600]


@pytest.mark.parametrize("shift", [1, 60, 1000, 2 ** 30])
@pytest.mark.parametrize("heads,page,T,window,opt", [
    (16, 16, 10, 64, dict(padded=True)), (3, 128, 33, 4, {}), (32, 64, 10, 1, dict(masked=True)), (16, 64, 10, 40, dict(tree=False)),
])
def test_windows_over_positions_ahead_of_the_keys(monkeypatch, heads, page, T, window, opt, shift):
    # a node's window counts positions, wherever its key lies: a node sees itself at least
    import tests.tree_cases as cases
    depths = cases.depths
    if opt.get("tree", True):
        monkeypatch.setattr(cases, "depths", lambda parent: [d + shift for d in depths(parent)])
    c = Case8(heads, page, AHEAD, T, window=window, **opt)
    if not opt.get("tree", True):                    # (blocks: nothing is seen behind the window)
        c.positions += shift
        o, lse = c.attention()
        rows = torch.from_numpy(np.repeat([[i + shift >= window for i in range(T)]] * c.n, heads, axis=1).reshape(c.n, -1))
        rows[1::2] = False
        rows = rows.flatten().cuda()
        assert shift < 60 or (o[rows] == 0).all() and torch.isneginf(lse[rows]).all()
        return
    c.check_attention(*c.attention())
