"""Pins of the oracle of the 8-bit cache and of verification (CPU)."""
import numpy as np
import pytest

from oracle import cache8 as O

torch = pytest.importorskip("torch")


def test_codes_are_the_types_own():
    x = np.concatenate([O.E4M3[:127], -O.E4M3[:127], np.linspace(-448, 448, 4001), 2.0 ** np.linspace(-14, 8.8, 997)])
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (O.to_e4m3(x.astype(np.float32)) == want).all()
    vals = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(vals, O.E4M3.astype(np.float32), equal_nan=True)


def test_a_rounding_is_off_by_half_a_step_and_reading_back_is_exact():
    rng = np.random.default_rng(0)
    e = torch.from_numpy((rng.normal(size=(200, 576)) * np.exp(rng.normal(size=(200, 1)) * 20)).astype(np.float32))
    e = e.bfloat16().double().numpy()
    codes, rope, scale = O.quantise(e)
    back = O.dequantise(codes, rope, scale)
    err = np.abs(back - e)[:, :512]
    assert (err <= np.maximum(2.0 ** -4 * np.abs(e[:, :512]), scale[:, None] * 2.0 ** -10)).all()
    assert (np.abs(e[:, :512]).max(axis=1) <= 448 * scale).all()
    assert ((np.abs(e[:, :512]).max(axis=1) > 224 * scale) | (scale == 2.0 ** -64)).all()
    assert (torch.from_numpy(back).bfloat16().double().numpy() == back).all()
    again = O.dequantise(*O.quantise(back))
    assert (again == back).all()


def test_entries_that_8_bits_do_not_hold_are_nan():
    e = np.ones((4, 576))
    e[0, 3], e[1, 570], e[2, 511] = np.nan, np.inf, 2.0 ** 127
    codes, _, scale = O.quantise(e)
    assert np.isnan(scale[:3]).all() and scale[3] == 2.0 ** -8 and (codes[:3] == 0).all()


def _law(target, draft, parent, T, V, n, seed):
    """Frequencies of the first token behind the context over n draws."""
    rng = np.random.default_rng(seed)
    count = np.zeros(V)
    for _ in range(n):
        if draft is None:
            tokens = list(np.argsort(-target[0], kind="stable")[:T])
        else:
            tokens = [rng.choice(V, p=draft[p + 1]) for p in parent]
        path, token = O.verify(target, draft, tokens, rng.random(T + 1), parent)
        count[tokens[path[0]] if path else token] += 1
    return count / n


@pytest.mark.parametrize("parent", [[-1, 0, 1], [-1, -1, -1], [-1, -1, 0]])
@pytest.mark.parametrize("certain", [False, True])
def test_tokens_follow_the_targets_law(parent, certain):
    # the kept tokens are the target's own, whatever the draft: frequencies of n draws
    # lie within 5 sqrt(p (1 - p) / n) of p
    rng = np.random.default_rng(3)
    V, T, n = 6, 3, 20000
    target = rng.dirichlet(np.ones(V), T + 1)
    draft = None if certain else rng.dirichlet(np.ones(V), T)
    if certain:
        parent = [-1] * T                       # siblings are distinct then
    f = _law(target, draft, parent, T, V, n, 11)
    assert (np.abs(f - target[0]) <= 5 * np.sqrt(target[0] * (1 - target[0]) / n)).all()


def test_closed_forms():
    p = np.array([[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.2, 0.3, 0.5]])
    q = np.array([[0.25, 0.5, 0.25], [0.0, 0.5, 0.5]])
    assert O.verify(p, q, [0, 1], [0.99, 0.99, 0.49]) == ([0, 1], 1)        # p >= q: kept; 0.2 <= 0.49 < 0.5
    assert O.verify(p, q, [1, 1], [0.6, 0.0, 0.3]) == ([], 0)               # 0.6 * 0.5 >= 0.25; left: token 0 alone
    assert O.verify(p, q, [0, 2], [0.0, 0.0, 0.3], first=7) == ([7], 1)     # nothing of token 2 in row 1
    assert O.verify(p, None, [1, 2], [0.3, 0.1, 0.9], parent=[-1, -1]) == ([1], 2)   # 0.1 * 0.75 < 0.25
    assert O.verify(np.zeros((1, 4)), None, [], [0.5]) == ([], -1)
    assert O.verify(p, q, [5, 0], [0.1, 0.1, 0.6], parent=[-1, -1]) == ([1], 2)
