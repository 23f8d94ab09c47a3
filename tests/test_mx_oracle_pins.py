"""Pins of the microscaled, norm and router oracles against hand values and
closed forms (no GPU)."""
import numpy as np
import pytest

from oracle import mx_oracle as M
from oracle import route_oracle as R


def test_grids():
    assert M.GRID4[-1] == 6 and M.GRID8[-1] == 448 and len(M.GRID8) == 127
    assert M.GRID8[1] == 2.0 ** -9 and M.GRID8[8] == 2.0 ** -6
    assert (np.diff(M.GRID8) > 0).all()


def test_scale_is_the_smallest_that_clips_nothing():
    v = np.zeros((1, 32 * 5))
    v[0, 0], v[0, 33], v[0, 70], v[0, 100] = 6.0, -6.0001, 448.0, 3.0     # 1, 2, 75 -> 128 (6 * 128 = 768), 0.5
    k = M.scale_exponents(v, 6.0)
    assert k.tolist() == [[0, 1, 7, -1, -127]]
    assert M.scale_exponents(v, 448.0).tolist() == [[-6, -6, 0, -7, -127]]
    assert M.scale_exponents(np.array([[np.inf], [np.nan], [3e38], [1e-45]]), 6.0).ravel().tolist() == [128, 128, 126, -127]


def test_ties_go_to_the_even_code():
    v = np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, -0.0]])
    codes, k = M.quantize(v, M.GRID4)
    assert k.tolist() == [[0]]
    assert codes.tolist() == [[7, 0, 2, 2, 4, 4, 6, 6, 8, 14, 8]]


@pytest.mark.parametrize("grid,half", [(M.GRID4, 2.0 ** -2), (M.GRID8, 2.0 ** -4)])
def test_rounding_is_within_half_a_step(grid, half):
    # relative half step of a normal value (one mantissa bit: 1/4, three: 1/16),
    # absolute half step below the smallest normal one
    v = np.random.default_rng(3).normal(size=(64, 256))
    codes, k = M.quantize(v, grid)
    d = np.abs(M.values(codes, k, grid) - v)
    unit = 2.0 ** np.repeat(k, 32, axis=1)
    assert (d <= np.maximum(half * np.abs(v), grid[1] / 2 * unit)).all()


def test_pack_places_every_nibble_and_scale():
    rng = np.random.default_rng(4)
    v = rng.normal(size=(150, 200))
    codes, k = M.quantize(v, M.GRID4)
    buf = M.pack4(codes, k)
    L = M.layout(150, 200, True)
    assert L == {"cols_padded": 256, "q_bytes": 32768, "s_offset": 32768, "s_bytes": 2048, "total": 34816}
    for r, c in [(0, 0), (127, 127), (128, 128), (149, 199), (5, 131)]:
        tile = (r // 128) * 2 + c // 128
        byte = buf[tile * 8192 + (r % 128) * 64 + (c % 128) // 2]
        assert (byte >> (4 * (c % 2))) & 15 == codes[r, c]
        b = c // 32
        assert buf[L["s_offset"] + tile * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] == k[r, b] + 127
    # rows of a tile's scale atom: 512 distinct places
    assert len(np.unique(M.scale_places(128, 128))) == 512


def test_rmsnorm_closed_form():
    h, y = M.rmsnorm(np.full((2, 8), 3.0), np.full((2, 8), 1.0), np.arange(8.0), eps=0.0)
    assert (h == 4).all() and np.allclose(y, np.arange(8.0))


def test_route_hand_values():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, g = R.route_select(l, None, 2, sigmoid=False)
    assert ids.tolist() == [[2, 1]] and np.allclose(g, [[4 / 6, 2 / 6]])
    ids, g = R.route_select(l, None, 2, sigmoid=False, renorm=False, scale=2.0)
    assert np.allclose(g, [[1.0, 0.5]])
    # the bias moves the choice, not the gate
    ids, g = R.route_select(l, [1.0, 0, 0, 0], 2, sigmoid=False)
    assert ids.tolist() == [[0, 2]] and np.allclose(g, [[1 / 5, 4 / 5]])
    # ties to the lower index, and to the lower group
    assert R.route_select(np.zeros((1, 6)), None, 3, True)[0].tolist() == [[0, 1, 2]]
    assert R.route_select(np.zeros((1, 6)), None, 2, True, 3, 1, 2)[0].tolist() == [[0, 1]]
    # groups: {0,1} sums to 1.0, {2,3} to 1.1 though expert 0 is the best
    b = [0.4, -0.4, 0.05, 0.05]
    assert R.route_select(np.zeros((1, 4)), b, 1, True, 2, 1, 2)[0].tolist() == [[2]]
    assert R.route_select(np.zeros((1, 4)), b, 1, True, 2, 1, 1)[0].tolist() == [[0]]
    # masked experts come last with gate 0; all masked: gates 0
    ids, g = R.route_select(np.array([[-np.inf, 1.0, -np.inf]]), None, 2, False)
    assert ids.tolist() == [[1, 0]] and g.tolist() == [[1.0, 0.0]]
    ids, g = R.route_select(np.full((1, 3), np.nan), None, 2, True)
    assert ids.tolist() == [[0, 1]] and g.tolist() == [[0.0, 0.0]]
