"""Pins of the 8-bit and routing oracles against independent statements of the definitions."""
import numpy as np
import pytest

from oracle import fp8_ref as F
from oracle import moe_ref as M


def test_e4m3_values_match_torch():
    torch = pytest.importorskip("torch")
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(v, nan=-1.0), np.nan_to_num(F.E4M3, nan=-1.0))
    assert np.nanmax(F.E4M3) == 448.0


def test_rounding_is_to_nearest_even():
    pos = F.E4M3[:127]
    assert np.array_equal(F.round_e4m3(pos), np.arange(127))
    mid = (pos[1:] + pos[:-1]) / 2
    even = np.arange(126) + (np.arange(126) % 2)
    assert np.array_equal(F.round_e4m3(mid), even)
    assert np.array_equal(F.round_e4m3(-mid), even | 128)
    assert np.array_equal(F.round_e4m3(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(F.round_e4m3(np.nextafter(mid, 1e9)), np.arange(126) + 1)
    rng = np.random.default_rng(0)
    v = rng.standard_normal(4000) * np.exp(rng.uniform(-9, 4, 4000))
    v = v.clip(-448, 448)
    near = np.abs(np.abs(v)[:, None] - pos[None]).argmin(1)      # no exact ties among these
    assert np.array_equal(F.round_e4m3(v) & 127, near)


@pytest.mark.parametrize("e8m0", [False, True])
def test_scales(e8m0):
    top = np.array([448.0, 449.0, 447.0, 1.0, 1e-30, 0.0, 3e38])
    s = F.block_scales(top, e8m0)
    assert s[0] == 1.0 and s[5] == 2.0 ** -126
    assert np.all(top / s <= 448 * (1 + 2 ** -23))
    if e8m0:
        assert np.array_equal(np.log2(s), np.round(np.log2(s)))
        assert s[1] == 2.0 and s[2] == 1.0 and np.all(top[:5] / s[:5] > 223)
    assert np.isnan(F.block_scales(np.inf, e8m0)) and np.isnan(F.block_scales(np.nan, e8m0))


def test_quantize_error_is_at_most_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((130, 272))
    for rows in (1, 128):
        q, s = F.ref_quantize(x, rows, False)
        d = F.dequantize(q, s, rows)
        sx = np.repeat(np.repeat(s, rows, 0)[:130], 128, 1)[:, :272]
        # half a step: 2^-4 of the value, or 2^-10 of the scale below the normal range
        assert np.all(np.abs(d - x) <= np.maximum(np.abs(x) * 2.0 ** -4, sx * 2.0 ** -10) * (1 + 1e-12))


def test_product_by_blocks():
    rng = np.random.default_rng(2)
    xq, wq = rng.integers(0, 126, (3, 300)).astype(np.uint8), rng.integers(0, 126, (140, 300)).astype(np.uint8)
    xs, ws = rng.random((3, 3)), rng.random((2, 3))
    y, _ = F.ref_matmul(xq, xs, wq, ws)
    for r, o in ((0, 0), (2, 127), (1, 128), (2, 139)):
        want = sum(xs[r, c // 128] * ws[o // 128, c // 128] * F.E4M3[xq[r, c]] * F.E4M3[wq[o, c]] for c in range(300))
        assert abs(y[r, o] - want) <= 1e-9 * abs(want)


def test_route_by_hand():
    l = np.array([1.0, 3.0, 3.0, 2.0])
    ids, w = M.ref_route_token(l, 2, renormalize=False)
    assert ids.tolist() == [1, 2] and np.allclose(w, np.exp(3.0) / np.exp(l).sum())
    ids, w = M.ref_route_token(l, 2, bias=np.array([0.0, 0.0, -1.0, 0.0]), scoring="sigmoid", scale=2.0)
    s = 1 / (1 + np.exp(-l))
    assert ids.tolist() == [1, 3] and np.allclose(w, 2 * s[[1, 3]] / (s[1] + s[3]))
    # groups {0, 1} and {2, 3}: by the best (3 and 3, the lower group), by two best (4 and 5)
    assert M.ref_route_token(l, 2, n_groups=2, top_groups=1)[0].tolist() == [1, 0]
    assert M.ref_route_token(l, 2, n_groups=2, top_groups=1, group_score="top2")[0].tolist() == [2, 3]
    # nothing left: ids -1
    ids, w = M.ref_route_token(np.array([-np.inf, np.nan, 0.5, -np.inf]), 3)
    assert ids.tolist() == [2, -1, -1] and w.tolist() == [1.0, 0.0, 0.0]


def test_group_and_combine_by_hand():
    ids = np.array([[1, 0], [1, 7], [0, 1]], dtype=np.int32)
    off, rows, place = M.ref_group(ids, 3)
    assert off.tolist() == [0, 2, 5, 5] and rows.tolist() == [0, 2, 0, 1, 2, -1]
    assert place.tolist() == [[2, 0], [3, -1], [1, 4]]
    flat = ids.reshape(-1)
    keep = np.flatnonzero(flat < 3)
    assert np.array_equal(rows[:5], keep[np.argsort(flat[keep], kind="stable")] // 2)
    y = np.arange(10.0).reshape(5, 2)
    out, _ = M.ref_combine(y, place, np.full((3, 2), 0.5))
    assert out.tolist() == [[2.0, 3.0], [3.0, 3.5], [5.0, 6.0]]
