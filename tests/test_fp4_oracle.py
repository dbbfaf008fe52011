"""Pins of the 4-bit floating-point and routing oracle (oracle/fp4.py): decoded
grids against torch's float8 types, nearest codes by brute force, tiles by
their definition, the sort by counting."""
import numpy as np
import pytest
import torch

from oracle import fp4


def test_e4m3_against_torch():
    b = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(fp4.e4m3_decode(b), want.astype(np.float64), equal_nan=True)
    rng = np.random.default_rng(0)
    v = np.concatenate([np.exp2(rng.uniform(-14, 8.8, 20000)), fp4._E4M3, (fp4._E4M3[1:] + fp4._E4M3[:-1]) / 2, [448, 449, 1e9]])
    v = v.astype(np.float32)
    want = torch.from_numpy(v).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp4.e4m3_encode(v.astype(np.float64)), want)


def test_e2m1_nearest_even():
    q = np.concatenate([np.linspace(-7, 7, 2801), (fp4.GRID[1:] + fp4.GRID[:-1]) / 2])
    for v, c in zip(q, fp4.e2m1_encode(q)):
        d = np.abs(fp4.GRID - abs(v))
        best = np.flatnonzero(d == d.min())
        assert (c & 7) == (best[0] if best.size == 1 else best[best % 2 == 0][0])
        assert (c >> 3) == np.signbit(v)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quantize_by_hand(fmt):
    n = fp4.BLOCK[fmt]
    x = np.zeros((2, n))
    x[0, :4] = [6, -3, 0.25, 0.75]      # scale 1: codes 7, 5 + sign, tie to 0, tie to 2
    x[1, 0] = 7.9                       # mx: saturates at 6; nv: 7.9 / 6 -> 1.375 (E4M3), code 6 * 1.375
    c, s, v = fp4.quantize(x, fmt)
    assert list(c[0, :4]) == [7, 13, 0, 2] and list(v[0, :4]) == [6, -3, 0, 1]
    assert s[0, 0] == (0x38 if fmt == "nv" else 127)
    assert v[1, 0] == (6 * 1.375 if fmt == "nv" else 6)
    assert np.array_equal(fp4.values(fp4.pack(c), fp4.tile(s), fmt), v)


def test_mx_scale_is_floor_log2():
    for a, e in [(1.0, -2), (1.99, -2), (2.0, -1), (2.0**-126, -127), (2.0**-149, -127), (3e38, 125)]:
        _, s, _ = fp4.quantize(np.full((1, 32), a).astype(np.float32).astype(np.float64), "mx")
        assert int(s[0, 0]) - 127 == e


def test_tiles_follow_the_definition():
    R, J = 300, 11
    s = np.random.default_rng(1).integers(0, 256, (R, J)).astype(np.uint8)
    t = fp4.tile(s)
    flat, kb = t.reshape(-1), t.shape[1]
    for r, j in [(0, 0), (31, 3), (32, 4), (127, 10), (128, 0), (299, 7)]:
        assert flat[((r // 128) * kb + j // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + j % 4] == s[r, j]
    assert np.array_equal(fp4.untile(t, R, J), s)


def test_sort_by_counting():
    ids = np.array([[2, 0], [2, -1], [5, 0], [0, 7]])
    pos, off, cnt = fp4.sort(ids, 6, 4)
    assert cnt.tolist() == [3, 0, 2, 0, 0, 1] and off.tolist() == [0, 4, 4, 8, 8, 8, 12]
    assert pos.tolist() == [[4, 0], [5, -1], [8, 1], [2, -1]]
