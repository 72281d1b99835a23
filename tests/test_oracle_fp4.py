"""Pins of the 4-bit oracle (oracle/fp4_ref.py): closed forms of the formats, a brute-force nearest
search, ties, saturation and the stored layout."""
import numpy as np
import pytest

from oracle import fp4_ref as f4


def test_e4m3_values():
    assert len(f4.E4M3) == 127 and f4.E4M3[-1] == 448 and f4.E4M3[1] == 2.0 ** -9 and f4.E4M3[8] == 2.0 ** -6
    assert f4.E4M3[0x38] == 1.0 and (np.diff(f4.E4M3) > 0).all()


def test_nearest_even_by_brute_force():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(0, 8, 500), np.arange(0, 64) / 8, [100.0]])
    for points in (f4.VALUES, f4.E4M3):
        w = np.concatenate([v, (points[1:] + points[:-1]) / 2])
        got = f4.nearest_even(points, w)
        for x, g in zip(w, got):
            d = np.abs(points - x)
            best = np.flatnonzero(d == d.min())
            assert g == (best[0] if len(best) == 1 else next(b for b in best if b % 2 == 0)), x


def test_mx_scale_is_the_ocp_conversion():
    """X = 2^(floor(log2 amax) - 2): 4 <= amax / X < 8, values past 6 saturate."""
    x = np.zeros((1, 32))
    for top, scale in ((4.0, 1.0), (6.0, 1.0), (7.999, 1.0), (8.0, 2.0), (3.999, 0.5), (1.0, 0.25)):
        x[0, 0] = top
        c, s, r = f4.quantize(x, "mxfp4")
        assert 2.0 ** (int(s[0, 0]) - 127) == scale and r[0] == 1
    x[0, 0] = 7.999
    assert f4.dequantize(*f4.quantize(x, "mxfp4"), "mxfp4")[0, 0] == 6.0
    x[0, 0] = 0
    assert f4.quantize(x, "mxfp4")[1][0, 0] == 127


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 32))
    x[0, :8] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0]
    c, _, _ = f4.quantize(x, "mxfp4")
    assert f4.VALUES[c[0, :8] & 7].tolist() == [4, 0, 1, 1, 2, 2, 4, 4] and c[0, 7] == 14


def test_nv_row_scale():
    for top, r in ((2688.0, 1.0), (2688.5, 2.0), (1344.0, 0.5), (1.0, 2.0 ** -11), (0.0, 1.0)):
        x = np.zeros((1, 16))
        x[0, 3] = top
        _, s, row = f4.quantize(x, "nvfp4")
        assert row[0] == r, top
        if top:
            assert s[0, 0] == np.abs(f4.E4M3 - top / 6 / r).argmin()
        assert top <= 2688 * row[0]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_error_bound(fmt):
    """Within half a code step of the block's scale (a quarter of the largest where MXFP4 saturates, and
    half an e4m3 step of it for NVFP4)."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 128)) * np.exp2(rng.uniform(-20, 20, (40, 1)))
    y = f4.dequantize(*f4.quantize(x, fmt), fmt)
    B = f4.BLOCK[fmt]
    top = np.abs(x).reshape(40, -1, B).max(axis=2)
    err = np.abs(x - y).reshape(40, -1, B).max(axis=2)
    assert (err <= top * (0.25 if fmt == "mxfp4" else 1 / 6 + 1 / 16)).all()


def test_infinite_and_nan_blocks():
    x = np.ones((2, 64))
    x[0, 5], x[0, 40] = np.inf, np.nan
    for fmt in ("mxfp4", "nvfp4"):
        y = f4.dequantize(*f4.quantize(x, fmt), fmt)
        assert np.isnan(y[0, :16]).all() and np.isfinite(y[0, 48:]).all() == (fmt == "nvfp4")
        assert (np.abs(y[1] - 1) <= 1 / 16).all()


def test_tile_layout():
    s = np.arange(200 * 5, dtype=np.int64).reshape(200, 5).astype(np.uint8) | 1
    t = f4.tile_scales(s)
    assert t.size == 2 * 2 * 512
    assert t[0] == s[0, 0] and t[3] == s[0, 3] and t[16] == s[1, 0] and t[4] == s[32, 0]
    assert t[512] == s[0, 4] and t[513] == 0 and t[2 * 512 + 16] == s[129, 0]


def test_packing():
    c = np.arange(16, dtype=np.uint8).reshape(1, 16)
    assert f4.pack_codes(c)[0].tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
