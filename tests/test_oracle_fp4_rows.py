"""The sampled-rows form of the oracle's 4-bit block gives the whole block's rows."""
import dataclasses

import numpy as np
import pytest

import zimage_inputs as zi
from oracle import fp4_ref as f4
from oracle import zimage_ref as ref


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("modulated,projections", [(True, True), (False, False)])
def test_rows_of_a_block(fmt, modulated, projections):
    d = dataclasses.replace(zi.TINY, ffn=704)
    keys = [k for k, _, _ in zi.block_specs("layers.0", d, modulated)]
    W = ref.Weights(zi.make_weights(d, seed=3, keys=keys, threads=2))
    x = zi.make_stream(d, 1, 24, seed=3)[0].astype(np.float64)
    c = zi.make_cond(d, 1, seed=3)[0].astype(np.float64) if modulated else None
    ang = ref.rope_angles(ref.position_ids(8, 4, 4), d.rope_axes)
    rows = np.array([0, 5, 15, 16, 23])
    whole = f4.block_forward(x, W, "layers.0", d, ang, c, fmt, projections)
    part = f4.block_forward_rows(x, W, "layers.0", d, ang, c, rows, fmt, projections)
    # products of other shapes may sum in another order, which can cross a border of the 4-bit grid
    assert np.linalg.norm(part - whole[rows]) <= 1e-3 * np.linalg.norm(whole[rows])
