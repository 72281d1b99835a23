"""4-bit projections at the model's own widths (3840 and 10240) and 1,024 rows or more, against oracle/fp4_ref.py.

Products over K = 10240: the tolerance of test_gpu_fp4.py.  A whole block, on sampled rows: the bars derived in
test_gpu_fp4_model.py (relative ones, at any width): QKV and w1|w3 7e-2 and cosine 0.995, every projection 0.2 and 0.98.
The update without x takes the FFN's difference whole where it outweighs the attention's: 4e-2 under the same bar with
QKV and w1|w3, 0.21 with every projection: bar 0.3, cosine 1 - 0.3^2 / 2 rounded down to 0.95."""
import os

import numpy as np
import pytest

from gpu_util import assert_parity, require_gpu, torch
import zimage_inputs as zi
from oracle import fp4_ref as f4
from oracle import zimage_ref as ref
from test_gpu_fp4 import check_product, random_matrix

pytestmark = pytest.mark.gpu
S_TXT, GRID = 32, 32  # 1,024 image tokens and their text: 1,056 rows


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from stream_diffusion_transformer_b200 import abi
    abi.lib()
    abi.clear_device_status()
    yield
    assert abi.device_status() == 0


@pytest.mark.parametrize("M,N,K", [(1, 3840, 10240), (33, 264, 10240), (128, 264, 10240), (129, 3840, 10240), (1153, 776, 10240)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_over_the_ffn_width(fmt, M, N, K):
    from stream_diffusion_transformer_b200 import model
    rng = np.random.default_rng(M + N + K)
    a, av = random_matrix(rng, M, K, fmt)
    b, bv = random_matrix(rng, N, K, fmt, 0.02)
    check_product(model.gemm_fp4(a, b), av, bv)


@pytest.fixture(scope="module")
def block():
    from stream_diffusion_transformer_b200 import model
    d, prefix = zi.FULL, "layers.0"
    bits = zi.make_weights(d, seed=51, keys=model.block_keys(prefix, True), threads=max(1, min(32, os.cpu_count() or 1)))
    cfg = model.make_config(d)
    x = zi.make_stream(d, 1, GRID * GRID + S_TXT, seed=51)
    return d, prefix, bits, cfg, model.DeviceBlock(cfg, prefix, bits, True, "cuda"), x, zi.make_cond(d, 1, seed=51)


@pytest.mark.slow
@pytest.mark.parametrize("fmt,projections", [("nvfp4", "all"), ("mxfp4", "all"), ("nvfp4", True)])
def test_block_at_full_width(block, fmt, projections):
    from stream_diffusion_transformer_b200 import model
    d, prefix, bits, cfg, blk, x, c = block
    four = blk.with_fp4(fmt, projections)
    S = x.shape[1]
    if projections == "all":  # the packed weight itself, on sampled rows
        some = np.array([0, 1, 127, 128, 2047, d.dim - 1])
        w2 = ref.Weights(bits)(f"{prefix}.feed_forward.w2.weight")[some]
        code = f4.quantize(w2, fmt)[0]
        np.testing.assert_array_equal(four.t["w2_4"].cpu().numpy()[some], f4.pack_codes(code))
    xt, ct = torch.from_numpy(x).cuda(), torch.from_numpy(c).cuda()
    pos = model.positions(S_TXT, GRID, GRID)
    # two workspaces holding different bytes: the result is what the call computes alone
    from stream_diffusion_transformer_b200 import abi
    need = abi.block_workspace_size(cfg, 1, S)
    got, again = (model.block_forward(cfg, four, ct, pos, xt, ws=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
                  for fill in (0x00, 0x5A))
    assert torch.equal(got, again)
    rows = np.array([0, 1, 31, 127, 128, 500, 1023, 1024, 1040, S - 1])
    ang = ref.rope_angles(ref.position_ids(S_TXT, GRID, GRID), d.rope_axes)
    x0 = x[0].astype(np.float64)
    want = f4.block_forward_rows(x0, ref.Weights(bits), prefix, d, ang, c[0].astype(np.float64), rows, fmt, projections == "all")
    rel, cos = (0.2, 0.98) if projections == "all" else (7e-2, 0.995)
    got = got[0].cpu().numpy()[rows]
    assert_parity(got, want, rel=rel, cos=cos, what=f"{fmt} {projections}")
    if projections == "all":
        rel, cos = 0.3, 0.95
    assert_parity(got - x0[rows], want - x0[rows], rel=rel, cos=cos, what=f"{fmt} {projections} update")
