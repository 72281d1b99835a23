"""GPU test of the 4-bit product where row scales are far from 1: NVFP4 rows from 2^-120 to 2^120 in every pairing.

An element may be off by what test_gpu_fp4.py allows (2^-8 of it and K 2^-23 sum |a b|) and, below bf16's normal
numbers, by half a step of 2^-133 and as much again for the fp32 result's own.  Past bf16's largest number it is
infinite."""
import numpy as np
import pytest

from gpu_util import require_gpu, torch
from oracle import fp4_ref as f4

pytestmark = pytest.mark.gpu
POWERS = [-120, -90, -74, -64, -40, -1, 0, 1, 40, 64, 74, 90, 120]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from stream_diffusion_transformer_b200 import abi
    abi.lib()
    abi.clear_device_status()
    yield
    assert abi.device_status() == 0


def rows(rng, n, K, cols):
    """n rows of random values in `cols`, row i times 2^POWERS[i mod 13]: a 4-bit matrix and its exact values (fp64)."""
    from stream_diffusion_transformer_b200 import model
    x = np.zeros((n, K))
    x[:, cols] = rng.standard_normal((n, K))[:, cols]
    x *= np.ldexp(1.0, np.array(POWERS)[np.arange(n) % len(POWERS)])[:, None]
    m = model.quantize_fp4(torch.from_numpy(x.astype(np.float32)).cuda())
    return m, torch.from_numpy(f4.rows_values(x.astype(np.float32), "nvfp4")).cuda()


@pytest.mark.parametrize("M,N,K", [(13, 104, 256), (29, 136, 4096), (60, 136, 96), (117, 136, 256), (600, 520, 256), (1300, 784, 96)])
def test_products_of_rows_of_any_size(M, N, K):
    from stream_diffusion_transformer_b200 import model
    rng = np.random.default_rng(M + N + K)
    everywhere = np.ones(K, bool)
    a, av = rows(rng, M, K, everywhere)
    b, bv = rows(rng, N, K, everywhere)
    got, want = model.gemm_fp4(a, b).double(), av @ bv.t()
    tol = 2.0 ** -8 * want.abs() + K * 2.0 ** -23 * (av.abs() @ bv.abs().t()) + 2.0 ** -133
    top = torch.finfo(torch.bfloat16).max
    finite, over = want.abs() + tol < top, want.abs() - tol > top * (1 + 2.0 ** -8)
    assert finite.any() and over.any()
    assert ((got - want).abs() <= tol)[finite].all(), float(((got - want).abs() / tol)[finite].nan_to_num(1e30).max())
    assert torch.equal(got[over], torch.copysign(torch.full_like(got[over], float("inf")), want[over]))
    # rows that share no column: zero whatever their scales
    half = np.arange(K) < K // 2
    got = model.gemm_fp4(rows(rng, M, K, half)[0], rows(rng, N, K, ~half)[0])
    assert (got == 0).all()
