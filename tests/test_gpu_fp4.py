"""GPU tests of the 4-bit rows and their product against oracle/fp4_ref.py and fp64 products.

Rows: codes, block scales, row scales and read-back values are bit-exact.  Product: the operands are exact in
fp64, so an element may be off by the rounding of its bf16 result (2^-8 of it) and by fp32 accumulation:
each of the K terms' additions rounds to at worst 2^-23 of the sum of magnitudes so far, K 2^-23 sum |a b| in all."""
import numpy as np
import pytest

from gpu_util import require_gpu, torch
from oracle import fp4_ref as f4

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from stream_diffusion_transformer_b200 import abi
    abi.lib()
    abi.clear_device_status()
    yield
    assert abi.device_status() == 0


def edge_rows(cols):
    """Ties in every block, values one fp32 step off a tie, saturation, zeros of both signs, tiny and huge
    rows, blocks that underflow beside large ones, infinities and NaN."""
    rng = np.random.default_rng(3)
    ties = np.array([6, 4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -2.5, -5, -0.0, 0.0] * 2, np.float32)
    base = np.tile(ties, -(-cols // 32))[:cols]
    rows = [base, np.nextafter(base, np.float32(np.inf)), np.nextafter(base, np.float32(-np.inf)), base * 448,
            np.nextafter(base * np.float32(448), np.float32(np.inf)), base * np.float32(2 ** -13), np.zeros(cols, np.float32),
            base * np.float32(1e-37), base * np.float32(1e-42), base * np.float32(5e37)]
    spread = (rng.standard_normal(cols) * np.exp2(rng.uniform(-30, 30, cols))).astype(np.float32)
    rows += [spread, np.where(np.arange(cols) < 16, 1e6, 1e-3).astype(np.float32)]
    # block maxima on and beside the borders between two e4m3 scales: 6 * midpoint * 2^k
    mids = (f4.E4M3[1:] + f4.E4M3[:-1]) / 2
    for step in (0, 1, -1):
        r = np.zeros(cols, np.float32)
        r[0] = 2688
        for j, c in enumerate(range(16, cols, 16)):
            v = np.float32(6 * mids[(j * 7) % len(mids)])
            r[c] = v if step == 0 else np.nextafter(v, np.float32(step * np.inf))
        rows.append(r)
    bad = spread.copy()
    bad[1], bad[cols - 1] = np.inf, np.nan
    rows.append(bad)
    return np.stack(rows).astype(np.float32)


def check_rows(x, fmt, bf16):
    from stream_diffusion_transformer_b200 import model
    t = torch.from_numpy(x).cuda()
    if bf16:
        t = t.bfloat16()
        x = t.float().cpu().numpy()
    m = model.quantize_fp4(t, fmt)
    code, stored, row = f4.quantize(x, fmt)
    np.testing.assert_array_equal(m.codes.cpu().numpy(), f4.pack_codes(code))
    np.testing.assert_array_equal(m.block_scales.cpu().numpy(), f4.tile_scales(stored))
    if fmt == "nvfp4":
        np.testing.assert_array_equal(m.row_scales.cpu().numpy().astype(np.float64), row)
    want = f4.dequantize(code, stored, row, fmt)
    np.testing.assert_array_equal(model.dequantize_fp4(m, torch.float32).cpu().numpy(), want.astype(np.float32))
    want16 = torch.from_numpy(want).to(torch.bfloat16).float().numpy()  # exact above the subnormal numbers
    np.testing.assert_array_equal(model.dequantize_fp4(m).float().cpu().numpy(), want16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("fmt", FMTS)
def test_rows_edges(fmt, bf16):
    for cols in (32, 96, 2592):
        check_rows(edge_rows(cols), fmt, bf16)


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (129, 160), (200, 1056), (5, 2560), (33, 3840), (7, 4128),
                                       (2, 10240), (1, 16384)])
@pytest.mark.parametrize("fmt", FMTS)
def test_rows_sizes(fmt, rows, cols):
    rng = np.random.default_rng(rows * cols)
    x = (rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32)
    check_rows(x, fmt, False)
    check_rows(x, fmt, True)


def random_matrix(rng, rows, cols, fmt, scale=1.0):
    """A random 4-bit matrix on the GPU and its exact values (fp64, on the GPU)."""
    from stream_diffusion_transformer_b200 import model
    x = (rng.standard_normal((rows, cols)) * scale * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32)
    code, stored, row = f4.quantize(x, fmt)
    m = model.Fp4Matrix(fmt, torch.from_numpy(f4.pack_codes(code)).cuda(), torch.from_numpy(f4.tile_scales(stored)).cuda(),
                        torch.from_numpy(row.astype(np.float32)).cuda() if fmt == "nvfp4" else None)
    return m, torch.from_numpy(f4.dequantize(code, stored, row, fmt)).cuda()


def check_product(got, a, b):
    want = a @ b.t()
    tol = 2.0 ** -8 * want.abs() + a.shape[1] * 2.0 ** -23 * (a.abs() @ b.abs().t())
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all() and (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 3840, 3840), (2, 136, 96), (16, 128, 256), (17, 264, 544), (33, 1000, 1184),
                                   (64, 256, 320), (65, 120, 2592), (128, 512, 768), (129, 384, 288), (300, 776, 1056),
                                   (513, 512, 512), (1000, 1032, 608), (1153, 3848, 2592)])
@pytest.mark.parametrize("fmt", FMTS)
def test_product(fmt, M, N, K):
    from stream_diffusion_transformer_b200 import model
    rng = np.random.default_rng(M + N + K)
    a, av = random_matrix(rng, M, K, fmt)
    b, bv = random_matrix(rng, N, K, fmt, 0.02)
    out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    check_product(model.gemm_fp4(a, b, out=out[:M]), av, bv)
    assert (out[M] == 7.0).all()  # rows behind the last stay as they were


@pytest.mark.parametrize("fmt", FMTS)
def test_product_scales_reach_their_own_elements(fmt):
    """Operands of ones whose scales alone differ: every row and block of both sides counts once."""
    from stream_diffusion_transformer_b200 import model
    for M, N, K in ((200, 392, 704), (700, 520, 704)):
        B, rng = f4.BLOCK[fmt], np.random.default_rng(5)
        sides = []
        for R in (M, N):
            code = np.full((R, K), 2, np.uint8)
            stored = (rng.integers(120, 135, (R, K // B)) if fmt == "mxfp4" else rng.integers(40, 80, (R, K // B))).astype(np.uint8)
            row = np.exp2(rng.integers(-3, 4, R)).astype(np.float64)
            if fmt == "mxfp4":
                row[:] = 1
            m = model.Fp4Matrix(fmt, torch.from_numpy(f4.pack_codes(code)).cuda(),
                                torch.from_numpy(f4.tile_scales(stored)).cuda(),
                                torch.from_numpy(row.astype(np.float32)).cuda() if fmt == "nvfp4" else None)
            sides.append((m, torch.from_numpy(f4.dequantize(code, stored, row, fmt)).cuda()))
        check_product(model.gemm_fp4(sides[0][0], sides[1][0]), sides[0][1], sides[1][1])


@pytest.mark.parametrize("M", [5, 600])
@pytest.mark.parametrize("fmt", FMTS)
def test_product_nan_stays_in_its_row(fmt, M):
    from stream_diffusion_transformer_b200 import model
    x = torch.randn(M, 256, device="cuda")
    x[3, 7] = float("inf")
    w = torch.randn(136, 256, device="cuda")
    w[10, 200] = float("nan")
    got = model.gemm_fp4(model.quantize_fp4(x, fmt), model.quantize_fp4(w, fmt))
    nan = torch.isnan(got)
    want = torch.zeros_like(nan)
    want[3], want[:, 10] = True, True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("fmt", FMTS)
def test_streams_graphs_and_repeats(fmt):
    """The same bits on another stream, from a captured graph replayed on new inputs, and with two calls at once."""
    from stream_diffusion_transformer_b200 import model
    w = model.quantize_fp4(torch.randn(520, 1056, device="cuda"), fmt)
    for M in (4, 70, 700):
        x, y = torch.randn(M, 1056, device="cuda"), torch.randn(M, 1056, device="cuda")
        want_x, want_y = (model.gemm_fp4(model.quantize_fp4(t, fmt), w) for t in (x, y))
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            gx = model.gemm_fp4(model.quantize_fp4(x, fmt), w)
        with torch.cuda.stream(s2):
            gy = model.gemm_fp4(model.quantize_fp4(y, fmt), w)
        torch.cuda.synchronize()
        assert torch.equal(gx, want_x) and torch.equal(gy, want_y)
        buf = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = model.gemm_fp4(model.quantize_fp4(buf, fmt), w)
        graph.replay()
        assert torch.equal(out, want_x)
        buf.copy_(y)
        graph.replay()
        assert torch.equal(out, want_y)


def test_empty_and_refusals():
    from stream_diffusion_transformer_b200 import model
    w = model.quantize_fp4(torch.randn(16, 64, device="cuda"))
    e = model.quantize_fp4(torch.empty(0, 64, device="cuda"))
    assert model.gemm_fp4(e, w).shape == (0, 16) and model.dequantize_fp4(e).shape == (0, 64)
    for bad in (lambda: model.quantize_fp4(torch.randn(4, 64)), lambda: model.quantize_fp4(torch.randn(4, 64, device="cuda").half()),
                lambda: model.quantize_fp4(torch.randn(4, 128, device="cuda")[:, ::2]), lambda: model.quantize_fp4(torch.randn(4, 64, device="cuda"), "fp4"),
                lambda: model.gemm_fp4(w, model.quantize_fp4(torch.randn(16, 64, device="cuda"), "mxfp4")),
                lambda: model.gemm_fp4(w, model.quantize_fp4(torch.randn(16, 96, device="cuda"))),
                lambda: model.gemm_fp4(w._replace(block_scales=w.block_scales[:-1]), w),
                lambda: model.gemm_fp4(w._replace(row_scales=None), w),
                lambda: model.gemm_fp4(w, w, out=torch.empty(16, 8, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    """More than 2^32 elements going in, and more than 2^31 coming out of a product: the last rows."""
    from stream_diffusion_transformer_b200 import model
    rows, cols = 262272, 16384
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-128:] = torch.randn(128, cols, device="cuda")
    m, tail = model.quantize_fp4(x, fmt), model.quantize_fp4(x[-128:].clone(), fmt)
    assert torch.equal(m.codes[-128:], tail.codes)
    assert torch.equal(m.block_scales[-tail.block_scales.numel():], tail.block_scales)
    if fmt == "nvfp4":
        assert torch.equal(m.row_scales[-128:], tail.row_scales)
    x.fill_(1.0)
    y = model.dequantize_fp4(m)
    assert torch.equal(y[-128:], model.dequantize_fp4(tail)) and not y[:128].any()
    del x, y, m
    a, b = model.quantize_fp4(torch.randn(70000, 64, device="cuda"), fmt), model.quantize_fp4(torch.randn(32768, 64, device="cuda"), fmt)
    got = model.gemm_fp4(a, b)[-200:].double()
    da, db = (model.dequantize_fp4(t, torch.float32).double() for t in (a, b))
    want, size = da[-200:] @ db.t(), da[-200:].abs() @ db.abs().t()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 64 * 2.0 ** -23 * size).all()
