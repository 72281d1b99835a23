"""GPU tests of 4-bit rows in numbers and widths where the kernels run by another plan (1,024 rows or more): every
byte is written, and sampled rows are bit-identical to oracle/fp4_ref.py (a row's result depends on that row alone)."""
import numpy as np
import pytest

from gpu_util import require_gpu, torch
from oracle import fp4_ref as f4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from stream_diffusion_transformer_b200 import abi
    abi.lib()
    abi.clear_device_status()
    yield
    assert abi.device_status() == 0


def untile(tiled, rows, blocks):
    """Block scales [rows, blocks] out of the stored layout, and whether all bytes outside the matrix are zero."""
    ty, tx = -(-rows // 128), -(-blocks // 4)
    full = tiled.reshape(ty, tx, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(ty * 128, tx * 4)
    return full[:rows, :blocks], not full[rows:].any() and not full[:, blocks:].any()


def quantize_into(x, fmt, fill):
    """zi_quantize_fp4 into buffers whose every byte is `fill`."""
    from stream_diffusion_transformer_b200 import abi, model
    f = {"mxfp4": abi.ZI_FP4_MX, "nvfp4": abi.ZI_FP4_NV}[fmt]
    rows, cols = x.shape
    q = torch.full((rows, cols // 2), fill, dtype=torch.uint8, device="cuda")
    bs = torch.full((abi.fp4_scale_size(f, rows, cols),), fill, dtype=torch.uint8, device="cuda")
    rs = torch.full((4 * rows,), fill, dtype=torch.uint8, device="cuda").view(torch.float32) if fmt == "nvfp4" else None
    abi.call("zi_quantize_fp4", f, x.data_ptr(), int(x.dtype == torch.bfloat16), rows, cols, q.data_ptr(), bs.data_ptr(),
             None if rs is None else rs.data_ptr(), torch.cuda.current_stream().cuda_stream)
    return model.Fp4Matrix(fmt, q, bs, rs)


@pytest.mark.parametrize("rows,cols", [(1023, 10240), (1024, 32), (1024, 160), (1024, 544), (1024, 768), (1153, 1056),
                                       (1024, 1280), (1024, 1536), (1025, 2560), (1024, 2944), (1153, 3840), (1024, 5120),
                                       (1024, 6144), (1153, 10240), (1024, 12288), (1024, 16384)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_every_column_of_many_rows(fmt, bf16, rows, cols):
    from stream_diffusion_transformer_b200 import model
    rng = np.random.default_rng(rows + cols)
    x = (rng.standard_normal((rows, cols), dtype=np.float32) * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32)
    x[rng.permutation(rows)[:rows // 2], cols - 5] *= 64  # rows whose largest value stands at their end
    t = torch.from_numpy(x).cuda()
    if bf16:
        t = t.bfloat16()
        x = t.float().cpu().numpy()
    m, other = quantize_into(t, fmt, 0xFF), quantize_into(t, fmt, 0x00)
    for a, b in zip(m[1:], other[1:]):
        assert a is None and b is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8)), "bytes left as they were"
    some = np.unique(np.concatenate([[0, 1, rows - 2, rows - 1], rng.integers(0, rows, 44)]))
    code, stored, row = f4.quantize(x[some], fmt)
    np.testing.assert_array_equal(m.codes.cpu().numpy()[some], f4.pack_codes(code))
    scales, clean = untile(m.block_scales.cpu().numpy(), rows, cols // f4.BLOCK[fmt])
    np.testing.assert_array_equal(scales[some], stored)
    assert clean
    if fmt == "nvfp4":
        np.testing.assert_array_equal(m.row_scales.cpu().numpy()[some].astype(np.float64), row)
    want = f4.dequantize(code, stored, row, fmt)
    np.testing.assert_array_equal(model.dequantize_fp4(m, torch.float32).cpu().numpy()[some], want.astype(np.float32))
    want16 = torch.from_numpy(want).to(torch.bfloat16).float().numpy()
    np.testing.assert_array_equal(model.dequantize_fp4(m).float().cpu().numpy()[some], want16)
