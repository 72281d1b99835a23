"""Argument checks of the 4-bit and masked-attention entry points: each is refused before anything reaches a
device, so they run without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def abi():
    from stream_diffusion_transformer_b200 import abi as a, build
    build.build()
    a.lib()
    return a


P = 1 << 20  # an aligned non-null address; never read: every call here fails its checks


def refused(abi, status, fn, *args):
    with pytest.raises(abi.ZiError) as e:
        abi.call(fn, *args)
    assert e.value.status == status, (fn, args, e.value.status)


def test_scale_size(abi):
    assert abi.fp4_scale_size(abi.ZI_FP4_MX, 1, 32) == 512
    assert abi.fp4_scale_size(abi.ZI_FP4_NV, 1, 32) == 512
    assert abi.fp4_scale_size(abi.ZI_FP4_NV, 129, 96) == 2 * 2 * 512
    assert abi.fp4_scale_size(abi.ZI_FP4_MX, 4128, 3840) == 33 * 30 * 512
    assert abi.fp4_scale_size(abi.ZI_FP4_NV, 0, 32) == 0
    n = ctypes.c_size_t()
    for status, args in ((abi.ZI_ERR_ARG, (2, 1, 32)), (abi.ZI_ERR_ARG, (0, -1, 32)), (abi.ZI_ERR_ARG, (0, 1, 0)),
                         (abi.ZI_ERR_SHAPE, (0, 1, 48)), (abi.ZI_ERR_SHAPE, (1, 1 << 30 | 1, 32))):
        refused(abi, status, "zi_fp4_scale_size", *args, ctypes.byref(n))
    refused(abi, abi.ZI_ERR_ARG, "zi_fp4_scale_size", 0, 1, 32, None)


def test_rows(abi):
    ok = [1, P, 1, 4, 64, P, P, P, None]  # format, x, bf16, rows, cols, codes, block scales, row scales, stream
    for fn, order in (("zi_quantize_fp4", lambda a: a), ("zi_dequantize_fp4", lambda a: [a[0], a[5], a[6], a[7], a[3], a[4],
                                                                                   a[1], a[2], a[8]])):
        def bad(status, **kw):
            a = list(ok)
            for i, v in kw.items():
                a[int(i[1:])] = v
            refused(abi, status, fn, *order(a))
        for i in ("_1", "_5", "_6", "_7"):
            bad(abi.ZI_ERR_ARG, **{i: None})
            bad(abi.ZI_ERR_ALIGN, **{i: P + 8})
        bad(abi.ZI_ERR_ARG, _0=2)
        bad(abi.ZI_ERR_ARG, _0=0)  # row scales given to MXFP4
        bad(abi.ZI_ERR_ARG, _2=2)
        bad(abi.ZI_ERR_ARG, _3=-1)
        bad(abi.ZI_ERR_ARG, _4=0)
        bad(abi.ZI_ERR_SHAPE, _4=48)
        bad(abi.ZI_ERR_SHAPE, _4=16416)
        bad(abi.ZI_ERR_SHAPE, _3=(1 << 30) + 1)


def test_product(abi):
    ok = [1, P, P, P, P, P, P, P, 4, 64, 64, None]

    def bad(status, **kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        refused(abi, status, "zi_gemm_fp4", *a)
    for i in range(1, 8):
        bad(abi.ZI_ERR_ARG, **{f"_{i}": None})
        bad(abi.ZI_ERR_ALIGN, **{f"_{i}": P + 4})
    bad(abi.ZI_ERR_ARG, _0=0)
    bad(abi.ZI_ERR_ARG, _0=0, _3=None)
    bad(abi.ZI_ERR_ARG, _8=-1)
    bad(abi.ZI_ERR_SHAPE, _9=60)
    bad(abi.ZI_ERR_SHAPE, _10=48)
    for i in ("_8", "_9", "_10"):
        bad(abi.ZI_ERR_SHAPE, **{i: (1 << 24) + 32})


def test_masked_attention(abi):
    def desc(**kw):
        d = abi.attention_desc_init()
        assert abs(d.scale - 128 ** -0.5) < 1e-7 and d.softcap == 0 and not d.d_slopes
        d.q = d.k = d.v = d.out = P
        d.batch, d.heads, d.kv_heads, d.q_len, d.kv_len = 2, 4, 2, 3, 5
        for t in ("q", "k", "v", "out"):
            for n, s in (("batch", 8192), ("row", 512), ("head", 128)):
                setattr(d, f"{t}_{n}_stride", s)
        for k, v in kw.items():
            setattr(d, k, v)
        return ctypes.byref(d)

    def bad(status, **kw):
        refused(abi, status, "zi_attention_masked", desc(**kw), None)
    refused(abi, abi.ZI_ERR_ARG, "zi_attention_masked", None, None)
    refused(abi, abi.ZI_ERR_ARG, "zi_attention_desc_init", None)
    for name in ("q", "k", "v", "out"):
        bad(abi.ZI_ERR_ARG, **{name: None})
        bad(abi.ZI_ERR_ALIGN, **{name: P + 8})
        for dim in ("batch", "row", "head"):
            bad(abi.ZI_ERR_ARG, **{f"{name}_{dim}_stride": 0})
            bad(abi.ZI_ERR_ARG, **{f"{name}_{dim}_stride": -512})
            bad(abi.ZI_ERR_ALIGN, **{f"{name}_{dim}_stride": 516})
            bad(abi.ZI_ERR_SHAPE, **{f"{name}_{dim}_stride": 1 << 36})
    for name in ("batch", "heads", "kv_heads", "q_len", "kv_len"):
        bad(abi.ZI_ERR_ARG, **{name: 0})
        bad(abi.ZI_ERR_ARG, **{name: -1})
    bad(abi.ZI_ERR_SHAPE, heads=5)
    bad(abi.ZI_ERR_SHAPE, batch=65536)
    bad(abi.ZI_ERR_SHAPE, q_len=(1 << 24) + 1)
    bad(abi.ZI_ERR_SHAPE, kv_len=(1 << 24) + 1)
    bad(abi.ZI_ERR_SHAPE, heads=256, kv_heads=1, q_len=1 << 23)
    for v in (0.0, -1.0, float("nan"), float("inf"), 1e-19, 2e18):
        bad(abi.ZI_ERR_ARG, scale=v)
    for v in (-1.0, float("nan"), float("inf"), 1e-40, 1e-19, 2e18):
        bad(abi.ZI_ERR_ARG, softcap=v)
    bad(abi.ZI_ERR_ARG, causal=2)
    bad(abi.ZI_ERR_ARG, d_prefix_len=P)
    bad(abi.ZI_ERR_ARG, d_q_doc=P)
    bad(abi.ZI_ERR_ARG, d_k_doc=P)
    for name in ("d_slopes", "d_kv_len"):
        bad(abi.ZI_ERR_ALIGN, **{name: P + 2})
