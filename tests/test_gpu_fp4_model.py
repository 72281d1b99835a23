"""GPU tests of blocks and models whose projections run in 4 bits, and of the new operators as one run.

Fused epilogues, tight: with x of rows +-1 the norm gives +-1 whatever the rounding, so the rows going into a
4-bit projection are the oracle's exactly; with w2 (or the output projection) zero the block shows the QKV (or the
gate and up) product alone, to the bf16 block's bars (rel-L2 2e-2, cosine 0.999).

Whole blocks.  A quantiser turns a relative difference e of its input into sqrt(e^2 + 0.8 e D), D its mean step
relative to the values' rms (a difference of e crosses a border with probability e / D and then costs D; 0.8 is the
mean |x| of a unit normal): D ~ 0.3 for blocks whose largest value lies between 4 and 8 steps of 1.  GPU and
oracle differ by 3e-3 first after the attention (bf16 probabilities and result); h before it agrees.
- QKV and w1|w3: h2 2.7e-2; the product of gate and up 1.5 times that, 4e-2; through w2 and the norm, added to an
  x1 of the same size without a difference: 2.8e-2.  Bar 7e-2, cosine 1 - bar^2 / 2 rounded down to 0.995.
- all: attention output 2.7e-2, so x1 2.7e-2, h2 8.5e-2, gate times up 0.125, into w2 0.21, the sum with x1 0.15.
  Bar 0.2, cosine 0.98.
A modulated block's gates scale the update, so its differences are smaller."""
import dataclasses

import numpy as np
import pytest

from gpu_util import assert_parity, require_gpu, torch
import zimage_inputs as zi
from oracle import fp4_ref as f4
from oracle import zimage_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from stream_diffusion_transformer_b200 import abi
    abi.lib()
    abi.clear_device_status()
    yield
    assert abi.device_status() == 0


def run_block(d, bits, x, fmt, projections, s_txt, gh, gw, seed, modulated):
    from stream_diffusion_transformer_b200 import model
    cfg, prefix = model.make_config(d), "layers.0"
    c = zi.make_cond(d, 1, seed=seed) if modulated else None
    blk = model.DeviceBlock(cfg, prefix, bits, modulated, "cuda")
    four = blk.with_fp4(fmt, projections)
    pos = model.positions(s_txt, gh, gw)
    xt, ct = torch.from_numpy(x).cuda(), None if c is None else torch.from_numpy(c).cuda()
    before = model.block_forward(cfg, blk, ct, pos, xt)
    got = model.block_forward(cfg, four, ct, pos, xt)
    assert torch.equal(model.block_forward(cfg, four, ct, pos, xt), got)
    assert torch.equal(model.block_forward(cfg, blk, ct, pos, xt), before)  # the bf16 block is as it was
    assert not torch.equal(got, before)
    ang = ref.rope_angles(ref.position_ids(s_txt, gh, gw), d.rope_axes)
    want = f4.block_forward(x[0].astype(np.float64), ref.Weights(bits), prefix, d, ang,
                            None if c is None else c[0].astype(np.float64), fmt, projections == "all")
    return got[0].cpu().numpy(), want


@pytest.mark.parametrize("part", ["qkv", "ffn"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_fused_epilogues(fmt, part):
    from stream_diffusion_transformer_b200 import model
    d = zi.TINY
    bits = dict(zi.make_weights(d, seed=41, keys=model.block_keys("layers.0", False), threads=4))
    for k in ("attention_norm1", "ffn_norm1"):
        bits[f"layers.0.{k}.weight"] = np.full_like(bits[f"layers.0.{k}.weight"], 0x3F80)  # gains 1
    zero = "layers.0.feed_forward.w2.weight" if part == "qkv" else "layers.0.attention.to_out.weight"
    bits[zero] = np.zeros_like(bits[zero])
    S = 256 + 44  # two row tiles, the second ragged
    rng = np.random.default_rng(6)
    x = rng.choice([-1.0, 1.0], (1, S, d.dim)).astype(np.float32)
    got, want = run_block(d, bits, x, fmt, True, 44, 16, 16, 41, False)
    assert_parity(got, want, what=f"{fmt} {part}")
    assert_parity(got - x[0], want - x[0], what=f"{fmt} {part} update")


@pytest.mark.parametrize("projections", [True, "all"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("modulated", [True, False])
def test_tiny_block(modulated, fmt, projections):
    from stream_diffusion_transformer_b200 import model
    d = zi.TINY
    bits = zi.make_weights(d, seed=42, keys=model.block_keys("layers.0", modulated), threads=4)
    x = zi.make_stream(d, 1, 96, seed=42)
    got, want = run_block(d, bits, x, fmt, projections, 32, 8, 8, 42, modulated)
    rel, cos = (0.2, 0.98) if projections == "all" else (7e-2, 0.995)
    assert_parity(got, want, rel=rel, cos=cos, what=f"{fmt} {projections} {modulated}")


def test_model_forward_graph_and_mixed_blocks():
    """A model in 4 bits near its bf16 parent, the same bits from a captured graph, and bf16 blocks beside 4-bit ones."""
    from stream_diffusion_transformer_b200 import abi, model
    d = dataclasses.replace(zi.TINY, n_noise=1, n_ctx=1, n_main=2)
    bits = zi.make_weights(d, seed=43, threads=4)
    dit = model.DiT(model.make_config(d), lambda keys: {k: bits[k] for k in keys})
    lat = torch.from_numpy(zi.make_latent(d, 2, 16, 16, seed=43)).cuda()
    txt = torch.from_numpy(zi.make_text(d, 2, 32, seed=43).view(np.int16)).cuda().view(torch.bfloat16)
    t = torch.tensor([0.3, 0.7], device="cuda")
    base = dit.forward(lat, t, txt)
    errs = {}
    for fmt in ("nvfp4", "mxfp4"):
        for projections in (True, "all"):
            four = dit.with_fp4(fmt, projections)
            y = four.forward(lat, t, txt)
            errs[fmt, projections] = float((y - base).norm() / base.norm())
            buf = torch.empty_like(y)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                four.forward(lat, t, txt, buf)
            graph.replay()
            assert torch.equal(buf, y)
    print(errs)
    assert torch.equal(dit.forward(lat, t, txt), base)
    assert all(0 < e < 0.5 for e in errs.values()) and errs["nvfp4", True] < errs["mxfp4", True]
    # the refiners in bf16, the main blocks in 4 bits: the library takes blocks of both kinds
    four = dit.with_fp4("nvfp4", "all")
    mixed = dit.with_fp4("nvfp4", "all")
    mixed.noise, mixed.ctx = dit.noise, dit.ctx
    mixed._bind()
    y = mixed.forward(lat, t, txt)
    assert torch.isfinite(y).all() and not torch.equal(y, four.forward(lat, t, txt)) and not torch.equal(y, base)


def test_4_bit_weights_are_checked():
    from stream_diffusion_transformer_b200 import abi, model
    d = zi.TINY
    bits = zi.make_weights(d, seed=44, keys=model.block_keys("layers.0", False), threads=4)
    cfg = model.make_config(d)
    blk = model.DeviceBlock(cfg, "layers.0", bits, False, "cuda")
    x = torch.from_numpy(zi.make_stream(d, 1, 96, seed=44)).cuda()
    pos = model.positions(32, 8, 8)
    for fmt, gone in (("nvfp4", "w_qkv4"), ("nvfp4", "b_13_4"), ("nvfp4", "r_qkv4"), ("nvfp4", "r_2_4"), ("mxfp4", "w2_4"),
                      ("mxfp4", "b_out4")):
        four = blk.with_fp4(fmt, "all")
        setattr(four.struct, gone, None)
        with pytest.raises(abi.ZiError) as e:
            model.block_forward(cfg, four, None, pos, x)
        assert e.value.status == abi.ZI_ERR_ARG
    four, eight = blk.with_fp4("nvfp4"), blk.with_e4m3(True)
    for f in ("w_qkv8", "s_qkv", "w13_8", "s_13"):
        setattr(four.struct, f, getattr(eight.struct, f))
    with pytest.raises(abi.ZiError):
        model.block_forward(cfg, four, None, pos, x)
    four = blk.with_fp4("nvfp4")
    four.struct.w13_4 += 8
    with pytest.raises(abi.ZiError) as e:
        model.block_forward(cfg, four, None, pos, x)
    assert e.value.status == abi.ZI_ERR_ALIGN
    with pytest.raises(ValueError):
        blk.with_fp4("nvfp4", False)


def test_run_of_the_operators_on_a_packed_stream():
    """Three documents packed into one stream: rows to 4 bits, QKV product, attention by documents straight from the
    fused projection, rows to 4 bits, output product.  Each step is held to its own tolerance on what the step before
    gave, and the whole run captured in a graph gives the same bits."""
    from stream_diffusion_transformer_b200 import model
    from test_gpu_attention_masked import check
    from test_gpu_fp4 import check_product
    S, H, Hk = 500, 4, 2
    D = H * 128
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = torch.randn((S, D), generator=g, device="cuda").bfloat16()
    wqkv = model.quantize_fp4(0.05 * torch.randn((D + 2 * Hk * 128, D), generator=g, device="cuda"))
    wout = model.quantize_fp4(0.05 * torch.randn((D, D), generator=g, device="cuda"))
    ids = torch.cat([torch.full((n,), i, dtype=torch.int32) for n, i in ((200, 0), (90, 1), (130, 2), (40, 0), (30, 1), (10, -1))])
    ids = ids[None].cuda()

    def run(x):
        qkv = model.gemm_fp4(model.quantize_fp4(x), wqkv)
        q = qkv[:, :D].view(1, S, H, 128)
        k = qkv[:, D:D + Hk * 128].view(1, S, Hk, 128)
        v = qkv[:, D + Hk * 128:].view(1, S, Hk, 128)
        att = model.attention_masked(q, k, v, softcap=30.0, q_doc=ids, k_doc=ids)
        return qkv, (q, k, v), att, model.gemm_fp4(model.quantize_fp4(att.view(S, D)), wout)

    def values(m):
        return model.dequantize_fp4(m, torch.float32).double()

    qkv, parts, att, out = run(x)
    check_product(qkv, values(model.quantize_fp4(x)), values(wqkv))
    assert torch.equal(check(*parts, softcap=30.0, q_doc=ids, k_doc=ids), att)
    check_product(out, values(model.quantize_fp4(att.view(S, D))), values(wout))
    assert (out[-10:] == 0).all()  # rows that see nothing stay zero through the product
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(buf)[3]
    graph.replay()
    assert torch.equal(got, out)
