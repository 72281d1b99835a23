"""GPU test of masked attention over a long stream (more heads than run side by side, more units than SMs), on sampled
rows against the formula in fp64, with the tolerance of test_gpu_attention_masked.py."""
import math

import pytest

from gpu_util import require_gpu, torch
from test_gpu_attention_masked import inputs, slopes_of

pytestmark = pytest.mark.gpu
N, H, CAP, PREFIX = 16896, 10, 30.0, 500  # K and V of ten heads: 86 MB


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from stream_diffusion_transformer_b200 import abi
    abi.lib()
    abi.clear_device_status()
    yield
    assert abi.device_status() == 0


@pytest.mark.parametrize("kind,Hk,m", [("cap and bias", 10, N), ("plain", 10, N), ("prefix", 2, N - 3), ("documents", 10, N)])
def test_sampled_rows(kind, Hk, m):
    from stream_diffusion_transformer_b200 import model
    n = N if kind != "prefix" else N - 100
    q, k, v = inputs(1, n, m, H, Hk, 30)
    kw = {}
    cap = kind in ("cap and bias", "prefix")
    if cap:
        kw["softcap"] = CAP
    if kind == "cap and bias":
        kw["slopes"] = slopes_of(H)
    if kind == "prefix":
        kw.update(causal=True, prefix_len=torch.tensor([PREFIX], dtype=torch.int32, device="cuda"))
    if kind == "documents":  # images of several sizes, their texts, padding
        sizes = [(3000, 0), (5000, 1), (4000, 2), (4500, 3), (77, 0), (77, 1), (77, 2), (77, 3)]
        ids = torch.cat([torch.full((s,), d, dtype=torch.int32) for s, d in sizes])
        ids = torch.cat([ids, torch.full((n - len(ids),), -1, dtype=torch.int32)])[None].cuda()
        kw["q_doc"] = kw["k_doc"] = ids
    got = model.attention_masked(q, k, v, **kw)
    assert torch.isfinite(got).all()
    rows = torch.tensor([0, 1, 127, 128, 255, 256, 3000, 7999, 8000, 12345, 16520, 16576, 16577, 16600, n - 1], device="cuda")
    place, j = (rows + m - n)[:, None], torch.arange(m, device="cuda")
    see = torch.ones(len(rows), m, dtype=torch.bool, device="cuda")
    if kind == "prefix":
        see = (j <= place) | (j < PREFIX)
    if kind == "documents":
        see = (ids[0, rows][:, None] == ids[0]) & (ids[0] >= 0)
    for h in range(H):
        qh, kh, vh = q[0, rows, h].double(), k[0, :, h * Hk // H].double(), v[0, :, h * Hk // H].double()
        s = qh @ kh.t() / math.sqrt(128)
        d = 2 * 128 * 2.0 ** -24 * (qh.abs() @ kh.abs().t()) / math.sqrt(128)
        if cap:
            s = CAP * torch.tanh(s / CAP)
            d = d + CAP * 2.0 ** -17
        if kind == "cap and bias":
            bias = kw["slopes"][h].double() * (place - j).abs()
            s, d = s - bias, d + bias * 2.0 ** -22
        d = d + s.abs() * 2.0 ** -21
        s = torch.where(see, s, -math.inf)
        top = s.amax(1, keepdim=True)
        w = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        o, A = w @ vh, w @ vh.abs()
        dmax = torch.where(w > 1e-7, d, 0.0).amax(1, keepdim=True)
        tol = 2.0 ** -8 * (o.abs() + A) + (2.0 ** -13 + 2 * dmax) * A + 1e-30
        off = (got[0, rows, h].double() - o).abs()
        assert (off <= tol).all(), (h, float((off / tol).max()))
    if kind == "documents":
        assert (got[0, 16808:] == 0).all()
