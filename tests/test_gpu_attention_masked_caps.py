"""GPU tests of masked attention's cap: caps far above the scores, and scores that the cap must not carry elsewhere.

Tolerances as in test_gpu_attention_masked.py but for the cap's share d of a score's error: at most 2^-17 of the cap
(the polynomial's 3.7e-6, and below that the exponential form's) and at most 2^-14 of the score itself (the
polynomial's 4.5e-5 < 2^-14; the series and the exponential form are within 10^-6)."""
import math

import pytest

from gpu_util import require_gpu, torch
from test_gpu_attention_masked import i32, inputs, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from stream_diffusion_transformer_b200 import abi
    abi.lib()
    abi.clear_device_status()
    yield
    assert abi.device_status() == 0


def causal_formula(q, k, v, cap, slopes=None):
    """(out, tolerance) in fp64 of one causal batch element with the cap's error bounded as above."""
    n, H, m, group = q.shape[1], q.shape[2], k.shape[1], q.shape[2] // k.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    j = torch.arange(m, device=q.device)
    place = torch.arange(n, device=q.device)[:, None] + m - n
    for h in range(H):
        qh, kh, vh = q[0, :, h].double(), k[0, :, h // group].double(), v[0, :, h // group].double()
        s = qh @ kh.t() / math.sqrt(128)
        d = 2 * 128 * 2.0 ** -24 * (qh.abs() @ kh.abs().t()) / math.sqrt(128)
        s = cap * torch.tanh(s / cap)
        d = d + (s.abs() * 2.0 ** -14).clamp(max=cap * 2.0 ** -17)
        if slopes is not None:
            bias = slopes[h].double() * (place - j).abs()
            s, d = s - bias, d + bias * 2.0 ** -22
        d = d + s.abs() * 2.0 ** -21
        w = torch.softmax(torch.where(j <= place, s, -math.inf), 1)
        o, A = w @ vh, w @ vh.abs()
        dmax = torch.where(w > 1e-7, d, 0.0).amax(1, keepdim=True)
        out[0, :, h] = o
        tol[0, :, h] = 2.0 ** -8 * (o.abs() + A) + (2.0 ** -13 + 2 * dmax) * A
    return out, tol


@pytest.mark.parametrize("n,m,H,Hk", [(1, 700, 4, 1), (2, 100, 2, 1), (300, 400, 2, 1), (130, 130, 3, 3)])
@pytest.mark.parametrize("cap", [0.5, 30.0, 800.0, 900.0, 1e4, 1e5, 1e6, 1e8, 2.0 ** 60])
def test_caps_of_any_size(cap, n, m, H, Hk):
    """Scores of a few units under caps that press them flat, bend them and leave them alone."""
    from stream_diffusion_transformer_b200 import model
    q, k, v = inputs(1, n, m, H, Hk, 20, spread=4.0)
    for slopes in (None, slopes_of(H)):
        got = model.attention_masked(q, k, v, softcap=cap, causal=True, slopes=slopes).double()
        want, tol = causal_formula(q, k, v, cap, slopes)
        assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())
        if cap >= 1e5:  # scores of 20 at most: tanh takes (20 / cap)^2 / 3 < 2^-26 of them
            free, tol0 = causal_formula(q, k, v, 2.0 ** 200, slopes)
            assert ((got - free).abs() <= tol0).all()


@pytest.mark.parametrize("slope", [False, True])
@pytest.mark.parametrize("n,m", [(2, 400), (300, 400)])
def test_hidden_keys_leave_a_capped_row_as_it_is(n, m, slope):
    """Bit for bit: keys past the end, later ones and those of other documents, however large their scores are."""
    from stream_diffusion_transformer_b200 import model
    q, k, v = inputs(1, n, m, 2, 1, 21)
    kw = dict(softcap=30.0, slopes=slopes_of(2) if slope else None)

    def with_loud(rows, by):
        k2, v2 = k.clone(), v.clone()
        k2[:, rows], v2[:, rows] = k2[:, rows] * by, v2[:, rows] * 100.0
        return k2, v2
    used = m - 70
    for by in (50.0, 2.0 ** 120, float("nan")):
        a = model.attention_masked(q, k, v, kv_len=i32(used), **kw)
        assert torch.equal(model.attention_masked(q, *with_loud(slice(used, m), by), kv_len=i32(used), **kw), a)
    a = model.attention_masked(q, k, v, causal=True, **kw)
    for last in (m - n, m - 1 - n // 2):  # the keys behind the one at place `last`
        got = model.attention_masked(q, *with_loud(slice(last + 1, m), 50.0), causal=True, **kw)
        seen = last - (m - n) + 1  # queries that stand at `last` or before
        assert torch.equal(got[:, :seen], a[:, :seen]) and not torch.equal(got, a)
    ids = (torch.arange(m, dtype=torch.int32, device="cuda") % 3)[None].contiguous()
    own = torch.full((1, n), 1, dtype=torch.int32, device="cuda")
    a = model.attention_masked(q, k, v, q_doc=own, k_doc=ids, **kw)
    assert torch.equal(model.attention_masked(q, *with_loud(ids[0] != 1, 50.0), q_doc=own, k_doc=ids, **kw), a)
