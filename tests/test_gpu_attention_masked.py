"""GPU tests of the masked attention against its formula in fp64.

Tolerance of an element, with w_j the exact softmax weights and A = sum_j w_j |v_j|: the result's rounding to
bf16 (2^-8 |o|), the probabilities' rounding to bf16 (2^-8 A) with their exponential (7.5e-5 < 2^-13), and
2 d A for scores that are off by at most d: the fp32 product of 128 terms (128 * 2^-24 * scale sum |q k|, twice
for the order of the sums), the cap's tanh (2^-17 of the cap) and the bias (2^-22 of it), and the roundings
of the score itself on its way (2^-21 of it)."""
import math

import pytest

from gpu_util import require_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from stream_diffusion_transformer_b200 import abi
    abi.lib()
    abi.clear_device_status()
    yield
    assert abi.device_status() == 0


def formula(q, k, v, scale=None, softcap=0.0, slopes=None, causal=False, prefix_len=None, kv_len=None, q_doc=None,
            k_doc=None):
    """(out, tolerance) in fp64, one head at a time."""
    B, n, H, _ = q.shape
    m, group = k.shape[1], H // k.shape[2]
    scale = 1 / math.sqrt(128) if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    j = torch.arange(m, device=q.device)
    for b in range(B):
        N = m if kv_len is None else min(max(int(kv_len[b]), 0), m)
        place = torch.arange(n, device=q.device)[:, None] + N - n
        see = (j < N).expand(n, m)
        if causal:
            see = see & ((j <= place) | (j < (int(prefix_len[b]) if prefix_len is not None else 0)))
        if q_doc is not None:
            see = see & (q_doc[b][:, None] == k_doc[b]) & (k_doc[b] >= 0)
        kb, vb = k[b].double().nan_to_num(0, 0, 0), v[b].double()
        seen = see.any(0)
        kb, vb = torch.where(seen[:, None, None], kb, 0.0), torch.where(seen[:, None, None], vb, 0.0)
        for h in range(H):
            s = scale * (q[b, :, h].double() @ kb[:, h // group].t())
            d = 2 * 128 * 2.0 ** -24 * scale * (q[b, :, h].double().abs() @ kb[:, h // group].abs().t())
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                d += softcap * 2.0 ** -17
            if slopes is not None:
                bias = slopes[h].double() * (place - j).abs()
                s = s - bias
                d += bias.abs() * 2.0 ** -22
            d += s.abs() * 2.0 ** -21
            s = torch.where(see, s, -math.inf)
            top = s.amax(1, keepdim=True)
            w = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
            o = w @ vb[:, h // group]
            A = w @ vb[:, h // group].abs()
            dmax = torch.where(w > 1e-7, d, 0.0).amax(1, keepdim=True)
            out[b, :, h] = o
            tol[b, :, h] = 2.0 ** -8 * (o.abs() + A) + (2.0 ** -13 + 2 * dmax) * A + 1e-30
    return out, tol


def check(q, k, v, **kw):
    from stream_diffusion_transformer_b200 import model
    got = model.attention_masked(q, k, v, **kw)
    want, tol = formula(q, k, v, **kw)
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all(), "not finite"
    assert (off <= tol).all(), float((off / tol).max())
    return got


def inputs(B, n, m, H, Hk, seed=0, spread=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1000 * n + m)
    q = (spread * torch.randn((B, n, H, 128), generator=g, device="cuda")).bfloat16()
    k = torch.randn((B, m, Hk, 128), generator=g, device="cuda").bfloat16()
    v = torch.randn((B, m, Hk, 128), generator=g, device="cuda").bfloat16()
    return q, k, v


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def slopes_of(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)


SIZES = [(1, 1, 1, 1, 1), (2, 1, 5, 2, 1), (1, 1, 1000, 10, 2), (2, 3, 129, 6, 6), (1, 17, 33, 3, 1), (1, 128, 128, 2, 2),
         (2, 130, 257, 4, 2), (1, 300, 555, 2, 1), (1, 257, 257, 1, 1), (1, 600, 640, 3, 3), (3, 5, 2000, 4, 1)]
KINDS = ["plain", "cap", "bias", "causal", "prefix", "lengths", "documents", "all"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,n,m,H,Hk", SIZES)
def test_sizes_and_masks(kind, B, n, m, H, Hk):
    q, k, v = inputs(B, n, m, H, Hk)
    kw = {}
    if kind in ("cap", "all"):
        kw["softcap"] = 20.0
    if kind in ("bias", "all"):
        kw["slopes"] = slopes_of(H)
    if kind in ("causal", "prefix", "all"):
        kw["causal"] = True
    if kind in ("prefix", "all"):
        kw["prefix_len"] = i32(*[(m * (b + 1)) // (B + 2) for b in range(B)])
    if kind in ("lengths", "all"):
        kw["kv_len"] = i32(*[m - (b * m) // 3 - m // 5 for b in range(B)])
    if kind in ("documents", "all"):
        g = torch.Generator().manual_seed(m)
        ids = torch.sort(torch.randint(-1, 4, (B, m), generator=g, dtype=torch.int32), dim=1)[0].cuda()
        kw["k_doc"], kw["q_doc"] = ids, ids[:, -n:].contiguous() if n <= m else ids.new_zeros(B, n)
    check(q, k, v, **kw)


def test_documents_in_any_order_and_images_before_texts():
    q, k, v = inputs(1, 700, 700, 2, 2, 1)
    ids = torch.cat([torch.full((n,), d, dtype=torch.int32) for n, d in
                     ((250, 0), (130, 1), (200, 2), (30, 0), (33, 1), (40, 2), (17, -1))])[None].cuda()
    got = check(q, k, v, q_doc=ids, k_doc=ids)
    assert (got[0, -17:] == 0).all()
    # a document's rows do not depend on what it is packed with
    own = (ids[0] == 1).nonzero()[:, 0]
    alone = check(q[:, own].contiguous(), k[:, own].contiguous(), v[:, own].contiguous())
    assert (got[0, own].double() - alone[0].double()).abs().max() < 2e-2
    shuffled = torch.randint(-2, 5, (1, 700), dtype=torch.int32, device="cuda")
    check(q, k, v, q_doc=shuffled, k_doc=shuffled, causal=True)


def test_rows_that_see_nothing_are_zero():
    for n, m in ((1, 64), (40, 300), (300, 300)):
        q, k, v = inputs(2, n, m, 2, 1, 2)
        got = check(q, k, v, kv_len=i32(0, m))
        assert (got[0] == 0).all() and (got[1] != 0).any()
        got = check(q, k, v, kv_len=i32(-5, 2 * m))
        assert (got[0] == 0).all()
        none = torch.full((2, m), -1, dtype=torch.int32, device="cuda")
        got = check(q, k, v, q_doc=torch.zeros((2, n), dtype=torch.int32, device="cuda"), k_doc=none)
        assert (got == 0).all()
        if n > 1:  # more queries than keys: the first ones stand before the first key
            got = check(q, k, v, kv_len=i32(n // 2, 1), causal=True)
            assert (got[1, :n - 1] == 0).all() and (got[1, n - 1] != 0).any()


def test_nan_in_rows_that_nobody_sees():
    for n, m, used in ((1, 500, 333), (130, 500, 333), (300, 400, 300)):
        q, k, v = inputs(1, n, m, 2, 2, 3)
        bad_k, bad_v = k.clone(), v.clone()
        bad_k[:, used:], bad_v[:, used:] = float("nan"), float("inf")
        want = check(q, k, v, kv_len=i32(used), causal=True)
        assert torch.equal(check(q, bad_k, bad_v, kv_len=i32(used), causal=True), want)
        ids = torch.zeros((1, m), dtype=torch.int32, device="cuda")
        ids[:, used:] = -1
        ids[:, 7] = -3
        bad_k[:, 7], bad_v[:, 7] = float("inf"), float("nan")
        q_ids = torch.zeros((1, n), dtype=torch.int32, device="cuda")
        got = check(q, bad_k, bad_v, q_doc=q_ids, k_doc=ids)
        assert torch.equal(got, check(q, k, v, q_doc=q_ids, k_doc=ids))
        bad_q = q.clone()
        if n > 1:  # a padded query: its NaN reaches no other row
            bad_q[:, 5], q_ids[:, 5] = float("nan"), -1
            got2 = check_finite(bad_q, k, v, q_doc=q_ids, k_doc=ids)
            assert (got2[:, 5] == 0).all()
            keep = [i for i in range(n) if i != 5]
            assert torch.equal(got2[:, keep], got[:, keep])


def check_finite(q, k, v, **kw):
    from stream_diffusion_transformer_b200 import model
    got = model.attention_masked(q, k, v, **kw)
    assert torch.isfinite(got).all()
    return got


@pytest.mark.parametrize("n", [1, 40, 300])
def test_strides(n):
    """Slices of a fused projection, [B, H, n, 128] layouts, a cache with room to grow, an output with gaps."""
    from stream_diffusion_transformer_b200 import model
    B, m, H, Hk = 2, 300, 4, 2
    q, k, v = inputs(B, n, m, H, Hk, 4)
    want = check(q, k, v, causal=True)
    fused = torch.zeros((B, m, (H + 2 * Hk) * 128), dtype=torch.bfloat16, device="cuda")
    fused[:, m - n:, :H * 128] = q.reshape(B, n, -1)
    fused[:, :, H * 128:(H + Hk) * 128], fused[:, :, (H + Hk) * 128:] = k.reshape(B, m, -1), v.reshape(B, m, -1)
    qs = fused[:, m - n:, :H * 128].unflatten(2, (H, 128))
    ks = fused[:, :, H * 128:(H + Hk) * 128].unflatten(2, (Hk, 128))
    vs = fused[:, :, (H + Hk) * 128:].unflatten(2, (Hk, 128))
    assert torch.equal(model.attention_masked(qs, ks, vs, causal=True), want)
    swap = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    assert torch.equal(model.attention_masked(*swap, causal=True), want)
    cache_k = torch.full((B, 1000, Hk, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    cache_v = cache_k.clone()
    cache_k[:, :m], cache_v[:, :m] = k, v
    assert torch.equal(model.attention_masked(q, cache_k[:, :m], cache_v[:, :m], causal=True), want)
    room = torch.full((B, n + 2, H + 1, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    view = room[:, 1:n + 1, :H, :128]
    model.attention_masked(q, k, v, causal=True, out=view)
    assert torch.equal(view, want)
    room[:, 1:n + 1, :H, :128] = 5.0
    assert (room == 5.0).all()  # nothing beside the output was written


def test_scores_far_out():
    """Scores of thousands, a cap far inside them, slopes that bury all but the nearest key."""
    q, k, v = inputs(1, 200, 260, 2, 2, 5, spread=60.0)
    check(q, k, v, softcap=10.0)
    check(q, k, v, softcap=1000.0, causal=True)
    check(q, k, v, slopes=torch.tensor([40.0, 0.0], device="cuda"))
    check(q, k, v, scale=2.0)
    q, k, v = inputs(1, 2, 260, 2, 2, 5, spread=60.0)
    check(q, k, v, softcap=10.0)
    check(q, k, v, slopes=torch.tensor([40.0, 0.0], device="cuda"), causal=True)


def test_scales_and_caps_at_the_ends_of_their_range():
    for n, m in ((2, 100), (300, 400)):
        q, k, v = inputs(1, n, m, 2, 1, 10)
        for kw in (dict(scale=2.0 ** -60), dict(softcap=2.0 ** -60), dict(softcap=2.0 ** 60), dict(scale=2.0 ** -60, softcap=2.0 ** 60),
                   dict(scale=2.0 ** -60, slopes=slopes_of(2)), dict(softcap=2.0 ** 60, slopes=slopes_of(2))):
            check(q, k, v, causal=True, **kw)


def test_documents_past_the_lists_of_key_tiles():
    """More key tiles (2,110) than the kernel lists by document: the later ones are masked one by one."""
    n, m = 300, 270000
    q, k, v = inputs(1, n, m, 1, 1, 11)
    ids = (torch.arange(m, dtype=torch.int32, device="cuda") // 90000)[None].contiguous()
    q_ids = torch.full((1, n), 2, dtype=torch.int32, device="cuda")
    q_ids[:, :20], q_ids[:, 20:40] = 0, 7
    got = check(q, k, v, q_doc=q_ids, k_doc=ids, kv_len=i32(m - 77), causal=True)
    assert (got[0, 20:40] == 0).all()


def test_first_call_of_a_process_may_be_captured():
    """Each kernel's first launch raises its shared-memory limit; that may happen while a stream is being captured."""
    import subprocess
    import sys
    from conftest import ROOT
    code = """
import torch
from stream_diffusion_transformer_b200 import model
x, w = torch.randn(700, 256, device="cuda"), torch.randn(264, 256, device="cuda")
q = torch.randn(1, 300, 2, 128, device="cuda").bfloat16()
torch.cuda.synchronize()
def run():
    a, b = model.quantize_fp4(x), model.quantize_fp4(w)
    return (model.gemm_fp4(a, b), model.gemm_fp4(model.quantize_fp4(x[:5]), b), model.attention_masked(q, q, q, softcap=9.0),
            model.attention_masked(q[:, :2], q, q))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_streams_graphs_and_repeats():
    """The same bits on another stream, from a captured graph on new inputs, and with two calls at once."""
    from stream_diffusion_transformer_b200 import model
    for n, m in ((1, 1500), (300, 400)):
        a, b = inputs(2, n, m, 4, 2, 6), inputs(2, n, m, 4, 2, 7)
        kw = dict(causal=True, softcap=30.0, kv_len=i32(m, m - 100))
        want_a, want_b = check(*a, **kw), check(*b, **kw)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            ga = model.attention_masked(*a, **kw)
        with torch.cuda.stream(s2):
            gb = model.attention_masked(*b, **kw)
        torch.cuda.synchronize()
        assert torch.equal(ga, want_a) and torch.equal(gb, want_b)
        buf = [t.clone() for t in a]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = model.attention_masked(*buf, **kw)
        graph.replay()
        assert torch.equal(out, want_a)
        for t, s in zip(buf, b):
            t.copy_(s)
        graph.replay()
        assert torch.equal(out, want_b)


def test_a_step_over_a_cache_equals_the_last_row():
    """One token at a time gives what the whole causal stream gives, within the two roundings."""
    from stream_diffusion_transformer_b200 import model
    q, k, v = inputs(1, 200, 200, 4, 2, 8)
    kw = dict(softcap=25.0, slopes=slopes_of(4), causal=True)
    whole = check(q, k, v, **kw)
    for t in (0, 1, 63, 127, 128, 199):
        one = check(q[:, t:t + 1].contiguous(), k, v, kv_len=i32(t + 1), **kw)
        assert (one[0, 0].double() - whole[0, t].double()).abs().max() < 3e-2


def test_refusals():
    from stream_diffusion_transformer_b200 import abi, model
    q, k, v = inputs(1, 4, 8, 4, 2)
    ids = torch.zeros((1, 8), dtype=torch.int32, device="cuda")
    for bad in (lambda: model.attention_masked(q.float(), k, v), lambda: model.attention_masked(q, k, v[:, :4]),
                lambda: model.attention_masked(q[..., ::2], k, v), lambda: model.attention_masked(q.cpu(), k, v),
                lambda: model.attention_masked(q, k, v, kv_len=torch.tensor([3], device="cuda")),
                lambda: model.attention_masked(q, k, v, slopes=torch.ones(3, device="cuda")),
                lambda: model.attention_masked(q, k, v, out=torch.empty_like(k))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: model.attention_masked(q[:, :, :3], k, v), lambda: model.attention_masked(q, k, v, k_doc=ids),
                lambda: model.attention_masked(q, k, v, prefix_len=i32(3)), lambda: model.attention_masked(q, k, v, softcap=-1.0),
                lambda: model.attention_masked(q, k, v, scale=float("nan")),
                lambda: model.attention_masked(q, k.expand(1, 8, 2, 128)[:, :1].expand(1, 8, 2, 128), v)):
        with pytest.raises(abi.ZiError):
            bad()


@pytest.mark.parametrize("n", [2, 300])
def test_offsets_past_32_bits(n):
    """Rows 2^24 elements apart in one buffer: the last ones stand past 2^32 elements (8 GB)."""
    from stream_diffusion_transformer_b200 import model
    m, step = 300, 1 << 24
    q, k, v = inputs(1, n, m, 2, 2, 11)
    want = check(q, k, v, causal=True)
    room = torch.empty(m * step, dtype=torch.bfloat16, device="cuda")
    views = []
    for i, t in enumerate((q, k, v, want)):
        views.append(room.as_strided((1, t.shape[1], 2, 128), (m * step, step, 128, 1), (m - t.shape[1]) * step + 256 * i))
    for view, t in zip(views, (q, k, v, torch.zeros_like(want))):
        view.copy_(t)
    model.attention_masked(*views[:3], causal=True, out=views[3])
    assert torch.equal(views[3], want)
    for view, t in zip(views, (q, k, v)):
        assert torch.equal(view, t)


@pytest.mark.parametrize("n", [1, 300])
def test_largest_biases(n):
    """A slope of 2^20 over 300 places (scores of 2^28.3) leaves each query its own place at any scale: the next key
    is behind by 2^20, so the result is v of that place, bit for bit."""
    from stream_diffusion_transformer_b200 import model
    q, k, v = inputs(1, n, 300, 2, 2, 12)
    slopes = torch.full((2,), 2.0 ** 20, device="cuda")
    for scale in (2.0 ** -60, 128 ** -0.5):
        for softcap in (0.0, 20.0):
            got = model.attention_masked(q, k, v, scale=scale, softcap=softcap, slopes=slopes)
            assert torch.equal(got, v[:, 300 - n:])
