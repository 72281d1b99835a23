"""GPU test of masked attention with nothing to attend: no batch element, no query, no key row."""
import pytest

from gpu_util import require_gpu, torch
from test_gpu_attention_masked import i32, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("B,n,m", [(0, 3, 5), (2, 0, 5), (0, 0, 0), (2, 3, 0), (1, 300, 0), (2, 0, 0)])
def test_empty_sizes(B, n, m):
    from stream_diffusion_transformer_b200 import model
    q = torch.randn(B, n, 4, 128, device="cuda").bfloat16()
    k = torch.randn(B, m, 2, 128, device="cuda").bfloat16()
    ids = lambda rows: torch.zeros(B, rows, dtype=torch.int32, device="cuda")
    for kw in ({}, dict(causal=True, prefix_len=i32(*[1] * B), kv_len=i32(*[m] * B)),
               dict(softcap=9.0, slopes=slopes_of(4), q_doc=ids(n), k_doc=ids(m))):
        got = model.attention_masked(q, k, k, **kw)
        assert got.shape == q.shape and got.dtype == torch.bfloat16 and (got == 0).all()
        room = torch.full((B, n + 2, 5, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        view = room[:, 1:n + 1, :4]
        assert model.attention_masked(q, k, k, out=view, **kw) is view and (view == 0).all()
        view.fill_(5.0)
        assert (room == 5.0).all()


def test_empty_sizes_are_checked_too():
    from stream_diffusion_transformer_b200 import model
    q = torch.randn(0, 3, 4, 128, device="cuda").bfloat16()
    k = torch.randn(0, 5, 2, 128, device="cuda").bfloat16()
    for bad in (lambda: model.attention_masked(q.float(), k, k), lambda: model.attention_masked(q, k, k[:, :4]),
                lambda: model.attention_masked(q, k, k, slopes=torch.ones(3, device="cuda")),
                lambda: model.attention_masked(q, k, k, out=torch.empty_like(k))):
        with pytest.raises(ValueError):
            bad()
