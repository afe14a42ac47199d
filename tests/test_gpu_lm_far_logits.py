"""Gradients of the softmax operators from a stored lse where the logits are
far from zero."""
import pytest
import torch

import gradient_compression_sgd_gc_gb300 as gc

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def _device(x, pad=0, start=0):
    N, V = x.shape
    buf = torch.full((start + N * (V + pad),), 77.0, dtype=x.dtype, device=DEV)
    d = buf[start:].view(N, V + pad)[:, :V]
    d.copy_(x)
    return d


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tau", [2.0, 64.0])
def test_one_logit_below_the_floor(dtype, tau):
    """One real logit of -2^60 tau / 2, all others masked: p = 1 there.  Every number is a power of two, so the results
    are exact."""
    V, at = 700, 300
    x = torch.full((3, V), -INF, dtype=dtype)
    x[:, at] = -2.0 ** 59 * tau * (1.0 if tau > 2 else 1.5)
    d = _device(x, 3, 1)
    ids = torch.tensor([at, -1, at], device=DEV)
    lp, H, lse = (torch.empty(3, device=DEV) for _ in range(3))
    gc.token_logprobs(d, ids, lp, entropy=H, lse=lse, temperature=tau)
    assert not lp.any() and not H.any()
    out = torch.full_like(d, 9.0)
    g, h = torch.tensor([1.0, 2.0, 0.5], device=DEV), torch.tensor([0.0, 0.0, 4.0], device=DEV)
    gc.token_logprobs_grad(d, ids, lse, H, g, h, out, temperature=tau)
    assert not out.any()

    # half of the teacher's mass on the real logit, half on a masked one
    top = torch.tensor([[at, 5]] * 3, dtype=torch.int32, device=DEV)
    t, w, loss = torch.zeros(3, 2, device=DEV), torch.ones(3, device=DEV), torch.empty(3, device=DEV)
    gc.distill_loss(d, top, t, loss, lse, temperature=tau)
    want = torch.zeros(3, V)
    want[:, at], want[:, 5] = 0.5 * tau, -0.5 * tau
    gc.distill_grad(d, top, t, lse, w, out, temperature=tau)
    assert torch.equal(out.cpu().float(), want)
    gc.distill_loss_grad(d, top, t, w, loss, out, temperature=tau)
    assert torch.equal(out.cpu().float(), want)
