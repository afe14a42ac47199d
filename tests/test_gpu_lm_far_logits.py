"""Gradients of the softmax operators from a stored lse where the logits are
far from zero: rows below -2^60, and rows whose lse, rounded to fp32, no longer
holds the logarithm of the sum.  Bounds: lm_helpers, with a term for lse's
rounding only below 1024."""
import pytest
import torch

import gradient_compression_sgd_gc_gb300 as gc
from lm_helpers import U, distill64, entropy64, round_tol, softmax64, sum_error

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


FAR = [-1e9, 1e9, -1e20, -1e30, 1e38, "lowest", -3000.0]


def _far_rows(V, dtype, far, seed):
    """Rows of one far value; of far values at three distances; of normal values; the far value with a few larger."""
    far = torch.finfo(dtype).min if far == "lowest" else far
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(6, V, generator=g) * 2.5).to(dtype)
    x[1] = far
    x[2] = far
    x[2, ::3] = far * (1.0 - 2.0 ** -7)              # apart by some units in the last place of bf16
    x[2, V // 2:] = -INF
    x[4] = far
    x[4, ::5] = torch.randn(x[4, ::5].shape, generator=g).to(dtype)       # far values beside usual ones
    x[5] = (x[5].float() + max(-4000.0, min(4000.0, far))).to(dtype)      # an offset that leaves the differences
    return x


def _from_max(x):
    """The rows less their largest entry, in 64 bits, which changes no softmax: at -1e20 a double's unit is 16384, and
    max + log(sum) would lose the logarithm."""
    x = x.double()
    return x - x.max(dim=1, keepdim=True).values


def _log_error(V, lse):
    """Absolute error of log p beside the sum's and its own rounding: that of lse below 1024, of the sum's logarithm
    above."""
    near = lse.abs() < 1024
    size = torch.where(near, lse.abs(), torch.zeros_like(lse)) + float(torch.log(torch.tensor(float(V))))
    return 8 * U * size[:, None]


def _p_error(V, lp, lse):
    """Relative error of p: the sum's, the exponent's rounding and the logarithm's."""
    return sum_error(V) + (16 + 4 * torch.nan_to_num(lp.abs(), posinf=0.0).clamp(max=200.0)) * U + _log_error(V, lse)


@pytest.mark.parametrize("V,tau", [(40, 1.0), (1003, 0.5), (1003, 100.0), (20_011, 1.0), (20_011, 100.0), (131_072, 0.5)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_log_probability_gradient_far_from_zero(V, dtype, tau):
    for k, far in enumerate(FAR):
        x = _far_rows(V, dtype, far, 10 * V + k)
        N = x.shape[0]
        gen = torch.Generator().manual_seed(k)
        ids = torch.randint(0, V, (N,), generator=gen)
        ids[2] = 0
        ids[5] = -1
        g, h = torch.randn(N, generator=gen), torch.randn(N, generator=gen)
        pad, start = (0, 0) if k % 2 else (3, 1)
        d = _device(x, pad, start)
        lpd, H, lse = (torch.empty(N, device=DEV) for _ in range(3))
        gc.token_logprobs(d, ids.to(DEV), lpd, entropy=H, lse=lse, temperature=tau)
        lse64, (_, _, lp, p) = softmax64(x, tau)[1], softmax64(_from_max(x), tau)
        one = torch.zeros_like(p)
        rows = torch.arange(N)[ids >= 0]
        one[rows, ids[rows]] = 1.0
        here = (ids >= 0).double()[:, None]
        H64 = entropy64(lp, p)[:, None]
        lp0 = torch.where(p == 0, torch.zeros_like(lp), lp)
        gd, hd = g.double()[:, None], h.double()[:, None]
        ref = (gd * here * (one - p) - hd * p * (lp0 + H64)) / tau
        base, rel = sum_error(V), _p_error(V, lp, lse64)
        tol = (gd.abs() * (p * rel + one * 4 * U) + hd.abs() * p * (rel + 8 * U) * (lp0.abs() + H64)
               + hd.abs() * p * (2 * base * (2 + H64) + base + 8 * U * lp0.abs() + _log_error(V, lse64))) / tau
        # a p below 2^-126 is zero
        tol = tol + 2.0 ** -126 * (gd.abs() + hd.abs() * (lp0.abs() + H64)) / tau + round_tol(dtype, ref)
        outs = []
        for out in (torch.full_like(d, 9.0), _device(torch.zeros_like(x), 2, 5), d):        # the last in place
            gc.token_logprobs_grad(d, ids.to(DEV), lse, H, g.to(DEV), h.to(DEV), out, temperature=tau)
            err = (out.cpu().double() - ref).abs()
            assert (err <= tol).all(), (far, float((err - tol).max()), int((err - tol).max(1).values.argmax()))
            outs.append(out.cpu())
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("V,tau", [(40, 1.0), (1003, 0.5), (1003, 100.0), (20_011, 1.0), (20_011, 100.0), (131_072, 0.5)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_distillation_gradient_far_from_zero(V, dtype, tau):
    K = 7
    for k, far in enumerate(FAR):
        x = _far_rows(V, dtype, far, 10 * V + k)
        N = x.shape[0]
        gen = torch.Generator().manual_seed(k)
        ids = torch.randint(0, V // 2, (N, K), generator=gen).int()
        t = torch.randn(N, K, generator=gen) * 2.5
        w = torch.rand(N, generator=gen) + 0.1
        w[3] = 0.0
        pad, start = (0, 0) if k % 2 else (3, 1)
        d = _device(x, pad, start)
        _, ref, _, p, qv = distill64(_from_max(x), ids, t, tau, w)
        lp = torch.log(p.clamp(min=1e-40))
        tol = w.double()[:, None] * tau * (p + qv) * (_p_error(V, lp, softmax64(x, tau)[1]) + (K + 40) * U)
        tol = tol + round_tol(dtype, ref) + 2.0 ** -126 * tau * w.double()[:, None]
        idd, td, wd = ids.to(DEV), t.to(DEV), w.to(DEV)
        loss, lse = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
        gc.distill_loss(d, idd, td, loss, lse, temperature=tau)
        for out in (torch.full_like(d, 9.0), _device(torch.zeros_like(x), 2, 5), d):        # the last in place
            gc.distill_grad(d, idd, td, lse, wd, out, temperature=tau)
            err = (out.cpu().double() - ref).abs()
            assert (err <= tol).all(), (far, float((err - tol).max()), int((err - tol).max(1).values.argmax()))
        d = _device(x, pad, start)
        gc.distill_loss_grad(d, idd, td, wd, loss, d, temperature=tau)
        assert ((d.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("N", [1, 700])
def test_gradients_of_many_rows_without_a_choice(N):
    """Rows filled with one mask value, among usual ones: uniform, whatever the value."""
    V = 5003
    x = torch.randn(N, V, generator=torch.Generator().manual_seed(1))
    x[::2] = -1e9
    x[1::6] = torch.finfo(F32).min
    d = _device(x)
    lp, H, lse = (torch.empty(N, device=DEV) for _ in range(3))
    ids = torch.full((N,), 7, device=DEV)
    gc.token_logprobs(d, ids, lp, entropy=H, lse=lse, temperature=0.5)
    out, g = torch.empty_like(d), torch.ones(N, device=DEV)
    gc.token_logprobs_grad(d, ids, lse, None, g, None, out, temperature=0.5)
    p = softmax64(_from_max(x), 0.5)[3]
    p[:, 7] -= 1.0
    assert ((out.cpu().double() + 2 * p).abs() <= 2 * (p.abs() + 1e-9) * (sum_error(V) + 8 * U * 40)).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_given_tokens_at_masked_logits(dtype):
    """The token's and the teacher's terms remain where the logit is -inf, in a usual row and in one of nothing else;
    other masked places have no gradient."""
    V, tau = 2500, 2.0
    x = torch.randn(4, V, generator=torch.Generator().manual_seed(3)).to(dtype)
    x[:, 100:200] = -INF
    x[1] = x[3] = -INF
    d = _device(x, 3, 1)
    ids = torch.tensor([150, 150, 5, -1], device=DEV)
    lp, H, lse = (torch.empty(4, device=DEV) for _ in range(3))
    gc.token_logprobs(d, ids, lp, entropy=H, lse=lse, temperature=tau)
    assert lp[0] == -INF and lp[1] == -INF and H[1] == 0 and lp[3] == 0
    out = torch.full_like(d, 9.0)
    g, h = torch.tensor([0.5, 0.25, 1.0, 4.0], device=DEV), torch.tensor([1.0, 8.0, 0.0, 8.0], device=DEV)
    gc.token_logprobs_grad(d, ids, lse, H, g, h, out, temperature=tau)
    out = out.cpu().float()
    assert out[0, 150] == 0.25 and out[1, 150] == 0.125        # g / tau, exact in both types
    masked = torch.isinf(x)
    masked[0, 150] = masked[1, 150] = False
    assert not out[masked].any() and torch.isfinite(out).all() and out[0, 5] != 0

    top = torch.tensor([[150, 5]] * 4, dtype=torch.int32, device=DEV)
    t, w, loss = torch.zeros(4, 2, device=DEV), torch.ones(4, device=DEV), torch.empty(4, device=DEV)
    gc.distill_loss(d, top, t, loss, lse, temperature=tau)
    assert (loss == INF).all()
    masked[:, 150] = masked[:, 5] = False
    for call in (lambda: gc.distill_grad(d, top, t, lse, w, out, temperature=tau),
                 lambda: gc.distill_loss_grad(d, top, t, w, loss, out, temperature=tau)):
        out = torch.full_like(d, 9.0)
        call()
        out = out.cpu().float()
        assert (out[:, 150] == -1.0).all() and (out[[1, 3], 5] == -1.0).all()      # -w tau q
        assert not out[masked].any() and torch.isfinite(out).all() and out[0, 6] > 0


@pytest.mark.parametrize("tau", [0.9, 7.0, 1.7, 0.3])
def test_lse_below_1024_is_rounded_once(tau):
    """lse within its own rounding (2^-15 from 512 to 1024) and the sum's error, at temperatures whose inverse is not
    an fp32 number; so the probabilities that a gradient forms from it sum to one as closely."""
    N, V = 300, 40
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(N, V, generator=gen) + (torch.linspace(520, 1000, N) * tau)[:, None]
    x[::2] *= -1.0
    d, ids = _device(x, 1, 3), torch.randint(0, V, (N,), generator=gen).to(DEV)
    lp, lse, loss = (torch.empty(N, device=DEV) for _ in range(3))
    top, t = ids[:, None].int().contiguous(), torch.zeros(N, 1, device=DEV)
    m = x.double().max(1).values
    want = m / tau + torch.log(torch.exp(_from_max(x) / tau).sum(1))
    tol = 2.0 ** -15 + sum_error(V)
    for call in (lambda: gc.token_logprobs(d, ids, lp, lse=lse, temperature=tau),
                 lambda: gc.distill_loss(d, top, t, loss, lse, temperature=tau)):
        lse.zero_()
        call()
        assert ((lse.cpu().double() - want).abs() <= tol).all()
    out, g = torch.empty_like(d), torch.ones(N, device=DEV)
    gc.token_logprobs_grad(d, ids, lse, None, g, None, out, temperature=tau)
    assert (out.cpu().double().sum(1).abs() * tau <= tol + 64 * U).all()
    gc.distill_grad(d, top, t, lse, g, out, temperature=tau)
    assert (out.cpu().double().sum(1).abs() / tau <= tol + 64 * U).all()
