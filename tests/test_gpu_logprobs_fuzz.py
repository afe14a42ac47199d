"""Seeded random configurations of the log probabilities and their gradient
against plain 64-bit forms: sizes, types, strides, starts, masks, ties, absent
tokens and numbers of alternatives drawn together.

Bounds as in lm_helpers and test_gpu_logprobs, with two properties of fp32 in
place: a log probability that leaves its range is -inf (the lowest value
divided by a temperature below 1), and a probability below 2^-126 may be zero,
which leaves its whole gradient out.  Results below fp32's or bf16's normal
range are rounded to a multiple of 2^-133 at worst."""
import pytest
import torch

import gradient_compression_sgd_gc_gb300 as gc
from lm_helpers import U, entropy64, round_tol, softmax64, sum_error, top64

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")
MAX32 = float(torch.finfo(F32).max)


class Draw:
    def __init__(self, case):
        self.g = torch.Generator().manual_seed(7000 + case)

    def whole(self, lo, hi):
        """Spread over the logarithm."""
        return max(lo, min(hi, round(lo * (hi / lo) ** float(torch.rand(1, generator=self.g)))))

    def one(self, *choices):
        return choices[int(torch.randint(0, len(choices), (1,), generator=self.g))]

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g)

    def chance(self, *shape):
        return torch.rand(*shape, generator=self.g)


def _place(x, pad, start):
    buf = torch.full((start + x.shape[0] * (x.shape[1] + pad),), 77.0, dtype=x.dtype, device=DEV)
    d = buf[start:].view(x.shape[0], x.shape[1] + pad)[:, :x.shape[1]]
    d.copy_(x)
    return d


def _draw_logits(r, N, V, dtype):
    """Logits, and which of them are not masked."""
    x = (r.normal(N, V) * r.one(0.5, 2.5, 8.0)).to(dtype)
    if r.one(True, False, False):
        x = (x * 2).round() / 2                                  # many ties
    keep = torch.ones(N, V, dtype=torch.bool)
    low = r.one(None, None, -INF, torch.finfo(dtype).min)
    if low is not None:
        keep = r.chance(N, V) < r.one(0.5, 0.05)
        keep[torch.arange(N), torch.randint(0, V, (N,), generator=r.g)] = True
        x = torch.where(keep, x, torch.full_like(x, low))
    return x, keep


@pytest.mark.parametrize("case", range(32))
def test_log_probabilities(case):
    r = Draw(case)
    dtype = r.one(F32, BF16)
    N, V = r.one((r.whole(1, 30), r.whole(1, 90_000)), (r.whole(150, 400), r.whole(1, 9000)), (700, r.whole(1, 3000)))
    K = min(V, r.one(0, 1, 7, 33, 64, 100, 128))
    tau = r.one(1.0, 0.7, 3.0)
    x, keep = _draw_logits(r, N, V, dtype)
    d = _place(x, r.one(0, 0, 1, 7, 64), r.one(0, 0, 1, 5))
    ids = torch.multinomial(keep.float(), 1, generator=r.g)[:, 0]
    ids[r.chance(N) < 0.1] = -1
    ids = ids.to(r.one(torch.int32, torch.int64))
    present = ids >= 0
    at = ids.clamp(min=0).long()[:, None]

    lp, H, lse = (torch.empty(N, device=DEV) for _ in range(3))
    ti, tl = torch.empty(N, K, dtype=torch.int32, device=DEV), torch.empty(N, K, device=DEV)
    gc.token_logprobs(d, ids.to(DEV), lp, entropy=H, lse=lse, top_ids=ti if K else None, top_logprobs=tl if K else None,
                      temperature=tau)
    _, lse64, lp64, p64 = softmax64(x, tau)
    H64, base = entropy64(lp64, p64), sum_error(V)
    lp64 = torch.where(lp64 < -MAX32, -INF, lp64)
    want = torch.where(present, lp64.gather(1, at)[:, 0], 0.0)
    assert ((lp.cpu().double() - want).abs() <= base + 4 * U * (1 + want.abs())).all()
    assert ((lse.cpu().double() - lse64).abs() <= base + 8 * U * lse64.abs()).all()
    assert ((H.cpu().double() - H64).abs() <= 2 * base * (2 + H64)).all()
    if K:
        best = top64(x, K)
        assert torch.equal(ti.cpu().long(), best)
        ref, got = lp64.gather(1, best), tl.cpu().double()
        fin = torch.isfinite(ref)
        assert torch.equal(got[~fin], ref[~fin])
        assert ((got - ref).abs()[fin] <= (base + 4 * U * (1 + ref.abs()))[fin]).all()

    # the gradient from what the forward pass has left, in fp32 as it is
    g, h = r.normal(N), r.normal(N)
    gd, hd = g.double()[:, None], h.double()[:, None]
    l0, H0 = lse.cpu().double()[:, None], H.cpu().double()[:, None]
    q = x.double() / tau - l0
    p = torch.exp(q)
    q = torch.where(p == 0, 0.0, q)
    one = torch.zeros_like(p).scatter_(1, at, present.double()[:, None])
    ref = (gd * (one - present.double()[:, None] * p) - hd * p * (q + H0)) / tau
    size = (gd.abs() * (one + p) + hd.abs() * p * (q.abs() + H0)) / tau
    tol = size * U * (24 + 4 * q.abs().clamp(max=200.0) + 4 * l0.abs()) + hd.abs() * p * U * (4 * l0.abs() + 4) / tau
    tol = tol + torch.where(p < 2.0 ** -125, size, 0.0) + round_tol(dtype, ref) + 2.0 ** -132
    out = torch.empty_like(d) if r.one(True, False) else _place(torch.zeros_like(x), 3, 2)
    for to in (out, d):                                          # the second in place
        gc.token_logprobs_grad(d, ids.to(DEV), lse, H, g.to(DEV), h.to(DEV), to, temperature=tau)
        assert ((to.cpu().double() - ref).abs() <= tol).all()
