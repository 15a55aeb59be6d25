"""Attention with a sliding window and sinks in 64 bits, with bounds on what the
kernels' roundings can do to each element.

Roundings (half a step: bf16 2^-8, relative): the forward rounds each weight to
bf16 before the product with V and the output once; sums and the normaliser are
fp32 of unrounded weights.  The backward recomputes P (rounded to bf16), rounds
dS = P o (dP - D) to bf16, sums in fp32 and rounds each gradient once; its D comes
from the rounded output.  fp32 effects (d-term score sums, 2^x to 2^-22, the
log-sum-exp that P is recomputed from) stay below FP32 = 4e-4 relative for the
scores drawn here: 128 terms of |q k| <= 20, times scale 0.09 and 2^-24 a term, is
1.4e-5 in a score, and the exponential turns an absolute error of a score into a
relative one of P; 4e-4 leaves a factor of 25 for correlated sums.
"""
import math

import torch

BF16 = 2.0 ** -8
FP32 = 4e-4
LSE_TOL = 4e-4


def visible(n_q, n_k, window, sinks, causal=True, device="cpu"):
    """[n_q, n_k] truth values; window None or 0: no window."""
    p = torch.arange(n_q, device=device)[:, None] + (n_k - n_q)
    j = torch.arange(n_k, device=device)[None]
    if not causal:
        return torch.ones(n_q, n_k, dtype=torch.bool, device=device)
    m = j <= p
    if window:
        m = m & ((p - j < window) | (j < sinks))
    return m


def _weights(q, k, scale, mask):
    """P [H, n_q, n_k] and lse [H, n_q]; q [n_q, H, d], k [n_k, H, d] in 64 bits."""
    s = torch.einsum("ihd,jhd->hij", q, k) * scale
    s = s.masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:2], -math.inf, dtype=s.dtype, device=s.device)
    p = torch.where(mask, torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None]),
                    torch.zeros((), dtype=s.dtype, device=s.device))
    return p, lse


def _spread(x, H):
    return x.double().repeat_interleave(H // x.shape[1], 1)


def forward(q, k, v, scale, mask):
    """One sequence: (o, lse, bound of o); q [n_q, H, d], k/v [n_k, Hk, d]."""
    H = q.shape[1]
    k, v = _spread(k, H), _spread(v, H)
    p, lse = _weights(q.double(), k, scale, mask)
    o = torch.einsum("hij,jhd->ihd", p, v)
    a = torch.einsum("hij,jhd->ihd", p, v.abs())
    return o, lse, (BF16 + FP32) * a + BF16 * o.abs() + 1e-6


def backward(q, k, v, dout, scale, mask):
    """One sequence: ((dq, dk, dv), their bounds)."""
    H, Hk = q.shape[1], k.shape[1]
    q, dout, kk, vv = q.double(), dout.double(), _spread(k, H), _spread(v, H)
    p, _ = _weights(q, kk, scale, mask)
    o = torch.einsum("hij,jhd->ihd", p, vv)
    a = torch.einsum("hij,jhd->ihd", p, vv.abs())
    dp = torch.einsum("ihd,jhd->hij", dout, vv)
    ds = p * (dp - (dout * o).sum(-1).T[..., None])
    # D = do . o from the rounded output; the rounded weights make o off by BF16 (a + |o|).
    dD = (dout.abs() * ((BF16 + FP32) * a + BF16 * o.abs())).sum(-1).T[..., None]
    # dP: fp32 sum of d terms.
    ddp = torch.einsum("ihd,jhd->hij", dout.abs(), vv.abs()) * 2.0 ** -20
    e_ds = (2 * BF16 + FP32) * ds.abs() + p * (dD + ddp)
    e_p = (BF16 + FP32) * p

    def group(x):
        return x.reshape(x.shape[0], Hk, H // Hk, x.shape[-1]).sum(2)
    dq = torch.einsum("hij,jhd->ihd", ds, kk) * scale
    dk = group(torch.einsum("hij,ihd->jhd", ds, q)) * scale
    dv = group(torch.einsum("hij,ihd->jhd", p, dout))
    bq = torch.einsum("hij,jhd->ihd", e_ds, kk.abs()) * scale + BF16 * dq.abs() + 1e-6
    bk = group(torch.einsum("hij,ihd->jhd", e_ds, q.abs())) * scale + BF16 * dk.abs() + 1e-6
    bv = group(torch.einsum("hij,ihd->jhd", e_p, dout.abs())) + BF16 * dv.abs() + 1e-6
    return (dq, dk, dv), (bq, bk, bv)


def check(got, ref, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), "%s: not finite" % what
    over = ((got - ref).abs() - bound).max().item() if got.numel() else -1.0
    worst = ((got - ref).abs() / bound).max().item() if got.numel() else 0.0
    assert over <= 0, "%s: %.3g times its bound" % (what, worst)


def check_lse(got, ref, what):
    empty = ref == -math.inf
    assert torch.equal(got == -math.inf, empty), "%s: rows without keys differ" % what
    d = (got.double() - ref).masked_fill(empty, 0.0).abs()
    assert d.numel() == 0 or d.max().item() <= LSE_TOL, "%s: lse off by %.3g" % (what, d.max().item())
