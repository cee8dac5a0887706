"""Plain 64-bit masked attention, its log-sum-exp and its gradients, written from
the definitions over the dense token mask (natural order, torch tensors).  Test
infrastructure for the gradient and cache tests; small grids only.

Every function also returns the sums of magnitudes from which the tests derive
their tolerances: bf16 rounds by at most 2^-8 of a value, fp32 by 2^-24."""
from __future__ import annotations

import math

import torch

BF16 = 2.0 ** -8
FP32 = 2.0 ** -24


def token_mask(T, H, W, gamma, Rt, radius, disk=False, frame=0, cached=None):
    """[heads, n, m]: query i (radius[:, i]) of the frames from `frame` on keeps key j of the first `cached` frames (all T by default)."""
    n = frame * H * W + torch.arange(radius.shape[1], device=radius.device)
    m = torch.arange((T if cached is None else cached) * H * W, device=radius.device)
    return pairs_kept(T, H, W, gamma, Rt, n, m, radius, disk)


def pairs_kept(T, H, W, gamma, Rt, n, m, radius, disk=False):
    split = lambda x: (x // (H * W), x // W % H, x % W)  # noqa: E731
    (tn, hn, wn), (tm, hm, wm) = split(n), split(m)
    dt = (tn[:, None] - tm[None]).abs()
    dh, dw = (hn[:, None] - hm[None]).abs(), (wn[:, None] - wm[None]).abs()
    keep = torch.zeros(radius.shape[0], len(n), len(m), dtype=torch.bool, device=radius.device)
    for delta in range(min(Rt, T - 1) + 1):
        s = torch.floor(radius.double() * math.pow(gamma, delta) + 1e-9)[..., None]
        near = (dh * dh + dw * dw)[None] <= s * s if disk else torch.maximum(dh, dw)[None] <= s
        keep |= (dt == delta)[None] & near & (radius >= 0)[..., None]
    return keep


def attention(q, k, v, keep, p_round=BF16):
    """(out, lse, bound of out before its own rounding, bound of lse); rows that keep nothing: 0 and -inf.
    p_round: what the probabilities are rounded by before the product with v (0: not rounded)."""
    q, k, v = q.double(), k.double(), v.double()
    d = q.shape[-1]
    x = (q @ k.mT / math.sqrt(d)).masked_fill(~keep, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse.nan_to_num(neginf=0.0)[..., None]).masked_fill(~keep, 0.0)
    out = p @ v
    # scores: d products summed in fp32 (d * 2^-24 of the sum of magnitudes), scaled once more
    dx = (q.abs() @ k.abs().mT / math.sqrt(d)) * ((d + 4) * FP32) + 2.0 ** -20 * (1 + x.masked_fill(~keep, 0.0).abs())
    # numerator and denominator each carry P's error; P is also rounded to bf16 (the numerator alone)
    err = (p * dx).sum(-1)
    out_err = (p * (p_round + dx)) @ v.abs() + (err + 2.0 ** -16)[..., None] * (p @ v.abs())
    lse_err = err + 2.0 ** -18 * (1 + lse.nan_to_num(neginf=0.0).abs())
    # a row of no keys has no error to allow
    return out, lse, out_err, lse_err


def gradients(q, k, v, out, lse, dout, keep):
    """((dq, dk, dv), their bounds before their own rounding) from the given out and lse."""
    q, k, v, out, lse, dout = (x.double() for x in (q, k, v, out, lse, dout))
    d = q.shape[-1]
    root = 1 / math.sqrt(d)
    x = q @ k.mT * root
    p = torch.exp(x - lse[..., None]).masked_fill(~keep, 0.0)
    dp, big = dout @ v.mT, dout.abs() @ v.abs().mT
    delta, big_d = (dout * out).sum(-1, keepdim=True), (dout * out).abs().sum(-1, keepdim=True)
    ds = p * (dp - delta)
    grads = (ds @ k * root, ds.mT @ q * root, p.mT @ dout)
    p_err = p * ((q.abs() @ k.abs().mT * root) * ((d + 4) * FP32) + 2.0 ** -20 * (1 + x.abs() + lse.abs()[..., None]))
    ds_err = p_err * (dp - delta).abs() + (p + p_err) * (big + big_d) * ((d + 4) * FP32)
    # rounded to bf16 for the products, then summed in fp32 over at most n rows
    sums = max(q.shape[1], k.shape[1]) * FP32
    ds_err, p_err = ds_err + (BF16 + sums) * (ds.abs() + ds_err), p_err + (BF16 + sums) * (p + p_err)
    return grads, (ds_err @ k.abs() * root, ds_err.mT @ q.abs() * root, p_err.mT @ dout.abs())


def check(got, ref, bound, name=""):
    """got within bound plus got's own rounding of ref."""
    got64 = got.double()
    nothing = ref == -math.inf
    assert torch.equal(got64 == -math.inf, nothing), name
    got64, ref, bound = (x.masked_fill(nothing, 0.0) for x in (got64, ref, bound))
    step = BF16 if got.dtype == torch.bfloat16 else FP32
    tol = bound * (1 + step) + ref.abs() * step + 1e-30
    over = (got64 - ref).abs() - tol
    assert torch.isfinite(got64).all(), name
    assert over.max() <= 0, f"{name}: {int((over > 0).sum())} of {over.numel()} beyond the bound, worst by {over.max():.3e} " \
                            f"(error {float((got64 - ref).abs().max()):.3e})"
