"""Plain 64-bit definitions of the operators around the linear layers, with the quantities
their error bounds need.  Everything runs in float64 torch on the inputs' device."""
import math

import torch

U32 = 2.0 ** -24


def unit(dtype):
    """Unit roundoff of a rounding to nearest."""
    return {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[dtype]


def least(dtype):
    """Half of the smallest subnormal: the absolute error of a rounding near zero."""
    return {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}[dtype]


def assert_within(got, ref, tol, what=""):
    got, ref, tol = got.double(), ref.double(), tol.double()
    assert got.shape == ref.shape
    assert not torch.isnan(got).any(), "%s: NaN" % what
    excess = (got - ref).abs() - tol
    worst = excess.max().item() if excess.numel() else 0.0
    assert worst <= 0, "%s: off by up to %g beyond the bound" % (what, worst)


def norm_rope(x, weight, eps, norm, cos, sin, interleaved):
    """x [T, H, D] in 64 bits -> (y, magnitude): magnitude bounds the terms of each y."""
    x = x.double()
    if norm:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            x = x * weight.double()
    if cos is None:
        return x, x.abs()
    half = cos.shape[1]
    y, mag = x.clone(), x.abs().clone()
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos.double()[:, None], sin.double()[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def attend(q, k, v, scale, seen, p_unit, p_least):
    """q [n, D], k and v [m, D], seen [n, m] bool -> (out, lse, tol) in 64 bits.

    tol bounds a kernel that sums in fp32 and rounds each softmax weight once to p_unit:
      * a score is a D-term fp32 dot product, scaled: off by (D + 8) u sum_d |q k| scale at
        most, and its exponential by another 2^-21 (approximate base-2 exponential, and the
        rounding of its argument, at most 2^-24 times an argument below 2^3 log2 e units per
        unit of score): a relative error eps of each weight, of the sum, and so 2 eps of out;
      * each weight rounded once: p_unit of sum_j w_j |v_j|, or p_least of an unnormalized
        weight (at most 1 for the largest) where it is subnormal;
      * the sum over keys in fp32: (m + 8) u sum_j w_j |v_j| at most.
    """
    q, k, v = q.double(), k.double(), v.double()
    k_seen = torch.where(seen.any(0)[:, None], k, torch.zeros_like(k))
    v_seen = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))
    k_seen, v_seen = torch.nan_to_num(k_seen), torch.nan_to_num(v_seen)
    score = (q @ k_seen.t() * scale).masked_fill(~seen, -math.inf)
    top = score.max(-1, keepdim=True).values if k.shape[0] else score.new_full((q.shape[0], 1), -math.inf)
    top0 = torch.where(top.isinf(), torch.zeros_like(top), top)
    e = torch.exp(score - top0)
    total = e.sum(-1, keepdim=True)
    safe = torch.where(total > 0, total, torch.ones_like(total))
    out = e @ v_seen / safe
    lse = (top + torch.log(total))[:, 0]
    mags = e @ v_seen.abs() / safe
    dot_abs = ((q.abs() @ k_seen.abs().t()) * abs(scale)).masked_fill(~seen, 0.0)
    dmax = dot_abs.max(-1, keepdim=True).values if k.shape[0] else torch.zeros_like(total)
    span = torch.where(seen, (top0 - score).nan_to_num(posinf=0.0), torch.zeros_like(score))
    smax = span.max(-1, keepdim=True).values if k.shape[0] else torch.zeros_like(total)
    eps = (q.shape[1] + 8) * U32 * dmax + 2.0 ** -21 + 4 * U32 * smax
    m = seen.sum(-1, keepdim=True)
    tol = (2 * eps + p_unit + (m + 8) * U32) * mags + p_least * m / safe * v_seen.abs().amax(0) if k.shape[0] \
        else torch.zeros_like(out)
    return out, lse, tol, (eps[:, 0] + (m[:, 0] + 8) * U32) + 2.0 ** -20 * (1 + lse.abs().nan_to_num(posinf=0.0))
