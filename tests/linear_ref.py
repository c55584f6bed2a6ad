"""Plain 64-bit forms of linear attention with a decay per head and of the block norm, on the CPU, with
error bounds derived from the number of fp32 roundings.

Every bound has the form c * u * A: u = 2^-24 (a rounding to nearest of fp32 is off by at most half a step,
u relative), A the sum of the absolute values of the terms that a value is made of, c the number of
roundings that the longest path from an input to that value can meet. bf16 outputs add 2^-8 of the value
(half a step of an 8-bit significand).
"""

import torch

U32 = 2.0 ** -24
UB16 = 2.0 ** -8


def recur(q, k, v, alpha, S, absolute=False, ckpt=-1):
    """One row. q, k [T, Hk, dk], v [T, H, dv], alpha [H] or [T, H], S [H, dv, dk]; returns (out [T, H, dv],
    state, state after ckpt tokens or None). With absolute the same over absolute values: the A above."""
    f = (lambda x: x.double().abs()) if absolute else (lambda x: x.double())
    T, H = v.shape[0], v.shape[1]
    group = H // k.shape[1]
    q, k = f(q).repeat_interleave(group, 1), f(k).repeat_interleave(group, 1)
    v, alpha, S = f(v), f(alpha).expand(T, H), f(S).clone()
    out = torch.zeros(T, H, v.shape[2], dtype=torch.float64)
    at = S.clone() if ckpt == 0 else None
    for t in range(T):
        S = S * alpha[t][:, None, None] + v[t][:, :, None] * k[t][:, None, :]
        out[t] = (S @ q[t][:, :, None])[:, :, 0]
        if t + 1 == ckpt:
            at = S.clone()
    return out, S, at


def roundings(T, dk):
    """Roundings on the longest path of a T-token row: two per token for a decay and an add to the state
    (token by token; the chunk form meets fewer), a product of dk terms and one of up to 64 tokens summed
    in any order, and 16 for the decay products inside a chunk and the scaling of a term."""
    return 2 * T + dk + 64 + 16


def check(got, ref, bound, what):
    """Every value within its bound."""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound
    worst = ((got - ref).abs() / bound.clamp_min(1e-300)).max().item() if got.numel() else 0.0
    assert not (over > 0).any(), f"{what}: {int((over > 0).sum())} of {got.numel()} values past their bound " \
                                 f"(largest {worst:.3g} times)"


def out_bound(A, T, dk, ref, bf16):
    """bf16 outputs may be formed from operands in two bf16 parts, hi = x rounded and lo = x - hi rounded: x - hi is
    within 2^-9 of x (half a step of 8 bits), the rounding of lo within 2^-9 of that, so each term is off by at
    most 2^-18 of itself (64 u) besides the fp32 roundings."""
    c = roundings(T, dk) + (64 if bf16 else 0)
    return c * U32 * A + (UB16 * ref.abs() * (1 + 1e-3) if bf16 else 0) + 1e-37


def gated(o, gate, weight, eps):
    """y = o / sqrt(mean o^2 + eps) * weight * sigmoid(gate) over the last axis."""
    y = o / ((o * o).mean(-1, keepdim=True) + eps).sqrt()
    return y * (weight.double() if weight is not None else 1.0) / (1 + torch.exp(-gate.double()))


def norm_ref(resid, z=None, w_post=None, gate=None, scale=1.0, w_pre=None, eps=1e-6):
    """(r', bound on |error of r'|, y or None, bound on |error of y|) before any rounding to bf16.

    The mean square of D positive terms is off by at most (D / threads + 20) u relative where a thread sums
    up to 64 of them and the partial sums meet up to 20 more additions; its root by half that. With the
    reciprocal, the products and an exponential good to 2 steps, 64 u covers a normalized, gated term."""
    r = resid.double()
    c = 64 * U32
    err = torch.zeros_like(r)
    if z is not None:
        t = z.double()
        if w_post is not None:
            t = t / ((t * t).mean(-1, keepdim=True) + eps).sqrt() * w_post.double()
        if gate is not None:
            t = t / (1 + torch.exp(-gate.double()))
        t = t * scale
        r = r + t
        err = c * t.abs() + U32 * r.abs()
    if w_pre is None:
        return r, err + 1e-37, None, None
    ms = (r * r).mean(-1, keepdim=True) + eps
    f = 1 / ms.sqrt()
    y = r * f * w_pre.double()
    df = err.square().mean(-1, keepdim=True).sqrt() * f  # relative change of f by the errors of r'
    yerr = (err * f * w_pre.double()).abs() * (1 + 1e-3) + (c + df * (1 + 1e-3)) * y.abs() + 1e-37
    return r, err + 1e-37, y, yerr
