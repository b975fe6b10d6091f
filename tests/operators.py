"""64-bit definitions of the operators around the quantized layers, with bounds
on how far a correct kernel can be from them, for the GPU tests.

u is half a step of a type relative to a value (bf16 2^-8, fp16 2^-11), F that of
float (2^-24). A bound counts the roundings that the operators document and a
generous count of float roundings for sums and elementary functions."""
from __future__ import annotations

import torch

F = 2.0 ** -24


def u(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tiny(dtype) -> float:
    """Half a step among the type's subnormal numbers."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def attention(q, k, v, q_lengths, k_lengths, causal, scale=None):
    """(o, bound), float64 [q rows, heads, dim], on the CPU. A hidden key takes no part at all."""
    dtype, dim, group = q.dtype, q.shape[2], q.shape[1] // k.shape[1]
    scale = dim ** -0.5 if scale is None else scale
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    o, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    q0 = k0 = 0
    for n, m in zip(q_lengths, k_lengths):
        i, j = torch.arange(n)[:, None], torch.arange(m)
        seen = j <= i + (m - n) if causal else torch.ones(n, m, dtype=torch.bool)
        for h in range(q.shape[1] if n and m else 0):
            qh, kh, vh = q[q0:q0 + n, h], k[k0:k0 + m, h // group], v[k0:k0 + m, h // group]
            s = torch.where(seen, scale * (qh @ kh.T), -torch.inf)
            rows = seen.any(1)
            p = torch.zeros(n, m, dtype=torch.float64)
            e = torch.exp(s[rows] - s[rows].max(1, keepdim=True).values)
            p[rows] = e / e.sum(1, keepdim=True)
            # 0 times anything is 0 for a key that is not seen
            finite = vh.isfinite().all(1)
            part = p[:, finite] @ vh[finite]
            for key in torch.nonzero(~finite).flatten().tolist():
                part = torch.where(seen[:, key:key + 1], part + p[:, key:key + 1] * vh[key], part)
            o[q0:q0 + n, h] = part
            # probabilities rounded to the type; scores off by the float roundings of
            # a product of `dim` terms, times two for numerator and denominator; the
            # exponential, the sums over the keys; the result's rounding
            size = (p[:, finite] @ vh[finite].abs())
            score = scale * (qh.abs() @ kh.abs().T)
            score = torch.where(seen & score.isfinite(), score, 0).amax(1, keepdim=True)
            slack = u(dtype) + 2 * (dim + 8) * F * score + 2.0 ** -18 + 4 * m * F
            bound[q0:q0 + n, h] = size * slack + u(dtype) * part.abs() + tiny(dtype)
            if dtype == torch.float16:  # small probabilities are subnormal: half a step of 2^-24 each; the sum is at least 1
                bound[q0:q0 + n, h] += 2.0 ** -25 * (seen[:, finite].double() @ vh[finite].abs())
        q0, k0 = q0 + n, k0 + m
    return o, bound


def activation(t, name):
    if name == "relu":
        return t.clamp_min(0)
    if name == "silu":
        return t / (1 + torch.exp(-t))
    if name == "gelu":
        return t * torch.special.erfc(-t * 0.5 ** 0.5) / 2
    if name == "gelu_tanh":
        return t / (1 + torch.exp(-2 * (2 / torch.pi) ** 0.5 * (t + 0.044715 * t ** 3)))
    return t


def linear(X, W, bias, name, residual):
    """(Y, bound) on the CPU. Every activation's slope is under 1.2 in size."""
    dtype, K = X.dtype, X.shape[1]
    X, W = X.detach().cpu().double(), W.detach().cpu().double()
    t, size = X @ W, X.abs() @ W.abs()
    if bias is not None:
        t, size = t + bias.cpu().double(), size + bias.cpu().double().abs()
    y = activation(t, name)
    # a float sum of K terms, one step each; a few roundings and the elementary functions of the activation
    bound = 1.2 * 2 * (K + 4) * F * size + 2.0 ** -18 * (y.abs() + (name is not None) * 2.0 ** -3)
    if residual is not None:
        y = y + residual.cpu().double()
        bound = bound + 2 * F * residual.cpu().double().abs()
    return y, bound * (1 + u(dtype)) + u(dtype) * y.abs() + tiny(dtype)


def residual_norm(x, y, sequence, gate=None, residual_scale=1.0, post_norm=None, post_weight=None, post_bias=None,
                  norm="rms", weight=None, bias=None, scale=None, shift=None, eps=1e-6):
    """((x', bound), (h, bound)) on the CPU; `sequence` is each row's sequence."""
    x_dtype, kind = x.dtype, y.dtype if y is not None else None
    wide = lambda t: None if t is None else t.detach().cpu().double()
    x, y, gate, post_weight, post_bias, weight, bias, scale, shift = map(
        wide, (x, y, gate, post_weight, post_bias, weight, bias, scale, shift))
    slack = 2.0 ** -18  # 64 float roundings: a sum in the order of a tree, square root, division, products

    def apply(t, t_err, which, w, b):
        """The norm of t, which is off by t_err, and how far it can be off."""
        if which is None:
            n, err = t, t_err
        else:
            c = t - t.mean(1, keepdim=True) if which == "layer" else t
            c_err = t_err + slack * (t.abs() + t.abs().mean(1, keepdim=True)) + t_err.mean(1, keepdim=True)
            r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
            n = c * r
            # the deviation's relative error is at most the values' (weighted by n) and the sums'
            err = r * c_err + n.abs() * (slack + r * c_err.pow(2).mean(1, keepdim=True).sqrt())
        if w is not None:
            n, err = n * w, err * w.abs()
        if b is not None:
            n, err = n + b, err + slack * b.abs()
        return n, err + slack * n.abs()

    x_err = torch.zeros_like(x)
    if y is not None:
        n, err = apply(y, torch.zeros_like(y), post_norm, post_weight, post_bias)
        if gate is not None:
            n, err = n * gate[sequence], err * gate[sequence].abs()
        x_err = err + slack * (n.abs() + (residual_scale * x).abs())
        x = residual_scale * x + n
    out_x = x, x_err + u(x_dtype) * (x.abs() + x_err) + tiny(x_dtype)
    if norm is None:
        return out_x, None
    h, err = apply(x, x_err, norm, weight, bias)
    if scale is not None:
        h, err = h * (1 + scale[sequence]), err * (1 + scale[sequence]).abs()
    if shift is not None:
        h, err = h + shift[sequence], err + slack * shift[sequence].abs()
    err = err + slack * h.abs()
    kind = kind or (x_dtype if x_dtype != torch.float32 else torch.bfloat16)
    return out_x, (h, err + u(kind) * (h.abs() + err) + tiny(kind))


def check(got, want, bound, what=""):
    """got within bound of want; the same infinities, NaN where want has them."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    odd = ~want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()), what
    assert torch.equal(got[odd & ~want.isnan()], want[odd & ~want.isnan()]), what
    off = torch.where(odd, 0, (got - want).abs() - bound)
    worst = off.argmax()
    assert off.max() <= 0, (f"{what}: {int((off > 0).sum())} of {off.numel()} values outside; at {worst.item()}: "
                            f"{got.flatten()[worst].item()} for {want.flatten()[worst].item()} +- {bound.flatten()[worst].item()}")
