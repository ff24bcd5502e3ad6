"""Plain 64-bit forms of the block operators (rotary positions, norms, 8-bit products) and the
rounding units their tests count in. Torch float64 on whatever device the inputs are on; no code
shared with the library."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24          # half a step of fp32, relative


def half_step(dtype: torch.dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tiny_step(dtype: torch.dtype) -> float:
    """Half the spacing of the type's smallest numbers (what a rounding near zero can be off by)."""
    fi = torch.finfo(dtype)
    return fi.smallest_normal * fi.eps / 2


def worst(got: torch.Tensor, ref: torch.Tensor, arith: torch.Tensor, dtype: torch.dtype) -> float:
    """Largest |got - ref| in units of its bound: one rounding to `dtype` plus the arithmetic bound."""
    bound = half_step(dtype) * (ref.abs() + arith) + arith + tiny_step(dtype)
    d = (got.double() - ref).abs() / bound
    return float(d.max()) if d.numel() else 0.0


def rotate(x, cs, rot, interleaved, inverse=False):
    """x [..., D] float64, cs [..., P, 2] float64 -> turned x, and |x1| + |x2| per channel."""
    P = rot // 2
    i = torch.arange(P, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
    c, s = cs[..., 0], cs[..., 1]
    s = -s if inverse else s
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    m = (x[..., a].abs() + x[..., b].abs()) * (c.abs() + s.abs())
    mag[..., a], mag[..., b] = m, m
    return y, mag


def stats(x, kind, eps):
    """mean, rstd [..., 1] of float64 rows."""
    zero = torch.zeros_like(x[..., :1])
    if kind == "none":
        return zero, zero + 1
    mean = x.mean(-1, keepdim=True) if kind == "layer" else zero
    return mean, 1 / ((x - mean).square().mean(-1, keepdim=True) + eps).sqrt()


def quantize(x):
    """int8 codes and fp32 scales of the rows of x, from the definition."""
    a = x.double().abs().amax(1) if x.shape[1] else x.new_zeros(x.shape[0]).double()
    bad = ~torch.isfinite(x.double()).all(1)
    scale = (a / 127).float()
    small = a < 2.0 ** -100
    scale[small] = 1.0
    q = (x.double() / scale.double()[:, None]).round()
    q[small | bad] = 0
    scale[bad] = float("nan")
    return q.to(torch.int8), scale
