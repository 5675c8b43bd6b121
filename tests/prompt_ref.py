"""Plain 64-bit forms of the prompt operators (rotary positions, norm, attention in the expanded form), with the error bounds the
GPU tests hold the kernels to."""
from __future__ import annotations

import math

import torch

STEP = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}       # spacing of subnormal numbers


def frequencies(dim, scaling="none", base=10000.0, factor=8.0, original=4096.0, fast=32.0, slow=1.0):
    """Radians a position of each pair, pair by pair."""
    out = []
    for j in range(dim // 2):
        f = base ** (-2 * j / dim)
        if scaling == "linear":
            f /= factor
        if scaling == "ntk" and dim > 2:
            f = (base * factor ** (dim / (dim - 2))) ** (-2 * j / dim)
        if scaling == "yarn":
            at = [dim * math.log(original / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast, slow)]
            low, high = max(0, math.floor(at[0])), min(dim - 1, math.ceil(at[1]))
            high = high if high > low else low + 0.001
            g = min(1.0, max(0.0, (j - low) / (high - low)))
            f = f * (1 - g) + f / factor * g
        out.append(f)
    return out


def rotate(x, position, f, layout, amplitude=1.0):
    """x [N, ..., dim] fp64 turned; and sum |a| + |b| of the pairs, laid out like x."""
    f = torch.tensor(f, dtype=torch.float64, device=x.device)
    w = position.double()[:, None] * f
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (-1,)
    c, s = torch.cos(w).view(shape), torch.sin(w).view(shape)
    half = x.shape[-1] // 2
    a, b = (x[..., :half], x[..., half:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    y, z, m = amplitude * (a * c - b * s), amplitude * (a * s + b * c), abs(amplitude) * (a.abs() + b.abs())
    if layout == "half":
        return torch.cat([y, z], -1), torch.cat([m, m], -1)
    return torch.stack([y, z], -1).flatten(-2), torch.stack([m, m], -1).flatten(-2)


def rotate_bound(out, size, dtype):
    """The angle is off by 2^-24 of itself (at most pi) where it is converted, sine and cosine by 2 ulp (2^-23), each of the two
    products and the amplitude by 2^-24: (pi + 2 + 3) 2^-24 < 2^-20.6 of |a| + |b|; then the rounding to the type."""
    return size * 2.0 ** -20.6 + out.abs() * torch.finfo(dtype).eps / 2 * 1.001 + STEP[dtype] / 2


def norm(x, gain, eps):
    return x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * gain


def norm_bound(out, dtype):
    """A sum of 512 positive terms in fp32 is off by at most 512 * 2^-24 of itself, its root by half of that; root, reciprocal, mean,
    eps and two products add 6 roundings of 2^-24 (root and reciprocal up to 2^-23); then the rounding to the type."""
    return out.abs() * ((256 + 10) * 2.0 ** -24 + torch.finfo(dtype).eps / 2) * 1.001 + STEP[dtype] / 2


def attention(q, k, r, v, new, seq, scale, dtype, weights="same"):
    """out [N][H][128], lse [N][H] and the bounds of both; q [N][H][192], k, v [M][H][128], r [M][64] in fp64.

    With p the weights and A = sum p |v|:
    * a score is a sum of 192 exact products in fp32 (each addition off by at most 2^-23 of the running magnitude, as the tensor
      cores may truncate) and one product with the scale, itself rounded: ds = 196 * 2^-23 * scale * sum |q k|;
    * a weight is exp2 of it (relative 2^-21: 2 ulp, and the argument's own rounding 2^-23 * (|s| log2 e + 16)) and is rounded to the
      type (eps / 2; below the type's normal range half of its spacing there, relative to the largest weight, which is at least 1/2);
    * the same errors without the rounding, and those of summing n weights (2^-23 n), are in the denominator;
    * the products with v sum in fp32 (2^-23 n), and the result is rounded (eps / 2).
    """
    N, H = q.shape[:2]
    eps, tiny = torch.finfo(dtype).eps, STEP[dtype]
    out, lse = torch.zeros((N, H, 128), dtype=torch.float64, device=q.device), torch.full((N, H), -math.inf, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    n0 = m0 = 0
    for t, length in zip(new, seq):
        for h in range(H):
            key = torch.cat([k[m0:m0 + length, h], r[m0:m0 + length]], 1)
            val = v[m0:m0 + length, h]
            for i0 in range(0, t, 512):
                i1 = min(t, i0 + 512)
                ends = torch.arange(length - t + i0 + 1, length - t + i1 + 1, device=q.device)
                rows = (ends > 0).nonzero()[:, 0]
                if not len(rows) or not length:
                    continue
                ends = ends[rows]
                at = n0 + i0 + rows
                hi = int(ends.max())
                seen = torch.arange(hi, device=q.device)[None] < ends[:, None]
                # (values that a row does not see stay out of its sums, whatever they are)
                kk, vv = torch.nan_to_num(key[:hi], 0.0, 0.0, 0.0), torch.nan_to_num(val[:hi], 0.0, 0.0, 0.0)
                s = q[at, h] @ kk.T * scale
                s = torch.where(seen, s, -math.inf)
                ds = 196 * 2.0 ** -23 * abs(scale) * torch.where(seen, q[at, h].abs() @ kk.abs().T, 0.0).amax(1)
                m = s.amax(1, keepdim=True)
                e = torch.exp(s - m)
                l = e.sum(1, keepdim=True)
                p = e / l
                o, A = p @ vv, p @ vv.abs()
                big = torch.where(seen, s.abs(), 0.0).amax(1)
                exp_err = 2 * ds + 2.0 ** -21 + 2.0 ** -22 * (1.5 * big + 16)
                count = 2.0 ** -23 * (ends + 64)
                rel = 2 * exp_err + eps / 2 + 2 * count
                out[at, h], lse[at, h] = o, (m + torch.log(l))[:, 0]
                tol[at, h] = rel[:, None] * A * 1.05 + eps / 2 * o.abs() * 1.05 + tiny * (seen.double() @ vv.abs()) + tiny
                tol_lse[at, h] = exp_err + count + 2.0 ** -22 * lse[at, h].abs() + 2.0 ** -22
        n0, m0 = n0 + t, m0 + length
    return out, lse, tol, tol_lse
