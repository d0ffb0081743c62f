"""64-bit form of the rotary operators and the error bound their outputs are held to."""
from __future__ import annotations

import torch

EPS_F32 = 2.0 ** -24  # half a step, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS_F32}


def rope(x, inv_freq, positions, axes=None, norm_w=None, eps=1e-6, mscale=1.0, interleaved=False):
    """(out, bound) of x [T, H, D]: the output in 64 bits, and what f32 arithmetic may be
    off by before the output is rounded.

    Angles: the argument of the cosine is rounded to f32 in half turns below 1 (2^-25 pi)
    and the functions are good to 2 steps (2^-23): 2^-22 together, times |a| + |b|.  Two
    products, a sum and mscale round another 4 times: (|a| + |b|) 2^-22.  The norm: D
    squares added up in runs of at most 32 and then over 32 lanes (at most 40 roundings, of which a root
    keeps half), then five more: 25 2^-24 relative.  In all at most 2^-19 (|a| + |b|) mscale."""
    x = x.double()
    T, H, D = x.shape
    half = inv_freq.numel()
    if norm_w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * norm_w.double()
    pos = positions.view(1, -1) if positions.dim() == 1 else positions
    out, bound = x.clone(), x.abs() * (2.0 ** -19 if norm_w is not None else 0.0)
    for j in range(half):
        i, k = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        ax = 0 if axes is None else int(axes[j])
        p = pos[ax] if 0 <= ax < pos.shape[0] else torch.zeros_like(pos[0])
        g = p.double() * inv_freq[j].double()
        c, s = torch.cos(g).view(T, 1), torch.sin(g).view(T, 1)
        a, b = x[:, :, i], x[:, :, k]
        out[:, :, i] = mscale * (a * c - b * s)
        out[:, :, k] = mscale * (b * c + a * s)
        far = (p.double().abs() * inv_freq[j].double().abs() * 2.0 ** -50).view(T, 1)
        bound[:, :, i] = bound[:, :, k] = (a.abs() + b.abs()) * abs(mscale) * (2.0 ** -19 + far)
    return out, bound


def check_rope(y, ref, dtype):
    out, bound = ref
    err = (y.double() - out).abs()
    tol = HALF_STEP[dtype] * out.abs() + bound * (1 + HALF_STEP[dtype])
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -134  # half the smallest subnormal step
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} outputs off, by up to {(err / tol.clamp(min=1e-300)).max().item():.2f} bounds"
