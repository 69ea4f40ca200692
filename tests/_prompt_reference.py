"""64-bit definitions of kvq_norm_rope and kvq_prompt_attention, and the bounds
that their results are held to."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}             # half a step of the smallest numbers


def norm_rope(x, weight, eps, pos, inv_freq, pair_axis, interleaved):
    """x [rows, H, D]; pos [axes, rows].  Returns the exact result and the size |n_a| + |n_b| of each channel's terms."""
    x = x.double().cpu()
    rows, _, D = x.shape
    if eps is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            x = x * weight.double().cpu()
    y, size = x.clone(), x.abs().clone()
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        phi = pos[pair_axis[i] if pair_axis else 0].double().cpu() * float(inv_freq[i])
        c, s = phi.cos()[:, None], phi.sin()[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def norm_rope_bound(y, size, dtype):
    """The result's rounding, and the kernel's binary32 steps: the sum of squares (19 additions and products in a row, halved by
    the root), the root (3), the scaling (2), sine and cosine (2 for the function, 1/2 for the angle) and the rotation (2),
    each 2^-24 of the terms: 19, taken as 24."""
    return U[dtype] * y.abs() + (1 + U[dtype]) * 24 * 2.0 ** -24 * size + TINY[dtype]


def prompt(q, k, v, scale, causal):
    """One sequence: q [n, Hq, D], k and v [n, Hkv, D] -> out, lse and (the size sum_j p_j |v_j|, the scores' bound) in 64 bits."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros((n, Hq, D), dtype=torch.float64, device=q.device)
    size = torch.zeros_like(out)
    lse = torch.zeros((n, Hq), dtype=torch.float64, device=q.device)
    reach = torch.zeros_like(lse)
    for h in range(Hq):
        qh, kh, vh = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        a = qh @ kh.T * scale
        seen = torch.ones((n, n), dtype=torch.bool, device=q.device)
        if causal:
            seen = seen.tril()
        a = a.masked_fill(~seen, -math.inf)
        lse[:, h] = a.logsumexp(-1)
        p = (a - lse[:, h, None]).exp()
        out[:, h] = p @ vh
        size[:, h] = p @ vh.abs()
        reach[:, h] = (qh.abs() @ kh.abs().T * abs(scale)).masked_fill(~seen, 0.0).amax(-1)
    return out, lse, size, reach


def prompt_bounds(out, lse, size, reach, top, n, D, dtype, out_dtype):
    """A weight is rounded to `dtype` (in fp16 with 2^6 of headroom below its smallest step: 2^-31 absolute a key, `top` the
    largest |v|).  A score is a sum of D fp32 products, whose additions may cut instead of round (2^-23 each), and takes one
    rounding more with the maximum and one in the exponential (2^-22): 2^-23 (D + 2) of sum |q k| scale + 2^-21.  The sums of
    n weights and of n products: 2^-23 n."""
    score = 2.0 ** -23 * (D + 2) * reach + 2.0 ** -21
    e = (U[dtype] + 2 * score + 2.0 ** -23 * n)[..., None] * size
    if dtype is torch.float16:
        e = e + n * 2.0 ** -31 * top
    return e + U[out_dtype] * (out.abs() + e) + TINY[out_dtype], score + 2.0 ** -23 * (n + lse.abs())
