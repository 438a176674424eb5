"""64-bit forms of the 8-bit cache, of attention with sinks and of drawing tokens, and how far the
kernels may be from them.  Tolerances count roundings, as in tests/target_ref.py."""
import math

import torch

from tests.target_ref import U32, half_step

BLOCK, TOP = 16, 448.0


def power(e):
    """2^e in float64, exactly (pow and ldexp of the GPU may be off by a last bit)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def least_scale(amax):
    """The least power of two s with amax <= 448 s (1 for 0): float64 in and out."""
    m, e = torch.frexp(amax / TOP)
    s = power(torch.where(m == 0.5, e - 1, e)).clamp(min=2.0 ** -126)
    return torch.where(amax > 0, s, torch.ones_like(s))


def round8(x):
    """float64 to the nearest e4m3 value, ties to even (4 significant bits, steps of 2^-9 below 2^-6)."""
    _, e = torch.frexp(torch.where(torch.isfinite(x), x, torch.zeros_like(x)))
    step = power((e - 4).clamp(min=-9))
    return torch.where(torch.isfinite(x), torch.round(x / step) * step, torch.full_like(x, math.nan))


def quantise(x):
    """[..., 16, dim] float64 -> values of codes, scale [...]"""
    a = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax((-1, -2))
    s = least_scale(a)
    return round8(x / s[..., None, None]), s


def rotate_exact(x, table, rot, interleaved):
    """x [n, heads, dim], table [n, 2, rot / 2] of these positions: float64, the table's entries as they are."""
    x, c, s = x.double().clone(), table[:, 0].double()[:, None], table[:, 1].double()[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2].clone(), x[..., 1:rot:2].clone()
        x[..., 0:rot:2], x[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2].clone(), x[..., rot // 2:rot].clone()
        x[..., :rot // 2], x[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return x


def visible(past, n, window, sinks, device):
    i = past + torch.arange(n, device=device)[:, None]
    j = torch.arange(past + n, device=device)[None]
    ok = j <= i
    if window:
        ok = ok & ((j > i - window) | (j < sinks))
    return ok


def attention(q, k, v, past, scale, window, sinks, eight=False, ratios=False):
    """q [n, Hq, D]; k, v [Hkv, past + n, D] float64 values.  Returns float64 [n, Hq, D] and its tolerance.

    As in target_ref.attention, with h half a step of what the weights are rounded to (8-bit cache: fp16), and of the
    scores' error two roundings more for the scales.  fp16 weights are kept 2^7 times as large and at most 2^8 above the
    row's reference, so that the largest is at least 2^7 and one below 2^-14 is off by up to 2^-25: 2^-32 of the
    largest's; with an 8-bit cache the weights are relative to the largest scale of a value, so this is of the largest
    value that can be.  ratios: values' scales are not powers of two, so that above 32 rows a cache head their quotients by
    the largest, and the values times these, are rounded to fp16: two half steps more."""
    n, Hq, D = q.shape
    Hkv, L = k.shape[0], k.shape[1]
    grp = Hq // Hkv
    dtype = q.dtype
    ok = visible(past, n, window, sinks, q.device)
    seen = ok.any(0)[None, :, None]
    k = torch.where(seen, k, torch.zeros_like(k)).repeat_interleave(grp, 0)
    v = torch.where(seen, v, torch.zeros_like(v)).repeat_interleave(grp, 0)
    q = q.double().transpose(0, 1)
    s = q @ k.transpose(1, 2) * scale
    s_abs = q.abs() @ k.abs().transpose(1, 2) * abs(scale)
    p = torch.softmax(s.masked_fill(~ok, -math.inf), -1)
    o = p @ v
    size = p @ v.abs()
    delta = s_abs.masked_fill(~ok, 0.0).amax(-1, keepdim=True) * (2 * D + (8 if eight else 4)) * U32
    h = half_step(torch.float16 if eight else dtype)
    tol = size * (h * (1 + eight * 2.0 ** -8 + 2 * ratios) + 2 * delta + 4 * (L + 64) * U32) + half_step(dtype) * o.abs() + 1e-30
    if dtype == torch.float16:  # the result's own absolute step
        tol = tol + 2.0 ** -25
    if eight or dtype == torch.float16:
        big = v.abs().amax((1, 2), keepdim=True) * (2 if eight else 1)  # (a scale's largest value: below twice the block's)
        tol = tol + 2.0 ** -31 * L * big
    return o.transpose(0, 1), tol.transpose(0, 1)


def sample(z, u, T, K, P, M):
    """One row: logits z [V] (float64), the settings as Python floats of the float32 that the call gets.
    Returns token, probability and how close the draw is to a border (relative to the mass)."""
    V = z.numel()
    if T == 0:
        return int((z == z.max()).nonzero()[0, 0]), 1.0, 1.0
    w = torch.exp((z - z.max()) / T)
    order = torch.argsort(-z, stable=True)
    order = order[torch.isfinite(z[order])]
    if 0 < K < V:
        order = order[:K]
    if P < 1.0:
        c = torch.cumsum(w[order], 0)
        order = order[:int(((c - w[order]) < P * c[-1]).sum())]
    order = order[w[order] >= M]
    ids = torch.sort(order)[0]
    c = torch.cumsum(w[ids], 0)
    v = u * float(c[-1])
    at = int((c <= v).sum())
    near = float((c - v).abs().min() / c[-1])
    return int(ids[at]), float(w[ids[at]] / c[-1]), near
