"""64-bit forms of the target-step operators, and how far the kernels may be from them.

Tolerances count roundings: a rounding to type t is off by at most eps(t) / 2 of the value.
"""
import math

import torch

U32 = 2.0 ** -24  # half a step of float32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def bits_of(words, V):
    """[..., W] int32 bit planes -> bool [..., V]"""
    t = torch.arange(V, device=words.device)
    return ((words[..., t >> 5] >> (t & 31).to(torch.int32)) & 1).bool()


def planes_of(flags):
    """bool [..., V] -> int32 bit planes [..., ceil(V / 32)]"""
    V = flags.shape[-1]
    W = (V + 31) // 32
    pad = torch.zeros(flags.shape[:-1] + (W * 32,), dtype=torch.int64, device=flags.device)
    pad[..., :V] = flags.long()
    w = (pad.reshape(flags.shape[:-1] + (W, 32)) << torch.arange(32, device=flags.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def process_logits(logits, prompt, output, draft, rep, freq, pres, bias, mask):
    """prompt, output: per-sequence id lists; draft [B, G] list; bias: per-sequence (id, value) lists;
    mask: bool [B, N, V] or None.  Returns the values in float64 and their tolerance before the last rounding."""
    B, N, V = logits.shape
    res = torch.empty((B, N, V), dtype=torch.float64)
    tol = torch.empty((B, N, V), dtype=torch.float64)
    x = logits.detach().cpu().double()
    for b in range(B):
        for i in range(N):
            cnt = torch.zeros(V, dtype=torch.float64)
            made = list(output[b]) + [t for t in (draft[b][:i] if draft is not None else [])]
            for t in made:
                if 0 <= t < V:
                    cnt[t] += 1
            seen = cnt > 0
            for t in prompt[b]:
                if 0 <= t < V:
                    seen[t] = True
            z = x[b, i].clone()
            z = torch.where(seen, torch.where(z > 0, z / rep[b], z * rep[b]), z)
            size = z.abs() + abs(freq[b]) * cnt + abs(pres[b])
            z = z - freq[b] * cnt - pres[b] * (cnt > 0)
            for t, v in bias[b]:
                if 0 <= t < V:
                    z[t] += v
                    size[t] += abs(v)
            # each partial result is rounded to float32 once: repetition, product, two differences, the biases'
            # sum (one addition an entry) and its addition
            tol[b, i] = (6 + len(bias[b])) * U32 * size
            if mask is not None:
                z[~mask[b, i].cpu()] = -math.inf
            res[b, i] = z
    return res, tol


def rotate(x, pos, freq, mscale, rot, interleaved):
    """x [n, heads, dim], pos [n], freq [rot / 2] float64.  Returns values and tolerance before the last rounding."""
    x = x.double()
    ang = pos.double()[:, None] * freq
    c, s = (ang.cos() * mscale)[:, None], (ang.sin() * mscale)[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    ra, rb = a * c - b * s, b * c + a * s
    # cosine and sine rounded to float32, two products and a sum: 3 roundings of each term; the angle itself is
    # formed in float64 from a float64 frequency (error far below)
    t = 3 * U32 * mscale * (a.abs() + b.abs()) + 1e-30
    y, tol = x.clone(), torch.zeros_like(x)
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
        tol[..., 0:rot:2] = tol[..., 1:rot:2] = t
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
        tol[..., :rot // 2] = tol[..., rot // 2:rot] = t
    return y, tol


def gather(pages, table_row, L, page_size):
    """[heads, L, dim] of a sequence's first L positions."""
    j = torch.arange(L, device=pages.device)
    return pages[table_row.long()[j // page_size], :, j % page_size].transpose(0, 1)


def attention(q, k, v, past, scale, window, dtype):
    """q [n, Hq, D]; k, v [Hkv, L, D] with L = past + n.  Returns float64 [n, Hq, D] and its tolerance.

    With p the weights and h half a step of the 16-bit type: the weights are rounded to it (h), a score is off by
    delta (its dot product's D float32 additions, each off by at most 2 half steps where the matrix unit cuts, and
    its scaling), which changes a weight by a factor within 1 + 2 delta; the L additions of a sum are off by 2 half
    steps of float32 each; the result is rounded once (h)."""
    n, Hq, D = q.shape
    Hkv, L = k.shape[0], k.shape[1]
    grp = Hq // Hkv
    k, v = k.double().repeat_interleave(grp, 0), v.double().repeat_interleave(grp, 0)
    q = q.double().transpose(0, 1)
    s = q @ k.transpose(1, 2) * scale
    s_abs = q.abs() @ k.abs().transpose(1, 2) * abs(scale)
    i = past + torch.arange(n, device=q.device)[:, None]
    j = torch.arange(L, device=q.device)[None]
    ok = j <= i
    if window:
        ok = ok & (j > i - window)
    p = torch.softmax(s.masked_fill(~ok, -math.inf), -1)
    v = torch.where(ok.any(0)[None, :, None], v, torch.zeros_like(v))
    o = p @ v
    size = p @ v.abs()
    delta = (s_abs.masked_fill(~ok, 0.0).amax(-1, keepdim=True)) * (2 * D + 4) * U32
    h = half_step(dtype)
    tol = size * (h + 2 * delta + 4 * (L + 64) * U32) + h * o.abs() + 1e-30
    if dtype == torch.float16:  # below the smallest normal weight a step is absolute
        tol = tol + 2.0 ** -24 * (v.abs().amax(1, keepdim=True) * L)
    return o.transpose(0, 1), tol.transpose(0, 1)
