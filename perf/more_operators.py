"""What is measured of the operators of the drafter's side and of small caches: drawing tokens, the
8-bit paged cache (append and attention), attention with a window and sinks.

``sample`` draws a token of each row from given random numbers, after temperature, top-k,
top-p and min-p.  ``rotate_append`` fills a cache of 8-bit codes with a scale for each 16
tokens and head, ``paged_attention`` reads it, and with ``sinks`` a sliding window keeps the
first tokens in sight.  Each case below is one step of one of them; ``run`` computes it in
elementary torch operations, or with the framework's kernels where ``own`` is set.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BLOCK = 16  # tokens that share a scale
_TOP = 448.0  # the largest e4m3 value


def _sv():
    import speculative_decoding_verification_20_gb300 as sv

    return sv


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one drafted token for each of a few sequences
        dict(name="sample_b4_n1_v32k", op="sample", B=4, N=1, V=32000, dtype="bf16", top_k=50, top_p=True, min_p=False),
        # a drafter's step, or plain decoding, of 256 sequences with settings of their own
        dict(name="sample_b256_n1_v128k", op="sample", B=256, N=1, V=128256, dtype="bf16", top_k=200, top_p=True,
             min_p=True),
        # every position of a round, fp32 logits, no top-k: nuclei of any size
        dict(name="sample_b24_n8_v152k", op="sample", B=24, N=8, V=151936, dtype="f32", top_k=0, top_p=True, min_p=True),
        # one token of a few sequences into the 8-bit cache
        dict(name="append8_b4_n1", op="append8", B=4, N=1, Hq=32, Hkv=8, D=128, rot=128, inter=False, dtype="bf16",
             page=16, past_lo=50, past_hi=4000, ragged=False),
        # a round of 256 sequences, gamma 7, ragged
        dict(name="append8_b256_n8", op="append8", B=256, N=8, Hq=32, Hkv=8, D=128, rot=128, inter=False, dtype="bf16",
             page=32, past_lo=0, past_hi=1000, ragged=True),
        # a chunk of two prompts, interleaved pairs on half of the head
        dict(name="append8_b2_n4096", op="append8", B=2, N=4096, Hq=32, Hkv=8, D=128, rot=64, inter=True, dtype="f16",
             page=64, past_lo=0, past_hi=20000, ragged=True),
        # plain decoding of one short sequence over the 8-bit cache: latency
        dict(name="attn8_b1_n1", op="attn8", B=1, N=1, Hq=32, Hkv=8, D=128, dtype="bf16", page=16, past_lo=700,
             past_hi=700, ragged=False, window=0, sinks=0),
        # a round of 64 sequences, gamma 7, mixed lengths
        dict(name="attn8_b64_n8", op="attn8", B=64, N=8, Hq=32, Hkv=8, D=128, dtype="bf16", page=16, past_lo=1500,
             past_hi=8200, ragged=True, window=0, sinks=0),
        # a round of two very long sequences, gamma 5: more rows a cache head
        dict(name="attn8_b2_n6_long", op="attn8", B=2, N=6, Hq=32, Hkv=4, D=128, dtype="bf16", page=64, past_lo=90001,
             past_hi=131000, ragged=False, window=0, sinks=0),
        # a chunk of two prompts behind earlier chunks
        dict(name="attn8_b2_n2048", op="attn8", B=2, N=2048, Hq=32, Hkv=8, D=128, dtype="f16", page=64, past_lo=4000,
             past_hi=6144, ragged=False, window=0, sinks=0),
        # a round over long texts through a window, the first tokens in sight
        dict(name="sinks_b48_n5", op="sinks", B=48, N=5, Hq=32, Hkv=8, D=128, dtype="bf16", page=32, past_lo=300,
             past_hi=16000, ragged=True, window=2048, sinks=4),
        # chunks of odd lengths, small heads in groups of five, sinks that end inside a page
        dict(name="sinks_b3_n777", op="sinks", B=3, N=777, Hq=20, Hkv=4, D=64, dtype="f16", page=48, past_lo=100,
             past_hi=6000, ragged=True, window=1500, sinks=70),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "append8", "attn8", "sinks"])
    ref = [work(c) for c in listed() if c["op"] == op]
    cap_b, cap_f = max(w["bytes"] for w in ref), max(w["flops"] for w in ref)
    while True:
        if op == "sample":
            case = dict(op=op, B=_logu(rng, 1, 256), N=rng.randint(1, 9), V=_logu(rng, 1000, 152000),
                        dtype=rng.choice(["bf16", "f32"]), top_k=rng.choice([0, 0, 1, 20, 50, 200, 2000]),
                        top_p=rng.random() < 0.5, min_p=rng.random() < 0.5)
        else:
            Hkv = rng.choice([1, 2, 4, 8])
            D = rng.choice([64, 128])
            N = rng.choice([1, rng.randint(2, 9), rng.randint(2, 9), _logu(rng, 10, 2100)])
            case = dict(op=op, B=_logu(rng, 1, 128), N=N, Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=D,
                        dtype=rng.choice(["bf16", "f16"]), page=rng.choice([16, 32, 48, 64, 128, 256]))
            lo = _logu(rng, 1, 20000)
            case.update(past_lo=lo - 1, past_hi=lo - 1 + _logu(rng, 1, 20000), ragged=rng.random() < 0.5)
            if op == "append8":
                case.update(rot=rng.choice([D, D // 2, D // 4]), inter=rng.random() < 0.5)
            elif op == "attn8":
                case.update(window=rng.choice([0, 0, _logu(rng, 1, 5000)]))
                case.update(sinks=rng.choice([0, _logu(rng, 1, 300)]) if case["window"] else 0)
            else:
                case.update(window=_logu(rng, 1, 5000), sinks=_logu(rng, 1, 300))
        w = work(case)
        if op in ("attn8", "sinks"):  # the whole cache is part of the state: 4 GB of it at most
            past, new = _spread(case)
            if 4 * (sum(past) + sum(new)) * case["Hkv"] * case["D"] > 4e9:
                continue
        if w["bytes"] <= cap_b and w["flops"] <= cap_f:
            return case


def _spread(case):
    """past[b], new[b]: lengths spread evenly over the case's range, in mixed order."""
    B, N = case["B"], case["N"]
    past, new = [], []
    for b in range(B):
        x = ((b + 1) * 0.6180339887498949) % 1.0 if B > 1 else 1.0
        y = ((b + 1) * 0.7548776662466927) % 1.0
        past.append(case["past_lo"] + int(x * (case["past_hi"] - case["past_lo"])))
        new.append(1 + int(y * N) if case["ragged"] else N)
    if case["ragged"]:
        new[0] = N
    return past, new


def _visible(past, n, window, sinks):
    """Visible keys summed over the n new tokens, and the number of distinct keys."""
    if not window:
        return n * past + n * (n + 1) // 2, past + n
    pairs = 0
    for i in range(n):
        own_window = min(past + i + 1, window)
        pairs += own_window + min(sinks, past + i + 1 - own_window)
    lo = max(0, past + 1 - window)
    return pairs, past + n - lo + min(sinks, lo)


def work(case):
    if case["op"] == "sample":
        B, N, V = case["B"], case["N"], case["V"]
        return {"bytes": B * N * V * (2 if case["dtype"] == "bf16" else 4) + 12 * B * N + 16 * B, "flops": 4 * B * N * V}
    past, new = _spread(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    T = sum(new)
    if case["op"] == "append8":
        held = sum(p % _BLOCK for p in past)  # tokens already in a block that gets more
        back = held + T  # tokens of the changed blocks: written as codes and read back as values
        n = 2 * 2 * T * Hq * D + 2 * 2 * T * Hkv * D + 4 * T * case["rot"]
        n += 2 * held * Hkv * D + 2 * back * Hkv * D + 2 * 2 * back * Hkv * D + 2 * 4 * Hkv * (back // _BLOCK + 1)
        return {"bytes": n, "flops": 3 * T * (Hq + Hkv) * case["rot"] + 4 * back * Hkv * D}
    pairs = keys = 0
    for p, n in zip(past, new):
        a, k = _visible(p, n, case["window"], case["sinks"])
        pairs, keys = pairs + a, keys + k
    per_key = D + 4 / _BLOCK if case["op"] == "attn8" else 2 * D
    return {"bytes": int(2 * keys * Hkv * per_key) + 2 * 2 * T * Hq * D, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _sample_inputs(case, seed):
    B, N, V = case["B"], case["N"], case["V"]
    g = _gen(seed)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")
    # logits fall with the logarithm of a token's rank, steeply where the text is predictable
    steep = 1.1 + 1.6 * rand(B, N, 1)
    z = torch.empty((B, N, V), device="cuda", dtype=_DT[case["dtype"]])
    for b in range(0, B, 16):
        n = min(16, B - b)
        z[b:b + n] = 12.0 - steep[b:b + n] * torch.log1p(V * rand(n, N, V)) + 0.3 * torch.randn(
            (n, N, V), generator=g, device="cuda")
    z[:, :, V - V // 100:] = -math.inf  # the padding of the vocabulary
    d = dict(logits=z, uniforms=rand(B, N))
    pick = lambda xs, dt: torch.tensor(xs, device="cuda", dtype=dt)[
        torch.randint(0, len(xs), (B,), generator=g, device="cuda")]
    d["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.2], torch.float32)
    k = case["top_k"]
    d["top_k"] = pick([k, max(1, k // 2), max(1, k // 5)], torch.int32) if k else None
    d["top_p"] = pick([0.8, 0.9, 0.95, 1.0], torch.float32) if case["top_p"] else None
    d["min_p"] = pick([0.0, 0.01, 0.05, 0.1], torch.float32) if case["min_p"] else None
    return d


def _power(e):
    """2^e in float64, exactly (its exponent bits; pow and ldexp of the GPU may be off by a last bit)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _least_scale(amax):
    """The least power of two s with amax <= 448 s (1 for a block of zeros); amax in float64."""
    m, e = torch.frexp(amax / _TOP)  # amax / 448 = m 2^e, m in [0.5, 1)
    s = _power(torch.where(m == 0.5, e - 1, e))
    return torch.where(amax > 0, s, torch.ones_like(s))


def _round8(x):
    """float64 values rounded to e4m3: 4 significant bits, steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(x)
    step = _power((e - 4).clamp_(min=-9))
    return torch.round(x / step) * step


def _cache_layout(case, g, whole):
    """Pages in random order.  whole: of all positions; otherwise only of those that an append touches, and
    the rest of a table's row names page 0, which holds nothing of theirs."""
    P = case["page"]
    past, new = _spread(case)
    need = [(p + n + P - 1) // P for p, n in zip(past, new)]
    first = [0 if whole else p // P for p in past]
    count = sum(n - f for n, f in zip(need, first))
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32) + (0 if whole else 1)
    table = torch.zeros((case["B"], max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, (n, f) in enumerate(zip(need, first)):
        table[b, f:n] = order[at:at + n - f]
        at += n - f
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return dict(page_table=table, past=past, new=new, cache_lens=i32(past), num_new=i32(new)), count + (0 if whole else 1)


def _pages8(shape, g):
    """Codes and scales of random values, quantised as an append does."""
    pages, H, P, D = shape
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((pages, H, P // _BLOCK), dtype=torch.float32, device="cuda")
    for i in range(0, pages, 4096):
        n = min(4096, pages - i)
        x = torch.empty((n, H, P // _BLOCK, _BLOCK * D), device="cuda").normal_(generator=g)
        # some blocks are louder than others
        x *= torch.exp2(torch.rand((n, H, P // _BLOCK, 1), generator=g, device="cuda") * 3.0 - 1.5)
        s = _least_scale(x.abs().amax(-1).double()).float()
        codes[i:i + n] = (x / s[..., None]).to(torch.float8_e4m3fn).reshape(n, H, P, D)
        scales[i:i + n] = s
    return codes, scales


def _chunk_inputs(case, seed):
    B, N, Hq, Hkv, D, P = (case[k] for k in ("B", "N", "Hq", "Hkv", "D", "page"))
    g, dt = _gen(seed), _DT[case["dtype"]]
    d, pages = _cache_layout(case, g, case["op"] != "append8")
    d["q"] = _randn((B, N, Hq, D), g, dt)
    shape = (pages, Hkv, P, D)
    if case["op"] == "sinks":
        d["k_pages"] = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
        d["v_pages"] = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    else:
        d["k_pages"], d["k_scales"] = _pages8(shape, g)
        d["v_pages"], d["v_scales"] = _pages8(shape, g)
    if case["op"] == "append8":
        d["k"], d["v"] = _randn((B, N, Hkv, D), g, dt), _randn((B, N, Hkv, D), g, dt)
        # cosines and sines of every position
        rot = case["rot"]
        freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
        ang = torch.arange(max(p + n for p, n in zip(d["past"], d["new"])), dtype=torch.float64,
                           device="cuda")[:, None] * freq
        d["table"] = torch.stack((ang.cos().float(), ang.sin().float()), 1).contiguous()
        # the changed blocks, for reading them back
        d["first"] = d["cache_lens"] // _BLOCK * _BLOCK
        d["count"] = d["cache_lens"] - d["first"] + d["num_new"]
    return d


def prepare(case, seed):
    s = dict(case=case)
    if case["op"] == "sample":
        s.update(_sample_inputs(case, seed))
        return s
    s.update(_chunk_inputs(case, seed))
    s["max_context"] = max(p + n for p, n in zip(s["past"], s["new"]))
    if own:
        if case["op"] == "sinks":
            s["cache"] = _sv().PagedCache.from_tensors(s["k_pages"], s["v_pages"])
        else:
            s["cache"] = _sv().PagedCache8.from_tensors(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"sample": _own_sample, "append8": _own_append, "attn8": _own_attn, "sinks": _own_attn}[op](s)
    return {"sample": _plain_sample, "append8": _plain_append, "attn8": _plain_attn, "sinks": _plain_attn}[op](s)


def _own_sample(s):
    return _sv().sample(s["logits"], s["uniforms"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])


def _own_append(s):
    c = s["case"]
    q = _sv().rotate_append(s["q"], s["k"], s["v"], s["table"], s["cache"], s["page_table"], s["cache_lens"],
                            s["num_new"], interleaved=c["inter"])
    k, v = _sv().read_cache(s["cache"], s["page_table"], s["first"], c["N"] + _BLOCK - 1, s["count"], dtype=q.dtype)
    return q, k, v


def _own_attn(s):
    c = s["case"]
    return _sv().paged_attention(s["q"], s["cache"], s["page_table"], s["cache_lens"], s["num_new"], window=c["window"],
                                 sinks=c["sinks"], max_context=s["max_context"])


def _plain_sample(s):
    B, N, V = s["logits"].shape
    rows = lambda x, none: torch.full((B * N, 1), none, device="cuda", dtype=torch.float64) if x is None else \
        x.double()[:, None].expand(B, N).reshape(B * N, 1)
    T, P, M = rows(s["temperature"], 1.0), rows(s["top_p"], 1.0), rows(s["min_p"], 0.0)
    K = rows(s["top_k"], 0.0).long()
    K = torch.where((K == 0) | (K > V), torch.full_like(K, V), K)
    K = torch.where(T == 0, torch.ones_like(K), K)  # greedy: the first of the largest
    # by falling logit, equal ones by their number; weights and their sums in 64 bits, since a token is drawn by
    # comparing sums of up to V of them
    z, order = torch.sort(s["logits"].reshape(B * N, V), dim=1, descending=True, stable=True)
    w = torch.exp((z.double() - z[:, :1].double()) / torch.where(T == 0, torch.ones_like(T), T))
    at = torch.arange(V, device="cuda")[None]
    w = torch.where(at < K, w, torch.zeros_like(w))
    before = torch.cumsum(w, 1) - w
    keep = (P >= 1.0) | (before < P * w.sum(1, keepdim=True))
    w = torch.where(keep & (w >= M), w, torch.zeros_like(w))
    # back in the order of the tokens
    w = torch.zeros_like(w).scatter_(1, order, w)
    c = torch.cumsum(w, 1)
    total = w.sum(1, keepdim=True)
    over = (c > s["uniforms"].reshape(B * N, 1).double() * total) & (w > 0)
    token = torch.where(over, at, torch.full_like(at, V)).amin(1)
    prob = (w.gather(1, token[:, None]) / total).float()
    return token.to(torch.int32).reshape(B, N), prob.reshape(B, N)


def _values(s, name):
    x = s[name + "_pages"].float()
    pages, H, P, D = x.shape
    return (x.reshape(pages, H, P // _BLOCK, _BLOCK, D) * s[name + "_scales"][..., None, None]).reshape(x.shape)


def _plain_append(s):
    c = s["case"]
    B, N, rot, P, D, H = c["B"], c["N"], c["rot"], c["page"], c["D"], c["Hkv"]
    i = torch.arange(N, device="cuda")[None]
    live = i < s["num_new"][:, None]
    pos = torch.where(live, s["cache_lens"][:, None].long() + i, torch.zeros((), dtype=torch.long, device="cuda"))
    cos, sin = s["table"][pos, 0][:, :, None], s["table"][pos, 1][:, :, None]

    def turn(x, c_, s_):
        if c["inter"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack((a * c_ - b * s_, a * s_ + b * c_), -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat((a * c_ - b * s_, a * s_ + b * c_), -1)
        return torch.cat((y, x[..., rot:]), -1)

    q = torch.where(live[..., None, None], turn(s["q"].float(), cos, sin), torch.zeros((), device="cuda")).to(s["q"].dtype)
    # The changed blocks: rows first[b] .. of every sequence, in 64 bits, since a value next to the border between two
    # codes goes to one or the other.
    R = (N + _BLOCK - 1 + _BLOCK - 1) // _BLOCK * _BLOCK  # rows of the blocks that a sequence can touch
    r = torch.arange(R, device="cuda")[None]
    inside = r < s["count"][:, None]
    held = r < (s["cache_lens"] - s["first"])[:, None]
    row = torch.where(inside, s["first"][:, None].long() + r, torch.zeros((), dtype=torch.long, device="cuda"))
    page = s["page_table"].gather(1, row // P).long()
    fresh = (r - (s["cache_lens"] - s["first"])[:, None].long()).clamp(0, N - 1)
    res = []
    for name, x in (("k", turn(s["k"].double(), cos.double(), sin.double())), ("v", s["v"].double())):
        codes, scales = s[name + "_pages"], s[name + "_scales"]
        old = codes[page, :, row % P].double() * scales[page, :, row % P // _BLOCK].double()[..., None]
        x = torch.where(held[..., None, None], old, x.gather(1, fresh[..., None, None].expand(B, R, H, D)))
        x = torch.where(inside[..., None, None], x, torch.zeros_like(x)).reshape(B, R // _BLOCK, _BLOCK, H, D)
        scale = _least_scale(x.abs().amax((2, 4)))  # [B, blocks, H]
        y = _round8(x / scale[:, :, None, :, None])
        bi, ri = inside.nonzero(as_tuple=True)
        codes[page[bi, ri], :, row[bi, ri] % P] = y.reshape(B, R, H, D)[bi, ri].float().to(codes.dtype)
        scales[page[bi, ri], :, row[bi, ri] % P // _BLOCK] = scale.float()[bi, ri // _BLOCK]
        y = (y * scale[:, :, None, :, None]).reshape(B, R, H, D)[:, :N + _BLOCK - 1]
        res.append(y.to(s["q"].dtype))
    return q, res[0], res[1]


def _plain_attn(s):
    c = s["case"]
    Hq, Hkv, D, w, sinks, P = c["Hq"], c["Hkv"], c["D"], c["window"], c["sinks"], c["page"]
    grp = Hq // Hkv
    out = torch.zeros_like(s["q"])
    for b, (past, n) in enumerate(zip(s["past"], s["new"])):
        L = past + n
        lo = max(0, past + 1 - w) if w else 0
        at = torch.arange(L, device="cuda")
        if lo > sinks:
            at = torch.cat((at[:sinks], at[lo:]))
        page, slot = s["page_table"][b][at // P].long(), at % P

        def values(name):
            x = s[name + "_pages"][page, :, slot].float()
            if c["op"] == "attn8":
                x = x * s[name + "_scales"][page, :, slot // _BLOCK][..., None]
            return x.transpose(0, 1)

        q = s["q"][b, :n].float().reshape(n, Hkv, grp, D).permute(1, 2, 0, 3).reshape(Hkv, grp * n, D)
        sc = torch.bmm(q, values("k").transpose(1, 2)) * (1.0 / math.sqrt(D))
        qp = past + torch.arange(n, device="cuda").repeat(grp)[:, None]
        ok = at[None] <= qp
        if w:
            ok = ok & ((at[None] > qp - w) | (at[None] < sinks))
        sc = sc.masked_fill_(~ok, -math.inf)
        sc = torch.exp_(sc - sc.amax(-1, keepdim=True))
        o = torch.bmm(sc, values("v")) / sc.sum(-1, keepdim=True)
        out[b, :n] = o.reshape(Hkv, grp, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D).to(out.dtype)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    return {"sample": _exact_sample, "append8": _exact_append, "attn8": _exact_attn, "sinks": _exact_attn}[case["op"]](
        case, seed)


def _exact_sample(case, seed):
    d = _sample_inputs(case, seed)
    B, N, V = case["B"], case["N"], case["V"]
    tokens = torch.empty((B, N), dtype=torch.int32, device="cuda")
    probs = torch.empty((B, N), dtype=torch.float64, device="cuda")
    of = lambda name, none: [none] * B if d[name] is None else d[name].tolist()
    T, K, P, M = of("temperature", 1.0), of("top_k", 0), of("top_p", 1.0), of("min_p", 0.0)
    for b in range(B):
        for i in range(N):
            z = d["logits"][b, i].double()
            if T[b] == 0.0:
                tokens[b, i] = (z == z.amax()).nonzero()[0, 0].to(torch.int32)
                probs[b, i] = 1.0
                continue
            p = torch.softmax(z / T[b], 0)
            rank = torch.argsort(z, descending=True, stable=True)
            if 0 < K[b] < V:
                rank = rank[:K[b]]
            if P[b] < 1.0:
                mass = p[rank]
                mass = torch.cumsum(mass / mass.sum(), 0)
                rank = rank[:int((mass < P[b]).sum()) + 1]
            rank = rank[p[rank] / p.amax() >= M[b]]
            ids = torch.sort(rank)[0]
            cdf = torch.cumsum(p[ids], 0)
            hit = int((cdf <= d["uniforms"][b, i].double() * cdf[-1]).sum())
            tokens[b, i] = ids[hit].to(torch.int32)
            probs[b, i] = p[ids[hit]] / cdf[-1]
    return tokens, probs


def _exact_append(case, seed):
    d = _chunk_inputs(case, seed)
    B, N, rot, P, H, D = case["B"], case["N"], case["rot"], case["page"], case["Hkv"], case["D"]
    q_out = torch.zeros(d["q"].shape, dtype=torch.float64, device="cuda")
    back = [torch.zeros((B, N + _BLOCK - 1, H, D), dtype=torch.float64, device="cuda") for _ in range(2)]
    for b, (past, n) in enumerate(zip(d["past"], d["new"])):
        tab = d["table"][past:past + n].double()
        unit = torch.complex(tab[:, 0], tab[:, 1])[:, None]

        def rotated(x):
            x = x.double().clone()
            head = x[..., :rot]
            if case["inter"]:
                z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * unit
                x[..., :rot] = torch.view_as_real(z).reshape(head.shape)
            else:
                z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * unit
                x[..., :rot] = torch.cat((z.real, z.imag), -1)
            return x

        q_out[b, :n] = rotated(d["q"][b, :n])
        first = past // _BLOCK * _BLOCK
        old = torch.arange(first, past, device="cuda")
        page, slot = d["page_table"][b].long()[old // P], old % P
        for x, name, dst in ((rotated(d["k"][b, :n]), "k", back[0]), (d["v"][b, :n].double(), "v", back[1])):
            kept = d[name + "_pages"][page, :, slot].double() * \
                d[name + "_scales"][page, :, slot // _BLOCK].double()[..., None]
            x = torch.cat((kept, x), 0)
            rows = x.shape[0]
            x = torch.cat((x, x.new_zeros((-rows % _BLOCK, H, D))), 0).reshape(-1, _BLOCK, H, D)
            peak = x.abs().amax((1, 3), keepdim=True)
            powers = torch.tensor([2.0 ** e for e in range(-60, 40)], dtype=torch.float64, device="cuda")
            scale = powers[torch.bucketize(peak, _TOP * powers)]  # the first that holds the block
            scale = torch.where(peak > 0, scale, torch.ones_like(scale))
            y = x / scale
            below = powers[torch.bucketize(y.abs().clamp(min=2.0 ** -6), powers, right=True) - 1]  # 2^e <= |y| < 2^(e + 1)
            y = torch.round(y / (below / 8)) * (below / 8) * scale
            dst[b, :rows] = y.reshape(-1, H, D)[:rows]
    return q_out, back[0], back[1]


def _exact_attn(case, seed):
    if work(case)["flops"] > 2e12:
        return None
    d = _chunk_inputs(case, seed)
    D, Hkv, P, w, sinks = case["D"], case["Hkv"], case["page"], case["window"], case["sinks"]
    grp = case["Hq"] // Hkv
    res = torch.zeros(d["q"].shape, dtype=torch.float64, device="cuda")
    for b, (past, n) in enumerate(zip(d["past"], d["new"])):
        keys = torch.arange(past + n, device="cuda")
        if w:
            keys = keys[(keys < sinks) | (keys > past - w)]
        page, slot = d["page_table"][b].long()[torch.div(keys, P, rounding_mode="floor")], keys % P
        step = max(1, int(2.5e8 / (grp * max(1, keys.numel()))))
        for h in range(Hkv):
            k, v = d["k_pages"][page, h, slot].double(), d["v_pages"][page, h, slot].double()
            if case["op"] == "attn8":
                k = k * d["k_scales"][page, h, slot // _BLOCK].double()[:, None]
                v = v * d["v_scales"][page, h, slot // _BLOCK].double()[:, None]
            for i in range(0, n, step):
                at = past + torch.arange(i, min(n, i + step), device="cuda")
                hide = keys[None] > at[:, None]
                if w:
                    hide = hide | ((keys[None] <= at[:, None] - w) & (keys[None] >= sinks))
                for g in range(grp):
                    x = d["q"][b, i:i + step][:min(n - i, step), h * grp + g].double() @ k.T / D ** 0.5
                    p = torch.softmax(x.masked_fill(hide, -math.inf), -1)
                    res[b, i:i + at.numel(), h * grp + g] = p @ v
    return res
