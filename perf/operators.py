"""What is measured of the target-step operators: logit processing, rotary append, paged attention.

Three operators stand around a verification call.  ``paged_attention`` runs the new
tokens of a round (or a chunk of a prompt) over the paged cache that ``rotate_append``
fills, and ``process_logits`` applies penalties, biases and grammar masks to the logits
before they are verified.  Each case below is one call of one of them; ``run`` computes
it in elementary torch operations, or with the framework's kernels where ``own`` is set.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _sv():
    import speculative_decoding_verification_20_gb300 as sv

    return sv


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a drafter's next-token logits, a few sequences: one small call per drafted token
        dict(name="logits_b4_n1_v32k", op="logits", B=4, N=1, V=32000, dtype="bf16", hist=300, bias=8, mask="row",
             penal=True),
        # a round of 256 sequences, gamma 7, every position with its own grammar mask
        dict(name="logits_b256_n8_v128k", op="logits", B=256, N=8, V=128256, dtype="bf16", hist=2000, bias=16,
             mask="pos", penal=True),
        # fp32 logits, gamma 8, long outputs, one mask per sequence
        dict(name="logits_b32_n9_v152k", op="logits", B=32, N=9, V=151936, dtype="f32", hist=9000, bias=300, mask="row",
             penal=True),
        # one token for each of a few sequences
        dict(name="rotate_b4_n1", op="rotate", B=4, N=1, Hq=32, Hkv=8, D=128, rot=128, inter=False, dtype="bf16",
             page=16, past_lo=50, past_hi=4000, ragged=False, scaling="none"),
        # a round of 256 sequences, gamma 7, ragged, far positions on a scaled table
        dict(name="rotate_b256_n8", op="rotate", B=256, N=8, Hq=32, Hkv=8, D=128, rot=128, inter=False, dtype="bf16",
             page=32, past_lo=0, past_hi=1000, ragged=True, scaling="yarn"),
        # a chunk of two prompts, interleaved pairs on half of the head
        dict(name="rotate_b2_n4096", op="rotate", B=2, N=4096, Hq=32, Hkv=8, D=128, rot=64, inter=True, dtype="f16",
             page=64, past_lo=0, past_hi=20000, ragged=True, scaling="linear"),
        # plain decoding of one short sequence: latency
        dict(name="attn_b1_n1", op="attn", B=1, N=1, Hq=32, Hkv=8, D=128, dtype="bf16", page=16, past_lo=700,
             past_hi=700, ragged=False, window=0),
        # a round of 64 sequences, gamma 7, mixed lengths
        dict(name="attn_b64_n8", op="attn", B=64, N=8, Hq=32, Hkv=8, D=128, dtype="bf16", page=16, past_lo=1500,
             past_hi=8200, ragged=True, window=0),
        # a round of two very long sequences, gamma 5: few rows, long axis
        dict(name="attn_b2_n6_long", op="attn", B=2, N=6, Hq=32, Hkv=4, D=128, dtype="bf16", page=64, past_lo=90001,
             past_hi=131000, ragged=False, window=0),
        # a chunk of two prompts behind earlier chunks
        dict(name="attn_b2_n2048", op="attn", B=2, N=2048, Hq=32, Hkv=8, D=128, dtype="bf16", page=64, past_lo=4000,
             past_hi=6144, ragged=False, window=0),
        # small heads in groups of five, a sliding window, chunks of odd lengths, odd pages
        dict(name="attn_b5_n333_window", op="attn", B=5, N=333, Hq=20, Hkv=4, D=64, dtype="f16", page=48, past_lo=10,
             past_hi=5000, ragged=True, window=1001),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logits", "rotate", "attn"])
    ref = [work(c) for c in listed() if c["op"] == op]
    cap_b, cap_f = max(w["bytes"] for w in ref), max(w["flops"] for w in ref)
    while True:
        if op == "logits":
            case = dict(op=op, B=_logu(rng, 1, 256), N=rng.randint(1, 9), V=_logu(rng, 1000, 152000),
                        dtype=rng.choice(["bf16", "f32"]), hist=_logu(rng, 1, 9000), bias=rng.choice([0, 1, 16, 300]),
                        mask=rng.choice(["none", "row", "pos"]), penal=rng.random() < 0.8)
        else:
            Hkv = rng.choice([1, 2, 4, 8])
            D = rng.choice([64, 128])
            N = rng.choice([1, rng.randint(2, 9), rng.randint(2, 9), _logu(rng, 10, 2100)])
            case = dict(op=op, B=_logu(rng, 1, 128), N=N, Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=D,
                        dtype=rng.choice(["bf16", "f16"]), page=rng.choice([16, 32, 48, 64, 128, 256]))
            lo = _logu(rng, 1, 20000)
            case.update(past_lo=lo - 1, past_hi=lo - 1 + _logu(rng, 1, 20000), ragged=rng.random() < 0.5)
            if op == "rotate":
                case.update(rot=rng.choice([D, D // 2, D // 4]), inter=rng.random() < 0.5,
                            scaling=rng.choice(["none", "linear", "yarn"]))
            else:
                case.update(window=rng.choice([0, 0, _logu(rng, 1, 5000)]))
        w = work(case)
        if op != "logits":  # the whole cache is part of the state: 4 GB of it at most
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


def _visible(past, n, window):
    """Visible keys summed over the n new tokens, and the number of distinct keys."""
    if not window:
        return n * past + n * (n + 1) // 2, past + n
    pairs = sum(min(past + i + 1, window) for i in range(n))
    return pairs, past + n - max(0, past + 1 - window)


def work(case):
    if case["op"] == "logits":
        B, N, V = case["B"], case["N"], case["V"]
        es = 2 if case["dtype"] == "bf16" else 4
        W = (V + 31) // 32
        n = 2 * B * N * V * es + 8 * B * case["bias"]
        n += {"none": 0, "row": 4 * B * W, "pos": 4 * B * N * W}[case["mask"]]
        if case["penal"]:  # which tokens were seen, as bits, and the counts of those that were output
            n += 2 * 4 * B * W + 4 * B * min(case["hist"], V)
        return {"bytes": n, "flops": 6 * B * N * V}
    past, new = _spread(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    T = sum(new)
    if case["op"] == "rotate":
        return {"bytes": 2 * 2 * T * (Hq + 2 * Hkv) * D + 4 * T * case["rot"], "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    pairs = keys = 0
    for p, n in zip(past, new):
        a, k = _visible(p, n, case["window"])
        pairs, keys = pairs + a, keys + k
    return {"bytes": 2 * 2 * keys * Hkv * D + 2 * 2 * T * Hq * D, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _logit_inputs(case, seed):
    B, N, V, H = case["B"], case["N"], case["V"], case["hist"]
    g = _gen(seed)
    d = {}
    d["logits"] = torch.empty(B, N, V, device="cuda", dtype=_DT[case["dtype"]])
    for b in range(0, B, 16):
        n = min(16, B - b)
        d["logits"][b:b + n] = 3.0 * torch.randn((n, N, V), generator=g, device="cuda")
    # tokens come by a power law: few ids make most of a text
    u = torch.rand((B, H), generator=g, device="cuda")
    d["tokens"] = (torch.exp(u * math.log(V)) - 1.0).to(torch.int32).clamp_(0, V - 1)
    d["total_lens"] = torch.randint((H + 1) // 2, H + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    d["prompt_lens"] = d["total_lens"] // 2
    u = torch.rand((B, max(N - 1, 1)), generator=g, device="cuda")
    d["draft_tokens"] = (torch.exp(u * math.log(V)) - 1.0).to(torch.int32).clamp_(0, V - 1)[:, :N - 1].contiguous()
    r = torch.rand((3, B), generator=g, device="cuda")
    d["repetition"], d["frequency"], d["presence"] = 1.0 + 0.5 * r[0], 0.6 * r[1], 0.8 * r[2]
    if case["bias"]:
        n = case["bias"]
        d["bias_ids"] = torch.randint(0, V, (B, n), generator=g, device="cuda", dtype=torch.int32).reshape(-1)
        d["bias_values"] = 5.0 * torch.randn((B * n,), generator=g, device="cuda")
        d["bias_offsets"] = torch.arange(B + 1, device="cuda", dtype=torch.int32) * n
    if case["mask"] != "none":
        # rows inside a string allow nearly everything, rows at a keyword nearly nothing
        shape = (B, N) if case["mask"] == "pos" else (B, 1)
        W = (V + 31) // 32
        level = torch.tensor([0.002, 0.3, 0.98], device="cuda")[
            torch.randint(0, 3, shape, generator=g, device="cuda")]
        bits = torch.zeros(shape + (W,), device="cuda", dtype=torch.int32)
        for k in range(32):
            on = torch.rand(shape + (W,), generator=g, device="cuda") < level[..., None]
            bits |= on.to(torch.int32) << k
        d["mask"] = bits if case["mask"] == "pos" else bits[:, 0].contiguous()
    return d


def _chunk_inputs(case, seed, cache_random):
    B, N, Hq, Hkv, D, P = (case[k] for k in ("B", "N", "Hq", "Hkv", "D", "page"))
    g, dt = _gen(seed), _DT[case["dtype"]]
    past, new = _spread(case)
    need = [(p + n + P - 1) // P for p, n in zip(past, new)]
    pages = sum(need)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    d = dict(page_table=table, past=past, new=new,
             cache_lens=torch.tensor(past, dtype=torch.int32, device="cuda"),
             num_new=torch.tensor(new, dtype=torch.int32, device="cuda"))
    d["q"] = _randn((B, N, Hq, D), g, dt)
    shape = (pages, Hkv, P, D)
    if cache_random:
        d["k_pages"] = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
        d["v_pages"] = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    else:
        d["k_pages"] = torch.zeros(shape, dtype=dt, device="cuda")
        d["v_pages"] = torch.zeros(shape, dtype=dt, device="cuda")
        d["k"], d["v"] = _randn((B, N, Hkv, D), g, dt), _randn((B, N, Hkv, D), g, dt)
    return d


_BASE = 10000.0
_YARN = dict(type="yarn", factor=8.0, original_length=4096)
_LINEAR = dict(type="linear", factor=4.0)


def _scaling(case):
    return {"none": None, "linear": _LINEAR, "yarn": _YARN}[case["scaling"]]


def _frequencies(case):
    """Angle per position of each pair and the factor on cos and sin, in Python floats."""
    half, rot = case["rot"] // 2, case["rot"]
    freq = [_BASE ** (-2.0 * j / rot) for j in range(half)]
    if case["scaling"] == "linear":
        return [f / _LINEAR["factor"] for f in freq], 1.0
    if case["scaling"] == "yarn":
        s, L = _YARN["factor"], _YARN["original_length"]

        def at(turns):  # the pair that makes so many turns over the original length
            return rot * math.log(L / (turns * 2.0 * math.pi)) / (2.0 * math.log(_BASE))

        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        out = []
        for j, f in enumerate(freq):
            ramp = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            out.append(f * (1.0 - ramp) + f / s * ramp)
        return out, 0.1 * math.log(s) + 1.0
    return freq, 1.0


def prepare(case, seed):
    s = dict(case=case)
    if case["op"] == "logits":
        d = _logit_inputs(case, seed)
        s.update(d)
        if case["penal"]:
            B, V = case["B"], case["V"]
            if own:
                s["history"] = _sv().TokenHistory(B, V, device="cuda")
                s["history"].load(d["tokens"], d["prompt_lens"], d["total_lens"])
            else:
                j = torch.arange(case["hist"], device="cuda")[None]
                out = ((j >= d["prompt_lens"][:, None]) & (j < d["total_lens"][:, None])).to(torch.int32)
                pro = (j < d["prompt_lens"][:, None]).to(torch.int32)
                at = d["tokens"].long()
                s["counts"] = torch.zeros((B, V), dtype=torch.int32, device="cuda").scatter_add_(1, at, out)
                s["prompt"] = torch.zeros((B, V), dtype=torch.int32, device="cuda").scatter_add_(1, at, pro) > 0
    else:
        d = _chunk_inputs(case, seed, case["op"] == "attn")
        s.update(d)
        s["max_context"] = max(p + n for p, n in zip(d["past"], d["new"]))
        if own:
            s["cache"] = _sv().PagedCache.from_tensors(d["k_pages"], d["v_pages"])
        if case["op"] == "rotate":
            if own:
                s["table"] = _sv().rotary_table(s["max_context"], case["rot"], base=_BASE, scaling=_scaling(case),
                                                device="cuda")
            else:
                freq, m = _frequencies(case)
                ang = torch.arange(s["max_context"], dtype=torch.float64, device="cuda")[:, None] * torch.tensor(
                    freq, dtype=torch.float64, device="cuda")
                s["cos"], s["sin"] = (ang.cos() * m).float(), (ang.sin() * m).float()
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"logits": _own_logits, "rotate": _own_rotate, "attn": _own_attn}[op](s)
    return {"logits": _plain_logits, "rotate": _plain_rotate, "attn": _plain_attn}[op](s)


def _own_logits(s):
    kw = {}
    if s["case"]["penal"]:
        kw = dict(history=s["history"], draft_tokens=s["draft_tokens"], repetition=s["repetition"],
                  frequency=s["frequency"], presence=s["presence"])
    if s["case"]["bias"]:
        kw["bias"] = (s["bias_ids"], s["bias_values"], s["bias_offsets"])
    return _sv().process_logits(s["logits"], mask=s.get("mask"), **kw)


def _own_rotate(s):
    c = s["case"]
    q = _sv().rotate_append(s["q"], s["k"], s["v"], s["table"], s["cache"], s["page_table"], s["cache_lens"],
                            s["num_new"], interleaved=c["inter"])
    return q, s["k_pages"], s["v_pages"]


def _own_attn(s):
    return _sv().paged_attention(s["q"], s["cache"], s["page_table"], s["cache_lens"], s["num_new"],
                                 window=s["case"]["window"], max_context=s["max_context"])


def _plain_logits(s):
    c = s["case"]
    B, N, V = c["B"], c["N"], c["V"]
    z = s["logits"].float()
    if c["penal"]:
        cnt = s["counts"][:, None].repeat(1, N, 1)
        one = torch.ones((B, 1), dtype=torch.int32, device="cuda")
        for i in range(1, N):
            at = s["draft_tokens"][:, i - 1:i].long()
            for j in range(i, N):
                cnt[:, j].scatter_add_(1, at, one)
        seen = s["prompt"][:, None] | (cnt > 0)
        r = s["repetition"][:, None, None]
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        z = z - s["frequency"][:, None, None] * cnt - s["presence"][:, None, None] * (cnt > 0)
    if c["bias"]:
        add = torch.zeros((B, V), device="cuda")
        row = torch.arange(B, device="cuda").repeat_interleave(c["bias"])
        add.index_put_((row, s["bias_ids"].long()), s["bias_values"], accumulate=True)
        z = z + add[:, None]
    if c["mask"] != "none":
        t = torch.arange(V, device="cuda")
        m = s["mask"] if c["mask"] == "pos" else s["mask"][:, None]
        ok = (m[..., t >> 5] >> (t & 31).to(torch.int32)) & 1
        z = torch.where(ok.bool(), z, torch.full((), -math.inf, device="cuda"))
    return z.to(s["logits"].dtype)


def _plain_rotate(s):
    c = s["case"]
    B, N, rot, P = c["B"], c["N"], c["rot"], c["page"]
    live = torch.arange(N, device="cuda")[None] < s["num_new"][:, None]
    pos = s["cache_lens"][:, None].long() + torch.arange(N, device="cuda")[None]
    at = torch.where(live, pos, torch.zeros_like(pos))
    cos, sin = s["cos"][at][:, :, None], s["sin"][at][:, :, None]

    def turn(x):
        x = x.float()
        h = rot // 2
        if c["inter"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = x[..., :h], x[..., h:rot]
            y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((y, x[..., rot:]), -1)

    q = torch.where(live[..., None, None], turn(s["q"]), torch.zeros((), device="cuda")).to(s["q"].dtype)
    k = turn(s["k"]).to(s["k"].dtype)
    bi, ti = live.nonzero(as_tuple=True)
    page = s["page_table"][bi, at[bi, ti] // P].long()
    slot = at[bi, ti] % P
    s["k_pages"][page, :, slot] = k[bi, ti]
    s["v_pages"][page, :, slot] = s["v"][bi, ti]
    return q, s["k_pages"], s["v_pages"]


def _plain_attn(s):
    c = s["case"]
    Hq, Hkv, D, w = c["Hq"], c["Hkv"], c["D"], c["window"]
    grp = Hq // Hkv
    out = torch.zeros_like(s["q"])
    for b, (past, n) in enumerate(zip(s["past"], s["new"])):
        L = past + n
        lo = max(0, past + 1 - w) if w else 0
        p0 = lo // c["page"]
        ids = s["page_table"][b, p0:(L + c["page"] - 1) // c["page"]].long()
        lo0 = p0 * c["page"]
        k = s["k_pages"][ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :L - lo0].float()
        v = s["v_pages"][ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :L - lo0].float()
        q = s["q"][b, :n].float().reshape(n, Hkv, grp, D).permute(1, 2, 0, 3).reshape(Hkv, grp * n, D)
        sc = torch.bmm(q, k.transpose(1, 2)) * (1.0 / math.sqrt(D))
        qp = past + torch.arange(n, device="cuda").repeat(grp)[:, None]
        kp = lo0 + torch.arange(L - lo0, device="cuda")[None]
        ok = (kp <= qp) & (kp > qp - w) if w else kp <= qp
        sc = sc.masked_fill_(~ok, -math.inf)
        sc = torch.exp_(sc - sc.amax(-1, keepdim=True))
        o = torch.bmm(sc, v) / sc.sum(-1, keepdim=True)
        out[b, :n] = o.reshape(Hkv, grp, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D).to(out.dtype)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    return {"logits": _exact_logits, "rotate": _exact_rotate, "attn": _exact_attn}[case["op"]](case, seed)


def _exact_logits(case, seed):
    d = _logit_inputs(case, seed)
    B, N, V = case["B"], case["N"], case["V"]
    res = torch.empty((B, N, V), dtype=torch.float64, device="cuda")
    pl, tl = d["prompt_lens"].tolist(), d["total_lens"].tolist()
    shifts = torch.arange(32, device="cuda", dtype=torch.int32)
    for b in range(B):
        toks = d["tokens"][b].long()
        in_prompt = torch.bincount(toks[:pl[b]], minlength=V) > 0
        in_output = torch.bincount(toks[pl[b]:tl[b]], minlength=V).double()
        for i in range(N):
            z = d["logits"][b, i].double()
            if case["penal"]:
                n = in_output + torch.bincount(d["draft_tokens"][b, :i].long(), minlength=V)
                factor = d["repetition"][b].double()
                hit = in_prompt | (n > 0)
                up, down = hit & (z > 0), hit & (z <= 0)
                z[up] /= factor
                z[down] *= factor
                z -= n * d["frequency"][b].double()
                z[n > 0] -= d["presence"][b].double()
            if case["bias"]:
                lo, hi = b * case["bias"], (b + 1) * case["bias"]
                z.index_add_(0, d["bias_ids"][lo:hi].long(), d["bias_values"][lo:hi].double())
            if case["mask"] != "none":
                words = d["mask"][b, i] if case["mask"] == "pos" else d["mask"][b]
                bits = ((words[:, None] >> shifts) & 1).reshape(-1)[:V]
                z[bits == 0] = -math.inf
            res[b, i] = z
    return res


def _exact_rotate(case, seed):
    d = _chunk_inputs(case, seed, False)
    B, N, rot, P = case["B"], case["N"], case["rot"], case["page"]
    freq, m = _frequencies(case)
    freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
    qo = torch.zeros(d["q"].shape, dtype=torch.float64, device="cuda")
    ko, vo = d["k_pages"].double(), d["v_pages"].double()
    for b, (past, n) in enumerate(zip(d["past"], d["new"])):
        pos = past + torch.arange(n, device="cuda")
        turn = m * torch.polar(torch.ones((n, 1, rot // 2), dtype=torch.float64, device="cuda"),
                               pos.double()[:, None, None] * freq)

        def rotated(x):
            x = x.double().clone()
            head = x[..., :rot]
            if case["inter"]:
                z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
                x[..., :rot] = torch.view_as_real(z).reshape(head.shape)
            else:
                z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
                x[..., :rot] = torch.cat((z.real, z.imag), -1)
            return x

        qo[b, :n] = rotated(d["q"][b, :n])
        page = d["page_table"][b].long()[torch.div(pos, P, rounding_mode="floor")]
        ko[page, :, pos % P] = rotated(d["k"][b, :n])
        vo[page, :, pos % P] = d["v"][b, :n].double()
    return qo, ko, vo


def _exact_attn(case, seed):
    if work(case)["flops"] > 2e12:
        return None
    d = _chunk_inputs(case, seed, True)
    D, Hkv, P, w = case["D"], case["Hkv"], case["page"], case["window"]
    grp = case["Hq"] // Hkv
    res = torch.zeros(d["q"].shape, dtype=torch.float64, device="cuda")
    for b, (past, n) in enumerate(zip(d["past"], d["new"])):
        keys = torch.arange(past + n, device="cuda")
        if w:
            keys = keys[max(0, past + 1 - w):]
        page, slot = d["page_table"][b].long()[torch.div(keys, P, rounding_mode="floor")], keys % P
        step = max(1, int(2.5e8 / (grp * max(1, keys.numel()))))
        for h in range(Hkv):
            k, v = d["k_pages"][page, h, slot].double(), d["v_pages"][page, h, slot].double()
            for i in range(0, n, step):
                at = past + torch.arange(i, min(n, i + step), device="cuda")
                hide = keys[None] > at[:, None]
                if w:
                    hide = hide | (keys[None] <= at[:, None] - w)
                for g in range(grp):
                    x = d["q"][b, i:i + step][:min(n - i, step), h * grp + g].double() @ k.T / D ** 0.5
                    p = torch.softmax(x.masked_fill(hide, -math.inf), -1)
                    res[b, i:i + at.numel(), h * grp + g] = p @ v
    return res
