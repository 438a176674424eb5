"""The target-step operators on a GPU against their 64-bit forms (tests/target_ref.py)."""
import math
import random
import struct

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import target_ref as ref

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_20_gb300 import _build

    _build.build()
    sv.load_library()


def check(got, want, tol, what=""):
    got, want, tol = got.double().cpu(), want.cpu(), tol.cpu()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got) & (got < 0), inf & (want < 0)), what
    d = torch.where(inf, torch.zeros_like(want), (got - want).abs())
    over = ~(d <= torch.where(inf, torch.ones_like(tol), tol))
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} off, worst {(d / tol)[over].max()} of tolerance"


# ---------------------------------------------------------------------------
# logits
# ---------------------------------------------------------------------------
def logit_case(B, N, V, dtype, seed, hist=40, nbias=5, mask="pos", draft=True):
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    d = dict(logits=(3 * torch.randn(B, N, V, generator=g)).to(dtype))
    # a few ids make most of the text, the first and the last id among them
    ids = [0, V - 1] + [rng.randrange(V) for _ in range(8)]
    tok = lambda n: [rng.choice(ids) if rng.random() < 0.7 else rng.randrange(V) for _ in range(n)]
    d["prompt"] = [tok(rng.randrange(hist + 1)) for _ in range(B)]
    d["output"] = [tok(rng.randrange(hist + 1)) for _ in range(B)]
    d["draft"] = [tok(max(N - 1, 1)) for _ in range(B)] if draft else None
    d["rep"] = [1.0 + 0.5 * rng.random() for _ in range(B)]
    d["freq"] = [rng.uniform(-1, 1) for _ in range(B)]
    d["pres"] = [rng.uniform(-1, 1) for _ in range(B)]
    f32 = lambda xs: [float(torch.tensor(x, dtype=F32)) for x in xs]
    d["rep"], d["freq"], d["pres"] = f32(d["rep"]), f32(d["freq"]), f32(d["pres"])
    d["bias"] = [list(zip(tok(n), f32([rng.uniform(-5, 5) for _ in range(n)])))
                 for n in [rng.randrange(nbias + 1) for _ in range(B)]]
    d["mask"] = None
    if mask:
        level = torch.tensor([0.0, 0.01, 0.5, 1.0])[torch.randint(0, 4, (B, N, 1), generator=g)]
        m = torch.rand(B, N, V, generator=g) < level
        d["mask"] = m if mask == "pos" else m[:, :1].expand(B, N, V).contiguous()
    return d


def history_of(d, V, slots=None, of=None):
    B = len(d["prompt"])
    h = sv.TokenHistory(slots or B, V)
    L = max(1, max(len(p) + len(o) for p, o in zip(d["prompt"], d["output"])))
    toks = torch.full((B, L), -7, dtype=torch.int32)
    for b in range(B):
        row = d["prompt"][b] + d["output"][b]
        toks[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
    h.load(toks.cuda(), [len(p) for p in d["prompt"]], [len(p) + len(o) for p, o in zip(d["prompt"], d["output"])], of)
    return h


def bias_of(d):
    ids = [t for row in d["bias"] for t, _ in row]
    vals = [v for row in d["bias"] for _, v in row]
    offs = [0]
    for row in d["bias"]:
        offs.append(offs[-1] + len(row))
    return (torch.tensor(ids, dtype=torch.int32).cuda(), torch.tensor(vals, dtype=F32).cuda(),
            torch.tensor(offs, dtype=torch.int32).cuda())


def run_logits(d, x, V, mask_kind="pos", **kw):
    m = None
    if d["mask"] is not None:
        m = ref.planes_of(d["mask"] if mask_kind == "pos" else d["mask"][:, 0]).cuda()
    return sv.process_logits(x, draft_tokens=None if d["draft"] is None else torch.tensor(d["draft"], dtype=torch.int32).cuda(),
                             repetition=d["rep"], frequency=d["freq"], presence=d["pres"], bias=bias_of(d), mask=m, **kw)


def want_logits(d):
    w, t = ref.process_logits(d["logits"], d["prompt"], d["output"], d["draft"], d["rep"], d["freq"], d["pres"], d["bias"],
                              d["mask"])
    return w, t + ref.half_step(d["logits"].dtype) * torch.where(torch.isinf(w), 0.0, w.abs()) * (1 + 2 ** -6)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,N,V,mask", [(1, 1, 1, "pos"), (2, 3, 7, "pos"), (3, 2, 33, "row"), (2, 9, 1000, "pos"),
                                        (3, 4, 8191, "pos"), (2, 2, 8193, None), (4, 1, 32000, "row"),
                                        (2, 8, 20011, "pos"), (1, 33, 515, "row")])
def test_logits_match(B, N, V, mask, dtype):
    d = logit_case(B, N, V, dtype, seed=B * 100 + N * 10 + V, mask=mask)
    got = run_logits(d, d["logits"].cuda(), V, mask, history=history_of(d, V))
    check(got, *want_logits(d))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_logits_large_launch_matches(dtype):
    """Enough rows that each thread takes several vectors."""
    B, N, V = 130, 16, 8193
    d = logit_case(B, N, V, dtype, seed=3, hist=30)
    got = run_logits(d, d["logits"].cuda(), V, history=history_of(d, V))
    check(got, *want_logits(d))


def test_logits_wide_launch_in_place_with_strides():
    B, N, V = 9, 4, 5003
    d = logit_case(B, N, V, BF, seed=11)
    big = torch.zeros(N, B, V + 13, dtype=BF, device="cuda")  # another order, padded, odd rows
    x = big.permute(1, 0, 2)[:, :, 5:5 + V]
    x.copy_(d["logits"])
    got = run_logits(d, x, V, history=history_of(d, V), out=x)
    assert got is x
    check(got, *want_logits(d))
    assert big[:, :, :5].abs().max() == 0 and big[:, :, 5 + V:].abs().max() == 0
    # rows whose output starts at another offset than their input
    y = torch.zeros(B, N, V + 3, dtype=BF, device="cuda")[:, :, 3:]
    got = run_logits(d, d["logits"].cuda(), V, history=history_of(d, V), out=y)
    check(got, *want_logits(d))


def test_logits_plain_copies_and_single_parts():
    B, N, V = 3, 2, 1003
    d = logit_case(B, N, V, F32, seed=5)
    x = d["logits"].cuda()
    assert torch.equal(sv.process_logits(x), x)
    none = dict(d, prompt=[[]] * B, output=[[]] * B, draft=None, rep=[1.0] * B, freq=[0.0] * B, pres=[0.0] * B,
                bias=[[]] * B, mask=None)
    for part in (dict(bias=d["bias"]), dict(mask=d["mask"]), dict(output=d["output"], freq=d["freq"]),
                 dict(prompt=d["prompt"], rep=d["rep"]), dict(draft=d["draft"], pres=d["pres"], rep=d["rep"])):
        e = dict(none, **part)
        kw = {}
        if e["prompt"] != none["prompt"] or e["output"] != none["output"]:
            kw["history"] = history_of(e, V)
        check(run_logits(e, x, V, **kw), *want_logits(e))


def test_logits_many_biases_and_repeats():
    """More biases in one chunk than its list holds, ids repeated and out of range."""
    V = 2000
    d = logit_case(2, 3, V, F32, seed=8)
    rng = random.Random(1)
    d["bias"] = [[(rng.randrange(40), rng.uniform(-1, 1)) for _ in range(3000)],
                 [(-1, 5.0), (V, 5.0), (2 ** 31 - 1, 1.0), (7, 1.5), (7, 2.25)]]
    d["bias"] = [[(t, float(torch.tensor(v, dtype=F32))) for t, v in row] for row in d["bias"]]
    check(run_logits(d, d["logits"].cuda(), V, history=history_of(d, V)), *want_logits(d))


def test_logits_special_values():
    x = torch.tensor([[[math.inf, -math.inf, math.nan, 0.0, -0.0, 1e38, -1e38, 2.0]]], device="cuda")
    h = sv.TokenHistory(1, 8)
    h.load([[0, 1, 2, 3, 4, 5, 6, 7]], [8], [8])
    allow = torch.tensor([[0b01111111]], dtype=torch.int32, device="cuda")
    z = sv.process_logits(x, history=h, repetition=2.0, mask=allow)[0, 0]
    assert z[0] == math.inf and z[1] == -math.inf and z[2].isnan() and z[3] == 0 and z[4] == 0
    assert z[5] == 5e37 and z[6] == -2e38 and z[7] == -math.inf
    # what the mask hides may be anything
    z = sv.process_logits(torch.full((1, 1, 8), math.nan, device="cuda"), mask=torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    assert bool((z == -math.inf).all())
    low = torch.full((1, 1, 8), torch.finfo(BF).min, dtype=BF, device="cuda")
    z = sv.process_logits(low, frequency=1.0, history=h, repetition=2.0)
    assert bool((z == -math.inf).all())


def test_logits_bad_sequences_get_nan_and_a_status():
    B, V = 7, 100
    x = torch.randn(B, 2, V, device="cuda")
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    h = sv.TokenHistory(3, V)
    rep = [1.0, 0.0, -1.0, math.nan, math.inf, 1.0, 1.0]
    freq = [0.0, 0.0, 0.0, 0.0, 0.0, math.nan, 0.0]
    slots = [2, 0, 0, 0, 0, 0, 3]
    z = sv.process_logits(x, history=h, slots=slots, repetition=rep, frequency=freq, row_status=st)
    assert st.tolist() == [0] + [sv.ROW_BAD_PENALTY] * 5 + [sv.ROW_BAD_SLOT]
    assert torch.equal(z[0], x[0]) and bool(z[1:].isnan().all())
    res = sv.spec_verify(z, torch.randn(B, 1, V, device="cuda"), torch.zeros(B, 1, dtype=torch.int32), 1.0, seed=1)
    assert res["row_status"][0] == 0 and bool((res["row_status"][1:] & sv.ROW_NONFINITE != 0).all())


def test_history_load_add_and_slots():
    V = 1000
    h = sv.TokenHistory(5, V)
    h.load(torch.tensor([[1, 2, 3, 2, 999], [5, 5, 5, 5, 5]], dtype=torch.int32, device="cuda"), [2, 0], [5, 3], [4, 1])
    c = h.counts.cpu()
    assert c[4, 1] == 0 and c[4, 2] == 1 and c[4, 3] == 1 and c[4, 999] == 1 and c[1, 5] == 3 and int(c.sum()) == 6
    seen = ref.bits_of(h.seen, V).cpu()
    assert seen[4].nonzero().flatten().tolist() == [1, 2, 3, 999] and seen[1].nonzero().flatten().tolist() == [5]
    h.add(torch.tensor([[7, 7, -1, -1], [1000, 5, 2 ** 31 - 1, -5]], dtype=torch.int32, device="cuda"), slots=[4, 1])
    c = h.counts.cpu()
    assert c[4, 7] == 2 and c[1, 5] == 4 and int(c.sum()) == 9
    h.add(torch.tensor([[9]], dtype=torch.int32, device="cuda"), slots=[5])  # no such slot: skipped
    h.add(torch.tensor([[9]], dtype=torch.int32, device="cuda"), slots=[-1])
    assert int(h.counts.sum()) == 9
    h.load(torch.zeros((1, 0), dtype=torch.int32, device="cuda"), slots=[4])  # an empty text empties the slot
    assert int(h.counts[4].sum()) == 0 and int(h.seen[4].abs().sum()) == 0 and int(h.counts[1].sum()) == 4
    with pytest.raises(ValueError):
        h.add(torch.zeros((6, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        sv.process_logits(torch.zeros(1, 1, V + 1, device="cuda"), history=h)


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------
def paged(B, N, Hq, Hkv, D, dtype, page, past, new, seed, order="hnd", spare=3, poison=True):
    """Random q, k, v of all positions, and a cache whose unused rows, pages and page ids are poison."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [(p + n + page - 1) // page for p, n in zip(past, new)]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    wide = max(max(need), 1) + 1
    table = torch.full((B, wide), -1 if poison else 0, dtype=torch.int32)
    shape = (pages, Hkv, page, D) if order == "hnd" else (pages, page, Hkv, D)
    kc = torch.full(shape, math.nan if poison else 0.0, dtype=dtype, device="cuda")
    vc = torch.full(shape, math.nan if poison else 0.0, dtype=dtype, device="cuda")
    if order == "nhd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    at = 0
    ks, vs = [], []
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]].to(torch.int32)
        at += need[b]
        L = past[b] + new[b]
        k = torch.randn(Hkv, L, D, generator=g, device="cuda").to(dtype)
        v = torch.randn(Hkv, L, D, generator=g, device="cuda").to(dtype)
        j = torch.arange(L, device="cuda")
        ids = table[b].cuda().long()[j // page]
        kc[ids, :, j % page] = k.transpose(0, 1)
        vc[ids, :, j % page] = v.transpose(0, 1)
        ks.append(k)
        vs.append(v)
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").to(dtype)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return dict(q=q, k=ks, v=vs, cache=sv.PagedCache.from_tensors(kc, vc), table=table.cuda(), lens=i32(past), new=i32(new))


def check_attention(s, past, new, window=0, scale=None, got=None, **kw):
    q = s["q"]
    D = q.shape[3]
    if got is None:
        got = sv.paged_attention(q, s["cache"], s["table"], s["lens"], s["new"], window=window, scale=scale, **kw)
    for b in range(q.shape[0]):
        n = new[b]
        assert bool((got[b, n:] == 0).all()), f"sequence {b}: rows past its new tokens"
        if n == 0:
            continue
        w, t = ref.attention(q[b, :n], s["k"][b], s["v"][b], past[b], 1 / math.sqrt(D) if scale is None else scale, window,
                             q.dtype)
        check(got[b, :n], w, t, f"sequence {b}")
    return got


SHAPES = [  # B, N, Hq, Hkv, D, page, past, new, window
    (1, 1, 1, 1, 64, 16, [0], [1], 0),
    (1, 1, 8, 8, 128, 16, [15], [1], 0),
    (2, 1, 8, 2, 128, 32, [16, 700], [1, 1], 0),
    (3, 1, 32, 8, 128, 16, [127, 128, 129], [1, 1, 1], 0),
    (3, 8, 8, 2, 64, 16, [0, 5, 1000], [8, 3, 1], 0),
    (4, 5, 6, 2, 128, 48, [3, 0, 511, 40], [5, 0, 4, 0], 0),
    (2, 6, 40, 8, 128, 64, [3001, 2000], [6, 6], 0),
    (2, 6, 35, 7, 64, 16, [300, 2000], [6, 2], 100),
    (2, 17, 16, 1, 128, 128, [0, 333], [17, 9], 0),
    (1, 130, 4, 4, 64, 16, [7], [130], 0),
    (2, 200, 6, 2, 128, 256, [0, 1000], [200, 77], 64),
    (1, 77, 12, 3, 128, 16, [500], [77], 1),
    (3, 300, 8, 2, 128, 64, [0, 129, 900], [300, 257, 1], 0),
    (2, 520, 5, 1, 64, 48, [100, 0], [520, 511], 0),
    (2, 300, 64, 1, 128, 16, [77, 0], [40, 300], 333),
    (1, 1100, 2, 2, 128, 32, [2500], [1100], 1000),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_attention_matches(shape, dtype):
    B, N, Hq, Hkv, D, page, past, new, window = shape
    s = paged(B, N, Hq, Hkv, D, dtype, page, past, new, seed=N + Hq)
    check_attention(s, past, new, window)


@pytest.mark.parametrize("N", [1, 8, 150])
def test_attention_layouts_strides_scale_and_out(N):
    B, Hq, Hkv, D = 2, 8, 2, 128
    past, new = [100, 260], [N, max(1, N - 3)]
    s = paged(B, N, Hq, Hkv, D, BF, 32, past, new, seed=4, order="nhd")
    want = check_attention(s, past, new, scale=0.2)
    fused = torch.randn(B, N, Hq + 2 * Hkv, D, device="cuda").to(BF)  # q inside a fused projection
    fused[:, :, :Hq] = s["q"]
    out = torch.full((N, B, Hq, D), 7.0, dtype=BF, device="cuda").transpose(0, 1)
    got = sv.paged_attention(fused[:, :, :Hq], s["cache"], s["table"], s["lens"], s["new"], scale=0.2, out=out,
                             max_context=max(p + n for p, n in zip(past, new)))
    assert got is out
    check_attention(s, past, new, scale=0.2, got=got)
    odd = torch.zeros(B * N * Hq * D + 3, dtype=BF, device="cuda")[3:].view(B, N, Hq, D)  # off a boundary: copied
    odd.copy_(s["q"])
    got = sv.paged_attention(odd, s["cache"], s["table"], s["lens"], s["new"], scale=0.2)
    assert torch.equal(got, want)
    # the drafter's view: batch expanded over one query
    one = s["q"][:1].expand(B, N, Hq, D)
    got = sv.paged_attention(one, s["cache"], s["table"], s["lens"], s["new"])
    check_attention(dict(s, q=one), past, new, got=got)


@pytest.mark.parametrize("N", [1, 6, 160])
def test_attention_many_sequences_of_mixed_lengths(N):
    B, Hq, Hkv, D, page = 300, 4, 2, 64, 16
    rng = random.Random(N)
    past = [rng.choice([0, 1, 15, 16, rng.randrange(400)]) for _ in range(B)]
    new = [rng.choice([0, 1, N, rng.randrange(N + 1)]) for _ in range(B)]
    s = paged(B, N, Hq, Hkv, D, BF, page, past, new, seed=N)
    check_attention(s, past, new)


@pytest.mark.parametrize("N,past", [(1, 40000), (6, 70001), (150, 30000)])
def test_attention_long_axis_is_joined_over_many_ctas(N, past):
    s = paged(1, N, 8, 1, 128, BF, 64, [past], [N], seed=past)
    check_attention(s, [past], [N])


@pytest.mark.parametrize("N", [1, 8, 140])
def test_attention_large_scores_and_one_key_rows(N):
    """Scores whose maximum grows along the keys, and far apart: the running maximum has to be followed."""
    past, D = 600, 128
    s = paged(1, N, 4, 1, D, BF, 16, [past], [N], seed=2)
    j = torch.arange(past + N, device="cuda")
    k = s["k"][0] * (1 + 20.0 * (j / (past + N)))[None, :, None]
    s["k"][0] = k.to(BF)
    ids = s["table"][0].long()[j // 16]
    s["cache"].k[ids, :, j % 16] = s["k"][0].transpose(0, 1)
    check_attention(s, [past], [N], scale=0.5)
    check_attention(s, [past], [N], window=1)


@pytest.mark.parametrize("N", [1, 8, 140])
def test_attention_bad_lengths_and_pages(N):
    B, page = 6, 16
    past, new = [100] * B, [N] * B
    s = paged(B, N, 8, 2, 64, BF, page, past, new, seed=9, poison=False)
    lens, cnt, table = s["lens"].clone(), s["new"].clone(), s["table"].clone()
    lens[1] = -1
    cnt[2] = N + 1
    cnt[3] = -2
    lens[4] = table.shape[1] * page - N + 1  # one position past the table
    table[5, 2] = s["cache"].pages  # one past the last page
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    got = sv.paged_attention(s["q"], s["cache"], table, lens, cnt, row_status=st)
    L, P = sv.ROW_BAD_LENGTH, sv.ROW_BAD_PAGE
    assert st.tolist() == [0, L, L, L, L, P]
    assert bool(got[1:6].isnan().all())
    w, t = ref.attention(s["q"][0], s["k"][0], s["v"][0], 100, 0.125, 0, BF)
    check(got[0], w, t)
    table[5, 2] = -(2 ** 31)
    st.zero_()
    got = sv.paged_attention(s["q"][5:], s["cache"], table[5:], lens[5:], cnt[5:], row_status=st[5:])
    assert st.tolist() == [0] * 5 + [P] and bool(got.isnan().all())


@pytest.mark.parametrize("N", [1, 8, 150])
def test_attention_is_repeatable_on_other_streams_and_in_graphs(N):
    past, new = [1000, 200], [N, N]
    s = paged(2, N, 8, 2, 128, BF, 32, past, new, seed=6)
    f = lambda **kw: sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], **kw)
    a = f()
    assert torch.equal(a, f())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = f(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(a, b)
    ws = torch.empty(sv.attention_workspace_size(2, N, 8, 2, 128), dtype=torch.uint8, device="cuda").fill_(255)
    assert torch.equal(a, f(workspace=ws))  # what a workspace holds before does not matter
    with pytest.raises(sv.SpecVerifyError):
        f(workspace=ws[:256])
    out = torch.zeros_like(a)
    with torch.cuda.stream(st):
        f(out=out)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(out=out)
    s["q"].copy_(torch.randn_like(s["q"]))
    graph.replay()
    check_attention(s, past, new, got=out)


@pytest.mark.parametrize("N", [1, 8, 150])
def test_attention_gives_up_a_wait_and_recovers(N):
    """A limit that no wait can keep: NaN and a status, and the next call is unaffected."""
    past, new = [3000, 200], [N, N]
    s = paged(2, N, 8, 2, 128, BF, 32, past, new, seed=6)
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    got = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], row_status=st, wait_limit_ns=1)
    # (a short sequence's waits may be over at the first look)
    assert st[0] == sv.ROW_INTERNAL and st[1] in (0, sv.ROW_INTERNAL)
    assert bool(got[0].isnan().any())
    st.zero_()
    check_attention(s, past, new, row_status=st)
    assert st.tolist() == [0, 0]


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,rot,page,order", [
    (1, 1, 1, 1, 64, 64, 16, "hnd"), (3, 5, 6, 2, 128, 128, 16, "nhd"), (2, 40, 5, 1, 128, 32, 48, "hnd"),
    (2, 7, 4, 4, 80, 16, 32, "hnd"), (2, 3, 3, 3, 256, 128, 64, "nhd"), (1, 300, 16, 8, 64, 32, 256, "hnd")])
def test_rotate_append_matches(B, N, Hq, Hkv, D, rot, page, order, inter, dtype):
    rng = random.Random(N)
    past = [rng.randrange(5000) for _ in range(B)]
    new = [N] + [rng.randrange(N + 1) for _ in range(B - 1)]
    s = paged(B, N, Hq, Hkv, D, dtype, page, [0] * B, [p + N for p in past], seed=1, order=order)
    scaling = dict(type="yarn", factor=4.0, original_length=2048) if rot == 128 else None
    table = sv.rotary_table(6000, rot, scaling=scaling)
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if scaling is None:
        freq, m = 10000.0 ** (-2 * j / rot), 1.0
    else:  # the frequencies are the table's own angle at position 1, in 64 bits
        ref_t = sv.rotary_table(2, rot, scaling=scaling)
        m = 0.1 * math.log(4.0) + 1.0
        at = lambda turns: rot * math.log(2048 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
        lo, hi = math.floor(at(32.0)), math.ceil(at(1.0))
        r = ((j - lo) / (hi - lo)).clamp(0, 1)
        freq = 10000.0 ** (-2 * j / rot)
        freq = freq * (1 - r) + freq / 4 * r
        assert torch.allclose(ref_t[1, 1].double(), freq.sin() * m, rtol=2.0 ** -22, atol=0)
    g = torch.Generator(device="cuda").manual_seed(5)
    k = torch.randn(B, N, Hkv, D, generator=g, device="cuda").to(dtype)
    v = torch.randn(B, N, Hkv, D, generator=g, device="cuda").to(dtype)
    cache = s["cache"]
    before_k, before_v = cache.k.clone(), cache.v.clone()
    lens = torch.tensor(past, dtype=torch.int32, device="cuda")
    cnt = torch.tensor(new, dtype=torch.int32, device="cuda")
    q = s["q"].clone()
    got = sv.rotate_append(q, k, v, table, cache, s["table"], lens, cnt, interleaved=inter)
    assert torch.equal(q, s["q"])
    h = ref.half_step(dtype)
    small = 2.0 ** -25 if dtype == HF else 0.0  # half the smallest float16
    touched = torch.zeros(cache.k.shape[0], page, dtype=torch.bool, device="cuda")
    for b in range(B):
        n = new[b]
        assert bool((got[b, n:] == 0).all())
        if n == 0:
            continue
        pos = past[b] + torch.arange(n, device="cuda")
        w, t = ref.rotate(q[b, :n], pos, freq, m, rot, inter)
        check(got[b, :n], w, t * (1 + h) + h * w.abs() + small, "q")
        w, t = ref.rotate(k[b, :n], pos, freq, m, rot, inter)
        ids = s["table"][b].long()[pos // page]
        check(cache.k[ids, :, pos % page], w, t * (1 + h) + h * w.abs() + small, "k")
        assert torch.equal(cache.v[ids, :, pos % page], v[b, :n])
        touched[ids, pos % page] = True
    keep = ~touched[:, None, :, None].expand_as(cache.k)
    eq = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert eq(cache.k[keep].contiguous(), before_k[keep].contiguous())
    assert eq(cache.v[keep].contiguous(), before_v[keep].contiguous())


def test_rotate_in_place_fused_and_streams():
    B, N, Hq, Hkv, D = 2, 6, 8, 2, 128
    s = paged(B, N, Hq, Hkv, D, BF, 16, [0, 0], [200, 200], seed=3)
    table = sv.rotary_table(400, 64)
    lens = torch.tensor([0, 190], dtype=torch.int32, device="cuda")
    qkv = torch.randn(B, N, (Hq + 2 * Hkv) * D, device="cuda").to(BF).view(B, N, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    want = sv.rotate_append(q, k, v, table, s["cache"], s["table"], lens)
    wk = s["cache"].k.clone()
    s["cache"].k.zero_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = sv.rotate_append(q, k, v, table, s["cache"], s["table"], lens, out=q, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert got is q and torch.equal(q, want)
    j = torch.arange(6, device="cuda")
    ids = s["table"][0].long()[j // 16]
    assert torch.equal(s["cache"].k[ids, :, j % 16], wk[ids, :, j % 16])


def test_rotate_bad_lengths_and_pages():
    B, N, page = 6, 4, 16
    s = paged(B, N, 4, 2, 64, BF, page, [0] * B, [100] * B, seed=3, poison=False)
    table = sv.rotary_table(90, 64)
    lens = torch.tensor([10, -1, 87, 10, 10, 86], dtype=torch.int32, device="cuda")  # 87 + 4 > 90
    cnt = torch.tensor([4, 4, 4, 5, 4, 4], dtype=torch.int32, device="cuda")
    pt = s["table"].clone()
    pt[4, 0] = -3
    k = torch.ones(B, N, 2, 64, dtype=BF, device="cuda")
    before = s["cache"].v.clone()
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    got = sv.rotate_append(s["q"], k, k, table, s["cache"], pt, lens, cnt, row_status=st)
    L, P = sv.ROW_BAD_LENGTH, sv.ROW_BAD_PAGE
    assert st.tolist() == [0, L, L, L, P, 0]
    for b in range(B):
        assert bool(got[b].isnan().all()) == (b in (1, 2, 3))
    changed = (s["cache"].v != before).any(-1).any(1).sum()
    assert int(changed) == 8  # sequences 0 and 5 wrote their four tokens


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_one_round_together():
    """Appends, attends, adjusts and verifies; the next round overwrites the rejected keys."""
    B, N, Hq, Hkv, D, page, V = 3, 4, 8, 2, 64, 16, 500
    torch.manual_seed(0)
    cache = sv.PagedCache(24, page, Hkv, D)
    pt = torch.randperm(24, device="cuda").to(torch.int32).view(B, 8)
    table = sv.rotary_table(128, D)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    history = sv.TokenHistory(B, V)
    head = torch.randn(Hq * D, V, device="cuda").to(BF) * 0.2
    keys, vals = [torch.zeros(Hkv, 0, D, device="cuda", dtype=BF) for _ in range(B)], None
    for step in range(4):
        q, k, v = (torch.randn(B, N, h, D, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
        past = lens.tolist()
        q = sv.rotate_append(q, k, v, table, cache, pt, lens)
        o = sv.paged_attention(q, cache, pt, lens, max_context=128)
        for b in range(B):
            kk = ref.gather(cache.k, pt[b], past[b] + N, page)
            assert torch.equal(kk[:, :past[b]], keys[b])  # what was accepted is still there
            w, t = ref.attention(q[b], kk, ref.gather(cache.v, pt[b], past[b] + N, page), past[b], 0.125, 0, BF)
            check(o[b], w, t)
        logits = (o.reshape(B, N, Hq * D) @ head).float()
        x = torch.randint(0, V, (B, N - 1), dtype=torch.int32, device="cuda")
        x[:, 0] = logits[:, 0].argmax(-1)
        z = sv.process_logits(logits, history=history, draft_tokens=x, repetition=1.0 + 1e-6, presence=0.0)
        res = sv.spec_verify(z, torch.randn(B, N - 1, V, device="cuda"), x, 0.0, seed=step)
        assert int(res["row_status"].abs().sum()) == 0
        history.add(res["out_tokens"])
        lens += res["accepted_len"] + 1
        keys = [ref.gather(cache.k, pt[b], int(lens[b]), page) for b in range(B)]
    assert int(history.counts.sum()) == int(lens.sum())


def test_short_calls_and_converted_calls_agree(monkeypatch):
    """Tensors that need no conversion go straight to the C entry points, and give what the general way gives."""
    from speculative_decoding_verification_20_gb300 import target as tg

    class General:
        logits = rotate = attention = staticmethod(lambda *a: None)

    class Direct:
        def __getattr__(self, name):
            def call(*a):
                res = getattr(short, name)(*a)
                assert res is not None, f"{name} was not served directly"
                return res
            return call

    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))
    B, N, Hq, Hkv, D, V = 3, 5, 8, 2, 128, 1000
    past, new = [40, 0, 77], [5, 3, 1]
    s = paged(B, N, Hq, Hkv, D, BF, 32, past, new, seed=8)
    k = torch.randn(B, N, Hkv, D, device="cuda").to(BF)
    table = sv.rotary_table(200, 64)
    d = logit_case(B, N, V, BF, seed=9)
    h = history_of(d, V, slots=4, of=[3, 0, 2])
    f32 = lambda x: torch.tensor(x, dtype=F32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    x, mask, bias = d["logits"].cuda(), ref.planes_of(d["mask"]).cuda(), bias_of(d)

    def calls(st):
        kw = dict(row_status=st)
        cache = sv.PagedCache.from_tensors(s["cache"].k.clone(), s["cache"].v.clone())
        q = sv.rotate_append(s["q"], k, k, table, cache, s["table"], s["lens"], s["new"], interleaved=True, **kw)
        o = sv.paged_attention(q, cache, s["table"], s["lens"], s["new"], window=50, scale=0.1, max_context=90, **kw)
        o2 = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], out=torch.empty_like(o))
        z = sv.process_logits(x, history=h, slots=i32([3, 0, 2]), draft_tokens=i32(d["draft"]), repetition=f32(d["rep"]),
                              frequency=f32(d["freq"]), presence=f32(d["pres"]), bias=bias, mask=mask, **kw)
        z2 = sv.process_logits(x[:, :1].contiguous(), slots=i32([9, 9, 9]))  # no history: its slots are not read
        return q, cache.k, o, o2, z, z2

    short = tg._short if not isinstance(tg._short, tg._Short) else None
    if short is None:
        tg._short.attention
        short = tg._short
    st = [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2)]
    monkeypatch.setattr(tg, "_short", Direct())
    a = calls(st[0])
    monkeypatch.setattr(tg, "_short", General())
    b = calls(st[1])
    assert all(same(p, r) for p, r in zip(a, b))
    assert torch.equal(st[0], st[1]) and not st[0].any()


def test_refusals_name_the_argument():
    s = paged(2, 3, 4, 2, 64, BF, 16, [20, 5], [3, 3], seed=2)
    host = sv.PagedCache.from_tensors(s["cache"].k.cpu(), s["cache"].v.cpu())
    k = torch.ones(2, 3, 2, 64, dtype=BF, device="cuda")
    table = sv.rotary_table(64, 64)
    at = lambda **kw: sv.paged_attention(**{**dict(q=s["q"], cache=s["cache"], page_table=s["table"],
                                                   cache_lens=s["lens"]), **kw})
    ro = lambda **kw: sv.rotate_append(**{**dict(q=s["q"], k=k, v=k, table=table, cache=s["cache"],
                                                 page_table=s["table"], cache_lens=s["lens"]), **kw})
    for call in (at, ro):
        for kw, error in ((dict(cache=host), ValueError), (dict(q=s["q"].to(HF)), TypeError),
                          (dict(q=s["q"][:1]), ValueError), (dict(page_table=s["table"][:1]), ValueError),
                          (dict(out=torch.empty(2, 3, 4, 64, device="cuda")), ValueError),
                          (dict(row_status=torch.zeros(2, device="cuda")), ValueError)):
            with pytest.raises(error):
                call(**kw)
    for kw in (dict(window=-1), dict(window="a"), dict(window=1.5), dict(scale="a"), dict(scale=math.nan),
               dict(q=s["q"][:, :, :3])):
        with pytest.raises((ValueError, TypeError, struct.error, sv.SpecVerifyError)):
            at(**kw)
    with pytest.raises(TypeError):
        ro(v=k.to(HF))
    with pytest.raises(ValueError):
        ro(table=table.double())
    x = torch.zeros(2, 3, 100, device="cuda")
    h = sv.TokenHistory(2, 99)
    for kw in (dict(history=h), dict(mask=torch.zeros(2, 3, device="cuda")), dict(out=x.to(BF)),
               dict(mask=torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda")),
               dict(draft_tokens=torch.zeros(2, 1, dtype=torch.int32, device="cuda")),
               dict(row_status=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            sv.process_logits(x, **kw)
    torch.cuda.synchronize()
