"""The 8-bit paged cache on a GPU: append, reading back, attention (tests/drafter_ref.py)."""
import math

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import drafter_ref as ref
from tests import target_ref

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
BLK = ref.BLOCK


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_20_gb300 import _build

    _build.build()
    sv.load_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def near(got, want, tol, what=""):
    got, want, tol = got.double().cpu(), want.cpu(), tol.cpu()
    over = ~((got - want).abs() <= tol)
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} off, worst {((got - want).abs() / tol)[over].max()}"


def bits(t):
    return t.contiguous().view(torch.uint8)


def empty_cache(pages, page, Hkv, D, order="hnd", poison=True):
    """Codes and scales that are NaN all over."""
    shape = (pages, Hkv, page, D) if order == "hnd" else (pages, page, Hkv, D)
    make = lambda: torch.full(shape, 0x7F if poison else 0, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    k, v = make(), make()
    if order == "nhd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    s = lambda: torch.full((pages, Hkv, page // BLK), math.nan if poison else 1.0, device="cuda")
    ks, vs = s(), s()
    if order == "nhd":  # scales in another order too
        ks, vs = (t.permute(1, 0, 2).contiguous().permute(1, 0, 2) for t in (ks, vs))
    return sv.PagedCache8.from_tensors(k, v, ks, vs)


def tables(past, new, page, seed, spare=3):
    need = [(p + n + page - 1) // page for p, n in zip(past, new)]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    t = torch.full((len(past), max(max(need), 1) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t.cuda(), pages


def hold(cache, table, b, first, k, v):
    """Writes values [L, H, D] (float64) to positions first .. of sequence b, quantised block by block; first a multiple
    of 16.  Returns what is held, float64 [H, L, D]."""
    L, page = k.shape[0], cache.page_size
    res = []
    for x, codes, scales in ((k, cache.k, cache.k_scales), (v, cache.v, cache.v_scales)):
        pad = torch.cat((x.double(), x.new_zeros((-L % BLK,) + x.shape[1:], dtype=torch.float64)))
        y, s = ref.quantise(pad.reshape(-1, BLK, *x.shape[1:]).transpose(1, 2))  # [blocks, H, 16, D], [blocks, H]
        j = first + torch.arange(L, device="cuda")
        pg = table[b].long()[j // page]
        flat = y.transpose(1, 2).reshape(-1, *x.shape[1:])[:L]
        codes[pg, :, j % page] = flat.float().to(torch.float8_e4m3fn)
        scales[pg, :, j % page // BLK] = s.repeat_interleave(BLK, 0)[:L].float()
        res.append((flat * s.repeat_interleave(BLK, 0)[:L, :, None]).transpose(0, 1))
    return res


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def expected_append(cache, table, past, new, k, v, tab, rot, inter):
    """Codes and scales after an append, from the definition, whole."""
    page = cache.page_size
    out = [cache.k.clone(), cache.v.clone(), cache.k_scales.clone(), cache.v_scales.clone()]
    for b, (p, n) in enumerate(zip(past, new)):
        if n == 0:
            continue
        kk = ref.rotate_exact(k[b, :n], tab[p:p + n], rot, inter)
        for x, codes, scales in ((kk, out[0], out[2]), (v[b, :n].double(), out[1], out[3])):
            for blk in range(p // BLK, (p + n - 1) // BLK + 1):
                j = torch.arange(blk * BLK, min((blk + 1) * BLK, p + n), device="cuda")
                pg, slot = int(table[b, blk * BLK // page]), j % page
                at = (slot // BLK)[0]
                old = codes[pg][:, slot].double() * scales[pg, :, at].double()[:, None, None]  # [H, m, D]
                fresh = x[(j - p).clamp(min=0)].transpose(0, 1)
                live = torch.where((j < p)[None, :, None], old, fresh)
                y, s = ref.quantise(live)
                same = (j < p)[None, :, None] & (s == scales[pg, :, at].double())[:, None, None]
                codes[pg, :, slot] = torch.where(same, codes[pg][:, slot].float(), y.float()).to(torch.float8_e4m3fn)
                scales[pg, :, at] = s.float()
    return out


CASES = [(1, 1, 4, 2, 128, 128, False, BF, 16, [0], [1], "hnd"), (3, 1, 4, 2, 64, 64, False, BF, 16, [15, 16, 31], [1, 1, 1], "hnd"),
         (3, 5, 8, 2, 128, 64, True, HF, 32, [13, 0, 100], [5, 0, 3], "nhd"),
         (2, 17, 2, 1, 96, 32, False, BF, 48, [47, 15], [17, 17], "hnd"), (2, 40, 3, 3, 256, 256, True, BF, 64, [7, 64], [40, 33], "nhd"),
         (1, 300, 2, 2, 128, 128, False, HF, 16, [5], [299], "hnd"), (2, 3, 2, 2, 16, 16, False, HF, 16, [1, 30], [3, 2], "hnd"),
         (2, 9, 5, 1, 240, 112, True, BF, 32, [3, 31], [9, 9], "hnd")]


@pytest.mark.parametrize("B,N,Hq,Hkv,D,rot,inter,dtype,page,past,new,order", CASES)
def test_append_codes_are_the_definitions(B, N, Hq, Hkv, D, rot, inter, dtype, page, past, new, order):
    g = torch.Generator(device="cuda").manual_seed(N + D)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * torch.exp2(
        4 * torch.rand(*s[:-1], 1, generator=g, device="cuda"))).to(dtype)
    q, k, v = r(B, N, Hq, D), r(B, N, Hkv, D), r(B, N, Hkv, D)
    table, pages = tables(past, new, page, seed=B + N)
    cache = empty_cache(pages, page, Hkv, D, order)
    for b, p in enumerate(past):  # what the first block holds, and rejected tokens behind it
        if p % BLK and new[b]:
            lo = p // BLK * BLK
            hold(cache, table, b, lo, 3 * r(BLK, Hkv, D), 40 * r(BLK, Hkv, D))
    tab = sv.rotary_table(max(p + n for p, n in zip(past, new)) + 1, rot)
    want = expected_append(cache, table, past, new, k, v, tab, rot, inter)
    got = sv.rotate_append(q, k, v, tab, cache, table, i32(past), i32(new), interleaved=inter)
    for t, w, name in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), want, ("k", "v", "k_scales", "v_scales")):
        assert torch.equal(bits(t), bits(w)), name
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    for b, (p, n) in enumerate(zip(past, new)):
        w, t = target_ref.rotate(q[b, :n], p + torch.arange(n, device="cuda"), 10000.0 ** (-2 * j / rot), 1.0, rot, inter)
        near(got[b, :n], w, t + target_ref.half_step(dtype) * w.abs() * (1 + 2 ** -6) + (2.0 ** -25 if dtype == HF else 0.0), "q")
        assert bool((got[b, n:] == 0).all())
    # again: the same positions, the same cache
    sv.rotate_append(q, k, v, tab, cache, table, i32(past), i32(new), interleaved=inter)
    for t, w in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), want):
        assert torch.equal(bits(t), bits(w))
    # and what it stands for
    first = i32([p // BLK * BLK for p in past])
    count = i32([p + n - p // BLK * BLK if n else 0 for p, n in zip(past, new)])
    kk, vv = sv.read_cache(cache, table, first, N + BLK, count, dtype=BF)
    for b, (p, n) in enumerate(zip(past, new)):
        c = int(count[b])
        j = int(first[b]) + torch.arange(c, device="cuda")
        pg = table[b].long()[j // page]
        for x, codes, scales in ((kk, cache.k, cache.k_scales), (vv, cache.v, cache.v_scales)):
            w = codes[pg, :, j % page].double() * scales[pg, :, j % page // BLK].double()[..., None]
            assert torch.equal(x[b, :c].double(), w)  # 4 bits and a power of two: exact in bf16
            assert bool((x[b, c:] == 0).all())


def test_append_special_values():
    D, page = 64, 16
    tab = sv.rotary_table(64, 64)
    cache = empty_cache(4, page, 1, D, poison=False)
    pt = i32([[2, 1, 0, 3]])
    v = torch.zeros(1, 16, 1, D, dtype=BF, device="cuda")
    k = torch.zeros_like(v)
    q = torch.zeros_like(v)
    sv.rotate_append(q, k, v, tab, cache, pt, i32([0]))  # zeros: scale 1
    assert float(cache.v_scales[2, 0, 0]) == 1.0 and bool((cache.v[2].float() == 0).all())
    v[0, 3, 0, 5], v[0, 4, 0, 6], v[0, 5, 0, 7], v[0, 6, 0, 8] = math.inf, -math.inf, math.nan, 1.0
    sv.rotate_append(q, k, v, tab, cache, pt, i32([0]))
    got = cache.v[2, 0].float()
    assert int(got.isnan().sum()) == 3 and got[3, 5].isnan() and got[4, 6].isnan() and got[5, 7].isnan()
    assert float(cache.v_scales[2, 0, 0]) == 2.0 ** -8 and float(got[6, 8]) == 256.0  # 1 <= 448 s
    for amax, s in ((448.0, 1.0), (450.0, 2.0), (224.0, 0.5), (1.75 * 2.0 ** 100, 2.0 ** 92), (2.0 ** -133, 2.0 ** -126),
                    (3.0e38, 2.0 ** 120)):
        v.zero_()
        v[0, 9, 0, 0] = -amax
        sv.rotate_append(q, k, v, tab, cache, pt, i32([0]))
        assert float(cache.v_scales[2, 0, 0]) == s, amax
        x = float(torch.tensor(amax, dtype=BF))
        assert float(cache.v[2, 0, 9, 0].float()) == -float(ref.round8(torch.tensor(x / s, dtype=torch.float64))), amax


def test_rejected_tokens_leave_no_trace():
    D, page = 128, 32
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda n, f=1.0: (f * torch.randn(1, n, 2, D, generator=g, device="cuda")).to(BF)
    tab = sv.rotary_table(100, D)
    pt = i32([[1, 0]])
    caches = [empty_cache(3, page, 2, D) for _ in "ab"]
    head, tail, loud = (r(20), r(20)), (r(5), r(5)), (r(9, 1000.0), r(9, 1000.0))
    for c in caches:
        sv.rotate_append(r(20), *head, tab, c, pt, i32([0]))
    sv.rotate_append(r(9), *loud, tab, caches[1], pt, i32([20]))  # a round whose tokens are rejected
    assert not torch.equal(caches[0].k_scales[1], caches[1].k_scales[1])
    for c in caches:
        sv.rotate_append(r(5), *tail, tab, c, pt, i32([20]))
    a, b = (sv.read_cache(c, pt, i32([0]), 25) for c in caches)
    scales = [c.k_scales[1].cpu() for c in caches]
    assert torch.equal(*scales)
    # what was small beside the loud tokens lost its last bits (below 2^-9 of their scale), nothing else
    assert torch.equal(a[0][:, 20:], b[0][:, 20:]) and torch.equal(a[1][:, 20:], b[1][:, 20:])
    top = max(float(x.float().abs().max()) for x in loud) * 2 ** 0.5
    lost = 2.0 ** -10 * 2 * top / 448
    assert float((a[0].float() - b[0].float()).abs().max()) <= lost and float((a[1].float() - b[1].float()).abs().max()) <= lost


def test_bad_lengths_and_pages():
    B, N, D, page = 6, 4, 64, 16
    tab = sv.rotary_table(40, D)
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda h: torch.randn(B, N, h, D, generator=g, device="cuda").to(BF)
    cache = empty_cache(9, page, 1, D, poison=False)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    table = i32([[0, 1, 2], [3, -1, 4], [5, 9, 6], [7, 7, 7], [7, 7, 7], [8, 8, 8]])
    lens, new = i32([0, 20, 14, -1, 10, 45]), i32([2, 4, 4, 1, 5, 4])
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = sv.rotate_append(r(2), r(1), r(1), tab, cache, table, lens, new, row_status=st)
    assert st.tolist() == [0, sv.ROW_BAD_PAGE, sv.ROW_BAD_PAGE] + [sv.ROW_BAD_LENGTH] * 3
    assert bool(q[3:].isnan().all()) and not bool(q[:3].isnan().any())
    touched = [0, 5]  # of sequence 2 the positions 14 and 15 lie on a good page
    for t, w in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), before):
        others = [p for p in range(9) if p not in touched]
        assert torch.equal(bits(t[others]), bits(w[others]))
        assert not torch.equal(bits(t[touched]), bits(w[touched]))
    st.zero_()
    k, v = sv.read_cache(cache, table, lens, N, new, row_status=st)
    assert st.tolist() == [0, sv.ROW_BAD_PAGE, sv.ROW_BAD_PAGE, sv.ROW_BAD_LENGTH, sv.ROW_BAD_LENGTH, sv.ROW_BAD_LENGTH]
    assert bool(k[3:].isnan().all()) and bool(v[1].isnan().all()) and not bool(k[0].isnan().any())
    assert bool(k[2, 2:].isnan().all()) and not bool(k[2, :2].isnan().any())
    sv.rotate_append(r(2)[:0], r(1)[:0], r(1)[:0], tab, cache, table[:0], lens[:0])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def paged8(B, N, Hq, Hkv, D, dtype, page, past, new, seed, order="hnd", scales="pow2"):
    """A cache whose unused rows, scales, pages and page ids are poison, and what it stands for."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    table, pages = tables(past, new, page, seed)
    cache = empty_cache(pages, page, Hkv, D, order)
    ks, vs = [], []
    for b, (p, n) in enumerate(zip(past, new)):
        L = p + n
        loud = lambda: torch.exp2(torch.randint(-3, 4, ((L + BLK - 1) // BLK, Hkv, 1), generator=g,
                                                device="cuda").float()).repeat_interleave(BLK, 0)[:L]
        x = [torch.randn(L, Hkv, D, generator=g, device="cuda"), torch.randn(L, Hkv, D, generator=g, device="cuda") * loud()]
        k, v = hold(cache, table, b, 0, *x) if L else (x[0].transpose(0, 1).double(), x[1].transpose(0, 1).double())
        if scales == "any" and L:  # any positive numbers, and a block of zeros by its scale
            j = torch.arange(L, device="cuda")
            pg = table[b].long()[j // page]
            for held, sc in ((k, cache.k_scales), (v, cache.v_scales)):
                f = 0.5 + torch.rand(Hkv, (L + BLK - 1) // BLK, generator=g, device="cuda")
                f[0, 0] = 0.0
                f = f.repeat_interleave(BLK, 1)[:, :L]
                new_s = (sc[pg, :, j % page // BLK] * f.T)
                old = sc[pg, :, j % page // BLK].double()
                sc[pg, :, j % page // BLK] = new_s
                held *= (new_s.double() / old).T[..., None]
        ks.append(k)
        vs.append(v)
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").to(dtype)
    return dict(q=q, k=ks, v=vs, cache=cache, table=table, lens=i32(past), new=i32(new))


def check8(s, past, new, window=0, sinks=0, scale=None, got=None, ratios=False, **kw):
    q = s["q"]
    D = q.shape[3]
    scale_ = 1 / math.sqrt(D) if scale is None else scale
    if got is None:
        got = sv.paged_attention(q, s["cache"], s["table"], s["lens"], s["new"], window=window, sinks=sinks, scale=scale, **kw)
    assert got.dtype == q.dtype
    for b in range(q.shape[0]):
        n = new[b]
        assert bool((got[b, n:] == 0).all()), f"sequence {b}: rows past its new tokens"
        if n:
            near(got[b, :n], *ref.attention(q[b, :n], s["k"][b], s["v"][b], past[b], scale_, window, sinks, eight=True,
                                            ratios=ratios), f"sequence {b}")


ATT = [(1, 1, 4, 1, 128, BF, 16, [0], [1]), (3, 1, 8, 2, 128, HF, 16, [0, 15, 700], [1, 1, 1]),
       (4, 5, 4, 2, 64, BF, 32, [0, 33, 127, 128], [5, 0, 3, 5]), (2, 8, 8, 2, 128, BF, 48, [1000, 250], [8, 7]),
       (2, 9, 20, 4, 64, HF, 16, [513, 95], [9, 9]), (2, 33, 4, 4, 128, BF, 64, [300, 2], [33, 20]),
       (1, 70, 8, 1, 128, HF, 128, [1234], [70]), (2, 300, 4, 2, 64, BF, 16, [77, 0], [300, 129]),
       (20, 2, 16, 8, 128, BF, 16, list(range(0, 400, 20)), [2] * 20), (2, 257, 6, 2, 128, BF, 32, [400, 129], [257, 256])]


@pytest.mark.parametrize("B,N,Hq,Hkv,D,dtype,page,past,new", ATT)
@pytest.mark.parametrize("order,scales", [("hnd", "pow2"), ("nhd", "any")])
def test_attention_matches(B, N, Hq, Hkv, D, dtype, page, past, new, order, scales):
    s = paged8(B, N, Hq, Hkv, D, dtype, page, past, new, seed=N + D, order=order, scales=scales)
    check8(s, past, new, ratios=scales == "any" and N * (Hq // Hkv) > 32)


@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 0), (100, 3), (130, 16), (200, 130), (64, 300), (500, 1), (3, 10 ** 12)])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,dtype,page,past,new",
                         [(3, 3, 8, 2, 128, BF, 16, [600, 10, 290], [3, 3, 2]), (2, 40, 8, 2, 64, HF, 48, [900, 70], [40, 39]),
                          (2, 200, 4, 2, 128, BF, 32, [777, 0], [200, 131])])
def test_attention_windows_and_sinks(B, N, Hq, Hkv, D, dtype, page, past, new, window, sinks):
    s = paged8(B, N, Hq, Hkv, D, dtype, page, past, new, seed=window)
    check8(s, past, new, window, sinks)


@pytest.mark.parametrize("N", [2, 30, 200])
def test_attention_scales_of_all_sizes(N):
    """Queries and scales far from 1, and values whose blocks grow along the sequence."""
    past, new = [500], [N]
    for dtype, qf, kf in ((BF, 1e20, 2.0 ** -40), (BF, 1e-25, 2.0 ** 60), (HF, 300.0, 2.0 ** -8)):
        s = paged8(1, N, 4, 1, 128, dtype, 32, past, new, seed=1)
        s["q"] = (s["q"].float() * qf).to(dtype)
        s["cache"].k_scales *= kf
        s["k"] = [x * kf for x in s["k"]]
        check8(s, past, new, scale=1 / (qf * kf * math.sqrt(128)))
    s = paged8(1, N, 4, 1, 128, BF, 32, past, new, seed=2)
    L = 500 + N
    up = torch.exp2((torch.arange((L + 15) // 16, device="cuda") // 2).float() - 12).repeat_interleave(16)[:L]
    j = torch.arange(L, device="cuda")
    pg = s["table"][0].long()[j // 32]
    s["cache"].v_scales[pg, 0, j % 32 // 16] = s["cache"].v_scales[pg, 0, j % 32 // 16] * up
    s["v"] = [s["v"][0] * up.double()[None, :, None]]
    check8(s, past, new)


@pytest.mark.parametrize("N", [1, 33, 150])
def test_attention_many_small_weights(N):
    """16000 keys of weight 2^-25 beside one of 1: they are a part of the result that does not vanish."""
    D, page, L = 64, 64, 16000 + N
    table, pages = tables([16000], [N], page, 0)
    cache = empty_cache(pages, page, 1, D)
    k = torch.zeros(L, 1, D, device="cuda")
    k[3, 0, 0] = 1.0
    v = torch.zeros(L, 1, D, device="cuda")
    v[:, :, 1] = 1.0
    v[3, :, 1] = 0.0
    v[3, :, 2] = 1.0
    kk, vv = hold(cache, table, 0, 0, k, v)
    q = torch.zeros(1, N, 1, D, dtype=BF, device="cuda")
    q[..., 0] = 25.0 * math.log(2)
    s = dict(q=q, k=[kk], v=[vv], cache=cache, table=table, lens=i32([16000]), new=i32([N]))
    check8(s, [16000], [N], scale=1.0)


@pytest.mark.parametrize("N", [2, 40, 200])
def test_attention_nan_keys_reach_who_sees_them(N):
    past, new = [200], [N]
    s = paged8(1, N, 2, 1, 64, BF, 16, past, new, seed=3)
    pos = 200 + N - 1  # the last token's own key
    codes = s["cache"].k.view(torch.uint8)
    codes[int(s["table"][0, pos // 16]), 0, pos % 16, 7] = 0x7F
    got = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"])
    assert bool(got[0, N - 1].isnan().all())
    s["k"][0][:, pos] = 0.0
    for b in range(1):
        w, t = ref.attention(s["q"][0, :N - 1], s["k"][0][:, :pos], s["v"][0][:, :pos], 200, 1 / 8, 0, 0, eight=True)
        near(got[0, :N - 1], w, t)


@pytest.mark.parametrize("N", [1, 40, 300])
def test_attention_bad_pages_and_lengths(N):
    past, new = [100, 200, 300, 5], [N, N, N, N]
    s = paged8(4, N, 4, 2, 64, BF, 16, past, new, seed=4)
    s["table"][1, 3] = s["cache"].pages
    s["lens"][2] = -3
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], row_status=st)
    assert st.tolist() == [0, sv.ROW_BAD_PAGE, sv.ROW_BAD_LENGTH, 0]
    assert bool(got[1].isnan().all()) and bool(got[2].isnan().all())
    for b in (0, 3):
        near(got[b], *ref.attention(s["q"][b], s["k"][b], s["v"][b], past[b], 1 / 8, 0, 0, eight=True))


def test_attention_streams_graphs_and_strides():
    past, new = [300, 40], [6, 5]
    s = paged8(2, 6, 8, 2, 128, BF, 16, past, new, seed=5)
    want = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"])
    check8(s, past, new, got=want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], max_context=400)
    s["lens"].copy_(i32([200, 33]))
    g.replay()
    torch.cuda.synchronize()
    s["k"] = [x[:, :p + 6] for x, p in zip(s["k"], [200, 33])]
    s["v"] = [x[:, :p + 6] for x, p in zip(s["v"], [200, 33])]
    s2 = dict(s, k=[s["k"][0], s["k"][1][:, :38]], v=[s["v"][0], s["v"][1][:, :38]])
    check8(s2, [200, 33], new, got=cap)
    big = torch.zeros(6, 2, 8, 136, dtype=BF, device="cuda")
    q2 = big.transpose(0, 1)[..., :128]
    q2.copy_(s["q"])
    out = torch.full((2, 6, 8, 144), 7.0, dtype=BF, device="cuda")
    got = sv.paged_attention(q2, s["cache"], s["table"], s["lens"], s["new"], out=out[..., :128])
    assert torch.equal(got, cap) and bool((out[..., 128:] == 7).all())


def test_a_drafting_step_end_to_end():
    """append -> attention with window and sinks -> logits -> sample -> verify, over the 8-bit cache, against the same in
    64 bits at the attention's output."""
    B, Hq, Hkv, D, V, G = 3, 4, 2, 64, 1000, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    cache = sv.PagedCache8(30, 16, Hkv, D)
    pt = torch.randperm(30, generator=torch.Generator().manual_seed(1))[:30].reshape(3, 10).to(torch.int32).cuda()
    tab = sv.rotary_table(160, D)
    head = (r(Hq * D, V) / 8).to(BF)
    lens = i32([0] * B)
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    history = sv.TokenHistory(B, V)

    def step(n):
        q, k, v = r(B, n, Hq, D).to(BF), r(B, n, Hkv, D).to(BF), r(B, n, Hkv, D).to(BF)
        q = sv.rotate_append(q, k, v, tab, cache, pt, lens, row_status=status)
        o = sv.paged_attention(q, cache, pt, lens, window=32, sinks=4, row_status=status)
        for b in range(B):
            p = int(lens[b])
            kk, vv = sv.read_cache(cache, pt[b:b + 1], i32([0]), p + n)
            near(o[b], *ref.attention(q[b], kk[0].double().transpose(0, 1), vv[0].double().transpose(0, 1), p, D ** -0.5, 32, 4,
                                      eight=True), f"sequence {b} at {p}")
        return sv.process_logits(o.reshape(B, n, -1)[:, -G - 1:] @ head, history=history, repetition=1.2, row_status=status)

    step(100)
    lens += 100
    for rnd in range(3):
        rows, toks = [], []
        start = lens.clone()
        for i in range(G):
            z = step(1)
            t, p = sv.sample(z, torch.rand(B, 1, generator=g, device="cuda"), 0.9, 50, 0.95, 0.0, row_status=status)
            rows.append(z)
            toks.append(t)
            lens += 1
        x = torch.cat(toks, 1)
        lens.copy_(start)
        z = step(G + 1)
        res = sv.spec_verify(z, torch.cat(rows, 1), x, 0.9, None, 50, 0.95, seed=rnd)
        history.add(res["out_tokens"])
        lens += res["accepted_len"] + 1
        status |= res["row_status"]
    assert status.tolist() == [0] * B


def test_append_next_to_borders_between_codes():
    """Rotated keys within 2^-25 of the middle between two codes, where the products' errors are steps of their sum, and
    such values drawn at random."""
    h = float.fromhex
    D = 32
    cases = [("0x1.13cp-1", "-0x1.2a4p-7", "0x1.c55fb2p-1", "0x1.dbcc8ep-2"), ("0x1.4ep+1", "0x1.2p-1", "0x1.c74276p-2", "0x1.ca9db4p-1"),
             ("-0x1.10cp+0", "-0x1.5b8p+1", "-0x1.bae2fap-3", "0x1.f3e27cp-1")]
    rng = torch.Generator().manual_seed(5)
    pairs = [tuple(map(h, c)) for c in cases]
    # b chosen so that a c - b s, or b c + a s, falls next to 17/16, 19/16, ... of a power of two
    while len(pairs) < 16 * 16 * 40:
        a, t = float(torch.randn((), generator=rng).half()), float(torch.rand((), generator=rng)) * 6.28
        c, s = float(torch.tensor(math.cos(t), dtype=F32)), float(torch.tensor(math.sin(t), dtype=F32))
        mid = (17 + 2 * int(torch.randint(0, 8, (), generator=rng))) / 16 * 2.0 ** -int(torch.randint(0, 4, (), generator=rng))
        b = float(torch.tensor((a * c - mid) / s).half())
        if abs(b) < 8 and abs(s) > 0.05:  # the sine that brings the middle nearest
            s = float(torch.tensor((a * c - mid) / b, dtype=F32)) if b else s
            if abs(s) < 1:
                pairs.append((a, b, c, s))
    n = len(pairs) // 16
    x = torch.tensor(pairs, dtype=torch.float64).reshape(n, 16, 4)
    k = torch.zeros(1, n, 1, D, dtype=HF, device="cuda")
    k[0, :, 0, :16], k[0, :, 0, 16:] = x[:, :, 0].to(HF), x[:, :, 1].to(HF)
    tab = torch.stack((x[:, :, 2].float(), x[:, :, 3].float()), 1).cuda()
    for inter in (False, True):
        kk = k if not inter else torch.stack((k[..., :16], k[..., 16:]), -1).flatten(-2)
        table, pages = tables([0], [n], 16, 0)
        cache = empty_cache(pages, 16, 1, D)
        want = expected_append(cache, table, [0], [n], kk, kk, tab, D, inter)
        sv.rotate_append(torch.zeros_like(kk), kk, kk, tab, cache, table, i32([0]), i32([n]), interleaved=inter)
        for t, w, name in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), want, ("k", "v", "k_scales", "v_scales")):
            assert torch.equal(bits(t), bits(w)), name
