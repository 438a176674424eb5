"""The 8-bit cache with scales that the caller set: any finite numbers, not powers of two."""
import math

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import drafter_ref as ref
from tests.test_cache8_gpu import bits, built, empty_cache, expected_append, i32  # noqa: F401  (built: the fixture)

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("D,inter", [(64, False), (160, True)])
def test_append_rounds_held_codes_once(D, inter):
    """A code times a scale of 24 bits has 28.  Each block's scale is chosen so that one of its codes times it is next to
    the middle between two codes of the new scale, within 32 bits' step of it, above or below."""
    B, H, past = 128, 4, 9
    g = torch.Generator().manual_seed(D)
    cache = empty_cache(B, 16, H, D)
    table = torch.randperm(B, generator=g).to(torch.int32)[:, None].cuda()
    for codes, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        c = torch.tensor([9.0, 10.0, 11.0, 13.0, 14.0, 15.0])[torch.randint(0, 6, (B, H), generator=g)]
        tie = 17.0 + 2.0 * torch.randint(0, 8, (B, H), generator=g)
        scales[:, :, 0] = (tie.double() / c.double()).float().cuda()
        x = torch.randint(-15, 16, (B, H, past, D), generator=g).float()
        x[:, :, ::2, ::3] = c[..., None, None] * torch.sign(x[:, :, ::2, ::3] + 0.5)
        codes[:, :, :past] = x.cuda().to(torch.float8_e4m3fn)
    k, v = (torch.randn(B, 1, H, D, generator=g).to(BF).cuda() for _ in "kv")
    k[..., 1], v[..., 3] = 300.0, -300.0  # (the new scale: 2^-1 or 1)
    # zeros under a scale beside which the new one vanishes
    cache.v[int(table[0, 0]), 0, :past] = torch.zeros(past, D, device="cuda").to(torch.float8_e4m3fn)
    cache.v_scales[int(table[0, 0]), 0, 0] = 3e38
    v[0, 0, 0] = 2.0 ** -60
    tab = sv.rotary_table(past + 1, 64)
    old = bits(cache.v).clone()
    want = expected_append(cache, table, [past] * B, [1] * B, k, v, tab, 64, inter)
    sv.rotate_append(torch.zeros_like(k), k, v, tab, cache, table, i32([past] * B), interleaved=inter)
    for t, w, name in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), want, ("k", "v", "k_scales", "v_scales")):
        assert torch.equal(bits(t), bits(w)), (name, int((bits(t) != bits(w)).sum()))
    assert not torch.equal(bits(cache.v), old)


def rounded(x, dtype):
    """float64 to the nearest bfloat16 or float16 number, ties to even, as float64."""
    p, least = (8, -133) if dtype == BF else (11, -24)
    _, e = torch.frexp(x)
    step = ref.power((e - p).clamp(min=least))
    y = torch.round(x / step) * step
    return torch.where(y.abs() > torch.finfo(dtype).max, torch.sign(y) * math.inf, y)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["ties", "any", "small", "large", "powers"])
def test_reading_back_rounds_once(dtype, kind):
    """Scales of 24 bits: such that a code times one is within 32 bits' step of the middle between two numbers of the
    result's type, and any, from products below the type's range to those above."""
    B, H, D, L = 40, 3, 64, 48
    g = torch.Generator().manual_seed(len(kind))
    cache = empty_cache(B * 3, 16, H, D)
    table = torch.randperm(3 * B, generator=g).to(torch.int32).reshape(B, 3).cuda()
    for codes, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        shape = (3 * B, H, 1)
        if kind == "ties":
            n = 8 if dtype == BF else 11
            c = torch.tensor([9.0, 10.0, 11.0, 13.0, 14.0, 15.0])[torch.randint(0, 6, shape, generator=g)]
            tie = 2.0 * torch.randint(1 << (n - 1), 1 << n, shape, generator=g) + 1
            s = (tie.double() / c.double()).float() * torch.exp2(torch.randint(-6, 3, shape, generator=g).float())
        else:
            lo, hi = dict(any=(-8, 5), small=(-149, -118) if dtype == BF else (-30, -14), powers=(-30, 7),
                          large=(110, 121) if dtype == BF else (6, 9))[kind]
            s = torch.exp2(torch.randint(lo, hi, shape, generator=g).float())
            if kind != "powers":
                s = s * (1 + torch.rand(shape, generator=g))
        scales.copy_(s)
        x = torch.randint(0, 256, codes.shape, generator=g).to(torch.uint8)
        codes.view(torch.uint8).copy_(torch.where(x & 0x7F == 0x7F, x - 1, x))
        if kind == "ties":
            codes[:, :, ::2] = c[..., None].cuda().to(torch.float8_e4m3fn)
    k, v = sv.read_cache(cache, table, i32([0] * B), L, dtype=dtype)
    assert k.dtype == v.dtype == dtype
    at = table.long()
    for got, codes, scales in ((k, cache.k, cache.k_scales), (v, cache.v, cache.v_scales)):
        x = codes[at].double() * scales[at][..., None].double()  # [B, 3, H, 16, D]
        want = rounded(x, dtype).transpose(2, 3).reshape(B, L, H, D)
        assert torch.equal(got.double(), want), int((got.double() != want).sum())


@pytest.mark.parametrize("heads,pages", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("blocks", [False, True])
def test_scales_may_share_memory_where_they_are_read(heads, pages, blocks):
    """One scale for all, for each page or for each head, expanded: as if it were written out.  blocks: one buffer for the
    blocks of a page, expanded over the others."""
    g = torch.Generator(device="cuda").manual_seed(3)
    P, H, S, D, B = 12, 2, 48, 64, 2
    make = lambda *s: 0.5 + torch.rand(*s, generator=g, device="cuda")
    shape = (P if pages else 1, H if heads else 1, S // 16 if blocks else 1)
    ks, vs = make(*shape).expand(P, H, S // 16), make(*shape).expand(P, H, S // 16)
    k, v = (torch.randn(P, H, S, D, generator=g, device="cuda").to(torch.float8_e4m3fn) for _ in "kv")
    shared = sv.PagedCache8.from_tensors(k, v, ks, vs)
    own = sv.PagedCache8.from_tensors(k, v, ks.clone(memory_format=torch.contiguous_format),
                                      vs.clone(memory_format=torch.contiguous_format))
    table = torch.randperm(P, generator=g, device="cuda").to(torch.int32).reshape(B, P // B)
    for N, lens in ((1, [17, 200]), (20, [100, 250]), (150, [0, 100])):
        q = torch.randn(B, N, 4, D, generator=g, device="cuda").to(BF)
        for kw in (dict(), dict(window=40, sinks=3)):
            want = sv.paged_attention(q, own, table, i32(lens), **kw)
            assert torch.equal(sv.paged_attention(q, shared, table, i32(lens), **kw), want)
        for x, y in zip(sv.read_cache(shared, table, i32(lens), N), sv.read_cache(own, table, i32(lens), N)):
            assert torch.equal(x, y)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = sv.paged_attention(q, shared, table, i32(lens), stream=st, **kw)
    st.synchronize()
    assert torch.equal(got, want)
    lens = i32(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sv.paged_attention(q, shared, table, lens, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    new = torch.randn(B, 3, H, D, generator=g, device="cuda").to(BF)
    with pytest.raises(ValueError, match="share a scale"):
        sv.rotate_append(new, new, new, sv.rotary_table(300, D), shared, table, i32([5, 60]))
