"""Edges of the 8-bit cache, of sinks and of drawing tokens: caches and logits past 32-bit offsets, queries that are not
finite beside others, blocks of zeros beside small values."""
import math

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import drafter_ref as ref
from tests.test_cache8_gpu import bits, built, check8, empty_cache, expected_append, hold, i32, near, paged8, tables  # noqa: F401
from tests.test_target_gpu import paged

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def test_a_cache_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes, and whose scales more than 2^28 numbers, behind the first."""
    H, S, D = 4, 16, 128
    pages = (1 << 32) // (H * S * D) + 40
    mem = [torch.empty(pages, H, S, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"]
    scales = [torch.empty(pages * 128, device="cuda").as_strided((pages, H, 1), (128, 2, 1)) for _ in "kv"]
    big = sv.PagedCache8.from_tensors(*mem, *scales)
    past, new, N = [100, 37], [9, 5], 9
    table = torch.tensor([[pages - 1 - 2 * i for i in range(8)], [pages - 2 - 2 * i for i in range(8)]], dtype=torch.int32,
                         device="cuda")
    table[0, 2], table[1, 1] = 0, 1
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda n, h: torch.randn(2, n, h, D, generator=g, device="cuda").to(BF)
    tab = sv.rotary_table(128, D)
    small = sv.PagedCache8(16, S, H, D)
    few = torch.arange(16, device="cuda").to(torch.int32).reshape(2, 8)
    k, v = r(112, H), r(112, H)
    for c, t in ((big, table), (small, few)):
        sv.rotate_append(torch.zeros_like(k), k, v, tab, c, t, i32([0, 0]), i32(past))
    q, k, v = r(N, 8), r(N, H), r(N, H)
    out = []
    for c, t in ((big, table), (small, few)):
        x = sv.rotate_append(q, k, v, tab, c, t, i32(past), i32(new))
        out.append([x, *sv.read_cache(c, t, i32([0, 0]), 112, i32([109, 42])),
                    sv.paged_attention(x, c, t, i32(past), i32(new)),
                    sv.paged_attention(x, c, t, i32(past), i32(new), window=30, sinks=20),
                    *(sv.paged_attention(x[:, :1].expand(2, n, 8, D).contiguous(), c, t, i32([5, 0])) for n in (37, 110))])
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_logits_past_32_bits(dtype):
    V, far = 5003, (1 << 32) + 8 * 13
    mem = torch.empty(far + (1 << 31) + V + 77, dtype=dtype, device="cuda")
    z = mem.as_strided((2, 2, V), (far, (1 << 31) + 77, 1))
    g = torch.Generator(device="cuda").manual_seed(1)
    z.copy_(3 * torch.randn(2, 2, V, generator=g, device="cuda"))
    u = torch.rand(2, 2, generator=g, device="cuda")
    for kw in (dict(top_k=40, top_p=0.9), dict(top_p=0.9), dict(top_k=4000), dict(min_p=0.01), dict(temperature=0.0)):
        for a, b in zip(sv.sample(z, u, **kw), sv.sample(z.clone(memory_format=torch.contiguous_format), u, **kw)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("eight,dtype", [(True, BF), (True, HF), (False, BF)])
@pytest.mark.parametrize("N", [2, 7, 20, 150])
def test_queries_that_are_not_finite_reach_no_other_row(N, eight, dtype, value):
    past, new = [300, 40], [N, N]
    s = (paged8 if eight else paged)(2, N, 4, 2, 64, dtype, 16, past, new, seed=N)
    call = lambda: sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], window=250, sinks=9)
    want = call()
    bad = [(0, 0, 1), (1, N - 1, 3), (1, N // 2, 0)]
    for b, i, h in bad:
        s["q"][b, i, h, 5] = value
    got = call()
    for b, i, h in bad:
        assert bool(got[b, i, h].isnan().all())
        got[b, i, h] = want[b, i, h]
    assert torch.equal(got, want)


@pytest.mark.parametrize("N", [1, 8, 30, 100])
@pytest.mark.parametrize("loud", [0, -8, -16, -22])
def test_blocks_of_zeros_count_with_their_scale(N, loud):
    """A block of zeros has scale 1.  Beside it values of size 2^loud are off by what the largest scale leaves them: up to 32
    rows a cache head a weight times its scale is off by 2^-25 where the row's largest weight is 2^7 or more, which is 448 *
    2^-32 of a value at most for each of L keys; above, a value is off by half a step of fp16, 2^-25 of 2^7 (the quotients
    of the scales are powers of two, above 2^-31, and exact)."""
    D, L, dtype = 64, 200 + N, BF
    table, pages = tables([200], [N], 16, 0)
    cache = empty_cache(pages, 16, 1, D)
    g = torch.Generator(device="cuda").manual_seed(N)
    k = torch.randn(L, 1, D, generator=g, device="cuda")
    v = 2.0 ** loud * torch.randn(L, 1, D, generator=g, device="cuda")
    v[32:64] = 0.0
    kk, vv = hold(cache, table, 0, 0, k, v)
    assert float(cache.v_scales[int(table[0, 2]), 0, 0]) == 1.0
    q = torch.randn(1, N, 4, D, generator=g, device="cuda").to(dtype)
    got = sv.paged_attention(q, cache, table, i32([200]), i32([N]))
    want, tol = ref.attention(q[0], kk, vv, 200, 1 / 8, 0, 0, eight=True)
    near(got[0], want, tol + 2.0 ** -32 * (448 * L if N * 4 <= 32 else 1))
