"""Attention with a window and sinks over the 16-bit cache, on a GPU (tests/drafter_ref.py)."""
import math

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import drafter_ref as ref
from tests.test_cache8_gpu import built, i32, near, paged8  # noqa: F401  (built: the fixture)
from tests.test_target_gpu import paged

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16

SHAPES = [(3, 1, 4, 1, 128, BF, 16, [0, 15, 900], [1, 1, 1]), (2, 8, 8, 2, 64, HF, 32, [700, 130], [8, 5]),
          (2, 12, 8, 4, 128, BF, 48, [1000, 60], [12, 12]), (2, 20, 10, 2, 64, BF, 16, [600, 129], [20, 3]),
          (1, 33, 3, 1, 128, HF, 128, [1300], [33]), (2, 130, 4, 2, 128, BF, 16, [500, 0], [130, 77]),
          (1, 400, 4, 2, 64, HF, 80, [333], [400])]


def check(s, past, new, window, sinks, got=None, **kw):
    D = s["q"].shape[3]
    if got is None:
        got = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], window=window, sinks=sinks, **kw)
    for b in range(s["q"].shape[0]):
        n = new[b]
        assert bool((got[b, n:] == 0).all())
        if n:
            near(got[b, :n], *ref.attention(s["q"][b, :n], s["k"][b].double(), s["v"][b].double(), past[b], 1 / math.sqrt(D),
                                            window, sinks), f"sequence {b}")
    return got


@pytest.mark.parametrize("window,sinks", [(1, 1), (37, 4), (128, 128), (100, 129), (200, 16), (65, 300), (1000, 7), (2, 10 ** 12)])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,dtype,page,past,new", SHAPES)
def test_sinks_match(B, N, Hq, Hkv, D, dtype, page, past, new, window, sinks):
    s = paged(B, N, Hq, Hkv, D, dtype, page, past, new, seed=N + window)
    check(s, past, new, window, sinks)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("N", [1, 10, 40, 150])
@pytest.mark.parametrize("window,sinks", [(50, 5), (130, 40), (300, 16)])
def test_pages_between_sinks_and_window_may_be_gone(N, window, sinks, eight):
    """Their entries are out of range, and what shares a page with visible positions may be NaN."""
    past, new, page = [1500], [N], 16
    make = paged8 if eight else paged
    s = make(1, N, 4, 1, 64, BF, page, past, new, seed=window)
    lo = 1500 + 1 - window
    for j in range(sinks, lo):
        p = int(s["table"][0, j // page])
        if p < 0:
            continue
        if eight:
            s["cache"].k.view(torch.uint8)[p, :, j % page] = 0x7F
            s["cache"].v.view(torch.uint8)[p, :, j % page] = 0x7F
        else:
            s["cache"].k[p, :, j % page] = math.nan
            s["cache"].v[p, :, j % page] = math.nan
    first, last = (sinks + page - 1) // page, lo // page
    s["table"][0, first:last] = 2 ** 31 - 1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], window=window, sinks=sinks, row_status=st)
    assert st.tolist() == [0]
    near(got[0], *ref.attention(s["q"][0], s["k"][0].double(), s["v"][0].double(), 1500, 1 / 8, window, sinks, eight=eight))


def test_sinks_without_effect_change_nothing():
    past, new = [700, 300], [9, 9]
    s = paged(2, 9, 8, 2, 128, BF, 16, past, new, seed=1)
    call = lambda **kw: sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], **kw)
    assert torch.equal(call(sinks=50), call())  # no window
    assert torch.equal(call(window=10000, sinks=50), call(window=10000))
    check(s, past, new, 10 ** 9, 10 ** 9)


def test_long_sequences_and_many_units():
    past, new = [70001, 5], [3, 3]
    s = paged(2, 3, 8, 2, 64, BF, 64, past, new, seed=2)
    check(s, past, new, 4096, 4)
    check(s, past, new, 20000, 3000, max_context=70004)
    past = [0, 100, 1000, 37] * 40
    s = paged(160, 2, 4, 2, 64, HF, 16, past, [2] * 160, seed=3)
    check(s, past, [2] * 160, 64, 20)
