"""Many small softmax weights beside a large one: what they add up to reaches the output."""
import math

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import target_ref as ref
from tests.test_target_gpu import check, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_20_gb300 import _build

    _build.build()
    sv.load_library()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gap", [10.0, 14.0, 17.5])
@pytest.mark.parametrize("N", [1, 12, 150])  # of 4 heads a cache head: one form of the kernel each
@pytest.mark.parametrize("first", [True, False])
def test_small_weights_add_up(N, gap, dtype, first):
    # as many units as CTAs, so that a row's keys are not spread over many running maxima
    B, Hkv, past, D, page = 40, 4, 16000, 64, 64
    L = past + N
    s = paged(B, N, 4 * Hkv, Hkv, D, dtype, page, [past] * B, [N] * B, seed=1, poison=False)
    at = 0 if first else past - 3  # the key with the large weight
    s["q"].zero_()
    s["q"][..., 0] = 8.0  # 1 / scale
    k = torch.zeros(Hkv, L, D, device="cuda")
    k[:, at, 0] = gap
    v = 1.0 + 0.25 * torch.randn(Hkv, L, D, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    v[:, at] = 0.0
    k, v = k.to(dtype), v.to(dtype)
    j = torch.arange(L, device="cuda")
    for b in range(B):
        ids = s["table"][b].long()[j // page]
        s["cache"].k[ids, :, j % page] = k.transpose(0, 1)
        s["cache"].v[ids, :, j % page] = v.transpose(0, 1)
    got = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"])
    w, t = ref.attention(s["q"][0], k, v, past, 1 / math.sqrt(D), 0, dtype)
    if dtype == torch.float16:
        # the smallest half step, 2^-25, stands for 2^-32 of the row's largest weight, and the sum is at least that
        # weight: instead of the 2^-24 that the general bound takes
        t = t - (2.0 ** -24 - 2.0 ** -32) * (v.double().abs().amax(1).repeat_interleave(4, 0) * L)
        assert float(t.max()) < float(w.abs().max()) / 8
    for b in (0, 17, B - 1):
        check(got[b], w, t, f"sequence {b}")
