"""A NaN or infinity among the keys reaches the tokens that see its position, and no others."""
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


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N", [3, 8, 20, 90])  # of 4 heads a cache head: each form of the kernel
def test_keys_that_are_not_numbers(N, D, value):
    past, page, window = 300, 16, 37
    s = paged(1, N, 8, 2, D, torch.bfloat16, page, [past], [N], seed=N)
    for at, w, hit in ((past + N // 2, 0, range(N // 2, N)),     # one of the new tokens: itself and those behind it
                       (past + 1 - window, window, range(1))):   # leaves the window of the second token
        kept = s["k"][0][:, at].clone()
        want, tol = ref.attention(s["q"][0], s["k"][0], s["v"][0], past, 1 / math.sqrt(D), w, torch.bfloat16)
        place = (s["table"][0, at // page].long(), slice(None), at % page)
        s["cache"].k[place] = value
        got = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], window=w)[0]
        s["cache"].k[place] = kept
        free = [i for i in range(N) if i not in hit]
        check(got[free], want[free], tol[free])
        if math.isnan(value):
            assert bool(got[list(hit)].isnan().all())
