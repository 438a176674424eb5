"""Waits of the attention kernels that run out: a row is right or NaN, and a sequence with NaN rows says so."""
import math
import random

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import target_ref as ref
from tests.test_target_gpu import check_attention, paged

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_20_gb300 import _build

    _build.build()
    sv.load_library()


# rows a cache head: 2 and 24 (warp-wide products), 48 and 128 (one row tile), 280 (two row tiles)
@pytest.mark.parametrize("N,group,D", [(1, 2, 64), (6, 4, 128), (12, 4, 64), (12, 4, 128), (32, 4, 128), (70, 4, 128)])
def test_rows_are_right_or_nan(N, group, D):
    Hkv, B = 2, 40
    rng = random.Random(N)
    past = [rng.choice([rng.randrange(1, 90), rng.randrange(130, 500), rng.randrange(2000, 3000)]) for _ in range(B)]
    new = [N] * B
    s = paged(B, N, Hkv * group, Hkv, D, BF, 32, past, new, seed=6)
    want = [ref.attention(s["q"][b], s["k"][b], s["v"][b], past[b], 1 / math.sqrt(D), 0, BF) for b in range(B)]
    w, t = torch.stack([x for x, _ in want]), torch.stack([x for _, x in want])
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    gave_up = 0
    for limit in [1] * 10 + [1000, 1500, 2000, 3000, 4000, 6000, 8000, 12000, 16000, 25000] * 3:  # ns
        st.zero_()
        got = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], row_status=st, wait_limit_ns=limit)
        nan = got.isnan()
        assert bool((((got.double() - w).abs() <= t) | nan).all()), limit
        assert torch.equal(nan.any(-1), nan.all(-1)), limit
        flagged = st != 0
        assert bool((st[flagged] == sv.ROW_INTERNAL).all()), limit
        assert not bool((nan.flatten(1).any(1) & ~flagged).any()), limit
        gave_up += int(flagged.any())
    assert gave_up >= 10  # a limit of one look is not kept by a cold start
    st.zero_()
    check_attention(s, past, new, row_status=st)
    assert not st.any()
