"""Attention over the 8-bit cache: many units a CTA, and waits that run out."""
import math
import random

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import drafter_ref as ref
from tests.test_cache8_gpu import built, check8, paged8  # noqa: F401  (built: the fixture)

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("kind", ["short", "mixed", "window"])
@pytest.mark.parametrize("N,group,D,dtype,page", [(2, 4, 128, BF, 16), (7, 4, 64, HF, 32), (12, 4, 128, BF, 48),
                                                  (17, 7, 64, BF, 16), (70, 4, 128, HF, 64)])
def test_many_units(N, group, D, dtype, page, kind):
    Hkv, B = 4, 90
    rng = random.Random(N)
    past = [rng.randrange(0, 90) if kind == "short" else rng.choice([0, 1, rng.randrange(200), rng.randrange(100, 1500)])
            for _ in range(B)]
    new = [rng.choice([0, 1, N, N, N]) for _ in range(B)]
    s = paged8(B, N, Hkv * group, Hkv, D, dtype, page, past, new, seed=N)
    check8(s, past, new, *((150, 20) if kind == "window" else (0, 0)))


@pytest.mark.parametrize("N,group,D", [(1, 2, 64), (6, 4, 128), (12, 4, 64), (12, 4, 128), (32, 4, 128), (70, 4, 128)])
def test_rows_are_right_or_nan_when_waits_run_out(N, group, D):
    Hkv, B = 2, 40
    rng = random.Random(N)
    past = [rng.choice([rng.randrange(1, 90), rng.randrange(130, 500), rng.randrange(2000, 3000)]) for _ in range(B)]
    new = [N] * B
    s = paged8(B, N, Hkv * group, Hkv, D, BF, 32, past, new, seed=6)
    want = [ref.attention(s["q"][b], s["k"][b], s["v"][b], past[b], 1 / math.sqrt(D), 0, 0, eight=True) for b in range(B)]
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
    check8(s, past, new, row_status=st)
    assert not st.any()
