"""bf16 queries over the 8-bit cache: elements far below their row's largest."""
import math

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import drafter_ref as ref
from tests.test_cache8_gpu import built, empty_cache, hold, i32, near, tables  # noqa: F401  (built: the fixture)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N", [1, 26, 60, 200])
def test_small_elements_beside_a_large_one(N, D):
    """Keys are 0 where the query is large, so that its small element alone makes the scores: row i's is 2^-j of the largest
    (times 1.99, all eight bits), j from 20 on, under a scale that brings the scores to about 4.

    A row enters as fp16 with its largest element in [2^14, 2^15): steps are 2^-24 there at least, so that an element of
    eight bits is exact from 2^-31 of the power of two below the largest on, and off by up to 2^-39 of it under that."""
    L = 40 + N
    g = torch.Generator(device="cuda").manual_seed(N)
    for j0 in (20, 31, 32, 36, 41):
        table, pages = tables([40], [N], 16, N)
        cache = empty_cache(pages, 16, 1, D)
        k = torch.zeros(L, 1, D, device="cuda")
        k[:, 0, 5] = torch.randint(-15, 16, (L,), generator=g, device="cuda").float() / 16
        v = torch.randn(L, 1, D, generator=g, device="cuda")
        kk, vv = hold(cache, table, 0, 0, k, v)
        q = torch.zeros(1, N, 2, D, device="cuda")
        q[..., 0] = 1.5
        q[..., 5] = 1.9921875 * 2.0 ** -j0
        q[:, :, 1] *= 2.0 ** 60  # the same a power of two away
        q = q.to(BF)
        scale = 4.0 / 2.0 ** -j0
        for h in range(2):
            sc = scale * (2.0 ** -60 if h else 1.0)
            x = q[:, :, h:h + 1].contiguous()
            got = sv.paged_attention(x, cache, table, i32([40]), i32([N]), scale=sc)
            want, tol = ref.attention(x[0], kk, vv, 40, sc, 0, 0, eight=True)
            off = 0.0 if j0 <= 31 else 2.0 ** -39 * (2.0 ** 60 if h else 1.0) * sc * float(kk.abs().max())
            # scores off by `off` at most: weights over their sum by a factor e^(2 off), and so a mean of the values
            size = float(vv.abs().max())
            near(got[0], want, tol + size * math.expm1(2 * off), f"2^-{j0}, head {h}")
