"""Drawing tokens where a draw falls next to a border: the weights' accuracy decides."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests.test_sample_gpu import built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.mark.parametrize("T", [0.45, 0.7, 1.0, 1.3, 5.0])
def test_draws_next_to_a_border(T):
    """Two tokens of weights w and 1, and the random number nearest to w / (1 + w): the first is drawn iff w (1 - u) > u.

    A weight is off by at most 2^-33.6 of itself and 0.54 steps of 2^-44; the margin asked for is 2^-33.5 and 2^-44.8 / w
    (float64's own error, some 2^-48 here, is in the difference)."""
    rng = np.random.default_rng(int(100 * T))
    T32 = np.float32(T)
    m = np.float32(rng.normal() * 8)
    x = (m + rng.uniform(-11, -2, 400000) * np.log(2) * T).astype(np.float32)
    w = np.exp((x.astype(np.float64) - float(m)) / float(T32))
    u = (w / (1 + w)).astype(np.float32)
    gap = (w * (1 - u.astype(np.float64)) - u) / u
    use = (np.abs(gap) > 2.0 ** -33.5 + 2.0 ** -44.8 / w) & (np.abs(gap) < 2.0 ** -30)
    n = int(use.sum())
    assert n > 1000
    z = torch.from_numpy(np.stack((x[use], np.full(n, m)), 1))[:, None].cuda()
    tok, prob = sv.sample(z, torch.from_numpy(u[use])[:, None].cuda(), T)
    want = torch.from_numpy(np.where(gap[use] > 0, 0, 1).astype(np.int32))
    assert torch.equal(tok[:, 0].cpu(), want), int((tok[:, 0].cpu() != want).sum())
