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


@pytest.mark.parametrize("m,high,low,least", [(7.7, "0x1.01800p-13", "0x1.017ffep-13", "0x1.5cab2cp-6"),
                                              (4.1, "0x1.ca800p-13", "0x1.ca7ffep-13", "0x1.07ad8cp-3")])
def test_min_p_between_weights_that_are_out_of_order(m, high, low, least):
    """At temperature 2 the weight of `high` comes out a step of 2^-44 or two below that of `low`, though it is the larger
    logit, and min-p's border lies between the two.  The nucleus ends with `low`; every row still gets a token: min-p
    takes nothing above a cut that it leaves, so the last token is the greater logit's."""
    V = 4096
    from speculative_decoding_verification_20_gb300 import target as tg

    z = torch.full((1, 1, V), -20.0)
    z[0, 0, 10], z[0, 0, 5], z[0, 0, V - 1] = m, float.fromhex(low), float.fromhex(high)
    w = float(np.exp((float.fromhex(high) - float(np.float32(m))) / 2))
    tail = (V - 3) * float(np.exp((-20.0 - m) / 2))
    P = torch.tensor([(1 + 1.5 * w) / (1 + 2 * w + tail)], device="cuda")  # reached in the middle of `low`
    M = torch.tensor([float.fromhex(least)], device="cuda")
    T = torch.tensor([2.0], device="cuda")
    z = z.cuda()
    u = torch.tensor([[1 - 0.25 * w / (1 + 2 * w)]], device="cuda")
    tok = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((1,), -7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = tg._SAMPLE.pack(tg._SAMPLE.size, z.data_ptr(), 0, 1, 1, V, V, V, u.data_ptr(), 1, T.data_ptr(), 0, P.data_ptr(),
                           M.data_ptr(), tok.data_ptr(), prob.data_ptr(), st.data_ptr())
    assert sv.load_library().spec_verify_sample(args, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert st.tolist() == [0] and tok.tolist() == [V - 1]
    assert abs(float(prob[0]) - w / (1 + 2 * w)) < 1e-6
