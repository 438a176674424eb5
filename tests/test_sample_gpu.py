"""Drawing tokens on a GPU against the 64-bit form (tests/drafter_ref.py)."""
import math

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import drafter_ref as ref
from tests.target_ref import U32

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# weights are off by 2^-40 of themselves and by 2^-45 of the largest: below V = 2^18 tokens borders move by
# 2^-40 + 2^18 * 2^-45 of the mass at most where every token is as likely as the largest (less otherwise)
NEAR = 2.0 ** -26


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_20_gb300 import _build

    _build.build()
    sv.load_library()


def rows(B, N, V, dtype, seed, kind="steep"):
    g = torch.Generator().manual_seed(seed)
    if kind == "steep":
        z = 12 - (1.1 + 1.6 * torch.rand(B, N, 1, generator=g)) * torch.log1p(V * torch.rand(B, N, V, generator=g))
    elif kind == "flat":
        z = 0.1 * torch.randn(B, N, V, generator=g)
    elif kind == "ties":  # few values
        z = torch.randint(-3, 3, (B, N, V), generator=g).float()
    elif kind == "equal":
        z = torch.full((B, N, V), -7.25)
    else:
        z = 4 * torch.randn(B, N, V, generator=g)
    if V > 8 and kind != "equal":
        z[:, :, torch.randperm(V, generator=g)[:V // 9]] = -math.inf
    u = torch.rand(B, N, generator=g)
    return z.to(dtype), u


def check(z, u, T, K, P, M, x=None, **kw):
    B, N, V = z.shape
    f32 = lambda xs, none: [none] * B if xs is None else torch.tensor(xs, dtype=F32).tolist()
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    tok, prob = sv.sample(z.cuda() if x is None else x, u.cuda(), T, K, P, M, row_status=st, **kw)
    assert st.tolist() == [0] * B and tok.dtype == torch.int32 and tok.shape == (B, N) and prob.dtype == F32
    T_, P_, M_ = f32(T, 1.0), f32(P, 1.0), f32(M, 0.0)
    K_ = [0] * B if K is None else K
    tok, prob = tok.cpu(), prob.cpu()
    for b in range(B):
        for i in range(N):
            t, p, near = ref.sample(z[b, i].double(), float(u[b, i]), T_[b], K_[b], P_[b], M_[b])
            assert near > NEAR, "the case is too close to a border"
            assert int(tok[b, i]) == t, (b, i, T_[b], K_[b], P_[b], M_[b], float(u[b, i]), float(prob[b, i]), p)
            # the ratio in 64 bits, rounded once
            assert abs(float(prob[b, i]) - p) <= p * U32 * 1.01


MIX = [(None, None, None, None), ([0.7] * 6, None, None, None), (None, [1, 2, 5, 50, 0, 40], None, None),
       (None, None, [0.9, 0.5, 0.05, 1.0, 0.99, 0.999], None), (None, None, None, [0.0, 1.0, 0.1, 0.01, 0.3, 1e-5]),
       ([0.0, 0.3, 0.8, 1.0, 1.3, 2.0], [0, 40, 7, 300, 50, 3], [0.9, 0.8, 1.0, 0.95, 0.7, 0.5],
        [0.0, 0.02, 0.1, 0.0, 0.01, 0.5]),
       ([1.0, 0.0, 3.0, 0.01, 1.5, 0.5], [0, 0, 5000, 20000, 0, 400], [0.95, 1.0, 0.9, 0.99, 0.3, 0.9999],
        [0.001, 0.0, 0.0, 0.0, 0.2, 0.0])]


@pytest.mark.parametrize("mix", range(len(MIX)))
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V,kind", [(1, "steep"), (7, "normal"), (33, "ties"), (2048, "flat"), (2049, "steep"),
                                    (5003, "ties"), (32000, "steep"), (50257, "normal"), (151936, "steep")])
def test_draws_match(V, kind, dtype, mix):
    z, u = rows(6, 2, V, dtype, seed=V + mix, kind=kind)
    check(z, u, *MIX[mix])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [262144, 100003])
def test_equal_and_flat_rows(V, dtype):
    """Borders by number alone: ties are cut by id, over all CTAs of a row; sums reach 2^62."""
    z, u = rows(6, 1, V, dtype, seed=5, kind="equal")
    u = torch.tensor([[0.0], [0.25], [0.5], [0.7500001], [1 - 2.0 ** -24], [2.0 ** -30]])
    T, K, P = 1.0, [0, 1, 1000, 70001, 0, 3], [1.0, 1.0, 0.5, 0.25, 0.7, 0.9]
    tok, prob = sv.sample(z.cuda(), u.cuda(), T, K, P)
    for b in range(6):
        n = K[b] or V
        n = math.ceil(float(torch.tensor(P[b], dtype=F32)) * n)
        assert int(tok[b, 0]) == int(float(u[b, 0]) * n), b
        assert abs(float(prob[b, 0]) - 1 / n) <= U32 / n
    z, u = rows(6, 1, V, dtype, seed=6, kind="flat")
    check(z, u, [1.0, 0.5, 2.0, 1.0, 1.0, 100.0], [0, 60000, 0, 3000, 90000, 0], [0.5, 0.9, 0.99999, 0.3, 1.0, 0.6],
          [0.0, 0.0, 0.0, 0.5, 0.7, 0.99])


def test_values_of_all_sizes():
    """Rows whose logits span the type: pivots by the order of floats as well as by value."""
    V = 40000
    g = torch.Generator().manual_seed(2)
    z = torch.exp2(torch.randint(-120, 100, (2, 1, V), generator=g).float()) * torch.randn(2, 1, V, generator=g).sign()
    z[1] = torch.where(torch.rand(1, V, generator=g) < 0.5, -0.0, 1e-42)
    z[0, 0, 77] = torch.finfo(F32).max
    u = torch.tensor([[0.9], [0.3333]])
    check(z, u, [1.0, 1.0], [30000, 25000], [0.999, 0.6], None)
    check(z, u, [1e30, 1.0], None, [0.7, 0.7], None)


def test_strides_and_alignment():
    V = 4999
    z, u = rows(5, 3, V, BF, seed=9)
    for off in (0, 1, 5):
        big = torch.full((3, 5, V + 11), math.nan, dtype=BF, device="cuda")
        x = big.permute(1, 0, 2)[:, :, off:off + V]
        x.copy_(z)
        check(z, u, [0.8] * 5, [50] * 5, [0.9] * 5, None, x=x)
        check(z, u, [0.8] * 5, None, [0.9] * 5, [0.01] * 5, x=x)
    y = torch.zeros(5, 3, V, 2, dtype=BF, device="cuda")[..., 0]  # converted
    y.copy_(z)
    check(z, u, [1.1] * 5, None, None, None, x=y)


def test_bad_rows():
    B, V = 12, 3000
    z, u = rows(B, 2, V, F32, seed=1)
    z[1, 0, 5] = math.nan
    z[2, 1, V - 1] = math.inf
    z[3, 0] = -math.inf
    u[4, 1], u[5, 0], u[6, 1] = 1.0, -0.1, math.nan
    T, K, P, M = [1.0] * B, [20] * B, [0.9] * B, [0.0] * B
    T[7], K[8], P[9], P[10], M[11] = -1.0, -1, 0.0, 1.1, math.nan
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    tok, prob = sv.sample(z.cuda(), u.cuda(), T, K, P, M, row_status=st)
    assert st.tolist() == [0, sv.ROW_NONFINITE, sv.ROW_NONFINITE, sv.ROW_NONFINITE, sv.ROW_BAD_UNIFORM, sv.ROW_BAD_UNIFORM,
                           sv.ROW_BAD_UNIFORM, sv.ROW_BAD_TEMPERATURE, sv.ROW_BAD_TOP_K, sv.ROW_BAD_TOP_P, sv.ROW_BAD_TOP_P,
                           sv.ROW_BAD_MIN_P]
    bad = [(1, 0), (2, 1), (3, 0), (4, 1), (5, 0), (6, 1)] + [(b, i) for b in range(7, 12) for i in range(2)]
    for b in range(B):
        for i in range(2):
            if (b, i) in bad:
                assert int(tok[b, i]) == -1 and math.isnan(float(prob[b, i]))
            else:
                t, p, near = ref.sample(z[b, i].double(), float(u[b, i]), 1.0, 20, float(torch.tensor(0.9, dtype=F32)), 0.0)
                assert near > NEAR and int(tok[b, i]) == t


def test_streams_graphs_and_many_rows():
    z, u = rows(300, 3, 3001, BF, seed=4)
    x, uu = z.cuda(), u.cuda()
    T = torch.full((300,), 0.9, device="cuda")
    K = torch.full((300,), 60, dtype=torch.int32, device="cuda")
    want = sv.sample(x, uu, T, K)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.sample(x, uu, T, K, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = sv.sample(x, uu, T, K)
    uu.copy_(1 - uu - 2.0 ** -25)
    want2 = sv.sample(x, uu, T, K)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap[0], want2[0]) and torch.equal(cap[1], want2[1]) and not torch.equal(want2[0], want[0])
    assert sv.sample(x[:0], uu[:0])[0].shape == (0, 3)


def test_draws_feed_verification():
    """Drafts from sample are what spec_verify takes them for: with the same logits on both sides all are accepted."""
    B, G, V = 64, 4, 5000
    z, u = rows(B, G + 1, V, F32, seed=8)
    z, u = z.cuda(), u.cuda()
    x, prob = sv.sample(z[:, :G], u[:, :G], 0.8, 40, 0.9)
    res = sv.spec_verify(z, z[:, :G].contiguous(), x, 0.8, None, 40, 0.9, seed=3)
    assert res["row_status"].tolist() == [0] * B
    assert res["accepted_len"].tolist() == [G] * B
    assert torch.equal(res["out_tokens"][:, :G], x) and bool((prob > 0).all())


def test_threads_and_rows_that_share_memory():
    """Calls of two threads on streams of their own; rows of logits that lie on one another."""
    import threading

    z, u = rows(20, 2, 9001, F32, seed=12)
    x, uu = z.cuda(), u.cuda()
    want = sv.sample(x, uu, 0.8, 30, 0.9)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(20):
            got = sv.sample(x, uu, 0.8, 30, 0.9, stream=s)
            s.synchronize()
            if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    one = x[:1, :1].expand(20, 2, 9001)
    tok, prob = sv.sample(one, uu, 0.8, None, 0.9)
    for b in range(20):
        for i in range(2):
            t, p, near = ref.sample(z[0, 0].double(), float(u[b, i]), float(torch.tensor(0.8, dtype=F32)), 0,
                                    float(torch.tensor(0.9, dtype=F32)), 0.0)
            assert near > NEAR and int(tok[b, i]) == t and abs(float(prob[b, i]) - p) <= p * U32 * 1.01


@pytest.mark.parametrize("V", [300, 70000])
def test_settings_at_the_ends_of_their_ranges(V):
    z, u = rows(6, 1, V, F32, seed=21)
    check(z, u, [1.0, 0.01, 1.0, 1.0, 1.0, 1000.0], [0, 0, V, V - 1, 1, 0], [1e-30, 1e-38, 1e-7, 1.0, 1e-40, 1 - 2.0 ** -24],
          [0.0, 0.0, 1e-30, 1e-40, 1.0, 1.0])
    u[:] = torch.tensor([[0.0], [1e-40], [2.0 ** -24], [1 - 2.0 ** -24], [1e-30], [2.0 ** -60]])
    tok, prob = sv.sample(z.cuda(), u.cuda(), 1.0, None, 0.999999, None)
    for b in range(6):  # (the first and the last kept token: the sums' ends, not between borders)
        w = torch.exp(z[b, 0].double() - z[b, 0].max().double())
        assert w[int(tok[b, 0])] > 0 and 0 < float(prob[b, 0]) <= 1
        if b != 3:
            assert int(tok[b, 0]) <= int((torch.cumsum(w, 0) > w.sum() * 2.0 ** -22).nonzero()[0, 0])
