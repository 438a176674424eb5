"""paged_attention with 33 to 128 query rows a cache head (new tokens x query heads sharing it), against its 64-bit
form: the key tiles of a unit go to two halves of a CTA in turn, and a CTA has one unit after the other."""
import math
import random

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import target_ref as ref
from tests.test_target_gpu import check, check_attention, paged

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_20_gb300 import _build

    _build.build()
    sv.load_library()


SHAPES = [  # B, N, Hq, Hkv, D, page, past, new, window
    (1, 33, 1, 1, 64, 16, [0], [33], 0),
    (2, 11, 6, 2, 128, 16, [0, 250], [11, 9], 0),
    (3, 9, 8, 2, 64, 48, [5, 0, 1000], [9, 0, 1], 0),
    (3, 12, 16, 4, 128, 48, [127, 128, 129], [12, 12, 12], 0),
    (2, 8, 16, 2, 64, 64, [700, 60], [8, 5], 100),
    (2, 64, 1, 1, 128, 32, [300, 2000], [64, 17], 5),
    (2, 100, 4, 4, 64, 256, [0, 900], [100, 77], 0),
    (2, 16, 16, 2, 128, 16, [0, 1111], [16, 16], 300),
    (1, 2, 64, 1, 128, 128, [4000], [2], 1),
    (4, 128, 2, 2, 64, 16, [3, 0, 511, 40], [128, 0, 100, 1], 0),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_shapes_match(shape, dtype):
    B, N, Hq, Hkv, D, page, past, new, window = shape
    s = paged(B, N, Hq, Hkv, D, dtype, page, past, new, seed=N + Hq)
    check_attention(s, past, new, window)


def lengths(kind, B, N, rng):
    """past[b], new[b] of a batch in which most units are one or two key tiles."""
    if kind == "short":
        past = [rng.randrange(1, 121 - N) for _ in range(B)]
    elif kind == "some longer":
        past = [rng.randrange(129, 600) if rng.random() < 0.1 else rng.randrange(1, 121 - N) for _ in range(B)]
    else:  # runs of one, two, four and eight short ones before a longer
        past = []
        while len(past) < B:
            past += [rng.randrange(1, 121 - N) for _ in range(rng.choice([1, 2, 4, 8]))] + [rng.randrange(140, 600)]
        past = past[:B]
    new = [rng.choice([N, N, N, 0, 1, rng.randrange(N + 1)]) for _ in range(B)]
    return past, new


@pytest.mark.parametrize("kind", ["short", "some longer", "runs"])
@pytest.mark.parametrize("N,group,D,dtype,page,window", [
    (11, 3, 128, BF, 16, 0), (12, 4, 64, HF, 48, 0), (8, 8, 128, HF, 16, 0), (8, 8, 64, BF, 48, 0),
    (16, 8, 128, BF, 48, 70), (32, 4, 64, HF, 16, 200), (9, 4, 128, BF, 16, 20)])
def test_many_short_units(N, group, D, dtype, page, window, kind):
    B, Hkv = 260, 4  # some seven units a CTA
    past, new = lengths(kind, B, N, random.Random(N * D))
    s = paged(B, N, Hkv * group, Hkv, D, dtype, page, past, new, seed=N)
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    a = check_attention(s, past, new, window, row_status=st)
    assert not st.any()
    b = sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], window=window)
    assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
def test_bad_lengths_and_pages(D):
    B, N, page = 200, 12, 16
    rng = random.Random(D)
    past = [rng.choice([rng.randrange(1, 100), rng.randrange(130, 400)]) for _ in range(B)]
    new = [N] * B
    s = paged(B, N, 16, 4, D, BF, page, past, new, seed=9, poison=False)
    lens, cnt, table = s["lens"].clone(), s["new"].clone(), s["table"].clone()
    want = [0] * B
    for b in range(0, B, 5):
        kind = b // 5 % 4
        if kind == 0:
            lens[b] = -1
        elif kind == 1:
            cnt[b] = N + 1
        elif kind == 2:
            lens[b] = table.shape[1] * page - N + 1  # one position past the table
        else:
            table[b, (past[b] + N - 1) // page] = s["cache"].pages if b % 40 == 15 else -5
        want[b] = sv.ROW_BAD_PAGE if kind == 3 else sv.ROW_BAD_LENGTH
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    got = sv.paged_attention(s["q"], s["cache"], table, lens, cnt, row_status=st)
    assert st.tolist() == want
    for b in range(B):
        if want[b]:
            assert bool(got[b].isnan().all()), b
        else:
            w, t = ref.attention(s["q"][b], s["k"][b], s["v"][b], past[b], D ** -0.5, 0, BF)
            check(got[b], w, t, f"sequence {b}")


def test_layouts_strides_scale_and_out():
    B, N, Hq, Hkv, D = 2, 12, 8, 2, 128
    past, new = [100, 260], [N, N - 3]
    s = paged(B, N, Hq, Hkv, D, BF, 32, past, new, seed=4, order="nhd")
    fused = torch.randn(B, N, Hq + 2 * Hkv, D, device="cuda").to(BF)  # q inside a fused projection
    fused[:, :, :Hq] = s["q"]
    out = torch.full((N, B, Hq, D), 7.0, dtype=BF, device="cuda").transpose(0, 1)
    got = sv.paged_attention(fused[:, :, :Hq], s["cache"], s["table"], s["lens"], s["new"], scale=0.2, out=out,
                             max_context=max(p + n for p, n in zip(past, new)))
    assert got is out
    check_attention(s, past, new, scale=0.2, got=got)


def test_large_scores_and_one_key_rows():
    """Scores whose maximum grows along the keys, and far apart: each half follows its own running maximum."""
    past, N, D = 600, 20, 128
    s = paged(1, N, 4, 1, D, BF, 16, [past], [N], seed=2)
    j = torch.arange(past + N, device="cuda")
    s["k"][0] = (s["k"][0] * (1 + 20.0 * (j / (past + N)))[None, :, None]).to(BF)
    s["cache"].k[s["table"][0].long()[j // 16], :, j % 16] = s["k"][0].transpose(0, 1)
    check_attention(s, [past], [N], scale=0.5)
    check_attention(s, [past], [N], window=1)


def test_other_streams_and_graphs():
    B, N = 90, 12
    rng = random.Random(3)
    past, new = [rng.randrange(1, 400) for _ in range(B)], [N] * B
    s = paged(B, N, 16, 4, 64, HF, 32, past, new, seed=6)
    f = lambda **kw: sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], **kw)
    a = f()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = f(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(a, b)
    out = torch.zeros_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(out=out)
    s["q"].copy_(torch.randn_like(s["q"]))
    graph.replay()
    check_attention(s, past, new, got=out)


def test_rows_of_a_tile_that_are_not_there():
    """Every count of rows around a warp's 32, one unit after the other."""
    B, N, Hkv, D = 128, 128, 2, 64
    past = [(7 * b) % 150 for b in range(B)]
    new = [b + 1 for b in range(B)]
    s = paged(B, N, Hkv, Hkv, D, BF, 16, past, new, seed=5)
    check_attention(s, past, new, scale=1 / math.sqrt(D))
