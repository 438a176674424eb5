"""Bit planes of process_logits whose last words have bits past the vocabulary."""
import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_20_gb300 import _build

    _build.build()
    sv.load_library()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 31, 33, 100, 2047, 8191, 8193, 32001])
@pytest.mark.parametrize("skew", [0, 1, 7])
def test_bits_past_the_vocabulary_are_ignored(V, skew, dtype):
    B, N, pad = 3, 2, 200
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(B, N, V, generator=g, device="cuda").to(dtype)
    room = torch.full((B, N, V + pad), 7.0, dtype=dtype, device="cuda")
    src, dst = room.clone()[:, :, skew:skew + V], room[:, :, skew:skew + V]
    src.copy_(x)
    h = sv.TokenHistory(B + 1, V)  # (the last slot's neighbour is there to be read by mistake)
    h.load(torch.randint(0, V, (B + 1, 40), generator=g, device="cuda", dtype=torch.int32))
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, (V + 31) // 32), generator=g, device="cuda", dtype=torch.int32)
    call = lambda out: sv.process_logits(src, history=h, repetition=1.5, frequency=0.25, presence=0.5, mask=mask, out=out)
    want = call(torch.empty(B, N, V, dtype=dtype, device="cuda"))
    t = torch.arange(32 * h.words, device="cuda").view(h.words, 32)
    past = ((t >= V).long() << torch.arange(32, device="cuda")).sum(1)
    h.seen |= torch.where(past >= 2 ** 31, past - 2 ** 32, past).to(torch.int32)
    assert torch.equal(call(dst), want)
    assert bool((room[:, :, :skew] == 7).all()) and bool((room[:, :, skew + V:] == 7).all())
