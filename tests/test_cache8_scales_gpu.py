"""The 8-bit cache with scales that the caller set: any finite numbers, not powers of two."""
import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests.test_cache8_gpu import bits, built, empty_cache, expected_append, i32  # noqa: F401  (built: the fixture)

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("D,inter", [(64, False), (160, True)])
def test_append_rounds_held_codes_once(D, inter):
    """A code times a scale of 24 bits has 28.  Each block's scale is chosen so that one of its codes times it is next to
    the middle between two codes of the new scale, within 32 bits' step of it, above or below."""
    B, H, past = 128, 4, 9
    g = torch.Generator().manual_seed(D)
    cache = empty_cache(B, 16, H, D)
    table = torch.randperm(B, generator=g).to(torch.int32)[:, None].cuda()
    for codes, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        c = torch.tensor([9.0, 10.0, 11.0, 13.0, 14.0, 15.0])[torch.randint(0, 6, (B, H), generator=g)]
        tie = 17.0 + 2.0 * torch.randint(0, 8, (B, H), generator=g)
        scales[:, :, 0] = (tie.double() / c.double()).float().cuda()
        x = torch.randint(-15, 16, (B, H, past, D), generator=g).float()
        x[:, :, ::2, ::3] = c[..., None, None] * torch.sign(x[:, :, ::2, ::3] + 0.5)
        codes[:, :, :past] = x.cuda().to(torch.float8_e4m3fn)
    k, v = (torch.randn(B, 1, H, D, generator=g).to(BF).cuda() for _ in "kv")
    k[..., 1], v[..., 3] = 300.0, -300.0  # (the new scale: 2^-1 or 1)
    # zeros under a scale beside which the new one vanishes
    cache.v[int(table[0, 0]), 0, :past] = torch.zeros(past, D, device="cuda").to(torch.float8_e4m3fn)
    cache.v_scales[int(table[0, 0]), 0, 0] = 3e38
    v[0, 0, 0] = 2.0 ** -60
    tab = sv.rotary_table(past + 1, 64)
    old = bits(cache.v).clone()
    want = expected_append(cache, table, [past] * B, [1] * B, k, v, tab, 64, inter)
    sv.rotate_append(torch.zeros_like(k), k, v, tab, cache, table, i32([past] * B), interleaved=inter)
    for t, w, name in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), want, ("k", "v", "k_scales", "v_scales")):
        assert torch.equal(bits(t), bits(w)), (name, int((bits(t) != bits(w)).sum()))
    assert not torch.equal(bits(cache.v), old)
