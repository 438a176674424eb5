"""What rejected tokens leave in a block of the 8-bit cache: not its scale, but what its tokens lost under it."""
import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests import drafter_ref as ref
from tests.test_cache8_gpu import built, empty_cache, i32  # noqa: F401  (built: the fixture)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("loud", [4.0, 2.0 ** 10, 2.0 ** 16])
def test_tokens_beside_rejected_ones_keep_what_their_scale_leaves(loud):
    """Behind 4 tokens a call appends 3 that are accepted and 5 loud ones that are not, all in one block; the next call writes
    over the loud ones.  The scale is then what a cache has that never saw them.  A value was rounded under each scale that
    it met, by at most 2^-4 of itself or, below 2^-6 of the scale, 2^-10 of that."""
    D, H = 64, 2
    g = torch.Generator(device="cuda").manual_seed(int(loud))
    r = lambda n: torch.randn(1, n, H, D, generator=g, device="cuda").to(BF)
    tab = sv.rotary_table(32, D)
    tab[:, 0], tab[:, 1] = 1.0, 0.0  # (no rotation: keys and values alike)
    pt = i32([[0]])
    first, kept, gone, last = ((r(n), r(n)) for n in (4, 3, 5, 2))
    for x in last:
        x[..., 0] = 6.0  # (the largest of what is live in the end: both caches end with one scale)
    both = lambda a, b: tuple(torch.cat((x, loud * y), 1) for x, y in zip(a, b))
    caches = [empty_cache(1, 16, H, D) for _ in "ab"]
    for c in caches:
        sv.rotate_append(r(4), *first, tab, c, pt, i32([0]))
    before = [t.clone() for t in (caches[0].k_scales, caches[0].v_scales)]
    sv.rotate_append(r(8), *both(kept, gone), tab, caches[0], pt, i32([4]))
    sv.rotate_append(r(3), *kept, tab, caches[1], pt, i32([4]))
    under = [t.clone() for t in (caches[0].k_scales, caches[0].v_scales)]
    for c in caches:
        sv.rotate_append(r(2), *last, tab, c, pt, i32([7]))
    assert torch.equal(caches[0].k_scales, caches[1].k_scales) and torch.equal(caches[0].v_scales, caches[1].v_scales)
    got, clean = (sv.read_cache(c, pt, i32([0]), 9) for c in caches)
    for i, *scales in ((0, before[0], under[0], caches[0].k_scales), (1, before[1], under[1], caches[0].v_scales)):
        s0, s1, s2 = (t[0, :, 0].double()[:, None] for t in scales)
        assert bool((s1 > s2).all())
        x = torch.cat((first[i], kept[i], last[i]), 1)[0].double()
        off = torch.zeros_like(x)
        for sc, rows in ((s0, slice(0, 4)), (s1, slice(0, 7)), (s2, slice(0, 9))):
            off[rows] += torch.maximum(2.0 ** -4 * (x.abs() + off)[rows], 2.0 ** -10 * sc + 0 * x[rows])
        assert bool(((got[i][0].double() - x).abs() <= off).all())
        assert torch.equal(got[i][:, 7:], clean[i][:, 7:])  # written after them: nothing of them is left
        # exactly: rounded under s1, then under s2
        y = ref.round8(ref.round8(x[4:7] / s1) * s1 / s2) * s2
        assert torch.equal(got[i][0, 4:7].double(), y)
        if loud >= 2.0 ** 16:
            assert not torch.equal(got[i][:, :7], clean[i][:, :7])
