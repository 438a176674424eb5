"""Refusals of the 8-bit cache, of sinks and of sampling, without a GPU: the C entry points return before they
enqueue anything, and the binding raises."""
import math
import os
import subprocess

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from speculative_decoding_verification_20_gb300 import target as tg

GOOD = 0x10000  # never dereferenced: the checks come first
CACHE = dict(k_pages=GOOD, v_pages=GOOD, pages=8, page_size=32, kp=4096, kh=2048, ks=64, vp=4096, vh=2048, vs=64,
             page_table=GOOD, pt_stride=4, pages_per_seq=4, cache_lens=GOOD, num_new=0)
SCALES = dict(sk=GOOD, sv=GOOD, skp=4, skh=2, svp=4, svh=2)
BAD_SCALES = [dict(sv=0), dict(sk=GOOD + 2), dict(skp=-1), dict(skh=1), dict(svh=0), dict(svp=1)]
BAD_CACHES = [dict(k_pages=0), dict(v_pages=GOOD + 8), dict(pages=0), dict(page_size=8), dict(page_size=24), dict(ks=72),
              dict(ks=48), dict(kh=1032), dict(page_table=0), dict(cache_lens=0), dict(vp=-16)]


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_20_gb300 import _build

    _build.build()
    return sv.load_library()


def pack(fmt, base, kw):
    d = dict(base)
    for k in kw:
        assert k in d, k
    d.update(kw)
    if d["size"] is None:
        d["size"] = fmt.size
    return fmt.pack(*d.values())


def test_structures_match_the_header(lib, tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "s.c"
    src.write_text('#include "spec_verify_target.h"\n#include <stdio.h>\nint main(void){printf("%zu %zu %zu %zu",'
                   "sizeof(sv_rotate_options),sizeof(sv_attention_options),sizeof(sv_read_args),sizeof(sv_sample_args));"
                   "return 0;}\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I" + os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert sizes == [tg._ROTATE_OPTIONS.size, tg._ATTENTION_OPTIONS.size, tg._READ.size, tg._SAMPLE.size]


def test_sample_refusals(lib):
    base = dict(size=None, logits=GOOD, dtype=0, B=2, N=3, V=100, sb=300, sn=100, u=GOOD, us=3, t=0, k=0, p=0, m=0, tok=GOOD,
                prob=0, status=0)
    f = lambda **kw: lib.spec_verify_sample(pack(tg._SAMPLE, base, kw), None)
    assert lib.spec_verify_sample(None, None) == -1
    assert f(size=8) == -1
    assert f(B=0) == 0
    assert f(dtype=2) == -2
    assert f(N=0) == -1
    assert f(V=0) == -1
    assert f(V=262145) == -4
    assert f(B=1 << 20, N=1 << 10) == -4
    for kw in (dict(logits=0), dict(u=0), dict(tok=0), dict(logits=GOOD + 2), dict(u=GOOD + 2), dict(tok=GOOD + 1),
               dict(prob=GOOD + 2), dict(sb=-1), dict(sn=-1), dict(us=-1)):
        assert f(**kw) == -1, kw


def test_read_refusals(lib):
    base = dict(size=None, ko=GOOD, vo=GOOD, dtype=1, B=2, N=3, Hkv=2, D=64, **CACHE, **SCALES, status=0)
    f = lambda **kw: lib.spec_verify_read_cache(pack(tg._READ, base, kw), None)
    assert lib.spec_verify_read_cache(None, None) == -1
    assert f(size=8) == -1
    assert f(B=0) == 0
    assert f(dtype=0) == -2
    assert f(N=0) == -1
    assert f(D=72) == -1
    assert f(D=272) == -4
    assert f(ko=GOOD + 8) == -1
    assert f(vo=0) == -1
    assert f(sk=0) == -1
    for kw in BAD_CACHES + BAD_SCALES:
        assert f(**kw) == -1, kw


def test_append_refusals(lib):
    base = dict(size=None, q=GOOD, qo=GOOD, k=GOOD, v=GOOD, dtype=1, B=2, N=3, Hq=4, Hkv=2, D=64, qb=768, qn=256, qh=64,
                ob=768, on=256, oh=64, kb=384, kn=128, khs=64, vb=384, vn=128, vhs=64, table=GOOD, tlen=100, rot=64,
                inter=0, **CACHE, status=0)
    opt = dict(size=None, **SCALES)
    f = lambda o={}, **kw: lib.spec_verify_rotate_append_ex(pack(tg._ROTATE, base, kw), pack(tg._ROTATE_OPTIONS, opt, o), None)
    assert lib.spec_verify_rotate_append_ex(None, None, None) == -1
    assert f(size=8) == -1
    assert f(dict(size=8)) == -1
    assert f(B=0) == 0
    assert f(dtype=3) == -2
    assert f(D=272, rot=64) == -4
    assert f(B=1 << 15, N=1 << 16) == -4  # more blocks than a launch has
    for kw in BAD_CACHES:
        assert f(**kw) == -1, kw
    for kw in BAD_SCALES:
        assert f(kw) == -1, kw


def test_attention_refusals(lib):
    base = dict(size=None, q=GOOD, out=GOOD, dtype=1, B=2, N=3, Hq=4, Hkv=2, D=64, qb=768, qn=256, qh=64, ob=768, on=256,
                oh=64, scale=0.125, window=0, max_context=0, **CACHE, ws=GOOD, wsb=1 << 40, status=0, wait=0)
    opt = dict(size=None, sinks=0, **SCALES)
    f = lambda o={}, **kw: lib.spec_verify_attention_ex(pack(tg._ATTENTION, base, kw), pack(tg._ATTENTION_OPTIONS, opt, o), None)
    assert lib.spec_verify_attention_ex(None, None, None) == -1
    assert f(size=8) == -1
    assert f(dict(size=8)) == -1
    assert f(dict(sinks=-1)) == -1
    assert f(B=0) == 0
    assert f(dtype=3) == -2
    assert f(D=96) == -2
    assert f(ws=0) == -5
    assert f(wsb=100) == -5
    for kw in BAD_CACHES:
        assert f(**kw) == -1, kw
    for kw in BAD_SCALES:
        assert f(kw) == -1, kw


def test_binding_refusals(lib):
    c = sv.PagedCache8(4, 32, 2, 64, device="cpu")
    assert (c.pages, c.page_size, c.kv_heads, c.head_dim) == (4, 32, 2, 64) and c.k_scales.shape == (4, 2, 2)
    good = (c.k, c.v, c.k_scales, c.v_scales)
    F8 = torch.float8_e4m3fn
    for bad in ((c.k.view(torch.uint8), c.v.view(torch.uint8), *good[2:]), (c.k, c.v.view(torch.uint8), *good[2:]),
                (c.k.view(torch.float8_e5m2), c.v.view(torch.float8_e5m2), *good[2:])):
        with pytest.raises((TypeError, ValueError)):
            sv.PagedCache8.from_tensors(*bad)
    wide = torch.zeros(4, 2, 32, 72, dtype=torch.uint8).view(F8)
    for bad in ((*good[:2], c.k_scales[:, :, :1], c.v_scales), (*good[:2], c.k_scales.double(), c.v_scales),
                (*good[:2], c.k_scales, torch.ones(4, 2, 4)[:, :, ::2]), (wide[..., :64], wide[..., :64], *good[2:]),
                (c.k[:, :, :, ::2], c.v[:, :, :, ::2], *good[2:])):
        with pytest.raises(ValueError):
            sv.PagedCache8.from_tensors(*bad)
    with pytest.raises(ValueError):
        sv.PagedCache8(4, 24, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        sv.read_cache(c, torch.zeros(1, 1, dtype=torch.int32), [0], 3)
    with pytest.raises(TypeError):
        sv.read_cache(sv.PagedCache(4, 32, 2, 64, device="cpu"), torch.zeros(1, 1, dtype=torch.int32), [0], 3)
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.paged_attention(q, c, None, None)
    with pytest.raises(ValueError):
        sv.rotate_append(q, q, q, None, c, None, None)
    with pytest.raises(ValueError):
        sv.sample(torch.zeros(1, 1, 8), torch.zeros(1, 1))


def test_the_definitions_quantise_as_torch_does():
    """The oracle's rounding against torch's own conversion (both round float32 values to nearest even)."""
    from tests import drafter_ref as ref

    g = torch.Generator().manual_seed(0)
    x = torch.cat((torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 8, (20000,), generator=g).float()),
                   torch.tensor([0.0, 448.0, -448.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -6, 15.5, 17.0, 18.0, 19.0])))
    x = x.clamp(-448, 448)
    assert torch.equal(ref.round8(x.double()).float(), x.to(torch.float8_e4m3fn).float())
    for amax, s in ((448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (3.5, 2.0 ** -7), (3.50001, 2.0 ** -6), (0.0, 1.0)):
        assert float(ref.least_scale(torch.tensor(amax, dtype=torch.float64))) == s
    assert math.isnan(float(ref.round8(torch.tensor(math.inf, dtype=torch.float64))))
