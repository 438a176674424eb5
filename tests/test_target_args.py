"""Refusals of the target-step operators, without a GPU: the C entry points return before
they enqueue anything, and the binding raises."""
import math
import struct

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from speculative_decoding_verification_20_gb300 import target as tg

GOOD = 0x10000  # never dereferenced: the checks come first
CACHE = dict(k_pages=GOOD, v_pages=GOOD, pages=8, page_size=16, kp=2048, kh=1024, ks=64, vp=2048, vh=1024, vs=64,
             page_table=GOOD, pt_stride=4, pages_per_seq=4, cache_lens=GOOD, num_new=0)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_20_gb300 import _build

    _build.build()
    return sv.load_library()


def _call(fn, fmt, base, **kw):
    d = dict(base)
    for k in kw:
        assert k in d, k
    d.update(kw)
    if d["size"] is None:
        d["size"] = fmt.size
    return fn(fmt.pack(*d.values()), None)


def test_structures_match_the_header(lib, tmp_path):
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "s.c"
    src.write_text('#include "spec_verify_target.h"\n#include <stdio.h>\nint main(void){printf("%zu %zu %zu %zu",'
                   "sizeof(sv_history_args),sizeof(sv_logits_args),sizeof(sv_rotate_args),sizeof(sv_attention_args));"
                   "return 0;}\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I" + os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert sizes == [tg._HISTORY.size, tg._LOGITS.size, tg._ROTATE.size, tg._ATTENTION.size]


def test_history_refusals(lib):
    base = dict(size=None, seen=GOOD, counts=GOOD, slots=4, words=4, V=100, slot_of=0, tokens=GOOD, B=2,
                L=5, stride=5, prompt=0, total=0, clear=0)
    f = lambda **kw: _call(lib.spec_verify_history_add, tg._HISTORY, base, **kw)
    assert lib.spec_verify_history_add(None, None) == -1
    assert f(size=8) == -1
    assert f(B=0) == 0
    assert f(words=3) == -1
    assert f(V=0) == -1
    assert f(B=5) == -1  # more rows than slots, and no slot_of
    assert f(seen=0) == -1
    assert f(tokens=0) == -1
    assert f(V=262145, words=10000) == -4
    assert f(B=65536, slots=70000) == -4


def test_logits_refusals(lib):
    base = dict(size=None, logits=GOOD, out=GOOD, dtype=0, B=2, N=3, V=100, lb=300, ln=100, ob=300, on=100, seen=0,
                counts=0, slots=0, words=0, slot_of=0, draft=0, ds=0, dl=0, rep=0, freq=0, pres=0, ids=0,
                vals=0, offs=0, nbias=0, mask=0, mb=0, mn=0, status=0)
    f = lambda **kw: _call(lib.spec_verify_process_logits, tg._LOGITS, base, **kw)
    assert lib.spec_verify_process_logits(None, None) == -1
    assert f(size=232) == -1
    assert f(B=0) == 0
    assert f(dtype=2) == -2
    assert f(N=0) == -1
    assert f(V=0) == -1
    assert f(N=34) == -4
    assert f(V=262145) == -4
    assert f(logits=0) == -1
    assert f(out=GOOD + 2) == -1
    assert f(on=99) == -1  # output rows on one another
    assert f(ob=0) == -1
    assert f(seen=GOOD, counts=GOOD, slots=4, words=3) == -1
    assert f(seen=GOOD, counts=GOOD, slots=1, words=4) == -1
    assert f(seen=GOOD, counts=0, slots=4, words=4) == -1
    assert f(ids=GOOD, vals=GOOD, offs=0, nbias=4) == -1
    assert f(ids=GOOD, vals=GOOD, offs=GOOD, nbias=-1) == -1
    assert f(draft=GOOD, ds=-1) == -1
    assert f(mask=GOOD, mb=-1) == -1


BAD_CACHES = [dict(k_pages=0), dict(v_pages=GOOD + 8), dict(pages=0), dict(page_size=8), dict(page_size=24),
              dict(ks=63), dict(vs=56), dict(kh=1025), dict(page_table=0), dict(pt_stride=3), dict(pages_per_seq=0),
              dict(cache_lens=0), dict(vp=-8)]


def test_rotate_refusals(lib):
    base = dict(size=None, q=GOOD, qo=GOOD, k=GOOD, v=GOOD, dtype=1, B=2, N=3, Hq=4, Hkv=2, D=64, qb=768, qn=256, qh=64,
                ob=768, on=256, oh=64, kb=384, kn=128, khs=64, vb=384, vn=128, vhs=64, table=GOOD, tlen=100, rot=64,
                inter=0, **CACHE, status=0)
    f = lambda **kw: _call(lib.spec_verify_rotate_append, tg._ROTATE, base, **kw)
    assert lib.spec_verify_rotate_append(None, None) == -1
    assert f(size=8) == -1
    assert f(B=0) == 0
    assert f(dtype=0) == -2
    assert f(N=0) == -1
    assert f(D=72) == -1
    assert f(D=272, rot=64) == -4
    assert f(rot=24) == -1
    assert f(rot=80) == -1
    assert f(q=GOOD + 8) == -1
    assert f(qn=257) == -1
    assert f(oh=0) == -1
    assert f(on=8) == -1
    assert f(table=GOOD + 4) == -1
    for kw in BAD_CACHES:
        assert f(**kw) == -1, kw


def test_attention_refusals(lib):
    base = dict(size=None, q=GOOD, out=GOOD, dtype=1, B=2, N=3, Hq=4, Hkv=2, D=64, qb=768, qn=256, qh=64, ob=768, on=256,
                oh=64, scale=0.125, window=0, max_context=0, **CACHE, ws=GOOD, wsb=1 << 40, status=0, wait=0)
    f = lambda **kw: _call(lib.spec_verify_attention, tg._ATTENTION, base, **kw)
    assert lib.spec_verify_attention(None, None) == -1
    assert f(size=8) == -1
    assert f(B=0) == 0
    assert f(dtype=0) == -2
    assert f(D=96) == -2
    assert f(Hq=5) == -1
    assert f(Hq=130) == -4  # 65 heads a cache head
    assert f(window=-1) == -1
    assert f(scale=0.0) == -1
    assert f(scale=math.nan) == -1
    assert f(scale=math.inf) == -1
    assert f(oh=56) == -1
    assert f(ob=8) == -1
    assert f(out=0) == -1
    assert f(ws=0) == -5
    assert f(wsb=100) == -5
    assert f(ws=GOOD + 16) == -1
    for kw in BAD_CACHES:
        assert f(**kw) == -1, kw


def test_attention_workspace_size(lib):
    assert sv.attention_workspace_size(1, 1, 32, 8, 128) > 0
    assert sv.attention_workspace_size(64, 8, 32, 8, 128) >= sv.attention_workspace_size(64, 1, 32, 8, 128)
    assert sv.attention_workspace_size(64, 1, 32, 8, 128) == sv.attention_workspace_size(1, 1, 32, 8, 128)
    assert sv.attention_workspace_size(1, 0, 32, 8, 128) == 0
    assert sv.attention_workspace_size(1, 1, 30, 8, 128) == 0
    assert sv.attention_workspace_size(1, 1, 32, 8, 96) == 0


def test_binding_refuses_cpu_tensors_and_bad_types(lib):
    with pytest.raises(ValueError):
        sv.process_logits(torch.zeros(1, 1, 8))
    with pytest.raises(ValueError):
        sv.TokenHistory(2, 8, device="cpu").add([[1, 2]])
    with pytest.raises(ValueError):
        sv.TokenHistory(0, 8, device="cpu")
    cache = sv.PagedCache(4, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        sv.paged_attention(torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), cache, None, None)
    with pytest.raises(ValueError):
        sv.rotate_append(torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), None, None, None, cache, None, None)
    with pytest.raises(ValueError):
        sv.PagedCache(4, 8, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        sv.PagedCache(4, 24, 2, 64, device="cpu")
    with pytest.raises(TypeError):
        sv.PagedCache(4, 16, 2, 64, dtype=torch.float32, device="cpu")
    k = torch.zeros(4, 2, 16, 68, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.PagedCache.from_tensors(k[..., :64], k[..., :64])  # rows of 136 bytes
    with pytest.raises(ValueError):
        sv.PagedCache.from_tensors(k.transpose(2, 3), k.transpose(2, 3))
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)  # another order of the same axes is fine
    assert sv.PagedCache.from_tensors(k.transpose(1, 2), k.transpose(1, 2)).page_size == 16


def test_rotary_table_values_and_refusals():
    t = sv.rotary_table(5000, 32, base=500.0, device="cpu")
    assert t.shape == (5000, 2, 16) and t.dtype == torch.float32
    for p in (0, 1, 77, 4999):
        for j in (0, 3, 15):
            a = p * 500.0 ** (-2.0 * j / 32)
            # a float64 angle below 5000 is off by at most 2^-40, its cosine rounded once to float32
            assert abs(t[p, 0, j].item() - math.cos(a)) < 2.0 ** -24 and abs(t[p, 1, j].item() - math.sin(a)) < 2.0 ** -24
    lin = sv.rotary_table(40, 32, scaling=dict(type="linear", factor=4.0), device="cpu")
    plain = sv.rotary_table(10, 32, device="cpu")
    assert torch.allclose(lin[::4], plain, rtol=0, atol=2.0 ** -22)
    ntk = sv.rotary_table(40, 32, scaling=dict(type="ntk", factor=4.0), device="cpu")
    # the fastest pair is unchanged, the slowest stretched by the factor
    assert torch.allclose(ntk[:, :, 0], sv.rotary_table(40, 32, device="cpu")[:, :, 0], rtol=0, atol=2.0 ** -22)
    assert torch.allclose(ntk[::4, :, 15], plain[:, :, 15], rtol=0, atol=2.0 ** -22)
    yarn = sv.rotary_table(64, 64, scaling=dict(type="yarn", factor=8.0, original_length=4096), device="cpu")
    m = 0.1 * math.log(8.0) + 1.0
    full = sv.rotary_table(64, 64, device="cpu")
    assert torch.allclose(yarn[:, :, 0], full[:, :, 0] * m, rtol=0, atol=2.0 ** -22)
    assert torch.allclose(yarn[::8, :, 31], full[:8, :, 31] * m, rtol=0, atol=2.0 ** -22)
    for bad in (dict(type="other", factor=2.0), dict(type="linear", factor=0.5), dict(type="linear", factor=math.nan)):
        with pytest.raises(ValueError):
            sv.rotary_table(8, 32, scaling=bad, device="cpu")
    for n, d in ((0, 32), (8, 31), (8, 0)):
        with pytest.raises(ValueError):
            sv.rotary_table(n, d, device="cpu")


def test_packed_layouts_are_runs_of_eight_byte_fields():
    for s in (tg._HISTORY, tg._LOGITS, tg._ROTATE, tg._ATTENTION):
        assert s.size % 8 == 0 and isinstance(s, struct.Struct)


def test_measured_cases_are_well_formed():
    """The measured cases and draws stay inside what the operators take."""
    import importlib.util
    import os
    import random

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("operators", os.path.join(root, "perf", "operators.py"))
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    rng = random.Random(7)
    cases = ops.listed() + [ops.draw(rng) for _ in range(60)]
    for c in cases:
        w = ops.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0
        if c["op"] != "logits":
            assert c["page"] % 16 == 0 and c["Hq"] % c["Hkv"] == 0 and c["D"] in (64, 128)
            past, new = ops._spread(c)
            assert max(new) == c["N"] and min(new) >= 1 and min(past) >= 0
