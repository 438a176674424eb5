"""Appending to and reading the 8-bit cache on other streams, from threads and in graphs; sinks in a graph."""
import threading

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from tests.test_cache8_gpu import bits, built, expected_append, i32, tables  # noqa: F401  (built: the fixture)
from tests.test_sinks_gpu import check
from tests.test_target_gpu import paged

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
NAMES = ("k", "v", "k_scales", "v_scales")


def step(seed, B=5, N=6, Hq=4, Hkv=2, D=64, page=32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    past, new = [0, 15, 31, 7, 100][:B], [N, 1, N - 1, 0, N][:B]
    table, pages = tables(past, new, page, seed)
    r = lambda h: torch.randn(B, N, h, D, generator=g, device="cuda").to(BF)
    cache = sv.PagedCache8(pages, page, Hkv, D)
    cache.k.copy_(torch.randn(pages, Hkv, page, D, generator=g, device="cuda").to(cache.k.dtype))
    cache.v.copy_(torch.randn(pages, Hkv, page, D, generator=g, device="cuda").to(cache.v.dtype))
    return dict(cache=cache, table=table, past=past, new=new, q=r(Hq), k=r(Hkv), v=r(Hkv), tab=sv.rotary_table(128, D),
                lens=i32(past), num=i32(new), first=i32([0] * B), count=i32([p + n for p, n in zip(past, new)]))


def expected(s):
    return expected_append(s["cache"], s["table"], s["past"], s["new"], s["k"], s["v"], s["tab"], 64, False)


def append(s, **kw):
    return sv.rotate_append(s["q"], s["k"], s["v"], s["tab"], s["cache"], s["table"], s["lens"], s["num"], **kw)


def read(s, **kw):
    return sv.read_cache(s["cache"], s["table"], s["first"], 106, s["count"], **kw)


def same(s, want):
    return all(torch.equal(bits(getattr(s["cache"], n)), bits(w)) for n, w in zip(NAMES, want))


def test_another_stream():
    s, t = step(1), step(1)
    want = expected(s)
    q = append(t)
    back = read(t)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, got_back = append(s, stream=st), read(s, stream=st)
    st.synchronize()
    assert same(s, want) and torch.equal(got, q)
    assert all(torch.equal(a, b) for a, b in zip(got_back, back))


def test_a_captured_step_is_replayed_on_new_tokens():
    """One capture: append, read back; the lengths advance between replays, the blocks are rescaled each time."""
    s = step(2)
    held = [getattr(s["cache"], n).clone() for n in NAMES]
    graph = torch.cuda.CUDAGraph()
    append(s)  # (loads what the first call loads)
    for n, t in zip(NAMES, held):
        getattr(s["cache"], n).copy_(t)
    with torch.cuda.graph(graph):
        q = append(s)
        back = read(s, dtype=HF)
    g = torch.Generator(device="cuda").manual_seed(9)
    for rnd in range(3):
        for n in ("q", "k", "v"):
            s[n].copy_((2.0 ** (3 * rnd)) * torch.randn(s[n].shape, generator=g, device="cuda"))
        want = expected(s)
        graph.replay()
        torch.cuda.synchronize()
        assert same(s, want), rnd
        again = append(dict(s, cache=sv.PagedCache8.from_tensors(*(t.clone() for t in want))))
        assert torch.equal(q, again)
        plain = read(s, dtype=HF)
        assert all(torch.equal(a, b) for a, b in zip(back, plain))


def test_threads():
    """Each thread appends to a cache of its own, on its own stream."""
    steps = [step(10 + i) for i in range(4)]
    wants = [expected(s) for s in steps]
    torch.cuda.synchronize()
    bad = []

    def work(s, want):
        st = torch.cuda.Stream()
        for _ in range(10):  # the same positions again: the same cache
            append(s, stream=st)
            read(s, stream=st)
        st.synchronize()
        if not same(s, want):
            bad.append(1)

    threads = [threading.Thread(target=work, args=a) for a in zip(steps, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("N", [1, 9, 40, 150])
def test_sinks_in_a_graph(N):
    past, new = [900, 500], [N, N]
    s = paged(2, N, 8, 2, 64, BF, 32, past, new, seed=N)
    call = lambda: sv.paged_attention(s["q"], s["cache"], s["table"], s["lens"], s["new"], window=200, sinks=5, max_context=1100)
    want = call()
    check(s, past, new, 200, 5, got=want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    call()  # (the stream's own call between capture and replay)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    s["q"].copy_(torch.randn(s["q"].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check(s, past, new, 200, 5, got=got)
    assert not torch.equal(got, want)
