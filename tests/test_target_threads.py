"""Two threads that call paged_attention on one stream, without a GPU: the C function is a stand-in that takes a
while between its two launches, as the real one may, since ctypes lets other threads run meanwhile."""
import threading
import time

import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from speculative_decoding_verification_20_gb300 import target as tg


class OnGpu(torch.Tensor):
    """A tensor that says it is on a GPU."""
    is_cuda = True


class Library:
    def __init__(self):
        self.launches = []

    def spec_verify_attention_workspace_size(self, *shape):
        return 4096

    def spec_verify_attention(self, packed, stream):
        workspace = tg._ATTENTION.unpack(packed)[-4]
        for kernel in ("attend", "join"):
            self.launches.append((workspace, threading.get_ident(), kernel))
            time.sleep(0.001)
        return 0


@pytest.mark.parametrize("own_workspace", [False, True])
def test_no_launch_of_another_thread_between_the_two(monkeypatch, own_workspace):
    lib = Library()
    monkeypatch.setattr(tg, "_library", lambda: lib)
    monkeypatch.setattr(tg, "_short", type("General", (), {"attention": staticmethod(lambda *a: None)}))
    monkeypatch.setattr(tg, "_current_device", lambda: None)
    monkeypatch.setattr(tg, "_raw_stream", lambda device: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(tg, "_workspaces", {})
    cache = sv.PagedCache(4, 16, 1, 64, device="cpu")
    pages, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    kw = dict(workspace=torch.empty(4096, dtype=torch.uint8)) if own_workspace else {}

    def calls():
        q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16).as_subclass(OnGpu)
        for _ in range(20):
            sv.paged_attention(q, cache, pages, lens, out=q, **kw)

    threads = [threading.Thread(target=calls) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(lib.launches) == 120 and len({w for w, _, _ in lib.launches}) == 1
    for first, second in zip(lib.launches[::2], lib.launches[1::2]):
        assert first[:2] == second[:2] and (first[2], second[2]) == ("attend", "join")
