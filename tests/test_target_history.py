"""A TokenHistory whose planes are replaced: the calls read the ones it holds then, and refuse planes that do not fit."""
import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from speculative_decoding_verification_20_gb300 import target as tg


class OnGpu(torch.Tensor):
    """A tensor that says it is on a GPU."""
    is_cuda = True


def misfits(slots, V, device):
    """Planes of another size, type or layout than a history's: (seen, counts)."""
    W = (V + 31) // 32
    z = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device=device)
    return [(z(slots, W - 1), z(slots, V)), (z(slots - 1, W), z(slots, V)), (z(slots, W), z(V)),
            (z(slots, W, dtype=torch.int64), z(slots, V)), (z(slots, W), z(slots, V, dtype=torch.float32)),
            (z(slots, 2 * W)[:, :W], z(slots, V)), (z(slots, W), z(V, slots).t())]


def test_the_general_way_reads_what_the_history_holds(monkeypatch):
    seen = []

    class Library:
        def spec_verify_history_add(self, packed, stream):
            seen.append(tg._HISTORY.unpack(packed)[1:6])
            return 0

        def spec_verify_process_logits(self, packed, stream):
            seen.append(tg._LOGITS.unpack(packed)[11:15])
            return 0

    monkeypatch.setattr(tg, "_library", Library)
    monkeypatch.setattr(tg, "_short", type("General", (), {"logits": staticmethod(lambda *a: None)}))
    monkeypatch.setattr(tg, "_current_device", lambda: None)
    monkeypatch.setattr(tg, "_raw_stream", lambda device: 7)
    h = sv.TokenHistory(3, 100, device="cpu")
    x = torch.zeros(2, 1, 100).as_subclass(OnGpu)
    gpu = lambda t: t.as_subclass(OnGpu)
    tokens = torch.zeros(2, 4, dtype=torch.int32)

    def calls():
        del seen[:]
        h.load(tokens), h.add(tokens)
        sv.process_logits(x, history=h, out=x)
        return seen

    def now():
        at = (h.seen.data_ptr(), h.counts.data_ptr(), h.counts.shape[0], h.seen.shape[1])
        return [at + (100,)] * 2 + [at]

    h.counts = gpu(h.counts)
    assert calls() == now() and (h.slots, h.vocab, h.words) == (3, 100, 4)
    h.seen, h.counts = torch.zeros(7, 9, dtype=torch.int32), gpu(torch.zeros(7, 100, dtype=torch.int32))
    assert calls() == now() and (h.slots, h.vocab, h.words) == (7, 100, 9)
    for s, c in misfits(3, 100, "cpu"):
        h.seen, h.counts = s, gpu(c)
        for call in (lambda: h.load(tokens), lambda: h.add(tokens), lambda: sv.process_logits(x, history=h, out=x)):
            with pytest.raises(ValueError):
                call()


@pytest.mark.gpu
def test_the_direct_way_refuses_planes_that_do_not_fit():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.randn(2, 1, 100, device="cuda")
    h = sv.TokenHistory(2, 100)
    for s, c in misfits(3, 100, "cuda"):
        h.seen, h.counts = s, c
        with pytest.raises(ValueError):
            sv.process_logits(x, history=h)
    h.seen, h.counts = (torch.zeros(3, n, dtype=torch.int32, device="cuda") for n in (5, 100))
    h.add(torch.tensor([[7, 7]], dtype=torch.int32, device="cuda"), slots=[1])
    z = sv.process_logits(x, history=h, frequency=torch.ones(2, device="cuda"))
    want = x.clone()
    want[1, 0, 7] -= 2
    assert torch.equal(z, want)
