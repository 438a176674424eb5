"""A PagedCache whose tensors are replaced: the calls read the ones it holds then.  Page tables with shared rows."""
import pytest
import torch

import speculative_decoding_verification_20_gb300 as sv
from speculative_decoding_verification_20_gb300 import target as tg


class OnGpu(torch.Tensor):
    """A tensor that says it is on a GPU."""
    is_cuda = True


class Library:
    """Keeps the cache's addresses, pages and page size of each call."""

    def __init__(self):
        self.seen = []

    def spec_verify_attention_workspace_size(self, *shape):
        return 4096

    def spec_verify_attention(self, packed, stream):
        self.seen.append(tg._ATTENTION.unpack(packed)[18:22])
        return 0

    def spec_verify_rotate_append(self, packed, stream):
        self.seen.append(tg._ROTATE.unpack(packed)[27:31])
        return 0


def test_the_general_way_reads_what_the_cache_holds(monkeypatch):
    lib = Library()
    monkeypatch.setattr(tg, "_library", lambda: lib)
    none = staticmethod(lambda *a: None)
    monkeypatch.setattr(tg, "_short", type("General", (), {"attention": none, "rotate": none}))
    monkeypatch.setattr(tg, "_current_device", lambda: None)
    monkeypatch.setattr(tg, "_raw_stream", lambda device: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(tg, "_workspaces", {})
    cache = sv.PagedCache(4, 16, 1, 64, device="cpu")
    pages, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16).as_subclass(OnGpu)
    table = sv.rotary_table(64, 64, device="cpu")

    def calls():
        del lib.seen[:]
        sv.paged_attention(q, cache, pages, lens)
        sv.rotate_append(q, q, q, table, cache, pages, lens)
        return lib.seen

    now = lambda: [(cache.k.data_ptr(), cache.v.data_ptr(), *cache.k.shape[::2])] * 2
    assert calls() == now()
    cache.k, cache.v = (torch.zeros(9, 1, 32, 64, dtype=torch.bfloat16) for _ in range(2))
    assert (cache.pages, cache.page_size, cache.kv_heads, cache.head_dim) == (9, 32, 1, 64) and calls() == now()
    cache.v.data = torch.zeros(9, 1, 32, 64, dtype=torch.bfloat16)
    assert calls() == now()
    cache.k = cache.k[:4]  # no longer alike
    for call in (lambda: sv.paged_attention(q, cache, pages, lens),
                 lambda: sv.rotate_append(q, q, q, table, cache, pages, lens)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("as_list", [False, True])  # lengths that need a conversion take the general way
def test_replaced_tensors_are_read_and_written(as_list):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    cache = sv.PagedCache(6, 16, 2, 64)
    cache.k.zero_(), cache.v.zero_()
    pages = torch.randperm(6, device="cuda").to(torch.int32)[None]
    lens = [40] if as_list else torch.tensor([40], dtype=torch.int32, device="cuda")
    table = sv.rotary_table(96, 64)
    q, k, v = rand(1, 5, 4, 64), rand(1, 5, 2, 64), rand(1, 5, 2, 64)
    old = cache.k, cache.v  # (kept, as a caller may)
    sv.paged_attention(q, cache, pages, lens)
    cache.k, cache.v = rand(6, 2, 16, 64), rand(6, 2, 16, 64)
    fresh = sv.PagedCache.from_tensors(cache.k.clone(), cache.v.clone())
    got, want = (sv.rotate_append(q, k, v, table, c, pages, lens) for c in (cache, fresh))
    assert torch.equal(got, want) and torch.equal(cache.k, fresh.k) and torch.equal(cache.v, fresh.v)
    assert torch.equal(sv.paged_attention(q, cache, pages, lens), sv.paged_attention(q, fresh, pages, lens))
    assert not old[0].any() and not old[1].any()


@pytest.mark.gpu
def test_sequences_may_share_a_row_of_the_page_table():
    """Samples of one prompt: an expanded row, and rows that overlap, are read as they are written."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    B = 3
    cache = sv.PagedCache.from_tensors(rand(8, 2, 16, 64), rand(8, 2, 16, 64))
    row = torch.randperm(8, device="cuda").to(torch.int32)
    lens = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    q = rand(B, 2, 4, 64)
    for table in (row[None, :4].expand(B, 4), row.as_strided((B, 4), (2, 1))):
        want = sv.paged_attention(q, cache, table.contiguous(), lens)
        assert torch.equal(sv.paged_attention(q, cache, table, lens), want)
        assert torch.equal(sv.paged_attention(q, cache, table, lens.tolist()), want)
    new = torch.tensor([1, 0, 0], dtype=torch.int32, device="cuda")  # the first writes, the others read
    k, t = rand(B, 2, 2, 64), sv.rotary_table(64, 64)
    other = sv.PagedCache.from_tensors(cache.k.clone(), cache.v.clone())
    a = sv.rotate_append(q, k, k, t, cache, row[None, :4].expand(B, 4), lens, new)
    b = sv.rotate_append(q, k, k, t, other, row[None, :4].repeat(B, 1), lens, new)
    assert torch.equal(a, b) and torch.equal(cache.k, other.k) and torch.equal(cache.v, other.v)
