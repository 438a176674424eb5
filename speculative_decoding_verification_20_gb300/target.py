"""Operators around one verification call: the target's attention over its paged cache,
the rotary positions that fill it, and what is done to the logits before they are verified.

A round with gamma drafts runs N = gamma + 1 new tokens of each sequence::

    q = sv.rotate_append(q, k, v, table, cache, page_table, cache_lens)      # every layer
    o = sv.paged_attention(q, cache, page_table, cache_lens, max_context=m)
    ...
    z = sv.process_logits(logits, history=history, draft_tokens=x, repetition=r, mask=grammar)
    res = sv.spec_verify(z, draft_logits, x, temperature, seed=step)
    history.add(res["out_tokens"])                                           # the -1s are skipped
    cache_lens += res["accepted_len"] + 1                                    # rejected keys are overwritten

N = 1 is the plain decoding step; a large N is a chunk of a prompt.  The arrays are those of
``include/spec_verify_target.h``, which states the formulas.  Nothing here synchronises,
and there is no CPU path.  ``row_status`` (int32 [B], zeroed by the caller) collects the
ROW_BAD_* bits of sequences whose data is bad; such a sequence gets NaN, which spec_verify
then reports as ROW_NONFINITE.
"""
from __future__ import annotations

import ctypes
import math
import struct
import threading
from typing import Optional, Tuple, Union

import torch

SV_F16 = 2

ROW_BAD_PENALTY = 0x100
ROW_BAD_SLOT = 0x200
ROW_BAD_LENGTH = 0x400
ROW_BAD_PAGE = 0x800
ROW_BAD_MIN_P = 0x1000
ROW_BAD_UNIFORM = 0x2000

SCALE_BLOCK = 16  # tokens that share a scale in an 8-bit cache (SV_SCALE_BLOCK)

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: SV_F16}

# the C structures are runs of 8-byte fields, filled in one go
_HISTORY = struct.Struct("<Q2Q3q2Q3q2Qq")
_LOGITS = struct.Struct("<Q2Q4q4q2Q2q2Q2q3Q3QqQ2qQ")
_CACHE = "2Q8qQ2q2Q"
_ROTATE = struct.Struct("<Q4Q6q12qQ3q" + _CACHE + "Q")
_ATTENTION = struct.Struct("<Q2Q6q6qd2q" + _CACHE + "QqQQ")
_SCALES = "2Q4q"
_ROTATE_OPTIONS = struct.Struct("<Q" + _SCALES)
_ATTENTION_OPTIONS = struct.Struct("<Qq" + _SCALES)
_READ = struct.Struct("<Q2Q5q" + _CACHE + _SCALES + "Q")
_SAMPLE = struct.Struct("<QQ6qQq7Q")
_NO_SCALES = (0, 0, 0, 0, 0, 0)


_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream
_lib = None


def _library():
    global _lib
    if _lib is None:
        from . import load_library

        _lib = load_library()
    return _lib


class _Short:
    """The calls in csrc/sv_bind.cpp, which serve tensors that need no conversion and answer None for others; loaded
    at the first use."""

    __slots__ = ()

    def __getattr__(self, name):
        global _short
        from . import _build

        lib = _library()
        try:
            from . import _bind
        except ImportError as e:
            raise RuntimeError(f"{_build.BIND} is missing or of another torch: build it with "
                               "__graft_entry__.build()") from e
        address = lambda fn: ctypes.cast(fn, ctypes.c_void_p).value
        _bind.setup(address(lib.spec_verify_process_logits), address(lib.spec_verify_rotate_append),
                    address(lib.spec_verify_attention), address(lib.spec_verify_attention_workspace_size),
                    address(lib.spec_verify_rotate_append_ex), address(lib.spec_verify_attention_ex),
                    address(lib.spec_verify_sample), address(lib.spec_verify_read_cache), _check)
        _short = _bind
        return getattr(_bind, name)


_short = _Short()


def _check(status: int) -> None:
    if status:
        from . import SpecVerifyError, strerror

        raise SpecVerifyError(status, strerror(status))


def _p(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _vec(x, B: int, dtype: torch.dtype, device, name: str) -> Optional[torch.Tensor]:
    """A per-sequence parameter as a contiguous device vector of B entries."""
    if x is None:
        return None
    if isinstance(x, torch.Tensor) and x.dtype == dtype and x.device == device and x.dim() == 1 and \
            x.shape[0] == B and x.is_contiguous():
        return x
    from . import _dev_vec

    return _dev_vec(x, B, dtype, device, name)


def _table(x: torch.Tensor, rows: int, cols: int, device, name: str) -> torch.Tensor:
    """An int32 device matrix of so many rows and at least so many columns, rows contiguous."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[0] != rows or x.shape[1] < cols:
        raise ValueError(f"{name} must be [{rows}, >= {cols}]")
    if x.dtype != torch.int32 or x.device != device:
        x = x.to(device=device, dtype=torch.int32)
    return x if x.stride(1) == 1 or x.shape[1] == 1 else x.contiguous()


def _page_table(x: torch.Tensor, B: int, device) -> torch.Tensor:
    """A page table with rows of their own: sequences that share one (an expanded row) get a copy each."""
    x = _table(x, B, 1, device, "page_table")
    return x if B < 2 or x.stride(0) >= x.shape[1] else x.contiguous()


def _status(row_status, B, device):
    if row_status is not None and (row_status.dtype != torch.int32 or row_status.device != device or
                                   tuple(row_status.shape) != (B,) or not row_status.is_contiguous()):
        raise ValueError("row_status must be a contiguous int32 CUDA tensor of B entries")
    return row_status


def _elsewhere(device: torch.device, stream, fn, args, kwargs):
    """The call on another stream than torch's current one (what it allocates belongs to that stream, what it is
    given is kept for it), or on another device than the current one."""
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device):
        if stream is not None and torch.cuda.current_device() != device.index:
            raise ValueError(f"the stream is not one of {device}")
        res = fn(*args, **kwargs)
        if stream is not None:
            for t in (*args, *kwargs.values()):
                for u in t if isinstance(t, (tuple, list)) else \
                        (t.k, t.v, t.k_scales, t.v_scales) if isinstance(t, PagedCache8) else \
                        (t.k, t.v) if isinstance(t, PagedCache) else \
                        (t.seen, t.counts) if isinstance(t, TokenHistory) else (t,):
                    if isinstance(u, torch.Tensor) and u.is_cuda:
                        u.record_stream(stream)
    return res


_workspaces: dict = {}
# A call of spec_verify_attention enqueues two kernels, the second of which joins what the first left in the workspace,
# and ctypes lets other threads run meanwhile: none may enqueue its own between them.
_attend_lock = threading.Lock()


def _workspace(nbytes: int, device: torch.device, raw: int) -> torch.Tensor:
    """Scratch of the calls on one stream, which follow one another; a call that is captured into a graph gets its own
    from the graph's memory, since replays may overlap with the stream's later calls."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, raw)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _workspaces[key] = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws


# ---------------------------------------------------------------------------
# logits
# ---------------------------------------------------------------------------
class TokenHistory:
    """The tokens that the penalties of ``process_logits`` count, for ``slots`` sequences.

    seen: int32 [slots, words], a bit plane (token t: bit t % 32 of word t // 32);
    counts: int32 [slots, V], occurrences in the output.
    """

    def __init__(self, slots: int, vocab: int, device="cuda"):
        if slots < 1 or vocab < 1:
            raise ValueError("slots and vocab must be positive")
        self.seen = torch.zeros((slots, (vocab + 127) // 128 * 4), dtype=torch.int32, device=device)
        self.counts = torch.zeros((slots, vocab), dtype=torch.int32, device=device)

    # seen and counts may be replaced: nothing is kept of them but the tensors
    slots = property(lambda self: self.counts.shape[0])
    vocab = property(lambda self: self.counts.shape[1])
    words = property(lambda self: self.seen.shape[1])

    def _planes(self) -> Tuple[int, int, int, int, int]:
        """The planes' addresses, slots, words and vocabulary, of what the history holds now."""
        seen, counts = self.seen, self.counts
        if seen.dim() != 2 or counts.dim() != 2 or seen.shape[0] != counts.shape[0] or \
                32 * seen.shape[1] < counts.shape[1] or seen.device != counts.device or \
                seen.dtype != torch.int32 or counts.dtype != torch.int32 or \
                not seen.is_contiguous() or not counts.is_contiguous():
            raise ValueError("seen must be int32 [slots, >= ceil(V / 32)] and counts int32 [slots, V], contiguous, on "
                             "one device")
        return seen.data_ptr(), counts.data_ptr(), seen.shape[0], seen.shape[1], counts.shape[1]

    def _call(self, tokens, prompt_lens, total_lens, slots, clear, stream):
        if not self.counts.is_cuda:
            raise ValueError("the history must be on a CUDA device")
        dev = self.counts.device
        if stream is not None or _current_device() != dev.index:
            return _elsewhere(dev, stream, TokenHistory._call, (self, tokens, prompt_lens, total_lens, slots, clear, None),
                              {})
        if not isinstance(tokens, torch.Tensor):
            tokens = torch.as_tensor(tokens, dtype=torch.int32)
        if tokens.dim() != 2:
            raise ValueError("tokens must be [B, L]")
        B, L = tokens.shape
        planes = self._planes()
        tokens = _table(tokens, B, L, dev, "tokens")
        slot_of = _vec(slots, B, torch.int32, dev, "slots")
        if slot_of is None and B > self.slots:
            raise ValueError(f"{B} rows but only {self.slots} slots")
        pl = _vec(prompt_lens, B, torch.int32, dev, "prompt_lens")
        tl = _vec(total_lens, B, torch.int32, dev, "total_lens")
        _check(_library().spec_verify_history_add(_HISTORY.pack(
            _HISTORY.size, *planes, _p(slot_of), _p(tokens), B, L, tokens.stride(0), _p(pl), _p(tl), int(clear)),
            _raw_stream(dev.index)))

    def load(self, tokens, prompt_lens=None, total_lens=None, slots=None, *, stream=None) -> None:
        """New sequences take their slots: of row b of tokens [B, L] the first prompt_lens[b] (default: none) are
        the prompt, those up to total_lens[b] (default: L) output.  slots [B] (default: row b, slot b)."""
        self._call(tokens, prompt_lens, total_lens, slots, True, stream)

    def add(self, tokens, total_lens=None, slots=None, *, stream=None) -> None:
        """Output tokens of a round, as spec_verify returns them: [B, L], ids outside [0, vocab) are skipped."""
        self._call(tokens, None, total_lens, slots, False, stream)


def process_logits(logits: torch.Tensor, *, history: Optional[TokenHistory] = None, slots=None,
                   draft_tokens: Optional[torch.Tensor] = None, repetition=None, frequency=None, presence=None,
                   bias: Optional[Tuple] = None, mask: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, row_status: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Penalties, biases and masks on logits [B, N, V] (float32 or bfloat16, CUDA, vocabulary contiguous).

    Row i of a sequence counts its history and draft_tokens[b, :i] (int32 [B, >= N - 1]).
    repetition, frequency, presence: per-sequence tensors, sequences or scalars.
    bias: (ids int32 [n], values float32 [n], offsets int32 [B + 1]), the added values of each sequence.
    mask: int32 [B, N, W] or [B, W], W >= ceil(V / 32), 1 = allowed: bit t % 32 of word t // 32 is token t's.
    out: where to write (may be ``logits``); by default a new tensor.  Returns it.
    """
    if stream is None:
        seen, counts = (None, None) if history is None else (history.seen, history.counts)
        ids, vals, offs = (None, None, None) if bias is None else bias
        res = _short.logits(logits, seen, counts, slots, draft_tokens, repetition, frequency, presence, ids, vals, offs,
                            mask, out, row_status)
        if res is not None:
            return res
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dim() != 3:
        raise ValueError("logits must be a CUDA tensor [B, N, V]")
    dev = logits.device
    if stream is not None or _current_device() != dev.index:
        return _elsewhere(dev, stream, process_logits, (logits,), dict(
            history=history, slots=slots, draft_tokens=draft_tokens, repetition=repetition, frequency=frequency,
            presence=presence, bias=bias, mask=mask, out=out, row_status=row_status))
    code = _DTYPE.get(logits.dtype)
    if code not in (0, 1):
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    B, N, V = logits.shape
    x = logits if logits.stride(2) == 1 or V == 1 else logits.contiguous()
    if out is None:
        out = torch.empty((B, N, V), dtype=logits.dtype, device=dev)
    elif out.shape != logits.shape or out.dtype != logits.dtype or out.device != dev or (V > 1 and out.stride(2) != 1):
        raise ValueError("out must have the logits' shape, type and device, and a contiguous vocabulary")
    seen = counts = slot_of = 0
    nslots = words = 0
    if history is not None:
        seen, counts, nslots, words, vocab = history._planes()
        if vocab != V or history.counts.device != dev:
            raise ValueError(f"the history is of {vocab} tokens on {history.counts.device}")
        slots = _vec(slots, B, torch.int32, dev, "slots")
        if slots is None and B > nslots:
            raise ValueError(f"{B} rows but only {nslots} slots")
        slot_of = _p(slots)
    toks = tstride = tlen = 0
    if draft_tokens is not None and N > 1:
        draft_tokens = _table(draft_tokens, B, N - 1, dev, "draft_tokens")
        toks, tstride, tlen = draft_tokens.data_ptr(), draft_tokens.stride(0), draft_tokens.shape[1]
    rep = _vec(repetition, B, torch.float32, dev, "repetition")
    freq = _vec(frequency, B, torch.float32, dev, "frequency")
    pres = _vec(presence, B, torch.float32, dev, "presence")
    ids = vals = offs = None
    nbias = 0
    if bias is not None:
        ids, vals, offs = bias
        nbias = len(ids)
        ids = _vec(ids, nbias, torch.int32, dev, "bias ids")
        vals = _vec(vals, len(vals), torch.float32, dev, "bias values")
        offs = _vec(offs, B + 1, torch.int32, dev, "bias offsets")
        if vals.shape[0] != nbias:
            raise ValueError("bias ids and values differ in length")
        if nbias == 0:
            ids = vals = offs = None
    msb = msn = 0
    if mask is not None:
        if mask.dtype != torch.int32 or mask.device != dev:
            raise ValueError("mask must be an int32 CUDA tensor")
        dims = mask.dim()
        if dims not in (2, 3) or mask.shape[0] != B or (dims == 3 and mask.shape[1] != N) or 32 * mask.shape[-1] < V:
            raise ValueError("mask must be [B, N, W] or [B, W] with W >= ceil(V / 32)")
        if mask.stride(-1) != 1 and mask.shape[-1] > 1:
            mask = mask.contiguous()
        msb, msn = mask.stride(0), (mask.stride(1) if dims == 3 else 0)
    _status(row_status, B, dev)
    xs, os = x.stride(), out.stride()
    _check(_library().spec_verify_process_logits(_LOGITS.pack(
        _LOGITS.size, x.data_ptr(), out.data_ptr(), code, B, N, V, xs[0], xs[1], os[0], os[1], seen, counts, nslots, words,
        slot_of, toks, tstride, tlen, _p(rep), _p(freq), _p(pres), _p(ids), _p(vals), _p(offs), nbias, _p(mask), msb, msn,
        _p(row_status)), _raw_stream(dev.index)))
    return out


# ---------------------------------------------------------------------------
# paged cache
# ---------------------------------------------------------------------------
class PagedCache:
    """Keys and values of one layer in pages: k, v [pages, kv_heads, page_size, head_dim], bfloat16 or float16.

    Position j of a sequence is row j % page_size of the page that its page table names at j // page_size.  The calls
    read k and v as they are then.
    """

    def __init__(self, pages: int, page_size: int, kv_heads: int, head_dim: int, dtype=torch.bfloat16, device="cuda"):
        shape = (pages, kv_heads, page_size, head_dim)
        self.k, self.v = torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device)
        _pages(self)

    @classmethod
    def from_tensors(cls, k: torch.Tensor, v: torch.Tensor) -> "PagedCache":
        """A cache over the caller's memory; any order of page, head and row in memory (views are fine), as long
        as the head dimension is contiguous and every row starts on a 16-byte boundary."""
        self = cls.__new__(cls)
        self.k, self.v = k, v
        _pages(self)
        return self

    # k and v may be replaced: nothing is kept of them but the tensors
    pages = property(lambda self: self.k.shape[0])
    kv_heads = property(lambda self: self.k.shape[1])
    page_size = property(lambda self: self.k.shape[2])
    head_dim = property(lambda self: self.k.shape[3])
    dtype = property(lambda self: self.k.dtype)
    device = property(lambda self: self.k.device)


class PagedCache8:
    """Keys and values of one layer in pages, held in 8 bits: k, v [pages, kv_heads, page_size, head_dim], float8_e4m3fn
    codes, and a scale for each 16 tokens and head: k_scales, v_scales float32 [pages, kv_heads, page_size / 16].

    A key is its code times its scale.  ``rotate_append`` keeps the scales at powers of two; ``paged_attention`` and
    ``read_cache`` take any that are finite and not negative.  Half the memory of a ``PagedCache``; attention over it takes
    about as long up to 32 rows a cache head (new tokens x query heads that share it), longer above.  A value is off by
    up to 2^-4 of itself or 2^-10 of its block's scale, whichever is more, for each scale that it was rounded under.  The
    calls read the tensors as they are then.
    """

    def __init__(self, pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
        shape = (pages, kv_heads, page_size, head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in "kv")
        self.k_scales, self.v_scales = (torch.ones((pages, kv_heads, page_size // SCALE_BLOCK), device=device)
                                        for _ in "kv")
        _check8(self)

    @classmethod
    def from_tensors(cls, k: torch.Tensor, v: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor) -> "PagedCache8":
        """A cache over the caller's memory; any order of page, head and row in memory (views are fine), as long as
        the head dimension is contiguous, every row starts on a 16-byte boundary and a head's scales are contiguous.
        Scales may share memory (one for each head, or one for all, expanded) in a cache that is only read: each call
        reads a copy of them, written out; ``rotate_append`` needs a scale for each block."""
        self = cls.__new__(cls)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        _check8(self)
        return self

    # the tensors may be replaced: nothing else is kept of them
    pages = property(lambda self: self.k.shape[0])
    kv_heads = property(lambda self: self.k.shape[1])
    page_size = property(lambda self: self.k.shape[2])
    head_dim = property(lambda self: self.k.shape[3])
    device = property(lambda self: self.k.device)


def _check8(cache: PagedCache8) -> None:
    k, v, ks, vs = cache.k, cache.v, cache.k_scales, cache.v_scales
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
        raise ValueError("k and v must be [pages, kv_heads, page_size, head_dim] of one shape, type and device")
    if k.dtype != torch.float8_e4m3fn:
        raise TypeError(f"the cache must be float8_e4m3fn, got {k.dtype}")
    if k.shape[2] < 16 or k.shape[2] % 16:
        raise ValueError(f"page_size must be a multiple of 16, got {k.shape[2]}")
    for t in (k, v):
        if t.stride(3) != 1 or t.data_ptr() % 16 or any(s % 16 for s in t.stride()[:3]):
            raise ValueError("rows of the cache must be contiguous and start on 16-byte boundaries")
    want = (k.shape[0], k.shape[1], k.shape[2] // SCALE_BLOCK)
    for t in (ks, vs):
        if t.dtype != torch.float32 or t.device != k.device or tuple(t.shape) != want or \
                (t.stride(2) > 1 and want[2] > 1):
            raise ValueError(f"scales must be float32 {list(want)} on the cache's device, a head's contiguous")


def _pages8(cache: PagedCache8, written: bool = False) -> Tuple[tuple, tuple, tuple]:
    """The head of the C description of a cache's pages, and that of its scales, of what it holds now; and the scales'
    tensors, to be kept until the call is enqueued."""
    _check8(cache)
    k, v = cache.k, cache.v
    scales = []
    for t in (cache.k_scales, cache.v_scales):
        n = t.shape[2]
        if (n > 1 and t.stride(2) != 1) or (t.shape[1] > 1 and t.stride(1) < n) or (t.shape[0] > 1 and t.stride(0) < n):
            if written:
                raise ValueError("blocks that share a scale cannot be appended to: each needs one of its own")
            t = t.contiguous()
        scales.append(t)
    ks, vs = scales
    return ((k.data_ptr(), v.data_ptr(), k.shape[0], k.shape[2], *k.stride()[:3], *v.stride()[:3]),
            (ks.data_ptr(), vs.data_ptr(), *ks.stride()[:2], *vs.stride()[:2]), (ks, vs))


def _of_cache(cache, q: torch.Tensor, written: bool = False) -> Tuple[tuple, Optional[tuple], torch.dtype, Optional[tuple]]:
    """A cache's C description, its scales' (None: 16 bits), the type of the queries, and what is to be kept until the
    call is enqueued."""
    if isinstance(cache, PagedCache8):
        pages, scales, held = _pages8(cache, written)
        if q.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
        return pages, scales, q.dtype, held
    return _pages(cache), None, cache.dtype, None


def _pages(cache: PagedCache) -> tuple:
    """The head of the C description of a cache: addresses, pages, page size and strides, of what it holds now."""
    k, v = cache.k, cache.v
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
        raise ValueError("k and v must be [pages, kv_heads, page_size, head_dim] of one shape, type and device")
    if k.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"the cache must be bfloat16 or float16, got {k.dtype}")
    if k.shape[2] < 16 or k.shape[2] % 16:
        raise ValueError(f"page_size must be a multiple of 16, got {k.shape[2]}")
    for t in (k, v):
        if t.stride(3) != 1 or t.data_ptr() % 16 or any(s % 8 for s in t.stride()[:3]):
            raise ValueError("rows of the cache must be contiguous and start on 16-byte boundaries")
    return (k.data_ptr(), v.data_ptr(), k.shape[0], k.shape[2], *k.stride()[:3], *v.stride()[:3])


def rotary_table(length: int, rotary_dim: int, base: float = 10000.0, scaling: Optional[dict] = None,
                 device="cuda") -> torch.Tensor:
    """float32 [length, 2, rotary_dim / 2]: the cosines and sines of positions 0 .. length - 1.

    Pair j turns by base^(-2j / rotary_dim) per position; the angles are formed in 64 bits.  scaling, for
    contexts longer than the model was trained on:
      {"type": "linear", "factor": s}    positions divided by s
      {"type": "ntk", "factor": s}       base * s^(d / (d - 2)): the slowest pair is stretched by s
      {"type": "yarn", "factor": s, "original_length": L, "beta_fast": 32, "beta_slow": 1}
          pairs that make more than beta_fast turns over L stay, those with fewer than beta_slow are stretched
          by s, a ramp between; cosines and sines are scaled by 0.1 ln(s) + 1 ("attention_factor" overrides)
    """
    if length < 1 or rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("length must be positive and rotary_dim even")
    d, half = rotary_dim, rotary_dim // 2
    j = torch.arange(half, dtype=torch.float64, device=device)
    mscale = 1.0
    freq = None
    if scaling is not None:
        kind, s = scaling.get("type"), float(scaling.get("factor", 1.0))
        if not s >= 1.0:
            raise ValueError("the scaling factor must be at least 1")
        if kind == "linear":
            freq = base ** (-2.0 * j / d) / s
        elif kind == "ntk":
            if d <= 2:
                raise ValueError("ntk scaling needs rotary_dim > 2")
            freq = (base * s ** (d / (d - 2.0))) ** (-2.0 * j / d)
        elif kind == "yarn":
            L = float(scaling["original_length"])

            def pair_of(turns):  # the (real-valued) pair that makes so many turns over L positions
                return d * math.log(L / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

            lo = max(math.floor(pair_of(float(scaling.get("beta_fast", 32.0)))), 0)
            hi = min(math.ceil(pair_of(float(scaling.get("beta_slow", 1.0)))), d - 1)
            ramp = ((j - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
            freq = base ** (-2.0 * j / d)
            freq = freq * (1.0 - ramp) + freq / s * ramp
            mscale = float(scaling.get("attention_factor", 0.1 * math.log(s) + 1.0))
        else:
            raise ValueError(f"unknown rotary scaling {kind!r}")
    else:
        freq = base ** (-2.0 * j / d)
    angle = torch.arange(length, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack(((angle.cos() * mscale).float(), (angle.sin() * mscale).float()), 1)


def _rows(t: torch.Tensor, name: str, shape, dtype, device) -> torch.Tensor:
    """[B, N, heads, dim] with contiguous, 16-byte aligned heads; a copy if it has not."""
    if not isinstance(t, torch.Tensor) or t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if t.dtype != dtype or t.device != device:
        raise TypeError(f"{name} must be {dtype} on {device} like the cache, got {t.dtype} on {t.device}")
    s = t.stride()
    if s[3] != 1 or (s[0] | s[1] | s[2]) & 7 or t.data_ptr() & 15:
        t = t.contiguous()
        if t.data_ptr() & 15:  # a contiguous view that starts off a boundary
            t = t.clone()
    return t


def _out_rows(out, shape, dtype, device):
    s = out.stride()
    if out.shape != shape or out.dtype != dtype or out.device != device or s[3] != 1 or \
            (s[0] | s[1] | s[2]) & 7 or out.data_ptr() & 15:
        raise ValueError("out must have q's shape, type and device, with contiguous, 16-byte aligned heads")
    return out


def rotate_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor,
                  cache: Union[PagedCache, PagedCache8], page_table: torch.Tensor, cache_lens: torch.Tensor, num_new: Optional[torch.Tensor] = None, *,
                  interleaved: bool = False, out: Optional[torch.Tensor] = None,
                  row_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotates q [B, N, q_heads, dim] and k [B, N, kv_heads, dim] by their positions, writes k and v to the cache.

    New token i of sequence b has position cache_lens[b] + i (int32 [B]); num_new [B] of the N are there
    (default: all).  table: from rotary_table, at least as long as the last position; its rotary_dim
    (a multiple of 16) may be less than dim.  Pairs are (j, j + rotary_dim / 2), or (2j, 2j + 1) with
    interleaved.  Returns the rotated q (``out``, which may be q; rows past num_new are zeros).
    Into a ``PagedCache8`` (q, k, v bfloat16 or float16) each block of 16 positions that gets new tokens gets a new
    scale, the least power of two that holds what is live in it after the call, and what it held is rescaled; blocks
    that two sequences write to must be different ones.  Tokens that are rejected later are live in their own call: the
    scale forgets them with the next one, but what was rounded beside them (held tokens, and accepted ones of that call)
    keeps what it lost under their scale, 2^-10 of it at most.
    """
    if stream is None:
        scales = (cache.k_scales, cache.v_scales) if isinstance(cache, PagedCache8) else (None, None)
        res = _short.rotate(q, k, v, table, cache.k, cache.v, page_table, cache_lens, num_new, interleaved, out,
                            row_status, *scales)
        if res is not None:
            return res
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 4:
        raise ValueError("q must be a CUDA tensor [B, N, q_heads, dim]")
    dev, shape = q.device, q.shape
    if stream is not None or _current_device() != dev.index:
        return _elsewhere(dev, stream, rotate_append, (q, k, v, table, cache, page_table, cache_lens, num_new), dict(
            interleaved=interleaved, out=out, row_status=row_status))
    B, N, Hq, D = shape
    pages, scales, dtype, _ = _of_cache(cache, q, written=True)
    if D != cache.head_dim or dev != cache.device:
        raise ValueError(f"the cache has heads of {cache.head_dim} on {cache.device}")
    if table.dim() != 3 or table.shape[1] != 2 or table.dtype != torch.float32 or table.device != dev or \
            not table.is_contiguous():
        raise ValueError("table must be a contiguous float32 CUDA tensor [length, 2, rotary_dim / 2]")
    tlen, _, half = table.shape
    if half % 8 or 2 * half > D or half < 8:
        raise ValueError(f"rotary_dim must be a multiple of 16 and at most {D}, got {2 * half}")
    kv = (B, N, cache.kv_heads, D)
    x = _rows(q, "q", shape, dtype, dev)
    k = _rows(k, "k", kv, dtype, dev)
    v = _rows(v, "v", kv, dtype, dev)
    o = torch.empty(shape, dtype=dtype, device=dev) if out is None else _out_rows(out, shape, dtype, dev)
    pt = _page_table(page_table, B, dev)
    lens = _vec(cache_lens, B, torch.int32, dev, "cache_lens")
    new = _vec(num_new, B, torch.int32, dev, "num_new")
    _status(row_status, B, dev)
    xs, os, ks, vs = x.stride(), o.stride(), k.stride(), v.stride()
    args = _ROTATE.pack(
        _ROTATE.size, x.data_ptr(), o.data_ptr(), k.data_ptr(), v.data_ptr(), _DTYPE[dtype], B, N, Hq, cache.kv_heads, D,
        xs[0], xs[1], xs[2], os[0], os[1], os[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], table.data_ptr(), tlen,
        2 * half, 1 if interleaved else 0, *pages, pt.data_ptr(), pt.stride(0), pt.shape[1], lens.data_ptr(),
        _p(new), _p(row_status))
    if scales is None:
        _check(_library().spec_verify_rotate_append(args, _raw_stream(dev.index)))
    else:
        _check(_library().spec_verify_rotate_append_ex(args, _ROTATE_OPTIONS.pack(_ROTATE_OPTIONS.size, *scales),
                                                       _raw_stream(dev.index)))
    return o


def read_cache(cache: PagedCache8, page_table: torch.Tensor, first, N: int, count: Optional[torch.Tensor] = None, *,
               dtype: torch.dtype = torch.bfloat16, row_status: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values that an 8-bit cache holds: k, v [B, N, kv_heads, dim] of positions first[b] .. first[b] + N - 1
    (int32 [B]; count [B] of the N are wanted, default all; the others are zeros), code times scale rounded to dtype."""
    if not isinstance(cache, PagedCache8):
        raise TypeError("read_cache takes a PagedCache8")
    if stream is None and dtype in (torch.bfloat16, torch.float16):
        res = _short.read(cache.k, cache.v, cache.k_scales, cache.v_scales, page_table, first, N, count,
                          dtype == torch.float16, row_status)
        if res is not None:
            return res
    if not cache.k.is_cuda:
        raise ValueError("the cache must be on a CUDA device")
    dev = cache.device
    if stream is not None or _current_device() != dev.index:
        return _elsewhere(dev, stream, read_cache, (cache, page_table, first, N, count), dict(dtype=dtype,
                                                                                              row_status=row_status))
    pages, scales, held = _pages8(cache)  # (held: until the call is enqueued)
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [B, pages a sequence]")
    B, H, D = page_table.shape[0], cache.kv_heads, cache.head_dim
    pt = _page_table(page_table, B, dev)
    lens = _vec(first, B, torch.int32, dev, "first")
    new = _vec(count, B, torch.int32, dev, "count")
    _status(row_status, B, dev)
    k, v = (torch.empty((B, N, H, D), dtype=dtype, device=dev) for _ in "kv")
    _check(_library().spec_verify_read_cache(_READ.pack(
        _READ.size, k.data_ptr(), v.data_ptr(), _DTYPE[dtype], B, N, H, D, *pages, pt.data_ptr(), pt.stride(0), pt.shape[1],
        lens.data_ptr(), _p(new), *scales, _p(row_status)), _raw_stream(dev.index)))
    return k, v


def attention_workspace_size(B: int, N: int, q_heads: int, kv_heads: int, dim: int) -> int:
    """Bytes of workspace that one paged_attention call of this shape needs (0 for a shape it does not take)."""
    return int(_library().spec_verify_attention_workspace_size(B, N, q_heads, kv_heads, dim))


def paged_attention(q: torch.Tensor, cache: Union[PagedCache, PagedCache8], page_table: torch.Tensor,
                    cache_lens: torch.Tensor, num_new: Optional[torch.Tensor] = None, *,
                    scale: Optional[float] = None, window: int = 0, sinks: int = 0,
                    max_context: Optional[int] = None, out: Optional[torch.Tensor] = None,
                    row_status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    wait_limit_ns: int = 0, stream=None) -> torch.Tensor:
    """Attention of the new tokens q [B, N, q_heads, dim] (dim 64 or 128) over the cache that holds their keys.

    Token i of sequence b sees the positions up to cache_lens[b] + i, with window > 0 only the last ``window``
    of them and the first ``sinks`` positions (pages between the two are not touched: their table entries may be
    anything).  Over a ``PagedCache8`` q is bfloat16 or float16 and the products are formed in float16 with 32-bit sums.
    scale: default 1 / sqrt(dim).  max_context: the host's upper bound of cache_lens + num_new
    (default: the page table's width); it only sizes the launch.  Rows past num_new are zeros.
    workspace: uint8 of attention_workspace_size() bytes; calls on one must not overlap on the GPU (default: one kept
    for each stream, or the graph's own memory while a graph is captured).  Threads may share a stream.
    """
    if stream is None and workspace is None:
        scales = (cache.k_scales, cache.v_scales) if isinstance(cache, PagedCache8) else (None, None)
        res = _short.attention(q, cache.k, cache.v, page_table, cache_lens, num_new, scale, window, max_context, out,
                               row_status, wait_limit_ns, sinks, *scales)
        if res is not None:
            return res
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 4:
        raise ValueError("q must be a CUDA tensor [B, N, q_heads, dim]")
    dev, shape = q.device, q.shape
    if stream is not None or _current_device() != dev.index:
        return _elsewhere(dev, stream, paged_attention, (q, cache, page_table, cache_lens, num_new), dict(
            scale=scale, window=window, sinks=sinks, max_context=max_context, out=out, row_status=row_status,
            workspace=workspace, wait_limit_ns=wait_limit_ns))
    B, N, Hq, D = shape
    (pages, scales, dtype, held), Hkv = _of_cache(cache, q), cache.kv_heads  # (held: until the call is enqueued)
    if D != cache.head_dim or dev != cache.device:
        raise ValueError(f"the cache has heads of {cache.head_dim} on {cache.device}")
    if Hq % Hkv:
        raise ValueError(f"{Hq} query heads cannot share {Hkv} cache heads evenly")
    if window < 0:
        raise ValueError("window must be 0 (none) or positive")
    if sinks < 0:
        raise ValueError("sinks must be 0 (none) or positive")
    x = _rows(q, "q", shape, dtype, dev)
    o = torch.empty(shape, dtype=dtype, device=dev) if out is None else _out_rows(out, shape, dtype, dev)
    pt = _page_table(page_table, B, dev)
    lens = _vec(cache_lens, B, torch.int32, dev, "cache_lens")
    new = _vec(num_new, B, torch.int32, dev, "num_new")
    _status(row_status, B, dev)
    lib, raw = _library(), _raw_stream(dev.index)
    xs, os = x.stride(), o.stride()
    with _attend_lock:
        if workspace is None:
            workspace = _workspace(lib.spec_verify_attention_workspace_size(B, N, Hq, Hkv, D), dev, raw)
        args = _ATTENTION.pack(
            _ATTENTION.size, x.data_ptr(), o.data_ptr(), _DTYPE[dtype], B, N, Hq, Hkv, D, xs[0], xs[1], xs[2],
            os[0], os[1], os[2], 1.0 / math.sqrt(D) if scale is None else float(scale), window, max_context or 0,
            *pages, pt.data_ptr(), pt.stride(0), pt.shape[1], lens.data_ptr(), _p(new), workspace.data_ptr(),
            workspace.numel(), _p(row_status), wait_limit_ns)
        if scales is None and not sinks:
            status = lib.spec_verify_attention(args, raw)
        else:
            status = lib.spec_verify_attention_ex(args, _ATTENTION_OPTIONS.pack(
                _ATTENTION_OPTIONS.size, sinks, *(scales or _NO_SCALES)), raw)
    _check(status)
    return o


# ---------------------------------------------------------------------------
# drawing tokens
# ---------------------------------------------------------------------------
def sample(logits: torch.Tensor, uniforms: torch.Tensor, temperature=None, top_k=None, top_p=None, min_p=None, *,
           row_status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """A token of every row of logits [B, N, V] (float32 or bfloat16, CUDA), from given random numbers.

    uniforms: float32 [B, N], each in [0, 1).  temperature (0: greedy), top_k (0: none), top_p, min_p: per-sequence
    tensors, sequences or scalars.  Kept are the top_k largest (of equal logits the lower id first), of these the
    shortest run of the likeliest with a mass of at least top_p of theirs, of these those at least min_p times as likely
    as the likeliest; the token is the first in the order of ids up to which the kept mass exceeds uniform times all of
    it.  Without min_p this is the q that spec_verify forms of the logits with the same temperature, top_k and top_p;
    it has no min_p, so drafts for it are drawn without one (with one the accepted text is not the target's).
    Returns tokens int32 [B, N] and the probability that each had, float32 [B, N].  Rows with a bad parameter or random
    number, a NaN or +inf logit or no finite logit get -1 and NaN (and their bits in row_status).
    """
    if stream is None:
        res = _short.sample(logits, uniforms, temperature, top_k, top_p, min_p, row_status)
        if res is not None:
            return res
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dim() != 3:
        raise ValueError("logits must be a CUDA tensor [B, N, V]")
    dev = logits.device
    if stream is not None or _current_device() != dev.index:
        return _elsewhere(dev, stream, sample, (logits, uniforms, temperature, top_k, top_p, min_p),
                          dict(row_status=row_status))
    code = _DTYPE.get(logits.dtype)
    if code not in (0, 1):
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    B, N, V = logits.shape
    x = logits if logits.stride(2) == 1 or V == 1 else logits.contiguous()
    if not isinstance(uniforms, torch.Tensor) or uniforms.dtype != torch.float32 or uniforms.device != dev or \
            tuple(uniforms.shape) != (B, N):
        raise ValueError(f"uniforms must be a float32 CUDA tensor [{B}, {N}]")
    if uniforms.stride(1) != 1 and N > 1:
        uniforms = uniforms.contiguous()
    t = _vec(temperature, B, torch.float32, dev, "temperature")
    k = _vec(top_k, B, torch.int32, dev, "top_k")
    p = _vec(top_p, B, torch.float32, dev, "top_p")
    m = _vec(min_p, B, torch.float32, dev, "min_p")
    _status(row_status, B, dev)
    tokens = torch.empty((B, N), dtype=torch.int32, device=dev)
    probs = torch.empty((B, N), dtype=torch.float32, device=dev)
    _check(_library().spec_verify_sample(_SAMPLE.pack(
        _SAMPLE.size, x.data_ptr(), code, B, N, V, x.stride(0), x.stride(1), uniforms.data_ptr(), uniforms.stride(0), _p(t),
        _p(k), _p(p), _p(m), tokens.data_ptr(), probs.data_ptr(), _p(row_status)), _raw_stream(dev.index)))
    return tokens, probs
