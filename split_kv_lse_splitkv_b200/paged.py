"""A paged key-value cache and the calls that serve tokens from it: append, page selection, decode attention.

:class:`PagedKV` holds the caches, the scratch and the status word and marshals tensors into the C ABI's
``splitkv_paged_*`` calls; every step runs in that library's kernels.
"""
from __future__ import annotations

import ctypes
import threading
from typing import Optional

import torch

from . import binding as B
from .binding import EINVAL, EUNSUPPORTED, SplitKVError

_COUNTERS = 1024  # bytes at the head of the workspace that have to be zero before its first use
_MOST = (1 << 31) - 1
_I32, _F32 = torch.int32, torch.float32
_append, _select, _decode = B._lib.splitkv_paged_append, B._lib.splitkv_paged_select, B._lib.splitkv_paged_decode

# torch.cuda.current_device(), current_stream(device).cuda_stream and torch.empty_strided(device="cuda"), without what is
# around them (0.8 us a tensor instead of 1.3 to 1.9, in calls of 8 to 13).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_empty = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None) or (
    lambda shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype, device="cuda"))


def rope_table(n_positions: int, rope_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """float32 [n_positions, rope_dim]: for position p the cosines, then the sines, of p * base^(-2i/rope_dim). The
    angles are formed in float64: at position 10^6 a float32 angle is off by 0.03."""
    if n_positions < 1 or rope_dim < 2 or rope_dim % 2 or not base > 0:
        raise SplitKVError(EINVAL, "rope_table")
    freq = float(base) ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device) / rope_dim)
    angle = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), 1).to(torch.float32)


def _need(ok, what: str) -> None:
    if not ok:
        raise SplitKVError(EINVAL, what)


# Status words by device index, [words, number taken] each. They are never given back: a captured graph goes on reading
# and writing the word of an object that is gone.
_WORDS = 128
_words = {}
_words_lock = threading.Lock()


def _status_word(device, index) -> torch.Tensor:
    with _words_lock:
        blocks = _words.setdefault(index, [])
        if not blocks or blocks[-1][1] == _WORDS:
            with torch.inference_mode(False):  # objects made outside of that mode share them
                words = torch.zeros(_WORDS, dtype=_I32, device=device)
            if device.type == "cuda":
                torch.cuda.current_stream(device).synchronize()  # the next ones may be taken on another stream
            blocks.append([words, 0])
        block = blocks[-1]
        block[1] += 1
        return block[0][block[1] - 1:block[1]]


class PagedKV:
    """The paged cache of one attention layer and its calls.

    ``k_cache`` and ``v_cache`` are [n_pages, n_kv_heads, page_size, head_dim] tensors of equal strides (any order
    of the outer dimensions in memory: pass a transposed view of a [n_pages, page_size, n_kv_heads, head_dim]
    tensor as it is); without them they are allocated here from ``n_pages``, ``dtype`` and ``device``. ``k_bounds``
    [n_pages, n_kv_heads, 2, head_dim] holds each page's smallest and largest key channel and is needed for
    :meth:`select` only (``bounds=True`` allocates it).

    Every call takes a page table (int32 [n_seqs, up to max_pages]: row b lists the pages of sequence b) and is
    enqueued on the current stream (``stream=``: on that one, which its tensors then belong to as well: they may be
    dropped at once; what it returns is that stream's); none synchronizes (making the object does). Lengths,
    tables and token lists are read on the device, so a call captured into a CUDA graph follows their values at each
    replay. The object's scratch is shared by its decode calls: on a change of stream the new one waits for the old
    one, and a captured call has scratch of its own. A stream given by its handle has to outlive the object. Results
    carry no autograd history. The object may be dropped while calls are under way; a graph that was captured from it
    needs the caches and bounds that it was captured with until its last replay is done. Errors that only the device sees collect in :attr:`status`;
    while it is not zero, calls do no work and what they return is not written (:meth:`check_status` raises; zero it to
    go on).
    """

    def __init__(self, n_q_heads, n_kv_heads, head_dim, page_size, max_seqs, max_pages, n_pages=None, dtype=None,
                 k_cache=None, v_cache=None, k_bounds=None, bounds=False, scale=None, device="cuda"):
        _need((k_cache is None) == (v_cache is None), "PagedKV: k_cache and v_cache come together")
        if k_cache is None:
            _need(n_pages is not None and n_pages > 0, "PagedKV: n_pages or the caches")
            dtype = torch.bfloat16 if dtype is None else dtype
            shape = (int(n_pages), int(n_kv_heads), int(page_size), int(head_dim))
            k_cache = torch.empty(shape, dtype=dtype, device=device)
            v_cache = torch.empty(shape, dtype=dtype, device=device)
        shape = (k_cache.shape[0], int(n_kv_heads), int(page_size), int(head_dim))
        _need(n_pages is None or n_pages == shape[0], "PagedKV: n_pages and the caches differ")
        _need(dtype is None or dtype == k_cache.dtype, "PagedKV: dtype and the caches differ")
        _need(tuple(k_cache.shape) == shape and tuple(v_cache.shape) == shape,
              f"PagedKV: caches of {tuple(k_cache.shape)} and {tuple(v_cache.shape)}, not {shape}")
        _need(v_cache.dtype == k_cache.dtype and v_cache.device == k_cache.device and
              v_cache.stride() == k_cache.stride() and k_cache.stride(3) == 1,
              "PagedKV: the caches need the same type, device and strides, and dense channels")
        if k_bounds is None and bounds:
            k_bounds = torch.empty(shape[0], shape[1], 2, shape[3], dtype=k_cache.dtype, device=k_cache.device)
        if k_bounds is not None:
            _need(tuple(k_bounds.shape) == (shape[0], shape[1], 2, shape[3]) and k_bounds.is_contiguous() and
                  k_bounds.dtype == k_cache.dtype and k_bounds.device == k_cache.device,
                  "PagedKV: k_bounds must be a dense [n_pages, n_kv_heads, 2, head_dim] tensor of the caches' type")
        self._k_cache, self._v_cache, self._k_bounds = k_cache, v_cache, k_bounds
        self.dtype, self.device = k_cache.dtype, k_cache.device
        self.n_q_heads, self.n_kv_heads, self.head_dim = int(n_q_heads), shape[1], shape[3]
        self.page_size, self.max_seqs, self.max_pages = shape[2], int(max_seqs), int(max_pages)
        self._scale = scale
        self._dev = k_cache.get_device()  # -1 on the CPU
        self._index = self._dev if self.device.type == "cuda" else None
        self._layouts = {}  # (table width, table stride) -> splitkv_paged
        whole = self._layout(self.max_pages, self.max_pages)
        self._ws_bytes = B._lib.splitkv_paged_workspace_size(whole, self.max_seqs)
        if self._ws_bytes == 0:  # let the library say what is wrong with the description
            raise SplitKVError(_decode(whole, self.max_seqs, *[0] * 14), "PagedKV")
        self._q_strides = (self.n_q_heads * self.head_dim, self.head_dim, 1)
        self._lock = threading.Lock()
        self._ws = self._stream = None
        self._streams = set()  # those that _first_on has seen
        if self._index is None:
            self._status = _status_word(self.device, None)
        else:  # the scratch, whose counters start at zero: before any stream's first call
            if torch.cuda.is_current_stream_capturing():
                raise SplitKVError(EINVAL, "PagedKV: made during a stream capture")
            self._status = _status_word(self.device, self._index)
            self._ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=self.device)
            self._ws[:_COUNTERS].zero_()
            self._ws_at = self._ws.data_ptr()
            self._stream = torch.cuda.current_stream(self.device)
            self._stream.synchronize()
        # The object's own tensors, which it keeps.
        self._k_at, self._v_at, self._status_at = k_cache.data_ptr(), v_cache.data_ptr(), self._status.data_ptr()
        self._bounds_at = None if k_bounds is None else k_bounds.data_ptr()

    # Read only: the kernels are called with the addresses of these tensors, taken once.
    k_cache = property(lambda self: self._k_cache)
    v_cache = property(lambda self: self._v_cache)
    k_bounds = property(lambda self: self._k_bounds)
    status = property(lambda self: self._status)

    # -- marshalling. These calls are made once per layer and token: checks are plain comparisons, texts are made only where
    # one fails, and the library is called with integers.
    def _layout(self, width: int, stride: int):
        got = self._layouts.get((width, stride))
        if got is None:
            st = self._k_cache.stride()
            got = ctypes.byref(B.make_paged(self.n_q_heads, self.n_kv_heads, self.head_dim, self.page_size,
                                            self._k_cache.shape[0], width, st[:3], stride, self._scale, self.dtype))
            if len(self._layouts) < 64:
                self._layouts[(width, stride)] = got
        return got

    def _on(self, fn, stream, *args):
        """fn(*args) with the cache's device current, on `stream` where one is given."""
        if self._index is None:
            raise SplitKVError(EINVAL, f"PagedKV: the cache is on {self.device}, not on a CUDA device")
        if stream is None:
            with torch.cuda.device(self._index):
                return fn(*args)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=self.device)
        _need(stream.device == self.device, "PagedKV: a stream of another device than the cache's")
        with torch.cuda.stream(stream):
            got = fn(*args)
            if not torch._C._cuda_isCurrentStreamCapturing():
                for t in args:  # may be dropped as soon as the call returns, and belong to another stream
                    if isinstance(t, torch.Tensor):
                        t.record_stream(stream)
            return got

    def _first_on(self, raw) -> None:
        """The first call on the current stream. The object may be dropped while work of its calls is under way, on streams
        other than those its tensors were allocated on: these are not to be given to anybody else before that is done."""
        if torch._C._cuda_isCurrentStreamCapturing():
            return  # a graph's replays are no work of this stream
        now = torch.cuda.current_stream(self.device)
        for t in (self._k_cache, self._v_cache, self._k_bounds, self._ws):
            if t is not None:
                t.record_stream(now)
        self._streams.add(raw)

    def _table(self, page_table, what):
        shape, strides = page_table.shape, page_table.stride()
        if (page_table.dtype is not _I32 or len(shape) != 2 or page_table.get_device() != self._dev or
                (shape[1] > 1 and strides[1] != 1)):
            raise SplitKVError(EINVAL, f"{what}: page_table must be an int32 [n_seqs, pages] tensor on the cache's "
                               "device, its rows dense")
        n, width = shape
        stride = strides[0] if n > 1 else width
        if n > self.max_seqs or not 1 <= width <= self.max_pages or stride < width:
            raise SplitKVError(EINVAL, f"{what}: a page table of {n} x {width}, {stride} apart; made for up to "
                               f"{self.max_seqs} x {self.max_pages}, apart")
        return n, self._layout(width, stride)

    def _list(self, t, n, what, name):
        if t.dtype is not _I32 or t.shape != (n,) or t.get_device() != self._dev or not t.is_contiguous():
            raise SplitKVError(EINVAL, f"{what}: {name} must be a dense int32 [{n}] tensor on the cache's device")

    def _rows(self, t, n, heads, what, name) -> int:
        """Stride between the tokens of a [n, heads, head_dim] tensor whose heads are dense."""
        d = self.head_dim
        if t.dtype is self.dtype and t.shape == (n, heads, d) and t.get_device() == self._dev:
            token, head, one = t.stride()
            if one == 1 and (head == d or heads == 1):
                return token if n > 1 else heads * d
        raise SplitKVError(EINVAL, f"{what}: {name} must be a {self.dtype} [{n}, {heads}, {d}] tensor on the cache's "
                           "device, each token's heads dense")

    def _out(self, t, shape, dtype, what, name):
        if t.shape != shape or t.dtype is not dtype or t.get_device() != self._dev or not t.is_contiguous():
            raise SplitKVError(EINVAL, f"{what}: {name} must be a dense {dtype} tensor of {shape} on the cache's device")

    # -- the calls
    def append(self, k, v, page_table, token_seq, token_pos, q=None, rope: Optional[torch.Tensor] = None,
               interleaved: bool = False, q_out=None, stream=None):
        """Writes the keys and values of new tokens ([n_tokens, n_kv_heads, head_dim]) to their sequences' pages:
        token i goes to position ``token_pos[i]`` of sequence ``token_seq[i]``, a row of ``page_table`` (< 0:
        padding). The tokens are strictly ascending by (sequence, position). With ``rope`` (:func:`rope_table`) the
        keys are rotated on the way, and ``q`` [n_tokens, n_q_heads, head_dim] into the tensor returned. The
        bounds of the pages written follow, where the object has bounds."""
        what = "PagedKV.append"
        n = k.shape[0] if k.dim() else 0
        n_seqs, layout = self._table(page_table, what)
        ks = self._rows(k, n, self.n_kv_heads, what, "k")
        vs = self._rows(v, n, self.n_kv_heads, what, "v")
        self._list(token_seq, n, what, "token_seq")
        self._list(token_pos, n, what, "token_pos")
        qs = rope_len = rope_dim = 0
        if rope is not None:
            if rope.dtype is not _F32 or rope.dim() != 2 or rope.get_device() != self._dev or not rope.is_contiguous():
                raise SplitKVError(EINVAL, f"{what}: rope must be a dense float32 [positions, rope_dim] tensor")
            rope_len, rope_dim = rope.shape
        if q is not None:
            qs = self._rows(q, n, self.n_q_heads, what, "q")
        elif q_out is not None:
            raise SplitKVError(EINVAL, f"{what}: q_out without q")
        if q_out is not None:
            self._out(q_out, (n, self.n_q_heads, self.head_dim), self.dtype, what, "q_out")
        index = self._index
        if stream is not None or index is None or _current_device() != index:
            return self._on(self.append, stream, k, v, page_table, token_seq, token_pos, q, rope, interleaved, q_out)
        if q is not None and q_out is None:
            q_out = _empty((n, self.n_q_heads, self.head_dim), self._q_strides, self.dtype)
        raw = _raw_stream(index)
        if raw not in self._streams:
            self._first_on(raw)
        rc = _append(layout, n_seqs, n, None if q is None else q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
                     None if rope is None else rope.data_ptr(), rope_dim, rope_len, 1 if interleaved else 0,
                     page_table.data_ptr(), token_seq.data_ptr(), token_pos.data_ptr(),
                     None if q is None else q_out.data_ptr(), self._k_at, self._v_at, self._bounds_at, self._status_at,
                     raw)
        if rc:
            raise SplitKVError(rc, "splitkv_paged_append")
        return q_out

    def select(self, q, page_table, seq_lens, n_select, keep_first=1, keep_last=1, pages=None, stream=None):
        """int32 [n_seqs, n_kv_heads, n_select]: the pages (indices into the sequence's row of ``page_table``) that
        the new token of each sequence reads at each kv head, ascending, then -1. The first ``keep_first`` and last
        ``keep_last`` pages are always among them, the others are those with the largest bound on their scores. An
        ``n_select`` below ``keep_first + keep_last`` cuts the kept ones off at their end: the newest page, which holds the
        token's own key, is the first to be left out."""
        what = "PagedKV.select"
        if self._k_bounds is None:
            raise SplitKVError(EINVAL, f"{what}: the cache has no bounds (PagedKV(..., bounds=True))")
        n, layout = self._table(page_table, what)
        qs = self._rows(q, n, self.n_q_heads, what, "q")
        self._list(seq_lens, n, what, "seq_lens")
        n_select = int(n_select)
        if n_select < 1 or keep_first < 0 or keep_last < 0:
            raise SplitKVError(EINVAL, f"{what}: n_select, keep_first, keep_last")
        if n_select > B.PAGED_MAX_SELECT_PAGES:  # before a result of that size is made
            raise SplitKVError(EUNSUPPORTED, f"{what}: n_select past {B.PAGED_MAX_SELECT_PAGES}")
        shape = (n, self.n_kv_heads, n_select)
        if pages is not None:
            self._out(pages, shape, _I32, what, "pages")
        index = self._index
        if stream is not None or index is None or _current_device() != index:
            return self._on(self.select, stream, q, page_table, seq_lens, n_select, keep_first, keep_last, pages)
        if pages is None:
            pages = _empty(shape, (self.n_kv_heads * n_select, n_select, 1), _I32)
        raw = _raw_stream(index)
        if raw not in self._streams:
            self._first_on(raw)
        # Scratch of the call alone: 8 bytes per page and kv head. No sequence has more pages than its row: any larger
        # number of kept ones says the same.
        ws = _empty((n * self.n_kv_heads * page_table.shape[1] * 2 + 4,), (1,), _I32)
        rc = _select(layout, n, q.data_ptr(), qs, self._bounds_at, page_table.data_ptr(), seq_lens.data_ptr(), n_select,
                     min(int(keep_first), _MOST), min(int(keep_last), _MOST), pages.data_ptr(), self._status_at,
                     ws.data_ptr(), ws.shape[0] * 4, raw)
        if rc:
            raise SplitKVError(rc, "splitkv_paged_select")
        return pages

    def decode(self, q, page_table, seq_lens, pages=None, o=None, lse=None, stream=None):
        """(o, lse): attention of one new token of each sequence (q [n_seqs, n_q_heads, head_dim]) over the sequence's
        cached keys, the first ``seq_lens[b]`` positions of row b, or over the pages of them that ``pages``
        (:meth:`select`) lists. A sequence without keys gets o = 0, lse = -inf. To attend several new tokens
        of a sequence, list its row once for each, with the length that the token sees."""
        what = "PagedKV.decode"
        n, layout = self._table(page_table, what)
        heads = self.n_q_heads
        qs = self._rows(q, n, heads, what, "q")
        self._list(seq_lens, n, what, "seq_lens")
        n_select, pages_at = 0, None
        if pages is not None:
            n_select = pages.shape[2] if pages.dim() == 3 else 0
            if n_select < 1:
                raise SplitKVError(EINVAL, f"{what}: pages must be [n_seqs, n_kv_heads, n_select]")
            if n_select > _MOST:
                raise SplitKVError(EUNSUPPORTED, f"{what}: n_select past 31 bits")
            self._out(pages, (n, self.n_kv_heads, n_select), _I32, what, "pages")
            pages_at = pages.data_ptr()
        if o is not None:
            self._out(o, (n, heads, self.head_dim), self.dtype, what, "o")
        if lse is not None:
            self._out(lse, (n, heads), _F32, what, "lse")
        index = self._index
        if stream is not None or index is None or _current_device() != index:
            return self._on(self.decode, stream, q, page_table, seq_lens, pages, o, lse)
        if o is None:
            o = _empty((n, heads, self.head_dim), self._q_strides, self.dtype)
        if lse is None:
            lse = _empty((n, heads), (heads, 1), _F32)
        raw = _raw_stream(index)
        if raw not in self._streams:
            self._first_on(raw)
        args = (layout, n, q.data_ptr(), qs, self._k_at, self._v_at, page_table.data_ptr(), seq_lens.data_ptr(), pages_at,
                n_select, o.data_ptr(), lse.data_ptr(), self._status_at)
        if torch._C._cuda_isCurrentStreamCapturing():
            # The graph may be replayed beside other work of this object.
            rc = self._decode_apart(args, raw)
        else:
            with self._lock:
                other = raw != self._stream.cuda_stream  # the scratch is used in turn
                if other and self._capturing(self._stream):
                    rc = self._decode_apart(args, raw)  # to wait for that stream now would be to join its capture
                else:
                    if other:
                        now = torch.cuda.current_stream(self.device)
                        now.wait_stream(self._stream)
                        self._stream = now
                    rc = _decode(*args, self._ws_at, self._ws_bytes, raw)
        if rc:
            raise SplitKVError(rc, "splitkv_paged_decode")
        return o, lse

    def _decode_apart(self, args, raw) -> int:
        """With scratch of the call's own, its counters zeroed on the stream."""
        ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=self.device)
        ws[:_COUNTERS].zero_()
        return _decode(*args, ws.data_ptr(), self._ws_bytes, raw)

    @staticmethod
    def _capturing(stream) -> bool:
        with torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()

    # -- host-side reads (synchronizing; for tests and reports)
    def status_value(self) -> int:
        return int(self._status.item())

    def check_status(self):
        st = self.status_value()
        if st:
            raise RuntimeError(f"device status word 0x{st:x}")
