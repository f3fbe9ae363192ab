"""A paged key-value cache on the device, and the attention that reads it.

Binding of the exl3_kv_* and exl3_paged_attention calls (include/exl3.h):
argument checks and marshalling only.  The bookkeeping -- page tables, lengths,
reference counts, free pages -- lives in device tensors and is read and written
by the kernels alone, so every call can be captured in a CUDA graph and none
waits for the host.  What the kernels find wrong (a bad list, too few pages) is
therefore reported by ``KvCache.check()``, which synchronises.

A step of a model with L layers, for a batch of sequences ``seqs``:

    cache.extend(seqs, m)                               # room for m tokens each
    for layer in range(L):
        ...                                             # q, k, v products
        cache.write(layer, seqs, k, v)
        o = cache.attention(layer, seqs, q, workspace=ws)
        ...                                             # o product, MLP
    cache.truncate(seqs, accepted)                      # drop rejected tokens

All calls work on the current CUDA device, which must be the cache's, and on
the current stream or the one given.  Inference only: no backward pass.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import exl3 as ex

MAX_LIST = 1024         # entries of a list of sequences

_F16, _I32 = torch.float16, torch.int32
_extend, _write, _truncate = ex._binding.kv_extend, ex._binding.kv_write, ex._binding.kv_truncate
_fork, _compact, _attention = ex._binding.kv_fork, ex._binding.kv_compact, ex._binding.paged_attention


class KvCache:
    """k, v: (n_layers, n_pages, n_heads, page_size, head_dim) fp16; table:
    (n_seqs, max_pages) int32; lens: (n_seqs,) int32; refs: (n_pages,) int32;
    free: (ceil(n_pages / 32),) int32 bits.  The cache takes the tensors as
    they are (``KvCache.empty`` makes and clears them); its scratch memory is
    cleared on the current stream."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                 refs: torch.Tensor, free: torch.Tensor):
        if k.dim() != 5 or table.dim() != 2:
            raise ValueError("expected k of (n_layers, n_pages, n_heads, page_size, head_dim) and table of "
                             "(n_seqs, max_pages)")
        n_layers, n_pages, n_heads, page_size, head_dim = k.shape
        n_seqs, max_pages = table.shape
        ex._expect(k, "k", torch.float16, k.shape)
        ex._expect(v, "v", torch.float16, k.shape)
        ex._expect(table, "table", torch.int32, (n_seqs, max_pages))
        ex._expect(lens, "lens", torch.int32, (n_seqs,))
        ex._expect(refs, "refs", torch.int32, (n_pages,))
        ex._expect(free, "free", torch.int32, ((n_pages + 31) // 32,))
        self.k, self.v, self.table, self.lens, self.refs, self.free = k, v, table, lens, refs, free
        self.n_layers, self.n_pages, self.n_heads = n_layers, n_pages, n_heads
        self.page_size, self.head_dim = page_size, head_dim
        self.n_seqs, self.max_pages = n_seqs, max_pages
        n = int(ex.lib.exl3_kv_scratch_bytes(n_pages))
        if n == 0:
            raise ex.Exl3Error(ex.EXL3_ERR_UNSUPPORTED, f"a cache of {n_pages} pages")
        self.scratch = torch.zeros(n, dtype=torch.uint8, device=k.device)
        self.device, self._index = k.device, k.get_device()
        self._scale = 1.0 / math.sqrt(head_dim)
        self._desc = ex.Cache(k.data_ptr(), v.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr(),
                              free.data_ptr(), self.scratch.data_ptr(), n_layers, n_pages, n_heads, page_size,
                              head_dim, n_seqs, max_pages)
        self._ref, self._at = ctypes.byref(self._desc), ctypes.addressof(self._desc)

    @classmethod
    def empty(cls, n_layers: int, n_pages: int, n_heads: int, page_size: int, head_dim: int, n_seqs: int,
              max_pages: int, device=None, stream=None) -> "KvCache":
        """An empty cache with memory of its own (zero-filled keys and values)."""
        if stream is not None:
            with torch.cuda.stream(stream):             # what is allocated here belongs to the stream that uses it
                return cls.empty(n_layers, n_pages, n_heads, page_size, head_dim, n_seqs, max_pages, device)
        device = device or "cuda"
        pool = lambda: torch.zeros((n_layers, n_pages, n_heads, page_size, head_dim), dtype=torch.float16, device=device)
        words = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)
        cache = cls(pool(), pool(), words(n_seqs, max_pages), words(n_seqs), words(n_pages), words((n_pages + 31) // 32))
        cache.reset()
        return cache

    # ------------------------------------------------------------ checks ---
    # Small calls are bound by the host, so each check is one condition on its
    # usual path.

    def _list(self, t: Optional[torch.Tensor], what: str, n: int) -> Optional[int]:
        """Checks a list of n int32 numbers; its address, None for no list."""
        if t is None:
            return None
        if t.dtype is _I32 and t.shape == (n,) and n <= MAX_LIST and t.is_contiguous() and t.get_device() == self._index:
            return t.data_ptr()
        if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{what}: expected a contiguous one-dimensional int32 tensor on {self.device}, got {t.dtype} "
                             f"of shape {tuple(t.shape)} on {t.device}")
        if t.shape[0] != n:
            raise ValueError(f"{what}: expected {n} entries, got {t.shape[0]}")
        raise ex.Exl3Error(ex.EXL3_ERR_UNSUPPORTED, f"{what}: a list of more than {MAX_LIST} entries")

    def _rows(self, t: torch.Tensor, what: str, n: int, heads: int):
        """Checks (n, m, heads, head_dim) rows, dense within a row; returns m and
        the strides between entries and between rows."""
        shape = t.shape
        if len(shape) != 4 or t.dtype is not _F16 or shape[0] != n or shape[2] != heads or \
                shape[3] != self.head_dim or t.get_device() != self._index:
            raise ValueError(f"{what}: expected fp16 of shape ({n}, m, {heads}, {self.head_dim}) on {self.device}, got "
                             f"{t.dtype} {tuple(shape)} on {t.device}")
        m, (s0, s1, s2, s3) = shape[1], t.stride()
        if m <= 1:
            s1 = 0
        if n <= 1:
            s0 = 0
        if s3 != 1 or (s2 != self.head_dim and heads > 1) or s1 % 8 or s0 % 8:
            raise ValueError(f"{what}: the heads of a row must lie one behind the other, rows and entries a multiple of "
                             f"8 elements apart; strides are {t.stride()}")
        return m, s0, s1

    @staticmethod
    def _alike(t: torch.Tensor, other: torch.Tensor) -> bool:
        return t.dtype is other.dtype and t.shape == other.shape and t.stride() == other.stride() and \
            t.get_device() == other.get_device()

    def _where(self, stream):
        """The stream's handle; the cache's device must be the current one."""
        if ex._current_device() != self._index:
            raise ValueError(f"the cache is on {self.device}, the current device is cuda:{torch.cuda.current_device()}")
        return ex._raw_stream(self._index) if stream is None else stream.cuda_stream

    @staticmethod
    def _entries(t: torch.Tensor, what: str) -> int:
        if t.dim() != 1:
            raise ValueError(f"{what}: expected a one-dimensional tensor, got shape {tuple(t.shape)}")
        return t.shape[0]

    # ------------------------------------------------------- bookkeeping ---

    def reset(self, stream=None):
        """No sequence holds anything, every page is free."""
        ex._check(ex.lib.exl3_kv_reset(self._ref, self._where(stream)), "exl3_kv_reset")

    def status(self, stream=None) -> int:
        """Synchronises, then reads and clears the fault word: EXL3_OK,
        EXL3_ERR_CACHE_FULL or EXL3_ERR_INDEX.  While it is set, ``extend``
        and ``write`` do nothing."""
        return int(ex.lib.exl3_kv_status(self._ref, self._where(stream)))

    def check(self, stream=None):
        """``status()`` as an exception."""
        ex._check(self.status(stream), "KvCache")

    def extend(self, seqs: torch.Tensor, m: int, counts: Optional[torch.Tensor] = None, stream=None):
        """Each sequence of ``seqs`` grows by ``m`` tokens (counts: by
        counts[b], 0..m), whose keys and values ``write`` then brings."""
        n = self._entries(seqs, "seqs")
        p, c, s = self._list(seqs, "seqs", n), self._list(counts, "counts", n), self._where(stream)
        if n:
            st = _extend(self._at, n, m, p, c, s)
            if st:
                ex._check(st, "exl3_kv_extend")

    def write(self, layer: int, seqs: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
              counts: Optional[torch.Tensor] = None, stream=None):
        """Keys and values (n, m, n_heads, head_dim) of the last m (counts:
        counts[b]) tokens of each sequence, those that ``extend`` made room
        for, in one layer.  (A page that several sequences hold is written for
        all of them.)"""
        n = self._entries(seqs, "seqs")
        p, c = self._list(seqs, "seqs", n), self._list(counts, "counts", n)
        m, bs, rs = self._rows(k, "k", n, self.n_heads)
        if not self._alike(v, k):
            raise ValueError("k and v must have the same type, device, shape and strides")
        s = self._where(stream)
        if n and m:
            st = _write(self._at, layer, n, m, p, c, k.data_ptr(), v.data_ptr(), bs, rs, s)
            if st:
                ex._check(st, "exl3_kv_write")

    def truncate(self, seqs: torch.Tensor, lens: Optional[torch.Tensor] = None, stream=None):
        """Each sequence keeps its first lens[b] tokens (None: it is freed)."""
        n = self._entries(seqs, "seqs")
        p, c, s = self._list(seqs, "seqs", n), self._list(lens, "lens", n), self._where(stream)
        if n:
            st = _truncate(self._at, n, p, c, s)
            if st:
                ex._check(st, "exl3_kv_truncate")

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None):
        """Each empty sequence dst[b] shares all of src[b] from now on."""
        n = self._entries(src, "src")
        p, d, s = self._list(src, "src", n), self._list(dst, "dst", n), self._where(stream)
        if n:
            st = _fork(self._at, n, p, d, s)
            if st:
                ex._check(st, "exl3_kv_fork")

    def compact(self, stream=None):
        """Moves pages so that the used ones are the first of the pool."""
        st = _compact(self._at, self._where(stream))
        if st:
            ex._check(st, "exl3_kv_compact")

    # --------------------------------------------------------- attention ---

    def attention_workspace(self, n: int, m: int, n_q_heads: int) -> torch.Tensor:
        """Zero-filled workspace for attention calls with up to m rows per
        sequence (any number n of sequences)."""
        if n < 0:
            raise ValueError("n: expected a number of sequences")
        need = [int(ex.lib.exl3_paged_attention_workspace_bytes(r, n_q_heads, self.n_heads, self.head_dim))
                for r in range(1, m + 1)]
        if not all(need) or not need:
            raise ex.Exl3Error(ex.EXL3_ERR_UNSUPPORTED, f"attention of {m} rows with {n_q_heads} heads")
        return torch.zeros(max(need), dtype=torch.uint8, device=self.device)

    def attention_launches(self, n: int, m: int, n_q_heads: int) -> int:
        """Kernel launches of one attention call of this size."""
        return int(ex.lib.exl3_paged_attention_launches(self._ref, n, m, n_q_heads))

    def attention(self, layer: int, seqs: torch.Tensor, q: torch.Tensor, counts: Optional[torch.Tensor] = None,
                  scale: Optional[float] = None, window: int = 0, sinks: int = 0, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of the last m (counts: counts[b]) tokens of each sequence,
        q: (n, m, n_q_heads, head_dim), over that sequence.  Row i sees the
        tokens up to its own; with ``window`` only the last ``window`` of them
        and the first ``sinks`` of the sequence.  scale: 1/sqrt(head_dim) by
        default.  lse: (n, m, n_q_heads) fp32, filled with the logarithms of
        the softmax sums.  Rows from counts[b] on are left as they were (in an
        ``out`` made here: zero).  ``out`` may be ``q``."""
        if stream is not None and (out is None or workspace is None):
            with torch.cuda.stream(stream):             # what is allocated here belongs to the stream that uses it
                return self.attention(layer, seqs, q, counts, scale, window, sinks, out, lse, workspace)
        n = self._entries(seqs, "seqs")
        p, c = self._list(seqs, "seqs", n), self._list(counts, "counts", n)
        heads = q.shape[2] if q.dim() == 4 else 0
        m, qb, qr = self._rows(q, "q", n, heads)
        if out is None:
            make = torch.empty if counts is None else torch.zeros
            out = make((n, m, heads, self.head_dim), dtype=torch.float16, device=self.device)
        if self._alike(out, q):
            ob, orow = qb, qr
        else:
            mo, ob, orow = self._rows(out, "out", n, heads)
            if mo != m:
                raise ValueError(f"out: expected {m} rows per sequence, got {mo}")
        if lse is not None:
            ex._expect(lse, "lse", torch.float32, (n, m, heads), self._index)
        s = self._where(stream)
        if n == 0 or m == 0:
            return out
        if workspace is None:
            workspace = self.attention_workspace(n, m, heads)
        st = _attention(self._at, layer, n, m, p, c, q.data_ptr(), qb, qr, heads, self._scale if scale is None else scale,
                        window, sinks, out.data_ptr(), ob, orow, None if lse is None else lse.data_ptr(),
                        workspace.data_ptr(), ex._room(workspace, self._index), s)
        if st:
            ex._check(st, "exl3_paged_attention")
        return out
