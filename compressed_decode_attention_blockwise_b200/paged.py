"""Paged K/V cache of many sequences of different lengths, and single-token
decode attention over it (``include/fc_paged.h``).

Where ``CodecKVCache`` holds a batch whose rows have one length, compressed,
a ``PagedKVCache`` holds sequences that come, grow, fork and go, in pages that
all layers share: bf16 or fp32 rows, or int8 rows with one fp32 scale per
(token, kv head). ``read`` hands a sequence over as the dense rows
``CodecKVCache.prefill`` takes.

A step opens a batch (``begin``: which slots grow by how many tokens), then
each layer writes its new tokens and attends (``append`` and ``attention``, or
``step`` for both in one launch). Device memory comes from torch; page
decisions and every byte of arithmetic are libfc's.
"""

from __future__ import annotations

import array
import ctypes
from typing import Optional

import torch

from . import _lib

_I64x4 = ctypes.c_int64 * 4
_FLOAT = {torch.bfloat16: _lib.FC_DTYPE_BF16, torch.float32: _lib.FC_DTYPE_F32}
_STORE = {"i8": torch.int8, "bf16": torch.bfloat16, "f32": torch.float32}


class PagedKVCache:
    """K and V of ``n_layers`` layers in ``n_pages`` pages of ``page_size``
    tokens, for up to ``n_slots`` sequences of up to ``max_pages`` pages.

    ``kv`` chooses the storage: "bf16", "f32" or "i8". Tokens have
    ``token_dtype`` (bf16 / f32 storage: that dtype). ``storage`` adopts the
    caller's tensors (k, v, k_scales, v_scales): (n_layers, n_pages, Hk,
    page_size, D) and, for "i8", fp32 (n_layers, n_pages, Hk, page_size).
    """

    def __init__(self, n_layers: int, n_slots: int, n_pages: int, Hk: int,
                 D: int, page_size: int = 16, max_pages: int = 0,
                 kv: str = "bf16", token_dtype: torch.dtype = torch.bfloat16,
                 device="cuda", storage=None):
        self.n_layers, self.n_slots, self.n_pages = n_layers, n_slots, n_pages
        self.Hk, self.D, self.page_size = Hk, D, page_size
        self.max_pages = max_pages or n_pages
        self.kv = kv
        store = _STORE.get(kv)
        if store is None:
            raise ValueError('kv must be "bf16", "f32" or "i8"')
        if kv != "i8":
            token_dtype = store
        if token_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("token_dtype must be bfloat16 or float32")
        self.token_dtype = token_dtype
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        shape = (n_layers, n_pages, Hk, page_size, D)
        if storage is None:
            self.k = torch.empty(shape, dtype=store, device=device)
            self.v = torch.empty(shape, dtype=store, device=device)
            self.k_scales = self.v_scales = None
            if kv == "i8":
                self.k_scales = torch.empty(shape[:4], dtype=torch.float32,
                                            device=device)
                self.v_scales = torch.empty_like(self.k_scales)
        else:
            self.k, self.v, self.k_scales, self.v_scales = storage
            self._check_storage(shape, store)
        i32 = dict(dtype=torch.int32)
        self.table = torch.empty((n_slots, self.max_pages), device=device,
                                 **i32)
        self.lens = torch.empty(n_slots, device=device, **i32)
        self._batch = torch.zeros((n_slots, 4), device=device, **i32)
        self._h_table = torch.full((n_slots, self.max_pages), -1, **i32)
        self._h_lens = torch.zeros(n_slots, **i32)
        self._h_refs = torch.zeros(n_pages, **i32)
        # (indexed without a tensor's cost)
        self._len_of = (ctypes.c_int32 * n_slots).from_address(
            self._h_lens.data_ptr())
        p = self.pages = _lib.FcPages()
        p.k, p.v = self.k.data_ptr(), self.v.data_ptr()
        if self.k_scales is not None:
            p.k_scales = self.k_scales.data_ptr()
            p.v_scales = self.v_scales.data_ptr()
            (p.scale_stride_layer, p.scale_stride_page,
             p.scale_stride_head) = self.k_scales.stride()[:3]
        p.dtype, p.page_size = _lib.dtype_code(store), page_size
        p.n_layers, p.n_pages, p.H, p.D = n_layers, n_pages, Hk, D
        p.stride_layer, p.stride_page, p.stride_head = self.k.stride()[:3]
        p.n_slots, p.max_pages = n_slots, self.max_pages
        p.table, p.lens = self.table.data_ptr(), self.lens.data_ptr()
        p.batch = self._batch.data_ptr()
        p.h_table = self._h_table.data_ptr()
        p.h_lens, p.h_refs = self._h_lens.data_ptr(), self._h_refs.data_ptr()
        self._lib = _lib.load()
        self._ref = ctypes.byref(p)
        self._index = -1 if device.type != "cuda" else device.index
        self._where = device if self._index < 0 else self._index
        self._rows = 0             # rows of the open batch (0: none)
        self._ws: dict = {}        # (stream, Hq) -> workspace
        self._graph_ws: dict = {}  # the same, of the capture self._capture
        self._capture = 0
        self._dense: dict = {}     # H -> strides of a dense (rows, H, 1, D)
        self.reset()

    def _check_storage(self, shape, store):
        pools = [(self.k, shape, store), (self.v, shape, store)]
        if self.kv == "i8":
            pools += [(self.k_scales, shape[:4], torch.float32),
                      (self.v_scales, shape[:4], torch.float32)]
        elif self.k_scales is not None or self.v_scales is not None:
            raise ValueError("scales belong to int8 storage only")
        for t, want, dt in pools:
            if t is None or tuple(t.shape) != tuple(want) or t.dtype != dt \
                    or t.device != self.device:
                raise ValueError("storage tensors must be %s %s on %s"
                                 % (tuple(want), dt, self.device))
            if t.stride(-1) != 1 or (t.dim() == 5 and
                                     t.stride(3) != self.D):
                raise ValueError("the rows of a page must be contiguous")
        for a, b in zip(pools[::2], pools[1::2]):
            if a[0].stride() != b[0].stride():
                raise ValueError("k and v must have the same strides")

    # -- the calls' device and stream ----------------------------------------
    def _stream(self) -> int:
        if self._index < 0:
            return 0
        return torch._C._cuda_getCurrentRawStream(self._index)

    def _on_device(self):
        """A guard that makes the cache's device the current one."""
        if self._index < 0 or torch._C._cuda_getDevice() == self._index:
            return _NO_GUARD
        return torch.cuda.device(self.device)

    # -- which sequences hold what -------------------------------------------
    def reset(self):
        """Empty every slot."""
        with self._on_device():
            _lib.fc_pages_reset(self.pages, self._stream())
        self._rows = 0

    def begin(self, slots, counts=None, rows: int = 0):
        """Open the batch of a step: row i is ``slots[i]``, which grows by
        ``counts[i]`` tokens (an int for all rows; one each by default).
        Missing pages are taken, a shared last page is copied first. ``rows``
        pads the batch with empty rows (for a captured graph of fixed size;
        a captured ``append`` writes no more tokens than it was given at its
        capture, a captured ``step`` one in a row: the batches it is replayed
        for may not have more).
        Raises FcError with FC_ERR_CAPACITY, nothing changed, when the pages
        do not suffice."""
        slots = _ints(slots)
        n = len(slots)
        if isinstance(counts, int):
            counts = array.array("i", [counts]) * n
        elif counts is not None:
            counts = _ints(counts)
            if len(counts) != n:
                raise ValueError("one count per slot")
        rows = rows or n
        with self._on_device():
            st = self._lib.fc_pages_begin(
                self._ref, slots.buffer_info()[0], None if counts is None
                else counts.buffer_info()[0], n, rows, self._stream())
        if st:
            raise _lib.FcError(st, "fc_pages_begin")
        self._rows = rows

    def fork(self, src, dst):
        """Slot ``dst[i]`` (empty) shares the pages of ``src[i]``."""
        src, dst = _ints(src), _ints(dst)
        if len(src) != len(dst):
            raise ValueError("one source per destination")
        with self._on_device():
            st = self._lib.fc_pages_fork(
                self._ref, src.buffer_info()[0], dst.buffer_info()[0],
                len(dst), self._stream())
        if st:
            raise _lib.FcError(st, "fc_pages_fork")
        self._rows = 0

    def free(self, slots):
        """Empty the slots; pages no other slot shares become free."""
        slots = _ints(slots)
        with self._on_device():
            st = self._lib.fc_pages_free(
                self._ref, slots.buffer_info()[0], len(slots), self._stream())
        if st:
            raise _lib.FcError(st, "fc_pages_free")
        self._rows = 0

    def crop(self, slot: int, tokens_to_remove: int):
        """Remove the last ``-tokens_to_remove`` tokens of a slot (a negative
        count, as ``CodecKVCache.crop``)."""
        if tokens_to_remove > 0:
            raise ValueError("crop takes a negative count of tokens to remove")
        with self._on_device():
            _lib.fc_pages_crop(self.pages, int(slot), int(tokens_to_remove),
                               self._stream())
        self._rows = int(self.pages.n_rows)

    def compact(self) -> int:
        """Pack the live pages to the front of the pools; returns how many
        there are."""
        with self._on_device():
            return _lib.fc_pages_compact(self.pages, self._stream())

    def save_map(self):
        """(table, lens): the host's copy of the map, for ``restore_map``."""
        return self._h_table.clone(), self._h_lens.clone()

    def restore_map(self, table: torch.Tensor, lens: torch.Tensor):
        """Take over a map: slot s holds ``lens[s]`` tokens in the pages
        ``table[s]`` names (CPU int32 tensors of the map's shapes)."""
        for t, like in ((table, self._h_table), (lens, self._h_lens)):
            if t.device.type != "cpu" or t.dtype != torch.int32 or \
                    t.shape != like.shape or not t.is_contiguous():
                raise ValueError("restore_map takes contiguous CPU int32 "
                                 "tensors of shape %s and %s" % (
                                     tuple(self._h_table.shape),
                                     tuple(self._h_lens.shape)))
        with self._on_device():
            _lib.fc_pages_restore(self.pages, table, lens, self._stream())
        self._rows = 0

    def seq_len(self, slot: int) -> int:
        return self._len_of[slot]

    @property
    def free_pages(self) -> int:
        return int(self.pages.n_free)

    @property
    def rows(self) -> int:
        """Rows of the open batch (0: none)."""
        return self._rows

    # -- a layer's data ------------------------------------------------------
    def _check_kind(self, k, v):
        if k.dtype != self.token_dtype or v.dtype != self.token_dtype:
            raise ValueError("tokens must be %s" % self.token_dtype)
        if k.get_device() != self._index or v.get_device() != self._index:
            raise ValueError("tokens must be on %s" % self.device)

    def append(self, k: torch.Tensor, v: torch.Tensor, layer: int = 0):
        """Write the open batch's new tokens: (B, Hk, M, D), whose B * M
        tokens are the rows' new tokens in order ((1, Hk, N, D) for packed
        prompts, (rows, Hk, m, D) for m tokens each)."""
        shape = k.shape
        if len(shape) != 4 or shape != v.shape or shape[1] != self.Hk or \
                shape[3] != self.D:
            raise ValueError("tokens must be (B, %d, M, %d), got %s and %s"
                             % (self.Hk, self.D, tuple(shape),
                                tuple(v.shape)))
        self._check_kind(k, v)
        with self._on_device():
            st = self._lib.fc_paged_append(
                self._ref, layer, k.data_ptr(), v.data_ptr(),
                _FLOAT[k.dtype], _I64x4(*k.stride()), _I64x4(*v.stride()),
                shape[0], shape[2], self._stream())
        if st:
            raise _lib.FcError(st, "fc_paged_append")

    def _dense_strides(self, H: int):
        d = self._dense[H] = _I64x4(H * self.D, self.D, self.D, 1)
        return d

    def _new_workspace(self, Hq: int):
        """(tensor, address, bytes) of a zeroed workspace."""
        n = _lib.fc_paged_workspace_bytes(Hq, self.Hk, self.D)
        if n == 0:
            raise _lib.FcError(_lib.FC_ERR_UNSUPPORTED,
                               "fc_paged_workspace_bytes")
        t = torch.zeros(n, dtype=torch.uint8, device=self.device)
        return t, t.data_ptr(), n

    def _refuse_query(self, q):
        raise ValueError(
            "q must be a bfloat16 or float32 (%d, Hq, 1, %d) tensor on %s for "
            "the open batch, got %s %s on %s" % (
                self._rows, self.D, self.device, q.dtype, tuple(q.shape),
                q.device))

    def _attend(self, q, new, layer, out, softmax_scale, window, sinks,
                out_dtype, lse):
        shape = q.shape
        code = _FLOAT.get(q.dtype)
        if code is None or len(shape) != 4 or shape[0] != self._rows or \
                shape[2] != 1 or shape[3] != self.D or \
                q.get_device() != self._index:
            self._refuse_query(q)
        Hq = shape[1]
        dense = self._dense.get(Hq) or self._dense_strides(Hq)
        if out is None:
            out = torch.empty_like(q, dtype=out_dtype,
                                   memory_format=torch.contiguous_format)
            strides = dense
        else:
            out_dtype = out.dtype
            if out.shape != shape or out.get_device() != self._index:
                raise ValueError("out must have q's shape %s, on %s"
                                 % (tuple(shape), self.device))
            strides = _I64x4(*out.stride())
        out_code = _FLOAT.get(out_dtype)
        if out_code is None:
            raise ValueError("out must be bfloat16 or float32")
        lse_ptr = None
        if lse is not None:
            if lse.shape != shape[:2] or lse.dtype != torch.float32 or \
                    lse.get_device() != self._index or \
                    not lse.is_contiguous():
                raise ValueError("lse must be a contiguous float32 (rows, Hq) "
                                 "tensor on %s" % self.device)
            lse_ptr = lse.data_ptr()
        if self._index >= 0 and torch._C._cuda_getDevice() != self._index:
            with torch.cuda.device(self.device):
                return self._attend(q, new, layer, out, softmax_scale, window,
                                    sinks, out_dtype, lse)
        s = self._stream()
        held = self._ws
        if self._index >= 0 and torch._C._cuda_isCurrentStreamCapturing():
            # the graph's own: graphs may be replayed side by side. Kept while
            # it is captured, so that its calls share one zeroing; after that
            # the graph's memory pool keeps the memory, as any temporary's.
            capture = self._lib.fc_paged_capture_id(s)
            if capture != self._capture:
                self._capture, self._graph_ws = capture, {}
            held = self._graph_ws
        ws = held.get((s, Hq))
        if ws is None:
            ws = held[s, Hq] = self._new_workspace(Hq)
        if softmax_scale is None:
            softmax_scale = 0.0
        qs = dense if q.is_contiguous() else _I64x4(*q.stride())
        if new is None:
            st = self._lib.fc_paged_attention(
                self._ref, layer, q.data_ptr(), code, qs, Hq, softmax_scale,
                window, sinks, ws[1], ws[2], out.data_ptr(), out_code,
                strides, lse_ptr, s)
        else:
            k, v = new
            new_dense = self._dense.get(self.Hk) or \
                self._dense_strides(self.Hk)
            st = self._lib.fc_paged_step(
                self._ref, layer, q.data_ptr(), code, qs, Hq, k.data_ptr(),
                v.data_ptr(), _FLOAT[k.dtype],
                new_dense if k.is_contiguous() else _I64x4(*k.stride()),
                new_dense if v.is_contiguous() else _I64x4(*v.stride()),
                softmax_scale, window, sinks, ws[1], ws[2], out.data_ptr(),
                out_code, strides, lse_ptr, s)
        if st:
            raise _lib.FcError(st, "fc_paged_attention" if new is None else
                               "fc_paged_step")
        return out

    def attention(self, q: torch.Tensor, layer: int = 0,
                  out: Optional[torch.Tensor] = None,
                  softmax_scale: Optional[float] = None, window: int = 0,
                  sinks: int = 0, out_dtype: torch.dtype = torch.float32,
                  lse: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of q (rows, Hq, 1, D), one token per row of the open
        batch, over the rows' sequences. ``window`` > 0 limits it to the last
        ``window`` tokens and the first ``sinks`` ones. ``lse`` (rows, Hq)
        receives the log of the softmax's sum. A row without tokens gives
        zeros (lse -inf)."""
        return self._attend(q, None, layer, out, softmax_scale, window, sinks,
                            out_dtype, lse)

    def step(self, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
             layer: int = 0, out: Optional[torch.Tensor] = None,
             softmax_scale: Optional[float] = None, window: int = 0,
             sinks: int = 0, out_dtype: torch.dtype = torch.float32,
             lse: Optional[torch.Tensor] = None) -> torch.Tensor:
        """``append`` of one token per row ((rows, Hk, 1, D)), then
        ``attention``, in one launch."""
        want = (self._rows, self.Hk, 1, self.D)
        if k_new.shape != want or v_new.shape != want:
            raise ValueError("step takes one new token per row, %s, got %s "
                             "and %s" % (want, tuple(k_new.shape),
                                         tuple(v_new.shape)))
        self._check_kind(k_new, v_new)
        return self._attend(q, (k_new, v_new), layer, out, softmax_scale,
                            window, sinks, out_dtype, lse)

    def read(self, slot: int, layer: int = 0,
             dtype: Optional[torch.dtype] = None):
        """(k, v) of one slot as dense (1, Hk, seq_len, D) rows in the token
        dtype (or ``dtype``)."""
        dt = dtype or self.token_dtype
        code = _FLOAT.get(dt)
        if code is None:
            raise ValueError("rows are read as bfloat16 or float32")
        T = self.seq_len(slot)
        k = torch.empty(1, self.Hk, T, self.D, dtype=dt, device=self._where)
        v = torch.empty_like(k)
        strides = _I64x4(self.Hk * T * self.D, T * self.D, self.D, 1)
        with self._on_device():
            st = self._lib.fc_paged_read(
                self._ref, layer, slot, k.data_ptr(), v.data_ptr(), code,
                strides, strides, T, self._stream())
        if st:
            raise _lib.FcError(st, "fc_paged_read")
        return k, v


class _NoGuard:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_NO_GUARD = _NoGuard()


def _ints(x):
    """A host int32 array of the integers in x (array.array converts several
    times faster than a ctypes array does)."""
    if isinstance(x, torch.Tensor):
        x = x.tolist()
    return array.array("i", x)
