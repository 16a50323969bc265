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

from typing import Optional

import torch

from . import _lib

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
        store = _STORE[kv]
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
        self._ws: dict = {}        # (stream, Hq) -> workspace
        self._ws_bytes: dict = {}  # Hq -> bytes
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
        return _lib._raw_stream(None, self.device)

    def _on_device(self):
        """A guard that makes the cache's device the current one."""
        if self.device.type != "cuda" or \
                torch.cuda.current_device() == self.device.index:
            return _NO_GUARD
        return torch.cuda.device(self.device)

    # -- which sequences hold what -------------------------------------------
    def reset(self):
        """Empty every slot."""
        with self._on_device():
            _lib.fc_pages_reset(self.pages, self._stream())

    def begin(self, slots, counts=None, rows: int = 0):
        """Open the batch of a step: row i is ``slots[i]``, which grows by
        ``counts[i]`` tokens (an int for all rows; one each by default).
        Missing pages are taken, a shared last page is copied first. ``rows``
        pads the batch with empty rows (for a captured graph of fixed size).
        Raises FcError with FC_ERR_CAPACITY, nothing changed, when the pages
        do not suffice."""
        slots = _ints(slots)
        if isinstance(counts, int):
            counts = [counts] * len(slots)
        elif counts is not None:
            counts = _ints(counts)
            if len(counts) != len(slots):
                raise ValueError("one count per slot")
        with self._on_device():
            _lib.fc_pages_begin(self.pages, slots, counts,
                                rows or len(slots), self._stream())

    def fork(self, src, dst):
        """Slot ``dst[i]`` (empty) shares the pages of ``src[i]``."""
        src, dst = _ints(src), _ints(dst)
        if len(src) != len(dst):
            raise ValueError("one source per destination")
        with self._on_device():
            _lib.fc_pages_fork(self.pages, src, dst, self._stream())

    def free(self, slots):
        """Empty the slots; pages no other slot shares become free."""
        with self._on_device():
            _lib.fc_pages_free(self.pages, _ints(slots), self._stream())

    def crop(self, slot: int, tokens_to_remove: int):
        """Remove the last ``-tokens_to_remove`` tokens of a slot (a negative
        count, as ``CodecKVCache.crop``)."""
        if tokens_to_remove > 0:
            raise ValueError("crop takes a negative count of tokens to remove")
        with self._on_device():
            _lib.fc_pages_crop(self.pages, int(slot), int(tokens_to_remove),
                               self._stream())

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

    def seq_len(self, slot: int) -> int:
        return int(self._h_lens[slot])

    @property
    def free_pages(self) -> int:
        return int(self.pages.n_free)

    @property
    def rows(self) -> int:
        """Rows of the open batch (0: none)."""
        return int(self.pages.n_rows)

    # -- a layer's data ------------------------------------------------------
    def _check_tokens(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.shape[1] != self.Hk or \
                k.shape[3] != self.D:
            raise ValueError("tokens must be (B, %d, M, %d), got %s and %s"
                             % (self.Hk, self.D, tuple(k.shape),
                                tuple(v.shape)))
        if k.dtype != self.token_dtype or v.dtype != self.token_dtype:
            raise ValueError("tokens must be %s" % self.token_dtype)
        if k.device != self.device or v.device != self.device:
            raise ValueError("tokens must be on %s" % self.device)

    def append(self, k: torch.Tensor, v: torch.Tensor, layer: int = 0):
        """Write the open batch's new tokens: (B, Hk, M, D), whose B * M
        tokens are the rows' new tokens in order ((1, Hk, N, D) for packed
        prompts, (rows, Hk, m, D) for m tokens each)."""
        self._check_tokens(k, v)
        with self._on_device():
            _lib.fc_paged_append(self.pages, layer, k, v, self._stream())

    def _workspace(self, Hq: int, stream: int) -> torch.Tensor:
        n = self._ws_bytes.get(Hq)
        if n is None:
            n = _lib.fc_paged_workspace_bytes(Hq, self.Hk, self.D)
            if n == 0:
                raise _lib.FcError(_lib.FC_ERR_UNSUPPORTED,
                                   "fc_paged_workspace_bytes")
            self._ws_bytes[Hq] = n
        if self.device.type == "cuda" and \
                torch._C._cuda_isCurrentStreamCapturing():
            # a graph's own: graphs may be replayed side by side
            return torch.zeros(n, dtype=torch.uint8, device=self.device)
        ws = self._ws.get((stream, Hq))
        if ws is None:
            ws = self._ws[stream, Hq] = torch.zeros(
                n, dtype=torch.uint8, device=self.device)
        return ws

    def _out(self, q, out, out_dtype, lse):
        if q.dim() != 4 or q.shape[0] != self.pages.n_rows or \
                q.shape[2] != 1 or q.shape[3] != self.D:
            raise ValueError("q must be (%d, Hq, 1, %d) for the open batch, "
                             "got %s" % (self.pages.n_rows, self.D,
                                         tuple(q.shape)))
        if q.device != self.device:
            raise ValueError("q must be on %s" % self.device)
        if q.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("q must be bfloat16 or float32")
        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype, device=self.device)
        elif out.shape != q.shape or out.device != self.device or \
                out.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out must be a bfloat16 or float32 tensor of "
                             "q's shape on %s" % self.device)
        if lse is not None and (lse.shape != q.shape[:2] or
                                lse.dtype != torch.float32 or
                                lse.device != self.device or
                                not lse.is_contiguous()):
            raise ValueError("lse must be a contiguous float32 (rows, Hq) "
                             "tensor on %s" % self.device)
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
        out = self._out(q, out, out_dtype, lse)
        with self._on_device():
            s = self._stream()
            _lib.fc_paged_attention(
                self.pages, layer, q, out, lse, 0.0 if softmax_scale is None
                else softmax_scale, window, sinks,
                self._workspace(q.shape[1], s), s)
        return out

    def step(self, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
             layer: int = 0, out: Optional[torch.Tensor] = None,
             softmax_scale: Optional[float] = None, window: int = 0,
             sinks: int = 0, out_dtype: torch.dtype = torch.float32,
             lse: Optional[torch.Tensor] = None) -> torch.Tensor:
        """``append`` of one token per row ((rows, Hk, 1, D)), then
        ``attention``, in one launch."""
        self._check_tokens(k_new, v_new)
        if k_new.shape[0] != self.pages.n_rows or k_new.shape[2] != 1:
            raise ValueError("step takes one new token per row")
        out = self._out(q, out, out_dtype, lse)
        with self._on_device():
            s = self._stream()
            _lib.fc_paged_step(
                self.pages, layer, q, k_new, v_new, out, lse,
                0.0 if softmax_scale is None else softmax_scale, window,
                sinks, self._workspace(q.shape[1], s), s)
        return out

    def read(self, slot: int, layer: int = 0,
             dtype: Optional[torch.dtype] = None):
        """(k, v) of one slot as dense (1, Hk, seq_len, D) rows in the token
        dtype (or ``dtype``)."""
        shape = (1, self.Hk, self.seq_len(slot), self.D)
        dt = dtype or self.token_dtype
        k = torch.empty(shape, dtype=dt, device=self.device)
        v = torch.empty(shape, dtype=dt, device=self.device)
        with self._on_device():
            _lib.fc_paged_read(self.pages, layer, int(slot), k, v,
                               self._stream())
        return k, v


class _NoGuard:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_NO_GUARD = _NoGuard()


def _ints(x):
    if isinstance(x, torch.Tensor):
        x = x.tolist()
    return [int(i) for i in x]
