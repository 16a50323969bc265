"""The paged cache's calls on the host: what they refuse, and that a failed
call leaves the host's map as it was. No kernel is launched here (device
addresses are fake, and without a GPU every launch fails with FC_ERR_CUDA)."""

import ctypes

import numpy as np
import pytest
import torch

from compressed_decode_attention_blockwise_b200 import _lib
from _paged import Model

FAKE = 0x10000  # aligned, never dereferenced here
DT = {"bf16": _lib.FC_DTYPE_BF16, "f32": _lib.FC_DTYPE_F32,
      "i8": _lib.FC_DTYPE_I8}

if torch.cuda.is_available():   # fake addresses must never reach a kernel
    pytest.skip("host checks with fake device addresses run without a GPU",
                allow_module_level=True)


class Host:
    """A descriptor over fake device memory with real host arrays."""

    def __init__(self, kv="bf16", slots=4, pages=8, max_pages=4, H=2, D=64,
                 P=16, layers=2):
        self.table = np.full((slots, max_pages), -1, np.int32)
        self.lens = np.zeros(slots, np.int32)
        self.refs = np.zeros(pages, np.int32)
        p = self.p = _lib.FcPages()
        p.k = p.v = p.table = p.lens = p.batch = FAKE
        if kv == "i8":
            p.k_scales = p.v_scales = FAKE
            p.scale_stride_head = P
            p.scale_stride_page = H * P
            p.scale_stride_layer = pages * H * P
        p.dtype, p.page_size = DT[kv], P
        p.n_layers, p.n_pages, p.H, p.D = layers, pages, H, D
        p.stride_head, p.stride_page = P * D, H * P * D
        p.stride_layer = pages * H * P * D
        p.n_slots, p.max_pages = slots, max_pages
        p.h_table = self.table.ctypes.data
        p.h_lens, p.h_refs = self.lens.ctypes.data, self.refs.ctypes.data
        p.n_free = pages

    def hold(self, rows, lens):
        """A map set directly (as an earlier call would have left it)."""
        for s, (row, n) in enumerate(zip(rows, lens)):
            self.table[s, :len(row)] = row
            self.lens[s] = n
            for g in row:
                self.refs[g] += 1
        self.p.n_free = int((self.refs == 0).sum())

    def state(self):
        f = bytes(self.p)
        return f, self.table.tobytes(), self.lens.tobytes(), \
            self.refs.tobytes()


def i32(*v):
    return (ctypes.c_int32 * max(1, len(v)))(*v)


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


@pytest.mark.parametrize("field,value,status", [
    ("k", None, "INVALID"), ("v", None, "INVALID"), ("table", None, "INVALID"),
    ("h_refs", None, "INVALID"), ("k", FAKE + 8, "INVALID"),
    ("batch", FAKE + 4, "INVALID"), ("dtype", 9, "INVALID"),
    ("k_scales", FAKE, "INVALID"), ("page_size", 0, "INVALID"),
    ("page_size", 24, "INVALID"), ("page_size", 4, "UNSUPPORTED"),
    ("page_size", 2048, "UNSUPPORTED"), ("D", 96, "UNSUPPORTED"),
    ("D", 512, "UNSUPPORTED"), ("n_layers", 0, "INVALID"),
    ("n_pages", 0, "INVALID"), ("n_slots", 0, "INVALID"),
    ("max_pages", 0, "INVALID"), ("H", 0, "INVALID"),
    ("stride_head", 16 * 64 - 8, "INVALID"),
    ("stride_page", 2 * 16 * 64 + 4, "INVALID"),
    ("stride_layer", -8, "INVALID"), ("max_pages", 1 << 28, "UNSUPPORTED"),
])
def test_bad_descriptors(field, value, status):
    h = Host()
    setattr(h.p, field, value)
    want = getattr(_lib, "FC_ERR_" + status)
    lib = _lib.load()
    assert lib.fc_pages_begin(h.p, i32(0), None, 1, 1, None) == want
    st = i64(2 * 64, 64, 64, 1)
    h.p.n_rows = 1
    assert lib.fc_paged_append(h.p, 0, FAKE, FAKE, DT["bf16"], st, st, 1, 1,
                               None) == want
    assert lib.fc_paged_read(h.p, 0, 0, FAKE, FAKE, DT["bf16"], st, st, 1,
                             None) == want


def test_int8_pages_need_scales():
    lib = _lib.load()
    for field in ("k_scales", "v_scales"):
        h = Host("i8")
        setattr(h.p, field, None)
        assert lib.fc_pages_free(h.p, i32(0), 1, None) == _lib.FC_ERR_INVALID
    h = Host("i8")
    h.p.scale_stride_head = 18
    assert lib.fc_pages_free(h.p, i32(0), 1, None) == _lib.FC_ERR_INVALID


def test_bookkeeping_refusals_change_nothing():
    lib = _lib.load()
    h = Host()
    h.hold([[0, 1], [2], [], [5]], [20, 7, 0, 16])
    before = h.state()
    inv, cap = _lib.FC_ERR_INVALID, _lib.FC_ERR_CAPACITY
    begin = lambda s, c, n, rows: lib.fc_pages_begin(
        h.p, None if s is None else i32(*s),
        None if c is None else i32(*c), n, rows, None)
    assert begin(None, None, 1, 1) == inv
    assert begin([0], None, 0, 1) == inv
    assert begin([0, 1], None, 2, 1) == inv          # fewer rows than slots
    assert begin([0], None, 1, 5) == inv             # more rows than slots
    assert begin([4], None, 1, 1) == inv
    assert begin([-1], None, 1, 1) == inv
    assert begin([1, 1], None, 2, 2) == inv          # the same slot twice
    assert begin([0], [-1], 1, 1) == inv
    assert begin([0], [4 * 16 - 20 + 1], 1, 1) == cap   # past a table row
    assert begin([0, 1, 2, 3], [44, 57, 64, 0], 4, 4) == cap  # past the pool
    fork = lambda s, d: lib.fc_pages_fork(h.p, i32(*s), i32(*d), len(d), None)
    assert fork([0], [1]) == inv                     # not empty
    assert fork([2], [2]) == inv
    assert fork([0, 1], [2, 2]) == inv
    assert fork([4], [2]) == inv and fork([0], [-1]) == inv
    assert lib.fc_pages_fork(h.p, None, i32(2), 1, None) == inv
    free = lambda *s: lib.fc_pages_free(h.p, i32(*s), len(s), None)
    assert free(4) == inv and free(0, 0) == inv and free(-1) == inv
    assert lib.fc_pages_crop(h.p, 0, 1, None) == inv
    assert lib.fc_pages_crop(h.p, 9, -1, None) == inv
    assert lib.fc_pages_crop(h.p, 0, 0, None) == _lib.FC_OK
    t = np.full((4, 4), -1, np.int32)
    n = np.zeros(4, np.int32)
    rest = lambda: lib.fc_pages_restore(h.p, t.ctypes.data, n.ctypes.data,
                                        None)
    n[0] = 17
    t[0, :2] = [3, 8]                                # a page out of range
    assert rest() == inv
    t[0, :2] = [3, 3]                                # twice in one slot
    assert rest() == inv
    n[0] = 65                                        # longer than a row
    assert rest() == inv
    n[0] = -1
    assert rest() == inv
    assert lib.fc_pages_restore(h.p, None, n.ctypes.data, None) == inv
    assert h.state() == before


def test_failed_launches_roll_the_map_back():
    """Without a GPU each launch fails: the host's map has to be unchanged,
    whatever the call had decided (pages taken, shared, dropped, moved)."""
    lib = _lib.load()
    h = Host(pages=12)
    h.hold([[0, 1], [0, 7], [], [5]], [20, 25, 0, 16])
    before = h.state()
    cuda = _lib.FC_ERR_CUDA
    assert lib.fc_pages_begin(h.p, i32(0, 1, 2), i32(1, 30, 3), 3, 4,
                              None) == cuda
    assert h.state() == before
    assert lib.fc_pages_fork(h.p, i32(0, 1), i32(2), 1, None) == cuda
    assert h.state() == before
    assert lib.fc_pages_free(h.p, i32(1, 0), 2, None) == cuda
    assert h.state() == before
    assert lib.fc_pages_crop(h.p, 1, -20, None) == cuda
    assert h.state() == before
    assert lib.fc_pages_compact(h.p, None, None) == cuda
    assert h.state() == before
    t, n = h.table.copy(), h.lens.copy()
    t[0, 0] = 9
    assert lib.fc_pages_restore(h.p, t.ctypes.data, n.ctypes.data,
                                None) == cuda
    assert h.state() == before
    assert lib.fc_pages_reset(h.p, None) == cuda
    assert h.state() == before


def _attention(h, **kw):
    D, H = int(h.p.D), int(h.p.H)
    a = dict(layer=0, q=FAKE, q_dtype=DT["bf16"], q_strides=i64(8 * D, D, D, 1),
             Hq=4 * H, scale=0.0, window=0, sinks=0, ws=FAKE, ws_bytes=1 << 30,
             out=FAKE, out_dtype=DT["f32"], out_strides=i64(8 * D, D, D, 1),
             lse=None)
    a.update(kw)
    return _lib.load().fc_paged_attention(
        h.p, a["layer"], a["q"], a["q_dtype"], a["q_strides"], a["Hq"],
        a["scale"], a["window"], a["sinks"], a["ws"], a["ws_bytes"], a["out"],
        a["out_dtype"], a["out_strides"], a["lse"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(layer=-1), "INVALID"), (dict(layer=2), "INVALID"),
    (dict(q=None), "INVALID"), (dict(out=None), "INVALID"),
    (dict(ws=None), "INVALID"), (dict(ws=FAKE + 16), "INVALID"),
    (dict(ws_bytes=64), "INVALID"), (dict(q_dtype=2), "INVALID"),
    (dict(out_dtype=2), "INVALID"), (dict(q=FAKE + 1), "INVALID"),
    (dict(out=FAKE + 2), "INVALID"), (dict(lse=FAKE + 2), "INVALID"),
    (dict(q_strides=i64(512, 64, 64, 2)), "INVALID"),
    (dict(out_strides=i64(512, 64, 64, 0)), "INVALID"),
    (dict(window=-1), "INVALID"), (dict(sinks=-1), "INVALID"),
    (dict(scale=float("nan")), "INVALID"), (dict(Hq=3), "INVALID"),
    (dict(Hq=0), "INVALID"), (dict(Hq=6), "UNSUPPORTED"),
    (dict(Hq=64), "UNSUPPORTED"),
])
def test_attention_refusals(kw, status):
    h = Host()
    h.p.n_rows = 1
    assert _attention(h, **kw) == getattr(_lib, "FC_ERR_" + status)


def test_data_calls_need_an_open_batch():
    h = Host()
    st = i64(128, 64, 64, 1)
    lib = _lib.load()
    assert _attention(h) == _lib.FC_ERR_INVALID
    assert lib.fc_paged_append(h.p, 0, FAKE, FAKE, DT["bf16"], st, st, 1, 1,
                               None) == _lib.FC_ERR_INVALID
    h.p.n_rows, h.p.n_tokens = 2, 5     # a batch that is not one token each
    append = lambda dt, B, M, k=FAKE: lib.fc_paged_append(
        h.p, 0, k, FAKE, dt, st, st, B, M, None)
    assert append(DT["bf16"], 1, 4) == _lib.FC_ERR_INVALID   # too few tokens
    assert append(DT["bf16"], 1 << 20, 1 << 20) == _lib.FC_ERR_INVALID
    assert append(DT["bf16"], -1, -5) == _lib.FC_ERR_INVALID
    assert append(DT["f32"], 1, 5) == _lib.FC_ERR_INVALID    # bf16 pages
    assert append(DT["i8"], 1, 5) == _lib.FC_ERR_INVALID
    assert append(DT["bf16"], 1, 5, None) == _lib.FC_ERR_INVALID
    assert append(DT["bf16"], 1, 5, FAKE + 1) == _lib.FC_ERR_INVALID
    D, H = 64, 2
    step = lib.fc_paged_step(
        h.p, 0, FAKE, DT["bf16"], i64(8 * D, D, D, 1), 4 * H, FAKE, FAKE,
        DT["bf16"], st, st, 0.0, 0, 0, FAKE, 1 << 30, FAKE, DT["f32"],
        i64(8 * D, D, D, 1), None, None)
    assert step == _lib.FC_ERR_INVALID


def test_read_refusals():
    h = Host()
    h.hold([[0, 1], [], [], []], [20, 0, 0, 0])
    lib = _lib.load()
    st = i64(0, 32 * 64, 64, 1)
    read = lambda **k: lib.fc_paged_read(
        h.p, k.get("layer", 0), k.get("slot", 0), k.get("k", FAKE), FAKE,
        k.get("dt", DT["bf16"]), k.get("st", st), st, k.get("T", 20), None)
    for kw in (dict(layer=2), dict(slot=4), dict(slot=-1), dict(k=None),
               dict(dt=DT["i8"]), dict(T=19), dict(k=FAKE + 8),
               dict(st=i64(0, 2048, 65, 1)), dict(st=i64(0, 2048, 64, 2))):
        assert read(**kw) == _lib.FC_ERR_INVALID, kw
    assert read(slot=1, T=0) == _lib.FC_OK    # nothing to read


def test_workspace_bytes():
    f = _lib.fc_paged_workspace_bytes
    assert f(8, 2, 64) > 0 and f(32, 2, 256) > f(16, 2, 256)
    assert f(6, 2, 64) == f(8, 0, 64) == f(8, 2, 100) == f(0, 2, 64) == 0


def test_model_copies_before_writing_shared_pages():
    """The tests' own model: two forks of one partly filled page."""
    m = Model(3, 6, 8, 4)
    assert m.begin([0], [11]) == (True, [])
    m.fork([0, 0], [1, 2])
    assert m.rows == [[0, 1]] * 3 and m.refs()[:3] == [3, 3, 0]
    ok, copies = m.begin([1, 2, 0], [1, 1, 1])
    assert ok and copies == [(1, 2), (1, 3)]      # the last one writes in place
    assert m.rows == [[0, 1], [0, 2], [0, 3]]
    m.crop(1, 8)
    assert m.rows[1] == [0] and m.refs() == [3, 1, 0, 1, 0, 0]
    assert m.compact() == 3 and m.rows[2] == [0, 2]
    assert not m.begin([0], [40])[0] and m.lens == [12, 8, 12]
