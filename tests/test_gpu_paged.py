"""The paged cache on the GPU against plain 64-bit forms (tests/_paged.py).

Pools start as NaN and pages lie in no order, so a read of a masked, free or
foreign token shows. Tolerances: ``_paged.attend_bound`` for attention; append,
read of unquantised pages and all bookkeeping are exact.
"""

import numpy as np
import pytest
import torch

from compressed_decode_attention_blockwise_b200 import (CodecKVCache, FcError,
                                                        PagedKVCache, _lib)
from _paged import (EPS, Model, attend, attend_bound, held, quantise, seen)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def rand(gen, *shape, dtype=F32):
    return torch.randn(shape, generator=gen).to(dtype)


class Filled:
    """A cache whose slots hold random sequences in shuffled pages, written
    straight into the pools; everything else in the pools is NaN (int8: scale
    NaN). ``hide`` (window, sinks) also poisons the masked tokens."""

    def __init__(self, lens, kv="bf16", Hk=2, D=128, page=16, layers=1,
                 seed=0, hide=None, spare=3, token_dtype=BF):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.kv, self.page = list(lens), kv, page
        need = [-(-n // page) for n in lens]
        total = sum(need) + spare
        order = torch.randperm(total, generator=gen).tolist()
        self.rows, at = [], 0
        for m in need:
            self.rows.append(order[at:at + m])
            at += m
        width = max(need + [0]) + 8
        self.cache = c = PagedKVCache(
            layers, len(lens), total, Hk, D, page_size=page, max_pages=width,
            kv=kv, token_dtype=token_dtype, device=DEV)
        tok = c.token_dtype
        self.k = [rand(gen, layers, n, Hk, D, dtype=tok) for n in lens]
        self.v = [rand(gen, layers, n, Hk, D, dtype=tok) + 0.25 for n in lens]
        self.v = [v.to(tok) for v in self.v]
        for pool, scales, rows in ((c.k, c.k_scales, self.k),
                                   (c.v, c.v_scales, self.v)):
            host = torch.full(pool.shape, float("nan")) if kv != "i8" else \
                torch.full(pool.shape, 77.0)
            sc = torch.full(pool.shape[:4], float("nan"))
            for row, x, n in zip(self.rows, rows, lens):
                live = set(seen(n, *hide)) if hide else range(n)
                for t in live:
                    if kv == "i8":
                        code, s = quantise(x[:, t])
                        host[:, row[t // page], :, t % page] = code.float()
                        sc[:, row[t // page], :, t % page] = s
                    else:
                        host[:, row[t // page], :, t % page] = x[:, t].float()
            pool.copy_(host.to(pool.dtype))
            if scales is not None:
                scales.copy_(sc)
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        for i, row in enumerate(self.rows):
            table[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
        c.restore_map(table, torch.tensor(lens, dtype=torch.int32))

    def values(self, slot, layer=0):
        f = lambda x: held(x[slot][layer], self.kv).numpy()
        return f(self.k), f(self.v)


def check_attention(got, q, f, G, slots=None, window=0, sinks=0, layer=0,
                    scale=None, lse=None, extra=None):
    """got (B, Hq, 1, D) against the plain form; ``extra``: (k, v) rows (one
    each) that follow a slot's tokens."""
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    slots = range(len(f.lens)) if slots is None else slots
    for i, s in enumerate(slots):
        k, v = f.values(s, layer)
        if extra is not None:
            k = np.concatenate([k, held(extra[0][i, :, 0], f.kv).numpy()[None]])
            v = np.concatenate([v, held(extra[1][i, :, 0], f.kv).numpy()[None]])
        ref, rl, mag, dots = attend(q[i, :, 0].double().cpu().numpy(), k, v, G,
                                    scale, window, sinks)
        g = got[i, :, 0].double().cpu().numpy()
        err = np.abs(g - ref)
        ok = err <= attend_bound(mag, dots, ref, len(k), D, got.dtype)
        assert ok.all(), "row %d: %d values off, worst %.3g at %.3g" % (
            i, (~ok).sum(), err[~ok].max(), np.abs(ref).max())
        if lse is not None:
            x = lse[i].double().cpu().numpy()
            if len(seen(len(k), window, sinks)) == 0:
                assert np.all(np.isneginf(x))
            else:
                tol = (6 * D / 16 + 5) * 2.0 ** -22 * dots + 2.0 ** -20 + \
                    2.0 ** -22 * np.abs(rl) + len(k) * 2.0 ** -24
                assert np.all(np.abs(x - rl) <= tol)


RAGGED = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 100, 257]


@pytest.mark.parametrize("kv", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_every_shape(kv, D, G):
    """Every page type, head size and group over lengths around the tile and
    page borders, empty sequences among them."""
    page = {1: 16, 2: 8, 4: 32, 8: 16, 16: 64}[G]
    f = Filled(RAGGED, kv, D=D, page=page, seed=D + G)
    gen = torch.Generator().manual_seed(5)
    dt = F32 if kv == "f32" else BF
    q = rand(gen, len(RAGGED), 2 * G, 1, D, dtype=dt)
    f.cache.begin(range(len(RAGGED)), 0)
    for out_dtype in (F32, BF):
        lse = torch.empty(len(RAGGED), 2 * G, device=DEV)
        got = f.cache.attention(q.to(DEV), out_dtype=out_dtype, lse=lse)
        check_attention(got, q, f, G, lse=lse)
        assert not got[0].any()                     # the empty sequence


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("window,sinks", [
    (1, 0), (1, 1), (5, 0), (16, 4), (17, 16), (40, 17), (100, 50), (300, 4),
    (64, 1000), (1 << 40, 1 << 40)])
def test_window_and_sinks(kv, window, sinks):
    """Masked tokens hold NaN: none may be read."""
    lens = RAGGED + [47, 48, 49, 130]
    f = Filled(lens, kv, page=8, hide=(window, sinks), seed=window % 97)
    gen = torch.Generator().manual_seed(6)
    q = rand(gen, len(lens), 8, 1, 128, dtype=BF)
    f.cache.begin(range(len(lens)), 0)
    got = f.cache.attention(q.to(DEV), window=window, sinks=sinks)
    check_attention(got, q, f, 4, window=window, sinks=sinks)


@pytest.mark.parametrize("kv,D,Hk,G,lens", [
    ("bf16", 128, 1, 8, [20011]),
    ("bf16", 128, 2, 4, [9000, 3, 0, 1200, 31]),
    ("i8", 128, 1, 16, [16384, 1]),
    ("f32", 64, 3, 2, [5003, 4999]),
    ("bf16", 256, 1, 16, [7001]),
    ("i8", 64, 5, 1, [3000] * 7),
])
def test_long_sequences_are_split_and_joined(kv, D, Hk, G, lens):
    f = Filled(lens, kv, Hk=Hk, D=D, page=32, seed=len(lens))
    gen = torch.Generator().manual_seed(7)
    q = rand(gen, len(lens), Hk * G, 1, D, dtype=BF)
    f.cache.begin(range(len(lens)), 0)
    lse = torch.empty(len(lens), Hk * G, device=DEV)
    got = [f.cache.attention(q.to(DEV), lse=lse) for _ in range(3)]
    check_attention(got[0], q, f, G, lse=lse)
    # the same inputs give the same bits, whichever CTA came last
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_many_short_sequences():
    """More segments than warps: most are finished by one warp alone."""
    gen = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 40, (300,), generator=gen).tolist()
    f = Filled(lens, Hk=8, D=64, page=8)
    q = rand(gen, 300, 8, 1, 64, dtype=BF)
    f.cache.begin(range(300), 0)
    check_attention(f.cache.attention(q.to(DEV)), q, f, 1)


@pytest.mark.parametrize("kv,n", [("f32", 512), ("i8", 1024), ("bf16", 496)])
def test_shares_that_end_with_the_table_lookahead(kv, n):
    """A warp takes the pages of 32 tiles (of 16 tokens) at a time; here every
    sequence has exactly 32 or 64 tiles, or one less, and there are as many
    sequences as the GPU has warps at work or a few more, so that shares end
    where a lookahead does."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 12 * sms + 5
    gen = torch.Generator().manual_seed(10)
    f = Filled([n] * 2, kv, Hk=1, D=32, seed=3)
    own = f.cache
    c = PagedKVCache(1, rows, own.n_pages, 1, 32, max_pages=own.max_pages,
                     kv=kv, token_dtype=BF, device=DEV,
                     storage=(own.k, own.v, own.k_scales, own.v_scales))
    # the two sequences' pages, shared by all rows
    table = own.save_map()[0].repeat(-(-rows // 2), 1)[:rows].contiguous()
    c.restore_map(table, torch.full((rows,), n, dtype=torch.int32))
    q = rand(gen, rows, 1, 1, 32, dtype=BF)
    c.begin(range(rows), 0)
    got = c.attention(q.to(DEV))
    some = [0, 1, 2, rows // 2, rows - 2, rows - 1]
    check_attention(got[some], q[some], f, 1, slots=[i % 2 for i in some])
    for odd in (0, 1):      # equal queries give equal outputs in every row
        qq = q[odd:odd + 1].expand(rows, 1, 1, 32).contiguous().to(DEV)
        o = c.attention(qq)[odd::2]
        err = (o - o[:1]).abs().max() / o.abs().max()
        assert float(err) <= 2.0 ** -17     # splits differ by rounding only


def test_strides_scale_and_alignment():
    """Queries and outputs at odd offsets and strides; what lies around the
    outputs stays."""
    f = Filled([33, 0, 90], Hk=2, D=64)
    gen = torch.Generator().manual_seed(9)
    f.cache.begin(range(3), 0)
    for dt in (BF, F32):
        for off in (0, 1, 3, 4):
            big = rand(gen, 3, 8, 1, 71, dtype=dt).to(DEV)
            q = big[..., off:off + 64]
            hold = torch.full((3, 11, 1, 69), 5.0, dtype=dt, device=DEV)
            out = hold[:, 2:10, :, off:off + 64]
            f.cache.attention(q, out=out, softmax_scale=0.3)
            check_attention(out, q.cpu(), f, 4, scale=0.3)
            hold[:, 2:10, :, off:off + 64] = 5.0
            assert bool((hold == 5.0).all())
    # head-major queries (transposed), and one query for all rows
    q = rand(gen, 8, 3, 1, 64, dtype=BF).to(DEV).transpose(0, 1)
    check_attention(f.cache.attention(q), q.cpu(), f, 4)
    q = rand(gen, 1, 8, 1, 64, dtype=BF).to(DEV).expand(3, 8, 1, 64)
    check_attention(f.cache.attention(q), q.cpu(), f, 4)


def test_large_scores_and_equal_scores():
    """Scores of +-300 (the running maximum is raised again and again) and
    scores that are all equal."""
    f = Filled([400, 400], Hk=1, D=128, seed=11)
    up = torch.linspace(-3, 3, 400)[:, None].to(BF)
    f.k[0] = (up * torch.ones(1, 128)).to(BF)[None, :, None]
    f.k[1] = torch.ones(1, 400, 1, 128, dtype=BF)
    for s in (0, 1):
        for t in range(400):
            f.cache.k[0, f.rows[s][t // 16], 0, t % 16] = f.k[s][0, t, 0].to(DEV)
    q = torch.full((2, 2, 1, 128), 9.0, dtype=BF)
    q[:, 1] = -9.0
    f.cache.begin([0, 1], 0)
    lse = torch.empty(2, 2, device=DEV)
    got = f.cache.attention(q.to(DEV), lse=lse)
    check_attention(got, q, f, 2, lse=lse)


@pytest.mark.parametrize("kv,tok", [("bf16", BF), ("f32", F32), ("i8", BF),
                                    ("i8", F32)])
@pytest.mark.parametrize("D", [32, 128, 256])
def test_step_is_append_then_attention(kv, tok, D):
    """The fused step against the plain form, and bit for bit against the two
    calls; two layers, new tokens that open a page, lengths from zero."""
    lens = [0, 1, 15, 16, 31, 200, 47]
    gen = torch.Generator().manual_seed(12)
    q = rand(gen, 2, 7, 8, 1, D, dtype=tok)
    k = rand(gen, 2, 7, 2, 1, D, dtype=tok)
    v = rand(gen, 2, 7, 2, 1, D, dtype=tok)
    outs, pools = [], []
    for fused in (True, False):
        f = Filled(lens, kv, D=D, layers=2, seed=13, spare=9, token_dtype=tok)
        f.cache.begin(range(7))
        for layer in (0, 1):
            args = [x[layer].to(DEV) for x in (q, k, v)]
            if fused:
                o = f.cache.step(*args, layer=layer, window=100, sinks=3)
            else:
                f.cache.append(args[1], args[2], layer=layer)
                o = f.cache.attention(args[0], layer=layer, window=100,
                                      sinks=3)
            check_attention(o, q[layer], f, 4, layer=layer, window=100,
                            sinks=3, extra=(k[layer], v[layer]))
            outs.append(o)
        pools.append((f.cache.k, f.cache.v, f.cache.k_scales,
                      f.cache.v_scales))
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    for a, b in zip(*pools):
        if a is not None:
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def expect_pool(f, kv, x_rows, old, scales_old, rows, lens, layer=0):
    """The pool after token rows x_rows[slot] (n, Hk, D) are at positions
    [lens - n, lens) of the slots' pages."""
    pool = old.clone().cpu()
    sc = None if scales_old is None else scales_old.clone().cpu()
    P = pool.shape[3]
    for s, x in x_rows.items():
        for j in range(x.shape[0]):
            t = lens[s] - x.shape[0] + j
            g = rows[s][t // P]
            if kv == "i8":
                code, scale = quantise(x[j])
                pool[layer, g, :, t % P] = code
                sc[layer, g, :, t % P] = scale
            else:
                pool[layer, g, :, t % P] = x[j].to(pool.dtype)
    return pool, sc


@pytest.mark.parametrize("kv", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("D,Hk,page", [(32, 3, 8), (64, 1, 16), (128, 8, 32),
                                       (256, 2, 128)])
def test_append_writes_exactly_the_new_tokens(kv, D, Hk, page):
    """Ragged counts (zero among them), packed and per-row layouts, strided
    and misaligned sources; nothing else in the pools changes."""
    lens = [0, 5, 16, 33, 0, 7]
    counts = [17, 3, 0, 40, 1, 9]
    f = Filled(lens, kv, Hk=Hk, D=D, page=page, layers=2, spare=30, seed=D)
    c = f.cache
    gen = torch.Generator().manual_seed(14)
    N = sum(counts)
    model = Model(6, c.n_pages, page, c.max_pages)
    model.rows, model.lens = [list(r) for r in f.rows], list(lens)
    c.begin(range(6), counts)
    assert model.begin(range(6), counts)[0]
    assert np.array_equal(c.table.cpu().numpy(), model.table())
    new = [n + m for n, m in zip(lens, counts)]
    assert c.lens.tolist() == new
    for source in ("packed", "odd", "spread"):
        x = [rand(gen, N, Hk, D, dtype=c.token_dtype) for _ in range(2)]
        if source == "packed":
            give = [y.to(DEV).transpose(0, 1)[None] for y in x]
        elif source == "odd":
            big = [torch.zeros(N, Hk, D + 3, dtype=c.token_dtype, device=DEV)
                   for _ in x]
            for b, y in zip(big, x):
                b[..., 1:D + 1] = y.to(DEV)
            give = [b[..., 1:D + 1].transpose(0, 1)[None] for b in big]
        else:   # (B, Hk, M, D) with more room than tokens
            M = 11
            B = -(-N // M)
            give = []
            for y in x:
                g = torch.zeros(B, Hk, M, D, dtype=c.token_dtype, device=DEV)
                flat = torch.zeros(B * M, Hk, D, dtype=c.token_dtype)
                flat[:N] = y
                g.copy_(flat.view(B, M, Hk, D).transpose(1, 2))
                give.append(g)
        old = [t.clone() if t is not None else None
               for t in (c.k, c.v, c.k_scales, c.v_scales)]
        c.append(*give, layer=1)
        ends = np.cumsum([0] + counts)
        for i, (pool, scales) in enumerate(((c.k, c.k_scales),
                                            (c.v, c.v_scales))):
            rows = {s: x[i][ends[s]:ends[s + 1]] for s in range(6)}
            want, sc = expect_pool(f, kv, rows, old[i], old[2 + i],
                                   model.rows, new, layer=1)
            assert torch.equal(pool.cpu().view(torch.uint8),
                               want.view(torch.uint8))
            if sc is not None:
                got = scales.cpu()
                assert torch.equal(got.isnan(), sc.isnan())
                ok = ~sc.isnan()
                # the fp32 rounding of absmax / 127 in 64 bits
                assert torch.equal(got[ok], sc[ok])


def test_int8_ties_zero_rows_and_nonfinite_rows():
    c = PagedKVCache(1, 1, 8, 1, 128, kv="i8", token_dtype=F32, device=DEV)
    c.begin([0], [9])
    x = torch.zeros(9, 128)
    # absmax 127: codes are the values, with exact halves (ties to even)
    x[0] = torch.arange(128) * 0.5 + 0.5
    x[0, 127] = -127.0
    x[1] = -x[0]
    x[2, 5] = 1e-45                                  # the smallest subnormal
    x[2, 6] = -1e-45
    x[3] = torch.linspace(-1, 1, 128) * 3e38
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    x[7] = torch.linspace(-2e-37, 1e-37, 128)
    gen = torch.Generator().manual_seed(1)
    x[8] = torch.randn(128, generator=gen)
    t = x.to(DEV)[None, None]                        # (1, 1, 9, 128)
    c.append(t, t)
    codes, scale = quantise(x)
    page = c.k[0, 0, 0, :9].cpu(), c.k_scales[0, 0, 0, :9].cpu()
    for r in (0, 1, 2, 3, 4, 7, 8):
        assert torch.equal(page[0][r], codes[r]), r
        assert page[1][r] == scale[r], r
    for r in (5, 6):                                 # inf, NaN
        assert not page[0][r].any() and page[1][r].isnan()


@pytest.mark.parametrize("kv", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("D", [32, 128, 256])
def test_read_returns_dense_rows(kv, D):
    f = Filled([0, 1, 8, 70, 257], kv, Hk=3, D=D, page=8, layers=2)
    for layer in (0, 1):
        for s, n in enumerate(f.lens):
            for dt in (BF, F32):
                got = f.cache.read(s, layer, dtype=dt)
                for g, ref in zip(got, f.values(s, layer)):
                    assert g.shape == (1, 3, n, D) and g.dtype == dt
                    ref = torch.from_numpy(ref).transpose(0, 1)[None]
                    err = (g.double().cpu() - ref).abs()
                    # one fp32 rounding of code * scale, one to the dtype
                    tol = (2.0 ** -24 + EPS[dt]) * ref.abs() * 1.001
                    if kv != "i8" and (dt == F32 or kv == "bf16"):
                        tol = torch.zeros_like(tol)
                    assert bool((err <= tol).all())


def test_bookkeeping_follows_the_model():
    """Random begins, forks, crops, frees and compactions against the model;
    every token carries its own value, so a page copied wrongly, shared when
    written or lost shows in the rows read back."""
    rng = np.random.default_rng(3)
    P, slots, pages = 8, 12, 26
    c = PagedKVCache(2, slots, pages, 2, 32, page_size=P, max_pages=9,
                     kv="f32", device=DEV)
    m = Model(slots, pages, P, 9)
    vals = [[] for _ in range(slots)]
    stamp, refused = 1.0, 0
    for it in range(160):
        op = rng.choice(["begin", "begin", "fork", "free", "crop", "compact"])
        if op == "begin":
            n = int(rng.integers(1, 6))
            ss = [int(s) for s in rng.permutation(slots)[:n]]
            cs = [int(x) for x in rng.integers(0, 14, n)]
            cs = [min(x, 72 - m.lens[s]) for s, x in zip(ss, cs)]
            ok, _ = m.begin(ss, cs)
            if not ok:
                refused += 1
                with pytest.raises(FcError) as e:
                    c.begin(ss, cs)
                assert e.value.status == _lib.FC_ERR_CAPACITY
            else:
                c.begin(ss, cs, rows=min(slots, n + it % 3))
                N = sum(cs)
                v = torch.arange(N, dtype=F32) + stamp
                stamp += N
                if N:
                    for layer in (0, 1):
                        x = (v + 0.25 * layer)[None, None, :, None] \
                            .expand(1, 2, N, 32).to(DEV)
                        c.append(x, -x, layer=layer)
                at = 0
                for s, k in zip(ss, cs):
                    vals[s] = vals[s] + v[at:at + k].tolist()
                    at += k
        elif op == "fork":
            empty = [s for s in range(slots) if not m.lens[s]]
            full = [s for s in range(slots) if m.lens[s]]
            if not empty or not full:
                continue
            dst = empty[:int(rng.integers(1, 4))]
            src = [int(rng.choice(full)) for _ in dst]
            m.fork(src, dst)
            c.fork(src, dst)
            for a, b in zip(src, dst):
                vals[b] = list(vals[a])
        elif op == "free":
            ss = [int(s) for s in rng.permutation(slots)[:2]]
            for s in ss:
                m.crop(s, 0)
                vals[s] = []
            c.free(ss)
        elif op == "crop":
            s, k = int(rng.integers(slots)), int(rng.integers(0, 20))
            keep = max(0, m.lens[s] - k)
            m.crop(s, keep)
            c.crop(s, -k)
            vals[s] = vals[s][:keep]
        else:
            assert c.compact() == m.compact()
        assert np.array_equal(c.table.cpu().numpy(), m.table())
        assert c.lens.tolist() == m.lens
        table, lens = c.save_map()
        assert np.array_equal(table.numpy(), m.table())
        assert lens.tolist() == m.lens
        assert c._h_refs.tolist() == m.refs()
        assert c.free_pages == m.refs().count(0)
        if it % 8 == 7:
            for s in range(slots):
                for layer in (0, 1):
                    k, v = c.read(s, layer)
                    want = torch.tensor(vals[s], dtype=F32) + 0.25 * layer
                    assert torch.equal(k[0, 1, :, 5].cpu(), want)
                    assert torch.equal(v[0, 0, :, 31].cpu(), -want)
    assert refused > 3 and stamp > 200


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_forks_write_to_their_own_copies(kv):
    """Parallel samples of one prompt: all layers' shared last page is copied,
    the source's rows stay, and each fork attends to its own tokens."""
    f = Filled([45, 0, 0, 0], kv, layers=3, spare=8, seed=20)
    c = f.cache
    gen = torch.Generator().manual_seed(21)
    c.fork([0, 0, 0], [1, 2, 3])
    assert c.rows == 0
    before = [c.read(0, layer) for layer in range(3)]
    c.begin([1, 2, 3])
    assert c.free_pages == 8 - 3
    for layer in range(3):
        q, k, v = (rand(gen, 3, h, 1, 128, dtype=BF) for h in (8, 2, 2))
        o = c.step(q.to(DEV), k.to(DEV), v.to(DEV), layer=layer)
        check_attention(o, q, f, 4, slots=[0, 0, 0], layer=layer, extra=(k, v))
        for a, b in zip(c.read(0, layer), before[layer]):
            assert torch.equal(a, b)


def test_restore_map_and_compact_across_launches():
    """More moved pages than one launch's list holds, in two layers."""
    n, P = 9000, 8
    c = PagedKVCache(2, 3, n, 1, 32, page_size=P, kv="f32", device=DEV)
    ids = torch.arange(n, dtype=F32, device=DEV)
    for layer in (0, 1):
        c.k[layer] = (ids + 0.5 * layer)[:, None, None, None]
        c.v[layer] = -(ids + 0.5 * layer)[:, None, None, None]
    g = torch.Generator().manual_seed(2)
    used = torch.randperm(n, generator=g)[:8500].to(torch.int32)
    used = used[used >= 400]                 # holes at the front as well
    cut = [0, 3000, 3001, len(used)]
    table = torch.full((3, n), -1, dtype=torch.int32)
    lens = torch.zeros(3, dtype=torch.int32)
    for s in range(3):
        part = used[cut[s]:cut[s + 1]]
        table[s, :len(part)] = part
        lens[s] = len(part) * P - (s + 1)
    c.restore_map(table, lens)
    m = Model(3, n, P, n)
    m.rows = [[int(x) for x in r[r >= 0]] for r in table]
    m.lens = lens.tolist()
    assert c.free_pages == n - len(used)
    assert c.compact() == m.compact() == len(used)
    assert np.array_equal(c.table.cpu().numpy(), m.table())
    for s in range(3):
        for layer in (0, 1):
            k, v = c.read(s, layer)
            want = table[s, :cut[s + 1] - cut[s]].float() + 0.5 * layer
            assert torch.equal(k[0, 0, ::P, 3].cpu(), want)
            assert torch.equal(v[0, 0, 2::P, 30].cpu(),
                               -want[:len(v[0, 0, 2::P])])
    assert c.compact() == len(used)          # nothing left to move


def test_captured_steps_are_replayed_after_each_begin():
    """A graph of two layers' steps over a padded batch, replayed with other
    slots and lengths, against the plain form and the eager calls."""
    f = Filled([40, 7, 0, 100, 21], layers=2, spare=12, seed=30)
    c = f.cache
    gen = torch.Generator().manual_seed(31)
    q = torch.zeros(2, 4, 8, 1, 128, dtype=BF, device=DEV)
    k, v = (torch.zeros(2, 4, 2, 1, 128, dtype=BF, device=DEV)
            for _ in range(2))
    outs = [torch.zeros(4, 8, 1, 128, device=DEV) for _ in range(2)]
    c.begin([2], rows=4)                     # the captured launches' shape
    saved = c.save_map()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        for call in (lambda: c.begin([2], rows=4), lambda: c.free([2]),
                     lambda: c.fork([0], [2]), c.compact, c.reset,
                     lambda: c.crop(0, -1), lambda: c.restore_map(*saved)):
            with pytest.raises(FcError):     # bookkeeping is not captured
                call()
        for layer in range(2):
            c.step(q[layer], k[layer], v[layer], layer=layer, out=outs[layer])
    torch.cuda.current_stream().wait_stream(side)
    c.crop(2, -1)                            # the token that was never written
    for slots in ([0, 3, 1], [4, 0], [1, 3, 0, 4]):
        c.begin(slots, rows=4)
        x = [rand(gen, 2, 4, h, 1, 128, dtype=BF) for h in (8, 2, 2)]
        for t, y in zip((q, k, v), x):
            t.copy_(y)
        g.replay()
        for layer in range(2):
            o = outs[layer]
            ex = (x[1][layer], x[2][layer])
            n = len(slots)
            check_attention(o[:n], x[0][layer], f, 4, slots=slots,
                            layer=layer, extra=ex)
            assert not o[n:].any()           # padding rows
            assert torch.equal(o, c.attention(q[layer], layer=layer))
        for i, s in enumerate(slots):        # the tokens are part of the slot
            f.k[s] = torch.cat([f.k[s], x[1][:, i, :, 0][:, None]], 1)
            f.v[s] = torch.cat([f.v[s], x[2][:, i, :, 0][:, None]], 1)


def test_replay_after_a_smaller_batch_leaves_the_other_slots():
    """Rows that a smaller batch no longer has are empty for a captured step of
    the larger one: it writes nothing to their slots."""
    f = Filled([40, 7, 30], spare=6, seed=32)
    c = f.cache
    gen = torch.Generator().manual_seed(33)
    x = [rand(gen, 3, h, 1, 128, dtype=BF).to(DEV) for h in (8, 2, 2)]
    c.begin([0, 1, 2])
    out = torch.zeros(3, 8, 1, 128, device=DEV)
    c.step(*x, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.step(*x, out=out)
    c.begin([1])
    keep = [[t.clone() for t in c.read(s)] for s in (0, 2)]
    x[1].add_(1.0)
    g.replay()
    assert not out[1:].any()
    for s, rows in zip((0, 2), keep):
        for a, b in zip(c.read(s), rows):
            assert torch.equal(a, b)
    assert torch.equal(c.read(1)[0][:, :, -1], x[1][0, :, 0][None])


def test_two_graphs_side_by_side():
    """Graphs captured on one stream and replayed on two at once: each has a
    workspace of its own."""
    f = Filled([5000, 80], layers=2, page=32, seed=42)
    gen = torch.Generator().manual_seed(43)
    q = rand(gen, 2, 8, 1, 128, dtype=BF).to(DEV)
    f.cache.begin([0, 1], 0)
    want = [f.cache.attention(q, layer=i) for i in (0, 1)]
    outs = [torch.zeros_like(w) for w in want]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            for _ in range(10):
                f.cache.attention(q, layer=i, out=outs[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("kv,Hk,G,page,D", [
    ("bf16", 7, 16, 1024, 64), ("i8", 13, 2, 256, 128), ("f32", 1, 1, 8, 256),
    ("i8", 3, 8, 8, 256), ("bf16", 33, 4, 64, 32)])
def test_odd_heads_and_page_sizes(kv, Hk, G, page, D):
    lens = [1030, 1, 15, 2047, 0, 300]
    f = Filled(lens, kv, Hk=Hk, D=D, page=page, seed=Hk, hide=(700, 9))
    gen = torch.Generator().manual_seed(Hk)
    dt = F32 if kv == "f32" else BF
    for qd in (dt, F32):
        q = rand(gen, 6, Hk * G, 1, D, dtype=qd)
        f.cache.begin(range(6), 0)
        got = f.cache.attention(q.to(DEV), window=700, sinks=9)
        check_attention(got, q, f, G, window=700, sinks=9)


def test_other_streams_and_concurrent_calls():
    """Two layers' attention on two streams at once: each stream has its own
    workspace."""
    f = Filled([6000, 50, 900], layers=2, page=32, seed=40)
    gen = torch.Generator().manual_seed(41)
    q = rand(gen, 3, 8, 1, 128, dtype=BF).to(DEV)
    f.cache.begin(range(3), 0)
    want = [f.cache.attention(q, layer=i) for i in (0, 1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(f.cache.attention(q, layer=i))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements per K: sequences in
    its last pages."""
    P, Hk, D = 128, 8, 128
    pages = (1 << 31) // (P * Hk * D) + 40
    c = PagedKVCache(1, 2, pages, Hk, D, page_size=P, max_pages=8, device=DEV)
    table = torch.full((2, 8), -1, dtype=torch.int32)
    table[0, :3] = torch.tensor([pages - 1, pages - 2, 5])
    table[1, :2] = torch.tensor([pages - 7, pages - 3])
    c.restore_map(table, torch.tensor([300, 200], dtype=torch.int32))
    gen = torch.Generator().manual_seed(50)

    class F:
        kv, lens = "bf16", [300, 200]
        k = [rand(gen, 1, n, Hk, D, dtype=BF) for n in lens]
        v = [rand(gen, 1, n, Hk, D, dtype=BF) for n in lens]

        def values(self, s, layer):
            return self.k[s][0].double().numpy(), self.v[s][0].double().numpy()

    f = F()
    c.crop(0, -300)
    c.crop(1, -200)
    c.restore_map(table, torch.zeros(2, dtype=torch.int32))
    # write through the cache: the map is taken over with the tokens counted
    c.restore_map(table, torch.tensor([300, 200], dtype=torch.int32))
    for s in (0, 1):
        for i, pool in ((0, c.k), (1, c.v)):
            x = (f.k, f.v)[i][s][0]
            for t0 in range(0, f.lens[s], P):
                part = x[t0:t0 + P].transpose(0, 1).to(DEV)
                pool[0, int(table[s, t0 // P]), :, :part.shape[1]] = part
    c.begin([0, 1], 0)
    q = rand(gen, 2, Hk, 1, D, dtype=BF)
    check_attention(c.attention(q.to(DEV)), q, f, 1)
    k, _ = c.read(0)
    assert torch.equal(k[0].cpu(), f.k[0][0].transpose(0, 1))


def test_hand_over_to_the_codec():
    """A sequence grown in pages, read as dense rows and archived by the
    lossless codec: the same attention on both sides."""
    c = PagedKVCache(1, 2, 40, 2, 64, kv="f32", device=DEV)
    gen = torch.Generator().manual_seed(60)
    k, v = rand(gen, 1, 2, 300, 64).to(DEV), rand(gen, 1, 2, 300, 64).to(DEV)
    c.begin([1], [250])
    c.append(k[:, :, :250], v[:, :, :250])
    for t in range(250, 300):
        c.begin([1])
        o = c.step(rand(gen, 1, 8, 1, 64).to(DEV), k[:, :, t:t + 1],
                   v[:, :, t:t + 1])
    kk, vv = c.read(1)
    assert torch.equal(kk, k) and torch.equal(vv, v)
    codec = CodecKVCache(1, 2, 64, R=8, S=8, coeff_k="f32", coeff_v="f32",
                         token_dtype=F32, device=DEV)
    codec.prefill(kk, vv)
    q = rand(gen, 1, 8, 1, 64).to(DEV)
    c.begin([1], 0)
    err = (codec.attention(q) - c.attention(q)).abs().max()
    assert float(err) <= 2e-3      # the codec path's own bar
    assert o.shape == (1, 8, 1, 64)


def test_adopted_storage_with_strides():
    """Pools that are views of a larger allocation (layers inside pages)."""
    big = torch.full((10, 2, 2, 3, 16, 64), float("nan"), dtype=BF, device=DEV)
    k = big[:, 0].permute(1, 0, 2, 3, 4)     # (layers, pages, Hk, P, D)
    v = big[:, 1].permute(1, 0, 2, 3, 4)
    c = PagedKVCache(2, 3, 10, 3, 64, device=DEV, max_pages=4,
                     storage=(k, v, None, None))
    gen = torch.Generator().manual_seed(70)
    x = rand(gen, 2, 1, 3, 60, 64, dtype=BF).to(DEV)
    c.begin([0, 2], [20, 40])
    for layer in (0, 1):
        c.append(x[layer], -x[layer], layer=layer)
    c.free([0])
    assert c.compact() == 3
    for layer in (0, 1):
        kk, vv = c.read(2, layer)
        assert torch.equal(kk, x[layer][:, :, 20:])
        assert torch.equal(vv, -x[layer][:, :, 20:])


def test_binding_refuses_wrong_tensors():
    f = Filled([5, 9], Hk=2, D=64)
    c = f.cache
    q = torch.zeros(2, 4, 1, 64, dtype=BF, device=DEV)
    t = torch.zeros(2, 2, 1, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        c.attention(q)                               # no batch is open
    c.begin([0, 1])
    bad = [lambda: c.attention(q[:1]), lambda: c.attention(q.half()),
           lambda: c.attention(q.cpu()), lambda: c.attention(q[..., :32]),
           lambda: c.attention(q, out=q[:, :2]),
           lambda: c.attention(q, lse=torch.zeros(2, 3, device=DEV)),
           lambda: c.append(t.float(), t.float()),
           lambda: c.append(t[:, :1], t[:, :1]),
           lambda: c.append(t.cpu(), t.cpu()),
           lambda: c.step(q, t[:1], t[:1]),
           lambda: c.begin([0, 1], [1]), lambda: c.crop(0, 1),
           lambda: c.restore_map(torch.zeros(2, 2, dtype=torch.int32),
                                 torch.zeros(2, dtype=torch.int32)),
           lambda: PagedKVCache(1, 1, 2, 2, 64, device=DEV,
                                storage=(q, q, None, None))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d" % i)
    for call in (lambda: c.attention(q, layer=1), lambda: c.begin([0, 0]),
                 lambda: c.attention(q[:, :3].contiguous()),
                 lambda: c.attention(q, window=-1)):
        with pytest.raises(FcError):
            call()
    c.begin([0, 1], 0)
    with pytest.raises(FcError):                     # no new tokens to write
        c.step(q, t, t)
