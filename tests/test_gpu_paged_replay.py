"""Captured launches of the paged cache, replayed after other batches."""

import ctypes

import pytest
import torch

from compressed_decode_attention_blockwise_b200 import PagedKVCache
from _paged import quantise

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def check_rows(c, want, kv):
    """The pools hold exactly want[slot] = (k, v), (n, Hk, D) each, in order;
    every other row of them is as it began (NaN, int8: code 77, scale NaN)."""
    table, lens = c.save_map()
    P = c.page_size
    for i, (pool, scales) in enumerate(((c.k, c.k_scales),
                                        (c.v, c.v_scales))):
        got = pool.cpu()
        ref = torch.full_like(got, 77 if kv == "i8" else float("nan"))
        if kv == "i8":
            sc = torch.full(scales.shape, float("nan"))
        for s, rows in want.items():
            assert lens[s] == len(rows[i])
            for t, x in enumerate(rows[i]):
                g = int(table[s, t // P])
                if kv == "i8":
                    ref[0, g, :, t % P], sc[0, g, :, t % P] = quantise(x)
                else:
                    ref[0, g, :, t % P] = x
        assert torch.equal(got.nan_to_num(9e9), ref.nan_to_num(9e9)) \
            if kv != "i8" else torch.equal(got, ref)
        if kv == "i8":
            assert torch.equal(scales.cpu().nan_to_num(9e9),
                               sc.nan_to_num(9e9))


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_append_captured_over_a_batch_without_tokens(kv):
    """A graph is captured while the open batch has no new tokens: the launch
    is in it all the same."""
    c = PagedKVCache(1, 2, 4, 2, 64, page_size=8, kv=kv, device=DEV)
    for pool in (c.k, c.v):
        pool.fill_(77 if kv == "i8" else float("nan"))
    for scales in (c.k_scales, c.v_scales):
        if scales is not None:
            scales.fill_(float("nan"))
    gen = torch.Generator().manual_seed(4)
    x = [torch.randn(6, 2, 64, generator=gen).to(BF) for _ in range(2)]
    k, v = (y.transpose(0, 1)[None].to(DEV) for y in x)
    c.begin([0, 1], 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(k, v)
    c.begin([1, 0], [4, 2])
    g.replay()
    check_rows(c, {1: [y[:4] for y in x], 0: [y[4:] for y in x]}, kv)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("rows,M,batches", [
    # batches that shrink and grow again, one token a row
    (8, 1, [[1] * 8, [1] * 2, [1] * 4, [1] * 8, [1]]),
    # more tokens in fewer rows than an earlier batch had
    (4, 4, [[4] * 4, [1], [16], [3, 0, 9], [0, 0, 1]]),
    # rows as they are after a reset, and after the first batch behind it
    (4, 1, [[1] * 4, None, [1] * 2, [1] * 3]),
    (6, 5, [[5, 0, 2], None, [7, 11], [1] * 6, None, [1, 29]]),
])
def test_captured_append_writes_every_token(kv, rows, M, batches):
    """An append captured over ``rows`` rows and rows * M tokens, replayed
    after each begin (None: a reset) of at most as many: each new token is in
    its page, and nothing else has been written."""
    Hk, D, P = 2, 64, 8
    c = PagedKVCache(1, rows, 40, Hk, D, page_size=P, max_pages=8, kv=kv,
                     device=DEV)

    def clear():
        for pool in (c.k, c.v):
            pool.fill_(77 if kv == "i8" else float("nan"))
        for scales in (c.k_scales, c.v_scales):
            if scales is not None:
                scales.fill_(float("nan"))

    clear()
    k, v = (torch.zeros(rows, Hk, M, D, dtype=BF, device=DEV)
            for _ in range(2))
    c.begin(range(rows), 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(k, v)
    gen = torch.Generator().manual_seed(rows + M)
    want = {}
    for counts in batches:
        if counts is None:
            c.reset()
            clear()
            want = {}
            continue
        slots = list(range(rows - 1, rows - 1 - len(counts), -1))
        c.begin(slots, counts)
        x = [torch.randn(rows * M, Hk, D, generator=gen).to(BF)
             for _ in range(2)]
        for t, y in zip((k, v), x):
            t.copy_(y.view(rows, M, Hk, D).transpose(1, 2))
        g.replay()
        at = 0
        for s, n in zip(slots, counts):
            old = want.get(s, (torch.empty(0, Hk, D, dtype=BF),) * 2)
            want[s] = tuple(torch.cat([o, y[at:at + n]])
                            for o, y in zip(old, x))
            at += n
        check_rows(c, want, kv)


def node_types(g):
    """The types of a kept graph's nodes (0: kernel, 2: memset)."""
    cu = ctypes.CDLL("libcuda.so.1")
    raw, n = ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    types = []
    for x in nodes:
        t = ctypes.c_int()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(x), ctypes.byref(t)) == 0
        types.append(t.value)
    return types


def filled(layers, lens, Hk=2, D=128, page=16):
    c = PagedKVCache(layers, len(lens), sum(-(-n // page) for n in lens) + 8,
                     Hk, D, page_size=page, device=DEV)
    gen = torch.Generator(DEV).manual_seed(sum(lens))
    c.begin(range(len(lens)), lens)
    for layer in range(layers):
        c.append(*(torch.randn(1, Hk, sum(lens), D, generator=gen, device=DEV)
                   .to(BF) for _ in range(2)), layer=layer)
    return c, gen


def test_a_captured_attention_is_one_launch():
    """Twelve layers in one graph are twelve kernels and what zeroes their
    workspace once; the next graph has a workspace of its own."""
    c, gen = filled(12, [3000, 70, 1])
    c.begin(range(3), 0)
    q = torch.randn(12, 3, 8, 1, 128, generator=gen, device=DEV).to(BF)
    want = [c.attention(q[i], layer=i) for i in range(12)]
    graphs, outs = [], []
    for _ in range(2):
        out = torch.zeros(12, 3, 8, 1, 128, device=DEV)
        g = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(g):
            for i in range(12):
                c.attention(q[i], layer=i, out=out[i])
        types = node_types(g)
        assert len(types) <= 13 and types.count(0) >= 12
        g.instantiate()
        graphs.append(g)
        outs.append(out)
    # side by side, eager calls among them
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        assert torch.equal(c.attention(q[0]), want[0])
    torch.cuda.synchronize()
    for out in outs:
        for o, w in zip(out, want):
            assert torch.equal(o, w)


def test_branches_of_one_capture_have_their_own_workspaces():
    """Two streams of one capture, whose launches may run at once, and two
    numbers of heads."""
    c, gen = filled(2, [4000, 900])
    c.begin([0, 1], 0)
    q = [torch.randn(2, h, 1, 128, generator=gen, device=DEV).to(BF)
         for h in (8, 4)]
    want = [[c.attention(x, layer=i) for x in q] for i in (0, 1)]
    outs = [[torch.zeros_like(w) for w in ws] for ws in want]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        for _ in range(10):
            for x, o in zip(q, outs[0]):
                c.attention(x, layer=0, out=o)
            with torch.cuda.stream(side):
                for x, o in zip(q, outs[1]):
                    c.attention(x, layer=1, out=o)
        main.wait_stream(side)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    for ws, os in zip(want, outs):
        for w, o in zip(ws, os):
            assert torch.equal(w, o)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_a_captured_step_attends_for_rows_without_a_token(kv):
    """A step captured over one token a row, replayed for a batch in which some
    rows have none: those rows only attend, and nothing of theirs is written."""
    c = PagedKVCache(1, 4, 60, 2, 64, kv=kv, device=DEV)
    gen = torch.Generator(DEV).manual_seed(9)
    lens = [33, 160, 16, 5]
    c.begin(range(4), lens)
    c.append(*(torch.randn(1, 2, sum(lens), 64, generator=gen, device=DEV)
               .to(BF) for _ in range(2)))
    q, k, v = (torch.randn(4, h, 1, 64, generator=gen, device=DEV).to(BF)
               for h in (8, 2, 2))
    out = torch.zeros(4, 8, 1, 64, device=DEV)
    c.begin(range(4))
    c.step(q, k, v, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.step(q, k, v, out=out)
    for counts in ([1, 0, 1, 0], [0, 0, 0, 0], [0, 1]):
        slots = list(range(len(counts)))
        before = [c.read(s) for s in range(4)]
        c.begin(slots, counts)
        k.add_(0.5)
        g.replay()
        want = c.attention(q[:len(counts)].contiguous())
        assert torch.equal(out[:len(counts)], want)
        assert not out[len(counts):].any()
        for s in range(4):
            n = before[s][0].shape[2]
            new = counts[s] if s < len(counts) else 0
            after = c.read(s)
            assert after[0].shape[2] == n + new
            for a, b in zip(after, before[s]):
                assert torch.equal(a[:, :, :n], b)
            if new and kv == "bf16":
                assert torch.equal(after[0][0, :, n], k[s, :, 0])
                assert torch.equal(after[1][0, :, n], v[s, :, 0])
