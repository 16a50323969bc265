"""Captured launches of the paged cache, replayed after other batches."""

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
