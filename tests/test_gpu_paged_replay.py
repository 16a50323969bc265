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
