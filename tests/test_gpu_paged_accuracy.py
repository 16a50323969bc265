"""How near the paged attention comes to 64 bits, in the 2-norm of each head.

The element-wise bounds of the other tests cover the worst case of every sum;
the limits here are what a correct kernel's errors add up to when roundings are
independent, so that a lost limb or a truncated running sum shows.

An fp32 output, per head, relative to its 2-norm. V has mean 1 and deviation 1,
so sum p |v| is 1.2 times the output and the deviations v - out are as large as
it; the scores' deviation is 2 (log2 domain: |s| < 16, half a step 2^-21), so at
200 tokens some six of them carry the sum, sqrt(sum p^2) <= 0.45, and at more
tokens fewer errors remain. In units of 1e-7:
  scores   D / 16 + 3 <= 19 roundings whose partial sums are half as large in
           the mean: sqrt(19 / 3) 2^-22 ln 2 = 4.2; the products of 16 channels
           are truncated at 2^-23 of sums a quarter as large: 4 of them, 2.7;
           together 5, times 0.45: 2.2
  e^x      2^-22 relative, times 0.45: 1.1
  p        three limbs 2^-24 (int8: two fp16 limbs, 2^-23): 0.3 (0.5)
  V sums   a tile's three products truncated at 2^-24 in the mean, times 1.2:
           2.1; at most 170 tiles of one warp added in fp32, the partial sums
           growing to the whole: sqrt(170 / 3) 2^-24 / sqrt(3) = 2.6
  l        as the tiles, 2.6; joins and the division: four of 2^-24, 0.7
Root of the squares: 4.9. The limit is 6. Two limbs of p instead of three leave
2^-17 / sqrt(3) sqrt(2) 0.45 = 20 at 200 tokens; running sums that stay in the
tensor cores lose 2^-24 a tile, 100 over 170 tiles.
"""

import pytest
import torch

from compressed_decode_attention_blockwise_b200 import PagedKVCache
from _paged import attend, attend_bound, held

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
LIMIT = 6e-7


def shared_cache(k, v, slots, kv, page=64):
    """A cache all of whose slots share the pages of one sequence, (n, Hk, D)
    tokens each of K and V."""
    n, Hk, D = k.shape
    need = -(-n // page)
    c = PagedKVCache(1, slots, need, Hk, D, page_size=page, max_pages=need + 1,
                     kv=kv, token_dtype=k.dtype, device=DEV)
    c.begin([0], [n])
    c.append(k.transpose(0, 1)[None], v.transpose(0, 1)[None])
    table, lens = c.save_map()
    c.restore_map(table[:1].repeat(slots, 1).contiguous(),
                  lens[:1].repeat(slots).contiguous())
    c.begin(range(slots), 0)
    return c


def exact(q, k, v, kv):
    """(B, Hq, D) in 64 bits; q (B, Hq, 1, D), k and v (n, Hk, D)."""
    B, Hq, _, D = q.shape
    Hk = k.shape[1]
    k, v = held(k, kv), held(v, kv)
    out = torch.empty(B, Hq, D, dtype=torch.float64, device=q.device)
    for h in range(Hk):
        g = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
        s = q[:, g, 0].double() @ k[:, h].T * D ** -0.5
        out[:, g] = torch.softmax(s, -1) @ v[:, h]
    return out


def off(got, ref):
    """The largest relative 2-norm of a head's error."""
    d = (got[:, :, 0].double() - ref).norm(dim=-1)
    return float((d / ref.norm(dim=-1)).max())


def tokens(gen, n, Hk, D, dtype):
    k = torch.randn(n, Hk, D, generator=gen, device=DEV)
    v = torch.randn(n, Hk, D, generator=gen, device=DEV) + 1.0
    return k.to(dtype), v.to(dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv,qd", [("bf16", BF), ("bf16", F32), ("f32", F32),
                                   ("i8", BF), ("i8", F32)])
@pytest.mark.parametrize("n,slots", [(200, 3), (8000, 40), (50000, 8)])
def test_fp32_results(D, kv, qd, n, slots):
    gen = torch.Generator(DEV).manual_seed(n + D)
    k, v = tokens(gen, n, 8, D, F32 if kv == "f32" else BF)
    c = shared_cache(k, v, slots, kv)
    q = (2.0 * torch.randn(slots, 16, 1, D, generator=gen, device=DEV)).to(qd)
    assert off(c.attention(q), exact(q, k, v, kv)) <= LIMIT


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("qd", [BF, F32])
def test_int8_queries_with_a_mean(D, G, qd):
    """Queries whose elements do not average out, and one large channel in K,
    whose codes leave the others few bits: a score is a small difference of
    what a bias on the codes would add to it."""
    gen = torch.Generator(DEV).manual_seed(D + G)
    k, v = tokens(gen, 2000, 2, D, BF)
    k[:, :, 5] *= 8.0
    c = shared_cache(k, v, 4, "i8")
    q = torch.randn(4, 2 * G, 1, D, generator=gen, device=DEV)
    q = (1.4 * q + 0.9).to(qd)
    assert off(c.attention(q), exact(q, k, v, "i8")) <= LIMIT


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first,count", [(0, 1), (0, 40), (333, 1), (700, 60),
                                         (999, 1)])
def test_int8_large_values_of_no_weight(D, first, count):
    """Tokens whose V rows are 2^20 times as large as the others' and whose
    scores are low by 90 for some heads of the group (they add nothing there)
    and high for others (they are the result)."""
    gen = torch.Generator(DEV).manual_seed(first + D)
    k, v = tokens(gen, 1000, 1, D, F32)
    base = 2.0 * torch.randn(D, generator=gen, device=DEV)
    big = slice(first, first + count)
    k[big] = 0.01 * k[big] - base * (90.0 * D ** 0.5 / float(base @ base))
    v[big] *= 2.0 ** 20
    c = shared_cache(k, v, 3, "i8")
    q = 0.2 * torch.randn(3, 8, 1, D, generator=gen, device=DEV)
    q[:, ::2] += base
    q[:, 1::2] -= base
    ref = exact(q, k, v, "i8")
    assert float(ref[:, ::2].abs().max()) < 100 < 1e5 < \
        float(ref[:, 1::2].abs().max())
    got = c.attention(q)
    assert off(got[:, ::2], ref[:, ::2]) <= LIMIT
    # The large tokens' scores are 90, 130 in the log2 domain, where half a step
    # is 2^-17 and not the 2^-21 that LIMIT counts: D / 16 + 3 roundings of a
    # score, of which p takes ln 2; ``count`` tokens of nearly equal weight.
    scores = ((D / 16 + 3) / 3) ** 0.5 * 2.0 ** -17 * 0.6932 / count ** 0.5
    assert off(got[:, 1::2], ref[:, 1::2]) <= LIMIT + scores


def test_int8_scales_over_the_whole_range():
    """V rows from 2^-100 to 2^100, each the whole result of its own sequence
    and of the tokens before it."""
    D = 64
    gen = torch.Generator(DEV).manual_seed(1)
    for lo, hi in ((-100, 100), (100, -100), (-100, -100), (100, 100)):
        k, v = tokens(gen, 120, 1, D, F32)
        e = torch.linspace(lo, hi, 120, device=DEV).round()
        v = v * torch.exp2(e)[:, None, None]
        c = shared_cache(k, v, 1, "i8", page=16)
        q = torch.randn(1, 4, 1, D, generator=gen, device=DEV)
        assert off(c.attention(q), exact(q, k, v, "i8")) <= LIMIT


def with_nonfinite(kv, D, qd, lens, edit, fused=False):
    """(output before, output after, q, k, v of slot 1) of a cache of two kv
    heads and eight query heads in which ``edit`` has changed q, k and v of
    slot 1 (fused: its last token comes by a step)."""
    gen = torch.Generator(DEV).manual_seed(D + lens[1])
    tok = F32 if kv == "f32" else BF
    k, v = tokens(gen, sum(lens), 2, D, tok)
    q = torch.randn(len(lens), 8, 1, D, generator=gen, device=DEV).to(qd)
    outs = []
    for changed in (False, True):
        if changed:
            at = slice(lens[0], lens[0] + lens[1])
            edit(q[1], k[at], v[at])
        c = PagedKVCache(1, len(lens), sum(lens) // 16 + 9, 2, D, kv=kv,
                         token_dtype=tok, device=DEV)
        c.begin(range(len(lens)), lens)
        c.append(k.transpose(0, 1)[None], v.transpose(0, 1)[None])
        if fused:
            last = torch.tensor(lens).cumsum(0) - 1
            for s in range(len(lens)):
                c.crop(s, -1)
            c.begin(range(len(lens)))
            outs.append(c.step(q, k[last][:, :, None], v[last][:, :, None]))
        else:
            c.begin(range(len(lens)), 0)
            outs.append(c.attention(q))
    return outs[0], outs[1], q[1], k[at], v[at]


def check_heads(got, q, k, v, heads, drop=None):
    """Heads of slot 1 against the plain form over the tokens but ``drop``;
    got (8, 1, D), channels that are not finite in v set to 0 there."""
    keep = [t for t in range(k.shape[0]) if t != drop]
    f = lambda x: x.double().cpu().numpy()
    D = q.shape[-1]
    v = torch.where(v.isfinite(), v, torch.zeros_like(v))
    k, v = k[keep], v[keep]
    ref, _, mag, dots = attend(f(q[:, 0]), f(k), f(v), 4, D ** -0.5)
    err = abs(f(got[:, 0]) - ref)
    ok = err <= attend_bound(mag, dots, ref, len(keep), D, F32)
    return ok[heads]


@pytest.mark.parametrize("kv,qd", [("bf16", BF), ("bf16", F32), ("f32", F32)])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("lens,at", [([300, 77, 130], 50), ([40, 1, 9], 0),
                                     ([9, 20011], 12345), ([300, 33, 5], 32)])
def test_infinite_values_are_the_formulas(kv, D, qd, lens, at):
    """An infinity in a seen K row is a score of minus or plus infinity (a
    token without weight; NaN), one in V an infinite output of its channel;
    the other channels, heads and rows have the values of the formula."""
    def k_edit(q, k, v):
        q[:, 0, 9] = q[:, 0, 9].abs() * torch.tensor(
            [1, 1, -1, 1, -1, 1, -1, 1], device=DEV, dtype=q.dtype)
        k[at, 1, 9] = float("-inf")
    old, got, q, k, v = with_nonfinite(kv, D, qd, lens, k_edit,
                                       fused=at == lens[1] - 1)
    rest = torch.ones(len(lens), 8, dtype=torch.bool, device=DEV)
    rest[1] = False
    assert torch.equal(got[rest], old[rest])
    assert got[1, [4, 6]].isnan().all()              # a score of +inf
    if lens[1] > 1:                                   # -inf: without the token
        assert check_heads(got[1], q, k, v, [5, 7], drop=at).all()
    assert check_heads(got[1], q, torch.nan_to_num(k), v, [0, 1, 2, 3]).all()

    def v_edit(q, k, v):
        v[at, 1, 9] = float("-inf")
        v[at, 0, 3] = float("inf")
    old, got, q, k, v = with_nonfinite(kv, D, qd, lens, v_edit,
                                       fused=at == lens[1] - 1)
    assert torch.equal(got[rest], old[rest])
    assert (got[1, 4:, 0, 9] == float("-inf")).all()
    assert (got[1, :4, 0, 3] == float("inf")).all()
    ok = check_heads(got[1], q, k, v, list(range(8)))
    ok[4:, 9] = ok[:4, 3] = True
    assert ok.all()


@pytest.mark.parametrize("kv", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("what", ["k", "v", "q"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_nonfinite_elements_stay_in_their_head(kv, what, bad):
    """A NaN (int8: or an infinity) in a seen row makes NaN of the outputs of
    its (row, kv head), or of its channel of them in V; one in a query of those
    of its head. All others keep their bits."""
    def edit(q, k, v):
        if what == "q":
            q[6, 0, 9] = bad
        else:
            (k if what == "k" else v)[50, 1, 9] = bad
    old, got, *_ = with_nonfinite(kv, 64, F32 if kv == "f32" else BF,
                                  [300, 77, 130], edit)
    head = torch.zeros(3, 8, dtype=torch.bool, device=DEV)
    head[1, 6 if what == "q" else slice(4, 8)] = True
    assert torch.equal(got[~head], old[~head])
    if bad != bad or kv == "i8":
        x = got[head][..., 9] if what == "v" and kv != "i8" else got[head]
        assert x.isnan().all()
