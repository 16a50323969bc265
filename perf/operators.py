"""The paged cache's operators as a serving program calls them, with their plain forms.

A cache of many sequences of different lengths keeps K and V in pages of
``page`` tokens, (layers, pages, Hk, page, D); a table row per sequence names
its pages in order. The operators are single-token attention over the pages
(optionally a sliding window and a few first tokens that stay visible), the
decode step (append the new token, then attend), the append of prompts, the
read of a sequence as dense rows, forking with copy on write, and compaction.

``own`` selects the framework's calls; otherwise the plain forms run:
elementary torch operations in 32 bits, rounded once at the end.
"""

import math
import random

import numpy as np
import torch

own = False

_STORE = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8}
_TOKEN = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.bfloat16}
_BYTES = {"bf16": 2, "f32": 4, "i8": 1}
DEV = "cuda:0"


# ------------------------------------------------------------------- cases

def listed():
    base = {"op": "attend", "kv": "bf16", "B": 8, "Hk": 8, "G": 4, "D": 128,
            "page": 16, "T": 4101, "ragged": True, "window": 0, "sinks": 0,
            "layers": 1, "out": "bf16"}
    c = lambda name, **kw: dict(base, name=name, **kw)
    return [
        # one short fp32 sequence without head sharing: latency of a call
        c("attend_short", kv="f32", B=1, Hk=4, G=1, D=64, T=256, ragged=False,
          out="f32"),
        # an ordinary serving batch of ragged sequences
        c("attend_batch"),
        # one long context alone on the GPU: the cache is split over all SMs
        c("attend_long", B=1, page=64, T=131075, ragged=False),
        # a large batch over an int8 cache: the largest read
        c("attend_large", kv="i8", B=64, G=8, page=32, T=8199, out="f32"),
        # long chats that see a window and their first tokens only
        c("attend_window", B=24, page=32, T=32768, window=1000, sinks=4),
        # a decode step of a busy server
        c("step_batch", op="step", B=64, T=2049),
        # a decode step of a few int8 sequences: latency, with quantisation
        c("step_few", op="step", kv="i8", B=4, T=700, out="f32"),
        # prompts arriving together, written to their pages
        c("append_prompts", op="append", B=8, page=32, T=8192),
        # a short prompt quantised to int8, then read back as dense rows
        c("append_read_i8", op="append_read", kv="i8", B=2, T=333),
        # a long sequence handed over as dense rows
        c("read_long", op="append_read", B=1, page=64, T=32768, ragged=False),
        # parallel samples: 8 prompts forked 8 times, the first new token of
        # each fork (copies every fork's shared last page in all layers)
        c("fork_samples", op="fork", B=8, forks=8, T=1003, layers=8),
        # a pool with holes packed to its front after sequences ended
        c("compact_pool", op="compact", B=48, T=1500, layers=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "step", "append",
                     "append_read", "fork", "compact"])
    c = {"op": op, "kv": rng.choice(["bf16", "bf16", "i8", "f32"]),
         "B": _log(rng, 1, 96), "Hk": rng.choice([1, 2, 4, 8]),
         "G": rng.choice([1, 2, 4, 8, 16]), "D": rng.choice([32, 64, 128, 256]),
         "page": rng.choice([8, 16, 32, 64, 128]), "T": _log(rng, 1, 60000),
         "ragged": rng.random() < 0.8, "window": 0, "sinks": 0, "layers": 1,
         "out": rng.choice(["bf16", "f32"])}
    if op in ("attend", "step") and rng.random() < 0.4:
        c["window"] = _log(rng, 1, 5000)
        c["sinks"] = rng.choice([0, 1, 4, 37])
    if op == "append_read":
        c["B"] = min(c["B"], 4)
    if op in ("fork", "compact"):
        c["layers"] = rng.choice([1, 2, 6])
        c["T"] = min(c["T"], 4000)
    if op == "fork":
        c["forks"] = rng.randint(1, 5)
    # a drawn case holds less than the largest listed one
    most = 4e8 if op in ("attend", "step") else 1e8
    while _pool_bytes(c) > most:
        if c["B"] > 1 and rng.random() < 0.5:
            c["B"] = max(1, c["B"] // 2)
        else:
            c["T"] = max(1, c["T"] // 2)
    return c


def _pool_bytes(c):
    return 2 * c["layers"] * c["B"] * c["T"] * c["Hk"] * c["D"] * _BYTES[c["kv"]]


def _lens(c):
    """Lengths of the case's sequences: T for all, or spread over [1, T] with
    one of them at T (and one empty slot where the batch is large)."""
    if not c["ragged"]:
        return [c["T"]] * c["B"]
    r = random.Random("%(B)d %(T)d %(page)d" % c)
    lens = [r.randint(max(1, c["T"] // 4), c["T"]) for _ in range(c["B"])]
    lens[r.randrange(c["B"])] = c["T"]
    if c["B"] >= 16 and c["op"] == "attend":
        lens[r.randrange(c["B"])] = 0
    return lens


def _visible(c, n):
    if not c["window"]:
        return n
    lo = max(0, n - c["window"])
    return n - lo + min(lo, c["sinks"])


def work(c):
    per = c["Hk"] * c["D"] * _BYTES[c["kv"]] + \
        (4 * c["Hk"] if c["kv"] == "i8" else 0)         # one of K, V
    tok = 4 if c["kv"] == "f32" else 2                  # a token's element
    lens, Hq = _lens(c), c["Hk"] * c["G"]
    dense = c["Hk"] * c["D"] * tok
    if c["op"] in ("attend", "step"):
        vis = sum(_visible(c, n) for n in lens)
        by = 2 * per * vis + c["B"] * Hq * c["D"] * \
            (tok + (4 if c["out"] == "f32" else 2))
        if c["op"] == "step":
            by += 2 * dense * c["B"]
        return {"bytes": by, "flops": 4 * Hq * c["D"] * vis}
    if c["op"] in ("append", "append_read"):
        by = 2 * (dense + per) * sum(lens)
        if c["op"] == "append_read":
            by += 2 * (dense + per) * sum(lens)
        return {"bytes": by, "flops": 0}
    page = 2 * per * c["page"] * c["layers"]
    if c["op"] == "fork":
        copies = sum(c["forks"] for n in lens if n % c["page"])
        return {"bytes": max(1, 2 * page * copies) + 8 * sum(
            -(-n // c["page"]) for n in lens) * c["forks"], "flops": 0}
    table, _, _ = _map(c, random.Random(1))
    live = sorted({p for row in table for p in row})
    moved = sum(p >= len(live) for p in live)
    return {"bytes": max(1, 2 * page * moved) + 8 * len(live), "flops": 0}


# ------------------------------------------------------------------ inputs

def _map(c, rng):
    """(table rows, lengths before the call, number of pages). Pages lie in
    the pool in no order, as after some time of serving. A step's table
    includes the page of its new token (the lowest free one, in row order)."""
    P = c["page"]
    lens = _lens(c)
    before = [n - 1 for n in lens] if c["op"] == "step" else lens
    if c["op"] in ("append", "append_read"):
        # an empty cache fills from its first page on
        rows, at = [], 0
        for n in lens:
            m = -(-n // P)
            rows.append(list(range(at, at + m)))
            at += m
        return rows, [0] * len(lens), at + 2
    need = [-(-n // P) for n in before]
    spare = c["B"] * (1 + c.get("forks", 0)) + 3
    if c["op"] == "compact":
        spare = sum(need) // 2 + 3        # a third of the pool is free
    total = sum(need) + spare
    order = list(range(total))
    if c["op"] == "compact":              # which pages are free: by the case
        random.Random("%(B)d %(T)d %(page)d %(layers)d" % c).shuffle(order)
        order = sorted(order[:sum(need)])
        rng.shuffle(order)
    else:
        rng.shuffle(order)
    rows, at = [], 0
    for m in need:
        rows.append(order[at:at + m])
        at += m
    if c["op"] == "step":
        free = sorted(set(range(total)) - {p for r in rows for p in r})
        for r, n in zip(rows, lens):
            if -(-n // P) > len(r):
                r.append(free.pop(0))
    return rows, before, total


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _quantise(x):
    """int8 codes and fp32 scales of rows (..., D); the rounding is decided in
    64 bits, where a code next to a border (bf16 rows hit exact ties) comes
    out as its definition says."""
    top = x.abs().amax(-1).double()
    safe = torch.where(top > 0, top, torch.ones_like(top))
    codes = torch.round(x.double() * 127.0 / safe[..., None])
    return codes.to(torch.int8), (top / 127.0).float()


def _inputs(c, seed):
    """Tensors of the case, on the GPU: the pool (with a bias per channel and
    one outlier channel per head, as caches have), table, lengths, queries and
    new tokens."""
    gen = torch.Generator(DEV).manual_seed(seed)
    rows, before, total = _map(c, random.Random(seed))
    H, P, D, L, Hq = c["Hk"], c["page"], c["D"], c["layers"], c["Hk"] * c["G"]
    tok = _TOKEN[c["kv"]]
    s = {"case": c, "rows": rows, "before": before, "pages": total}
    bias = 0.5 * _normal(gen, 2, H, 1, D)
    gain = torch.ones(2, H, 1, D, device=DEV)
    gain.scatter_(3, torch.randint(D, (2, H, 1, 1), generator=gen, device=DEV), 4.0)
    writes = c["op"] in ("append", "append_read")
    for i, name in enumerate("kv"):
        if writes:
            x = torch.zeros(L, total, H, P, D, device=DEV)
        else:
            x = (_normal(gen, L, total, H, P, D) + bias[i]) * gain[i]
        if c["kv"] == "i8":
            s[name], s[name + "s"] = _quantise(x)
        else:
            s[name], s[name + "s"] = x.to(_STORE[c["kv"]]), None
        del x
    n_slots = c["B"] * (1 + c.get("forks", 0))
    lens = _lens(c)
    width = max([-(-(n + 1) // P) for n in lens] + [1]) + 1
    table = np.full((n_slots, width), -1, np.int32)
    for r, row in enumerate(rows):
        table[r, :len(row)] = row
    hold = np.zeros(n_slots, np.int32)
    hold[:c["B"]] = before
    s["table0"], s["lens0"] = torch.from_numpy(table), torch.from_numpy(hold)
    s["table"], s["lens"] = s["table0"].to(DEV), torch.tensor(lens, device=DEV)
    s["lens_all"] = s["lens0"].to(DEV)
    if c["op"] in ("attend", "step"):
        s["q"] = (2.0 * _normal(gen, c["B"], Hq, 1, D)).to(tok)
    if c["op"] == "step":
        s["kn"] = (_normal(gen, c["B"], H, 1, D) + bias[0, :, :]).to(tok)
        s["vn"] = (_normal(gen, c["B"], H, 1, D) + bias[1, :, :]).to(tok)
    if writes:
        N = sum(lens)      # packed tokens (N, H, D), seen as (1, H, N, D)
        s["kn"] = (_normal(gen, N, H, D) + bias[0, :, 0]).to(tok) \
            .transpose(0, 1)[None]
        s["vn"] = (_normal(gen, N, H, D) + bias[1, :, 0]).to(tok) \
            .transpose(0, 1)[None]
        at = np.concatenate([np.arange(n) for n in lens])
        of = np.repeat(np.arange(c["B"]), lens)
        s["at"] = torch.from_numpy(at).to(DEV)
        s["of"] = torch.from_numpy(of).to(DEV)
    if c["op"] == "fork":
        s["src"] = [b for b in range(c["B"]) for _ in range(c["forks"])]
        s["dst"] = list(range(c["B"], n_slots))
        s["src_d"] = torch.tensor(s["src"], device=DEV)
        s["dst_d"] = torch.tensor(s["dst"], device=DEV)
    return s


def prepare(c, seed):
    s = _inputs(c, seed)
    if own:
        from compressed_decode_attention_blockwise_b200 import PagedKVCache
        cache = PagedKVCache(
            c["layers"], s["table0"].shape[0], s["pages"], c["Hk"], c["D"],
            page_size=c["page"], max_pages=s["table0"].shape[1], kv=c["kv"],
            token_dtype=_TOKEN[c["kv"]], device=DEV,
            storage=(s["k"], s["v"], s["ks"], s["vs"]))
        cache.restore_map(s["table0"], s["lens0"])
        if c["op"] == "attend":
            cache.begin(range(c["B"]), 0)
        elif c["op"] == "step":
            cache.begin(range(c["B"]))
        elif c["op"] in ("append", "append_read"):
            cache.begin(range(c["B"]), _lens(c))
        s["cache"] = cache
        s["out_dtype"] = torch.float32 if c["out"] == "f32" else torch.bfloat16
    return s


# --------------------------------------------------------------- plain forms

def _dense(s, name, rows):
    """(B, H, T, D) in 32 bits: the pages of table rows `rows`, in order."""
    t = rows.clamp(min=0).long()
    x = s[name][0][t].float()                       # (B, n, H, P, D)
    if s[name + "s"] is not None:
        x = x * s[name + "s"][0][t][..., None]
    B, n, H, P, D = x.shape
    return x.transpose(1, 2).reshape(B, H, n * P, D)


def _plain_attend(s):
    c = s["case"]
    B, H, G, D = c["B"], c["Hk"], c["G"], c["D"]
    k = _dense(s, "k", s["table"][:B])
    v = _dense(s, "v", s["table"][:B])
    pos = torch.arange(k.shape[2], device=k.device)
    lens = s["lens"][:, None]
    seen = pos < lens
    if c["window"]:
        seen = seen & ((pos >= lens - c["window"]) | (pos < c["sinks"]))
    q = s["q"].float().reshape(B, H, G, D)
    x = torch.matmul(q, k.transpose(2, 3)) * D ** -0.5
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.reshape(B, H * G, 1, D).to(
        torch.float32 if c["out"] == "f32" else torch.bfloat16)


def _plain_write(s, slots, at, kn, vn):
    """Writes (N, H, D) tokens to positions `at` of table rows `slots`."""
    P = s["case"]["page"]
    page = s["table"][slots, at // P].long()
    for name, x in (("k", kn), ("v", vn)):
        x = x.float()
        if s[name + "s"] is not None:
            x, scale = _quantise(x)
            s[name + "s"][0][page, :, at % P] = scale
        s[name][0][page, :, at % P] = x.to(s[name].dtype)


def _plain_read(s):
    outs = []
    for b, n in enumerate(_lens(s["case"])):
        outs.append([_dense(s, name, s["table"][b:b + 1])[:, :, :n]
                     .to(s["kn"].dtype) for name in "kv"])
    return outs


def _plain_fork(s):
    """Table rows and lengths after the forks and their next token's page;
    the shared last pages copied in all layers."""
    P = s["case"]["page"]
    table, lens = s["table"].clone(), s["lens_all"].clone()
    table[s["dst_d"]] = table[s["src_d"]]
    lens[s["dst_d"]] = lens[s["src_d"]]
    refs = torch.bincount(table[table >= 0].long(), minlength=s["pages"])
    free = torch.nonzero(refs == 0)[:, 0]
    at = lens[s["dst_d"]].long()
    new = free[:at.numel()]
    old = table[s["dst_d"], at // P].long()
    part = at % P != 0
    for name in ("k", "v", "ks", "vs"):
        if s[name] is not None:
            s[name][:, new[part]] = s[name][:, old[part]]
    table[s["dst_d"], at // P] = new.int()
    lens[s["dst_d"]] += 1
    return table, lens, s["k"], s["v"]


def _plain_compact(s):
    table = s["table"].clone()
    refs = torch.bincount(table[table >= 0].long(), minlength=s["pages"])
    live = torch.nonzero(refs)[:, 0]
    n = live.numel()
    src = live[live >= n]
    dst = torch.nonzero(refs[:n] == 0)[:, 0]
    to = torch.arange(s["pages"], device=table.device)
    to[src] = dst
    table = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table)
    for name in ("k", "v", "ks", "vs"):
        if s[name] is not None:
            s[name][:, dst] = s[name][:, src]
    return table, s["k"], s["v"]


def _plain(s):
    c = s["case"]
    if c["op"] == "attend":
        return _plain_attend(s)
    if c["op"] == "step":
        slots = torch.arange(c["B"], device=s["lens"].device)
        _plain_write(s, slots, s["lens"] - 1, s["kn"][:, :, 0], s["vn"][:, :, 0])
        return _step_outputs(s, _plain_attend(s))
    if c["op"] in ("append", "append_read"):
        _plain_write(s, s["of"], s["at"], s["kn"][0].transpose(0, 1),
                     s["vn"][0].transpose(0, 1))
        return (s["k"], s["v"]) if c["op"] == "append" and c["kv"] != "i8" \
            else _plain_read(s)
    return _plain_fork(s) if c["op"] == "fork" else _plain_compact(s)


def _step_outputs(s, out):
    """The step's output and the pool it wrote to (an int8 pool's values show
    in the output of the token that was just written)."""
    return (out,) if s["ks"] is not None else (out, s["k"], s["v"])


def run(s):
    if not own:
        return _plain(s)
    c, cache = s["case"], s["cache"]
    if c["op"] == "attend":
        return cache.attention(s["q"], window=c["window"], sinks=c["sinks"],
                               out_dtype=s["out_dtype"])
    if c["op"] == "step":
        return _step_outputs(s, cache.step(
            s["q"], s["kn"], s["vn"], window=c["window"], sinks=c["sinks"],
            out_dtype=s["out_dtype"]))
    if c["op"] in ("append", "append_read"):
        cache.append(s["kn"], s["vn"])
        if c["op"] == "append" and c["kv"] != "i8":
            return s["k"], s["v"]
        return [list(cache.read(b)) for b in range(c["B"])]
    if c["op"] == "fork":
        cache.free(s["dst"])          # what an earlier pass had forked
        cache.fork(s["src"], s["dst"])
        cache.begin(s["dst"])
        return cache.table, cache.lens, s["k"], s["v"]
    # a pool taken over with its map (an earlier pass had packed it)
    cache.restore_map(s["table0"], s["lens0"])
    cache.compact()
    return cache.table, s["k"], s["v"]


# -------------------------------------------------------------------- exact

def _rows64(s, name, b, n):
    """(n, H, D) in 64 bits: token t of row b from its page, one index each."""
    P = s["case"]["page"]
    t = torch.arange(n, device=DEV)
    page = torch.tensor(s["rows"][b], device=DEV, dtype=torch.long)[t // P]
    x = s[name][0][page, :, t % P].double()
    if s[name + "s"] is not None:
        x = x * s[name + "s"][0][page, :, t % P].double()[..., None]
    return x


def _held64(c, x):
    """What the cache holds for new tokens x (..., D), in 64 bits."""
    x = x.double()
    if c["kv"] != "i8":
        return x
    top = x.abs().amax(-1, keepdim=True)
    code = torch.round((127.0 * x) / top.clamp(min=1e-300))
    return code * (top / 127.0).float().double()


def exact(c, seed):
    if c["op"] in ("fork", "compact"):
        return None                       # copies and whole numbers
    s = _inputs(c, seed)
    lens = _lens(c)
    if c["op"] in ("append", "append_read"):
        kv = [_held64(c, s[n][0]) for n in ("kn", "vn")]      # (H, N, D)
        ends = np.cumsum([0] + lens)
        if c["op"] == "append_read" or c["kv"] == "i8":
            return [[x[None, :, a:b] for x in kv]
                    for a, b in zip(ends[:-1], ends[1:])]
        pools = []
        for x in kv:
            pool = torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV)
            for b, n in enumerate(lens):
                for i, p in enumerate(s["rows"][b]):
                    part = x[:, ends[b] + i * c["page"]:
                             min(ends[b] + (i + 1) * c["page"], ends[b + 1])]
                    pool[0, p, :, :part.shape[1]] = part
            pools.append(pool)
        return tuple(pools)
    B, H, G, D = c["B"], c["Hk"], c["G"], c["D"]
    out = torch.zeros(B, H * G, 1, D, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        keep = [t for t in range(min(c["sinks"], n))] if c["window"] else []
        first = max(0, n - c["window"]) if c["window"] else 0
        keep = torch.tensor([t for t in keep if t < first], dtype=torch.long,
                            device=DEV)
        keep = torch.cat([keep, torch.arange(first, n, device=DEV)])
        k, v = (_rows64(s, name, b, n) for name in "kv")
        if c["op"] == "step":
            k[-1], v[-1] = (_held64(c, s[i][b, :, 0]) for i in ("kn", "vn"))
        k, v = k[keep], v[keep]
        for h in range(H):
            q = s["q"][b, h * G:(h + 1) * G, 0].double()
            w = torch.softmax(q @ k[:, h].T / math.sqrt(D), dim=-1)
            out[b, h * G:(h + 1) * G, 0] = w @ v[:, h]
    if c["op"] == "step":
        return (out,) if c["kv"] == "i8" else (out, None, None)
    return out
