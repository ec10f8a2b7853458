"""Timed cases of the 8-bit paged KV cache of the verify pass: block tables and slot maps built on the GPU
(kv_slots), the commit of accepted tokens into the cache (kv_commit), and the attention of one token or of a
draft tree over it (kv_attention).

The cache is a pool of pages of P tokens. Per page, KV head and side (0 = K, 1 = V) it holds P * D E4M3 bytes and
one scale, a power of two; K is stored [D/16][P][16] and V [P/16][D][16], both in 16-byte groups. `run` computes each
operator in its plain form (elementary torch operations in 32 bits) or, where `own` is set, through the package.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
#: Every request's page list holds this many more entries than its longest length needs.
SPARE_BLOCKS = 2


# ---------------------------------------------------------------- the cases

def listed():
    proj = {"hq": 40, "hkv": 8, "d": 128}   # the served model's attention layers (QKV 7,168 = 40 + 2 * 8 heads of 128)
    return [
        # a chat turn that decodes alone: the latency of one short call
        {"name": "decode 1 x 1k", "op": "attention", "b": 1, "rows": 1, "len": 1000, "ragged": False, "page": 16, **proj},
        # a full decode batch over contexts of very different lengths: the cache's bytes
        {"name": "decode 64 x 8k ragged", "op": "attention", "b": 64, "rows": 1, "len": 8192, "ragged": True, "page": 64, **proj},
        # the staircase's shortest tree at its longest context
        {"name": "tree 8 x 32k", "op": "attention", "b": 1, "rows": 8, "len": 32768, "ragged": False, "page": 64, **proj},
        # the staircase's tallest tree at its shortest context: one verify pass of one request
        {"name": "tree 32 x 1k", "op": "attention", "b": 1, "rows": 32, "len": 1024, "ragged": False, "page": 32, **proj},
        # several requests sharing one verify pass, tall trees over long contexts: bytes and products alike
        {"name": "tree 32, 8 x 32k ragged", "op": "attention", "b": 8, "rows": 32, "len": 32768, "ragged": True, "page": 64, **proj},
        # a smaller model's heads, small pages, trees of 1 to 16 rows, a few requests with nothing cached yet
        {"name": "tree 16, 24 x 3k ragged", "op": "attention", "b": 24, "rows": 16, "len": 3001, "ragged": True, "page": 16,
         "hq": 16, "hkv": 4, "d": 64},
        # one accepted path of a verify pass
        {"name": "commit 1 x 5", "op": "commit", "b": 1, "tokens": 5, "ragged": False, "prefix": 700, "page": 16, "hkv": 8, "d": 128},
        # the accepted paths of a whole batch
        {"name": "commit 64 x 16 ragged", "op": "commit", "b": 64, "tokens": 16, "ragged": True, "prefix": 300, "page": 64, "hkv": 8, "d": 128},
        # a prompt's keys and values
        {"name": "commit 2 x 16k", "op": "commit", "b": 2, "tokens": 16384, "ragged": False, "prefix": 33, "page": 64, "hkv": 8, "d": 128},
        # a small batch after a verify pass: a few tokens each
        {"name": "slots 8 x 8", "op": "slots", "b": 8, "grow": 8, "len": 2000, "page": 16},
        # a large batch: prompts arrive, requests end
        {"name": "slots 1000 x 300", "op": "slots", "b": 1000, "grow": 300, "len": 4000, "page": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "commit", "slots"])
    page = rng.choice([16, 32, 64, 128])
    if op == "slots":
        return {"op": op, "b": _log(rng, 1, 1000), "grow": _log(rng, 1, 300), "len": _log(rng, 1, 4000), "page": page}
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128])
    if op == "commit":
        b = _log(rng, 1, 64)
        return {"op": op, "b": b, "tokens": _log(rng, 1, min(16384, 32768 // b)), "ragged": rng.random() < 0.5,
                "prefix": _log(rng, 1, 700), "page": page, "hkv": hkv, "d": d}
    b, rows = _log(rng, 1, 64), rng.choice([1, 1, 8, 16, 24, 32, rng.randint(2, 31)])
    most = min(32768, 262144 // b, 1_800_000 // (b * rows))
    return {"op": op, "b": b, "rows": rows, "len": _log(rng, 16, most), "ragged": rng.random() < 0.5, "page": page,
            "hq": hkv * rng.choice([1, 2, 4, 5]), "hkv": hkv, "d": d}


def _spread(n, lo, hi, ragged, key):
    """n whole numbers of lo..hi, fixed by the case alone: hi everywhere, or spread over the range."""
    if not ragged:
        return np.full(n, hi, np.int64)
    x = np.random.RandomState(1000 * key + n).uniform(0.0, 1.0, n)
    v = np.round(lo + (hi - lo) * x).astype(np.int64)
    v[n // 2] = hi
    return v


def _lens(c):
    """Cached tokens of each request of an attention case; in a ragged one every twelfth has none yet."""
    v = _spread(c["b"], 1, c["len"], c["ragged"], 1)
    if c["ragged"] and c["b"] > 12:
        v[5::12] = 0
    return v


def _rows(c):
    return _spread(c["b"], 1, c["rows"], c["ragged"], 2)


def _added(c):
    return _spread(c["b"], 1, c["tokens"], c["ragged"], 3)


def _prefixes(c):
    return _spread(c["b"], 0, c["prefix"], True, 4)


def _wants(c):
    """(lengths held, lengths wanted) of a slots case: most requests grow, every ninth ends, every fifth stays."""
    have = _spread(c["b"], 1, c["len"], True, 5)
    want = have + _spread(c["b"], 1, c["grow"], True, 6)
    i = np.arange(c["b"])
    want = np.where(i % 5 == 3, have, want)
    return have, np.where(i % 9 == 4, 0, want)


def work(c):
    if c["op"] == "attention":
        lens, rows = _lens(c), _rows(c)
        blocks = -(-lens // c["page"])
        per = c["hkv"] * c["d"]
        b = 2 * per * int(lens.sum()) + 8 * c["hkv"] * int(blocks.sum()) + 4 * int(blocks.sum())   # cache, scales, tables
        b += int(rows.sum()) * (2 * 2 * c["hq"] * c["d"] + 2 * 2 * per + 4) + 8 * c["b"]          # q, out, new K and V, masks
        return {"bytes": b, "flops": 4.0 * c["d"] * c["hq"] * float((rows * (lens + (rows + 1) / 2)).sum())}
    if c["op"] == "commit":
        n, per = int(_added(c).sum()), c["hkv"] * c["d"]
        pages = int((-(-(_prefixes(c) + _added(c)) // c["page"]) - _prefixes(c) // c["page"]).sum())
        return {"bytes": n * (2 * 2 * per + 2 * per + 8) + pages * 8 * c["hkv"], "flops": 4.0 * n * per}
    have, want = _wants(c)
    hb, wb = -(-have // c["page"]), -(-want // c["page"])
    up, down = int(np.maximum(want - have, 0).sum()), int(np.maximum(have - want, 0).sum())
    pages = int(np.abs(wb - hb).sum())
    # two calls: lengths in and out, slots out, page ids moved between stack and table, starts
    return {"bytes": 2 * (12 * c["b"] + 4 * c["b"] + 8 * pages) + 4 * (up + down), "flops": 0.0}


# ---------------------------------------------------------------- inputs

def _i32(v):
    return torch.tensor(np.asarray(v, np.int32), device=DEV)


def _power(e):
    """2^e of whole numbers e, exactly, as float32."""
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e.int())


def _pool(n_pages, c, gen):
    """A pool of pages of earlier tokens: E4M3 bytes of normal values, each page and head with a range of its own, and a few
    channels of K larger than the rest; scales are powers of two."""
    shape = (n_pages, c["hkv"], 2, c["page"] * c["d"])
    x = torch.randn(shape, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn((n_pages, c["hkv"], 2, 1), generator=gen, device=DEV))
    keys = x[:, :, 0].view(n_pages, c["hkv"], c["d"] // 16, c["page"], 16)
    keys[:, :, 1, :, 3] *= 4.0
    scales = _power(torch.ceil(torch.log2(x.abs().amax(-1) / 448.0)).clamp(min=-60.0))
    pages = (x / scales[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return pages, scales


def _tables(blocks, n_pages, width, gen):
    """Pages dealt out to requests in a random order: (table, the pages left, in the order of the stack)."""
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(blocks), width), -1, dtype=torch.int32, device=DEV)
    used = int(blocks.sum())
    b = np.repeat(np.arange(len(blocks)), blocks)
    j = np.arange(used) - np.repeat(np.cumsum(blocks) - blocks, blocks)
    table[torch.from_numpy(b).to(DEV), torch.from_numpy(j).to(DEV)] = order[:used]
    return table, order[used:]


def _tree_masks(rows, gen_seed):
    """Ancestor masks of random draft trees: node 0 is the root, the others hang below an earlier node."""
    rs = random.Random(gen_seed)
    out = []
    for t in rows:
        m = []
        for i in range(int(t)):
            m.append((1 << i) | (m[rs.randrange(max(0, i - 4), i)] if i else 0))
        out += m
    return np.array(out, np.uint32)


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "slots":
        have, want = _wants(c)
        most = -(-np.maximum(have, want) // c["page"])
        blocks = -(-have // c["page"])
        n_pages, width = int(most.sum()) + 7, int(most.max()) + SPARE_BLOCKS
        table, left = _tables(blocks, n_pages, width, gen)
        free = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        free[: left.numel()] = left
        room = int(max(np.maximum(want - have, 0).sum(), np.maximum(have - want, 0).sum())) + 3
        s.update(lens=_i32(have), have=_i32(have), want=_i32(want), table=table, free=free, n_free=_i32([left.numel()]),
                 slots=[torch.zeros(room, dtype=torch.int32, device=DEV) for _ in range(2)],
                 starts=[torch.zeros(c["b"] + 1, dtype=torch.int32, device=DEV) for _ in range(2)],
                 info=[torch.zeros(4, dtype=torch.int32, device=DEV) for _ in range(2)])
        return s
    if c["op"] == "commit":
        pre, add = _prefixes(c), _added(c)
        blocks = -(-(pre + add) // c["page"])
        n_pages = int(blocks.sum()) + 5
        s["pages"], s["scales"] = _pool(n_pages, c, gen)
        table, _ = _tables(blocks, n_pages, int(blocks.max()), gen)
        b = np.repeat(np.arange(c["b"]), add)
        pos = np.arange(int(add.sum())) - np.repeat(np.cumsum(add) - add, add) + np.repeat(pre, add)
        b, pos = torch.from_numpy(b).to(DEV), torch.from_numpy(pos).to(DEV)
        s["slots"] = (table[b, pos // c["page"]].long() * c["page"] + pos % c["page"]).to(torch.int32)
        n, per = int(add.sum()), c["hkv"] * c["d"]
        # rows of the projection's output: queries (here as many heads), keys, values side by side; the accepted
        # nodes are some of the rows
        rows = n if c["tokens"] > 64 else n + 9
        qkv = torch.randn((rows, 3 * per), generator=gen, device=DEV)
        qkv[:, per + 19 :: c["d"]] *= 4.0
        s["qkv"] = qkv.to(torch.bfloat16)
        s["k"] = s["qkv"][:, per : 2 * per].view(rows, c["hkv"], c["d"])
        s["v"] = s["qkv"][:, 2 * per :].view(rows, c["hkv"], c["d"])
        s["src"] = None if c["tokens"] > 64 else torch.randperm(rows, generator=gen, device=DEV)[:n].to(torch.int32)
    else:
        lens, rows = _lens(c), _rows(c)
        blocks = -(-lens // c["page"])
        n_pages = max(1, int(blocks.sum()))
        s["pages"], s["scales"] = _pool(n_pages, c, gen)
        s["table"], _ = _tables(blocks, n_pages, int(blocks.max()) + SPARE_BLOCKS, gen)
        s["lens"], s["row_start"] = _i32(lens), _i32(np.concatenate([[0], np.cumsum(rows)]))
        r, per = int(rows.sum()), c["hkv"] * c["d"]
        qkv = torch.randn((r, c["hq"] * c["d"] + 2 * per), generator=gen, device=DEV)
        s["qkv"] = qkv.to(torch.bfloat16)
        a = c["hq"] * c["d"]
        s["q"] = s["qkv"][:, :a].view(r, c["hq"], c["d"])
        s["k"] = s["qkv"][:, a : a + per].view(r, c["hkv"], c["d"])
        s["v"] = s["qkv"][:, a + per :].view(r, c["hkv"], c["d"])
        s["mask"] = torch.from_numpy(_tree_masks(rows, seed).view(np.int32)).to(DEV)
    return s


# ---------------------------------------------------------------- one pass

def _keys(bytes_, c):
    """E4M3 values of K pages [..., P * D] as float32 [..., P, D]."""
    x = bytes_.view(torch.float8_e4m3fn).to(torch.float32).view(*bytes_.shape[:-1], c["d"] // 16, c["page"], 16)
    return x.transpose(-3, -2).flatten(-2)


def _values(bytes_, c):
    """E4M3 values of V pages [..., P * D] as float32 [..., P, D]."""
    x = bytes_.view(torch.float8_e4m3fn).to(torch.float32).view(*bytes_.shape[:-1], c["page"] // 16, c["d"], 16)
    return x.transpose(-2, -1).flatten(-3, -2)


def _plain_attention(s):
    c = s["c"]
    b, t, g, d, p = c["b"], c["rows"], c["hq"] // c["hkv"], c["d"], c["page"]
    ids = s["table"].clamp(min=0).long()
    n = ids.shape[1] * p
    sc = s["scales"][ids]                                                       # [b, blocks, hkv, 2]
    k = _keys(s["pages"][ids][:, :, :, 0], c) * sc[..., 0, None, None]          # [b, blocks, hkv, p, d]
    v = _values(s["pages"][ids][:, :, :, 1], c) * sc[..., 1, None, None]
    k, v = (x.permute(0, 2, 1, 3, 4).reshape(b, c["hkv"], n, d) for x in (k, v))
    at = torch.arange(t, device=DEV)
    count = (s["row_start"][1:] - s["row_start"][:-1]).long()
    row = (s["row_start"][:-1, None].long() + at).clamp(max=s["q"].shape[0] - 1)   # [b, t]
    there = at < count[:, None]
    q = s["q"][row].float().view(b, t, c["hkv"], g, d).permute(0, 2, 1, 3, 4).reshape(b, c["hkv"], t * g, d)
    kn, vn = (s[x][row].float().permute(0, 2, 1, 3) for x in ("k", "v"))           # [b, hkv, t, d]
    old = torch.einsum("bhrd,bhnd->bhrn", q, k) * d ** -0.5
    old = old.masked_fill((torch.arange(n, device=DEV) >= s["lens"][:, None])[:, None, None], -math.inf)
    new = torch.einsum("bhrd,bhnd->bhrn", q, kn).view(b, c["hkv"], t, g, t) * d ** -0.5
    sees = ((s["mask"][row][:, :, None] >> at) & 1).bool() & there[:, None, :]     # [b, t, t]
    new = new.masked_fill(~sees[:, None, :, None, :], -math.inf).view(b, c["hkv"], t * g, t)
    top = torch.maximum(old.amax(-1, keepdim=True), new.amax(-1, keepdim=True))
    top = top.masked_fill(top == -math.inf, 0.0)
    old, new = torch.exp(old - top), torch.exp(new - top)
    total = old.sum(-1, keepdim=True) + new.sum(-1, keepdim=True)
    y = torch.einsum("bhrn,bhnd->bhrd", old, v) + torch.einsum("bhrn,bhnd->bhrd", new, vn)
    y = torch.where(total > 0, y / total, 0.0).view(b, c["hkv"], t, g, d).permute(0, 2, 1, 3, 4)
    return y.reshape(b, t, c["hq"], d)[there].to(torch.bfloat16)


def _exponent(top):
    """The smallest e in -60..60 with top <= 448 * 2^e, as float32."""
    m, e = torch.frexp(top)
    e = e - 9 + (m > 0.875)                       # 448 = 0.875 * 2^9
    return torch.where(top > 0, e, -60).clamp(-60, 60).float()


def _plain_commit(s):
    c = s["c"]
    p, d, h = c["page"], c["d"], c["hkv"]
    k, v = (s[x].float() if s["src"] is None else s[x][s["src"].long()].float() for x in ("k", "v"))
    page, off = s["slots"].long() // p, s["slots"].long() % p
    ids, at = torch.unique(page, return_inverse=True)
    first = torch.full((ids.numel(),), p, device=DEV).scatter_reduce(0, at, off, "amin")
    tops = torch.zeros((ids.numel(), h, 2), device=DEV)
    for i, x in enumerate((k, v)):
        tops[..., i].scatter_reduce_(0, at[:, None].expand(-1, h), x.abs().amax(-1), "amax")
    e = _exponent(tops)
    held = (torch.frexp(s["scales"][ids])[1] - 1).float()
    e = torch.where((first == 0)[:, None, None], e, torch.maximum(e, held))
    old = s["pages"][ids]
    before = torch.arange(p, device=DEV) < first[:, None]                       # [pages, p]
    new = old.clone()
    for i, (x, values) in enumerate(((k, _keys), (v, _values))):
        moved = values(old[:, :, i], c) * _power(held - e)[..., i, None, None]
        put = torch.zeros((ids.numel(), p, h, d), device=DEV)
        put[at, off] = x * _power(-e[at][..., i])[..., None]
        there = torch.zeros((ids.numel(), p), dtype=torch.bool, device=DEV)
        there[at, off] = True
        y = torch.where(there[:, None, :, None], put.transpose(1, 2), moved).to(torch.float8_e4m3fn).view(torch.uint8)
        if i == 0:
            y, keep = y.view(-1, h, p, d // 16, 16).transpose(2, 3), (there | before)[:, None, None, :, None]
        else:
            y, keep = y.view(-1, h, p // 16, 16, d).transpose(3, 4), (there | before).view(-1, 1, p // 16, 1, 16)
        new[:, :, i] = torch.where(keep, y, old[:, :, i].view(y.shape)).reshape(new[:, :, i].shape)
    s["pages"][ids], s["scales"][ids] = new, _power(e)
    return s["pages"].view(torch.float8_e4m3fn), s["scales"]


def _plain_slots(s, want, i):
    p, n_pages = s["c"]["page"], s["free"].numel()
    lens, table, free, n_free = s["lens"].long(), s["table"], s["free"], s["n_free"].long()
    want = want.long()
    held, need = (lens + p - 1) // p, (want + p - 1) // p
    # pages of requests that shrink go back on the stack, the last one first
    gone = (held - need).clamp(min=0)
    each = torch.repeat_interleave(torch.arange(gone.numel(), device=DEV), gone)
    j = torch.arange(each.numel(), device=DEV)
    block = need[each] + j - (gone.cumsum(0) - gone)[each]
    free[n_free + each.numel() - 1 - j] = table[each, block]
    table[each, block] = -1
    top = n_free + each.numel()
    # pages of requests that grow come off its top
    more = (need - held).clamp(min=0)
    each = torch.repeat_interleave(torch.arange(more.numel(), device=DEV), more)
    j = torch.arange(each.numel(), device=DEV)
    table[each, held[each] + j - (more.cumsum(0) - more)[each]] = free[top - 1 - j]
    s["n_free"].copy_(top - each.numel())
    added = (want - lens).clamp(min=0)
    ends = added.cumsum(0)
    each = torch.repeat_interleave(torch.arange(added.numel(), device=DEV), added)
    pos = lens[each] + torch.arange(each.numel(), device=DEV) - (ends - added)[each]
    s["slots"][i].fill_(-1)
    s["slots"][i][: each.numel()] = table[each, pos // p] * p + (pos % p).int()
    s["starts"][i][0] = 0
    s["starts"][i][1:] = ends
    s["info"][i].zero_()
    s["lens"].copy_(want)


def run(s):
    op = s["c"]["op"]
    if own:
        import nvfp4_weight_gemm_b200 as tl
        cache = tl.KvCache(s["pages"], s["scales"], s["c"]["page"]) if op != "slots" else None
    if op == "attention":
        if own:
            return tl.kv_attention(s["q"], cache, s["table"], s["lens"], s["k"], s["v"], mask=s["mask"],
                                   row_start=s["row_start"], max_rows=s["c"]["rows"])
        return _plain_attention(s)
    if op == "commit":
        if own:
            tl.kv_commit(cache, s["k"], s["v"], s["slots"], src=s["src"])
            return s["pages"].view(torch.float8_e4m3fn), s["scales"]
        return _plain_commit(s)
    # requests grow and end, and then the lengths are taken back: one pass leaves the lengths as they were
    for i, want in ((0, s["want"]), (1, s["have"])):
        if own:
            tl.kv_slots(s["lens"], want, s["table"], s["free"], s["n_free"], s["c"]["page"], s["slots"][i], s["starts"][i],
                        s["info"][i])
        else:
            _plain_slots(s, want, i)
    return s["slots"], s["starts"], s["info"], s["table"], s["free"], s["n_free"], s["lens"]


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3_table():
    v = np.empty(256)
    for i in range(256):
        e, m = (i >> 3) & 15, i & 7
        x = math.nan if i & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[i] = -x if i & 128 else x
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _to_e4m3(x):
    """The nearest E4M3 value (ties to even) of each of x (64 bits, magnitudes up to 448)."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def exact(c, seed):
    if c["op"] == "slots":
        return None
    s = prepare(c, seed)
    table, p, d, h = _e4m3_table(), c["page"], c["d"], c["hkv"]
    if c["op"] == "attention":
        out = torch.zeros((s["q"].shape[0], c["hq"], d), dtype=torch.float64, device=DEV)
        starts, lens = s["row_start"].tolist(), s["lens"].tolist()
        bits = (s["mask"].long()[:, None] >> torch.arange(32, device=DEV)) & 1
        for b, n in enumerate(lens):
            lo, hi = starts[b], starts[b + 1]
            ids = s["table"][b, : -(-n // p)].long()
            for j in range(h):
                k = torch.cat([table[s["pages"][ids, j, 0].long()].view(-1, d // 16, p, 16).permute(0, 2, 1, 3).reshape(-1, p, d)
                               .mul(s["scales"][ids, j, 0].double()[:, None, None]).reshape(-1, d)[:n], s["k"][lo:hi, j].double()])
                v = torch.cat([table[s["pages"][ids, j, 1].long()].view(-1, p // 16, d, 16).permute(0, 1, 3, 2).reshape(-1, p, d)
                               .mul(s["scales"][ids, j, 1].double()[:, None, None]).reshape(-1, d)[:n], s["v"][lo:hi, j].double()])
                g = c["hq"] // h
                z = s["q"][lo:hi, j * g : (j + 1) * g].double() @ k.T / math.sqrt(d)
                blind = torch.cat([torch.zeros((hi - lo, n), dtype=torch.bool, device=DEV), bits[lo:hi, : hi - lo] == 0], 1)
                out[lo:hi, j * g : (j + 1) * g] = torch.softmax(z.masked_fill(blind[:, None], -math.inf), -1) @ v
        return out
    pages, scales = table[s["pages"].long()], s["scales"].double()
    src = torch.arange(s["slots"].numel(), device=DEV) if s["src"] is None else s["src"].long()
    slots = s["slots"].tolist()
    i = 0
    while i < len(slots):
        page, off = divmod(slots[i], p)
        m = 1
        while i + m < len(slots) and slots[i + m] == slots[i] + m and off + m < p:
            m += 1
        for side, x in enumerate((s["k"], s["v"])):
            y = x[src[i : i + m]].double()                                     # [m, h, d]
            scale = torch.tensor([2.0 ** next(i for i in range(-60, 61) if top <= 448.0 * 2.0 ** i)
                                  for top in y.abs().amax((0, 2)).tolist()], dtype=torch.float64, device=DEV)
            was = scales[page, :, side]
            scale = scale if off == 0 else torch.maximum(scale, was)
            if side == 0:
                view = pages[page, :, 0].view(h, d // 16, p, 16).permute(0, 2, 1, 3)      # [h, p, d/16, 16]
                y = y.view(m, h, d // 16, 16).transpose(0, 1)
            else:
                view = pages[page, :, 1].view(h, p // 16, d, 16).permute(0, 1, 3, 2).reshape(h, p, d)
                y = y.transpose(0, 1)
            f = lambda t: scale.view(-1, *[1] * (t.dim() - 1))  # noqa: E731
            w = view.clone()
            w[:, :off] = _to_e4m3(view[:, :off] * f(view).reciprocal() * was.view(-1, *[1] * (view.dim() - 1)))
            w[:, off : off + m] = _to_e4m3(y / f(y))
            if side == 0:
                pages[page, :, 0] = w.permute(0, 2, 1, 3).reshape(h, p * d)
            else:
                pages[page, :, 1] = w.view(h, p // 16, 16, d).transpose(2, 3).reshape(h, p * d)
            scales[page, :, side] = scale
        i += m
    return pages, scales
