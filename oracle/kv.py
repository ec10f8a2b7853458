"""Plain 64-bit statements of the 8-bit paged KV cache: slot maps, commits, tree attention.

Written from the definitions in include/tl_nvfp4.h, one request, page and token at a time; they share no
code with the library.
"""

from __future__ import annotations

import math

import numpy as np


def e4m3_table() -> np.ndarray:
    """The 256 E4M3 values ("fn"): S EEEE MMM, bias 7, no infinities, S.1111.111 NaN."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if b & 0x7F == 0x7F else m / 512.0 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        out[b] = -x if b & 0x80 else x
    return out


TABLE = e4m3_table()


def e4m3_bytes(x: np.ndarray) -> np.ndarray:
    """Bytes of the nearest E4M3 values, ties to the even byte; magnitudes over 448 give 448, NaN gives 0x7F."""
    x = np.asarray(x, np.float64)
    mags = TABLE[:127]
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.searchsorted(mags, a)                     # mags[hi - 1] < a <= mags[hi]
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mags[lo], mags[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    out = pick.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), out)


def place_k(t: int, c: np.ndarray, P: int) -> np.ndarray:
    """Byte of channel c of the token at place t within a page's K side."""
    return (c // 16) * P * 16 + t * 16 + c % 16


def place_v(t: int, c: np.ndarray, D: int) -> np.ndarray:
    """Byte of channel c of the token at place t within a page's V side."""
    return (t // 16) * D * 16 + c * 16 + t % 16


def slots(lens, want, P, table, free, n_free, max_slots):
    """(lens, table, free, n_free, slots, starts, info) after one call; the inputs are left alone."""
    lens, table, free = [int(x) for x in lens], np.array(table), np.array(free)
    B, width, n_pages = len(lens), table.shape[1], len(free)
    refused = [lens[b] < 0 or want[b] < 0 or lens[b] > width * P or want[b] > width * P for b in range(B)]
    goal = [lens[b] if refused[b] else int(want[b]) for b in range(B)]
    pages = lambda n: -(-n // P)  # noqa: E731
    gone = [(b, j) for b in range(B) if not refused[b] for j in range(pages(goal[b]), pages(lens[b]))]
    more = [(b, j) for b in range(B) if not refused[b] for j in range(pages(lens[b]), pages(goal[b]))]
    grow = sum(max(0, goal[b] - lens[b]) for b in range(B))
    out = np.full(max_slots, -1, np.int64)
    starts = [0] * (B + 1)
    if n_free < 0 or n_free + len(gone) > n_pages:
        info = [8 + (4 if any(refused) else 0) + (2 if grow > max_slots else 0), 0, max(0, grow - max_slots), sum(refused)]
        return lens, table, free, n_free, out, starts, info
    top = n_free + len(gone)
    for i, (b, j) in enumerate(gone):
        free[top - 1 - i] = table[b, j]
        table[b, j] = -1
    short, lack = max(0, len(more) - top), max(0, grow - max_slots)
    info = [(1 if short else 0) + (2 if lack else 0) + (4 if any(refused) else 0), short, lack, sum(refused)]
    ok = not short and not lack
    n = 0
    if ok:
        for i, (b, j) in enumerate(more):
            table[b, j] = free[top - 1 - i]
        top -= len(more)
    for b in range(B):
        starts[b] = n
        if goal[b] > lens[b] and ok:
            for pos in range(lens[b], goal[b]):
                out[n] = table[b, pos // P] * P + pos % P
                n += 1
        if goal[b] < lens[b] or ok:
            lens[b] = goal[b]
    starts[B] = n
    return lens, table, free, top, out, starts, info


def commit(pages, scales, P, k, v, slots_, src=None):
    """(pages, scales) after a commit; k, v float [rows, heads, D] (any values a bf16 holds)."""
    pages, scales = np.array(pages), np.array(scales)
    heads, D = k.shape[1], k.shape[2]
    c = np.arange(D)
    i, n = 0, len(slots_)
    while i < n:
        if slots_[i] < 0 or slots_[i] >= pages.shape[0] * P:
            i += 1
            continue
        page, off = divmod(int(slots_[i]), P)
        m = 1
        while i + m < n and off + m < P and slots_[i + m] == slots_[i] + m:
            m += 1
        for side, x in enumerate((k, v)):
            place = (lambda t: place_k(t, c, P)) if side == 0 else (lambda t: place_v(t, c, D))
            for h in range(heads):
                rows = [np.asarray(x[src[i + t] if src is not None else i + t, h], np.float64) for t in range(m)]
                top = max(float(np.max(np.abs(r[np.isfinite(r)]), initial=0.0)) for r in rows)
                e = next((q for q in range(-60, 61) if top <= 448.0 * 2.0 ** q), 60)
                if off:
                    was = int(math.log2(scales[page, h, side]))
                    if e > was:
                        for t in range(off):
                            at = place(t)
                            pages[page, h, side, at] = e4m3_bytes(TABLE[pages[page, h, side, at]] * 2.0 ** (was - e))
                    e = max(e, was)
                for t, r in enumerate(rows):
                    r = np.where(np.isfinite(r), r, np.nan)
                    pages[page, h, side, place(off + t)] = e4m3_bytes(r * 2.0 ** -e)
                scales[page, h, side] = 2.0 ** e
        i += m
    return pages, scales


def cached(pages, scales, P, D, ids, n, head, side):
    """The first n tokens' K or V of one head, float64 [n, D]."""
    c, out = np.arange(D), np.empty((n, D))
    for t in range(n):
        p, o = int(ids[t // P]), t % P
        at = place_k(o, c, P) if side == 0 else place_v(o, c, D)
        out[t] = TABLE[pages[p, head, side, at]] * float(scales[p, head, side])
    return out


def attention(q, pages, scales, P, table, lens, k_new, v_new, masks, row_start, scale):
    """(out, weight, size, reach): out float64 [R, heads, D]; weight = sum p |v| / sum p; of what the row sees, size
    [R, heads] = the largest scale * sum |q k| and reach = the largest scale * max |q| * sum |k|: what the error of a
    computed result is measured by."""
    R, Hq, D = q.shape
    heads = pages.shape[1]
    g = Hq // heads
    out, weight, size, reach = np.zeros((R, Hq, D)), np.zeros((R, Hq, D)), np.zeros((R, Hq)), np.zeros((R, Hq))
    for b, n in enumerate(lens):
        lo, hi = int(row_start[b]), int(row_start[b + 1])
        for h in range(heads):
            kc = cached(pages, scales, P, D, table[b], int(n), h, 0)
            vc = cached(pages, scales, P, D, table[b], int(n), h, 1)
            for i in range(lo, hi):
                see = [] if k_new is None else [j for j in range(hi - lo) if (int(masks[i]) >> j) & 1]
                k = np.concatenate([kc] + [np.asarray(k_new[lo + j, h], np.float64)[None] for j in see])
                v = np.concatenate([vc] + [np.asarray(v_new[lo + j, h], np.float64)[None] for j in see])
                if not len(k):
                    continue
                for a in range(h * g, (h + 1) * g):
                    x = np.asarray(q[i, a], np.float64)
                    s = scale * (k @ x)
                    p = np.exp(s - np.max(s))
                    out[i, a] = p @ v / p.sum()
                    weight[i, a] = p @ np.abs(v) / p.sum()
                    size[i, a] = abs(scale) * np.max(np.abs(k) @ np.abs(x))
                    reach[i, a] = abs(scale) * np.max(np.abs(x)) * np.max(np.abs(k).sum(1))
    return out, weight, size, reach
