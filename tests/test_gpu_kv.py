"""The 8-bit paged KV cache on the GPU (tl_kv_slots, tl_kv_commit, tl_kv_attention through the binding) against the plain
64-bit statements in oracle/kv.py.

Bars. Slot maps and commits are exact: every page id, slot, byte and scale is compared. Attention, per element, with W = sum
p |v| / sum p, A = the largest scale * sum |q k| of the row and C = the largest scale * max |q| * sum |k|, from the oracle,
over n cached tokens of D channels:

    |y - y_ref| <= 2^-8 |y_ref| + W (2^-11 + 4 * 2^-24 * (D A + n) + 2^-19 + 2^-16.8 C)

The terms: bf16 output, half a step 2^-8. Weights p rounded to f16 for the product with V, half a step 2^-11. A score is D
products (exact in fp32) summed in fp32, each addition within 2^-23 (a truncating adder), so it is off by D 2^-23 A and its p by
as much, once above and once below the division: 4 * 2^-24 D A. Sums over n tokens above and below: the same with n. exp2, its
argument's rounding, the division and the factors: within 2^-19 for arguments up to 2^4, times W. Q is held in two E4M3
terms under a scale that brings the row's largest magnitude above 224: the second term's smallest step is 2^-9, so an element
is off by at most 2^-10 / 224 < 2^-17.8 of the largest, a score by 2^-17.8 C, and y by twice that (above and below the
division).
"""

import math

import numpy as np
import pytest
import torch

from oracle import kv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import nvfp4_weight_gemm_b200 as tl  # noqa: E402

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _init():
    from nvfp4_weight_gemm_b200 import build
    build.build()
    tl.init(0)
    yield
    tl.check_device_error()


def _i32(v):
    return torch.tensor(np.asarray(v, np.int64).astype(np.int32), device=DEV)


def _bf16(a):
    """float array -> (bf16 tensor on the GPU, its values as float64)."""
    t = torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.to(torch.float64).numpy()


# ---------------------------------------------------------------- block tables and slot maps

def _slots_state(rs, B, P, top, spare=5, width_spare=1):
    lens = rs.integers(0, top + 1, B)
    blocks = -(-lens // P)
    width = max(1, -(-top // P)) + width_spare
    n_pages = int(blocks.sum()) + B * width // 2 + spare
    order = rs.permutation(n_pages)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, : blocks[b]] = order[at : at + blocks[b]]
        at += blocks[b]
    free = np.full(n_pages, 77)
    free[: n_pages - at] = order[at:]
    return lens, table, free, n_pages - at


def _run_slots(lens, want, P, table, free, n_free, room):
    dl, dt, df, dn = _i32(lens), _i32(table), _i32(free), _i32([n_free])
    s, st, info = (torch.full((n,), 123456, dtype=torch.int32, device=DEV) for n in (room, len(lens) + 1, 4))
    tl.kv_slots(dl, _i32(want), dt, df, dn, P, s, st, info)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (dl, dt, df, dn, s, st, info)]


def _check_slots(lens, want, P, table, free, n_free, room):
    ref = kv.slots(lens, want, P, table, free, n_free, room)
    got = _run_slots(lens, want, P, table, free, n_free, room)
    assert got[0].tolist() == list(ref[0])
    assert np.array_equal(got[1], ref[1]) and np.array_equal(got[2], ref[2]) and int(got[3][0]) == ref[3]
    assert np.array_equal(got[4], ref[4]) and got[5].tolist() == list(ref[5]) and got[6].tolist() == list(ref[6])
    return got, ref


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("B,top", [(1, 1), (1, 1000), (7, 40), (33, 300), (1024, 90)])
def test_slots_match_the_plain_statement(P, B, top):
    rs = np.random.default_rng(B * 1000 + P)
    lens, table, free, n = _slots_state(rs, B, P, top)
    want = np.where(rs.random(B) < 0.2, 0, np.clip(lens + rs.integers(-top // 3 - 1, top // 3 + 2, B), 0, top))
    grow = int(np.maximum(want - lens, 0).sum())
    got, ref = _check_slots(lens, want, P, table, free, n, grow + 3)
    assert ref[6][0] in (0, 1)
    # back again: growth and return undo each other where no pages were both returned and taken
    if ref[6][0] == 0 and (want >= lens).all():
        back, _ = _check_slots(ref[0], lens, P, ref[1], ref[2], ref[3], 5)
        assert np.array_equal(back[1], table)


def test_slots_many_tokens_share_the_work_of_several_blocks():
    # more slots than one block deals out at once: prompts of thousands of tokens next to requests that end
    rs = np.random.default_rng(5)
    lens, table, free, n = _slots_state(rs, 600, 16, 500, spare=20000, width_spare=400)
    want = np.where(np.arange(600) % 7 == 2, 0, lens + rs.integers(0, 600, 600))
    want[11] = lens[11] + 6000
    got, ref = _check_slots(lens, want, 16, table, free, n, int(np.maximum(want - lens, 0).sum()) + 1000)
    assert ref[6] == [0, 0, 0, 0]
    # returned exactly
    assert _check_slots(ref[0], lens, 16, ref[1], ref[2], ref[3], 40000)[1][6] == [0, 0, 0, 0]


@pytest.mark.parametrize("room", [1, 2047, 2048, 2049, 4097, 8193, 9001])
def test_slots_of_every_number_of_blocks(room):
    # the arrays' room sets how many blocks deal the slots out, whether they are filled or not
    rs = np.random.default_rng(room)
    lens, table, free, n = _slots_state(rs, 70, 32, 200, spare=2000, width_spare=200)
    want = lens + rs.integers(0, 5, 70)
    want[5] += max(0, room - int((want - lens).sum()) - int(rs.integers(0, 3)))
    want[9] = 0
    _check_slots(lens, want, 32, table, free, n, room)


def test_slots_refuse_and_leave():
    table, free = np.array([[0, -1, -1], [1, -1, -1]]), np.array([2, 9, 9, 9])
    for lens, want, n, room in (([16, 16], [32, 32], 1, 99), ([16, 16], [18, 8], 1, 1), ([16, 16], [49, 18], 1, 9),
                                ([-1, 16], [3, 17], 1, 9), ([16, 16], [-5, 17], 1, 9), ([16, 16], [0, 0], 3, 9), ([16, 16], [17, 16], -1, 9),
                                ([16, 16], [16, 16], 1, 0), ([16, 60], [16, 0], 1, 4)):
        _check_slots(np.array(lens), np.array(want), 16, table, free, n, room)


# ---------------------------------------------------------------- commits

def _rand_pool(rs, n_pages, heads, P, D, spread=2.0):
    """A pool as commits leave it: bytes without NaN, scales powers of two around 2^-7."""
    pages = rs.integers(0, 256, (n_pages, heads, 2, P * D), dtype=np.uint8)
    pages = np.where(pages & 0x7F == 0x7F, pages - 1, pages).astype(np.uint8)
    scales = (2.0 ** np.round(rs.normal(-7, spread, (n_pages, heads, 2)))).astype(np.float32)
    return pages, scales


def _check_commit(pages, scales, P, k, v, slots, src=None, pad=0):
    heads, D = k.shape[1:]
    n = k.shape[0]
    both = np.concatenate([k.reshape(n, -1), np.zeros((n, pad)), v.reshape(n, -1)], 1)
    d, h = _bf16(both)
    dk = d[:, : heads * D].view(n, heads, D)
    dv = d[:, heads * D + pad :].view(n, heads, D)
    kh, vh = h[:, : heads * D].reshape(n, heads, D), h[:, heads * D + pad :].reshape(n, heads, D)
    dp, ds = torch.from_numpy(pages.copy()).to(DEV), torch.from_numpy(scales.copy()).to(DEV)
    tl.kv_commit(tl.KvCache(dp, ds, P), dk, dv, _i32(slots), None if src is None else _i32(src))
    torch.cuda.synchronize()
    rp, rsc = kv.commit(pages, scales, P, kh, vh, list(slots), src)
    gp, gs = dp.cpu().numpy(), ds.cpu().numpy()
    assert np.array_equal(gs, rsc)
    same = kv.TABLE[gp] == kv.TABLE[rp]
    assert (same | ((gp & 0x7F == 0x7F) & (rp & 0x7F == 0x7F))).all(), np.argwhere(gp != rp)[:5]
    return gp, gs


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("off,n", [(0, 1), (5, 1), (15, 2), (0, 16), (3, 13), (7, 150), (0, 300)])
def test_commit_bytes_are_the_plain_statements(D, P, off, n):
    rs = np.random.default_rng(D + P + 17 * off + n)
    pages, scales = _rand_pool(rs, 24, 2, P, D)
    ids = rs.permutation(24)
    pos = off + np.arange(n)
    slots = ids[pos // P] * P + pos % P
    k, v = rs.normal(0, 1, (n, 2, D)), rs.normal(0, 3, (n, 2, D))
    k[:, :, 7] *= 20.0
    _check_commit(pages, scales, P, k, v, slots)


def test_commit_of_many_requests_with_gaps_sources_and_strides():
    rs = np.random.default_rng(9)
    P, D, H = 32, 128, 3
    pages, scales = _rand_pool(rs, 90, H, P, D)
    ids, slots = rs.permutation(90), []
    for b in range(40):
        lo = int(rs.integers(0, 40))
        pos = lo + np.arange(int(rs.integers(0, 24)))
        slots += list(ids[2 * b + pos // P] * P + pos % P) + [-1] * int(rs.integers(0, 3))
    n = len(slots)
    src = rs.integers(0, n + 6, n)
    k, v = rs.normal(0, 1, (n + 6, H, D)), rs.normal(0, 1, (n + 6, H, D))
    _check_commit(pages, scales, P, k, v, np.array(slots), src=list(src), pad=40)


def test_commit_long_prompts_take_the_page_chunks():
    rs = np.random.default_rng(10)
    for P in (16, 128):
        pages, scales = _rand_pool(rs, 2200 // P + 8, 1, P, 64)
        ids = rs.permutation(len(pages))
        slots = np.zeros(0, int)
        at = 0
        for o, m in ((0, 700), (9, 690), (1, 1), (15, 300)):
            pos = o + np.arange(m)
            slots = np.concatenate([slots, ids[at + pos // P] * P + pos % P])
            at += -(-(o + m) // P)
        n = len(slots)
        _check_commit(pages, scales, P, rs.normal(0, 1, (n, 1, 64)), rs.normal(0, 1, (n, 1, 64)), slots)


@pytest.mark.parametrize("P,H,D,n", [(16, 8, 64, 330), (64, 8, 128, 450), (64, 16, 64, 900), (128, 4, 128, 1500)])
def test_commit_short_runs_of_which_a_block_writes_several(P, H, D, n):
    # requests of 1 to 20 tokens behind none or some, of magnitudes far apart (scales grow), a few values not finite
    rs = np.random.default_rng(P + n)
    n_pages = 2 * n // P + n // 4 + 8
    pages, scales = _rand_pool(rs, n_pages, H, P, D)
    ids, slots, size, at = rs.permutation(n_pages), [], [], 0
    while len(slots) < n:
        pos = int(rs.integers(0, P)) * int(rs.integers(0, 2)) + np.arange(int(rs.integers(1, 21)))
        if at + pos[-1] // P >= n_pages:
            break
        slots += list(ids[at + pos // P] * P + pos % P)
        size += [2.0 ** int(rs.integers(-9, 9))] * len(pos)
        at += pos[-1] // P + 1
    m = len(slots)
    k, v = rs.normal(0, 1, (2, m, H, D)) * np.array(size)[None, :, None, None]
    for x in (k, v):
        for value in (np.nan, np.inf, -np.inf):
            x[rs.integers(0, m, 5), rs.integers(0, H, 5), rs.integers(0, D, 5)] = value
    _check_commit(pages, scales, P, k, v, np.array(slots))


@pytest.mark.parametrize("P", [16, 64])
def test_commit_extremes(P):
    rs = np.random.default_rng(11)
    D = 64
    pages, scales = _rand_pool(rs, 8, 1, P, D)
    scales[1], scales[2], scales[3] = 2.0 ** -60, 2.0 ** 60, 2.0 ** 3
    n = 6
    k, v = rs.normal(0, 1, (n, 1, D)), rs.normal(0, 1, (n, 1, D))
    k[0, 0, 3], v[0, 0, 4] = np.nan, np.inf            # NaN bytes; the scale comes from the finite values
    k[1], v[1, 0, 9] = 0.0, -np.inf
    k[2, 0, 5], v[2] = 3e38, 0.0                       # over 448 * 2^60: saturates
    k[3], v[3] = 1e-30, 1e-38                          # under the smallest scale
    k[4, 0, :] = np.where(np.arange(D) % 2, 448.0, -448.0)
    v[5, 0, :] = 449.0
    # a page of its own each (fresh), then the same rows behind tokens that are there already
    _check_commit(pages, scales, P, k, v, np.array([P * 1, P * 2, P * 3, P * 4, P * 5, P * 6]))
    _check_commit(pages, scales, P, k, v, np.array([P * 1 + 5, P * 2 + 5, P * 3 + 5, P * 4 + 5, P * 5 + 15, P * 6 + 9]))
    _check_commit(pages, scales, P, k, v, P * 3 + 4 + np.arange(6))


def test_commit_flags_what_is_out_of_range():
    rs = np.random.default_rng(12)
    pages, scales = _rand_pool(rs, 4, 1, 16, 64)
    k = v = rs.normal(0, 1, (2, 1, 64))
    _check_commit(pages, scales, 16, k, v, np.array([64, 17]))      # slot 64 is behind the pool: nothing written
    with pytest.raises(tl.TlError, match="DEVICE_FAULT"):
        tl.check_device_error()
    d, _ = _bf16(k)
    c = tl.KvCache(torch.from_numpy(pages.copy()).to(DEV), torch.from_numpy(scales.copy()).to(DEV), 16)
    tl.kv_commit(c, d, d, _i32([16]), src=_i32([2]))                # row 2 of 2: zeros
    with pytest.raises(tl.TlError, match="DEVICE_FAULT"):
        tl.check_device_error()
    assert not (c.pages[1, 0, 0].view(-1, 16, 16)[:, 0] & 0x7F).any()
    tl.check_device_error()


# ---------------------------------------------------------------- attention

def _tree_masks(rs, rows):
    out = []
    for t in rows:
        m = []
        for i in range(t):
            m.append((1 << i) | (m[int(rs.integers(0, i))] if i else 0))
        out += m
    return np.array(out, np.int64)


class Case:
    """Inputs of one attention call on the GPU and in the oracle's form."""

    def __init__(self, seed, lens, rows, hq, hkv, D, P, new=True, masks=None, spread=1.0, q_size=1.0, extra_pages=3):
        rs = self.rs = np.random.default_rng(seed)
        self.lens, self.rows, self.P, self.D, self.hq, self.hkv = list(lens), list(rows), P, D, hq, hkv
        B, R = len(lens), int(sum(rows))
        blocks = [-(-n // P) for n in lens]
        n_pages = sum(blocks) + extra_pages
        self.pages, self.scales = _rand_pool(rs, n_pages, hkv, P, D, spread)
        # normal values instead of all bytes: scores of ordinary size
        self.pages = kv.e4m3_bytes(rs.normal(0, 60, self.pages.shape)).reshape(self.pages.shape)
        ids, at = rs.permutation(n_pages), 0
        self.table = np.full((B, max(blocks + [1]) + 1), -1)
        for b in range(B):
            self.table[b, : blocks[b]] = ids[at : at + blocks[b]]
            at += blocks[b]
        # what lies behind a request's last token in its last page must not matter
        for b, n in enumerate(lens):
            if n % P:
                page = self.table[b, blocks[b] - 1]
                for t in range(n % P, P):
                    self.pages[page, :, 0][:, kv.place_k(t, np.arange(D), P)] = 0x7F
                    self.pages[page, :, 1][:, kv.place_v(t, np.arange(D), D)] = 0xFF
        self.start = np.concatenate([[0], np.cumsum(rows)])
        self.q = rs.normal(0, q_size, (R, hq, D))
        self.kn, self.vn = (rs.normal(0, 1, (R, hkv, D)) for _ in range(2)) if new else (None, None)
        self.masks = _tree_masks(rs, rows) if masks is None else np.asarray(masks)
        self.scale = D ** -0.5

    def device(self):
        self.dq, self.qv = _bf16(self.q)
        if self.kn is not None:
            self.dkn, self.knv = _bf16(self.kn)
            self.dvn, self.vnv = _bf16(self.vn)
        else:
            self.dkn = self.dvn = self.knv = self.vnv = None
        self.cache = tl.KvCache(torch.from_numpy(self.pages).to(DEV), torch.from_numpy(self.scales).to(DEV), self.P)
        self.dtable, self.dlens, self.dstart = _i32(self.table), _i32(self.lens), _i32(self.start)
        self.dmask = torch.from_numpy(self.masks.astype(np.uint32).view(np.int32)).to(DEV)
        return self

    def run(self, **kw):
        args = dict(mask=self.dmask, row_start=self.dstart, max_rows=max(self.rows + [1]), scale=self.scale)
        args.update(kw)
        y = tl.kv_attention(self.dq, self.cache, self.dtable, self.dlens, self.dkn, self.dvn, **args)
        torch.cuda.synchronize()
        return y

    def reference(self):
        return kv.attention(self.qv, self.pages, self.scales, self.P, self.table, self.lens, self.knv, self.vnv, self.masks,
                            self.start, self.scale)

    def check(self, y, ref=None):
        out, weight, size, reach = self.reference() if ref is None else ref
        n = np.zeros(len(out))
        for b, m in enumerate(self.lens):
            n[self.start[b] : self.start[b + 1]] = m + 32
        off = 2.0 ** -11 + 4 * 2.0 ** -24 * (self.D * size + n[:, None]) + 2.0 ** -19 + 2.0 ** -16.8 * reach
        bar = 2.0 ** -8 * np.abs(out) + weight * off[..., None]
        got = y.float().cpu().numpy().astype(np.float64)
        bad = ~(np.abs(got - out) <= bar)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], out[bad][:4], bar[bad][:4])


HEADS = [(1, 1), (5, 1), (4, 4), (16, 2), (10, 2)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 127, 128, 129, 300])
def test_attention_one_row(D, P, n):
    c = Case(n + P, [n], [1], 10, 2, D, P).device()
    c.check(c.run())


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("rows", [2, 7, 8, 16, 24, 31, 32])
def test_attention_trees(hq, hkv, rows):
    c = Case(100 * hq + rows, [133], [rows], hq, hkv, 128 if rows % 2 else 64, 32).device()
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 128])
def test_attention_ragged_batch(D):
    lens = [0, 1, 640, 128, 77, 0, 1025, 16, 33, 127]
    rows = [3, 1, 32, 0, 8, 1, 5, 32, 0, 2]
    c = Case(7, lens, rows, 10, 2, D, 16).device()
    c.check(c.run())


@pytest.mark.parametrize("D,hq,hkv,rows", [(64, 16, 4, 16), (128, 10, 2, 32), (64, 2, 2, 1)])
def test_attention_many_tiles_and_requests_a_block(D, hq, hkv, rows):
    # every block walks over several requests and heads, and over several tiles of most of them
    rs = np.random.default_rng(D + rows)
    n = 12
    c = Case(6, [int(x) for x in rs.integers(0, 3000, n)], [int(x) for x in rs.integers(1, rows + 1, n)], hq, hkv, D, 16).device()
    y = c.run()
    c.check(y)
    for _ in range(5):
        assert torch.equal(y, c.run())


def test_attention_long_context_and_many_requests():
    c = Case(8, [9000], [4], 5, 1, 128, 64).device()
    c.check(c.run())
    rs = np.random.default_rng(3)
    c = Case(9, [int(x) for x in rs.integers(0, 60, 300)], [1] * 300, 2, 1, 64, 16).device()
    c.check(c.run(row_start=None, max_rows=None))


def test_attention_largest_group_and_tree():
    c = Case(10, [200, 3], [32, 32], 32, 2, 128, 64).device()    # 16 query heads a KV head: 512 rows a unit
    c.check(c.run())


def test_attention_without_new_rows_and_with_causal_default():
    c = Case(11, [40, 0, 5], [1, 2, 3], 4, 2, 64, 16, new=False).device()
    y = c.run()
    assert not y[1:3].any()                                       # nothing to see: zeros
    c.check(y)
    rows = [4, 1, 32]
    c = Case(12, [40, 0, 5], rows, 4, 2, 64, 16, masks=np.concatenate([(2 << np.arange(t)) - 1 for t in rows])).device()
    c.check(c.run(mask=None))
    assert torch.equal(c.run(mask=None), c.run())


def test_attention_rows_that_see_nothing_and_nan_in_unseen_nodes():
    # node 1 holds NaN and infinities and only itself sees it; node 2 sees nothing at all; bits behind the tree do not count
    masks = [0x1, 0x2, 0x0, 0xFFFFFFF9 & ~0x2]
    for n in (0, 40):
        c = Case(13, [n], [4], 4, 2, 128, 16, masks=masks)
        c.kn[1], c.vn[1] = np.nan, np.inf
        c.kn[2, 0, 3] = np.inf
        c.device()
        y = c.run()
        masks_seen = [0x1, 0x2, 0x0, 0x9]
        c.masks = np.array(masks_seen)
        out, weight, size, reach = c.reference()
        got = y.float().cpu().numpy()
        assert np.isnan(got[1]).all()
        keep = [0, 2, 3]
        assert np.isfinite(got[keep]).all()
        if n == 0:
            assert not got[2].any()
        out[1] = weight[1] = size[1] = reach[1] = 0.0
        z = y.clone()
        z[1] = 0
        c.check(z, (out, weight, size, reach))


def test_attention_nan_in_a_seen_token_reaches_every_row_of_its_head_only():
    c = Case(14, [50], [2], 4, 2, 64, 16)
    page = c.table[0, 1]
    c.pages[page, 1, 0][kv.place_k(3, np.array([5]), 16)] = 0x7F      # token 19, head 1: K
    c.device()
    got = c.run().float().cpu().numpy()
    assert np.isnan(got[:, 2:]).all() and np.isfinite(got[:, :2]).all()
    c = Case(15, [50], [2], 4, 2, 64, 16)
    page = c.table[0, 1]
    c.pages[page, 0, 1][kv.place_v(3, np.array([5]), 64)] = 0xFF      # V: one channel
    c.device()
    got = c.run().float().cpu().numpy()
    assert np.isnan(got[:, :2, 5]).all() and np.isfinite(got[:, 2:]).all()
    assert np.isfinite(np.delete(got[:, :2], 5, 2)).all()


@pytest.mark.parametrize("q_size", [1e-30, 0.02, 12.0])
def test_attention_sizes_of_scores_and_scales(q_size):
    # peaked and flat softmaxes; page scales many binades apart, so that V of some pages is far larger than of others
    c = Case(16, [700, 129], [6, 1], 4, 2, 128, 16, spread=6.0, q_size=q_size).device()
    # K scales stay moderate: only V differs
    c.scales[..., 0] = 2.0 ** -6
    c.device()
    c.check(c.run())


def test_attention_weights_far_below_the_largest():
    # The weight p vs of a token's bytes is held in f16, at 2^8 or more for the row's largest of a part (the reference lags it
    # by up to 2^7, never leads): from 2^-22 of the largest down it is off by up to half a subnormal step, 2^-25 / 2^8 of the
    # largest, whatever it is itself. That shows in channels where the bytes of the tokens with large weights are zero.
    c = Case(31, [400], [5], 4, 2, 64, 16, spread=6.0, q_size=6.0)
    c.scales[..., 0] = 2.0 ** -7
    for page in range(len(c.pages)):
        for h in range(2):
            if c.scales[page, h, 1] > 2.0 ** -7:
                for t in range(16):
                    c.pages[page, h, 1][kv.place_v(t, np.arange(8), 64)] = 0
    c.device()
    out, weight, size, reach = c.reference()
    largest = np.zeros((5, 4))
    for i in range(5):
        for h in range(4):
            k = kv.cached(c.pages, c.scales, 16, 64, c.table[0], 400, h // 2, 0) @ c.qv[i, h] * c.scale
            own = np.array([c.knv[j, h // 2] @ c.qv[i, h] * c.scale for j in range(5) if c.masks[i] >> j & 1])
            top = max(k.max(), own.max())
            vs = c.scales[c.table[0][np.arange(400) // 16], h // 2, 1].astype(np.float64)
            largest[i, h] = (np.exp(k - top) * vs).max() / (np.exp(k - top).sum() + np.exp(own - top).sum())
    off = 2.0 ** -11 + 4 * 2.0 ** -24 * (64 * size + 432) + 2.0 ** -19 + 2.0 ** -16.8 * reach
    bar = 2.0 ** -8 * np.abs(out) + weight * off[..., None] + (400 * 448 * 2.0 ** -33 * largest)[..., None]
    assert (np.abs(c.run().double().cpu().numpy() - out) <= bar).all()


def test_attention_rows_of_very_different_sizes():
    # rows of one tree whose queries differ by 2^80 in size: each row's scores are as exact as alone
    c = Case(17, [300], [8], 4, 2, 64, 32)
    c.q *= (2.0 ** np.linspace(-40, 4, 8))[:, None, None]
    c.q[5] *= 2.0 ** -60
    c.device()
    c.check(c.run())


def test_attention_sink_and_long_tail():
    # one token far above all others, whose many small weights still add up to a fifth of the sum
    c = Case(18, [4096], [1], 1, 1, 64, 64)
    c.scales[:] = 2.0 ** -6
    c.q[:] = 0.0
    c.q[0, 0, 0] = 8.0
    k0 = np.zeros(c.pages[:, 0, 0].shape, np.uint8)
    c.pages[:, 0, 0] = k0
    first = c.table[0, 0]
    c.pages[first, 0, 0][kv.place_k(0, np.array([0]), 64)] = int(kv.e4m3_bytes(np.array([608.0 / 1.0]))[0])
    c.scales[first, 0, 0] = 2.0 ** -5                  # s = 8 * 448 / 32 / 8 = 14: e^14 is 1.2e6 against 4095 ones
    c.device()
    c.check(c.run())


def test_attention_scores_that_grow_along_the_cache():
    # each tile's largest score is above all before it: the running maximum moves in every tile, up and then down
    for up in (True, False):
        c = Case(19, [1100], [5], 4, 1, 64, 16)
        c.pages[:, 0, 0] = 0
        for t in range(1100):
            level = (t if up else 1100 - t) / 1100.0
            c.pages[c.table[0, t // 16], 0, 0][kv.place_k(t % 16, np.array([0]), 16)] = int(kv.e4m3_bytes(np.array([440.0 * level]))[0])
        c.scales[..., 0] = 2.0 ** -3
        c.q[:, :, 0] = np.abs(c.q[:, :, 0]) * 6.0
        c.device()
        c.check(c.run())


def test_attention_strided_rows_and_rows_left_alone():
    c = Case(20, [30, 70], [2, 3], 10, 2, 128, 16).device()
    plain = c.run()
    qkv = torch.zeros((7, (10 + 2 * 2) * 128 + 24), dtype=torch.bfloat16, device=DEV)
    out = torch.full((7, 10 * 128 + 8), 9.0, dtype=torch.bfloat16, device=DEV)
    qkv[1:6, :1280], qkv[1:6, 1280:1536], qkv[1:6, 1544:1800] = c.dq.view(5, -1), c.dkn.view(5, -1), c.dvn.view(5, -1)
    mask = torch.zeros(7, dtype=torch.int32, device=DEV)
    mask[1:6] = c.dmask
    # a row in front of the first request and one behind the last belong to nobody
    tl.kv_attention(qkv[:, :1280].unflatten(1, (10, 128)), c.cache, c.dtable, c.dlens, qkv[:, 1280:1536].unflatten(1, (2, 128)),
                    qkv[:, 1544:1800].unflatten(1, (2, 128)), mask=mask, row_start=c.dstart + 1, max_rows=3, scale=c.scale,
                    out=out[:, :1280].unflatten(1, (10, 128)))
    torch.cuda.synchronize()
    assert torch.equal(out[1:6, :1280].reshape(5, 10, 128), plain)
    assert (out[0] == 9.0).all() and (out[6] == 9.0).all() and (out[:, 1280:] == 9.0).all()


def test_attention_flags_bad_pages_and_rows_and_stays_in_bounds():
    c = Case(21, [100, 40], [2, 2], 4, 2, 64, 16).device()
    good = c.run()
    t = c.dtable.clone()
    t[0, 2], t[0, 3] = -1, 10 ** 9
    y = tl.kv_attention(c.dq, c.cache, t, c.dlens, c.dkn, c.dvn, mask=c.dmask, row_start=c.dstart, max_rows=2)
    with pytest.raises(tl.TlError, match="DEVICE_FAULT"):
        tl.check_device_error()
    assert torch.equal(y[2:], good[2:])
    for start in ([0, 3, 4], [0, 2, 5], [-1, 2, 4], [0, 2, 1]):     # too many rows, behind R, in front, backwards
        tl.kv_attention(c.dq, c.cache, c.dtable, c.dlens, c.dkn, c.dvn, mask=c.dmask, row_start=_i32(start), max_rows=2)
        with pytest.raises(tl.TlError, match="DEVICE_FAULT"):
            tl.check_device_error()
    # lengths outside the table are cut
    over = c.run()
    c.dlens[1] = -7
    cut = c.run()
    assert torch.equal(over[:2], cut[:2]) and torch.isfinite(cut.float()).all()
    tl.check_device_error()


def test_attention_equal_calls_give_equal_bits_and_graphs_replay():
    a, b = Case(22, [500, 30], [8, 8], 10, 2, 128, 64).device(), Case(23, [90, 800], [8, 8], 10, 2, 128, 64).device()
    ya, yb = a.run(), b.run()
    assert torch.equal(ya, a.run())
    outs, graphs = [], []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(tl.kv_attention(c.dq, c.cache, c.dtable, c.dlens, c.dkn, c.dvn, mask=c.dmask, row_start=c.dstart, max_rows=8))
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):      # two graphs at once: each has a workspace of its own
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ya) and torch.equal(outs[1], yb)
    # lengths are read when the graph runs
    a.dlens[0] = 77
    graphs[0].replay()
    torch.cuda.synchronize()
    a.lens[0] = 77
    a.check(outs[0])


def test_attention_on_another_stream():
    c = Case(24, [300], [4], 4, 2, 128, 32).device()
    y = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = tl.kv_attention(c.dq, c.cache, c.dtable, c.dlens, c.dkn, c.dvn, mask=c.dmask, stream=s)
    s.synchronize()
    assert torch.equal(y, z)


def test_pool_over_four_gigabytes():
    # page offsets that pass 32 bits: a request in the last pages of a 5 GB pool
    P, D, H = 128, 128, 8
    n_pages = 5 * 2 ** 30 // (H * 2 * P * D)
    cache = tl.KvCache.empty(n_pages, H, D, P, device=DEV)
    rs = np.random.default_rng(25)
    n = 200
    k, v = _bf16(rs.normal(0, 1, (n, H, D))), _bf16(rs.normal(0, 1, (n, H, D)))
    ids = [n_pages - 1, n_pages - 2]
    slots = np.array([ids[t // P] * P + t % P for t in range(n)])
    tl.kv_commit(cache, k[0], v[0], _i32(slots))
    q, qv = _bf16(rs.normal(0, 1, (1, H, D)))
    y = tl.kv_attention(q, cache, _i32([ids]), _i32([n]))
    torch.cuda.synchronize()
    small_p, small_s = kv.commit(np.zeros((2, H, 2, P * D), np.uint8), np.ones((2, H, 2), np.float32), P, k[1], v[1], list(range(n)))
    assert np.array_equal(cache.pages[ids].cpu().numpy()[0], small_p[0])
    assert np.array_equal(cache.scales[ids].cpu().numpy(), small_s)
    c = Case(26, [n], [1], H, H, D, P)
    c.pages, c.scales, c.table, c.qv, c.knv, c.vnv = small_p, small_s, np.array([[0, 1]]), qv, None, None
    c.masks = np.zeros(1, np.int64)
    c.check(y)


# ---------------------------------------------------------------- together

def test_a_served_batch_round_by_round():
    """Slot maps, prompt commits, tree attention and path commits as a serving loop uses them, against attention over the
    cache that the plain statements build."""
    rs = np.random.default_rng(30)
    B, P, D, H, HQ = 4, 16, 64, 2, 6
    n_pages, width = 40, 10
    cache = tl.KvCache.empty(n_pages, H, D, P, device=DEV)
    cache.pages.fill_(0x7F)
    cache.scales.fill_(float("nan"))
    lens, table = _i32([0] * B), _i32(np.full((B, width), -1))
    free, n_free = _i32(np.arange(n_pages)), _i32([n_pages])
    h = dict(lens=[0] * B, table=np.full((B, width), -1), free=np.arange(n_pages), n=n_pages,
             pages=np.full((n_pages, H, 2, P * D), 0x7F, np.uint8), scales=np.ones((n_pages, H, 2), np.float32))

    def move(want, rows_k, rows_v, hk, hv, src):
        room = 64
        s, st, info = (torch.zeros(m, dtype=torch.int32, device=DEV) for m in (room, B + 1, 4))
        tl.kv_slots(lens, _i32(want), table, free, n_free, P, s, st, info)
        ref = kv.slots(h["lens"], want, P, h["table"], h["free"], h["n"], room)
        h["lens"], h["table"], h["free"], h["n"] = ref[:4]
        assert ref[6] == [0, 0, 0, 0]
        if rows_k is not None:
            src = np.concatenate([src, np.zeros(room - len(src))]).astype(int)
            tl.kv_commit(cache, rows_k, rows_v, s, src=_i32(src))
            h["pages"], h["scales"] = kv.commit(h["pages"], h["scales"], P, hk, hv, list(ref[4]), list(src))
        torch.cuda.synchronize()
        assert table.cpu().numpy().tolist() == h["table"].tolist() and s.cpu().numpy().tolist() == ref[4].tolist()

    prompts = [20, 3, 17, 16]
    (k, hk), (v, hv) = (_bf16(rs.normal(0, 1, (sum(prompts), H, D))) for _ in range(2))
    move(prompts, k, v, hk, hv, np.arange(sum(prompts)))
    for rnd in range(4):
        rows = [int(x) for x in rs.integers(1, 9, B)]
        c = Case(40 + rnd, [0] * B, rows, HQ, H, D, P)
        c.lens, c.table, c.pages, c.scales = h["lens"], h["table"], h["pages"], h["scales"]
        c.device()
        c.cache, c.dtable, c.dlens = cache, table, lens
        c.check(c.run())
        # accept a path of each tree; request 2 ends in round 1 and starts again in round 2
        src, want = [], list(h["lens"])
        for b in range(B):
            path = [i for i in range(rows[b]) if (int(c.masks[c.start[b + 1] - 1]) >> i) & 1]
            if rnd == 1 and b == 2:
                want[b] = 0
                continue
            src += [int(c.start[b]) + i for i in path]
            want[b] += len(path)
        move(want, c.dkn, c.dvn, c.knv, c.vnv, np.array(src))
    tl.check_device_error()
    got = cache.pages.cpu().numpy()
    used = h["table"][h["table"] >= 0]
    assert np.array_equal(cache.scales.cpu().numpy()[used], h["scales"][used])
    assert np.array_equal(got[used], h["pages"][used])


def _wrong(t):
    """Tensors that differ from t in one thing: type, layout, shape, device."""
    twice = torch.stack([t, t], -1)
    out = [t.float() if t.dtype is torch.int32 else t.half(), t[None], t.cpu()]
    if t.numel() > 1:                                       # one element is contiguous whatever its stride
        out += [twice[..., 0], t[:-1]]
    return out


def test_binding_refuses_wrong_tensors():
    i = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=DEV)  # noqa: E731
    good = dict(lens=i(3), want=i(3), table=i(3, 2), free_pages=i(6), n_free=i(1), slots=i(9), starts=i(4), info=i(4))
    tl.kv_slots(page_tokens=16, **good)
    for name, t in good.items():
        for k, bad in enumerate(_wrong(t)):
            if k == 4 and name in ("free_pages", "slots"):
                continue                                    # any length will do
            with pytest.raises(ValueError):
                tl.kv_slots(page_tokens=16, **{**good, name: bad})
    x = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    cache = tl.KvCache(torch.zeros((6, 2, 2, 1024), dtype=torch.uint8, device=DEV), torch.ones((6, 2, 2), device=DEV), 16)
    good = dict(k=x(5, 2, 64), v=x(5, 2, 64), slots=i(5) - 1)
    tl.kv_commit(cache, **good)
    for name, t in good.items():
        for k, bad in enumerate(_wrong(t)):
            if not (k == 4 and name == "slots"):            # fewer slots than rows will do
                with pytest.raises(ValueError):
                    tl.kv_commit(cache, **{**good, name: bad})
    good = dict(q=x(5, 4, 64), table=i(2, 3), lens=i(2), k_new=x(5, 2, 64), v_new=x(5, 2, 64), mask=i(5), row_start=i(3), out=x(5, 4, 64))
    tl.kv_attention(cache=cache, max_rows=4, **good)
    for name, t in good.items():
        for bad in _wrong(t):
            with pytest.raises(ValueError):
                tl.kv_attention(cache=cache, max_rows=4, **{**good, name: bad})
    with pytest.raises(ValueError):
        tl.kv_attention(cache=cache, max_rows=4, workspace=x(99999), **good)
    # one row: its stride says nothing, and need not agree
    one = dict(q=x(1, 4, 64), table=i(1, 3), lens=i(1), k_new=x(2, 2, 64)[:1], v_new=x(1, 4, 64)[:, :2], out=x(1, 4, 64))
    tl.kv_attention(cache=cache, **one)
    torch.cuda.synchronize()
    tl.check_device_error()
