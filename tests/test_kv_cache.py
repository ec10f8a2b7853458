"""8-bit paged KV cache on the host: refusals of the C ABI and of the binding, workspace sizes, and the plain 64-bit
statements (oracle/kv.py) against hand-worked values. Nothing here reaches CUDA."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv

A = 1 << 20  # fake, aligned addresses: never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    from nvfp4_weight_gemm_b200 import build, _lib
    build.build()
    return _lib.lib()


def _at(i):
    return (1 << 40) + (i << 34)   # far enough apart for any of the sizes below


def _cache(**kw):
    from nvfp4_weight_gemm_b200._lib import KvCacheC
    d = dict(pages=_at(0), scales=_at(1), n_pages=100, page_tokens=64, n_kv_heads=8, head_dim=128)
    d.update(kw)
    return KvCacheC(*d.values())


# ---------------------------------------------------------------- refusals

def test_slots_refuses(L):
    def call(lens=_at(0), want=_at(1), B=8, P=16, table=_at(2), width=100, free=_at(3), n_pages=50, n_free=_at(4), slots=_at(5),
             room=64, starts=_at(6), info=_at(7)):
        return L.tl_kv_slots(lens, want, B, P, table, width, free, n_pages, n_free, slots, room, starts, info, None)
    assert call(B=0) == 1 and call(B=1025) == 1
    assert call(P=48) == 3 and call(P=8) == 3 and call(P=0) == 3
    assert call(width=0) == 1 and call(width=1 << 27) == 1
    assert call(n_pages=0) == 1 and call(n_pages=1 << 27) == 1
    assert call(room=-1) == 1
    for name in ("lens", "want", "table", "free", "n_free", "slots", "starts", "info"):
        assert call(**{name: None}) == 1
        assert call(**{name: A + 2}) == 2
    assert call(want=_at(0)) == 1                       # lengths over the wanted lengths
    assert call(slots=_at(5), starts=_at(5) + 4 * 63) == 1
    assert "overlap" in L.tl_last_error_message().decode()


def test_commit_refuses(L):
    def call(c=None, k=_at(2), v=_at(3), stride=8 * 128, rows=32, src=None, slots=_at(4), n=16, **kw):
        return L.tl_kv_commit(ctypes.byref(c or _cache(**kw)), k, v, stride, rows, src, slots, n, None)
    assert call(n=-1) == 1 and call(n=(1 << 24) + 1) == 1
    assert call(n=0, k=None, v=None, slots=None) == 0   # nothing to commit: a no-op before any CUDA call
    assert call(page_tokens=48) == 3 and call(head_dim=96) == 3
    assert call(n_kv_heads=0) == 1 and call(n_kv_heads=257) == 1
    assert call(n_pages=0) == 1 and call(n_pages=1 << 25) == 1
    assert call(pages=None) == 1 and call(scales=None) == 1
    assert call(pages=_at(0) + 8) == 2 and call(scales=_at(1) + 4) == 2
    assert call(stride=1016) == 1 and call(stride=1028) == 1
    assert call(rows=0) == 1 and call(rows=15) == 1 and call(rows=0, src=_at(5)) == 1
    assert call(k=None) == 1 and call(v=None) == 1 and call(slots=None) == 1
    assert call(k=_at(2) + 2) == 2 and call(v=_at(3) + 8) == 2 and call(slots=_at(4) + 1) == 2 and call(src=_at(5) + 2) == 2
    assert call(k=_at(0) + 4096) == 1 and call(slots=_at(1)) == 1 and call(scales=_at(0) + 64) == 1
    assert L.tl_kv_commit(None, _at(2), _at(3), 1024, 32, None, _at(4), 16, None) == 1


def test_attention_refuses(L):
    need = ctypes.c_size_t()
    assert L.tl_kv_attention_workspace(ctypes.byref(_cache()), 40, 4, 32, ctypes.byref(need)) == 0
    def call(q=_at(2), qs=40 * 128, hq=40, table=_at(3), width=200, lens=_at(4), B=4, kn=_at(5), vn=_at(6), ns=8 * 128, mask=_at(7),
             start=_at(8), R=100, rows=32, scale=0.1, out=_at(9), os=40 * 128, ws=_at(10), wb=need.value, **kw):
        return L.tl_kv_attention(q, qs, hq, ctypes.byref(_cache(**kw)), table, width, lens, B, kn, vn, ns, mask, start, R, rows,
                                 ctypes.c_float(scale), out, os, ws, wb, None)
    assert call(R=0) == 0 and call(R=-1) == 1
    assert call(start=None) == 1                        # 100 rows are not 4 x 32
    assert call(hq=39) == 1 and call(hq=0) == 1 and call(hq=8 * 17) == 3
    assert call(B=0) == 1 and call(B=1025) == 1 and call(rows=0) == 1 and call(rows=33) == 1
    assert call(width=0) == 1 and call(width=1 << 26) == 1
    assert call(head_dim=256) == 3 and call(page_tokens=256) == 3
    assert call(scale=math.nan) == 1 and call(scale=math.inf) == 1
    assert call(kn=None) == 1 and call(vn=None) == 1
    for name in ("q", "table", "lens", "out", "ws"):
        assert call(**{name: None}) == 1
    assert call(q=_at(2) + 8) == 2 and call(kn=_at(5) + 2) == 2 and call(vn=_at(6) + 4) == 2 and call(out=_at(9) + 2) == 2
    assert call(ws=_at(10) + 16) == 2 and call(lens=_at(4) + 2) == 2 and call(mask=_at(7) + 1) == 2
    assert call(qs=5112) == 1 and call(qs=5124) == 1 and call(os=1024) == 1 and call(ns=1000) == 1
    assert call(wb=need.value - 1) == 1
    assert call(out=_at(2) + 5120 * 2) == 1 and call(out=_at(0)) == 1 and call(out=_at(5)) == 1 and call(out=_at(6)) == 1
    assert call(ws=_at(3)) == 1 and call(ws=_at(9)) == 1
    assert "overlap" in L.tl_last_error_message().decode()


def test_attention_refuses_more_work_than_it_counts_in_32_bits(L):
    # 1024 requests x 8 KV heads x 7 tiles of 80 rows, each of 16 + 9 a tile of 128 tokens, at most 4e9 in all: 7748 tiles
    for tiles, code in ((7748, 1), (7749, 3)):
        assert L.tl_kv_attention(_at(2), 128 * 128, 128, ctypes.byref(_cache()), _at(3), 2 * tiles, _at(4), 1024, None, None, 0, None,
                                 _at(8), 100, 32, ctypes.c_float(0.1), _at(9), 128 * 128, _at(10), 16, None) == code
    assert "too large for one call" in L.tl_last_error_message().decode()


def test_workspace_grows_with_its_sizes(L):
    def need(hq, B, rows, **kw):
        n = ctypes.c_size_t()
        assert L.tl_kv_attention_workspace(ctypes.byref(_cache(**kw)), hq, B, rows, ctypes.byref(n)) == 0
        return n.value
    base = need(40, 1, 1)
    assert base > 0 and need(40, 2, 1) > base and need(40, 1, 32) > base and need(40, 1, 1, head_dim=64) < base
    # room for every row's part once a request and once a CTA
    assert need(40, 64, 32) >= 64 * 32 * 40 * (128 + 2) * 4
    n = ctypes.c_size_t()
    assert L.tl_kv_attention_workspace(ctypes.byref(_cache()), 12, 1, 1, ctypes.byref(n)) == 1
    assert L.tl_kv_attention_workspace(ctypes.byref(_cache()), 40, 1, 1, None) == 1


def test_binding_refuses_what_the_library_cannot_see():
    import nvfp4_weight_gemm_b200 as tl
    with pytest.raises(ValueError):
        tl.KvCache(torch.zeros((4, 2, 2, 1024), dtype=torch.int8), torch.ones((4, 2, 2)), 16)
    with pytest.raises(ValueError):
        tl.KvCache(torch.zeros((4, 2, 2, 1000), dtype=torch.uint8), torch.ones((4, 2, 2)), 16)
    with pytest.raises(ValueError):
        tl.KvCache(torch.zeros((4, 2, 2, 1024), dtype=torch.uint8), torch.ones((4, 2)), 16)
    c = tl.KvCache(torch.zeros((4, 2, 2, 1024), dtype=torch.uint8), torch.ones((4, 2, 2)), 16)
    assert (c.n_pages, c.kv_heads, c.head_dim) == (4, 2, 64)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        tl.kv_commit(c, x.float(), x, i)
    with pytest.raises(ValueError):
        tl.kv_commit(c, x, x, i.long())
    with pytest.raises(ValueError):
        tl.kv_commit(c, x, x[:, :, ::2], i)
    with pytest.raises(ValueError):
        tl.kv_commit(c, x, x, i)                        # host tensors
    with pytest.raises(ValueError):
        tl.kv_attention(x, c, i[None], i[:1], k_new=x)  # keys without values
    with pytest.raises(ValueError):
        tl.kv_attention(x, c, i[None], i[:1], row_start=i[:2])   # no max_rows
    with pytest.raises(ValueError):
        tl.kv_slots(i, i, i[:, None], i, i[:1], 16, i, i, i)     # starts and info too short


# ---------------------------------------------------------------- the plain statements

def test_e4m3_bytes_against_the_table_and_ties():
    t = kv.TABLE
    for b in range(256):
        if not math.isnan(t[b]):
            assert int(kv.e4m3_bytes(np.array([t[b]]))[0]) == b
    # halfway values go to the even byte; beyond the largest value it stays; NaN
    mids = (t[:126] + t[1:127]) / 2
    got = kv.e4m3_bytes(mids)
    assert all(int(g) in (i, i + 1) and int(g) % 2 == 0 for i, g in enumerate(got))
    assert [int(b) for b in kv.e4m3_bytes(np.array([1e9, -1e9, np.nan, 2.0 ** -10, 2.0 ** -11]))] == [0x7E, 0xFE, 0x7F, 0, 0]


def test_places_cover_a_page_once():
    for D in (64, 128):
        for P in (16, 32, 64, 128):
            c = np.arange(D)
            for place in (lambda t: kv.place_k(t, c, P), lambda t: kv.place_v(t, c, D)):
                seen = np.concatenate([place(t) for t in range(P)])
                assert np.array_equal(np.sort(seen), np.arange(P * D))


def test_slots_hand_worked():
    # pages of 16: request 0 grows 15 -> 18 (one page), request 1 ends (two pages back), request 2 starts with 1 token
    table = np.array([[4, -1, -1], [7, 2, -1], [-1, -1, -1]])
    free = np.array([5, 6, 0, 0, 0, 0, 0, 0])
    lens, table2, free2, n, slots, starts, info = kv.slots([15, 20, 0], [18, 0, 1], 16, table, free, 2, 6)
    # returned: page 7, then 2, the first at the top: stack 5 6 2 7; taken: 7 for request 0, 2 for request 2
    assert lens == [18, 0, 1] and n == 2 and info == [0, 0, 0, 0]
    assert table2.tolist() == [[4, 7, -1], [-1, -1, -1], [2, -1, -1]]
    assert slots.tolist() == [4 * 16 + 15, 7 * 16, 7 * 16 + 1, 2 * 16, -1, -1] and starts == [0, 3, 3, 4]
    # and back again
    back = kv.slots(lens, [15, 20, 0], 16, table2, free2, n, 20)
    assert back[0] == [15, 20, 0] and back[3] == 2 and sorted(back[1][back[1] >= 0].tolist()) == [2, 4, 7]


def test_slots_refusals_hand_worked():
    table, free = np.array([[0, -1], [1, -1]]), np.array([2, 9, 9, 9])
    lens, t, f, n, s, st, info = kv.slots([16, 16], [32, 32], 16, table, free, 1, 99)
    assert lens == [16, 16] and n == 1 and info == [1, 1, 0, 0] and s.max() == -1 and st == [0, 0, 0]
    lens, t, f, n, s, st, info = kv.slots([16, 16], [18, 8], 16, table, free, 1, 1)
    assert lens == [16, 8] and n == 1 and info == [2, 0, 1, 0] and t.tolist() == table.tolist()
    lens, t, f, n, s, st, info = kv.slots([16, 16], [40, 18], 16, table, free, 1, 9)
    assert lens == [16, 18] and info == [4, 0, 0, 1] and s[:2].tolist() == [32, 33] and st == [0, 0, 2]
    lens, t, f, n, s, st, info = kv.slots([16, 16], [0, 0], 16, table, free, 3, 9)
    assert lens == [16, 16] and info == [8, 0, 0, 0] and n == 3


def test_commit_hand_worked():
    P, D = 16, 64
    pages, scales = np.full((2, 1, 2, P * D), 0x7F, np.uint8), np.ones((2, 1, 2), np.float32)
    k = np.zeros((2, 1, D)); v = np.zeros((2, 1, D))
    k[0, 0, 0], k[1, 0, 17] = 448.0, -1.0        # largest 448: scale 1
    v[0, 0, 1], v[1, 0, 1] = 449.0, np.inf       # largest finite 449: scale 2; the infinity becomes NaN
    p, s = kv.commit(pages, scales, P, k, v, [16, 17])
    assert s[1, 0].tolist() == [1.0, 2.0] and s[0, 0].tolist() == [1.0, 1.0]
    assert p[1, 0, 0, 0] == 0x7E and p[1, 0, 0, 1 * P * 16 + 1 * 16 + 1] == 0xB8
    assert kv.TABLE[p[1, 0, 1, 16]] == 224.0 and p[1, 0, 1, 17] == 0x7F      # 224.5 to 224 (steps of 16), NaN
    assert (p[0] == 0x7F).all() and p[1, 0, 0, 2 * 16] == 0x7F               # nothing else is touched
    # a third token 4 times larger: the page moves to scale 4, -1 becomes -0.25
    k3 = np.zeros((1, 1, D)); k3[0, 0, 5] = 1792.0
    p2, s2 = kv.commit(p, s, P, k3, np.zeros((1, 1, D)), [18])
    assert s2[1, 0].tolist() == [4.0, 2.0] and kv.TABLE[p2[1, 0, 0, 0]] == 112.0
    assert kv.TABLE[p2[1, 0, 0, 1 * P * 16 + 16 + 1]] == -0.25 and p2[1, 0, 1, 17] == 0x7F


def test_attention_hand_worked():
    P, D = 16, 64
    pages, scales = np.zeros((1, 1, 2, P * D), np.uint8), np.full((1, 1, 2), 1.0, np.float32)
    one = int(kv.e4m3_bytes(np.array([1.0]))[0])
    pages[0, 0, 0, kv.place_k(0, np.array([0]), P)] = one    # token 0: k = e_0
    pages[0, 0, 1, kv.place_v(0, np.array([3]), D)] = one    # token 0: v = e_3
    q = np.zeros((2, 1, D)); q[0, 0, 0] = math.log(3.0)
    kn = np.zeros((2, 1, D)); vn = np.zeros((2, 1, D)); vn[0, 0, 5] = 2.0; vn[1] = np.nan
    out, _, _, _ = kv.attention(q, pages, scales, P, np.array([[0]]), [1], kn, vn, [1, 0], [0, 2], 1.0)
    # row 0: token 0 with weight 3, itself with weight 1; row 1 sees token 0 alone
    assert np.allclose(out[0, 0, [3, 5]], [0.75, 0.5]) and np.allclose(out[1, 0, 3], 1.0) and np.isfinite(out).all()
    out, _, _, _ = kv.attention(q, pages, scales, P, np.array([[0]]), [0], kn, vn, [1, 0], [0, 2], 1.0)
    assert out[0, 0, 5] == 2.0 and not out[1].any()          # nothing to see: zeros
