"""The 8-bit paged KV cache on the GPU at the edges of what its interface allows, against the plain statements in oracle/kv.py
(bars: test_gpu_kv.py)."""

import numpy as np
import pytest
import torch

from oracle import kv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import nvfp4_weight_gemm_b200 as tl  # noqa: E402
from test_gpu_kv import Case  # noqa: E402

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

def test_slots_of_a_table_with_more_than_2_to_32_entries():
    # 1,024 requests x (2^22 + 1) pages: the sums of pages asked for, and of pages held, can pass 2^32
    B, P, width = 1024, 16, 2 ** 22 + 1
    table = torch.empty((B, width), dtype=torch.int32, device=DEV)
    room = 200

    def call(lens, want, head, free, n_free):
        table[:, :8] = _i32(head)
        df, dl, dn = _i32(free), _i32(lens), _i32([n_free])
        s, st, info = (torch.full((n,), 123456, dtype=torch.int32, device=DEV) for n in (room, B + 1, 4))
        tl.kv_slots(dl, _i32(want), table, df, dn, P, s, st, info)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in (dl, table[:, :8], df, dn, s, st, info)]

    free = np.arange(64) + 7
    head = np.full((B, 8), -1)
    full = width * P
    # all ask for every page their row of the table has room for: nothing moves
    got = call([0] * B, [full] * B, head, free, 5)
    assert got[6].tolist() == [3, 2 ** 31 - 1, 2 ** 31 - 1, 0]
    assert not got[0].any() and (got[1] == -1).all() and np.array_equal(got[2], free) and got[3][0] == 5
    assert (got[4] == -1).all() and not got[5].any()
    # all claim to hold such lengths and end, so that 2^32 + 5 pages would be returned to a stack for 64: nothing moves
    lens = [full if b < 5 else full - P for b in range(B)]
    got = call(lens, [0] * B, head, free, 5)
    assert got[6].tolist() == [8, 0, 0, 0]
    assert got[0].tolist() == lens and (got[1] == -1).all() and np.array_equal(got[2], free) and got[3][0] == 5
    # ordinary lengths: as with a narrow table
    rs = np.random.default_rng(1)
    lens, want = rs.integers(0, 3, B) * (np.arange(B) % 40 == 3) * 30, np.zeros(B, int)
    want[::90] = 9
    want[3], want[83] = lens[3] + 20, lens[83] + 7
    blocks = -(-lens // P)
    ids = np.arange(int(blocks.sum()) + 40)
    at = 0
    for b in range(B):
        head[b, : blocks[b]] = ids[at : at + blocks[b]]
        at += blocks[b]
    free = np.concatenate([ids[at:], np.full(at, 3)])
    got, ref = call(lens, want, head, free, 40), kv.slots(lens, want, P, head, free, 40, room)
    assert ref[6] == [0, 0, 0, 0] and (want < lens).any()
    for x, y in zip(got, ref):
        assert np.array_equal(np.ravel(x), np.ravel(y))


# ---------------------------------------------------------------- attention

def test_attention_on_another_stream_leaves_memory_that_the_current_one_still_uses():
    # tensors of the sizes of the output and of the workspace are freed while a copy of them is still queued on the current
    # stream: the call on the other stream, which does not wait for that copy, must not get their blocks
    c = Case(24, [300, 9], [4, 2], 4, 2, 128, 32).device()
    good = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    size = tl.kv_attention_workspace(c.cache, 4, 2, 4)
    for _ in range(3):
        shapes = [good.shape, ((size + 1) // 2,)]
        held = [torch.full(s, 7.0 + i, dtype=torch.bfloat16, device=DEV) for i, s in enumerate(shapes)]
        torch.cuda.synchronize()
        torch.cuda._sleep(30_000_000)
        copies = [t.clone() for t in held]
        del held
        y = tl.kv_attention(c.dq, c.cache, c.dtable, c.dlens, c.dkn, c.dvn, mask=c.dmask, row_start=c.dstart, max_rows=4, stream=side)
        side.synchronize()
        z = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(y, good) and torch.equal(z, good)
        for i, t in enumerate(copies):
            assert (t == 7.0 + i).all()


@pytest.mark.parametrize("n", [0, 1, 40, 300])
def test_attention_own_nodes_whose_score_is_minus_infinity(n):
    # a score of minus infinity is a weight of zero: beside cached tokens or nodes with finite scores it changes nothing, and
    # alone it leaves 0 / 0
    c = Case(27, [n], [4], 4, 2, 64, 16, masks=[0x1, 0x2, 0x6, 0xC])
    c.q[:, :, 3] = -0.1 - np.abs(c.q[:, :, 3])
    c.kn[:3, :, 3] = np.inf
    c.device()
    y = c.run().double()
    c.masks = np.array([0x0, 0x0, 0x0, 0x8])        # the nodes whose scores are finite
    if n == 0:
        assert torch.isnan(y[:3]).all()
        y[:3] = 0.0
    c.check(y)


@pytest.mark.parametrize("at", [0, 4100, 8191])
@pytest.mark.parametrize("apart", [5, 12])
def test_attention_sink_beside_a_tail_that_weighs_a_quarter(at, apart):
    # One token's score is 10 above those of 8,191 others, whose small weights add up to a quarter of the sum; the scale of V in
    # the sink's page is 2^5 or 2^12 times the others', so the weights of their bytes are 2^-19 or 2^-26 of the sink's: in f16 without
    # the shift by 2^8 they would be subnormal, or zero. In half of the channels the sink's V is zero and the tail's has one sign,
    # so that a result without the tail's V is off by all of it there; one without the tail's weights in the sum is off by a third
    # elsewhere. 296 requests share the pages, so that a block's share of the work is two whole requests and the tail stands behind
    # the sink's reference. The bar has one more term: a weight is held to half a subnormal step of f16, 2^-25, at 2^8 for the largest.
    P, n, B = 64, 8192, 296
    c = Case(28, [n], [1], 1, 1, 64, P, new=False)
    rs = c.rs
    page = int(c.table[0, at // P])
    c.scales[..., 0], c.scales[..., 1] = 2.0 ** -5, 2.0 ** (-7 - apart)
    c.scales[page, 0, 1] = 2.0 ** -7
    c.q[:] = 0.0
    c.q[0, 0, 0], c.q[0, 0, 1] = 8.0, 0.25
    v = rs.normal(0, 60, c.pages[:, 0, 1].shape).reshape(-1, P // 16, 64, 16)
    v[:, :, :32] = np.abs(v[:, :, :32]) + 20.0
    v[page] /= 2.0 ** min(apart, 8)                                   # the tail's tokens beside the sink
    k = rs.normal(0, 60, c.pages[:, 0, 0].shape).reshape(-1, 4, P, 16)
    k[:, 0, :, 0] = 0.0
    k[page, 0, at % P, 0] = 320.0                                     # s = 8 * 320 / 32 / 8 = 10
    v[page, at % P // 16, :32, at % 16], v[page, at % P // 16, 32:, at % 16] = 0.0, 3.0
    c.pages[:, 0, 0], c.pages[:, 0, 1] = (kv.e4m3_bytes(x).reshape(len(x), -1) for x in (k, v))
    c.device()
    out, weight, size, reach = c.reference()
    kc, vc = (kv.cached(c.pages, c.scales, P, 64, c.table[0], n, 0, side) for side in (0, 1))
    s = c.scale * (kc @ c.qv[0, 0])
    p = np.exp(s - s.max())
    own, vs = c.scales[c.table[0][np.arange(n) // P], 0, 1, None].astype(np.float64), float(c.scales[page, 0, 1])
    off = 2.0 ** -11 + 4 * 2.0 ** -24 * (64 * size + n) + 2.0 ** -19 + 2.0 ** -16.8 * reach
    bar = (2.0 ** -8 * np.abs(out) + weight * off[..., None])[0, 0] + 2.0 ** -33 * vs * np.abs(vc / own).sum(0) / p.sum()
    # what the tail is to the result, on the host
    assert s.argmax() == at and 0.2 < 1 - p[at] / p.sum() < 0.3
    assert np.median(p * own[:, 0]) < 2.0 ** (-14 - apart) * vs
    without_v, without_l = p[at] * vc[at] / p.sum(), p @ vc / p[at]
    assert (np.abs(without_v - out[0, 0]) > 8 * bar)[:32].all() and (np.abs(without_l - out[0, 0]) > 8 * bar).all()
    y = tl.kv_attention(c.dq.expand(B, 1, 64).contiguous(), c.cache, _i32(np.tile(c.table, (B, 1))), _i32([n] * B), scale=c.scale)
    torch.cuda.synchronize()
    assert (np.abs(y[:, 0].double().cpu().numpy() - out[0, 0]) <= bar).all()


def test_attention_sums_of_a_long_context_keep_their_bits():
    # 148 requests of 2^22 tokens (one page again and again) whose V has one sign: a block adds up a whole request. The MMA cuts off
    # each product at its accumulator's last bit, at most 2^-23 of it, and one accumulator takes 2^16 products: at most 2^-7 of W. A
    # thread adds up 2^9 weights below, each sum within 2^-24: 2^-14 with the joining of the parts.
    P, D, n, B = 128, 64, 2 ** 22, 148
    c = Case(29, [P], [1], 1, 1, D, P, new=False, extra_pages=0)
    c.scales[:] = 2.0 ** -6
    c.pages[:, :, 1] &= 0x7F
    c.device()
    out, weight, size, reach = c.reference()
    off = 2.0 ** -7 + 2.0 ** -14 + 2.0 ** -11 + 4 * 2.0 ** -24 * D * size + 2.0 ** -19 + 2.0 ** -16.8 * reach
    bar = 2.0 ** -8 * np.abs(out) + weight * off[..., None]
    y = tl.kv_attention(c.dq.expand(B, 1, D).contiguous(), c.cache, torch.full((B, n // P), int(c.table[0, 0]), dtype=torch.int32, device=DEV),
                        torch.full((B,), n, dtype=torch.int32, device=DEV), scale=c.scale)
    torch.cuda.synchronize()
    assert (np.abs(y.double().cpu().numpy() - out) <= bar).all()


@pytest.mark.parametrize("D,hq,hkv,rows,B,times", [(64, 2, 2, 1, 50, 200), (128, 10, 2, 32, 12, 160), (64, 16, 4, 3, 30, 90), (128, 4, 4, 9, 40, 70)])
def test_attention_blocks_that_join_many_parts_of_a_request(D, hq, hkv, rows, B, times):
    # contexts of `times` times the same 4,000 tokens, of which a block takes several times what one accumulator takes, beside short
    # ones; the weights are those of the 4,000 tokens. Scales of V far apart, so that the parts' references differ.
    P, n = 16, 4000
    c = Case(30 + rows, [n], [rows], hq, hkv, D, P, new=False, spread=3.0, q_size=2.0, extra_pages=0)
    c.scales[..., 0] = 2.0 ** -6
    c.device()
    out, weight, size, reach = c.reference()
    off = 2.0 ** -7 + 2.0 ** -14 + 2.0 ** -11 + 4 * 2.0 ** -24 * D * size + 2.0 ** -19 + 2.0 ** -16.8 * reach
    # the weights' own limit, as where they are far below the largest: half a subnormal step of f16, 2^-25, at 2^8 for the largest
    small = np.zeros(out.shape)
    for h in range(hkv):
        k, v = (kv.cached(c.pages, c.scales, P, D, c.table[0], n, h, side) for side in (0, 1))
        vs = c.scales[c.table[0][np.arange(n) // P], h, 1].astype(np.float64)
        for i in range(rows):
            for a in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                p = np.exp(c.scale * (k @ c.qv[i, a]) - (c.scale * (k @ c.qv[i, a])).max())
                small[i, a] = 2.0 ** -33 * (p * vs).max() * np.abs(v / vs[:, None]).sum(0) / p.sum()
    bar = 2.0 ** -8 * np.abs(out) + weight * off[..., None] + small
    few = [1 if b % 5 == 2 else times for b in range(B)]
    table = np.full((B, times * n // P), -1)
    for b in range(B):
        table[b, : few[b] * n // P] = np.tile(c.table[0, : n // P], few[b])
    args = (c.dq.repeat(B, 1, 1), c.cache, _i32(table), _i32([f * n for f in few]))
    y = tl.kv_attention(*args, scale=c.scale)
    torch.cuda.synchronize()
    got = y.double().cpu().numpy().reshape(B, rows, hq, D)
    assert (np.abs(got - out) <= bar).all()
    assert torch.equal(y, tl.kv_attention(*args, scale=c.scale))


def test_attention_nan_in_one_part_of_a_block_reaches_the_row():
    # NaN in a token of the first, of a middle and of the last of the parts that a block joins
    P, D, n, B = 128, 64, 128 * 1400, 148
    c = Case(31, [3 * P], [1], 1, 1, D, P, new=False, extra_pages=0).device()
    ids = [int(x) for x in c.table[0, :3]]
    c.cache.pages[ids[1], 0, 0, 0] = 0x7F                                     # K
    c.cache.pages[ids[2], 0, 1].view(P // 16, D, 16)[0, 5, 0] = 0x7F          # V, channel 5
    table = np.full((B, n // P), ids[0])
    at = {3: (0, 1), 9: (600, 1), 20: (1399, 1), 31: (10, 2), 40: (800, 2), 60: (1398, 2)}
    for b, (j, which) in at.items():
        table[b, j] = ids[which]
    y = tl.kv_attention(c.dq.expand(B, 1, D).contiguous(), c.cache, _i32(table), _i32([n] * B), scale=c.scale)[:, 0].float().cpu().numpy()
    for b in range(B):
        j, which = at.get(b, (0, 0))
        bad = np.isnan(y[b])
        assert bad.all() if which == 1 else bad[5] and bad.sum() == 1 if which == 2 else not bad.any()


def test_attention_of_one_request_for_seconds():
    # 2^30 - 128 tokens, 52 heads, all in one page: the longest call there is. Scores are all zero and V is one value a channel, so
    # every sum is exact.
    H, D, P, width = 52, 64, 128, 2 ** 23 - 1
    cache = tl.KvCache(torch.zeros((1, H, 2, P * D), dtype=torch.uint8, device=DEV), torch.full((1, H, 2), 0.125, device=DEV), P)
    v = cache.pages[0, :, 1].view(H, P // 16, D, 16)
    v[:, :, :, :] = 0x38                            # 1.0
    v[:, :, 3::5] = 0xC4                            # -3.0
    want = torch.full((D,), 0.125, device=DEV)
    want[3::5] = -0.375
    q = torch.randn((1, H, D), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    y = tl.kv_attention(q, cache, torch.zeros((1, width), dtype=torch.int32, device=DEV), _i32([width * P]))
    tl.check_device_error()
    assert (y.float() == want).all()
