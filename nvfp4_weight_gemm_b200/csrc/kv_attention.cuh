// kv_attention.cuh -- attention of one token or of a draft tree's rows over the 8-bit paged KV cache
// (layout: kv_cache.cuh).
//
// A verify pass checks the rows of a draft tree in one forward pass (TandemLLM docs v0.12.0, "What
// TandemLLM is", section 1.2). In its attention layers a row sees every cached token of its request and,
// of the tree, the nodes that its mask names (its ancestors and itself), whose K and V are fresh bf16 rows:
//
//     s_t = c q . (e4m3(k_t) ks)  t < len,     s_j = c q . k_new_j  for j in mask,
//     out = (sum p v) / (sum p),               p = exp(s - max s)
//
// In base 2, with w = s log2(e) + log2(vs) the log-weight of the bytes of V (vs the page's V scale), the
// sums over any part of the cached tokens are held as (m, l, O):
//
//     O = sum 2^(w - m) e4m3(v),    l = sum 2^(s log2(e) - m),    out = O / l
//
// The maximum m is taken over w, not s: a product 2^(w - m) e4m3(v) is then at most 448 however the
// pages' scales differ. Parts are joined by rescaling with 2^(m - max m).
//
// Two launches: kv_attention_kernel streams the cache and writes one (m, l, O) per part and row;
// kv_merge_kernel adds the tree and joins the parts.
//
// Work. A unit is (request, KV head, row tile): the rows of a request and KV head are its rows times the head's
// query heads, row r = i * G + g, in the fewest row tiles that hold them, evenly; the cached tokens are cut into
// tiles of 128. The tiles of all units form one list, in which a tile weighs what its rows make it cost and a unit some
// more for its beginning and end; each CTA takes an equal, contiguous share of the weight (the tiles that begin in it),
// so requests of unequal lengths and trees fill the GPU evenly. The part of unit u on CTA g goes to slot u + g: going
// along the list, each step moves to the next unit or the next CTA, so no two parts meet.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include "gemm_tc.cuh"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace tl {

constexpr int KV_TILE = 128;          // cached tokens of a tile
// Tiles of a segment at most. The MMA truncates each product against its accumulator, so that sums of values of one sign lose
// some 2^-27 of themselves a token: 0.65% over 2^20 tokens in one accumulator, 2.5% over 2^22. Over 2^16 it is 2^-11, and what
// follows is added to the part in fp32 by the softmax warps. (4 requests of 2^20 tokens with trees of 32 rows: 4.73 ms, as with one
// segment a part; with 256 tiles 4.79.)
constexpr int KV_SEG_TILES = 512;
constexpr int KV_MAX_ROWS = 32;       // rows of one request: the bits of a mask
constexpr float KV_LOG2E = 1.4426950408889634f;

struct KvAttnParams {
    const __nv_bfloat16* q;       // [R][Hq][D], rows q_stride elements apart
    const uint8_t* pages;
    const float* scales;
    const int* table;             // [B][width]
    const int* lens;              // [B]
    const __nv_bfloat16* k_new;   // [R][Hkv][D], rows new_stride apart, or null
    const __nv_bfloat16* v_new;
    const unsigned* mask;         // [R], or null: row i sees rows 0..i
    const int* row_start;         // [B + 1], or null: max_rows rows each
    __nv_bfloat16* out;           // [R][Hq][D], rows out_stride apart
    float* part_o;                // [slots][NT][D]
    float2* part_ml;              // [slots][NT]
    int* err;
    long long q_stride, new_stride, out_stride;
    float scale;                  // c * log2(e)
    int B, width, n_pages, page_log2, heads, group, R, max_rows, ctas, row_tiles, nt;   // row tiles of the largest request
};

// Request b: its rows (0 where the offsets are invalid) and the cached tokens they attend to (0 without rows). Its loads
// do not wait for one another.
struct KvRequest {
    int first, rows, len;
    bool bad;
    __device__ __forceinline__ KvRequest(const KvAttnParams& p, int b) {
        const int held = p.lens[b];
        first = b * p.max_rows;
        rows = p.max_rows;
        bad = false;
        if (p.row_start) {
            const int r0 = p.row_start[b], r1 = p.row_start[b + 1];
            bad = r0 < 0 || r1 < r0 || r1 - r0 > p.max_rows || r1 > p.R;
            first = r0;
            rows = bad ? 0 : r1 - r0;
        }
        const long long room = (long long)p.width << p.page_log2;
        len = (rows == 0 || held < 0) ? 0 : (int)(held < room ? held : room);
    }
};

__device__ __forceinline__ int kv_tiles(int len) { return (int)(((unsigned)len + KV_TILE - 1) / KV_TILE); }

// Weights, in about 0.18 us: a tile's share that does not depend on its rows, and a unit's beginning and end. (Of 6, 9,
// 12, 16 and 22 for the latter: 24 requests of about 3k tokens in 34.8, 33.2, 31.0, 31.2 and 32.7 us,
// a mix of long and short ones in 74, 69, 62, 51 and 52.)
constexpr int KV_W_TILE = 4, KV_W_UNIT = 16;

// How the rows of a request are cut for row tiles of at most `most` rows, and what its units weigh. (The host keeps the
// weight of a whole call below 2^32.)
struct KvShape {
    int row_tiles, nt;      // row tiles, and rows of each (a multiple of 16; the last may hold fewer)
    unsigned tile_w, unit_w;
    __device__ __forceinline__ KvShape() {}
    __device__ __forceinline__ KvShape(int rows, int tiles, int most) {
        row_tiles = (rows + most - 1) / most;
        nt = row_tiles <= 1 ? (rows + 15) / 16 * 16 : ((rows + row_tiles - 1) / row_tiles + 15) / 16 * 16;
        tile_w = KV_W_TILE + nt / 16;
        unit_w = KV_W_UNIT + tiles * tile_w;
    }
    // Of a unit that begins at weight 0, the first tile that begins at `x` or behind it.
    __device__ __forceinline__ int tile_from(unsigned x, int tiles) const {
        if (x == 0) return 0;
        if (x >= unit_w) return tiles;
        return x <= KV_W_UNIT + tile_w ? 1 : (int)((x - KV_W_UNIT + tile_w - 1) / tile_w);
    }
};

// The shares of the CTAs: of `total`, CTA g has start(g) .. start(g + 1), equal to within one.
struct KvShares {
    unsigned q, r;
    __device__ __forceinline__ KvShares(unsigned total, int ctas) : q(total / ctas), r(total % ctas) {}
    __device__ __forceinline__ unsigned start(int g) const { return (unsigned)g * q + min((unsigned)g, r); }
    __device__ __forceinline__ int owner(unsigned x) const { return x < r * (q + 1) ? (int)(x / (q + 1)) : (int)(r + (x - r * (q + 1)) / q); }
};

// One step of a walk along a range of the tile list: tiles k0..k1 of row tile rt of (b, head), KV_SEG_TILES of them at most.
struct __align__(16) KvSeg {
    int b, head, rt, k0, k1, nt, n_rows;
    short valid;    // tokens of its last tile (128 unless it is the unit's last)
    short more;     // to be added to the unit's part, which the segments in front of it began
};

struct KvWalk {
    const unsigned* pre;     // [B + 1] weight of the requests in front
    const int* len;          // [B]
    const uint8_t* rows;     // [B]
    int B, heads, group, most;
    unsigned end;
    int b, head, rt, k;      // next: tile k of unit (b, head, rt)
    int tiles;               // of request b
    unsigned at;             // where its unit begins
    bool more;               // some of its unit's tiles went out in the segment in front
    KvShape s;
    __device__ __forceinline__ void look() {
        tiles = kv_tiles(len[b]);
        s = KvShape((int)rows[b] * group, tiles, most);
    }
    __device__ __forceinline__ KvWalk(const KvAttnParams& p, const unsigned* pre_, const int* len_, const uint8_t* rows_, unsigned begin,
                                      unsigned end_, int most_)
        : pre(pre_), len(len_), rows(rows_), B(p.B), heads(p.heads), group(p.group), most(most_), end(end_), b(p.B), head(0), rt(0), k(0),
          tiles(0), at(0), more(false) {
        if (begin >= end) return;
        int lo = 0, hi = B;
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= begin) lo = mid; else hi = mid;
        }
        b = lo;
        look();
        const unsigned in = begin - pre[b], j = in / s.unit_w;
        head = (int)(j / s.row_tiles);
        rt = (int)(j - head * s.row_tiles);
        at = pre[b] + j * s.unit_w;
        k = s.tile_from(begin - at, tiles);
        if (k == tiles) step();
    }
    // on to the next unit
    __device__ __forceinline__ void step() {
        k = 0;
        at += s.unit_w;
        if (++rt < s.row_tiles) return;
        rt = 0;
        if (++head < heads) return;
        head = 0;
        ++b;
#pragma unroll 1
        while (b < B && pre[b + 1] == pre[b]) ++b;
        if (b < B) look();
    }
    __device__ __forceinline__ bool next(KvSeg& g) {
        if (b >= B || at >= end) return false;
        const int k1 = min(s.tile_from(end - at, tiles), k + KV_SEG_TILES);
        if (k1 <= k) return false;
        g.b = b;
        g.head = head;
        g.rt = rt;
        g.k0 = k;
        g.k1 = k1;
        g.nt = s.nt;
        g.n_rows = min((int)rows[b] * group - rt * s.nt, s.nt);
        g.valid = (short)(k1 == tiles ? ((len[b] - 1) & (KV_TILE - 1)) + 1 : KV_TILE);
        g.more = more;
        k = k1;
        more = k != tiles;
        if (!more) step();
        return true;
    }
};

// ---------------------------------------------------------------- the streaming kernel
//
// Both products run on the tensor cores with the cache as operand A and the rows as operand B, so that
// few rows cost little (an MMA is 128 tokens or channels times NT rows, NT a multiple of 16):
//
//     S^T [token][row]   = K  [token][channel] . Q^T      E4M3: A = the cache's bytes, moved to tensor memory as they are
//     O^T [channel][row] = V^T [channel][token] . P^T     f16:  A = V in tensor memory,  B = P in shared memory
//
// K is never converted: Q is. (Operand A in shared memory would have to have K's 128 tokens side by side: a tile's pages in
// pieces of 16 channels, and bulk copies that small, 18 a tile, were 23% slower for one row than moving K from whole pages.)
// Each row of Q is scaled by a power of two that brings its largest magnitude into (224, 448] and written as the sum of two E4M3 terms, the second holding what the first left over. A bf16 value
// has 8 significant bits and a term holds 4, so the sum is exact for elements down to 2^-10 of the largest; the
// others are within 2^-10 in that scale, 2^-17.8 of the row's largest. Both terms multiply the same K into one fp32
// accumulator (products of E4M3 are exact in it).
// P would lose too much in E4M3: it keeps f16 (11 bits against the output's 8), after a scaling that leaves 2^-22 of
// the largest weight normal, and V becomes f16 on the way (every E4M3 value is an f16 value). The sums l take
// p before that rounding. S, O and l are fp32.
//
// The reference m of a row's weights is kept as long as no log-weight of a tile passes it by more than
// KV_SLACK; only then (and in a segment's first tile) are the tile's maxima found across lanes, and O and
// l rescaled. So most tiles need one comparison a score and one vote.
//
// Roles (one CTA of 16 warps per SM; registers are moved between the warpgroups, KvCfg):
//   * warp 0        walks the CTA's share of the list and publishes its segments (a unit's tiles, KvSeg) in a ring that the
//                   other roles follow (the walk in every role was code of 8 KB each, and instruction fetches a bound);
//                   producer: a page's K and V of the head are one contiguous piece, brought in by one bulk copy;
//                   tiles of 128 tokens, a ring of stages. Scales follow by cp.async.
//   * warp 1        issues the MMAs of S^T, warp 2 those of O^T (each waits for other roles).
//   * warp 3        the rows: Q of the next segment to one of two buffers in shared memory. The first segment's Q is
//                   brought in by the softmax warps, which have nothing to do yet.
//   * warps 4..7    movers: K (lane = token), then V, converted (lane = channel), 16 bytes of a lane at a time.
//   * warps 8..15   softmax: two groups of four warps, half of the blocks of 8 rows each, lane = token; blocks without
//                   rows are passed over. A group also reads its rows of O (lane = channel) when a segment ends and writes
//                   the part.
// Bound: for a few rows the cache's bytes (64 requests of up to 8k tokens, 8 KV heads of 128, one row each: 107 us, 80% of
// what a copy reaches). A tile of 128 tokens and 128 channels takes 0.82 us with 16 rows, 1.17 with 48 and 1.72 with 80, of
// which memory needs 0.74. With many rows it is the softmax's: its warps go through one step after another, and no unit is busy
// half the time. In cycles of a tile of 80 rows (of 40), by time stamps in the kernel, two groups' average: 280 (170) of wait for
// the scores, 470 (340) of their load, 510 (300) of scale and maximum, 230 (150) of vote, 185 (105) until the weights, 720 (550)
// of exponentials and weights, 160 (95) of fence and arrival, 250 (280) until the next wait: 2,800 (2,000) of the 2,910 (2,040)
// that such a tile takes with the stamps. Rows as operand A, padded to 128 and a row a thread (no votes, no exchange across
// lanes), took 1.81 us; the groups on alternate tiles, four groups on two tiles, or three groups on thirds of the rows 1.99 and more.
// Every mbarrier wait is bounded; after one has run out the others return at once, every role runs to its end
// (so no named barrier is left waiting), and the status word is set.

constexpr float KV_SLACK = 7.0f;       // P is at most 2^(KV_SLACK + KV_P_SHIFT), f16's largest value is 2^16 - 32
constexpr float KV_P_SHIFT = 8.0f;

template <int D, int NT>
struct KvCfg {
    static constexpr int WARPS = 16, THREADS = 32 * WARPS;
    // registers a thread: 128 at launch (512 over the four warpgroups), then dealt out by need
    static constexpr int REGS_CONTROL = 96, REGS_MOVE = 96, REGS_SOFTMAX = 160;
    static_assert(REGS_CONTROL + REGS_MOVE + 2 * REGS_SOFTMAX <= 512, "registers of the launch");
    static constexpr int NH = NT / 2;                          // rows of a softmax group
    static constexpr int NB = NT / 16;                         // blocks of 8 rows of a softmax group at most
    static constexpr int STAGE_BYTES = 2 * KV_TILE * D;
    static constexpr int QSTEPS = 2 * D / 32;                  // MMAs of S^T: 32 channels each, both terms
    static constexpr int Q_BYTES = NT * D * 2;                 // slabs of [NT] 128-byte rows, swizzled: the first terms, the second
    static constexpr int P_BYTES = NT * KV_TILE * 2;
    // tiles in flight between movers, MMAs and softmax: what tensor memory holds
    static constexpr int PER_TILE = D / 4 + KV_TILE / 2 + NT;
    static constexpr int BUFS = (4 * PER_TILE + NT <= 512) ? 4 : (3 * PER_TILE + NT <= 512) ? 3 : 2;
    // S^T runs up to BUFS tiles (so perhaps BUFS segments) ahead of the softmax, and Q two segments ahead of S^T
    static constexpr int ROWF_RING = 8;
    // page scales: the producer is up to STAGES tiles ahead of S^T, and that BUFS ahead of the softmax
    static constexpr int SCALE_RING = 16;
    static constexpr int SEG_RING = 16;
    static constexpr int SMALL_BYTES = (KV_MAX_BATCH + 4) * 4 + 5 * KV_MAX_BATCH   // weight in front, tokens, rows
                                     + SCALE_RING * 8 * 8                 // page scales
                                     + ROWF_RING * NT * 4                 // row factors
                                     + 2 * NT * 4                         // -m, rescaling factors
                                     + 2 * 4 * NH * 4                     // a group's four warps' maxima or sums
                                     + SEG_RING * 32                      // segments
                                     + 768;                               // barriers
    static constexpr int FIXED = 2 * Q_BYTES + BUFS * P_BYTES + SMALL_BYTES + 1024 /*align*/;
    static constexpr int FIT = (232448 - FIXED) / STAGE_BYTES;
    static constexpr int STAGES = FIT < 8 ? FIT : 8;
    static_assert(ROWF_RING >= BUFS + 3 && SCALE_RING >= STAGES + BUFS, "rings");
    static constexpr int SMEM_BYTES = FIXED + STAGES * STAGE_BYTES;
    // without the rows (bits 17 up: rows / 8)
    static constexpr uint32_t IDESC_QK = (1u << 4) /*fp32*/ | ((128u >> 4) << 24);         // E4M3 x E4M3
    static constexpr uint32_t IDESC_PV = idesc_f16(0u /*f16*/, 128u, 0u) | (1u << 16);     // B: rows fastest
    // P lies token by token, rows fastest (a softmax thread holds one token's rows): atoms of 8 tokens x 16 rows,
    // 32 bytes a token, 32-byte swizzle; the atoms of 8 tokens side by side, then the next 8 tokens
    static constexpr int P_ATOM = 256, P_STEP = (NT / 16) * P_ATOM;
    // tensor memory columns: K tiles, V tiles, S^T, one O^T
    static constexpr int K_COL = 0, K_COLS = D / 4;
    static constexpr int V_COL = BUFS * K_COLS, V_COLS = KV_TILE / 2;
    static constexpr int S_COL = V_COL + BUFS * V_COLS;
    static constexpr int O_COL = S_COL + BUFS * NT;
    static constexpr int TMEM_COLS = 512;
    static_assert(O_COL + NT <= TMEM_COLS, "tensor memory budget");
    static_assert(NT % 16 == 0 && NH % 8 == 0, "MMA and store shapes");
    static_assert(STAGES >= 3 && STAGES <= 8, "shared memory budget");
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                   "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}

// Two fp32 values in one register pair: Blackwell's packed fp32 arithmetic does both in one instruction.
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float kv_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float kv_lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float kv_warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void kv_group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool kv_group_any(int id, bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(id), "r"((uint32_t)mine) : "memory");
    return r != 0;
}
__device__ __forceinline__ void sts_128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// Shared-memory matrix descriptor of an operand whose rows are fastest, 32-byte swizzle: `mn` bytes between
// groups of 16 rows, `k` bytes between groups of 8 along the summed axis.
__device__ __forceinline__ uint64_t smem_desc_mn_sw32(uint32_t saddr, uint32_t mn, uint32_t k) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(mn >> 4) << 16) | ((uint64_t)(k >> 4) << 32) | ((uint64_t)1u << 46) |
           ((uint64_t)6u << 61);
}
// Two f16 values (a in the low half).
__device__ __forceinline__ uint32_t kv_pack_f16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Sixteen E4M3 bytes -> eight f16x2 words.
__device__ __forceinline__ void kv_decode16(uint4 q, uint32_t* out) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(out[2 * j]), "=r"(out[2 * j + 1]) : "r"(w[j]));
}

// Bounded wait that also gives up when another role has aborted the CTA. A poll sleeps in hardware for some 4 microseconds,
// so the limit is about a second: no wait lasts longer than a segment, 0.9 ms.
__device__ __forceinline__ bool kv_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
    for (uint32_t i = 0; i < (TL_WAIT_LIMIT >> 4); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 15u && *abort_flag) return false;
    }
    return false;
}

// The first n bytes of a word (none for n <= 0), zeros behind them.
__device__ __forceinline__ uint32_t kv_first_bytes(uint32_t w, int n) {
    return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u);
}

// D[tmem] (+)= A[tmem] * B[smem], fp32 accumulate, by the one lane whose `on` is set, of a converged warp: f16 operands, and
// E4M3 ones. (The predicate in the instruction: 16 to 42 cycles an MMA of 16 to 80 rows back to back; in a branch of that lane
// 25 to 42, and 127 where the compiler did not know the warp's index as uniform.)
__device__ __forceinline__ void mma_f16_if(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on) : "memory");
}
__device__ __forceinline__ void mma_f8_if(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on) : "memory");
}
// Arrive once on `bar` when every MMA issued so far by that lane has completed.
__device__ __forceinline__ void mma_commit_if(uint32_t on, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"(on) : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

// Eight values a lane -> over the warp's lanes, the combination of value 4 * (lane & 1) + (lane & 2) + (lane >> 2 & 1) in
// every lane: three exchanges that halve the values, two that do not (nine shuffles against forty one by one).
template <typename Op>
__device__ __forceinline__ float kv_across8(float (&v)[8], int lane, Op op) {
#pragma unroll
    for (int w = 4, d = 1; w; w >>= 1, d <<= 1) {
#pragma unroll
        for (int j = 0; j < w; ++j) {
            const bool hi = lane & d;
            v[j] = op(hi ? v[j + w] : v[j], __shfl_xor_sync(0xFFFFFFFFu, hi ? v[j] : v[j + w], d));
        }
    }
    v[0] = op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 8));
    return op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 16));
}

// Bounded wait that does not mind an abort: for work in flight that has to end before the CTA may.
__device__ __forceinline__ bool kv_drain(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
    for (uint32_t i = 0; i < (TL_WAIT_LIMIT >> 4); ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}

__device__ __forceinline__ uint64_t kv_uniform64(uint64_t v) {
    return ((uint64_t)__shfl_sync(0xFFFFFFFFu, (uint32_t)(v >> 32), 0) << 32) | (uint64_t)__shfl_sync(0xFFFFFFFFu, (uint32_t)v, 0);
}

// Ring position of a tile: buffer and parity of its use.
template <int N>
struct KvRing {
    uint32_t i = 0, par = 0;
    __device__ __forceinline__ void step() {
        if (++i == N) { i = 0; par ^= 1u; }
    }
};

// The Q rows of a segment's row tile into shared memory as two E4M3 terms, each row scaled by a power of two; rowf[n]
// undoes the scale. D = 128: a slab of 128-byte rows for each term; D = 64: one slab, both terms side by side (128-byte
// swizzle). A row with a non-finite element gets a NaN factor. By `threads` threads (a multiple of 32): the bf16 rows
// are first copied, all at once, to where their terms will lie (a row's 2 D bytes are as many as its terms'); then
// the lanes of a row read all of it and write it back as terms.
template <int D, int NT>
__device__ __forceinline__ void kv_load_rows(const KvAttnParams& p, const KvSeg& sg, int t, int threads, uint8_t* q_sm, float* rowf) {
    constexpr int LPR = D / 8;                 // lanes of a row, 8 channels each
    const int first = p.row_start ? __ldg(p.row_start + sg.b) : sg.b * p.max_rows;
    const int c = t % LPR, step = threads / LPR;
    const unsigned inv_group = (65536u + p.group - 1) / p.group;     // r / group = r * inv_group >> 16 for r < 512, group <= 16
    const __nv_bfloat16* const q0 = p.q + (size_t)first * p.q_stride + (size_t)(sg.head * p.group) * D + 8 * c;
    const int r0 = sg.rt * sg.nt, nt = sg.nt;
    // 16-byte unit of the row that this lane copies; for D = 128 the second half of a row lies in the second slab
    const uint32_t unit = c & 7, slab = (uint32_t)(c >> 3) * (NT * 128);
#pragma unroll 1
    for (int n = t / LPR; n < nt; n += step) {
        const unsigned r = r0 + n, node = r * inv_group >> 16;
        const bool there = n < sg.n_rows;
        const __nv_bfloat16* const from = there ? q0 + (size_t)node * p.q_stride + (size_t)(r - node * p.group) * D : p.q;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(q_sm + slab + n * 128 + (unit << 4))), "l"(from),
                     "r"(there ? 16 : 0) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    const int c2 = (D == 128) ? c : c + 8;
    const uint32_t slab2 = (D == 128) ? NT * 128 : 0;
    // nt is a multiple of 16 and a warp's rows are a power of two up to 8: whole warps leave the loop together
#pragma unroll 1
    for (int n = t / LPR; n < nt; n += step) {
        const uint4 q = *reinterpret_cast<const uint4*>(q_sm + slab + n * 128 + (unit << 4));    // this lane's own copy
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) m = __vmaxu2(m, w[v] & 0x7FFF7FFFu);
        unsigned top = max(m & 0xFFFFu, m >> 16);
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        // the smallest e with top <= 448 * 2^e: the significand's 7 bits behind the point against 1.75
        const int e = max((int)(top >> 7) - 127, -100) - 8 + ((top & 0x7Fu) > 0x60u);
        const float f = kv_pow2(-e);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float x = __int_as_float((int)(w[v] << 16)) * f, y = __int_as_float((int)(w[v] & 0xFFFF0000u)) * f;
            const uint32_t a = kv_e4m3x2(x, y), h = kv_f16x2(a);
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h));
            const uint32_t b = kv_e4m3x2(x - back.x, y - back.y);
            hi[v >> 1] = (v & 1) ? (hi[v >> 1] | (a << 16)) : a;
            lo[v >> 1] = (v & 1) ? (lo[v >> 1] | (b << 16)) : b;
        }
        // the shuffles above are the point where all lanes of the row hold its elements
        uint8_t* const row = q_sm + n * 128;
        *reinterpret_cast<uint2*>(row + (((c >> 1) ^ (n & 7)) << 4) + (c & 1) * 8) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(row + slab2 + (((c2 >> 1) ^ (n & 7)) << 4) + (c & 1) * 8) = make_uint2(lo[0], lo[1]);
        if (c == 0) rowf[n] = top < 0x7F80u ? p.scale * kv_pow2(e) : __int_as_float(0x7FC00000);
    }
    fence_proxy_async_smem();
}

template <int D, int NT>
__global__ void __launch_bounds__(KvCfg<D, NT>::THREADS, 1) kv_attention_kernel(const __grid_constant__ KvAttnParams p) {
    using C = KvCfg<D, NT>;
    constexpr int NH = C::NH;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int BUFS = C::BUFS;
    uint8_t* const q_sm = smem;
    uint8_t* const p_sm = q_sm + 2 * C::Q_BYTES;
    uint8_t* const stages = p_sm + BUFS * C::P_BYTES;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(stages + C::STAGES * C::STAGE_BYTES);
    uint64_t* const kvfull = bars;               // [8] a stage's bytes and scales landed
    uint64_t* const kvempty = kvfull + 8;        // [8] read by the movers
    uint64_t* const kready = kvempty + 8;        // [4] K tile in tensor memory
    uint64_t* const qkdone = kready + 4;         // [4] S^T complete (and the K tile free)
    uint64_t* const vready = qkdone + 4;         // [4] V tile in tensor memory
    uint64_t* const pready = vready + 4;         // [4] P in shared memory, O rescaled if need be
    uint64_t* const pvdone = pready + 4;         // [4] O^T has the tile (and the V tile and P are free)
    uint64_t* const qready = pvdone + 4;         // [2] Q of a segment in shared memory
    uint64_t* const qfree = qready + 2;          // [2] its last S^T is complete
    uint64_t* const ofull = qfree + 2;           // [1] a segment's O^T is complete
    uint64_t* const oempty = ofull + 1;          // [1] read by the softmax warps
    uint64_t* const segfull = oempty + 1;        // [SEG_RING] a segment is published
    uint64_t* const segempty = segfull + C::SEG_RING;   // [SEG_RING] the softmax warps, the last to follow, are done with it
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(segempty + C::SEG_RING);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float2* const page_scale = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(bars) + 768);   // [SCALE_RING][8] (K, V)
    KvSeg* const segs = reinterpret_cast<KvSeg*>(page_scale + C::SCALE_RING * 8);            // [SEG_RING]
    float* const rowf = reinterpret_cast<float*>(segs + C::SEG_RING);            // [ROWF_RING][NT]: score = S * rowf * K scale
    float* const negm = rowf + C::ROWF_RING * NT;                                            // [NT] -m
    float* const resc = negm + NT;                                                           // [NT]
    float* const red = resc + NT;                                                            // [2][4][NH]
    unsigned* const pre = reinterpret_cast<unsigned*>(red + 8 * NH);                         // [B + 1]
    int* const len_of = reinterpret_cast<int*>(pre + KV_MAX_BATCH + 4);                      // [B]
    uint8_t* const rows8 = reinterpret_cast<uint8_t*>(len_of + KV_MAX_BATCH);                // [B]

    // the warp's index from one lane: the compiler then knows the roles' code as uniform, which an MMA's operands have to be
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    // the merge may be brought up now; it waits for this launch's parts by itself
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) { mbar_init(&kvfull[i], 33); mbar_init(&kvempty[i], 4); }
        for (int i = 0; i < BUFS; ++i) {
            mbar_init(&kready[i], 4); mbar_init(&qkdone[i], 1);
            mbar_init(&vready[i], 4); mbar_init(&pready[i], 8); mbar_init(&pvdone[i], 1);
        }
        for (int i = 0; i < 2; ++i) { mbar_init(&qready[i], 2); mbar_init(&qfree[i], 1); }
        mbar_init(ofull, 1); mbar_init(oempty, 8);
        for (int i = 0; i < C::SEG_RING; ++i) { mbar_init(&segfull[i], 1); mbar_init(&segempty[i], 8); }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += C::THREADS) {
        const KvRequest rq(p, b);
        const KvShape sh(rq.rows * p.group, kv_tiles(rq.len), NT);
        rows8[b] = (uint8_t)rq.rows;
        len_of[b] = rq.len;
        pre[b + 1] = rq.len > 0 ? (unsigned)(p.heads * sh.row_tiles) * sh.unit_w : 0u;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int g = blockIdx.x;
    // segment number `i` of the CTA, once it is published; false: there is none (or the CTA has aborted)
    auto segment = [&](uint32_t i, KvSeg& sg) -> bool {
        const uint32_t at = i % C::SEG_RING;
        if (!__all_sync(0xFFFFFFFFu, kv_wait(&segfull[at], (i / C::SEG_RING) & 1u, abort_flag))) return false;
        sg = segs[at];
        return sg.k1 > 0;
    };
    KvSeg sg;

    if (warp < 4) {
        regs_dec<C::REGS_CONTROL>();
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            const uint64_t pol = p.row_tiles > 1 ? policy_evict_normal() : policy_evict_first();
            const int per_tile = KV_TILE >> p.page_log2;
            const uint32_t page_bytes = 2u * D << p.page_log2;
            const uint32_t stage0 = smem_u32(stages);
            int s = 0;
            uint32_t ph = 0, issued = 0, last_ph = 0, tile = 0;
            // inclusive scan of the weights
            unsigned carry = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                unsigned v = (b0 + lane < p.B) ? pre[b0 + lane + 1] : 0u;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const unsigned o = __shfl_up_sync(0xFFFFFFFFu, v, d);
                    if (lane >= d) v += o;
                }
                v += carry;
                if (b0 + lane < p.B) pre[b0 + lane + 1] = v;
                carry = __shfl_sync(0xFFFFFFFFu, v, 31);
            }
            if (lane == 0) pre[0] = 0;
            __syncwarp();
            const KvShares shares(carry, p.ctas);
            KvWalk walk(p, pre, len_of, rows8, shares.start(g), shares.start(g + 1), NT);
            uint32_t seg = 0;
            // the next segment, published for the others; k1 of 0 marks the end
            auto publish = [&]() -> bool {
                const bool there = walk.next(sg);
                const uint32_t at = seg % C::SEG_RING;
                if (!__all_sync(0xFFFFFFFFu, kv_wait(&segempty[at], ((seg / C::SEG_RING) & 1u) ^ 1u, abort_flag))) {
                    if (lane == 0) tc_fail(p.err, abort_flag, TL_DEV_ERR_TIMEOUT_PRODUCER);
                    return false;
                }
                if (lane == 0) {
                    if (!there) sg.k1 = 0;
                    segs[at] = sg;
                    mbar_arrive(&segfull[at]);
                }
                __syncwarp();
                ++seg;
                return there;
            };
            bool more = publish();
            int k = more ? sg.k0 : 0;
            // the page that this lane brings in of tile k: looked up a tile ahead
            auto look = [&](int& n) -> int {
                n = min((int)(((unsigned)len_of[sg.b] + (1u << p.page_log2) - 1) >> p.page_log2) - k * per_tile, per_tile);
                return lane < n ? __ldg(p.table + (size_t)sg.b * p.width + (size_t)k * per_tile + lane) : 0;
            };
            int n = 0, id = more ? look(n) : 0;
#pragma unroll 1
            while (more) {
                const int cur_n = n, head = sg.head;
                int page = id;
                if (++k == sg.k1) {
                    more = publish();
                    k = sg.k0;
                }
                if (more) id = look(n);
                if (page < 0 || page >= p.n_pages) {
                    atomicCAS(p.err, 0, TL_DEV_ERR_KV_PAGE);
                    page = 0;
                }
                if (!__all_sync(0xFFFFFFFFu, kv_wait(&kvempty[s], ph ^ 1u, abort_flag))) {
                    if (lane == 0) tc_fail(p.err, abort_flag, TL_DEV_ERR_TIMEOUT_PRODUCER);
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&kvfull[s], page_bytes * (uint32_t)cur_n);
                __syncwarp();
                if (lane < cur_n) {
                    const size_t unit = (size_t)page * p.heads + head;
                    bulk_load_s(stage0 + (uint32_t)(s * C::STAGE_BYTES) + page_bytes * (uint32_t)lane, p.pages + unit * page_bytes,
                                page_bytes, &kvfull[s], pol);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(page_scale + 8 * (tile % C::SCALE_RING) + lane)),
                                 "l"(p.scales + 2 * unit) : "memory");
                }
                ++tile;
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&kvfull[s])) : "memory");
                issued |= 1u << s;
                last_ph = (last_ph & ~(1u << s)) | (ph << s);
                if (++s == C::STAGES) { s = 0; ph ^= 1u; }
            }
            // every issued copy must land before the CTA can leave
#pragma unroll 1
            for (int i = 0; i < C::STAGES; ++i)
                if ((issued >> i) & 1u)
                    if (!kv_drain(&kvfull[i], (last_ph >> i) & 1u))
                        if (lane == 0) tc_fail(p.err, abort_flag, TL_DEV_ERR_TIMEOUT_DRAIN);
        } else if (warp < 3) {
            // ------------------------------------------------------------ MMA issuers
            const uint32_t tmem_u = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            const uint64_t qdesc = kv_uniform64(smem_desc_k_sw128(smem_u32(q_sm)));
            const uint64_t pdesc = kv_uniform64(smem_desc_mn_sw32(smem_u32(p_sm), C::P_ATOM, C::P_STEP));
            const uint32_t leader = elect_one() ? 1u : 0u;
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                if (ok && !__all_sync(0xFFFFFFFFu, kv_wait(bar, parity, abort_flag))) {
                    if (lane == 0) tc_fail(p.err, abort_flag, TL_DEV_ERR_TIMEOUT_MMA);
                    ok = false;
                }
            };
            KvRing<BUFS> ring;
            uint32_t seg = 0;
            uint64_t* last_bar = nullptr;
            uint32_t last_par = 0;
#pragma unroll 1
            while (ok && segment(seg, sg)) {
                const uint32_t n_bits = (uint32_t)(sg.nt >> 3) << 17;
#pragma unroll 1
                for (int k = sg.k0; k < sg.k1; ++k) {
                    const uint32_t b = ring.i;
                    if (warp == 1) {
                        if (k == sg.k0) wait(&qready[seg & 1u], (seg >> 1) & 1u);
                        wait(&kready[b], ring.par);
                        wait(&pvdone[b], ring.par ^ 1u);          // S^T's buffer and P's: O^T has the tile that lay there last
                        if (!ok) break;
                        tc_fence_after();
                        {
                            const uint64_t qd = qdesc + (uint64_t)((seg & 1u) * (C::Q_BYTES >> 4));
                            const uint32_t d = tmem_u + (uint32_t)(C::S_COL) + b * NT, a = tmem_u + (uint32_t)C::K_COL + b * C::K_COLS;
#pragma unroll
                            for (int i = 0; i < C::QSTEPS; ++i)
                                mma_f8_if(leader, d, a + 8u * (i % (D / 32)), qd + (uint64_t)(((i >> 2) * NT * 128 + (i & 3) * 32) >> 4),
                                          C::IDESC_QK | n_bits, i ? 1u : 0u);
                            mma_commit_if(leader, &qkdone[b]);
                            if (k + 1 == sg.k1) mma_commit_if(leader, &qfree[seg & 1u]);
                        }
                        last_bar = &qkdone[b];
                    } else {
                        if (k == sg.k0) wait(oempty, (seg & 1u) ^ 1u);
                        wait(&vready[b], ring.par);
                        wait(&pready[b], ring.par);
                        if (!ok) break;
                        tc_fence_after();
                        {
                            const uint64_t pd = pdesc + (uint64_t)(b * (C::P_BYTES >> 4));
#pragma unroll
                            for (int i = 0; i < KV_TILE / 16; ++i)
                                mma_f16_if(leader, tmem_u + (uint32_t)C::O_COL, tmem_u + (uint32_t)(C::V_COL + 8 * i) + b * C::V_COLS,
                                           pd + (uint64_t)((2 * i * C::P_STEP) >> 4), C::IDESC_PV | n_bits, (i || k != sg.k0) ? 1u : 0u);
                            mma_commit_if(leader, &pvdone[b]);
                            if (k + 1 == sg.k1) mma_commit_if(leader, ofull);
                        }
                        last_bar = &pvdone[b];
                    }
                    last_par = ring.par;
                    __syncwarp();
                    ring.step();
                }
                ++seg;
            }
            // no MMA may still run when tensor memory is released: the barrier of this warp's last ones
            if (last_bar && !__all_sync(0xFFFFFFFFu, kv_drain(last_bar, last_par)) && lane == 0)
                tc_fail(p.err, abort_flag, TL_DEV_ERR_TIMEOUT_DRAIN);
        } else {
            // ------------------------------------------------------------ rows
            uint32_t seg = 0;
#pragma unroll 1
            while (segment(seg, sg)) {
                if (seg > 0) {
                    if (!__all_sync(0xFFFFFFFFu, kv_wait(&qfree[seg & 1u], ((seg >> 1) & 1u) ^ 1u, abort_flag))) {
                        if (lane == 0) tc_fail(p.err, abort_flag, TL_DEV_ERR_TIMEOUT_PRODUCER);
                        break;
                    }
                    kv_load_rows<D, NT>(p, sg, lane, 32, q_sm + (seg & 1u) * C::Q_BYTES, rowf + (seg % C::ROWF_RING) * NT);
                    __syncwarp();
                    if (lane < 2) mbar_arrive(&qready[seg & 1u]);
                }
                ++seg;
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ movers
        regs_dec<C::REGS_MOVE>();
        const int qd = warp & 3, r = 32 * qd + lane;             // token of the tile; channel
        const uint32_t t_lane = tmem + ((uint32_t)(32 * qd) << 16);
        const int pl = p.page_log2;
        const uint32_t page_bytes = 2u * D << pl;
        const uint32_t k_off = (uint32_t)(r >> pl) * page_bytes + (uint32_t)(r & ((1 << pl) - 1)) * 16u;
        KvRing<C::STAGES> stage;
        KvRing<BUFS> ring;
        uint32_t seg = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (!__all_sync(0xFFFFFFFFu, kv_wait(bar, parity, abort_flag))) {
                if (lane == 0) tc_fail(p.err, abort_flag, TL_DEV_ERR_TIMEOUT_DEQUANT);
                ok = false;
            }
        };
#pragma unroll 1
        while (ok && segment(seg++, sg)) {
#pragma unroll 1
            for (int k = sg.k0; k < sg.k1; ++k, stage.step(), ring.step()) {
                const uint32_t b = ring.i;
                wait(&kvfull[stage.i], stage.par);
                if (!ok) break;
                const uint8_t* const st = stages + stage.i * C::STAGE_BYTES;
                uint32_t out[32];
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    *reinterpret_cast<uint4*>(out + 4 * c) = *reinterpret_cast<const uint4*>(st + k_off + ((16u * c) << pl));
                wait(&qkdone[b], ring.par ^ 1u);                  // the S^T that read this K buffer last
                if (!ok) break;
                tc_fence_after();
                if (D == 128) tmem_st32(t_lane + (uint32_t)C::K_COL + b * C::K_COLS, out);
                else tmem_st16(t_lane + (uint32_t)C::K_COL + b * C::K_COLS, out);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&kready[b]);
                // tokens behind the request's last one count nothing, whatever their bytes are
                const int valid = (k + 1 == sg.k1) ? sg.valid : KV_TILE;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    if (D == 128 || qd < 2) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int tt = 64 * half + 16 * c;
                            uint4 w = *reinterpret_cast<const uint4*>(st + (uint32_t)(tt >> pl) * page_bytes + (uint32_t)(D << pl) +
                                                                      (uint32_t)((tt & ((1 << pl) - 1)) >> 4) * (16u * D) + 16u * r);
                            if (valid < KV_TILE) {
                                w.x = kv_first_bytes(w.x, valid - tt);
                                w.y = kv_first_bytes(w.y, valid - tt - 4);
                                w.z = kv_first_bytes(w.z, valid - tt - 8);
                                w.w = kv_first_bytes(w.w, valid - tt - 12);
                            }
                            kv_decode16(w, out + 8 * c);
                        }
                    }
                    if (half == 0) {
                        // the O^T that read this V buffer last; a quarter without channels waits too, for an arrival ahead
                        // of its phase would complete another tile's
                        wait(&pvdone[b], ring.par ^ 1u);
                        if (!ok) break;
                        tc_fence_after();
                    } else {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&kvempty[stage.i]);
                    }
                    if (D == 128 || qd < 2) tmem_st32(t_lane + (uint32_t)C::V_COL + b * C::V_COLS + 32u * half, out);
                }
                if (!ok) break;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&vready[b]);
            }
        }
        tmem_wait_st();
    } else {
        // ------------------------------------------------------------ softmax
        regs_inc<C::REGS_SOFTMAX>();
        const int grp = (warp - 8) >> 2, qd = warp & 3, t = 32 * qd + lane;     // token of the tile; channel
        const int bar_id = 1 + grp;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * qd) << 16);
        // this token's rows in P: 16-byte units of 8 rows, two a 32-byte line, swapped in every other four tokens
        const uint32_t p_line = smem_u32(p_sm) + (uint32_t)((t >> 3) * C::P_STEP + (t & 7) * 32);
        float* const g_negm = negm + grp * NH;        // this group's rows, block by block
        float* const g_resc = resc + grp * NH;
        float* const g_red = red + grp * 4 * NH;
        uint32_t n = 0, seg = 0;
        KvRing<BUFS> ring;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            // a failure is recorded and the warp goes on: the group's barriers need all of its warps
            if (!__all_sync(0xFFFFFFFFu, kv_wait(bar, parity, abort_flag)) && lane == 0)
                tc_fail(p.err, abort_flag, TL_DEV_ERR_TIMEOUT_EPILOGUE);
        };
        // whether there is a segment is for the group to agree on, after an abort too: its barriers need all of its warps
#pragma unroll 1
        while (!kv_group_any(bar_id, !segment(seg, sg))) {
            if (seg == 0) {
                kv_load_rows<D, NT>(p, sg, (int)threadIdx.x - 256, 256, q_sm, rowf);
                kv_group_sync(bar_id);
                if (t == 0) mbar_arrive(&qready[0]);
            }
            // this group's blocks of 8 rows: nb of them from row c0 (the first group has one more if they are odd)
            const int blocks = (sg.n_rows + 7) >> 3;
            const int nb = grp ? blocks >> 1 : (blocks + 1) >> 1, c0 = grp ? 8 * ((blocks + 1) >> 1) : 0;
            // where a block lies in this token's lines of P
            auto p_unit = [&](int j) -> uint32_t {
                const uint32_t u = (uint32_t)(c0 >> 3) + j;
                return (u >> 1) * C::P_ATOM + (((u ^ (t >> 2)) & 1u) << 4);
            };
            float l[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) l[i] = 0.0f;
            uint32_t was_b = 0, was_par = 0;       // the tile before: its buffer
#pragma unroll 1
            for (int k = sg.k0; k < sg.k1; ++k) {
                const uint32_t b = ring.i;
                const bool first = k == sg.k0;
                wait(&qkdone[b], ring.par);
                tc_fence_after();
                const uint32_t s_at = t_lane + (uint32_t)(C::S_COL + c0) + b * NT;
                const float* const rf_at = rowf + (seg % C::ROWF_RING) * NT + c0;
                const float2 sc = page_scale[8 * (n % C::SCALE_RING) + (t >> p.page_log2)];
                const int valid = (k + 1 == sg.k1) ? sg.valid : KV_TILE;
                const bool live = t < valid;
                const float vs = live ? sc.y : 1.0f;
                const float lv = kv_lg2(vs);
                const uint64_t ks2 = f2_pack(sc.x, sc.x);
                float x[NH];
                // Twice where the reference moves (in a segment's first tile it always does, and x is not needed before). The
                // state is kept opaque, so that the code of x is there once: instruction fetches are a bound.
                uint32_t move = first ? 1u : 0u, moved = 0;
#pragma unroll 1
                for (;;) {
                    asm volatile("" : "+r"(move), "+r"(moved));
                    if (!move) {
                        // x = score - m; a full group's blocks in one piece (without branches between them the loads and the
                        // chains of different blocks overlap), others one by one
                        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        auto scores = [&](int j) {
#pragma unroll
                            for (int i = 8 * j; i < 8 * j + 8; i += 4) {
                                const float4 rf = *reinterpret_cast<const float4*>(rf_at + i);
                                const float4 nm = *reinterpret_cast<const float4*>(g_negm + i);
                                f2_unpack(f2_fma(f2_mul(f2_pack(x[i], x[i + 1]), ks2), f2_pack(rf.x, rf.y), f2_pack(nm.x, nm.y)), x[i], x[i + 1]);
                                f2_unpack(f2_fma(f2_mul(f2_pack(x[i + 2], x[i + 3]), ks2), f2_pack(rf.z, rf.w), f2_pack(nm.z, nm.w)), x[i + 2],
                                          x[i + 3]);
                            }
#pragma unroll
                            for (int i = 8 * j; i < 8 * j + 8; ++i) tops[i & 3] = fmaxf(tops[i & 3], x[i]);
                        };
                        if (nb == C::NB) {
#pragma unroll
                            for (int j = 0; j + 1 < C::NB; j += 2) tmem_ld16f(s_at + 8 * j, x + 8 * j);
                            if (C::NB & 1) tmem_ld8(s_at + 8 * (C::NB - 1), x + 8 * (C::NB - 1));
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < C::NB; ++j) scores(j);
                        } else {
#pragma unroll
                            for (int j = 0; j + 1 < C::NB; ++j)
                                if (j < nb) {
                                    tmem_ld8(s_at + 8 * j, x + 8 * j);
                                    tmem_wait_ld();
                                    scores(j);
                                }
                        }
                        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                        if (moved || !kv_group_any(bar_id, live && top + lv > KV_SLACK)) break;
                    }
                    move = 0;
                    moved = 1;
                    // the reference moves: maxima of the log-weights over the tile's tokens, block by block
#pragma unroll 1
                    for (int j = 0; j < nb; ++j) {
                        float v[8];
                        tmem_ld8(s_at + 8 * j, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = live ? fmaf(v[i] * sc.x, rf_at[8 * j + i], lv) : -INFINITY;
                        const float w = kv_across8(v, lane, [](float a_, float b_) { return fmaxf(a_, b_); });
                        if (lane < 8) g_red[qd * NH + 8 * j + ((lane & 1) << 2) + (lane & 2) + (lane >> 2)] = w;
                    }
                    kv_group_sync(bar_id);
                    if (t < 8 * nb) {
                        const float* const rd = g_red + t;
                        const float old = first ? -INFINITY : -g_negm[t];
                        const float now = fmaxf(old, fmaxf(fmaxf(rd[0], rd[NH]), fmaxf(rd[2 * NH], rd[3 * NH])));
                        // what O and l shrink by (nothing is held yet under an old m of minus infinity)
                        g_resc[t] = (old == -INFINITY) ? 0.0f : kv_ex2(old - now);
                        g_negm[t] = -now;
                    }
                    kv_group_sync(bar_id);
                    if (!first) {
                        wait(&pvdone[was_b], was_par);                // O holds every tile before this one
                        tc_fence_after();
#pragma unroll 1
                        for (int j = 0; j < nb; ++j) {
                            float o[8];
                            tmem_ld8(t_lane + (uint32_t)(C::O_COL + c0) + 8 * j, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] *= g_resc[8 * j + i];
                            tmem_st8(t_lane + (uint32_t)(C::O_COL + c0) + 8 * j, o);
                        }
                        tmem_wait_st();
#pragma unroll
                        for (int i = 0; i < NH; ++i) l[i] *= g_resc[i];        // rows without work hold nothing that counts
                    }
                }
                if (!live) {
#pragma unroll
                    for (int i = 0; i < NH; ++i) x[i] = -INFINITY;
                }
                const float vs8 = vs * 256.0f;                    // 2^KV_P_SHIFT
                const uint64_t vs2 = f2_pack(vs8, vs8);
                const uint32_t at = p_line + b * C::P_BYTES;
                auto weights = [&](int j) {
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const int c = 8 * j + i;
                        const uint64_t e2 = f2_pack(kv_ex2(x[c]), kv_ex2(x[c + 1]));
                        f2_unpack(f2_add(f2_pack(l[c], l[c + 1]), e2), l[c], l[c + 1]);
                        float w0, w1;
                        f2_unpack(f2_mul(e2, vs2), w0, w1);
                        h[i >> 1] = kv_pack_f16(w0, w1);
                    }
                    sts_128(at + p_unit(j), h[0], h[1], h[2], h[3]);
                };
                if (nb == C::NB) {
#pragma unroll
                    for (int j = 0; j < C::NB; ++j) weights(j);
                } else {
#pragma unroll
                    for (int j = 0; j + 1 < C::NB; ++j)
                        if (j < nb) weights(j);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pready[b]);
                was_b = b;
                was_par = ring.par;
                ++n;
                ring.step();
            }
            // the segment's part: l over the lanes and warps, O as it lies
#pragma unroll
            for (int j = 0; j < C::NB; ++j) {
                if (j < nb) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = l[8 * j + i];
                    const float w = kv_across8(v, lane, [](float a_, float b_) { return a_ + b_; });
                    if (lane < 8) g_red[qd * NH + 8 * j + ((lane & 1) << 2) + (lane & 2) + (lane >> 2)] = w;
                }
            }
            const size_t slot = (((size_t)sg.b * p.heads + sg.head) * p.row_tiles + sg.rt + g) * NT;
            kv_group_sync(bar_id);
            const int row = c0 + t;
            if (!sg.more) {
                if (t < 8 * nb && row < sg.n_rows) {
                    const float* const rd = g_red + t;
                    p.part_ml[slot + row] = make_float2(-g_negm[t] - KV_P_SHIFT, 256.0f * ((rd[0] + rd[NH]) + (rd[2 * NH] + rd[3 * NH])));
                }
                wait(ofull, seg & 1u);
                tc_fence_after();
#pragma unroll 1
                for (int j = 0; j < nb; ++j) {
                    float o[8];
                    tmem_ld8(t_lane + (uint32_t)(C::O_COL + c0) + 8 * j, o);
                    tmem_wait_ld();
                    if (D == 128 || qd < 2) {
                        float* const to = p.part_o + (slot + 8 * j + c0) * D + t;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (8 * j + c0 + i < sg.n_rows) to[i * D] = o[i];
                    }
                }
            } else {
                // joined with what these threads have written of the part; where an m is minus infinity there is nothing to join,
                // but a NaN counts
                if (t < 8 * nb && row < sg.n_rows) {
                    const float* const rd = g_red + t;
                    const float2 had = p.part_ml[slot + row];
                    const float m = -g_negm[t] - KV_P_SHIFT, top = fmaxf(had.x, m);
                    const float f0 = (had.x == -INFINITY) ? 0.0f : kv_ex2(had.x - top), f1 = (m == -INFINITY) ? 0.0f : kv_ex2(m - top);
                    p.part_ml[slot + row] = make_float2(top, had.y * f0 + 256.0f * ((rd[0] + rd[NH]) + (rd[2 * NH] + rd[3 * NH])) * f1);
                    g_resc[t] = f0;
                    g_negm[t] = f1;
                }
                kv_group_sync(bar_id);
                wait(ofull, seg & 1u);
                tc_fence_after();
#pragma unroll 1
                for (int j = 0; j < nb; ++j) {
                    float o[8], had[8];
                    float* const to = p.part_o + (slot + 8 * j + c0) * D + t;
                    tmem_ld8(t_lane + (uint32_t)(C::O_COL + c0) + 8 * j, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) had[i] = ((D == 128 || qd < 2) && 8 * j + c0 + i < sg.n_rows) ? to[i * D] : 0.0f;
                    tmem_wait_ld();
                    if (D == 128 || qd < 2) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (8 * j + c0 + i < sg.n_rows) to[i * D] = fmaf(had[i], g_resc[8 * j + i], o[i] * g_negm[8 * j + i]);
                    }
                }
            }
            tc_fence_before();
            kv_group_sync(bar_id);            // red and negm may change again
            if (lane == 0) { mbar_arrive(oempty); mbar_arrive(&segempty[seg % C::SEG_RING]); }
            ++seg;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// One warp per row of a unit, a CTA's rows all of one unit, so that they share the tree's K and V of the KV head in
// shared memory: the scores of the nodes that the row sees (a lane a node), their softmax and V in fp32, then the
// parts of the cached tokens, in list order. What the mask leaves out is never used, so nothing of it (an infinity, a
// NaN) reaches the row. A row that sees nothing at all gives zeros. Latency-bound, so all loads that do not depend on one
// another are in flight at once. It is launched early, but the streaming kernel has all registers of an SM: the tree's part
// runs while other SMs still stream.
constexpr int KV_MERGE_WARPS = 8, KV_MERGE_THREADS = 32 * KV_MERGE_WARPS;

template <int D>
__global__ void __launch_bounds__(KV_MERGE_THREADS) kv_merge_kernel(const KvAttnParams p, int chunks) {
    constexpr int E = D / 32;                            // channels of a lane
    constexpr int RP = D + 8;                            // padded row: 16-byte reads of eight rows spread over the banks
    constexpr int LOADS = KV_MAX_ROWS * D / 8 / KV_MERGE_THREADS;     // 16-byte pieces of K a thread, and of V, at most
    __shared__ __align__(16) __nv_bfloat16 kn[KV_MAX_ROWS * RP], vn[KV_MAX_ROWS * RP], qn[KV_MERGE_WARPS * D];
    __shared__ unsigned sums[2][KV_MERGE_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x, head = blockIdx.y / chunks, chunk = blockIdx.y % chunks;
    // this request, and its place in the tile list
    const KvRequest rq(p, b);
    unsigned before = 0, all = 0;
#pragma unroll 1
    for (int i = tid; i < p.B; i += KV_MERGE_THREADS) {
        const KvRequest other(p, i);
        KvShape sh(other.rows * p.group, kv_tiles(other.len), p.nt);
        const unsigned w = other.len > 0 ? (unsigned)(p.heads * sh.row_tiles) * sh.unit_w : 0u;
        all += w;
        if (i < b) before += w;
    }
    const int first = rq.first, rows = rq.rows;
    if (rq.bad && tid == 0 && blockIdx.y == 0) atomicCAS(p.err, 0, TL_DEV_ERR_KV_ROWS);
    // every CTA waits for the streaming kernel, so that this launch never ends before it
    if (chunk * KV_MERGE_WARPS >= rows * p.group) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int r = chunk * KV_MERGE_WARPS + warp, i = r / p.group, h = head * p.group + r % p.group;
    const int row = first + i;
    const bool works = r < rows * p.group;
    unsigned bits = 0;
    if (p.k_new) {
        // all that the tree's part reads, in one go
        uint4 kq[LOADS], vq[LOADS], qq = make_uint4(0, 0, 0, 0);
        const size_t base = (size_t)first * p.new_stride + (size_t)head * D;
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int e = tid + u * KV_MERGE_THREADS, j = e / (D / 8), c = e % (D / 8);
            if (j < rows) {
                kq[u] = __ldg(reinterpret_cast<const uint4*>(p.k_new + base + (size_t)j * p.new_stride + 8 * c));
                vq[u] = __ldg(reinterpret_cast<const uint4*>(p.v_new + base + (size_t)j * p.new_stride + 8 * c));
            }
        }
        if (works) {
            if (lane < D / 8) qq = __ldg(reinterpret_cast<const uint4*>(p.q + (size_t)row * p.q_stride + (size_t)h * D) + lane);
            bits = p.mask ? __ldg(p.mask + row) : (2u << i) - 1u;
            if (rows < 32) bits &= (1u << rows) - 1u;
        }
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int e = tid + u * KV_MERGE_THREADS, j = e / (D / 8), c = e % (D / 8);
            if (j < rows) {
                *reinterpret_cast<uint4*>(kn + j * RP + 8 * c) = kq[u];
                *reinterpret_cast<uint4*>(vn + j * RP + 8 * c) = vq[u];
            }
        }
        if (lane < D / 8) *reinterpret_cast<uint4*>(qn + warp * D + 8 * lane) = qq;
    }
    all = __reduce_add_sync(0xFFFFFFFFu, all);
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    if (lane == 0) { sums[0][warp] = all; sums[1][warp] = before; }
    __syncthreads();
    if (!works) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    all = before = 0;
#pragma unroll
    for (int u = 0; u < KV_MERGE_WARPS; ++u) { all += sums[0][u]; before += sums[1][u]; }

    float m = -INFINITY, l = 0.0f;
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    if (bits) {
        const bool sees = (bits >> lane) & 1u;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (sees) {
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) {
                const uint4 a = *reinterpret_cast<const uint4*>(kn + lane * RP + 8 * c), w = *reinterpret_cast<const uint4*>(qn + warp * D + 8 * c);
                const uint32_t ka[4] = {a.x, a.y, a.z, a.w}, qa[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    acc[u] = fmaf(__int_as_float((int)(ka[u] & 0xFFFF0000u)), __int_as_float((int)(qa[u] & 0xFFFF0000u)),
                                  fmaf(__int_as_float((int)(ka[u] << 16)), __int_as_float((int)(qa[u] << 16)), acc[u]));
            }
        }
        const float s = sees ? ((acc[0] + acc[1]) + (acc[2] + acc[3])) * p.scale : -INFINITY;
        m = kv_warp_max(s);
        // where every node's score is minus infinity they weigh nothing beside cached tokens; alone they leave 0 / 0
        const float pr = sees ? exp2f(s - ((m == -INFINITY && rq.len > 0) ? 0.0f : m)) : 0.0f;
        l = pr;
#pragma unroll
        for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        for (unsigned todo = bits; todo;) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = todo ? __ffs(todo) - 1 : 0;
                const float w = todo ? __shfl_sync(0xFFFFFFFFu, pr, j) : 0.0f;
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const uint32_t x = todo ? *reinterpret_cast<const uint32_t*>(vn + j * RP + E * lane + e) : 0u;
                    o[e] = fmaf(w, __int_as_float((int)(x << 16)), o[e]);
                    o[e + 1] = fmaf(w, __int_as_float((int)(x & 0xFFFF0000u)), o[e + 1]);
                }
                todo &= todo - 1;
            }
        }
    }
    // the parts of the cached tokens: a lane looks at a part (whether the CTA had a tile of the unit, and its m and l), then
    // all lanes add the parts' O in order, eight loads in flight, the first eight beside those of m and l
    const int tiles = kv_tiles(rq.len);
    const KvShape sh(rows * p.group, tiles, p.nt);
    const int rt = r / sh.nt, n = r - rt * sh.nt;
    const unsigned at0 = before + (unsigned)(head * sh.row_tiles + rt) * sh.unit_w;
    const long long slot0 = ((long long)b * p.heads + head) * p.row_tiles + rt;
    const KvShares shares(all, p.ctas);
    int g0 = 0, g1 = -1;
    if (rq.len > 0) {
        g0 = shares.owner(at0);
        g1 = shares.owner(at0 + sh.unit_w - 1);
    }
    bool waits = true;
    for (int gb = g0; gb <= g1; gb += 32) {
        const int g = gb + lane;
        float2 ml = make_float2(-INFINITY, 0.0f);
        bool has = false;
        if (g <= g1) {
            const unsigned lo = shares.start(g), hi = shares.start(g + 1);
            has = sh.tile_from(lo > at0 ? lo - at0 : 0u, tiles) < sh.tile_from(hi > at0 ? hi - at0 : 0u, tiles);
        }
        unsigned todo = __ballot_sync(0xFFFFFFFFu, has);
        if (waits) asm volatile("griddepcontrol.wait;" ::: "memory");
        waits = false;
        if (has) ml = __ldcg(p.part_ml + (size_t)(slot0 + g) * p.nt + n);
        float f = 0.0f;
        bool fresh = true;
        while (todo) {
            float2 x[8][E / 2];
            unsigned left = todo;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int src = left ? __ffs(left) - 1 : 0;
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    x[u][e / 2] = left ? __ldcg(reinterpret_cast<const float2*>(p.part_o + ((size_t)(slot0 + gb + src) * p.nt + n) * D + E * lane + e))
                                       : make_float2(0.0f, 0.0f);
                left &= left - 1;
            }
            if (fresh) {
                const float top = fmaxf(m, kv_warp_max(ml.x));
                // a part or tree without weight (m of minus infinity) counts nothing, but a NaN of it counts
                const float f0 = (m == -INFINITY) ? 0.0f : exp2f(m - top);
                f = (ml.x == -INFINITY) ? 0.0f : exp2f(ml.x - top);
                float sum = ml.y * f;
#pragma unroll
                for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
                m = top;
                l = l * f0 + sum;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] *= f0;
                fresh = false;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float fu = todo ? __shfl_sync(0xFFFFFFFFu, f, __ffs(todo) - 1) : 0.0f;
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    o[e] = fmaf(x[u][e / 2].x, fu, o[e]);
                    o[e + 1] = fmaf(x[u][e / 2].y, fu, o[e + 1]);
                }
                todo &= todo - 1;
            }
        }
    }
    if (waits) asm volatile("griddepcontrol.wait;" ::: "memory");
    const float inv = (m == -INFINITY && l == 0.0f) ? 0.0f : 1.0f / l;
    __nv_bfloat16* const to = p.out + (size_t)row * p.out_stride + (size_t)h * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<__nv_bfloat162*>(to + e) = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
}

}  // namespace tl
