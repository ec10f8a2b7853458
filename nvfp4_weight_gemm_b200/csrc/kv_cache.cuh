// kv_cache.cuh -- the 8-bit paged KV cache of the verify pass: block tables and slot maps
// (kv_slots_kernel) and the commit of accepted tokens (kv_commit_kernel).
//
// 16 of the served model's 64 layers are attention layers (TandemLLM docs v0.12.0, "What TandemLLM
// is", section 1.1). Their keys and values live in a pool of pages of P tokens. One page holds,
// per KV head, 2 * P * D E4M3 bytes and two scales:
//
//     pages  uint8 [n_pages][Hkv][2][P * D]   side 0: K as [D/16][P][16], side 1: V as [P/16][D][16]
//     scales float [n_pages][Hkv][2]          powers of two, 2^-60 .. 2^60
//
// Both sides are cut into 16-byte groups: a K group is one token's 16 consecutive channels, a V group
// one channel's 16 consecutive tokens. A warp whose lanes are 32 tokens (K) or 32 channels (V) then
// reads shared memory in 512-byte rows without bank conflicts, and each lane's 16 bytes are
// consecutive along the axis that the product sums over.
//
// The scale is a power of two: E4M3 is a floating format, so a finer scale would buy no relative
// precision, and moving a page to a larger scale (below) only shifts exponents, which is exact for
// every value that stays normal.
#pragma once
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

namespace tl {

constexpr int KV_MAX_BATCH = 1024;
constexpr int KV_EXP_MIN = -60, KV_EXP_MAX = 60;

constexpr int TL_DEV_ERR_KV_SLOT = 0x301;   // a slot or source row outside its range (commit)
constexpr int TL_DEV_ERR_KV_PAGE = 0x302;   // a page id outside 0..n_pages-1 (attention)
constexpr int TL_DEV_ERR_KV_ROWS = 0x303;   // row offsets that do not fit R or max_rows (attention)

// ---------------------------------------------------------------- block tables and slot maps

struct KvSlotsParams {
    int* lens;          // [B] in/out: tokens held
    const int* want;    // [B] tokens wanted
    int* table;         // [B][width] in/out
    int* free_pages;    // [n_pages] in/out: a stack
    int* n_free;        // in/out: its height
    int* slots;         // [max_slots] out
    int* starts;        // [B + 1] out
    int* info;          // [4] out
    int B, width, page_log2, n_pages, max_slots;
};

constexpr int KV_SLOTS_THREADS = 1024;
constexpr int KV_SLOTS_A_CTA = 2048;        // slots of a CTA before the cluster grows (up to 8 CTAs)

// Inclusive scan of one value a thread over the block (1024 threads); `total` gets the sum.
__device__ __forceinline__ unsigned long long kv_block_scan(unsigned long long v, unsigned long long* warp_sums,
                                                            unsigned long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += o;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        unsigned long long s = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long o = __shfl_up_sync(0xFFFFFFFFu, s, d);
            if (lane >= d) s += o;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    if (warp > 0) v += warp_sums[warp - 1];
    *total = warp_sums[31];
    __syncthreads();
    return v;
}

// The request whose half-open range of the exclusive prefix sums `pre` ([B + 1], pre[B] = total)
// holds i: the largest b with pre[b] <= i.
__device__ __forceinline__ int kv_find(const int* pre, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// One thread a request; the pages and slots of all requests are then dealt out over the threads of
// the launch, each finding its request in the prefix sums. Launched as one CTA, or as one cluster of
// CTAs that repeat the scan and share the dealing out when there are many slots. Latency-bound: a
// few dependent reads of the request arrays, the stack and the table. Two calls of 64 requests with 8 slots each: 16.5 us
// on one CTA, as on eight; of 1000 requests with 8 slots each 84 us on one and 29 on eight, with 300 each 142 and 35.
__global__ void __launch_bounds__(KV_SLOTS_THREADS, 1) kv_slots_kernel(const KvSlotsParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    __shared__ unsigned long long warp_sums[32];
    __shared__ int pre_add[KV_MAX_BATCH + 1], pre_more[KV_MAX_BATCH + 1], pre_gone[KV_MAX_BATCH + 1];
    __shared__ int len_of[KV_MAX_BATCH], want_of[KV_MAX_BATCH];
    const int b = threadIdx.x;
    const int P = 1 << p.page_log2;
    const long long room = (long long)p.width * P;
    const int n_free = *p.n_free;
    int len = 0, want = 0;
    bool refused = false;
    if (b < p.B) {
        len = p.lens[b];
        want = p.want[b];
        refused = len < 0 || want < 0 || len > room || want > room;
        if (refused) want = len;
        len_of[b] = len;
        want_of[b] = want;
    }
    const int held = refused ? 0 : (int)(((long long)len + P - 1) >> p.page_log2);
    const int need = refused ? 0 : (int)(((long long)want + P - 1) >> p.page_log2);
    const unsigned long long add = (!refused && want > len) ? (unsigned long long)(want - len) : 0ull;
    const unsigned long long more = need > held ? need - held : 0, gone = held > need ? held - need : 0;
    unsigned long long adds, pages;
    const unsigned long long add_end = kv_block_scan(add, warp_sums, &adds);
    unsigned long long more_end, gone_end;
    long long n_more, n_gone;
    if ((long long)p.B * p.width <= 0xFFFFFFFFll) {
        // both sums are of pages that the table has entries for, so 32 bits hold either: one scan for both
        const unsigned long long page_end = kv_block_scan(more | (gone << 32), warp_sums, &pages);
        more_end = page_end & 0xFFFFFFFFull;
        gone_end = page_end >> 32;
        n_more = (long long)(pages & 0xFFFFFFFFull);
        n_gone = (long long)(pages >> 32);
    } else {
        more_end = kv_block_scan(more, warp_sums, &pages);
        n_more = (long long)pages;
        gone_end = kv_block_scan(gone, warp_sums, &pages);
        n_gone = (long long)pages;
    }
    const int n_refused = __syncthreads_count(refused);
    const bool corrupt = n_free < 0 || n_free + n_gone > p.n_pages;
    const long long top = n_free + n_gone;
    const long long pages_missing = n_more > top ? n_more - top : 0;
    const long long slots_missing = adds > (unsigned long long)p.max_slots ? (long long)adds - p.max_slots : 0;
    const bool grows = !corrupt && pages_missing == 0 && slots_missing == 0;
    if (b < p.B) {
        pre_add[b] = grows ? (int)(add_end - add) : 0;
        pre_more[b] = grows ? (int)(more_end - more) : 0;
        pre_gone[b] = corrupt ? 0 : (int)(gone_end - gone);
    }
    if (b == 0) {
        pre_add[p.B] = grows ? (int)adds : 0;
        pre_more[p.B] = grows ? (int)n_more : 0;
        pre_gone[p.B] = corrupt ? 0 : (int)n_gone;
    }
    __syncthreads();
    const int t0 = rank * KV_SLOTS_THREADS + threadIdx.x, step = ranks * KV_SLOTS_THREADS;
    // every CTA has read the state: it may change now
    if (ranks > 1) cluster.sync();
    // pages of requests that shrink go back on the stack, the last one first, so that a later growth by
    // as much takes the same pages again
    for (int i = t0; i < pre_gone[p.B]; i += step) {
        const int r = kv_find(pre_gone, p.B, i);
        int* const entry = p.table + (size_t)r * p.width + ((want_of[r] + P - 1) >> p.page_log2) + (i - pre_gone[r]);
        p.free_pages[top - 1 - i] = *entry;
        *entry = -1;
    }
    if (ranks > 1) cluster.sync(); else __syncthreads();
    for (int i = t0; i < pre_more[p.B]; i += step) {
        const int r = kv_find(pre_more, p.B, i);
        p.table[(size_t)r * p.width + ((len_of[r] + P - 1) >> p.page_log2) + (i - pre_more[r])] =
            __ldcg(p.free_pages + (top - 1 - i));
    }
    if (rank == 0) {
        if (b < p.B) {
            p.starts[b] = pre_add[b];
            if (!refused && !corrupt && (grows || want < len)) p.lens[b] = want;
        }
        if (b == 0) {
            p.starts[p.B] = pre_add[p.B];
            if (!corrupt) *p.n_free = (int)(top - pre_more[p.B]);
            p.info[0] = (corrupt ? 8 : 0) | (n_refused ? 4 : 0) | (slots_missing ? 2 : 0) | (pages_missing && !corrupt ? 1 : 0);
            p.info[1] = corrupt ? 0 : pages_missing > 0x7FFFFFFF ? 0x7FFFFFFF : (int)pages_missing;
            p.info[2] = slots_missing > 0x7FFFFFFF ? 0x7FFFFFFF : (int)slots_missing;
            p.info[3] = n_refused;
        }
    }
    if (ranks > 1) cluster.sync(); else __syncthreads();
    // a warp takes 128 slots at a time, 32 side by side; a lane searches for the first and looks whether the request of
    // the last one still holds the next
    const int n_slots = pre_add[p.B], lane = b & 31;
    for (long long i0 = (t0 >> 5) * 128; i0 < p.max_slots; i0 += 4 * step) {
        int page[4], r = 0;
        int pos[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long i = i0 + 32 * u + lane;
            page[u] = -1;
            pos[u] = 0;
            if (i < n_slots) {
                if (u == 0 || i >= pre_add[r + 1]) r = kv_find(pre_add, p.B, (int)i);
                pos[u] = len_of[r] + ((int)i - pre_add[r]);
                page[u] = __ldcg(p.table + (size_t)r * p.width + (pos[u] >> p.page_log2));
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long i = i0 + 32 * u + lane;
            if (i < p.max_slots) p.slots[i] = page[u] >= 0 ? (page[u] << p.page_log2) + (pos[u] & (P - 1)) : -1;
        }
    }
}

// ---------------------------------------------------------------- commit

struct KvCommitParams {
    uint8_t* pages;
    float* scales;
    const __nv_bfloat16* k;   // [n_rows][Hkv][D], rows `stride` elements apart
    const __nv_bfloat16* v;
    const int* src;           // [n] source row of each token, or null (token i is row i)
    const int* slots;         // [n] where each token goes, < 0: nowhere
    int* err;
    long long stride;
    int n_rows, n, n_pages, page_log2, heads, chunk;
};

constexpr int KV_COMMIT_THREADS = 128;

// The exponent that commit gives a block of values whose largest finite magnitude is `top`: the
// smallest e in KV_EXP_MIN .. KV_EXP_MAX with top <= 448 * 2^e.
__device__ __forceinline__ int kv_exponent(float top) {
    int e;
    const float m = frexpf(top, &e);          // top = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = (top > 0.0f) ? e - 9 + (m > 0.875f) : KV_EXP_MIN;
    return min(max(e, KV_EXP_MIN), KV_EXP_MAX);
}

__device__ __forceinline__ float kv_pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// Two E4M3 bytes, round to nearest even, largest magnitude 448; NaN stays NaN (a in the low byte).
__device__ __forceinline__ uint32_t kv_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Two E4M3 bytes -> two f16 values (exact).
__device__ __forceinline__ uint32_t kv_f16x2(uint32_t two_bytes) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two_bytes));
    return h;
}

// A bf16 value times `inv`; an infinity becomes a NaN (E4M3 has no infinity).
__device__ __forceinline__ float kv_scaled(uint32_t bits16, float inv) {
    const float x = __int_as_float((int)(bits16 << 16));
    return ((bits16 & 0x7F80u) == 0x7F80u) ? __int_as_float(0x7FC00000) : x * inv;
}

// Two E4M3 bytes of bf16 values (in the upper halves) times `inv`. ODD: there may be infinities and NaN.
template <bool ODD>
__device__ __forceinline__ uint32_t kv_bytes2(uint32_t a, uint32_t b, float inv) {
    if (ODD) return kv_e4m3x2(kv_scaled(a >> 16, inv), kv_scaled(b >> 16, inv));
    return kv_e4m3x2(__int_as_float((int)a) * inv, __int_as_float((int)b) * inv);
}

// Four bytes of a page moved to a scale 2^shift times smaller in value (shift <= 0): every value is
// multiplied by 2^shift and rounded to E4M3 again (exact unless it becomes subnormal).
__device__ __forceinline__ uint32_t kv_moved(uint32_t w, float factor) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t h = kv_f16x2((w >> (16 * i)) & 0xFFFFu);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        out |= kv_e4m3x2(f.x * factor, f.y * factor) << (16 * i);
    }
    return out;
}

// One CTA per (chunk of tokens, KV head and side). Consecutive tokens that go to consecutive places
// of one page form a run, and a CTA writes the runs that begin in its chunk: it brings the run's
// rows of its head into shared memory, finds their largest finite magnitude, and with it the page's
// scale, moves the bytes that the page holds already if the scale grew, and writes the new ones.
// A page whose first token is written takes no notice of what it held. Bytes behind the run stay.
// A page has one run in a call: the caller keeps its tokens together. (Two runs of a page, with tokens that go nowhere between
// them, would change one scale from two CTAs. A search of the list for them, so that one CTA writes them in turn, was right but
// cost calls without any: 2.8 -> 3.2 us for 5 tokens, replayed back to back, 43 -> 47 to 56 for 2 x 16k.)
// A page whose scale grows is read and written once more. For prompts the rows' bytes are the bound (bf16 in, E4M3 out:
// 2 x 16k tokens of 8 heads take 44 us, 31 at copy speed), so the instructions an element are few: maxima and the test for
// infinities on packed halves, two channels of V a thread; 64 registers keep eight CTAs on an SM. For a few tokens it is
// latency, two dependent reads (slots, rows) and the page's: 5 us for 5 tokens.
template <int D>
__global__ void __launch_bounds__(KV_COMMIT_THREADS, 8) kv_commit_kernel(const KvCommitParams p) {
    constexpr int RP = D + 8;                     // padded row in elements: 16-byte column reads of 8 lanes spread over the banks
    extern __shared__ __align__(16) __nv_bfloat16 rows[];      // [P][RP], in 16-byte pieces
    __shared__ int sl[2 * KV_COMMIT_THREADS];     // slots of tokens i0 - 1 .. i0 + chunk + P - 2, all that a run may reach
    __shared__ unsigned begins[4];                // bit i of word i / 32: a run begins at token i of the chunk
    __shared__ unsigned tops[4];
    const int P = 1 << p.page_log2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.y >> 1, side = blockIdx.y & 1;
    const int i0 = blockIdx.x * p.chunk;
    const long long places = (long long)p.n_pages << p.page_log2;
    const __nv_bfloat16* const x = (side ? p.v : p.k) + (size_t)head * D;

#pragma unroll
    for (int j = tid; j < 2 * KV_COMMIT_THREADS; j += KV_COMMIT_THREADS) {
        const int i = i0 - 1 + j;
        sl[j] = (j < p.chunk + P && i >= 0 && i < p.n) ? __ldg(p.slots + i) : -2;      // -2: follows nothing
    }
    __syncthreads();
    {
        bool begin = false;
        if (tid < p.chunk) {
            const int s = sl[tid + 1];
            if (s >= places) atomicCAS(p.err, 0, TL_DEV_ERR_KV_SLOT);
            begin = s >= 0 && s < places && ((s & (P - 1)) == 0 || sl[tid] != s - 1);
        }
        const unsigned m = __ballot_sync(0xFFFFFFFFu, begin);
        if (lane == 0) begins[warp] = m;
    }
    __syncthreads();
    for (int w = 0; w < KV_COMMIT_THREADS / 32; ++w) {
        for (unsigned todo = begins[w]; todo; todo &= todo - 1) {
            const int first = i0 + 32 * w + __ffs(todo) - 1;
            const int slot = sl[first - i0 + 1];
            const int page = slot >> p.page_log2, off = slot & (P - 1);
            // the run's length
            int m = 1;
            {
                const int most = min(P - off, p.n - first);
                bool goes = tid >= 1 && tid < most && sl[first - i0 + 1 + tid] == slot + tid;
                const unsigned g = __ballot_sync(0xFFFFFFFFu, goes || tid == 0);
                __shared__ unsigned follows[4];
                if (lane == 0) follows[warp] = g;
                __syncthreads();
                m = 0;
                for (int u = 0; u < 4; ++u) {
                    const unsigned f = follows[u];
                    if (f == 0xFFFFFFFFu) { m += 32; continue; }
                    m += __ffs(~f) - 1;
                    break;
                }
                m = min(m, most);
            }
            uint8_t* const at = p.pages + (((size_t)page * p.heads + head) * 2 + side) * ((size_t)P * D);
            float* const scale = p.scales + ((size_t)page * p.heads + head) * 2 + side;
            const float was = off ? *scale : 0.0f;
            // rows into shared memory, eight loads of a thread in flight, and the largest finite magnitude (bf16 magnitudes
            // order as integers)
            unsigned top = 0, top2 = 0;             // top2: of the elements in lower and in upper halves
            bool outside = false;                   // a row that is not there
            constexpr int LPR = D / 8, STEP = KV_COMMIT_THREADS / LPR;      // lanes of a row, rows at a time
            const int c = tid % LPR;
#pragma unroll 1
            for (int t0 = tid / LPR; t0 < m; t0 += 8 * STEP) {
                uint4 q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int t = t0 + j * STEP;
                    q[j] = make_uint4(0, 0, 0, 0);
                    if (t < m) {
                        const int row = p.src ? __ldg(p.src + first + t) : first + t;
                        if (row >= 0 && row < p.n_rows)
                            q[j] = __ldcs(reinterpret_cast<const uint4*>(x + (size_t)row * p.stride + 8 * c));
                        else
                            outside = true;
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (t0 + j * STEP < m) *reinterpret_cast<uint4*>(rows + (t0 + j * STEP) * RP + 8 * c) = q[j];
                    top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(q[j].x & 0x7FFF7FFFu, q[j].y & 0x7FFF7FFFu),
                                                   __vmaxu2(q[j].z & 0x7FFF7FFFu, q[j].w & 0x7FFF7FFFu)));
                }
            }
            if (outside) atomicCAS(p.err, 0, TL_DEV_ERR_KV_SLOT);
            top = max(top2 & 0xFFFFu, top2 >> 16);
            const bool odd = __syncthreads_or(top >= 0x7F80u);      // there are infinities or NaN: the largest of the others
            if (odd) {
                top = 0;
                for (int e = tid; e < m * D; e += KV_COMMIT_THREADS) {
                    const unsigned h = reinterpret_cast<const unsigned short*>(rows)[(e / D) * RP + e % D] & 0x7FFFu;
                    if (h < 0x7F80u) top = max(top, h);
                }
            }
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            if (lane == 0) tops[warp] = top;
            __syncthreads();
            top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
            int e = kv_exponent(__int_as_float((int)(top << 16)));
            int e_was = e;
            if (off) {
                e_was = min(max((int)((__float_as_int(was) >> 23) & 0xFF) - 127, KV_EXP_MIN), KV_EXP_MAX);
                e = max(e, e_was);
            }
            const float inv = kv_pow2(-e), factor = kv_pow2(max(e_was - e, -126));
            if (off > 0 && e_was != e) {
                // the bytes in front of the run move to the page's new scale, two 16-byte groups of a thread in flight
                const int n_old = side ? ((off + 15) >> 4) * D : off * (D / 16);
                const unsigned inv_off = ((1u << 20) + off - 1) / off;      // u / off = u * inv_off >> 20 for u < 1024, off < 128
#pragma unroll 1
                for (int u0 = tid; u0 < n_old; u0 += 2 * KV_COMMIT_THREADS) {
                    uint4* at_u[2];
                    uint4 q[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int u = u0 + j * KV_COMMIT_THREADS, cu = (int)((unsigned)u * inv_off >> 20);
                        at_u[j] = reinterpret_cast<uint4*>(at) + (side ? u : cu * P + (u - cu * off));
                        if (u < n_old) q[j] = *at_u[j];
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int u = u0 + j * KV_COMMIT_THREADS;
                        if (u >= n_old) break;
                        uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // of a V group that the run begins in, the bytes from there on stay
                            const int nb = side ? min(max(off - (u / D * 16 + 4 * i), 0), 4) : 4;
                            const uint32_t keep = nb == 4 ? 0xFFFFFFFFu : (1u << (8 * nb)) - 1u;
                            w[i] = (kv_moved(w[i], factor) & keep) | (w[i] & ~keep);
                        }
                        *at_u[j] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncthreads();      // the run writes single bytes of such a group
            }
            if (side == 0) {
                // K: 16-byte groups (16 channels of a token), tokens fastest
                const unsigned inv_m = ((1u << 20) + m - 1) / m;      // u / m = u * inv_m >> 20 for u < 1024, m <= 128
                auto convert = [&](auto odd_) {
                    constexpr bool ODD = decltype(odd_)::value;
#pragma unroll 1
                    for (int u = tid; u < m * (D / 16); u += KV_COMMIT_THREADS) {
                        const int c = (int)((unsigned)u * inv_m >> 20), t = u - c * m;
                        const uint4 a = *reinterpret_cast<const uint4*>(rows + t * RP + 16 * c);
                        const uint4 b = *reinterpret_cast<const uint4*>(rows + t * RP + 16 * c + 8);
                        const uint32_t in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                        uint32_t out[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            out[j] = kv_bytes2<ODD>(in[2 * j] << 16, in[2 * j] & 0xFFFF0000u, inv) |
                                     (kv_bytes2<ODD>(in[2 * j + 1] << 16, in[2 * j + 1] & 0xFFFF0000u, inv) << 16);
                        *reinterpret_cast<uint4*>(at + ((size_t)c * P + off + t) * 16) = make_uint4(out[0], out[1], out[2], out[3]);
                    }
                };
                if (odd) convert(std::true_type{}); else convert(std::false_type{});
            } else {
                // V: 16-byte groups (16 tokens of a channel), channels fastest; a group that the run fills in part
                // keeps its other bytes
                const unsigned short* const bits = reinterpret_cast<const unsigned short*>(rows);
                const int g0 = off >> 4, g1 = (off + m + 15) >> 4;
                auto convert = [&](auto odd_) {
                    constexpr bool ODD = decltype(odd_)::value;
#pragma unroll 1
                    for (int u = tid; u < (g1 - g0) * (D / 2); u += KV_COMMIT_THREADS) {
                        const int g = g0 + u / (D / 2), d = 2 * (u % (D / 2));             // two channels of a group
                        const int lo = max(16 * g, off), hi = min(16 * g + 16, off + m);   // places of the run in the group
                        if (hi - lo == 16) {
                            const unsigned short* const from = bits + (lo - off) * RP + d;
                            uint32_t w[16], out[8];
#pragma unroll
                            for (int t = 0; t < 16; ++t) w[t] = *reinterpret_cast<const uint32_t*>(from + t * RP);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t* const v = w + 4 * j;
                                out[j] = kv_bytes2<ODD>(v[0] << 16, v[1] << 16, inv) | (kv_bytes2<ODD>(v[2] << 16, v[3] << 16, inv) << 16);
                                out[4 + j] = kv_bytes2<ODD>(v[0] & 0xFFFF0000u, v[1] & 0xFFFF0000u, inv) |
                                             (kv_bytes2<ODD>(v[2] & 0xFFFF0000u, v[3] & 0xFFFF0000u, inv) << 16);
                            }
                            uint4* const to = reinterpret_cast<uint4*>(at + ((size_t)g * D + d) * 16);
                            to[0] = make_uint4(out[0], out[1], out[2], out[3]);
                            to[1] = make_uint4(out[4], out[5], out[6], out[7]);
                            continue;
                        }
                        // a group that the run fills in part: its bytes one by one, the others stay
                        uint8_t* const to = at + ((size_t)g * D + d) * 16;
#pragma unroll 2
                        for (int t = lo; t < hi; ++t) {
                            const uint32_t two = *reinterpret_cast<const uint32_t*>(bits + (t - off) * RP + d);
                            const uint32_t y = kv_bytes2<ODD>(two << 16, two & 0xFFFF0000u, inv);
                            to[t - 16 * g] = (uint8_t)y;
                            to[t - 16 * g + 16] = (uint8_t)(y >> 8);
                        }
                    }
                };
                if (odd) convert(std::true_type{}); else convert(std::false_type{});
            }
            if (tid == 0) *scale = kv_pow2(e);
            __syncthreads();   // the next run reuses the rows
        }
    }
}

}  // namespace tl
