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
// Work. A unit is (request, KV head); its cached tokens are cut into tiles of 128. The tiles of all
// units form one list, cut into equal contiguous ranges, one for each group of CTAs, so requests of
// unequal lengths fill the GPU evenly. The group's CTAs take a row tile of the unit's rows each (the
// rows of a unit are the request's rows times the query heads of its KV head, row r = i * G + g). The
// part of unit u in range g goes to slot u + g: going along the list, each step moves to the next unit
// or the next range, so no two parts meet.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace tl {

constexpr int KV_TILE = 128;          // cached tokens of a tile
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
    float* part_o;                // [slots][row tiles][NT][D]
    float2* part_ml;              // [slots][row tiles][NT]
    int* err;
    long long q_stride, new_stride, out_stride;
    float scale;                  // c * log2(e)
    int B, width, n_pages, page_log2, heads, group, R, max_rows, groups, row_tiles, nt;
};

// The rows of request b: first row and count (0 where the offsets are invalid).
__device__ __forceinline__ int kv_rows_of(const KvAttnParams& p, int b, int* first, bool* bad) {
    if (!p.row_start) {
        *first = b * p.max_rows;
        return p.max_rows;
    }
    const int r0 = p.row_start[b], r1 = p.row_start[b + 1];
    *first = r0;
    if (r0 < 0 || r1 < r0 || r1 - r0 > p.max_rows || r1 > p.R) {
        *bad = true;
        return 0;
    }
    return r1 - r0;
}

// The cached tokens of request b that its rows attend to (0 if it has no rows).
__device__ __forceinline__ int kv_len_of(const KvAttnParams& p, int b) {
    int first;
    bool bad = false;
    if (kv_rows_of(p, b, &first, &bad) == 0) return 0;
    const long long room = (long long)p.width << p.page_log2;
    const int len = p.lens[b];
    return len < 0 ? 0 : (int)(len < room ? len : room);
}

__device__ __forceinline__ int kv_tiles(int len) { return (int)(((long long)len + KV_TILE - 1) / KV_TILE); }

__device__ __forceinline__ long long kv_range_start(long long g, long long total, long long groups) {
    return g * total / groups;
}

// One step of a walk along a range of the tile list: tiles k0..k1 of unit (b, head).
struct KvSeg {
    int b, head, k0, k1, tiles;
};

struct KvSegIter {
    const int* pre;      // [B + 1] tiles of the requests in front (per head)
    int B, heads, b;
    long long t, end;
    __device__ __forceinline__ KvSegIter(const int* pre_, int B_, int heads_, long long begin, long long end_)
        : pre(pre_), B(B_), heads(heads_), b(0), t(begin), end(end_) {
        if (t < end) b = kv_find(pre, B, (int)(t / heads));
    }
    __device__ __forceinline__ bool next(KvSeg& s) {
        if (t >= end) return false;
        while ((long long)heads * pre[b + 1] <= t) ++b;
        const int tiles = pre[b + 1] - pre[b];
        const long long in = t - (long long)heads * pre[b];
        s.b = b;
        s.tiles = tiles;
        s.head = (int)(in / tiles);
        s.k0 = (int)(in - (long long)s.head * tiles);
        const long long left = end - t;
        s.k1 = (left < tiles - s.k0) ? s.k0 + (int)left : tiles;
        t += s.k1 - s.k0;
        return true;
    }
};

// The simple form of the streaming kernel: fp32 on CUDA cores, one row tile of 16 rows a CTA.
constexpr int KV_SIMT_NT = 16;

template <int D>
__global__ void __launch_bounds__(KV_TILE) kv_attention_kernel(const KvAttnParams p) {
    __shared__ int pre[KV_MAX_BATCH + 1];
    __shared__ float qs[KV_SIMT_NT][D];
    __shared__ float ps[KV_SIMT_NT][KV_TILE];
    __shared__ float red[4][KV_SIMT_NT];
    __shared__ const uint8_t* page_at[KV_TILE / 16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = 1 << p.page_log2;
    for (int b = tid; b < p.B; b += KV_TILE) pre[b + 1] = kv_tiles(kv_len_of(p, b));
    __syncthreads();
    if (tid == 0) {
        pre[0] = 0;
        for (int b = 0; b < p.B; ++b) pre[b + 1] += pre[b];
    }
    __syncthreads();
    const long long total = (long long)p.heads * pre[p.B];
    const long long groups = p.groups < total ? p.groups : total;
    const int g = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
    if (g >= groups) return;
    KvSegIter it(pre, p.B, p.heads, kv_range_start(g, total, groups), kv_range_start(g + 1, total, groups));
    KvSeg s;
    while (it.next(s)) {
        int first;
        bool bad = false;
        const int rows = kv_rows_of(p, s.b, &first, &bad) * p.group;
        const int r0 = rt * p.nt, n_rows = min(rows - r0, p.nt);
        if (n_rows <= 0) continue;
        const int len = kv_len_of(p, s.b);
        for (int e = tid; e < KV_SIMT_NT * D; e += KV_TILE) {
            const int n = e / D, d = e % D;
            float v = 0.0f;
            if (n < n_rows) {
                const int i = (r0 + n) / p.group, gq = (r0 + n) % p.group;
                v = __bfloat162float(p.q[(size_t)(first + i) * p.q_stride + (size_t)(s.head * p.group + gq) * D + d]) * p.scale;
            }
            qs[n][d] = v;
        }
        float o[KV_SIMT_NT], m[KV_SIMT_NT], l[KV_SIMT_NT];
#pragma unroll
        for (int n = 0; n < KV_SIMT_NT; ++n) { o[n] = 0.0f; m[n] = -INFINITY; l[n] = 0.0f; }
        for (int k = s.k0; k < s.k1; ++k) {
            __syncthreads();
            const int t = k * KV_TILE + tid;
            const int blk = min(t, len - 1) >> p.page_log2;
            int page = p.table[(size_t)s.b * p.width + blk];
            if (page < 0 || page >= p.n_pages) {
                atomicCAS(p.err, 0, TL_DEV_ERR_KV_PAGE);
                page = 0;
            }
            const uint8_t* const at = p.pages + ((size_t)page * p.heads + s.head) * 2 * ((size_t)P * D);
            if ((tid & 15) == 0) page_at[tid / 16] = at + (size_t)P * D;
            const float ks = p.scales[((size_t)page * p.heads + s.head) * 2];
            const float vs = p.scales[((size_t)page * p.heads + s.head) * 2 + 1];
            const float lv = log2f(vs);
            float w[KV_SIMT_NT];
#pragma unroll
            for (int n = 0; n < KV_SIMT_NT; ++n) w[n] = 0.0f;
            for (int c = 0; c < D / 16; ++c) {
                const uint4 q4 = *reinterpret_cast<const uint4*>(at + ((size_t)c * P + (t & (P - 1))) * 16);
                const uint32_t in[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const uint32_t h = kv_f16x2((in[u >> 1] >> (16 * (u & 1))) & 0xFFFFu);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
#pragma unroll
                    for (int n = 0; n < KV_SIMT_NT; ++n)
                        w[n] = fmaf(f.y, qs[n][16 * c + 2 * u + 1], fmaf(f.x, qs[n][16 * c + 2 * u], w[n]));
                }
            }
#pragma unroll
            for (int n = 0; n < KV_SIMT_NT; ++n) {
                w[n] = (t < len) ? fmaf(w[n], ks, lv) : -INFINITY;
                float x = w[n];
#pragma unroll
                for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
                if (lane == 0) red[warp][n] = x;
            }
            __syncthreads();
            float alpha[KV_SIMT_NT];
#pragma unroll
            for (int n = 0; n < KV_SIMT_NT; ++n) {
                const float top = fmaxf(m[n], fmaxf(fmaxf(red[0][n], red[1][n]), fmaxf(red[2][n], red[3][n])));
                alpha[n] = (m[n] == -INFINITY) ? 0.0f : exp2f(m[n] - top);
                m[n] = top;
                const float pr = (t < len) ? exp2f(w[n] - top) : 0.0f;
                l[n] = fmaf(l[n], alpha[n], (t < len) ? pr / vs : 0.0f);
                ps[n][tid] = pr;
            }
            __syncthreads();
            if (tid < D) {
#pragma unroll
                for (int n = 0; n < KV_SIMT_NT; ++n) o[n] *= alpha[n];
                const int valid = min(len - k * KV_TILE, KV_TILE);
                for (int c = 0; c < (valid + 15) / 16; ++c) {
                    const int place = (k * KV_TILE + 16 * c) & (P - 1);
                    const uint4 q4 = *reinterpret_cast<const uint4*>(page_at[c] + ((size_t)(place >> 4) * D + tid) * 16);
                    const uint32_t in[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const uint32_t h = kv_f16x2((in[u >> 1] >> (16 * (u & 1))) & 0xFFFFu);
                        float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                        const int at_t = 16 * c + 2 * u;
                        if (at_t >= valid) f.x = 0.0f;
                        if (at_t + 1 >= valid) f.y = 0.0f;
#pragma unroll
                        for (int n = 0; n < KV_SIMT_NT; ++n)
                            o[n] = fmaf(f.y, ps[n][at_t + 1], fmaf(f.x, ps[n][at_t], o[n]));
                    }
                }
            }
        }
        __syncthreads();
        const size_t slot = ((size_t)s.b * p.heads + s.head + g) * p.row_tiles + rt;
#pragma unroll
        for (int n = 0; n < KV_SIMT_NT; ++n) {
            if (n >= n_rows) break;
            float x = l[n];
#pragma unroll
            for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
            if (lane == 0) red[warp][n] = x;
            if (tid < D) p.part_o[(slot * p.nt + n) * D + tid] = o[n];
        }
        __syncthreads();
        if (tid < n_rows)
            p.part_ml[slot * p.nt + tid] = make_float2(0.0f, (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]));
        if (tid == 0)
            for (int n = 0; n < n_rows; ++n) p.part_ml[slot * p.nt + n].x = m[n];
    }
}

// One warp per (row, query head): the scores of the tree nodes that the row sees (a lane a node), their
// softmax and V in fp32, then the parts of the cached tokens, in list order. A node that the mask leaves
// out is never read, so nothing of it (an infinity, a NaN) reaches the row. A row that sees nothing at
// all gives zeros.
constexpr int KV_MERGE_THREADS = 256;

template <int D>
__global__ void __launch_bounds__(KV_MERGE_THREADS) kv_merge_kernel(const KvAttnParams p) {
    constexpr int E = D / 32;                            // channels of a lane
    __shared__ long long sums[2][KV_MERGE_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x;
    int first;
    bool bad = false;
    const int rows = kv_rows_of(p, b, &first, &bad);
    if (bad && tid == 0 && blockIdx.y == 0) atomicCAS(p.err, 0, TL_DEV_ERR_KV_ROWS);
    const int per = blockIdx.y * (KV_MERGE_THREADS / 32) + warp;    // (row, query head) of the request
    if (blockIdx.y * (KV_MERGE_THREADS / 32) >= rows * p.heads * p.group) return;
    // this request's place in the tile list
    long long before = 0, all = 0;
    for (int i = tid; i < p.B; i += KV_MERGE_THREADS) {
        const int n = kv_tiles(kv_len_of(p, i));
        all += n;
        if (i < b) before += n;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
        before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
    }
    if (lane == 0) { sums[0][warp] = all; sums[1][warp] = before; }
    __syncthreads();
    all = before = 0;
#pragma unroll
    for (int u = 0; u < KV_MERGE_THREADS / 32; ++u) { all += sums[0][u]; before += sums[1][u]; }
    const int hq = p.heads * p.group;
    const bool mine = per < rows * hq;
    const int i = mine ? per / hq : 0, h = mine ? per % hq : 0, head = h / p.group;
    const int row = first + i;

    float m = -INFINITY, l = 0.0f;
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    if (mine && p.k_new) {
        unsigned bits = p.mask ? p.mask[row] : (2u << i) - 1u;
        if (rows < 32) bits &= (1u << rows) - 1u;
        float s = -INFINITY;
        if ((bits >> lane) & 1u) {
            const uint4* const kr = reinterpret_cast<const uint4*>(p.k_new + (size_t)(first + lane) * p.new_stride + (size_t)head * D);
            const uint4* const qr = reinterpret_cast<const uint4*>(p.q + (size_t)row * p.q_stride + (size_t)h * D);
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint4 a = __ldg(kr + c), w = __ldg(qr + c);
                const uint32_t ka[4] = {a.x, a.y, a.z, a.w}, qa[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    acc[u] = fmaf(__int_as_float((int)(ka[u] & 0xFFFF0000u)), __int_as_float((int)(qa[u] & 0xFFFF0000u)),
                                  fmaf(__int_as_float((int)(ka[u] << 16)), __int_as_float((int)(qa[u] << 16)), acc[u]));
            }
            s = ((acc[0] + acc[1]) + (acc[2] + acc[3])) * p.scale;
        }
        float top = s;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const float pr = ((bits >> lane) & 1u) ? exp2f(s - top) : 0.0f;
        float sum = pr;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (bits) { m = top; l = sum; }
        for (unsigned todo = bits; todo; todo &= todo - 1) {
            const int j = __ffs(todo) - 1;
            const float w = __shfl_sync(0xFFFFFFFFu, pr, j);
            const __nv_bfloat16* const vr = p.v_new + (size_t)(first + j) * p.new_stride + (size_t)head * D + E * lane;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const uint32_t x = __ldg(reinterpret_cast<const unsigned*>(vr + e));
                o[e] = fmaf(w, __int_as_float((int)(x << 16)), o[e]);
                o[e + 1] = fmaf(w, __int_as_float((int)(x & 0xFFFF0000u)), o[e + 1]);
            }
        }
    }
    // the parts of the cached tokens
    const int len = kv_len_of(p, b);
    if (!mine) return;
    if (len > 0) {
        const int tiles = kv_tiles(len);
        const long long total = (long long)p.heads * all, groups = p.groups < total ? p.groups : total;
        const long long a = (long long)p.heads * before + (long long)head * tiles, z = a + tiles;
        const int g0 = (int)(((a + 1) * groups - 1) / total), g1 = (int)((z * groups - 1) / total);
        const int r = i * p.group + h % p.group, rt = r / p.nt, n = r % p.nt;
        for (int g = g0; g <= g1; ++g) {
            const size_t at = (((size_t)b * p.heads + head + g) * p.row_tiles + rt) * p.nt + n;
            const float2 ml = __ldcg(p.part_ml + at);
            const float top = fmaxf(m, ml.x);
            // a part or tree without weight (m of minus infinity) counts nothing
            const float f0 = (m == -INFINITY) ? 0.0f : exp2f(m - top), f1 = (ml.x == -INFINITY) ? 0.0f : exp2f(ml.x - top);
            m = top;
            l = l * f0 + ml.y * f1;
            const float* const po = p.part_o + at * D + E * lane;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 x = __ldcg(reinterpret_cast<const float2*>(po + e));
                o[e] = o[e] * f0 + x.x * f1;
                o[e + 1] = o[e + 1] * f0 + x.y * f1;
            }
        }
    }
    const float inv = (m == -INFINITY && l == 0.0f) ? 0.0f : 1.0f / l;
    __nv_bfloat16* const to = p.out + (size_t)row * p.out_stride + (size_t)h * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<__nv_bfloat162*>(to + e) = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
}

}  // namespace tl
