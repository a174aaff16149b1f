// attention.cuh -- attention over the 4-bit cache.
// Part of libqknorm.so; included by kv4.cu.
#pragma once

#include "cache.cuh"

namespace {

struct AttentionArgs {
    const void *q;
    int64_t T, row_stride, out_stride;
    int Hq, group;  // query heads, and query heads to a key/value head
    Pool pool;
    const int32_t *page_table;
    int64_t table_stride, max_pages;
    const int32_t *kv_lens;
    int B;
    const int32_t *q_starts;
    int max_q;
    float scale;
    void *out;
    float *lse;
    float *row_lse;  // [B][max_q][Hq], in the workspace
    float *scores;
};

// Sequence b's cached rows and query tokens, taken into the ranges the buffers have.
__device__ __forceinline__ int kv_len(const AttentionArgs &a, int b)
{
    const int64_t most = a.max_pages << a.pool.log2_page;
    const int n = a.kv_lens[b];
    return n < 0 ? 0 : (n > most ? (int)most : n);
}
__device__ __forceinline__ void q_range(const AttentionArgs &a, int b, int64_t &start, int &count)
{
    if (a.q_starts == nullptr) {
        start = b;
        count = 1;
        return;
    }
    const int64_t s = a.q_starts[b], e = a.q_starts[b + 1];
    start = s < 0 ? 0 : (s > a.T ? a.T : s);
    const int64_t end = e < start ? start : (e > a.T ? a.T : e);
    count = end - start > a.max_q ? a.max_q : (int)(end - start);
}

template <typename TS>
__device__ __forceinline__ float load_one(const TS *p);
template <>
__device__ __forceinline__ float load_one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float load_one(const __half *p) { return __half2float(*p); }
template <>
__device__ __forceinline__ float load_one(const float *p) { return *p; }
template <>
__device__ __forceinline__ float load_one(const __nv_fp8_e4m3 *p) { return (float)*p; }
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float f) { *p = __float2bfloat16_rn(f); }
__device__ __forceinline__ void store_one(__half *p, float f) { *p = __float2half_rn(f); }
__device__ __forceinline__ void store_one(float *p, float f) { *p = f; }
__device__ __forceinline__ void store_one(__nv_fp8_e4m3 *p, float f) { *p = __nv_fp8_e4m3(f); }

constexpr int kSimpleWarps = 4;

// A row of the cache: lane l's D/32 elements and the row's pair.
template <int D>
__device__ __forceinline__ bool load_row(const AttentionArgs &a, const int32_t *table, int hk,
                                         int kv, int j, int lane, float (&x)[D / 32])
{
    const int64_t page = table[j >> a.pool.log2_page];
    if (!page_ok(a.pool, page)) {
        if (lane == 0) atomicAdd(&g_kv4_bad_pages, 1u);
        return false;
    }
    const int off = j & ((1 << a.pool.log2_page) - 1);
    const uint8_t *blk = a.pool.base + page * a.pool.page_bytes + (int64_t)hk * a.pool.head_bytes +
                         (off / kBlockRows) * kBlockBytes<D>;
    const int row = off % kBlockRows;
    float scale, mid;
    unpack_params(*reinterpret_cast<const uint32_t *>(blk + 16 * D + kv * 64 + row * 4), scale, mid);
    const uint8_t *c = blk + kv * 8 * D + row * (D / 2) + lane * (D / 64);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        x[2 * i] = fmaf(scale, (float)((int)(c[i] & 15) - 8), mid);
        x[2 * i + 1] = fmaf(scale, (float)((int)(c[i] >> 4) - 8), mid);
    }
    return true;
}

// One block per (sequence, query token, query head); each warp takes every
// fourth row with a softmax of its own, and the four are joined at the end.
template <typename TS, int D>
__global__ void __launch_bounds__(kSimpleWarps * 32)
qkn_kv4_attention_kernel(AttentionArgs a)
{
    constexpr int kE = D / 32;
    pdl_wait_then_release();
    const int b = blockIdx.x, i = blockIdx.y, h = blockIdx.z;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int64_t start;
    int count;
    q_range(a, b, start, count);
    if (i >= count) return;
    const int sees = kv_len(a, b) - count + i + 1;
    const int64_t t = start + i;
    const int hk = h / a.group;
    float q[kE], acc[kE] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e)
        q[e] = load_one(static_cast<const TS *>(a.q) + t * a.row_stride + (int64_t)h * D +
                        lane * kE + e);
    const int32_t *table = a.page_table + b * a.table_stride;
    for (int j = warp; j < sees; j += kSimpleWarps) {
        float x[kE];
        if (!load_row<D>(a, table, hk, 0, j, lane, x)) continue;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e) s = fmaf(q[e], x[e], s);
        s = group_sum<32>(s) * a.scale;
        const float top = fmaxf(m, s);
        const float ref = top == -INFINITY ? 0.f : top;
        const float old = expf(m - ref), p = expf(s - ref);
        load_row<D>(a, table, hk, 1, j, lane, x);
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] = fmaf(acc[e], old, p * x[e]);
        l = fmaf(l, old, p);
        m = top;
    }
    __shared__ float part[kSimpleWarps][D + 2];
#pragma unroll
    for (int e = 0; e < kE; ++e) part[warp][lane * kE + e] = acc[e];
    if (lane == 0) {
        part[warp][D] = m;
        part[warp][D + 1] = l;
    }
    __syncthreads();
    float top = -INFINITY;
    for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, part[w][D]);
    const float ref = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w) total += part[w][D + 1] * expf(part[w][D] - ref);
    for (int d = threadIdx.x; d < D; d += kSimpleWarps * 32) {
        float o = 0.f;
        for (int w = 0; w < kSimpleWarps; ++w) o += part[w][d] * expf(part[w][D] - ref);
        store_one(static_cast<TS *>(a.out) + t * a.out_stride + (int64_t)h * D + d,
                  total == 0.f ? 0.f : o / total);
    }
    if (threadIdx.x == 0) {
        const float lse = ref + logf(total);
        if (a.lse != nullptr) a.lse[t * a.Hq + h] = lse;
        a.row_lse[((int64_t)b * a.max_q + i) * a.Hq + h] = lse;
    }
}

// One warp per cached row: its weight under every query row that sees it.
template <typename TS, int D>
__global__ void __launch_bounds__(kSimpleWarps * 32)
qkn_kv4_scores_kernel(AttentionArgs a)
{
    constexpr int kE = D / 32;
    pdl_wait_then_release();
    const int b = blockIdx.x, hk = blockIdx.y;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int64_t start;
    int count;
    q_range(a, b, start, count);
    const int n = kv_len(a, b);
    const int32_t *table = a.page_table + b * a.table_stride;
    for (int j = blockIdx.z * kSimpleWarps + warp; j < n; j += gridDim.z * kSimpleWarps) {
        float x[kE], add = 0.f;
        if (!load_row<D>(a, table, hk, 0, j, lane, x)) continue;
        for (int i = 0; i < count; ++i) {
            if (j >= n - count + i + 1) continue;
            for (int g = 0; g < a.group; ++g) {
                const int h = hk * a.group + g;
                const TS *q = static_cast<const TS *>(a.q) + (start + i) * a.row_stride +
                              (int64_t)h * D + lane * kE;
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < kE; ++e) s = fmaf(load_one(q + e), x[e], s);
                s = group_sum<32>(s) * a.scale;
                add += expf(s - a.row_lse[((int64_t)b * a.max_q + i) * a.Hq + h]);
            }
        }
        const int64_t page = table[j >> a.pool.log2_page];
        const int off = j & ((1 << a.pool.log2_page) - 1);
        if (lane == 0) a.scores[((page * a.pool.Hk + hk) << a.pool.log2_page) + off] += add;
    }
}

}  // namespace
