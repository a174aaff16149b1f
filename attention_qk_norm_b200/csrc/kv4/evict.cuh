// evict.cuh -- eviction by accumulated attention weight: the choice of the
// kept rows and their copy to other pages.
// Part of libqknorm.so; included by kv4.cu.
#pragma once

#include "cache.cuh"

namespace {

struct EvictArgs {
    Pool pool;
    float *scores;
    const int32_t *page_table;
    int64_t table_stride, max_pages;
    const int32_t *kv_lens;
    const int32_t *dst_table;
    int64_t dst_stride;
    int64_t B;
    int budget, recent;
    int32_t *new_lens, *kept;
};

__device__ __forceinline__ int evict_len(const EvictArgs &a, int64_t b)
{
    const int64_t most = a.max_pages << a.pool.log2_page;
    const int n = a.kv_lens[b];
    return n < 0 ? 0 : (n > most ? (int)most : n);
}

// A score as a whole number in the same order; NaN is 0, below all others.
__device__ __forceinline__ uint32_t score_key(float s)
{
    const uint32_t u = __float_as_uint(s + 0.f);  // -0 counts as +0
    if (s != s) return 0u;
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

constexpr int kSelectThreads = 512;

__device__ __forceinline__ uint32_t row_key(const EvictArgs &a, const int32_t *table, int hk, int j)
{
    const int64_t page = table[j >> a.pool.log2_page];
    if (!page_ok(a.pool, page)) return 0u;
    const int off = j & ((1 << a.pool.log2_page) - 1);
    return score_key(a.scores[((page * a.pool.Hk + hk) << a.pool.log2_page) + off]);
}

// Exclusive sum of `flag` over the block, and its total.
__device__ __forceinline__ int block_rank(bool flag, int *sums, int &total)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t m = __ballot_sync(0xffffffffu, flag);
    __syncthreads();
    if (lane == 0) sums[warp] = __popc(m);
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
        if (w == warp) before = total;
        total += sums[w];
    }
    return before + __popc(m & ((1u << lane) - 1));
}

// One block per (sequence, head): the k-th largest key by four passes over
// its 8-bit digits, then the kept rows' numbers in order.
__global__ void __launch_bounds__(kSelectThreads) qkn_kv4_select_kernel(EvictArgs a)
{
    __shared__ int hist[256];
    __shared__ int sums[kSelectThreads / 32];
    __shared__ int s_digit, s_left;
    pdl_wait_then_release();
    const int64_t b = blockIdx.x / a.pool.Hk;
    const int hk = (int)(blockIdx.x % a.pool.Hk);
    const int n = evict_len(a, b);
    const int32_t *table = a.page_table + b * a.table_stride;
    int32_t *kept = a.kept + (b * a.pool.Hk + hk) * a.budget;
    const int keep = n < a.budget ? n : a.budget;
    if (hk == 0 && threadIdx.x == 0) a.new_lens[b] = keep;
    if (n <= a.budget) {
        for (int j = threadIdx.x; j < a.budget; j += kSelectThreads) kept[j] = j < n ? j : -1;
        return;
    }
    const int old = n - a.recent;            // rows that compete
    int left = a.budget - a.recent;          // how many of them stay
    uint32_t prefix = 0, mask = 0;
    if (left > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = threadIdx.x; i < 256; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
            for (int j = threadIdx.x; j < old; j += kSelectThreads) {
                const uint32_t key = row_key(a, table, hk, j);
                if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                int d = 255, above = 0;
                while (d > 0 && above + hist[d] < left) above += hist[d--];
                s_digit = d;
                s_left = left - above;
            }
            __syncthreads();
            prefix |= (uint32_t)s_digit << shift;
            mask |= 255u << shift;
            left = s_left;
        }
    } else {
        prefix = 0xffffffffu;
        left = 0;
    }
    // Rows above the border key stay, and the first `left` of those on it.
    int out = 0, ties = 0;
    for (int base = 0; base < n; base += kSelectThreads) {
        const int j = base + threadIdx.x;
        const uint32_t key = j < old ? row_key(a, table, hk, j) : 0u;
        const bool tie = j < old && key == prefix;
        int total;
        const int rank = block_rank(tie, sums, total);
        const bool stay = j < n && (j >= old || key > prefix || (tie && ties + rank < left));
        ties += total;
        const int at = block_rank(stay, sums, total);
        if (stay) kept[out + at] = j;
        out += total;
    }
}

// Copies of the kept rows: D/16 lanes to a row, a lane copies 16 bytes of its
// codes (half the lanes K, half V), and the first three the parameters and
// the score.
template <int D>
__global__ void __launch_bounds__(256) qkn_kv4_move_kernel(EvictArgs a)
{
    constexpr int kLanes = D / 16;
    pdl_wait_then_release();
    const int64_t rows = a.B * a.pool.Hk * a.budget;
    const int lane = threadIdx.x % kLanes;
    const int mask = (1 << a.pool.log2_page) - 1;
    for (int64_t r = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / kLanes; r < rows;
         r += (int64_t)gridDim.x * blockDim.x / kLanes) {
        const int src = a.kept[r];
        if (src < 0) continue;
        const int64_t item = r / a.budget;
        const int dst = (int)(r - item * a.budget);
        const int64_t b = item / a.pool.Hk;
        const int hk = (int)(item - b * a.pool.Hk);
        const int64_t from = a.page_table[b * a.table_stride + (src >> a.pool.log2_page)];
        const int64_t to = a.dst_table[b * a.dst_stride + (dst >> a.pool.log2_page)];
        if (!page_ok(a.pool, from) || !page_ok(a.pool, to)) {
            if (lane == 0) atomicAdd(&g_kv4_bad_pages, 1u);
            continue;
        }
        const int so = src & mask, to_off = dst & mask;
        const uint8_t *sb = a.pool.base + from * a.pool.page_bytes +
                            (int64_t)hk * a.pool.head_bytes + so / kBlockRows * kBlockBytes<D>;
        uint8_t *db = a.pool.base + to * a.pool.page_bytes + (int64_t)hk * a.pool.head_bytes +
                      to_off / kBlockRows * kBlockBytes<D>;
        const int sr = so % kBlockRows, dr = to_off % kBlockRows;
        const int kv = lane / (kLanes / 2), part = lane % (kLanes / 2);
        const int at = kv * 8 * D + part * 16;
        const uint4 codes = *reinterpret_cast<const uint4 *>(sb + at + sr * (D / 2));
        uint32_t word = 0;
        if (lane < 2)
            word = *reinterpret_cast<const uint32_t *>(sb + 16 * D + lane * 64 + sr * 4);
        else if (lane == 2)
            word = __float_as_uint(
                a.scores[((from * a.pool.Hk + hk) << a.pool.log2_page) + so]);
        *reinterpret_cast<uint4 *>(db + at + dr * (D / 2)) = codes;
        if (lane < 2)
            *reinterpret_cast<uint32_t *>(db + 16 * D + lane * 64 + dr * 4) = word;
        else if (lane == 2)
            a.scores[((to * a.pool.Hk + hk) << a.pool.log2_page) + to_off] = __uint_as_float(word);
    }
}

}  // namespace
