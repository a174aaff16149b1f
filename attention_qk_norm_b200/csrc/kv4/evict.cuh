// evict.cuh -- eviction by accumulated attention weight: the choice of the
// kept rows and their copy to other pages.
// Part of libqknorm.so; included by kv4.cu.
#pragma once

#include <cooperative_groups.h>

#include "cache.cuh"

namespace {

namespace cg = cooperative_groups;

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

constexpr int kEvictThreads = 512;
// Rows that always stay: above every score's key.
constexpr uint32_t kNewestKey = 0xffffffffu;

__device__ __forceinline__ uint32_t row_key(const EvictArgs &a, const int32_t *table, int hk, int j)
{
    const int64_t page = table[j >> a.pool.log2_page];
    if (!page_ok(a.pool, page)) return 0u;
    const int off = j & ((1 << a.pool.log2_page) - 1);
    return score_key(a.scores[((page * a.pool.Hk + hk) << a.pool.log2_page) + off]);
}

// The copy of kept rows [r0, r1) of one head, source(r) the row that becomes
// row r: a warp to a block of 16 rows where they go, so that the parameters
// and scores are written as whole lines; D/16 lanes to a row's codes, 16 bytes
// each.  The next block's rows are looked up while this one's are under way.
template <int D, typename Source>
__device__ __forceinline__ void move_rows(const EvictArgs &a, int64_t b, int hk, int r0, int r1,
                                          int warp, int warps, Source source)
{
    constexpr int kLanes = D / 16;          // 16-byte pieces of a row's K and V codes
    constexpr int kRows = 32 / kLanes;      // rows of codes a warp copies at once
    constexpr int kTimes = kBlockRows / kRows;
    const int lane = threadIdx.x % 32;
    const int mask = (1 << a.pool.log2_page) - 1;
    const int32_t *table = a.page_table + b * a.table_stride;
    const int32_t *to_table = a.dst_table + b * a.dst_stride;
    uint8_t *head = a.pool.base + (int64_t)hk * a.pool.head_bytes;
    const int piece = lane % kLanes;  // K's pieces of a row, then V's
    const int code_at = piece / (kLanes / 2) * 8 * D + piece % (kLanes / 2) * 16;
    // Lane l looks row l % 16 of a block up: its page (-1: none) and place.
    int page, off, to;
    const auto look = [&](int blk) {
        const int r = blk * kBlockRows + lane % kBlockRows;
        page = to = -1;
        off = 0;
        if (blk * kBlockRows >= r1) return;
        to = to_table[blk * kBlockRows >> a.pool.log2_page];
        if (r >= r0 && r < r1) {
            const int src = source(r);
            page = table[src >> a.pool.log2_page];
            off = src & mask;
        }
    };
    int blk = r0 / kBlockRows + warp;
    look(blk);
    for (; blk * kBlockRows < r1; blk += warps) {
        const bool there = blk * kBlockRows + lane % kBlockRows >= r0 &&
                           blk * kBlockRows + lane % kBlockRows < r1;
        if (there && lane < kBlockRows && !(page_ok(a.pool, page) && page_ok(a.pool, to)))
            atomicAdd(&g_kv4_bad_pages, 1u);
        const int dst = to, from = page_ok(a.pool, page) && page_ok(a.pool, to) ? page : -1;
        const int from_off = off;
        uint4 codes[kTimes];
        uint32_t have = 0;
#pragma unroll
        for (int i = 0; i < kTimes; ++i) {
            const int p = __shfl_sync(0xffffffffu, from, i * kRows + lane / kLanes);
            const int o = __shfl_sync(0xffffffffu, from_off, i * kRows + lane / kLanes);
            if (p >= 0) {
                have |= 1u << i;
                codes[i] = *reinterpret_cast<const uint4 *>(
                    head + p * a.pool.page_bytes + o / kBlockRows * kBlockBytes<D> + code_at +
                    o % kBlockRows * (D / 2));
            }
        }
        uint32_t par = 0;
        float score = 0.f;
        if (from >= 0) {
            par = *reinterpret_cast<const uint32_t *>(
                head + from * a.pool.page_bytes + from_off / kBlockRows * kBlockBytes<D> + 16 * D +
                lane / kBlockRows * 64 + from_off % kBlockRows * 4);
            if (lane < kBlockRows)
                score = a.scores[(((int64_t)from * a.pool.Hk + hk) << a.pool.log2_page) + from_off];
        }
        look(blk + warps);
        const int dst_off = blk * kBlockRows & mask;
        uint8_t *db = head + dst * a.pool.page_bytes + dst_off / kBlockRows * kBlockBytes<D>;
#pragma unroll
        for (int i = 0; i < kTimes; ++i)
            if (have >> i & 1u)
                *reinterpret_cast<uint4 *>(db + code_at + (i * kRows + lane / kLanes) * (D / 2)) =
                    codes[i];
        if (from >= 0) {
            *reinterpret_cast<uint32_t *>(db + 16 * D + lane * 4) = par;
            if (lane < kBlockRows)
                a.scores[(((int64_t)dst * a.pool.Hk + hk) << a.pool.log2_page) + dst_off + lane] =
                    score;
        }
    }
}

// One cluster per (sequence, head).  Its blocks hold equal runs of the rows'
// keys in shared memory.  The border (the budget-th largest key) is found in
// three digits of 11, 11 and 10 bits: each block counts its keys by digit, and
// each adds a share of the bins up over the blocks.  (Counting the keys at or above
// three candidates, two bits at a time and sixteen rounds, measured 110 us for
// 64 sequences x 8 heads of up to 8192 rows where the digits measured 85.)
// Then each block knows how many of its rows stay and how many stay before
// them, lists its rows in place of their keys, and copies them.
constexpr int kBins = 2048;

// Words from one thread's keys to the next's: `each`, made an odd number of
// 16-byte steps so that eight lanes' loads fall on different banks.
__host__ __device__ __forceinline__ int key_stride(int each) { return each % 8 == 0 ? each + 4 : each; }

// kCluster: more than one block, each with an SM to itself and registers to
// match; else two to an SM, whose counting and copying overlap.  (256 threads
// and four blocks to an SM measured 115 us, 512 and three 119, with 1024 in a
// cluster 88 us for 2 sequences of 131072 where 512 measured 63.)
template <int D, bool kCluster>
__global__ void __launch_bounds__(kEvictThreads, 2)
qkn_kv4_evict_kernel(const EvictArgs a)
{
    constexpr int kWarpsOf = kEvictThreads / 32;
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ __align__(16) int hist[kBins];  // this block's counts of one digit
    __shared__ __align__(16) int sums[kCluster ? kBins / 2 : 1];  // the cluster's, this block's bins
    __shared__ int warp_gt[kWarpsOf], warp_eq[kWarpsOf];
    __shared__ int block_gt, block_eq, s_digit, s_left;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = kCluster ? (int)cluster.num_blocks() : 1;
    const int rank = kCluster ? (int)cluster.block_rank() : 0;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    for (int i = tid; i < kBins; i += kEvictThreads) hist[i] = 0;
    pdl_wait_then_release();

    const int64_t item = blockIdx.x / blocks;
    const int64_t b = item / a.pool.Hk;
    const int hk = (int)(item - b * a.pool.Hk);
    const int n = evict_len(a, b);
    const int32_t *table = a.page_table + b * a.table_stride;
    int32_t *kept = a.kept + item * a.budget;
    const int keep = n < a.budget ? n : a.budget;
    if (hk == 0 && rank == 0 && tid == 0) a.new_lens[b] = keep;
    for (int j = keep + rank * kEvictThreads + tid; j < a.budget; j += blocks * kEvictThreads)
        kept[j] = -1;
    if (n <= a.budget) {  // all stay; the same for every block of the cluster
        const int per = ((n + blocks - 1) / blocks + 15) / 16 * 16;
        const int r0 = min(n, rank * per), r1 = min(n, r0 + per);
        for (int j = r0 + tid; j < r1; j += kEvictThreads) kept[j] = j;
        move_rows<D>(a, b, hk, r0, r1, warp, kWarpsOf, [](int r) { return r; });
        return;
    }

    // This block's rows, four to a load; a thread's share is `each` in a row.
    const int each = ((n + blocks * kEvictThreads - 1) / (blocks * kEvictThreads) + 3) / 4 * 4;
    const int stride = key_stride(each);
    const int r0 = min(n, rank * each * kEvictThreads);
    const int old = n - a.recent;
#pragma unroll 4
    for (int i = tid * 4; i < each * kEvictThreads; i += kEvictThreads * 4) {
        const int j = r0 + i;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        bool ok = false;
        if (j < n) {
            const int64_t page = table[j >> a.pool.log2_page];
            ok = page_ok(a.pool, page);
            if (ok)
                s = *reinterpret_cast<const float4 *>(
                    a.scores + ((page * a.pool.Hk + hk) << a.pool.log2_page) +
                    (j & ((1 << a.pool.log2_page) - 1)));
        }
        const float f[4] = {s.x, s.y, s.z, s.w};
        uint32_t k[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            k[e] = j + e >= n ? 0u : (j + e >= old ? kNewestKey : (ok ? score_key(f[e]) : 0u));
        const int owner = i / each;
        *reinterpret_cast<uint4 *>(keys + owner * stride + (i - owner * each)) =
            make_uint4(k[0], k[1], k[2], k[3]);
    }
    __syncthreads();

    // Rows behind the last have key 0 too, but sit behind every row of key 0,
    // and there are budget rows before them.
    const uint32_t *mine = keys + tid * stride;
    uint32_t border = 0;
    int left = a.budget;  // how many of the keys that share the border's digits so far stay
#pragma unroll
    for (int digit = 0; digit < 3; ++digit) {
        const int shift = digit == 0 ? 21 : (digit == 1 ? 10 : 0);
        const uint32_t bins = digit == 2 ? 1023u : 2047u;
        const uint32_t mask = digit == 0 ? 0u : (digit == 1 ? 0xffe00000u : 0xfffffc00u);
        for (int i = 0; i < each; i += 4) {
            const uint4 k = *reinterpret_cast<const uint4 *>(mine + i);
            if ((k.x & mask) == border) atomicAdd(&hist[k.x >> shift & bins], 1);
            if ((k.y & mask) == border) atomicAdd(&hist[k.y >> shift & bins], 1);
            if ((k.z & mask) == border) atomicAdd(&hist[k.z >> shift & bins], 1);
            if ((k.w & mask) == border) atomicAdd(&hist[k.w >> shift & bins], 1);
        }
        __syncthreads();
        // Four bins to a thread, the highest first.
        const int bin = kBins - 4 - 4 * tid;
        int4 c = *reinterpret_cast<const int4 *>(&hist[bin]);
        if constexpr (kCluster) {
            // Each block adds up an equal share of the bins, and reads the others'.
            const int share = kBins / blocks;
            cluster.sync();
            for (int i = tid * 4; i < share; i += kEvictThreads * 4) {
                int4 x = make_int4(0, 0, 0, 0);
#pragma unroll 8
                for (int r = 0; r < blocks; ++r) {
                    const int4 y = *reinterpret_cast<const int4 *>(
                        cluster.map_shared_rank(&hist[rank * share + i], r));
                    x.x += y.x;
                    x.y += y.y;
                    x.z += y.z;
                    x.w += y.w;
                }
                *reinterpret_cast<int4 *>(&sums[i]) = x;
            }
            cluster.sync();
            c = *reinterpret_cast<const int4 *>(
                cluster.map_shared_rank(&sums[bin % share], bin / share));
        }
        *reinterpret_cast<int4 *>(&hist[bin]) = make_int4(0, 0, 0, 0);  // for the next digit
        const int own = c.x + c.y + c.z + c.w;
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) warp_gt[warp] = sum;
        __syncthreads();
        int above = sum - own;
#pragma unroll
        for (int w = 0; w < kWarpsOf; ++w)
            if (w < warp) above += warp_gt[w];
        if (above < left && left <= above + own) {  // the border's digit is one of these four
            int d = bin + 3;
            const int four[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (d == bin + 3 - e && above + four[e] < left) {
                    above += four[e];
                    --d;
                }
            s_digit = d;
            s_left = left - above;
        }
        __syncthreads();
        border |= (uint32_t)s_digit << shift;
        left = s_left;
    }
    const int ties = left;  // of the rows on the border, the first ones stay

    // Ranks: rows above and on the border, by thread, warp, block.
    int gt = 0, eq = 0;
    for (int i = 0; i < each; i += 4) {
        const uint4 k = *reinterpret_cast<const uint4 *>(mine + i);
        gt += (k.x > border) + (k.y > border) + (k.z > border) + (k.w > border);
        eq += (k.x == border) + (k.y == border) + (k.z == border) + (k.w == border);
    }
    int gt_sum = gt, eq_sum = eq;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, gt_sum, o);
        const int y = __shfl_up_sync(0xffffffffu, eq_sum, o);
        if (lane >= o) {
            gt_sum += x;
            eq_sum += y;
        }
    }
    if (lane == 31) {
        warp_gt[warp] = gt_sum;
        warp_eq[warp] = eq_sum;
    }
    __syncthreads();
    int gt_before = gt_sum - gt, eq_before = eq_sum - eq, gt_all = 0, eq_all = 0;
#pragma unroll
    for (int w = 0; w < kWarpsOf; ++w) {
        if (w < warp) {
            gt_before += warp_gt[w];
            eq_before += warp_eq[w];
        }
        gt_all += warp_gt[w];
        eq_all += warp_eq[w];
    }
    int gt_blocks = 0, eq_blocks = 0;  // in the blocks before this one
    if constexpr (kCluster) {
        if (tid == 0) {
            block_gt = gt_all;
            block_eq = eq_all;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            gt_blocks += *cluster.map_shared_rank(&block_gt, r);
            eq_blocks += *cluster.map_shared_rank(&block_eq, r);
        }
        cluster.sync();  // no block leaves while another reads its counts
    }
    // The block's kept rows are [first, first + kept_here) of the head's.
    const int first = gt_blocks + min(eq_blocks, ties);
    const int last = gt_blocks + gt_all + min(eq_blocks + eq_all, ties);
    // Which of the thread's rows stay (`each` is at most 80), then their list
    // in place of the keys.
    uint32_t stay[3] = {};
    int e = eq_blocks + eq_before;
    for (int i = 0; i < each; ++i) {
        const uint32_t k = mine[i];
        const bool on = k == border;
        if (k > border || (on && e < ties)) stay[i / 32] |= 1u << (i % 32);
        e += on;
    }
    int at = gt_blocks + gt_before + min(eq_blocks + eq_before, ties) - first;
    __syncthreads();
#pragma unroll
    for (int word = 0; word < 3; ++word)
        for (uint32_t m = stay[word]; m != 0; m &= m - 1)
            keys[at++] = (uint32_t)(r0 + tid * each + word * 32 + __ffs(m) - 1);
    __syncthreads();
    for (int i = tid; i < last - first; i += kEvictThreads) kept[first + i] = (int32_t)keys[i];
    if constexpr (kCluster) {
        // The blocks copy equal shares: the newest rows all stay, and all lie in
        // the last blocks' runs.  (The barrier makes the list visible.)
        cluster.sync();
        const int share = ((a.budget + blocks - 1) / blocks + kBlockRows - 1) / kBlockRows * kBlockRows;
        const int m0 = min(a.budget, rank * share), m1 = min(a.budget, m0 + share);
        move_rows<D>(a, b, hk, m0, m1, warp, kWarpsOf, [&](int r) { return __ldcg(kept + r); });
    } else {
        move_rows<D>(a, b, hk, first, last, warp, kWarpsOf, [&](int r) { return (int)keys[r]; });
    }
}

// Sequences too long for a cluster's shared memory: the same choice by one
// block over the scores in memory, and a copy of its own.
__device__ __forceinline__ int block_rank(bool flag, int *sums, int &total)
{
    // Exclusive sum of `flag` over the block, and its total.
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t m = __ballot_sync(0xffffffffu, flag);
    __syncthreads();
    if (lane == 0) sums[warp] = __popc(m);
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kEvictThreads / 32; ++w) {
        if (w == warp) before = total;
        total += sums[w];
    }
    return before + __popc(m & ((1u << lane) - 1));
}

__global__ void __launch_bounds__(kEvictThreads) qkn_kv4_select_kernel(const EvictArgs a)
{
    __shared__ int hist[256];
    __shared__ int sums[kEvictThreads / 32];
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
        for (int j = threadIdx.x; j < a.budget; j += kEvictThreads) kept[j] = j < n ? j : -1;
        return;
    }
    const int old = n - a.recent;
    int left = a.budget;
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kEvictThreads) hist[i] = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kEvictThreads) {
            const uint32_t key = j < old ? row_key(a, table, hk, j) : kNewestKey;
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
    // Rows above the border key stay, and the first `left` of those on it.
    int out = 0, ties = 0;
    for (int base = 0; base < n; base += kEvictThreads) {
        const int j = base + threadIdx.x;
        const uint32_t key = j < old ? row_key(a, table, hk, j) : kNewestKey;
        const bool tie = j < n && key == prefix;
        int total;
        const int rank = block_rank(tie, sums, total);
        const bool stay = j < n && (key > prefix || (tie && ties + rank < left));
        ties += total;
        const int at = block_rank(stay, sums, total);
        if (stay) kept[out + at] = j;
        out += total;
    }
}

template <int D>
__global__ void __launch_bounds__(kEvictThreads) qkn_kv4_move_kernel(const EvictArgs a)
{
    pdl_wait_then_release();
    const int64_t item = blockIdx.x;
    const int64_t b = item / a.pool.Hk;
    const int n = evict_len(a, b), keep = n < a.budget ? n : a.budget;
    const int32_t *kept = a.kept + item * a.budget;
    const int warps = gridDim.y * (kEvictThreads / 32);
    move_rows<D>(a, b, (int)(item - b * a.pool.Hk), 0, keep,
                 blockIdx.y * (kEvictThreads / 32) + threadIdx.x / 32, warps,
                 [&](int r) { return kept[r]; });
}

}  // namespace
