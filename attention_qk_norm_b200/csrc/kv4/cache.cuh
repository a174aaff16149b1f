// cache.cuh -- the 4-bit key/value cache's layout, the append kernel (per-head
// QK-Norm with the cache store as its epilogue) and the read-back kernel.
// Part of libqknorm.so; included by kv4.cu.
#pragma once

#include "../storage.cuh"

namespace {

// Where things lie in a pool (include/qknorm_kv4.h).
struct Pool {
    uint8_t *base;
    int64_t pages;
    int64_t page_bytes;  // one page, all heads
    int head_bytes;      // one page of one head
    int log2_page;       // page_size = 1 << log2_page
    int Hk;
};

constexpr int kBlockRows = 16;
template <int D>
constexpr int kBlockBytes = 16 * D + 128;

// Pages and slots outside the pool that kernels met.
__device__ unsigned int g_kv4_bad_pages;

__device__ __forceinline__ bool page_ok(const Pool &pool, int64_t page)
{
    return page >= 0 && page < pool.pages;
}

// ------------------------------------------------------------- row format --
// The held form of a row of fp32 values spread over kWidth lanes of a
// sub-warp, kN to a lane: its codes, and the step and middle before the row's
// factor.  Every operation rounds on its own (no contraction into fma), so
// that the codes are those of the header's formula bit for bit.
struct RowParams {
    float step, mid;
};

template <int kWidth, int kN>
__device__ __forceinline__ RowParams row_params(const float (&y)[kN])
{
    float lo = y[0], hi = y[0];
    bool finite = true;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
        lo = fminf(lo, y[e]);
        hi = fmaxf(hi, y[e]);
        finite = finite && fabsf(y[e]) <= 3.402823466e38f;
    }
    // A row that is not finite spreads as NaN through the two shuffles.
    int bad = finite ? 0 : 1;
#pragma unroll
    for (int o = kWidth / 2; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    }
    RowParams p;
    p.step = __fmul_rn(__fsub_rn(__fmul_rn(hi, 0.5f), __fmul_rn(lo, 0.5f)), 2.0f / 15.0f);
    if (p.step < 1.17549435e-38f) p.step = 0.f;
    p.mid = fmaf(8.f, p.step, lo);  // 8 * step is exact, but may not fit fp32 by itself
    if (bad) p.step = p.mid = __int_as_float(0x7fffffff);
    return p;
}

// Eight codes in one word, element 0 in the lowest nibble.
__device__ __forceinline__ uint32_t row_code(float y, const RowParams &p, float inv)
{
    float c = rintf(__fmul_rn(__fsub_rn(y, p.mid), inv));
    c = fminf(fmaxf(c, -8.f), 7.f);  // NaN becomes -8
    return (uint32_t)((int)c + 8);
}

// {scale, mid} as stored: bf16 each, scale in the low half.
__device__ __forceinline__ uint32_t pack_params(float scale, float mid)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(scale, mid);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void unpack_params(uint32_t w, float &scale, float &mid)
{
    scale = __uint_as_float(w << 16);
    mid = __uint_as_float(w & 0xffff0000u);
}

// ----------------------------------------------------------------- append --
constexpr int kAppendThreads = 256;

// One sub-warp holds a (token, head) row, as in the per-head QK-Norm kernel,
// and visits rows with a grid stride, kAppendRows at a time in flight.  A row
// is read once: its sum of squares, its extremes and its codes all come from
// the same registers.  kNorm: heads [0, Hq) queries, [Hq, Hq+Hk) keys, both
// normalised in place, then values; otherwise the rows are the key and value
// heads alone and nothing is written back.
template <typename TS, int D, bool kNorm>
__global__ void __launch_bounds__(kAppendThreads)
qkn_kv4_append_kernel(TS *__restrict__ qkv, int64_t row_stride, int64_t T, int Hq, int Hk,
                      const float *__restrict__ gamma_q, const float *__restrict__ gamma_k,
                      float eps, const int64_t *__restrict__ slots, Pool pool,
                      float *__restrict__ scores)
{
    using S = Storage<TS>;
    constexpr int kVec = S::kVec;
    constexpr int kNV = D / kVec;
    constexpr int kLPR = kNV < 32 ? kNV : 32;
    constexpr int kVPL = kNV / kLPR;
    constexpr int kEPL = kVPL * kVec;
    constexpr bool kPacked = kVec == 16;  // the per-head kernel's order of sums
    pdl_wait_then_release();

    const int heads = kNorm ? Hq + 2 * Hk : 2 * Hk;
    const int first = kNorm ? 0 : Hq;
    const uint64_t tid = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int lane = (int)(tid % kLPR);
    const uint64_t groups = (uint64_t)gridDim.x * blockDim.x / kLPR;
    const uint64_t rows = (uint64_t)T * heads;
    int64_t t = (int64_t)((tid / kLPR) / heads);
    int h = (int)((tid / kLPR) - (uint64_t)t * heads) + first;
    const int64_t dt = (int64_t)(groups / heads);
    const int dh = (int)(groups - (uint64_t)dt * heads);

    // Whole warps take each step together (the shuffles need every lane).
    for (uint64_t base = 0; base < rows; base += groups) {
        const bool live = t < T;
        const bool is_q = kNorm && h < Hq;
        const bool is_v = h >= Hq + Hk;
        uint4 *ptr = reinterpret_cast<uint4 *>(qkv + t * row_stride + (int64_t)h * D) + lane;
        float f[kVPL][kVec];
#pragma unroll
        for (int v = 0; v < kVPL; ++v)
            S::unpack(live ? load_stream(ptr + v * kLPR) : zero_vec<uint4>(), f[v]);
        float rinv = 1.f;
        float y[kEPL];
#pragma unroll
        for (int v = 0; v < kVPL; ++v)
#pragma unroll
            for (int e = 0; e < kVec; ++e) y[v * kVec + e] = f[v][e];
        if constexpr (kNorm) {
            float s = 0.f;
            if constexpr (kPacked) {
                uint64_t acc = f2_pack(0.f, 0.f);
#pragma unroll
                for (int v = 0; v < kVPL; ++v) sumsq_acc(acc, f[v]);
                s = sumsq_total(acc);
            } else {
#pragma unroll
                for (int v = 0; v < kVPL; ++v)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) s = fmaf(f[v][e], f[v][e], s);
            }
            s = group_sum<kLPR>(s);
            if (!is_v) {
                rinv = rsqrtf(s / (float)D + eps);
                const float *gamma = is_q ? gamma_q : gamma_k;
#pragma unroll
                for (int v = 0; v < kVPL; ++v) {
                    float g[kVec], o[kVec];
                    load_gamma<kVec>(gamma + (lane + v * kLPR) * kVec, g);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        o[e] = __fmul_rn(__fmul_rn(f[v][e], rinv), g[e]);
                        y[v * kVec + e] = __fmul_rn(f[v][e], g[e]);
                    }
                    if (live) store_stream(ptr + v * kLPR, S::pack(o));
                }
            }
        }
        // Extremes over the sub-warp: every lane takes part, query rows too.
        RowParams p = row_params<kLPR, kEPL>(y);
        if (live && !is_q) {
            const int64_t slot = slots[t];
            const int64_t page = slot >> pool.log2_page;
            if (slot >= 0 && page < pool.pages) {
                const int kv = is_v ? 1 : 0;
                const int hk = h - Hq - kv * Hk;
                const int off = (int)(slot & ((1 << pool.log2_page) - 1));
                uint8_t *blk = pool.base + page * pool.page_bytes +
                               (int64_t)hk * pool.head_bytes +
                               (off / kBlockRows) * kBlockBytes<D>;
                const int row = off % kBlockRows;
                const float inv = p.step > 0.f ? __fdiv_rn(1.f, p.step) : 0.f;
                uint8_t *codes = blk + kv * 8 * D + row * (D / 2);
#pragma unroll
                for (int v = 0; v < kVPL; ++v) {
                    uint32_t w[(kVec + 7) / 8] = {};
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        w[e / 8] |= row_code(y[v * kVec + e], p, inv) << (4 * (e % 8));
                    uint8_t *at = codes + (lane + v * kLPR) * (kVec / 2);
                    if constexpr (kVec == 4)
                        *reinterpret_cast<uint16_t *>(at) = (uint16_t)w[0];
                    else if constexpr (kVec == 8)
                        *reinterpret_cast<uint32_t *>(at) = w[0];
                    else
                        *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
                }
                if (lane == 0) {
                    *reinterpret_cast<uint32_t *>(blk + 16 * D + kv * 64 + row * 4) =
                        pack_params(p.step * rinv, p.mid * rinv);
                    if (scores != nullptr && kv == 0)
                        scores[((page * pool.Hk + hk) << pool.log2_page) + off] = 0.f;
                }
            } else if (slot >= 0 && lane == 0) {
                atomicAdd(&g_kv4_bad_pages, 1u);
            }
        }
        t += dt;
        h += dh;
        if (h >= heads + first) {
            h -= heads;
            t += 1;
        }
    }
}

// ------------------------------------------------------------------- read --
// One sub-warp per (slot, head, K or V) row: kVec elements of the output type
// to a lane.
template <typename TS, int D>
__global__ void __launch_bounds__(kAppendThreads)
qkn_kv4_read_kernel(Pool pool, const int64_t *__restrict__ slots, int64_t N,
                    TS *__restrict__ k, TS *__restrict__ v, int64_t row_stride)
{
    using S = Storage<TS>;
    constexpr int kVec = S::kVec;
    constexpr int kNV = D / kVec;
    constexpr int kLPR = kNV < 32 ? kNV : 32;
    constexpr int kVPL = kNV / kLPR;
    pdl_wait_then_release();
    const uint64_t tid = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int lane = (int)(tid % kLPR);
    const uint64_t groups = (uint64_t)gridDim.x * blockDim.x / kLPR;
    const uint64_t rows = (uint64_t)N * 2 * pool.Hk;
    for (uint64_t r = tid / kLPR; r < rows; r += groups) {
        const int64_t i = (int64_t)(r / (2 * pool.Hk));
        const int part = (int)(r - (uint64_t)i * 2 * pool.Hk);
        const int kv = part >= pool.Hk ? 1 : 0;
        const int hk = part - kv * pool.Hk;
        TS *out = kv ? v : k;
        if (out == nullptr) continue;
        const int64_t slot = slots[i];
        const int64_t page = slot >> pool.log2_page;
        const bool ok = slot >= 0 && page < pool.pages;
        const int off = (int)(slot & ((1 << pool.log2_page) - 1));
        const uint8_t *blk = pool.base + (ok ? page : 0) * pool.page_bytes +
                             (int64_t)hk * pool.head_bytes + (off / kBlockRows) * kBlockBytes<D>;
        const int row = off % kBlockRows;
        float scale = 0.f, mid = 0.f;
        if (ok)
            unpack_params(*reinterpret_cast<const uint32_t *>(blk + 16 * D + kv * 64 + row * 4),
                          scale, mid);
        else if (slot >= 0 && lane == 0 && hk == 0)
            atomicAdd(&g_kv4_bad_pages, 1u);
        const uint8_t *codes = blk + kv * 8 * D + row * (D / 2);
        uint4 *to = reinterpret_cast<uint4 *>(out + i * row_stride + (int64_t)hk * D);
#pragma unroll
        for (int j = 0; j < kVPL; ++j) {
            uint32_t w[(kVec + 7) / 8] = {};
            const uint8_t *at = codes + (lane + j * kLPR) * (kVec / 2);
            if (ok) {
                if constexpr (kVec == 4) {
                    w[0] = *reinterpret_cast<const uint16_t *>(at);
                } else if constexpr (kVec == 8) {
                    w[0] = *reinterpret_cast<const uint32_t *>(at);
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(at);
                    w[0] = u.x;
                    w[1] = u.y;
                }
            }
            float f[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                f[e] = fmaf(scale, (float)((int)((w[e / 8] >> (4 * (e % 8))) & 15u) - 8), mid);
            store_stream(to + lane + j * kLPR, S::pack(f));
        }
    }
}

}  // namespace
