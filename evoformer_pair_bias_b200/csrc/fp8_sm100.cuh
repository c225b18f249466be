// fp8_sm100.cuh -- the product of two e4m3 matrices with a scale per block of 128
// along the summed axis, on tcgen05:
//
//   y[r,o] = sum_b sx[r,b] * sw[o,b] * (sum_{k in b} x[r,k] w[o,k]) + bias[o]
//
// sx has one scale per row and block; sw one per 128 x 128 block (SW_ROWS = false,
// a layer's weight) or one per row and block (SW_ROWS = true, the operands of a
// weight's gradient).  The scales are any fp32 numbers, so they cannot enter the
// tensor core's own block scaling (powers of two): every block's product leaves
// TMEM once and is added, scaled, into fp32 registers, while the tensor core
// works on the next block in the other half of TMEM.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "sm100.cuh"
#include "tma_maps.cuh"

namespace evo {
namespace fp8 {

using namespace evo::sm100;

constexpr int BM = 128;            // rows of y a tile
constexpr int BK = 128;            // one scale block of the summed axis: 128 bytes, one swizzle span
enum : unsigned int { kLinTimeout = 0x5000u };

struct LinParams {
    int M, N, K;                   // y [M, N], summed axis K
    const void *x, *w;             // codes, for the tensor maps
    int64_t ldx, ldw;
    const float* sx;               // [M, K/128] with strides
    int64_t sx_row, sx_grp;
    const float* sw;               // [N or N/128, K/128] with strides
    int64_t sw_row, sw_grp;
    const float* bias;             // [N] or null
    void* y;                       // bf16 or fp32 [M, N]
    int64_t ldy;
};

// kind::f8f6f4, e4m3 x e4m3 -> fp32, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}
// ---------------------------------------------------------------- split kernel
// One 128 x 128 tile of y per cluster; the S CTAs of the cluster each sum a run of
// blocks, and join their fp32 results through distributed shared memory in rank
// order (the same bits on every run, one launch, no workspace).  S = 1 where there
// are tiles enough.  Roles: warp 0 TMA, warp 1 MMA, warps 4-11 add up the blocks
// (warp % 4 is the quarter of TMEM lanes a warp may read, (warp - 4) / 4 its half
// of the 128 columns).
namespace split {

constexpr int BN = 128;
constexpr int STAGES = 6;
constexpr int STAGE_BYTES = (BM + BN) * BK;
constexpr int THREADS = 384;
constexpr int SWB_OFF = STAGES * STAGE_BYTES;              // 64 column scales for each of 8 warps
constexpr int BAR_OFF = SWB_OFF + 8 * 64 * 4;
constexpr int MISC_OFF = BAR_OFF + (2 * STAGES + 5) * 8;
constexpr int SMEM = MISC_OFF + 16 + 1024;
static_assert(STAGES * STAGE_BYTES >= BM * BN * 4, "the joined tile lies over the stages");
static_assert(SMEM <= 232448, "shared memory budget");

// float4 chunk `ch` of row `r` of the fp32 tile: chunks permuted by the row, so that lanes
// holding one chunk of 32 rows, or 32 chunks of one row, meet different banks
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int r, int ch) {
    return base + (uint32_t)(r * 512 + ((ch ^ (r & 31)) << 4));
}

template <typename T, bool SW_ROWS>
__global__ void __launch_bounds__(THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                  const LinParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int tile = (int)(blockIdx.x / S), tn = (p.N + BN - 1) / BN;
    const int m0 = tile / tn * BM, n0 = tile % tn * BN;
    const int kb_all = (p.K + BK - 1) / BK;
    const int kb0 = (int)((int64_t)kb_all * rank / S), kb1 = (int)((int64_t)kb_all * (rank + 1) / S);
    auto bar_full = [&](int i) { return base + BAR_OFF + 8u * i; };
    auto bar_empty = [&](int i) { return base + BAR_OFF + 8u * (STAGES + i); };
    auto bar_accf = [&](int b) { return base + BAR_OFF + 8u * (2 * STAGES + b); };
    auto bar_acce = [&](int b) { return base + BAR_OFF + 8u * (2 * STAGES + 2 + b); };
    const uint32_t bar_done = base + BAR_OFF + 8u * (2 * STAGES + 4);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + MISC_OFF + 4);

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(bar_full(i), 1);
            mbar_init(bar_empty(i), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_accf(b), 1);
            mbar_init(bar_acce(b), 8);
        }
        mbar_init(bar_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(base + MISC_OFF, 2 * BN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    float acc[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0.f;
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row = 32 * quarter + lane;                   // of the tile

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&tm_x);
            prefetch_tmap(&tm_w);
            bool ok = true;
            int n = 0;
            for (int kb = kb0; ok && kb < kb1; ++kb, ++n) {
                const int st = n % STAGES;
                ok = mbar_wait(bar_empty(st), (uint32_t)(((n / STAGES) & 1) ^ 1), abort_flag, kLinTimeout | 0x01);
                if (!ok) break;
                const uint32_t dst = base + st * STAGE_BYTES;
                mbar_arrive_expect_tx(bar_full(st), STAGE_BYTES);
                tma_load_2d(dst, &tm_x, bar_full(st), kb * BK, m0);
                tma_load_2d(dst + BM * BK, &tm_w, bar_full(st), kb * BK, n0);
            }
            // the loads still in flight land before shared memory is released or reused
            volatile int no_abort = 0;
            for (int u = n > STAGES ? n - STAGES : 0; u < n; ++u)
                mbar_wait(bar_full(u % STAGES), (uint32_t)((u / STAGES) & 1), &no_abort, kLinTimeout | 0x02);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t IDESC = idesc_e4m3(BM, BN);
            bool ok = true;
            int n = 0;
            for (int kb = kb0; ok && kb < kb1; ++kb, ++n) {
                const int st = n % STAGES, b = n & 1;
                ok = mbar_wait(bar_acce(b), (uint32_t)(((n >> 1) & 1) ^ 1), abort_flag, kLinTimeout | 0x03);
                if (ok) ok = mbar_wait(bar_full(st), (uint32_t)((n / STAGES) & 1), abort_flag, kLinTimeout | 0x04);
                if (!ok) break;
                tc_fence_after();
                const uint32_t a = base + st * STAGE_BYTES;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f8(tmem + (uint32_t)(b * BN), smem_desc(a + kk * 32, 16, 1024, kSw128),
                           smem_desc(a + BM * BK + kk * 32, 16, 1024, kSw128), IDESC, kk > 0 ? 1u : 0u);
                mma_commit(bar_empty(st));
                mma_commit(bar_accf(b));
            }
            volatile int no_abort = 0;
            mma_commit(bar_done);
            mbar_wait(bar_done, 0, &no_abort, kLinTimeout | 0x05);
        }
    } else if (warp >= 4) {
        const bool live = m0 + row < p.M;
        const float* sx = p.sx + (int64_t)(live ? m0 + row : 0) * p.sx_row;
        // SW_ROWS: lane l fetches the scales of columns l and 32 + l of this warp's 64, and the warp
        // shares them through its own slice of shared memory; else one scale for the whole tile
        const int c_lo = n0 + 64 * half + lane;
        const float* sw = p.sw + (SW_ROWS ? (int64_t)min(c_lo, p.N - 1) : (int64_t)(n0 / 128)) * p.sw_row;
        const float* sw_hi = p.sw + (SW_ROWS ? (int64_t)min(c_lo + 32, p.N - 1) : (int64_t)0) * p.sw_row;
        float* swb = reinterpret_cast<float*>(gbase + SWB_OFF) + 64 * (warp - 4);
        float a_next = 0.f, w_next = 0.f, h_next = 0.f;
        if (kb0 < kb1) {
            a_next = __ldg(sx + kb0 * p.sx_grp);
            w_next = __ldg(sw + kb0 * p.sw_grp);
            if (SW_ROWS) h_next = __ldg(sw_hi + kb0 * p.sw_grp);
        }
        int n = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++n) {
            const int b = n & 1;
            float f = a_next;
            if (SW_ROWS) {
                __syncwarp();                              // the last block's scales have been read
                swb[lane] = w_next;
                swb[32 + lane] = h_next;
                __syncwarp();
            } else {
                f *= w_next;
            }
            if (kb + 1 < kb1) {
                a_next = __ldg(sx + (kb + 1) * p.sx_grp);
                w_next = __ldg(sw + (kb + 1) * p.sw_grp);
                if (SW_ROWS) h_next = __ldg(sw_hi + (kb + 1) * p.sw_grp);
            }
            const bool ok = mbar_wait(bar_accf(b), (uint32_t)((n >> 1) & 1), abort_flag, kLinTimeout | 0x06);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t ta = tmem + (uint32_t)(b * BN + 64 * half) + ((uint32_t)(32 * quarter) << 16);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t v[32];
                tmem_ld32_sync(ta + 32 * c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float t = __uint_as_float(v[i]);
                    if (SW_ROWS) t *= swb[32 * c + i];
                    acc[32 * c + i] = fmaf(t, f, acc[32 * c + i]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_acce(b));
        }
    }
    // every load has landed and every MMA is done: the stages take the fp32 tile
    __syncthreads();
    if (warp >= 4 && m0 + row < p.M) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sts128(tile_addr(base, row, 16 * half + i), __float_as_uint(acc[4 * i]), __float_as_uint(acc[4 * i + 1]),
                   __float_as_uint(acc[4 * i + 2]), __float_as_uint(acc[4 * i + 3]));
    }
    if (S > 1)
        cluster_sync();
    else
        __syncthreads();
    const int rows = min(BM, p.M - m0);
    T* y = static_cast<T*>(p.y);
    const bool vec = p.ldy % 4 == 0 && (reinterpret_cast<uintptr_t>(p.y) & (4 * sizeof(T) - 1)) == 0;
    for (int idx = rank * THREADS + (int)threadIdx.x; idx < rows * 32; idx += S * THREADS) {
        const int r = idx >> 5, ch = idx & 31, c = n0 + 4 * ch;
        if (c >= p.N) continue;
        const uint32_t at = tile_addr(base, r, ch);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < S; ++k) {
            const float4 v = ld_cluster(at, (uint32_t)k);
            o[0] += v.x;
            o[1] += v.y;
            o[2] += v.z;
            o[3] += v.w;
        }
        if (p.bias) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < p.N) o[e] += __ldg(p.bias + c + e);
        }
        T* out = y + (int64_t)(m0 + r) * p.ldy + c;
        if (vec && c + 4 <= p.N) {
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
            else
                *reinterpret_cast<float4*>(out) = make_float4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < p.N) Elem<T>::store(out + e, o[e]);
        }
    }
    tc_fence_before();
    if (S > 1)
        cluster_sync();                                    // peers have read this CTA's tile
    else
        __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 2 * BN);
    }
}

}  // namespace split

// ----------------------------------------------------------------- wide kernel
// Persistent, one CTA per SM, 128 x 256 tiles of y, the columns of a row block in
// succession.  Roles: warp 0 TMA, warp 1 MMA, warp 2 the scales of the coming blocks
// and warp 3 the bias of the coming tile (cp.async into shared memory), warps 4-11
// add up the blocks and write the tile (warp % 4: the quarter of TMEM lanes;
// (warp - 4) / 4: the half of the 256 columns, one scale block of w).  While they write
// a tile, the next tile's first two blocks are multiplied.  y leaves through boxes of
// 32 rows in shared memory: by TMA where y's rows are 16-byte aligned, else by the
// warp, a row at a time.
//
// The summing warps hold 128 sums each and nothing that comes from global memory:
// scales or bias fetched into their own registers spilled, and waited for the load
// at the spill (131072 x 256 x 1024: 107-125 us, against TODO us).
namespace wide {

constexpr int BN = 256;
constexpr int STAGE_BYTES = (BM + BN) * BK;
constexpr int SUM_WARPS = 16;                              // 4 column groups x 4 lane quarters
constexpr int COLS = 4 * BN / SUM_WARPS;                   // columns a summing warp holds
constexpr int THREADS = 32 * (4 + SUM_WARPS);
constexpr int RING = 8;                                    // blocks whose scales are held
constexpr int SLOT = (BM + BN) * 4;                        // 128 scales of x, then 2 or 256 of w
// Shared memory: S stages, X boxes of 32 rows x BB bytes for each summing warp.
template <int S, int X, int BB>
struct Layout {
    static constexpr int stages = S, boxes = X, box_cols = BB, box = 32 * BB;
    static constexpr int stg_off = S * STAGE_BYTES;
    static constexpr int ring_off = stg_off + SUM_WARPS * X * box;
    static constexpr int bias_off = ring_off + RING * SLOT;
    static constexpr int bar_off = bias_off + 2 * BN * 4;
    static constexpr int n_bars = 2 * S + 2 * RING + 4 + 4 + 1;
    static constexpr int misc_off = bar_off + n_bars * 8;
    static constexpr int smem = misc_off + 16 + 1024;
    static_assert(smem <= 232448, "shared memory budget");
};
using Short = Layout<3, 1, 128>;
// registers per thread: 96 at launch (20 warps), handed from the control warps to the others
constexpr int LAUNCH_REGS = 96, CTRL_REGS = 32, SUM_REGS = 112;
static_assert(4 * CTRL_REGS + SUM_WARPS * SUM_REGS <= (4 + SUM_WARPS) * LAUNCH_REGS, "register split");

__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` (which counts the arriving threads) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T, bool SW_ROWS, class L>
__global__ void __launch_bounds__(THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                  const __grid_constant__ CUtensorMap tm_y, const LinParams p, const int tma_out) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    constexpr int STAGES = L::stages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tn = (p.N + BN - 1) / BN, tiles = (p.M + BM - 1) / BM * tn;
    const int nkb = (p.K + BK - 1) / BK;
    auto bar = [&](int i) { return base + L::bar_off + 8u * i; };
    auto bar_full = [&](uint32_t i) { return bar(i); };
    auto bar_empty = [&](uint32_t i) { return bar(STAGES + i); };
    auto bar_sfull = [&](uint32_t i) { return bar(2 * STAGES + i); };
    auto bar_sempty = [&](uint32_t i) { return bar(2 * STAGES + RING + i); };
    auto bar_accf = [&](uint32_t b) { return bar(2 * STAGES + 2 * RING + b); };
    auto bar_acce = [&](uint32_t b) { return bar(2 * STAGES + 2 * RING + 2 + b); };
    auto bar_bfull = [&](uint32_t b) { return bar(2 * STAGES + 2 * RING + 4 + b); };
    auto bar_bempty = [&](uint32_t b) { return bar(2 * STAGES + 2 * RING + 6 + b); };
    const uint32_t bar_done = bar(2 * STAGES + 2 * RING + 8);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + L::misc_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::misc_off + 4);

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(bar_full(i), 1);
            mbar_init(bar_empty(i), 1);
        }
        for (int i = 0; i < RING; ++i) {
            mbar_init(bar_sfull(i), 32);
            mbar_init(bar_sempty(i), SUM_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_accf(b), 1);
            mbar_init(bar_acce(b), SUM_WARPS);
            mbar_init(bar_bfull(b), 32);
            mbar_init(bar_bempty(b), SUM_WARPS);
        }
        mbar_init(bar_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(base + L::misc_off, 2 * BN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        regs_decrease<CTRL_REGS>();
        bool ok = true;
        uint32_t n = 0;
        if (warp == 0 && lane == 0) {
            prefetch_tmap(&tm_x);
            prefetch_tmap(&tm_w);
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const int m0 = t / tn * BM, n0 = t % tn * BN;
                for (int kb = 0; ok && kb < nkb; ++kb, ++n) {
                    const uint32_t st = n % STAGES;
                    ok = mbar_wait(bar_empty(st), ((n / STAGES) & 1) ^ 1, abort_flag, kLinTimeout | 0x11);
                    if (!ok) break;
                    const uint32_t dst = base + st * STAGE_BYTES;
                    mbar_arrive_expect_tx(bar_full(st), STAGE_BYTES);
                    tma_load_2d(dst, &tm_x, bar_full(st), kb * BK, m0);
                    tma_load_2d(dst + BM * BK, &tm_w, bar_full(st), kb * BK, n0);
                }
            }
            // the loads still in flight land before shared memory is released
            volatile int no_abort = 0;
            for (uint32_t u = n > STAGES ? n - STAGES : 0; u < n; ++u)
                mbar_wait(bar_full(u % STAGES), (u / STAGES) & 1, &no_abort, kLinTimeout | 0x12);
        } else if (warp == 1 && lane == 0) {
            constexpr uint32_t IDESC = idesc_e4m3(BM, BN);
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                for (int kb = 0; kb < nkb; ++kb, ++n) {
                    const uint32_t st = n % STAGES, b = n & 1;
                    ok = mbar_wait(bar_acce(b), ((n >> 1) & 1) ^ 1, abort_flag, kLinTimeout | 0x13);
                    if (ok) ok = mbar_wait(bar_full(st), (n / STAGES) & 1, abort_flag, kLinTimeout | 0x14);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = base + st * STAGE_BYTES;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8(tmem + b * BN, smem_desc(a + kk * 32, 16, 1024, kSw128),
                               smem_desc(a + BM * BK + kk * 32, 16, 1024, kSw128), IDESC, kk > 0 ? 1u : 0u);
                    mma_commit(bar_empty(st));
                    mma_commit(bar_accf(b));
                }
            }
            volatile int no_abort = 0;
            mma_commit(bar_done);
            mbar_wait(bar_done, 0, &no_abort, kLinTimeout | 0x15);
        } else if (warp == 2) {
            constexpr int WS = SW_ROWS ? 8 : 1;            // scales of w a lane fetches
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const int m0 = t / tn * BM, n0 = t % tn * BN;
                const float *fx[4], *fw[WS];
#pragma unroll
                for (int i = 0; i < 4; ++i) fx[i] = p.sx + (int64_t)min(m0 + lane + 32 * i, p.M - 1) * p.sx_row;
#pragma unroll
                for (int i = 0; i < WS; ++i)
                    fw[i] = p.sw + (int64_t)(SW_ROWS ? min(n0 + lane + 32 * i, p.N - 1)
                                                     : min(n0 + 128 * (lane & 1), p.N - 1) / 128) * p.sw_row;
                for (int kb = 0; kb < nkb; ++kb, ++n) {
                    const uint32_t st = n % RING, dst = base + L::ring_off + st * SLOT + 4 * lane;
                    ok = mbar_wait(bar_sempty(st), ((n / RING) & 1) ^ 1, abort_flag, kLinTimeout | 0x17);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i) cp_async4(dst + 128 * i, fx[i] + kb * p.sx_grp);
#pragma unroll
                    for (int i = 0; i < WS; ++i)
                        if (SW_ROWS || lane < 2) cp_async4(dst + 4 * BM + 128 * i, fw[i] + kb * p.sw_grp);
                    cp_async_arrive(bar_sfull(st));
                }
            }
            cp_async_wait_all();
        } else if (warp == 3 && p.bias) {
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++n) {
                const int n0 = t % tn * BN;
                const uint32_t b = n & 1, dst = base + L::bias_off + b * BN * 4 + 4 * lane;
                ok = mbar_wait(bar_bempty(b), ((n >> 1) & 1) ^ 1, abort_flag, kLinTimeout | 0x18);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 8; ++i) cp_async4(dst + 128 * i, p.bias + min(n0 + lane + 32 * i, p.N - 1));
                cp_async_arrive(bar_bfull(b));
            }
            cp_async_wait_all();
        }
    } else {
        regs_increase<SUM_REGS>();
        const int quarter = warp & 3, col_w = ((warp - 4) >> 2) * COLS;   // this warp's lanes and columns of the tile
        const uint32_t stg = base + L::stg_off + (uint32_t)(warp - 4) * L::boxes * L::box;
        if (lane == 0) prefetch_tmap(&tm_y);
        bool ok = true;
        uint32_t n = 0, tile_no = 0;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++tile_no) {
            uint64_t acc[COLS / 2];
#pragma unroll
            for (int i = 0; i < COLS / 2; ++i) acc[i] = 0;
#pragma unroll 1
            for (int kb = 0; kb < nkb; ++kb, ++n) {
                const uint32_t b = n & 1, rs = n % RING;
                ok = mbar_wait(bar_sfull(rs), (n / RING) & 1, abort_flag, kLinTimeout | 0x19);
                const float* ring = reinterpret_cast<const float*>(gbase + L::ring_off + rs * SLOT);
                float f = ring[32 * quarter + lane];
                if (!SW_ROWS) f *= ring[BM + col_w / 128];
                if (ok) ok = mbar_wait(bar_accf(b), (n >> 1) & 1, abort_flag, kLinTimeout | 0x16);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t f2v = f2(f, f);
                const uint32_t ta = tmem + b * BN + (uint32_t)col_w + ((uint32_t)(32 * quarter) << 16);
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32_sync(ta + 32 * c, v);
                    if (c == COLS / 32 - 1) {              // everything has been read: the buffer is free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_acce(b));
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        uint64_t t0 = f2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                        uint64_t t1 = f2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                        if (SW_ROWS) {
                            const float4 s = *reinterpret_cast<const float4*>(ring + BM + col_w + 32 * c + i);
                            t0 = fmul2(t0, f2(s.x, s.y));
                            t1 = fmul2(t1, f2(s.z, s.w));
                        }
                        uint64_t* a = acc + 16 * c + i / 2;
                        a[0] = ffma2(t0, f2v, a[0]);
                        a[1] = ffma2(t1, f2v, a[1]);
                    }
                }
                __syncwarp();                              // the slot's scales have been read
                if (lane == 0) mbar_arrive(bar_sempty(rs));
            }
            if (!ok) break;
            // ------------------------------------------------ the tile leaves
            constexpr int CPB = L::box_cols / sizeof(T), CH = L::box_cols / 16;   // columns, 16-byte chunks a box
            const int row0 = t / tn * BM + 32 * quarter, col0 = t % tn * BN + col_w;
            const float* bias_s = reinterpret_cast<const float*>(gbase + L::bias_off) + (tile_no & 1) * BN + col_w;
            if (p.bias) {
                ok = mbar_wait(bar_bfull(tile_no & 1), (tile_no >> 1) & 1, abort_flag, kLinTimeout | 0x1a);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            // chunk `ch` of row `r` in a box, as TMA's swizzle of that width places it
            auto place = [&](uint32_t box, int r, int ch) {
                return box + r * L::box_cols + ((ch ^ (L::box_cols == 128 ? r & 7 : (r >> 1) & 3)) << 4);
            };
#pragma unroll
            for (int g = 0; g < COLS / CPB; ++g) {
                const int c0 = col0 + g * CPB;
                const uint32_t box = stg + (uint32_t)(g % L::boxes) * L::box;
                if (tma_out) {
                    if (lane == 0) bulk_wait_read<L::boxes - 1>();   // the store that last read the box is done with it
                    __syncwarp();
                }
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {          // this lane's row
                    constexpr int E = 16 / sizeof(T);
                    uint64_t o2[E / 2];
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) o2[e] = acc[(g * CPB + ch * E) / 2 + e];
                    if (p.bias) {
#pragma unroll
                        for (int e = 0; e < E; e += 4) {
                            const float4 v = *reinterpret_cast<const float4*>(bias_s + g * CPB + ch * E + e);
                            o2[e / 2] = fadd2(o2[e / 2], f2(v.x, v.y));
                            o2[e / 2 + 1] = fadd2(o2[e / 2 + 1], f2(v.z, v.w));
                        }
                    }
                    float o[E];
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        o[e] = f2lo(o2[e / 2]);
                        o[e + 1] = f2hi(o2[e / 2]);
                    }
                    const uint32_t at = place(box, lane, ch);
                    if constexpr (sizeof(T) == 2)
                        sts128(at, pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
                    else
                        sts128(at, __float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3]));
                }
                if (tma_out) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (row0 < p.M && c0 < p.N) tma_store_2d(&tm_y, box, c0, row0);
                        bulk_commit();                     // also of nothing, so that the wait above keeps its distance
                    }
                } else {
                    __syncwarp();
                    constexpr int LPR = L::box_cols / 4;   // lanes a row, one 32-bit word each
                    const int rows = min(32, p.M - row0), w = lane % LPR;
                    for (int r = lane / LPR; r < 32; r += 32 / LPR) {
                        uint32_t v;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(place(box, r, w >> 2) + (w & 3) * 4));
                        const uint32_t next = __shfl_down_sync(0xffffffffu, v, 1);
                        if (r >= rows) continue;
                        T* out = static_cast<T*>(p.y) + (int64_t)(row0 + r) * p.ldy + c0;
                        if constexpr (sizeof(T) == 4) {
                            if (c0 + w < p.N) out[w] = __uint_as_float(v);
                        } else {
                            uint16_t* o16 = reinterpret_cast<uint16_t*>(out);
                            const int c = c0 + 2 * w;
                            if ((reinterpret_cast<uintptr_t>(out) & 3) == 0) {
                                if (c + 1 < p.N)
                                    *reinterpret_cast<uint32_t*>(o16 + 2 * w) = v;
                                else if (c < p.N)
                                    o16[2 * w] = (uint16_t)v;
                            } else {                       // pairs start at odd columns
                                if (w == 0 && c < p.N) o16[0] = (uint16_t)v;
                                if (w < LPR - 1 && c + 2 < p.N)
                                    *reinterpret_cast<uint32_t*>(o16 + 2 * w + 1) = (v >> 16) | (next << 16);
                                else if (c + 1 < p.N)
                                    o16[2 * w + 1] = (uint16_t)(v >> 16);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            if (p.bias) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_bempty(tile_no & 1));
            }
        }
        if (lane == 0) bulk_wait<0>();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 2 * BN);
    }
}

}  // namespace wide
}  // namespace fp8
}  // namespace evo
