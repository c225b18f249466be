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
    int parts;                     // Parts: runs of blocks; y is then fp32 [parts * (M up to whole tiles), N]
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
// ------------------------------------------------------------------ the kernel
// One CTA per SM, tiles of 128 x BN of y.  Roles: warp 0 TMA, warp 1 MMA, warp 2 the
// scales of the coming blocks and warp 3 the bias of the coming tile (cp.async into
// shared memory), the warps from 4 on add up the blocks (warp % 4: the quarter of TMEM
// lanes a warp may read; (warp - 4) / 4: its share of the columns) and write the tile.
//
// Wide   256 columns, persistent: the tiles of a row block in succession.  While one is
//        written the next one's first two blocks are multiplied.  y leaves through
//        boxes of 32 rows in shared memory, by TMA where its rows are 16-byte aligned,
//        else by the warp a row at a time.
// Split  128 columns, one tile per cluster, for calls with few tiles (few rows, or a
//        weight's gradient): the CTAs of the cluster each sum a run of blocks and join
//        their fp32 results through distributed shared memory in rank order -- the same
//        bits on every run, one launch, no workspace.  The summing warps work in two
//        groups on alternate blocks, so that each waits half as often.
// Parts  256 columns, for long sums into few tiles: items of a tile and a run of blocks fill
//        the GPU whatever the number of tiles is (clusters of 8 leave a quarter of it idle),
//        and their fp32 results go to a workspace, which sum_parts_kernel adds in order.
//
// The summing warps are what bounds the long sums: a block's 128 x BN results are read
// from TMEM and added in the time the tensor core takes for the next (512 cycles at BN =
// 256).  Sixteen warps of 64 columns share a tile's way out best, eight of 128 columns hold
// twice the registers and need fewer instructions a block.  Both builds in turn on one GPU,
// calls in a row under the power cap, bf16, us with sixteen and eight: 131072 x 256 x 1024
// 71.6 and 73.4, 32768 x 1024 x 2048 97.1 and 94.3, 16384 x 1280 x 4096 114.6 and 111.0,
// 8191 x 4096 x 8192 315 and 303.  Long begins above a sum of 1024, where its gain passes 3 %;
// from 512 to 1024 eight lead by 1 to 3 %.  The warps hold their sums and nothing that comes
// from global memory: scales and bias fetched into their own registers spilled and waited for
// the load at the spill (131072 x 256 x 1024 125 us, 8191 x 4096 x 8192 350).
constexpr int RING = 8;                                    // blocks whose scales are held
enum Mode { WHOLE, JOINED, PARTS };
template <int BN_, int STAGES_, Mode MODE, int WARPS>
struct Config {
    static constexpr int BN = BN_, STAGES = STAGES_;
    static constexpr int SUM_WARPS = WARPS;                // column groups x 4 lane quarters
    static constexpr int THREADS = 32 * (4 + SUM_WARPS);
    // registers per thread: at launch, and as handed from the control warps to the others
    static constexpr int LAUNCH_REGS = WARPS == 16 ? 96 : 168;
    static constexpr int CTRL_REGS = WARPS == 16 ? 32 : 56, SUM_REGS = WARPS == 16 ? 112 : 216;
    static_assert(4 * CTRL_REGS + SUM_WARPS * SUM_REGS <= (4 + SUM_WARPS) * LAUNCH_REGS, "register split");
    static_assert(LAUNCH_REGS * THREADS <= 65536, "registers of an SM");
    static constexpr bool JOIN = MODE == JOINED;           // a cluster's CTAs join one tile
    static constexpr bool PART = MODE == PARTS;            // each item sums a run of blocks into the workspace
    static constexpr int GROUPS = JOIN ? 2 : 1;            // groups of summing warps, which take the blocks in turn
    static constexpr int GROUP_WARPS = SUM_WARPS / GROUPS;
    static constexpr int COLS = 4 * BN / GROUP_WARPS;      // columns a summing warp holds
    static constexpr int BUFS = 512 / BN;                  // blocks' results in TMEM
    static constexpr int STAGE_BYTES = (BM + BN) * BK;
    static constexpr int SLOT = (BM + BN) * 4;             // 128 scales of x, then BN / 128 or BN of w
    static constexpr int BOX = 32 * 128, BOXES = 16 / WARPS;   // of a warp; JOIN: the tile lies over the stages instead
    static constexpr int READ = WARPS == 16 ? 32 : 64;     // columns read from TMEM at a time
    static constexpr int stg_off = STAGES * STAGE_BYTES;
    static constexpr int ring_off = stg_off + (JOIN ? 0 : SUM_WARPS * BOXES * BOX);
    static constexpr int bias_off = ring_off + RING * SLOT;
    static constexpr int bar_off = bias_off + 2 * BN * 4;
    static constexpr int n_bars = 2 * STAGES + 2 * RING + 2 * BUFS + 5;
    static constexpr int misc_off = bar_off + n_bars * 8;
    static constexpr int smem = misc_off + 16 + 1024;
    static_assert(smem <= 232448, "shared memory budget");
    static_assert(!JOIN || (BN == 128 && stg_off >= GROUPS * BM * BN * 4), "the groups' tiles lie over the stages");
};
using Wide = Config<256, 3, WHOLE, 16>;
using Long = Config<256, 3, WHOLE, 8>;                     // Wide, for sums of more than 1024
using Split = Config<128, 6, JOINED, 16>;
using Parts = Config<256, 3, PARTS, 8>;

__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const float* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on `bar` (which counts the arriving threads) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// float4 chunk `ch` of row `r` of the joined tile: chunks permuted by the row, so that lanes
// holding one chunk of 32 rows, or 32 chunks of one row, meet different banks
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int r, int ch) {
    return base + (uint32_t)(r * 512 + ((ch ^ (r & 31)) << 4));
}

template <typename T, bool SW_ROWS, class L>
__global__ void __launch_bounds__(L::THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                  const __grid_constant__ CUtensorMap tm_y, const LinParams p, const int tma_out) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    constexpr int BN = L::BN, COLS = L::COLS, STAGES = L::STAGES, BUFS = L::BUFS;
    // through a shuffle, so that the compiler knows it is the same for the warp (uniform registers)
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int tn = (p.N + BN - 1) / BN, tiles = (p.M + BM - 1) / BM * tn;
    const int all_kb = (p.K + BK - 1) / BK;
    // this CTA's tiles t0, t0 + step, ... and of each the blocks kb0 .. kb1 - 1
    const int S = L::JOIN ? (int)cluster_size() : 1, rank = L::JOIN ? (int)cluster_rank() : 0;
    const int t0 = (int)blockIdx.x / S, step = L::JOIN ? tiles : (int)gridDim.x;
    const int kb0_c = (int)((int64_t)all_kb * rank / S), kb1_c = (int)((int64_t)all_kb * (rank + 1) / S);
    // Parts: item t is part t % parts of tile t / parts
    const int parts = L::PART ? p.parts : 1, items = tiles * parts;
    auto first_kb = [&](int t) { return L::PART ? (int)((int64_t)all_kb * (t % parts) / parts) : kb0_c; };
    auto end_kb = [&](int t) { return L::PART ? (int)((int64_t)all_kb * (t % parts + 1) / parts) : kb1_c; };
    auto bar = [&](int i) { return base + L::bar_off + 8u * i; };
    auto bar_full = [&](uint32_t i) { return bar(i); };
    auto bar_empty = [&](uint32_t i) { return bar(STAGES + i); };
    auto bar_sfull = [&](uint32_t i) { return bar(2 * STAGES + i); };
    auto bar_sempty = [&](uint32_t i) { return bar(2 * STAGES + RING + i); };
    auto bar_accf = [&](uint32_t b) { return bar(2 * STAGES + 2 * RING + b); };
    auto bar_acce = [&](uint32_t b) { return bar(2 * STAGES + 2 * RING + BUFS + b); };
    auto bar_bfull = [&](uint32_t b) { return bar(2 * STAGES + 2 * RING + 2 * BUFS + b); };
    auto bar_bempty = [&](uint32_t b) { return bar(2 * STAGES + 2 * RING + 2 * BUFS + 2 + b); };
    const uint32_t bar_done = bar(2 * STAGES + 2 * RING + 2 * BUFS + 4);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + L::misc_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::misc_off + 4);

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(bar_full(i), 1);
            mbar_init(bar_empty(i), 1);
        }
        for (int i = 0; i < RING; ++i) {
            mbar_init(bar_sfull(i), 32);
            mbar_init(bar_sempty(i), L::GROUP_WARPS);
        }
        for (int b = 0; b < BUFS; ++b) {
            mbar_init(bar_accf(b), 1);
            mbar_init(bar_acce(b), L::GROUP_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_bfull(b), 32);
            mbar_init(bar_bempty(b), L::SUM_WARPS);
        }
        mbar_init(bar_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(base + L::misc_off, BUFS * BN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        regs_decrease<L::CTRL_REGS>();
        bool ok = true;
        uint32_t n = 0;
        if (warp == 0 && lane == 0) {
            prefetch_tmap(&tm_x);
            prefetch_tmap(&tm_w);
            for (int t = t0; ok && t < items; t += step) {
                const int tile = t / parts, m0 = tile / tn * BM, n0 = tile % tn * BN, kb0 = first_kb(t), kb1 = end_kb(t);
                for (int kb = kb0; ok && kb < kb1; ++kb, ++n) {
                    const uint32_t st = n % STAGES;
                    ok = mbar_wait(bar_empty(st), ((n / STAGES) & 1) ^ 1, abort_flag, kLinTimeout | 0x11);
                    if (!ok) break;
                    const uint32_t dst = base + st * L::STAGE_BYTES;
                    mbar_arrive_expect_tx(bar_full(st), L::STAGE_BYTES);
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
            for (int t = t0; ok && t < items; t += step) {
                const int kb0 = first_kb(t), kb1 = end_kb(t);
                for (int kb = kb0; kb < kb1; ++kb, ++n) {
                    const uint32_t st = n % STAGES, b = n % BUFS;
                    ok = mbar_wait(bar_acce(b), ((n / BUFS) & 1) ^ 1, abort_flag, kLinTimeout | 0x13);
                    if (ok) ok = mbar_wait(bar_full(st), (n / STAGES) & 1, abort_flag, kLinTimeout | 0x14);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = base + st * L::STAGE_BYTES;
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
            // C scales of the rows from r0 on (the last row again past `rows`), block by block: 16
            // bytes a copy where the rows' scales lie side by side and aligned (12 single copies a
            // block held 1024 x 131072 x 256 up: 69 us, 3 wide ones 60), else one for each row.  The
            // control warps have 32 registers: a pointer for each copy would spill, and take the
            // summing warps' code along with it.
            auto side = [](const float* src, int64_t s_row, int64_t s_grp, int r0, int C, int rows) {
                return s_row == 1 && s_grp % 4 == 0 && r0 + C <= rows && (reinterpret_cast<uintptr_t>(src) & 15) == 0;
            };
            auto copy = [&](uint32_t dst, const float* src, bool wide, int r0, int rows, int64_t s_row, auto count) {
                constexpr int C = decltype(count)::value;
                if (wide) {
#pragma unroll
                    for (int i = 0; i < C / 128; ++i) cp_async16(dst + 16 * lane + 512 * i, src + r0 + 4 * lane + 128 * i);
                } else {
#pragma unroll 1
                    for (int i = lane; i < C; i += 32) cp_async4(dst + 4 * i, src + (int64_t)min(r0 + i, rows - 1) * s_row);
                }
            };
            for (int t = t0; ok && t < items; t += step) {
                const int tile = t / parts, m0 = tile / tn * BM, n0 = tile % tn * BN, kb0 = first_kb(t), kb1 = end_kb(t);
                const bool x_wide = side(p.sx, p.sx_row, p.sx_grp, m0, BM, p.M);
                const bool w_wide = SW_ROWS && side(p.sw, p.sw_row, p.sw_grp, n0, BN, p.N);
                const float* sx = p.sx + kb0 * p.sx_grp;
                const float* sw = p.sw + kb0 * p.sw_grp;
                if (!SW_ROWS) sw += (int64_t)(min(n0 + 128 * (lane & (BN / 128 - 1)), p.N - 1) / 128) * p.sw_row;
                for (int kb = kb0; kb < kb1; ++kb, ++n, sx += p.sx_grp, sw += p.sw_grp) {
                    const uint32_t st = n % RING, dst = base + L::ring_off + st * L::SLOT;
                    ok = mbar_wait(bar_sempty(st), ((n / RING) & 1) ^ 1, abort_flag, kLinTimeout | 0x17);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    copy(dst, sx, x_wide, m0, p.M, p.sx_row, std::integral_constant<int, BM>{});
                    if (SW_ROWS)
                        copy(dst + 4 * BM, sw, w_wide, n0, p.N, p.sw_row, std::integral_constant<int, BN>{});
                    else if (lane < BN / 128)
                        cp_async4(dst + 4 * BM + 4 * lane, sw);
                    cp_async_arrive(bar_sfull(st));
                }
            }
            cp_async_wait_all();
        } else if (warp == 3 && p.bias && !L::JOIN) {
            for (int t = t0; ok && t < items; t += step, ++n) {
                const int n0 = t / parts % tn * BN;
                const uint32_t b = n & 1, dst = base + L::bias_off + b * BN * 4 + 4 * lane;
                ok = mbar_wait(bar_bempty(b), ((n >> 1) & 1) ^ 1, abort_flag, kLinTimeout | 0x18);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < BN / 32; ++i) cp_async4(dst + 128 * i, p.bias + min(n0 + lane + 32 * i, p.N - 1));
                cp_async_arrive(bar_bfull(b));
            }
            cp_async_wait_all();
        }
    } else {
        regs_increase<L::SUM_REGS>();
        // this warp's lanes and columns of the tile, and its group
        const int quarter = warp & 3, col_w = ((warp - 4) % L::GROUP_WARPS >> 2) * COLS, group = (warp - 4) / L::GROUP_WARPS;
        const uint32_t boxes = base + L::stg_off + (uint32_t)(warp - 4) * L::BOXES * L::BOX;
        if (!L::JOIN && lane == 0) prefetch_tmap(&tm_y);
        bool ok = true;
        uint32_t n = (uint32_t)group, tile_no = 0;
        for (int t = t0; ok && t < items; t += step, ++tile_no) {
            uint64_t acc[COLS / 2];
#pragma unroll
            for (int i = 0; i < COLS / 2; ++i) acc[i] = 0;
            const int tile = t / parts, kb0 = first_kb(t), kb1 = end_kb(t);
            const bool live = (!L::JOIN && !L::PART) || tile / tn * BM + 32 * quarter < p.M;   // else no row of y: only arrivals
#pragma unroll 1
            for (int kb = kb0 + group; kb < kb1; kb += L::GROUPS, n += L::GROUPS) {
                const uint32_t b = n % BUFS, rs = n % RING;
                ok = mbar_wait(bar_sfull(rs), (n / RING) & 1, abort_flag, kLinTimeout | 0x19);
                const float* ring = reinterpret_cast<const float*>(gbase + L::ring_off + rs * L::SLOT);
                float f = ring[32 * quarter + lane];
                if (!SW_ROWS) f *= ring[BM + col_w / 128];
                if (ok) ok = mbar_wait(bar_accf(b), (n / BUFS) & 1, abort_flag, kLinTimeout | 0x16);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t f2v = f2(f, f);
                const uint32_t ta = tmem + b * BN + (uint32_t)col_w + ((uint32_t)(32 * quarter) << 16);
                if (!live) {
                    if (lane == 0) {
                        mbar_arrive(bar_acce(b));
                        mbar_arrive(bar_sempty(rs));
                    }
                    continue;
                }
                auto release = [&]() {                     // everything has been read: the buffer is free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_acce(b));
                };
                if constexpr (SW_ROWS) {
                    // sixteen columns at a time, their scales (the same for the whole warp) fetched
                    // before the results, so that one wait covers both
#pragma unroll
                    for (int c = 0; c < COLS / 16; ++c) {
                        uint32_t v[16];
                        float4 s[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[i] = *reinterpret_cast<const float4*>(ring + BM + col_w + 16 * c + 4 * i);
                        tmem_ld16_sync(ta + 16 * c, v);
                        if (c == COLS / 16 - 1) release();
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const uint64_t t0 = fmul2(f2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), f2(s[i / 4].x, s[i / 4].y));
                            const uint64_t t1 = fmul2(f2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), f2(s[i / 4].z, s[i / 4].w));
                            uint64_t* a = acc + 8 * c + i / 2;
                            a[0] = ffma2(t0, f2v, a[0]);
                            a[1] = ffma2(t1, f2v, a[1]);
                        }
                    }
                } else {
                    constexpr int W = L::READ;
#pragma unroll
                    for (int c = 0; c < COLS / W; ++c) {
                        uint32_t v[W];
                        if constexpr (W == 64)
                            tmem_ld32x2_sync(ta + W * c, ta + W * c + 32, v);
                        else
                            tmem_ld32_sync(ta + W * c, v);
                        if (c == COLS / W - 1) release();
#pragma unroll
                        for (int i = 0; i < W; i += 4) {
                            const uint64_t t0 = f2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                            const uint64_t t1 = f2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                            uint64_t* a = acc + (W * c + i) / 2;
                            a[0] = ffma2(t0, f2v, a[0]);
                            a[1] = ffma2(t1, f2v, a[1]);
                        }
                    }
                }
                __syncwarp();                              // the slot's scales have been read
                if (lane == 0) mbar_arrive(bar_sempty(rs));
            }
            if (!ok) break;
            if constexpr (L::JOIN) {
                // once every MMA is done every load has been used too: the stages take the fp32 tile,
                // one of each group
                ok = mbar_wait(bar_done, 0, abort_flag, kLinTimeout | 0x1b);
                ok = __all_sync(0xffffffffu, ok);
                const int row = 32 * quarter + lane;
                if (ok && tile / tn * BM + row < p.M) {
#pragma unroll
                    for (int i = 0; i < COLS / 4; ++i)
                        sts128(tile_addr(base + (uint32_t)(group * BM * BN * 4), row, col_w / 4 + i), __float_as_uint(f2lo(acc[2 * i])),
                               __float_as_uint(f2hi(acc[2 * i])), __float_as_uint(f2lo(acc[2 * i + 1])),
                               __float_as_uint(f2hi(acc[2 * i + 1])));
                }
                break;
            }
            // ------------------------------------------------ the tile leaves
            constexpr int CPB = 128 / sizeof(T);           // columns a box
            const int row0 = tile / tn * BM + 32 * quarter, col0 = tile % tn * BN + col_w;
            const int out0 = L::PART ? t % parts * ((p.M + BM - 1) / BM * BM) + row0 : row0;   // the row of y that row0 becomes
            const float* bias_s = reinterpret_cast<const float*>(gbase + L::bias_off) + (tile_no & 1) * BN + col_w;
            if (p.bias) {
                ok = mbar_wait(bar_bfull(tile_no & 1), (tile_no >> 1) & 1, abort_flag, kLinTimeout | 0x1a);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            // chunk `ch` of row `r` in a box, as TMA's 128-byte swizzle places it
            uint32_t box = boxes;
            auto place = [&](int r, int ch) {
                return box + r * 128 + ((ch ^ (r & 7)) << 4);
            };
#pragma unroll
            for (int g = 0; g < COLS / CPB; ++g) {
                const int c0 = col0 + g * CPB;
                box = boxes + (uint32_t)(g % L::BOXES) * L::BOX;
                if (tma_out) {
                    if (lane == 0) bulk_wait_read<L::BOXES - 1>();   // the store that last read the box is done with it
                    __syncwarp();
                }
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) {           // this lane's row
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
                    const uint32_t at = place(lane, ch);
                    if constexpr (sizeof(T) == 2)
                        sts128(at, pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
                    else
                        sts128(at, __float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3]));
                }
                if (tma_out) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (row0 < p.M && c0 < p.N) tma_store_2d(&tm_y, box, c0, out0);
                        bulk_commit();                     // also of nothing, so that the wait above keeps its distance
                    }
                } else {
                    __syncwarp();
                    const int rows = min(32, p.M - row0), w = lane;   // a 32-bit word of the row
                    for (int r = 0; r < rows; ++r) {
                        uint32_t v;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(place(r, w >> 2) + (w & 3) * 4));
                        const uint32_t next = __shfl_down_sync(0xffffffffu, v, 1);
                        T* out = static_cast<T*>(p.y) + (int64_t)(out0 + r) * p.ldy + c0;
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
                                if (w < 31 && c + 2 < p.N)
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
        if (!L::JOIN && lane == 0) bulk_wait<0>();
    }
    __syncwarp();                                          // one lane of the first warps comes late
    if constexpr (L::JOIN) {
        const int m0 = t0 / tn * BM, n0 = t0 % tn * BN;
        cluster_sync();
        const int rows = min(BM, p.M - m0);
        T* y = static_cast<T*>(p.y);
        const bool vec = (p.M == 1 || p.ldy % 4 == 0) && (reinterpret_cast<uintptr_t>(p.y) & (4 * sizeof(T) - 1)) == 0;
        for (int idx = rank * L::THREADS + (int)threadIdx.x; idx < rows * 32; idx += S * L::THREADS) {
            const int r = idx >> 5, ch = idx & 31, c = n0 + 4 * ch;
            if (c >= p.N) continue;
            const uint32_t at = tile_addr(base, r, ch);
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < L::GROUPS * S; ++k) {
                const float4 v = ld_cluster(at + (uint32_t)(k % L::GROUPS * BM * BN * 4), (uint32_t)(k / L::GROUPS));
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
    }
    tc_fence_before();
    if (L::JOIN)
        cluster_sync();                                    // peers have read this CTA's tile
    else
        __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, BUFS * BN);
    }
}

// y = the parts of Parts, added in order, + bias.  One thread per four columns; the parts were
// written just before and lie in L2.
template <typename T>
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* part, int64_t ld, int64_t part_rows, int parts,
                                                        const LinParams p) {
    const int64_t per_row = (p.N + 3) / 4, items = p.M * per_row;
    const bool vec = (p.M == 1 || p.ldy % 4 == 0) && (reinterpret_cast<uintptr_t>(p.y) & (4 * sizeof(T) - 1)) == 0;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < items; t += (int64_t)gridDim.x * 256) {
        const int64_t r = t / per_row, c = (t - r * per_row) * 4;
        const float* at = part + r * ld + c;
        float4 o = *reinterpret_cast<const float4*>(at);
#pragma unroll 8
        for (int k = 1; k < parts; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(at + k * part_rows * ld);
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
        }
        float f[4] = {o.x, o.y, o.z, o.w};
        if (p.bias) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < p.N) f[e] += __ldg(p.bias + c + e);
        }
        T* out = static_cast<T*>(p.y) + r * p.ldy + c;
        if (vec && c + 4 <= p.N) {
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
            else
                *reinterpret_cast<float4*>(out) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < p.N) Elem<T>::store(out + e, f[e]);
        }
    }
}

// ------------------------------------------------------------- one or two rows of x
// The same product for single tokens, bound by reading w once: no tensor core, whose tiles would
// be nearly empty and whose blocks' results would be read one by one.  A warp takes R rows of w
// and every KS-th chunk of 512 codes of them, a lane 16 codes of each (one scale block), as exact
// products of halves added in fp32 (one instruction each on sm_100a); the lanes are added by
// shuffles, the KS warps in order.  What counts is bytes on their way: four chunks of two rows in
// each of 32 warps an SM read 1 x 8192 x 8192 in 18.6 us, two of four rows in 24 warps in 26.8
// (and left a second wave), with the codes converted to fp32 in 28.8; the tiles took 22.7.
namespace few {

constexpr int R = 2, CHUNK = 512, WARPS = 8;

struct Codes16 {
    uint32_t w[4];
    // codes k .. k + 15 of a row, zeros from K on; nothing behind the row's last code is read
    template <bool WHOLE>
    __device__ __forceinline__ void load(const uint8_t* row, int k, int K) {
        if (WHOLE || k + 16 <= K) {
            const uint4 a = *reinterpret_cast<const uint4*>(row + k);
            w[0] = a.x;
            w[1] = a.y;
            w[2] = a.z;
            w[3] = a.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = 0;
#pragma unroll
            for (int i = 0; i < 15; ++i)
                if (k + i < K) w[i >> 2] |= (uint32_t)row[k + i] << (8 * (i & 3));
        }
    }
    // as 16 halves, which hold every e4m3 value
    __device__ __forceinline__ void halves(uint32_t* h) const {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[i]) : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
    }
};
// a + the product of two halves, one rounding.
__device__ __forceinline__ float fma_half(uint16_t x, uint16_t y, float a) {
    asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(a) : "h"(x), "h"(y));
    return a;
}

template <typename T, bool SW_ROWS, int M>
__global__ void __launch_bounds__(32 * WARPS, M == 1 ? 4 : 2) linear_kernel(const LinParams p, const int ks) {
    __shared__ float join[WARPS][R * M];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp / ks, part = warp - sub * ks;       // the block's sub-th R rows, this warp's chunks
    const int64_t n0 = ((int64_t)blockIdx.x * (WARPS / ks) + sub) * R;
    const uint8_t *x[M], *w[R];
    const float *sx[M], *sw[R];
#pragma unroll
    for (int m = 0; m < M; ++m) {                            // a row past the last one repeats it
        const int r = min(m, p.M - 1);
        x[m] = static_cast<const uint8_t*>(p.x) + r * p.ldx;
        sx[m] = p.sx + r * p.sx_row;
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int64_t n = min(n0 + j, (int64_t)p.N - 1);
        w[j] = static_cast<const uint8_t*>(p.w) + n * p.ldw;
        sw[j] = p.sw + (SW_ROWS ? n : n / 128) * p.sw_row;
    }
    float acc[R][M];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int m = 0; m < M; ++m) acc[j][m] = 0.f;
    auto add = [&](int k, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        Codes16 cw[R], cx[M];
        float fw[R], f[M];
        const int64_t b = k / BK;
#pragma unroll
        for (int j = 0; j < R; ++j) cw[j].template load<WHOLE>(w[j], k, p.K);
#pragma unroll
        for (int m = 0; m < M; ++m) cx[m].template load<WHOLE>(x[m], k, p.K);
#pragma unroll
        for (int j = 0; j < R; ++j) fw[j] = __ldg(sw[j] + b * p.sw_grp);
#pragma unroll
        for (int m = 0; m < M; ++m) f[m] = __ldg(sx[m] + b * p.sx_grp);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            uint32_t v[8];
            cw[j].halves(v);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                uint32_t u[8];
                cx[m].halves(u);                             // once for all j: the compiler keeps it
                float a = 0.f, c = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a = fma_half((uint16_t)v[i], (uint16_t)u[i], a);
                    c = fma_half((uint16_t)(v[i] >> 16), (uint16_t)(u[i] >> 16), c);
                }
                acc[j][m] = fmaf(a + c, f[m] * fw[j], acc[j][m]);
            }
        }
    };
    if (n0 < p.N) {
        const int last = p.K / CHUNK * CHUNK;                // whole chunks first, without a test a load
        int k = part * CHUNK + 16 * lane;
#pragma unroll (M == 1 ? 4 : 2)
        for (; k < last; k += ks * CHUNK) add(k, std::true_type{});
        if (k < p.K) add(k, std::false_type{});
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) acc[j][m] += __shfl_xor_sync(0xffffffffu, acc[j][m], o);
            if (lane == 0) join[warp][j * M + m] = acc[j][m];
        }
    __syncthreads();
    if (part == 0 && lane < R * M) {
        float s = 0.f;
        for (int i = 0; i < ks; ++i) s += join[warp + i][lane];
        const int m = lane % M;
        const int64_t n = n0 + lane / M;
        if (m < p.M && n < p.N) {
            if (p.bias) s += __ldg(p.bias + n);
            Elem<T>::store(static_cast<T*>(p.y) + m * p.ldy + n, s);
        }
    }
}

}  // namespace few
}  // namespace fp8
}  // namespace evo
