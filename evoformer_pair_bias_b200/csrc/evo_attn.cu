// evo_attn.cu -- C-ABI entry points, argument validation and launch layer.
//
// The whole library is one translation unit (it includes every kernel
// header), so the device status word and all kernels share one module.
//
// Call shapes handled here (all through strides, no copies):
//   MSA-row attention          rows s = MSA sequences
//   triangle, starting node    rows s = pair rows
//   triangle, ending node      transposed pair: s and n strides swapped
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "evo_attn.h"
#include "common.cuh"
#include "simt.cuh"
#include "sm100.cuh"
#include "tma_maps.cuh"
#include "timing.cuh"
#include "fwd_sm100.cuh"
#include "bwd_sm100.cuh"
#include "proj_sm100.cuh"
#include "trimul_sm100.cuh"
#include "partials.cuh"
#include "fp8_rows.cuh"
#include "fp8_sm100.cuh"

#define EVO_VERSION 10100

namespace {

using evo::Strides;

std::atomic<uint64_t> g_launches{0};
std::atomic<uint64_t> g_wait_limit_ns{EVO_WAIT_LIMIT_NS};

// 2^x through the FMA-pipe exponential of the attention kernels, two values per call.
__global__ void exp2_fma_kernel(const float* __restrict__ x, float* __restrict__ y, int64_t n) {
    for (int64_t i = 2 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x); i < n;
         i += 2 * (int64_t)gridDim.x * blockDim.x) {
        const float a = x[i], b = i + 1 < n ? x[i + 1] : 0.0f;
        const uint64_t r = evo::sm100::exp2_poly2(evo::sm100::f2(a, b));
        y[i] = evo::sm100::f2lo(r);
        if (i + 1 < n) y[i + 1] = evo::sm100::f2hi(r);
    }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

Strides to_strides(const evo_strides_t& s) { return Strides{s.b, s.s, s.n, s.h}; }

bool strides_ok(const evo_strides_t* s) {
    return s && s->b >= 0 && s->s >= 0 && s->n >= 0 && s->h >= 0;
}

bool strides_mult(const evo_strides_t* s, int64_t m) {
    return s->b % m == 0 && s->s % m == 0 && s->n % m == 0 && s->h % m == 0;
}

// Every element of a [B,S,N,H,C] view must be addressed at most once: the
// strides must not make two logical rows of the output overlap.  (Inputs may
// alias freely.)  Checked by sorting the four (extent, stride) pairs.
bool non_overlapping(const evo_shape_t& sh, const evo_strides_t& st) {
    struct D { int64_t n, s; };
    D d[5] = {{sh.B, st.b}, {sh.S, st.s}, {sh.N, st.n}, {sh.H, st.h}, {sh.C, 1}};
    std::sort(d, d + 5, [](const D& a, const D& b) { return a.s < b.s; });
    int64_t span = 1;  // elements covered by the inner dims so far
    for (auto& e : d) {
        if (e.n == 1) continue;
        if (e.s < span) return false;
        span = e.s * e.n;
    }
    return true;
}

evo_status_t check_shape(const evo_shape_t* sh) {
    if (!sh) return EVO_ERR_INVALID_ARG;
    if (sh->B < 0 || sh->S < 0 || sh->N < 0 || sh->H < 0 || sh->C < 1) return EVO_ERR_INVALID_ARG;
    if (sh->B > 65535 || sh->S > (1 << 30) || sh->N > (1 << 30) || sh->H > 65535) return EVO_ERR_UNSUPPORTED;
    if (sh->B * sh->H > 65535) return EVO_ERR_UNSUPPORTED;
    return EVO_OK;
}

bool empty_call(const evo_shape_t* sh) { return sh->B == 0 || sh->S == 0 || sh->N == 0 || sh->H == 0; }

template <typename K>
cudaError_t set_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// ---------------------------------------------------------------- forward
evo_status_t fwd_f32(const evo_shape_t& sh, const void* q, const void* k, const void* v, const void* g,
                     const evo_strides_t& in, const void* mask, const void* bias, void* out,
                     const evo_strides_t& os, float* lse, cudaStream_t stream) {
    evo::simt::Args a{};
    a.B = (int)sh.B; a.S = (int)sh.S; a.N = (int)sh.N; a.H = (int)sh.H; a.C = (int)sh.C;
    a.q = q; a.k = k; a.v = v; a.g = g; a.in = to_strides(in);
    a.mask = mask; a.bias = bias; a.out_w = out; a.os = to_strides(os); a.lse = lse;
    dim3 grid((unsigned)((sh.N + evo::simt::kRowsPerCta - 1) / evo::simt::kRowsPerCta), (unsigned)sh.S,
              (unsigned)(sh.B * sh.H));
    {
        evo::timing::Scope t(EVO_PHASE_FWD_MAIN, stream);
        evo::simt::fwd_kernel<float><<<grid, evo::simt::kWarps * 32, 0, stream>>>(a);
    }
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
    return n;
}

template <int NSUB, bool HM, bool HB>
evo_status_t launch_fwd_bf16(const CUtensorMap* maps, const evo::fwd::Params& p, cudaStream_t stream) {
    using L = evo::fwd::Layout<NSUB>;
    auto kern = evo::fwd::fwd_bf16_kernel<NSUB, HM, HB>;
    static cudaError_t attr = set_smem(kern, L::bytes);
    if (attr != cudaSuccess) return EVO_ERR_CUDA;
    // The kernel's setmaxnreg split assumes exactly L::launch_regs registers per
    // thread at launch; any other count could make the increase wait forever.
    static int regs = [&] {
        cudaFuncAttributes fa{};
        return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : -1;
    }();
    if (regs != L::launch_regs) return EVO_ERR_UNSUPPORTED;
    const int grid = std::min(p.n_items, sm_count());
    {
        evo::timing::Scope t(EVO_PHASE_FWD_MAIN, stream);
        kern<<<grid, L::threads, L::bytes, stream>>>(maps[0], maps[1], maps[2], maps[3], maps[4], maps[5], p);
    }
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

constexpr int kFwdNsub = 2;

evo_status_t fwd_bf16(const evo_shape_t& sh, const void* q, const void* k, const void* v, const void* g,
                      const evo_strides_t& in, const void* mask, const void* bias, void* out, void* out_lo,
                      const evo_strides_t& os, float* lse, cudaStream_t stream) {
    if (sh.C != evo::fwd::HD || sh.N % 8 != 0) return EVO_ERR_UNSUPPORTED;
    if (!strides_mult(&in, 8) || !strides_mult(&os, 8)) return EVO_ERR_UNSUPPORTED;
    for (const void* ptr : {q, k, v, g, (const void*)out}) if (!aligned(ptr, 16)) return EVO_ERR_UNSUPPORTED;
    if (out_lo && !aligned(out_lo, 16)) return EVO_ERR_UNSUPPORTED;
    if ((mask && !aligned(mask, 16)) || (bias && !aligned(bias, 16))) return EVO_ERR_UNSUPPORTED;
    const int64_t n_it = (sh.N + evo::fwd::BM - 1) / evo::fwd::BM;
    const int64_t n_sg = (sh.S + kFwdNsub - 1) / kFwdNsub;
    const int64_t n_items = sh.B * sh.H * n_sg * n_it;
    if (n_items > (int64_t)1 << 30) return EVO_ERR_UNSUPPORTED;
    CUtensorMap maps[6];
    std::memset(maps, 0, sizeof(maps));
    if (!evo::tma::rows_bf16(&maps[0], q, sh, in, evo::fwd::BM, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !evo::tma::rows_bf16(&maps[1], k, sh, in, evo::fwd::BN, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !evo::tma::rows_bf16(&maps[2], v, sh, in, evo::fwd::BN, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !evo::tma::rows_bf16(&maps[5], g, sh, in, evo::fwd::BM, CU_TENSOR_MAP_SWIZZLE_64B))
        return EVO_ERR_CUDA;
    if (bias && !evo::tma::square_bf16(&maps[3], bias, sh, evo::fwd::BM)) return EVO_ERR_CUDA;
    if (mask && !evo::tma::mask_bf16(&maps[4], mask, sh, 64)) return EVO_ERR_CUDA;
    evo::fwd::Params p{};
    p.B = (int)sh.B; p.S = (int)sh.S; p.N = (int)sh.N; p.H = (int)sh.H;
    p.n_kv = (int)((sh.N + evo::fwd::BN - 1) / evo::fwd::BN);
    p.n_it = (int)n_it;
    p.n_sg = (int)n_sg;
    p.n_items = (int)n_items;
    p.scale = 1.0f / sqrtf((float)sh.C);
    p.r_bf16 = __bfloat162float(__float2bfloat16_rn(sqrtf((float)sh.C)));
    p.r2_bf16 = __bfloat162float(__float2bfloat16_rn(sqrtf((float)sh.C) - p.r_bf16));
    p.g = static_cast<const __nv_bfloat16*>(g);
    p.in = to_strides(in);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.out_lo = static_cast<__nv_bfloat16*>(out_lo);
    p.os = to_strides(os);
    p.lse = lse;
    p.wait_ns = g_wait_limit_ns.load();
    if (mask && bias) return launch_fwd_bf16<kFwdNsub, true, true>(maps, p, stream);
    if (mask) return launch_fwd_bf16<kFwdNsub, true, false>(maps, p, stream);
    if (bias) return launch_fwd_bf16<kFwdNsub, false, true>(maps, p, stream);
    return launch_fwd_bf16<kFwdNsub, false, false>(maps, p, stream);
}

// ---------------------------------------------------------------- backward
struct BwdWorkspace {
    size_t d_off, nl_off, doa_off, dol_off, dqacc_off, biast_off, part_off, total;
    int groups, db_groups;
};

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

BwdWorkspace bwd_workspace(const evo_shape_t& sh, evo_dtype_t dt) {
    BwdWorkspace w{};
    const size_t rows = (size_t)sh.B * sh.S * sh.H * sh.N;       // logit rows
    const size_t T = rows * (size_t)sh.C;                         // elements of a per-row tensor
    const size_t pair = (size_t)sh.B * sh.H * sh.N * sh.N;
    size_t off = 0;
    w.d_off = off;
    off = align256(off + rows * 4);
    if (dt == EVO_DTYPE_BF16) {
        // row terms -D and nl are stored with the query axis padded to whole tiles
        const size_t padded_rows = (size_t)sh.B * sh.S * sh.H * (size_t)((sh.N + 127) / 128 * 128);
        off = align256(w.d_off + padded_rows * 4);
        w.groups = evo::bwd::num_groups(sh.B, sh.S, sh.N, sh.H);
        // the d_pair_bias kernel's row groups, chosen for a 148-SM B200 (a pure function
        // of the shape, so that the workspace size never depends on the device)
        w.db_groups = evo::dbias::num_groups(sh.B, sh.S, sh.N, sh.H, 148);
        w.nl_off = off;
        off = align256(off + padded_rows * 4);
        w.doa_off = off;
        off = align256(off + T * 2);
        w.dol_off = off;
        off = align256(off + T * 2);
        w.dqacc_off = off;
        off = align256(off + T * 4);
        w.biast_off = off;
        off = align256(off + pair * 2);
        w.part_off = off;
        off = align256(off + pair * 4 * (size_t)(w.db_groups > 1 ? w.db_groups : 0));
    }
    w.total = off;
    return w;
}

evo_status_t bwd_f32(const evo_shape_t& sh, evo::simt::Args a, cudaStream_t stream) {
    (void)sh;
    const int64_t rows = (int64_t)a.B * a.S * a.N * a.H;
    evo::simt::bwd_pre_kernel<float><<<(unsigned)((rows + 255) / 256), 256, 0, stream>>>(a);
    const dim3 grid((unsigned)((a.N + evo::simt::kRowsPerCta - 1) / evo::simt::kRowsPerCta), (unsigned)a.S,
                    (unsigned)(a.B * a.H));
    evo::simt::bwd_dq_kernel<float><<<grid, evo::simt::kWarps * 32, 0, stream>>>(a);
    evo::simt::bwd_dkdv_kernel<float><<<grid, evo::simt::kWarps * 32, 0, stream>>>(a);
    const dim3 gb((unsigned)((a.N + 127) / 128), (unsigned)a.N, (unsigned)(a.B * a.H));
    evo::simt::bwd_dbias_kernel<float><<<gb, 128, 0, stream>>>(a);
    g_launches += 4;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

// ---------------------------------------------------------------- fused pre-attention projection
// maps[0]: w [c_in, n_out], boxes of 64 columns x 64 rows; maps[1]: y [rows, n_out] (pitch ldy),
// boxes of 64 columns x 32 rows.  Persistent grid: n_groups x (CTAs per group), at most one per SM.
template <int BNO, int CIN>
evo_status_t launch_ln_linear(const CUtensorMap* maps, const evo::proj::LnParams& p, cudaStream_t stream) {
    using L = evo::proj::PLayout<BNO, CIN>;
    auto kern = evo::proj::ln_linear_kernel<BNO, CIN>;
    static cudaError_t attr = set_smem(kern, L::bytes);
    if (attr != cudaSuccess) return EVO_ERR_CUDA;
    const int64_t nrb = (p.rows + evo::proj::BM - 1) / evo::proj::BM;
    // the widest column group whose w chunks stay resident; else all columns in one group
    const int nsl = p.n_out / BNO, kc = CIN / evo::proj::KBOX;
    int gsl = nsl;
    if (nsl * kc > L::NW) {
        for (int g = nsl; g >= 1; --g)
            if (nsl % g == 0 && g * kc <= L::NW) { gsl = g; break; }
    }
    evo::proj::LnParams q = p;
    q.gsl = gsl;
    const int64_t ngr = nsl / gsl;
    const int64_t grid = ngr * std::min<int64_t>(nrb, std::max<int64_t>(1, sm_count() / ngr));
    if (grid > 0x7fffffff) return EVO_ERR_UNSUPPORTED;
    {
        evo::timing::Scope t(EVO_PHASE_PROJ, stream);
        kern<<<(unsigned)grid, evo::proj::THREADS, L::bytes, stream>>>(maps[0], maps[1], q);
    }
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

template <int BNO>
evo_status_t launch_ln_linear_cin(const CUtensorMap* maps, const evo::proj::LnParams& p, cudaStream_t stream) {
    switch (p.c_in) {
        case 64: return launch_ln_linear<BNO, 64>(maps, p, stream);
        case 128: return launch_ln_linear<BNO, 128>(maps, p, stream);
        case 192: return launch_ln_linear<BNO, 192>(maps, p, stream);
        case 256: return launch_ln_linear<BNO, 256>(maps, p, stream);
    }
    return EVO_ERR_UNSUPPORTED;
}

template <int CPL, int LPR, int HQ>
evo_status_t launch_pair_bias(const evo::proj::PbParams& p, int64_t total, cudaStream_t stream) {
    auto kern = evo::proj::pair_bias_kernel<CPL, LPR, HQ>;
    static cudaError_t attr = set_smem(kern, evo::proj::PB_SMEM);
    if (attr != cudaSuccess) return EVO_ERR_CUDA;
    const int64_t blocks = (total + evo::proj::PB_ROWS - 1) / evo::proj::PB_ROWS;
    const size_t shm = (size_t)p.c_z * 4 * HQ * sizeof(float) + (size_t)4 * HQ * evo::proj::PB_ROWS * 2;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, evo::proj::PB_THREADS, shm) != cudaSuccess)
        return EVO_ERR_CUDA;
    const int grid = (int)std::min<int64_t>(blocks, (int64_t)sm_count() * std::max(per_sm, 1));
    {
        evo::timing::Scope t(EVO_PHASE_PAIR_BIAS, stream);
        kern<<<grid, evo::proj::PB_THREADS, shm, stream>>>(p);
    }
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

template <int HQ>
evo_status_t launch_pair_bias_rows(const evo::proj::PbParams& p, int64_t total, cudaStream_t stream) {
    auto kern = evo::proj::pair_bias_rows_kernel<HQ>;
    static cudaError_t attr = set_smem(kern, evo::proj::PBR_SMEM);
    if (attr != cudaSuccess) return EVO_ERR_CUDA;
    const int64_t ch = p.c_z / 8;
    const size_t shm = (size_t)evo::proj::PBR_THREADS * (ch | 1) * 16 + (size_t)p.c_z * 4 * HQ * 4 +
                       (size_t)(1 + evo::proj::PBR_THREADS / 32) * 4 * HQ * 4;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, evo::proj::PBR_THREADS, shm) != cudaSuccess)
        return EVO_ERR_CUDA;
    const int64_t blocks = (total + evo::proj::PBR_THREADS - 1) / evo::proj::PBR_THREADS;
    const int grid = (int)std::min<int64_t>(blocks, (int64_t)sm_count() * std::max(per_sm, 1));
    {
        evo::timing::Scope t(EVO_PHASE_PAIR_BIAS, stream);
        kern<<<grid, evo::proj::PBR_THREADS, shm, stream>>>(p);
    }
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

template <int CPL, int LPR>
evo_status_t launch_pair_bias_h(const evo::proj::PbParams& p, int64_t total, cudaStream_t stream) {
    switch ((p.H + 3) / 4) {
        case 1: return launch_pair_bias<CPL, LPR, 1>(p, total, stream);
        case 2: return launch_pair_bias<CPL, LPR, 2>(p, total, stream);
        case 3: return launch_pair_bias<CPL, LPR, 3>(p, total, stream);
        case 4: return launch_pair_bias<CPL, LPR, 4>(p, total, stream);
    }
    return EVO_ERR_UNSUPPORTED;
}

// z[m] (M x Nc) = scale * a[m]^T b[m] (incoming: a, b are K x M, K x Nc) or a[m] b[m]^T
// (outgoing: a, b are M x K, Nc x K) for the `batch` matrices m, on the tri_mul kernel.
evo_status_t launch_contraction(const void* a, const void* bb, void* z, int64_t M, int64_t Nc, int64_t K,
                                int64_t batch, bool incoming, float scale, int phase, cudaStream_t stream) {
    using namespace evo::trimul;
    CUtensorMap maps[3];
    std::memset(maps, 0, sizeof(maps));
    const bool ok = incoming ? (evo::tma::batch_bf16(&maps[0], a, M, K, batch, 64, 64) &&
                                evo::tma::batch_bf16(&maps[1], bb, Nc, K, batch, 64, 64))
                             : (evo::tma::batch_bf16(&maps[0], a, K, M, batch, 64, BM) &&
                                evo::tma::batch_bf16(&maps[1], bb, K, Nc, batch, 64, BN));
    if (!ok || !evo::tma::batch_bf16(&maps[2], z, Nc, M, batch, 64, 32)) return EVO_ERR_CUDA;
    TriParams p{};
    p.M = (int)M; p.Nc = (int)Nc; p.K = (int)K; p.BC = (int)batch; p.incoming = incoming ? 1 : 0; p.scale = scale;
    p.tiles_i = (int)((M + BM - 1) / BM); p.tiles_j = (int)((Nc + BN - 1) / BN);
    const int64_t tiles = batch * p.tiles_i * p.tiles_j;
    static cudaError_t attr = set_smem(tri_mul_kernel, TLayout::bytes);
    if (attr != cudaSuccess) return EVO_ERR_CUDA;
    const int grid = (int)std::min<int64_t>(tiles, sm_count());
    {
        evo::timing::Scope t(phase, stream);
        tri_mul_kernel<<<grid, THREADS, TLayout::bytes, stream>>>(maps[0], maps[1], maps[2], p);
    }
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

// ---------------------------------------------------------------- 8-bit projection
bool dtype_ok(evo_dtype_t d) { return d == EVO_DTYPE_BF16 || d == EVO_DTYPE_F32; }
int64_t elem_bytes(evo_dtype_t d) { return d == EVO_DTYPE_BF16 ? 2 : 4; }

// Whether rows of `cols` elements at pitch `ld` can be moved in 16-byte pieces.
bool rows_vec(const void* ptr, int64_t cols, int64_t ld, int64_t e) {
    return !ptr || (aligned(ptr, 16) && cols * e % 16 == 0 && ld * e % 16 == 0);
}
// The same, where a pitch that is never stepped along (one row) does not matter.
bool rows_vec(const void* ptr, int64_t rows, int64_t cols, int64_t ld, int64_t e) {
    return rows_vec(ptr, cols, rows > 1 ? ld : 0, e);
}

// How a row is held: nv fragments of 256 columns in each of wpr warps, and the threads of a block.
struct RowSplit {
    int nv, wpr, threads;
};
constexpr int64_t kMaxRowCols = 32768;
// Forward: as many rows as fit in blocks of 8 warps, two fragments per warp above 2048 columns, up to
// 16 warps (9763 rows of 4097 columns in fp32: four fragments in five warps took 251 us where this
// takes 151).
// Above 8192 columns up to 32 warps of four, whose registers spill (4096 x 12288 in bf16: 162 us, 55 at
// the copy's rate).
RowSplit row_split(int64_t cols) {
    const int chunks = (int)((cols + 255) / 256);
    const int nv = chunks <= 8 ? 1 : chunks <= 32 ? 2 : 4, wpr = (chunks + nv - 1) / nv;
    return {nv, wpr, 32 * (wpr <= 8 ? 8 / wpr * wpr : wpr)};
}
// Backward: twice the values per column, so one fragment per warp up to 8192 columns; above, four,
// which spill (4096 x 12288 in bf16: 281 us, 62 at the copy's rate).
RowSplit row_split_bwd(int64_t cols) {
    const int chunks = (int)((cols + 255) / 256);
    const int nv = chunks <= 32 ? 1 : 4, wpr = (chunks + nv - 1) / nv;
    return {nv, wpr, 32 * (wpr <= 8 ? 8 / wpr * wpr : wpr)};
}

// Blocks for `rows` of which a block takes `per` at a time: at most what runs at once.  The answer for
// each block size is kept by the kernel's launcher (asking costs a microsecond).
using Resident = std::atomic<int>[33];
template <typename K>
int walking_grid(K kernel, int threads, int64_t rows, int64_t per, Resident& kept) {
    int n = kept[threads / 32].load();
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess || n < 1) n = 1;
        kept[threads / 32].store(n);
    }
    return (int)std::min<int64_t>((rows + per - 1) / per, (int64_t)sm_count() * n);
}

// f(T{}, VEC) with the call's type and alignment as types.
template <typename F>
void by_type(evo_dtype_t dtype, bool vec, F f) {
    auto with = [&](auto t) { vec ? f(t, std::true_type{}) : f(t, std::false_type{}); };
    dtype == EVO_DTYPE_BF16 ? with(__nv_bfloat16{}) : with(float{});
}

template <typename T, bool VEC, int NV, int R, int THREADS, bool SMALL>
void launch_norm_eps(const evo::fp8::NormParams& p, const RowSplit& s, cudaStream_t stream) {
    auto kern = evo::fp8::add_rms_norm_kernel<T, VEC, NV, R, THREADS, SMALL>;
    static Resident kept;
    const int grid = walking_grid(kern, s.threads, p.rows, s.threads / 32 / s.wpr * R, kept);
    kern<<<grid, s.threads, 0, stream>>>(p, s.wpr);
}
template <typename T, bool VEC, int NV, int R, int THREADS>
void launch_norm_as(const evo::fp8::NormParams& p, const RowSplit& s, cudaStream_t stream) {
    if (p.eps < 0x1p-20f) return launch_norm_eps<T, VEC, NV, R, THREADS, true>(p, s, stream);
    return launch_norm_eps<T, VEC, NV, R, THREADS, false>(p, s, stream);
}
template <typename T, bool VEC>
void launch_norm(const evo::fp8::NormParams& p, const RowSplit& s, cudaStream_t stream) {
    constexpr int R = sizeof(T) == 2 ? 2 : 1;    // fp32 rows fill the registers one at a time
    if (s.nv == 4) return launch_norm_as<T, VEC, 4, 1, 1024>(p, s, stream);
    if (s.threads > 256) return launch_norm_as<T, VEC, 2, 1, 512>(p, s, stream);
    if (s.wpr == 1) return launch_norm_as<T, VEC, 1, R, 256>(p, s, stream);
    if (s.nv == 1) return launch_norm_as<T, VEC, 1, 1, 256>(p, s, stream);
    return launch_norm_as<T, VEC, 2, 1, 256>(p, s, stream);
}

template <typename T, bool VEC, int NV, int R, int THREADS>
void launch_norm_bwd_as(const evo::fp8::NormBwdParams& p, const RowSplit& s, int grid, cudaStream_t stream) {
    const int warps = s.threads / 32;
    const size_t shm = p.part && warps > s.wpr ? (size_t)warps * NV * 256 * sizeof(float) : 0;
    evo::fp8::rms_bwd_kernel<T, VEC, NV, R, THREADS><<<grid, s.threads, shm, stream>>>(p, s.wpr);
}
template <typename T, bool VEC>
void launch_norm_bwd(const evo::fp8::NormBwdParams& p, const RowSplit& s, int grid, cudaStream_t stream) {
    constexpr int R = sizeof(T) == 2 ? 2 : 1;
    if (s.nv == 4) return launch_norm_bwd_as<T, VEC, 4, 1, 1024>(p, s, grid, stream);
    if (s.threads > 640) return launch_norm_bwd_as<T, VEC, 1, 1, 1024>(p, s, grid, stream);
    if (s.wpr == 1) return launch_norm_bwd_as<T, VEC, 1, R, 256>(p, s, grid, stream);
    return launch_norm_bwd_as<T, VEC, 1, 1, 640>(p, s, grid, stream);
}
// Blocks of the norm's backward, each of which leaves one partial row of d_weight: a pure
// function of the sizes (for the workspace query), for either type.
int64_t norm_bwd_blocks(int64_t rows, int64_t cols) {
    const RowSplit s = row_split_bwd(cols);
    const int64_t per = s.threads / 32 / s.wpr;
    return std::min<int64_t>((rows + per - 1) / per, 148 * (s.threads <= 256 ? 2 : 1));
}

template <typename T, bool VEC>
void launch_quantize(const evo::fp8::QuantParams& p, bool square, cudaStream_t s) {
    using namespace evo::fp8;
    const unsigned grid = (unsigned)((p.rows + 127) / 128 * ((p.cols + 127) / 128));
    if (!p.qt && !square)
        quantize_tile_kernel<T, VEC, false, true, false><<<grid, 512, 0, s>>>(p);
    else if (!p.qt)
        quantize_tile_kernel<T, VEC, true, true, false><<<grid, 512, 0, s>>>(p);
    else if (square && p.q)
        quantize_tile_kernel<T, VEC, true, true, true><<<grid, 512, 0, s>>>(p);
    else if (square)
        quantize_tile_kernel<T, VEC, true, false, true><<<grid, 512, 0, s>>>(p);
    else if (p.q)
        quantize_tile_kernel<T, VEC, false, true, true><<<grid, 512, 0, s>>>(p);
    else
        quantize_tile_kernel<T, VEC, false, false, true><<<grid, 512, 0, s>>>(p);
}

// The checks and the launch that evo_quantize_fp8 and evo_quantize_fp8_both share: p.q, p.qt or both.
evo_status_t quantize(const evo::fp8::QuantParams& p, evo_dtype_t dtype, bool square, cudaStream_t s) {
    const int64_t e = elem_bytes(dtype);
    if (!p.x || p.ldx < 0 || !aligned(p.x, e)) return EVO_ERR_INVALID_ARG;
    auto bad = [](const void* q, int64_t ld, int64_t rows, int64_t cols, const float* sc, int64_t sr, int64_t sg) {
        return q && (!sc || (rows > 1 && ld < cols) || sr < 1 || sg < 1 || !aligned(sc, 4));
    };
    if (bad(p.q, p.ldq, p.rows, p.cols, p.scale, p.s_row, p.s_grp) ||
        bad(p.qt, p.ldqt, p.cols, p.rows, p.scale_t, p.st_row, p.st_grp))
        return EVO_ERR_INVALID_ARG;
    if (!aligned(p.q, 16) || !aligned(p.qt, 16) || (p.q && p.rows > 1 && p.ldq % 16 != 0) ||
        (p.qt && p.cols > 1 && p.ldqt % 16 != 0))
        return EVO_ERR_UNSUPPORTED;
    if ((p.rows + 127) / 128 > 0x7fffffff / ((p.cols + 127) / 128)) return EVO_ERR_UNSUPPORTED;
    const bool vec = rows_vec(p.x, p.rows, p.cols, p.ldx, e);
    by_type(dtype, vec, [&](auto t, auto v) { launch_quantize<decltype(t), decltype(v)::value>(p, square, s); });
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

// Dynamic shared memory above 48 KB is granted per kernel and device.
template <typename K>
bool grant_smem(K kernel, int bytes, std::atomic<uint64_t>* granted) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return false;
    const uint64_t bit = 1ull << (dev & 63);
    if (granted[dev >> 6].load() & bit) return true;
    if (set_smem(kernel, bytes) != cudaSuccess) return false;
    granted[dev >> 6].fetch_or(bit);
    return true;
}

// The kernel hands registers between its warps, which only works out when it was compiled to
// the count that the split was written for.  S: CTAs that join a tile.
template <typename T, bool SW_ROWS, class L>
evo_status_t launch_linear_as(const evo::fp8::LinParams& p, int S, cudaStream_t stream) {
    namespace f8 = evo::fp8;
    auto kern = f8::linear_kernel<T, SW_ROWS, L>;
    static std::atomic<uint64_t> granted[4];
    if (!grant_smem(kern, L::smem, granted)) return EVO_ERR_CUDA;
    static const int regs = [&] {
        cudaFuncAttributes fa{};
        return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs != L::LAUNCH_REGS) return EVO_ERR_CUDA;
    const int64_t tm = (p.M + f8::BM - 1) / f8::BM;
    const int64_t tiles = tm * ((p.N + L::BN - 1) / L::BN) * (L::PART ? p.parts : 1);
    if (tiles * S > 0x7fffffff - 65536) return EVO_ERR_UNSUPPORTED;
    const int64_t y_rows = L::PART ? tm * f8::BM * p.parts : p.M;
    const int64_t e = sizeof(T);
    const bool tma_out = !L::JOIN && aligned(p.y, 16) && (p.M == 1 || p.ldy * e % 16 == 0);
    CUtensorMap maps[3];
    std::memset(maps, 0, sizeof(maps));
    if (!evo::tma::matrix_u8(&maps[0], p.x, p.M, p.K, p.ldx, f8::BM) ||
        !evo::tma::matrix_u8(&maps[1], p.w, p.N, p.K, p.ldw, L::BN) ||
        (tma_out && !evo::tma::boxes_out(&maps[2], p.y, y_rows, p.N, p.ldy, (int)e)))
        return EVO_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(L::JOIN ? tiles * S : std::min<int64_t>(tiles, sm_count())));
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)S;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], p, tma_out ? 1 : 0);
    g_launches += 1;
    return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

// Largest size of a product's axis: every index and step of the kernels stays below 2^31.
constexpr int64_t kMaxProduct = (int64_t)0x7fffffff - 65536;

// Which form a product takes: Few with S warps a row of w, Wide (S = 1), Split with S CTAs a tile, or
// Parts with S runs a tile.
struct LinPlan {
    enum Form { FEW, WIDE, SPLIT, PARTS } form;
    int S;
    size_t workspace;            // bytes
    int64_t ld;                  // Parts: pitch of the workspace's rows
};
// A pure function of the sizes.  Up to two rows: Few (1 x 8192 x 8192 18.3 us, in parts 22.7; two
// rows 23.4 and 23.3; four 34.9 and 24).  Else the costs are in blocks of 128 x 256 x 128 on one SM
// (0.6 us): a block of 128 columns takes as long as one of 256 (both wait more than they add), a
// CTA's start, last step and end about five, a second launch with its pass over the parts four more.
// The counts of SMs and of clusters at once are a B200's.
// Measured both ways: 1024 x 131072 x 256 takes 99 us in clusters of 6, 57 in parts.
LinPlan plan_linear(int64_t M, int64_t N, int64_t K) {
    namespace f8 = evo::fp8;
    // clusters of 1 to 8 CTAs that run at once on 148 SMs (a cluster lies in one GPC)
    static const int at_once[9] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
    const int64_t tm = (M + f8::BM - 1) / f8::BM, blocks = (K + f8::BK - 1) / f8::BK;
    const int64_t wide = tm * ((N + 255) / 256), narrow = tm * ((N + 127) / 128);
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    if (M <= 2) {
        // enough warps to keep the GPU's loads in flight, each with a chunk at least
        int ks = 1;
        while (ks < f8::few::WARPS && N * ks < 148 * 16 * f8::few::R && K > ks * f8::few::CHUNK) ks *= 2;
        return {LinPlan::FEW, ks, 0, 0};
    }
    LinPlan best{LinPlan::WIDE, 1, 0, 0};
    int64_t t_best = up(wide, 148) * (blocks + 5);
    if (narrow > 148) return best;
    for (int S = 1; S <= 8 && (S == 1 || blocks >= 2 * S); ++S) {
        const int64_t t = up(narrow, at_once[S]) * (up(blocks, S) + 5);
        if (t < t_best) {
            t_best = t;
            best = {LinPlan::SPLIT, S, 0, 0};
        }
    }
    const int64_t S = std::min<int64_t>(148 / std::max<int64_t>(wide, 1), blocks / 2);
    if (S > 1 && up(blocks, S) + 9 < t_best) {
        const int64_t ld = up(N, 4) * 4;
        best = {LinPlan::PARTS, (int)S, (size_t)(S * tm * f8::BM * ld) * sizeof(float), ld};
    }
    return best;
}

template <typename T, bool SW_ROWS>
evo_status_t launch_linear_few(const evo::fp8::LinParams& p, int ks, cudaStream_t stream) {
    namespace few = evo::fp8::few;
    const int64_t rows = (int64_t)few::R * (few::WARPS / ks);
    const unsigned grid = (unsigned)((p.N + rows - 1) / rows);
    if (p.M == 1) few::linear_kernel<T, SW_ROWS, 1><<<grid, 32 * few::WARPS, 0, stream>>>(p, ks);
    else few::linear_kernel<T, SW_ROWS, 2><<<grid, 32 * few::WARPS, 0, stream>>>(p, ks);
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

template <typename T, bool SW_ROWS>
evo_status_t launch_linear(const evo::fp8::LinParams& p, const LinPlan& plan, void* workspace, cudaStream_t stream) {
    namespace f8 = evo::fp8;
    if (plan.form == LinPlan::FEW) return launch_linear_few<T, SW_ROWS>(p, plan.S, stream);
    if (plan.form == LinPlan::WIDE)                        // both sides are measured beside linear_kernel
        return p.K > 8 * f8::BK ? launch_linear_as<T, SW_ROWS, f8::Long>(p, 1, stream)
                                : launch_linear_as<T, SW_ROWS, f8::Wide>(p, 1, stream);
    if (plan.form == LinPlan::SPLIT) return launch_linear_as<T, SW_ROWS, f8::Split>(p, plan.S, stream);
    f8::LinParams parts = p;
    parts.y = workspace;
    parts.ldy = plan.ld;
    parts.bias = nullptr;
    parts.parts = plan.S;
    const evo_status_t st = launch_linear_as<float, SW_ROWS, f8::Parts>(parts, 1, stream);
    if (st != EVO_OK) return st;
    const int64_t items = (int64_t)p.M * ((p.N + 3) / 4), rows = (int64_t)(p.M + f8::BM - 1) / f8::BM * f8::BM;
    const int grid = (int)std::min<int64_t>((items + 255) / 256, 148 * 8);
    f8::sum_parts_kernel<T><<<grid, 256, 0, stream>>>(static_cast<const float*>(workspace), plan.ld, rows, plan.S, p);
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

}  // namespace

extern "C" {

const char* evo_status_string(evo_status_t s) {
    switch (s) {
        case EVO_OK: return "EVO_OK";
        case EVO_ERR_INVALID_ARG: return "EVO_ERR_INVALID_ARG";
        case EVO_ERR_UNSUPPORTED: return "EVO_ERR_UNSUPPORTED";
        case EVO_ERR_WORKSPACE_TOO_SMALL: return "EVO_ERR_WORKSPACE_TOO_SMALL";
        case EVO_ERR_CUDA: return "EVO_ERR_CUDA";
        case EVO_ERR_DEVICE_TIMEOUT: return "EVO_ERR_DEVICE_TIMEOUT";
    }
    return "EVO_ERR_UNKNOWN";
}

int evo_attn_version(void) { return EVO_VERSION; }

uint64_t evo_attn_set_wait_limit_ns(uint64_t ns) { return g_wait_limit_ns.exchange(ns); }

evo_status_t evo_exp2_fma(const float* x, float* y, int64_t n, void* stream) {
    if (n < 0 || (n > 0 && (!x || !y))) return EVO_ERR_INVALID_ARG;
    if (n == 0) return EVO_OK;
    if (!aligned(x, 4) || !aligned(y, 4)) return EVO_ERR_INVALID_ARG;
    const int blocks = (int)std::min<int64_t>((n + 511) / 512, 148 * 8);
    exp2_fma_kernel<<<blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(x, y, n);
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

uint64_t evo_attn_launch_count(void) { return g_launches.load(); }

evo_status_t evo_attn_timing_enable(int on) { return evo::timing::enable(on); }

evo_status_t evo_attn_timing_collect(evo_timing_t* out) { return evo::timing::collect(out); }

evo_status_t evo_attn_device_status(int clear) {
    if (cudaDeviceSynchronize() != cudaSuccess) return EVO_ERR_CUDA;
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_evo_status, sizeof(v)) != cudaSuccess) return EVO_ERR_CUDA;
    if (clear) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_evo_status, &z, sizeof(z)) != cudaSuccess) return EVO_ERR_CUDA;
    }
    return v == 0 ? EVO_OK : EVO_ERR_DEVICE_TIMEOUT;
}

size_t evo_attn_bwd_workspace_bytes(const evo_shape_t* shape, evo_dtype_t dtype) {
    if (check_shape(shape) != EVO_OK) return 0;
    if (dtype != EVO_DTYPE_BF16 && dtype != EVO_DTYPE_F32) return 0;
    return bwd_workspace(*shape, dtype).total;
}

evo_status_t evo_attn_fwd(const evo_shape_t* shape, evo_dtype_t dtype, const void* q, const void* k,
                          const void* v, const void* g, const evo_strides_t* in_str, const void* mask_bias,
                          const void* pair_bias, void* out, void* out_lo, const evo_strides_t* out_str, float* lse,
                          void* stream) {
    evo_status_t st = check_shape(shape);
    if (st != EVO_OK) return st;
    if (dtype != EVO_DTYPE_BF16 && dtype != EVO_DTYPE_F32) return EVO_ERR_INVALID_ARG;
    if (!strides_ok(in_str) || !strides_ok(out_str)) return EVO_ERR_INVALID_ARG;
    if (empty_call(shape)) return EVO_OK;
    if (!q || !k || !v || !g || !out || !lse) return EVO_ERR_INVALID_ARG;
    if (!non_overlapping(*shape, *out_str)) return EVO_ERR_INVALID_ARG;
    if (!aligned(lse, 4)) return EVO_ERR_INVALID_ARG;
    if (out_lo && out_lo == out) return EVO_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == EVO_DTYPE_F32) {
        if (shape->C > evo::simt::kMaxC) return EVO_ERR_UNSUPPORTED;
        for (const void* p : {q, k, v, g, (const void*)out})
            if (!aligned(p, 4)) return EVO_ERR_INVALID_ARG;
        if (shape->S > 65535) return EVO_ERR_UNSUPPORTED;
        return fwd_f32(*shape, q, k, v, g, *in_str, mask_bias, pair_bias, out, *out_str, lse, s);
    }
    return fwd_bf16(*shape, q, k, v, g, *in_str, mask_bias, pair_bias, out, out_lo, *out_str, lse, s);
}

evo_status_t evo_attn_bwd(const evo_shape_t* shape, evo_dtype_t dtype, const void* q, const void* k,
                          const void* v, const void* g, const evo_strides_t* in_str, const void* mask_bias,
                          const void* pair_bias, const void* out, const void* out_lo, const void* dout,
                          const evo_strides_t* out_str, const float* lse, void* dq, void* dk, void* dv,
                          void* dg, const evo_strides_t* grad_str, float* d_pair_bias, void* workspace,
                          size_t workspace_bytes, void* stream) {
    evo_status_t st = check_shape(shape);
    if (st != EVO_OK) return st;
    if (dtype != EVO_DTYPE_BF16 && dtype != EVO_DTYPE_F32) return EVO_ERR_INVALID_ARG;
    if (!strides_ok(in_str) || !strides_ok(out_str) || !strides_ok(grad_str)) return EVO_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (shape->B == 0 || shape->H == 0 || shape->N == 0) return EVO_OK;
    if (!d_pair_bias || !aligned(d_pair_bias, 4)) return EVO_ERR_INVALID_ARG;
    const size_t pair_bytes = (size_t)shape->B * shape->H * shape->N * shape->N * sizeof(float);
    if (shape->S == 0) {
        return cudaMemsetAsync(d_pair_bias, 0, pair_bytes, s) == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
    }
    if (!q || !k || !v || !g || !out || !dout || !lse || !dq || !dk || !dv || !dg) return EVO_ERR_INVALID_ARG;
    if (!non_overlapping(*shape, *grad_str)) return EVO_ERR_INVALID_ARG;
    const BwdWorkspace ws = bwd_workspace(*shape, dtype);
    if (ws.total > 0 && (!workspace || workspace_bytes < ws.total)) return EVO_ERR_WORKSPACE_TOO_SMALL;
    if (workspace && !aligned(workspace, 256)) return EVO_ERR_INVALID_ARG;
    if (!aligned(lse, 4)) return EVO_ERR_INVALID_ARG;

    evo::simt::Args a{};
    a.B = (int)shape->B; a.S = (int)shape->S; a.N = (int)shape->N; a.H = (int)shape->H; a.C = (int)shape->C;
    a.q = q; a.k = k; a.v = v; a.g = g; a.in = to_strides(*in_str);
    a.mask = mask_bias; a.bias = pair_bias; a.out = out; a.dout = dout; a.os = to_strides(*out_str);
    a.lse = const_cast<float*>(lse);
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.gs = to_strides(*grad_str);
    a.dbias = d_pair_bias;
    a.D = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.d_off);
    if (dtype == EVO_DTYPE_F32) {
        if (shape->C > evo::simt::kMaxC) return EVO_ERR_UNSUPPORTED;
        for (const void* p : {q, k, v, g, out, dout, (const void*)dq, (const void*)dk, (const void*)dv,
                              (const void*)dg})
            if (!aligned(p, 4)) return EVO_ERR_INVALID_ARG;
        if (shape->S > 65535 || shape->N > 65535) return EVO_ERR_UNSUPPORTED;
        evo::timing::Scope t(EVO_PHASE_BWD_ALL, s);
        return bwd_f32(*shape, a, s);
    }
    evo::bwd::Call c{};
    c.shape = *shape;
    c.q = q; c.k = k; c.v = v; c.g = g; c.in = *in_str;
    c.mask = mask_bias; c.bias = pair_bias; c.out = out; c.out_lo = out_lo; c.dout = dout; c.os = *out_str;
    c.lse = lse;
    c.dq = dq; c.dk = dk; c.dv = dv; c.dg = dg; c.gs = *grad_str; c.dbias = d_pair_bias;
    c.ws = static_cast<char*>(workspace);
    c.d_off = ws.d_off; c.nl_off = ws.nl_off; c.doa_off = ws.doa_off; c.dol_off = ws.dol_off;
    c.dqacc_off = ws.dqacc_off;
    c.biast_off = ws.biast_off; c.part_off = ws.part_off; c.groups = ws.groups; c.db_groups = ws.db_groups;
    c.wait_ns = g_wait_limit_ns.load();
    int launched = 0;
    evo_status_t rs;
    {
        evo::timing::Scope t(EVO_PHASE_BWD_ALL, s);
        rs = evo::bwd::run(c, s, &launched);
    }
    g_launches += (uint64_t)launched;
    return rs;
}

// ---------------------------------------------------------------- no-allocation backward
// Scratch area of evo_attn_bwd_noalloc.  Host code must not pass the array's
// name to a kernel: on the host it is only a stand-in for the device object,
// whose address is looked up once per device below.
static __device__ __align__(256) unsigned char g_evo_noalloc_ws[EVO_ATTN_NOALLOC_WORKSPACE_BYTES];

static std::mutex g_noalloc_mu;
struct NoallocSlot {
    unsigned long long ctx_id;   // the context the address belongs to (0: none yet)
    void* addr;
};
static NoallocSlot g_noalloc_slot[256] = {};

// Identifier of the calling thread's current context, unique among the
// contexts this process creates (cuCtxGetId), or 0 when it cannot be had.  A
// context created after cudaDeviceReset gets a new identifier, so an address
// cached for the old context is never reused.
static unsigned long long current_ctx_id() {
    static std::once_flag once;
    static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
    static PFN_cuCtxGetId_v12000 get_id = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
        p = nullptr;
        if (cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
    });
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (!get_current || !get_id || get_current(&ctx) != CUDA_SUCCESS || !ctx || get_id(ctx, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

// Device address of the scratch array in the current device's context.  It
// is looked up (cudaGetSymbolAddress, with that device current) on the first
// call in each context and cached; a later call in the same context reuses
// it, a call in a new context (after cudaDeviceReset) looks it up again.
// Without a context identifier it is looked up on every call.
static evo_status_t noalloc_workspace(void** addr) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return EVO_ERR_CUDA;
    if (dev < 0 || dev >= 256) return EVO_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    unsigned long long id = current_ctx_id();
    NoallocSlot& slot = g_noalloc_slot[dev];
    if (id == 0 || slot.ctx_id != id || !slot.addr) {
        void* a = nullptr;
        if (cudaGetSymbolAddress(&a, g_evo_noalloc_ws) != cudaSuccess || !a) return EVO_ERR_CUDA;
        if (id == 0) id = current_ctx_id();      // the lookup may have made the context current
        slot.ctx_id = id;
        slot.addr = a;
    }
    *addr = slot.addr;
    return EVO_OK;
}

evo_status_t evo_ln_linear(int64_t rows, int64_t c_in, int64_t n_out, const void* x, const float* ln_w,
                           const float* ln_b, float eps, const void* w, const float* bias, void* y, int64_t ldy,
                           void* stream) {
    if (rows < 0 || c_in <= 0 || n_out <= 0 || ldy < n_out || !(eps >= 0.f)) return EVO_ERR_INVALID_ARG;
    if (rows == 0) return EVO_OK;
    if (!x || !w || !y) return EVO_ERR_INVALID_ARG;
    if (c_in % evo::proj::KBOX != 0 || c_in > evo::proj::MAX_CIN || n_out % 128 != 0 || ldy % 8 != 0)
        return EVO_ERR_UNSUPPORTED;
    if (rows > (int64_t)0x7fffffff - evo::proj::BM || n_out > (int64_t)0x7fffffff) return EVO_ERR_UNSUPPORTED;
    for (const void* q : {x, w, (const void*)y})
        if (!aligned(q, 16)) return EVO_ERR_UNSUPPORTED;
    if (bias && !aligned(bias, 16)) return EVO_ERR_UNSUPPORTED;      // read as float4
    for (const void* q : {(const void*)ln_w, (const void*)ln_b})
        if (q && !aligned(q, 4)) return EVO_ERR_INVALID_ARG;
    CUtensorMap maps[2];
    std::memset(maps, 0, sizeof(maps));
    if (!evo::tma::matrix_bf16(&maps[0], w, c_in, n_out, n_out, 64) ||
        !evo::tma::matrix_bf16(&maps[1], y, rows, n_out, ldy, 32))
        return EVO_ERR_CUDA;
    evo::proj::LnParams p{};
    p.rows = (int)rows; p.c_in = (int)c_in; p.n_out = (int)n_out; p.eps = eps;
    p.x = static_cast<const __nv_bfloat16*>(x); p.ln_w = ln_w; p.ln_b = ln_b; p.bias = bias;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return n_out % 256 == 0 ? launch_ln_linear_cin<256>(maps, p, s) : launch_ln_linear_cin<128>(maps, p, s);
}

evo_status_t evo_ln_pair_bias(int64_t B, int64_t N, int64_t c_z, int64_t H, const void* z, const float* ln_w,
                              const float* ln_b, float eps, const void* w, const float* bias, void* pair_bias,
                              void* stream) {
    if (B < 0 || N < 0 || c_z <= 0 || H <= 0 || !(eps >= 0.f)) return EVO_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return EVO_OK;
    if (!z || !w || !pair_bias) return EVO_ERR_INVALID_ARG;
    if (c_z % 8 != 0 || c_z > 1024 || H > evo::proj::PB_MAX_H) return EVO_ERR_UNSUPPORTED;
    if (!aligned(z, 16) || !aligned(w, 2) || !aligned(pair_bias, 2)) return EVO_ERR_UNSUPPORTED;
    evo::proj::PbParams p{};
    p.B = (int)B; p.N = (int)N; p.c_z = (int)c_z; p.H = (int)H; p.eps = eps;
    p.z = static_cast<const __nv_bfloat16*>(z); p.ln_w = ln_w; p.ln_b = ln_b;
    p.w = static_cast<const __nv_bfloat16*>(w); p.bias = bias;
    p.out = static_cast<__nv_bfloat16*>(pair_bias);
    const int64_t total = B * N * N;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t chunks = c_z / 8;
    if (c_z <= evo::proj::PBR_MAX_CZ) {
        switch ((H + 3) / 4) {
            case 1: return launch_pair_bias_rows<1>(p, total, s);
            case 2: return launch_pair_bias_rows<2>(p, total, s);
            case 3: return launch_pair_bias_rows<3>(p, total, s);
            default: return launch_pair_bias_rows<4>(p, total, s);
        }
    }
    if (chunks > 64) return launch_pair_bias_h<4, 32>(p, total, s);
    if (chunks > 32) return launch_pair_bias_h<2, 32>(p, total, s);
    if (chunks > 16) return launch_pair_bias_h<1, 32>(p, total, s);
    if (chunks > 8) return launch_pair_bias_h<1, 16>(p, total, s);
    if (chunks > 4) return launch_pair_bias_h<1, 8>(p, total, s);
    if (chunks > 2) return launch_pair_bias_h<1, 4>(p, total, s);
    return launch_pair_bias_h<1, 2>(p, total, s);    // at least 2 lanes per row: 16 rows per warp step
}

evo_status_t evo_tri_mul(int64_t B, int64_t C, int64_t N, const void* a, const void* bb, int incoming,
                         void* z, void* stream) {
    if (B < 0 || C < 0 || N < 0) return EVO_ERR_INVALID_ARG;
    if (B == 0 || C == 0 || N == 0) return EVO_OK;
    if (!a || !bb || !z) return EVO_ERR_INVALID_ARG;
    const int64_t BC = B * C;
    if (N % 8 != 0 || BC > (int64_t)0x7fffffff || N > (int64_t)0x7fffffff / 2) return EVO_ERR_UNSUPPORTED;
    for (const void* q : {a, bb, (const void*)z})
        if (!aligned(q, 16)) return EVO_ERR_UNSUPPORTED;
    const bool in = incoming != 0;
    return launch_contraction(a, bb, z, N, N, N, BC, in, 1.f, EVO_PHASE_TRI_MUL, static_cast<cudaStream_t>(stream));
}

evo_status_t evo_outer_product_mean(int64_t B, int64_t S, int64_t N, int64_t Ca, int64_t Cb, const void* a,
                                    const void* bb, void* out, void* stream) {
    if (B < 0 || S < 0 || N < 0 || Ca <= 0 || Cb <= 0) return EVO_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return EVO_OK;
    if (S == 0 || !a || !bb || !out) return EVO_ERR_INVALID_ARG;
    const int64_t M = N * Ca, Nc = N * Cb;
    if (M % 8 != 0 || Nc % 8 != 0 || M > (int64_t)0x7fffffff / 2 || Nc > (int64_t)0x7fffffff / 2 ||
        S > (int64_t)0x7fffffff || B > (int64_t)0x7fffffff)
        return EVO_ERR_UNSUPPORTED;
    for (const void* q : {a, bb, (const void*)out})
        if (!aligned(q, 16)) return EVO_ERR_UNSUPPORTED;
    // out[b, (i, c1), (j, c2)] = (1/S) sum_s a[b, s, (i, c1)] bb[b, s, (j, c2)]: the MN-major contraction
    return launch_contraction(a, bb, out, M, Nc, S, B, true, (float)(1.0 / (double)S), EVO_PHASE_OPM,
                              static_cast<cudaStream_t>(stream));
}

evo_status_t evo_sum_partials(int64_t count, const float* const* parts, int64_t n, float* out, void* stream) {
    static_assert(EVO_MAX_PARTIALS == evo::partials::MAX_PARTS, "partials limit");
    if (count < 1 || n < 0 || !parts || !out) return EVO_ERR_INVALID_ARG;
    if (count > EVO_MAX_PARTIALS) return EVO_ERR_UNSUPPORTED;
    evo::partials::Params p{};
    bool vec = aligned(out, 16);
    for (int64_t r = 0; r < count; ++r) {
        if (!parts[r]) return EVO_ERR_INVALID_ARG;
        if (!aligned(parts[r], 4)) return EVO_ERR_UNSUPPORTED;
        vec = vec && aligned(parts[r], 16);
        p.part[r] = parts[r];
    }
    if (!aligned(out, 4)) return EVO_ERR_UNSUPPORTED;
    if (n == 0) return EVO_OK;
    p.out = out;
    p.n = n;
    p.count = (int)count;
    p.vec = vec ? 1 : 0;
    const int64_t items = vec ? n / 4 + n % 4 : n;
    const int blocks = (int)std::min<int64_t>((items + 255) / 256, 148 * 8);
    evo::partials::sum_kernel<<<blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

evo_status_t evo_attn_bwd_noalloc(const evo_shape_t* shape, evo_dtype_t dtype, const void* q, const void* k,
                                  const void* v, const void* g, const evo_strides_t* in_str, const void* mask_bias,
                                  const void* pair_bias, const void* out, const void* out_lo, const void* dout,
                                  const evo_strides_t* out_str, const float* lse, void* dq, void* dk, void* dv,
                                  void* dg, const evo_strides_t* grad_str, float* d_pair_bias, void* stream) {
    const evo_status_t st = check_shape(shape);
    if (st != EVO_OK) return st;
    if (dtype != EVO_DTYPE_BF16 && dtype != EVO_DTYPE_F32) return EVO_ERR_INVALID_ARG;
    if (evo_attn_bwd_workspace_bytes(shape, dtype) > EVO_ATTN_NOALLOC_WORKSPACE_BYTES)
        return EVO_ERR_WORKSPACE_TOO_SMALL;
    void* ws = nullptr;
    const evo_status_t wst = noalloc_workspace(&ws);
    if (wst != EVO_OK) return wst;
    return evo_attn_bwd(shape, dtype, q, k, v, g, in_str, mask_bias, pair_bias, out, out_lo, dout, out_str, lse,
                        dq, dk, dv, dg, grad_str, d_pair_bias, ws, EVO_ATTN_NOALLOC_WORKSPACE_BYTES, stream);
}

evo_status_t evo_add_rms_norm_fp8(int64_t rows, int64_t cols, evo_dtype_t dtype, const void* x, int64_t ldx,
                                  const void* residual, int64_t ldr, const void* weight, evo_dtype_t w_dtype,
                                  float eps, void* q, int64_t ldq, float* scale, int64_t scale_row,
                                  int64_t scale_group, void* h, int64_t ldh, void* n, int64_t ldn, float* rstd,
                                  void* stream) {
    if (rows < 0 || cols < 1 || !dtype_ok(dtype) || !dtype_ok(w_dtype) || !(eps >= 0.f)) return EVO_ERR_INVALID_ARG;
    if (rows == 0) return EVO_OK;
    if (!x || !q || !scale || scale_row < 1 || scale_group < 1) return EVO_ERR_INVALID_ARG;
    if (ldx < 0 || (residual && ldr < 0) || (rows > 1 && (ldq < cols || (h && ldh < cols) || (n && ldn < cols))))
        return EVO_ERR_INVALID_ARG;
    if (cols > kMaxRowCols || !aligned(q, 16) || (rows > 1 && ldq % 16 != 0)) return EVO_ERR_UNSUPPORTED;
    const int64_t e = elem_bytes(dtype);
    for (const void* t : {x, residual, (const void*)h, (const void*)n})
        if (!aligned(t, e)) return EVO_ERR_INVALID_ARG;
    if (!aligned(weight, elem_bytes(w_dtype)) || !aligned(scale, 4) || !aligned(rstd, 4)) return EVO_ERR_INVALID_ARG;
    evo::fp8::NormParams p{};
    p.rows = rows; p.cols = cols; p.x = x; p.res = residual; p.ldx = ldx; p.ldres = ldr;
    p.w = weight; p.w_bf16 = w_dtype == EVO_DTYPE_BF16; p.eps = eps; p.inv_cols = 1.0f / (float)cols;
    p.q = static_cast<uint8_t*>(q); p.ldq = ldq;
    p.scale = scale; p.s_row = scale_row; p.s_grp = scale_group;
    p.h = h; p.n = n; p.ldh = ldh; p.ldn = ldn; p.rstd = rstd;
    const RowSplit split = row_split(cols);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = rows_vec(x, rows, cols, ldx, e) && rows_vec(residual, rows, cols, ldr, e) &&
                     rows_vec(h, rows, cols, ldh, e) && rows_vec(n, rows, cols, ldn, e);
    by_type(dtype, vec, [&](auto t, auto v) { launch_norm<decltype(t), decltype(v)::value>(p, split, s); });
    g_launches += 1;
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

size_t evo_add_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1 || cols > kMaxRowCols) return 0;
    return (size_t)(norm_bwd_blocks(rows, cols) * cols) * sizeof(float);
}

evo_status_t evo_add_rms_norm_bwd(int64_t rows, int64_t cols, evo_dtype_t dtype, const void* dy, int64_t lddy,
                                  const void* dh, int64_t lddh, const void* h, int64_t ldh, const float* rstd,
                                  const void* weight, evo_dtype_t w_dtype, void* dx, int64_t lddx, void* dweight,
                                  evo_dtype_t dw_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (rows < 0 || cols < 1 || !dtype_ok(dtype) || !dtype_ok(w_dtype) || !dtype_ok(dw_dtype)) return EVO_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!aligned(dweight, elem_bytes(dw_dtype))) return EVO_ERR_INVALID_ARG;
    if (cols > kMaxRowCols) return EVO_ERR_UNSUPPORTED;
    if (rows == 0) {
        if (dweight && cudaMemsetAsync(dweight, 0, (size_t)(cols * elem_bytes(dw_dtype)), s) != cudaSuccess) return EVO_ERR_CUDA;
        return EVO_OK;
    }
    if (!dy || !h || !rstd || !dx || lddy < 0 || ldh < 0 || (dh && lddh < 0) || (rows > 1 && lddx < cols))
        return EVO_ERR_INVALID_ARG;
    const int64_t e = elem_bytes(dtype);
    for (const void* t : {dy, dh, h, (const void*)dx})
        if (!aligned(t, e)) return EVO_ERR_INVALID_ARG;
    if (!aligned(weight, elem_bytes(w_dtype)) || !aligned(rstd, 4)) return EVO_ERR_INVALID_ARG;
    if (dweight) {
        if (!workspace || workspace_bytes < evo_add_rms_norm_bwd_workspace_bytes(rows, cols))
            return EVO_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 16)) return EVO_ERR_INVALID_ARG;
    }
    evo::fp8::NormBwdParams p{};
    p.rows = rows; p.cols = cols; p.dy = dy; p.dh = dh; p.h = h;
    p.lddy = lddy; p.lddh = lddh; p.ldh = ldh; p.rstd = rstd;
    p.w = weight; p.w_bf16 = w_dtype == EVO_DTYPE_BF16; p.inv_cols = 1.0f / (float)cols; p.dx = dx; p.lddx = lddx;
    p.part = dweight ? static_cast<float*>(workspace) : nullptr;
    const RowSplit split = row_split_bwd(cols);
    const int blocks = (int)norm_bwd_blocks(rows, cols);
    const bool vec = rows_vec(dy, rows, cols, lddy, e) && rows_vec(dh, rows, cols, lddh, e) &&
                     rows_vec(h, rows, cols, ldh, e) && rows_vec(dx, rows, cols, lddx, e);
    by_type(dtype, vec, [&](auto t, auto v) { launch_norm_bwd<decltype(t), decltype(v)::value>(p, split, blocks, s); });
    g_launches += 1;
    if (dweight) {
        const unsigned grid = (unsigned)((cols + 31) / 32);
        if (dw_dtype == EVO_DTYPE_BF16)
            evo::fp8::sum_columns_kernel<<<grid, 1024, 0, s>>>(p.part, blocks, cols, static_cast<__nv_bfloat16*>(dweight));
        else
            evo::fp8::sum_columns_kernel<<<grid, 1024, 0, s>>>(p.part, blocks, cols, static_cast<float*>(dweight));
        g_launches += 1;
    }
    return cudaGetLastError() == cudaSuccess ? EVO_OK : EVO_ERR_CUDA;
}

evo_status_t evo_quantize_fp8(int64_t rows, int64_t cols, evo_dtype_t dtype, const void* x, int64_t ldx, int square,
                              int transpose, void* q, int64_t ldq, float* scale, int64_t scale_row,
                              int64_t scale_group, void* stream) {
    if (rows < 0 || cols < 0 || !dtype_ok(dtype)) return EVO_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return EVO_OK;
    if (!q) return EVO_ERR_INVALID_ARG;
    evo::fp8::QuantParams p{};
    p.rows = rows; p.cols = cols; p.x = x; p.ldx = ldx;
    if (transpose) {
        p.qt = static_cast<uint8_t*>(q); p.ldqt = ldq; p.scale_t = scale; p.st_row = scale_row; p.st_grp = scale_group;
    } else {
        p.q = static_cast<uint8_t*>(q); p.ldq = ldq; p.scale = scale; p.s_row = scale_row; p.s_grp = scale_group;
    }
    return quantize(p, dtype, square != 0, static_cast<cudaStream_t>(stream));
}

evo_status_t evo_quantize_fp8_both(int64_t rows, int64_t cols, evo_dtype_t dtype, const void* x, int64_t ldx,
                                   int square, void* q, int64_t ldq, float* scale, int64_t scale_row,
                                   int64_t scale_group, void* q_t, int64_t ldq_t, float* scale_t,
                                   int64_t scale_t_row, int64_t scale_t_group, void* stream) {
    if (rows < 0 || cols < 0 || !dtype_ok(dtype)) return EVO_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return EVO_OK;
    if (!q || !q_t) return EVO_ERR_INVALID_ARG;
    evo::fp8::QuantParams p{};
    p.rows = rows; p.cols = cols; p.x = x; p.ldx = ldx;
    p.q = static_cast<uint8_t*>(q); p.ldq = ldq; p.scale = scale; p.s_row = scale_row; p.s_grp = scale_group;
    p.qt = static_cast<uint8_t*>(q_t); p.ldqt = ldq_t; p.scale_t = scale_t;
    p.st_row = scale_t_row; p.st_grp = scale_t_group;
    return quantize(p, dtype, square != 0, static_cast<cudaStream_t>(stream));
}

// Zeros in rows x cols elements of e bytes at a pitch of ld elements.
static bool zero_matrix(void* p, int64_t rows, int64_t cols, int64_t ld, int64_t e, void* stream) {
    return cudaMemset2DAsync(p, (size_t)((rows > 1 ? ld : cols) * e), 0, (size_t)(cols * e), (size_t)rows,
                             static_cast<cudaStream_t>(stream)) == cudaSuccess;
}

// Where evo_fp8_linear_bwd keeps its operands in the workspace.
struct BwdOperands {
    int64_t ld_n, ld_m;          // pitches of dy's codes, and of both transposes
    size_t dy, dys, dyt, dyts, xt, xts, work, total;
    BwdOperands(int64_t M, int64_t N, int64_t K, bool dx, bool dw) {
        const int64_t gn = (N + 127) / 128, gm = (M + 127) / 128;
        ld_n = (N + 15) / 16 * 16;
        ld_m = (M + 15) / 16 * 16;
        size_t at = 0;
        auto take = [&](bool want, int64_t bytes) {
            const size_t here = at;
            if (want) at += align256((size_t)bytes);
            return here;
        };
        dy = take(dx, M * ld_n);
        dys = take(dx, M * gn * 4);
        dyt = take(dw, N * ld_m);
        dyts = take(dw, N * gm * 4);
        xt = take(dw, K * ld_m);
        xts = take(dw, K * gm * 4);
        work = at;
        total = at + std::max(dx ? plan_linear(M, K, N).workspace : 0, dw ? plan_linear(N, K, M).workspace : 0);
    }
};

size_t evo_fp8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    return M < 1 || N < 1 || K < 1 || M > kMaxProduct || N > kMaxProduct || K > kMaxProduct ? 0 : plan_linear(M, N, K).workspace;
}

evo_status_t evo_fp8_linear(int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const float* x_scale,
                            int64_t x_scale_row, int64_t x_scale_group, const void* w, int64_t ldw,
                            const float* w_scale, int64_t w_scale_row, int64_t w_scale_group, int w_scale_rows,
                            const float* bias, evo_dtype_t y_dtype, void* y, int64_t ldy, void* workspace,
                            size_t workspace_bytes, void* stream) {
    if (M < 0 || N < 0 || K < 1 || !dtype_ok(y_dtype)) return EVO_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return EVO_OK;
    if (!x || !x_scale || !w || !w_scale || !y) return EVO_ERR_INVALID_ARG;
    if ((M > 1 && (ldx < K || ldy < N)) || (N > 1 && ldw < K)) return EVO_ERR_INVALID_ARG;
    if (x_scale_row < 0 || x_scale_group < 0 || w_scale_row < 0 || w_scale_group < 0) return EVO_ERR_INVALID_ARG;
    if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) || !aligned(y, elem_bytes(y_dtype)))
        return EVO_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || (M > 1 && ldx % 16 != 0) || (N > 1 && ldw % 16 != 0))
        return EVO_ERR_UNSUPPORTED;
    if (M > kMaxProduct || N > kMaxProduct || K > kMaxProduct) return EVO_ERR_UNSUPPORTED;
    const LinPlan plan = plan_linear(M, N, K);
    if (plan.workspace > 0 && (!workspace || workspace_bytes < plan.workspace)) return EVO_ERR_WORKSPACE_TOO_SMALL;
    if (plan.workspace > 0 && !aligned(workspace, 256)) return EVO_ERR_INVALID_ARG;
    evo::fp8::LinParams p{};
    p.M = (int)M; p.N = (int)N; p.K = (int)K;
    p.x = x; p.ldx = ldx; p.w = w; p.ldw = ldw;
    p.sx = x_scale; p.sx_row = x_scale_row; p.sx_grp = x_scale_group;
    p.sw = w_scale; p.sw_row = w_scale_row; p.sw_grp = w_scale_group;
    p.bias = bias; p.y = y; p.ldy = ldy;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (y_dtype == EVO_DTYPE_BF16)
        return w_scale_rows ? launch_linear<__nv_bfloat16, true>(p, plan, workspace, s) : launch_linear<__nv_bfloat16, false>(p, plan, workspace, s);
    return w_scale_rows ? launch_linear<float, true>(p, plan, workspace, s) : launch_linear<float, false>(p, plan, workspace, s);
}

size_t evo_fp8_linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int want_dx, int want_dw) {
    if (M < 1 || N < 1 || K < 1 || M > kMaxProduct || N > kMaxProduct || K > kMaxProduct) return 0;
    return BwdOperands(M, N, K, want_dx != 0, want_dw != 0).total;
}

evo_status_t evo_fp8_linear_bwd(int64_t M, int64_t N, int64_t K, evo_dtype_t dtype, const void* dy, int64_t lddy,
                                const void* x, int64_t ldx, const void* w_t, int64_t ldw_t, const float* w_t_scale,
                                int64_t w_t_scale_row, int64_t w_t_scale_group, void* dx, int64_t lddx, void* dw,
                                evo_dtype_t dw_dtype, int64_t lddw, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (M < 0 || N < 0 || K < 1 || !dtype_ok(dtype) || !dtype_ok(dw_dtype)) return EVO_ERR_INVALID_ARG;
    if (!dx && !dw) return EVO_OK;
    if (dw && N > 1 && lddw < K) return EVO_ERR_INVALID_ARG;
    if (M == 0 || N == 0) {                                 // the empty sums: dw without rows, dx without outputs
        if (dw && N > 0 && !zero_matrix(dw, N, K, lddw, elem_bytes(dw_dtype), stream)) return EVO_ERR_CUDA;
        if (!dx || M == 0) return EVO_OK;
        if ((M > 1 && lddx < K) || !aligned(dx, elem_bytes(dtype))) return EVO_ERR_INVALID_ARG;
        // a dx that the runtime does not know (where there is no device, none is known) is not written
        cudaPointerAttributes at{};
        if (cudaPointerGetAttributes(&at, dx) != cudaSuccess || at.type == cudaMemoryTypeUnregistered) {
            cudaGetLastError();
            return EVO_OK;
        }
        return zero_matrix(dx, M, K, lddx, elem_bytes(dtype), stream) ? EVO_OK : EVO_ERR_CUDA;
    }
    if (M > kMaxProduct || N > kMaxProduct || K > kMaxProduct) return EVO_ERR_UNSUPPORTED;
    if (!dy || (dw && !x) || (dx && (!w_t || !w_t_scale)) || (dx && M > 1 && lddx < K)) return EVO_ERR_INVALID_ARG;
    if ((dx && !aligned(dx, elem_bytes(dtype))) || (dw && !aligned(dw, elem_bytes(dw_dtype)))) return EVO_ERR_INVALID_ARG;
    // everything the calls below would refuse, before the first of them enqueues anything
    if (lddy < 0 || !aligned(dy, elem_bytes(dtype)) || (dw && (ldx < 0 || !aligned(x, elem_bytes(dtype)))))
        return EVO_ERR_INVALID_ARG;
    if (dx && ((K > 1 && ldw_t < N) || w_t_scale_row < 0 || w_t_scale_group < 0 || !aligned(w_t_scale, 4)))
        return EVO_ERR_INVALID_ARG;
    if (dx && (!aligned(w_t, 16) || (K > 1 && ldw_t % 16 != 0))) return EVO_ERR_UNSUPPORTED;
    const BwdOperands o(M, N, K, dx != nullptr, dw != nullptr);
    if (!workspace || workspace_bytes < o.total) return EVO_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 256)) return EVO_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    auto f = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    const size_t work = workspace_bytes - o.work;
    evo_status_t st;
    if (dx && dw)
        st = evo_quantize_fp8_both(M, N, dtype, dy, lddy, 0, ws + o.dy, o.ld_n, f(o.dys), 1, M, ws + o.dyt, o.ld_m,
                                   f(o.dyts), 1, N, stream);
    else if (dx)
        st = evo_quantize_fp8(M, N, dtype, dy, lddy, 0, 0, ws + o.dy, o.ld_n, f(o.dys), 1, M, stream);
    else
        st = evo_quantize_fp8(M, N, dtype, dy, lddy, 0, 1, ws + o.dyt, o.ld_m, f(o.dyts), 1, N, stream);
    if (st == EVO_OK && dx)
        st = evo_fp8_linear(M, K, N, ws + o.dy, o.ld_n, f(o.dys), 1, M, w_t, ldw_t, w_t_scale, w_t_scale_row,
                            w_t_scale_group, 0, nullptr, dtype, dx, lddx, ws + o.work, work, stream);
    if (st == EVO_OK && dw)
        st = evo_quantize_fp8(M, K, dtype, x, ldx, 0, 1, ws + o.xt, o.ld_m, f(o.xts), 1, K, stream);
    if (st == EVO_OK && dw)
        st = evo_fp8_linear(N, K, M, ws + o.dyt, o.ld_m, f(o.dyts), 1, N, ws + o.xt, o.ld_m, f(o.xts), 1, K, 1, nullptr,
                            dw_dtype, dw, lddw, ws + o.work, work, stream);
    return st;
}

}  // extern "C"
