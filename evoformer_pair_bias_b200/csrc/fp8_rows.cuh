// fp8_rows.cuh -- the memory-bound operators around the 8-bit projection:
//   add_rms_norm_kernel   h = x + residual, n = h / rms(h) * weight, n in e4m3
//                         with one scale per row and 128 channels
//   rms_bwd_kernel        its gradients (and sum_columns_kernel for d_weight)
//   quantize_*_kernel     a matrix in e4m3 with 1 x 128 or 128 x 128 scales, as
//                         it lies or transposed
//
// A group whose largest magnitude is m (held at LEAST or above) keeps
//   q = e4m3(448 * v / m),   scale = m / 448.
// The quotient is correctly rounded before the one rounding to e4m3: with
// inv = 1/m rounded, q0 = t * inv and the remainder t - q0 * m taken by a fused
// multiply-add, q0 + remainder * inv is the rounded quotient (Markstein's
// correction step).  bf16 values make ties in e4m3 often enough to matter (448 =
// 7 * 64, so v = 3m/2^k is one); a plain product with 1/m would break them
// either way.  t = 0.875 v cannot overflow and is exact for bf16 v; the factor
// 512 that is left is exact.  In the norm the row's 1 / rms cancels out of
// v / m, so the quotient is that of u = h * weight, exact in fp32 for bf16.
//
// All of these move each byte once and are bound by HBM.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "sm100.cuh"

namespace evo {
namespace fp8 {

constexpr int GROUP = 128;
constexpr float LEAST = 7.888609052210118e-31f;   // 2^-100: the smallest maximum a group is given
constexpr float TOP = 448.0f;                     // largest e4m3 value

// Two values as e4m3, `lo` in the low byte; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// 448 * v / m, correctly rounded; inv = 1 / m.
__device__ __forceinline__ float quotient(float v, float m, float inv) {
    const float t = 0.875f * v;
    const float q = t * inv;
    return fmaf(fmaf(-q, m, t), inv, q) * 512.0f;
}
// Four quotients as e4m3 bytes.
__device__ __forceinline__ uint32_t e4m3x4(const float* v, float m, float inv) {
    return e4m3x2(quotient(v[0], m, inv), quotient(v[1], m, inv)) |
           (e4m3x2(quotient(v[2], m, inv), quotient(v[3], m, inv)) << 16);
}
// |v| as an integer that orders like it, with NaN above infinity above the rest:
// the largest of a group is NaN as soon as one value is.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// A group's maximum as a divisor: at least LEAST, NaN where it is not finite.
__device__ __forceinline__ float divisor(uint32_t mag) {
    return mag >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : fmaxf(__uint_as_float(mag), LEAST);
}

// ------------------------------------------------------------- row fragments
// A warp holds 256 columns of a row, 8 values a lane.
//   VEC   lane l holds columns 8l .. 8l + 7 (16-byte loads): a 128-group is a half warp
//   else  lane l holds columns l + 32e (single loads, coalesced): values 0..3 lie in
//         the first group, 4..7 in the second
// VEC wants every row 16-byte aligned and the row's bytes a multiple of 16.
template <bool VEC>
__device__ __forceinline__ int frag_col(int lane, int e) {
    return VEC ? 8 * lane + e : lane + 32 * e;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load_frag(const T* row, int64_t c0, int64_t cols, int lane, float* v) {
    if constexpr (VEC && sizeof(T) == 2) {
        const int64_t c = c0 + 8 * lane;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (c < cols) w = *reinterpret_cast<const uint4*>(row + c);
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = sm100::bf16lo(a[e]);
            v[2 * e + 1] = sm100::bf16hi(a[e]);
        }
    } else if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t c = c0 + 8 * lane + 4 * h;
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < cols) w = *reinterpret_cast<const float4*>(row + c);
            v[4 * h] = w.x;
            v[4 * h + 1] = w.y;
            v[4 * h + 2] = w.z;
            v[4 * h + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = c0 + lane + 32 * e;
            v[e] = c < cols ? Elem<T>::load(row + c) : 0.f;
        }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_frag(T* row, int64_t c0, int64_t cols, int lane, const float* v) {
    if constexpr (VEC && sizeof(T) == 2) {
        const int64_t c = c0 + 8 * lane;
        if (c < cols)
            *reinterpret_cast<uint4*>(row + c) =
                make_uint4(sm100::pack_bf16(v[0], v[1]), sm100::pack_bf16(v[2], v[3]), sm100::pack_bf16(v[4], v[5]),
                           sm100::pack_bf16(v[6], v[7]));
    } else if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t c = c0 + 8 * lane + 4 * h;
            if (c < cols)
                *reinterpret_cast<float4*>(row + c) = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = c0 + lane + 32 * e;
            if (c < cols) Elem<T>::store(row + c, v[e]);
        }
    }
}

// v rounded to T and back.
template <typename T>
__device__ __forceinline__ float rounded(float v) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(__float2bfloat16_rn(v));
    return v;
}

// Largest magnitude of each value's group: mag[0] for values 0..3, mag[1] for 4..7.
template <bool VEC>
__device__ __forceinline__ void group_max(const float* v, uint32_t* mag) {
    uint32_t a = 0, b = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        a = max(a, magnitude(v[e]));
        b = max(b, magnitude(v[4 + e]));
    }
    if (VEC) {                                   // one group in this half warp
        a = max(a, b);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        b = a;
    } else {
        a = __reduce_max_sync(0xffffffffu, a);
        b = __reduce_max_sync(0xffffffffu, b);
    }
    mag[0] = a;
    mag[1] = b;
}

// The fragment's quotients, d[0] / d[1] the divisors of its two halves, as bytes of q's row.
// q rows are 16-byte aligned; only columns below `cols` are written.
template <bool VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int64_t c0, int64_t cols, int lane, const float* v,
                                           const float* d) {
    const float i0 = __frcp_rn(d[0]), i1 = VEC ? i0 : __frcp_rn(d[1]);
    const uint32_t lo = e4m3x4(v, d[0], i0), hi = e4m3x4(v + 4, d[1], i1);
    if (VEC) {
        const int64_t c = c0 + 8 * lane;
        if (c + 8 <= cols)
            *reinterpret_cast<uint2*>(row + c) = make_uint2(lo, hi);
        else if (c < cols)                       // fp32 rows end on multiples of 4
            *reinterpret_cast<uint32_t*>(row + c) = lo;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = c0 + lane + 32 * e;
            if (c < cols) row[c] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
        }
    }
}

// The scales of the fragment's two groups, from the lanes that own them.
template <bool VEC>
__device__ __forceinline__ void store_scales(float* s, int64_t stride, int64_t c0, int64_t cols, int lane,
                                             const float* sc) {
    const int64_t g = c0 / GROUP;
    if ((lane & 15) == 0) {
        const int h = lane >> 4;
        if (c0 + GROUP * h < cols) s[(g + h) * stride] = VEC ? sc[0] : sc[h];
    }
}

// ------------------------------------------------------------- add, norm, quantise
struct NormParams {
    int64_t rows, cols;
    const void *x, *res;         // T [rows, cols], res may be null
    int64_t ldx, ldres;
    const void* w;               // [cols], bf16 or fp32, or null (ones)
    int w_bf16;
    float eps;
    uint8_t* q;                  // e4m3 [rows, cols]
    int64_t ldq;
    float* scale;                // [rows, groups] with strides
    int64_t s_row, s_grp;
    void *h, *n;                 // T [rows, cols] or null
    int64_t ldh, ldn;
    float* rstd;                 // [rows] or null
};

__device__ __forceinline__ float load_w(const void* w, int bf16, int64_t c) {
    if (!w) return 1.f;
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]) : static_cast<const float*>(w)[c];
}

// Sum of one value per lane over the `wpr` warps of a row (a power of two).  Every warp of
// the block calls it; `slot` alternates so that one barrier per call is enough.
__device__ __forceinline__ float row_sum(float v, int wpr, int warp, float* buf) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (wpr == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    const int w0 = warp & ~(wpr - 1);
    float s = 0.f;
    for (int i = 0; i < wpr; ++i) s += buf[w0 + i];
    return s;
}

// wpr warps (a power of two) hold a row, NV fragments of 256 columns each; a block holds
// (blockDim / 32) / wpr rows at a time and walks the rows with the grid.  The weight stays
// in registers.
template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const NormParams p, const int wpr) {
    __shared__ float buf[2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (blockDim.x >> 5) / wpr, sub = warp / wpr, part = warp & (wpr - 1);
    float w[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = (int64_t)(i * wpr + part) * 256 + frag_col<VEC>(lane, e);
            w[i][e] = c < p.cols ? load_w(p.w, p.w_bf16, c) : 0.f;
        }
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < p.rows; r0 += (int64_t)gridDim.x * per, turn ^= 1) {
        const int64_t r = r0 + sub;
        const bool live = r < p.rows;
        float h[NV][8];
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c0 = (int64_t)(i * wpr + part) * 256;
            const int64_t lim = live ? p.cols : 0;
            load_frag<T, VEC>(static_cast<const T*>(p.x) + r * p.ldx, c0, lim, lane, h[i]);
            if (p.res) {
                float a[8];
                load_frag<T, VEC>(static_cast<const T*>(p.res) + r * p.ldres, c0, lim, lane, a);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] = rounded<T>(h[i][e] + a[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sq = fmaf(h[i][e], h[i][e], sq);
        }
        sq = row_sum(sq, wpr, warp, buf[turn]);
        const float rstd = __frsqrt_rn(__fdiv_rn(sq, (float)p.cols) + p.eps);
        if (!live) continue;                     // no barrier below
        const float floor_u = __fdiv_rn(LEAST, rstd);
        if (p.rstd && part == 0 && lane == 0) p.rstd[r] = rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c0 = (int64_t)(i * wpr + part) * 256;
            if (c0 >= p.cols) break;
            if (p.h) store_frag<T, VEC>(static_cast<T*>(p.h) + r * p.ldh, c0, p.cols, lane, h[i]);
            if (p.n) {
                float n[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) n[e] = h[i][e] * rstd * w[i][e];
                store_frag<T, VEC>(static_cast<T*>(p.n) + r * p.ldn, c0, p.cols, lane, n);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] *= w[i][e];
            uint32_t mag[2];
            group_max<VEC>(h[i], mag);
            float d[2], sc[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                d[g] = mag[g] >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : fmaxf(__uint_as_float(mag[g]), floor_u);
                sc[g] = __fdiv_rn(d[g] * rstd, TOP);
            }
            store_e4m3<VEC>(p.q + r * p.ldq, c0, p.cols, lane, h[i], d);
            store_scales<VEC>(p.scale + r * p.s_row, p.s_grp, c0, p.cols, lane, sc);
        }
    }
}

// ------------------------------------------------------------- gradients of the norm
struct NormBwdParams {
    int64_t rows, cols;
    const void *dy, *dh, *h;     // T [rows, cols]; dh may be null
    int64_t lddy, lddh, ldh;
    const float* rstd;           // [rows]
    const void* w;
    int w_bf16;
    void* dx;                    // T [rows, cols]
    int64_t lddx;
    float* part;                 // fp32 [gridDim.x, cols] partial sums of d_weight, or null
};

// dx = dh + rstd * (g - n * mean(g n)), g = dy * w, n = h * rstd.  Each warp adds up dy * n of
// the rows it meets in registers; a block's rows are joined in shared memory and leave one
// partial row, and sum_columns_kernel adds the partial rows in order: no atomics, the same
// bits on every run.
template <typename T, bool VEC, int NV>
__global__ void __launch_bounds__(1024) rms_bwd_kernel(const NormBwdParams p, const int wpr) {
    __shared__ float buf[2][32];
    extern __shared__ float join[];              // [warps][NV][256] when a block holds several rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (blockDim.x >> 5) / wpr, sub = warp / wpr, part = warp & (wpr - 1);
    float w[NV][8], dw[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = (int64_t)(i * wpr + part) * 256 + frag_col<VEC>(lane, e);
            w[i][e] = c < p.cols ? load_w(p.w, p.w_bf16, c) : 0.f;
            dw[i][e] = 0.f;
        }
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < p.rows; r0 += (int64_t)gridDim.x * per, turn ^= 1) {
        const int64_t r = r0 + sub;
        const bool live = r < p.rows;
        const float rstd = live ? p.rstd[r] : 0.f;
        float dy[NV][8], n[NV][8];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c0 = (int64_t)(i * wpr + part) * 256;
            const int64_t lim = live ? p.cols : 0;
            load_frag<T, VEC>(static_cast<const T*>(p.dy) + r * p.lddy, c0, lim, lane, dy[i]);
            load_frag<T, VEC>(static_cast<const T*>(p.h) + r * p.ldh, c0, lim, lane, n[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[i][e] *= rstd;
                if (live) dw[i][e] = fmaf(dy[i][e], n[i][e], dw[i][e]);
                dy[i][e] *= w[i][e];
                dot = fmaf(dy[i][e], n[i][e], dot);
            }
        }
        dot = row_sum(dot, wpr, warp, buf[turn]);
        if (!live) continue;
        const float mean = __fdiv_rn(dot, (float)p.cols);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c0 = (int64_t)(i * wpr + part) * 256;
            if (c0 >= p.cols) break;
            float a[8];
            if (p.dh) {
                load_frag<T, VEC>(static_cast<const T*>(p.dh) + r * p.lddh, c0, p.cols, lane, a);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = fmaf(rstd, fmaf(-n[i][e], mean, dy[i][e]), a[e]);
            store_frag<T, VEC>(static_cast<T*>(p.dx) + r * p.lddx, c0, p.cols, lane, a);
        }
    }
    if (!p.part) return;
    float* out = p.part + (int64_t)blockIdx.x * p.cols;
    if (per > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) join[(warp * NV + i) * 256 + frag_col<VEC>(lane, e)] = dw[i][e];
        __syncthreads();
        // column c of the row lies with warp (c / 256) % wpr of each row, fragment (c / 256) / wpr
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            const int f = (int)(c >> 8), o = ((f & (wpr - 1)) * NV + f / wpr) * 256 + (int)(c & 255);
            float s = 0.f;
            for (int k = 0; k < per; ++k) s += join[k * wpr * NV * 256 + o];
            out[c] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t c = (int64_t)(i * wpr + part) * 256 + frag_col<VEC>(lane, e);
                if (c < p.cols) out[c] = dw[i][e];
            }
    }
}

// out[c] = sum over the n partial rows, in a fixed order: 32 threads a column, each every 32nd row.
template <typename T>
__global__ void __launch_bounds__(1024) sum_columns_kernel(const float* part, int64_t n, int64_t cols, T* out) {
    __shared__ float s[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    float a = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int64_t r = ty; r < n; r += 32) a += part[r * cols + c];
    }
    s[ty][tx] = a;
    __syncthreads();
    a = s[tx][ty];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    const int64_t cc = (int64_t)blockIdx.x * 32 + ty;
    if (tx == 0 && cc < cols) Elem<T>::store(out + cc, a);
}

// ------------------------------------------------------------- quantise
struct QuantParams {
    int64_t rows, cols;          // of x
    const void* x;               // T [rows, cols]
    int64_t ldx;
    uint8_t* q;                  // e4m3 [rows, cols]
    int64_t ldq;
    float* scale;                // [rows or blocks, groups] with strides
    int64_t s_row, s_grp;
    uint8_t* qt;                 // e4m3 [cols, rows], the transpose
    int64_t ldqt;
    float* scale_t;              // [cols or blocks, groups] with strides
    int64_t st_row, st_grp;
};

// 1 x 128 groups along the rows: a warp takes 256 columns of a row at a time.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t chunks = (p.cols + 255) / 256, items = p.rows * chunks;
    for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < items; t += (int64_t)gridDim.x * 8) {
        const int64_t r = t / chunks, c0 = (t - r * chunks) * 256;
        float v[8], d[2], sc[2];
        load_frag<T, VEC>(static_cast<const T*>(p.x) + r * p.ldx, c0, p.cols, lane, v);
        uint32_t mag[2];
        group_max<VEC>(v, mag);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            d[g] = divisor(mag[g]);
            sc[g] = __fdiv_rn(d[g], TOP);
        }
        store_e4m3<VEC>(p.q + r * p.ldq, c0, p.cols, lane, v, d);
        store_scales<VEC>(p.scale + r * p.s_row, p.s_grp, c0, p.cols, lane, sc);
    }
}

// A 128 x 128 tile of x in one block of 512 threads, TC columns x TR rows a thread:
//   bf16 VEC  8 columns x 4 rows (16-byte loads, 16 lanes a row), kept as loaded
//   fp32 VEC  4 columns x 8 rows (16-byte loads, a warp a row)
//   else      columns l + 32j, 8 rows (single loads, a warp a row)
template <typename T, bool VEC>
struct Tile {
    static constexpr bool PACKED = VEC && sizeof(T) == 2;
    static constexpr int TC = PACKED ? 8 : 4;
    static constexpr int TR = 32 / TC;
    static constexpr int LPR = 128 / TC;         // lanes a row
    uint32_t v[TR][4];                           // four bf16 pairs or four floats

    static __device__ __forceinline__ int col(int lane, int j) { return VEC ? (lane % LPR) * TC + j : lane + 32 * j; }
    static __device__ __forceinline__ int row(int warp, int lane) { return warp * 8 + (lane / LPR) * TR; }

    __device__ __forceinline__ void load(const QuantParams& p, int64_t r0, int64_t c0, int warp, int lane) {
        const int64_t r = r0 + row(warp, lane);
#pragma unroll
        for (int i = 0; i < TR; ++i) {
            const T* x = static_cast<const T*>(p.x) + (r + i) * p.ldx;
            const bool live = r + i < p.rows;
            if constexpr (VEC) {
                const int64_t c = c0 + col(lane, 0);
                uint4 w = make_uint4(0, 0, 0, 0);
                if (live && c < p.cols) w = *reinterpret_cast<const uint4*>(x + c);
                v[i][0] = w.x;
                v[i][1] = w.y;
                v[i][2] = w.z;
                v[i][3] = w.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t c = c0 + col(lane, j);
                    v[i][j] = live && c < p.cols ? __float_as_uint(Elem<T>::load(x + c)) : 0u;
                }
            }
        }
    }
    __device__ __forceinline__ float at(int i, int j) const {
        if constexpr (PACKED) return j & 1 ? sm100::bf16hi(v[i][j / 2]) : sm100::bf16lo(v[i][j / 2]);
        return __uint_as_float(v[i][j]);
    }
    // Magnitudes as integers that order like them: pairs of 16 bits (PACKED) or one of 32.
    static __device__ __forceinline__ uint32_t mag(uint32_t w) { return w & (PACKED ? 0x7fff7fffu : 0x7fffffffu); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return PACKED ? __vmaxu2(a, b) : max(a, b); }
    // The larger of a pair (PACKED), as the bits of a float.
    static __device__ __forceinline__ uint32_t widest(uint32_t m) {
        return PACKED ? max(m << 16, m & 0xffff0000u) : m;
    }
};

// 128 x 128 blocks (SQUARE), or 1 x 128 groups along the columns for q and along the rows for the
// transpose.  ROWS writes q, TRANSPOSE the transpose, through shared memory.
template <typename T, bool VEC, bool SQUARE, bool ROWS, bool TRANSPOSE>
__global__ void __launch_bounds__(512, 2) quantize_tile_kernel(const QuantParams p) {
    using L = Tile<T, VEC>;
    constexpr int PITCH = 132;                   // bytes of a transposed column: 33 words, so columns meet other banks
    constexpr int W = L::PACKED ? 64 : 128;      // words of a warp's column maxima
    constexpr bool BY_COL = TRANSPOSE && !SQUARE;
    __shared__ uint32_t cmax[BY_COL ? 16 : 1][BY_COL ? W + 2 : 16];
    __shared__ float dv[BY_COL ? 128 : 1], iv[BY_COL ? 128 : 1];
    __shared__ uint32_t tq[TRANSPOSE ? 128 * PITCH / 4 : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tc = (p.cols + 127) / 128;
    const int64_t br = blockIdx.x / tc, bc = blockIdx.x - br * tc;
    const int64_t r0 = br * 128, c0 = bc * 128;
    L t;
    t.load(p, r0, c0, warp, lane);
    if constexpr (SQUARE) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < L::TR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) m = L::larger(m, L::mag(t.v[i][j]));
        m = __reduce_max_sync(0xffffffffu, L::widest(m));
        if (lane == 0) cmax[0][warp] = m;
        __syncthreads();
        if (warp == 0) {
            m = __reduce_max_sync(0xffffffffu, lane < 16 ? cmax[0][lane] : 0u);
            if (lane == 0) {
                const float d = divisor(m);
                dv[0] = d;
                iv[0] = __frcp_rn(d);
                if (ROWS) p.scale[br * p.s_row + bc * p.s_grp] = __fdiv_rn(d, TOP);
                if (TRANSPOSE) p.scale_t[bc * p.st_row + br * p.st_grp] = __fdiv_rn(d, TOP);
            }
        }
        __syncthreads();
    } else if constexpr (TRANSPOSE) {
        uint32_t m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[j] = L::mag(t.v[0][j]);
#pragma unroll
            for (int i = 1; i < L::TR; ++i) m[j] = L::larger(m[j], L::mag(t.v[i][j]));
            if (L::LPR == 16) m[j] = L::larger(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        }
        if (L::LPR == 32 || lane < 16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) cmax[warp][L::PACKED ? 4 * lane + j : L::col(lane, j)] = m[j];
        }
        __syncthreads();
        // four threads a column, four warps' maxima each
        const int c = threadIdx.x >> 2, part = threadIdx.x & 3;
        uint32_t a = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) a = L::larger(a, cmax[4 * part + k][L::PACKED ? c >> 1 : c]);
        a = L::larger(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = L::larger(a, __shfl_xor_sync(0xffffffffu, a, 2));
        if (L::PACKED) a = c & 1 ? a & 0xffff0000u : a << 16;
        if (part == 0) {
            const float d = divisor(a);
            dv[c] = d;
            iv[c] = __frcp_rn(d);
            if (c0 + c < p.cols) p.scale_t[(c0 + c) * p.st_row + br * p.st_grp] = __fdiv_rn(d, TOP);
        }
        __syncthreads();
    }
    const int rr = L::row(warp, lane);
    if constexpr (TRANSPOSE) {
#pragma unroll
        for (int j = 0; j < L::TC; ++j) {
            const int c = L::col(lane, j);
            const float d = dv[SQUARE ? 0 : c], inv = iv[SQUARE ? 0 : c];
#pragma unroll
            for (int i = 0; i < L::TR; i += 4) {
                const float f[4] = {t.at(i, j), t.at(i + 1, j), t.at(i + 2, j), t.at(i + 3, j)};
                tq[c * (PITCH / 4) + (rr + i) / 4] = e4m3x4(f, d, inv);
            }
        }
        __syncthreads();
        // a warp writes 128 bytes of an output row at a time
        const int64_t r = r0 + 4 * lane;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = warp * 8 + k;
            if (c0 + c >= p.cols) break;
            uint8_t* out = p.qt + (c0 + c) * p.ldqt + r;
            const uint32_t b = tq[c * (PITCH / 4) + lane];
            if (r + 4 <= p.rows) {
                *reinterpret_cast<uint32_t*>(out) = b;
            } else {
                for (int e = 0; e < 4; ++e)
                    if (r + e < p.rows) out[e] = (uint8_t)(b >> (8 * e));
            }
        }
    }
    if constexpr (ROWS) {
#pragma unroll
        for (int i = 0; i < L::TR; ++i) {
            const int64_t r = r0 + rr + i;
            float d = SQUARE ? dv[0] : 0.f, inv = SQUARE ? iv[0] : 0.f;
            if constexpr (!SQUARE) {             // the row's group: 16 or 32 lanes hold it
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) m = L::larger(m, L::mag(t.v[i][j]));
                m = L::widest(m);
                if (L::LPR == 32) {
                    m = __reduce_max_sync(0xffffffffu, m);
                } else {
#pragma unroll
                    for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                }
                d = divisor(m);
                inv = __frcp_rn(d);
                if (lane % L::LPR == 0 && r < p.rows) p.scale[r * p.s_row + bc * p.s_grp] = __fdiv_rn(d, TOP);
            }
            if (r >= p.rows) continue;
            uint8_t* out = p.q + r * p.ldq;
            float f[L::TC];
#pragma unroll
            for (int j = 0; j < L::TC; ++j) f[j] = t.at(i, j);
            if constexpr (VEC) {
                const int64_t c = c0 + L::col(lane, 0);
                if (c < p.cols) {
                    if constexpr (L::TC == 8)
                        *reinterpret_cast<uint2*>(out + c) = make_uint2(e4m3x4(f, d, inv), e4m3x4(f + 4, d, inv));
                    else
                        *reinterpret_cast<uint32_t*>(out + c) = e4m3x4(f, d, inv);
                }
            } else {
                const uint32_t b = e4m3x4(f, d, inv);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t c = c0 + L::col(lane, j);
                    if (c < p.cols) out[c] = (uint8_t)(b >> (8 * j));
                }
            }
        }
    }
}

}  // namespace fp8
}  // namespace evo
