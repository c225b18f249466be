// fp8_rows.cuh -- the memory-bound operators around the 8-bit projection:
//   add_rms_norm_kernel   h = x + residual, n = h / rms(h) * weight, n in e4m3
//                         with one scale per row and 128 channels
//   rms_bwd_kernel        its gradients (and sum_columns_kernel for d_weight)
//   quantize_tile_kernel  a matrix in e4m3 with 1 x 128 or 128 x 128 scales, as
//                         it lies or transposed
//
// A group whose largest magnitude is m (held at LEAST or above) keeps
//   q = e4m3(448 * v / m),   scale = m / 448.
// The quotient is rounded once to fp32 before the one rounding to e4m3.  With
// M = m / 512, t = 0.875 v and inv an approximate 1 / M, q0 = t * inv and the
// remainder t - q0 * M by a fused multiply-add, q0 + remainder * inv is the
// rounded quotient (Markstein's correction step; it leaves 2^-21 of a unit in the
// last place).  bf16 values make ties in e4m3 often enough to matter (448 =
// 7 * 64, so v = 3m/2^k is one); a plain product with 1/m would break them
// either way.  t is exact for bf16 v (fp32 values have a form of their own) and cannot
// overflow, and neither M nor inv
// leaves the normal range.  In the norm the row's 1 / rms cancels out of v / m,
// so the quotient is that of u = h * weight, exact in fp32 for bf16; its least
// maximum is LEAST * rms, and rows of a rms so small that its M would be
// subnormal are taken up by a power of two first.
//
// All of these move each byte once and are bound by HBM, next to it by the
// instructions: at 6.4 TB/s an SM has some 17 issue slots a value, so sums and
// products run on pairs (f32x2), bf16 adds on pairs too, and 1 / rms and 1 / M
// come from the approximate unit (2^-22), which the quotient above corrects.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "sm100.cuh"

namespace evo {
namespace fp8 {

using sm100::f2;
using sm100::f2hi;
using sm100::f2lo;
using sm100::fadd2;
using sm100::ffma2;
using sm100::fmul2;

constexpr int GROUP = 128;
constexpr float LEAST = 7.888609052210118e-31f;   // 2^-100: the smallest maximum a group is given
constexpr float TOP = 448.0f;                     // largest e4m3 value

__device__ __forceinline__ uint64_t twice(float v) { return f2(v, v); }
// Approximate reciprocal and reciprocal square root (hardware, normal range).
__device__ __forceinline__ float fast_rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Two values as e4m3, the low one in the low byte; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2(uint64_t v) { return e4m3x2(f2lo(v), f2hi(v)); }
// A group's divisor, ready for use on pairs: M = m / 512 (negated) and about 1 / M.
__device__ __forceinline__ float neg_of(float m) { return m * (-1.0f / 512.0f); }
__device__ __forceinline__ float inv_of(float m) { return fast_rcp(m * (1.0f / 512.0f)); }
struct Divisor {
    uint64_t neg, inv;
    __device__ __forceinline__ explicit Divisor(float m) : neg(twice(neg_of(m))), inv(twice(inv_of(m))) {}
    __device__ __forceinline__ Divisor(uint64_t n, uint64_t i) : neg(n), inv(i) {}   // another group for each of the pair
};
// 448 * v / m of a pair, rounded.  EXACT: 0.875 v is a float, as from bf16 values.  Else the remainder
// is taken in two steps, v - q M and that less v / 8: the first lies near v / 8 and rounds by 2^-27 v,
// the second is exact, so that the quotient is within 0.65 of a unit in the last place, and exact
// where it is a float (with 0.875 v rounded it missed ties by a unit; the rounding of 0.875 v carried
// along takes two more instructions: 131072 x 1024 117 -> 125 us).
template <bool EXACT>
__device__ __forceinline__ uint64_t quotient(uint64_t v, const Divisor& d) {
    if constexpr (EXACT) {
        const uint64_t t = fmul2(v, twice(0.875f)), q = fmul2(t, d.inv);
        return ffma2(ffma2(q, d.neg, t), d.inv, q);
    } else {
        const uint64_t q = fmul2(v, fmul2(d.inv, twice(0.875f)));
        return ffma2(ffma2(v, twice(-0.125f), ffma2(q, d.neg, v)), d.inv, q);
    }
}
// The same of v + low: what the norm's fp32 products have beyond v.
__device__ __forceinline__ uint64_t quotient(uint64_t v, uint64_t low, const Divisor& d) {
    const uint64_t c = twice(0.875f), t = fmul2(v, c), q = fmul2(t, d.inv);
    const uint64_t left = ffma2(c, low, ffma2(c, v, t ^ 0x8000000080000000ull));
    return ffma2(fadd2(ffma2(q, d.neg, t), left), d.inv, q);
}
// Four quotients as e4m3 bytes.
template <bool EXACT>
__device__ __forceinline__ uint32_t e4m3x4(uint64_t a, uint64_t b, const Divisor& d) {
    return e4m3x2(quotient<EXACT>(a, d)) | (e4m3x2(quotient<EXACT>(b, d)) << 16);
}
// |v| as an integer that orders like it, with NaN above infinity above the rest:
// the largest of a group is NaN as soon as one value is.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t magnitude(uint64_t v) { return max(magnitude(f2lo(v)), magnitude(f2hi(v))); }
// A group's maximum as a divisor: at least `least`, NaN where it is not finite.
__device__ __forceinline__ float divisor(uint32_t mag, float least = LEAST) {
    return mag >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : fmaxf(__uint_as_float(mag), least);
}

// ------------------------------------------------------------- row fragments
// A warp holds 256 columns of a row, 8 values a lane.
//   run   lane l holds columns 8l .. 8l + 7: a 128-group is a half warp.  bf16, and fp32 where VEC
//   else  lane l holds columns l + 32e (single loads, coalesced): values 0..3 lie in
//         the first group, 4..7 in the second
// VEC: every row is 16-byte aligned and the row's bytes are a multiple of 16, so a run is read
// 16 bytes at a time.  Other bf16 rows are read by aligned words, with a single value at either
// end of a run that starts at an odd one.
// Raw is a fragment as loaded, so that the next one can be on its way meanwhile.
template <typename T, bool VEC>
constexpr bool kRun = VEC || sizeof(T) == 2;
template <bool RUN>
__device__ __forceinline__ int frag_col(int lane, int e) {
    return RUN ? 8 * lane + e : lane + 32 * e;
}

// Eight bf16 values from p, of which the first `n` exist, as four pairs; zeros for the others.
__device__ __forceinline__ void load_run(const __nv_bfloat16* p, int64_t n, uint32_t* w) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    if (n >= 8) {
        if ((reinterpret_cast<uintptr_t>(h) & 2) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(h + 2 * i);
        } else {
            const uint32_t first = h[0], last = h[7];
            uint32_t m[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) m[i] = *reinterpret_cast<const uint32_t*>(h + 1 + 2 * i);
            w[0] = first | (m[0] << 16);
            w[1] = __funnelshift_r(m[0], m[1], 16);
            w[2] = __funnelshift_r(m[1], m[2], 16);
            w[3] = (m[2] >> 16) | (last << 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = 0;
            if (2 * i < n) w[i] = h[2 * i];
            if (2 * i + 1 < n) w[i] |= (uint32_t)h[2 * i + 1] << 16;
        }
    }
}
__device__ __forceinline__ void store_run(__nv_bfloat16* p, int64_t n, const uint32_t* w) {
    uint16_t* h = reinterpret_cast<uint16_t*>(p);
    if (n >= 8) {
        if ((reinterpret_cast<uintptr_t>(h) & 2) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(h + 2 * i) = w[i];
        } else {
            h[0] = (uint16_t)w[0];
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(h + 1 + 2 * i) = __funnelshift_r(w[i], w[i + 1], 16);
            h[7] = (uint16_t)(w[3] >> 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) h[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}
// Eight codes to q's row at column c (a multiple of 8; rows are 16-byte aligned), below `cols` only.
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t c, int64_t cols, uint32_t lo, uint32_t hi) {
    if (c + 8 <= cols) {
        *reinterpret_cast<uint2*>(row + c) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < cols) row[c + e] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
    }
}

template <typename T, bool VEC>
struct Raw {
    static constexpr bool PACKED = sizeof(T) == 2;
    static constexpr int N = PACKED ? 4 : 8;     // words: bf16 pairs or floats
    uint32_t w[N];

    __device__ __forceinline__ void load(const T* row, int64_t c0, int64_t cols, int lane) {
        if constexpr (VEC) {
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                const int64_t c = c0 + 8 * lane + 4 * h;
                uint4 a = make_uint4(0, 0, 0, 0);
                if (c < cols) a = *reinterpret_cast<const uint4*>(row + c);
                w[4 * h] = a.x;
                w[4 * h + 1] = a.y;
                w[4 * h + 2] = a.z;
                w[4 * h + 3] = a.w;
            }
        } else if constexpr (PACKED) {
            load_run(row + c0 + 8 * lane, cols - c0 - 8 * lane, w);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t c = c0 + lane + 32 * e;
                w[e] = c < cols ? __float_as_uint(Elem<T>::load(row + c)) : 0u;
            }
        }
    }
    __device__ __forceinline__ void store(T* row, int64_t c0, int64_t cols, int lane) const {
        if constexpr (VEC) {
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                const int64_t c = c0 + 8 * lane + 4 * h;
                if (c < cols) *reinterpret_cast<uint4*>(row + c) = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
            }
        } else if constexpr (PACKED) {
            store_run(row + c0 + 8 * lane, cols - c0 - 8 * lane, w);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t c = c0 + lane + 32 * e;
                if (c < cols) Elem<T>::store(row + c, __uint_as_float(w[e]));
            }
        }
    }
    // Values 2i and 2i + 1.
    __device__ __forceinline__ uint64_t pair(int i) const {
        if constexpr (PACKED) return sm100::bf16x2_to_f2(w[i]);
        return f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    // Sets values 2i and 2i + 1, rounded to T.
    __device__ __forceinline__ void set(int i, uint64_t v) {
        if constexpr (PACKED) {
            w[i] = sm100::pack_bf16(f2lo(v), f2hi(v));
        } else {
            w[2 * i] = __float_as_uint(f2lo(v));
            w[2 * i + 1] = __float_as_uint(f2hi(v));
        }
    }
    // this + o, rounded to T.
    __device__ __forceinline__ void add(const Raw& o) {
        if constexpr (PACKED) {                  // each half: one fp32 sum, rounded
#pragma unroll
            for (int i = 0; i < 4; ++i) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(o.w[i]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) set(i, fadd2(pair(i), o.pair(i)));
        }
    }
};

// Largest magnitude of each value's group: mag[0] for values 0..3, mag[1] for 4..7.
template <bool RUN>
__device__ __forceinline__ void group_max(const uint64_t* v, uint32_t* mag) {
    uint32_t a = max(magnitude(v[0]), magnitude(v[1])), b = max(magnitude(v[2]), magnitude(v[3]));
    if (RUN) {                                   // one group in this half warp
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

// The fragment's quotients, m[0] / m[1] the divisors of its two halves, as bytes of q's row.
// q rows are 16-byte aligned; only columns below `cols` are written.  `low`: what is left of each
// value beyond fp32, or null.
template <bool RUN>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int64_t c0, int64_t cols, int lane, const uint64_t* v,
                                           const float* m, const uint64_t* low = nullptr) {
    auto four = [&](int i, const Divisor& d) {
        if (!low) return e4m3x4<true>(v[i], v[i + 1], d);
        return e4m3x2(quotient(v[i], low[i], d)) | (e4m3x2(quotient(v[i + 1], low[i + 1], d)) << 16);
    };
    const Divisor d0(m[0]);
    const uint32_t lo = four(0, d0);
    uint32_t hi;
    if (RUN)
        hi = four(2, d0);
    else
        hi = four(2, Divisor(m[1]));
    if (RUN) {
        store_codes(row, c0 + 8 * lane, cols, lo, hi);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = c0 + lane + 32 * e;
            if (c < cols) row[c] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
        }
    }
}

// The scales of the fragment's two groups, from the lanes that own them.
template <bool RUN>
__device__ __forceinline__ void store_scales(float* s, int64_t stride, int64_t c0, int64_t cols, int lane,
                                             const float* sc) {
    const int64_t g = c0 / GROUP;
    if ((lane & 15) == 0) {
        const int h = lane >> 4;
        if (c0 + GROUP * h < cols) s[(g + h) * stride] = RUN ? sc[0] : sc[h];
    }
}

// ------------------------------------------------------------- add, norm, quantise
struct NormParams {
    int64_t rows, cols;
    const void *x, *res;         // T [rows, cols], res may be null
    int64_t ldx, ldres;
    const void* w;               // [cols], bf16 or fp32, or null (ones)
    int w_bf16;
    float eps, inv_cols;
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
// The weight of a lane's columns, in pairs; zero beyond the row.
template <bool RUN, int NV>
__device__ __forceinline__ void load_weight(const void* w, int bf16, int64_t cols, int wpr, int part, int lane,
                                            uint64_t (*out)[4]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t c0 = (int64_t)(i * wpr + part) * 256;
            const int64_t a = c0 + frag_col<RUN>(lane, 2 * e), b = c0 + frag_col<RUN>(lane, 2 * e + 1);
            out[i][e] = f2(a < cols ? load_w(w, bf16, a) : 0.f, b < cols ? load_w(w, bf16, b) : 0.f);
        }
}

// Sum of one value per lane over the `wpr` warps of a row, the first of them `first`.  Every warp
// of the block calls it; the caller alternates `buf`, so that one barrier per call is enough.
__device__ __forceinline__ float row_sum(float v, int wpr, int warp, int first, float* buf) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (wpr == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < wpr; ++i) s += buf[first + i];
    return s;
}

// A row lies with wpr warps, NV fragments of 256 columns each; a block of at most THREADS threads
// takes blockDim / 32 / wpr * R rows at a time (R rows per warp, only with wpr == 1) and walks the
// rows with the grid.  The weight stays in registers, and the next rows are loaded while these are
// worked on: at 32 warps of one row an SM has 32 KB on its way, too little for HBM's latency
// (196608 x 256 in bf16: 104 us; two rows a warp and the loads ahead 65, with three blocks an SM
// 61.5, of 54.9 at the copy's rate).
//
// SMALL, for eps below 2^-20: rows may have a smaller rms than 2^-10.  They go up by the power of two
// that leaves the rms at (1/2, 1]: exact, and u and its divisors, down to 2^-100 / 512 of the rms, stay
// in the normal range.  Any row times a factor takes 65 us there, so a larger eps does without.
template <typename T, bool VEC, int NV, int R, int THREADS, bool SMALL>
__global__ void __launch_bounds__(THREADS, THREADS != 256 ? 1 : R == 2 ? 3 : NV <= 2 ? 2 : 1) add_rms_norm_kernel(const NormParams p, const int wpr) {
    __shared__ float buf[2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = warp / wpr * wpr, part = warp - first;
    const int per = (int)(blockDim.x >> 5) / wpr * R, sub = warp / wpr * R;
    const int64_t step = (int64_t)gridDim.x * per;
    uint64_t w[NV][4];
    load_weight<kRun<T, VEC>, NV>(p.w, p.w_bf16, p.cols, wpr, part, lane, w);
    Raw<T, VEC> x[R][NV], res[R][NV];
    auto load = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c0 = (int64_t)(i * wpr + part) * 256, lim = r + k < p.rows ? p.cols : 0;
                x[k][i].load(static_cast<const T*>(p.x) + (r + k) * p.ldx, c0, lim, lane);
                if (p.res) res[k][i].load(static_cast<const T*>(p.res) + (r + k) * p.ldres, c0, lim, lane);
            }
    };
    int64_t r = (int64_t)blockIdx.x * per + sub;
    load(r);
    int turn = 0;
    // every warp makes the same number of turns, for the barrier in row_sum
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < p.rows; r0 += step, r += step, turn ^= 1) {
        Raw<T, VEC> h[R][NV];
        float rstd[R], up[R], rs[R], least[R], per_m[R];
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                h[k][i] = x[k][i];
                if (p.res) h[k][i].add(res[k][i]);
            }
        load(r + step);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            uint64_t sq = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) sq = ffma2(h[k][i].pair(e), h[k][i].pair(e), sq);
            const float ms = row_sum(f2lo(sq) + f2hi(sq), wpr, warp, first, buf[turn]) * p.inv_cols + p.eps;
            rstd[k] = rsqrtf(ms);
            up[k] = 1.f;                                   // the row's factor, and what it leaves of 1 / rms
            rs[k] = rstd[k];
            if (SMALL) {
                const uint32_t e = min(max(__float_as_uint(rstd[k]) & 0x7f800000u, 0x3f800000u), 0x7e800000u);
                up[k] = __uint_as_float(e);
                rs[k] *= __uint_as_float(0x7f000000u - e); // 1 / up
            }
            least[k] = LEAST * (ms * rstd[k] * up[k]);     // LEAST / rs: the least maximum of u = n / rs
            per_m[k] = least[k] == least[k] ? rs[k] * (1.0f / TOP) : least[k];     // NaN where ms is 0 or infinite
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t row = r + k;
            if (row >= p.rows) continue;                   // no barrier below
            if (p.rstd && part == 0 && lane == 0) p.rstd[row] = rstd[k];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c0 = (int64_t)(i * wpr + part) * 256;
                if (c0 >= p.cols) break;
                if (p.h) h[k][i].store(static_cast<T*>(p.h) + row * p.ldh, c0, p.cols, lane);
                uint64_t v[4], u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = h[k][i].pair(e);
                    if (SMALL) v[e] = fmul2(v[e], twice(up[k]));
                    u[e] = fmul2(v[e], w[i][e]);
                }
                if (p.n) {
                    Raw<T, VEC> n;
#pragma unroll
                    for (int e = 0; e < 4; ++e) n.set(e, fmul2(u[e], twice(rs[k])));
                    n.store(static_cast<T*>(p.n) + row * p.ldn, c0, p.cols, lane);
                }
                uint32_t mag[2];
                group_max<kRun<T, VEC>>(u, mag);
                float m[2], sc[2];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    m[g] = divisor(mag[g], least[k]);
                    sc[g] = m[g] * per_m[k];
                }
                if constexpr (sizeof(T) == 4) {            // fp32: u is rounded, its rest goes into the quotient
                    uint64_t low[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) low[e] = ffma2(v[e], w[i][e], u[e] ^ 0x8000000080000000ull);
                    store_e4m3<kRun<T, VEC>>(p.q + row * p.ldq, c0, p.cols, lane, u, m, low);
                } else {
                    store_e4m3<kRun<T, VEC>>(p.q + row * p.ldq, c0, p.cols, lane, u, m);
                }
                store_scales<kRun<T, VEC>>(p.scale + row * p.s_row, p.s_grp, c0, p.cols, lane, sc);
            }
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
    float inv_cols;
    void* dx;                    // T [rows, cols]
    int64_t lddx;
    float* part;                 // fp32 [gridDim.x, cols] partial sums of d_weight, or null
};

// dx = dh + rstd * (g - n * mean(g n)), g = dy * w, n = h * rstd.  Each warp adds up dy * n of
// the rows it meets in registers; a block's rows are joined in shared memory and leave one
// partial row, and sum_columns_kernel adds the partial rows in order: no atomics, the same
// bits on every run.  Layout and loads ahead as in the forward: 196608 x 256 in bf16 takes 70 us
// (62.5 at the copy's rate), 92 without the loads ahead; a third block per SM spills (116).
template <typename T, bool VEC, int NV, int R, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1) rms_bwd_kernel(const NormBwdParams p, const int wpr) {
    __shared__ float buf[2][32];
    extern __shared__ float join[];              // [warps][NV][256] when a block holds several rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = warp / wpr * wpr, part = warp - first;
    const int rows_b = (int)(blockDim.x >> 5) / wpr, per = rows_b * R, sub = warp / wpr * R;
    const int64_t step = (int64_t)gridDim.x * per;
    uint64_t w[NV][4], dw[NV][4];
    load_weight<kRun<T, VEC>, NV>(p.w, p.w_bf16, p.cols, wpr, part, lane, w);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[i][e] = 0;
    Raw<T, VEC> dy[R][NV], h[R][NV], dh[R][NV];
    float rs[R];
    auto load = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const bool live = r + k < p.rows;
            rs[k] = live ? p.rstd[r + k] : 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c0 = (int64_t)(i * wpr + part) * 256, lim = live ? p.cols : 0;
                dy[k][i].load(static_cast<const T*>(p.dy) + (r + k) * p.lddy, c0, lim, lane);
                h[k][i].load(static_cast<const T*>(p.h) + (r + k) * p.ldh, c0, lim, lane);
                if (p.dh) dh[k][i].load(static_cast<const T*>(p.dh) + (r + k) * p.lddh, c0, lim, lane);
            }
        }
    };
    constexpr bool AHEAD = THREADS <= 640;       // else the registers do not hold two rows
    int64_t r = (int64_t)blockIdx.x * per + sub;
    if (AHEAD) load(r);
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < p.rows; r0 += step, r += step, turn ^= 1) {
        if (!AHEAD) load(r);
        uint64_t g[R][NV][4], n[R][NV][4], a[R][NV][4];
        float rstd[R], mean[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            rstd[k] = rs[k];
            const uint64_t rs2 = twice(rs[k]);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {              // a row past the end is all zeros
                    n[k][i][e] = fmul2(h[k][i].pair(e), rs2);
                    const uint64_t y = dy[k][i].pair(e);
                    dw[i][e] = ffma2(y, n[k][i][e], dw[i][e]);
                    g[k][i][e] = fmul2(y, w[i][e]);
                    a[k][i][e] = p.dh ? dh[k][i].pair(e) : 0;
                }
        }
        if (AHEAD) load(r + step);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            uint64_t dot = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) dot = ffma2(g[k][i][e], n[k][i][e], dot);
            mean[k] = row_sum(f2lo(dot) + f2hi(dot), wpr, warp, first, buf[turn]) * p.inv_cols;
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t row = r + k;
            if (row >= p.rows) continue;
            const uint64_t neg = twice(-mean[k]), rs2 = twice(rstd[k]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c0 = (int64_t)(i * wpr + part) * 256;
                if (c0 >= p.cols) break;
                Raw<T, VEC> o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o.set(e, ffma2(rs2, ffma2(n[k][i][e], neg, g[k][i][e]), a[k][i][e]));
                o.store(static_cast<T*>(p.dx) + row * p.lddx, c0, p.cols, lane);
            }
        }
    }
    if (!p.part) return;
    float* out = p.part + (int64_t)blockIdx.x * p.cols;
    if (rows_b > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                join[(warp * NV + i) * 256 + frag_col<kRun<T, VEC>>(lane, 2 * e)] = f2lo(dw[i][e]);
                join[(warp * NV + i) * 256 + frag_col<kRun<T, VEC>>(lane, 2 * e + 1)] = f2hi(dw[i][e]);
            }
        __syncthreads();
        // column c of the row lies with warp (c / 256) % wpr of each row, fragment (c / 256) / wpr
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            const int f = (int)(c >> 8), o = (f % wpr * NV + f / wpr) * 256 + (int)(c & 255);
            float s = 0.f;
            for (int k = 0; k < rows_b; ++k) s += join[k * wpr * NV * 256 + o];
            out[c] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t c0 = (int64_t)(i * wpr + part) * 256;
                const int64_t ca = c0 + frag_col<kRun<T, VEC>>(lane, 2 * e), cb = c0 + frag_col<kRun<T, VEC>>(lane, 2 * e + 1);
                if (ca < p.cols) out[ca] = f2lo(dw[i][e]);
                if (cb < p.cols) out[cb] = f2hi(dw[i][e]);
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

// A 128 x 128 tile of x in one block of 512 threads, TC columns x TR rows a thread:
//   bf16      8 columns x 4 rows (16-byte loads where VEC, 16 lanes a row), kept as loaded
//   fp32 VEC  4 columns x 8 rows (16-byte loads, a warp a row)
//   else      columns l + 32j, 8 rows (single loads, a warp a row)
template <typename T, bool VEC>
struct Tile {
    static constexpr bool PACKED = sizeof(T) == 2, RUN = kRun<T, VEC>;
    static constexpr int TC = PACKED ? 8 : 4;
    static constexpr int TR = 32 / TC;
    static constexpr int LPR = 128 / TC;         // lanes a row
    uint32_t v[TR][4];                           // four bf16 pairs or four floats

    static __device__ __forceinline__ int col(int lane, int j) { return RUN ? (lane % LPR) * TC + j : lane + 32 * j; }
    static __device__ __forceinline__ int row(int warp, int lane) { return warp * 8 + (lane / LPR) * TR; }

    __device__ __forceinline__ void load(const QuantParams& p, int64_t r0, int64_t c0, int warp, int lane) {
        const int64_t r = r0 + row(warp, lane), c = c0 + col(lane, 0);
        const int rows = (int)min((int64_t)TR, p.rows - r);
        const T* x = static_cast<const T*>(p.x) + r * p.ldx + (RUN ? c : c0);
#pragma unroll
        for (int i = 0; i < TR; ++i, x += p.ldx) {
            const bool live = i < rows && c < p.cols;
            if constexpr (VEC) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (live) w = *reinterpret_cast<const uint4*>(x);
                v[i][0] = w.x;
                v[i][1] = w.y;
                v[i][2] = w.z;
                v[i][3] = w.w;
            } else if constexpr (PACKED) {
                load_run(x, live ? p.cols - c : 0, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i][j] = live && c + 32 * j < p.cols ? __float_as_uint(Elem<T>::load(x + col(lane, j))) : 0u;
            }
        }
    }
    // Columns 2j and 2j + 1 of row i.
    __device__ __forceinline__ uint64_t pair(int i, int j) const {
        if constexpr (PACKED) return sm100::bf16x2_to_f2(v[i][j]);
        return f2(__uint_as_float(v[i][2 * j]), __uint_as_float(v[i][2 * j + 1]));
    }
    // Where word w (four rows) of column c lies in the transposed tile: rotated by the lane that
    // writes the column, so that a warp's words, and a column's, meet 32 banks.
    static __device__ __forceinline__ int owner(int c) { return PACKED ? c >> 3 : RUN ? c >> 2 : c & 31; }
    static __device__ __forceinline__ int spot(int c, int w) { return c * 32 + (w ^ (PACKED ? 2 * owner(c) : owner(c))); }
    // The divisors of a lane's j-th column pair lie together, those of the lanes side by side: index
    // of column c's float (its M, and two further its 1 / M).
    static __device__ __forceinline__ int pair_at(int lane, int j) { return 4 * (j * LPR + lane % LPR); }
    static __device__ __forceinline__ int divisor_at(int c) {
        return RUN ? pair_at(owner(c), (c % TC) >> 1) + (c & 1) : pair_at(c & 31, c >> 6) + ((c >> 5) & 1);
    }
    // Magnitudes as integers that order like them: pairs of 16 bits (PACKED) or one of 32.
    static __device__ __forceinline__ uint32_t mag(uint32_t w) { return w & (PACKED ? 0x7fff7fffu : 0x7fffffffu); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        if (!PACKED) return max(a, b);
        asm("max.u16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return a;
    }
    // The larger of a pair (PACKED), as the bits of a float.
    static __device__ __forceinline__ uint32_t widest(uint32_t m) {
        return PACKED ? max(m << 16, m & 0xffff0000u) : m;
    }
};

// 128 x 128 blocks (SQUARE), or 1 x 128 groups along the columns for q and along the rows for the
// transpose.  ROWS writes q, TRANSPOSE the transpose, through shared memory.  ROWS alone, in 1 x 128
// groups, needs neither shared memory nor a barrier (40000 x 1000 in bf16: 28 us; a warp for 256
// columns of a row at a time took 51).  The transposing form is
// bound by its instructions (15 a value; 131072 x 1024 in bf16: 85 us, 63 at the copy's rate): column
// pairs go through the quotient together, three blocks an SM (bf16) cover each other's barriers.
// Walking the tiles with the next one on its way in registers took 115 us, for the blocks it costs.
template <typename T, bool VEC, bool SQUARE, bool ROWS, bool TRANSPOSE>
__global__ void __launch_bounds__(512, Tile<T, VEC>::PACKED && !(ROWS && TRANSPOSE) ? 3 : 2) quantize_tile_kernel(const QuantParams p) {
    using L = Tile<T, VEC>;
    constexpr int W = L::PACKED ? 64 : 128;      // words of a warp's column maxima
    constexpr bool BY_COL = TRANSPOSE && !SQUARE;
    __shared__ uint32_t cmax[BY_COL ? 16 : 1][BY_COL ? W + 2 : 16];
    __shared__ __align__(16) float dv[BY_COL ? 256 : 1];   // BY_COL: M and 1 / M of every column
    __shared__ uint32_t tq[TRANSPOSE ? 128 * 32 : 1];
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
                if (ROWS) p.scale[br * p.s_row + bc * p.s_grp] = d * (1.0f / TOP);
                if (TRANSPOSE) p.scale_t[bc * p.st_row + br * p.st_grp] = d * (1.0f / TOP);
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
            dv[L::divisor_at(c)] = neg_of(d);
            dv[L::divisor_at(c) + 2] = inv_of(d);
            if (c0 + c < p.cols) p.scale_t[(c0 + c) * p.st_row + br * p.st_grp] = d * (1.0f / TOP);
        }
        __syncthreads();
    }
    const int rr = L::row(warp, lane);
    if constexpr (TRANSPOSE) {
#pragma unroll
        for (int j = 0; j < L::TC / 2; ++j) {
            const int c = L::col(lane, 2 * j), c1 = L::col(lane, 2 * j + 1);
            Divisor d(0, 0);
            if constexpr (SQUARE) {
                d = Divisor(dv[0]);
            } else {
                const float4 f = *reinterpret_cast<const float4*>(dv + L::pair_at(lane, j));
                d = Divisor(f2(f.x, f.y), f2(f.z, f.w));
            }
#pragma unroll
            for (int i = 0; i < L::TR; i += 4) {
                uint64_t q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) q[k] = quotient<L::PACKED>(t.pair(i + k, j), d);
                tq[L::spot(c, (rr + i) / 4)] = e4m3x2(f2lo(q[0]), f2lo(q[1])) | (e4m3x2(f2lo(q[2]), f2lo(q[3])) << 16);
                tq[L::spot(c1, (rr + i) / 4)] = e4m3x2(f2hi(q[0]), f2hi(q[1])) | (e4m3x2(f2hi(q[2]), f2hi(q[3])) << 16);
            }
        }
        __syncthreads();
        // a warp writes 128 bytes of an output row at a time
        const int64_t r = r0 + 4 * lane;
        const int cols = (int)min((int64_t)8, p.cols - c0 - warp * 8);
        uint8_t* out = p.qt + (c0 + warp * 8) * p.ldqt + r;
        const bool whole = r + 4 <= p.rows;
#pragma unroll
        for (int k = 0; k < 8; ++k, out += p.ldqt) {
            if (k >= cols) break;
            const uint32_t b = tq[L::spot(warp * 8 + k, lane)];
            if (whole) {
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
            float m_row = SQUARE ? dv[0] : 0.f;
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
                m_row = divisor(m);
                if (lane % L::LPR == 0 && r < p.rows) p.scale[r * p.s_row + bc * p.s_grp] = m_row * (1.0f / TOP);
            }
            if (r >= p.rows) continue;
            uint8_t* out = p.q + r * p.ldq;
            const Divisor d(m_row);
            uint64_t f[L::TC / 2];
#pragma unroll
            for (int j = 0; j < L::TC / 2; ++j) f[j] = t.pair(i, j);
            if constexpr (L::PACKED) {
                store_codes(out, c0 + L::col(lane, 0), p.cols, e4m3x4<true>(f[0], f[1], d), e4m3x4<true>(f[2], f[3], d));
            } else if constexpr (VEC) {
                const int64_t c = c0 + L::col(lane, 0);
                if (c < p.cols) *reinterpret_cast<uint32_t*>(out + c) = e4m3x4<false>(f[0], f[1], d);
            } else {
                const uint32_t b = e4m3x4<false>(f[0], f[1], d);
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
