// RMSNorm, with or without the residual's addition, writing 8-bit values
// (e4m3 or int8) and their scales.
//
//   s = x + residual (fp32; the residual is stored back as bf16), or s = x
//   y = s * rsqrt(mean(s^2) + eps) * w              (fp32, never rounded to bf16)
//   scale = max(max|y| / Q, 2^-100), Q = 448 (e4m3) or 127 (int8), over the
//           row or over each group of 128 columns
//   q = y / scale, rounded to nearest (ties to even)
//
// Bound by memory: 7 bytes per element with the residual (x, residual in and
// out, q), 3 without.  The row stays in registers as the products s * w, and
// since max|y| = rstd * max|s w| the largest product is found in the same
// pass as the sum of squares: a row takes one reduction, not two.  The
// largest magnitude is compared as bit patterns, where NaN and infinity order
// above every number, so neither is lost the way fmaxf loses a NaN.
#include "common.cuh"
#include "pairs.cuh"
#include "pdl.cuh"
#include "tokens.h"

namespace nf {
namespace {

constexpr float kScaleMin = 0x1p-100f;  // a group of zeros still has a scale that can be divided by

__device__ __forceinline__ bool finite_bits(float f) {
    return (__float_as_uint(f) & 0x7F800000u) != 0x7F800000u;
}

// Four values to four bytes, the first in the lowest.  |v| <= Q up to one
// rounding of y / scale, which rounds back to Q.
template <bool INT8>
__device__ __forceinline__ uint32_t quant4(float2 a, float2 b) {
    if constexpr (INT8) {
        // adding 1.5 * 2^23 leaves the integer nearest to v (ties to even) in the low bits
        const float2 magic = make_float2(12582912.f, 12582912.f);
        a = __fadd2_rn(a, magic);
        b = __fadd2_rn(b, magic);
        const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    } else {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
        return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
}

// The scale of a group whose largest |s w| has the bits `top`.
template <bool INT8>
__device__ __forceinline__ float scale_of(uint32_t top, float rstd) {
    const float v = __uint_as_float(top) * rstd * (INT8 ? 1.0f / 127.0f : 1.0f / 448.0f);
    return v < kScaleMin ? kScaleMin : v;  // false for NaN, which stays
}

// y / scale = s w * first * second.  rstd stands in y and in the scale alike,
// so the quotient is s w * (Q / max|s w|): fewer roundings than y / scale has.
// Where max|s w| is so small that Q over it could overflow, or the scale is
// the smallest one, the factors are rstd and 1 / scale, one after the other
// (their product alone could overflow).
struct Factors {
    float first, second;
};
template <bool INT8>
__device__ __forceinline__ Factors factors(float top, float rstd, float scale) {
    Factors f;
    const bool direct = top >= kScaleMin && scale > kScaleMin;
    f.first = direct ? 1.f : rstd;
    f.second = __fdiv_rn(direct ? (INT8 ? 127.f : 448.f) : 1.f, direct ? top : scale);
    return f;
}

// A row per blockDim.x threads (a multiple of 32), blockDim.y rows per CTA
// (more than one only where a row is one warp).  Thread t holds the vectors
// k * T + t, k < VPT, so 16 neighbouring lanes hold a group of 128 columns.
// MAXT bounds the CTA size, so that rows of up to 512 threads (hidden 16384 at
// four vectors per thread) keep a larger register budget.
template <int VPT, int MAXT, bool RES, bool INT8, bool GROUPED>
__global__ void __launch_bounds__(MAXT)
norm_q8_rows(const Q8Args a) {
    __shared__ float red_sum[32];
    __shared__ uint32_t red_top[32];
    const int T = blockDim.x, t = threadIdx.x;
    const int H = a.hidden, NV = H / kVec;
    const float inv_h = 1.0f / static_cast<float>(H);
    grid_dep_wait();
    grid_dep_release();
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows; row += step) {
        const uint16_t* xr = a.x + row * H;
        uint16_t* rr = RES ? a.res + row * H : nullptr;
        uint4 xv[VPT], rv[RES ? VPT : 1];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * T + t;
            xv[k] = make_uint4(0, 0, 0, 0);
            if constexpr (RES) rv[k] = xv[k];
            if (v < NV) {
                xv[k] = ld_stream(xr + v * kVec);
                if constexpr (RES) rv[k] = ld_stream(rr + v * kVec);
            }
        }
        float2 p[VPT][4];  // s * w
        uint32_t top[VPT];
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * T + t;
            top[k] = 0;
            float2 s[4], wf[4];
            unpack8x2(xv[k], s);
            if constexpr (RES) {
                float2 r[4];
                unpack8x2(rv[k], r);
#pragma unroll
                for (int q = 0; q < 4; ++q) s[q] = __fadd2_rn(s[q], r[q]);
                if (v < NV) st_stream(rr + v * kVec, pack8x2(s));
            }
            unpack8x2(v < NV ? ld_param(a.w + v * kVec) : make_uint4(0, 0, 0, 0), wf);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                ss = __ffma2_rn(s[q], s[q], ss);
                p[k][q] = __fmul2_rn(s[q], wf[q]);
                top[k] = max(top[k], max(__float_as_uint(p[k][q].x) & 0x7FFFFFFFu,
                                         __float_as_uint(p[k][q].y) & 0x7FFFFFFFu));
            }
        }
        float sum[1] = {ss.x + ss.y};
        uint32_t row_top = 0;
        warp_sum<1>(sum);
        if constexpr (GROUPED) {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int off = 8; off > 0; off >>= 1)
                    top[k] = max(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], off));
        } else {
#pragma unroll
            for (int k = 0; k < VPT; ++k) row_top = max(row_top, top[k]);
            row_top = __reduce_max_sync(0xFFFFFFFFu, row_top);
        }
        if (T > 32) {
            const int warp = t >> 5, nw = T >> 5;
            if ((t & 31) == 0) {
                red_sum[warp] = sum[0];
                if constexpr (!GROUPED) red_top[warp] = row_top;
            }
            __syncthreads();
            sum[0] = 0.f;
            for (int i = 0; i < nw; ++i) {
                sum[0] += red_sum[i];
                if constexpr (!GROUPED) row_top = max(row_top, red_top[i]);
            }
        }
        // a sum that is not finite (NaN, infinity, or values beyond 1.8e19 whose
        // squares overflow) has no norm: every scale of the row is NaN, every q 0
        const float rstd = finite_bits(sum[0]) ? rsqrtf(sum[0] * inv_h + a.eps) : __uint_as_float(0x7FC00000u);
        float row_scale = 0.f;
        if constexpr (!GROUPED) {
            row_scale = scale_of<INT8>(row_top, rstd);
            if (t == 0) a.scale[row] = row_scale;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * T + t;
            float scale = row_scale;
            if constexpr (GROUPED) {
                scale = scale_of<INT8>(top[k], rstd);
                if ((t & 15) == 0 && v < NV) a.scale[row * a.groups + v / 16] = scale;
            }
            const float t_max = __uint_as_float(GROUPED ? top[k] : row_top);
            const Factors f = factors<INT8>(t_max, rstd, scale);
            const float2 f1 = make_float2(f.first, f.first), f2 = make_float2(f.second, f.second);
            float2 o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = __fmul2_rn(__fmul2_rn(p[k][q], f1), f2);
            uint2 bytes = make_uint2(quant4<INT8>(o[0], o[1]), quant4<INT8>(o[2], o[3]));
            if (!finite_bits(scale)) bytes = make_uint2(0, 0);
            if (v < NV) __stcs(reinterpret_cast<uint2*>(a.q + row * H + v * kVec), bytes);
        }
        if (T > 32) __syncthreads();  // the reduction buffers are reused by the next row
    }
}

template <int VPT, int MAXT, bool RES, bool INT8, bool GROUPED>
cudaError_t go(const Q8Args& a, int threads, int rows_per_cta, cudaStream_t st) {
    const int64_t blocks = (a.rows + rows_per_cta - 1) / rows_per_cta;
    const unsigned grid = static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF);
    return launch_with_pdl(norm_q8_rows<VPT, MAXT, RES, INT8, GROUPED>, dim3(grid), dim3(threads, rows_per_cta), 0, st, a);
}

template <int VPT, int MAXT>
cudaError_t go(const Q8Args& a, bool int8, bool grouped, int threads, int rpc, cudaStream_t st) {
    const int pick = (a.res ? 4 : 0) | (int8 ? 2 : 0) | (grouped ? 1 : 0);
    switch (pick) {
        case 0: return go<VPT, MAXT, false, false, false>(a, threads, rpc, st);
        case 1: return go<VPT, MAXT, false, false, true>(a, threads, rpc, st);
        case 2: return go<VPT, MAXT, false, true, false>(a, threads, rpc, st);
        case 3: return go<VPT, MAXT, false, true, true>(a, threads, rpc, st);
        case 4: return go<VPT, MAXT, true, false, false>(a, threads, rpc, st);
        case 5: return go<VPT, MAXT, true, false, true>(a, threads, rpc, st);
        case 6: return go<VPT, MAXT, true, true, false>(a, threads, rpc, st);
        default: return go<VPT, MAXT, true, true, true>(a, threads, rpc, st);
    }
}

}  // namespace

cudaError_t launch_norm_q8(const Q8Args& a, bool int8, bool grouped, int sms, cudaStream_t st) {
    (void)sms;
    const int nv = a.hidden / kVec;
    const auto threads = [nv](int vpt) { return ((nv + vpt - 1) / vpt + 31) / 32 * 32; };
    if (a.rows <= 256 && threads(2) <= 1024) return go<2, 1024>(a, int8, grouped, threads(2), 1, st);
    const int t = threads(4);
    if (t > 512) return go<4, 1024>(a, int8, grouped, t, 1, st);
    return go<4, 512>(a, int8, grouped, t, t == 32 ? 4 : 1, st);
}

}  // namespace nf
