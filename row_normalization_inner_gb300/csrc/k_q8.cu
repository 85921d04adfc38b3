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
// out, q), 3 without (16384 x 8192 e4m3 with group scales on a GB300: 136 us,
// 6.9 TB/s, with the residual, 66 us, 6.1 TB/s, without).  The row stays in registers as the products s * w, and
// since max|y| = rstd * max|s w| the largest product is found in the same
// pass as the sum of squares: a row takes one reduction, not two.  The
// largest magnitude is compared as bit patterns, where NaN and infinity order
// above every number, so neither is lost the way fmaxf loses a NaN.
#include <atomic>

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

// rstd stands in y and in the scale alike, so y / scale is s w * (Q / max|s w|):
// fewer roundings than dividing y has.  Only a maximum so small or so large
// that the quotient could leave fp32, or a smallest scale, takes y itself.
// Q / max is divided exactly where a row has one (no time at any size; 15% to
// 30% fewer values that round to the neighbour of the exact result's) and is an
// approximate reciprocal where every thread computes its group's: exact there,
// 16384 x 8192 e4m3 would take 72.1 us for 66.3 and 12% fewer such values.
__device__ __forceinline__ bool plain_range(float top, float scale) {
    return top >= kScaleMin && top <= 0x1p100f && scale > kScaleMin;
}
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest magnitude of three, a NaN standing above every number.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// a * b + c of bf16 a, b in fp32 (the product of two bf16 is exact there).
__device__ __forceinline__ float fma_bf16(uint16_t a, uint16_t b, float c) {
    float d;
    asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"(a), "h"(b), "f"(c));
    return d;
}

// The ring's share of an SM: shared memory (each CTA needs some 1.7 KB
// besides) and threads, for which its kernels are compiled.  Fewer threads
// than would fit, since more made it slower (16384 x 4096: 512 threads 34.0
// us, 768 34.6 us, 1024 43.7 us; 5120: 39.4, 42.0, 56.0 us), except that rows
// of 193 to 384 threads take 768 (8192: 512 threads 66.8 us, 768 62.7 us; with
// group scales 66.1 and 73.9 us) and longer ones what 1024 give.  Every row
// length gets three stages or more.
constexpr int kRingBytes = 200 * 1024;
constexpr int kRingMaxStages = 8;
constexpr int ring_threads(int maxt, bool grouped) {
    return maxt <= 192 || (maxt <= 256 && grouped) ? 512 : maxt <= 384 ? 768 : 1024;
}
constexpr bool three_stages(int ctas, int threads) { return kRingBytes / ctas / (4 * threads * 16) >= 3; }
static_assert(three_stages(4, 128) && three_stages(3, 160) && three_stages(2, 192) && three_stages(3, 256) &&
              three_stages(2, 384) && three_stages(2, 512) && three_stages(1, 1024), "stages");
// Shorter rows stay with the row-per-CTA form (16384 x 1024: 10.3 us; the ring 11.3 us).
constexpr int kRingMinThreads = 128;

__device__ __forceinline__ void bulk_copy(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_addr(to)), "l"(from), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}

// The row of a thread: vectors k * T + t, k < VPT, so that 16 neighbouring
// lanes hold a group of 128 columns.
// RING: the products take the mixed-precision form (with it the ring was
// faster, 16384 x 8192 71 -> 63 us, and the row-per-CTA form slower, 16384 x
// 4096 34 -> 38 us), and the weight's vectors are the caller's where KEEPW (a
// CTA's threads keep them for all their rows) or read here.
template <int VPT, bool RES, bool INT8, bool GROUPED, bool RING, bool KEEPW>
struct Q8Row {
    float2 p[VPT][4];    // s * w
    uint32_t top[VPT];   // bits of the largest |s w| of the vector; GROUPED: of its group
    float sum;           // of squares
    uint32_t row_top;

    // From the loaded vectors; stores the residual.
    __device__ __forceinline__ void products(const Q8Args& a, int64_t row, const uint4 (&xv)[VPT],
                                             const uint4 (&rv)[RES ? VPT : 1], const uint4 (&wk)[KEEPW ? VPT : 1],
                                             int T, int t) {
        const int NV = a.hidden / kVec;
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * T + t;
            uint4 wv;
            if constexpr (KEEPW) wv = wk[k];
            else wv = v < NV ? ld_param(a.w + v * kVec) : make_uint4(0, 0, 0, 0);
            if constexpr (RING && !RES) {
                const uint32_t xs[4] = {xv[k].x, xv[k].y, xv[k].z, xv[k].w}, ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint16_t xl = xs[q] & 0xFFFF, xh = xs[q] >> 16, wl = ws[q] & 0xFFFF, wh = ws[q] >> 16;
                    ss.x = fma_bf16(xl, xl, ss.x);
                    ss.y = fma_bf16(xh, xh, ss.y);
                    p[k][q] = make_float2(fma_bf16(xl, wl, 0.f), fma_bf16(xh, wh, 0.f));
                }
            } else {
                float2 s[4], wf[4];
                unpack8x2(xv[k], s);
                if constexpr (RES) {
                    float2 r[4];
                    unpack8x2(rv[k], r);
#pragma unroll
                    for (int q = 0; q < 4; ++q) s[q] = __fadd2_rn(s[q], r[q]);
                    if (v < NV) st_stream(a.res + row * a.hidden + v * kVec, pack8x2(s));
                }
                unpack8x2(wv, wf);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    ss = __ffma2_rn(s[q], s[q], ss);
                    p[k][q] = __fmul2_rn(s[q], wf[q]);
                }
            }
            float m = max3_abs(p[k][0].x, p[k][0].y, p[k][1].x);
            m = max3_abs(m, p[k][1].y, p[k][2].x);
            m = max3_abs(m, p[k][2].y, p[k][3].x);
            top[k] = __float_as_uint(max3_abs(m, p[k][3].y, 0.f)) & 0x7FFFFFFFu;
        }
        sum = ss.x + ss.y;
        row_top = 0;
    }

    // Over the warp, and (GROUPED) over the group's 16 lanes.
    __device__ __forceinline__ void reduce_warp() {
        float v[1] = {sum};
        warp_sum<1>(v);
        sum = v[0];
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
    }

    // The warps' values, in a fixed order, on either side of a CTA barrier.
    __device__ __forceinline__ void leave(float* red_sum, uint32_t* red_top, int t) const {
        if ((t & 31) == 0) {
            red_sum[t >> 5] = sum;
            if constexpr (!GROUPED) red_top[t >> 5] = row_top;
        }
    }
    // The buffers hold zeros behind the warps' entries.
    __device__ __forceinline__ void collect(const float* red_sum, const uint32_t* red_top, int warps) {
        sum = 0.f;
        for (int i = 0; i < warps; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(red_sum + i);
            sum += (f.x + f.y) + (f.z + f.w);
            if constexpr (!GROUPED) {
                const uint4 u = *reinterpret_cast<const uint4*>(red_top + i);
                row_top = max(max(row_top, u.x), max(max(u.y, u.z), u.w));
            }
        }
    }

    // Scales and 8-bit values.
    __device__ __forceinline__ void finish(const Q8Args& a, int64_t row, int T, int t) const {
        const int H = a.hidden, NV = H / kVec;
        // a sum that is not finite (NaN, infinity, or values beyond 1.8e19 whose
        // squares overflow) has no norm: every scale of the row is NaN, every q 0
        const float rstd = finite_bits(sum) ? rsqrtf(sum * (1.0f / static_cast<float>(H)) + a.eps)
                                            : __uint_as_float(0x7FC00000u);
        float row_scale = 0.f, factor = 0.f;
        bool range = true;
        if constexpr (!GROUPED) {
            const float top_value = __uint_as_float(row_top);
            row_scale = scale_of<INT8>(row_top, rstd);
            range = plain_range(top_value, row_scale);
            factor = __fdiv_rn(INT8 ? 127.f : 448.f, top_value);
            if (t == 0) a.scale[row] = row_scale;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * T + t;
            float scale = row_scale;
            if constexpr (GROUPED) {
                const float top_value = __uint_as_float(top[k]);
                scale = scale_of<INT8>(top[k], rstd);
                range = plain_range(top_value, scale);
                factor = (INT8 ? 127.f : 448.f) * reciprocal(top_value);
                if ((t & 15) == 0 && v < NV) a.scale[row * a.groups + v / 16] = scale;
            }
            float2 o[4];
            if (range) {
                const float2 f = make_float2(factor, factor);
#pragma unroll
                for (int q = 0; q < 4; ++q) o[q] = __fmul2_rn(p[k][q], f);
            } else {
                // one factor after the other: their product could overflow
                const float inv = __frcp_rn(scale);
                const float2 f1 = make_float2(rstd, rstd), f2 = make_float2(inv, inv);
#pragma unroll
                for (int q = 0; q < 4; ++q) o[q] = __fmul2_rn(__fmul2_rn(p[k][q], f1), f2);
            }
            uint2 bytes = make_uint2(quant4<INT8>(o[0], o[1]), quant4<INT8>(o[2], o[3]));
            if (!range && !finite_bits(scale)) bytes = make_uint2(0, 0);
            if (v < NV) __stcs(reinterpret_cast<uint2*>(a.q + row * H + v * kVec), bytes);
        }
    }
};

// A row per blockDim.x threads (a multiple of 32), loaded into registers;
// blockDim.y rows per CTA, more than one only where a row is one warp.
template <int VPT, int MAXT, bool RES, bool INT8, bool GROUPED>
__global__ void __launch_bounds__(MAXT)
norm_q8_rows(const Q8Args a) {
    __shared__ __align__(16) float red_sum[32];
    __shared__ __align__(16) uint32_t red_top[32];
    const int T = blockDim.x, t = threadIdx.x, NV = a.hidden / kVec;
    if (t < 32) red_sum[t] = red_top[t] = 0;
    __syncthreads();
    grid_dep_wait();
    grid_dep_release();
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows; row += step) {
        uint4 xv[VPT], rv[RES ? VPT : 1];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * T + t;
            xv[k] = make_uint4(0, 0, 0, 0);
            if constexpr (RES) rv[k] = xv[k];
            if (v < NV) {
                xv[k] = ld_stream(a.x + row * a.hidden + v * kVec);
                if constexpr (RES) rv[k] = ld_stream(a.res + row * a.hidden + v * kVec);
            }
        }
        Q8Row<VPT, RES, INT8, GROUPED, false, false> r;
        const uint4 none[1] = {};
        r.products(a, row, xv, rv, none, T, t);
        r.reduce_warp();
        if (T > 32) {
            r.leave(red_sum, red_top, t);
            __syncthreads();
            r.collect(red_sum, red_top, T >> 5);
        }
        r.finish(a, row, T, t);
        if (T > 32) __syncthreads();  // the reduction buffers are reused by the next row
    }
}

// Calls of many rows without the residual: one wave of CTAs that walk the rows blockIdx.x, +
// gridDim.x, ..., each row brought into a ring of `stages` rows in shared
// memory by bulk copies that thread 0 issues.  A row's loads, its reduction
// and its stores take turns in a CTA, and with a row per CTA too few bytes
// are in flight where only 3 bytes move per element; the ring keeps rows in
// flight whatever the CTA is doing (16384 x 5120: 45.8 -> 39.4 us, x 12288: 127
// -> 93 us; with the residual, 7 bytes per element, the row-per-CTA form runs
// at the copy rate: 16384 x 8192 133 us, the ring 148 us).  One barrier per row: behind it every
// thread has read the row's stage, which is then refilled, and the reduction
// buffers alternate.
template <int VPT, int MAXT, bool INT8, bool GROUPED>
__global__ void __launch_bounds__(MAXT, ring_threads(MAXT, GROUPED) / MAXT)
norm_q8_ring(const Q8Args a, int stages) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) float red_sum[2][32];
    __shared__ __align__(16) uint32_t red_top[2][32];
    __shared__ __align__(8) uint64_t full[kRingMaxStages];
    const int T = blockDim.x, t = threadIdx.x, NV = a.hidden / kVec;
    const uint32_t row_bytes = a.hidden * 2;
    if (t < 32) red_sum[0][t] = red_sum[1][t] = red_top[0][t] = red_top[1][t] = 0;
    if (t == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_release();
    const auto row_of = [&](int64_t i) { return blockIdx.x + i * gridDim.x; };
    const auto fetch = [&](int64_t i, int s) {  // the i-th row of this CTA into stage s, by thread 0
        const int64_t row = row_of(i);
        if (row >= a.rows) return;
        uint8_t* to = ring + static_cast<size_t>(s) * row_bytes;
        mbar_arrive_expect_tx(&full[s], row_bytes);
        bulk_copy(to, a.x + row * a.hidden, row_bytes, &full[s]);
    };
    if (t == 0)
        for (int s = 0; s < stages; ++s) fetch(s, s);
    // (at 384 threads with group scales, and above, the registers they take cost more)
    constexpr bool kKeepW = MAXT <= 256 || (MAXT == 384 && !GROUPED);
    uint4 wv[kKeepW ? VPT : 1];
    if constexpr (kKeepW) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            wv[k] = k * T + t < NV ? ld_param(a.w + (k * T + t) * kVec) : make_uint4(0, 0, 0, 0);
    }
    int stage = 0;
    uint32_t parity = 0;
    for (int64_t i = 0; row_of(i) < a.rows; ++i) {
        const int64_t row = row_of(i);
        const bool ok = mbar_wait(&full[stage], parity, kWaitLimitNs);
        const uint8_t* from = ring + static_cast<size_t>(stage) * row_bytes;
        uint4 xv[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int v = k * T + t;
            xv[k] = make_uint4(0, 0, 0, 0);
            if (v < NV && ok) xv[k] = *reinterpret_cast<const uint4*>(from + v * 16);
        }
        const uint4 none[1] = {};  // no residual
        Q8Row<VPT, false, INT8, GROUPED, true, kKeepW> r;
        if (ok) r.products(a, row, xv, none, wv, T, t);
        __syncwarp();
        r.reduce_warp();
        r.leave(red_sum[i & 1], red_top[i & 1], t);
        const bool failed = __syncthreads_or(!ok);
        r.collect(red_sum[i & 1], red_top[i & 1], T >> 5);
        if (failed) {  // a copy did not arrive: say so, give those in flight a last chance, and leave
            if (t == 0) {
                record_status(a.status, kStatusTimeout);
                for (int k = 0; k < stages && row_of(i + k) < a.rows; ++k)
                    mbar_wait(&full[(stage + k) % stages], stage + k < stages ? parity : parity ^ 1, kWaitLimitNs / 4);
            }
            return;
        }
        if (t == 0) fetch(i + stages, stage);
        if (++stage == stages) {
            stage = 0;
            parity ^= 1;
        }
        r.finish(a, row, T, t);
    }
}

template <int VPT, int MAXT, bool RES, bool INT8, bool GROUPED>
cudaError_t go(const Q8Args& a, int threads, int sms, cudaStream_t st) {
    if constexpr (VPT > 2 && !RES) {
        const int ctas = ring_threads(MAXT, GROUPED) / threads, stage_bytes = a.hidden * 2;
        const int64_t wave = static_cast<int64_t>(ctas) * sms;
        if (threads >= kRingMinThreads && a.rows >= 2 * wave) {  // every resident CTA has several rows
            const auto kernel = norm_q8_ring<VPT, MAXT, INT8, GROUPED>;
            static std::atomic<bool> set[64];
            int dev = 0;
            if (cudaError_t e = cudaGetDevice(&dev)) return e;
            if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
            if (!set[dev].load(std::memory_order_acquire)) {
                if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes))
                    return e;
                set[dev].store(true, std::memory_order_release);
            }
            const int fit = kRingBytes / ctas / stage_bytes, stages = fit < kRingMaxStages ? fit : kRingMaxStages;
            return launch_with_pdl(kernel, dim3(static_cast<unsigned>(wave)), dim3(threads),
                                   static_cast<size_t>(stages) * stage_bytes, st, a, stages);
        }
    }
    const int rpc = VPT > 2 && threads == 32 ? 4 : 1;
    const int64_t blocks = (a.rows + rpc - 1) / rpc;
    const unsigned grid = static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF);
    return launch_with_pdl(norm_q8_rows<VPT, MAXT, RES, INT8, GROUPED>, dim3(grid), dim3(threads, rpc), 0, st, a);
}

template <int VPT, int MAXT>
cudaError_t go(const Q8Args& a, bool int8, bool grouped, int threads, int sms, cudaStream_t st) {
    const int pick = (a.res ? 4 : 0) | (int8 ? 2 : 0) | (grouped ? 1 : 0);
    switch (pick) {
        case 0: return go<VPT, MAXT, false, false, false>(a, threads, sms, st);
        case 1: return go<VPT, MAXT, false, false, true>(a, threads, sms, st);
        case 2: return go<VPT, MAXT, false, true, false>(a, threads, sms, st);
        case 3: return go<VPT, MAXT, false, true, true>(a, threads, sms, st);
        case 4: return go<VPT, MAXT, true, false, false>(a, threads, sms, st);
        case 5: return go<VPT, MAXT, true, false, true>(a, threads, sms, st);
        case 6: return go<VPT, MAXT, true, true, false>(a, threads, sms, st);
        default: return go<VPT, MAXT, true, true, true>(a, threads, sms, st);
    }
}

}  // namespace

cudaError_t launch_norm_q8(const Q8Args& a, bool int8, bool grouped, int sms, cudaStream_t st) {
    const int nv = a.hidden / kVec;
    const auto threads = [nv](int vpt) { return ((nv + vpt - 1) / vpt + 31) / 32 * 32; };
    if (a.rows <= 256 && threads(2) <= 1024) return go<2, 1024>(a, int8, grouped, threads(2), sms, st);
    const int t = threads(4);
    if (t > 384) return go<4, 1024>(a, int8, grouped, t, sms, st);
    if (t > 256) return go<4, 384>(a, int8, grouped, t, sms, st);
    if (t > 192) return go<4, 256>(a, int8, grouped, t, sms, st);
    return go<4, 192>(a, int8, grouped, t, sms, st);
}

}  // namespace nf
