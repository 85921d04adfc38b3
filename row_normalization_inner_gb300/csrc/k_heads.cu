// Attention heads: rotation by position, RMSNorm of each head, and the append
// of keys and values to a paged cache, in one pass over the heads of a token.
//
//   n = x * rsqrt(mean(x^2) + eps) * w       (a segment with a weight; else n = x)
//   y = the pairs of n turned by the token's angles, the rest of n
//   out = y rounded once, in the heads' type; or, for an 8-bit cache,
//   scale = max(max|y| / Q, 2^-100), q = y / scale rounded to nearest
//
// Bound by memory: each element is read once and written once.  A warp takes a
// token and up to `passes` times 32 / G of its heads (heads.cuh), so that the
// token's angles -- two sines and cosines a lane at 64 pairs -- are computed
// once for all of them and wait in shared memory; a group of G lanes holds a
// row, and the row's sums stay in the warp.
#include <algorithm>

#include "heads.cuh"

namespace nf {
namespace {

constexpr int kWarps = 4;  // per CTA
constexpr float kScaleMin = 0x1p-100f;

__device__ __forceinline__ bool finite_bits(uint32_t b) { return (b & 0x7F800000u) != 0x7F800000u; }

// The scale of a row whose largest |y| has the bits `top`; NaN where that is not finite.
__device__ __forceinline__ float row_scale(uint32_t top, bool int8) {
    return finite_bits(top) ? fmaxf(__fdiv_rn(__uint_as_float(top), int8 ? 127.f : 448.f), kScaleMin) : __uint_as_float(0x7FC00000u);
}

// y / scale in fp32, rounded once, without a division for each element: the
// product with 1 / scale, corrected by its own remainder (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990).  Rows of 16-bit values often have quotients that lie exactly between
// two 8-bit values; a product alone would miss these.  An infinite or NaN
// `inverse` never gets here: such rows are stored as zeros.
__device__ __forceinline__ float quotient(float y, float scale, float inverse) {
    const float q = y * inverse;
    return fmaf(fmaf(-q, scale, y), inverse, q);
}

__device__ __forceinline__ uint32_t quant2(float y0, float y1, float scale, float inverse, bool fine, bool int8) {
    const float a = fine ? quotient(y0, scale, inverse) : 0.f, b = fine ? quotient(y1, scale, inverse) : 0.f;
    if (int8) return (static_cast<uint32_t>(__float2int_rn(a)) & 0xFF) | ((static_cast<uint32_t>(__float2int_rn(b)) & 0xFF) << 8);
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(b), "f"(a));
    return v;
}

template <int W>
__device__ __forceinline__ void store_quantized(uint8_t* p, const float2 (&y)[W / 2], float scale, float inverse, bool fine, bool int8) {
    uint32_t q[W / 4];
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
        q[i] = quant2(y[2 * i].x, y[2 * i].y, scale, inverse, fine, int8) |
               (quant2(y[2 * i + 1].x, y[2 * i + 1].y, scale, inverse, fine, int8) << 16);
    if constexpr (W == 8) *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(p) = q[0];
}

__device__ __forceinline__ uint32_t top_of(uint32_t top, float2 v) {
    return max(top, max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))));
}

// Where a token of an append stands.
struct Place {
    bool used;      // the token belongs to a sequence
    bool stored;    // and has a page
    int64_t position, page;
    int slot;
};

// The place of a token of sequence `seq`, which begins at token `first` and has
// `past` tokens before it (negative: the token is padding).
__device__ __forceinline__ Place place_in(const HeadsArgs& a, uint32_t token, int seq, int first, int past) {
    Place p{};
    p.used = past >= 0;
    if (!p.used) return p;
    p.position = static_cast<int64_t>(past) + (static_cast<int64_t>(token) - first);
    const uint32_t place = static_cast<uint32_t>(p.position);  // below 2^32: both terms are below 2^31
    const uint32_t column = place / static_cast<uint32_t>(a.page_size);
    p.slot = static_cast<int>(place - column * static_cast<uint32_t>(a.page_size));
    if (column < static_cast<uint32_t>(a.max_pages)) {
        p.page = a.table[seq * a.table_stride + column];
        p.stored = p.page >= 0 && p.page < a.pages;
    }
    return p;
}

// All lanes of a warp call this.  The sequence of a token is the last one that
// starts at or before it; the starts are searched 32 ways at a time, and the
// last 32 candidates' lengths come with them, so that the step costs one load's
// latency for each factor of 32 of the sequences and one for the page.
__device__ __forceinline__ Place find_place(const HeadsArgs& a, uint32_t token, int lane) {
    bool used;
    int seq, first, past;
    if (a.starts) {
        const int behind = a.starts[a.seqs];
        int lo = 0, n = a.seqs;  // the answer is in [lo, lo + n)
        for (;;) {
            const int step = (n + 31) / 32;
            const bool in = lane * step < n;
            const int at = lo + lane * step;
            const int start = in ? a.starts[at] : 0;
            const int held = in && step == 1 ? a.past[at] : 0;
            const uint32_t votes = __ballot_sync(0xFFFFFFFFu, in && start <= static_cast<int64_t>(token)) | 1u;
            const int k = 31 - __clz(votes);
            lo += k * step;
            n = min(step, n - k * step);
            first = __shfl_sync(0xFFFFFFFFu, start, k);
            past = __shfl_sync(0xFFFFFFFFu, held, k);
            if (step == 1) break;
        }
        seq = lo;
        used = first >= 0 && first <= static_cast<int64_t>(token) && static_cast<int64_t>(token) < behind;
    } else {
        seq = first = static_cast<int>(token);
        used = seq < a.seqs;
        past = used ? a.past[seq] : 0;
    }
    return place_in(a, token, seq, first, used ? past : -1);
}

// The row of head `h`: input, output and its scale.
template <typename T>
__device__ __forceinline__ const T* row_in(const HeadSegment& s, uint32_t batch, uint32_t at, int h) {
    return static_cast<const T*>(s.in) + batch * s.in_batch + at * s.in_token + h * s.in_head;
}

constexpr int kPasses = 4;     // most rows of a group in a share: so many are in flight
constexpr int kMaxWarps = 5;  // per CTA

// A CTA takes `per_cta` tokens, its warps their shares: so many rows of queries,
// keys or values.  The angles of a token are computed once, by all the warps
// that need them, while the rows are on their way.
template <typename T, bool INTER, bool APPEND, int GT>
__global__ void __launch_bounds__(kMaxWarps * 32, 4) heads_rows(const __grid_constant__ HeadsArgs a, int lanes) {
    constexpr int W = Elem<T>::W, P = W / 2;
    const int G = GT ? GT : lanes;
    extern __shared__ float4 tables[];  // [per_cta][2][pairs]
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x >> 5) / a.per_cta;
    const int nth = warp / warps, share = warp - nth * warps;  // the warp's token in the CTA
    const uint32_t group = a.turns == 1 ? blockIdx.x : blockIdx.x / a.turns;
    const uint32_t token = group * a.per_cta + nth;
    const int rows = 32 / G, j = lane & (G - 1), lane_row = lane / G;
    const uint32_t batch = APPEND ? 0 : token / a.tokens, at = token - batch * a.tokens;
    // the warp's share: queries, keys or values, and which rows of them
    int chunk = static_cast<int>(blockIdx.x - group * a.turns) * warps + share, si = 0;
    const bool real = token < a.total && chunk < a.chunks;
    if (!real) chunk = 0;
    while (chunk >= a.seg[si].chunks) chunk -= a.seg[si++].chunks;
    const HeadSegment& s = a.seg[si];
    const int pairs = s.rotate ? a.rope.pairs : 0;
    const LaneVectors<W, INTER> v(j, a.dim, pairs);
    const int head = chunk * a.passes * rows + lane_row;
    const int passes = min(a.passes, (s.heads - chunk * a.passes * rows + rows - 1) / rows);
    uint4 xa[kPasses], xb[kPasses];
    const T* in = row_in<T>(s, batch, at, head);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        xa[p] = xb[p] = make_uint4(0, 0, 0, 0);
        if (real && p < passes && head + p * rows < s.heads) {
            const T* row = in + p * rows * s.in_head;
            if (v.has_a) xa[p] = ld_stream(row + v.a);
            if (v.has_b) xb[p] = ld_stream(row + v.b);
        }
    }
    Place place{};
    if (APPEND && token < a.total) place = find_place(a, token, lane);
    float* table = reinterpret_cast<float*>(tables) + nth * 2 * a.rope.pairs;
    if (a.rope.pairs) {
        if (token < a.total) {
            const int64_t position = APPEND && !a.rope.positions ? place.position : position_at(a.rope, batch, at);
            fill_turns(table, a.rope, a.rope.pairs, position, a.rope.direction, share * 32 + lane, warps * 32);
        }
        __syncthreads();
    }
    if (!real || (APPEND && (!place.used || (s.cache && !place.stored)))) return;
    LaneTurns<W, INTER> t;
    if (pairs) t.read(table, pairs, v);
    const bool norm = s.weight != nullptr;
    uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
    if (norm) {
        if (v.has_a) wa = ld_param(static_cast<const T*>(s.weight) + v.a);
        if (v.has_b) wb = ld_param(static_cast<const T*>(s.weight) + v.b);
    }
    const float mean_of = 1.f / a.dim;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        if (p >= passes) break;
        const bool here = head + p * rows < s.heads;
        float2 fa[P], fb[P];
        Elem<T>::unpack(xa[p], fa);
        Elem<T>::unpack(xb[p], fb);
        if (norm) {
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                ss = __ffma2_rn(fa[i], fa[i], ss);
                ss = __ffma2_rn(fb[i], fb[i], ss);
            }
            const float r = rsqrtf(sum_lanes(ss.x + ss.y, G) * mean_of + a.eps);
            const float2 rstd = make_float2(r, r);
            float2 ga[P], gb[P];
            Elem<T>::unpack(wa, ga);
            Elem<T>::unpack(wb, gb);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                fa[i] = __fmul2_rn(__fmul2_rn(fa[i], rstd), ga[i]);
                fb[i] = __fmul2_rn(__fmul2_rn(fb[i], rstd), gb[i]);
            }
        }
        if (pairs) t.turn(fa, fb, v);
        if (APPEND && s.cache) {
            const int64_t row = place.page * s.out_batch + place.slot * s.out_token + (head + p * rows) * s.out_head;
            if (a.format != kCacheSame) {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < P; ++i) top = top_of(top_of(top, fa[i]), fb[i]);
#pragma unroll
                for (int off = G >> 1; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
                const bool int8 = a.format == kCacheInt8, fine = finite_bits(top);
                const float scale = row_scale(top, int8), inverse = __fdiv_rn(1.f, scale);
                uint8_t* out = static_cast<uint8_t*>(s.out) + row;
                if (here && v.has_a) store_quantized<W>(out + v.a, fa, scale, inverse, fine, int8);
                if (here && v.has_b) store_quantized<W>(out + v.b, fb, scale, inverse, fine, int8);
                if (here && j == 0) s.scale[place.page * s.scale_page + place.slot * s.scale_slot + (head + p * rows) * s.scale_head] = scale;
            } else {
                T* out = static_cast<T*>(s.out) + row;
                if (here && v.has_a) *reinterpret_cast<uint4*>(out + v.a) = norm || pairs ? Elem<T>::pack(fa) : xa[p];
                if (here && v.has_b) *reinterpret_cast<uint4*>(out + v.b) = norm || pairs ? Elem<T>::pack(fb) : xb[p];
            }
        } else {
            T* out = static_cast<T*>(s.out) + batch * s.out_batch + at * s.out_token + (head + p * rows) * s.out_head;
            if (here && v.has_a) st_stream(out + v.a, Elem<T>::pack(fa));
            if (here && v.has_b) st_stream(out + v.b, Elem<T>::pack(fb));
        }
    }
}

// Any head size, stride and alignment: a warp holds one row in shared memory,
// element by element, and computes its angles itself.  For rows whose vectors
// do not fall on 16 bytes, or whose rotated halves are no whole vectors.
template <typename T, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32) heads_elements(const __grid_constant__ HeadsArgs a) {
    extern __shared__ float staged[];
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31;
    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const uint32_t token = unit / a.chunks;
    if (token >= a.total) return;
    int head = static_cast<int>(unit - token * a.chunks), si = 0;
    while (head >= a.seg[si].heads) head -= a.seg[si++].heads;
    const HeadSegment& s = a.seg[si];
    const uint32_t batch = token / a.tokens, at = token - batch * a.tokens;
    Place place{};
    if constexpr (APPEND) {
        place = find_place(a, token, lane);
        if (!place.used || (s.cache && !place.stored)) return;
    }
    const int dim = a.dim, pairs = s.rotate ? a.rope.pairs : 0;
    float* row = staged + (threadIdx.x >> 5) * dim;
    const T* in = row_in<T>(s, batch, at, head);
    float ss = 0.f;
    for (int i = lane; i < dim; i += 32) {
        const float x = Elem<T>::load(in + i);
        row[i] = x;
        ss += x * x;
    }
    if (s.weight) {
        const float rstd = rsqrtf(sum_lanes(ss, 32) * (1.f / dim) + a.eps);
        for (int i = lane; i < dim; i += 32) row[i] *= rstd * Elem<T>::load(static_cast<const T*>(s.weight) + i);
    }
    __syncwarp();
    if (pairs) {
        const int64_t position = APPEND && !a.rope.positions ? place.position : position_at(a.rope, batch, at);
        for (int p = lane; p < pairs; p += 32) {
            const float2 t = turn_of(a.rope.rates[p], position, a.rope.magnitude, a.rope.direction);
            const int ia = a.rope.interleaved ? 2 * p : p, ib = a.rope.interleaved ? 2 * p + 1 : p + pairs;
            const float x = row[ia], y = row[ib];
            row[ia] = x * t.x - y * t.y;
            row[ib] = y * t.x + x * t.y;
        }
        __syncwarp();
    }
    if (APPEND && s.cache) {
        const int64_t first = place.page * s.out_batch + place.slot * s.out_token + head * s.out_head;
        if (a.format != kCacheSame) {
            uint32_t top = 0;
            for (int i = lane; i < dim; i += 32) top = max(top, __float_as_uint(fabsf(row[i])));
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            const bool int8 = a.format == kCacheInt8, fine = finite_bits(top);
            const float scale = row_scale(top, int8), inverse = __fdiv_rn(1.f, scale);
            uint8_t* out = static_cast<uint8_t*>(s.out) + first;
            for (int i = lane; i < dim; i += 32) out[i] = static_cast<uint8_t>(quant2(row[i], 0.f, scale, inverse, fine, int8));
            if (lane == 0) s.scale[place.page * s.scale_page + place.slot * s.scale_slot + head * s.scale_head] = scale;
        } else {
            T* out = static_cast<T*>(s.out) + first;
            for (int i = lane; i < dim; i += 32) {
                if (s.weight || pairs) Elem<T>::store(out + i, row[i]);
                else out[i] = in[i];
            }
        }
    } else {
        T* out = static_cast<T*>(s.out) + batch * s.out_batch + at * s.out_token + head * s.out_head;
        for (int i = lane; i < dim; i += 32) Elem<T>::store(out + i, row[i]);
    }
}

bool fits(const void* p, int64_t s0, int64_t s1, int64_t s2, int elements, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && s0 % elements == 0 && s1 % elements == 0 && s2 % elements == 0;
}

// Whether every row falls on whole 16-byte vectors (8-bit rows: on W bytes).
bool whole_vectors(const HeadsArgs& a, int W) {
    if (a.dim % W || (a.dim / W + 1) / 2 > 32 || (!a.rope.interleaved && a.rope.pairs % W)) return false;
    for (int i = 0; i < a.segments; ++i) {
        const HeadSegment& s = a.seg[i];
        if (!fits(s.in, s.in_batch, s.in_token, s.in_head, W, 16)) return false;
        if (!fits(s.out, s.out_batch, s.out_token, s.out_head, W, s.cache && a.format != kCacheSame ? W : 16)) return false;
        if (reinterpret_cast<uintptr_t>(s.weight) % 16) return false;
    }
    return true;
}

template <typename T, bool INTER, bool APPEND>
cudaError_t launch_lanes(const HeadsArgs& a, int G, dim3 grid, dim3 block, size_t smem, cudaStream_t st) {
    switch (G) {  // the common heads: 128 elements, 256 (bf16) and 64 (fp32)
        case 8: return launch_with_pdl(heads_rows<T, INTER, APPEND, 8>, grid, block, smem, st, a, G);
        case 16: return launch_with_pdl(heads_rows<T, INTER, APPEND, 16>, grid, block, smem, st, a, G);
        default: return launch_with_pdl(heads_rows<T, INTER, APPEND, 0>, grid, block, smem, st, a, G);
    }
}

template <typename T, bool APPEND>
cudaError_t launch(HeadsArgs a, int sms, cudaStream_t st) {
    constexpr int W = Elem<T>::W;
    if (!whole_vectors(a, W)) {
        a.chunks = 0;
        for (int i = 0; i < a.segments; ++i) a.chunks += a.seg[i].heads;
        const int64_t units = static_cast<int64_t>(a.total) * a.chunks;
        return launch_with_pdl(heads_elements<T, APPEND>, dim3(static_cast<unsigned>((units + kWarps - 1) / kWarps)), dim3(kWarps * 32),
                               kWarps * a.dim * sizeof(float), st, a);
    }
    const int G = lanes_for((a.dim / W + 1) / 2), rows = 32 / G;
    // As many rows to a share as leave every SM its warps: each pass more
    // spreads what a warp does before its rows over more of them.
    for (a.passes = kPasses;; a.passes /= 2) {
        a.chunks = 0;
        for (int i = 0; i < a.segments; ++i) {
            a.seg[i].chunks = (a.seg[i].heads + rows * a.passes - 1) / (rows * a.passes);
            a.chunks += a.seg[i].chunks;
        }
        if (a.passes == 1 || static_cast<int64_t>(a.total) * a.chunks >= 64 * sms) break;
    }
    // a warp to each share, in several CTAs where a token has many; tokens of few shares side by side in a CTA of four warps or more
    a.turns = (a.chunks + kMaxWarps - 1) / kMaxWarps;
    const int warps = (a.chunks + a.turns - 1) / a.turns;
    a.per_cta = warps >= 4 ? 1 : 4 / warps;
    const dim3 grid((a.total + a.per_cta - 1) / a.per_cta * a.turns), block(warps * a.per_cta * 32);
    const size_t smem = a.per_cta * a.rope.pairs * sizeof(float2);
    return a.rope.interleaved ? launch_lanes<T, true, APPEND>(a, G, grid, block, smem, st) : launch_lanes<T, false, APPEND>(a, G, grid, block, smem, st);
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs& a, bool f32, bool append, int sms, cudaStream_t st) {
    if (f32) return append ? launch<float, true>(a, sms, st) : launch<float, false>(a, sms, st);
    return append ? launch<uint16_t, true>(a, sms, st) : launch<uint16_t, false>(a, sms, st);
}

}  // namespace nf
