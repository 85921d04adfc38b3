// Attention heads: rotation by position, RMSNorm of each head, and the append
// of keys and values to a paged cache, in one pass over the heads of a token.
//
//   n = x * rsqrt(mean(x^2) + eps) * w       (a segment with a weight; else n = x)
//   y = the pairs of n turned by the token's angles, the rest of n
//   out = y rounded once, in the heads' type; or, for an 8-bit cache,
//   scale = max(max|y| / Q, 2^-100), q = y / scale rounded to nearest
//
// Bound by memory: each element is read once and written once (16384 tokens of
// 64 + 8 heads of 128 in bf16: turned 89.0 us, 6.8 TB/s, a copy's rate; normalized
// too 96.5 us, 6.3 TB/s).  A group of lanes holds a row (heads.cuh), so that its
// sums stay in the warp; a warp has four rows of every group in flight.  What it
// does before them -- its share, addresses, angles, weights -- is a good half of
// its instructions and the reason for most of what follows: the angles are
// computed once for a token's warps, the weights are folded into them, and few
// heads share a warp with other tokens' (16384 tokens of 8 + 2 heads: 16 us, 25
// with a warp to each).
#pragma once

#include <algorithm>

#include "heads.cuh"

namespace nf {
namespace {

constexpr int kWarps = 4;  // per CTA
constexpr float kScaleMin = 0x1p-100f;

__device__ __forceinline__ bool finite_bits(uint32_t b) { return (b & 0x7F800000u) != 0x7F800000u; }

// y / d rounded to fp32 once, given about 1 / d: the product with it, corrected
// by its own remainder (P. Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990).  Rows of 16-bit values often have
// quotients that lie exactly between two 8-bit values; a product alone would
// miss these.
__device__ __forceinline__ float quotient(float y, float d, float inverse) {
    const float q = y * inverse;
    return fmaf(fmaf(-q, d, y), inverse, q);
}
__device__ __forceinline__ float about_inverse(float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}

// The scale of a row whose largest |y| has the bits `top`; NaN where that is not finite.
__device__ __forceinline__ float row_scale(bool int8, uint32_t top) {
    const float most = int8 ? 127.f : 448.f, inverse = int8 ? 1.f / 127.f : 1.f / 448.f;
    return finite_bits(top) ? fmaxf(quotient(__uint_as_float(top), most, inverse), kScaleMin) : __uint_as_float(0x7FC00000u);
}

// Two elements in 8 bits, in the lower half of the result's 16 bits each's byte.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(b), "f"(a));
    return v;
}
// |y| <= 127 to the nearest integer, ties to even, in the lower 8 bits of the
// result: where fp32 numbers are one apart, the sum's own rounding is that.
__device__ __forceinline__ uint32_t int8_bits(float y) { return __float_as_uint(y + 0x1.8p23f); }
__device__ __forceinline__ uint32_t int8_pair(float a, float b) { return __byte_perm(int8_bits(a), int8_bits(b), 0x0040); }

// W elements (divided by the row's scale) in 8 bits; `keep`: all bits, or none.
template <bool INT8, int W>
__device__ __forceinline__ void store_8(uint8_t* p, const float (&v)[W], uint32_t keep) {
    uint32_t q[W / 4];
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
        const float *f = v + 4 * i;
        const uint32_t lower = INT8 ? int8_pair(f[0], f[1]) : e4m3_pair(f[0], f[1]), upper = INT8 ? int8_pair(f[2], f[3]) : e4m3_pair(f[2], f[3]);
        q[i] = __byte_perm(lower, upper, 0x5410) & keep;
    }
    if constexpr (W == 8) *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(p) = q[0];
}

// The largest magnitude of three, a NaN standing above every number.
__device__ __forceinline__ float largest(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A row in 8 bits, and its scale; with a NaN or an infinity its elements are zeros.
// All lanes of its group call this.
template <bool INTER, int GT, int P>
__device__ __forceinline__ void store_row_8(bool int8, uint8_t* to, float* scale_to, float2 (&x)[P], float2 (&y)[P], int G, int lane, bool here,
                                            bool first_lane, const LaneVectors<2 * P, INTER, GT != 0>& v) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) m = largest(largest(m, x[i].x, x[i].y), y[i].x, y[i].y);
    uint32_t top = __float_as_uint(m) & 0x7FFFFFFFu;  // as integers: a NaN stands above every number here too
    top = max_lanes<GT>(top, G, lane);
    const float scale = row_scale(int8, top), by = about_inverse(scale);
    const float2 d = make_float2(-scale, -scale), inverse = make_float2(by, by);
#pragma unroll
    for (int i = 0; i < P; ++i) {  // quotient(), two at a time
        const float2 qx = __fmul2_rn(x[i], inverse), qy = __fmul2_rn(y[i], inverse);
        x[i] = __ffma2_rn(__ffma2_rn(qx, d, x[i]), inverse, qx);
        y[i] = __ffma2_rn(__ffma2_rn(qy, d, y[i]), inverse, qy);
    }
    float a[2 * P], b[2 * P];
    in_order<2 * P, INTER>(x, y, a, b);
    const uint32_t keep = finite_bits(top) ? 0xFFFFFFFFu : 0u;
    if (int8) {
        if (here && v.has_a()) store_8<true>(to + v.a, a, keep);
        if (here && v.has_b()) store_8<true>(to + v.b, b, keep);
    } else {
        if (here && v.has_a()) store_8<false>(to + v.a, a, keep);
        if (here && v.has_b()) store_8<false>(to + v.b, b, keep);
    }
    if (here && first_lane) *scale_to = scale;
}

// Where a token of an append stands.
struct Place {
    int64_t position;  // in its sequence
    int64_t entry;     // of the table, for its page; -1: it has none
    int slot;          // -1: the token belongs to no sequence
};

// The place of a token of sequence `seq`, which begins at token `first` and has
// `past` tokens before it (negative: the token is padding).
__device__ __forceinline__ Place place_in(const HeadsArgs& a, int token, int seq, int first, int past) {
    Place p{0, -1, -1};
    if (past < 0) return p;
    const uint32_t place = static_cast<uint32_t>(past) + static_cast<uint32_t>(token - first);  // both below 2^31
    const uint32_t column = divide(place, a.by_page);
    p.position = place;
    p.slot = static_cast<int>(place - column * static_cast<uint32_t>(a.page_size));
    if (column < static_cast<uint32_t>(a.max_pages)) p.entry = seq * a.table_stride + column;
    return p;
}

// Its page, or -1 where the cache has none for it.  Only those ask that store there.
__device__ __forceinline__ int page_of(const HeadsArgs& a, const Place& p) {
    if (p.entry < 0) return -1;
    const int page = a.table[p.entry];
    return static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages) ? page : -1;
}

// All lanes of a warp call this.  The sequence of a token is the last one that
// starts at or before it; the starts are searched 32 ways at a time, and the
// last 32 candidates' lengths come with them, so that the step costs one load's
// latency for each factor of 32 of the sequences.
__device__ __forceinline__ Place find_place(const HeadsArgs& a, int token, int lane) {
    if (!a.starts) return place_in(a, token, token, token, token < a.seqs ? a.past[token] : -1);
    const int behind = a.starts[a.seqs];
    int lo = 0, n = a.seqs, first, past;  // the answer is in [lo, lo + n)
    for (;;) {
        const int step = (n + 31) / 32;
        const bool in = lane * step < n;
        const int at = lo + lane * step;
        const int start = in ? a.starts[at] : 0;
        const int held = in && step == 1 ? a.past[at] : 0;
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, in && start <= token) | 1u;
        const int k = 31 - __clz(votes);
        lo += k * step;
        n = min(step, n - k * step);
        first = __shfl_sync(0xFFFFFFFFu, start, k);
        past = __shfl_sync(0xFFFFFFFFu, held, k);
        if (step == 1) break;
    }
    return place_in(a, token, lo, first, first >= 0 && first <= token && token < behind ? past : -1);
}

// What a kernel is compiled for: the code that stores rows in 8 bits takes
// registers that other calls' rows want (an append of 8192 tokens of 32 + 8 + 8
// heads to a bf16 cache 34.0 us, with both in one kernel 34.7).
constexpr int kNoCache = 0, kCacheOfType = 1, kCache8Bits = 2;

// Warps of a CTA at most, and CTAs that the registers of an SM hold (80 a thread,
// some spilled).  With 3, 5 (of 96 registers) and 9 warps 16384 tokens of 64 + 8
// heads take 97, 95 and 95 us, of 32 + 8 heads 50, 52 and 52 turned and 54, 57 and
// 57 normalized too.  An append to an 8-bit cache (8192 tokens of 64 + 8 + 8) takes
// 59 us, with six CTAs of more registers 62.
constexpr int kMaxWarps = 3;
constexpr int kMinCtas = 7;
// Rows in 8 bits take twice the instructions: a share has half as many of them,
// so that its warp is not the one that the others' CTA waits for.
constexpr int rows_8(int rows) { return rows > 1 ? rows / 2 : 1; }
// Shares of four rows per SM from which these are taken rather than single rows
// (us, four rows / one): 256 tokens of 32 + 8 heads, five to an SM, turned 2.4 /
// 2.7, normalized too 3.0 / 3.1, 1024 tokens 4.3 / 6.0 and 5.0 / 6.8; appended with
// 8 + 8 heads, 320 tokens, six to an SM, 3.6 / 3.5, to an 8-bit cache 4.4 / 3.6,
// 384 tokens 3.7 / 4.4 and 4.5 / 4.9.
constexpr int64_t many_shares(bool append) { return append ? 7 : 4; }

// 1 over a row's root mean square.
template <typename T, bool INTER, int GT>
__device__ __forceinline__ float rstd_of(uint4 a, uint4 b, int G, int lane, float mean_of, float eps) {
    constexpr int P = Elem<T, INTER>::W / 2;
    float2 x[P], y[P];
    Elem<T, false>::unpack(a, b, x, y);
    float2 ss = __fmul2_rn(x[0], x[0]);
    ss = __ffma2_rn(y[0], y[0], ss);
#pragma unroll
    for (int i = 1; i < P; ++i) ss = __ffma2_rn(y[i], y[i], __ffma2_rn(x[i], x[i], ss));
    return rsqrtf(sum_lanes<GT>(ss.x + ss.y, G, lane) * mean_of + eps);
}

// A row of a lane's group: over its root mean square, weighted and turned.
template <typename T, bool INTER, bool FULL, bool NORM, int P>
__device__ __forceinline__ void turn_row(uint4 a, uint4 b, float rstd, const LaneFactors<2 * P, INTER, FULL>& f, float2 (&x)[P], float2 (&y)[P]) {
    Elem<T, INTER>::unpack(a, b, x, y);
    if constexpr (NORM) {
        const float2 r = make_float2(rstd, rstd);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = __fmul2_rn(x[i], r), y[i] = __fmul2_rn(y[i], r);
    }
    f.apply(x, y);
}

// N such rows, rounded to vectors again.  Without a branch between them, so that
// one is waited for under another's arithmetic.
template <typename T, bool INTER, int GT, bool NORM, int N, int M>
__device__ __forceinline__ void turn_rows(uint4 (&a)[M], uint4 (&b)[M], const float (&rstd)[M], const LaneFactors<Elem<T, INTER>::W, INTER, GT != 0>& f,
                                          int G, int lane, float mean_of, float eps) {
    constexpr int P = Elem<T, INTER>::W / 2;
#pragma unroll
    for (int p = 0; p < N; ++p) {
        float2 x[P], y[P];
        const float r = NORM && M > 1 ? rstd_of<T, INTER, GT>(a[p], b[p], G, lane, mean_of, eps) : rstd[p];
        turn_row<T, INTER, GT != 0, NORM, P>(a[p], b[p], r, f, x, y);
        Elem<T, INTER>::pack(x, y, a[p], b[p]);
    }
}

constexpr int kMaxTokens = 8;  // of a CTA
// One token, with keys and values in one share or not; several; several with
// both in one share (the code for that took 8% where it was not used).
constexpr int kOneToken = 0, kSeveralTokens = 1, kSeveralJoined = 2;

// A CTA takes `per_cta` tokens (several CTAs take turns where there is more to
// do), its warps their shares: N rows for each group of lanes, of queries, keys
// or values.  A share is part of a token, pass after pass of 32 / G heads; or,
// where a token has fewer heads, several tokens, each on as many groups as it
// needs, so that a few heads fill a warp too.  An append's share of two passes of
// keys takes the values' two as well.  The angles are computed once for
// all the warps that need them, while the rows are on their way.
// GT: lanes of a group, each with both its vectors; 0: a power of two that the
// host gives, some lanes without one or both.
// TOKENS: what a CTA has.
template <typename T, bool INTER, int CACHE, int GT, int N, int TOKENS>
__global__ void __launch_bounds__(kMaxWarps * 32, kMinCtas) heads_rows(const __grid_constant__ HeadsArgs a, int lanes) {
    constexpr int W = Elem<T, INTER>::W, P = W / 2;
    constexpr bool FULL = GT != 0, APPEND = CACHE != kNoCache, SEVERAL = TOKENS != kOneToken;
    const int G = FULL ? GT : lanes;
    extern __shared__ float4 tables[];  // [per_cta][2][pairs]
    __shared__ Place places[APPEND ? SEVERAL ? kMaxTokens : 1 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint32_t cta_of_tokens = divide(blockIdx.x, a.by_turns), first_token = SEVERAL ? cta_of_tokens * a.per_cta : cta_of_tokens;
    const int tokens = SEVERAL ? min(a.per_cta, static_cast<int>(a.total - first_token)) : 1;
    const int rows = 32 / G, group = lane / G, j = lane - group * G;
    // the warp's share: queries, keys or values, which tokens and which rows of them
    int share = static_cast<int>(blockIdx.x - cta_of_tokens * a.turns) * warps + warp, si = 0;
    bool real = share < a.shares;
    if (!real) share = 0;
    while (share >= a.seg[si].shares) share -= a.seg[si++].shares;
    const HeadSegment& s = a.seg[si];
    constexpr int H = APPEND && N > 1 && TOKENS != kSeveralTokens ? N / 2 : N;  // rows of a half
    const bool both = H < N && s.with_next;                                     // keys in the first half, values in the second
    constexpr int M = CACHE == kCache8Bits ? rows_8(N) : N;     // rows of a share that goes to the cache
    const int most = both ? H : s.cache ? M : N;
    const HeadSegment& s2 = a.seg[H < N ? si + both : si];
    // The lane's token in the CTA and its first head, how far its next head is, and
    // how many heads the share has for a group at most.  Lanes without a row of
    // their own (behind the last whole group, or the last token) are not `mine`:
    // they load along with the share's first, and store nothing.
    int nth = 0, head, step = rows, passes;
    bool mine, whole;  // whole: every group has N rows
    if (!SEVERAL || s.per_token) {
        if (SEVERAL) nth = share / s.per_token;
        const int first = (share - (SEVERAL ? nth * s.per_token : 0)) * most * rows;
        if (SEVERAL) real = real && nth < tokens;
        mine = (FULL && 32 % (GT ? GT : 1) == 0) || group < rows;
        head = first + (mine ? group : 0);
        passes = min(most, (s.heads - first + rows - 1) / rows);
        whole = real && first + most * rows <= s.heads;
    } else {
        const int in_share = (group * s.groups_factor) >> 10, first = share * s.tokens_of_share;  // group / groups_of_token
        nth = first + in_share;
        real = real && first < tokens;
        mine = in_share < s.tokens_of_share && nth < tokens;
        if (!mine) nth = first;
        step = s.groups_of_token;
        head = mine ? group - in_share * step : 0;
        passes = (s.heads + step - 1) / step;
        whole = real && s.heads == most * step;
    }
    if (SEVERAL && !real) nth = 0;
    const uint32_t token = first_token + nth;
    const uint32_t batch = APPEND ? 0 : divide(token, a.by_tokens), at = token - batch * a.tokens;
    const int pairs = s.rotate ? a.rope.pairs : 0;
    const LaneVectors<W, INTER, FULL> v(j, FULL ? 2 * W * GT : a.dim, pairs);
    // Nothing before this touches memory: it runs under the kernel ahead (a decode
    // step's rotation 1.49 us, with the wait first 1.74).
    grid_dep_wait();
    grid_dep_release();
    // what the angles need; for a single row it is asked for first, as it is waited for first
    const int thread = threadIdx.x, threads = warps * 32;
    int64_t position = 0;
    uint64_t rate = 0;
    const auto ask = [&] {
        if (thread < a.rope.pairs * tokens) {  // of the thread's first pair
            const int t = SEVERAL ? thread / a.rope.pairs : 0;
            if (a.rope.positions) position = SEVERAL ? position_of(a, first_token + t) : position_at(a.rope, batch, at);
            rate = a.rope.rates[thread - t * a.rope.pairs];
        }
    };
    if (N == 1) ask();
    uint4 xa[N], xb[N];
    {
        const T* in = static_cast<const T*>(s.in) + batch * s.in_batch + at * s.in_token;
        if (H < N && both) {
            const T* in2 = static_cast<const T*>(s2.in) + at * s2.in_token;
#pragma unroll
            for (int p = 0; p < H; ++p) {
                xa[p] = xb[p] = xa[H + p] = xb[H + p] = make_uint4(0, 0, 0, 0);
                if (p < passes) {
                    const int h = whole ? head + p * step : min(head + p * step, s.heads - 1);
                    const T *row = in + h * s.in_head, *row2 = in2 + h * s2.in_head;
                    if (v.has_a()) xa[p] = ld_stream(row + v.a);
                    if (v.has_b()) xb[p] = ld_stream(row + v.b);
                    if (v.has_a()) xa[H + p] = ld_stream(row2 + v.a);
                    if (v.has_b()) xb[H + p] = ld_stream(row2 + v.b);
                }
            }
        } else if (FULL && whole) {
            const T* row = in + head * s.in_head;
            const int64_t further = step * s.in_head;
#pragma unroll
            for (int p = 0; p < N; ++p, row += further) {
                if (M < N && p == M && s.cache) break;
                xa[p] = ld_stream(row + v.a), xb[p] = ld_stream(row + v.b);
            }
        } else {
#pragma unroll
            for (int p = 0; p < N; ++p) {
                xa[p] = xb[p] = make_uint4(0, 0, 0, 0);
                if (real && p < passes) {  // the same for all lanes; a head behind the last is the last, which is in the share
                    const T* row = in + min(head + p * step, s.heads - 1) * s.in_head;
                    if (v.has_a()) xa[p] = ld_stream(row + v.a);
                    if (v.has_b()) xb[p] = ld_stream(row + v.b);
                }
            }
        }
    }
    if (N > 1) ask();
    const T* weight = static_cast<const T*>(s.weight);
    Place place{0, -1, -1};
    if constexpr (APPEND) {
        for (int t = warp; t < tokens; t += warps) {  // a warp to a token
            place = find_place(a, static_cast<int>(first_token) + t, lane);
            if (lane == 0) places[t] = place;
        }
        __syncthreads();
        place = places[nth];
    }
    if (a.rope.pairs) {
        float* table = reinterpret_cast<float*>(tables);
        for (int i = thread; i < a.rope.pairs * tokens; i += threads) {
            const int t = SEVERAL ? i / a.rope.pairs : 0, p = i - t * a.rope.pairs;
            if (i != thread) {
                if (SEVERAL && a.rope.positions) position = position_of(a, first_token + t);
                rate = a.rope.rates[p];
            }
            if (APPEND && !a.rope.positions) position = places[t].position;
            const float2 cs = turn_of(rate, position, a.rope.magnitude, a.rope.direction);
            table[2 * t * a.rope.pairs + p] = cs.x;
            table[(2 * t + 1) * a.rope.pairs + p] = cs.y;
        }
    }
    const float* table = reinterpret_cast<const float*>(tables) + 2 * nth * a.rope.pairs;
    const float mean_of = 1.f / (FULL ? 2 * W * GT : a.dim);
    // A single row's norm does not wait for the angles (2% of a decode step); of
    // four rows it would be computed from values that are unpacked once more (4%
    // slower at 16384 tokens of 72 heads).
    float rstd[N] = {};
    if (N == 1 && weight) rstd[0] = rstd_of<T, INTER, GT>(xa[0], xb[0], G, lane, mean_of, a.eps);
    if (a.rope.pairs) __syncthreads();
    if (!real) return;
    const int page = APPEND && s.cache ? page_of(a, place) : 0;
    if (APPEND && (place.slot < 0 || page < 0)) {  // padding, or no page: nothing is stored
        if (!SEVERAL || s.per_token) return;       // the whole warp's token
        mine = false;
    }
    const bool half = N > 2 && passes <= 2;
    T* out = static_cast<T*>(s.out);
    if (APPEND && s.cache) {
        const int64_t cell = page * s.out_batch + place.slot * s.out_token;
        if constexpr (CACHE == kCache8Bits) {
            const bool int8 = a.format == kCacheInt8;
            if (H < N && both) {  // the values first: they need no factors, whose registers the keys take then
                uint8_t* q = static_cast<uint8_t*>(s2.out) + page * s2.out_batch + place.slot * s2.out_token + head * s2.out_head;
                float* scale = s2.scale + page * s2.scale_page + place.slot * s2.scale_slot + head * s2.scale_head;
#pragma unroll
                for (int p = 0; p < H; ++p, q += step * s2.out_head, scale += step * s2.scale_head) {
                    if (p >= passes) break;
                    float2 x[P], y[P];
                    Elem<T, INTER>::unpack(xa[H % N + p], xb[H % N + p], x, y);
                    store_row_8<INTER, GT, P>(int8, q, scale, x, y, G, lane, mine && head + p * step < s.heads, j == 0, v);
                }
            }
            LaneFactors<W, INTER, FULL> f;
            if (weight || pairs) f.read(weight, table, pairs, v);
            uint8_t* q = static_cast<uint8_t*>(s.out) + cell + head * s.out_head;
            float* scale = s.scale + page * s.scale_page + place.slot * s.scale_slot + head * s.scale_head;
#pragma unroll
            for (int p = 0; p < M; ++p, q += step * s.out_head, scale += step * s.scale_head) {
                if (p >= passes) break;
                float2 x[P], y[P];
                if (weight) {
                    const float r = N > 1 ? rstd_of<T, INTER, GT>(xa[p], xb[p], G, lane, mean_of, a.eps) : rstd[p];
                    turn_row<T, INTER, FULL, true, P>(xa[p], xb[p], r, f, x, y);
                } else if (pairs) {
                    turn_row<T, INTER, FULL, false, P>(xa[p], xb[p], 1.f, f, x, y);
                } else {
                    Elem<T, INTER>::unpack(xa[p], xb[p], x, y);
                }
                store_row_8<INTER, GT, P>(int8, q, scale, x, y, G, lane, mine && head + p * step < s.heads, j == 0, v);
            }
            return;
        }
        out += cell;
    } else {
        out += batch * s.out_batch + at * s.out_token;
    }
    if (weight || pairs) {  // else the rows go as they are
        LaneFactors<W, INTER, FULL> f;
        f.read(weight, table, pairs, v);
        if (weight) {
            if (half) turn_rows<T, INTER, GT, true, (N + 1) / 2>(xa, xb, rstd, f, G, lane, mean_of, a.eps);
            else turn_rows<T, INTER, GT, true, N>(xa, xb, rstd, f, G, lane, mean_of, a.eps);
        } else {
            if (H < N && both) turn_rows<T, INTER, GT, false, H>(xa, xb, rstd, f, G, lane, mean_of, a.eps);
            else turn_rows<T, INTER, GT, false, N>(xa, xb, rstd, f, G, lane, mean_of, a.eps);
        }
    }
    if (H < N && both) {
        T* out2 = static_cast<T*>(s2.out) + page * s2.out_batch + place.slot * s2.out_token;
#pragma unroll
        for (int p = 0; p < H; ++p) {
            const int h = head + p * step;
            if (mine && h < s.heads) {
                T *row = out + h * s.out_head, *row2 = out2 + h * s2.out_head;
                if (v.has_a()) st_stream(row + v.a, xa[p]);
                if (v.has_b()) st_stream(row + v.b, xb[p]);
                if (v.has_a()) st_stream(row2 + v.a, xa[H + p]);
                if (v.has_b()) st_stream(row2 + v.b, xb[H + p]);
            }
        }
    } else if (FULL && whole) {
        if (mine) {
            T* row = out + head * s.out_head;
            const int64_t further = step * s.out_head;
#pragma unroll
            for (int p = 0; p < N; ++p, row += further) st_stream(row + v.a, xa[p]), st_stream(row + v.b, xb[p]);
        }
    } else {
#pragma unroll
        for (int p = 0; p < N; ++p) {
            if (mine && head + p * step < s.heads) {
                T* row = out + (head + p * step) * s.out_head;
                if (v.has_a()) st_stream(row + v.a, xa[p]);
                if (v.has_b()) st_stream(row + v.b, xb[p]);
            }
        }
    }
}

// Any head size, stride and alignment: a warp holds one row in shared memory,
// element by element.  For rows whose vectors do not fall on 16 bytes, or whose
// rotated halves are no whole vectors.  A CTA takes a token, each of its warps
// `heads` rows, and the angles are computed once (16384 tokens of 32 heads of 128
// from odd addresses: 113 us, with angles for every row 196; whole vectors 42).
template <typename T, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32) heads_elements(const __grid_constant__ HeadsArgs a, int heads) {
    extern __shared__ float staged[];  // [kWarps][dim], then [2][pairs]
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dim = a.dim;
    const uint32_t token = divide(blockIdx.x, a.by_turns), batch = APPEND ? 0 : divide(token, a.by_tokens), at = token - batch * a.tokens;
    Place place{0, -1, -1};
    if constexpr (APPEND) {
        place = find_place(a, static_cast<int>(token), lane);
        if (place.slot < 0) return;  // the whole CTA's token
    }
    float* const row = staged + warp * dim;
    float* const table = staged + kWarps * dim;
    if (a.rope.pairs) {
        const int64_t position = APPEND && !a.rope.positions ? place.position : position_at(a.rope, batch, at);
        fill_turns(table, a.rope, a.rope.pairs, position, a.rope.direction, threadIdx.x, kWarps * 32);
        __syncthreads();
    }
    int next = static_cast<int>(blockIdx.x - token * a.turns) * kWarps * heads + warp;
    for (int n = 0; n < heads && next < a.shares; ++n, next += kWarps) {
        int head = next, si = 0;
        while (head >= a.seg[si].heads) head -= a.seg[si++].heads;
        const HeadSegment& s = a.seg[si];
        const int page = APPEND && s.cache ? page_of(a, place) : 0;
        if (page < 0) continue;
        const int pairs = s.rotate ? a.rope.pairs : 0;
        const T* in = static_cast<const T*>(s.in) + batch * s.in_batch + at * s.in_token + head * s.in_head;
        float ss = 0.f;
        for (int i = lane; i < dim; i += 32) {
            const float x = load_element(in + i);
            row[i] = x;
            ss += x * x;
        }
        if (s.weight) {
            const float rstd = rsqrtf(sum_lanes<32>(ss, 32, lane) * (1.f / dim) + a.eps);
            for (int i = lane; i < dim; i += 32) row[i] *= rstd * load_element(static_cast<const T*>(s.weight) + i);
        }
        __syncwarp();
        if (pairs) {
            for (int p = lane; p < pairs; p += 32) {
                const int ia = a.rope.interleaved ? 2 * p : p, ib = a.rope.interleaved ? 2 * p + 1 : p + pairs;
                const float x = row[ia], y = row[ib], c = table[p], t = table[pairs + p];
                row[ia] = fmaf(y, -t, __fmul_rn(x, c));  // rounded as in the vector kernel
                row[ib] = fmaf(x, t, __fmul_rn(y, c));
            }
            __syncwarp();
        }
        if (APPEND && s.cache) {
            const int64_t first = page * s.out_batch + place.slot * s.out_token + head * s.out_head;
            if (a.format != kCacheSame) {
                uint32_t top = 0;
                for (int i = lane; i < dim; i += 32) top = max(top, __float_as_uint(fabsf(row[i])));
                top = __reduce_max_sync(0xFFFFFFFFu, top);
                const bool int8 = a.format == kCacheInt8, fine = finite_bits(top);
                const float scale = row_scale(int8, top), inverse = about_inverse(scale);
                uint8_t* out = static_cast<uint8_t*>(s.out) + first;
                for (int i = lane; i < dim; i += 32) {
                    const float q = quotient(row[i], scale, inverse);
                    out[i] = fine ? static_cast<uint8_t>(int8 ? int8_bits(q) : e4m3_pair(q, 0.f)) : 0;
                }
                if (lane == 0) s.scale[page * s.scale_page + place.slot * s.scale_slot + head * s.scale_head] = scale;
            } else {
                T* out = static_cast<T*>(s.out) + first;
                for (int i = lane; i < dim; i += 32) {
                    if (s.weight || pairs) store_element(out + i, row[i]);
                    else out[i] = in[i];
                }
            }
        } else {
            T* out = static_cast<T*>(s.out) + batch * s.out_batch + at * s.out_token + head * s.out_head;
            for (int i = lane; i < dim; i += 32) store_element(out + i, row[i]);
        }
        __syncwarp();  // before the next row takes its place
    }
}

bool fits(const void* p, int64_t s0, int64_t s1, int64_t s2, int elements, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && s0 % elements == 0 && s1 % elements == 0 && s2 % elements == 0;
}

// Whether every row falls on whole 16-byte vectors (8-bit rows: on W bytes), each
// with all its pairs turned or none.
bool whole_vectors(const HeadsArgs& a, int W) {
    if (a.dim % W || (a.dim / W + 1) / 2 > 32 || a.rope.pairs % (a.rope.interleaved ? W / 2 : W)) return false;
    for (int i = 0; i < a.segments; ++i) {
        const HeadSegment& s = a.seg[i];
        if (!fits(s.in, s.in_batch, s.in_token, s.in_head, W, 16)) return false;
        if (!fits(s.out, s.out_batch, s.out_token, s.out_head, W, s.cache && a.format != kCacheSame ? W : 16)) return false;
        if (reinterpret_cast<uintptr_t>(s.weight) % 16) return false;
    }
    return true;
}

// How one set's rows of `tokens` tokens are shared out, `most` rows to a group.
inline void share_out_set(HeadSegment& s, int tokens, int most, int rows) {
    s.with_next = false;
    s.per_token = (s.heads + rows * most - 1) / (rows * most);
    s.shares = tokens * s.per_token;
    if (tokens == 1) return;
    s.groups_of_token = (s.heads + most - 1) / most;
    s.groups_factor = 1024 / s.groups_of_token + 1;  // n * this >> 10 is n / groups_of_token for n and that below 32
    s.tokens_of_share = std::min(tokens, rows / s.groups_of_token);
    if (s.tokens_of_share > 1) s.per_token = 0, s.shares = (tokens + s.tokens_of_share - 1) / s.tokens_of_share;
}

inline int turns_of(int shares) { return (shares + kMaxWarps - 1) / kMaxWarps; }

// Shares the rows of `tokens` tokens out among warps, `passes` to a group.
inline void share_out_tokens(HeadsArgs& a, int tokens, int passes, int rows) {
    a.per_cta = tokens;
    a.shares = 0;
    for (int i = 0; i < a.segments; ++i) {
        HeadSegment& s = a.seg[i];
        share_out_set(s, tokens, s.cache && a.format != kCacheSame ? rows_8(passes) : passes, rows);
        a.shares += s.shares;
    }
}

// An append's keys and values together, where that takes fewer CTAs, or fewer
// warps of a token's one (8192 tokens of 32 + 8 + 8 heads to an 8-bit cache 38 us,
// apart 40); else such a share only lasts longer than the others (64 + 8 + 8 heads
// 63, apart 59).
inline bool join_keys_and_values(HeadsArgs& a, int passes, int rows) {
    if (a.segments < 2 || !a.seg[a.segments - 1].cache) return false;
    HeadSegment &k = a.seg[a.segments - 2], &v = a.seg[a.segments - 1], joined = k;
    share_out_set(joined, a.per_cta, passes / 2, rows);
    const int shares = a.shares - k.shares - v.shares + joined.shares;
    if (turns_of(shares) == turns_of(a.shares) && !(a.per_cta == 1 && shares < a.shares && a.shares <= kMaxWarps)) return false;
    k = joined;
    k.with_next = true;
    v.shares = 0;
    a.shares = shares;
    return true;
}

// Rows of a group to a share, and the tokens to a CTA.  Four rows where that
// leaves every SM its warps: they are in flight together and spread what a warp
// does before them.  Then the tokens that take the fewest instructions each (some
// 300 for a share before its rows, 90 for 32 angles, which every CTA of the tokens
// computes), by a tenth.  Several tokens' keys and values are joined where there
// are more warps than run at a time (appends of 8 + 1 + 1 heads, us, joined / apart:
// 8192 tokens 12.8 / 15.3, 2500 6.3 / 7.2, 2200 5.0 / 4.6) and that is a fifth
// less than token by token (16 + 4 + 4 heads, an eighth less, 24.0 and 21.1).
inline int share_out(HeadsArgs& a, int rows, int64_t many, int sms) {
    const auto shares = [&] { return (static_cast<int64_t>(a.total) + a.per_cta - 1) / a.per_cta * a.shares; };
    const auto cost = [&] { return (300.0 * a.shares + 90.0 * turns_of(a.shares) * ((a.per_cta * a.rope.pairs + 31) / 32)) / a.per_cta; };
    share_out_tokens(a, 1, 4, rows);
    join_keys_and_values(a, 4, rows);
    if (shares() < many * sms) {
        share_out_tokens(a, 1, 1, rows);
        return 1;
    }
    const double one = cost();
    const auto most = [&](int tokens) { return tokens <= kMaxTokens && tokens * a.rope.pairs <= 1024; };
    double least = one;
    int64_t warps = shares();
    int best = 1;
    bool joined = true;
    for (int tokens = 2; most(tokens); ++tokens) {
        share_out_tokens(a, tokens, 4, rows);
        if (shares() < many * sms) break;
        if (cost() < 0.9 * least) best = tokens, least = cost(), warps = shares(), joined = false;
    }
    for (int tokens = 2; warps > (kMinCtas + 1) * kMaxWarps * sms && most(tokens); ++tokens) {
        share_out_tokens(a, tokens, 4, rows);
        if (!join_keys_and_values(a, 4, rows)) continue;
        if (shares() < many * sms) break;
        if (cost() < 0.9 * least && cost() < 0.8 * one) best = tokens, least = cost(), joined = true;
    }
    share_out_tokens(a, best, 4, rows);
    if (joined) join_keys_and_values(a, 4, rows);
    return 4;
}

template <typename T, bool INTER, int CACHE, int GT>
cudaError_t launch_rows(const HeadsArgs& a, int passes, int G, dim3 grid, dim3 block, size_t smem, cudaStream_t st) {
    if (passes == 1) return launch_args(heads_rows<T, INTER, CACHE, GT, 1, kOneToken>, grid, block, smem, st, a, G);
    if (a.per_cta == 1) return launch_args(heads_rows<T, INTER, CACHE, GT, 4, kOneToken>, grid, block, smem, st, a, G);
    if constexpr (CACHE != kNoCache) {
        if (a.seg[a.segments - 2].with_next) return launch_args(heads_rows<T, INTER, CACHE, GT, 4, kSeveralJoined>, grid, block, smem, st, a, G);
    }
    return launch_args(heads_rows<T, INTER, CACHE, GT, 4, kSeveralTokens>, grid, block, smem, st, a, G);
}

// The head sizes with kernels of their own: 64, 80, 96, 112 and 128, in bf16 192 and 256 too.
template <typename T, bool INTER, int CACHE>
cudaError_t launch_lanes(const HeadsArgs& a, int passes, int lanes, dim3 grid, dim3 block, size_t smem, cudaStream_t st) {
    const int own = own_lanes<Elem<T, INTER>::W>(a.dim);
#define NF_LANES(n) \
    if (own == n) return launch_rows<T, INTER, CACHE, n>(a, passes, n, grid, block, smem, st);
    if constexpr (sizeof(T) == 2) {
        NF_EACH_LANES_bf16(NF_LANES)
    } else {
        NF_EACH_LANES_f32(NF_LANES)
    }
#undef NF_LANES
    return launch_rows<T, INTER, CACHE, 0>(a, passes, lanes, grid, block, smem, st);
}

template <typename T, int CACHE>
cudaError_t launch_heads_rows(HeadsArgs& a, int sms, cudaStream_t st) {
    constexpr int W = Elem<T, false>::W;
    constexpr bool APPEND = CACHE != kNoCache;
    if (APPEND) a.by_page = Divider(a.page_size);
    a.by_tokens = Divider(a.tokens);
    if (!whole_vectors(a, W)) {
        a.shares = 0;
        for (int i = 0; i < a.segments; ++i) a.shares += a.seg[i].heads;
        // eight rows to a warp where every SM has its warps all the same
        const int heads = static_cast<int64_t>(a.total) * a.shares >= 256 * static_cast<int64_t>(sms) ? 8 : 1;
        a.turns = (a.shares + kWarps * heads - 1) / (kWarps * heads);
        a.by_turns = Divider(a.turns);
        return launch_args(heads_elements<T, APPEND>, dim3(a.total * a.turns), dim3(kWarps * 32),
                           (kWarps * a.dim + 2 * a.rope.pairs) * sizeof(float), st, a, heads);
    }
    const int G = lanes_of<W>(a.dim), rows = 32 / G;
    const int passes = share_out(a, rows, many_shares(APPEND), sms);
    a.turns = turns_of(a.shares);
    const int warps = (a.shares + a.turns - 1) / a.turns;
    a.by_turns = Divider(a.turns);
    const dim3 grid((a.total + a.per_cta - 1) / a.per_cta * a.turns), block(warps * 32);
    const size_t smem = a.per_cta * a.rope.pairs * sizeof(float2);
    return a.rope.interleaved ? launch_lanes<T, true, CACHE>(a, passes, G, grid, block, smem, st)
                              : launch_lanes<T, false, CACHE>(a, passes, G, grid, block, smem, st);
}

}  // namespace
}  // namespace nf
