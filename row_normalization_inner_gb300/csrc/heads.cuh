// What the kernels on attention heads share: the lanes' vectors of a row, and
// the angles.
//
// A row is one head of one token, `dim` elements.  A group of G lanes (of which
// sizes, stands at the end of this file) holds it, each lane two 16-byte vectors a
// and b, chosen so that a lane can turn its elements without another's:
//   half layout (pairs i, i + pairs):  a = elements j W.., b = pairs + j W..
//     for lane j below pairs / W, then the elements behind the rotated ones,
//     two vectors to a lane;
//   interleaved (pairs 2i, 2i + 1): a and b are any two vectors.
// Either way a lane has W pairs (x, y): in the half layout x from a and y from
// b, interleaved the even elements of a and b and the odd ones.  A vector's
// pairs are all turned, or none.
//
// Angles.  A pair turns by position * frequency.  `rates` holds frequencies as
// the share of a turn per position, in units of 2^-64, so that the 64-bit
// product position * rate IS the angle modulo a turn: exact for every position
// up to the rate's own rounding (2^-65 turns per position), with no reduction
// of large angles, no table of angles and no limit to a context.
#pragma once

#include "common.cuh"
#include "heads.h"
#include "pairs.cuh"
#include "pdl.cuh"

namespace nf {

__device__ __forceinline__ uint32_t divide(uint32_t n, const Divider& d) {
    return d.m ? static_cast<uint32_t>(__umul64hi(n, d.m)) : n;
}

// A lane's two vectors as pairs (x, y) in fp32, two pairs to a register pair for
// the packed arithmetic.
template <typename T, bool INTER> struct Elem;
template <bool INTER> struct Elem<uint16_t, INTER> {  // bf16
    static constexpr int W = 8;
    static __device__ __forceinline__ void unpack(uint4 a, uint4 b, float2 (&x)[4], float2 (&y)[4]) {
        if constexpr (INTER) {
            x[0] = make_float2(bf_lo(a.x), bf_lo(a.y)), y[0] = make_float2(bf_hi(a.x), bf_hi(a.y));
            x[1] = make_float2(bf_lo(a.z), bf_lo(a.w)), y[1] = make_float2(bf_hi(a.z), bf_hi(a.w));
            x[2] = make_float2(bf_lo(b.x), bf_lo(b.y)), y[2] = make_float2(bf_hi(b.x), bf_hi(b.y));
            x[3] = make_float2(bf_lo(b.z), bf_lo(b.w)), y[3] = make_float2(bf_hi(b.z), bf_hi(b.w));
        } else {
            unpack8x2(a, x);
            unpack8x2(b, y);
        }
    }
    static __device__ __forceinline__ void pack(const float2 (&x)[4], const float2 (&y)[4], uint4& a, uint4& b) {
        if constexpr (INTER) {
            a = make_uint4(pack2(x[0].x, y[0].x), pack2(x[0].y, y[0].y), pack2(x[1].x, y[1].x), pack2(x[1].y, y[1].y));
            b = make_uint4(pack2(x[2].x, y[2].x), pack2(x[2].y, y[2].y), pack2(x[3].x, y[3].x), pack2(x[3].y, y[3].y));
        } else {
            a = pack8x2(x);
            b = pack8x2(y);
        }
    }
};
template <bool INTER> struct Elem<float, INTER> {
    static constexpr int W = 4;
    static __device__ __forceinline__ float f(uint32_t u) { return __uint_as_float(u); }
    static __device__ __forceinline__ uint32_t u(float v) { return __float_as_uint(v); }
    static __device__ __forceinline__ void unpack(uint4 a, uint4 b, float2 (&x)[2], float2 (&y)[2]) {
        if constexpr (INTER) {
            x[0] = make_float2(f(a.x), f(a.z)), y[0] = make_float2(f(a.y), f(a.w));
            x[1] = make_float2(f(b.x), f(b.z)), y[1] = make_float2(f(b.y), f(b.w));
        } else {
            x[0] = make_float2(f(a.x), f(a.y)), x[1] = make_float2(f(a.z), f(a.w));
            y[0] = make_float2(f(b.x), f(b.y)), y[1] = make_float2(f(b.z), f(b.w));
        }
    }
    static __device__ __forceinline__ void pack(const float2 (&x)[2], const float2 (&y)[2], uint4& a, uint4& b) {
        if constexpr (INTER) {
            a = make_uint4(u(x[0].x), u(y[0].x), u(x[0].y), u(y[0].y));
            b = make_uint4(u(x[1].x), u(y[1].x), u(x[1].y), u(y[1].y));
        } else {
            a = make_uint4(u(x[0].x), u(x[0].y), u(x[1].x), u(x[1].y));
            b = make_uint4(u(y[0].x), u(y[0].y), u(y[1].x), u(y[1].y));
        }
    }
};
__device__ __forceinline__ float load_element(const uint16_t* p) { return bf_lo(*p); }
__device__ __forceinline__ float load_element(const float* p) { return *p; }
__device__ __forceinline__ void store_element(uint16_t* p, float f) { *p = static_cast<uint16_t>(pack2(f, 0.f) & 0xFFFF); }
__device__ __forceinline__ void store_element(float* p, float f) { *p = f; }

// (cos, sin) of a pair at a position, both times `magnitude`.  The angle's upper
// 32 bits (rounded) are a quarter and the rest to it; that and the lower 32 (signed)
// are x in [-1/2, 1/2] quarters, off by 1.5 * 2^-24 of itself at most.  On it the Taylor
// series of sin and cos of h x, h = pi / 2, to x^9 and x^10 (what is left out is
// below 2^-29 and 2^-30), the sine's first coefficient in two parts.  Both are off by
// 1.25 steps of 2^-24 at most over 4 million angles (0.28 in the square mean, rounding
// alone 0.24), and by 2.2 of their own value, however small: the slow pairs of the
// first positions turn by 1e-6, of which the upper 32 bits alone keep nine.  x as one
// 64-bit integer made to a float is off by 2^-24 and takes 3% in calls of few heads.
__device__ __forceinline__ float2 turn_of(uint64_t rate, int64_t position, float magnitude, float direction) {
    constexpr double h = 1.57079632679489661923, h2 = h * h, h3 = h * h2, h4 = h2 * h2;
    constexpr float first = static_cast<float>(h), rest = static_cast<float>(h - static_cast<double>(first));
    const uint64_t angle = rate * static_cast<uint64_t>(position);
    const uint32_t upper = static_cast<uint32_t>((angle + (1ull << 31)) >> 32), quarter = (upper + (1u << 29)) >> 30;
    const int32_t rest_of_upper = static_cast<int32_t>(upper << 2), lower = static_cast<int32_t>(static_cast<uint32_t>(angle));
    const float x = fmaf(static_cast<float>(lower), 0x1p-62f, static_cast<float>(rest_of_upper) * 0x1p-32f), z = x * x;
    float s = static_cast<float>(h4 * h4 * h / 362880);
    s = fmaf(s, z, static_cast<float>(-h3 * h4 / 5040));
    s = fmaf(s, z, static_cast<float>(h * h4 / 120));
    s = fmaf(s, z, static_cast<float>(-h3 / 6));
    s = fmaf(x, first, x * fmaf(s, z, rest));
    float c = static_cast<float>(-h4 * h4 * h2 / 3628800);
    c = fmaf(c, z, static_cast<float>(h4 * h4 / 40320));
    c = fmaf(c, z, static_cast<float>(-h2 * h4 / 720));
    c = fmaf(c, z, static_cast<float>(h4 / 24));
    c = fmaf(c, z, static_cast<float>(-h2 / 2));
    c = fmaf(c, z, 1.f);
    const float cosine = __uint_as_float(__float_as_uint(quarter & 1 ? s : c) ^ ((quarter + 1 & 2) << 30));
    const float sine = __uint_as_float(__float_as_uint(quarter & 1 ? c : s) ^ ((quarter & 2) << 30));
    return make_float2(cosine * magnitude, sine * (magnitude * direction));
}

__device__ __forceinline__ int64_t position_at(const Rotation& r, uint32_t batch, uint32_t token) {
    const int64_t at = batch * r.position_batch + token;
    return r.wide ? static_cast<const int64_t*>(r.positions)[at] : static_cast<const int32_t*>(r.positions)[at];
}

__device__ __forceinline__ int64_t position_of(const HeadsArgs& a, uint32_t token) {
    const uint32_t batch = divide(token, a.by_tokens);
    return position_at(a.rope, batch, token - batch * a.tokens);
}

// Lane j's two vectors: where they start, whether they are there, and whether
// their pairs are turned.  FULL: every lane of a group has both.
template <int W, bool INTER, bool FULL>
struct LaneVectors {
    int a, b;
    bool in_a, in_b;
    bool turn_a, turn_b;  // of the first and the second half of the lane's pairs
    __device__ __forceinline__ LaneVectors(int j, int dim, int pairs) {
        const int vectors = dim / W, items = (vectors + 1) / 2;
        if constexpr (INTER) {
            a = j * W;
            b = (items + j) * W;
            in_a = j < items;
            in_b = in_a && items + j < vectors;
            turn_a = in_a && a < 2 * pairs;
            turn_b = in_b && b < 2 * pairs;
        } else {
            const int turned = pairs / W, rest = vectors - 2 * turned, rest_items = (rest + 1) / 2;
            turn_a = turn_b = j < turned;
            a = turn_a ? j * W : (turned + j) * W;
            b = turn_a ? (turned + j) * W : (turned + rest_items + j) * W;
            in_a = j < turned + rest_items;
            in_b = in_a && (turn_a || turned + rest_items + j < vectors);
        }
    }
    __device__ __forceinline__ bool has_a() const { return FULL || in_a; }
    __device__ __forceinline__ bool has_b() const { return FULL || in_b; }
};

// A token's angles in shared memory: `pairs` cosines, then as many sines, by
// `threads` threads of which this is number `t`.
__device__ __forceinline__ void fill_turns(float* table, const Rotation& r, int pairs, int64_t position, float direction, int t, int threads) {
    for (int p = t; p < pairs; p += threads) {
        const float2 cs = turn_of(r.rates[p], position, r.magnitude, direction);
        table[p] = cs.x;
        table[pairs + p] = cs.y;
    }
}

// The lane's cosines and sines from that table (pairs and the vectors' first
// pairs are whole multiples of what is read at once).  Pairs that are not turned
// get (1, 0).
template <int W, bool INTER, bool FULL>
__device__ __forceinline__ void read_turns(const float* table, int pairs, const LaneVectors<W, INTER, FULL>& v, float2 (&c)[W / 2], float2 (&s)[W / 2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // the first and the second half of the lane's pairs
        const bool on = h ? v.turn_b : v.turn_a;
        const float* from = table + (!INTER ? v.a + h * (W / 2) : (h ? v.b : v.a) / 2);
        if constexpr (W == 8) {
            const float4 cc = on ? *reinterpret_cast<const float4*>(from) : make_float4(1.f, 1.f, 1.f, 1.f);
            const float4 ss = on ? *reinterpret_cast<const float4*>(from + pairs) : make_float4(0.f, 0.f, 0.f, 0.f);
            c[2 * h] = make_float2(cc.x, cc.y), c[2 * h + 1] = make_float2(cc.z, cc.w);
            s[2 * h] = make_float2(ss.x, ss.y), s[2 * h + 1] = make_float2(ss.z, ss.w);
        } else {
            c[h] = on ? *reinterpret_cast<const float2*>(from) : make_float2(1.f, 1.f);
            s[h] = on ? *reinterpret_cast<const float2*>(from + pairs) : make_float2(0.f, 0.f);
        }
    }
}

// A lane's factors at a token, the weights folded into the angles:
//   x' = x xc + y ys,   y' = y yc + x xs
// which takes a product per element out of every row.  A pair that is not
// turned takes xc and yc alone, whatever stands in its other element.
template <int W, bool INTER, bool FULL>
struct LaneFactors {
    static constexpr int P = W / 2;
    float2 xc[P], ys[P], yc[P], xs[P];
    bool turn_a, turn_b;
    template <typename T>
    __device__ __forceinline__ void read(const T* weight, const float* table, int pairs, const LaneVectors<W, INTER, FULL>& v) {
        float2 c[P], s[P];
        turn_a = v.turn_a, turn_b = v.turn_b;
        if (pairs) {
            read_turns<W, INTER, FULL>(table, pairs, v, c, s);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) c[i] = make_float2(1.f, 1.f), s[i] = make_float2(0.f, 0.f);
        }
        if (weight) {
            uint4 ua = make_uint4(0, 0, 0, 0), ub = ua;
            if (v.has_a()) ua = ld_param(weight + v.a);
            if (v.has_b()) ub = ld_param(weight + v.b);
            float2 x[P], y[P];
            Elem<T, INTER>::unpack(ua, ub, x, y);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                xc[i] = __fmul2_rn(x[i], c[i]);
                yc[i] = __fmul2_rn(y[i], c[i]);
                xs[i] = __fmul2_rn(x[i], s[i]);
                ys[i] = __fmul2_rn(y[i], make_float2(-s[i].x, -s[i].y));
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) xc[i] = yc[i] = c[i], xs[i] = s[i], ys[i] = make_float2(-s[i].x, -s[i].y);
        }
    }
    __device__ __forceinline__ void apply(float2 (&x)[P], float2 (&y)[P]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h ? turn_b : turn_a) {
#pragma unroll
                for (int i = h * P / 2; i < (h + 1) * P / 2; ++i) {
                    const float2 u = x[i];
                    x[i] = __ffma2_rn(y[i], ys[i], __fmul2_rn(u, xc[i]));
                    y[i] = __ffma2_rn(u, xs[i], __fmul2_rn(y[i], yc[i]));
                }
            } else {
#pragma unroll
                for (int i = h * P / 2; i < (h + 1) * P / 2; ++i) x[i] = __fmul2_rn(x[i], xc[i]), y[i] = __fmul2_rn(y[i], yc[i]);
            }
        }
    }
};

// The elements of vectors a and b in their order.
template <int W, bool INTER>
__device__ __forceinline__ void in_order(const float2 (&x)[W / 2], const float2 (&y)[W / 2], float (&a)[W], float (&b)[W]) {
    const float *xf = reinterpret_cast<const float*>(x), *yf = reinterpret_cast<const float*>(y);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        a[i] = !INTER ? xf[i] : i % 2 ? yf[i / 2] : xf[i / 2];
        b[i] = !INTER ? yf[i] : i % 2 ? yf[W / 2 + i / 2] : xf[W / 2 + i / 2];
    }
}

// Over the G lanes of a lane's group; all lanes of the warp call this, and every
// lane of a group gets the same value.  Where G is no power of two the group's
// first lane gathers it and hands it on.
template <int GT, typename V, typename Op>
__device__ __forceinline__ V over_lanes(V v, int G, int lane, Op op) {
    if constexpr (GT == 0 || (GT & (GT - 1)) == 0) {
#pragma unroll
        for (int off = G >> 1; off > 0; off >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
        return v;
    } else {
        const int j = lane % GT;
#pragma unroll
        for (int off = GT > 8 ? 8 : 4; off > 0; off >>= 1) {
            const V w = __shfl_down_sync(0xFFFFFFFFu, v, off);
            if (j + off < GT) v = op(v, w);
        }
        return __shfl_sync(0xFFFFFFFFu, v, lane - j);
    }
}
template <int GT>
__device__ __forceinline__ float sum_lanes(float v, int G, int lane) {
    return over_lanes<GT>(v, G, lane, [](float a, float b) { return a + b; });
}
template <int GT>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v, int G, int lane) {
    return over_lanes<GT>(v, G, lane, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint4* to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// As launch_with_pdl, the arguments (600 bytes) handed to the driver where they are.
template <typename Args>
cudaError_t launch_args(void (*kernel)(Args, int), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Args& args, int lanes) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* pointers[] = {const_cast<Args*>(&args), &lanes};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), pointers);
}

constexpr int kNoHead = 1 << 30;  // of a lane without a row; far from overflow when passes are added

// Lanes of a group.  Sizes whose lanes all have two whole vectors and that heads
// come in have kernels compiled for them; 5, 6, 7, 10, 12 or 14 lanes leave a few
// of a warp's idle (heads of 80 in bf16: six rows of five lanes, where groups of
// eight held four).  Others take the next power of two.
#define NF_EACH_LANES_bf16(X) X(4) X(5) X(6) X(7) X(8) X(12) X(16)
#define NF_EACH_LANES_f32(X) X(8) X(10) X(12) X(14) X(16)
template <int W>
inline int own_lanes(int dim) {
    if (dim % (2 * W)) return 0;
    const int n = dim / (2 * W);
    bool own = false;
#define NF_IS(m) own = own || n == m;
    if (W == 8) { NF_EACH_LANES_bf16(NF_IS) } else { NF_EACH_LANES_f32(NF_IS) }
#undef NF_IS
    return own ? n : 0;
}
template <int W>
inline int lanes_of(int dim) {
    if (const int own = own_lanes<W>(dim)) return own;
    int g = 1;
    while (g < (dim / W + 1) / 2) g *= 2;
    return g;
}

}  // namespace nf
