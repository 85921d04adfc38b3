// What the kernels on attention heads share: the lanes' vectors of a row, and
// the angles.
//
// A row is one head of one token, `dim` elements.  A group of G lanes (a power
// of two) holds it, each lane two 16-byte vectors a and b, chosen so that a
// lane can turn its elements without another's:
//   half layout (pairs i, i + pairs):  a = elements j W.., b = pairs + j W..
//     for lane j below pairs / W, then the elements behind the rotated ones,
//     two vectors to a lane;
//   interleaved (pairs 2i, 2i + 1): a and b are any two vectors.
//
// Angles.  A pair turns by position * frequency.  `rates` holds frequencies as
// the share of a turn per position, in units of 2^-64, so that the 64-bit
// product position * rate IS the angle modulo a turn: exact for every position
// up to the rate's own rounding (2^-65 turns per position), with no reduction
// of large angles, no table of angles and no limit to a context.  Its signed
// value over 2^63 is the angle in half turns, which sincospif takes.
#pragma once

#include "common.cuh"
#include "heads.h"
#include "pairs.cuh"
#include "pdl.cuh"

namespace nf {

// A 16-byte vector as W elements in fp32, in pairs for the packed arithmetic.
template <typename T> struct Elem;
template <> struct Elem<uint16_t> {  // bf16
    static constexpr int W = 8;
    static __device__ __forceinline__ void unpack(uint4 v, float2 (&f)[4]) { unpack8x2(v, f); }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[4]) { return pack8x2(f); }
    static __device__ __forceinline__ float load(const uint16_t* p) { return bf_lo(*p); }
    static __device__ __forceinline__ void store(uint16_t* p, float f) { *p = static_cast<uint16_t>(pack2(f, 0.f) & 0xFFFF); }
};
template <> struct Elem<float> {
    static constexpr int W = 4;
    static __device__ __forceinline__ void unpack(uint4 v, float2 (&f)[2]) {
        f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[2]) {
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    }
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ void store(float* p, float f) { *p = f; }
};

// (cos, sin) of a pair at a position, both times `magnitude`.  sincospif takes
// the angle's upper 24 bits, which fp32 holds exactly; the rest, below 2^-24 half
// turns, turns its result on to first order (what is left out is below 2^-46).
__device__ __forceinline__ float2 turn_of(uint64_t rate, int64_t position, float magnitude, float direction) {
    const uint64_t angle = rate * static_cast<uint64_t>(position);
    const int64_t upper = static_cast<int64_t>(angle + (1ull << 39)) >> 40;
    const int64_t rest = static_cast<int64_t>(angle - (static_cast<uint64_t>(upper) << 40));
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(upper)) * 0x1p-23f, &s, &c);
    const float r = __ll2float_rn(rest) * (3.14159265f * 0x1p-63f);
    return make_float2((c - s * r) * magnitude, (s + c * r) * magnitude * direction);
}

__device__ __forceinline__ int64_t position_at(const Rotation& r, uint32_t batch, uint32_t token) {
    const int64_t at = batch * r.position_batch + token;
    return r.wide ? static_cast<const int64_t*>(r.positions)[at] : static_cast<const int32_t*>(r.positions)[at];
}

// Lane j's two vectors: where they start, whether they are there, and how many
// pairs of each are turned (half layout: W of a, with b, or none).
template <int W, bool INTER>
struct LaneVectors {
    int a, b;
    bool has_a, has_b;
    int turned_a, turned_b;
    __device__ __forceinline__ LaneVectors(int j, int dim, int pairs) {
        const int vectors = dim / W, items = (vectors + 1) / 2;
        if constexpr (INTER) {
            a = j * W;
            b = (items + j) * W;
            has_a = j < items;
            has_b = has_a && items + j < vectors;
            turned_a = has_a ? max(0, min(W / 2, pairs - a / 2)) : 0;
            turned_b = has_b ? max(0, min(W / 2, pairs - b / 2)) : 0;
        } else {
            const int turned = pairs / W, rest = vectors - 2 * turned, rest_items = (rest + 1) / 2;
            const bool t = j < turned;
            a = t ? j * W : (turned + j) * W;
            b = t ? (turned + j) * W : (turned + rest_items + j) * W;
            has_a = j < turned + rest_items;
            has_b = has_a && (t || turned + rest_items + j < vectors);
            turned_a = t ? W : 0;
            turned_b = 0;
        }
    }
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

// A lane's angles from that table.  Elements that are not turned are left as
// they are, whatever stands beside them.
template <int W, bool INTER>
struct LaneTurns {
    float2 c[W / 2], s[W / 2];  // of pairs 2i and 2i + 1; interleaved: those of a, then those of b
    __device__ __forceinline__ void read(const float* table, int pairs, const LaneVectors<W, INTER>& v) {
        if constexpr (INTER) {
            float* cf = reinterpret_cast<float*>(c);
            float* sf = reinterpret_cast<float*>(s);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const bool on = i < W / 2 ? i < v.turned_a : i - W / 2 < v.turned_b;
                const int p = i < W / 2 ? v.a / 2 + i : v.b / 2 + i - W / 2;
                cf[i] = on ? table[p] : 1.f;
                sf[i] = on ? table[pairs + p] : 0.f;
            }
        } else if (v.turned_a) {  // pairs is a multiple of W here, and so is a
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const float4 cc = *reinterpret_cast<const float4*>(table + v.a + 4 * i);
                const float4 ss = *reinterpret_cast<const float4*>(table + pairs + v.a + 4 * i);
                c[2 * i] = make_float2(cc.x, cc.y);
                c[2 * i + 1] = make_float2(cc.z, cc.w);
                s[2 * i] = make_float2(ss.x, ss.y);
                s[2 * i + 1] = make_float2(ss.z, ss.w);
            }
        }
    }
    static __device__ __forceinline__ float2 turned(float2 v, float c, float s) { return make_float2(v.x * c - v.y * s, v.y * c + v.x * s); }
    __device__ __forceinline__ void turn(float2 (&a)[W / 2], float2 (&b)[W / 2], const LaneVectors<W, INTER>& v) const {
        if constexpr (INTER) {
            const float* cf = reinterpret_cast<const float*>(c);
            const float* sf = reinterpret_cast<const float*>(s);
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                if (i < v.turned_a) a[i] = turned(a[i], cf[i], sf[i]);
                if (i < v.turned_b) b[i] = turned(b[i], cf[W / 2 + i], sf[W / 2 + i]);
            }
        } else if (v.turned_a) {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                const float2 x = a[i], y = b[i], t = __fmul2_rn(y, s[i]);
                a[i] = __ffma2_rn(x, c[i], make_float2(-t.x, -t.y));
                b[i] = __ffma2_rn(y, c[i], __fmul2_rn(x, s[i]));
            }
        }
    }
};

// Sum over the G lanes of a group; every lane gets the same value.
__device__ __forceinline__ float sum_lanes(float v, int G) {
#pragma unroll
    for (int off = G >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint4* to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

inline int lanes_for(int items) {
    int g = 1;
    while (g < items) g *= 2;
    return g;
}

}  // namespace nf
