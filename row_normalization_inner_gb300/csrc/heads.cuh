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
// value over 2^63 is the angle in half turns, as sincospif takes it.
#pragma once

#include "common.cuh"
#include "heads.h"
#include "pdl.cuh"

namespace nf {

template <typename T> struct Elem;
template <> struct Elem<uint16_t> {  // bf16
    static constexpr int W = 8;
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) { unpack8(v, f); }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) { return pack8(f); }
    static __device__ __forceinline__ float load(const uint16_t* p) { return bf_lo(*p); }
    static __device__ __forceinline__ void store(uint16_t* p, float f) { *p = static_cast<uint16_t>(pack2(f, 0.f) & 0xFFFF); }
};
template <> struct Elem<float> {
    static constexpr int W = 4;
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ void store(float* p, float f) { *p = f; }
};

// (cos, sin) of a pair at a position, both times `magnitude`.
__device__ __forceinline__ float2 turn_of(uint64_t rate, int64_t position, float magnitude, float direction) {
    const int64_t angle = static_cast<int64_t>(rate * static_cast<uint64_t>(position));
    float s, c;
    sincospif(__ll2float_rn(angle) * 0x1p-63f, &s, &c);
    return make_float2(c * magnitude, s * magnitude * direction);
}

__device__ __forceinline__ int64_t position_at(const Rotation& r, uint32_t token, uint32_t tokens) {
    const uint32_t batch = token / tokens;
    const int64_t at = batch * r.position_batch + (token - batch * tokens);
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

// A lane's angles, from the warp's table of the token's.
template <int W, bool INTER>
struct LaneTurns {
    float c[W], s[W];  // interleaved: those of a, then those of b
    __device__ __forceinline__ void read(const float2* table, const LaneVectors<W, INTER>& v) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            bool on;
            int p;
            if constexpr (INTER) {
                on = i < W / 2 ? i < v.turned_a : i - W / 2 < v.turned_b;
                p = i < W / 2 ? v.a / 2 + i : v.b / 2 + i - W / 2;
            } else {
                on = v.turned_a > 0;
                p = v.a + i;
            }
            const float2 t = on ? table[p] : make_float2(1.f, 0.f);
            c[i] = t.x;
            s[i] = t.y;
        }
    }
    // Elements that are not turned are left as they are, whatever stands beside them.
    __device__ __forceinline__ void turn(float (&a)[W], float (&b)[W], const LaneVectors<W, INTER>& v) const {
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                const float x = a[2 * i], y = a[2 * i + 1];
                if (i < v.turned_a) {
                    a[2 * i] = x * c[i] - y * s[i];
                    a[2 * i + 1] = y * c[i] + x * s[i];
                }
                const float z = b[2 * i], w = b[2 * i + 1];
                if (i < v.turned_b) {
                    b[2 * i] = z * c[W / 2 + i] - w * s[W / 2 + i];
                    b[2 * i + 1] = w * c[W / 2 + i] + z * s[W / 2 + i];
                }
            }
        } else {
            const bool on = v.turned_a > 0;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float x = a[i], y = b[i];
                a[i] = on ? x * c[i] - y * s[i] : x;
                b[i] = on ? y * c[i] + x * s[i] : y;
            }
        }
    }
};

// Sum over the G lanes of a group; every lane gets the same value.
__device__ __forceinline__ float sum_lanes(float v, int G) {
    for (int off = G >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

inline int lanes_for(int items) {
    int g = 1;
    while (g < items) g *= 2;
    return g;
}

}  // namespace nf
