// Gradient of the RMSNorm of attention heads with the rotation behind it.  With
// the angles turned back, g = R(-t) dy, and n = x * rstd:
//
//   dweight = sum over all rows of g n                       (fp32)
//   dx      = rstd (g w - n mean(g w n))
//
// x is read again rather than saved as n: rstd comes out of the same pass.
//
// Bound by memory: dy and x are read once, dx written once.  A fixed number of
// CTAs walk the rows, each warp a stretch of its own in token order (so that a
// token's angles serve all its heads that the warp meets) and each lane with
// its columns' sums of g n in registers.  The rows ahead come through a ring in
// shared memory, each lane copying what it will read itself, so that no barrier
// stands between a copy and its use.  A CTA's sums go to the workspace, and a
// second launch adds them up: every sum has a fixed order.
#include <algorithm>

#include "heads.cuh"

namespace nf {
namespace {

constexpr int kWarps = 4;
constexpr int kCtasPerSm = 4;
constexpr int kStages = 4;

// What a warp walks: passes [first, end) of its segment, `per_token` to a token.
struct Stretch {
    int64_t first, end;
};
__device__ __forceinline__ Stretch stretch_of(int64_t passes, int warp, int warps) {
    return {passes * warp / warps, passes * (warp + 1) / warps};
}

// The CTA's sums over its warps, in their order, to the workspace.
__device__ __forceinline__ void leave_partials(const float* sums, float* out, int dim) {
    __syncthreads();
    for (int i = threadIdx.x; i < dim; i += kWarps * 32) {
        float s = sums[i];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) s += sums[w * dim + i];
        out[i] = s;
    }
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) heads_grad_rows(const __grid_constant__ HeadsGradArgs a, int G) {
    constexpr int W = Elem<T>::W;
    extern __shared__ uint4 ring[];  // [kStages][4][threads], then the turns
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp_in = threadIdx.x >> 5;
    int cta = blockIdx.x, si = 0;
    if (cta >= a.seg[0].ctas) cta -= a.seg[0].ctas, si = 1;
    const HeadGradSegment& s = a.seg[si];
    const int rows = 32 / G, j = lane & (G - 1), per_token = (s.heads + rows - 1) / rows;
    const Stretch r = stretch_of(static_cast<int64_t>(a.total) * per_token, cta * kWarps + warp_in, s.ctas * kWarps);
    const int pairs = a.rope.pairs;
    const LaneVectors<W, INTER> v(j, a.dim, pairs);
    float* table = reinterpret_cast<float*>(ring + kStages * 4 * kWarps * 32) + warp_in * 2 * pairs;

    uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
    if (v.has_a) wa = ld_param(static_cast<const T*>(s.weight) + v.a);
    if (v.has_b) wb = ld_param(static_cast<const T*>(s.weight) + v.b);
    float2 da[W / 2], db[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) da[i] = db[i] = make_float2(0.f, 0.f);

    if (r.first < r.end) {
        const float mean_of = 1.f / a.dim;
        uint32_t token = static_cast<uint32_t>(r.first / per_token);
        int pass = static_cast<int>(r.first - static_cast<int64_t>(token) * per_token);
        // the pass that is copied next
        uint32_t next_token = token;
        int next_pass = pass;
        int64_t left = r.end - r.first;
        const auto copy = [&](int stage) {
            if (left > 0) {
                const uint32_t batch = next_token / a.tokens, at = next_token - batch * a.tokens;
                const int head = next_pass * rows + lane / G;
                const bool here = head < s.heads;
                const T* y = static_cast<const T*>(s.dy) + batch * s.dy_batch + at * s.dy_token + (here ? head * s.dy_head : 0);
                const T* x = static_cast<const T*>(s.x) + batch * s.x_batch + at * s.x_token + (here ? head * s.x_head : 0);
                uint4* to = ring + stage * 4 * kWarps * 32 + threadIdx.x;
                const bool ha = here && v.has_a, hb = here && v.has_b;
                copy16(to, y + (ha ? v.a : 0), ha);
                copy16(to + kWarps * 32, y + (hb ? v.b : 0), hb);
                copy16(to + 2 * kWarps * 32, x + (ha ? v.a : 0), ha);
                copy16(to + 3 * kWarps * 32, x + (hb ? v.b : 0), hb);
                if (++next_pass == per_token) next_pass = 0, ++next_token;
                --left;
            }
            copies_commit();  // a group for every stage, empty ones behind the last pass
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) copy(i);
        int64_t position = pairs ? position_at(a.rope, token / a.tokens, token % a.tokens) : 0;
        bool fresh = true;
        LaneTurns<W, INTER> t;
        int stage = 0;
        for (int64_t p = r.first; p < r.end; ++p) {
            if (fresh && pairs) {
                __syncwarp();
                fill_turns(table, a.rope, pairs, position, -1.f, lane, 32);
                __syncwarp();
                t.read(table, pairs, v);
            }
            const uint32_t batch = token / a.tokens, at = token - batch * a.tokens;
            const int head = pass * rows + lane / G;
            fresh = ++pass == per_token;
            if (fresh) {
                pass = 0, ++token;
                if (pairs && p + 1 < r.end) position = position_at(a.rope, token / a.tokens, token % a.tokens);
            }
            copies_wait<kStages - 2>();
            const uint4* from = ring + stage * 4 * kWarps * 32 + threadIdx.x;
            float2 ga[W / 2], gb[W / 2], xa[W / 2], xb[W / 2], fa[W / 2], fb[W / 2];
            Elem<T>::unpack(from[0], ga);
            Elem<T>::unpack(from[kWarps * 32], gb);
            Elem<T>::unpack(from[2 * kWarps * 32], xa);
            Elem<T>::unpack(from[3 * kWarps * 32], xb);
            // into the stage before, whose rows are done with
            copy(stage ? stage - 1 : kStages - 1);
            stage = stage == kStages - 1 ? 0 : stage + 1;
            if (pairs) t.turn(ga, gb, v);
            Elem<T>::unpack(wa, fa);
            Elem<T>::unpack(wb, fb);
            float2 ss2 = make_float2(0.f, 0.f), dot2 = ss2;
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                ss2 = __ffma2_rn(xa[i], xa[i], ss2);
                ss2 = __ffma2_rn(xb[i], xb[i], ss2);
                fa[i] = __fmul2_rn(fa[i], ga[i]);
                fb[i] = __fmul2_rn(fb[i], gb[i]);
                dot2 = __ffma2_rn(fa[i], xa[i], dot2);
                dot2 = __ffma2_rn(fb[i], xb[i], dot2);
            }
            float ss = ss2.x + ss2.y, dot = dot2.x + dot2.y;
            for (int off = G >> 1; off > 0; off >>= 1) {
                ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
                dot += __shfl_xor_sync(0xFFFFFFFFu, dot, off);
            }
            const float rs = rsqrtf(ss * mean_of + a.eps), m = -dot * rs * mean_of;
            const float2 rstd = make_float2(rs, rs), mean = make_float2(m, m);
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                const float2 na = __fmul2_rn(xa[i], rstd), nb = __fmul2_rn(xb[i], rstd);
                da[i] = __ffma2_rn(ga[i], na, da[i]);
                db[i] = __ffma2_rn(gb[i], nb, db[i]);
                fa[i] = __fmul2_rn(rstd, __ffma2_rn(na, mean, fa[i]));
                fb[i] = __fmul2_rn(rstd, __ffma2_rn(nb, mean, fb[i]));
            }
            if (head < s.heads) {
                T* dx = static_cast<T*>(s.dx) + batch * s.dx_batch + at * s.dx_token + head * s.dx_head;
                if (v.has_a) st_stream(dx + v.a, Elem<T>::pack(fa));
                if (v.has_b) st_stream(dx + v.b, Elem<T>::pack(fb));
            }
        }
        copies_wait<0>();
    }
    for (int off = G; off < 32; off <<= 1) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            da[i].x += __shfl_xor_sync(0xFFFFFFFFu, da[i].x, off);
            da[i].y += __shfl_xor_sync(0xFFFFFFFFu, da[i].y, off);
            db[i].x += __shfl_xor_sync(0xFFFFFFFFu, db[i].x, off);
            db[i].y += __shfl_xor_sync(0xFFFFFFFFu, db[i].y, off);
        }
    }
    __syncthreads();  // the ring is done with: the sums take its place
    float* sums = reinterpret_cast<float*>(ring);
    if (lane < G) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            if (v.has_a) *reinterpret_cast<float2*>(sums + warp_in * a.dim + v.a + 2 * i) = da[i];
            if (v.has_b) *reinterpret_cast<float2*>(sums + warp_in * a.dim + v.b + 2 * i) = db[i];
        }
    }
    leave_partials(sums, a.partials + static_cast<int64_t>(blockIdx.x) * a.dim, a.dim);
}

// Any head size, stride and alignment: a warp's row in shared memory, element
// by element (as heads_elements).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) heads_grad_elements(const __grid_constant__ HeadsGradArgs a) {
    extern __shared__ float staged[];
    grid_dep_wait();
    grid_dep_release();
    constexpr int kPerLane = kHeadMaxDim / 32;
    const int lane = threadIdx.x & 31, warp_in = threadIdx.x >> 5, dim = a.dim, pairs = a.rope.pairs;
    int cta = blockIdx.x, si = 0;
    if (cta >= a.seg[0].ctas) cta -= a.seg[0].ctas, si = 1;
    const HeadGradSegment& s = a.seg[si];
    const Stretch r = stretch_of(static_cast<int64_t>(a.total) * s.heads, cta * kWarps + warp_in, s.ctas * kWarps);
    float* g = staged + warp_in * dim;
    float dw[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) dw[i] = 0.f;
    for (int64_t p = r.first; p < r.end; ++p) {
        const uint32_t token = static_cast<uint32_t>(p / s.heads), batch = token / a.tokens, at = token - batch * a.tokens;
        const int head = static_cast<int>(p - static_cast<int64_t>(token) * s.heads);
        const T* y = static_cast<const T*>(s.dy) + batch * s.dy_batch + at * s.dy_token + head * s.dy_head;
        const T* x = static_cast<const T*>(s.x) + batch * s.x_batch + at * s.x_token + head * s.x_head;
        T* dx = static_cast<T*>(s.dx) + batch * s.dx_batch + at * s.dx_token + head * s.dx_head;
        __syncwarp();
        for (int i = lane; i < dim; i += 32) g[i] = Elem<T>::load(y + i);
        __syncwarp();
        if (pairs) {
            const int64_t position = position_at(a.rope, token / a.tokens, token % a.tokens);
            for (int q = lane; q < pairs; q += 32) {
                const float2 t = turn_of(a.rope.rates[q], position, a.rope.magnitude, -1.f);
                const int ia = a.rope.interleaved ? 2 * q : q, ib = a.rope.interleaved ? 2 * q + 1 : q + pairs;
                const float u = g[ia], w = g[ib];
                g[ia] = u * t.x - w * t.y;
                g[ib] = w * t.x + u * t.y;
            }
            __syncwarp();
        }
        float ss = 0.f, dot = 0.f;
        for (int i = lane; i < dim; i += 32) {
            const float xi = Elem<T>::load(x + i);
            ss += xi * xi;
            dot += g[i] * Elem<T>::load(static_cast<const T*>(s.weight) + i) * xi;
        }
        ss = sum_lanes(ss, 32);
        dot = sum_lanes(dot, 32);
        const float rstd = rsqrtf(ss / dim + a.eps), mean = dot * rstd / dim;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
            const int i = lane + 32 * k;
            if (i < dim) {
                const float n = Elem<T>::load(x + i) * rstd;
                dw[k] += g[i] * n;
                Elem<T>::store(dx + i, rstd * (g[i] * Elem<T>::load(static_cast<const T*>(s.weight) + i) - n * mean));
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kPerLane; ++k)
        if (lane + 32 * k < dim) g[lane + 32 * k] = dw[k];
    leave_partials(staged, a.partials + static_cast<int64_t>(blockIdx.x) * dim, dim);
}

// dweight[i] = sum of its segment's partials: 32 columns to a CTA, 32 warps
// over the partials, then over the warps, in a fixed order.
__global__ void __launch_bounds__(1024) heads_grad_sum(const __grid_constant__ HeadsGradArgs a) {
    __shared__ float part[32][33];
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, column = blockIdx.x * 32 + lane;
    const HeadGradSegment& s = a.seg[blockIdx.y];
    const float* from = a.partials + static_cast<int64_t>(blockIdx.y ? a.seg[0].ctas : 0) * a.dim + column;
    float sum = 0.f;
    if (column < a.dim) {
#pragma unroll 8
        for (int p = warp; p < s.ctas; p += 32) sum += __ldcg(from + static_cast<int64_t>(p) * a.dim);
    }
    part[warp][lane] = sum;
    __syncthreads();
    sum = sum_lanes(part[lane][warp], 32);
    if (lane == 0 && blockIdx.x * 32 + warp < a.dim) s.dweight[blockIdx.x * 32 + warp] = sum;
}

bool fits(const void* p, int64_t s0, int64_t s1, int64_t s2, int W) {
    return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && s0 % W == 0 && s1 % W == 0 && s2 % W == 0;
}

bool whole_vectors(const HeadsGradArgs& a, int W) {
    if (a.dim % W || (a.dim / W + 1) / 2 > 32 || (!a.rope.interleaved && a.rope.pairs % W)) return false;
    for (int i = 0; i < a.segments; ++i) {
        const HeadGradSegment& s = a.seg[i];
        if (!fits(s.dx, s.dx_batch, s.dx_token, s.dx_head, W) || !fits(s.dy, s.dy_batch, s.dy_token, s.dy_head, W) ||
            !fits(s.x, s.x_batch, s.x_token, s.x_head, W) || reinterpret_cast<uintptr_t>(s.weight) % 16)
            return false;
    }
    return true;
}

template <typename T>
cudaError_t launch(HeadsGradArgs a, int sms, cudaStream_t st) {
    constexpr int W = Elem<T>::W;
    const bool vectors = whole_vectors(a, W);
    const int G = vectors ? lanes_for((a.dim / W + 1) / 2) : 32, rows = 32 / G;
    // CTAs in proportion to the segments' passes, two passes to a warp at least
    int64_t passes[2] = {0, 0};
    for (int i = 0; i < a.segments; ++i) passes[i] = static_cast<int64_t>(a.total) * ((a.seg[i].heads + rows - 1) / rows);
    const int64_t all = passes[0] + passes[1], most = static_cast<int64_t>(sms) * kCtasPerSm;
    const int64_t ctas = std::max<int64_t>(a.segments, std::min(most, (all + 2 * kWarps - 1) / (2 * kWarps)));
    a.seg[0].ctas = static_cast<int>(ctas);
    if (a.segments == 2) {
        const int64_t share = all ? (ctas * passes[1] + all / 2) / all : 1;
        a.seg[1].ctas = static_cast<int>(std::max<int64_t>(1, std::min(ctas - 1, share)));
        a.seg[0].ctas -= a.seg[1].ctas;
    }
    const dim3 grid(static_cast<unsigned>(ctas)), block(kWarps * 32);
    cudaError_t e;
    if (!vectors) {
        e = launch_with_pdl(heads_grad_elements<T>, grid, block, kWarps * a.dim * sizeof(float), st, a);
    } else {
        const size_t smem = kStages * 4 * kWarps * 32 * sizeof(uint4) + kWarps * a.rope.pairs * sizeof(float2);
        e = a.rope.interleaved ? launch_with_pdl(heads_grad_rows<T, true>, grid, block, smem, st, a, G)
                               : launch_with_pdl(heads_grad_rows<T, false>, grid, block, smem, st, a, G);
    }
    if (e != cudaSuccess) return e;
    return launch_with_pdl(heads_grad_sum, dim3((a.dim + 31) / 32, a.segments), dim3(1024), 0, st, a);
}

}  // namespace

size_t heads_grad_workspace(int64_t dim, int sms) {
    return static_cast<size_t>(sms) * kCtasPerSm * static_cast<size_t>(dim) * sizeof(float);
}

cudaError_t launch_heads_grad(const HeadsGradArgs& a, bool f32, int sms, cudaStream_t st) {
    return f32 ? launch<float>(a, sms, st) : launch<uint16_t>(a, sms, st);
}

}  // namespace nf
