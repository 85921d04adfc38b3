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
#pragma once

#include <algorithm>

#include "heads.cuh"

namespace nf {
namespace {

constexpr int kWarps = 4;
// Three CTAs to an SM and two passes ahead (16384 tokens of 72 heads of 128: 140 us;
// four CTAs, whose registers spill a little, 144, two 166; with four one pass
// ahead 165 and three 157, with five CTAs 220).
constexpr int kCtasPerSm = 3;
constexpr int kStages = 3;
// What a token's angles take, in passes: where only passes counted, the CTAs of 8
// key heads (two passes a token) were the last ones (0: 181 us with four CTAs to
// an SM, 1 165; with three CTAs 1 140, 2 141, 4 144).
constexpr int kTurnPasses = 1;

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

// Summed over the groups of a warp, in their order; the first one's lanes get it.
__device__ __forceinline__ float2 over_groups(float2 v, int G, int rows) {
    float2 s = v;
    for (int r = 1; r < rows; ++r) {
        s.x += __shfl_down_sync(0xFFFFFFFFu, v.x, r * G);
        s.y += __shfl_down_sync(0xFFFFFFFFu, v.y, r * G);
    }
    return s;
}

// A row of one of the walk's tensors, for the lane that holds it: `step` further
// with every pass of a token.
template <typename T>
struct RowPointer {
    T* p;
    int64_t step, next;  // to the next pass, and from behind a token's last pass to the next token's first
    __device__ __forceinline__ RowPointer(void* base, int64_t batch_stride, int64_t token_stride, int64_t head_stride, uint32_t batch, uint32_t token,
                                          int pass, int rows, int lane_row, int per_token)
        : step(rows * head_stride), next(token_stride - per_token * step) {
        p = static_cast<T*>(base) + batch * batch_stride + token * token_stride + (pass * rows + lane_row) * head_stride;
    }
};

template <typename T, bool INTER, int GT>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) heads_grad_rows(const __grid_constant__ HeadsGradArgs a, int lanes) {
    constexpr int W = Elem<T, INTER>::W, P = W / 2;
    constexpr bool FULL = GT != 0;
    const int G = FULL ? GT : lanes;
    constexpr int kSlot = 4 * kWarps * 32;  // vectors of a stage
    extern __shared__ uint4 ring[];         // [kStages][4][threads], then the turns
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp_in = threadIdx.x >> 5;
    int cta = blockIdx.x, si = 0;
    if (cta >= a.seg[0].ctas) cta -= a.seg[0].ctas, si = 1;
    const HeadGradSegment& s = a.seg[si];
    const int rows = 32 / G, lane_row = lane / G, j = lane - lane_row * G, per_token = (s.heads + rows - 1) / rows;
    const int first_head = lane_row < rows ? lane_row : kNoHead;  // lanes behind the last whole group hold none
    const Stretch r = stretch_of(static_cast<int64_t>(a.total) * per_token, cta * kWarps + warp_in, s.ctas * kWarps);
    const int pairs = a.rope.pairs;
    const LaneVectors<W, INTER, FULL> v(j, FULL ? 2 * W * GT : a.dim, pairs);
    float* table = reinterpret_cast<float*>(ring + kStages * kSlot) + warp_in * 2 * pairs;

    float2 dwx[P], dwy[P];
#pragma unroll
    for (int i = 0; i < P; ++i) dwx[i] = dwy[i] = make_float2(0.f, 0.f);

    if (r.first < r.end) {  // a call without rows may have null pointers
        uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
        if (v.has_a()) wa = ld_param(static_cast<const T*>(s.weight) + v.a);
        if (v.has_b()) wb = ld_param(static_cast<const T*>(s.weight) + v.b);
        const float mean_of = 1.f / (FULL ? 2 * W * GT : a.dim);
        uint32_t token = static_cast<uint32_t>(r.first / per_token);
        int pass = static_cast<int>(r.first - static_cast<int64_t>(token) * per_token), left = static_cast<int>(r.end - r.first);
        uint32_t batch = divide(token, a.by_tokens), at = token - batch * a.tokens;
        // the rows that are copied next, kStages - 1 passes ahead
        RowPointer<const T> y(const_cast<void*>(s.dy), s.dy_batch, s.dy_token, s.dy_head, batch, at, pass, rows, lane_row, per_token);
        RowPointer<const T> x(const_cast<void*>(s.x), s.x_batch, s.x_token, s.x_head, batch, at, pass, rows, lane_row, per_token);
        int ahead_head = pass * rows + first_head, ahead_pass = pass, ahead_left = left;
        uint32_t ahead_at = at;
        const auto copy = [&](int stage) {
            if (ahead_left > 0) {
                const bool here = ahead_head < s.heads;
                uint4* to = ring + stage * kSlot + threadIdx.x;
                const T* yp = here ? y.p : static_cast<const T*>(s.dy);
                const T* xp = here ? x.p : static_cast<const T*>(s.x);
                const bool ha = here && v.has_a(), hb = here && v.has_b();
                copy16(to, yp + (ha ? v.a : 0), ha);
                copy16(to + kWarps * 32, yp + (hb ? v.b : 0), hb);
                copy16(to + 2 * kWarps * 32, xp + (ha ? v.a : 0), ha);
                copy16(to + 3 * kWarps * 32, xp + (hb ? v.b : 0), hb);
                y.p += y.step, x.p += x.step, ahead_head += rows;
                if (++ahead_pass == per_token) {
                    ahead_pass = 0, ahead_head = first_head;
                    y.p += y.next, x.p += x.next;
                    if (++ahead_at == static_cast<uint32_t>(a.tokens)) {
                        ahead_at = 0;
                        y.p += s.dy_batch - a.tokens * s.dy_token, x.p += s.x_batch - a.tokens * s.x_token;
                    }
                }
                --ahead_left;
            }
            copies_commit();  // a group for every stage, empty ones behind the last pass
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) copy(i);
        RowPointer<T> dx(s.dx, s.dx_batch, s.dx_token, s.dx_head, batch, at, pass, rows, lane_row, per_token);
        int64_t position = pairs ? position_at(a.rope, batch, at) : 0;
        int stage = 0;
        while (left > 0) {  // a token
            float2 c[P], sn[P];
            if (pairs) {
                __syncwarp();
                fill_turns(table, a.rope, pairs, position, 1.f, lane, 32);
                __syncwarp();
                read_turns<W, INTER, FULL>(table, pairs, v, c, sn);
            }
            const int passes = min(left, per_token - pass);
            left -= passes;
            int head = pass * rows + first_head;
            if (++at == static_cast<uint32_t>(a.tokens)) at = 0, ++batch;
            if (pairs && left > 0) position = position_at(a.rope, batch, at);  // the next token's, on its way meanwhile
            for (int p = 0; p < passes; ++p) {
                copies_wait<kStages - 2>();
                const uint4* from = ring + stage * kSlot + threadIdx.x;
                float2 gx[P], gy[P], xx[P], xy[P], fx[P], fy[P];
                Elem<T, INTER>::unpack(from[0], from[kWarps * 32], gx, gy);
                Elem<T, INTER>::unpack(from[2 * kWarps * 32], from[3 * kWarps * 32], xx, xy);
                // into the stage before, whose rows are done with
                copy(stage ? stage - 1 : kStages - 1);
                stage = stage == kStages - 1 ? 0 : stage + 1;
                if (pairs) {  // turned back
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h ? v.turn_b : v.turn_a) {
#pragma unroll
                            for (int i = h * P / 2; i < (h + 1) * P / 2; ++i) {
                                const float2 u = gx[i], t = __fmul2_rn(u, sn[i]);
                                gx[i] = __ffma2_rn(gy[i], sn[i], __fmul2_rn(u, c[i]));
                                gy[i] = __ffma2_rn(gy[i], c[i], make_float2(-t.x, -t.y));
                            }
                        }
                    }
                }
                Elem<T, INTER>::unpack(wa, wb, fx, fy);
                float2 ss2 = make_float2(0.f, 0.f), dot2 = ss2;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    ss2 = __ffma2_rn(xx[i], xx[i], ss2);
                    ss2 = __ffma2_rn(xy[i], xy[i], ss2);
                    fx[i] = __fmul2_rn(fx[i], gx[i]);
                    fy[i] = __fmul2_rn(fy[i], gy[i]);
                    dot2 = __ffma2_rn(fx[i], xx[i], dot2);
                    dot2 = __ffma2_rn(fy[i], xy[i], dot2);
                }
                float ss = ss2.x + ss2.y, dot = dot2.x + dot2.y;
                ss = sum_lanes<GT>(ss, G, lane);
                dot = sum_lanes<GT>(dot, G, lane);
                const float rs = rsqrtf(ss * mean_of + a.eps), m = -dot * rs * mean_of;
                const float2 rstd = make_float2(rs, rs), mean = make_float2(m, m);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float2 nx = __fmul2_rn(xx[i], rstd), ny = __fmul2_rn(xy[i], rstd);
                    dwx[i] = __ffma2_rn(gx[i], nx, dwx[i]);
                    dwy[i] = __ffma2_rn(gy[i], ny, dwy[i]);
                    fx[i] = __fmul2_rn(rstd, __ffma2_rn(nx, mean, fx[i]));
                    fy[i] = __fmul2_rn(rstd, __ffma2_rn(ny, mean, fy[i]));
                }
                if (head < s.heads) {
                    uint4 oa, ob;
                    Elem<T, INTER>::pack(fx, fy, oa, ob);
                    if (v.has_a()) st_stream(dx.p + v.a, oa);
                    if (v.has_b()) st_stream(dx.p + v.b, ob);
                }
                dx.p += dx.step, head += rows;
            }
            pass = 0;
            dx.p += dx.next;
            if (at == 0) dx.p += s.dx_batch - a.tokens * s.dx_token;
        }
        copies_wait<0>();
    }
    // the groups' sums to the first one's lanes
#pragma unroll
    for (int i = 0; i < P; ++i) dwx[i] = over_groups(dwx[i], G, rows), dwy[i] = over_groups(dwy[i], G, rows);
    __syncthreads();  // the ring is done with: the sums take its place
    float* sums = reinterpret_cast<float*>(ring);
    if (lane < G) {
        float da[W], db[W];
        in_order<W, INTER>(dwx, dwy, da, db);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (v.has_a()) sums[warp_in * a.dim + v.a + i] = da[i];
            if (v.has_b()) sums[warp_in * a.dim + v.b + i] = db[i];
        }
    }
    leave_partials(sums, a.partials + static_cast<int64_t>(blockIdx.x) * a.dim, a.dim);
}

// Any head size, stride and alignment: a warp's row in shared memory, element
// by element (as heads_elements), its token's angles beside it; the next row is
// loaded meanwhile (16384 tokens of 32 heads of 128 from odd addresses: 333 us,
// 837 without; whole vectors 55).
template <typename T, int kPerLane>
__global__ void __launch_bounds__(kWarps * 32) heads_grad_elements(const __grid_constant__ HeadsGradArgs a) {
    extern __shared__ float staged[];
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp_in = threadIdx.x >> 5, dim = a.dim, pairs = a.rope.pairs;
    int cta = blockIdx.x, si = 0;
    if (cta >= a.seg[0].ctas) cta -= a.seg[0].ctas, si = 1;
    const HeadGradSegment& s = a.seg[si];
    const Stretch r = stretch_of(static_cast<int64_t>(a.total) * s.heads, cta * kWarps + warp_in, s.ctas * kWarps);
    float* const g = staged + warp_in * dim;
    float* const table = staged + kWarps * dim + warp_in * 2 * pairs;
    float dw[kPerLane], w[kPerLane], x[kPerLane], y[kPerLane];  // elements lane + 32 k; x and y of the row that is next
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        dw[k] = 0.f;
        w[k] = r.first < r.end && lane + 32 * k < dim ? load_element(static_cast<const T*>(s.weight) + lane + 32 * k) : 0.f;
    }
    uint32_t token = static_cast<uint32_t>(r.first / s.heads), batch = divide(token, a.by_tokens), at = token - batch * a.tokens;
    int head = static_cast<int>(r.first - static_cast<int64_t>(token) * s.heads);
    const auto load = [&] {
        const T* yp = static_cast<const T*>(s.dy) + batch * s.dy_batch + at * s.dy_token + head * s.dy_head;
        const T* xp = static_cast<const T*>(s.x) + batch * s.x_batch + at * s.x_token + head * s.x_head;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
            const int i = lane + 32 * k;
            x[k] = i < dim ? load_element(xp + i) : 0.f;
            y[k] = i < dim ? load_element(yp + i) : 0.f;
        }
    };
    if (r.first < r.end) load();
    bool fresh = true;  // a token's first row
    for (int64_t p = r.first; p < r.end; ++p) {
        T* dx = static_cast<T*>(s.dx) + batch * s.dx_batch + at * s.dx_token + head * s.dx_head;
        __syncwarp();
        if (fresh && pairs) fill_turns(table, a.rope, pairs, position_at(a.rope, batch, at), -1.f, lane, 32);
        float now[kPerLane];
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
            now[k] = x[k];
            if (lane + 32 * k < dim) g[lane + 32 * k] = y[k];
        }
        fresh = ++head == s.heads;
        if (fresh) {
            head = 0;
            batch = divide(++token, a.by_tokens), at = token - batch * a.tokens;
        }
        if (p + 1 < r.end) load();
        __syncwarp();
        if (pairs) {
            for (int q = lane; q < pairs; q += 32) {
                const int ia = a.rope.interleaved ? 2 * q : q, ib = a.rope.interleaved ? 2 * q + 1 : q + pairs;
                const float u = g[ia], v = g[ib], c = table[q], t = table[pairs + q];
                g[ia] = u * c - v * t;
                g[ib] = v * c + u * t;
            }
            __syncwarp();
        }
        float ss = 0.f, dot = 0.f, gk[kPerLane];
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
            gk[k] = lane + 32 * k < dim ? g[lane + 32 * k] : 0.f;
            ss += now[k] * now[k];
            dot += gk[k] * w[k] * now[k];
        }
        ss = sum_lanes<32>(ss, 32, lane);
        dot = sum_lanes<32>(dot, 32, lane);
        const float rstd = rsqrtf(ss / dim + a.eps), mean = dot * rstd / dim;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
            const float n = now[k] * rstd;
            dw[k] += gk[k] * n;
            if (lane + 32 * k < dim) store_element(dx + lane + 32 * k, rstd * (gk[k] * w[k] - n * mean));
        }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kPerLane; ++k)
        if (lane + 32 * k < dim) g[lane + 32 * k] = dw[k];
    leave_partials(staged, a.partials + static_cast<int64_t>(blockIdx.x) * dim, dim);
}

bool fits(const void* p, int64_t s0, int64_t s1, int64_t s2, int W) {
    return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && s0 % W == 0 && s1 % W == 0 && s2 % W == 0;
}

bool whole_vectors(const HeadsGradArgs& a, int W) {
    if (a.dim % W || (a.dim / W + 1) / 2 > 32 || a.rope.pairs % (a.rope.interleaved ? W / 2 : W)) return false;
    for (int i = 0; i < a.segments; ++i) {
        const HeadGradSegment& s = a.seg[i];
        if (!fits(s.dx, s.dx_batch, s.dx_token, s.dx_head, W) || !fits(s.dy, s.dy_batch, s.dy_token, s.dy_head, W) ||
            !fits(s.x, s.x_batch, s.x_token, s.x_head, W) || reinterpret_cast<uintptr_t>(s.weight) % 16)
            return false;
    }
    return true;
}

template <typename T, bool INTER>
cudaError_t launch_lanes(const HeadsGradArgs& a, int G, dim3 grid, cudaStream_t st) {
    const size_t smem = kStages * 4 * kWarps * 32 * sizeof(uint4) + kWarps * a.rope.pairs * sizeof(float2);
    const int own = own_lanes<Elem<T, INTER>::W>(a.dim);
#define NF_LANES(n) \
    if (own == n) return launch_args(heads_grad_rows<T, INTER, n>, grid, dim3(kWarps * 32), smem, st, a, n);
    if constexpr (sizeof(T) == 2) {
        NF_EACH_LANES_bf16(NF_LANES)
    } else {
        NF_EACH_LANES_f32(NF_LANES)
    }
#undef NF_LANES
    return launch_args(heads_grad_rows<T, INTER, 0>, grid, dim3(kWarps * 32), smem, st, a, G);
}

template <typename T>
cudaError_t launch_heads_grad_rows(HeadsGradArgs& a, int sms, cudaStream_t st) {
    constexpr int W = Elem<T, false>::W;
    const bool vectors = whole_vectors(a, W);
    const int G = vectors ? lanes_of<W>(a.dim) : 32, rows = 32 / G;
    a.by_tokens = Divider(a.tokens);
    // CTAs in proportion to the segments' work, two passes to a warp at least.
    int64_t work[2] = {0, 0}, passes = 0;
    for (int i = 0; i < a.segments; ++i) {
        const int64_t per_token = (a.seg[i].heads + rows - 1) / rows;
        passes += a.total * per_token;
        work[i] = a.total * (per_token + (vectors && a.rope.pairs ? kTurnPasses : 0));
    }
    const int64_t all = work[0] + work[1], most = static_cast<int64_t>(sms) * kCtasPerSm;
    const int64_t ctas = std::max<int64_t>(a.segments, std::min(most, (passes + 2 * kWarps - 1) / (2 * kWarps)));
    a.seg[0].ctas = static_cast<int>(ctas);
    if (a.segments == 2) {
        const int64_t share = all ? (ctas * work[1] + all / 2) / all : 1;
        a.seg[1].ctas = static_cast<int>(std::max<int64_t>(1, std::min(ctas - 1, share)));
        a.seg[0].ctas -= a.seg[1].ctas;
    }
    const dim3 grid(static_cast<unsigned>(ctas));
    if (!vectors) {
        const size_t smem = kWarps * (a.dim + 2 * a.rope.pairs) * sizeof(float);
        return a.dim <= 128 ? launch_with_pdl(heads_grad_elements<T, 4>, grid, dim3(kWarps * 32), smem, st, a)
                            : launch_with_pdl(heads_grad_elements<T, kHeadMaxDim / 32>, grid, dim3(kWarps * 32), smem, st, a);
    }
    return a.rope.interleaved ? launch_lanes<T, true>(a, G, grid, st) : launch_lanes<T, false>(a, G, grid, st);
}

}  // namespace
}  // namespace nf
