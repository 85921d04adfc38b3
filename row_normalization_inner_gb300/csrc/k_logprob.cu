// Log probabilities of given tokens, with entropy and top alternatives, and
// the gradient of both.
//
// Forward, per row of logits l at temperature T, with m = max l and
// d_j = (l_j - m) / T:
//     S = sum_j exp(d_j),  U = sum_j exp(d_j) d_j
//     logprob = d_t - log S,   entropy = log S - U / S,   stats = (m, log S)
// and the `top` largest logits, a tie going to the lower index.  One pass
// over the row: a thread keeps a running maximum and rescales its sums where
// it grows; powers of two stand for powers of e (d in units of ln 2).  d is
// the difference first and the product after, so that its error is relative
// to d itself.  S is an fp32 sum and log S is off by S's relative error, 1e-7
// to 1e-5 with the row's length and spread: a log probability nearer to 0 than
// that has no digits of its own (and where all else adds less than 2^-24, is 0).
//
// Bound by memory: the logits are read once (8192 x 131072 bf16 on a GB300
// 303 us, 7.1 TB/s; 16 x 131072 4.4 us, with 5 alternatives 7.5 us: latency).
// A row belongs to a CTA, or, where there are few rows, to a cluster of 2, 4
// or 8 CTAs that join their sums through distributed shared memory.
//
// The alternatives need no second pass: the sums need the maximum of every
// batch of vectors anyway, so each thread leaves the maxima of up to kSlots
// stretches of its elements in shared memory.  The top-th largest of the
// threads' maxima is a lower bound for the alternatives; only the stretches
// that reach it (little more than `top` of them) are read again, from L2,
// and what reaches the bound there is sorted as 64-bit keys (value, then
// index from the end), all distinct.  Reading all elements of the threads
// that reach the bound instead took 85 us more at 4096 x 131072 with 20
// alternatives.
//
// Backward: with p_j = exp(d_j - log S),
//     dl_j = ( g (1[j = t] - p_j) - h p_j (log p_j + H) ) / T
// for gradients g of logprob and h of entropy (H): one read, one write.
#include <cfloat>

#include <cooperative_groups.h>

#include "common.cuh"
#include "pairs.cuh"
#include "pdl.cuh"
#include "tokens.h"

namespace nf {
namespace {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// d is held at this or above: a power of two of it is 0, and its product
// with 0 is 0 where that of -infinity would be NaN
constexpr float kLowest = -16384.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max(x, kLowest), a NaN staying NaN.
__device__ __forceinline__ float hold(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(kLowest));
    return y;
}

// Element access of a 16-byte vector of bf16 or fp32 logits.
template <bool F32> struct Elem;
template <> struct Elem<false> {
    static constexpr int N = 8;
    using T = uint16_t;
    static constexpr uint32_t kNone = 0xFF80FF80u;  // -infinity in every element
    static __device__ __forceinline__ void unpack(uint4 v, float2 (&f)[4]) { unpack8x2(v, f); }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[4]) { return pack8x2(f); }
    // the largest element of N vectors (a NaN is passed over)
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&v)[N]) {
        __nv_bfloat162 m = max2(max2(as2(v[0].x), as2(v[0].y)), max2(as2(v[0].z), as2(v[0].w)));
#pragma unroll
        for (int k = 1; k < N; ++k)
            m = max2(m, max2(max2(as2(v[k].x), as2(v[k].y)), max2(as2(v[k].z), as2(v[k].w))));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ __nv_bfloat162 as2(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
    static __device__ __forceinline__ __nv_bfloat162 max2(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmax2(a, b); }
    static __device__ __forceinline__ float value(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
    static __device__ __forceinline__ uint16_t bits(float f) { return static_cast<uint16_t>(pack2(f, 0.f)); }
};
template <> struct Elem<true> {
    static constexpr int N = 4;
    using T = float;
    static constexpr uint32_t kNone = 0xFF800000u;
    static __device__ __forceinline__ void unpack(uint4 v, float2 (&f)[2]) {
        f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[2]) {
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                          __float_as_uint(f[1].y));
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&v)[N]) {
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < N; ++k)
            m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(v[k].x)), fmaxf(__uint_as_float(v[k].y), __uint_as_float(v[k].z))),
                      __uint_as_float(v[k].w));
        return m;
    }
    static __device__ __forceinline__ float value(float f) { return f; }
    static __device__ __forceinline__ float bits(float f) { return f; }
};

// A row of `n` elements that starts anywhere, as 16-byte vectors counted from
// the boundary at or below its start: element j is element j + lead of the
// vectors.  Only the first and the last vector can be partial; their missing
// elements are neither read nor written.
template <bool F32>
struct Row {
    using E = Elem<F32>;
    using T = typename E::T;
    const T* base;  // of element 0
    int lead;
    int n;
    __device__ __forceinline__ Row(const void* p, int64_t offset, int n_) {
        base = static_cast<const T*>(p) + offset;
        lead = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(T));
        n = n_;
    }
    __device__ __forceinline__ int vectors() const { return (lead + n + E::N - 1) / E::N; }
    __device__ __forceinline__ bool full(int v) const { return v * E::N >= lead && (v + 1) * E::N <= lead + n; }
    __device__ __forceinline__ uint4 load(int v) const {
        const int j0 = v * E::N - lead;
        if (full(v)) return ld_stream(base + j0);
        uint4 r = make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
        T* e = reinterpret_cast<T*>(&r);
#pragma unroll
        for (int k = 0; k < E::N; ++k)
            if (j0 + k >= 0 && j0 + k < n) e[k] = base[j0 + k];
        return r;
    }
};

// ---- forward ---------------------------------------------------------------------
constexpr int kFwdMaxThreads = 256;
// Resident CTAs per SM.  Five, at 48 registers, keep more of the row's bytes in
// flight (8192 x 131072 bf16: 303 us, four 319 us); with the alternatives, and
// in fp32 (half the arithmetic per byte), four at 64 registers were faster
// (4096 x 131072 bf16 with 20 alternatives 191 against 211 us, 1000 x 100003
// fp32 66 against 71 us).
constexpr int fwd_min_ctas(bool f32, bool top) { return f32 || top ? 4 : 5; }
constexpr int kFwdBatch = 4;   // vectors in flight per thread
constexpr int kTopMax = kLogprobMaxTop;

// An order-preserving integer of a float, and back.  Zeros of both signs are
// equal logits (and the running maximum, a comparison of values, keeps
// whichever came first), so both stand as +0, which adding +0 makes of them.
__device__ __forceinline__ uint32_t order_of(float f) {
    const uint32_t b = __float_as_uint(f + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ float key_value(uint64_t key) { return float_of(static_cast<uint32_t>(key >> 32)); }
__device__ __forceinline__ int key_index(uint64_t key) { return static_cast<int>(~static_cast<uint32_t>(key)); }

// Sums of exponentials of d (units of ln 2) below the maximum m.
struct Part {
    float m, s, u;
};

// The running sums of a thread.
struct Sums {
    float m;
    float2 s, u;
};

// Adds a batch of vectors.  Without HOLD an entry of -infinity (or one so far
// below the maximum that their difference overflows) turns u into NaN, by
// 0 * -infinity, and is found that way: testing every entry costs more than
// the rest of its arithmetic allows.
template <bool F32, bool HOLD, int N>
__device__ __forceinline__ void add_batch(Sums& p, const uint4 (&raw)[N], float c) {
    using E = Elem<F32>;
    const float2 nm = make_float2(-p.m, -p.m), c2 = make_float2(c, c);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float2 f[E::N / 2];
        E::unpack(raw[k], f);
#pragma unroll
        for (int q = 0; q < E::N / 2; ++q) {
            float2 d = __fmul2_rn(__fadd2_rn(f[q], nm), c2);
            if constexpr (HOLD) d = make_float2(hold(d.x), hold(d.y));
            const float2 e = make_float2(ex2(d.x), ex2(d.y));
            p.s = __fadd2_rn(p.s, e);
            p.u = __ffma2_rn(e, d, p.u);
        }
    }
}

// The batch's largest element.
template <bool F32, int N>
__device__ __forceinline__ float take_batch(Sums& p, const uint4 (&raw)[N], float c, bool& masked) {
    const float top = Elem<F32>::template largest<N>(raw);
    if (top > p.m) {
        const float d = hold((p.m - top) * c), g = ex2(d);
        const float2 d2 = make_float2(d, d), g2 = make_float2(g, g);
        p.u = __fmul2_rn(g2, __ffma2_rn(p.s, d2, p.u));
        p.s = __fmul2_rn(p.s, g2);
        p.m = top;
    }
    const Sums before = p;
    if (!masked) {
        add_batch<F32, false, N>(p, raw, c);
        masked = isnan(p.u.x + p.u.y);  // from here on this thread's row is taken with HOLD
        if (!masked) return top;
        p = before;
    }
    add_batch<F32, true, N>(p, raw, c);
    return top;
}

// p with the maximum m.
__device__ __forceinline__ Part rebase(Part p, float m, float c) {
    const float d = hold((p.m - m) * c), f = ex2(d);
    return Part{m, p.s * f, f * (p.u + p.s * d)};
}

// The warp's sums, in a fixed order, in every lane.
__device__ __forceinline__ Part warp_join(Part p, float c) {
    p = rebase(p, float_of(__reduce_max_sync(0xFFFFFFFFu, order_of(p.m))), c);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        p.s += __shfl_xor_sync(0xFFFFFFFFu, p.s, off);
        p.u += __shfl_xor_sync(0xFFFFFFFFu, p.u, off);
    }
    return p;
}

constexpr int kSlots = 16;
// The shared memory of the alternatives, laid out for T threads and `slots`
// stretches of each (rows of one batch need one, and more CTAs then fit).
struct TopShared {
    uint64_t* best;        // [kTopMax]
    uint64_t* cand;        // [capacity]: one round's candidates and those kept
    uint32_t* thread_max;  // [T], as order_of()
    float* slot;           // [slots][T]: largest element of each stretch
    uint16_t* list;        // [slots * T]: the stretches that reach the bound, slot * T + thread
    int *n_cand, *n_list;
    uint32_t* bound;
    int capacity;
    static constexpr __host__ __device__ int room(int threads, int per_vector) { return threads * per_vector + kTopMax; }
    static constexpr __host__ __device__ size_t bytes(int threads, int per_vector, int slots) {
        return 16 + 8 * (kTopMax + room(threads, per_vector)) + 4 * threads + 6 * slots * threads;
    }
    __device__ __forceinline__ TopShared(unsigned char* at, int threads, int per_vector, int slots) {
        n_cand = reinterpret_cast<int*>(at);
        n_list = n_cand + 1;
        bound = reinterpret_cast<uint32_t*>(n_cand + 2);
        capacity = room(threads, per_vector);
        best = reinterpret_cast<uint64_t*>(at + 16);
        cand = best + kTopMax;
        thread_max = reinterpret_cast<uint32_t*>(cand + capacity);
        slot = reinterpret_cast<float*>(thread_max + threads);
        list = reinterpret_cast<uint16_t*>(slot + slots * threads);
    }
};

// The elements of vector v that reach `low`, as keys, to the candidates;
// n_cand counts those that do not fit too.
template <bool F32>
__device__ __forceinline__ void push_top(const TopShared& sh, const Row<F32>& r, int v, uint4 raw, uint64_t low) {
    using E = Elem<F32>;
    float2 f[E::N / 2];
    E::unpack(raw, f);
    const int j0 = v * E::N - r.lead;
    const auto key_of = [&](int q) {
        return (static_cast<uint64_t>(order_of(q & 1 ? f[q / 2].y : f[q / 2].x)) << 32) | ~static_cast<uint32_t>(j0 + q);
    };
    // one addition for the vector: those of a row of equal elements come one after the other
    uint32_t reach = 0;
#pragma unroll
    for (int q = 0; q < E::N; ++q)
        reach |= static_cast<uint32_t>((q & 1 ? f[q / 2].y : f[q / 2].x) > -INFINITY && key_of(q) >= low) << q;
    if (reach == 0) return;
    int at = atomicAdd(sh.n_cand, __popc(reach));
#pragma unroll
    for (int q = 0; q < E::N; ++q) {
        if (!((reach >> q) & 1)) continue;
        if (at < sh.capacity) sh.cand[at] = key_of(q);
        ++at;
    }
}

// The `top` largest of cand[0, n), sorted, to best (0 where there are fewer).
// Every thread calls; synchronized on return.
__device__ __forceinline__ void sort_top(uint64_t* cand, int n, int top, uint64_t* best, int* n_kept) {
    const int t = threadIdx.x, T = blockDim.x;
    if (n > 256) {
        // the top-th largest key (they are distinct) bit by bit below the bits
        // that all share, then only what reaches it
        __shared__ int part[2][kFwdMaxThreads / 32];
        __shared__ uint2 differ[kFwdMaxThreads / 32];
        const int lane = t & 31, warp = t >> 5, warps = T >> 5;
        const uint64_t one = cand[0];
        uint64_t d = 0;
        for (int i = t; i < n; i += T) d |= cand[i] ^ one;
        const uint32_t hi = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(d >> 32));
        const uint32_t lo = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(d));
        if (lane == 0) differ[warp] = make_uint2(hi, lo);
        __syncthreads();
        const uint2 mine_d = lane < warps ? differ[lane] : make_uint2(0, 0);
        d = static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, mine_d.x)) << 32 | __reduce_or_sync(0xFFFFFFFFu, mine_d.y);
        const int first = 63 - __clzll(static_cast<long long>(d));
        uint64_t bound = first == 63 ? 0 : one >> (first + 1) << (first + 1);
        for (int b = first; b >= 0; --b) {
            const uint64_t test = bound | (1ull << b);
            int mine = 0;
            for (int i = t; i < n; i += T) mine += cand[i] >= test;
            mine = __reduce_add_sync(0xFFFFFFFFu, mine);
            if (lane == 0) part[b & 1][warp] = mine;
            __syncthreads();
            if (static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, lane < warps ? part[b & 1][lane] : 0)) >= top) bound = test;
        }
        // at most 9 of a thread's: n <= 8 T + kTopMax
        constexpr int kEach = 9;
        uint64_t keep[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) keep[k] = t + k * T < n && cand[t + k * T] >= bound ? cand[t + k * T] : 0;
        if (t == 0) *n_kept = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (keep[k]) cand[atomicAdd(n_kept, 1)] = keep[k];
        __syncthreads();
        n = *n_kept;
    }
    if (t < top) best[t] = 0;
    __syncthreads();
    for (int i = t; i < n; i += T) {
        const uint64_t key = cand[i];
        int above = 0;
        for (int k = 0; k < n; ++k) above += cand[k] > key;
        if (above < top) best[above] = key;
    }
    __syncthreads();
}

struct LogprobFwd {
    float* logprob;
    float* entropy;
    float2* stats;
    float* top_logprob;
    int64_t* top_ids;
    const void* logits;
    const void* targets;
    int64_t rows, stride;
    int vocab, top;
    float inv_t;
    int slots;  // of the alternatives' shared memory
    bool wide;
};

__device__ __forceinline__ int64_t target_at(const void* ids, bool wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

template <bool F32, bool TOP, bool CLUSTER>
__global__ void __launch_bounds__(kFwdMaxThreads, fwd_min_ctas(F32, TOP))
token_logprob_rows(const LogprobFwd a) {
    using E = Elem<F32>;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Part warps[kFwdMaxThreads / 32];
    __shared__ Part mine;
    const int t = threadIdx.x, T = blockDim.x, lane = t & 31, warp = t >> 5;
    const TopShared sh(smem, T, E::N, a.slots);  // only with TOP
    int ctas = 1, rank = 0;
    if constexpr (CLUSTER) {
        ctas = cg::this_cluster().num_blocks();
        rank = cg::this_cluster().block_rank();
    }
    const float c = a.inv_t * kLog2e;
    grid_dep_wait();
    grid_dep_release();
    for (int64_t row = blockIdx.x / ctas; row < a.rows; row += gridDim.x / ctas) {
        const Row<F32> r(a.logits, row * a.stride, a.vocab);
        const int nv = r.vectors();
        const int per = (nv + ctas - 1) / ctas;
        const int v0 = min(nv, rank * per), v1 = min(nv, v0 + per);
        // the thread's elements: vectors v0 + t + i * T
        Sums sums = {-FLT_MAX, make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        bool masked = false;
        // whole vectors are [f0, f1); a thread's first is v0 + t, or one step
        // on where that is the row's partial first vector
        const int f0 = v0 + (v0 < v1 && !r.full(v0)), f1 = v1 - (v1 > f0 && !r.full(v1 - 1));
        const auto first_of = [&](int thread) { return v0 + thread < f0 ? v0 + thread + T : v0 + thread; };
        const bool short_row = v1 - v0 <= kFwdBatch * T;  // one batch per thread, the partial vectors with it
        int shift = 0;                                    // batches per slot, as a power of two
        while ((v1 - v0) / (kFwdBatch * T) >> shift >= kSlots) ++shift;
        int slots = 0;
        if (short_row) {
            uint4 raw[kFwdBatch];
#pragma unroll
            for (int k = 0; k < kFwdBatch; ++k)
                raw[k] = v0 + t + k * T < v1 ? r.load(v0 + t + k * T) : make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
            masked = true;
            const float top = take_batch<F32, kFwdBatch>(sums, raw, c, masked);
            if constexpr (TOP) sh.slot[t] = top;
            slots = 1;
        } else {
            const uint4* src = reinterpret_cast<const uint4*>(r.base - r.lead);
            int v = first_of(t), batch = 0;
            float most = -INFINITY;
            for (; v + (kFwdBatch - 1) * T < f1; v += kFwdBatch * T) {
                uint4 raw[kFwdBatch];
#pragma unroll
                for (int k = 0; k < kFwdBatch; ++k) raw[k] = ld_stream(src + v + k * T);
                const float top = take_batch<F32, kFwdBatch>(sums, raw, c, masked);
                if constexpr (TOP) {
                    most = fmaxf(most, top);
                    ++batch;
                    if ((batch & ((1 << shift) - 1)) == 0) {
                        sh.slot[slots++ * T + t] = most;
                        most = -INFINITY;
                    }
                }
            }
            if (v < f1) {
                uint4 raw[kFwdBatch];
#pragma unroll
                for (int k = 0; k < kFwdBatch; ++k)
                    raw[k] = v + k * T < f1 ? ld_stream(src + v + k * T) : make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
                masked = true;  // the filling
                most = fmaxf(most, take_batch<F32, kFwdBatch>(sums, raw, c, masked));
                ++batch;
            }
            if constexpr (TOP) {
                if (slots << shift < batch) sh.slot[slots++ * T + t] = most;
            }
            if ((t == 0 && v0 < f0) || (f1 < v1 && t == (v1 - 1 - v0) % T)) {
                uint4 raw[2];
                raw[0] = raw[1] = make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
                if (t == 0 && v0 < f0) raw[0] = r.load(v0);
                if (f1 < v1 && t == (v1 - 1 - v0) % T) raw[1] = r.load(v1 - 1);
                masked = true;
                take_batch<F32, 2>(sums, raw, c, masked);
            }
        }
        // warp, then CTA, then cluster, each in a fixed order
        Part p = warp_join(Part{sums.m, sums.s.x + sums.s.y, sums.u.x + sums.u.y}, c);
        if (lane == 0) warps[warp] = p;
        const uint32_t ord = order_of(sums.m);
        if constexpr (TOP) {
            sh.thread_max[t] = ord;
            if (t == 0) *sh.n_list = *sh.n_cand = 0;
        }
        __syncthreads();
        if (warp == 0) {
            p = warp_join(lane < T / 32 ? warps[lane] : Part{-FLT_MAX, 0.f, 0.f}, c);
            if (lane == 0) mine = p;
        }
        if constexpr (TOP) {
            if (warp == T / 32 - 1) {
                // A bound that `top` threads' maxima reach, bit by bit below the
                // bits that all maxima share; a few more than `top` will do.
                constexpr int kEach = kFwdMaxThreads / 32;
                uint32_t x[kEach];
                uint32_t least = 0xFFFFFFFFu, most = 0;
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    x[i] = i * 32 < T ? sh.thread_max[i * 32 + lane] : 0;
                    if (i * 32 < T) least = min(least, x[i]);
                    most = max(most, x[i]);
                }
                least = __reduce_min_sync(0xFFFFFFFFu, least);
                most = __reduce_max_sync(0xFFFFFFFFu, most);
                uint32_t bound = least;
                if (least != most) {
                    int bit = 31 - __clz(least ^ most);
                    bound = bit == 31 ? 0 : most >> (bit + 1) << (bit + 1);
                    for (; bit >= 0; --bit) {
                        const uint32_t test = bound | (1u << bit);
                        int n = 0;
#pragma unroll
                        for (int i = 0; i < kEach; ++i) n += x[i] >= test;
                        n = __reduce_add_sync(0xFFFFFFFFu, n);
                        if (n < a.top) continue;
                        bound = test;
                        if (n <= a.top + 8) break;
                    }
                }
                if (lane == 0) *sh.bound = bound;
            }
            __syncthreads();
            const uint32_t bound = *sh.bound;
            if (ord >= bound) {
                int reach = 0;
                for (int i = 0; i < slots; ++i) reach += order_of(sh.slot[i * T + t]) >= bound;
                int at = reach ? atomicAdd(sh.n_list, reach) : 0;
                for (int i = 0; i < slots; ++i)
                    if (order_of(sh.slot[i * T + t]) >= bound) sh.list[at++] = static_cast<uint16_t>(i * T + t);
            }
            __syncthreads();
            // read these stretches again, and the partial vectors
            const int edges = short_row ? 0 : (v0 < f0) + (f1 < v1);
            const int per_log = shift + 2;  // vectors of a stretch
            static_assert(kFwdBatch == 4, "per_log");
            const int items = (*sh.n_list << per_log) + edges;
            uint64_t low = static_cast<uint64_t>(bound) << 32;  // keys below are out
            const auto vector_of = [&](int i) {  // v1: none
                if (i < edges) return i == 0 && v0 < f0 ? v0 : v1 - 1;
                if (i >= items) return v1;
                i -= edges;
                const int code = sh.list[i >> per_log], slot = code / T, thread = code - slot * T;
                const int v = (short_row ? v0 + thread : first_of(thread)) + ((slot << per_log) + (i & ((1 << per_log) - 1))) * T;
                return v < (short_row ? v1 : f1) ? v : v1;
            };
            for (int i0 = t; i0 < items; i0 += T) {
                if (*const_cast<volatile int*>(sh.n_cand) > sh.capacity) break;  // the rounds below will do it
                const int v = vector_of(i0);
                if (v < v1) push_top<F32>(sh, r, v, r.load(v), low);
            }
            __syncthreads();
            int n = *sh.n_cand;
            __syncthreads();
            if (n <= sh.capacity) {
                sort_top(sh.cand, n, a.top, sh.best, sh.n_cand);
            } else {
                // more than fit (many equal elements): again in rounds, keeping
                // the best of each
                if (t == 0) *sh.n_cand = 0;
                for (int i0 = 0; i0 < items; i0 += T) {
                    __syncthreads();
                    const int v = vector_of(i0 + t);
                    if (v < v1) push_top<F32>(sh, r, v, r.load(v), low);
                    __syncthreads();
                    n = *sh.n_cand;
                    const bool last = i0 + T >= items;
                    if (last || n + T * E::N > sh.capacity) {  // the next round might not fit
                        __syncthreads();
                        sort_top(sh.cand, n, a.top, sh.best, sh.n_cand);
                        const int kept = min(n, a.top);
                        if (t < kept) sh.cand[t] = sh.best[t];
                        if (kept == a.top) low = max(low, sh.best[a.top - 1]);
                        if (t == 0) *sh.n_cand = kept;
                    }
                }
                __syncthreads();
            }
        } else {
            __syncthreads();
        }
        Part all = mine;
        if constexpr (CLUSTER) {
            cg::cluster_group cluster = cg::this_cluster();
            cluster.sync();
            if (rank == 0) {
                // every warp: lane i takes CTA i's sums
                all = warp_join(lane < ctas ? *cluster.map_shared_rank(&mine, lane) : Part{-FLT_MAX, 0.f, 0.f}, c);
                if constexpr (TOP) {
                    for (int i = t; i < ctas * a.top; i += T)
                        sh.cand[i] = cluster.map_shared_rank(sh.best, i / a.top)[i % a.top];
                }
            }
            cluster.sync();  // the other CTAs' shared memory has been read
            if constexpr (TOP) {
                // ranks of missing alternatives (key 0) lie behind all others
                if (rank == 0) sort_top(sh.cand, ctas * a.top, a.top, sh.best, sh.n_cand);
            }
        }
        if (rank == 0) {
            const bool none = all.s == 0.f;   // every entry masked
            const bool bad = isnan(all.s);
            const float log_s = logf(all.s);  // -infinity where none
            if (t == 0) {
                const int64_t target = target_at(a.targets, a.wide, row);
                float lp = 0.f;
                if (target >= 0 && target < a.vocab)
                    lp = none ? -INFINITY : (E::value(r.base[target]) - all.m) * a.inv_t - log_s;
                a.logprob[row] = bad ? all.s : lp;
                a.entropy[row] = none ? 0.f : log_s - kLn2 * (all.u / all.s);
                a.stats[row] = make_float2(none ? -INFINITY : all.m, log_s);
            }
            if constexpr (TOP) {
                if (t < a.top) {
                    const uint64_t key = sh.best[t];
                    a.top_logprob[row * a.top + t] =
                        bad ? all.s : key ? (key_value(key) - all.m) * a.inv_t - log_s : -INFINITY;
                    a.top_ids[row * a.top + t] = key && !bad ? key_index(key) : -1;
                }
            }
        }
        __syncthreads();  // the shared memory is reused by the next row
    }
}

// ---- backward --------------------------------------------------------------------
// Two forms.  The largest calls give a CTA of 256 threads kBwdSpan batches of
// a row in turn (4096 x 131072 bf16, launches one after the other: 317 us;
// with a CTA per batch 334 us), all others a batch to a CTA of 128 threads
// (2048 x 131072: 159 against 162 us; 300 x 32003 fp32 in a graph: 10.4
// against 12.6 us).  Both keep 1536 threads of 40 registers on an SM (four
// CTAs of 256 threads at 52 registers: 343 us).
constexpr int kBwdBatch = 4;
constexpr int kBwdSpan = 4;
constexpr int64_t kBwdMinWork = 10000;  // CTAs with a span each
constexpr int bwd_threads(bool spans) { return spans ? 256 : 128; }

struct LogprobBwd {
    void* out;
    const void* logits;
    const void* targets;
    const float2* stats;
    const float* entropy;
    const float* d_logprob;
    const float* d_entropy;  // or null
    int64_t rows, stride, out_stride;
    int vocab, chunks;       // stretches of a row, a CTA each
    float inv_t;
    bool wide;
};

template <bool F32, bool SPANS>
__global__ void __launch_bounds__(bwd_threads(SPANS), 1536 / bwd_threads(SPANS))
token_logprob_grad(const LogprobBwd a) {
    using E = Elem<F32>;
    using T = typename E::T;
    grid_dep_wait();
    grid_dep_release();
    const int threads = blockDim.x;
    const int64_t work = a.rows * a.chunks;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int64_t row = w / a.chunks;
        const int chunk = static_cast<int>(w - row * a.chunks);
        const Row<F32> r(a.logits, row * a.stride, a.vocab);
        T* out = static_cast<T*>(a.out) + row * a.out_stride;
        const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(r.base) & 15);
        const int nv = r.vectors();
        const float2 st = a.stats[row];
        const int64_t target = target_at(a.targets, a.wide, row);
        const bool none = st.x == -INFINITY;  // a row without entries: its gradient is 0
        const bool known = target >= 0 && target < a.vocab && !none;
        const float g = known ? a.d_logprob[row] : 0.f;
        const float h = a.d_entropy && !none ? a.d_entropy[row] : 0.f;
        const float m = none ? 0.f : st.x, log2_s = none ? 0.f : st.y * kLog2e;
        // dl = p (A + B log2 p), p = 2^(log2 p)
        const float A = -a.inv_t * (h != 0.f ? fmaf(h, a.entropy[row], g) : g);
        const float B = -a.inv_t * h * kLn2;
        const float c = a.inv_t * kLog2e;
        const float2 c2 = make_float2(c, c), nm = make_float2(-m, -m), ns = make_float2(-log2_s, -log2_s);
        const float2 A2 = make_float2(A, A), B2 = make_float2(B, B);
        const auto batch = [&](int first) {
            uint4 raw[kBwdBatch];
#pragma unroll
            for (int k = 0; k < kBwdBatch; ++k)
                if (first + k * threads < nv) raw[k] = r.load(first + k * threads);
#pragma unroll
            for (int k = 0; k < kBwdBatch; ++k) {
                const int v = first + k * threads;
                if (v >= nv) continue;
                const int j0 = v * E::N - r.lead;
                float2 f[E::N / 2];
                E::unpack(raw[k], f);
#pragma unroll
                for (int q = 0; q < E::N / 2; ++q) {
                    float2 d = __fadd2_rn(__fmul2_rn(__fadd2_rn(f[q], nm), c2), ns);
                    d = make_float2(hold(d.x), hold(d.y));
                    const float2 p = make_float2(ex2(d.x), ex2(d.y));
                    f[q] = __fmul2_rn(p, __ffma2_rn(B2, d, A2));
                }
                if (known && target >= j0 && target < j0 + E::N) {
                    const int at = static_cast<int>(target - j0);
#pragma unroll
                    for (int q = 0; q < E::N / 2; ++q) {
                        if (at == 2 * q) f[q].x = fmaf(g, a.inv_t, f[q].x);
                        if (at == 2 * q + 1) f[q].y = fmaf(g, a.inv_t, f[q].y);
                    }
                }
                if (same && r.full(v)) {
                    st_stream(out + j0, E::pack(f));
                } else {
#pragma unroll
                    for (int q = 0; q < E::N; ++q)
                        if (j0 + q >= 0 && j0 + q < a.vocab) out[j0 + q] = E::bits(q & 1 ? f[q / 2].y : f[q / 2].x);
                }
            }
        };
        const int step = threads * kBwdBatch;
        if constexpr (SPANS) {
            const int64_t begin = static_cast<int64_t>(chunk) * kBwdSpan * step;
            const int end = static_cast<int>(begin + kBwdSpan * step < nv ? begin + kBwdSpan * step : nv);
            for (int first = static_cast<int>(begin) + threadIdx.x; first < end; first += step) batch(first);
        } else {
            batch(chunk * step + threadIdx.x);
        }
    }
}

template <bool F32, bool TOP, bool CLUSTER>
cudaError_t fwd(const LogprobFwd& a, int threads, int ctas, cudaStream_t st) {
    const auto k = token_logprob_rows<F32, TOP, CLUSTER>;
    constexpr int n = Elem<F32>::N;
    static_assert(TopShared::bytes(kFwdMaxThreads, 8, kSlots) <= 47 * 1024, "within the default limit of shared memory");
    const size_t smem = TOP ? TopShared::bytes(threads, n, a.slots) : 0;
    const int64_t most = 0x7FFFFFFF / ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.rows < most ? a.rows : most) * ctas));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <bool F32>
cudaError_t fwd(const LogprobFwd& a, int threads, int ctas, cudaStream_t st) {
    if (a.top) return ctas > 1 ? fwd<F32, true, true>(a, threads, ctas, st) : fwd<F32, true, false>(a, threads, ctas, st);
    return ctas > 1 ? fwd<F32, false, true>(a, threads, ctas, st) : fwd<F32, false, false>(a, threads, ctas, st);
}

}  // namespace

cudaError_t launch_token_logprob_fwd(float* logprob, float* entropy, float* stats, float* top_logprob,
                                     int64_t* top_ids, const void* logits, bool f32, const void* targets,
                                     bool wide, int64_t rows, int64_t vocab, int64_t stride, float temperature,
                                     int top, int sms, cudaStream_t st) {
    LogprobFwd a{};
    a.logprob = logprob;
    a.entropy = entropy;
    a.stats = reinterpret_cast<float2*>(stats);
    a.top_logprob = top_logprob;
    a.top_ids = top_ids;
    a.logits = logits;
    a.targets = targets;
    a.rows = rows;
    a.stride = stride;
    a.vocab = static_cast<int>(vocab);
    a.top = top;
    a.inv_t = 1.0f / temperature;
    a.wide = wide;
    const int64_t nv = vocab / (f32 ? 4 : 8) + 1;
    // Few rows: the largest CTA that has a batch per thread.  Where the rows
    // fill the GPU anyway, smaller CTAs, up to eight batches a thread (32
    // threads: four), so that more rows are in flight beside the one whose
    // sums are joined: 4096 x 1000 bf16 7.9 -> 4.7 us, with 5 alternatives
    // 20.1 -> 9.4 us; 4096 x 10000 25.8 -> 18.9 us; 256 x 32000 with 20
    // alternatives would go from 8.1 to 10.5 us.
    int threads = 32;
    if (rows >= 10 * static_cast<int64_t>(sms)) {
        while (threads < kFwdMaxThreads && nv > threads * kFwdBatch * (threads == 32 ? 4 : 8)) threads *= 2;
    } else {
        threads = 128;
        while (threads < kFwdMaxThreads && threads * kFwdBatch < nv) threads *= 2;
    }
    // Few rows: more CTAs per row, while two per SM leave each thread a vector,
    // or a full wave of them sixteen (160 x 131072 bf16 18.3 -> 11.9 us, 256 x
    // 131072 19.2 -> 17.7 us; beyond a wave it was slower: 350 x 131072 fp32
    // with 5 alternatives 38 -> 48 us).
    int ctas = 1;
    const int64_t wave = static_cast<int64_t>(fwd_min_ctas(f32, top != 0)) * sms;
    const auto fits = [&](int64_t c) {
        return (rows * c <= 2 * static_cast<int64_t>(sms) && nv >= c * threads) ||
               (rows * c <= wave && nv >= c * threads * 16);
    };
    while (ctas < 8 && fits(2 * ctas))
        ctas *= 2;
    // a row, or a CTA's share of one, of at most a batch per thread has one stretch (an unaligned row: one vector more)
    a.slots = (nv + 1 + ctas - 1) / ctas <= threads * kFwdBatch ? 1 : kSlots;
    return f32 ? fwd<true>(a, threads, ctas, st) : fwd<false>(a, threads, ctas, st);
}

cudaError_t launch_token_logprob_bwd(void* out, const void* logits, bool f32, const void* targets, bool wide,
                                     const float* stats, const float* entropy, const float* d_logprob,
                                     const float* d_entropy, int64_t rows, int64_t vocab, int64_t stride,
                                     int64_t out_stride, float temperature, cudaStream_t st) {
    LogprobBwd a{};
    a.out = out;
    a.logits = logits;
    a.targets = targets;
    a.stats = reinterpret_cast<const float2*>(stats);
    a.entropy = entropy;
    a.d_logprob = d_logprob;
    a.d_entropy = d_entropy;
    a.rows = rows;
    a.stride = stride;
    a.out_stride = out_stride;
    a.vocab = static_cast<int>(vocab);
    a.inv_t = 1.0f / temperature;
    a.wide = wide;
    const int n = f32 ? 4 : 8;
    // rows that do not all start on a 16-byte boundary can take one vector more
    const bool even = reinterpret_cast<uintptr_t>(logits) % 16 == 0 && (stride % n == 0 || rows == 1);
    const int64_t nv = (vocab + n - 1) / n + (even ? 0 : 1);
    const auto count = [nv](int64_t vectors) { return (nv + vectors - 1) / vectors; };
    const int64_t stretch = static_cast<int64_t>(bwd_threads(true)) * kBwdBatch * kBwdSpan;
    const bool spans = nv >= stretch && rows * count(stretch) >= kBwdMinWork;
    int threads = spans ? bwd_threads(true) : 32;
    while (threads < bwd_threads(false) && threads * kBwdBatch < nv) threads *= 2;
    a.chunks = static_cast<int>(count(spans ? stretch : threads * kBwdBatch));
    const int64_t work = rows * a.chunks;
    const dim3 grid(static_cast<unsigned>(work < 0x7FFFFFFF ? work : 0x7FFFFFFF));
    if (spans)
        return f32 ? launch_with_pdl(token_logprob_grad<true, true>, grid, dim3(threads), 0, st, a)
                   : launch_with_pdl(token_logprob_grad<false, true>, grid, dim3(threads), 0, st, a);
    return f32 ? launch_with_pdl(token_logprob_grad<true, false>, grid, dim3(threads), 0, st, a)
               : launch_with_pdl(token_logprob_grad<false, false>, grid, dim3(threads), 0, st, a);
}

}  // namespace nf
