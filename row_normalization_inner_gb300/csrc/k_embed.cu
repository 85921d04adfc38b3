// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: y[i] = bf16(scale * table[ids[i]]); an id outside [0, vocab)
// gives a row of zeros.  A gather of rows, bound by memory: 2 bytes read
// (once per distinct id) and 2 written per element.
//
// Backward: dtable[v] (+)= scale * sum over { i : ids[i] = v } of dy[i].  The
// tokens are sorted by id, stably, so that equal ids become a run in token
// order; every run is summed in fp32 in that order, which makes the result
// deterministic where atomics on the table would not be.  Launches:
//   1. the sort: one CTA up to kSortOne tokens (every radix pass in shared
//      memory), above that two launches per radix pass (digit counts of each
//      tile, then a stable scatter whose CTAs each add up the counts of the
//      tiles before theirs);
//   2. the sums: the sorted tokens are cut into chunks of equal length, a CTA
//      per chunk and slice of columns.  A run inside one chunk is written at
//      once; the pieces of a run that crosses chunks go to the workspace.
//      Where the table's gradient is overwritten, further CTAs of the same
//      launch write zeros into the rows no token names;
//   3. the join: the pieces of each crossing run are added in order.
// A chunk rather than a run per CTA, because word frequencies are uneven:
// one id can hold several percent of a batch.  Bound by memory: dy read
// once, the rows with tokens (or all rows) written once.
#include <atomic>

#include "common.cuh"
#include "pairs.cuh"
#include "pdl.cuh"
#include "tokens.h"

namespace nf {
namespace {

__device__ __forceinline__ int64_t id_at(const void* ids, bool wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

// ---- forward -------------------------------------------------------------------
constexpr int kFwdThreads = 128;
constexpr int kFwdUnroll = 4;

// blockDim = (threads over a row's vectors, tokens of the CTA)
__global__ void __launch_bounds__(kFwdThreads)
embedding_rows(uint16_t* __restrict__ y, const void* __restrict__ ids, bool wide,
               const uint16_t* __restrict__ table, int64_t tokens, int64_t vocab, int nv, float scale) {
    grid_dep_wait();
    grid_dep_release();
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    const float2 s2 = make_float2(scale, scale);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; i < tokens; i += step) {
        const int64_t id = id_at(ids, wide, i);
        const bool known = id >= 0 && id < vocab;
        const uint16_t* row = table + (known ? id : 0) * nv * kVec;
        uint16_t* out = y + i * nv * kVec;
        for (int v0 = threadIdx.x; v0 < nv; v0 += kFwdUnroll * blockDim.x) {
            uint4 r[kFwdUnroll];
#pragma unroll
            for (int k = 0; k < kFwdUnroll; ++k) {
                const int v = v0 + k * blockDim.x;
                r[k] = make_uint4(0, 0, 0, 0);
                if (known && v < nv) r[k] = ld_param(row + v * kVec);
            }
#pragma unroll
            for (int k = 0; k < kFwdUnroll; ++k) {
                const int v = v0 + k * blockDim.x;
                if (v >= nv) continue;
                if (known) {
                    float2 f[4];
                    unpack8x2(r[k], f);
#pragma unroll
                    for (int q = 0; q < 4; ++q) f[q] = __fmul2_rn(f[q], s2);
                    r[k] = pack8x2(f);
                }
                st_stream(out + v * kVec, r[k]);
            }
        }
    }
}

// ---- the sort --------------------------------------------------------------------
// LSD radix sort of (id, token) pairs.  Ids outside [0, vocab) become the key
// `vocab`, which sorts behind every row of the table.
constexpr int kBins = 1024;  // digits of up to 10 bits
constexpr int kBinBits = 10;

__device__ __forceinline__ uint32_t key_of(const void* ids, bool wide, int64_t i, int64_t vocab) {
    const int64_t id = id_at(ids, wide, i);
    return static_cast<uint32_t>(id >= 0 && id < vocab ? id : vocab);
}

// Lanes of the warp whose digit is this lane's.
__device__ __forceinline__ uint32_t lanes_like(uint32_t digit) { return __match_any_sync(0xFFFFFFFFu, digit); }

// Stable ranks of a tile's digits (key >> shift) & (bins - 1).  Warp w holds
// the items [w * 32 * ITEMS, (w + 1) * 32 * ITEMS) of the tile, item k of a
// lane at k * 32 + lane; bit k of `valid` says whether the lane has it.
// counts: `bins` of each warp, zeroed here.  On return the low 16 bits of
// rank[k] are the number of items of the same digit before this one in its
// warp (the high 16 are kept), counts[w * bins + d] is the number of items of
// digit d in the warps before w, and total[d] the tile's items of digit d.
template <int THREADS, int ITEMS>
__device__ __forceinline__ void rank_tile(const uint32_t (&key)[ITEMS], uint32_t valid, int shift, int bins,
                                          uint16_t* counts, uint32_t* total, uint32_t (&rank)[ITEMS]) {
    constexpr int kWarps = THREADS / 32;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    uint32_t* words = reinterpret_cast<uint32_t*>(counts);
    for (int i = t; i < kWarps * bins / 2; i += THREADS) words[i] = 0;
    __syncthreads();
    uint16_t* mine = counts + warp * bins;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const bool have = (valid >> k) & 1;
        // lanes past the end match each other only
        const uint32_t d = have ? (key[k] >> shift) & (bins - 1) : kBins;
        const uint32_t like = lanes_like(d);
        const int before = __popc(like & ((1u << lane) - 1));
        const uint32_t c = have ? mine[d] : 0;
        __syncwarp();
        if (have && before == 0) mine[d] = static_cast<uint16_t>(c + __popc(like));
        __syncwarp();
        rank[k] = (rank[k] & 0xFFFF0000u) | (c + before);
    }
    __syncthreads();
    for (int d = t; d < bins; d += THREADS) {
        uint32_t sum = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t c = counts[w * bins + d];
            counts[w * bins + d] = static_cast<uint16_t>(sum);
            sum += c;
        }
        total[d] = sum;
    }
    __syncthreads();
}

// Exclusive prefix sum of bins <= 2 * THREADS values in shared memory, by the
// whole CTA.  The values must be visible on entry; synchronized on return.
template <int THREADS>
__device__ __forceinline__ void scan_bins(uint32_t* values, int bins, uint32_t* warp_sums) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const uint32_t a = 2 * t < bins ? values[2 * t] : 0, b = 2 * t + 1 < bins ? values[2 * t + 1] : 0;
    uint32_t run = a + b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, run, off);
        if (lane >= off) run += up;
    }
    if (lane == 31) warp_sums[warp] = run;
    __syncthreads();
    const uint32_t w = lane < warp ? warp_sums[lane] : 0;
    run += __reduce_add_sync(0xFFFFFFFFu, w);
    if (2 * t < bins) values[2 * t] = run - a - b;
    if (2 * t + 1 < bins) values[2 * t + 1] = run - b;
    __syncthreads();
}

// One CTA sorts all tokens: every pass in shared memory.  A thread holds
// ITEMS of them; small batches take the variant with the fewest.
constexpr int kSortOne = 16384;
template <int THREADS, int ITEMS>
constexpr size_t sort_one_smem(int bins) {
    return static_cast<size_t>(THREADS) * ITEMS * 6 + static_cast<size_t>(THREADS / 32) * bins * 2 + bins * 4 + 128;
}

template <int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS)
sort_one(const void* __restrict__ ids, bool wide, int n, int64_t vocab, int bits, int passes,
         uint32_t* __restrict__ keys_out, uint32_t* __restrict__ at_out) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int bins = 1 << bits;
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
    uint32_t* total = keys + THREADS * ITEMS;
    uint32_t* warp_sums = total + bins;
    uint16_t* at = reinterpret_cast<uint16_t*>(warp_sums + 32);  // at most kSortOne tokens: 16 bits
    uint16_t* counts = at + THREADS * ITEMS;
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t key[ITEMS], pr[ITEMS];  // pr: the token in the high 16 bits, its rank in the low
    uint32_t valid = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = (warp * ITEMS + k) * 32 + lane;
        const bool have = i < n;
        valid |= static_cast<uint32_t>(have) << k;
        key[k] = have ? key_of(ids, wide, i, vocab) : 0;
        pr[k] = static_cast<uint32_t>(i) << 16;
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * bits;
        rank_tile<THREADS, ITEMS>(key, valid, shift, bins, counts, total, pr);
        scan_bins<THREADS>(total, bins, warp_sums);
        const bool last = p == passes - 1;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            if (!((valid >> k) & 1)) continue;
            const uint32_t d = (key[k] >> shift) & (bins - 1);
            const uint32_t to = total[d] + counts[warp * bins + d] + (pr[k] & 0xFFFFu);
            if (last) {
                keys_out[to] = key[k];
                at_out[to] = pr[k] >> 16;
            } else {
                keys[to] = key[k];
                at[to] = static_cast<uint16_t>(pr[k] >> 16);
            }
        }
        if (last) break;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = (warp * ITEMS + k) * 32 + lane;
            if ((valid >> k) & 1) {
                key[k] = keys[i];
                pr[k] = static_cast<uint32_t>(at[i]) << 16;
            }
        }
    }
}

// Tiles of many-CTA sorts.
constexpr int kTileThreads = 512;
constexpr int kTileItems = 8;
constexpr int kTile = kTileThreads * kTileItems;  // 4096

__global__ void __launch_bounds__(kTileThreads)
sort_count(const void* __restrict__ ids, bool wide, const uint32_t* __restrict__ keys_in, int64_t n,
           int64_t vocab, int shift, int bits, uint32_t* __restrict__ hist) {
    __shared__ uint32_t bins[kBins];
    grid_dep_wait();
    grid_dep_release();
    for (int d = threadIdx.x; d < kBins; d += kTileThreads) bins[d] = 0;
    __syncthreads();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile;
#pragma unroll
    for (int k = 0; k < kTileItems; ++k) {
        const int64_t i = base + k * kTileThreads + threadIdx.x;
        const bool ok = i < n;
        const uint32_t key = !ok ? 0 : keys_in ? keys_in[i] : key_of(ids, wide, i, vocab);
        const uint32_t d = ok ? (key >> shift) & ((1u << bits) - 1) : kBins;
        // one addition per distinct digit of the warp
        const uint32_t like = lanes_like(d);
        if (ok && __popc(like & ((1u << (threadIdx.x & 31)) - 1)) == 0) atomicAdd(&bins[d], __popc(like));
    }
    __syncthreads();
    for (int d = threadIdx.x; d < 1 << bits; d += kTileThreads)
        hist[(static_cast<int64_t>(blockIdx.x) << bits) + d] = bins[d];
}

__global__ void __launch_bounds__(kTileThreads)
sort_scatter(const void* __restrict__ ids, bool wide, const uint32_t* __restrict__ keys_in,
             const uint32_t* __restrict__ at_in, int64_t n, int64_t vocab, int shift, int bits, int tiles,
             const uint32_t* __restrict__ hist, uint32_t* __restrict__ keys_out,
             uint32_t* __restrict__ at_out) {
    __shared__ __align__(4) uint16_t counts[kTileThreads / 32 * kBins];
    __shared__ uint32_t total[kBins], first[kBins], warp_sums[32];
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile;
    const int bins = 1 << bits;
    uint32_t key[kTileItems], pos[kTileItems], rank[kTileItems];
    uint32_t valid = 0;
#pragma unroll
    for (int k = 0; k < kTileItems; ++k) {
        const int64_t i = base + (warp * kTileItems + k) * 32 + lane;
        const bool have = i < n;
        valid |= static_cast<uint32_t>(have) << k;
        key[k] = !have ? 0 : keys_in ? keys_in[i] : key_of(ids, wide, i, vocab);
        pos[k] = !have ? 0 : at_in ? at_in[i] : static_cast<uint32_t>(i);
        rank[k] = 0;
    }
    rank_tile<kTileThreads, kTileItems>(key, valid, shift, bins, counts, total, rank);
    // all tiles' items of a digit, and those of the tiles before this one
    for (int d = threadIdx.x; d < bins; d += kTileThreads) {
        uint32_t all = 0, before = 0;
#pragma unroll 8
        for (int i = 0; i < tiles; ++i) {
            const uint32_t c = hist[static_cast<int64_t>(i) * bins + d];
            all += c;
            if (i < static_cast<int>(blockIdx.x)) before += c;
        }
        total[d] = all;
        first[d] = before;
    }
    __syncthreads();
    scan_bins<kTileThreads>(total, bins, warp_sums);
#pragma unroll
    for (int k = 0; k < kTileItems; ++k) {
        if (!((valid >> k) & 1)) continue;
        const uint32_t d = (key[k] >> shift) & (bins - 1);
        const uint32_t to = total[d] + first[d] + counts[warp * bins + d] + rank[k];
        keys_out[to] = key[k];
        at_out[to] = pos[k];
    }
}

// ---- the sums --------------------------------------------------------------------
constexpr int kSumThreads = 128;   // threads of a column slice, 8 columns each
constexpr int kSumBatch = 4;       // rows of dy in flight per thread
constexpr int kSumPart = 256;      // tokens whose ids and numbers are staged at once
constexpr int kZeroRows = 16;      // rows per CTA that writes zeros

struct EmbedBwd {
    void* dtable;
    const uint16_t* dy;
    const uint32_t* keys;
    const uint32_t* at;
    float* pieces;       // [chunks][2][hidden]: a chunk's first and last piece of a crossing run
    int64_t tokens, vocab;
    int hidden, chunk, slices;
    int64_t chunks;
    float scale;
};

// One table row's 8 columns: (old +) scale * acc.  The old values are loaded
// apart, so that a batch of rows has its loads in flight together.
template <bool F32, bool ADD>
struct Old {
    static constexpr int N = F32 ? 2 : 1;  // 16-byte vectors
    uint4 v[ADD ? N : 1];
    static __device__ __forceinline__ uint4* place(const EmbedBwd& a, uint32_t key, int col) {
        return static_cast<uint4*>(a.dtable) + (static_cast<int64_t>(key) * (a.hidden / kVec) + col) * N;
    }
    __device__ __forceinline__ void load(const EmbedBwd& a, uint32_t key, int col) {
        const uint4* p = place(a, key, col);
        if constexpr (ADD) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = ld_stream(p + i);
        }
    }
    __device__ __forceinline__ void put(const EmbedBwd& a, uint32_t key, int col, const float2 (&acc)[4]) const {
        const float2 s2 = make_float2(a.scale, a.scale);
        float2 o[4];
        if constexpr (ADD && F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                o[2 * i] = make_float2(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
                o[2 * i + 1] = make_float2(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
            }
        } else if constexpr (ADD) {
            unpack8x2(v[0], o);
        } else {
            o[0] = o[1] = o[2] = o[3] = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = __ffma2_rn(acc[q], s2, o[q]);
        uint4* p = place(a, key, col);
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                st_stream(p + i, make_uint4(__float_as_uint(o[2 * i].x), __float_as_uint(o[2 * i].y),
                                            __float_as_uint(o[2 * i + 1].x), __float_as_uint(o[2 * i + 1].y)));
        } else {
            st_stream(p, pack8x2(o));
        }
    }
};

__device__ __forceinline__ void put_piece(float* pieces, int v, const float2 (&acc)[4]) {
    float4* p = reinterpret_cast<float4*>(pieces + static_cast<int64_t>(v) * kVec);
    p[0] = make_float4(acc[0].x, acc[0].y, acc[1].x, acc[1].y);
    p[1] = make_float4(acc[2].x, acc[2].y, acc[3].x, acc[3].y);
}

// First sorted position whose key is >= want, by one warp: 32 probes a step.
__device__ __forceinline__ int64_t lower_bound_warp(const uint32_t* keys, int64_t lo, int64_t hi, uint32_t want) {
    const int lane = threadIdx.x & 31;
    while (lo < hi) {
        const int64_t len = hi - lo, step = (len + 31) / 32;
        const int64_t i = lo + lane * step;
        const bool below = i < hi && keys[i] < want;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, below));  // keys ascend: the first n lanes
        if (n == 0) return lo;
        const int64_t next = lo + n * step;
        lo = lo + (n - 1) * step + 1;
        hi = next < hi ? next : hi;
    }
    return lo;
}

// CTAs [0, chunks * slices): the sums.  CTAs above: zeros for the table's
// rows without tokens, kZeroRows each.
template <bool F32, bool ADD>
__global__ void __launch_bounds__(kSumThreads)
embedding_sums(const EmbedBwd a) {
    __shared__ uint32_t touched[kZeroRows];
    __shared__ uint32_t keys[kSumPart + kSumBatch], at[kSumPart];  // keys: one more than the part's
    __shared__ int64_t range[2];
    grid_dep_wait();
    grid_dep_release();
    const int nv = a.hidden / kVec;
    const int64_t work = a.chunks * a.slices;
    if (!ADD && static_cast<int64_t>(blockIdx.x) >= work) {
        const int64_t r0 = (static_cast<int64_t>(blockIdx.x) - work) * kZeroRows;
        const int64_t r1 = r0 + kZeroRows < a.vocab ? r0 + kZeroRows : a.vocab;
        if (threadIdx.x < kZeroRows) touched[threadIdx.x] = 0;
        if (threadIdx.x < 64) {
            const int64_t b = lower_bound_warp(a.keys, 0, a.tokens, static_cast<uint32_t>(threadIdx.x < 32 ? r0 : r1));
            if ((threadIdx.x & 31) == 0) range[threadIdx.x >> 5] = b;
        }
        __syncthreads();
        for (int64_t i = range[0] + threadIdx.x; i < range[1]; i += kSumThreads) touched[a.keys[i] - r0] = 1;
        __syncthreads();
        const int per = F32 ? nv * 2 : nv;  // 16-byte vectors of a row
        for (int r = 0; r < r1 - r0; ++r) {
            if (touched[r]) continue;
            uint4* p = static_cast<uint4*>(a.dtable) + (r0 + r) * per;
            for (int v = threadIdx.x; v < per; v += kSumThreads) __stcs(p + v, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    const int64_t c = static_cast<int64_t>(blockIdx.x) / a.slices;
    const int v = static_cast<int>(blockIdx.x % a.slices) * kSumThreads + threadIdx.x;
    const int64_t begin = c * a.chunk;
    const int64_t end = begin + a.chunk < a.tokens ? begin + a.chunk : a.tokens;
    const uint32_t none = static_cast<uint32_t>(a.vocab);
    const uint32_t before = begin > 0 ? a.keys[begin - 1] : none;
    const uint32_t first = a.keys[begin];
    float2 acc[4] = {};
    for (int64_t part = begin; part < end; part += kSumPart) {
        const int n = static_cast<int>(end - part < kSumPart ? end - part : kSumPart);
        __syncthreads();  // the part before this one has been read
        for (int i = threadIdx.x; i < kSumPart + kSumBatch; i += kSumThreads) {
            keys[i] = part + i < a.tokens && i <= n ? a.keys[part + i] : none;
            if (i < n) at[i] = a.at[part + i];
        }
        __syncthreads();
        if (v >= nv) continue;
        for (int i = 0; i < n; i += kSumBatch) {
            if (keys[i] == none) break;
            uint4 d[kSumBatch];
            Old<F32, ADD> old[kSumBatch];
#pragma unroll
            for (int k = 0; k < kSumBatch; ++k) {
                const uint32_t key = keys[i + k];
                if (i + k >= n || key == none) continue;
                d[k] = ld_stream(a.dy + (static_cast<int64_t>(at[i + k]) * nv + v) * kVec);
                if (ADD && keys[i + k + 1] != key && !(key == first && before == first)) old[k].load(a, key, v);
            }
#pragma unroll
            for (int k = 0; k < kSumBatch; ++k) {
                const uint32_t key = keys[i + k];
                if (i + k >= n || key == none) break;
                float2 f[4];
                unpack8x2(d[k], f);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[q] = __fadd2_rn(acc[q], f[q]);
                const bool head = key == first && before == first;  // the run began in an earlier chunk
                if (keys[i + k + 1] != key) {                       // and ends here
                    if (head) put_piece(a.pieces + c * 2 * a.hidden, v, acc);
                    else old[k].put(a, key, v, acc);
                    acc[0] = acc[1] = acc[2] = acc[3] = make_float2(0.f, 0.f);
                } else if (part + i + k + 1 == end) {               // it goes on in the next chunk
                    put_piece(a.pieces + (c * 2 + (head ? 0 : 1)) * a.hidden, v, acc);
                }
            }
        }
    }
}

// The runs that cross chunks: the chunk in which a run begins adds its last
// piece and the first pieces of the chunks the run goes on through, in order.
template <bool F32, bool ADD>
__global__ void __launch_bounds__(kSumThreads)
embedding_join(const EmbedBwd a) {
    __shared__ int64_t last;
    grid_dep_wait();
    grid_dep_release();
    const int nv = a.hidden / kVec;
    const int64_t c = static_cast<int64_t>(blockIdx.x) / a.slices;
    const int v = static_cast<int>(blockIdx.x % a.slices) * kSumThreads + threadIdx.x;
    const int64_t begin = c * a.chunk, end = begin + a.chunk;
    if (end >= a.tokens) return;
    const uint32_t key = a.keys[end - 1];
    if (key >= a.vocab || a.keys[end] != key) return;                       // no run goes on
    if (a.keys[begin] == key && begin > 0 && a.keys[begin - 1] == key) return;  // it began earlier
    if (threadIdx.x < 32) {
        const int64_t stop = lower_bound_warp(a.keys, end, a.tokens, key + 1);
        if (threadIdx.x == 0) last = (stop - 1) / a.chunk;  // the chunk of the run's last token
    }
    __syncthreads();
    if (v >= nv) return;
    const float* p = a.pieces + (c * 2 + 1) * a.hidden + static_cast<int64_t>(v) * kVec;
    float2 acc[4];
    {
        const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
        acc[0] = make_float2(x.x, x.y);
        acc[1] = make_float2(x.z, x.w);
        acc[2] = make_float2(y.x, y.y);
        acc[3] = make_float2(y.z, y.w);
    }
    p += a.hidden;  // the next chunk's first piece
#pragma unroll 4
    for (int64_t i = c + 1; i <= last; ++i, p += 2 * static_cast<int64_t>(a.hidden)) {
        const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
        acc[0] = __fadd2_rn(acc[0], make_float2(x.x, x.y));
        acc[1] = __fadd2_rn(acc[1], make_float2(x.z, x.w));
        acc[2] = __fadd2_rn(acc[2], make_float2(y.x, y.y));
        acc[3] = __fadd2_rn(acc[3], make_float2(y.z, y.w));
    }
    Old<F32, ADD> old;
    old.load(a, key, v);
    old.put(a, key, v, acc);
}

int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

// Chunks of the sums: long enough that the pieces stay a small share of dy,
// short enough that every SM has several.
int chunk_rows(int64_t tokens, int slices, int sms) {
    int64_t c = tokens * slices / (static_cast<int64_t>(sms) * 16);
    int chunk = 8;
    while (chunk < 256 && chunk * 2 <= c) chunk *= 2;
    while ((tokens + chunk - 1) / chunk * slices > 0x3FFFFFFF) chunk *= 2;
    return chunk;
}

struct Layout {
    int slices, chunk;
    int64_t chunks, tiles;
    int64_t keys, at, keys2, at2, hist, pieces, bytes;  // byte offsets, total
};

Layout layout(int64_t tokens, int64_t hidden, int sms) {
    Layout l{};
    const int nv = static_cast<int>(hidden / kVec);
    l.slices = (nv + kSumThreads - 1) / kSumThreads;
    l.chunk = chunk_rows(tokens, l.slices, sms);
    l.chunks = (tokens + l.chunk - 1) / l.chunk;
    l.tiles = tokens > kSortOne ? (tokens + kTile - 1) / kTile : 0;
    int64_t at = 0;
    const auto take = [&at](int64_t bytes) { const int64_t o = at; at += round16(bytes); return o; };
    l.keys = take(tokens * 4);
    l.at = take(tokens * 4);
    l.keys2 = take(l.tiles ? tokens * 4 : 0);
    l.at2 = take(l.tiles ? tokens * 4 : 0);
    l.hist = take(l.tiles * kBins * 4);
    l.pieces = take(l.chunks * 2 * hidden * 4);
    l.bytes = at;
    return l;
}

template <int THREADS, int ITEMS>
cudaError_t sort_in_one(const void* ids, bool wide, int n, int64_t vocab, int bits, int passes, uint32_t* keys,
                        uint32_t* at, cudaStream_t st) {
    static_assert(THREADS * ITEMS <= kSortOne && kBins <= 2 * THREADS, "16-bit token numbers; two bins a thread");
    static std::atomic<bool> set[64];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const auto kernel = sort_one<THREADS, ITEMS>;
    if (!set[dev].load(std::memory_order_acquire)) {
        if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(sort_one_smem<THREADS, ITEMS>(kBins))))
            return e;
        set[dev].store(true, std::memory_order_release);
    }
    return launch_with_pdl(kernel, dim3(1), dim3(THREADS), sort_one_smem<THREADS, ITEMS>(1 << bits), st, ids, wide, n,
                           vocab, bits, passes, keys, at);
}

template <bool F32, bool ADD>
cudaError_t sums(const EmbedBwd& e, cudaStream_t st) {
    const int64_t work = e.chunks * e.slices;
    const int64_t zero = ADD ? 0 : (e.vocab + kZeroRows - 1) / kZeroRows;
    if (cudaError_t err = launch_with_pdl(embedding_sums<F32, ADD>, dim3(static_cast<unsigned>(work + zero)),
                                          dim3(kSumThreads), 0, st, e))
        return err;
    if (e.chunks <= 1) return cudaSuccess;
    return launch_with_pdl(embedding_join<F32, ADD>, dim3(static_cast<unsigned>(work)), dim3(kSumThreads), 0, st, e);
}

}  // namespace

cudaError_t launch_embedding_fwd(void* y, const void* ids, bool wide, const void* table, int64_t tokens,
                                 int64_t vocab, int64_t hidden, float scale, cudaStream_t st) {
    const int nv = static_cast<int>(hidden / kVec);
    int bx = 32;  // threads over a row: at most kFwdUnroll vectors each where the CTA allows
    while (bx < kFwdThreads && bx * kFwdUnroll < nv) bx *= 2;
    const int by = kFwdThreads / bx;
    const int64_t blocks = (tokens + by - 1) / by;
    const unsigned grid = static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF);
    return launch_with_pdl(embedding_rows, dim3(grid), dim3(bx, by), 0, st, static_cast<uint16_t*>(y), ids, wide,
                           static_cast<const uint16_t*>(table), tokens, vocab, nv, scale);
}

size_t embedding_bwd_workspace(int64_t tokens, int64_t hidden, int sms) {
    return static_cast<size_t>(layout(tokens, hidden, sms).bytes);
}

cudaError_t launch_embedding_bwd(void* dtable, bool f32, bool add, const void* dy, const void* ids, bool wide,
                                 int64_t tokens, int64_t vocab, int64_t hidden, float scale, void* workspace,
                                 int sms, cudaStream_t st) {
    const Layout l = layout(tokens, hidden, sms);
    char* ws = static_cast<char*>(workspace);
    const auto u32 = [ws](int64_t o) { return reinterpret_cast<uint32_t*>(ws + o); };
    int width = 1;  // bits of the largest key, `vocab`
    while ((vocab >> width) != 0) ++width;
    const int passes = (width + kBinBits - 1) / kBinBits;
    const int bits = (width + passes - 1) / passes;
    const uint32_t *keys = u32(l.keys), *at = u32(l.at);
    if (tokens == 0) {
        if (add) return cudaSuccess;
    } else if (!l.tiles) {
        const int n = static_cast<int>(tokens);
        const cudaError_t e = n <= 2048   ? sort_in_one<512, 4>(ids, wide, n, vocab, bits, passes, u32(l.keys), u32(l.at), st)
                              : n <= 4096 ? sort_in_one<1024, 4>(ids, wide, n, vocab, bits, passes, u32(l.keys), u32(l.at), st)
                                          : sort_in_one<1024, 16>(ids, wide, n, vocab, bits, passes, u32(l.keys), u32(l.at), st);
        if (e != cudaSuccess) return e;
    } else {
        uint32_t *to_keys = u32(l.keys), *to_at = u32(l.at), *other_keys = u32(l.keys2), *other_at = u32(l.at2);
        const uint32_t *from_keys = nullptr, *from_at = nullptr;
        const dim3 grid(static_cast<unsigned>(l.tiles));
        for (int p = 0; p < passes; ++p) {
            if (cudaError_t e = launch_with_pdl(sort_count, grid, dim3(kTileThreads), 0, st, ids, wide, from_keys,
                                                tokens, vocab, p * bits, bits, u32(l.hist)))
                return e;
            if (cudaError_t e = launch_with_pdl(sort_scatter, grid, dim3(kTileThreads), 0, st, ids, wide, from_keys,
                                                from_at, tokens, vocab, p * bits, bits, static_cast<int>(l.tiles),
                                                static_cast<const uint32_t*>(u32(l.hist)), to_keys, to_at))
                return e;
            from_keys = keys = to_keys;
            from_at = at = to_at;
            uint32_t *k = to_keys, *a = to_at;
            to_keys = other_keys;
            to_at = other_at;
            other_keys = k;
            other_at = a;
        }
    }
    EmbedBwd e{};
    e.dtable = dtable;
    e.dy = static_cast<const uint16_t*>(dy);
    e.keys = keys;
    e.at = at;
    e.pieces = reinterpret_cast<float*>(ws + l.pieces);
    e.tokens = tokens;
    e.vocab = vocab;
    e.hidden = static_cast<int>(hidden);
    e.chunk = l.chunk;
    e.slices = l.slices;
    e.chunks = l.chunks;
    e.scale = scale;
    if (f32) return add ? sums<true, true>(e, st) : sums<true, false>(e, st);
    return add ? sums<false, true>(e, st) : sums<false, false>(e, st);
}

}  // namespace nf
