// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: y[i] = bf16(scale * table[ids[i]]); an id outside [0, vocab)
// gives a row of zeros.  A gather of rows, bound by memory: 2 bytes read
// (once per distinct id) and 2 written per element.
//
// Backward: dtable[v] (+)= scale * sum over { i : ids[i] = v } of dy[i].  The
// tokens are sorted by id, stably, so that equal ids become a run in token
// order; every run is summed in fp32, its pieces in that order and the pieces'
// sums in a fixed grouping, which makes the result deterministic where atomics
// on the table would not be (bits depend on where the pieces end, and so on the
// SM count).  Up to kDirect
// tokens need no sort (embedding_direct).  The launches of the others:
//   1. the sort: up to kSortRank tokens by counting, up to kSortCluster radix
//      passes in the shared memory of one cluster of CTAs, above that two
//      launches per radix pass (digit counts of each tile, then a stable
//      scatter whose CTAs each add up the counts of the tiles before theirs),
//      and from kOffsetTiles tiles on a third between them for those sums;
//   2. the sums: the sorted tokens are cut into chunks of equal length, a CTA
//      per chunk and slice of columns.  A run inside one chunk is written at
//      once; the pieces of a run that crosses chunks go to the workspace.
//      Where the table's gradient is overwritten, further CTAs of the same
//      launch write zeros into the rows no token names;
//   3. the join: the pieces of each crossing run are added in order.
// A chunk rather than a run per CTA, because word frequencies are uneven:
// one id can hold several percent of a batch.  Bound by memory: dy read
// once, the rows with tokens (or all rows) written once.  One GB300: lookup
// of 32768 x 8192 118 us (6.2 TB/s), gradient of 16384 x 4096 written to
// 131072 fp32 rows 322 us (7.1 TB/s), of 65536 x 4096 added to them 243 us
// (4.9 TB/s, latency of the rows in the sums), to bf16 rows 233 us (3.7 TB/s).
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "pairs.cuh"
#include "pdl.cuh"
#include "tokens.h"

namespace nf {
namespace {

namespace cg = cooperative_groups;

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

// Lanes of the warp that have an item and this lane's digit of `bits` bits,
// from one vote per bit (__match_any_sync took five times as long: the whole
// sort of 16384 tokens 46 us).
__device__ __forceinline__ uint32_t lanes_like(uint32_t digit, bool have, int bits) {
    uint32_t like = __ballot_sync(0xFFFFFFFFu, have);
#pragma unroll
    for (int b = 0; b < kBinBits; ++b) {
        if (b >= bits) break;
        const bool one = (digit >> b) & 1;
        const uint32_t ones = __ballot_sync(0xFFFFFFFFu, one);
        like &= one ? ones : ~ones;
    }
    return like;
}

// Stable ranks of a tile's digits, `bits` bits of the key above `shift`
// (bins = 2^bits).  Warp w holds
// the items [w * 32 * ITEMS, (w + 1) * 32 * ITEMS) of the tile, item k of a
// lane at k * 32 + lane; bit k of `valid` says whether the lane has it.
// counts: `bins` of each warp, zeroed here.  On return the low 16 bits of
// rank[k] are the number of items of the same digit before this one in its
// warp (the high 16 are kept), counts[w * bins + d] is the number of items of
// digit d in the warps before w, and total[d] the tile's items of digit d.
template <int THREADS, int ITEMS>
__device__ __forceinline__ void rank_tile(const uint32_t (&key)[ITEMS], uint32_t valid, int shift, int bits,
                                          uint16_t* counts, uint32_t* total, uint32_t (&rank)[ITEMS]) {
    constexpr int kWarps = THREADS / 32;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, bins = 1 << bits;
    uint32_t* words = reinterpret_cast<uint32_t*>(counts);
    for (int i = t; i < kWarps * bins / 2; i += THREADS) words[i] = 0;
    __syncthreads();
    uint16_t* mine = counts + warp * bins;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const bool have = (valid >> k) & 1;
        const uint32_t d = (key[k] >> shift) & (bins - 1);
        const uint32_t like = lanes_like(d, have, bits);
        const int before = __popc(like & ((1u << lane) - 1));
        const uint32_t c = have ? mine[d] : 0;
        __syncwarp();
        if (have && before == 0) mine[d] = static_cast<uint16_t>(c + __popc(like));
        __syncwarp();
        rank[k] = (rank[k] & 0xFFFF0000u) | (c + before);
    }
    __syncthreads();
    for (int d = t; d < bins; d += THREADS) {
        uint16_t c[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) c[w] = counts[w * bins + d];
        uint32_t sum = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            counts[w * bins + d] = static_cast<uint16_t>(sum);
            sum += c[w];
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

// Up to kSortRank tokens: a token's place is the number of tokens before it
// in the order, counted against all of them.  A CTA takes 32 tokens, one per
// lane, its warps each a stretch of the tokens.  4096 tokens take the GPU
// 17 million comparisons, less than the latency of the radix passes
// (2000 tokens and 8 columns, all three launches: 13.8 -> 9.5 us).
constexpr int kSortRank = 4096;
constexpr int kRankThreads = 256;

__global__ void __launch_bounds__(kRankThreads)
sort_by_rank(const void* __restrict__ ids, bool wide, int n, int64_t vocab, uint32_t* __restrict__ keys_out,
             uint32_t* __restrict__ at_out, uint32_t* __restrict__ crossings) {
    __shared__ __align__(16) uint32_t keys[kSortRank];
    __shared__ int counts[kRankThreads / 32][32];
    grid_dep_wait();
    grid_dep_release();
    if (blockIdx.x == 0 && threadIdx.x == 0) *crossings = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int whole = (n + 3) / 4 * 4;
    for (int i = threadIdx.x; i < whole; i += kRankThreads)
        keys[i] = i < n ? key_of(ids, wide, i, vocab) : 0xFFFFFFFFu;  // behind every key
    __syncthreads();
    const int block = blockIdx.x * 32, token = block + lane;
    const uint32_t key = token < n ? keys[token] : 0;
    // of the tokens before this CTA's, those with the same key come first; of
    // those behind, they do not (key <= 2^30: no overflow)
    int count = 0;
    const uint4* four = reinterpret_cast<const uint4*>(keys);
    const int per = (whole / 4 + kRankThreads / 32 - 1) / (kRankThreads / 32);
    const int i0 = warp * per, i1 = min(i0 + per, whole / 4);
    const auto add = [&](int from, int to, uint32_t bound) {
#pragma unroll 4
        for (int i = from; i < to; ++i) {
            const uint4 k = four[i];
            count += (k.x < bound) + (k.y < bound) + (k.z < bound) + (k.w < bound);
        }
    };
    const int b0 = block / 4, b1 = min(block / 4 + 8, whole / 4);
    add(i0, min(i1, b0), key + 1);
    for (int i = max(i0, b0) * 4; i < min(i1, b1) * 4; ++i) count += keys[i] < key + (i < token);
    add(max(i0, b1), i1, key);
    counts[warp][lane] = count;
    __syncthreads();
    if (warp == 0 && token < n) {
#pragma unroll
        for (int w = 1; w < kRankThreads / 32; ++w) count += counts[w][lane];
        keys_out[count] = key;
        at_out[count] = token;
    }
}

// Up to kSortCluster tokens: one cluster of 1, 2, 4 or 8 CTAs, every pass in
// its shared memory.  CTA r holds the places [r * kTile, (r + 1) * kTile) of
// the order so far.  In a pass a CTA brings its tokens into digit order, the
// CTAs read each other's digit counts, and every token goes to its place, in
// whichever CTA that lies, through distributed shared memory: neighbours in
// digit order go to neighbouring places, where writing them straight from
// the registers took one transaction each (65536 tokens: 42 us).
constexpr int kSortThreads = 512;
constexpr int kSortCtas = 8;
constexpr int kSortCluster = 32768;
template <int ITEMS>
constexpr size_t sort_cluster_smem(int bins) {
    return static_cast<size_t>(kSortThreads) * ITEMS * 16 + static_cast<size_t>(kSortThreads / 32) * bins * 2 + 3 * bins * 4 + 128;
}

template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads, 1)
sort_cluster(const void* __restrict__ ids, bool wide, int n, int64_t vocab, int bits, int passes,
             uint32_t* __restrict__ keys_out, uint32_t* __restrict__ at_out, uint32_t* __restrict__ crossings) {
    constexpr int kTile = kSortThreads * ITEMS;
    extern __shared__ __align__(16) unsigned char smem[];
    const int bins = 1 << bits;
    uint64_t* order = reinterpret_cast<uint64_t*>(smem);  // this CTA's tokens in digit order: (key, token)
    uint64_t* place = order + kTile;                      // the tokens whose places are this CTA's
    uint32_t* total = reinterpret_cast<uint32_t*>(place + kTile);  // this CTA's items of each digit
    uint32_t* local = total + bins;                       // of smaller digits
    uint32_t* start = local + bins;                       // the place of the digit's first item of this CTA, less local
    uint32_t* warp_sums = start + bins;
    uint16_t* counts = reinterpret_cast<uint16_t*>(warp_sums + 32);
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), cta = cluster.block_rank();
    grid_dep_wait();
    grid_dep_release();
    if (cta == 0 && threadIdx.x == 0) *crossings = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int held = min(max(n - cta * kTile, 0), kTile);  // places of this CTA
    uint32_t key[ITEMS], token[ITEMS], rank[ITEMS];
    uint32_t valid = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int j = (warp * ITEMS + k) * 32 + lane;
        const bool have = j < held;
        valid |= static_cast<uint32_t>(have) << k;
        token[k] = cta * kTile + j;
        key[k] = have ? key_of(ids, wide, token[k], vocab) : 0;
        rank[k] = 0;
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * bits;
        const auto digit_of = [&](uint32_t k) { return (k >> shift) & (bins - 1); };
        rank_tile<kSortThreads, ITEMS>(key, valid, shift, bits, counts, total, rank);
        for (int d = threadIdx.x; d < bins; d += kSortThreads) local[d] = total[d];
        __syncthreads();
        scan_bins<kSortThreads>(local, bins, warp_sums);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            if (!((valid >> k) & 1)) continue;
            const uint32_t d = digit_of(key[k]);
            order[local[d] + counts[warp * bins + d] + (rank[k] & 0xFFFFu)] = static_cast<uint64_t>(key[k]) << 32 | token[k];
        }
        cluster.sync();
        uint32_t mine[2];  // bins <= 2 * kSortThreads
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int d = threadIdx.x + h * kSortThreads;
            if (d >= bins) break;
            uint32_t all = 0, before = 0;
#pragma unroll
            for (int i = 0; i < kSortCtas; ++i) {
                if (i >= ctas) break;
                const uint32_t c = cluster.map_shared_rank(total, i)[d];
                all += c;
                if (i < cta) before += c;
            }
            start[d] = all;
            mine[h] = before - local[d];
        }
        __syncthreads();
        scan_bins<kSortThreads>(start, bins, warp_sums);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int d = threadIdx.x + h * kSortThreads;
            if (d < bins) start[d] += mine[h];
        }
        __syncthreads();
        const bool last = p == passes - 1;
        for (int j = threadIdx.x; j < held; j += kSortThreads) {
            const uint64_t item = order[j];
            const uint32_t k = static_cast<uint32_t>(item >> 32), to = start[digit_of(k)] + j;
            if (last) {
                keys_out[to] = k;
                at_out[to] = static_cast<uint32_t>(item);
            } else {
                cluster.map_shared_rank(place, to / kTile)[to % kTile] = item;
            }
        }
        cluster.sync();  // all tokens are placed, and the counts have been read
        if (last) break;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            if ((valid >> k) & 1) {
                const uint64_t item = place[(warp * ITEMS + k) * 32 + lane];
                key[k] = static_cast<uint32_t>(item >> 32);
                token[k] = static_cast<uint32_t>(item);
            }
        }
    }
}

// Tiles of many-CTA sorts: 2048 tokens.  Tiles of 4096 were slower (65536
// tokens and 8 columns, the whole call: 43 against 33 us; 16 million: 2154
// against 1795 us).
constexpr int kTileThreads = 512;
constexpr int kTileItems = 4;
constexpr int kTile = kTileThreads * kTileItems;
// From this many tiles on a launch of its own adds up the tiles' counts; below,
// every CTA of the scatter adds up those of the tiles before its own, which
// saves a launch but grows with the square of the tiles (8 columns, the whole
// call, with the launch and without: 65536 tokens 34.5 and 32.8 us, 131072
// 45.7 and 47.5 us, a million 153 and 317 us, 16 million 1.8 and 36.9 ms).
constexpr int kOffsetTiles = 64;

__global__ void __launch_bounds__(kTileThreads)
sort_count(const void* __restrict__ ids, bool wide, const uint32_t* __restrict__ keys_in, int64_t n,
           int64_t vocab, int shift, int bits, uint32_t* __restrict__ hist, uint32_t* __restrict__ crossings) {
    __shared__ uint32_t bins[kBins];
    grid_dep_wait();
    grid_dep_release();
    if (blockIdx.x == 0 && threadIdx.x == 0) *crossings = 0;
    for (int d = threadIdx.x; d < kBins; d += kTileThreads) bins[d] = 0;
    __syncthreads();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile;
#pragma unroll
    for (int k = 0; k < kTileItems; ++k) {
        const int64_t i = base + k * kTileThreads + threadIdx.x;
        if (i < n) {
            const uint32_t key = keys_in ? keys_in[i] : key_of(ids, wide, i, vocab);
            atomicAdd(&bins[(key >> shift) & ((1u << bits) - 1)], 1u);  // a count: its order does not matter
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < 1 << bits; d += kTileThreads)
        hist[(static_cast<int64_t>(blockIdx.x) << bits) + d] = bins[d];
}

// The counts of each digit in the tiles before each tile, in place of the
// tiles' own, and behind them the counts of all tiles.  A CTA takes 32 digits,
// its warps each a stretch of the tiles.
constexpr int kOffsetWarps = 32;
__global__ void __launch_bounds__(kOffsetWarps * 32)
sort_offsets(uint32_t* __restrict__ hist, int bins, int tiles) {
    __shared__ uint32_t sums[kOffsetWarps][32];
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    const int per = (tiles + kOffsetWarps - 1) / kOffsetWarps;
    const int i0 = min(warp * per, tiles), i1 = min(i0 + per, tiles);
    uint32_t sum = 0;
    if (d < bins) {
#pragma unroll 16
        for (int i = i0; i < i1; ++i) sum += hist[static_cast<int64_t>(i) * bins + d];
    }
    sums[warp][lane] = sum;
    __syncthreads();
    uint32_t run = 0;
    for (int w = 0; w < warp; ++w) run += sums[w][lane];
    if (d >= bins) return;
    if (warp == kOffsetWarps - 1) hist[static_cast<int64_t>(tiles) * bins + d] = run + sum;
    constexpr int kBatch = 16;  // in flight
    for (int i = i0; i < i1; i += kBatch) {
        uint32_t c[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) c[k] = i + k < i1 ? hist[static_cast<int64_t>(i + k) * bins + d] : 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (i + k < i1) hist[static_cast<int64_t>(i + k) * bins + d] = run;
            run += c[k];
        }
    }
}

__global__ void __launch_bounds__(kTileThreads)
sort_scatter(const void* __restrict__ ids, bool wide, const uint32_t* __restrict__ keys_in,
             const uint32_t* __restrict__ at_in, int64_t n, int64_t vocab, int shift, int bits, int tiles,
             bool offsets, const uint32_t* __restrict__ hist, uint32_t* __restrict__ keys_out,
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
    rank_tile<kTileThreads, kTileItems>(key, valid, shift, bits, counts, total, rank);
    // all tiles' items of a digit, and those of the tiles before this one
    for (int d = threadIdx.x; d < bins; d += kTileThreads) {
        uint32_t all = 0, before = 0;
        if (offsets) {
            all = hist[static_cast<int64_t>(tiles) * bins + d];
            before = hist[static_cast<int64_t>(blockIdx.x) * bins + d];
        } else {
#pragma unroll 16
            for (int i = 0; i < tiles; ++i) {
                const uint32_t c = hist[static_cast<int64_t>(i) * bins + d];
                all += c;
                if (i < static_cast<int>(blockIdx.x)) before += c;
            }
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
// A CTA that writes zeros takes rows of kZeroBytes together, and never more
// than kZeroRows (the gradient of 16384 x 4096 written to 131072 fp32 rows with
// 128, 32 and 16 KB: 333, 320 and 318 us; of 300 x 4096: 279, 276 and 354 us;
// 16 rows whatever their length took 49 us where 126725 rows of 192 bytes take
// 5.5).
constexpr int kZeroBytes = 32 * 1024;
constexpr int kZeroRows = 1024;

struct EmbedBwd {
    void* dtable;
    const uint16_t* dy;
    const uint32_t* keys;
    const uint32_t* at;
    float* pieces;        // [chunks][2][hidden]: a chunk's first and last piece of a crossing run
    uint32_t* crossings;  // how many chunks a crossing run begins in, then (4 further on) which
    int64_t tokens, vocab;
    int hidden, chunk, slices;
    int zero_rows;        // per CTA that writes zeros
    int64_t chunks;
    float scale;
};

// One table row's 8 columns: (old +) scale * acc.  A bf16 row's old values are
// loaded apart, so that a batch of rows has its loads in flight together; an
// fp32 row is added to in L2 (a row is one thread's, so the order of such
// additions cannot matter).
template <bool F32, bool ADD>
struct Old {
    static constexpr int N = F32 ? 2 : 1;  // 16-byte vectors
    uint4 v;
    static __device__ __forceinline__ uint4* place(const EmbedBwd& a, uint32_t key, int col) {
        return static_cast<uint4*>(a.dtable) + (static_cast<int64_t>(key) * (a.hidden / kVec) + col) * N;
    }
    __device__ __forceinline__ void load(const EmbedBwd& a, uint32_t key, int col) {
        if constexpr (ADD && !F32) v = ld_stream(place(a, key, col));
    }
    __device__ __forceinline__ void put(const EmbedBwd& a, uint32_t key, int col, const float2 (&acc)[4]) const {
        const float2 s2 = make_float2(a.scale, a.scale);
        float2 o[4];
        if constexpr (ADD && !F32) {
            unpack8x2(v, o);
        } else {
            o[0] = o[1] = o[2] = o[3] = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = __ffma2_rn(acc[q], s2, o[q]);
        uint4* p = place(a, key, col);
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (ADD)
                    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p + i), "f"(o[2 * i].x),
                                 "f"(o[2 * i].y), "f"(o[2 * i + 1].x), "f"(o[2 * i + 1].y) : "memory");
                else
                    st_stream(p + i, make_uint4(__float_as_uint(o[2 * i].x), __float_as_uint(o[2 * i].y),
                                                __float_as_uint(o[2 * i + 1].x), __float_as_uint(o[2 * i + 1].y)));
            }
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

// Zeros into the table's rows [r0, r1) that have no tokens, by the whole CTA:
// touched[r - r0] says which have (only looked at where `any` does).
template <bool F32>
__device__ __forceinline__ void zero_rows(const EmbedBwd& a, int64_t r0, int64_t r1, const uint8_t* touched, bool any) {
    const int per = a.hidden / kVec * (F32 ? 2 : 1), total = static_cast<int>(r1 - r0) * per;  // 16-byte vectors
    uint4* p = static_cast<uint4*>(a.dtable) + r0 * per;
    const int T = blockDim.x, down = T / per, along = T % per;
    int row = threadIdx.x / per, col = threadIdx.x % per;
    for (int i = threadIdx.x; i < total; i += T) {
        if (!any || !touched[row]) __stcs(p + i, make_uint4(0, 0, 0, 0));
        row += down;
        col += along;
        if (col >= per) {
            col -= per;
            ++row;
        }
    }
}

// touched[r - r0] = 1 for the rows r of [r0, r0 + rows) that are among the n
// sorted keys, by the whole CTA; touched is 0 before, and no key lies outside.
// Few keys are walked.  Many, the most frequent ids' of a large batch, would
// keep this one CTA busy behind all others, so there a thread searches the keys
// for its rows, kSearch at a time (more took registers from the sums).  A round
// of searches takes as long as a walk of some 16384 keys (131072 fp32 rows of 8
// columns, the whole call, walks alone and with searches: 4 million words 914
// and 523 us, a million 218 and 161 us; 65536 words are walked, 36 us, where
// searches alone take 38.5 us).
constexpr uint32_t kWalkKeys = 16384;
constexpr int kSearch = 2;
__device__ __forceinline__ void mark_touched(const uint32_t* keys, uint32_t n, uint32_t r0, int rows, uint8_t* touched) {
    const int round = kSearch * kSumThreads;
    if (n <= kWalkKeys * ((rows + round - 1) / round)) {
        for (uint32_t i = threadIdx.x; i < n; i += kSumThreads) touched[keys[i] - r0] = 1;
        return;
    }
    for (int r = threadIdx.x; r < rows; r += round) {
        uint32_t at[kSearch] = {};  // keys below the row's lie in [0, at + len) at most, and all of [0, at) do
        for (uint32_t len = n; len > 0;) {
            const uint32_t half = len - len / 2;
#pragma unroll
            for (int k = 0; k < kSearch; ++k)
                if (keys[at[k] + half - 1] < r0 + r + k * kSumThreads) at[k] += half;
            len -= half;
        }
#pragma unroll
        for (int k = 0; k < kSearch; ++k)
            if (at[k] < n && keys[at[k]] == r0 + r + k * kSumThreads) touched[r + k * kSumThreads] = 1;
    }
}

// CTAs [0, chunks * slices): the sums.  CTAs above: zeros for the table's
// rows without tokens, zero_rows each.
template <bool F32, bool ADD>
__global__ void __launch_bounds__(kSumThreads)
embedding_sums(const EmbedBwd a) {
    __shared__ uint8_t touched[kZeroRows];
    __shared__ uint32_t keys[kSumPart + kSumBatch], at[kSumPart];  // keys: one more than the part's
    __shared__ int64_t range[2];
    grid_dep_wait();
    grid_dep_release();
    const int nv = a.hidden / kVec;
    const int64_t work = a.chunks * a.slices;
    if (!ADD && static_cast<int64_t>(blockIdx.x) >= work) {
        const int64_t r0 = (static_cast<int64_t>(blockIdx.x) - work) * a.zero_rows;
        const int64_t r1 = r0 + a.zero_rows < a.vocab ? r0 + a.zero_rows : a.vocab;
        for (int r = threadIdx.x; r < a.zero_rows; r += kSumThreads) touched[r] = 0;
        if (threadIdx.x < 64) {
            const int64_t b = lower_bound_warp(a.keys, 0, a.tokens, static_cast<uint32_t>(threadIdx.x < 32 ? r0 : r1));
            if ((threadIdx.x & 31) == 0) range[threadIdx.x >> 5] = b;
        }
        __syncthreads();
        mark_touched(a.keys + range[0], static_cast<uint32_t>(range[1] - range[0]), static_cast<uint32_t>(r0), a.zero_rows, touched);
        __syncthreads();
        zero_rows<F32>(a, r0, r1, touched, range[0] < range[1]);
        return;
    }
    const int64_t c = static_cast<int64_t>(blockIdx.x) / a.slices;
    const int v = static_cast<int>(blockIdx.x % a.slices) * kSumThreads + threadIdx.x;
    const int64_t begin = c * a.chunk;
    const int64_t end = begin + a.chunk < a.tokens ? begin + a.chunk : a.tokens;
    const uint32_t none = static_cast<uint32_t>(a.vocab);
    const uint32_t before = begin > 0 ? a.keys[begin - 1] : none;
    const uint32_t first = a.keys[begin];
    if (blockIdx.x % a.slices == 0 && threadIdx.x == 0) {
        const uint32_t key = a.keys[end - 1], after = end < a.tokens ? a.keys[end] : none;
        // the last run goes on, and began here
        if (key != none && after == key && !(first == key && before == key))
            a.crossings[4 + atomicAdd(a.crossings, 1u)] = static_cast<uint32_t>(c);
    }
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

// The runs that cross chunks: the last piece of the chunk in which a run
// begins and the first pieces of the chunks it goes on through, in order.  A
// CTA takes 32 column vectors of a run; its warps each add a stretch of the
// pieces, so that a run of thousands of tokens is not one long chain.
constexpr int kJoinWarps = 8;
template <bool F32, bool ADD>
__global__ void __launch_bounds__(kJoinWarps * 32)
embedding_join(const EmbedBwd a) {
    __shared__ float2 sums[kJoinWarps][4][32];
    // no early release: with the next kernel's CTAs resident beside these, a
    // call of 4096 tokens and 4096 columns took 32 us instead of 20
    grid_dep_wait();
    const int nv = a.hidden / kVec, slices = (nv + 31) / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t work = static_cast<int64_t>(*a.crossings) * slices;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int64_t c = a.crossings[4 + w / slices];
        const int v = static_cast<int>(w % slices) * 32 + lane;
        const uint32_t key = a.keys[(c + 1) * a.chunk];
        int64_t pieces = 1;  // and one for each following chunk that the run's id opens
        for (;;) {
            const int64_t at = (c + pieces + lane) * a.chunk;
            const uint32_t open = __ballot_sync(0xFFFFFFFFu, at < a.tokens && a.keys[at] == key);
            const int n = open == 0xFFFFFFFFu ? 32 : __ffs(~open) - 1;
            pieces += n;
            if (n < 32) break;
        }
        const int64_t per = (pieces + kJoinWarps - 1) / kJoinWarps;
        const int64_t p0 = warp * per, p1 = p0 + per < pieces ? p0 + per : pieces;
        float2 acc[4] = {};
        if (v < nv) {
#pragma unroll 4
            for (int64_t i = p0; i < p1; ++i) {
                const float4* p = reinterpret_cast<const float4*>(a.pieces + ((c + i) * 2 + (i == 0)) * a.hidden + v * kVec);
                const float4 x = p[0], y = p[1];
                acc[0] = __fadd2_rn(acc[0], make_float2(x.x, x.y));
                acc[1] = __fadd2_rn(acc[1], make_float2(x.z, x.w));
                acc[2] = __fadd2_rn(acc[2], make_float2(y.x, y.y));
                acc[3] = __fadd2_rn(acc[3], make_float2(y.z, y.w));
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) sums[warp][q][lane] = acc[q];
        __syncthreads();
        if (warp == 0 && v < nv) {
            Old<F32, ADD> old;
            old.load(a, key, v);
            for (int i = 1; i < kJoinWarps; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[q] = __fadd2_rn(acc[q], sums[i][q][lane]);
            old.put(a, key, v, acc);
        }
        __syncthreads();
    }
}

// ---- few tokens: one launch, no sort ------------------------------------------------
// Up to kDirect tokens a warp takes a token and 512 columns, and looks for the
// token's id among all of them, which lie in shared memory: where it stands
// earlier too, another warp has the run; else the warp adds up the id's rows in
// token order.  A run of more than kDirectRun rows is left to the whole CTA: its
// warps each add a stretch, and the stretches are joined in order.  A CTA's
// tokens are far apart, because the first tokens of a batch begin its longest
// runs.  Bound by latency: one launch against three.  The search grows with the
// square of the tokens and with the columns, hence the limit (2048 columns
// added to bf16, against the sort: 16 tokens 2.6 and 6.0 us, 200 4.5 and 9.7,
// 512 7.1 and 10.7, 1000 8.6 and 12.0, 2000 16.5 and 14.3; 8192 columns: 512
// 11.7 and 12.3, 1000 19.1 and 16.4).  Runs of 16 rows for a warp were slower
// (16 equal ids 4.6 for 3.0 us), of 4 too (64 words 4.1 for 3.6 us).
constexpr int kDirect = 512;
constexpr int kDirectThreads = 256, kDirectCtas = 3;
constexpr int kDirectWarps = kDirectThreads / 32;
constexpr int kDirectRun = 8;
constexpr int kDirectVectors = 64;  // of a warp's columns, two per lane
constexpr int kDirectBatch = 4;     // rows in flight

// Rows at[0, n) of dy added to acc, in order.
__device__ __forceinline__ void add_rows(const EmbedBwd& a, const uint16_t* at, int n, int v, int nv, float2 (&acc)[2][4]) {
    for (int i = 0; i < n; i += kDirectBatch) {
        uint4 d[kDirectBatch][2];
#pragma unroll
        for (int k = 0; k < kDirectBatch; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (i + k < n && v + 32 * h < nv)
                    d[k][h] = ld_stream(a.dy + (static_cast<int64_t>(at[i + k]) * nv + v + 32 * h) * kVec);
#pragma unroll
        for (int k = 0; k < kDirectBatch; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (i + k >= n || v + 32 * h >= nv) continue;
                float2 f[4];
                unpack8x2(d[k][h], f);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[h][q] = __fadd2_rn(acc[h][q], f[q]);
            }
    }
}

// CTAs [0, blocks * slices): the sums.  CTAs above: zeros, as in embedding_sums.
template <bool F32, bool ADD>
__global__ void __launch_bounds__(kDirectThreads, kDirectCtas)
embedding_direct(const EmbedBwd a, const void* __restrict__ ids, bool wide, int blocks) {
    __shared__ __align__(16) uint32_t keys[kDirect];
    __shared__ float2 sums[kDirectWarps][2][4][32];
    __shared__ uint16_t list[kDirect];                       // a long run's tokens
    __shared__ uint16_t short_list[kDirectWarps][kDirectRun];
    __shared__ uint16_t queue[kDirect / kDirectRun];         // the first tokens of this CTA's long runs
    __shared__ int queued, counts[kDirectWarps];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, n = static_cast<int>(a.tokens), nv = a.hidden / kVec;
    grid_dep_wait();
    grid_dep_release();
    if (!ADD && blockIdx.x >= static_cast<unsigned>(blocks * a.slices)) {
        uint8_t* touched = reinterpret_cast<uint8_t*>(sums);
        static_assert(sizeof(sums) >= kZeroRows, "touched");
        const int64_t r0 = static_cast<int64_t>(blockIdx.x - blocks * a.slices) * a.zero_rows;
        const int64_t r1 = r0 + a.zero_rows < a.vocab ? r0 + a.zero_rows : a.vocab;
        for (int r = t; r < a.zero_rows; r += kDirectThreads) touched[r] = 0;
        __syncthreads();
        bool any = false;
        for (int i = t; i < n; i += kDirectThreads) {
            const uint32_t key = key_of(ids, wide, i, a.vocab);
            if (key >= r0 && key < r1) {
                touched[key - r0] = 1;
                any = true;
            }
        }
        any = __syncthreads_or(any);
        zero_rows<F32>(a, r0, r1, touched, any);
        return;
    }
    const uint32_t none = static_cast<uint32_t>(a.vocab);
    const int whole = (n + kDirectThreads - 1) / kDirectThreads * kDirectThreads;  // keys, with some that no token has
    for (int i = t; i < whole; i += kDirectThreads) keys[i] = i < n ? key_of(ids, wide, i, a.vocab) : 0xFFFFFFFFu;
    if (t == 0) queued = 0;
    __syncthreads();
    const int slice = blockIdx.x % a.slices, block = blockIdx.x / a.slices;
    const int v = slice * kDirectVectors + lane;
    const uint4* four = reinterpret_cast<const uint4*>(keys);
    for (int i = block + warp * blocks; i < n; i += kDirectWarps * blocks) {
        const uint32_t key = keys[i];
        if (key == none) continue;
        int before = 0, after = 0;
        for (int p = lane; p < whole / 4; p += 32) {
            const uint4 k = four[p];
            const int same = (k.x == key) + (k.y == key) + (k.z == key) + (k.w == key);
            if (p < i / 4) before += same;
            else if (p > i / 4) after += same;
            else {
                before += (i % 4 > 0 && k.x == key) + (i % 4 > 1 && k.y == key) + (i % 4 > 2 && k.z == key);
                after += (i % 4 < 1 && k.y == key) + (i % 4 < 2 && k.z == key) + (i % 4 < 3 && k.w == key);
            }
        }
        if (__any_sync(0xFFFFFFFFu, before > 0)) continue;
        const int rows = 1 + __reduce_add_sync(0xFFFFFFFFu, after);
        if (rows > kDirectRun) {
            if (lane == 0) queue[atomicAdd(&queued, 1)] = static_cast<uint16_t>(i);
            continue;
        }
        uint16_t* mine = short_list[warp];
        if (lane == 0) mine[0] = static_cast<uint16_t>(i);
        for (int found = 1, p = (i + 1) / 32 * 32; found < rows; p += 32) {
            const bool is = p + lane > i && keys[p + lane] == key;
            const uint32_t which = __ballot_sync(0xFFFFFFFFu, is);
            if (is) mine[found + __popc(which & ((1u << lane) - 1))] = static_cast<uint16_t>(p + lane);
            found += __popc(which);
        }
        __syncwarp();
        Old<F32, ADD> old[2];
        float2 acc[2][4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (v + 32 * h < nv) old[h].load(a, key, v + 32 * h);
        add_rows(a, mine, rows, v, nv, acc);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (v + 32 * h < nv) old[h].put(a, key, v + 32 * h, acc[h]);
        __syncwarp();  // the list has been read
    }
    __syncthreads();
    for (int k = 0; k < queued; ++k) {
        const uint32_t key = keys[queue[k]];
        const int per = whole / kDirectWarps, p0 = warp * per;  // a multiple of 32
        int found = 0;
        for (int p = p0; p < p0 + per; p += 32) found += __popc(__ballot_sync(0xFFFFFFFFu, keys[p + lane] == key));
        if (lane == 0) counts[warp] = found;
        __syncthreads();
        int at = 0, rows = 0;
        for (int w = 0; w < kDirectWarps; ++w) {
            if (w == warp) at = rows;
            rows += counts[w];
        }
        for (int p = p0; p < p0 + per; p += 32) {
            const bool is = keys[p + lane] == key;
            const uint32_t which = __ballot_sync(0xFFFFFFFFu, is);
            if (is) list[at + __popc(which & ((1u << lane) - 1))] = static_cast<uint16_t>(p + lane);
            at += __popc(which);
        }
        __syncthreads();
        const int share = (rows + kDirectWarps - 1) / kDirectWarps, first = min(warp * share, rows);
        float2 acc[2][4] = {};
        add_rows(a, list + first, min(share, rows - first), v, nv, acc);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q) sums[warp][h][q][lane] = acc[h][q];
        __syncthreads();
        if (warp < 2 && v + 32 * warp < nv) {
            Old<F32, ADD> old;
            old.load(a, key, v + 32 * warp);
            float2 sum[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                sum[q] = sums[0][warp][q][lane];
                for (int w = 1; w < kDirectWarps; ++w) sum[q] = __fadd2_rn(sum[q], sums[w][warp][q][lane]);
            }
            old.put(a, key, v + 32 * warp, sum);
        }
        __syncthreads();  // counts, list and sums are used again
    }
}

int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

constexpr int kChunksPerSm = 4;
// Chunks of the sums: long enough that the pieces stay a small share of dy,
// short enough that every SM has several.
int chunk_rows(int64_t tokens, int slices, int sms) {
    int64_t c = tokens * slices / (static_cast<int64_t>(sms) * kChunksPerSm);
    int chunk = 8;
    while (chunk < 256 && chunk * 2 <= c) chunk *= 2;
    while ((tokens + chunk - 1) / chunk * slices > 0x3FFFFFFF) chunk *= 2;
    return chunk;
}

struct Layout {
    int slices, chunk;
    int64_t chunks, tiles;
    int64_t keys, at, keys2, at2, hist, crossings, pieces, bytes;  // byte offsets, total
};

Layout layout(int64_t tokens, int64_t hidden, int sms) {
    Layout l{};
    const int nv = static_cast<int>(hidden / kVec);
    l.slices = (nv + kSumThreads - 1) / kSumThreads;
    l.chunk = chunk_rows(tokens, l.slices, sms);
    l.chunks = (tokens + l.chunk - 1) / l.chunk;
    l.tiles = tokens > kSortCluster ? (tokens + kTile - 1) / kTile : 0;
    int64_t at = 0;
    const auto take = [&at](int64_t bytes) { const int64_t o = at; at += round16(bytes); return o; };
    l.keys = take(tokens * 4);
    l.at = take(tokens * 4);
    l.keys2 = take(l.tiles ? tokens * 4 : 0);
    l.at2 = take(l.tiles ? tokens * 4 : 0);
    l.hist = take(l.tiles ? (l.tiles + 1) * kBins * 4 : 0);
    l.crossings = take((4 + l.chunks) * 4);
    l.pieces = take(l.chunks * 2 * hidden * 4);
    l.bytes = at;
    return l;
}

template <int ITEMS>
cudaError_t sort_in_cluster(const void* ids, bool wide, int n, int64_t vocab, int bits, int passes, uint32_t* keys,
                            uint32_t* at, uint32_t* crossings, cudaStream_t st) {
    static_assert(kSortThreads * ITEMS * kSortCtas <= kSortCluster && kBins <= 2 * kSortThreads, "two bins a thread");
    static std::atomic<bool> set[64];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const auto kernel = sort_cluster<ITEMS>;
    if (!set[dev].load(std::memory_order_acquire)) {
        if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(sort_cluster_smem<ITEMS>(kBins))))
            return e;
        set[dev].store(true, std::memory_order_release);
    }
    unsigned ctas = 1;
    while (static_cast<int>(ctas) * kSortThreads * ITEMS < n) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sort_cluster_smem<ITEMS>(1 << bits);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, ids, wide, n, vocab, bits, passes, keys, at, crossings);
}

template <bool F32, bool ADD>
cudaError_t sums(const EmbedBwd& e, int sms, cudaStream_t st) {
    const int64_t work = e.chunks * e.slices;
    const int64_t zero = ADD ? 0 : (e.vocab + e.zero_rows - 1) / e.zero_rows;
    if (cudaError_t err = launch_with_pdl(embedding_sums<F32, ADD>, dim3(static_cast<unsigned>(work + zero)),
                                          dim3(kSumThreads), 0, st, e))
        return err;
    if (e.chunks <= 1) return cudaSuccess;
    // one crossing run per chunk at most; as many CTAs as stay resident take them in turn
    const int64_t joins = (e.chunks - 1) * ((e.hidden / kVec + 31) / 32), wave = static_cast<int64_t>(sms) * 8;
    return launch_with_pdl(embedding_join<F32, ADD>, dim3(static_cast<unsigned>(joins < wave ? joins : wave)),
                           dim3(kJoinWarps * 32), 0, st, e);
}

template <bool F32, bool ADD>
cudaError_t direct(EmbedBwd e, const void* ids, bool wide, int sms, cudaStream_t st) {
    e.slices = (e.hidden / kVec + kDirectVectors - 1) / kDirectVectors;
    // a token per warp, in one wave of CTAs where more would not all fit
    const int64_t most = kDirectCtas * static_cast<int64_t>(sms) / e.slices;
    int64_t blocks = (e.tokens + kDirectWarps - 1) / kDirectWarps;
    if (blocks > most) blocks = most > 0 ? most : 1;
    const int64_t zero = ADD ? 0 : (e.vocab + e.zero_rows - 1) / e.zero_rows;
    return launch_with_pdl(embedding_direct<F32, ADD>, dim3(static_cast<unsigned>(blocks * e.slices + zero)),
                           dim3(kDirectThreads), 0, st, e, ids, wide, static_cast<int>(blocks));
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
    EmbedBwd e{};
    e.dtable = dtable;
    e.dy = static_cast<const uint16_t*>(dy);
    e.tokens = tokens;
    e.vocab = vocab;
    e.hidden = static_cast<int>(hidden);
    e.scale = scale;
    const int64_t fit = kZeroBytes / (hidden * (f32 ? 4 : 2));
    e.zero_rows = static_cast<int>(fit < 1 ? 1 : fit > kZeroRows ? kZeroRows : fit);
    if (tokens > 0 && tokens <= kDirect) {
        if (f32) return add ? direct<true, true>(e, ids, wide, sms, st) : direct<true, false>(e, ids, wide, sms, st);
        return add ? direct<false, true>(e, ids, wide, sms, st) : direct<false, false>(e, ids, wide, sms, st);
    }
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
        const auto sort = n <= 4 * kSortThreads * kSortCtas ? sort_in_cluster<4> : sort_in_cluster<8>;
        const cudaError_t e =
            n <= kSortRank ? launch_with_pdl(sort_by_rank, dim3((n + 31) / 32), dim3(kRankThreads), 0, st, ids, wide, n,
                                             vocab, u32(l.keys), u32(l.at), u32(l.crossings))
                           : sort(ids, wide, n, vocab, bits, passes, u32(l.keys), u32(l.at), u32(l.crossings), st);
        if (e != cudaSuccess) return e;
    } else {
        uint32_t *to_keys = u32(l.keys), *to_at = u32(l.at), *other_keys = u32(l.keys2), *other_at = u32(l.at2);
        const uint32_t *from_keys = nullptr, *from_at = nullptr;
        const dim3 grid(static_cast<unsigned>(l.tiles));
        const bool offsets = l.tiles >= kOffsetTiles;
        for (int p = 0; p < passes; ++p) {
            if (cudaError_t e = launch_with_pdl(sort_count, grid, dim3(kTileThreads), 0, st, ids, wide, from_keys,
                                                tokens, vocab, p * bits, bits, u32(l.hist), u32(l.crossings)))
                return e;
            if (offsets) {
                const dim3 digits(((1 << bits) + 31) / 32);
                if (cudaError_t e = launch_with_pdl(sort_offsets, digits, dim3(kOffsetWarps * 32), 0, st, u32(l.hist),
                                                    1 << bits, static_cast<int>(l.tiles)))
                    return e;
            }
            if (cudaError_t e = launch_with_pdl(sort_scatter, grid, dim3(kTileThreads), 0, st, ids, wide, from_keys,
                                                from_at, tokens, vocab, p * bits, bits, static_cast<int>(l.tiles), offsets,
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
    e.keys = keys;
    e.at = at;
    e.pieces = reinterpret_cast<float*>(ws + l.pieces);
    e.crossings = u32(l.crossings);
    e.chunk = l.chunk;
    e.slices = l.slices;
    e.chunks = l.chunks;
    if (f32) return add ? sums<true, true>(e, sms, st) : sums<true, false>(e, sms, st);
    return add ? sums<false, true>(e, sms, st) : sums<false, false>(e, sms, st);
}

}  // namespace nf
