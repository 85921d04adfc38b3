// Host-side launchers of the operators on attention heads: the rotation by
// positions, the RMSNorm of each head with the rotation, and the append to a
// paged cache.  Internal to libnf.so: the entry points (api_heads.cu) validate
// arguments and call these.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace nf {

constexpr int kHeadMaxDim = 512;
constexpr int kMaxSegments = 3;

// n / d for 32-bit n by a product (set up on the host): with M = ceil(2^64 / d)
// the upper half of n * M is the quotient, as n (M d - 2^64) < 2^64.
struct Divider {
    uint64_t m;  // 0: d is 1
    uint32_t d;
    Divider() = default;
    explicit Divider(uint32_t by) : m(by > 1 ? ~0ull / by + 1 : 0), d(by) {}
};

// One set of heads of a call: queries, keys or values.  Strides in elements.
struct HeadSegment {
    const void* in;
    void* out;
    const void* weight;  // null: not normalized
    int64_t in_batch, in_token, in_head;
    int64_t out_batch, out_token, out_head;  // a cache: page, slot and head strides
    float* scale;                            // an 8-bit cache: per row
    int64_t scale_page, scale_slot, scale_head;
    int heads;
    // How a call's launcher shares out the rows (heads_rows.cuh).
    int shares;           // of a CTA's tokens
    int per_token;        // shares of a token; 0: a share holds several tokens,
    int tokens_of_share;  //   so many,
    int groups_of_token;  //   each on so many groups of lanes
    int groups_factor;
    bool rotate;
    bool cache;      // out is a paged cache
    bool with_next;  // its one share of a token has the next segment's rows too, in the second half of its passes
};

// The gradient of one set of normalized heads.
struct HeadGradSegment {
    void* dx;
    const void* dy;
    const void* x;
    const void* weight;
    float* dweight;
    int64_t dx_batch, dx_token, dx_head;
    int64_t dy_batch, dy_token, dy_head;
    int64_t x_batch, x_token, x_head;
    int heads;
    int ctas;  // set by the launcher
};

struct Rotation {
    const uint64_t* rates;  // [pairs]
    int pairs;              // 0: no rotation
    float magnitude;
    float direction;  // 1, or -1 to turn back
    bool interleaved;
    const void* positions;  // null in an append: the place in the sequence
    bool wide;              // 64-bit positions
    int64_t position_batch;
};

enum CacheFormat { kCacheSame = 0, kCacheE4M3 = 1, kCacheInt8 = 2 };

struct HeadsArgs {
    HeadSegment seg[kMaxSegments];
    Rotation rope;
    int segments;
    int dim;
    int tokens;      // per batch
    uint32_t total;  // batch * tokens
    int shares;      // of a CTA's tokens, over all segments (set by the launcher, and the five below)
    int per_cta;     // tokens
    int turns;       // CTAs that take these shares
    Divider by_tokens, by_turns, by_page;
    float eps;
    // an append
    const int32_t* starts;  // null: one token per sequence
    const int32_t* past;
    const int32_t* table;
    int64_t table_stride;
    int64_t pages;
    int seqs, max_pages, page_size;
    CacheFormat format;
};
// `append`: the call has a sequence per token, and segments that go to a cache.
cudaError_t launch_heads(HeadsArgs& a, bool f32, bool append, int sms, cudaStream_t st);
// By type, each in a file of its own so that they are compiled side by side.
cudaError_t launch_heads_bf16(HeadsArgs& a, int sms, cudaStream_t st);
cudaError_t launch_heads_f32(HeadsArgs& a, int sms, cudaStream_t st);
cudaError_t launch_append_bf16(HeadsArgs& a, int sms, cudaStream_t st);
cudaError_t launch_append_f32(HeadsArgs& a, int sms, cudaStream_t st);
cudaError_t launch_append_8_bf16(HeadsArgs& a, int sms, cudaStream_t st);
cudaError_t launch_append_8_f32(HeadsArgs& a, int sms, cudaStream_t st);

struct HeadsGradArgs {
    HeadGradSegment seg[2];
    Rotation rope;
    int segments;
    int dim;
    int tokens;
    uint32_t total;
    Divider by_tokens;  // set by the launcher
    float eps;
    float* partials;  // [CTAs][dim]
};
size_t heads_grad_workspace(int64_t dim, int sms);
cudaError_t launch_heads_grad(HeadsGradArgs& a, bool f32, int sms, cudaStream_t st);
// The passes over the rows, by type; a.seg[].ctas partials of each segment are left in a.partials.
cudaError_t launch_heads_grad_bf16(HeadsGradArgs& a, int sms, cudaStream_t st);
cudaError_t launch_heads_grad_f32(HeadsGradArgs& a, int sms, cudaStream_t st);

}  // namespace nf
