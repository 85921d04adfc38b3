// Host-side launchers of the token-side row operators: RMSNorm with an
// 8-bit output, the embedding lookup and its gradient, token log
// probabilities and their gradient.  Internal to libnf.so: the entry points
// (api_tokens.cu) validate arguments and call these.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace nf {

// RMSNorm (res null) or fused residual add + RMSNorm with an 8-bit output.
// group: columns that share a scale (kQ8Group), or 0 for the whole row.
constexpr int64_t kQ8MaxHidden = 32768;
constexpr int kQ8Group = 128;
struct Q8Args {
    uint8_t* q;
    float* scale;
    const uint16_t* x;
    uint16_t* res;
    const uint16_t* w;
    int64_t rows;
    int hidden;
    int* status;  // the device status word
    int groups;   // scales per row
    float eps;
};
cudaError_t launch_norm_q8(const Q8Args& a, bool int8, bool grouped, int sms, cudaStream_t st);

// Largest embedding calls.
constexpr int64_t kEmbedMaxHidden = 1 << 20;
constexpr int64_t kEmbedMaxTokens = 0x7FFFFFFF;
constexpr int64_t kEmbedMaxVocab = 1 << 30;
// Embedding lookup: y[i] = bf16(scale * table[ids[i]]).  wide: 64-bit ids.
cudaError_t launch_embedding_fwd(void* y, const void* ids, bool wide, const void* table, int64_t tokens,
                                 int64_t vocab, int64_t hidden, float scale, cudaStream_t st);
// Its gradient: dtable (fp32 or bf16) is overwritten, or added to (add).
size_t embedding_bwd_workspace(int64_t tokens, int64_t hidden, int sms);
cudaError_t launch_embedding_bwd(void* dtable, bool f32, bool add, const void* dy, const void* ids, bool wide,
                                 int64_t tokens, int64_t vocab, int64_t hidden, float scale, void* workspace,
                                 int sms, cudaStream_t st);

// Log probabilities of given tokens with entropy and alternatives (top 0 to
// kLogprobMaxTop), and the gradient.  Strides in elements.
constexpr int64_t kLogprobMaxVocab = 1 << 30;
constexpr int kLogprobMaxTop = 32;
cudaError_t launch_token_logprob_fwd(float* logprob, float* entropy, float* stats, float* top_logprob,
                                     int64_t* top_ids, const void* logits, bool f32, const void* targets,
                                     bool wide, int64_t rows, int64_t vocab, int64_t stride, float temperature,
                                     int top, int sms, cudaStream_t st);
cudaError_t launch_token_logprob_bwd(void* out, const void* logits, bool f32, const void* targets, bool wide,
                                     const float* stats, const float* entropy, const float* d_logprob,
                                     const float* d_entropy, int64_t rows, int64_t vocab, int64_t stride,
                                     int64_t out_stride, float temperature, cudaStream_t st);

}  // namespace nf
