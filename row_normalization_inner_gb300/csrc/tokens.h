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
    int groups;  // scales per row
    float eps;
};
cudaError_t launch_norm_q8(const Q8Args& a, bool int8, bool grouped, int sms, cudaStream_t st);

}  // namespace nf
