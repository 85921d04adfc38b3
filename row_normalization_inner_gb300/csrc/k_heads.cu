// Rotation and norm of attention heads (bf16), and the choice of the type.
#include "heads_rows.cuh"

namespace nf {

cudaError_t launch_heads_bf16(HeadsArgs& a, int sms, cudaStream_t st) { return launch_heads_rows<uint16_t, kNoCache>(a, sms, st); }

cudaError_t launch_heads(HeadsArgs& a, bool f32, bool append, int sms, cudaStream_t st) {
    if (!append) return f32 ? launch_heads_f32(a, sms, st) : launch_heads_bf16(a, sms, st);
    if (a.format == kCacheSame) return f32 ? launch_append_f32(a, sms, st) : launch_append_bf16(a, sms, st);
    return f32 ? launch_append_8_f32(a, sms, st) : launch_append_8_bf16(a, sms, st);
}

}  // namespace nf
