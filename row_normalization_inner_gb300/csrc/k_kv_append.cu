// Appends of bf16 keys and values to a paged cache of their type.
#include "heads_rows.cuh"

namespace nf {

cudaError_t launch_append_bf16(HeadsArgs& a, int sms, cudaStream_t st) { return launch_heads_rows<uint16_t, kCacheOfType>(a, sms, st); }

}  // namespace nf
