// Appends of f32 keys and values to a paged cache of their type.
#include "heads_rows.cuh"

namespace nf {

cudaError_t launch_append_f32(HeadsArgs& a, int sms, cudaStream_t st) { return launch_heads_rows<float, kCacheOfType>(a, sms, st); }

}  // namespace nf
