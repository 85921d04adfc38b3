// Appends of fp32 keys and values to a paged cache.
#include "heads_rows.cuh"

namespace nf {

cudaError_t launch_append_f32(HeadsArgs& a, int sms, cudaStream_t st) { return launch_heads_rows<float, true>(a, sms, st); }

}  // namespace nf
