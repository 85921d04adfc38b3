// Appends of f32 keys and values to a paged cache of 8-bit rows.
#include "heads_rows.cuh"

namespace nf {

cudaError_t launch_append_8_f32(HeadsArgs& a, int sms, cudaStream_t st) { return launch_heads_rows<float, kCache8Bits>(a, sms, st); }

}  // namespace nf
