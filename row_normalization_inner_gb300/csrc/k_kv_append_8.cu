// Appends of bf16 keys and values to a paged cache of 8-bit rows.
#include "heads_rows.cuh"

namespace nf {

cudaError_t launch_append_8_bf16(HeadsArgs& a, int sms, cudaStream_t st) { return launch_heads_rows<uint16_t, kCache8Bits>(a, sms, st); }

}  // namespace nf
