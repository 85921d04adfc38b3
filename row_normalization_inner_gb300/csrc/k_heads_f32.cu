// Rotation and norm of attention heads in fp32.
#include "heads_rows.cuh"

namespace nf {

cudaError_t launch_heads_f32(HeadsArgs& a, int sms, cudaStream_t st) { return launch_heads_rows<float, kNoCache>(a, sms, st); }

}  // namespace nf
