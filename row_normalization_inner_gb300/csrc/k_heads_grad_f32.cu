// Gradient of normalized attention heads in fp32.
#include "heads_grad.cuh"

namespace nf {

cudaError_t launch_heads_grad_f32(HeadsGradArgs& a, int sms, cudaStream_t st) { return launch_heads_grad_rows<float>(a, sms, st); }

}  // namespace nf
