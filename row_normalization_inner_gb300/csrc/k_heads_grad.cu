// Gradient of normalized attention heads (bf16), the last sum of the weights'
// gradients, and the choice of the type.
#include "heads_grad.cuh"

namespace nf {
namespace {

// dweight: the sum of a segment's partials, V columns to a CTA.  A thread adds up
// every 256th partial, all of them on their way at once (two of 456), then the
// warp its lanes' and the CTA its warps', in a fixed order (456 partials of 128
// columns, cold and alone: 5.4 us; with 32 columns to a CTA of 32 warps the sums took
// 2.5 times as long).
constexpr int kSumThreads = 256;
template <int V>
__global__ void __launch_bounds__(kSumThreads) heads_grad_sum(const __grid_constant__ HeadsGradArgs a) {
    __shared__ float part[kSumThreads / 32][V];
    grid_dep_wait();
    grid_dep_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, column = blockIdx.x * V;
    const HeadGradSegment& s = a.seg[blockIdx.y];
    const float* from = a.partials + static_cast<int64_t>(blockIdx.y ? a.seg[0].ctas : 0) * a.dim + column;
    float sum[V] = {};
#pragma unroll 4
    for (int p = threadIdx.x; p < s.ctas; p += kSumThreads) {
        if constexpr (V == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(from + static_cast<int64_t>(p) * a.dim));
            sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
        } else {
            sum[0] += __ldcg(from + static_cast<int64_t>(p) * a.dim);
        }
    }
    warp_sum<V>(sum);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) part[warp][i] = sum[i];
    }
    __syncthreads();
    if (threadIdx.x < V) {
        float t = part[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kSumThreads / 32; ++w) t += part[w][threadIdx.x];
        s.dweight[column + threadIdx.x] = t;
    }
}

}  // namespace

size_t heads_grad_workspace(int64_t dim, int sms) {
    return static_cast<size_t>(sms) * kCtasPerSm * static_cast<size_t>(dim) * sizeof(float);
}

cudaError_t launch_heads_grad_bf16(HeadsGradArgs& a, int sms, cudaStream_t st) { return launch_heads_grad_rows<uint16_t>(a, sms, st); }

cudaError_t launch_heads_grad(HeadsGradArgs& a, bool f32, int sms, cudaStream_t st) {
    if (const cudaError_t e = f32 ? launch_heads_grad_f32(a, sms, st) : launch_heads_grad_bf16(a, sms, st)) return e;
    return a.dim % 4 || reinterpret_cast<uintptr_t>(a.partials) % 16
               ? launch_with_pdl(heads_grad_sum<1>, dim3(a.dim, a.segments), dim3(kSumThreads), 0, st, a)
               : launch_with_pdl(heads_grad_sum<4>, dim3(a.dim / 4, a.segments), dim3(kSumThreads), 0, st, a);
}

}  // namespace nf
