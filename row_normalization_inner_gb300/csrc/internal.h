// Entry-point internals shared between the C ABI translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nf.h"

namespace nf {

// SM count of the current device, cached per device.
nf_status device_sm_count(int* sms);

// Address of the current device's status word, cached per device.
nf_status device_status_addr(int** addr);

inline nf_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NF_OK : NF_ERR_CUDA; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Span {
    const void* p;
    int64_t bytes;
};

inline bool overlap(Span a, Span b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

// Overlap allowed only as the exact same buffer.
inline bool bad_overlap_except_alias(Span out, Span in) {
    if (out.p == in.p && out.bytes == in.bytes) return false;
    return overlap(out, in);
}

// The LayerNorm backward behind nf_layernorm_bwd and
// nf_layernorm_bwd_noalloc.  With `scratch` null it is nf_layernorm_bwd.
// With `scratch` set, the workspace is a fixed area of `workspace_bytes`
// bytes owned by the library: `workspace` is ignored, every argument is
// checked first, a plan whose partials need more than the area returns
// NF_ERR_WORKSPACE_TOO_SMALL, and only then is the area's address fetched
// with scratch().
nf_status layernorm_bwd_impl(void* dx, float* dgamma, float* dbeta, const void* dy, const void* x,
                             const float* mean, const float* rstd, const void* gamma, int64_t rows,
                             int64_t hidden, void* workspace, size_t workspace_bytes,
                             nf_status (*scratch)(void**), nf_stream stream);

}  // namespace nf
