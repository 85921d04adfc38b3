// C ABI of the token-side row operators: argument validation and dispatch.
// As in api.cu, every argument is checked before anything is launched.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/nf.h"
#include "internal.h"
#include "tokens.h"

namespace nf {
namespace {

nf_status norm_q8(void* q, float* scale, const void* x, void* residual, bool fused, const void* weight,
                  int64_t rows, int64_t hidden, float eps, nf_q8_format format, int64_t group,
                  nf_stream stream) {
    if (hidden < 8 || hidden % 8 != 0 || hidden > kQ8MaxHidden) return NF_ERR_UNSUPPORTED_HIDDEN;
    if (rows < 0 || rows > (INT64_MAX / 8) / hidden) return NF_ERR_INVALID_ARG;
    if (!(std::isfinite(eps) && eps > 0.f)) return NF_ERR_INVALID_ARG;
    if (format != NF_Q8_E4M3 && format != NF_Q8_INT8) return NF_ERR_INVALID_ARG;
    if (group != 0 && group != kQ8Group) return NF_ERR_INVALID_ARG;
    if (rows == 0) return NF_OK;
    if (!q || !scale || !x || !weight || (fused && !residual)) return NF_ERR_INVALID_ARG;
    if (!aligned(q, 8) || !aligned(scale, 4) || !aligned(x, 16) || !aligned(weight, 16) ||
        !aligned(residual, 16))
        return NF_ERR_MISALIGNED;
    const int64_t groups = group ? (hidden + group - 1) / group : 1;
    const int64_t act = rows * hidden * 2;
    const Span outs[] = {{q, rows * hidden}, {scale, rows * groups * 4}, {residual, fused ? act : 0}};
    const Span ins[] = {{x, act}, {weight, hidden * 2}};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return NF_ERR_INVALID_ARG;
        for (const Span& in : ins)
            if (overlap(outs[i], in)) return NF_ERR_INVALID_ARG;
    }
    int sms;
    if (nf_status st = device_sm_count(&sms)) return st;
    Q8Args a{};
    a.q = static_cast<uint8_t*>(q);
    a.scale = scale;
    a.x = static_cast<const uint16_t*>(x);
    a.res = fused ? static_cast<uint16_t*>(residual) : nullptr;
    a.w = static_cast<const uint16_t*>(weight);
    a.rows = rows;
    a.hidden = static_cast<int>(hidden);
    a.groups = static_cast<int>(groups);
    a.eps = eps;
    return from_cuda(launch_norm_q8(a, format == NF_Q8_INT8, group != 0, sms,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace nf

using namespace nf;

extern "C" {

nf_status nf_rmsnorm_q8(void* q, float* scale, const void* x, const void* weight, int64_t rows,
                        int64_t hidden, float eps, nf_q8_format format, int64_t group,
                        nf_stream stream) {
    return norm_q8(q, scale, x, nullptr, false, weight, rows, hidden, eps, format, group, stream);
}

nf_status nf_fused_add_rmsnorm_q8(void* q, float* scale, const void* x, void* residual,
                                  const void* weight, int64_t rows, int64_t hidden, float eps,
                                  nf_q8_format format, int64_t group, nf_stream stream) {
    return norm_q8(q, scale, x, residual, true, weight, rows, hidden, eps, format, group, stream);
}

}  // extern "C"
