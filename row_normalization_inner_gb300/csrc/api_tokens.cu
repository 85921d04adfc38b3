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
    if (nf_status st = device_status_addr(&a.status)) return st;
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

// The sizes an embedding call takes: token numbers and table rows are kept in
// 32 bits (a row number of the table's size marks tokens without a row).
nf_status embedding_checks(int64_t tokens, int64_t vocab, int64_t hidden, float scale, int32_t id_bytes) {
    if (hidden < 8 || hidden % 8 != 0 || hidden > kEmbedMaxHidden) return NF_ERR_UNSUPPORTED_HIDDEN;
    if (tokens < 0 || tokens > kEmbedMaxTokens || vocab < 1 || vocab > kEmbedMaxVocab)
        return NF_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || (id_bytes != 4 && id_bytes != 8)) return NF_ERR_INVALID_ARG;
    return NF_OK;
}

nf_status logprob_checks(nf_dtype type, int32_t id_bytes, int64_t rows, int64_t vocab, int64_t stride,
                         float temperature) {
    if ((type != NF_BF16 && type != NF_F32) || (id_bytes != 4 && id_bytes != 8)) return NF_ERR_INVALID_ARG;
    if (rows < 0 || vocab < 1 || vocab > kLogprobMaxVocab || stride < vocab) return NF_ERR_INVALID_ARG;
    // every size in bytes stays in 64 bits (the alternatives of a row take 8 * kLogprobMaxTop)
    constexpr int64_t kMost = INT64_MAX / (8 * kLogprobMaxTop);
    if (stride > kMost || rows > kMost / stride) return NF_ERR_INVALID_ARG;
    if (!(temperature >= 0x1p-64f && temperature <= 0x1p64f)) return NF_ERR_INVALID_ARG;
    return NF_OK;
}

// Bytes from a strided matrix's first element to behind its last.
int64_t strided_bytes(int64_t rows, int64_t vocab, int64_t stride, int64_t size) {
    return ((rows - 1) * stride + vocab) * size;
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

nf_status nf_embedding_fwd(void* y, const void* ids, int32_t id_bytes, const void* table, int64_t tokens,
                           int64_t vocab, int64_t hidden, float scale, nf_stream stream) {
    if (nf_status st = embedding_checks(tokens, vocab, hidden, scale, id_bytes)) return st;
    if (tokens == 0) return NF_OK;
    if (!y || !ids || !table) return NF_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(table, 16) || !aligned(ids, id_bytes)) return NF_ERR_MISALIGNED;
    const Span out{y, tokens * hidden * 2};
    if (overlap(out, {ids, tokens * id_bytes}) || overlap(out, {table, vocab * hidden * 2}))
        return NF_ERR_INVALID_ARG;
    return from_cuda(launch_embedding_fwd(y, ids, id_bytes == 8, table, tokens, vocab, hidden, scale,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

size_t nf_embedding_bwd_workspace_size(int64_t tokens, int64_t hidden) {
    if (tokens <= 0 || tokens > kEmbedMaxTokens || hidden < 8 || hidden % 8 != 0 || hidden > kEmbedMaxHidden)
        return 0;
    int sms;
    if (device_sm_count(&sms) != NF_OK) return 0;
    return embedding_bwd_workspace(tokens, hidden, sms);
}

nf_status nf_embedding_bwd(void* dtable, nf_dtype dtable_type, int32_t accumulate, const void* dy,
                           const void* ids, int32_t id_bytes, int64_t tokens, int64_t vocab, int64_t hidden,
                           float scale, void* workspace, size_t workspace_bytes, nf_stream stream) {
    if (nf_status st = embedding_checks(tokens, vocab, hidden, scale, id_bytes)) return st;
    if ((dtable_type != NF_BF16 && dtable_type != NF_F32) || (accumulate != 0 && accumulate != 1))
        return NF_ERR_INVALID_ARG;
    if (tokens == 0 && accumulate) return NF_OK;
    if (!dtable || (tokens > 0 && (!dy || !ids || !workspace))) return NF_ERR_INVALID_ARG;
    if (!aligned(dtable, 16) || !aligned(dy, 16) || !aligned(ids, id_bytes) || !aligned(workspace, 16))
        return NF_ERR_MISALIGNED;
    int sms;
    if (nf_status st = device_sm_count(&sms)) return st;
    const size_t need = tokens ? embedding_bwd_workspace(tokens, hidden, sms) : 0;
    if (workspace_bytes < need) return NF_ERR_WORKSPACE_TOO_SMALL;
    const Span grad{dtable, vocab * hidden * (dtable_type == NF_F32 ? 4 : 2)};
    const Span ws{workspace, static_cast<int64_t>(need)};
    for (const Span& in : {Span{dy, tokens * hidden * 2}, Span{ids, tokens * id_bytes}})
        if (overlap(grad, in) || overlap(ws, in)) return NF_ERR_INVALID_ARG;
    if (overlap(grad, ws)) return NF_ERR_INVALID_ARG;
    return from_cuda(launch_embedding_bwd(dtable, dtable_type == NF_F32, accumulate != 0, dy, ids, id_bytes == 8,
                                          tokens, vocab, hidden, scale, workspace, sms,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

nf_status nf_token_logprob_fwd(float* logprob, float* entropy, float* stats, float* top_logprob,
                               int64_t* top_ids, const void* logits, nf_dtype type, int64_t stride,
                               const void* targets, int32_t id_bytes, int64_t rows, int64_t vocab,
                               float temperature, int32_t top, nf_stream stream) {
    if (nf_status st = logprob_checks(type, id_bytes, rows, vocab, stride, temperature)) return st;
    if (top < 0 || top > kLogprobMaxTop) return NF_ERR_INVALID_ARG;
    if (rows == 0) return NF_OK;
    if (!logprob || !entropy || !stats || !logits || !targets || (top && (!top_logprob || !top_ids)))
        return NF_ERR_INVALID_ARG;
    const int size = type == NF_F32 ? 4 : 2;
    if (!aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(stats, 8) || !aligned(logits, size) ||
        !aligned(targets, id_bytes) || (top && (!aligned(top_logprob, 4) || !aligned(top_ids, 8))))
        return NF_ERR_MISALIGNED;
    const Span outs[] = {{logprob, rows * 4}, {entropy, rows * 4}, {stats, rows * 8},
                         {top ? top_logprob : nullptr, rows * top * 4}, {top ? top_ids : nullptr, rows * top * 8}};
    const Span ins[] = {{logits, strided_bytes(rows, vocab, stride, size)}, {targets, rows * id_bytes}};
    for (int i = 0; i < 5; ++i) {
        for (int j = i + 1; j < 5; ++j)
            if (overlap(outs[i], outs[j])) return NF_ERR_INVALID_ARG;
        for (const Span& in : ins)
            if (overlap(outs[i], in)) return NF_ERR_INVALID_ARG;
    }
    int sms;
    if (nf_status st = device_sm_count(&sms)) return st;
    return from_cuda(launch_token_logprob_fwd(logprob, entropy, stats, top_logprob, top_ids, logits,
                                              type == NF_F32, targets, id_bytes == 8, rows, vocab, stride,
                                              temperature, top, sms, reinterpret_cast<cudaStream_t>(stream)));
}

nf_status nf_token_logprob_bwd(void* dlogits, int64_t dstride, const void* logits, nf_dtype type,
                               int64_t stride, const void* targets, int32_t id_bytes, const float* stats,
                               const float* entropy, const float* d_logprob, const float* d_entropy,
                               int64_t rows, int64_t vocab, float temperature, nf_stream stream) {
    if (nf_status st = logprob_checks(type, id_bytes, rows, vocab, stride, temperature)) return st;
    if (nf_status st = logprob_checks(type, id_bytes, rows, vocab, dstride, temperature)) return st;
    if (rows == 0) return NF_OK;
    if (!dlogits || !logits || !targets || !stats || !d_logprob || (d_entropy && !entropy)) return NF_ERR_INVALID_ARG;
    const int size = type == NF_F32 ? 4 : 2;
    if (!aligned(dlogits, size) || !aligned(logits, size) || !aligned(targets, id_bytes) || !aligned(stats, 8) ||
        !aligned(d_logprob, 4) || !aligned(d_entropy, 4) || (d_entropy && !aligned(entropy, 4)))
        return NF_ERR_MISALIGNED;
    const Span out{dlogits, strided_bytes(rows, vocab, dstride, size)};
    // dlogits may be the logits themselves: every element is read before it is written, by the thread that writes it
    if (!(dlogits == logits && dstride == stride) && overlap(out, {logits, strided_bytes(rows, vocab, stride, size)}))
        return NF_ERR_INVALID_ARG;
    for (const Span& in : {Span{targets, rows * id_bytes}, Span{stats, rows * 8}, Span{d_logprob, rows * 4},
                           Span{d_entropy, rows * 4}, Span{d_entropy ? entropy : nullptr, rows * 4}})
        if (overlap(out, in)) return NF_ERR_INVALID_ARG;
    return from_cuda(launch_token_logprob_bwd(dlogits, logits, type == NF_F32, targets, id_bytes == 8, stats,
                                              entropy, d_logprob, d_entropy, rows, vocab, stride, dstride,
                                              temperature, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
