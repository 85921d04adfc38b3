// C ABI of the operators on attention heads: argument validation and dispatch.
// As in api.cu, every argument is checked before anything is launched.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "../../include/nf.h"
#include "heads.h"
#include "internal.h"
#include "pair.h"

namespace nf {
namespace {

constexpr int64_t kMostStride = int64_t{1} << 40;
constexpr int64_t kMostRows = 0x7FFFFFFF;
constexpr int64_t kMostSeqs = 1 << 30;
constexpr int64_t kMostHeads = 1 << 20;  // of a set: the kernels step from head to head in 32 bits

// What a set of rows covers: up to three dimensions over rows of `inner`
// bytes.  Extents fit 128 bits whatever the arguments.
using Wide = __int128;
struct Region {
    uintptr_t base;
    int64_t n[3];       // sizes, outer first
    int64_t stride[3];  // in bytes; 0 for dimensions of one
    int64_t inner;
    Wide extent() const {
        Wide e = inner;
        for (int i = 0; i < 3; ++i) e += static_cast<Wide>(n[i] - 1) * stride[i];
        return e;
    }
};

Region region(const void* p, int64_t n0, int64_t n1, int64_t n2, int64_t s0, int64_t s1, int64_t s2, int64_t inner, int64_t size) {
    return {reinterpret_cast<uintptr_t>(p), {n0, n1, n2},
            {n0 > 1 ? s0 * size : 0, n1 > 1 ? s1 * size : 0, n2 > 1 ? s2 * size : 0}, inner * size};
}
Region flat(const void* p, int64_t bytes) { return region(p, 1, 1, 1, 0, 0, 0, bytes, 1); }

bool same(const Region& a, const Region& b) {
    if (a.base != b.base || a.inner != b.inner) return false;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || a.stride[i] != b.stride[i]) return false;
    return true;
}

// Whether two sets share a byte.  A row of b begins `at` bytes behind one of a, at = the
// distance of their bases and so many of every stride: of b's forwards, of a's back.
// The strides are gone through from the largest to the smallest, each only as often
// as what is left of them can make up for.  For sets whose rows do not share bytes
// among themselves that is a few times; where it is not, `tries` run out and the
// sets are taken to overlap.
struct Meeting {
    struct Step {
        Wide by, least, most;  // so many of it
        Wide low, high;        // what the steps behind this one come to
    };
    Step steps[6];
    int n = 0, tries = 256;
    Wide first, last;  // the distances at which two rows share a byte

    Meeting(const Region& a, const Region& b) : first(1 - static_cast<Wide>(b.inner)), last(static_cast<Wide>(a.inner) - 1) {
        for (int d = 0; d < 3; ++d) {
            if (a.stride[d]) add(a.stride[d], 1 - static_cast<Wide>(a.n[d]), 0);
            if (b.stride[d]) add(b.stride[d], 0, static_cast<Wide>(b.n[d]) - 1);
        }
        std::sort(steps, steps + n, [](const Step& x, const Step& y) { return x.by > y.by; });
        Wide low = 0, high = 0;
        for (int i = n - 1; i >= 0; --i) {
            steps[i].low = low, steps[i].high = high;
            low += steps[i].by * steps[i].least, high += steps[i].by * steps[i].most;
        }
    }
    void add(Wide by, Wide least, Wide most) {  // a stride that both have is one step
        for (int i = 0; i < n; ++i)
            if (steps[i].by == by) {
                steps[i].least += least, steps[i].most += most;
                return;
            }
        steps[n++] = {by, least, most, 0, 0};
    }
    static Wide down(Wide x, Wide by) { return x >= 0 ? x / by : -((by - 1 - x) / by); }
    bool at(Wide distance, int i = 0) {
        if (i == n) return first <= distance && distance <= last;
        const Step& s = steps[i];
        Wide from = -down(distance + s.high - first, s.by), to = down(last - s.low - distance, s.by);
        if (from < s.least) from = s.least;
        if (to > s.most) to = s.most;
        for (Wide k = from; k <= to; ++k)
            if (--tries < 0 || at(distance + k * s.by, i + 1)) return true;
        return false;
    }
};

__attribute__((noinline)) bool meet(const Region& a, const Region& b) {
    const Wide delta = static_cast<Wide>(b.base) - static_cast<Wide>(a.base);
    // Mostly (queries beside keys in one buffer) a stride that both have says it at once: within one step of it, what the
    // strides that are no whole multiples of it cover is apart.  (The checks of a rotation in place 0.2 us so, 0.8 without.)
    for (int d = 0; d < 3; ++d) {
        const int64_t step = a.stride[d];
        if (step == 0 || step != b.stride[d] || delta <= -step || delta >= step) continue;
        Wide ea = a.inner, eb = b.inner;
        for (int o = 0; o < 3; ++o) {
            if (a.stride[o] >= step ? a.stride[o] % step : 1) ea += static_cast<Wide>(a.n[o] - 1) * a.stride[o];
            if (b.stride[o] >= step ? b.stride[o] % step : 1) eb += static_cast<Wide>(b.n[o] - 1) * b.stride[o];
        }
        const Wide at = delta < 0 ? delta + step : delta;
        if (at >= ea && at + eb <= step) return false;
    }
    return Meeting(a, b).at(delta);
}

// Whether an output's own rows are apart: in the order of the strides, each
// dimension steps over what the ones inside it cover.
bool rows_apart(const Region& a) {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (a.stride[order[j]] > a.stride[order[j + 1]]) std::swap(order[j], order[j + 1]);
    Wide covered = a.inner;
    for (int d : order) {
        if (a.n[d] <= 1) continue;
        if (a.stride[d] < covered) return false;
        covered += static_cast<Wide>(a.n[d] - 1) * a.stride[d];
    }
    return true;
}

// The regions of a call: each output against everything else.
struct Regions {
    static constexpr int kMost = 24;
    Region r[kMost];
    bool out[kMost];
    int own[kMost];  // an input that the output may be, or the output it may stand for
    Wide behind[kMost];  // the first address behind it
    int n = 0;
    // `twin`: outputs and inputs of the same twin may be one another
    void add(const Region& x, bool is_out, int twin = 0) {
        if (!x.base) return;
        r[n] = x;
        out[n] = is_out;
        behind[n] = x.base + x.extent();
        own[n++] = twin;
    }
    bool sound() const {
        for (int i = 0; i < n; ++i) {
            if (!out[i]) continue;
            if (!rows_apart(r[i])) return false;
            for (int j = 0; j < n; ++j) {
                if (j == i || (out[j] && j < i) || r[j].base >= behind[i] || r[i].base >= behind[j]) continue;
                if (!out[j] && own[i] && own[i] == own[j] && same(r[i], r[j])) continue;
                if (meet(r[i], r[j])) return false;
            }
        }
        return true;
    }
};

bool stride_ok(int64_t s) { return s >= 0 && s <= kMostStride; }
bool heads_ok(const nf_heads* h) {
    return h->heads >= 1 && h->heads <= kMostHeads && stride_ok(h->batch_stride) && stride_ok(h->token_stride) && stride_ok(h->head_stride);
}
Region region_of(const nf_heads* h, int64_t batch, int64_t tokens, int64_t dim, int64_t size) {
    return region(h->data, batch, tokens, h->heads, h->batch_stride, h->token_stride, h->head_stride, dim, size);
}

// The sizes of a call; `heads` over all sets.
nf_status sizes_ok(nf_dtype type, int64_t batch, int64_t tokens, int64_t head_dim, int64_t heads) {
    if (head_dim < 1 || head_dim > kHeadMaxDim) return NF_ERR_UNSUPPORTED_HIDDEN;
    if (type != NF_BF16 && type != NF_F32) return NF_ERR_INVALID_ARG;
    if (batch < 0 || tokens < 0 || batch > kMostRows || tokens > kMostRows || heads < 1 || heads > kMostRows) return NF_ERR_INVALID_ARG;
    if (batch * tokens > kMostRows / heads) return NF_ERR_INVALID_ARG;
    return NF_OK;
}

nf_status rope_ok(const nf_rope* r, int64_t head_dim) {
    if (!r) return NF_OK;
    if (r->dim < 0 || r->dim % 2 || r->dim > head_dim) return NF_ERR_INVALID_ARG;
    if (r->layout != NF_ROPE_HALF && r->layout != NF_ROPE_INTERLEAVED) return NF_ERR_INVALID_ARG;
    if (r->dim == 0) return NF_OK;
    if (!std::isfinite(r->magnitude)) return NF_ERR_INVALID_ARG;
    if (r->positions && ((r->position_bytes != 4 && r->position_bytes != 8) || !stride_ok(r->position_stride))) return NF_ERR_INVALID_ARG;
    return NF_OK;
}
// `places`: without positions, the call has the tokens' places.
nf_status rope_pointers(const nf_rope* r, bool places) {
    if (!r || r->dim == 0) return NF_OK;
    if (!r->rates || (!r->positions && !places)) return NF_ERR_INVALID_ARG;
    if (!aligned(r->rates, 8) || (r->positions && !aligned(r->positions, r->position_bytes))) return NF_ERR_MISALIGNED;
    return NF_OK;
}
void add_rope(Regions& all, const nf_rope* r, int64_t batch, int64_t tokens) {
    if (!r || r->dim == 0) return;
    all.add(flat(r->rates, r->dim / 2 * 8), false);
    if (r->positions) all.add(region(r->positions, batch, 1, 1, r->position_stride, 0, 0, tokens, r->position_bytes), false);
}
Rotation rotation_of(const nf_rope* r, float direction) {
    Rotation x{};
    if (!r || r->dim == 0) return x;
    x.rates = r->rates;
    x.pairs = r->dim / 2;
    x.magnitude = r->magnitude;
    x.direction = direction;
    x.interleaved = r->layout == NF_ROPE_INTERLEAVED;
    x.positions = r->positions;
    x.wide = r->position_bytes == 8;
    x.position_batch = r->position_stride;
    return x;
}

bool eps_ok(float eps) { return std::isfinite(eps) && eps > 0.f; }

// A stride that is ever taken: that of a dimension of one may be anything.
int64_t taken(int64_t stride, int64_t n) { return n > 1 ? stride : 0; }

HeadSegment segment_of(const nf_heads* out, const nf_heads* in, const void* weight, int64_t batch, int64_t tokens) {
    HeadSegment s{};
    s.in = in->data;
    s.in_batch = taken(in->batch_stride, batch), s.in_token = taken(in->token_stride, tokens), s.in_head = taken(in->head_stride, in->heads);
    s.weight = weight;
    s.heads = in->heads;
    s.rotate = true;
    if (out) {
        s.out = out->data;
        s.out_batch = taken(out->batch_stride, batch), s.out_token = taken(out->token_stride, tokens), s.out_head = taken(out->head_stride, in->heads);
    }
    return s;
}

// Rotation with or without the norm: queries and keys to their outputs.
nf_status heads_call(const nf_heads* q_out, const nf_heads* q, const void* q_weight, const nf_heads* k_out, const nf_heads* k,
                     const void* k_weight, bool norm, nf_dtype type, int64_t batch, int64_t tokens, int64_t head_dim, float eps,
                     const nf_rope* rope, float direction, nf_stream stream) {
    if (!q_out || !q || !k_out != !k || (!norm && !rope)) return NF_ERR_INVALID_ARG;
    const nf_heads* outs[2] = {q_out, k_out};
    const nf_heads* ins[2] = {q, k};
    const void* weights[2] = {q_weight, k_weight};
    const int sets = k ? 2 : 1;
    int64_t heads = 0;
    for (int i = 0; i < sets; ++i) {
        if (!heads_ok(outs[i]) || !heads_ok(ins[i]) || outs[i]->heads != ins[i]->heads) return NF_ERR_INVALID_ARG;
        heads += ins[i]->heads;
    }
    if (nf_status st = sizes_ok(type, batch, tokens, head_dim, heads)) return st;
    if (nf_status st = rope_ok(rope, head_dim)) return st;
    if (norm && !eps_ok(eps)) return NF_ERR_INVALID_ARG;
    if (batch * tokens == 0) return NF_OK;
    const int size = type == NF_F32 ? 4 : 2;
    for (int i = 0; i < sets; ++i)
        if (!outs[i]->data || !ins[i]->data || (norm && !weights[i])) return NF_ERR_INVALID_ARG;
    for (int i = 0; i < sets; ++i)
        if (!aligned(outs[i]->data, size) || !aligned(ins[i]->data, size) || (norm && !aligned(weights[i], size))) return NF_ERR_MISALIGNED;
    if (nf_status st = rope_pointers(rope, false)) return st;
    Regions all;
    for (int i = 0; i < sets; ++i) {
        all.add(region_of(outs[i], batch, tokens, head_dim, size), true, i + 1);
        all.add(region_of(ins[i], batch, tokens, head_dim, size), false, i + 1);
        if (norm) all.add(flat(weights[i], head_dim * size), false);
    }
    add_rope(all, rope, batch, tokens);
    if (!all.sound()) return NF_ERR_INVALID_ARG;
    int sms;
    if (nf_status st = device_sm_count(&sms)) return st;
    HeadsArgs a{};
    for (int i = 0; i < sets; ++i) a.seg[i] = segment_of(outs[i], ins[i], norm ? weights[i] : nullptr, batch, tokens);
    a.segments = sets;
    a.rope = rotation_of(rope, direction);
    a.dim = static_cast<int>(head_dim);
    a.tokens = static_cast<int>(tokens);
    a.total = static_cast<uint32_t>(batch * tokens);
    a.eps = eps;
    return from_cuda(launch_heads(a, type == NF_F32, false, sms, reinterpret_cast<cudaStream_t>(stream)));
}

bool pages_ok(const nf_pages* c, bool scaled) {
    return stride_ok(c->page_stride) && stride_ok(c->slot_stride) && stride_ok(c->head_stride) &&
           (!scaled || (stride_ok(c->scale_page_stride) && stride_ok(c->scale_slot_stride) && stride_ok(c->scale_head_stride)));
}

// Radians per position to the share of a turn in units of 2^-64, modulo a turn:
// the nearest one, as far as 104 bits tell.
uint64_t rate_of(Pair frequency) {
    const bool back = frequency.hi < 0.0;
    const Pair turns = (back ? -frequency : frequency) / two_pi();
    const Pair part = turns - std::floor(turns.hi);  // in [-2^-53, 1)
    // in two halves, as 2^64 itself is not an integer that fits
    const double high = std::floor(part.hi * 0x1p32);
    const Pair low = scaled(scaled(part, 32) - high, 32);
    const uint64_t rate = (static_cast<uint64_t>(static_cast<int64_t>(high)) << 32) + static_cast<uint64_t>(std::llround(low.hi + low.lo));
    return back ? ~rate + 1 : rate;
}

}  // namespace
}  // namespace nf

using namespace nf;

extern "C" {

nf_status nf_rope_rates(uint64_t* rates, int32_t dim, double base, nf_rope_scaling scaling, double factor,
                        double length, double low, double high) {
    if (!rates || dim < 2 || dim % 2 || dim > kHeadMaxDim || !(std::isfinite(base) && base > 1.0)) return NF_ERR_INVALID_ARG;
    if (scaling < NF_ROPE_PLAIN || scaling > NF_ROPE_PARTS) return NF_ERR_INVALID_ARG;
    if (scaling != NF_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0)) return NF_ERR_INVALID_ARG;
    if (scaling == NF_ROPE_NTK && (dim < 4 || !std::isfinite(base * std::pow(factor, dim / (dim - 2.0))))) return NF_ERR_INVALID_ARG;
    if (scaling == NF_ROPE_PARTS &&
        !(std::isfinite(length) && length > 0.0 && std::isfinite(low) && std::isfinite(high) && low >= 0.0 && low < high))
        return NF_ERR_INVALID_ARG;
    Pair log_base = logarithm(base);
    if (scaling == NF_ROPE_NTK) log_base = log_base + logarithm(factor) * static_cast<double>(dim) / static_cast<double>(dim - 2);
    for (int i = 0; i < dim / 2; ++i) {
        Pair f = exponential(log_base * (-2.0 * i) / static_cast<double>(dim));
        if (scaling == NF_ROPE_LINEAR) f = f / factor;
        if (scaling == NF_ROPE_PARTS) {
            const Pair keep = (f * length / two_pi() - low) / (Pair(high) - low), slow = f / factor;
            if (keep.hi <= 0.0) f = slow;
            else if (keep.hi < 1.0) f = slow + keep * (f - slow);
        }
        rates[i] = rate_of(f);
    }
    return NF_OK;
}

nf_status nf_rope_rates_of(uint64_t* rates, const double* frequencies, int32_t count) {
    if (!rates || !frequencies || count < 0 || count > kHeadMaxDim / 2) return NF_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i)
        if (!(std::fabs(frequencies[i]) < 0x1p20)) return NF_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) rates[i] = rate_of(frequencies[i]);
    return NF_OK;
}

nf_status nf_rope_fwd(const nf_heads* q_out, const nf_heads* q, const nf_heads* k_out, const nf_heads* k,
                      nf_dtype type, int64_t batch, int64_t tokens, int64_t head_dim, const nf_rope* rope,
                      nf_stream stream) {
    return heads_call(q_out, q, nullptr, k_out, k, nullptr, false, type, batch, tokens, head_dim, 0.f, rope, 1.f, stream);
}

nf_status nf_rope_bwd(const nf_heads* dq, const nf_heads* dq_out, const nf_heads* dk, const nf_heads* dk_out,
                      nf_dtype type, int64_t batch, int64_t tokens, int64_t head_dim, const nf_rope* rope,
                      nf_stream stream) {
    return heads_call(dq, dq_out, nullptr, dk, dk_out, nullptr, false, type, batch, tokens, head_dim, 0.f, rope, -1.f, stream);
}

nf_status nf_qk_rmsnorm_rope_fwd(const nf_heads* q_out, const nf_heads* q, const void* q_weight,
                                 const nf_heads* k_out, const nf_heads* k, const void* k_weight, nf_dtype type,
                                 int64_t batch, int64_t tokens, int64_t head_dim, float eps,
                                 const nf_rope* rope, nf_stream stream) {
    return heads_call(q_out, q, q_weight, k_out, k, k_weight, true, type, batch, tokens, head_dim, eps, rope, 1.f, stream);
}

size_t nf_qk_rmsnorm_rope_bwd_workspace_size(int64_t head_dim) {
    int sms;
    if (head_dim < 1 || head_dim > kHeadMaxDim || device_sm_count(&sms) != NF_OK) return 0;
    return heads_grad_workspace(head_dim, sms);
}

nf_status nf_qk_rmsnorm_rope_bwd(const nf_heads* dq, float* dq_weight, const nf_heads* dq_out, const nf_heads* q,
                                 const void* q_weight, const nf_heads* dk, float* dk_weight,
                                 const nf_heads* dk_out, const nf_heads* k, const void* k_weight, nf_dtype type,
                                 int64_t batch, int64_t tokens, int64_t head_dim, float eps, const nf_rope* rope,
                                 void* workspace, size_t workspace_bytes, nf_stream stream) {
    if (!dq || !dq_out || !q || !dk != !k || !dk_out != !k) return NF_ERR_INVALID_ARG;
    const nf_heads* dxs[2] = {dq, dk};
    const nf_heads* dys[2] = {dq_out, dk_out};
    const nf_heads* xs[2] = {q, k};
    const void* weights[2] = {q_weight, k_weight};
    float* dweights[2] = {dq_weight, dk_weight};
    const int sets = k ? 2 : 1;
    int64_t heads = 0;
    for (int i = 0; i < sets; ++i) {
        if (!heads_ok(dxs[i]) || !heads_ok(dys[i]) || !heads_ok(xs[i])) return NF_ERR_INVALID_ARG;
        if (dxs[i]->heads != xs[i]->heads || dys[i]->heads != xs[i]->heads) return NF_ERR_INVALID_ARG;
        heads += xs[i]->heads;
    }
    if (nf_status st = sizes_ok(type, batch, tokens, head_dim, heads)) return st;
    if (nf_status st = rope_ok(rope, head_dim)) return st;
    if (!eps_ok(eps)) return NF_ERR_INVALID_ARG;
    const bool some = batch * tokens > 0;
    const int size = type == NF_F32 ? 4 : 2;
    for (int i = 0; i < sets; ++i)
        if (!dweights[i] || (some && (!dxs[i]->data || !dys[i]->data || !xs[i]->data || !weights[i]))) return NF_ERR_INVALID_ARG;
    if (!workspace) return NF_ERR_INVALID_ARG;
    for (int i = 0; i < sets; ++i)
        if (!aligned(dweights[i], 4) || (some && (!aligned(dxs[i]->data, size) || !aligned(dys[i]->data, size) ||
                                                  !aligned(xs[i]->data, size) || !aligned(weights[i], size))))
            return NF_ERR_MISALIGNED;
    if (!aligned(workspace, 4)) return NF_ERR_MISALIGNED;
    if (some)
        if (nf_status st = rope_pointers(rope, false)) return st;
    Regions all;
    for (int i = 0; i < sets; ++i) {
        all.add(flat(dweights[i], head_dim * 4), true);
        if (!some) continue;
        all.add(region_of(dxs[i], batch, tokens, head_dim, size), true, i + 1);
        all.add(region_of(dys[i], batch, tokens, head_dim, size), false, i + 1);
        all.add(region_of(xs[i], batch, tokens, head_dim, size), false, i + 1);
        all.add(flat(weights[i], head_dim * size), false);
    }
    if (some) add_rope(all, rope, batch, tokens);
    if (!all.sound()) return NF_ERR_INVALID_ARG;
    int sms;
    if (nf_status st = device_sm_count(&sms)) return st;
    const size_t need = heads_grad_workspace(head_dim, sms);
    if (workspace_bytes < need) return NF_ERR_WORKSPACE_TOO_SMALL;
    all.add(flat(workspace, static_cast<int64_t>(need)), true);
    if (!all.sound()) return NF_ERR_INVALID_ARG;
    HeadsGradArgs a{};
    for (int i = 0; i < sets; ++i) {
        HeadGradSegment& s = a.seg[i];
        s.dx = dxs[i]->data, s.dy = dys[i]->data, s.x = xs[i]->data;
        s.weight = weights[i], s.dweight = dweights[i];
        s.heads = xs[i]->heads;
        s.dx_batch = taken(dxs[i]->batch_stride, batch), s.dx_token = taken(dxs[i]->token_stride, tokens), s.dx_head = taken(dxs[i]->head_stride, s.heads);
        s.dy_batch = taken(dys[i]->batch_stride, batch), s.dy_token = taken(dys[i]->token_stride, tokens), s.dy_head = taken(dys[i]->head_stride, s.heads);
        s.x_batch = taken(xs[i]->batch_stride, batch), s.x_token = taken(xs[i]->token_stride, tokens), s.x_head = taken(xs[i]->head_stride, s.heads);
    }
    a.segments = sets;
    a.rope = rotation_of(rope, -1.f);
    a.dim = static_cast<int>(head_dim);
    a.tokens = static_cast<int>(tokens);
    a.total = static_cast<uint32_t>(batch * tokens);
    a.eps = eps;
    a.partials = static_cast<float*>(workspace);
    return from_cuda(launch_heads_grad(a, type == NF_F32, sms, reinterpret_cast<cudaStream_t>(stream)));
}

nf_status nf_kv_append(const nf_pages* k_cache, const nf_pages* v_cache, nf_cache_type cache_type, int64_t pages,
                       int32_t page_size, const nf_heads* k, const nf_heads* v, const void* k_weight,
                       const nf_heads* q_out, const nf_heads* q, const void* q_weight, nf_dtype type,
                       int64_t tokens, int64_t seqs, int64_t head_dim, const int32_t* starts,
                       const int32_t* past, const int32_t* table, int64_t table_stride, int32_t max_pages,
                       float eps, const nf_rope* rope, nf_stream stream) {
    if (!k_cache || !v_cache || !k || !v || !q_out != !q || (q_weight && !q)) return NF_ERR_INVALID_ARG;
    if (cache_type != NF_CACHE_SAME && cache_type != NF_CACHE_E4M3 && cache_type != NF_CACHE_INT8) return NF_ERR_INVALID_ARG;
    const bool scaled = cache_type != NF_CACHE_SAME;
    if (!heads_ok(k) || !heads_ok(v) || k->heads != v->heads || !pages_ok(k_cache, scaled) || !pages_ok(v_cache, scaled)) return NF_ERR_INVALID_ARG;
    if (q && (!heads_ok(q) || !heads_ok(q_out) || q->heads != q_out->heads)) return NF_ERR_INVALID_ARG;
    const int64_t heads = 2 * static_cast<int64_t>(k->heads) + (q ? q->heads : 0);
    if (nf_status st = sizes_ok(type, 1, tokens, head_dim, heads)) return st;
    if (nf_status st = rope_ok(rope, head_dim)) return st;
    if ((k_weight || q_weight) && !eps_ok(eps)) return NF_ERR_INVALID_ARG;
    if (pages < 0 || pages > kMostRows || page_size < 1 || seqs < 0 || seqs > kMostSeqs || max_pages < 0 ||
        !stride_ok(table_stride) || (seqs > 1 && table_stride < max_pages))
        return NF_ERR_INVALID_ARG;
    if (tokens == 0 || seqs == 0) return NF_OK;
    const int size = type == NF_F32 ? 4 : 2, cell = scaled ? 1 : size;
    if (!k->data || !v->data || !past || (max_pages > 0 && !table) || (q && (!q->data || !q_out->data))) return NF_ERR_INVALID_ARG;
    const nf_pages* caches[2] = {k_cache, v_cache};
    for (const nf_pages* c : caches)
        if (pages > 0 && (!c->data || (scaled && !c->scale))) return NF_ERR_INVALID_ARG;
    if (!aligned(k->data, size) || !aligned(v->data, size) || !aligned(k_weight, size) || !aligned(q_weight, size) ||
        !aligned(starts, 4) || !aligned(past, 4) || !aligned(table, 4) || (q && (!aligned(q->data, size) || !aligned(q_out->data, size))))
        return NF_ERR_MISALIGNED;
    for (const nf_pages* c : caches)
        if (!aligned(c->data, cell) || (scaled && !aligned(c->scale, 4))) return NF_ERR_MISALIGNED;
    if (nf_status st = rope_pointers(rope, true)) return st;
    Regions all;
    if (pages > 0) {
        for (const nf_pages* c : caches) {
            all.add(region(c->data, pages, page_size, k->heads, c->page_stride, c->slot_stride, c->head_stride, head_dim, cell), true);
            if (scaled)
                all.add(region(c->scale, pages, page_size, k->heads, c->scale_page_stride, c->scale_slot_stride, c->scale_head_stride, 1, 4), true);
        }
    }
    if (q) {
        all.add(region_of(q_out, 1, tokens, head_dim, size), true, 1);
        all.add(region_of(q, 1, tokens, head_dim, size), false, 1);
        if (q_weight) all.add(flat(q_weight, head_dim * size), false);
    }
    all.add(region_of(k, 1, tokens, head_dim, size), false);
    all.add(region_of(v, 1, tokens, head_dim, size), false);
    if (k_weight) all.add(flat(k_weight, head_dim * size), false);
    if (starts) all.add(flat(starts, (seqs + 1) * 4), false);
    all.add(flat(past, seqs * 4), false);
    if (max_pages > 0) all.add(region(table, seqs, 1, 1, table_stride, 0, 0, max_pages, 4), false);
    add_rope(all, rope, 1, tokens);
    if (!all.sound()) return NF_ERR_INVALID_ARG;
    int sms;
    if (nf_status st = device_sm_count(&sms)) return st;
    HeadsArgs a{};
    if (q) a.seg[a.segments++] = segment_of(q_out, q, q_weight, 1, tokens);
    for (int i = 0; i < 2; ++i) {
        HeadSegment& s = a.seg[a.segments++];
        s = segment_of(nullptr, i ? v : k, i ? nullptr : k_weight, 1, tokens);
        const nf_pages* c = caches[i];
        s.out = c->data;
        s.out_batch = taken(c->page_stride, pages), s.out_token = taken(c->slot_stride, page_size), s.out_head = taken(c->head_stride, k->heads);
        s.scale = c->scale;
        s.scale_page = c->scale_page_stride, s.scale_slot = c->scale_slot_stride, s.scale_head = c->scale_head_stride;
        s.rotate = i == 0;
        s.cache = true;
    }
    a.rope = rotation_of(rope, 1.f);
    a.dim = static_cast<int>(head_dim);
    a.tokens = static_cast<int>(tokens);
    a.total = static_cast<uint32_t>(tokens);
    a.eps = eps;
    a.starts = starts;
    a.past = past;
    a.table = table;
    a.table_stride = table_stride;
    a.pages = pages;
    a.seqs = static_cast<int>(seqs);
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.format = static_cast<CacheFormat>(cache_type);
    return from_cuda(launch_heads(a, type == NF_F32, true, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
