// The C-ABI of the calls at the vocabulary matrix: argument checks and
// launches. Declared and documented in include/zdo_vocab.h.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "checks.h"
#include "vocab.h"
#include "zdo_vocab.h"

namespace zdo {
namespace {

bool in_range(int64_t x, int64_t lo, int64_t hi) { return x >= lo && x <= hi; }

int out_of_range(const char *fn, const char *what, int64_t lo, int64_t hi) {
    return fail(ZDO_EINVAL, std::string(fn) + ": " + what + " must be in [" + std::to_string(lo) + ", " +
                                std::to_string(hi) + "]");
}

// The matrix within its parameter: where it starts in the flat buffer, and the
// parameter's elements.
struct Matrix {
    int64_t start = 0, numel = 0;
};

int take_matrix(const zdo_plan *p, int32_t param, int64_t vocab, int64_t dim, const char *fn, Matrix &m) {
    if (param < 0 || size_t(param) >= p->param_numel.size())
        return fail(ZDO_EINVAL, std::string(fn) + ": param_index must be in [0, " +
                                    std::to_string(p->param_numel.size()) + ")");
    if (!in_range(vocab, 1, kVocabMaxRows))
        return out_of_range(fn, "vocab", 1, kVocabMaxRows);
    if (!in_range(dim, 1, kVocabMaxDim))
        return out_of_range(fn, "dim", 1, kVocabMaxDim);
    m.numel = p->param_numel[size_t(param)];
    if (vocab * dim > m.numel)
        return fail(ZDO_EINVAL, std::string(fn) + ": vocab * dim = " + std::to_string(vocab * dim) +
                                    ", but the parameter has " + std::to_string(m.numel) + " elements");
    // parameters lie one after the other in their bucket, and buckets where
    // the plan put them
    size_t bucket = 0;
    int64_t filled = 0;
    for (int32_t i = 0; i < param; ++i) {
        filled += p->param_numel[size_t(i)];
        if (filled >= p->buckets[bucket].numel) {
            ++bucket;
            filled = 0;
        }
    }
    m.start = p->buckets[bucket].offset + filled;
    return ZDO_OK;
}

int check_count(int64_t n, int64_t most, const char *fn) {
    return in_range(n, 0, most) ? ZDO_OK : out_of_range(fn, "n", 0, most);
}

// An array with one element a token; with n = 0 it may be NULL.
int check_array(const void *p, int64_t n, int64_t elem_bytes, const char *fn, const char *what) {
    if (!p && n > 0)
        return fail(ZDO_EINVAL, std::string(fn) + ": " + what + " is NULL");
    if (!aligned_to(p, uintptr_t(elem_bytes)))
        return fail(ZDO_EALIGN, std::string(fn) + ": " + what + " is not " + std::to_string(elem_bytes) +
                                    "-byte aligned");
    return ZDO_OK;
}

int check_type(int32_t type, const char *fn, const char *what) {
    if (type != ZDO_BF16 && type != ZDO_F32)
        return fail(ZDO_EINVAL, std::string(fn) + ": " + what + " must be ZDO_BF16 or ZDO_F32");
    return ZDO_OK;
}

int64_t bytes_of(int32_t type) { return type == ZDO_F32 ? 4 : 2; }

// n rows of dim elements, one every `stride`.
int check_rows(const void *p, int64_t n, int64_t dim, int64_t stride, int32_t type, const char *fn, const char *what) {
    if (int rc = check_array(p, n, bytes_of(type), fn, what))
        return rc;
    if (n > 1 && !in_range(stride, dim, kVocabMaxStride))
        return out_of_range(fn, (std::string(what) + "'s stride").c_str(), dim, kVocabMaxStride);
    return ZDO_OK;
}

// The cross entropy's arguments, as far as W and the number of tokens go.
CeArgs args_at(const uint16_t *w, int64_t vocab, int64_t dim, int64_t n) {
    CeArgs a{};
    a.w = w;
    a.vocab = vocab;
    a.dim = dim;
    a.n = n;
    a.in_place = rows_in_place(w, dim);
    a.layout = ce_layout(n, vocab, dim, a.in_place);
    return a;
}

}  // namespace
}  // namespace zdo

using namespace zdo;

extern "C" {

int embedding_lookup(const zdo_plan *plan, int32_t param_index, int64_t vocab, int64_t dim, const uint16_t *params,
                     const int64_t *tokens, int64_t n, float scale, void *out, int32_t out_type, int64_t out_stride,
                     void *stream) {
    return guarded([&] {
        const char *fn = "embedding_lookup";
        Matrix w;
        if (int rc = check_plan(plan, fn))
            return rc;
        if (int rc = take_matrix(plan, param_index, vocab, dim, fn, w))
            return rc;
        if (int rc = check_count(n, kVocabMaxN, fn))
            return rc;
        if (int rc = check_ptr(params, fn, "params"))
            return rc;
        if (int rc = check_array(tokens, n, 8, fn, "tokens"))
            return rc;
        if (int rc = check_type(out_type, fn, "out_type"))
            return rc;
        if (int rc = check_rows(out, n, dim, out_stride, out_type, fn, "out"))
            return rc;
        Buffers bufs;
        bufs.reads(span_of(params, plan->buffer_numel, 2), "params");
        bufs.reads(span_of(tokens, n, 8), "tokens");
        bufs.writes(span_of_rows(out, n, dim, out_stride, bytes_of(out_type)), "out");
        if (int rc = bufs.check(fn))
            return rc;
        LookupArgs a{};
        a.w = params + w.start;
        a.vocab = vocab;
        a.dim = dim;
        a.tokens = tokens;
        a.n = n;
        a.scale = scale;
        a.out = out;
        a.f32 = out_type == ZDO_F32;
        a.stride = out_stride;
        return launch_result(launch_lookup(a, static_cast<hipStream_t>(stream)), fn);
    });
}

int64_t zdo_embedding_grad_workspace_bytes(int64_t n, int64_t dim) {
    if (!in_range(n, 0, kVocabMaxN) || !in_range(dim, 1, kVocabMaxDim))
        return -1;
    return rows_layout(n, dim).bytes;
}

int embedding_grad(const zdo_plan *plan, int32_t param_index, int64_t vocab, int64_t dim, const int64_t *tokens,
                   int64_t n, const void *grad_out, int32_t grad_type, int64_t grad_stride, float scale,
                   int32_t accumulate, uint16_t *grads, void *workspace, void *stream) {
    return guarded([&] {
        const char *fn = "embedding_grad";
        Matrix w;
        if (int rc = check_plan(plan, fn))
            return rc;
        if (int rc = take_matrix(plan, param_index, vocab, dim, fn, w))
            return rc;
        if (int rc = check_count(n, kVocabMaxN, fn))
            return rc;
        if (int rc = check_array(tokens, n, 8, fn, "tokens"))
            return rc;
        if (int rc = check_type(grad_type, fn, "grad_type"))
            return rc;
        if (int rc = check_rows(grad_out, n, dim, grad_stride, grad_type, fn, "grad_out"))
            return rc;
        if (int rc = check_ptr(grads, fn, "grads"))
            return rc;
        if (int rc = check_ptr(workspace, fn, "workspace"))
            return rc;
        Buffers bufs;
        bufs.reads(span_of(tokens, n, 8), "tokens");
        bufs.reads(span_of_rows(grad_out, n, dim, grad_stride, bytes_of(grad_type)), "grad_out");
        bufs.writes(span_of(grads, plan->buffer_numel, 2), "grads");
        bufs.writes(span_of(workspace, rows_layout(n, dim).bytes, 1), "workspace");
        if (int rc = bufs.check(fn))
            return rc;
        RowsArgs a{};
        a.g = grads + w.start;
        a.numel = w.numel;
        a.vocab = vocab;
        a.dim = dim;
        a.tokens = tokens;
        a.n = n;
        a.x = grad_out;
        a.f32 = grad_type == ZDO_F32;
        a.stride = grad_stride;
        a.scale = scale;
        a.accumulate = accumulate != 0;
        a.workspace = workspace;
        return launch_result(launch_rows(a, static_cast<hipStream_t>(stream)), fn);
    });
}

int64_t zdo_linear_cross_entropy_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
    if (!in_range(n, 0, kCeMaxN) || !in_range(vocab, 1, kVocabMaxRows) || !in_range(dim, 1, kVocabMaxDim))
        return -1;
    return ce_workspace_bytes(n, vocab, dim);
}

int linear_cross_entropy(const zdo_plan *plan, int32_t param_index, int64_t vocab, int64_t dim,
                         const uint16_t *params, const uint16_t *hidden, int64_t hidden_stride,
                         const int64_t *targets, int64_t n, float *loss, float *lse, void *workspace, void *stream) {
    return guarded([&] {
        const char *fn = "linear_cross_entropy";
        Matrix w;
        if (int rc = check_plan(plan, fn))
            return rc;
        if (int rc = take_matrix(plan, param_index, vocab, dim, fn, w))
            return rc;
        if (int rc = check_count(n, kCeMaxN, fn))
            return rc;
        if (int rc = check_ptr(params, fn, "params"))
            return rc;
        if (int rc = check_rows(hidden, n, dim, hidden_stride, ZDO_BF16, fn, "hidden"))
            return rc;
        if (int rc = check_array(targets, n, 8, fn, "targets"))
            return rc;
        if (int rc = check_array(loss, n, 4, fn, "loss"))
            return rc;
        if (int rc = check_array(lse, n, 4, fn, "lse"))
            return rc;
        if (int rc = check_ptr(workspace, fn, "workspace"))
            return rc;
        CeArgs a = args_at(params + w.start, vocab, dim, n);
        Buffers bufs;
        bufs.reads(span_of(params, plan->buffer_numel, 2), "params");
        bufs.reads(span_of_rows(hidden, n, dim, hidden_stride, bytes_of(ZDO_BF16)), "hidden");
        bufs.reads(span_of(targets, n, 8), "targets");
        bufs.writes(span_of(loss, n, 4), "loss");
        bufs.writes(span_of(lse, n, 4), "lse");
        bufs.writes(span_of(workspace, a.layout.bytes, 1), "workspace");
        if (int rc = bufs.check(fn))
            return rc;
        a.hidden = hidden;
        a.hidden_stride = hidden_stride;
        a.targets = targets;
        a.loss = loss;
        a.lse = lse;
        a.workspace = static_cast<char *>(workspace);
        return launch_result(launch_ce(a, static_cast<hipStream_t>(stream)), fn);
    });
}

int linear_cross_entropy_grad(const zdo_plan *plan, int32_t param_index, int64_t vocab, int64_t dim,
                              const uint16_t *params, const uint16_t *hidden, int64_t hidden_stride,
                              const int64_t *targets, int64_t n, const float *lse, const float *grad_loss,
                              void *grad_hidden, int32_t grad_hidden_type, int64_t grad_hidden_stride,
                              int32_t accumulate, uint16_t *grads, void *workspace, void *stream) {
    return guarded([&] {
        const char *fn = "linear_cross_entropy_grad";
        Matrix w;
        if (int rc = check_plan(plan, fn))
            return rc;
        if (int rc = take_matrix(plan, param_index, vocab, dim, fn, w))
            return rc;
        if (int rc = check_count(n, kCeMaxN, fn))
            return rc;
        if (int rc = check_ptr(params, fn, "params"))
            return rc;
        if (int rc = check_rows(hidden, n, dim, hidden_stride, ZDO_BF16, fn, "hidden"))
            return rc;
        if (int rc = check_array(targets, n, 8, fn, "targets"))
            return rc;
        if (int rc = check_array(lse, n, 4, fn, "lse"))
            return rc;
        if (int rc = check_array(grad_loss, n, 4, fn, "grad_loss"))
            return rc;
        if (!grad_hidden && !grads && n > 0)   // with n = 0 an empty grad_hidden may be NULL
            return fail(ZDO_EINVAL, std::string(fn) + ": grad_hidden and grads are both NULL");
        if (grad_hidden) {
            if (int rc = check_type(grad_hidden_type, fn, "grad_hidden_type"))
                return rc;
            if (int rc = check_rows(grad_hidden, n, dim, grad_hidden_stride, grad_hidden_type, fn, "grad_hidden"))
                return rc;
        }
        if (grads)
            if (int rc = check_ptr(grads, fn, "grads"))
                return rc;
        if (int rc = check_ptr(workspace, fn, "workspace"))
            return rc;
        CeArgs a = args_at(params + w.start, vocab, dim, n);
        Buffers bufs;
        bufs.reads(span_of(params, plan->buffer_numel, 2), "params");
        bufs.reads(span_of_rows(hidden, n, dim, hidden_stride, bytes_of(ZDO_BF16)), "hidden");
        bufs.reads(span_of(targets, n, 8), "targets");
        bufs.reads(span_of(lse, n, 4), "lse");
        bufs.reads(span_of(grad_loss, n, 4), "grad_loss");
        if (grad_hidden)
            bufs.writes(span_of_rows(grad_hidden, n, dim, grad_hidden_stride, bytes_of(grad_hidden_type)), "grad_hidden");
        if (grads)
            bufs.writes(span_of(grads, plan->buffer_numel, 2), "grads");
        bufs.writes(span_of(workspace, a.layout.bytes, 1), "workspace");
        if (int rc = bufs.check(fn))
            return rc;
        a.hidden = hidden;
        a.hidden_stride = hidden_stride;
        a.targets = targets;
        a.lse = const_cast<float *>(lse);   // read only by the gradient
        a.grad_loss = grad_loss;
        a.grad_hidden = grad_hidden;
        a.f32 = grad_hidden_type == ZDO_F32;
        a.grad_hidden_stride = grad_hidden_stride;
        a.grads = grads ? grads + w.start : nullptr;
        a.numel = w.numel;
        a.accumulate = accumulate != 0;
        a.workspace = static_cast<char *>(workspace);
        return launch_result(launch_ce_grad(a, static_cast<hipStream_t>(stream)), fn);
    });
}

}  // extern "C"
