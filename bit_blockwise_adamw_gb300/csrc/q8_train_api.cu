// q8_train_api.cu -- the extern "C" entry points declared in
// include/q8train.h: argument checks, then the launchers.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <new>
#include <vector>

#include "q8_internal.h"
#include "q8_train.h"

namespace {

using q8::cuda_fail;
using q8::fail;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxSize = int64_t(1) << 30;
constexpr int64_t kMaxTokens = int64_t(1) << 40;

// A row matrix: non-NULL (unless it has no rows), on its element's own
// alignment, rows that do not overlap.
int check_rows(const void* p, int64_t elem, int64_t rows, int64_t cols, int64_t stride, const char* name)
{
    if (rows == 0) return Q8_OK;
    if (!p) return fail(Q8_ERR_NULL, std::string(name) + " is NULL");
    if (!aligned(p, static_cast<uintptr_t>(elem))) return fail(Q8_ERR_ALIGN, std::string(name) + " is not aligned to its elements");
    if (stride < cols || stride >= kMaxTokens) return fail(Q8_ERR_SIZE, std::string(name) + "'s row stride must be at least its row's length, and below 2^40");
    return Q8_OK;
}

int check_vec(const void* p, const char* name)
{
    if (!aligned(p, 2)) return fail(Q8_ERR_ALIGN, std::string(name) + " must be 2-byte aligned");
    return Q8_OK;
}

int check_workspace(const void* p, int64_t have, int64_t need)
{
    if (need == 0) return Q8_OK;
    if (!p) return fail(Q8_ERR_NULL, "workspace is NULL");
    if (!aligned(p, 256)) return fail(Q8_ERR_ALIGN, "workspace must be 256-byte aligned");
    if (have < need) return fail(Q8_ERR_SIZE, "workspace_bytes is less than the call needs");
    return Q8_OK;
}

int check_ff(const q8_gated_ff* f)
{
    if (!f) return fail(Q8_ERR_NULL, "q8_gated_ff is NULL");
    if (f->tokens < 0 || f->tokens >= kMaxSize) return fail(Q8_ERR_SIZE, "tokens must lie in [0, 2^30)");
    if (f->d_model < 1 || f->d_model >= kMaxSize || f->d_ff < 1 || f->d_ff >= kMaxSize)
        return fail(Q8_ERR_SIZE, "d_model and d_ff must lie in [1, 2^30)");
    if (f->act != Q8_SILU && f->act != Q8_GELU_TANH && f->act != Q8_GELU)
        return fail(Q8_ERR_ARG, "act must be Q8_SILU, Q8_GELU_TANH or Q8_GELU");
    int rc = check_rows(f->x, 2, f->tokens, f->d_model, f->x_stride, "x");
    if (rc == Q8_OK) rc = check_rows(f->w_gate, 2, f->d_ff, f->d_model, f->d_model, "w_gate");
    if (rc == Q8_OK) rc = check_rows(f->w_up, 2, f->d_ff, f->d_model, f->d_model, "w_up");
    return rc;
}

int check_norm(const q8_block_norm* n)
{
    if (!n) return fail(Q8_ERR_NULL, "q8_block_norm is NULL");
    if (n->tokens < 0 || n->tokens >= kMaxTokens) return fail(Q8_ERR_SIZE, "tokens must lie in [0, 2^40)");
    if (n->dim < 1 || n->dim > Q8_NORM_MAX_DIM) return fail(Q8_ERR_SIZE, "dim must lie in [1, Q8_NORM_MAX_DIM]");
    for (int k : {n->post_kind, n->pre_kind})
        if (k != Q8_NORM_NONE && k != Q8_NORM_RMS && k != Q8_NORM_LAYER)
            return fail(Q8_ERR_ARG, "post_kind and pre_kind must be Q8_NORM_NONE, Q8_NORM_RMS or Q8_NORM_LAYER");
    if (n->residual_dtype != Q8_BF16 && n->residual_dtype != Q8_F32)
        return fail(Q8_ERR_ARG, "residual_dtype must be Q8_BF16 or Q8_F32");
    if (!std::isfinite(n->eps) || n->eps < 0.0f) return fail(Q8_ERR_ARG, "eps must be finite and >= 0");
    if (!std::isfinite(n->residual_scale)) return fail(Q8_ERR_ARG, "residual_scale must be finite");
    if ((n->post_kind == Q8_NORM_NONE && (n->post_weight || n->post_bias)) ||
        (n->pre_kind == Q8_NORM_NONE && (n->pre_weight || n->pre_bias)))
        return fail(Q8_ERR_ARG, "a Q8_NORM_NONE norm takes no weight and no bias");
    if (n->gate && (n->gate_tokens < 1 || n->gate_tokens >= kMaxTokens))
        return fail(Q8_ERR_SIZE, "gate_tokens must lie in [1, 2^40)");
    int rc = check_rows(n->residual, n->residual_dtype == Q8_F32 ? 4 : 2, n->tokens, n->dim, n->residual_stride, "residual");
    if (rc == Q8_OK) rc = check_rows(n->y, 2, n->tokens, n->dim, n->y_stride, "y");
    const struct { const void* p; const char* name; } vecs[] = {
        {n->post_weight, "post_weight"}, {n->post_bias, "post_bias"}, {n->pre_weight, "pre_weight"},
        {n->pre_bias, "pre_bias"}, {n->gate, "gate"}};
    for (const auto& v : vecs)
        if (rc == Q8_OK) rc = check_vec(v.p, v.name);
    return rc;
}

int check_norm_grads(const q8_block_norm* n, const q8_block_norm_grads* g)
{
    if (!g) return fail(Q8_ERR_NULL, "q8_block_norm_grads is NULL");
    if ((n->post_kind == Q8_NORM_NONE && (g->d_post_weight || g->d_post_bias)) ||
        (n->pre_kind == Q8_NORM_NONE && (g->d_pre_weight || g->d_pre_bias)) || (!n->gate && g->d_gate))
        return fail(Q8_ERR_ARG, "a gradient is asked for that has nothing to be the gradient of");
    const int64_t re = n->residual_dtype == Q8_F32 ? 4 : 2;
    const struct { const void* p; int64_t elem, stride; const char* name; } rows[] = {
        {g->d_residual_out, re, g->d_residual_out_stride, "d_residual_out"}, {g->dz, 2, g->dz_stride, "dz"},
        {g->d_residual, re, g->d_residual_stride, "d_residual"}, {g->d_y, 2, g->d_y_stride, "d_y"}};
    int rc = Q8_OK;
    for (const auto& r : rows)
        if (rc == Q8_OK && r.p) rc = check_rows(r.p, r.elem, n->tokens, n->dim, r.stride, r.name);
    const struct { const void* p; const char* name; } vecs[] = {
        {g->d_post_weight, "d_post_weight"}, {g->d_post_bias, "d_post_bias"}, {g->d_pre_weight, "d_pre_weight"},
        {g->d_pre_bias, "d_pre_bias"}, {g->d_gate, "d_gate"}};
    for (const auto& v : vecs)
        if (rc == Q8_OK) rc = check_vec(v.p, v.name);
    return rc;
}

int check_distill(const q8_distill_topk* d)
{
    if (!d) return fail(Q8_ERR_NULL, "q8_distill_topk is NULL");
    if (d->rows < 0 || d->rows >= kMaxTokens) return fail(Q8_ERR_SIZE, "rows must lie in [0, 2^40)");
    if (d->vocab < 1 || d->vocab >= (int64_t(1) << 31)) return fail(Q8_ERR_SIZE, "vocab must lie in [1, 2^31)");
    if (d->k < 0 || d->k > Q8_DISTILL_MAX_K) return fail(Q8_ERR_SIZE, "k must lie in [0, Q8_DISTILL_MAX_K]");
    if (d->logits_dtype != Q8_BF16 && d->logits_dtype != Q8_F32)
        return fail(Q8_ERR_ARG, "logits_dtype must be Q8_BF16 or Q8_F32");
    if (!std::isfinite(d->temperature) || d->temperature <= 0.0f) return fail(Q8_ERR_ARG, "temperature must be finite and > 0");
    if (!std::isfinite(d->kd_weight) || d->kd_weight < 0.0f || !std::isfinite(d->ce_weight) || d->ce_weight < 0.0f)
        return fail(Q8_ERR_ARG, "kd_weight and ce_weight must be finite and >= 0");
    int rc = check_rows(d->logits, d->logits_dtype == Q8_F32 ? 4 : 2, d->rows, d->vocab, d->logits_stride, "logits");
    if (rc != Q8_OK || d->rows == 0) return rc;
    if (d->k > 0 && (!d->teacher_ids || !d->teacher_logits)) return fail(Q8_ERR_NULL, "teacher_ids and teacher_logits must be non-NULL");
    if (!aligned(d->teacher_ids, 8) || !aligned(d->labels, 8)) return fail(Q8_ERR_ALIGN, "teacher_ids and labels must be 8-byte aligned");
    if (!aligned(d->teacher_logits, 4) || !aligned(d->row_weight, 4))
        return fail(Q8_ERR_ALIGN, "teacher_logits and row_weight must be 4-byte aligned");
    return Q8_OK;
}

int check_embedding(const q8_embedding* e)
{
    if (!e) return fail(Q8_ERR_NULL, "q8_embedding is NULL");
    if (e->tokens < 0 || e->tokens >= kMaxSize) return fail(Q8_ERR_SIZE, "tokens must lie in [0, 2^30)");
    if (e->vocab < 1 || e->vocab >= (int64_t(1) << 31)) return fail(Q8_ERR_SIZE, "vocab must lie in [1, 2^31)");
    if (e->dim < 1 || e->dim >= kMaxSize) return fail(Q8_ERR_SIZE, "dim must lie in [1, 2^30)");
    if (e->dtype != Q8_BF16 && e->dtype != Q8_F32) return fail(Q8_ERR_ARG, "dtype must be Q8_BF16 or Q8_F32");
    if (!std::isfinite(e->scale)) return fail(Q8_ERR_ARG, "scale must be finite");
    if (e->tokens > 0 && !e->ids) return fail(Q8_ERR_NULL, "ids is NULL");
    if (!aligned(e->ids, 8)) return fail(Q8_ERR_ALIGN, "ids must be 8-byte aligned");
    return Q8_OK;
}

std::string entry(const char* what, int i) { return std::string(what) + " (gradient " + std::to_string(i) + ")"; }

int check_grads(const q8_grad* list, int count, bool clip)
{
    if (count < 0) return fail(Q8_ERR_SIZE, "count must be >= 0");
    if (count > 0 && !list) return fail(Q8_ERR_NULL, "list is NULL");
    for (int i = 0; i < count; ++i) {
        const q8_grad& g = list[i];
        if (g.numel < 0 || g.numel >= kMaxTokens) return fail(Q8_ERR_SIZE, entry("numel must lie in [0, 2^40)", i));
        if (g.grad_dtype != Q8_BF16 && g.grad_dtype != Q8_F32)
            return fail(Q8_ERR_ARG, entry("grad_dtype must be Q8_BF16 or Q8_F32", i));
        if (clip && g.out_dtype != Q8_BF16 && g.out_dtype != Q8_F32)
            return fail(Q8_ERR_ARG, entry("out_dtype must be Q8_BF16 or Q8_F32", i));
        if (g.numel == 0) continue;
        if (!g.grad) return fail(Q8_ERR_NULL, entry("grad is NULL", i));
        if (!aligned(g.grad, g.grad_dtype == Q8_F32 ? 4 : 2)) return fail(Q8_ERR_ALIGN, entry("grad is not aligned to its elements", i));
        if (!clip) continue;
        if (!g.out) return fail(Q8_ERR_NULL, entry("out is NULL", i));
        if (!aligned(g.out, g.out_dtype == Q8_F32 ? 4 : 2)) return fail(Q8_ERR_ALIGN, entry("out is not aligned to its elements", i));
        if (g.out == g.grad && g.out_dtype != g.grad_dtype) return fail(Q8_ERR_ARG, entry("out over grad must have grad's type", i));
    }
    return Q8_OK;
}

// What clipping writes, in bytes, and the entry that it is of.
struct Span {
    uintptr_t begin, end;
    int entry;
};

Span span_of(const void* p, int64_t numel, int32_t dtype, int i)
{
    const uintptr_t begin = reinterpret_cast<uintptr_t>(p);
    return {begin, begin + static_cast<uintptr_t>(numel) * (dtype == Q8_F32 ? 4 : 2), i};
}

// Outputs that overlap one another or a gradient (but their own at the same
// address) would be read and written by several CTAs in no order.  Outputs in the
// order of their addresses, apart from the gradients, as those of one buffer are,
// take a look or two at each; else they are sorted (580 entries: 2 or 12 us on the host).
int check_overlaps(const q8_grad* list, int count)
{
    uintptr_t first = UINTPTR_MAX, last = 0;
    bool apart = true;
    for (int i = 0; i < count; ++i) {
        if (list[i].numel == 0) continue;
        const Span o = span_of(list[i].out, list[i].numel, list[i].out_dtype, i);
        apart = apart && o.begin >= last;
        first = std::min(first, o.begin);
        last = std::max(last, o.end);
    }
    const auto among = [&](const q8_grad& g, const Span& s) { return g.numel && g.out != g.grad && s.end > first && s.begin < last; };
    for (int i = 0; apart && i < count; ++i) apart = !among(list[i], span_of(list[i].grad, list[i].numel, list[i].grad_dtype, i));
    if (apart) return Q8_OK;
    try {
        std::vector<Span> outs;
        outs.reserve(static_cast<size_t>(count));
        for (int i = 0; i < count; ++i)
            if (list[i].numel) outs.push_back(span_of(list[i].out, list[i].numel, list[i].out_dtype, i));
        std::sort(outs.begin(), outs.end(), [](const Span& a, const Span& b) { return a.begin != b.begin ? a.begin < b.begin : a.entry < b.entry; });
        for (size_t k = 1; k < outs.size(); ++k)
            if (outs[k].begin < outs[k - 1].end) return fail(Q8_ERR_ARG, entry("out overlaps another's out", outs[k].entry));
        for (int i = 0; i < count; ++i) {
            const Span s = span_of(list[i].grad, list[i].numel, list[i].grad_dtype, i);
            if (!among(list[i], s)) continue;
            // the last output that begins before the gradient ends
            const auto o = std::partition_point(outs.begin(), outs.end(), [&](const Span& x) { return x.begin < s.end; });
            if (o != outs.begin() && (o - 1)->end > s.begin) return fail(Q8_ERR_ARG, entry("grad overlaps an out", i));
        }
    } catch (const std::bad_alloc&) {
        return fail(Q8_ERR_SIZE, "no host memory for a list of so many gradients");
    }
    return Q8_OK;
}

int check_norm_output(const float* norm)
{
    if (!norm) return fail(Q8_ERR_NULL, "norm is NULL");
    if (!aligned(norm, 4)) return fail(Q8_ERR_ALIGN, "norm must be 4-byte aligned");
    return Q8_OK;
}

std::mutex g_lock;
std::map<int, q8::DeviceInfo> g_devices;

}  // namespace

namespace q8 {

cudaError_t device_info(DeviceInfo* out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_lock);
    DeviceInfo& d = g_devices[dev];
    if (!d.sms && (e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if (!d.fault) {
        void* p = nullptr;
        if ((e = cudaHostAlloc(&p, sizeof(int32_t), cudaHostAllocMapped)) != cudaSuccess) return e;
        d.fault = static_cast<int32_t*>(p);
        *d.fault = 0;
    }
    *out = d;
    return cudaSuccess;
}

cudaError_t earlier_fault(int32_t* fault)
{
    volatile int32_t* f = fault;
    if (*f == 0) return cudaSuccess;
    *f = 0;
    return cudaErrorLaunchTimeout;
}

}  // namespace q8

extern "C" {

int64_t q8_gated_ff_workspace(const q8_gated_ff* ff, int backward)
{
    if (backward != 0 && backward != 1) return fail(Q8_ERR_ARG, "backward must be 0 or 1");
    const int rc = check_ff(ff);
    return rc != Q8_OK ? rc : q8::ff_workspace(*ff, backward != 0);
}

int q8_gated_ff_forward(const q8_gated_ff* ff, uint16_t* h, int64_t h_stride, float* saved, q8_stream_t stream)
{
    int rc = check_ff(ff);
    if (rc != Q8_OK) return rc;
    if ((rc = check_rows(h, 2, ff->tokens, ff->d_ff, h_stride, "h")) != Q8_OK) return rc;
    if (!aligned(saved, 4)) return fail(Q8_ERR_ALIGN, "saved must be 4-byte aligned");
    if ((rc = check_workspace(ff->workspace, ff->workspace_bytes, q8::ff_workspace(*ff, false))) != Q8_OK) return rc;
    if (ff->tokens == 0) return Q8_OK;
    const cudaError_t err = q8::launch_ff_forward(*ff, h, h_stride, saved, stream);
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_gated_ff_forward launch");
}

int q8_gated_ff_backward(const q8_gated_ff* ff, const uint16_t* dh, int64_t dh_stride, const float* saved,
                         uint16_t* dx, int64_t dx_stride, uint16_t* dw_gate, uint16_t* dw_up, q8_stream_t stream)
{
    int rc = check_ff(ff);
    if (rc != Q8_OK) return rc;
    if ((rc = check_rows(dh, 2, ff->tokens, ff->d_ff, dh_stride, "dh")) != Q8_OK) return rc;
    if (dx && (rc = check_rows(dx, 2, ff->tokens, ff->d_model, dx_stride, "dx")) != Q8_OK) return rc;
    if ((rc = check_vec(dw_gate, "dw_gate")) != Q8_OK || (rc = check_vec(dw_up, "dw_up")) != Q8_OK) return rc;
    if (!aligned(saved, 4)) return fail(Q8_ERR_ALIGN, "saved must be 4-byte aligned");
    if ((rc = check_workspace(ff->workspace, ff->workspace_bytes, q8::ff_workspace(*ff, true))) != Q8_OK) return rc;
    const q8::FfBackward b{dh, dh_stride, saved, dx, dx_stride, dw_gate, dw_up};
    cudaError_t err = cudaSuccess;
    if (ff->tokens == 0) {                       // sums over no tokens
        const size_t bytes = static_cast<size_t>(ff->d_ff) * ff->d_model * 2;
        if (dw_gate) err = cudaMemsetAsync(dw_gate, 0, bytes, stream);
        if (err == cudaSuccess && dw_up) err = cudaMemsetAsync(dw_up, 0, bytes, stream);
    } else if (dx || dw_gate || dw_up) {
        err = q8::launch_ff_backward(*ff, b, stream);
    }
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_gated_ff_backward launch");
}

int q8_block_norm_forward(const q8_block_norm* bn, void* residual_out, int64_t residual_out_stride, uint16_t* z,
                          int64_t z_stride, q8_stream_t stream)
{
    int rc = check_norm(bn);
    if (rc != Q8_OK) return rc;
    if (residual_out && (rc = check_rows(residual_out, bn->residual_dtype == Q8_F32 ? 4 : 2, bn->tokens, bn->dim,
                                         residual_out_stride, "residual_out")) != Q8_OK)
        return rc;
    if (z && (rc = check_rows(z, 2, bn->tokens, bn->dim, z_stride, "z")) != Q8_OK) return rc;
    if (bn->tokens == 0 || (!residual_out && !z)) return Q8_OK;
    const cudaError_t err = q8::launch_norm_forward(*bn, residual_out, residual_out_stride, z, z_stride, stream);
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_block_norm_forward launch");
}

int64_t q8_block_norm_workspace(const q8_block_norm* bn, const q8_block_norm_grads* g)
{
    int rc = check_norm(bn);
    if (rc == Q8_OK) rc = check_norm_grads(bn, g);
    return rc != Q8_OK ? rc : q8::norm_workspace(*bn, *g);
}

int q8_block_norm_backward(const q8_block_norm* bn, const q8_block_norm_grads* g, q8_stream_t stream)
{
    int rc = check_norm(bn);
    if (rc == Q8_OK) rc = check_norm_grads(bn, g);
    if (rc != Q8_OK) return rc;
    if ((rc = check_workspace(g->workspace, g->workspace_bytes, q8::norm_workspace(*bn, *g))) != Q8_OK) return rc;
    cudaError_t err = cudaSuccess;
    if (bn->tokens == 0) {                       // sums over no tokens (a gate then has no rows)
        for (uint16_t* p : {g->d_post_weight, g->d_post_bias, g->d_pre_weight, g->d_pre_bias})
            if (p && err == cudaSuccess) err = cudaMemsetAsync(p, 0, static_cast<size_t>(bn->dim) * 2, stream);
    } else {
        err = q8::launch_norm_backward(*bn, *g, stream);
    }
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_block_norm_backward launch");
}

int q8_distill_topk_forward(const q8_distill_topk* d, float* loss, float* stats, void* dlogits,
                            int64_t dlogits_stride, q8_stream_t stream)
{
    int rc = check_distill(d);
    if (rc != Q8_OK || d->rows == 0) return rc;
    if (!loss) return fail(Q8_ERR_NULL, "loss is NULL");
    if (!aligned(loss, 4) || !aligned(stats, 4)) return fail(Q8_ERR_ALIGN, "loss and stats must be 4-byte aligned");
    if (dlogits && (rc = check_rows(dlogits, d->logits_dtype == Q8_F32 ? 4 : 2, d->rows, d->vocab, dlogits_stride,
                                    "dlogits")) != Q8_OK)
        return rc;
    const cudaError_t err = q8::launch_distill(*d, loss, stats, nullptr, dlogits, dlogits_stride, stream);
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_distill_topk_forward launch");
}

int q8_distill_topk_backward(const q8_distill_topk* d, const float* stats, void* dlogits, int64_t dlogits_stride,
                             q8_stream_t stream)
{
    int rc = check_distill(d);
    if (rc != Q8_OK || d->rows == 0) return rc;
    if (!stats) return fail(Q8_ERR_NULL, "stats is NULL");
    if (!aligned(stats, 4)) return fail(Q8_ERR_ALIGN, "stats must be 4-byte aligned");
    if ((rc = check_rows(dlogits, d->logits_dtype == Q8_F32 ? 4 : 2, d->rows, d->vocab, dlogits_stride, "dlogits")) != Q8_OK)
        return rc;
    const cudaError_t err = q8::launch_distill(*d, nullptr, nullptr, stats, dlogits, dlogits_stride, stream);
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_distill_topk_backward launch");
}

int q8_embedding_forward(const q8_embedding* e, const uint16_t* table, void* out, int64_t out_stride,
                         q8_stream_t stream)
{
    int rc = check_embedding(e);
    if (rc == Q8_OK) rc = check_rows(table, 2, e->vocab, e->dim, e->dim, "table");
    if (rc == Q8_OK) rc = check_rows(out, e->dtype == Q8_F32 ? 4 : 2, e->tokens, e->dim, out_stride, "out");
    if (rc != Q8_OK || e->tokens == 0) return rc;
    const cudaError_t err = q8::launch_embed_forward(*e, table, out, out_stride, stream);
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_embedding_forward launch");
}

int64_t q8_embedding_workspace(const q8_embedding* e)
{
    const int rc = check_embedding(e);
    return rc != Q8_OK ? rc : q8::embed_workspace(*e);
}

int q8_embedding_backward(const q8_embedding* e, const void* dout, int64_t dout_stride, uint16_t* dtable,
                          int accumulate, void* workspace, int64_t workspace_bytes, q8_stream_t stream)
{
    int rc = check_embedding(e);
    if (rc != Q8_OK) return rc;
    if (accumulate != 0 && accumulate != 1) return fail(Q8_ERR_ARG, "accumulate must be 0 or 1");
    if ((rc = check_rows(dout, e->dtype == Q8_F32 ? 4 : 2, e->tokens, e->dim, dout_stride, "dout")) != Q8_OK) return rc;
    if ((rc = check_rows(dtable, 2, e->vocab, e->dim, e->dim, "dtable")) != Q8_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, q8::embed_workspace(*e))) != Q8_OK) return rc;
    cudaError_t err = cudaSuccess;
    if (e->tokens == 0) {                        // sums over no tokens
        if (!accumulate) err = cudaMemsetAsync(dtable, 0, static_cast<size_t>(e->vocab) * e->dim * 2, stream);
    } else {
        err = q8::launch_embed_backward(*e, dout, dout_stride, dtable, accumulate != 0, workspace, stream);
    }
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_embedding_backward launch");
}

int64_t q8_grad_norm_workspace(int count)
{
    if (count < 0) return fail(Q8_ERR_SIZE, "count must be >= 0");
    return q8::grads_workspace(count);
}

int q8_grad_norm(const q8_grad* list, int count, float* norm, void* workspace, int64_t workspace_bytes,
                 q8_stream_t stream)
{
    int rc = check_grads(list, count, false);
    if (rc == Q8_OK) rc = check_norm_output(norm);
    if (rc == Q8_OK) rc = check_workspace(workspace, workspace_bytes, q8::grads_workspace(count));
    if (rc != Q8_OK) return rc;
    const cudaError_t err = q8::launch_grads(list, count, false, 0.0, norm, workspace, stream);
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_grad_norm launch");
}

int q8_clip_grads(const q8_grad* list, int count, double max_norm, float* norm, void* workspace,
                  int64_t workspace_bytes, q8_stream_t stream)
{
    int rc = check_grads(list, count, true);
    if (rc == Q8_OK) rc = check_overlaps(list, count);
    if (rc == Q8_OK && !(max_norm >= 0.0)) rc = fail(Q8_ERR_ARG, "max_norm must be >= 0");
    if (rc == Q8_OK) rc = check_norm_output(norm);
    if (rc == Q8_OK) rc = check_workspace(workspace, workspace_bytes, q8::grads_workspace(count));
    if (rc != Q8_OK) return rc;
    const cudaError_t err = q8::launch_grads(list, count, true, max_norm, norm, workspace, stream);
    return err == cudaSuccess ? Q8_OK : cuda_fail(err, "q8_clip_grads launch");
}

}  // extern "C"
