// q8_distill.cu -- distillation from a teacher's top logits
// (include/q8train.h), forward and backward: one CTA to a row.
#include <algorithm>

#include "q8_internal.h"
#include "q8_train.h"

namespace q8 {

namespace {

constexpr int kRowThreads = 512;

template <bool MAX>
__device__ float cta_reduce(float v)
{
    __shared__ float part[kRowThreads / 32];
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
    for (int i = 1; i < kRowThreads / 32; ++i) v = MAX ? fmaxf(v, part[i]) : v + part[i];
    return v;
}

template <typename T>
__device__ __forceinline__ float load(const T* p, int64_t i);
template <>
__device__ __forceinline__ float load<float>(const float* p, int64_t i) { return p[i]; }
template <>
__device__ __forceinline__ float load<uint16_t>(const uint16_t* p, int64_t i) { return bf16_to_float(p[i]); }
__device__ __forceinline__ void store(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store(uint16_t* p, int64_t i, float v) { p[i] = float_to_bf16(v); }

template <typename T>
__global__ void __launch_bounds__(kRowThreads) distill_kernel(const q8_distill_topk d, float* loss, float* stats_out,
                                                              const float* stats_in, T* grad, int64_t grad_stride)
{
    __shared__ float s_p[Q8_DISTILL_MAX_K], s_z[Q8_DISTILL_MAX_K];
    __shared__ int s_id[Q8_DISTILL_MAX_K];
    const int K = static_cast<int>(d.k);
    const float it = 1.0f / d.temperature;
    for (int64_t t = blockIdx.x; t < d.rows; t += gridDim.x) {
        const T* z = static_cast<const T*>(d.logits) + t * d.logits_stride;
        __syncthreads();
        float top = -INFINITY;
        for (int k = threadIdx.x; k < K; k += kRowThreads) {
            const int64_t id = d.kd_weight > 0.0f ? d.teacher_ids[t * K + k] : -1;
            const bool ok = id >= 0 && id < d.vocab;
            s_id[k] = ok ? static_cast<int>(id) : -1;
            s_p[k] = ok ? d.teacher_logits[t * K + k] * it : -INFINITY;
            s_z[k] = ok ? load(z, id) : 0.0f;
            top = fmaxf(top, s_p[k]);
        }
        top = cta_reduce<true>(top);
        const bool taught = top > -INFINITY;
        float sum = 0.0f;
        for (int k = threadIdx.x; k < K; k += kRowThreads) sum += taught ? expf(s_p[k] - top) : 0.0f;
        const float logsum = logf(cta_reduce<false>(sum));
        const int64_t label = d.labels && d.ce_weight > 0.0f ? d.labels[t] : -1;
        const bool labelled = label >= 0 && label < d.vocab;
        const float zl = labelled ? load(z, label) : 0.0f;

        float lse1 = 0.0f, lset = 0.0f;
        if (stats_in) {
            lse1 = stats_in[2 * t];
            lset = stats_in[2 * t + 1];
        } else {
            float m = -INFINITY;
            for (int64_t j = threadIdx.x; j < d.vocab; j += kRowThreads) m = fmaxf(m, load(z, j));
            m = cta_reduce<true>(m);
            float a = 0.0f, b = 0.0f;
            for (int64_t j = threadIdx.x; j < d.vocab; j += kRowThreads) {
                const float v = load(z, j) - m;
                a += expf(v);
                b += expf(v * it);
            }
            a = cta_reduce<false>(a);
            b = cta_reduce<false>(b);
            lse1 = d.ce_weight > 0.0f ? m + logf(a) : 0.0f;
            lset = d.kd_weight > 0.0f ? m * it + logf(b) : 0.0f;
        }
        // entry k: p_k and the loss's sum
        float part = 0.0f;
        for (int k = threadIdx.x; k < K; k += kRowThreads) {
            const float logp = s_p[k] - top - logsum;
            const float p = taught ? expf(logp) : 0.0f;
            s_p[k] = p;
            if (p > 0.0f) part += p * (logp - (s_z[k] * it - lset));
        }
        part = cta_reduce<false>(part);                  // and s_p is written
        if (loss && threadIdx.x == 0) {
            loss[t] = (taught ? d.kd_weight * d.temperature * d.temperature * part : 0.0f) +
                      (labelled ? d.ce_weight * (lse1 - zl) : 0.0f);
            if (stats_out) {
                stats_out[2 * t] = lse1;
                stats_out[2 * t + 1] = lset;
            }
        }
        if (!grad) continue;
        const float w = d.row_weight ? d.row_weight[t] : 1.0f;
        const float ckd = taught ? w * d.kd_weight * d.temperature : 0.0f, cce = labelled ? w * d.ce_weight : 0.0f;
        T* out = grad + t * grad_stride;
        auto base = [&](float v) {
            float r = 0.0f;
            if (taught) r = ckd * expf(v * it - lset);
            if (labelled) r = fmaf(cce, expf(v - lse1), r);
            return r;
        };
        for (int64_t j = threadIdx.x; j < d.vocab; j += kRowThreads) store(out, j, base(load(z, j)));
        __syncthreads();
        // the entries' own terms, once for each id, and the label's
        for (int k = threadIdx.x; k < K; k += kRowThreads) {
            const int id = s_id[k];
            bool first = id >= 0;
            float p = 0.0f;
            for (int i = 0; i < K; ++i)
                if (s_id[i] == id) {
                    first = first && i >= k;
                    p += s_p[i];
                }
            if (first && taught) store(out, id, base(s_z[k]) - ckd * p - (id == label ? cce : 0.0f));
        }
        if (threadIdx.x == 0 && labelled) {
            bool entry = false;
            for (int i = 0; i < K; ++i) entry = entry || (taught && s_id[i] == label);
            if (!entry) store(out, label, base(zl) - cce);
        }
    }
}

template <typename T>
cudaError_t launch(const q8_distill_topk& d, float* loss, float* stats_out, const float* stats_in, void* grad,
                   int64_t grad_stride, cudaStream_t st)
{
    int grid = 0;
    const cudaError_t e = persistent_grid(reinterpret_cast<const void*>(distill_kernel<T>), kRowThreads, 0, &grid);
    if (e != cudaSuccess) return e;
    distill_kernel<T><<<static_cast<unsigned>(std::min<int64_t>(d.rows, grid)), kRowThreads, 0, st>>>(
        d, loss, stats_out, stats_in, static_cast<T*>(grad), grad_stride);
    return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_distill()
{
    int g = 0;
    const cudaError_t e = persistent_grid(reinterpret_cast<const void*>(distill_kernel<uint16_t>), kRowThreads, 0, &g);
    return e != cudaSuccess ? e : persistent_grid(reinterpret_cast<const void*>(distill_kernel<float>), kRowThreads, 0, &g);
}

cudaError_t launch_distill(const q8_distill_topk& d, float* loss, float* stats_out, const float* stats_in,
                           void* dlogits, int64_t dlogits_stride, cudaStream_t st)
{
    return d.logits_dtype == Q8_F32 ? launch<float>(d, loss, stats_out, stats_in, dlogits, dlogits_stride, st)
                                    : launch<uint16_t>(d, loss, stats_out, stats_in, dlogits, dlogits_stride, st);
}

}  // namespace q8
