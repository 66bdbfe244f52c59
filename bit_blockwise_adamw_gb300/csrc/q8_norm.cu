// q8_norm.cu -- the norms around a block's gate and residual
// (include/q8train.h), forward and backward: one CTA to a row.
#include <algorithm>

#include "q8_internal.h"
#include "q8_train.h"

namespace q8 {

namespace {

constexpr int kRowThreads = 256;

// The sum of v over the CTA, in every thread.
__device__ float cta_sum(float v)
{
    __shared__ float part[kRowThreads / 32];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < kRowThreads / 32; ++i) s += part[i];
    return s;
}

__device__ __forceinline__ float load_res(const void* p, int64_t i, int dtype)
{
    return dtype == Q8_F32 ? static_cast<const float*>(p)[i] : bf16_to_float(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ void store_res(void* p, int64_t i, int dtype, float v)
{
    if (dtype == Q8_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = float_to_bf16(v);
}

__device__ __forceinline__ float vec(const uint16_t* p, int64_t i, float none) { return p ? bf16_to_float(p[i]) : none; }

// Mean (0 unless layer) and reciprocal root of the row s(0 .. dim - 1).
template <typename Row>
__device__ float2 row_stats(Row s, int dim, int kind, float eps)
{
    if (kind == Q8_NORM_NONE) return make_float2(0.0f, 1.0f);
    float mu = 0.0f;
    if (kind == Q8_NORM_LAYER) {
        float a = 0.0f;
        for (int j = threadIdx.x; j < dim; j += kRowThreads) a += s(j);
        mu = cta_sum(a) / dim;
    }
    float q = 0.0f;
    for (int j = threadIdx.x; j < dim; j += kRowThreads) q = fmaf(s(j) - mu, s(j) - mu, q);
    return make_float2(mu, 1.0f / sqrtf(cta_sum(q) / dim + eps));
}

// r' into sr, and both rows' statistics.
__device__ void row_forward(const q8_block_norm& n, int64_t t, float* sr, float2* post, float2* pre)
{
    const int dim = static_cast<int>(n.dim);
    const uint16_t* y = n.y + t * n.y_stride;
    *post = row_stats([&](int j) { return bf16_to_float(y[j]); }, dim, n.post_kind, n.eps);
    const uint16_t* gate = n.gate ? n.gate + t / n.gate_tokens * n.dim : nullptr;
    for (int j = threadIdx.x; j < dim; j += kRowThreads) {
        const float v = fmaf((bf16_to_float(y[j]) - post->x) * post->y, vec(n.post_weight, j, 1.0f), vec(n.post_bias, j, 0.0f));
        sr[j] = fmaf(n.residual_scale, load_res(n.residual, t * n.residual_stride + j, n.residual_dtype),
                     vec(gate, j, 1.0f) * v);
    }
    *pre = row_stats([&](int j) { return sr[j]; }, dim, n.pre_kind, n.eps);
}

__global__ void __launch_bounds__(kRowThreads) norm_forward_kernel(const q8_block_norm n, void* r_out, int64_t r_stride,
                                                                   uint16_t* z, int64_t z_stride)
{
    extern __shared__ float sr[];
    for (int64_t t = blockIdx.x; t < n.tokens; t += gridDim.x) {
        float2 post, pre;
        row_forward(n, t, sr, &post, &pre);
        for (int j = threadIdx.x; j < n.dim; j += kRowThreads) {
            if (r_out) store_res(r_out, t * r_stride + j, n.residual_dtype, sr[j]);
            if (z) z[t * z_stride + j] = float_to_bf16(fmaf((sr[j] - pre.x) * pre.y, vec(n.pre_weight, j, 1.0f),
                                                            vec(n.pre_bias, j, 0.0f)));
        }
    }
}

// The gradient of a normalised row's input: rs (dn - c1 - v c2).
__device__ float2 norm_terms(float sum, float dot, int dim, int kind)
{
    return make_float2(kind == Q8_NORM_LAYER ? sum / dim : 0.0f, kind == Q8_NORM_NONE ? 0.0f : dot / dim);
}

// Rows of one CTA: a contiguous run of tokens.  Each column's sums over them go
// to partial[c][blockIdx.x][dim], c = post_w, post_b, pre_w, pre_b, gate; a
// gate's run never crosses into another group (runs are cut by group).
__global__ void __launch_bounds__(kRowThreads) norm_backward_kernel(const q8_block_norm n, const q8_block_norm_grads g,
                                                                    int64_t group, int64_t run, int64_t runs_per_group,
                                                                    float* partial)
{
    extern __shared__ float sr[];
    const int dim = static_cast<int>(n.dim);
    const int64_t next = static_cast<int64_t>(gridDim.x) * dim;
    float* sums = partial + static_cast<int64_t>(blockIdx.x) * dim;
    for (int c = 0; c < 5; ++c)
        for (int j = threadIdx.x; j < dim; j += kRowThreads) sums[c * next + j] = 0.0f;
    const int64_t first = blockIdx.x / runs_per_group * group + blockIdx.x % runs_per_group * run;
    const int64_t stop = min(min(first + run, (blockIdx.x / runs_per_group + 1) * group), n.tokens);
    for (int64_t t = first; t < stop; ++t) {
        float2 post, pre;
        row_forward(n, t, sr, &post, &pre);
        const uint16_t* gate = n.gate ? n.gate + t / n.gate_tokens * n.dim : nullptr;
        const uint16_t* y = n.y + t * n.y_stride;
        auto d_pre = [&](int j) { return g.dz ? bf16_to_float(g.dz[t * g.dz_stride + j]) : 0.0f; };
        float a = 0.0f, b = 0.0f;
        for (int j = threadIdx.x; j < dim; j += kRowThreads) {
            const float dn = d_pre(j) * vec(n.pre_weight, j, 1.0f);
            a += dn;
            b = fmaf(dn, (sr[j] - pre.x) * pre.y, b);
        }
        const float sa = cta_sum(a), sb = cta_sum(b);
        const float2 c = norm_terms(sa, sb, dim, n.pre_kind);
        a = b = 0.0f;
        for (int j = threadIdx.x; j < dim; j += kRowThreads) {
            const float dz = d_pre(j), rn = (sr[j] - pre.x) * pre.y, yn = (bf16_to_float(y[j]) - post.x) * post.y;
            float d = pre.y * (dz * vec(n.pre_weight, j, 1.0f) - c.x - rn * c.y);
            if (g.d_residual_out) d += load_res(g.d_residual_out, t * g.d_residual_out_stride + j, n.residual_dtype);
            if (g.d_residual) store_res(g.d_residual, t * g.d_residual_stride + j, n.residual_dtype, n.residual_scale * d);
            const float dp = d * vec(gate, j, 1.0f), w = vec(n.post_weight, j, 1.0f);
            sums[j] += dp * yn;
            sums[next + j] += dp;
            sums[2 * next + j] += dz * rn;
            sums[3 * next + j] += dz;
            sums[4 * next + j] += d * fmaf(yn, w, vec(n.post_bias, j, 0.0f));
            sr[j] = dp * w;                        // the gradient of the normalised y
            a += dp * w;
            b = fmaf(dp * w, yn, b);
        }
        const float ta = cta_sum(a), tb = cta_sum(b);
        const float2 e = norm_terms(ta, tb, dim, n.post_kind);
        if (g.d_y)
            for (int j = threadIdx.x; j < dim; j += kRowThreads)
                g.d_y[t * g.d_y_stride + j] = float_to_bf16(post.y * (sr[j] - e.x - (bf16_to_float(y[j]) - post.x) * post.y * e.y));
        __syncthreads();
    }
}

// out[r, j] = the sum of `count` consecutive rows of partial, for row r.
__global__ void norm_sum_kernel(const float* partial, int64_t rows, int64_t count, int64_t dim, uint16_t* out)
{
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < rows * dim;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        float s = 0.0f;
        for (int64_t c = 0; c < count; ++c) s += partial[(i / dim * count + c) * dim + i % dim];
        out[i] = float_to_bf16(s);
    }
}

struct Runs {
    int64_t group, run, per_group, ctas;
};

Runs plan(const q8_block_norm& n)
{
    Runs r;
    r.group = n.gate && n.gate_tokens < n.tokens ? n.gate_tokens : n.tokens;
    const int64_t groups = (n.tokens + r.group - 1) / r.group;
    r.per_group = groups >= 304 ? 1 : std::min<int64_t>(r.group, (304 + groups - 1) / groups);
    r.run = (r.group + r.per_group - 1) / r.per_group;
    r.ctas = groups * r.per_group;
    return r;
}

}  // namespace

cudaError_t prepare_norm()
{
    int g = 0;
    return cudaSuccess == persistent_grid(reinterpret_cast<const void*>(norm_forward_kernel), kRowThreads, 0, &g)
               ? cudaSuccess : cudaGetLastError();
}

cudaError_t launch_norm_forward(const q8_block_norm& n, void* residual_out, int64_t residual_out_stride, uint16_t* z,
                                int64_t z_stride, cudaStream_t st)
{
    const int smem = static_cast<int>(n.dim * 4);
    cudaError_t e = cudaFuncSetAttribute(norm_forward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    norm_forward_kernel<<<static_cast<unsigned>(std::min<int64_t>(n.tokens, 152 * 8)), kRowThreads, smem, st>>>(
        n, residual_out, residual_out_stride, z, z_stride);
    return cudaGetLastError();
}

int64_t norm_workspace(const q8_block_norm& n, const q8_block_norm_grads&)
{
    return n.tokens == 0 ? 0 : plan(n).ctas * n.dim * 5 * 4;
}

cudaError_t launch_norm_backward(const q8_block_norm& n, const q8_block_norm_grads& g, cudaStream_t st)
{
    const Runs r = plan(n);
    float* partial = static_cast<float*>(g.workspace);
    const int smem = static_cast<int>(n.dim * 4);
    cudaError_t e = cudaFuncSetAttribute(norm_backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    norm_backward_kernel<<<static_cast<unsigned>(r.ctas), kRowThreads, smem, st>>>(n, g, r.group, r.run, r.per_group, partial);
    uint16_t* outs[5] = {g.d_post_weight, g.d_post_bias, g.d_pre_weight, g.d_pre_bias, g.d_gate};
    for (int c = 0; c < 5; ++c) {
        if (!outs[c]) continue;
        const int64_t rows = c == 4 ? r.ctas / r.per_group : 1;
        norm_sum_kernel<<<static_cast<unsigned>(std::min<int64_t>((rows * n.dim + 127) / 128, 152 * 16)), 128, 0, st>>>(
            partial + c * r.ctas * n.dim, rows, c == 4 ? r.per_group : r.ctas, n.dim, outs[c]);
    }
    return cudaGetLastError();
}

}  // namespace q8
