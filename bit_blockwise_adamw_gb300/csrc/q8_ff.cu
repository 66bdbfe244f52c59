// q8_ff.cu -- the gated feed-forward product (include/q8train.h), forward and
// backward, as plain tiled fp32 products.
#include "q8_internal.h"
#include "q8_train.h"

namespace q8 {

namespace {

constexpr int kTile = 64, kStep = 16;

// act(g) and act'(g).
__device__ __forceinline__ float2 activation(float g, int act)
{
    if (act == Q8_SILU) {
        const float s = 1.0f / (1.0f + __expf(-g));
        return make_float2(g * s, s * fmaf(g, 1.0f - s, 1.0f));
    }
    if (act == Q8_GELU_TANH) {
        // 1/2 (1 + tanh(t)) = sigmoid(2 t)
        constexpr float c = 1.5957691216057308f;              // 2 sqrt(2/pi)
        const float g2 = g * g;
        const float s = 1.0f / (1.0f + __expf(-c * g * fmaf(0.044715f, g2, 1.0f)));
        return make_float2(g * s, s + g * s * (1.0f - s) * c * fmaf(3.0f * 0.044715f, g2, 1.0f));
    }
    const float cdf = 0.5f * erfcf(-0.70710678118654752f * g);
    return make_float2(g * cdf, fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), cdf));
}

// C[m, n] = sum over the segments s of sum_k A_s(m, k) B_s(n, k), with the
// operands' strides given: one 64 x 64 tile to a CTA, 4 x 4 to a thread.
struct Operand {
    const uint16_t* p[2];
    int64_t row, col;             // stride of m (or n), and of k
};

__device__ __forceinline__ void tile_product(const uint16_t* a, int64_t am, int64_t ak, const uint16_t* b, int64_t bn,
                                             int64_t bk, int64_t m0, int64_t n0, int64_t M, int64_t N, int64_t K,
                                             float acc[4][4])
{
    __shared__ float sa[kStep][kTile + 4], sb[kStep][kTile + 4];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t k0 = 0; k0 < K; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
            const int r = i / kStep, k = i % kStep;
            sa[k][r] = m0 + r < M && k0 + k < K ? bf16_to_float(a[(m0 + r) * am + (k0 + k) * ak]) : 0.0f;
            sb[k][r] = n0 + r < N && k0 + k < K ? bf16_to_float(b[(n0 + r) * bn + (k0 + k) * bk]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
}

// h (and g, u for the backward call), or with dh given dg and du.
__global__ void __launch_bounds__(256) ff_dual_kernel(const q8_gated_ff f, uint16_t* h, int64_t h_stride, float* saved,
                                                      const uint16_t* dh, int64_t dh_stride, uint16_t* dg, uint16_t* du)
{
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile; m0 < f.tokens; m0 += static_cast<int64_t>(gridDim.y) * kTile) {
        float g[4][4] = {}, u[4][4] = {};
        tile_product(f.x, f.x_stride, 1, f.w_gate, f.d_model, 1, m0, n0, f.tokens, f.d_ff, f.d_model, g);
        tile_product(f.x, f.x_stride, 1, f.w_up, f.d_model, 1, m0, n0, f.tokens, f.d_ff, f.d_model, u);
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
                if (m >= f.tokens || n >= f.d_ff) continue;
                const float2 a = activation(g[i][j], f.act);
                if (dh) {
                    const float d = bf16_to_float(dh[m * dh_stride + n]);
                    dg[m * f.d_ff + n] = float_to_bf16(d * u[i][j] * a.y);
                    du[m * f.d_ff + n] = float_to_bf16(d * a.x);
                } else {
                    h[m * h_stride + n] = float_to_bf16(a.x * u[i][j]);
                    if (saved) {
                        saved[m * f.d_ff + n] = g[i][j];
                        saved[(f.tokens + m) * f.d_ff + n] = u[i][j];
                    }
                }
            }
    }
}

// dg and du from the saved g and u.
__global__ void __launch_bounds__(256) ff_gates_kernel(const float* saved, const uint16_t* dh, int64_t dh_stride,
                                                       int64_t tokens, int64_t d_ff, int act, uint16_t* dg, uint16_t* du)
{
    const int64_t n = tokens * d_ff;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const float2 a = activation(saved[i], act);
        const float d = bf16_to_float(dh[i / d_ff * dh_stride + i % d_ff]);
        dg[i] = float_to_bf16(d * saved[n + i] * a.y);
        du[i] = float_to_bf16(d * a.x);
    }
}

__global__ void __launch_bounds__(256) ff_product_kernel(const Operand a, const Operand b, int segments, int64_t M,
                                                         int64_t N, int64_t K, uint16_t* c, int64_t c_stride)
{
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile; m0 < M; m0 += static_cast<int64_t>(gridDim.y) * kTile) {
        float acc[4][4] = {};
        for (int s = 0; s < segments; ++s)
            tile_product(a.p[s], a.row, a.col, b.p[s], b.row, b.col, m0, n0, M, N, K, acc);
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j)
                if (m0 + ty * 4 + i < M && n0 + tx * 4 + j < N)
                    c[(m0 + ty * 4 + i) * c_stride + n0 + tx * 4 + j] = float_to_bf16(acc[i][j]);
    }
}

dim3 tiles(int64_t M, int64_t N)
{
    const int64_t y = (M + kTile - 1) / kTile;
    return dim3(static_cast<unsigned>((N + kTile - 1) / kTile), static_cast<unsigned>(y < 65535 ? y : 65535));
}

}  // namespace

cudaError_t prepare_ff() { return cudaSuccess; }

int64_t ff_workspace(const q8_gated_ff& f, bool backward) { return backward ? 2 * f.tokens * f.d_ff * 2 : 0; }

cudaError_t launch_ff_forward(const q8_gated_ff& f, uint16_t* h, int64_t h_stride, float* saved, cudaStream_t st)
{
    ff_dual_kernel<<<tiles(f.tokens, f.d_ff), 256, 0, st>>>(f, h, h_stride, saved, nullptr, 0, nullptr, nullptr);
    return cudaGetLastError();
}

cudaError_t launch_ff_backward(const q8_gated_ff& f, const FfBackward& b, cudaStream_t st)
{
    uint16_t* dg = static_cast<uint16_t*>(f.workspace);
    uint16_t* du = dg + f.tokens * f.d_ff;
    if (b.saved)
        ff_gates_kernel<<<152 * 8, 256, 0, st>>>(b.saved, b.dh, b.dh_stride, f.tokens, f.d_ff, f.act, dg, du);
    else
        ff_dual_kernel<<<tiles(f.tokens, f.d_ff), 256, 0, st>>>(f, nullptr, 0, nullptr, b.dh, b.dh_stride, dg, du);
    if (b.dx)
        ff_product_kernel<<<tiles(f.tokens, f.d_model), 256, 0, st>>>(
            Operand{{dg, du}, f.d_ff, 1}, Operand{{f.w_gate, f.w_up}, 1, f.d_model}, 2, f.tokens, f.d_model, f.d_ff,
            b.dx, b.dx_stride);
    const uint16_t* d[2] = {dg, du};
    uint16_t* dw[2] = {b.dw_gate, b.dw_up};
    for (int i = 0; i < 2; ++i)
        if (dw[i])
            ff_product_kernel<<<tiles(f.d_ff, f.d_model), 256, 0, st>>>(
                Operand{{d[i], nullptr}, 1, f.d_ff}, Operand{{f.x, nullptr}, 1, f.x_stride}, 1, f.d_ff, f.d_model,
                f.tokens, dw[i], f.d_model);
    return cudaGetLastError();
}

}  // namespace q8
