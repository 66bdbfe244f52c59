// q8_embed.cu -- the token embedding: out[t] = scale * W[ids[t]], and the
// gradient of its table, dW[v] = scale * sum of dout[t] over the t with
// ids[t] = v (include/q8train.h).
//
// Neither does arithmetic worth counting: both are bound by the bytes of the
// rows that they move.
#include <algorithm>

#include "q8_internal.h"
#include "q8_train.h"

namespace q8 {

namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ float load(const uint16_t* p) { return bf16_to_float(*p); }
__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ void store(uint16_t* p, float x) { *p = float_to_bf16(x); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }

// A warp for each row.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) lookup_kernel(q8_embedding e, const uint16_t* table, T* out, int64_t out_stride)
{
    const int lane = threadIdx.x % 32;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
    for (int64_t t = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) / 32; t < e.tokens; t += warps) {
        const int64_t id = e.ids[t];
        const bool known = id >= 0 && id < e.vocab;
        const uint16_t* row = table + (known ? id : 0) * e.dim;
        for (int64_t c = lane; c < e.dim; c += 32) store(out + t * out_stride + c, known ? __fmul_rn(e.scale, load(row + c)) : 0.0f);
    }
}

// A warp for each token and 128 columns: the first token of its id adds up the
// rows of all later ones, in their order.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) scatter_kernel(q8_embedding e, const T* dout, int64_t stride, uint16_t* dtable, bool accumulate)
{
    const int lane = threadIdx.x % 32;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
    for (int64_t t = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) / 32; t < e.tokens; t += warps) {
        const int64_t id = e.ids[t];
        if (id < 0 || id >= e.vocab) continue;
        bool first = true;
        for (int64_t i = 0; first && i < t; i += 32) first = !__any_sync(~0u, i + lane < t && e.ids[i + lane] == id);
        if (!first) continue;
        for (int64_t c0 = static_cast<int64_t>(blockIdx.y) * 128; c0 < e.dim; c0 += static_cast<int64_t>(gridDim.y) * 128) {
            float sum[4] = {};
            for (int64_t i = t / 32 * 32; i < e.tokens; i += 32) {
                uint32_t same = __ballot_sync(~0u, i + lane < e.tokens && e.ids[i + lane] == id);
                for (; same; same &= same - 1) {
                    const T* row = dout + (i + __ffs(same) - 1) * stride;
                    for (int j = 0; j < 4; ++j)
                        if (c0 + j * 32 + lane < e.dim) sum[j] = __fadd_rn(sum[j], load(row + c0 + j * 32 + lane));
                }
            }
            for (int j = 0; j < 4; ++j) {
                const int64_t c = c0 + j * 32 + lane;
                if (c < e.dim) store(dtable + id * e.dim + c, accumulate ? __fmaf_rn(e.scale, sum[j], load(dtable + id * e.dim + c)) : __fmul_rn(e.scale, sum[j]));
            }
        }
    }
}

template <typename T>
cudaError_t lookup(const q8_embedding& e, const uint16_t* table, void* out, int64_t out_stride, cudaStream_t st)
{
    int grid = 0;
    const cudaError_t err = persistent_grid(reinterpret_cast<const void*>(lookup_kernel<T>), kRowThreads, 0, &grid);
    if (err != cudaSuccess) return err;
    grid = static_cast<int>(std::min<int64_t>(grid, (e.tokens + 7) / 8));
    lookup_kernel<T><<<grid, kRowThreads, 0, st>>>(e, table, static_cast<T*>(out), out_stride);
    return cudaGetLastError();
}

template <typename T>
cudaError_t scatter(const q8_embedding& e, const void* dout, int64_t stride, uint16_t* dtable, bool accumulate, cudaStream_t st)
{
    int grid = 0;
    const cudaError_t err = persistent_grid(reinterpret_cast<const void*>(scatter_kernel<T>), kRowThreads, 0, &grid);
    if (err != cudaSuccess) return err;
    grid = static_cast<int>(std::min<int64_t>(grid, (e.tokens + 7) / 8));
    const int tiles = static_cast<int>(std::min<int64_t>((e.dim + 127) / 128, 64));
    scatter_kernel<T><<<dim3(grid, tiles), kRowThreads, 0, st>>>(e, static_cast<const T*>(dout), stride, dtable, accumulate);
    return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_embed()
{
    int g = 0;
    for (const void* k : {reinterpret_cast<const void*>(lookup_kernel<uint16_t>), reinterpret_cast<const void*>(lookup_kernel<float>),
                          reinterpret_cast<const void*>(scatter_kernel<uint16_t>), reinterpret_cast<const void*>(scatter_kernel<float>)}) {
        const cudaError_t e = persistent_grid(k, kRowThreads, 0, &g);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_embed_forward(const q8_embedding& e, const uint16_t* table, void* out, int64_t out_stride, cudaStream_t st)
{
    return e.dtype == Q8_F32 ? lookup<float>(e, table, out, out_stride, st) : lookup<uint16_t>(e, table, out, out_stride, st);
}

int64_t embed_workspace(const q8_embedding&) { return 0; }

cudaError_t launch_embed_backward(const q8_embedding& e, const void* dout, int64_t dout_stride, uint16_t* dtable,
                                  bool accumulate, void*, cudaStream_t st)
{
    if (!accumulate) {
        const cudaError_t err = cudaMemsetAsync(dtable, 0, static_cast<size_t>(e.vocab) * e.dim * 2, st);
        if (err != cudaSuccess) return err;
    }
    return e.dtype == Q8_F32 ? scatter<float>(e, dout, dout_stride, dtable, accumulate, st)
                             : scatter<uint16_t>(e, dout, dout_stride, dtable, accumulate, st);
}

}  // namespace q8
