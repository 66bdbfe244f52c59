// q8_grads.cu -- the 2-norm of all gradients of a list, and their clipping
// (include/q8train.h).
//
// norm = sqrt(sum g^2), c = min(1, max_norm / (norm + 1e-6)), out = c * g: two
// operations an element, so both are bound by the gradients' bytes.
//
// A list travels as kernel parameters, kMaxGrads tensors to a launch.  It is
// cut into chunks of kChunk elements; each CTA takes a contiguous run of them
// and leaves one sum of squares in the workspace, in double; whoever needs the
// norm adds these up in one fixed order.
#include <algorithm>
#include <memory>

#include "q8_internal.h"
#include "q8_train.h"

namespace q8 {

namespace {

constexpr int kGradThreads = 256;
constexpr int kOwnElems = 64;                              // elements that a thread adds up in fp32
constexpr int kChunk = kGradThreads * kOwnElems;
constexpr int kMaxGrads = 768;
constexpr int kMaxParts = 1024;                            // CTAs of one launch, at most

struct Grad {
    const void* g;
    void* out;
    int64_t n;
};

struct GradArgs {
    double* parts;             // sums of squares: kMaxParts of each launch
    float* norm;
    double max_norm;
    int64_t nchunks;
    int32_t nt;
    int32_t parts_at;          // this launch's place in parts
    int32_t nparts;            // all launches' sums
    int64_t start[kMaxGrads + 1];
    uint8_t f32[kMaxGrads];    // bit 0: g is float32; bit 1: out is
    Grad d[kMaxGrads];
};
static_assert(sizeof(GradArgs) <= 32764, "kernel parameter space");

__device__ __forceinline__ int find(const int64_t* start, int nt, int64_t chunk)
{
    int lo = 0, hi = nt;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= chunk) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ float load(const void* p, bool f32, int64_t i)
{
    return f32 ? static_cast<const float*>(p)[i] : bf16_to_float(static_cast<const uint16_t*>(p)[i]);
}

__device__ double block_sum(double x, double* s)
{
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(~0u, x, o);
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = x;
    __syncthreads();
    double sum = 0.0;
    for (int w = 0; w < kGradThreads / 32; ++w) sum += s[w];
    __syncthreads();
    return sum;
}

// The squares of one thread's elements first, first + kGradThreads, ... of a
// chunk that ends at `last`.
__device__ double squares(const void* g, bool f32, int64_t first, int64_t last)
{
    float sum = 0.0f;
    for (int64_t i = first; i < last; i += kGradThreads) {
        const float x = load(g, f32, i);
        sum = __fmaf_rn(x, x, sum);
    }
    if (sum >= 0x1p-70f && sum <= 0x1p126f) return sum;
    // squares may have left fp32's range: the largest magnitude picks a power of
    // two that brings all of them, or all that count, back into it
    uint32_t top = 0;
    for (int64_t i = first; i < last; i += kGradThreads) top = max(top, __float_as_uint(load(g, f32, i)) & 0x7FFFFFFFu);
    const int exponent = static_cast<int>(top >> 23) - 127;
    if (top == 0 || exponent == 128) return sum;
    const int k = max(-126, min(126, -exponent));
    const float scale = __int_as_float((127 + k) << 23);
    sum = 0.0f;
    for (int64_t i = first; i < last; i += kGradThreads) {
        const float x = __fmul_rn(load(g, f32, i), scale);
        sum = __fmaf_rn(x, x, sum);
    }
    return ldexp(static_cast<double>(sum), -2 * k);
}

__global__ void __launch_bounds__(kGradThreads) squares_kernel(const __grid_constant__ GradArgs a)
{
    __shared__ double s[kGradThreads / 32];
    const int64_t begin = blockIdx.x * a.nchunks / gridDim.x;
    const int64_t end = (blockIdx.x + 1) * a.nchunks / gridDim.x;
    double sum = 0.0;
    int t = begin < end ? find(a.start, a.nt, begin) : 0;
    for (int64_t c = begin; c < end; ++c) {
        while (c >= a.start[t + 1]) ++t;
        const int64_t first = (c - a.start[t]) * kChunk;
        sum += squares(a.d[t].g, a.f32[t] & 1, first + threadIdx.x, min(first + kChunk, a.d[t].n));
    }
    sum = block_sum(sum, s);
    if (threadIdx.x == 0) a.parts[a.parts_at + blockIdx.x] = sum;
}

__device__ double total(const double* parts, int n, double* s)
{
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kGradThreads) sum += parts[i];
    return sqrt(block_sum(sum, s));
}

__global__ void __launch_bounds__(kGradThreads) norm_kernel(const double* parts, int n, float* norm)
{
    __shared__ double s[kGradThreads / 32];
    const double x = total(parts, n, s);
    if (threadIdx.x == 0) *norm = static_cast<float>(x);
}

__global__ void __launch_bounds__(kGradThreads) clip_kernel(const __grid_constant__ GradArgs a)
{
    __shared__ double s[kGradThreads / 32];
    const double norm = total(a.parts, a.nparts, s);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = static_cast<float>(norm);
    const double ratio = a.max_norm / (norm + 1e-6);
    const float c = ratio >= 1.0 ? 1.0f : static_cast<float>(ratio);       // NaN stays NaN
    const int64_t begin = blockIdx.x * a.nchunks / gridDim.x;
    const int64_t end = (blockIdx.x + 1) * a.nchunks / gridDim.x;
    int t = begin < end ? find(a.start, a.nt, begin) : 0;
    for (int64_t k = begin; k < end; ++k) {
        while (k >= a.start[t + 1]) ++t;
        const Grad& d = a.d[t];
        if (c == 1.0f && d.out == d.g) continue;
        const int64_t first = (k - a.start[t]) * kChunk, last = min(first + kChunk, d.n);
        for (int64_t i = first + threadIdx.x; i < last; i += kGradThreads) {
            const float x = __fmul_rn(load(d.g, a.f32[t] & 1, i), c);
            if (a.f32[t] & 2) static_cast<float*>(d.out)[i] = x;
            else static_cast<uint16_t*>(d.out)[i] = float_to_bf16(x);
        }
    }
}

}  // namespace

cudaError_t prepare_grads()
{
    int g = 0;
    for (const void* k : {reinterpret_cast<const void*>(squares_kernel), reinterpret_cast<const void*>(norm_kernel),
                          reinterpret_cast<const void*>(clip_kernel)}) {
        const cudaError_t e = persistent_grid(k, kGradThreads, 0, &g);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int64_t grads_workspace(int count) { return (static_cast<int64_t>(count) / kMaxGrads + 1) * kMaxParts * 8; }

cudaError_t launch_grads(const q8_grad* list, int count, bool clip, double max_norm, float* norm, void* workspace,
                         cudaStream_t st)
{
    int grid = 0;
    cudaError_t e = persistent_grid(reinterpret_cast<const void*>(squares_kernel), kGradThreads, 0, &grid);
    if (e != cudaSuccess) return e;
    grid = std::min(grid, kMaxParts);
    std::unique_ptr<GradArgs> a(new GradArgs());
    a->parts = static_cast<double*>(workspace);
    a->norm = norm;
    a->max_norm = max_norm;
    int parts = 0;
    for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
        int at = 0;
        for (int i = 0; i < count;) {
            a->nt = 0;
            a->start[0] = 0;
            for (; i < count && a->nt < kMaxGrads; ++i) {
                if (list[i].numel == 0) continue;
                const int n = a->nt++;
                a->d[n] = Grad{list[i].grad, list[i].out, list[i].numel};
                a->f32[n] = static_cast<uint8_t>((list[i].grad_dtype == Q8_F32 ? 1 : 0) | (list[i].out_dtype == Q8_F32 ? 2 : 0));
                a->start[n + 1] = a->start[n] + (list[i].numel + kChunk - 1) / kChunk;
            }
            a->nchunks = a->start[a->nt];
            if (a->nchunks == 0) continue;
            const int ctas = static_cast<int>(std::min<int64_t>(grid, a->nchunks));
            a->parts_at = at;
            at += ctas;
            a->nparts = parts;
            if (pass == 0) squares_kernel<<<ctas, kGradThreads, 0, st>>>(*a);
            else clip_kernel<<<ctas, kGradThreads, 0, st>>>(*a);
        }
        parts = at;
    }
    if (!clip || parts == 0) norm_kernel<<<1, kGradThreads, 0, st>>>(a->parts, parts, norm);
    return cudaGetLastError();
}

}  // namespace q8
