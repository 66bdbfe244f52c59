// q8_grads.cu -- the 2-norm of all gradients of a list, and their clipping
// (include/q8train.h).
//
// norm = sqrt(sum g^2), c = min(1, max_norm / (norm + 1e-6)), out = c * g: two
// operations an element, so both are bound by the gradients' bytes.
//
// A list travels as kernel parameters, kMaxGrads tensors to a launch.  Each
// tensor is cut into chunks of 32 KB that start on 16 bytes (the few
// elements before the first and behind the last whole vector of eight go one by
// one).  The CTAs take the chunks in turn, and each leaves one sum of squares in
// the workspace, in double; whoever needs the norm adds these up, without double
// arithmetic.  Clipping reads the gradients a second time, a CTA for each chunk,
// each launch's from the end backwards, so that what was read last, and is still
// in L2, comes first.  (Of several launches the first comes first: lists beyond
// 768 tensors find only the last launch's end in L2, if that.)  Every CTA of the
// clipping adds up all launches' sums: 7680 tensors of 20000 bf16 take 471 us, as
// one tensor 134; 76800 of them 12.6 ms, as one 1.33.
//
// Measured: the norm of 6.66e9 bf16 1.80 ms (7.4 TB/s of reads); clipping of
// 1.56e9 bf16 1.35 ms (9.35 GB moved, 6.9 TB/s; with as many CTAs as run at
// once, each with chunks in turn, 1.44 ms), of 40 million float32 to bf16 59 us
// (L2 has 60 of their 161 MB left; 62 us without).
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <limits>

#include "q8_device.cuh"
#include "q8_internal.h"
#include "q8_train.h"

namespace q8 {

namespace {

constexpr int kGradThreads = 256;
constexpr int kVecElems = 8;
// Vectors that a thread has in flight: 128 bytes of either type.
template <typename T> constexpr int kVecs = 16 / sizeof(T);
template <typename T> constexpr int kChunk = kGradThreads * kVecElems * kVecs<T>;
constexpr int kChunkBytes = kGradThreads * 128;
constexpr int kKeepBytes = 60 << 20;                  // of L2's 126 MB
constexpr int kPerSm = 3;                                  // CTAs of an SM that add up (four: 3 % slower)
constexpr int kClipPerSm = 6;                              // that clip (four: 3 % slower)
constexpr int kMaxGrads = 768;
constexpr int kMaxParts = 1024;                            // CTAs of one launch, at most

// A launch's time on the host grows with its parameters: short lists travel in
// short ones, with room for so many tensors (a norm of 64 tensors takes the host
// 7.9 us instead of 9.3).
constexpr int kFewGrads = 64;

struct Grad {
    const void* g;
    void* out;
    int64_t n;
};

// How a tensor's elements lie: the first `lead` come before a 16-byte boundary.
enum : uint8_t { kF32 = 1, kOutF32 = 2, kOutVec = 4 };     // kOutVec: out's vectors start on 16 bytes, too
struct Kind {
    uint8_t flags, lead;
};

template <int ROOM>
struct GradArgs {
    double* parts;             // sums of squares: kMaxParts of each launch
    float* norm;
    int64_t nchunks;
    float max_norm;
    int32_t each;              // chunks of a CTA of clip_kernel
    int32_t keep;              // the launch's last chunks, which L2 is to keep for the second pass
    int32_t nt;
    int32_t parts_at;          // this launch's place in parts
    int32_t nparts;            // all launches' sums
    uint16_t at[kMaxParts];                // the tensor of each CTA's first chunk
    uint16_t at_end[kMaxParts];            // and of the last chunks, from the end
    int64_t start[ROOM + 1];               // each tensor's first chunk
    Kind kind[ROOM];
    Grad d[ROOM];
};
static_assert(sizeof(GradArgs<kMaxGrads>) <= 32764, "kernel parameter space");

__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = float_to_bf16(x); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// Eight elements as they lie in memory: one 16-byte vector of bf16, two of float32.
template <typename T>
struct Eight {
    static constexpr int kWords = sizeof(T) / 2;
    uint4 w[kWords];

    // Loads that clipping may write over.  KEEP: L2 is to keep the line; else it
    // is the first to go.
    template <bool KEEP>
    __device__ __forceinline__ void read(const T* p)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = KEEP ? reinterpret_cast<const uint4*>(p)[i] : __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ float2 pair(int i) const
    {
        if constexpr (sizeof(T) == 2) {
            const uint32_t x = i == 0 ? w[0].x : i == 1 ? w[0].y : i == 2 ? w[0].z : w[0].w;
            return bf16x2(x);
        } else {
            const uint4& v = w[i / 2];
            return i % 2 ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w)) : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        }
    }
};

template <typename T>
__device__ __forceinline__ void add_squares(const Eight<T>& v, float2 (&sum)[2])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = v.pair(i);
        sum[i % 2] = __ffma2_rn(x, x, sum[i % 2]);
    }
}

// The squares of a thread's vectors p, p + kGradThreads * 8, ... before `stop`
// again, where their sum shows that some may have left fp32's range: the largest
// magnitude picks a power of two that brings all of them, or all that count,
// back into it.  Out of line, and read again, so that the loop keeps its registers.
// Zeros and values below some 4e-12 come here, too, and take longer: the norm of
// 50257 x 4096 bf16 62 us, 94 with nine rows of ten zeros, 108 of zeros alone, 194
// of values near 1e-13 (float32 121, 194, 217 and 387).
template <typename T>
__device__ __noinline__ double squares_scaled(const T* p, const T* stop)
{
    uint32_t top = 0;
    for (const T* q = p; q < stop; q += kGradThreads * kVecElems)
        for (int i = 0; i < kVecElems; ++i) top = max(top, __float_as_uint(load1(q + i)) & 0x7FFFFFFFu);
    const int exponent = static_cast<int>(top >> 23) - 127;
    if (top == 0) return 0.0;
    const int k = exponent == 128 ? 0 : max(-126, min(126, -exponent));       // infinity and NaN stay what they are
    const float scale = __int_as_float((127 + k) << 23);
    float sum = 0.0f;
    for (const T* q = p; q < stop; q += kGradThreads * kVecElems)
        for (int i = 0; i < kVecElems; ++i) {
            const float x = __fmul_rn(load1(q + i), scale);
            sum = __fmaf_rn(x, x, sum);
        }
    return static_cast<double>(sum) * __longlong_as_double(static_cast<int64_t>(1023 - 2 * k) << 52);
}

// A thread's sum of squares: hi + lo in fp32, lo what hi's roundings lost (Knuth's
// two-sum), and what came out of range for them in double.  This GPU adds some
// sixty floats in the time of one double: sums in double alone cost 6 us of a
// clipping of 8 MB.
struct Sum {
    float hi = 0.0f, lo = 0.0f;
    double rare = 0.0;
    bool any = false;

    __device__ __forceinline__ void add(float x)
    {
        const float t = __fadd_rn(hi, x), b = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(x, b)));
        hi = t;
    }
    // 2^90 leaves room for 2^36 summands
    static __device__ __forceinline__ bool in_range(float s) { return s >= 0x1p-70f && s <= 0x1p90f; }
    __device__ __forceinline__ void add_rare(double x)
    {
        rare += x;
        any = true;
    }
    // One element's square.
    __device__ __forceinline__ void add1(float x)
    {
        const float s = __fmul_rn(x, x);
        if (in_range(s)) add(s);
        else if (x != 0.0f) add_rare(static_cast<double>(x) * static_cast<double>(x));
    }
};

template <bool KEEP, typename T>
__device__ __forceinline__ void chunk_squares(Sum& total, const T* g, int64_t n, int lead, int64_t chunk)
{
    const int64_t first = lead + chunk * kChunk<T>;
    const T* p = g + first + threadIdx.x * kVecElems;
    const T* stop = p + kChunk<T>;
    float2 sum[2] = {};
    if (first + kChunk<T> <= n) {
        Eight<T> v[kVecs<T>];
#pragma unroll
        for (int j = 0; j < kVecs<T>; ++j) v[j].template read<KEEP>(p + j * kGradThreads * kVecElems);
#pragma unroll
        for (int j = 0; j < kVecs<T>; ++j) add_squares(v[j], sum);
    } else {
        const int64_t whole = first + (max(n - first, int64_t(0)) / kVecElems) * kVecElems;
        stop = g + whole;
#pragma unroll 2
        for (const T* q = p; q < stop; q += kGradThreads * kVecElems) {
            Eight<T> v;
            v.template read<KEEP>(q);
            add_squares(v, sum);
        }
        if (whole + threadIdx.x < n) total.add1(load1(g + whole + threadIdx.x));
    }
    if (chunk == 0 && static_cast<int>(threadIdx.x) < lead && threadIdx.x < n) total.add1(load1(g + threadIdx.x));
    const float s = __fadd_rn(__fadd_rn(sum[0].x, sum[0].y), __fadd_rn(sum[1].x, sum[1].y));
    if (Sum::in_range(s)) {
        total.add(s);
    } else {
        const double x = squares_scaled(p, stop);
        if (x != 0.0) total.add_rare(x);
    }
}

// The CTA's sum, to thread 0.
__device__ __forceinline__ double block_sum(Sum x)
{
    __shared__ float2 s[kGradThreads / 32];
    __shared__ double r[kGradThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int o = 16; o > 0; o /= 2) {
        const float hi = __shfl_xor_sync(~0u, x.hi, o), lo = __shfl_xor_sync(~0u, x.lo, o);
        x.add(hi);
        x.lo = __fadd_rn(x.lo, lo);
    }
    if (lane == 0) s[warp] = make_float2(x.hi, x.lo);
    const bool any = __syncthreads_or(x.any);
    if (any) {
        for (int o = 16; o > 0; o /= 2) x.rare += __shfl_xor_sync(~0u, x.rare, o);
        if (lane == 0) r[warp] = x.rare;
        __syncthreads();
    }
    double sum = 0.0;
    if (threadIdx.x == 0) {
        Sum t;
        for (int w = 0; w < kGradThreads / 32; ++w) {
            t.add(s[w].x);
            t.lo = __fadd_rn(t.lo, s[w].y);
        }
        sum = static_cast<double>(t.hi) + static_cast<double>(t.lo);
        if (any)
            for (int w = 0; w < kGradThreads / 32; ++w) sum += r[w];
    }
    return sum;
}

// Kernels of one call follow one another closely: the next one's CTAs take the
// places that this one's leave, and wait until all of its memory is there.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int ROOM>
__global__ void __launch_bounds__(kGradThreads, kPerSm) squares_kernel(const __grid_constant__ GradArgs<ROOM> a)
{
    let_next_start();
    const int64_t keep = a.nchunks - a.keep;
    Sum sum;
    int t = a.at[blockIdx.x];
    for (int64_t c = blockIdx.x; c < a.nchunks; c += gridDim.x) {
        while (c >= a.start[t + 1]) ++t;
        const Grad& d = a.d[t];
        const Kind k = a.kind[t];
        const int64_t i = c - a.start[t];
        if (k.flags & kF32) {
            if (c < keep) chunk_squares<false>(sum, static_cast<const float*>(d.g), d.n, k.lead, i);
            else chunk_squares<true>(sum, static_cast<const float*>(d.g), d.n, k.lead, i);
        } else {
            if (c < keep) chunk_squares<false>(sum, static_cast<const uint16_t*>(d.g), d.n, k.lead, i);
            else chunk_squares<true>(sum, static_cast<const uint16_t*>(d.g), d.n, k.lead, i);
        }
    }
    const double x = block_sum(sum);
    if (threadIdx.x == 0) a.parts[a.parts_at + blockIdx.x] = x;
}

// The square root of the sum of `n` parts, to all threads of the CTA: the sum and
// its root are rounded once each, however many parts there are.  The parts are
// added as whole numbers (integer operations on a double's bits, no double
// arithmetic), in units of 2^-58 of the largest part's power of two, their upper
// and lower 32 bits apart; a thread's sum of up to 2^b parts then travels as 54
// bits, in halves whose sums over a warp fit 32 bits.  What the 256 threads cut
// off is less than 2^(b - 45) of the sum: nothing beside fp32's 2^-24 below 2^27
// parts.  (Threads and warps that add in fp32, 13 roundings and one for every 256
// parts: 12.9 instead of 13.0 us for a clipping of 20 MB.)
__device__ __forceinline__ float norm_of(const double* parts, int n)
{
    __shared__ int top[kGradThreads / 32];
    __shared__ uint2 sums[kGradThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint64_t* bits = reinterpret_cast<const uint64_t*>(parts);
    int e = 0;                                             // the largest exponent, as doubles keep it; infinity's, and above it NaN
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kGradThreads) {
        const uint64_t x = bits[i];
        const int f = static_cast<int>(x >> 52) & 0x7FF;
        e = max(e, f == 0x7FF && x << 12 ? 0x800 : f);
    }
    e = __reduce_max_sync(~0u, e);
    if (lane == 0) top[warp] = e;
    __syncthreads();
    for (int w = 0; w < kGradThreads / 32; ++w) e = max(e, top[w]);
    if (e >= 0x7FF) return e == 0x7FF ? INFINITY : NAN;
    unsigned long long hi = 0, lo = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kGradThreads) {
        const uint64_t x = bits[i];
        const int f = static_cast<int>(x >> 52);
        const uint64_t m = f == 0 ? 0 : ((x & ((uint64_t(1) << 52) - 1)) | uint64_t(1) << 52) << 6 >> min(63, e - f);
        hi += m >> 32;
        lo += m & 0xFFFFFFFFu;
    }
    hi += lo >> 32;
    const int many = (n + kGradThreads - 1) / kGradThreads, b = many > 1 ? 32 - __clz(many - 1) : 0;
    const unsigned long long t = hi << (27 - b) | static_cast<uint32_t>(lo) >> (5 + b);
    const uint32_t t1 = __reduce_add_sync(~0u, static_cast<uint32_t>(t >> 27)), t0 = __reduce_add_sync(~0u, static_cast<uint32_t>(t) & 0x7FFFFFFu);
    if (lane == 0) sums[warp] = make_uint2(t1, t0);
    __syncthreads();
    unsigned long long upper = 0, lower = 0;
#pragma unroll
    for (int w = 0; w < kGradThreads / 32; ++w) {
        upper += sums[w].x;
        lower += sums[w].y;
    }
    float sum = __ull2float_rn((upper << 27) + lower);
    int k = e - 1023 - 58 + 5 + b;                         // the sum is `sum` * 2^k
    if (k & 1) {
        sum = __fadd_rn(sum, sum);
        --k;
    }
    // sqrt(sum) * 2^(k / 2), the power in two steps: that of a subnormal norm is none
    const int h0 = max(-126, min(127, k / 2)), h1 = max(-126, min(127, k / 2 - h0));
    return __fmul_rn(__fmul_rn(__fsqrt_rn(sum), __uint_as_float(static_cast<uint32_t>(127 + h0) << 23)),
                     __uint_as_float(static_cast<uint32_t>(127 + h1) << 23));
}

__global__ void __launch_bounds__(kGradThreads) norm_kernel(const double* parts, int n, float* norm)
{
    wait_for_previous();
    const float x = norm_of(parts, n);
    if (threadIdx.x == 0) *norm = x;
}

__device__ __forceinline__ uint32_t bf16_pair(float2 x)
{
    return static_cast<uint32_t>(float_to_bf16(x.x)) | static_cast<uint32_t>(float_to_bf16(x.y)) << 16;
}

template <typename T>
__device__ __forceinline__ void write8(const Eight<T>& v, float2 c, uint16_t* p, bool vec)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_pair(__fmul2_rn(v.pair(i), c));
    if (vec) {
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i % 2)));
    }
}

template <typename T>
__device__ __forceinline__ void write8(const Eight<T>& v, float2 c, float* p, bool vec)
{
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 x = __fmul2_rn(v.pair(i), c), y = __fmul2_rn(v.pair(i + 1), c);
        if (vec) {
            __stcs(reinterpret_cast<float4*>(p + 2 * i), make_float4(x.x, x.y, y.x, y.y));
        } else {
            p[2 * i] = x.x;
            p[2 * i + 1] = x.y;
            p[2 * i + 2] = y.x;
            p[2 * i + 3] = y.y;
        }
    }
}

template <typename T, typename O>
__device__ __noinline__ void chunk_clip(const T* g, O* out, int64_t n, int lead, bool vec, int64_t chunk, float c)
{
    constexpr int kStep = kGradThreads * kVecElems;
    const int64_t first = lead + chunk * kChunk<T>;
    const int64_t at = first + threadIdx.x * kVecElems;
    if (first + kChunk<T> <= n) {
        Eight<T> v[kVecs<T>];
#pragma unroll
        for (int j = 0; j < kVecs<T>; ++j) v[j].template read<false>(g + at + j * kStep);
#pragma unroll
        for (int j = 0; j < kVecs<T>; ++j) write8(v[j], splat(c), out + at + j * kStep, vec);
    } else {
        const int64_t whole = first + (max(n - first, int64_t(0)) / kVecElems) * kVecElems;
#pragma unroll 2
        for (int64_t i = at; i < whole; i += kStep) {
            Eight<T> v;
            v.template read<false>(g + i);
            write8(v, splat(c), out + i, vec);
        }
        if (whole + threadIdx.x < n) store1(out + whole + threadIdx.x, __fmul_rn(load1(g + whole + threadIdx.x), c));
    }
    if (chunk == 0 && static_cast<int>(threadIdx.x) < lead && threadIdx.x < n) store1(out + threadIdx.x, __fmul_rn(load1(g + threadIdx.x), c));
}

template <typename T>
__device__ __forceinline__ void chunk_clip(const T* g, const Grad& d, Kind k, int64_t chunk, float c)
{
    const bool vec = k.flags & kOutVec;
    if (k.flags & kOutF32) chunk_clip(g, static_cast<float*>(d.out), d.n, k.lead, vec, chunk, c);
    else chunk_clip(g, static_cast<uint16_t*>(d.out), d.n, k.lead, vec, chunk, c);
}

template <int ROOM>
__global__ void __launch_bounds__(kGradThreads, kClipPerSm) clip_kernel(const __grid_constant__ GradArgs<ROOM> a)
{
    int64_t c = a.nchunks - 1 - static_cast<int64_t>(blockIdx.x) * a.each;
    int t = 0;
    if (blockIdx.x < kMaxParts) {
        t = a.at_end[blockIdx.x];
    } else {
        for (int hi = a.nt; hi - t > 1;) {
            const int mid = (t + hi) / 2;
            if (a.start[mid] <= c) t = mid; else hi = mid;
        }
    }
    wait_for_previous();
    const float norm = norm_of(a.parts, a.nparts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
    const float ratio = __fdiv_rn(a.max_norm, __fadd_rn(norm, 1e-6f));
    const float f = ratio >= 1.0f ? 1.0f : ratio;                          // NaN stays NaN
    for (const int64_t stop = max(int64_t(0), c + 1 - a.each); c >= stop; --c) {
        while (c < a.start[t]) --t;
        const Grad& d = a.d[t];
        const Kind k = a.kind[t];
        if (f == 1.0f && d.out == d.g) continue;
        if (k.flags & kF32) chunk_clip(static_cast<const float*>(d.g), d, k, c - a.start[t], f);
        else chunk_clip(static_cast<const uint16_t*>(d.g), d, k, c - a.start[t], f);
    }
}

// The kernel after another one of the same call (wait_for_previous).
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), int grid, cudaStream_t st, const Args&... args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kGradThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// An entry's place in a launch: its vectors' alignment and its chunks.
template <int ROOM>
void add(GradArgs<ROOM>& a, const q8_grad& g)
{
    const int size = g.grad_dtype == Q8_F32 ? 4 : 2, out_size = g.out_dtype == Q8_F32 ? 4 : 2;
    const int lead = static_cast<int>((16 - reinterpret_cast<uintptr_t>(g.grad) % 16) % 16) / size;
    const bool vec = (reinterpret_cast<uintptr_t>(g.out) + lead * out_size) % 16 == 0;
    const int chunk = size == 4 ? kChunk<float> : kChunk<uint16_t>;
    const int n = a.nt++;
    a.d[n] = Grad{g.grad, g.out, g.numel};
    a.kind[n] = Kind{static_cast<uint8_t>((size == 4 ? kF32 : 0) | (out_size == 4 ? kOutF32 : 0) | (vec ? kOutVec : 0)),
                     static_cast<uint8_t>(lead)};
    a.start[n + 1] = a.start[n] + std::max<int64_t>(1, (g.numel - lead + chunk - 1) / chunk);
}

template <int ROOM>
cudaError_t run_grads(const q8_grad* list, int count, bool clip, double max_norm, float* norm, void* workspace, cudaStream_t st)
{
    int grid = 0;
    cudaError_t e = persistent_grid(reinterpret_cast<const void*>(squares_kernel<ROOM>), kGradThreads, 0, &grid);
    if (e != cudaSuccess) return e;
    grid = std::min(grid, kMaxParts);
    GradArgs<ROOM> a;
    a.parts = static_cast<double*>(workspace);
    a.norm = norm;
    a.max_norm = static_cast<float>(std::isinf(max_norm) ? max_norm : std::min(max_norm, static_cast<double>(FLT_MAX)));
    a.nparts = 0;
    bool in_place = clip;
    for (int i = 0; i < count && in_place; ++i) in_place = list[i].out == list[i].grad;
    int parts = 0;
    for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
        bool first = true;
        for (int i = 0; i < count;) {
            if (pass == 0 || count > ROOM) {               // the second pass finds a list of one launch as the first left it
                a.nt = 0;
                a.start[0] = 0;
                for (; i < count && a.nt < ROOM; ++i)
                    if (list[i].numel) add(a, list[i]);
                a.nchunks = a.start[a.nt];
            } else {
                i = count;
            }
            if (a.nchunks == 0) continue;
            if (a.nchunks > std::numeric_limits<int32_t>::max()) return cudaErrorInvalidConfiguration;
            // in place there may be nothing to write, and CTAs that only come to
            // see that are to be few (1.6e9 bf16 with c = 1: 473 us, the norm alone
            // 446; with a CTA for each chunk 661)
            a.each = in_place ? static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(16, a.nchunks / 1024))) : 1;
            const int ctas = static_cast<int>(pass == 0 ? std::min<int64_t>(grid, a.nchunks) : (a.nchunks + a.each - 1) / a.each);
            for (int b = 0, t = 0; pass == 0 && b < ctas; ++b) {
                while (b >= a.start[t + 1]) ++t;
                a.at[b] = static_cast<uint16_t>(t);
            }
            for (int b = 0, t = a.nt - 1; pass == 1 && b < ctas && b < kMaxParts; ++b) {
                while (a.nchunks - 1 - static_cast<int64_t>(b) * a.each < a.start[t]) --t;
                a.at_end[b] = static_cast<uint16_t>(t);
            }
            if (pass == 0) {
                a.parts_at = parts;
                a.keep = clip ? kKeepBytes / kChunkBytes : 0;
                parts += ctas;
                squares_kernel<ROOM><<<ctas, kGradThreads, 0, st>>>(a);
            } else if (first) {
                if ((e = launch_after(clip_kernel<ROOM>, ctas, st, a)) != cudaSuccess) return e;
                first = false;
            } else {
                clip_kernel<ROOM><<<ctas, kGradThreads, 0, st>>>(a);
            }
        }
        a.nparts = parts;
    }
    if (parts == 0) norm_kernel<<<1, kGradThreads, 0, st>>>(a.parts, 0, norm);
    else if (!clip) e = launch_after(norm_kernel, 1, st, static_cast<const double*>(a.parts), parts, norm);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int ROOM>
cudaError_t prepare_room()
{
    int g = 0;
    const cudaError_t e = persistent_grid(reinterpret_cast<const void*>(squares_kernel<ROOM>), kGradThreads, 0, &g);
    return e != cudaSuccess ? e : persistent_grid(reinterpret_cast<const void*>(clip_kernel<ROOM>), kGradThreads, 0, &g);
}

}  // namespace

cudaError_t prepare_grads()
{
    int g = 0;
    cudaError_t e = persistent_grid(reinterpret_cast<const void*>(norm_kernel), kGradThreads, 0, &g);
    if (e == cudaSuccess) e = prepare_room<kFewGrads>();
    return e == cudaSuccess ? prepare_room<kMaxGrads>() : e;
}

int64_t grads_workspace(int count) { return (static_cast<int64_t>(count) / kMaxGrads + 1) * kMaxParts * 8; }

cudaError_t launch_grads(const q8_grad* list, int count, bool clip, double max_norm, float* norm, void* workspace,
                         cudaStream_t st)
{
    return count <= kFewGrads ? run_grads<kFewGrads>(list, count, clip, max_norm, norm, workspace, st)
                              : run_grads<kMaxGrads>(list, count, clip, max_norm, norm, workspace, st);
}

}  // namespace q8
