// q8_norm.cu -- the norms around a block's gate and residual
// (include/q8train.h), forward and backward.
//
// The kernels give a row to a CTA of dim / E threads, E elements of fixed
// columns to each, and walk over rows; the next row's loads are in flight while
// a row is worked on, and several CTAs on an SM cover each other's reductions.
// A row is read once: its statistics come from registers (a layer norm's
// variance from the deviations, not from a difference of sums).  Bytes bound
// both directions: forward 8, backward 12 bytes an element in bf16.  16384 x
// 4096: forward 85 us, 6.3 TB/s (93 % of a copy's rate); backward with RMS norms
// and 8 gates 228 us, 3.5 TB/s: four reductions a row, one after another, and the
// sums' reads and writes in shared memory; no unit is above 62 %, it waits.
//
// The backward kernels recompute both norms from r and y and sum the weights'
// gradients over its rows, in shared memory (each column has one thread, so
// nothing is shared in fact; registers would leave room for half the CTAs).
// A CTA's rows are consecutive, so that a gate's group ends inside a CTA (and
// is written there) or is one of the two that reach over its ends.  norm_sum
// adds up the CTAs' sums, in their order.
#include <algorithm>
#include <mutex>
#include <set>

#include "q8_internal.h"
#include "q8_tc.cuh"
#include "q8_train.h"

namespace q8 {

namespace {

struct Forward {
    q8_block_norm n;
    void* residual_out;
    uint16_t* z;
    int64_t residual_out_stride, z_stride;
};

// Sums over the CTA's rows, each [dim] a CTA: which of them are wanted, and
// where they go (partial[index among the wanted][cta][dim]).
enum Sum { kPostWeight, kPostBias, kPreWeight, kPreBias, kGate, kSums };

struct Backward {
    q8_block_norm n;
    q8_block_norm_grads g;
    float* partial;                  // the weights' sums, a row of dim for each CTA
    float* gate_partial;             // [cta][2][dim]: groups that reach over the CTA's first and last row
    float* scratch;                  // [cta][wanted sums][dim], where shared memory does not hold them
    int32_t at[kSums];               // index among the wanted sums, -1: not wanted
    int32_t wanted;
    int32_t* fault;
};

// ------------------------------------------------------- a thread's columns

// E elements of a row of T: with VEC 8, chunks of eight, (i * threads + thread)
// apart (rows and pointers on 16 bytes, dim a multiple of eight); with VEC 1,
// single elements.  Raw is what is held while a load is in flight.
template <typename T, int VEC, int E>
struct Raw;

template <int E>
struct Raw<uint16_t, 8, E> {
    uint4 q[E / 8];
    __device__ __forceinline__ void load(const uint16_t* row, int dim)
    {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * 8;
            q[i] = c < dim ? __ldcs(reinterpret_cast<const uint4*>(row + c)) : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void get(float (&v)[E]) const
    {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    }
};

template <int E>
struct Raw<float, 8, E> {
    float4 q[E / 4];
    __device__ __forceinline__ void load(const float* row, int dim)
    {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const int c = ((i / 2) * blockDim.x + threadIdx.x) * 8 + (i & 1) * 4;
            q[i] = c < dim ? __ldcs(reinterpret_cast<const float4*>(row + c)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    }
    __device__ __forceinline__ void get(float (&v)[E]) const
    {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            v[4 * i] = q[i].x;
            v[4 * i + 1] = q[i].y;
            v[4 * i + 2] = q[i].z;
            v[4 * i + 3] = q[i].w;
        }
    }
};

template <typename T, int E>
struct Raw<T, 1, E> {
    T q[E];
    __device__ __forceinline__ void load(const T* row, int dim)
    {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            q[i] = c < dim ? row[c] : T(0);
        }
    }
    __device__ __forceinline__ void get(float (&v)[E]) const
    {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if constexpr (sizeof(T) == 2) v[i] = bf16_to_float(q[i]);
            else v[i] = q[i];
        }
    }
};

// Whether the thread's element i exists.
template <int VEC>
__device__ __forceinline__ bool inside(int i, int dim)
{
    return VEC == 8 ? static_cast<int>((i / 8) * blockDim.x + threadIdx.x) * 8 < dim
                    : static_cast<int>(i * blockDim.x + threadIdx.x) < dim;
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int VEC, int E>
__device__ __forceinline__ void put(uint16_t* row, int dim, const float (&v)[E])
{
    if constexpr (VEC == 8) {
#pragma unroll
        for (int i = 0; i < E; i += 8)
            if (inside<8>(i, dim))
                __stcs(reinterpret_cast<uint4*>(row + ((i / 8) * blockDim.x + threadIdx.x) * 8),
                       make_uint4(pack2(v[i], v[i + 1]), pack2(v[i + 2], v[i + 3]), pack2(v[i + 4], v[i + 5]),
                                  pack2(v[i + 6], v[i + 7])));
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (inside<1>(i, dim)) row[i * blockDim.x + threadIdx.x] = float_to_bf16(v[i]);
    }
}

template <int VEC, int E>
__device__ __forceinline__ void put(float* row, int dim, const float (&v)[E])
{
    if constexpr (VEC == 8) {
#pragma unroll
        for (int i = 0; i < E; i += 4)
            if (inside<8>(i, dim))
                __stcs(reinterpret_cast<float4*>(row + ((i / 8) * blockDim.x + threadIdx.x) * 8 + (i & 4)),
                       make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (inside<1>(i, dim)) row[i * blockDim.x + threadIdx.x] = v[i];
    }
}

// A vector of all channels (weights, biases, a gate's row): it stays in cache.
template <int VEC, int E>
__device__ __forceinline__ void channels(const uint16_t* p, int dim, float none, float (&v)[E])
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = none;
        return;
    }
    if constexpr (VEC == 8) {
        Raw<uint16_t, 8, E> r;
#pragma unroll
        for (int i = 0; i < E / 8; ++i)
            r.q[i] = inside<8>(8 * i, dim) ? __ldg(reinterpret_cast<const uint4*>(p) + i * blockDim.x + threadIdx.x)
                                           : make_uint4(0, 0, 0, 0);
        r.get(v);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = inside<1>(i, dim) ? bf16_to_float(__ldg(p + i * blockDim.x + threadIdx.x)) : 0.0f;
    }
}

// --------------------------------------------------------------- reductions

// K sums over the CTA, in every thread: one barrier, for which two buffers take
// turns (a buffer is written again only after the barrier that follows its
// reading).
struct Reducer {
    float* part;                     // [2][32][2]
    int turn = 0;

    template <int K>
    __device__ __forceinline__ void sum(float (&s)[K])
    {
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < K; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], o);
        if (warps == 1) return;
        float* p = part + turn * 64;
        turn ^= 1;
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) p[2 * (threadIdx.x >> 5) + k] = s[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] = lane < warps ? p[2 * lane + k] : 0.0f;
        for (int o = 16; o > 0; o >>= 1)
            if (o < warps || o == 1)
#pragma unroll
                for (int k = 0; k < K; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], o);
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] = __shfl_sync(0xFFFFFFFFu, s[k], 0);
    }
};

// v becomes (v - mean) / root (elements that do not exist: 0); the reciprocal
// root is returned.
template <int VEC, int E>
__device__ __forceinline__ float normalise(float (&v)[E], int dim, float inv_dim, int kind, float eps, Reducer& red)
{
    if (kind == Q8_NORM_NONE) return 1.0f;
    if (kind == Q8_NORM_LAYER) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] += v[i];
        red.sum(s);
        const float mean = s[0] * inv_dim;
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = inside<VEC>(i, dim) ? v[i] - mean : 0.0f;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < E; ++i) q[0] = fmaf(v[i], v[i], q[0]);
    red.sum(q);
    const float rs = rsqrtf(fmaf(q[0], inv_dim, eps));
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= rs;
    return rs;
}

// ------------------------------------------------------------------- forward

template <typename R, int VEC, int E, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : 1) norm_forward_kernel(const __grid_constant__ Forward a)
{
    __shared__ float s_part[128];
    Reducer red{s_part};
    const q8_block_norm& n = a.n;
    const int dim = static_cast<int>(n.dim);
    const float inv_dim = 1.0f / dim;
    const R* residual = static_cast<const R*>(n.residual);
    R* out = static_cast<R*>(a.residual_out);
    Raw<uint16_t, VEC, E> y_next;
    Raw<R, VEC, E> r_next;
    int64_t t = blockIdx.x;
    y_next.load(n.y + t * n.y_stride, dim);
    r_next.load(residual + t * n.residual_stride, dim);
    for (; t < n.tokens; t += gridDim.x) {
        float v[E], r[E], w[E];
        y_next.get(v);
        r_next.get(r);
        const int64_t next = t + gridDim.x;
        if (next < n.tokens) {
            y_next.load(n.y + next * n.y_stride, dim);
            r_next.load(residual + next * n.residual_stride, dim);
        }
        normalise<VEC>(v, dim, inv_dim, n.post_kind, n.eps, red);
        if (n.post_weight) {
            channels<VEC>(n.post_weight, dim, 1.0f, w);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] *= w[i];
        }
        if (n.post_bias) {
            channels<VEC>(n.post_bias, dim, 0.0f, w);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] += w[i];
        }
        if (n.gate) {
            channels<VEC>(n.gate + t / n.gate_tokens * n.dim, dim, 1.0f, w);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = fmaf(n.residual_scale, r[i], v[i]);
        if (out) put<VEC>(out + t * a.residual_out_stride, dim, v);
        if (!a.z) continue;
        normalise<VEC>(v, dim, inv_dim, n.pre_kind, n.eps, red);
        if (n.pre_weight) {
            channels<VEC>(n.pre_weight, dim, 1.0f, w);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] *= w[i];
        }
        if (n.pre_bias) {
            channels<VEC>(n.pre_bias, dim, 0.0f, w);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] += w[i];
        }
        put<VEC>(a.z + t * a.z_stride, dim, v);
    }
}

// ------------------------------------------------------------------ backward

constexpr int64_t kMostCtas = 16384;

// Rows [first, stop) of CTA c of `ctas`.
__host__ __device__ __forceinline__ int64_t first_row(int64_t tokens, int64_t c, int64_t ctas)
{
    const uint32_t n = static_cast<uint32_t>(ctas);          // at most kMostCtas: the product fits
    return tokens / ctas * c + static_cast<uint32_t>(tokens % ctas) * static_cast<uint32_t>(c) / n;
}

// The backward kernel works on eight elements (a chunk) at a time, in packed
// fp32 pairs: what it keeps of a row between its reductions is y, dz and dr' as
// they came and one fp32 value an element.  Beside the next row's loads that is
// more than 128 registers at E = 16 (140 to 360 bytes a thread are spilled with
// vectors, 788 to 1006 with single elements) and far more than 64 at the wider
// shapes (624 to 4438 bytes): it takes the rows that the staged kernel below
// does not.  RMS, bf16: 4096 x 16384 452 us, 2048 x 32768 1359 us (120 us of
// bytes each), 12007 x 4097 1560 us (88 us).
struct Eight {
    float2 v[4];
};

template <int E>
__device__ __forceinline__ Eight chunk_of(const Raw<uint16_t, 8, E>& r, int c)
{
    const uint32_t w[4] = {r.q[c].x, r.q[c].y, r.q[c].z, r.q[c].w};
    Eight e;
#pragma unroll
    for (int j = 0; j < 4; ++j) e.v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    return e;
}
template <int E>
__device__ __forceinline__ Eight chunk_of(const Raw<float, 8, E>& r, int c)
{
    const float4 a = r.q[2 * c], b = r.q[2 * c + 1];
    return Eight{{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}
template <typename T, int E>
__device__ __forceinline__ Eight chunk_of(const Raw<T, 1, E>& r, int c)
{
    float v[E];
    r.get(v);
    Eight e;
#pragma unroll
    for (int j = 0; j < 4; ++j) e.v[j] = make_float2(v[8 * c + 2 * j], v[8 * c + 2 * j + 1]);
    return e;
}

// The column of element j of chunk c.
template <int VEC>
__device__ __forceinline__ int column(int c, int j)
{
    return VEC == 8 ? (c * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8 + j
                    : (8 * c + j) * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
}

template <int VEC>
__device__ __forceinline__ Eight channels(const uint16_t* p, int dim, int c)
{
    Eight e;
    if constexpr (VEC == 8) {
        Raw<uint16_t, 8, 8> r;
        r.q[0] = column<8>(c, 0) < dim ? __ldg(reinterpret_cast<const uint4*>(p + column<8>(c, 0))) : make_uint4(0, 0, 0, 0);
        return chunk_of(r, 0);
    } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = column<1>(c, j) < dim ? bf16_to_float(__ldg(p + column<1>(c, j))) : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) e.v[j] = make_float2(v[2 * j], v[2 * j + 1]);
        return e;
    }
}

template <int VEC>
__device__ __forceinline__ void put(uint16_t* row, int dim, int c, const Eight& e)
{
    if constexpr (VEC == 8) {
        if (column<8>(c, 0) < dim)
            __stcs(reinterpret_cast<uint4*>(row + column<8>(c, 0)),
                   make_uint4(pack2(e.v[0].x, e.v[0].y), pack2(e.v[1].x, e.v[1].y), pack2(e.v[2].x, e.v[2].y),
                              pack2(e.v[3].x, e.v[3].y)));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (column<1>(c, j) < dim) row[column<1>(c, j)] = float_to_bf16(j & 1 ? e.v[j / 2].y : e.v[j / 2].x);
    }
}
template <int VEC>
__device__ __forceinline__ void put(float* row, int dim, int c, const Eight& e)
{
    if constexpr (VEC == 8) {
        if (column<8>(c, 0) < dim) {
            float4* p = reinterpret_cast<float4*>(row + column<8>(c, 0));
            __stcs(p, make_float4(e.v[0].x, e.v[0].y, e.v[1].x, e.v[1].y));
            __stcs(p + 1, make_float4(e.v[2].x, e.v[2].y, e.v[3].x, e.v[3].y));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (column<1>(c, j) < dim) row[column<1>(c, j)] = j & 1 ? e.v[j / 2].y : e.v[j / 2].x;
    }
}

// Sums of a chunk's columns: two 16-byte halves, each of consecutive threads on
// consecutive addresses; the columns' order among them is the threads' own.
__device__ __forceinline__ float4* sums_at(float* sums, int c, int half)
{
    return reinterpret_cast<float4*>(sums) + (2 * c + half) * blockDim.x + threadIdx.x;
}
__device__ __forceinline__ void accumulate(float* sums, int c, const Eight& e)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float4* p = sums_at(sums, c, h);
        const float4 s = *p;
        const float2 a = __fadd2_rn(make_float2(s.x, s.y), e.v[2 * h]), b = __fadd2_rn(make_float2(s.z, s.w), e.v[2 * h + 1]);
        *p = make_float4(a.x, a.y, b.x, b.y);
    }
}

// The thread's columns of the sums, which are set to zero, into a row of dim.
template <int VEC, int E, typename Out>
__device__ __forceinline__ void flush(float* sums, int dim, Out* row)
{
#pragma unroll
    for (int c = 0; c < E / 8; ++c) {
        const float4 a = *sums_at(sums, c, 0), b = *sums_at(sums, c, 1);
        *sums_at(sums, c, 0) = *sums_at(sums, c, 1) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const Eight e{{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
        if (VEC == 8 && (reinterpret_cast<uintptr_t>(row) & 15) != 0) {       // a gate's gradient may lie on any address
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (column<VEC>(c, j) < dim) {
                    const float v = j & 1 ? e.v[j / 2].y : e.v[j / 2].x;
                    if constexpr (sizeof(Out) == 2) row[column<VEC>(c, j)] = float_to_bf16(v);
                    else row[column<VEC>(c, j)] = v;
                }
        } else {
            put<VEC>(row, dim, c, e);
        }
    }
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ Eight operator*(const Eight& a, const Eight& b)
{
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = __fmul2_rn(a.v[j], b.v[j]);
    return r;
}
__device__ __forceinline__ Eight operator*(const Eight& a, float b)
{
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = __fmul2_rn(a.v[j], both(b));
    return r;
}
__device__ __forceinline__ Eight operator+(const Eight& a, const Eight& b)
{
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = __fadd2_rn(a.v[j], b.v[j]);
    return r;
}
__device__ __forceinline__ Eight operator+(const Eight& a, float b)
{
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = __fadd2_rn(a.v[j], both(b));
    return r;
}
// a b + c
__device__ __forceinline__ Eight fma8(const Eight& a, const Eight& b, const Eight& c)
{
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = __ffma2_rn(a.v[j], b.v[j], c.v[j]);
    return r;
}
__device__ __forceinline__ Eight fma8(const Eight& a, float b, const Eight& c)
{
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = __ffma2_rn(a.v[j], both(b), c.v[j]);
    return r;
}
__device__ __forceinline__ void add_dot(float2& s, const Eight& a, const Eight& b)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) s = __ffma2_rn(a.v[j], b.v[j], s);
}
__device__ __forceinline__ void add_all(float2& s, const Eight& a)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) s = __fadd2_rn(s, a.v[j]);
}
// Elements past the row's end become 0.
template <int VEC>
__device__ __forceinline__ Eight masked(const Eight& a, int c, int dim)
{
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        r.v[j] = make_float2(column<VEC>(c, 2 * j) < dim ? a.v[j].x : 0.0f, column<VEC>(c, 2 * j + 1) < dim ? a.v[j].y : 0.0f);
    return r;
}

// A vector of all channels as it lies in memory; ones where there is none.
template <int VEC, int E>
__device__ __forceinline__ void hold(Raw<uint16_t, VEC, E>& r, const uint16_t* p, int dim)
{
    if (p) {
        r.load(p, dim);
    } else if constexpr (VEC == 8) {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) r.q[i] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) r.q[i] = 0x3F80;
    }
}

// LAYER: one of the two norms is a layer norm (its means cost reductions that
// other launches do without).  The weights and the gate's row stay in registers:
// read again for each row, their latencies were what a row took longest for.
// Rows off 16 bytes come one element at a time: 3001 x 1601, layer norms, float32
// residual, 70 us for 86 MB, by instructions and six reductions a row.
template <typename R, int VEC, int E, int MAXT, bool LAYER>
__global__ void __launch_bounds__(MAXT, 1) norm_backward_kernel(const __grid_constant__ Backward a)
{
    constexpr int C = E / 8;
    extern __shared__ float4 s_sums4[];
    __shared__ float s_part[128];
    Reducer red{s_part};
    const q8_block_norm& n = a.n;
    const q8_block_norm_grads& g = a.g;
    const int dim = static_cast<int>(n.dim), span = E * blockDim.x;
    const float inv_dim = 1.0f / dim;
    float* sums = a.scratch ? a.scratch + static_cast<int64_t>(blockIdx.x) * a.wanted * span : reinterpret_cast<float*>(s_sums4);
    for (int i = threadIdx.x; i < a.wanted * span; i += blockDim.x) sums[i] = 0.0f;
    __syncthreads();
    const auto sum_of = [&](int which) { return sums + a.at[which] * span; };

    const R* residual = static_cast<const R*>(n.residual);
    const R* dr_out = static_cast<const R*>(g.d_residual_out);
    R* dr = static_cast<R*>(g.d_residual);
    const int64_t first = first_row(n.tokens, blockIdx.x, gridDim.x), stop = first_row(n.tokens, blockIdx.x + 1, gridDim.x);
    int64_t group = n.gate ? first / n.gate_tokens : 0;
    int64_t group_end = n.gate ? (group + 1) * n.gate_tokens : n.tokens;
    const int64_t first_group = group;

    // the group's gate gradient: to its place where the CTA has all of the group,
    // else to the CTA's own part
    const auto flush_gate = [&](int64_t end) {
        if (a.at[kGate] < 0) return;
        if (group * n.gate_tokens >= first && (end == group_end || end == n.tokens))
            flush<VEC, E>(sum_of(kGate), dim, g.d_gate + group * n.dim);
        else
            flush<VEC, E>(sum_of(kGate), dim, a.gate_partial + (2 * static_cast<int64_t>(blockIdx.x) + (group != first_group)) * n.dim);
    };
    const auto reduce = [&](float2 s) {
        float t[1] = {s.x + s.y};
        red.sum(t);
        return t[0];
    };
    const auto reduce_two = [&](float2 a, float2 b) {
        float t[2] = {a.x + a.y, b.x + b.y};
        red.sum(t);
        return make_float2(t[0], t[1]);
    };

    Raw<uint16_t, VEC, E> y_next, dz_next{};
    Raw<R, VEC, E> r_next, dr_next{};
    const auto load = [&](int64_t t) {
        y_next.load(n.y + t * n.y_stride, dim);
        r_next.load(residual + t * n.residual_stride, dim);
        if (g.dz) dz_next.load(g.dz + t * g.dz_stride, dim);
        if (dr_out) dr_next.load(dr_out + t * g.d_residual_out_stride, dim);
    };
    load(first);
    Raw<uint16_t, VEC, E> w, gate, pw;
    hold(w, n.post_weight, dim);
    hold(pw, n.pre_weight, dim);
    hold(gate, n.gate ? n.gate + group * n.dim : nullptr, dim);
    for (int64_t t = first; t < stop; ++t) {
        if (t == group_end) {
            flush_gate(t);
            ++group;
            group_end += n.gate_tokens;
            hold(gate, n.gate + group * n.dim, dim);
        }
        const Raw<uint16_t, VEC, E> y = y_next, dz = dz_next;
        const Raw<R, VEC, E> r = r_next, dro = dr_next;
        if (t + 1 < stop) load(t + 1);
        // y's statistics
        float y_rs = 1.0f, y_mean = 0.0f;
        const bool y_layer = LAYER && n.post_kind == Q8_NORM_LAYER, r_layer = LAYER && n.pre_kind == Q8_NORM_LAYER;
        if (n.post_kind != Q8_NORM_NONE) {
            if (y_layer) {
                float2 s = both(0.0f);
#pragma unroll
                for (int c = 0; c < C; ++c) add_all(s, chunk_of(y, c));
                y_mean = reduce(s) * inv_dim;
            }
            float2 s = both(0.0f);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                Eight e = chunk_of(y, c);
                if (y_layer) e = masked<VEC>(e + -y_mean, c, dim);
                add_dot(s, e, e);
            }
            y_rs = rsqrtf(fmaf(reduce(s), inv_dim, n.eps));
        }
        const auto yn_of = [&](int c) {
            const Eight e = chunk_of(y, c);
            return (y_layer ? e + -y_mean : e) * y_rs;
        };
        // r', then normalised
        Eight rn[C];
        {
            float2 s = both(0.0f);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                Eight p = yn_of(c) * chunk_of(w, c);
                if (n.post_bias) p = p + channels<VEC>(n.post_bias, dim, c);
                rn[c] = fma8(chunk_of(r, c), n.residual_scale, p * chunk_of(gate, c));
                if (LAYER) rn[c] = masked<VEC>(rn[c], c, dim);
                if (r_layer) add_all(s, rn[c]);
                else add_dot(s, rn[c], rn[c]);
            }
            if (r_layer) {
                const float mean = reduce(s) * inv_dim;
                s = both(0.0f);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    rn[c] = masked<VEC>(rn[c] + -mean, c, dim);
                    add_dot(s, rn[c], rn[c]);
                }
            }
            if (n.pre_kind != Q8_NORM_NONE) s.x = reduce(s);
            const float rs = n.pre_kind == Q8_NORM_NONE ? 1.0f : rsqrtf(fmaf(s.x, inv_dim, n.eps));
#pragma unroll
            for (int c = 0; c < C; ++c) rn[c] = rn[c] * rs;
            // d, the gradient of r', comes from dz through the norm
            float dot = 0.0f, mean = 0.0f;
            if (g.dz) {
                float2 sd = both(0.0f), sm = both(0.0f);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    Eight e = chunk_of(dz, c);
                    if (a.at[kPreBias] >= 0) accumulate(sum_of(kPreBias), c, e);
                    if (a.at[kPreWeight] >= 0) accumulate(sum_of(kPreWeight), c, e * rn[c]);
                    e = e * chunk_of(pw, c);
                    add_dot(sd, e, rn[c]);
                    if (r_layer) add_all(sm, e);
                }
                if (r_layer) {
                    const float2 both_sums = reduce_two(sd, sm);
                    dot = both_sums.x * inv_dim;
                    mean = both_sums.y * inv_dim;
                } else if (n.pre_kind != Q8_NORM_NONE) {
                    dot = reduce(sd) * inv_dim;
                }
            }
            // d, dr, and the gradient of the normalised y (kept in rn)
            float2 sd = both(0.0f), sm = both(0.0f);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                Eight d = chunk_of(dro, c);
                if (g.dz) {
                    Eight e = chunk_of(dz, c) * chunk_of(pw, c);
                    e = fma8(rn[c], -dot, r_layer ? e + -mean : e);
                    d = fma8(e, rs, d);
                }
                if (dr) put<VEC>(dr + t * g.d_residual_stride, dim, c, d * n.residual_scale);
                const Eight yn = yn_of(c);
                const Eight dw = d * chunk_of(w, c), gc = chunk_of(gate, c);
                if (a.at[kGate] >= 0) {
                    Eight p = dw * yn;
                    if (n.post_bias) p = fma8(d, channels<VEC>(n.post_bias, dim, c), p);
                    accumulate(sum_of(kGate), c, p);
                }
                if (a.at[kPostBias] >= 0) accumulate(sum_of(kPostBias), c, d * gc);
                if (a.at[kPostWeight] >= 0) accumulate(sum_of(kPostWeight), c, d * gc * yn);
                d = dw * gc;
                if (LAYER) d = masked<VEC>(d, c, dim);
                add_dot(sd, d, yn);
                if (y_layer) add_all(sm, d);
                rn[c] = d;
            }
            if (!g.d_y) continue;
            dot = mean = 0.0f;
            if (y_layer) {
                const float2 both_sums = reduce_two(sd, sm);
                dot = both_sums.x * inv_dim;
                mean = both_sums.y * inv_dim;
            } else if (n.post_kind != Q8_NORM_NONE) {
                dot = reduce(sd) * inv_dim;
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const Eight e = fma8(yn_of(c), -dot, y_layer ? rn[c] + -mean : rn[c]);
                put<VEC>(g.d_y + t * g.d_y_stride, dim, c, e * y_rs);
            }
        }
    }
    if (first < stop) flush_gate(stop);
    for (int which = 0; which < kGate; ++which)
        if (a.at[which] >= 0)
            flush<VEC, E>(sum_of(which), dim, a.partial + (static_cast<int64_t>(a.at[which]) * gridDim.x + blockIdx.x) * n.dim);
}

// The same with the rows staged: one thread copies the four rows of the next
// token to shared memory (bulk copies) while this one's are worked on, so that a
// thread holds eight columns in 64 registers and an SM 32 warps; with the rows
// in registers 16 warps wait for one another's reductions half of the time
// (16384 x 4096 with three sums: 303 us with the rows in registers, 228 us
// staged).  Rows on 16 bytes.
template <typename R, bool LAYER, int MAXT, int CTAS>
__global__ void __launch_bounds__(MAXT, CTAS) norm_staged_kernel(const __grid_constant__ Backward a)
{
    extern __shared__ float4 s_sums4[];
    __shared__ float s_part[128];
    __shared__ __align__(8) uint64_t s_full[2];
    Reducer red{s_part};
    const q8_block_norm& n = a.n;
    const q8_block_norm_grads& g = a.g;
    const int dim = static_cast<int>(n.dim), span = 8 * blockDim.x, tid = threadIdx.x;
    const float inv_dim = 1.0f / dim;
    const bool mine = tid * 8 < dim;
    float* sums = reinterpret_cast<float*>(s_sums4);
    for (int i = tid; i < a.wanted * span; i += blockDim.x) sums[i] = 0.0f;
    const auto sum_of = [&](int which) { return sums + a.at[which] * span; };
    // a stage: y, dz, r, dr'
    uint8_t* stages = reinterpret_cast<uint8_t*>(sums + a.wanted * span);
    const int half = dim * 2, wide = dim * static_cast<int>(sizeof(R)), stage_bytes = 2 * half + 2 * wide;

    const int64_t first = first_row(n.tokens, blockIdx.x, gridDim.x), stop = first_row(n.tokens, blockIdx.x + 1, gridDim.x);
    int64_t group = n.gate ? first / n.gate_tokens : 0;
    int64_t group_end = n.gate ? (group + 1) * n.gate_tokens : n.tokens;
    const int64_t first_group = group;
    const auto flush_gate = [&](int64_t end) {
        if (a.at[kGate] < 0) return;
        if (group * n.gate_tokens >= first && (end == group_end || end == n.tokens))
            flush<8, 8>(sum_of(kGate), dim, g.d_gate + group * n.dim);
        else
            flush<8, 8>(sum_of(kGate), dim, a.gate_partial + (2 * static_cast<int64_t>(blockIdx.x) + (group != first_group)) * n.dim);
    };
    const auto reduce = [&](float2 s) {
        float t[1] = {s.x + s.y};
        red.sum(t);
        return t[0];
    };
    const auto reduce_two = [&](float2 a, float2 b) {
        float t[2] = {a.x + a.y, b.x + b.y};
        red.sum(t);
        return make_float2(t[0], t[1]);
    };
    const auto fetch = [&](int64_t t, int stage) {
        const uint32_t bar = smem_addr(&s_full[stage]), to = smem_addr(stages + stage * stage_bytes);
        bar_expect(bar, half + wide + (g.dz ? half : 0) + (g.d_residual_out ? wide : 0));
        bulk_load(to, n.y + t * n.y_stride, half, bar);
        if (g.dz) bulk_load(to + half, g.dz + t * g.dz_stride, half, bar);
        bulk_load(to + 2 * half, static_cast<const R*>(n.residual) + t * n.residual_stride, wide, bar);
        if (g.d_residual_out)
            bulk_load(to + 2 * half + wide, static_cast<const R*>(g.d_residual_out) + t * g.d_residual_out_stride, wide, bar);
    };
    if (tid == 0) {
        bar_init(smem_addr(&s_full[0]), 1);
        bar_init(smem_addr(&s_full[1]), 1);
        bar_init_fence();
    }
    __syncthreads();
    if (tid == 0) fetch(first, 0);

    Raw<uint16_t, 8, 8> w, gate, pw;
    hold(w, n.post_weight, dim);
    hold(pw, n.pre_weight, dim);
    hold(gate, n.gate ? n.gate + group * n.dim : nullptr, dim);
    R* dr = static_cast<R*>(g.d_residual);
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t t = first; t < stop; ++t) {
        if (t == group_end) {
            flush_gate(t);
            ++group;
            group_end += n.gate_tokens;
            hold(gate, n.gate + group * n.dim, dim);
        }
        const uint8_t* at = stages + stage * stage_bytes;
        const auto eight = [&](const uint8_t* p) {
            Raw<uint16_t, 8, 8> r;
            r.q[0] = mine ? reinterpret_cast<const uint4*>(p)[tid] : make_uint4(0, 0, 0, 0);
            return chunk_of(r, 0);
        };
        const auto eight_r = [&](const uint8_t* p) {
            Raw<R, 8, 8> r;
            if constexpr (sizeof(R) == 2) {
                return eight(p);
            } else {
                r.q[0] = mine ? reinterpret_cast<const float4*>(p)[2 * tid] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                r.q[1] = mine ? reinterpret_cast<const float4*>(p)[2 * tid + 1] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                return chunk_of(r, 0);
            }
        };
        if (ok) ok = bar_wait(smem_addr(&s_full[stage]), phase);

        // y's statistics
        const bool y_layer = LAYER && n.post_kind == Q8_NORM_LAYER, r_layer = LAYER && n.pre_kind == Q8_NORM_LAYER;
        float y_rs = 1.0f, y_mean = 0.0f;
        if (y_layer) {
            float2 s = both(0.0f);
            add_all(s, eight(at));
            y_mean = reduce(s) * inv_dim;
        }
        float2 s = both(0.0f);
        {
            Eight e = eight(at);
            if (y_layer) e = masked<8>(e + -y_mean, 0, dim);
            add_dot(s, e, e);
        }
        const float y_sq = reduce(s);                // all have left the row before: its stage is free
        if (n.post_kind != Q8_NORM_NONE) y_rs = rsqrtf(fmaf(y_sq, inv_dim, n.eps));
        if (tid == 0 && t + 1 < stop) fetch(t + 1, stage ^ 1);
        const auto yn_of = [&]() {
            const Eight e = eight(at);
            return (y_layer ? e + -y_mean : e) * y_rs;
        };

        // r', then normalised
        Eight rn;
        {
            Eight p = yn_of() * chunk_of(w, 0);
            if (n.post_bias) p = p + channels<8>(n.post_bias, dim, 0);
            rn = fma8(eight_r(at + 2 * half), n.residual_scale, p * chunk_of(gate, 0));
            if (LAYER) rn = masked<8>(rn, 0, dim);       // past the row's end a layer norm of y leaves -mean
        }
        float rs = 1.0f;
        if (n.pre_kind != Q8_NORM_NONE) {
            if (r_layer) {
                s = both(0.0f);
                add_all(s, rn);
                rn = masked<8>(rn + -(reduce(s) * inv_dim), 0, dim);
            }
            s = both(0.0f);
            add_dot(s, rn, rn);
            rs = rsqrtf(fmaf(reduce(s), inv_dim, n.eps));
            rn = rn * rs;
        }

        // d, the gradient of r': from dz through the norm, and from dr'
        Eight d = g.d_residual_out ? eight_r(at + 2 * half + wide) : Eight{};
        if (g.dz) {
            Eight e = eight(at + half);
            if (a.at[kPreBias] >= 0) accumulate(sum_of(kPreBias), 0, e);
            if (a.at[kPreWeight] >= 0) accumulate(sum_of(kPreWeight), 0, e * rn);
            e = e * chunk_of(pw, 0);
            if (n.pre_kind != Q8_NORM_NONE) {
                s = both(0.0f);
                add_dot(s, e, rn);
                if (r_layer) {
                    float2 m = both(0.0f);
                    add_all(m, e);
                    s = reduce_two(s, m);
                    e = e + -(s.y * inv_dim);
                } else {
                    s.x = reduce(s);
                }
                e = fma8(rn, -(s.x * inv_dim), e);
            }
            d = fma8(e, rs, d);
        }
        if (dr) put<8>(dr + t * g.d_residual_stride, dim, 0, d * n.residual_scale);
        const Eight yn = yn_of(), gc = chunk_of(gate, 0);
        const Eight dw = d * chunk_of(w, 0);
        if (a.at[kGate] >= 0) {
            Eight p = dw * yn;
            if (n.post_bias) p = fma8(d, channels<8>(n.post_bias, dim, 0), p);
            accumulate(sum_of(kGate), 0, p);
        }
        if (a.at[kPostBias] >= 0) accumulate(sum_of(kPostBias), 0, d * gc);
        if (a.at[kPostWeight] >= 0) accumulate(sum_of(kPostWeight), 0, d * gc * yn);
        d = dw * gc;
        if (g.d_y) {
            if (n.post_kind != Q8_NORM_NONE) {
                if (LAYER) d = masked<8>(d, 0, dim);
                s = both(0.0f);
                add_dot(s, d, yn);
                if (y_layer) {
                    float2 m = both(0.0f);
                    add_all(m, d);
                    s = reduce_two(s, m);
                    d = d + -(s.y * inv_dim);
                } else {
                    s.x = reduce(s);
                }
                d = fma8(yn, -(s.x * inv_dim), d) * y_rs;
            }
            put<8>(g.d_y + t * g.d_y_stride, dim, 0, d);
        }
        if ((stage ^= 1) == 0) phase ^= 1;
    }
    if (!ok) {                                       // leave no copy in flight
        atomicExch_system(a.fault, 1);
        bar_wait(smem_addr(&s_full[stage]), phase);
        bar_wait(smem_addr(&s_full[stage ^ 1]), phase ^ stage ^ 1);
    }
    if (first < stop) flush_gate(stop);
    for (int which = 0; which < kGate; ++which)
        if (a.at[which] >= 0)
            flush<8, 8>(sum_of(which), dim, a.partial + (static_cast<int64_t>(a.at[which]) * gridDim.x + blockIdx.x) * n.dim);
}

// What the CTAs have of each sum, added up: 32 columns to a block, its 16 warps
// take every 16th CTA, and their sums are added in order.  Blocks
// [0, count * column blocks): the weights' sums.  Then the gate: only a group
// that more than one CTA has rows of is summed here.  Where groups are fewer
// than CTAs, the same for each group; else a block for each CTA's end, which a
// group may reach over, with all columns.
struct SumArgs {
    const float *partial, *gate_partial;
    uint16_t *out[kGate], *gate_out;
    int64_t ctas, dim, tokens, gate_tokens, column_blocks;
    int32_t count;                   // of the weights' sums
};

__global__ void __launch_bounds__(512) norm_sum_kernel(const __grid_constant__ SumArgs a)
{
    __shared__ float part[16][33];
    const int64_t dim = a.dim, block = blockIdx.x;
    const int64_t col = block % a.column_blocks * 32 + threadIdx.x, which = block / a.column_blocks;
    const auto first = [&](int64_t c) { return first_row(a.tokens, c, a.ctas); };
    const float* p;
    uint16_t* out;
    int64_t from = threadIdx.y, stop = a.ctas, step = dim;
    float s = 0.0f;
    if (which < a.count) {
        p = a.partial + which * a.ctas * dim + col;
        out = a.out[which];
    } else {
        const int64_t groups = (a.tokens + a.gate_tokens - 1) / a.gate_tokens;
        const bool few = groups < a.ctas;
        int64_t begin, cta;                          // the group's first row, and the CTA that has it
        if (few) {
            begin = (which - a.count) * a.gate_tokens;       // below 2^40, the CTAs at most 2^14
            cta = begin * a.ctas / a.tokens;                 // or one beside it
            while (cta + 1 < a.ctas && first(cta + 1) <= begin) ++cta;
            while (first(cta) > begin) --cta;
        } else {
            cta = block - a.count * a.column_blocks;
            begin = first(cta + 1) / a.gate_tokens * a.gate_tokens;
            if (begin == first(cta + 1) || begin < first(cta)) return;
        }
        const int64_t end = min(begin + a.gate_tokens, a.tokens);
        if (cta + 1 == a.ctas || first(cta + 1) >= end) return;      // written by the CTA itself
        stop = min(a.ctas, (end - 1) * a.ctas / a.tokens + 2);
        while (first(stop - 1) >= end) --stop;
        // the first CTA's part lies in its second place unless the group is its first
        const float* head = a.gate_partial + (2 * cta + (first(cta) < begin)) * dim;
        out = a.gate_out + begin / a.gate_tokens * dim;
        if (!few) {
            for (int64_t c = threadIdx.y * 32 + threadIdx.x; c < dim; c += 512) {
                s = head[c];
                for (int64_t k = cta + 1; k < stop; ++k) s += a.gate_partial[2 * k * dim + c];
                out[c] = float_to_bf16(s);
            }
            return;
        }
        if (threadIdx.y == 0 && col < dim) s = head[col];
        p = a.gate_partial + col;
        from += cta + 1;
        step = 2 * dim;
    }
    if (col < dim) {
#pragma unroll 8
        for (int64_t c = from; c < stop; c += 16) s += p[c * step];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < dim) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += part[i][threadIdx.x];
        out[col] = float_to_bf16(s);
    }
}

// ------------------------------------------------------------------------- host

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool on16(const void* p, int64_t stride, int64_t elem) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * elem % 16 == 0; }

// Eight columns at a time: everything on 16 bytes.
bool vectors(const q8_block_norm& n)
{
    const int64_t elem = n.residual_dtype == Q8_F32 ? 4 : 2;
    bool ok = n.dim % 8 == 0 && on16(n.residual, n.residual_stride, elem) && on16(n.y, n.y_stride, 2);
    for (const void* p : {n.post_weight, n.post_bias, n.pre_weight, n.pre_bias, n.gate}) ok = ok && on16(p, 0, 2);
    return ok;
}

bool backward_vectors(const q8_block_norm& n, const q8_block_norm_grads& g)
{
    const int64_t elem = n.residual_dtype == Q8_F32 ? 4 : 2;
    return vectors(n) && on16(g.d_residual_out, g.d_residual_out ? g.d_residual_out_stride : 0, elem) &&
           on16(g.dz, g.dz ? g.dz_stride : 0, 2) && on16(g.d_residual, g.d_residual ? g.d_residual_stride : 0, elem) &&
           on16(g.d_y, g.d_y ? g.d_y_stride : 0, 2);
}

using ForwardKernel = void (*)(Forward);
using BackwardKernel = void (*)(Backward);

struct Shape {
    int elements, most;              // to a thread, threads at most
};

// Few threads a row, for each warp's reductions cost as much as four of its
// elements; rows up to 4096 columns leave several CTAs to an SM.
Shape forward_shape(int64_t dim)
{
    return dim <= 4096 ? Shape{16, 256} : dim <= 8192 ? Shape{16, 512} : dim <= 16384 ? Shape{32, 512} : Shape{64, 512};
}

Shape backward_shape(int64_t dim, bool vec)
{
    if (!vec && dim <= 4096) return Shape{8, 512};           // single elements take a register each
    return dim <= 8192 ? Shape{16, 512} : dim <= 16384 ? Shape{16, 1024} : Shape{32, 1024};
}

int threads_of(int64_t dim, int elements) { return static_cast<int>(ceil_div(ceil_div(dim, elements), 32) * 32); }

template <typename R, int VEC>
ForwardKernel forward_kernel(int64_t dim)
{
    const Shape s = forward_shape(dim);
    if (s.most == 256) return norm_forward_kernel<R, VEC, 16, 256>;
    return s.elements == 16 ? norm_forward_kernel<R, VEC, 16, 512>
                            : s.elements == 32 ? norm_forward_kernel<R, VEC, 32, 512> : norm_forward_kernel<R, VEC, 64, 512>;
}

template <typename R, int VEC, bool LAYER>
BackwardKernel backward_kernel(int64_t dim)
{
    const Shape s = backward_shape(dim, VEC == 8);
    if constexpr (VEC == 1)
        if (s.elements == 8) return norm_backward_kernel<R, VEC, 8, 512, LAYER>;
    return s.most == 512 ? norm_backward_kernel<R, VEC, 16, 512, LAYER>
                         : s.elements == 16 ? norm_backward_kernel<R, VEC, 16, 1024, LAYER> : norm_backward_kernel<R, VEC, 32, 1024, LAYER>;
}

ForwardKernel forward_kernel(bool f32, bool vec, int64_t dim)
{
    if (f32) return vec ? forward_kernel<float, 8>(dim) : forward_kernel<float, 1>(dim);
    return vec ? forward_kernel<uint16_t, 8>(dim) : forward_kernel<uint16_t, 1>(dim);
}

BackwardKernel backward_kernel(bool f32, bool vec, bool layer, int64_t dim)
{
    if (f32)
        return vec ? (layer ? backward_kernel<float, 8, true>(dim) : backward_kernel<float, 8, false>(dim))
                   : (layer ? backward_kernel<float, 1, true>(dim) : backward_kernel<float, 1, false>(dim));
    return vec ? (layer ? backward_kernel<uint16_t, 8, true>(dim) : backward_kernel<uint16_t, 8, false>(dim))
               : (layer ? backward_kernel<uint16_t, 1, true>(dim) : backward_kernel<uint16_t, 1, false>(dim));
}

// The staged kernel: rows up to 4096 columns in CTAs of which an SM holds two or
// more, up to 8192 in one.
template <typename R>
BackwardKernel staged_kernel(bool layer, int threads)
{
    if (threads <= 512) return layer ? norm_staged_kernel<R, true, 512, 2> : norm_staged_kernel<R, false, 512, 2>;
    return layer ? norm_staged_kernel<R, true, 1024, 1> : norm_staged_kernel<R, false, 1024, 1>;
}

BackwardKernel staged_kernel(bool f32, bool layer, int threads)
{
    return f32 ? staged_kernel<float>(layer, threads) : staged_kernel<uint16_t>(layer, threads);
}

// What the backward kernel does: a function of sizes, strides and pointers
// alone, for the workspace is sized by it.  As many CTAs as are resident.
constexpr int64_t kMostShared = 227 * 1024 - 1024;

struct Plan {
    int64_t ctas, span;              // span: columns of a sum as the CTA keeps it
    int threads, wanted, at[kSums];
    bool staged, vec, shared;        // shared: the sums lie in shared memory
    int64_t smem, partial, gate_partial, scratch, bytes;
};

Plan plan(const q8_block_norm& n, const q8_block_norm_grads& g, int sms)
{
    Plan p{};
    const uint16_t* outs[kSums] = {g.d_post_weight, g.d_post_bias, g.d_pre_weight, g.d_pre_bias, g.d_gate};
    for (int i = 0; i < kSums; ++i) p.at[i] = outs[i] ? p.wanted++ : -1;
    p.vec = backward_vectors(n, g);
    const int64_t stages = 2 * n.dim * (4 + 2 * (n.residual_dtype == Q8_F32 ? 4 : 2));
    int64_t resident;                                        // CTAs to an SM, by their threads
    p.threads = threads_of(n.dim, 8);
    p.span = p.threads * int64_t(8);
    p.smem = p.wanted * p.span * 4 + stages;
    p.staged = p.vec && p.threads <= 1024 && p.smem <= kMostShared;
    if (p.staged) {
        resident = 1024 / p.threads;
        p.shared = true;
    } else {
        const Shape s = backward_shape(n.dim, p.vec);
        p.threads = threads_of(n.dim, s.elements);
        p.span = static_cast<int64_t>(p.threads) * s.elements;
        p.smem = p.wanted * p.span * 4;
        p.shared = p.smem <= kMostShared;
        if (!p.shared) p.smem = 0;
        resident = std::max(1, s.most / p.threads);
    }
    resident = std::min<int64_t>({resident, 16, 228 * 1024 / (p.smem + 2048)});
    // past two CTAs to an SM, four rows to a CTA at least: each CTA's sums are
    // written and read once more
    p.ctas = std::min<int64_t>({n.tokens, kMostCtas, sms * std::max<int64_t>(1, resident),
                                std::max<int64_t>(2 * sms, ceil_div(n.tokens, 4))});
    auto take = [&](int64_t floats) {
        const int64_t at = p.bytes;
        p.bytes += ceil_div(floats * 4, 256) * 256;
        return at;
    };
    p.partial = take((p.wanted - (p.at[kGate] >= 0)) * p.ctas * n.dim);
    p.gate_partial = take(p.at[kGate] >= 0 ? 2 * p.ctas * n.dim : 0);
    p.scratch = take(p.shared ? 0 : p.ctas * p.wanted * p.span);
    return p;
}

int sm_count()
{
    DeviceInfo d;                                            // sizes do not need a GPU: 152 SMs where there is none
    if (device_info(&d) == cudaSuccess) return d.sms;
    cudaGetLastError();
    return 152;
}

}  // namespace

// Once for each device: kernels' shared-memory limits, launch configurations.
cudaError_t prepare_norm()
{
    static std::mutex lock;
    static std::set<int> done;
    int dev = 0, grid = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> guard(lock);
    if (done.count(dev)) return cudaSuccess;
    for (bool f32 : {false, true})
        for (bool vec : {false, true})
            for (int64_t dim : {4096, 8192, 16384, 32768}) {
                const Shape s = forward_shape(dim);
                if (e == cudaSuccess)
                    e = persistent_grid(reinterpret_cast<const void*>(forward_kernel(f32, vec, dim)), s.most, 0, &grid);
                for (bool layer : {false, true}) {
                    if (e == cudaSuccess)
                        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(staged_kernel(f32, layer, dim <= 4096 ? 512 : 1024)),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
                    if (e == cudaSuccess)
                        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(backward_kernel(f32, vec, layer, dim)),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
                }
            }
    if (e == cudaSuccess) done.insert(dev);
    return e;
}

cudaError_t launch_norm_forward(const q8_block_norm& n, void* residual_out, int64_t residual_out_stride, uint16_t* z,
                                int64_t z_stride, cudaStream_t st)
{
    const bool f32 = n.residual_dtype == Q8_F32;
    const bool vec = vectors(n) && on16(residual_out, residual_out ? residual_out_stride : 0, f32 ? 4 : 2) &&
                     on16(z, z ? z_stride : 0, 2);
    const ForwardKernel k = forward_kernel(f32, vec, n.dim);
    const int threads = threads_of(n.dim, forward_shape(n.dim).elements);
    int grid = 0;
    const cudaError_t e = persistent_grid(reinterpret_cast<const void*>(k), threads, 0, &grid);
    if (e != cudaSuccess) return e;
    k<<<static_cast<unsigned>(std::min<int64_t>(n.tokens, grid)), threads, 0, st>>>(
        Forward{n, residual_out, z, residual_out_stride, z_stride});
    return cudaGetLastError();
}

int64_t norm_workspace(const q8_block_norm& n, const q8_block_norm_grads& g)
{
    return n.tokens == 0 ? 0 : plan(n, g, sm_count()).bytes;
}

cudaError_t launch_norm_backward(const q8_block_norm& n, const q8_block_norm_grads& g, cudaStream_t st)
{
    const bool f32 = n.residual_dtype == Q8_F32;
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    if (e == cudaSuccess) e = earlier_fault(dev.fault);
    if (e != cudaSuccess) return e;
    const Plan p = plan(n, g, dev.sms);
    uint8_t* ws = static_cast<uint8_t*>(g.workspace);
    Backward a{};
    a.n = n;
    a.g = g;
    a.partial = reinterpret_cast<float*>(ws + p.partial);
    a.gate_partial = reinterpret_cast<float*>(ws + p.gate_partial);
    a.scratch = p.shared ? nullptr : reinterpret_cast<float*>(ws + p.scratch);
    a.wanted = p.wanted;
    for (int i = 0; i < kSums; ++i) a.at[i] = p.at[i];
    a.fault = dev.fault;
    const bool layer = n.post_kind == Q8_NORM_LAYER || n.pre_kind == Q8_NORM_LAYER;
    const BackwardKernel k = p.staged ? staged_kernel(f32, layer, p.threads) : backward_kernel(f32, p.vec, layer, n.dim);
    if ((e = prepare_norm()) != cudaSuccess) return e;
    k<<<static_cast<unsigned>(p.ctas), p.threads, static_cast<size_t>(p.smem), st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    SumArgs s{a.partial, a.gate_partial, {}, g.d_gate, p.ctas, n.dim, n.tokens, std::max<int64_t>(1, n.gate_tokens),
              ceil_div(n.dim, 32), 0};
    uint16_t* outs[kGate] = {g.d_post_weight, g.d_post_bias, g.d_pre_weight, g.d_pre_bias};
    for (uint16_t* o : outs)
        if (o) s.out[s.count++] = o;
    int64_t blocks = s.count * s.column_blocks;
    if (g.d_gate && p.ctas > 1 && n.gate_tokens > 1) {       // a group of one row has one CTA
        const int64_t groups = ceil_div(n.tokens, n.gate_tokens);
        blocks += groups < p.ctas ? groups * s.column_blocks : p.ctas - 1;
    }
    if (blocks) norm_sum_kernel<<<static_cast<unsigned>(blocks), dim3(32, 16), 0, st>>>(s);
    return cudaGetLastError();
}

}  // namespace q8
