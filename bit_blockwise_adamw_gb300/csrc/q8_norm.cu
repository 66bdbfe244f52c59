// q8_norm.cu -- the norms around a block's gate and residual
// (include/q8train.h), forward and backward.
//
// Both kernels give a row to a CTA of dim / E threads, E elements of fixed
// columns to each, and walk over rows; the next row's loads are in flight while
// a row is worked on, and several CTAs on an SM cover each other's reductions.
// A row is read once: its statistics come from registers (a layer norm's
// variance from the deviations, not from a difference of sums).  Bytes bound
// both: forward 8, backward 12 bytes an element in bf16.
//
// The backward kernel recomputes both norms from r and y and sums the weights'
// gradients over its rows, in shared memory (each column has one thread, so
// nothing is shared in fact; registers would leave room for half the CTAs).
// A CTA's rows are consecutive, so that a gate's group ends inside a CTA (and
// is written there) or is one of the two that reach over its ends.  norm_sum
// and gate_sum add up the CTAs' sums, in their order.
#include <algorithm>

#include "q8_internal.h"
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
    const float rs = 1.0f / sqrtf(fmaf(q[0], inv_dim, eps));
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

// Rows [first, stop) of CTA c of `ctas`.
__host__ __device__ __forceinline__ int64_t first_row(int64_t tokens, int64_t c, int64_t ctas)
{
    return tokens / ctas * c + tokens % ctas * c / ctas;
}

// Where the thread keeps the sums of its columns: in shared memory, four
// columns to an access with VEC 8.
template <int VEC, int E>
__device__ __forceinline__ void accumulate(float* sums, int dim, const float (&v)[E])
{
    if constexpr (VEC == 8) {
#pragma unroll
        for (int i = 0; i < E; i += 4)
            if (inside<8>(i, dim)) {
                // halves of a chunk apart: consecutive threads on consecutive 16 bytes
                float4* p = reinterpret_cast<float4*>(sums) + ((i / 4) * blockDim.x + threadIdx.x);
                float4 s = *p;
                s.x += v[i];
                s.y += v[i + 1];
                s.z += v[i + 2];
                s.w += v[i + 3];
                *p = s;
            }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (inside<1>(i, dim)) sums[i * blockDim.x + threadIdx.x] += v[i];
    }
}

// The thread's columns of the sums, which are set to zero, into a row of dim.
template <int VEC, int E, typename Out>
__device__ __forceinline__ void flush(float* sums, int dim, Out* row)
{
    float v[E];
    if constexpr (VEC == 8) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            float4* p = reinterpret_cast<float4*>(sums) + ((i / 4) * blockDim.x + threadIdx.x);
            const float4 s = *p;
            v[i] = s.x;
            v[i + 1] = s.y;
            v[i + 2] = s.z;
            v[i + 3] = s.w;
            *p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            v[i] = sums[i * blockDim.x + threadIdx.x];
            sums[i * blockDim.x + threadIdx.x] = 0.0f;
        }
    }
    if constexpr (sizeof(Out) == 2 && VEC == 8) {
        // a gate's gradient may lie on any address
        if ((reinterpret_cast<uintptr_t>(row) & 15) != 0) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (inside<8>(i, dim)) row[((i / 8) * blockDim.x + threadIdx.x) * 8 + (i & 7)] = float_to_bf16(v[i]);
            return;
        }
    }
    put<VEC>(row, dim, v);
}

template <typename R, int VEC, int E, int MAXT, int CTAS>
__global__ void __launch_bounds__(MAXT, CTAS) norm_backward_kernel(const __grid_constant__ Backward a)
{
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
    int64_t group_end = n.gate ? (group + 1) * n.gate_tokens : n.tokens;      // tokens * 2 at most: no overflow
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

    Raw<uint16_t, VEC, E> y_next, dz_next;
    Raw<R, VEC, E> r_next, dr_next;
    const auto load = [&](int64_t t) {
        y_next.load(n.y + t * n.y_stride, dim);
        r_next.load(residual + t * n.residual_stride, dim);
        if (g.dz) dz_next.load(g.dz + t * g.dz_stride, dim);
        if (dr_out) dr_next.load(dr_out + t * g.d_residual_out_stride, dim);
    };
    load(first);
    for (int64_t t = first; t < stop; ++t) {
        if (t == group_end) {
            flush_gate(t);
            ++group;
            group_end += n.gate_tokens;
        }
        float yn[E], rn[E], dz[E], d[E], w[E], gate[E];
        y_next.get(yn);
        r_next.get(rn);
#pragma unroll
        for (int i = 0; i < E; ++i) dz[i] = d[i] = 0.0f;
        if (g.dz) dz_next.get(dz);
        if (dr_out) dr_next.get(d);
        if (t + 1 < stop) load(t + 1);

        // both norms again
        const float y_rs = normalise<VEC>(yn, dim, inv_dim, n.post_kind, n.eps, red);
        channels<VEC>(n.gate ? n.gate + group * n.dim : nullptr, dim, 1.0f, gate);
        channels<VEC>(n.post_weight, dim, 1.0f, w);
        if (n.post_bias) {
            float bias[E];
            channels<VEC>(n.post_bias, dim, 0.0f, bias);
#pragma unroll
            for (int i = 0; i < E; ++i) rn[i] = fmaf(n.residual_scale, rn[i], gate[i] * fmaf(yn[i], w[i], bias[i]));
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) rn[i] = fmaf(n.residual_scale, rn[i], gate[i] * (yn[i] * w[i]));
        }
        const float r_rs = normalise<VEC>(rn, dim, inv_dim, n.pre_kind, n.eps, red);

        // d: the gradient of r'
        if (g.dz) {
            if (a.at[kPreBias] >= 0) accumulate<VEC>(sum_of(kPreBias), dim, dz);
            if (a.at[kPreWeight] >= 0) {
                float p[E];
#pragma unroll
                for (int i = 0; i < E; ++i) p[i] = dz[i] * rn[i];
                accumulate<VEC>(sum_of(kPreWeight), dim, p);
            }
            if (n.pre_weight) {
                float pw[E];
                channels<VEC>(n.pre_weight, dim, 1.0f, pw);
#pragma unroll
                for (int i = 0; i < E; ++i) dz[i] *= pw[i];
            }
            if (n.pre_kind != Q8_NORM_NONE) {
                float s[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    s[0] = fmaf(dz[i], rn[i], s[0]);
                    s[1] += dz[i];
                }
                red.sum(s);
                const float dot = s[0] * inv_dim, mean = n.pre_kind == Q8_NORM_LAYER ? s[1] * inv_dim : 0.0f;
#pragma unroll
                for (int i = 0; i < E; ++i) d[i] = fmaf(r_rs, fmaf(-rn[i], dot, dz[i] - mean), d[i]);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) d[i] += dz[i];
            }
        }
        if (dr) {
#pragma unroll
            for (int i = 0; i < E; ++i) dz[i] = n.residual_scale * d[i];
            put<VEC>(dr + t * g.d_residual_stride, dim, dz);
        }
        if (a.at[kGate] >= 0) {
            if (n.post_bias) {
                channels<VEC>(n.post_bias, dim, 0.0f, dz);
#pragma unroll
                for (int i = 0; i < E; ++i) dz[i] = d[i] * fmaf(yn[i], w[i], dz[i]);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) dz[i] = d[i] * (yn[i] * w[i]);
            }
            accumulate<VEC>(sum_of(kGate), dim, dz);
        }
        // d: the gradient of N_post(y), then of the normalised y
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] *= gate[i];
        if (a.at[kPostBias] >= 0) accumulate<VEC>(sum_of(kPostBias), dim, d);
        if (a.at[kPostWeight] >= 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) dz[i] = d[i] * yn[i];
            accumulate<VEC>(sum_of(kPostWeight), dim, dz);
        }
        if (!g.d_y) continue;
        if (n.post_kind != Q8_NORM_NONE) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < E; ++i) {
                d[i] *= w[i];
                s[0] = fmaf(d[i], yn[i], s[0]);
                s[1] += inside<VEC>(i, dim) ? d[i] : 0.0f;
            }
            red.sum(s);
            const float dot = s[0] * inv_dim, mean = n.post_kind == Q8_NORM_LAYER ? s[1] * inv_dim : 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) d[i] = y_rs * fmaf(-yn[i], dot, d[i] - mean);
        }
        put<VEC>(g.d_y + t * g.d_y_stride, dim, d);
    }
    if (first < stop) flush_gate(stop);
    for (int which = 0; which < kGate; ++which)
        if (a.at[which] >= 0)
            flush<VEC, E>(sum_of(which), dim, a.partial + (static_cast<int64_t>(a.at[which]) * gridDim.x + blockIdx.x) * n.dim);
}

// Columns of the CTAs' sums: 32 columns to a block, its 16 warps take every
// 16th row, and their sums are added in order.
struct SumArgs {
    const float* partial;
    uint16_t* out[kGate];
    int64_t rows, dim;
};

__device__ __forceinline__ void sum_columns(float s, int64_t col, int64_t dim, uint16_t* out)
{
    __shared__ float part[16][33];
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < dim) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += part[i][threadIdx.x];
        out[col] = float_to_bf16(s);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(512) norm_sum_kernel(const __grid_constant__ SumArgs a)
{
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    const float* p = a.partial + blockIdx.y * a.rows * a.dim + col;
    float s = 0.0f;
    if (col < a.dim) {
#pragma unroll 4
        for (int64_t r = threadIdx.y; r < a.rows; r += 16) s += p[r * a.dim];
    }
    sum_columns(s, col, a.dim, a.out[blockIdx.y]);
}

// The gradient of the gate of each group that more than one CTA has rows of: the
// y index runs over the groups, or, where these are more, over the CTAs' ends.
__global__ void __launch_bounds__(512) gate_sum_kernel(const float* partial, int64_t tokens, int64_t gate_tokens, int64_t ctas,
                                                       int64_t dim, uint16_t* out)
{
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    const int64_t groups = (tokens + gate_tokens - 1) / gate_tokens;
    int64_t begin, cta;                              // the group's first row, and the CTA that has it
    if (groups < ctas) {
        begin = blockIdx.y * gate_tokens;
        cta = begin * ctas / tokens;                 // or one beside it
        while (cta + 1 < ctas && first_row(tokens, cta + 1, ctas) <= begin) ++cta;
        while (first_row(tokens, cta, ctas) > begin) --cta;
    } else {
        cta = blockIdx.y;
        const int64_t next = first_row(tokens, cta + 1, ctas);
        begin = next / gate_tokens * gate_tokens;
        if (begin == next || begin < first_row(tokens, cta, ctas)) return;
    }
    const int64_t end = min(begin + gate_tokens, tokens);
    if (cta + 1 == ctas || first_row(tokens, cta + 1, ctas) >= end) return;     // written by the CTA itself
    float s = 0.0f;
    if (col < dim)
        for (int64_t c = cta + threadIdx.y; c < ctas && first_row(tokens, c, ctas) < end; c += 16)
            s += partial[(2 * c + (first_row(tokens, c, ctas) < begin)) * dim + col];
    sum_columns(s, col, dim, out + begin / gate_tokens * dim);
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

Shape backward_shape(int64_t dim)
{
    return dim <= 4096 ? Shape{8, 512} : dim <= 8192 ? Shape{16, 512} : dim <= 16384 ? Shape{16, 1024} : Shape{32, 1024};
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

template <typename R, int VEC>
BackwardKernel backward_kernel(int64_t dim)
{
    const Shape s = backward_shape(dim);
    if (s.elements == 8) return norm_backward_kernel<R, VEC, 8, 512, 2>;
    return s.most == 512 ? norm_backward_kernel<R, VEC, 16, 512, 1>
                         : s.elements == 16 ? norm_backward_kernel<R, VEC, 16, 1024, 1> : norm_backward_kernel<R, VEC, 32, 1024, 1>;
}

ForwardKernel forward_kernel(bool f32, bool vec, int64_t dim)
{
    if (f32) return vec ? forward_kernel<float, 8>(dim) : forward_kernel<float, 1>(dim);
    return vec ? forward_kernel<uint16_t, 8>(dim) : forward_kernel<uint16_t, 1>(dim);
}

BackwardKernel backward_kernel(bool f32, bool vec, int64_t dim)
{
    if (f32) return vec ? backward_kernel<float, 8>(dim) : backward_kernel<float, 1>(dim);
    return vec ? backward_kernel<uint16_t, 8>(dim) : backward_kernel<uint16_t, 1>(dim);
}

// CTAs of the backward kernel: a function of sizes alone, for the workspace is
// sized by it; as many as are resident where their sums lie in shared memory.
constexpr int64_t kSums227 = 227 * 1024 - 1024;

struct Plan {
    int64_t ctas, span;              // span: columns of a sum as the CTA keeps it
    int threads, wanted, at[kSums];
    bool shared;
    int64_t smem, partial, gate_partial, scratch, bytes;
};

Plan plan(const q8_block_norm& n, const q8_block_norm_grads& g, int sms)
{
    Plan p{};
    const Shape s = backward_shape(n.dim);
    p.threads = threads_of(n.dim, s.elements);
    p.span = static_cast<int64_t>(p.threads) * s.elements;
    const uint16_t* outs[kSums] = {g.d_post_weight, g.d_post_bias, g.d_pre_weight, g.d_pre_bias, g.d_gate};
    for (int i = 0; i < kSums; ++i) p.at[i] = outs[i] ? p.wanted++ : -1;
    p.smem = p.wanted * p.span * 4;
    p.shared = p.smem <= kSums227;
    const int64_t by_threads = std::max(1, (s.elements == 8 ? 1024 : s.most) / p.threads);
    const int64_t by_smem = p.shared && p.smem ? std::max<int64_t>(1, 227 * 1024 / (p.smem + 2048)) : by_threads;
    p.ctas = std::min<int64_t>(n.tokens, sms * std::min<int64_t>(16, std::min(by_threads, by_smem)));
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

cudaError_t prepare_norm()
{
    cudaError_t e = cudaSuccess;
    int grid = 0;
    for (bool f32 : {false, true})
        for (bool vec : {false, true})
            for (int64_t dim : {4096, 8192, 16384, 32768}) {
                const Shape s = forward_shape(dim);
                if (e == cudaSuccess)
                    e = persistent_grid(reinterpret_cast<const void*>(forward_kernel(f32, vec, dim)), s.most, 0, &grid);
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(backward_kernel(f32, vec, dim)),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSums227);
            }
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
    const int64_t elem = f32 ? 4 : 2;
    const bool vec = vectors(n) && on16(g.d_residual_out, g.d_residual_out ? g.d_residual_out_stride : 0, elem) &&
                     on16(g.dz, g.dz ? g.dz_stride : 0, 2) && on16(g.d_residual, g.d_residual ? g.d_residual_stride : 0, elem) &&
                     on16(g.d_y, g.d_y ? g.d_y_stride : 0, 2);
    const Plan p = plan(n, g, sm_count());
    uint8_t* ws = static_cast<uint8_t*>(g.workspace);
    Backward a{};
    a.n = n;
    a.g = g;
    a.partial = reinterpret_cast<float*>(ws + p.partial);
    a.gate_partial = reinterpret_cast<float*>(ws + p.gate_partial);
    a.scratch = p.shared ? nullptr : reinterpret_cast<float*>(ws + p.scratch);
    a.wanted = p.wanted;
    for (int i = 0; i < kSums; ++i) a.at[i] = p.at[i];
    const BackwardKernel k = backward_kernel(f32, vec, n.dim);
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize, kSums227);
    if (e != cudaSuccess) return e;
    k<<<static_cast<unsigned>(p.ctas), p.threads, p.shared ? static_cast<size_t>(p.smem) : 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const unsigned blocks = static_cast<unsigned>(ceil_div(n.dim, 32));
    SumArgs s{a.partial, {}, p.ctas, n.dim};
    uint16_t* outs[kGate] = {g.d_post_weight, g.d_post_bias, g.d_pre_weight, g.d_pre_bias};
    int count = 0;
    for (uint16_t* o : outs)
        if (o) s.out[count++] = o;
    if (count) norm_sum_kernel<<<dim3(blocks, count), dim3(32, 16), 0, st>>>(s);
    if (g.d_gate && p.ctas > 1) {
        // only groups that reach from one CTA into the next have anything to add
        const int64_t groups = ceil_div(n.tokens, n.gate_tokens);
        gate_sum_kernel<<<dim3(blocks, static_cast<unsigned>(groups < p.ctas ? groups : p.ctas - 1)), dim3(32, 16), 0, st>>>(
            a.gate_partial, n.tokens, n.gate_tokens, p.ctas, n.dim, g.d_gate);
    }
    return cudaGetLastError();
}

}  // namespace q8
