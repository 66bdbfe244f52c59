// q8_distill.cu -- distillation from a teacher's top logits
// (include/q8train.h), forward and backward.
//
// The row kernel reads a row of logits from memory once.  A cluster of 1, 2, 4
// or 8 CTAs shares a row; each keeps its slice in shared memory.  Pass 1 runs
// over the slice as its chunks arrive, with a running maximum and the sums of
// exp relative to it (one for each of the two temperatures, 1 and tau, that the
// terms need); the cluster's CTAs exchange maximum and sums; pass 2 makes the
// gradient from shared memory and gives each chunk back, which the next row's
// load then fills.  One further warp of each CTA issues the loads (untiled bulk
// copies) and prepares the next row's teacher: ids, log p_k, the logits at the
// ids.  So loads, pass 1, pass 2's stores and the teacher's latencies overlap.
// The gradient is q scaled for every element; the K entries and the label
// differ from it by their own terms and are written once more after pass 2.
//
// Vocabularies too wide for eight CTAs' shared memory take wide_kernel, which
// reads the row again for each pass.
#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "q8_internal.h"
#include "q8_tc.cuh"
#include "q8_train.h"

namespace q8 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ float load(const T* p, int64_t i);
template <>
__device__ __forceinline__ float load<float>(const float* p, int64_t i) { return p[i]; }
template <>
__device__ __forceinline__ float load<uint16_t>(const uint16_t* p, int64_t i) { return bf16_to_float(p[i]); }
__device__ __forceinline__ void store(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store(uint16_t* p, int64_t i, float v) { p[i] = float_to_bf16(v); }

// 16 bytes of a row: eight bf16 or four float.
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[8])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[4])
{
    v[0] = __uint_as_float(q.x);
    v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z);
    v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack(const float (&v)[8])
{
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack(const float (&v)[4])
{
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// ---------------------------------------------------------------- row kernel

// A row as bulk copies may move it: `head` elements up to the first 16-byte
// boundary, `vecs` whole 16-byte vectors, `tail` elements after them.
template <typename T>
struct RowSpan {
    static constexpr int kPer = 16 / sizeof(T);
    int head, tail, vecs;
    __device__ RowSpan(const T* p, int vocab)
    {
        head = min(vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / static_cast<int>(sizeof(T)));
        vecs = (vocab - head) / kPer;
        tail = vocab - head - vecs * kPer;
    }
};

constexpr int kMaxChunks = 16;
constexpr int kMaxCluster = 8;

struct RowArgs {
    q8_distill_topk d;
    float* loss;
    float* stats_out;
    const float* stats_in;           // backward alone: no pass 1
    void* grad;
    int64_t grad_stride;
    int32_t slice_vecs;              // 16-byte vectors of a slice at most
    int32_t* fault;
};

// The maximum, and the sums of 2^(c (x - max)) for c = log2(e) (s1) and
// log2(e) / tau (st); with one temperature only st is kept.  The difference is
// formed before it is scaled: logits near the type's lowest value would
// overflow c * max.
struct Softmax {
    float max, s1, st;
};

__device__ __forceinline__ float rescale(float from, float to, float c)
{
    return from == -INFINITY ? 0.0f : exp2_approx((from - to) * c);     // nothing but -inf (or NaN) so far
}

template <bool DUAL>
__device__ __forceinline__ void merge(Softmax& a, const Softmax& b, float c1, float ct)
{
    const float m = fmaxf(a.max, b.max);
    if (DUAL) a.s1 = a.s1 * rescale(a.max, m, c1) + b.s1 * rescale(b.max, m, c1);
    a.st = a.st * rescale(a.max, m, ct) + b.st * rescale(b.max, m, ct);
    a.max = m;
}

template <bool DUAL>
__device__ __forceinline__ void merge_lanes(Softmax& m, int lanes, float c1, float ct)
{
    for (int o = lanes / 2; o > 0; o >>= 1) {
        Softmax q{__shfl_xor_sync(0xFFFFFFFFu, m.max, o), 0.0f, __shfl_xor_sync(0xFFFFFFFFu, m.st, o)};
        if (DUAL) q.s1 = __shfl_xor_sync(0xFFFFFFFFu, m.s1, o);
        merge<DUAL>(m, q, c1, ct);
    }
}

__device__ __forceinline__ float2 exp2_pair(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// With one temperature (DUAL false) c1 is not used and ct is the temperature of
// whatever terms there are.
template <typename T, bool GRAD, bool DUAL, int NT>
__global__ void __launch_bounds__(NT + 32, NT == 512 ? 2 : 8) row_kernel(const __grid_constant__ RowArgs args)
{
    using Span = RowSpan<T>;
    constexpr int kPer = Span::kPer;
    constexpr int kChunkVecs = 2 * NT;
    constexpr int kWarps = NT / 32;
    const q8_distill_topk& d = args.d;

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_full[kMaxChunks], s_empty[kMaxChunks], s_taught[2], s_used[2], s_xch[2];
    __shared__ Softmax s_part[2][kWarps];
    __shared__ Softmax s_peer[2][kMaxCluster];
    struct Teacher {
        float weight, label_z, lse1, lset;
        int label;                   // -1: no such term
        int taught;
    };
    __shared__ Teacher s_teacher[2];

    const int K = d.kd_weight > 0.0f ? static_cast<int>(d.k) : 0;
    const int K4 = (K + 3) & ~3;
    const int vocab = static_cast<int>(d.vocab);
    const uint4* buf = reinterpret_cast<const uint4*>(smem);
    float* s_logp = reinterpret_cast<float*>(smem + static_cast<size_t>(args.slice_vecs) * 16);     // [2][K4]
    float* s_z = s_logp + 2 * K4;                                                                   // [2][K4]
    int* s_id = reinterpret_cast<int*>(s_z + 2 * K4);                                               // [2][K4]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank, ranks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    const int64_t first_row = blockIdx.x / ranks, rows = gridDim.x / ranks;
    const float it = 1.0f / d.temperature;
    const bool kd = d.kd_weight > 0.0f;
    const float c1 = kLog2e, ct = DUAL || kd ? it * kLog2e : kLog2e;

    if (tid == 0) {
        for (int c = 0; c < kMaxChunks; ++c) {
            bar_init(smem_addr(&s_full[c]), 1);
            bar_init(smem_addr(&s_empty[c]), kWarps);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(smem_addr(&s_taught[b]), 1);
            bar_init(smem_addr(&s_used[b]), kWarps);
            bar_init(smem_addr(&s_xch[b]), ranks);
        }
        bar_init_fence();
    }
    __syncthreads();
    if (ranks > 1) cluster_sync();

    const auto row_of = [&](int64_t t) { return static_cast<const T*>(d.logits) + t * d.logits_stride; };
    // this CTA's vectors of the row
    const auto slice = [&](const Span& s, int* v0, int* v1) {
        *v0 = static_cast<int>(static_cast<int64_t>(s.vecs) * rank / ranks);
        *v1 = static_cast<int>(static_cast<int64_t>(s.vecs) * (rank + 1) / ranks);
    };
    // A wait that runs out makes every later one pass at once: the rows that are
    // left are walked through with whatever is in shared memory, so that all
    // barriers still meet and the kernel ends; the host hears of it.
    bool ok = true;
    const auto wait = [&](const uint64_t* bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait(smem_addr(bar), parity));
    };

    if (warp == kWarps) {
        // ------------------------------------------------ loads and the teacher
        uint32_t used_phase = 1;                     // a buffer's first wait passes
        uint32_t loads = 0, loaded = 0;              // bit c: the number of chunk c's loads, mod 2; whether there was one
        const auto load_row = [&](int64_t t) {
            const T* p = row_of(t);
            const Span s(p, vocab);
            int v0, v1;
            slice(s, &v0, &v1);
            const T* from = p + s.head + static_cast<int64_t>(v0) * kPer;
            for (int c = 0; c * kChunkVecs < v1 - v0; ++c) {
                wait(&s_empty[c], ((loads >> c) & 1) ^ 1);
                if (!ok) return;
                loads ^= 1u << c;
                loaded |= 1u << c;
                if (lane == 0) {
                    const uint32_t bytes = static_cast<uint32_t>(min(kChunkVecs, v1 - v0 - c * kChunkVecs)) * 16;
                    bar_expect(smem_addr(&s_full[c]), bytes);
                    bulk_load(smem_addr(smem) + c * kChunkVecs * 16, from + static_cast<int64_t>(c) * kChunkVecs * kPer, bytes,
                              smem_addr(&s_full[c]));
                }
                __syncwarp();
            }
        };
        const auto teach_row = [&](int64_t t, int b) {
            wait(&s_used[b], used_phase);
            const T* p = row_of(t);
            float *logp = s_logp + b * K4, *z = s_z + b * K4;
            int* ids = s_id + b * K4;
            float top = -INFINITY;
            for (int k = lane; k < K4; k += 32) {
                const int64_t id = k < K ? d.teacher_ids[t * K + k] : -1;
                const bool in = id >= 0 && id < vocab;
                ids[k] = in ? static_cast<int>(id) : -1;
                logp[k] = in ? d.teacher_logits[t * K + k] * it : -INFINITY;
                z[k] = in ? load(p, id) : 0.0f;
                top = fmaxf(top, logp[k]);
            }
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const bool taught = top > -INFINITY;
            float sum = 0.0f;
            if (taught)
                for (int k = lane; k < K; k += 32) sum += expf(logp[k] - top);
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (taught) {
                const float logsum = logf(sum);
                for (int k = lane; k < K; k += 32) logp[k] = (logp[k] - top) - logsum;
            }
            if (lane == 0) {
                Teacher& r = s_teacher[b];
                const int64_t label = d.labels && d.ce_weight > 0.0f ? d.labels[t] : -1;
                r.label = label >= 0 && label < vocab ? static_cast<int>(label) : -1;
                r.label_z = r.label >= 0 ? load(p, r.label) : 0.0f;
                r.weight = d.row_weight ? d.row_weight[t] : 1.0f;
                r.taught = taught;
                r.lse1 = args.stats_in ? args.stats_in[2 * t] : 0.0f;
                r.lset = args.stats_in ? args.stats_in[2 * t + 1] : 0.0f;
            }
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&s_taught[b]));
        };
        int64_t t = first_row;
        int b = 0;
        load_row(t);                                 // the grid has no more clusters than rows
        teach_row(t, b);
        while (t + rows < d.rows) {
            t += rows;
            if ((b ^= 1) == 0) used_phase ^= 1;
            teach_row(t, b);
            load_row(t);
        }
        // no copy may be in flight when the CTA ends: each was waited for by the
        // threads that read it, or, where those gave up, is now
        for (int c = 0; c < kMaxChunks; ++c)
            if (!ok && (loaded >> c) & 1) bar_wait(smem_addr(&s_full[c]), ((loads >> c) & 1) ^ 1);
    } else {
        // ------------------------------------------------------ pass 1, pass 2
        int turn = 0;
        uint32_t full_phase = 0;                     // bit c: the parity of chunk c's next wait
        for (int64_t t = first_row; t < d.rows; t += rows, ++turn) {
            const int b = turn & 1;
            const uint32_t pair_phase = (turn >> 1) & 1;
            const T* p = row_of(t);
            const Span s(p, vocab);
            int v0, v1;
            slice(s, &v0, &v1);
            // the elements before and after the vectors: one to a thread
            int edge = -1;
            if (rank == 0 && tid < s.head) edge = tid;
            if (rank == ranks - 1 && tid >= 8 && tid - 8 < s.tail) edge = vocab - s.tail + tid - 8;
            const float edge_z = edge >= 0 ? load(p, edge) : 0.0f;

            Softmax m{-INFINITY, 0.0f, 0.0f};
            if (!args.stats_in) {
                if (edge >= 0 && edge_z != -INFINITY) {
                    const float one = edge_z - edge_z + 1.0f;       // NaN where it is not finite
                    m = Softmax{edge_z, one, one};
                }
                for (int c = 0; c * kChunkVecs < v1 - v0; ++c) {
                    wait(&s_full[c], (full_phase >> c) & 1);
                    const int n = v1 - v0 - c * kChunkVecs;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int at = i * NT + tid;
                        if (at >= n) continue;
                        float v[kPer];
                        unpack(buf[c * kChunkVecs + at], v);
                        float top = v[0];
#pragma unroll
                        for (int j = 1; j < kPer; ++j) top = fmaxf(top, v[j]);
                        if (top > m.max) {
                            if (DUAL) m.s1 *= rescale(m.max, top, c1);
                            m.st *= rescale(m.max, top, ct);
                            m.max = top;
                        }
                        const float2 less = both(m.max == -INFINITY ? 0.0f : -m.max);
                        float2 a1 = both(0.0f), at2 = both(0.0f);
#pragma unroll
                        for (int j = 0; j < kPer; j += 2) {
                            const float2 x = __fadd2_rn(make_float2(v[j], v[j + 1]), less);
                            if (DUAL) a1 = __fadd2_rn(a1, exp2_pair(__fmul2_rn(x, both(c1))));
                            at2 = __fadd2_rn(at2, exp2_pair(__fmul2_rn(x, both(ct))));
                        }
                        m.s1 += a1.x + a1.y;
                        m.st += at2.x + at2.y;
                    }
                    if (!GRAD) {
                        full_phase ^= 1u << c;
                        __syncwarp();
                        if (lane == 0) bar_arrive(smem_addr(&s_empty[c]));
                    }
                }
                merge_lanes<DUAL>(m, 32, c1, ct);
                if (lane == 0) s_part[b][warp] = m;
                asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
                m = lane < kWarps ? s_part[b][lane] : Softmax{-INFINITY, 0.0f, 0.0f};
                merge_lanes<DUAL>(m, 32, c1, ct);
                if (ranks > 1) {
                    // to every CTA of the cluster; a buffer is written again two
                    // rows on, after all have read it
                    if (tid < static_cast<int>(ranks)) {
                        const uint32_t to = peer_addr(smem_addr(&s_peer[b][rank]), tid);
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(m.max) : "memory");
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(m.s1) : "memory");
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(m.st) : "memory");
                        bar_arrive_cluster(peer_addr(smem_addr(&s_xch[b]), tid));
                    }
                    __syncwarp();
                    wait(&s_xch[b], pair_phase);
                    m = lane < static_cast<int>(ranks) ? s_peer[b][lane] : Softmax{-INFINITY, 0.0f, 0.0f};
                    merge_lanes<DUAL>(m, 32, c1, ct);
                }
                if (m.max == -INFINITY) m.s1 = m.st = NAN;       // a row of -inf
            }
            wait(&s_taught[b], pair_phase);
            const Teacher r = s_teacher[b];
            const float *logp = s_logp + b * K4, *z = s_z + b * K4;
            const int* ids = s_id + b * K4;
            if (!DUAL) m.s1 = m.st;

            if (args.loss && rank == 0 && warp == 0) {
                // log q_id = z/tau - lse: relative to the maximum, where both are small
                const float ls1 = logf(m.s1), lst = logf(m.st);
                float part = 0.0f;
                if (r.taught)
                    for (int k = lane; k < K; k += 32) {
                        const float l = logp[k];
                        if (l > -INFINITY) part += expf(l) * (l - ((z[k] - m.max) * it - lst));
                    }
                for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
                if (lane == 0) {
                    args.loss[t] = (r.taught ? d.kd_weight * d.temperature * d.temperature * part : 0.0f) +
                                   (r.label >= 0 ? d.ce_weight * (ls1 + (m.max - r.label_z)) : 0.0f);
                    if (args.stats_out) {
                        args.stats_out[2 * t] = d.ce_weight > 0.0f ? m.max + ls1 : 0.0f;
                        args.stats_out[2 * t + 1] = kd ? m.max * it + lst : 0.0f;
                    }
                }
            }

            if (GRAD) {
                // gradient of an element: ft 2^((x at + bt) gt) + f1 2^((x + b1) c1)
                float ft = r.taught ? r.weight * d.kd_weight * d.temperature : 0.0f;
                float f1 = r.label >= 0 ? r.weight * d.ce_weight : 0.0f;
                const float own_t = ft, own_1 = f1;               // the entries' and the label's own factors
                float at = 1.0f, bt = -m.max, gt = ct, b1 = -m.max;
                if (args.stats_in) {
                    at = kd ? it : 1.0f;
                    bt = kd ? -r.lset : -r.lse1;
                    gt = kLog2e;
                    b1 = -r.lse1;
                } else {
                    ft = ft == 0.0f ? 0.0f : ft / m.st;
                    f1 = f1 == 0.0f ? 0.0f : f1 / m.s1;
                }
                if (!DUAL) ft += f1;
                const bool zero = ft == 0.0f && (!DUAL || f1 == 0.0f);    // 0 whatever the logits are
                const auto slope2 = [&](float2 x) {
                    if (zero) return both(0.0f);
                    float2 g = __fmul2_rn(both(ft), exp2_pair(__fmul2_rn(__ffma2_rn(x, both(at), both(bt)), both(gt))));
                    if (DUAL) g = __ffma2_rn(both(f1), exp2_pair(__fmul2_rn(__fadd2_rn(x, both(b1)), both(c1))), g);
                    return g;
                };
                const auto slope = [&](float x) { return slope2(both(x)).x; };
                T* out = static_cast<T*>(args.grad) + t * args.grad_stride;
                T* body = out + s.head + static_cast<int64_t>(v0) * kPer;
                const bool whole = (reinterpret_cast<uintptr_t>(body) & 15) == 0;
                for (int c = 0; c * kChunkVecs < v1 - v0; ++c) {
                    if (args.stats_in) wait(&s_full[c], (full_phase >> c) & 1);
                    full_phase ^= 1u << c;
                    const int n = v1 - v0 - c * kChunkVecs;
                    uint4 q[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (i * NT + tid < n) q[i] = buf[c * kChunkVecs + i * NT + tid];
                    __syncwarp();
                    if (lane == 0) bar_arrive(smem_addr(&s_empty[c]));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int to = c * kChunkVecs + i * NT + tid;
                        if (i * NT + tid >= n) continue;
                        float v[kPer];
                        unpack(q[i], v);
#pragma unroll
                        for (int j = 0; j < kPer; j += 2) {
                            const float2 g = slope2(make_float2(v[j], v[j + 1]));
                            v[j] = g.x;
                            v[j + 1] = g.y;
                        }
                        if (whole) {
                            __stcs(reinterpret_cast<uint4*>(body) + to, pack(v));
                        } else {
#pragma unroll
                            for (int j = 0; j < kPer; ++j) store(body, static_cast<int64_t>(to) * kPer + j, v[j]);
                        }
                    }
                }
                if (edge >= 0) store(out, edge, slope(edge_z));
                asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
                // the entries' own terms, once for each id, and the label's
                const int lo = rank == 0 ? 0 : s.head + v0 * kPer, hi = rank == ranks - 1 ? vocab : s.head + v1 * kPer;
                if (r.taught)
                    for (int k = tid; k < K; k += NT) {
                        const int id = ids[k];
                        if (id < lo || id >= hi) continue;
                        bool first = true;
                        float pk = 0.0f;
                        for (int i = 0; i < K4; i += 4) {
                            const int4 w = *reinterpret_cast<const int4*>(ids + i);
                            if (w.x == id) { first = first && i >= k; pk += expf(logp[i]); }
                            if (w.y == id) { first = first && i + 1 >= k; pk += expf(logp[i + 1]); }
                            if (w.z == id) { first = first && i + 2 >= k; pk += expf(logp[i + 2]); }
                            if (w.w == id) { first = first && i + 3 >= k; pk += expf(logp[i + 3]); }
                        }
                        if (first) store(out, id, slope(z[k]) - own_t * pk - (id == r.label ? own_1 : 0.0f));
                    }
                if (tid == 0 && r.label >= lo && r.label < hi) {
                    bool entry = false;
                    if (r.taught)
                        for (int i = 0; i < K; ++i) entry = entry || ids[i] == r.label;
                    if (!entry) store(out, r.label, slope(r.label_z) - own_1);
                }
            }
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&s_used[b]));
        }
    }
    if (!ok) atomicExch_system(args.fault, 1);
    __syncwarp();
    if (ranks > 1) cluster_sync();                   // no CTA ends while another may still write to it
}

// ---------------------------------------------------------------- wide kernel

constexpr int kWideThreads = 512;

template <bool MAX>
__device__ float cta_reduce(float v)
{
    __shared__ float part[kWideThreads / 32];
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
    for (int i = 1; i < kWideThreads / 32; ++i) v = MAX ? fmaxf(v, part[i]) : v + part[i];
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads) wide_kernel(const q8_distill_topk d, float* loss, float* stats_out,
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
        for (int k = threadIdx.x; k < K; k += kWideThreads) {
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
        for (int k = threadIdx.x; k < K; k += kWideThreads) sum += taught ? expf(s_p[k] - top) : 0.0f;
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
            for (int64_t j = threadIdx.x; j < d.vocab; j += kWideThreads) m = fmaxf(m, load(z, j));
            m = cta_reduce<true>(m);
            float a = 0.0f, b = 0.0f;
            for (int64_t j = threadIdx.x; j < d.vocab; j += kWideThreads) {
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
        for (int k = threadIdx.x; k < K; k += kWideThreads) {
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
        for (int64_t j = threadIdx.x; j < d.vocab; j += kWideThreads) store(out, j, base(load(z, j)));
        __syncthreads();
        // the entries' own terms, once for each id, and the label's
        for (int k = threadIdx.x; k < K; k += kWideThreads) {
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

// ------------------------------------------------------------------------- host

// A row's slices: the fewest CTAs whose share of the row leaves room for two
// CTAs on an SM (113 KB each with 1 KB kept by the system), else for one (226).
constexpr int64_t kShared2 = 113 * 1024, kShared1 = 226 * 1024, kStatic = 2 * 1024;

struct Config {
    int ctas = 0, threads = 0;       // CTAs to a row (0: the wide kernel), threads of the passes
    int slice_vecs = 0;
    size_t smem = 0;
};

Config configure(const q8_distill_topk& d, int sms)
{
    const int64_t elem = d.logits_dtype == Q8_F32 ? 4 : 2;
    const int64_t vecs = d.vocab * elem / 16;
    const int64_t teacher = 24 * ((d.k + 3) & ~int64_t(3));
    Config c;
    for (int64_t room : {kShared2, kShared1}) {
        for (int n = 1; n <= kMaxCluster && !c.ctas; n *= 2)
            if ((vecs + n - 1) / n * 16 + teacher + kStatic <= room && (vecs + n - 1) / n <= int64_t(kMaxChunks) * 1024) c.ctas = n;
        if (c.ctas) break;
    }
    if (!c.ctas) return c;
    // few rows: more CTAs to each, while a slice stays at least 8 KB
    while (c.ctas < kMaxCluster && d.rows * c.ctas * 2 <= sms && vecs / (2 * c.ctas) >= 512) c.ctas *= 2;
    c.slice_vecs = static_cast<int>((vecs + c.ctas - 1) / c.ctas);
    c.threads = c.slice_vecs <= 1024 ? 128 : 512;
    c.smem = static_cast<size_t>(c.slice_vecs) * 16 + static_cast<size_t>(teacher);
    return c;
}

cudaError_t allow_shared(const void* kernel)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kShared1 - kStatic));
}

// Clusters of `ctas` that run at once, cached by kernel, device and shape.
std::mutex g_lock;
std::map<std::tuple<const void*, int, int, size_t>, int> g_clusters;

cudaError_t clusters_at_once(const void* kernel, const cudaLaunchConfig_t& cfg, int ctas, int* out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const auto key = std::make_tuple(kernel, dev, ctas, cfg.dynamicSmemBytes);
    std::lock_guard<std::mutex> lock(g_lock);
    const auto at = g_clusters.find(key);
    if (at != g_clusters.end()) {
        *out = at->second;
        return cudaSuccess;
    }
    int n = 0;
    if ((e = allow_shared(kernel)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
    if (n <= 0) return cudaErrorInvalidConfiguration;
    g_clusters.emplace(key, n);
    *out = n;
    return cudaSuccess;
}

using RowKernel = void (*)(RowArgs);

template <typename T, int NT>
RowKernel row_kernel_of(bool grad, bool dual)
{
    return grad ? (dual ? row_kernel<T, true, true, NT> : row_kernel<T, true, false, NT>)
                : (dual ? row_kernel<T, false, true, NT> : row_kernel<T, false, false, NT>);
}

template <typename T>
RowKernel row_kernel_of(bool grad, bool dual, int threads)
{
    return threads == 128 ? row_kernel_of<T, 128>(grad, dual) : row_kernel_of<T, 512>(grad, dual);
}

template <typename T>
cudaError_t launch_wide(const q8_distill_topk& d, float* loss, float* stats_out, const float* stats_in, void* grad,
                        int64_t grad_stride, cudaStream_t st)
{
    int grid = 0;
    const cudaError_t e = persistent_grid(reinterpret_cast<const void*>(wide_kernel<T>), kWideThreads, 0, &grid);
    if (e != cudaSuccess) return e;
    wide_kernel<T><<<static_cast<unsigned>(std::min<int64_t>(d.rows, grid)), kWideThreads, 0, st>>>(
        d, loss, stats_out, stats_in, static_cast<T*>(grad), grad_stride);
    return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_distill()
{
    cudaError_t e = cudaSuccess;
    for (bool f32 : {false, true})
        for (bool grad : {false, true})
            for (bool dual : {false, true})
                for (int threads : {128, 512}) {
                    const RowKernel k = f32 ? row_kernel_of<float>(grad, dual, threads) : row_kernel_of<uint16_t>(grad, dual, threads);
                    if (e == cudaSuccess) e = allow_shared(reinterpret_cast<const void*>(k));
                }
    int g = 0;
    DeviceInfo dev;
    if (e == cudaSuccess) e = persistent_grid(reinterpret_cast<const void*>(wide_kernel<uint16_t>), kWideThreads, 0, &g);
    if (e == cudaSuccess) e = persistent_grid(reinterpret_cast<const void*>(wide_kernel<float>), kWideThreads, 0, &g);
    if (e == cudaSuccess) e = device_info(&dev);
    return e;
}

cudaError_t launch_distill(const q8_distill_topk& d, float* loss, float* stats_out, const float* stats_in,
                           void* dlogits, int64_t dlogits_stride, cudaStream_t st)
{
    static_assert(kMaxCluster == 8, "portable cluster size");
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    if (e == cudaSuccess) e = earlier_fault(dev.fault);
    if (e != cudaSuccess) return e;
    const Config c = configure(d, dev.sms);
    const bool f32 = d.logits_dtype == Q8_F32;
    if (!c.ctas)
        return f32 ? launch_wide<float>(d, loss, stats_out, stats_in, dlogits, dlogits_stride, st)
                   : launch_wide<uint16_t>(d, loss, stats_out, stats_in, dlogits, dlogits_stride, st);
    const bool dual = d.kd_weight > 0.0f && d.ce_weight > 0.0f && d.temperature != 1.0f;
    const RowKernel k = f32 ? row_kernel_of<float>(dlogits != nullptr, dual, c.threads)
                            : row_kernel_of<uint16_t>(dlogits != nullptr, dual, c.threads);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(c.ctas), 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(static_cast<unsigned>(c.threads + 32));
    cfg.gridDim = dim3(static_cast<unsigned>(c.ctas));
    cfg.dynamicSmemBytes = c.smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int at_once = 0;
    if ((e = clusters_at_once(reinterpret_cast<const void*>(k), cfg, c.ctas, &at_once)) != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(c.ctas * std::min<int64_t>(d.rows, at_once)));
    RowArgs a{};
    a.d = d;
    a.loss = loss;
    a.stats_out = stats_out;
    a.stats_in = stats_in;
    a.grad = dlogits;
    a.grad_stride = dlogits_stride;
    a.slice_vecs = c.slice_vecs;
    a.fault = dev.fault;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace q8
