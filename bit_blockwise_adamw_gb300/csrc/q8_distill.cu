// q8_distill.cu -- distillation from a teacher's top logits
// (include/q8train.h), forward and backward.
//
// The row kernel reads a row of logits from memory once.  Its threads make two
// passes: pass 1 keeps a running maximum and the sums of exp relative to it
// (one for each of the two temperatures, 1 and tau, that the terms need); pass 2
// makes the gradient.  The row comes through a ring of chunks in shared memory,
// loaded by untiled bulk copies that one further warp issues; another prepares
// the rows' teacher: ids, log p_k, the logits at the ids.  A cluster of 1, 2, 4
// or 8 CTAs shares a row where it is wide or rows are few; the CTAs exchange
// their maximum and sums.
//   kForward   pass 1 alone; a chunk goes back to the loads once it is read.
//   kTrain     the row stays in the ring between the passes, and pass 1 of the
//              next row runs chunk by chunk beside pass 2 of this one: with the
//              passes apart, all CTAs come to store at the same time and to
//              leave memory idle at the same time (8192 x 50257 bf16, loss and
//              gradient at two temperatures: 424 us apart, 395 us together).
//   kStream    pass 2 alone, from the forward call's statistics; or, for rows
//              too wide for eight CTAs' shared memory, both passes with the row
//              loaded twice.
// The gradient is q scaled for every element; the K entries and the label
// differ from it by their own terms and are written once more after pass 2.
//
// Measured: forward, 4096 x 50257 bf16, 72 us, 5.7 TB/s (85 % of a copy's rate),
// near both memory's and instruction issue's limit.  Loss and gradient at two
// temperatures, 8192 x 50257 bf16, 396 us for 1.65 GB: 22 instructions an element,
// four exponentials among them, from 16 warps an SM, which are too few to cover
// their latencies (issue 60 %, special-function units 45 %, DRAM 47 %).  float32,
// 1001 x 128001, loss and then gradient, 272 us; the two calls read the logits
// twice, 228 us of bytes.
#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "q8_distill_plan.h"
#include "q8_internal.h"
#include "q8_tc.cuh"
#include "q8_train.h"

namespace q8 {

using namespace distill;

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

// 16 bytes of a row, eight bf16 or four float, as float.
__device__ __forceinline__ void unpack(const uint4& q, float* v, const uint16_t*)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& q, float* v, const float*)
{
    v[0] = __uint_as_float(q.x);
    v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z);
    v[3] = __uint_as_float(q.w);
}
// The largest of N vectors' elements (NaN aside).
template <int N>
__device__ __forceinline__ float largest(const uint4 (&q)[N], const uint16_t*)
{
    const auto pair = [](const uint32_t& w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    __nv_bfloat162 top = pair(q[0].x);
#pragma unroll
    for (int i = 0; i < N; ++i)
        top = __hmax2(top, __hmax2(__hmax2(pair(q[i].x), pair(q[i].y)), __hmax2(pair(q[i].z), pair(q[i].w))));
    const float2 t = __bfloat1622float2(top);
    return fmaxf(t.x, t.y);
}
template <int N>
__device__ __forceinline__ float largest(const uint4 (&q)[N], const float*)
{
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
        top = fmaxf(top, fmaxf(fmaxf(__uint_as_float(q[i].x), __uint_as_float(q[i].y)),
                               fmaxf(__uint_as_float(q[i].z), __uint_as_float(q[i].w))));
    return top;
}
// 16 bytes of -inf.
__device__ __forceinline__ uint4 infinities(const uint16_t*) { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
__device__ __forceinline__ uint4 infinities(const float*) { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack(const float* v, const uint16_t*)
{
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack(const float* v, const float*)
{
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// The elements of a packed vector, one by one.
__device__ __forceinline__ void scatter(uint16_t* p, const uint4& q)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ void scatter(float* p, const uint4& q)
{
    p[0] = __uint_as_float(q.x);
    p[1] = __uint_as_float(q.y);
    p[2] = __uint_as_float(q.z);
    p[3] = __uint_as_float(q.w);
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

constexpr int kDropped = 0x7FFFDEAD;  // marks, for a moment, an entry whose id an earlier one has (a NaN no conversion gives)

struct RowArgs {
    q8_distill_topk d;
    float* loss;
    float* stats_out;
    const float* stats_in;           // kStream: the backward call's; NULL: both passes
    void* grad;
    int64_t grad_stride;
    int32_t slots, chunk;            // of the ring; 16-byte vectors of each
    int32_t seen;                    // places of the table of a row's ids
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

// Over each group of `lanes` lanes; all groups hold the same, so the warp's
// maximum is theirs.
template <bool DUAL>
__device__ __forceinline__ void merge_lanes(Softmax& m, int lanes, float c1, float ct)
{
    float top;
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(top) : "f"(m.max));
    if (DUAL) m.s1 *= rescale(m.max, top, c1);
    m.st *= rescale(m.max, top, ct);
    for (int o = lanes / 2; o > 0; o >>= 1) {
        if (DUAL) m.s1 += __shfl_xor_sync(0xFFFFFFFFu, m.s1, o);
        m.st += __shfl_xor_sync(0xFFFFFFFFu, m.st, o);
    }
    m.max = top;
}

__device__ __forceinline__ float2 exp2_pair(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// With one temperature (DUAL false) c1 is not used and ct is the temperature of
// whatever terms there are.
template <typename T, int MODE, bool DUAL, int SHAPE>
__global__ void __launch_bounds__(threads_of(SHAPE) + kOwn, ctas_per_sm(SHAPE)) row_kernel(const __grid_constant__ RowArgs args)
{
    constexpr bool GRAD = MODE != kForward;
    using Span = RowSpan<T>;
    constexpr int kPer = Span::kPer;
    constexpr int NT = threads_of(SHAPE);
    constexpr int kVecs = chunk_vectors(SHAPE, sizeof(T));
    constexpr int kWarps = NT / 32;
    const q8_distill_topk& d = args.d;

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_full[kMaxSlots], s_empty[kMaxSlots], s_taught[kTeachers], s_used[kTeachers], s_xch[2];
    __shared__ Softmax s_part[2][kWarps];
    __shared__ Softmax s_peer[2][kMaxCluster];
    struct Teacher {
        float own_t, own_1;          // weight of the row's teacher and label terms in the gradient, 0: none
        float label_z, lse1, lset;
        int taught, labelled;
    };
    __shared__ Teacher s_teacher[kTeachers];

    const int K = d.kd_weight > 0.0f ? static_cast<int>(d.k) : 0;
    const int E = (K + 4) & ~3;                       // entries and the label's place (index K), as a multiple of four
    const int vocab = static_cast<int>(d.vocab);
    const uint4* buf = reinterpret_cast<const uint4*>(smem);
    float* s_logp = reinterpret_cast<float*>(smem + static_cast<size_t>(args.slots) * args.chunk * 16);     // [kTeachers][E] each
    float* s_z = s_logp + kTeachers * E;
    float* s_own = s_z + kTeachers * E;                       // the entry's own part of the gradient
    int* s_id = reinterpret_cast<int*>(s_own + kTeachers * E);
    float* s_raw_l = reinterpret_cast<float*>(s_id + kTeachers * E);            // [2][E] each: as they come
    int64_t* s_raw_id = reinterpret_cast<int64_t*>(s_raw_l + 2 * E);
    int* s_seen = reinterpret_cast<int*>(s_raw_id + 2 * E);                       // [args.seen], a power of two above 2 K: the ids of a row, hashed

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank, ranks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    const int64_t first_row = blockIdx.x / ranks, rows = gridDim.x / ranks;
    const float it = 1.0f / d.temperature;
    const bool kd = d.kd_weight > 0.0f;
    const float c1 = kLog2e, ct = DUAL || kd ? it * kLog2e : kLog2e;

    if (tid == 0) {
        for (int c = 0; c < kMaxSlots; ++c) {
            bar_init(smem_addr(&s_full[c]), 1);
            bar_init(smem_addr(&s_empty[c]), kWarps);
        }
        for (int b = 0; b < kTeachers; ++b) {
            bar_init(smem_addr(&s_taught[b]), 1);
            bar_init(smem_addr(&s_used[b]), kWarps);
        }
        for (int b = 0; b < 2; ++b) bar_init(smem_addr(&s_xch[b]), ranks);
        bar_init_fence();
    }
    __syncthreads();
    if (ranks > 1) cluster_sync();

    const auto row_of = [&](int64_t t) { return static_cast<const T*>(d.logits) + t * d.logits_stride; };
    // this CTA's vectors of the row (ranks is a power of two)
    const int shift = __ffs(ranks) - 1;
    const auto slice = [&](const Span& s, int* v0, int* v1) {
        const int share = (s.vecs + static_cast<int>(ranks) - 1) >> shift;
        *v0 = min(s.vecs, share * static_cast<int>(rank));
        *v1 = min(s.vecs, *v0 + share);
    };
    // A wait that runs out makes every later one pass at once: the rows that are
    // left are walked through with whatever is in shared memory, so that all
    // barriers still meet and the kernel ends; the host hears of it.
    bool ok = true;
    const int slots = args.slots, chunk = args.chunk;
    const auto wait = [&](const uint64_t* bar, uint32_t parity) {
        if (ok) ok = bar_wait(smem_addr(bar), parity);
    };

    if (warp == kWarps) {
        // ---------------------------------------------------------- the loads
        int slot = 0;
        uint32_t turn = 0;                           // how often the ring went round, mod 2
        for (int64_t t = first_row; t < d.rows && lane == 0; t += rows) {
            const T* p = row_of(t);
            const Span s(p, vocab);
            int v0, v1;
            slice(s, &v0, &v1);
            const int times = MODE == kStream && !args.stats_in ? 2 : 1;
            for (int i = 0; i < times && ok; ++i) {
                const T* from = p + s.head + static_cast<int64_t>(v0) * kPer;
                for (int left = v1 - v0; left > 0; left -= chunk) {
                    if (!(ok = bar_wait_idle(smem_addr(&s_empty[slot]), turn ^ 1))) break;
                    const uint32_t bytes = static_cast<uint32_t>(min(chunk, left)) * 16;
                    bar_expect(smem_addr(&s_full[slot]), bytes);
                    bulk_load(smem_addr(smem) + slot * chunk * 16, from, bytes, smem_addr(&s_full[slot]));
                    from += chunk * kPer;
                    if (++slot == slots) slot = 0, turn ^= 1;
                }
            }
            if (!ok) break;
        }
        // no copy may be in flight when the CTA ends: each was waited for by the
        // threads that read it, or, where those gave up, is now
        for (int c = 0; c < slots && !ok; ++c) bar_wait(smem_addr(&s_full[c]), c < slot ? turn : turn ^ 1);
    } else if (warp == kWarps + 1) {
        // --------------------------------------------------------- the teacher
        // A row's entries come from memory in two dependent steps (the ids, the
        // logits at the ids).  Ids and teacher logits are copied to shared memory
        // two rows before they are needed, the logits of the first kAhead * 32 of
        // them are read one row before and not looked at until then, so that
        // neither latency is waited for.
        constexpr int kAhead = 4;
        T zs[kAhead], label_zs;
        int64_t label_ahead = -1, label_next = -1;
        const auto inside = [&](int64_t id) { return id >= 0 && id < vocab; };
        const auto fetch = [&](int64_t t, int at) {
            if (t < d.rows)
                for (int k = lane; k < K; k += 32) {
                    copy_async<8>(smem_addr(s_raw_id + at * E + k), d.teacher_ids + t * K + k);
                    copy_async<4>(smem_addr(s_raw_l + at * E + k), d.teacher_logits + t * K + k);
                }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        const auto gather = [&](int64_t t, int at) {
            if (t >= d.rows) return;
            const T* p = row_of(t);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int k = lane + 32 * i;
                if (k < K && inside(s_raw_id[at * E + k])) zs[i] = p[s_raw_id[at * E + k]];
            }
            if (inside(label_next)) label_zs = p[label_next];
        };
        const auto label_of = [&](int64_t t) {
            return t < d.rows && d.labels && d.ce_weight > 0.0f ? d.labels[t] : -1;
        };
        const auto clear_seen = [&]() {
            for (int i = lane; i < args.seen; i += 32) s_seen[i] = -1;
            __syncwarp();
        };
        // whether the id was there before
        const auto see = [&](int id) {
            for (uint32_t place = static_cast<uint32_t>(id) * 2654435761u >> 8;; ++place) {
                const int was = atomicCAS(&s_seen[place & (args.seen - 1)], -1, id);
                if (was == -1) return false;
                if (was == id) return true;
            }
        };
        int b = 0, at = 0;                           // of the prepared rows, and of the copies
        uint32_t used_phase = 1;                     // a buffer's first wait passes
        fetch(first_row, 0);
        fetch(first_row + rows, 1);
        label_next = label_of(first_row);
        label_ahead = label_of(first_row + rows);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        gather(first_row, 0);
        if (GRAD) clear_seen();
        for (int64_t t = first_row; t < d.rows; t += rows) {
            const float weight = d.row_weight ? d.row_weight[t] : 1.0f;
            if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait_idle(smem_addr(&s_used[b]), used_phase));
            float *logp = s_logp + b * E, *z = s_z + b * E, *own = s_own + b * E;
            int* ids = s_id + b * E;
            float top = -INFINITY;
            for (int k = lane; k < K; k += 32) {
                const int64_t v = s_raw_id[at * E + k];
                const bool in = inside(v);
                const float l = in ? s_raw_l[at * E + k] * it : -INFINITY;
                ids[k] = in ? static_cast<int>(v) : -1;
                logp[k] = l;
                top = fmaxf(top, l);
                if (k >= 32 * kAhead) z[k] = in ? load(row_of(t), v) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int k = lane + 32 * i;
                if (k < K) z[k] = ids[k] >= 0 ? load(&zs[i], 0) : 0.0f;
            }
            const bool labelled = inside(label_next);
            const int label = labelled ? static_cast<int>(label_next) : -1;
            const float label_z = labelled ? load(&label_zs, 0) : 0.0f;
            label_next = label_ahead;
            label_ahead = label_of(t + 2 * rows);
            __syncwarp();
            fetch(t + 2 * rows, at);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            at ^= 1;
            gather(t + rows, at);
            asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(top) : "f"(top));
            const bool taught = top > -INFINITY;
            const float own_t = taught ? weight * d.kd_weight * d.temperature : 0.0f;
            const float own_1 = labelled ? weight * d.ce_weight : 0.0f;
            float logsum = 0.0f;
            if (taught) {
                float sum = 0.0f;
                for (int k = lane; k < K; k += 32) sum += exp2_approx((logp[k] - top) * kLog2e);
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                logsum = logf(sum);
            }
            // log p_k, and what the entry has of its own: own_t p_k, and the label's
            // part where it is the label; entries of no teacher are none
            bool again = false, entry = false;
            for (int k = lane; k < K; k += 32) {
                logp[k] = (logp[k] - top) - logsum;
                if (!GRAD) continue;
                if (!taught) ids[k] = -1;
                if (ids[k] >= 0) {
                    again = see(ids[k]) || again;
                    entry = entry || ids[k] == label;
                }
                own[k] = own_t * exp2_approx(logp[k] * kLog2e) + (ids[k] == label ? own_1 : 0.0f);
            }
            if (GRAD) {
                entry = __any_sync(0xFFFFFFFFu, entry);
                if (__any_sync(0xFFFFFFFFu, again)) {
                    // an id that appears twice: its first entry takes the sum of all,
                    // in their order, and the others are dropped
                    for (int k0 = 0; k0 < K; k0 += 32) {
                        const int k = k0 + lane, mine = k < K ? ids[k] : -1;
                        if (mine < 0) continue;
                        bool first = true;
                        float sum = mine == label ? own_1 : 0.0f;
                        for (int i = 0; i < K; ++i)
                            if (ids[i] == mine) {
                                first = first && i >= k;
                                sum += own_t * exp2_approx(logp[i] * kLog2e);
                            }
                        own[k] = sum;
                        z[k] = first ? z[k] : __int_as_float(kDropped);
                    }
                    __syncwarp();
                    for (int k = lane; k < K; k += 32)
                        if (__float_as_int(z[k]) == kDropped) ids[k] = -1, z[k] = load(row_of(t), d.teacher_ids[t * K + k]);
                }
                if (lane == 0) {
                    ids[K] = labelled && !entry ? label : -1;
                    z[K] = label_z;
                    own[K] = own_1;
                }
            }
            if (lane == 0) {
                Teacher& r = s_teacher[b];
                r.own_t = own_t;
                r.own_1 = own_1;
                r.label_z = label_z;
                r.taught = taught;
                r.labelled = labelled;
                r.lse1 = args.stats_in ? args.stats_in[2 * t] : 0.0f;
                r.lset = args.stats_in ? args.stats_in[2 * t + 1] : 0.0f;
            }
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&s_taught[b]));
            if (GRAD) clear_seen();
            if (++b == kTeachers) b = 0, used_phase ^= 1;
        }
    } else {
        // ------------------------------------------------------ pass 1, pass 2
        // A place in the ring, and the parity of its round.
        struct Place {
            int slot = 0;
            uint32_t phase = 0;
        };
        const auto step = [&](Place& at) {
            if (++at.slot == slots) at.slot = 0, at.phase ^= 1;
        };
        const auto await = [&](const Place& at) { wait(&s_full[at.slot], at.phase); };
        const auto give_back = [&](const Place& at) {
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&s_empty[at.slot]));
        };

        // The elements before and after a row's vectors go one to a thread; they
        // are read a row ahead.
        struct Edge {
            int at = -1;
            float z = 0.0f;
        };
        // A row's part here: n vectors from element `begin` on, elements [lo, hi)
        // with the edges, its gradient's row.
        struct Row {
            int n = 0, begin = 0, lo = 0, hi = 0;
            T* out = nullptr;
        };
        const auto part_of = [&](int64_t t) {
            Row r;
            const Span s(row_of(t), vocab);
            int v0, v1;
            slice(s, &v0, &v1);
            r.n = v1 - v0;
            r.begin = s.head + v0 * kPer;
            r.lo = rank == 0 ? 0 : r.begin;
            r.hi = rank == ranks - 1 ? vocab : s.head + v1 * kPer;
            if (GRAD) r.out = static_cast<T*>(args.grad) + t * args.grad_stride;
            return r;
        };
        const auto edge_of = [&](int64_t t) {
            Edge e;
            if (t < d.rows && tid < 16) {
                const T* p = row_of(t);
                const Span s(p, vocab);
                if (rank == 0 && tid < s.head) e.at = tid;
                if (rank == ranks - 1 && tid >= 8 && tid - 8 < s.tail) e.at = vocab - s.tail + tid - 8;
                if (e.at >= 0) e.z = load(p, e.at);
            }
            return e;
        };

        const auto start = [&](const Edge& e) {
            Softmax m{-INFINITY, 0.0f, 0.0f};
            if (e.at >= 0 && e.z != -INFINITY) {
                const float one = e.z - e.z + 1.0f;                 // NaN where it is not finite
                m = Softmax{e.z, one, one};
            }
            return m;
        };

        // Pass 1 over the n vectors of a chunk: a whole one has kVecs to a thread,
        // taken together; the vectors of a row's last chunk go one by one.
        const auto take_vectors = [&](Softmax& m, const auto& q) {
            constexpr int N = sizeof(q) / sizeof(uint4);
            const T* kind = nullptr;
            const float top = largest<N>(q, kind);
            if (top > m.max) {
                if (DUAL) m.s1 *= rescale(m.max, top, c1);
                m.st *= rescale(m.max, top, ct);
                m.max = top;
            }
            const float2 less = both(m.max == -INFINITY ? 0.0f : -m.max);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float v[kPer];
                unpack(q[i], v, kind);
                float2 a1 = both(0.0f), at = both(0.0f);
#pragma unroll
                for (int j = 0; j < kPer; j += 2) {
                    const float2 x = __fadd2_rn(make_float2(v[j], v[j + 1]), less);
                    if (DUAL) a1 = __fadd2_rn(a1, exp2_pair(__fmul2_rn(x, both(c1))));
                    at = __fadd2_rn(at, exp2_pair(__fmul2_rn(x, both(ct))));
                }
                if (DUAL) m.s1 += a1.x + a1.y;
                m.st += at.x + at.y;
            }
        };
        const auto take = [&](Softmax& m, int slot, int n) {
            const uint4* from = buf + slot * chunk + tid;
            if (n == kVecs * NT) {
                uint4 q[kVecs];
#pragma unroll
                for (int i = 0; i < kVecs; ++i) q[i] = from[i * NT];
                take_vectors(m, q);
            } else {
#pragma unroll 1
                for (int i = tid; i < n; i += NT, from += NT) {
                    const uint4 q[1] = {*from};
                    take_vectors(m, q);
                }
            }
        };

        int b = 0;                                    // of the prepared teachers
        uint32_t taught_phase = 0;
        const auto next_teacher = [&]() {
            if (++b == kTeachers) b = 0, taught_phase ^= 1;
        };

        // The row's maximum and sums, from all threads of all CTAs.  Every thread
        // has then left the pass before it (one barrier).
        int parity = 0;
        uint32_t xch_phase = 0;
        const auto reduce = [&](Softmax& m) {
            merge_lanes<DUAL>(m, 32, c1, ct);
            if (lane == 0) s_part[parity][warp] = m;
            asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
            m = s_part[parity][lane % kWarps];
            merge_lanes<DUAL>(m, kWarps, c1, ct);
            if (ranks > 1) {
                // to every CTA of the cluster; a buffer is written again two rows
                // on, after all have read it.  The gradient may be written over
                // the logits, and a teacher reads them anywhere in the row: a CTA
                // tells the others to go on only when its own teacher is done
                // (most rows' has been for a row)
                if (tid < static_cast<int>(ranks)) {
                    if (GRAD) wait(&s_taught[b], taught_phase);
                    const uint32_t to = peer_addr(smem_addr(&s_peer[parity][rank]), tid);
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(m.max) : "memory");
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(m.s1) : "memory");
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(m.st) : "memory");
                    bar_arrive_cluster(peer_addr(smem_addr(&s_xch[parity]), tid));
                }
                __syncwarp();
                if (ok) ok = bar_wait<true>(smem_addr(&s_xch[parity]), xch_phase);
                m = s_peer[parity][lane & (ranks - 1)];
                merge_lanes<DUAL>(m, ranks, c1, ct);
            }
            if (m.max == -INFINITY) m.s1 = m.st = NAN;              // a row of -inf
            if (!DUAL) m.s1 = m.st;
            if ((parity ^= 1) == 0) xch_phase ^= 1;
        };

        // The loss, by the last warp of the first CTA.
        const auto write_loss = [&](int64_t t, const Softmax& m, int b) {
            if (!args.loss || rank != 0 || warp != kWarps - 1) return;
            // log q_id = z/tau - lse: relative to the maximum, where both are small
            const Teacher& r = s_teacher[b];
            const float *logp = s_logp + b * E, *z = s_z + b * E;
            const float ls1 = logf(m.s1), lst = logf(m.st);
            float part = 0.0f;
            if (r.taught)
                for (int k = lane; k < K; k += 32) {
                    // no weight adds nothing, also where l is finite and the student's
                    // logit -inf
                    const float l = logp[k], p = expf(l);
                    if (p > 0.0f) part += p * (l - ((z[k] - m.max) * it - lst));
                }
            for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
            if (lane == 0) {
                args.loss[t] = (r.taught ? d.kd_weight * d.temperature * d.temperature * part : 0.0f) +
                               (r.labelled ? d.ce_weight * (ls1 + (m.max - r.label_z)) : 0.0f);
                if (args.stats_out) {
                    args.stats_out[2 * t] = d.ce_weight > 0.0f ? m.max + ls1 : 0.0f;
                    args.stats_out[2 * t + 1] = kd ? m.max * it + lst : 0.0f;
                }
            }
        };

        // The gradient of an element: ft 2^((x at + bt) gt) + f1 2^((x + b1) c1).
        struct Slope {
            float ft = 0.0f, f1 = 0.0f, at = 1.0f, bt = 0.0f, gt = 0.0f, b1 = 0.0f;
        };
        const auto slope_of = [&](const Softmax& m, const Teacher& r) {
            Slope s;
            s.ft = r.own_t;
            s.f1 = r.own_1;
            if (MODE == kStream && args.stats_in) {
                s.at = kd ? it : 1.0f;
                s.bt = kd ? -r.lset : -r.lse1;
                s.gt = kLog2e;
                s.b1 = -r.lse1;
            } else {
                s.bt = s.b1 = -m.max;
                s.gt = ct;
                s.ft = s.ft == 0.0f ? 0.0f : __fdividef(s.ft, m.st);
                s.f1 = s.f1 == 0.0f ? 0.0f : __fdividef(s.f1, m.s1);
            }
            if (!DUAL) s.ft += s.f1;
            return s;
        };
        // 0 whatever the logits are, for a row that has no term
        const auto idle = [&](const Slope& s) { return s.ft == 0.0f && (!DUAL || s.f1 == 0.0f); };
        const auto slope2 = [&](const Slope& s, float2 x) {
            const float2 e = MODE == kStream ? __ffma2_rn(x, both(s.at), both(s.bt)) : __fadd2_rn(x, both(s.bt));
            float2 g = __fmul2_rn(both(s.ft), exp2_pair(__fmul2_rn(e, both(s.gt))));
            if (DUAL) g = __ffma2_rn(both(s.f1), exp2_pair(__fmul2_rn(__fadd2_rn(x, both(s.b1)), both(c1))), g);
            return g;
        };
        const auto slope1 = [&](const Slope& s, float x) { return idle(s) ? 0.0f : slope2(s, both(x)).x; };

        // Pass 2 over the n vectors of a chunk, whose gradient goes to `out`.
        const auto vector_slope = [&](const Slope& s, const uint4& q, bool none) {
            const T* kind = nullptr;
            float v[kPer];
            unpack(q, v, kind);
#pragma unroll
            for (int j = 0; j < kPer; j += 2) {
                const float2 g = slope2(s, make_float2(v[j], v[j + 1]));
                v[j] = g.x;
                v[j + 1] = g.y;
            }
            return none ? make_uint4(0, 0, 0, 0) : pack(v, kind);
        };
        const auto give = [&](const Slope& s, int slot, int n, T* out) {
            const uint4* from = buf + slot * chunk + tid;
            uint4* to = reinterpret_cast<uint4*>(out) + tid;
            const bool none = idle(s);
            if ((reinterpret_cast<uintptr_t>(out) & 15) != 0) {
#pragma unroll 1
                for (int i = tid; i < n; i += NT, from += NT, to += NT) scatter(reinterpret_cast<T*>(to), vector_slope(s, *from, none));
            } else if (n == kVecs * NT) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i) __stcs(to + i * NT, vector_slope(s, from[i * NT], none));
            } else {
#pragma unroll 1
                for (int i = tid; i < n; i += NT, from += NT, to += NT) __stcs(to, vector_slope(s, *from, none));
            }
        };

        // What the entries and the label have of their own, after the whole row's
        // pass 2 in every thread.
        const auto own_terms = [&](const Row& r, const Slope& s, int b) {
            const int* ids = s_id + b * E;
            const float *own = s_own + b * E, *z = s_z + b * E;
            for (int k = tid; k <= K; k += NT) {
                const int id = ids[k];
                if (id >= r.lo && id < r.hi) store(r.out, id, slope1(s, z[k]) - own[k]);
            }
        };
        const auto used = [&](int b) {
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&s_used[b]));
        };

        const auto edge_slope = [&](const Row& r, const Slope& s, const Edge& e) {
            if (e.at >= 0) store(r.out, e.at, slope1(s, e.z));
        };

        Place read;                                   // of the pass that reads first
        if (MODE == kTrain) {
            Place write;                              // of pass 2
            Edge edge = edge_of(first_row), ahead = edge_of(first_row + rows);
            Row cur = part_of(first_row), before;
            Softmax m = start(edge);
            for (int c = 0; c < cur.n; c += chunk) {
                await(read);
                take(m, read.slot, min(chunk, cur.n - c));
                step(read);
            }
            Slope slope;                              // of the row before, whose own terms are still to be written
            int before_b = -1;
            for (int64_t t = first_row; t < d.rows; t += rows) {
                reduce(m);
                if (before_b >= 0) {
                    own_terms(before, slope, before_b);
                    used(before_b);
                }
                wait(&s_taught[b], taught_phase);
                write_loss(t, m, b);
                slope = slope_of(m, s_teacher[b]);
                const Row next = t + rows < d.rows ? part_of(t + rows) : Row{};
                const Edge e = edge;
                edge = ahead;
                ahead = edge_of(t + 2 * rows);
                m = start(edge);
                T* out = cur.out + cur.begin;
                for (int c = 0; c < cur.n || c < next.n; c += chunk) {
                    if (c < next.n) {
                        await(read);
                        take(m, read.slot, min(chunk, next.n - c));
                        step(read);
                    }
                    if (c < cur.n) {
                        give(slope, write.slot, min(chunk, cur.n - c), out);
                        give_back(write);
                        step(write);
                        out += chunk * kPer;
                    }
                }
                edge_slope(cur, slope, e);
                before = cur;
                cur = next;
                before_b = b;
                next_teacher();
            }
            asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
            own_terms(before, slope, before_b);
            used(before_b);
        } else {
            const bool first_pass = MODE == kForward || !args.stats_in;
            Edge ahead = edge_of(first_row);
            for (int64_t t = first_row; t < d.rows; t += rows) {
                const Edge e = ahead;
                ahead = edge_of(t + rows);
                const Row cur = part_of(t);
                Softmax m = start(e);
                if (first_pass) {
                    for (int c = 0; c < cur.n; c += chunk) {
                        await(read);
                        take(m, read.slot, min(chunk, cur.n - c));
                        give_back(read);
                        step(read);
                    }
                    reduce(m);
                }
                wait(&s_taught[b], taught_phase);
                write_loss(t, m, b);
                if (MODE == kStream) {
                    const Slope slope = slope_of(m, s_teacher[b]);
                    T* out = cur.out + cur.begin;
                    for (int c = 0; c < cur.n; c += chunk) {
                        await(read);
                        give(slope, read.slot, min(chunk, cur.n - c), out);
                        give_back(read);
                        step(read);
                        out += chunk * kPer;
                    }
                    edge_slope(cur, slope, e);
                    asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
                    own_terms(cur, slope, b);
                }
                used(b);
                next_teacher();
            }
        }
    }
    if (!ok) atomicExch_system(args.fault, 1);
    __syncwarp();
    if (ranks > 1) cluster_sync();                   // no CTA ends while another may still write to it
}

// ------------------------------------------------------------------------- host

cudaError_t allow_shared(const void* kernel)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSm - kOfCta));
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

template <typename T, int MODE>
RowKernel row_kernel_of(bool dual, int shape)
{
    switch (kernel_shape(MODE, shape)) {
        case kFifth: return dual ? row_kernel<T, MODE, true, kFifth> : row_kernel<T, MODE, false, kFifth>;
        case kHalf: return dual ? row_kernel<T, MODE, true, kHalf> : row_kernel<T, MODE, false, kHalf>;
        default: return dual ? row_kernel<T, kTrain, true, kWhole> : row_kernel<T, kTrain, false, kWhole>;
    }
}

RowKernel row_kernel_of(bool f32, int mode, bool dual, int shape)
{
    if (f32)
        return mode == kForward ? row_kernel_of<float, kForward>(dual, shape)
                                : mode == kTrain ? row_kernel_of<float, kTrain>(dual, shape)
                                                 : row_kernel_of<float, kStream>(dual, shape);
    return mode == kForward ? row_kernel_of<uint16_t, kForward>(dual, shape)
                            : mode == kTrain ? row_kernel_of<uint16_t, kTrain>(dual, shape)
                                             : row_kernel_of<uint16_t, kStream>(dual, shape);
}

}  // namespace

cudaError_t prepare_distill()
{
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    for (bool f32 : {false, true})
        for (int mode : {kForward, kTrain, kStream})
            for (bool dual : {false, true})
                for (int shape : {kFifth, kHalf, kWhole})
                    if (e == cudaSuccess)
                        e = allow_shared(reinterpret_cast<const void*>(row_kernel_of(f32, mode, dual, shape)));
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
    const Config c = configure(d, dlogits != nullptr, stats_in == nullptr, dev.sms);
    if (!c.usable) return cudaErrorInvalidConfiguration;
    const bool dual = d.kd_weight > 0.0f && d.ce_weight > 0.0f && d.temperature != 1.0f;
    const RowKernel k = row_kernel_of(d.logits_dtype == Q8_F32, c.mode, dual, c.shape);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(c.ctas), 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(static_cast<unsigned>(threads_of(c.shape) + kOwn));
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
    a.slots = c.slots;
    a.chunk = c.chunk;
    a.seen = c.seen;
    a.fault = dev.fault;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace q8
