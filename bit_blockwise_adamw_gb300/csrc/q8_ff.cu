// q8_ff.cu -- the gated feed-forward product (include/q8train.h), forward and
// backward.
//
// Four matrix products carry it, all on one persistent tcgen05 kernel over
// pairs of CTAs (tile_kernel):
//   kForward  [g | u] = x [w_gate | w_up]^T       epilogue: h = act(g) u
//   kGates    the same product again              epilogue: dg, du from dh
//   kProducts dx = dg w_gate + du w_up            one accumulation over 2 d_ff
//             dw_gate = dg^T x, dw_up = du^T x    two batches, in the same launch
// A pair owns a 256 x 256 tile of the result: each CTA holds 128 rows of A and
// half of B's 256 rows, and the pair's tensor cores read both halves, so each
// operand byte is fetched once for twice the products.  In kForward and kGates
// the 256 columns are 128 of g beside the same 128 of u (CTA 0 loads w_gate's
// rows, CTA 1 w_up's), so that one thread of the epilogue finds g and u of its
// element in its own tensor-memory lane and no intermediate leaves the chip.
// Operands stay as they lie in memory: an operand whose M or N index is
// contiguous (the weights for dx, everything for dw) is loaded in boxes of
// 64 of that index by 64 of K and given to the tensor core as MN-major.
//
// Roles: warp 0 loads (TMA, a ring of six 32 KB stages in each CTA), warp 1 of
// the pair's first CTA issues the products, eight warps run the epilogue from
// tensor memory, whose 512 columns hold two accumulators, so that a tile's
// epilogue runs under the next tile's products.
//
// The tensor cores bound it where tiles are many: 8192 tokens, 4096 x 16384,
// forward and backward, 4.18 ms or 1.58 PFLOP/s, at the board's power limit.
// With few tiles the last round does: 1023 tokens, 1600 x 6400, 121 us for
// 63.7 us of products at their peak rate, 200 forward tiles on 76 pairs.
#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>

#include <cudaTypedefs.h>

#include "q8_internal.h"
#include "q8_tc.cuh"
#include "q8_train.h"

namespace q8 {

namespace {

constexpr int kPairM = 256, kPairN = 256, kStepK = 64;     // a pair's tile; K to a stage
constexpr int kHalf = 128;                                 // a CTA's rows of A, and of B
constexpr int kStages = 6;
constexpr int kOperandBytes = kHalf * kStepK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kChunkBytes = 64 * kStepK * 2;               // 64 of M or N by 64 of K
constexpr int kEpilogueWarps = 8;
constexpr int kTileThreads = 64 + 32 * kEpilogueWarps;
constexpr int kTileSmem = kStages * kStageBytes + 1024 + 256 + kEpilogueWarps * 32 * 17 * 4;
constexpr int kRaster = 8;                                 // row tiles that share a sweep over the columns

constexpr int kMostPairs = 160;

enum Mode { kForward, kGates, kProducts };
enum { kInput, kWeight };                                  // the jobs of kProducts: dx, and the weights' gradients

// One product: its tiles, by batch and by part of K.
struct Job {
    CUtensorMap a[2], b[2];          // kForward, kGates: a[0]; b by CTA.  kInput: by segment.  kWeight: a by batch, b[0]
    int32_t m_tiles, n_tiles, batches, splits;
    int32_t k_steps, segments;       // stages of one segment, and segments
    int64_t M, N;                    // of one batch's result (N = d_ff where two accumulators share a tile)
    uint16_t* out[2];
    int64_t out_stride;
    float* partial;                  // splits > 1: [batch, split, M, N]

    __host__ __device__ int64_t units() const { return static_cast<int64_t>(batches) * splits * m_tiles * n_tiles; }
};

struct TileArgs {
    Job job[2];                      // kForward, kGates: the first alone
    // Pairs take every pairs-th unit of the first job; the last `late` of them,
    // which have one unit less there, then take more of the second: all pairs take
    // every pairs-th for `rounds` rounds, then the late ones alone the rest.
    int32_t rounds, late;
    float* save;                     // kForward: g [M, N], then u, or NULL
    const uint16_t* dh;              // kGates
    int64_t dh_stride;
    int32_t act;
    int32_t* fault;                  // host-mapped: set when a wait ran out
};

// act(g) and act'(g).  __expf and the reciprocal are within a few units of 2^-23
// of their results; the reciprocal also of subnormal ones, where __fdividef gives
// 0 (past a denominator of 2^126): times the tanh form's inner derivative, some
// hundreds there, such a result is a normal number.
__device__ __forceinline__ float sigmoid(float t)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-t)));
    return r;
}

// Phi(g) = erfc(-g / sqrt(2)) / 2, with erfc(z) = t exp(-z^2 + P(t)),
// t = 1 / (1 + z / 2), z >= 0: the Chebyshev fit of Press et al., "Numerical
// Recipes", 6.2, within 1.2e-7 of erfc relatively everywhere; no branches, where
// erfcf's cost 5 us of 37 us of the forward product at 1023 tokens, 1600 x 6400.
__device__ __forceinline__ float normal_cdf(float g)
{
    const float z = fabsf(g) * 0.70710678118654752f, t = __fdividef(1.0f, fmaf(0.5f, z, 1.0f));
    float p = fmaf(t, 0.17087277f, -0.82215223f);
    p = fmaf(t, p, 1.48851587f);
    p = fmaf(t, p, -1.13520398f);
    p = fmaf(t, p, 0.27886807f);
    p = fmaf(t, p, -0.18628806f);
    p = fmaf(t, p, 0.09678418f);
    p = fmaf(t, p, 0.37409196f);
    p = fmaf(t, p, 1.00002368f);
    p = fmaf(t, p, -1.26551223f);
    const float half = 0.5f * t * __expf(fmaf(-z, z, p));
    return g < 0.0f ? half : 1.0f - half;
}

__device__ __forceinline__ float act_value(float g, int act)
{
    if (act == Q8_SILU) return g * sigmoid(g);
    if (act == Q8_GELU_TANH)       // (1 + tanh t)/2 = sigmoid(2 t)
        return g * sigmoid(1.5957691216057308f * g * fmaf(0.044715f, g * g, 1.0f));
    return g * normal_cdf(g);
}

__device__ __forceinline__ float2 act_both(float g, int act)
{
    if (act == Q8_SILU) {
        const float s = sigmoid(g);
        return make_float2(g * s, s * fmaf(g, 1.0f - s, 1.0f));
    }
    if (act == Q8_GELU_TANH) {
        // g^2 bounded: past 1e15 the sigmoid is 0 or 1, and infinity times s (1 - s) would be NaN
        const float g2 = fminf(g * g, 1e30f), s = sigmoid(1.5957691216057308f * g * fmaf(0.044715f, g2, 1.0f));
        return make_float2(g * s, s + g * s * (1.0f - s) * 1.5957691216057308f * fmaf(0.134145f, g2, 1.0f));
    }
    const float cdf = normal_cdf(g);
    return make_float2(g * cdf, fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), cdf));
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store32(void* p, const uint32_t r[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}

__device__ __forceinline__ void store16(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    *reinterpret_cast<uint4*>(p) = make_uint4(a, b, c, d);
}

// 32 consecutive elements of a row on 16 bytes.
__device__ __forceinline__ void store_row(uint16_t* p, const float v[32])
{
    uint32_t r[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) r[j] = pack2(v[2 * j], v[2 * j + 1]);
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        store32(p, r);
        store32(p + 16, r + 8);
    } else {
#pragma unroll
        for (int j = 0; j < 16; j += 4) store16(p + 2 * j, r[j], r[j + 1], r[j + 2], r[j + 3]);
    }
}

__device__ __forceinline__ void store_row(float* p, const float v[32])
{
    const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) store32(p + j, r + j);
    } else {
#pragma unroll
        for (int j = 0; j < 32; j += 4) store16(p + j, r[j], r[j + 1], r[j + 2], r[j + 3]);
    }
}

// A warp's 32 x 32 elements (a row to a lane) to rows `stride` apart, of which
// `rows` and of whose columns `cols` exist.  Rows on 16 bytes are stored lane by
// lane; others, and a matrix's last columns, go through the warp's shared memory
// so that a store still covers consecutive addresses (2968 tokens, 927 x 8576:
// element by element from the lanes the two backward products took 318 us).
constexpr int kTurnWords = 32 * 17;

template <typename T>
__device__ __forceinline__ void store_block(T* p, int64_t stride, int64_t rows, int64_t cols, const float v[32], float* turn, int lane)
{
    if (cols >= 32 && ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride * sizeof(T))) & 15) == 0) {
        if (lane < rows) store_row(p + lane * stride, v);
        return;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) turn[lane * 17 + j] = v[16 * half + j];
        __syncwarp();
        const int col = lane & 15;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = 2 * i + (lane >> 4);
            if (row < rows && 16 * half + col < cols) {
                const float x = turn[row * 17 + col];
                if constexpr (sizeof(T) == 2) p[row * stride + 16 * half + col] = float_to_bf16(x);
                else p[row * stride + 16 * half + col] = x;
            }
        }
    }
}

__device__ __forceinline__ void load_row(const uint16_t* p, float v[32], int64_t left)
{
    if (left >= 32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < left ? bf16_to_float(p[i]) : 0.0f;
    }
}

// One unit of work: a tile of one batch, over one of `splits` parts of K.
struct Unit {
    int batch, split, m, n, k0, k1;
};

__device__ __forceinline__ Unit unit_of(const Job& a, int i)
{
    Unit u;
    const int tiles = a.m_tiles * a.n_tiles;
    const int t = i % tiles;
    u.split = i / tiles % a.splits;
    u.batch = i / tiles / a.splits;
    // kRaster row tiles by all columns at a time, column by column: the tiles
    // that run at once share rows of both operands, which L2 then holds
    const int band = t / (kRaster * a.n_tiles), first = band * kRaster;
    const int rows = min(kRaster, a.m_tiles - first), in = t - first * a.n_tiles;
    u.m = first + in % rows;
    u.n = in / rows;
    const int64_t steps = static_cast<int64_t>(a.k_steps) * a.segments;
    u.k0 = static_cast<int>(steps * u.split / a.splits);
    u.k1 = static_cast<int>(steps * (u.split + 1) / a.splits);
    return u;
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ TileArgs args)
{
    constexpr bool kDual = MODE != kProducts;

    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;      // 128-byte swizzle: 1024-byte aligned stages
    const uint32_t bars = base + kStages * kStageBytes;
    const auto full = [&](int s) { return bars + 8 * s; };
    const auto empty = [&](int s) { return bars + 8 * (kStages + s); };
    const auto acc_full = [&](int b) { return bars + 8 * (2 * kStages + b); };
    const auto acc_empty = [&](int b) { return bars + 8 * (2 * kStages + 2 + b); };
    const uint32_t done = bars + 8 * (2 * kStages + 4);
    const uint32_t tmem_slot = done + 8;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    // the pair's units, in the same order in every role; body returns false to stop
    const auto for_units = [&](auto&& body) {
        const int units = static_cast<int>(args.job[0].units());           // checked to fit
        for (int i = pair; i < units; i += pairs)
            if (!body(args.job[0], 0, i)) return;
        if (kDual) return;
        // from the last pair on, so that neighbours work on neighbouring tiles
        const int second = static_cast<int>(args.job[1].units()), from = pairs - 1 - pair, common = args.rounds * pairs;
        for (int i = from; i < min(second, common); i += pairs)
            if (!body(args.job[1], 1, i)) return;
        for (int i = common + from; from < args.late && i < second; i += args.late)
            if (!body(args.job[1], 1, i)) return;
    };

    if (warp == 0) {
        if (elect()) {
            for (int s = 0; s < kStages; ++s) {
                bar_init(full(s), 1);
                bar_init(empty(s), 1);
            }
            for (int b = 0; b < 2; ++b) {
                bar_init(acc_full(b), 1);
                bar_init(acc_empty(b), 2 * kEpilogueWarps);
            }
            bar_init(done, 1);
            bar_init_fence();
            tma_prefetch_map(&args.job[0].a[0]);
            tma_prefetch_map(&args.job[0].b[0]);
        }
    } else if (warp == 1) {
        tmem_alloc_all(tmem_slot);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));

    bool ok = true;
    if (warp == 0) {
        if (elect()) {
            int s = 0;
            uint32_t phase = 1;                       // an empty stage's first wait passes
            for_units([&](const Job& job, int which, int i) {
                const Unit u = unit_of(job, i);
                const bool input = !kDual && which == kInput, weight = !kDual && which == kWeight;
                const int m0 = u.m * kPairM + static_cast<int>(rank) * kHalf;
                const int n0 = kDual ? u.n * kHalf : u.n * kPairN + static_cast<int>(rank) * kHalf;
                for (int k = u.k0; k < u.k1; ++k) {
                    if (!(ok = bar_wait(empty(s), phase))) return false;
                    if (rank == 0) bar_expect(full(s), 2 * kStageBytes);
                    const uint32_t bar = peer_addr(full(s), 0);
                    const int seg = input ? k / job.k_steps : 0;
                    const int x = (k - seg * job.k_steps) * kStepK;
                    const CUtensorMap* a = &job.a[weight ? u.batch : seg];
                    const CUtensorMap* b = &job.b[kDual ? rank : seg];
                    const uint32_t sa = base + s * kStageBytes, sb = sa + kOperandBytes;
                    if (weight) {
                        tma_load(sa, a, m0, x, bar);
                        tma_load(sa + kChunkBytes, a, m0 + 64, x, bar);
                    } else {
                        tma_load(sa, a, x, m0, bar);
                    }
                    if (!kDual) {
                        tma_load(sb, b, n0, x, bar);
                        tma_load(sb + kChunkBytes, b, n0 + 64, x, bar);
                    } else {
                        tma_load(sb, b, x, n0, bar);
                    }
                    if (++s == kStages) s = 0, phase ^= 1;
                }
                return true;
            });
            // no load may be in flight when the CTA ends: every stage loaded
            // has been given back (the products over it have completed)
            for (int i = 0; i < kStages; ++i) {
                ok = bar_wait(empty(s), phase) && ok;
                if (++s == kStages) s = 0, phase ^= 1;
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect()) {
            int s = 0, b = 0;
            uint32_t phase = 0, acc_phase = 1;
            for_units([&](const Job& job, int which, int i) {
                const Unit u = unit_of(job, i);
                // K-major: 8 rows of 128 bytes to a swizzle atom, K = 16 is 32 bytes on;
                // MN-major: 8 of K by 64 of M to an atom, K = 16 is two atoms on
                const bool a_mn = !kDual && which == kWeight;
                const uint32_t desc = kDual ? mma_desc(false, false, kPairM, kPairN)
                                            : a_mn ? mma_desc(true, true, kPairM, kPairN) : mma_desc(false, true, kPairM, kPairN);
                const uint32_t a_step = a_mn ? 2048 : 32, a_lead = a_mn ? kChunkBytes : 16;
                constexpr uint32_t b_step = kDual ? 32 : 2048, b_lead = kDual ? 16 : kChunkBytes;
                if (!(ok = bar_wait<true>(acc_empty(b), acc_phase))) return false;
                tc_fence_after();
                const uint32_t d = tmem + b * kPairN;
                for (int k = u.k0; k < u.k1; ++k) {
                    if (!(ok = bar_wait(full(s), phase))) return false;
                    tc_fence_after();
                    const uint32_t sa = base + s * kStageBytes, sb = sa + kOperandBytes;
#pragma unroll
                    for (int j = 0; j < kStepK / 16; ++j)
                        mma_pair(d, smem_desc(sa + j * a_step, a_lead, 1024), smem_desc(sb + j * b_step, b_lead, 1024), desc,
                                 k > u.k0 || j > 0);
                    mma_commit_pair(empty(s));
                    if (++s == kStages) s = 0, phase ^= 1;
                }
                mma_commit_pair(acc_full(b));
                if (++b == 2) b = 0, acc_phase ^= 1;
                return true;
            });
            mma_commit_pair(done);
            ok = bar_wait(done, 0) && ok;                // tensor memory is freed after this
        }
    } else {
        const int quad = warp & 3, half = (warp - 2) >> 2;       // 32 lanes, and half of the columns
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        float* turn = reinterpret_cast<float*>(raw + (bars + 256 - smem_addr(raw))) + (warp - 2) * kTurnWords;
        int b = 0;
        uint32_t phase = 0;
        for_units([&](const Job& job, int which, int i) {
            const Unit u = unit_of(job, i);
            const int64_t m = static_cast<int64_t>(u.m) * kPairM + rank * kHalf + quad * 32, rows = job.M - m;
            if (!(ok = __all_sync(0xFFFFFFFFu, bar_wait(acc_full(b), phase)))) return false;
            tc_fence_after();
            const uint32_t t = lanes + b * kPairN;
            constexpr int kChunks = kDual ? 2 : 4;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
                float v[32], w[32];
                const int col = (half * kChunks + c) * 32;
                const int64_t n = static_cast<int64_t>(u.n) * (kDual ? kHalf : kPairN) + col;
                const int64_t left = job.N - n;
                tmem_load32(t + col, v);
                if (kDual) tmem_load32(t + kHalf + col, w);
                tmem_load_wait();
                if (c == kChunks - 1) {                  // read out: the products may write here again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive_cluster(peer_addr(acc_empty(b), 0));
                }
                if (rows <= 0 || left <= 0) continue;    // for all of the warp
                if (MODE == kForward) {
                    if (args.save) {
                        store_block(args.save + m * job.N + n, job.N, rows, left, v, turn, lane);
                        store_block(args.save + (job.M + m) * job.N + n, job.N, rows, left, w, turn, lane);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = act_value(v[j], args.act) * w[j];
                    store_block(job.out[0] + m * job.out_stride + n, job.out_stride, rows, left, v, turn, lane);
                } else if (MODE == kGates) {
                    float d[32];
                    load_row(args.dh + (m + lane) * args.dh_stride + n, d, lane < rows ? left : 0);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float2 a = act_both(v[j], args.act);
                        v[j] = d[j] * w[j] * a.y;
                        w[j] = d[j] * a.x;
                    }
                    store_block(job.out[0] + m * job.out_stride + n, job.out_stride, rows, left, v, turn, lane);
                    store_block(job.out[1] + m * job.out_stride + n, job.out_stride, rows, left, w, turn, lane);
                } else if (job.splits > 1) {
                    store_block(job.partial + ((static_cast<int64_t>(u.batch) * job.splits + u.split) * job.M + m) * job.N + n, job.N,
                                rows, left, v, turn, lane);
                } else {
                    store_block(job.out[u.batch] + m * job.out_stride + n, job.out_stride, rows, left, v, turn, lane);
                }
            }
            if (++b == 2) b = 0, phase ^= 1;
            return true;
        });
        // the second CTA's copy of the last arrival: it must land before the CTA ends
        if (rank == 1 && warp == 2) ok = bar_wait(done, 0) && ok;
    }
    if (!ok) atomicExch_system(args.fault, 1);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) tmem_free_all(tmem);
}

// ------------------------------------------------------------ few tokens
//
// Up to 128 tokens the weights' bytes bound the forward product.  The weights
// are the tensor core's M then (64 rows of w_gate over the same 64 of w_up: one
// 128-row tile), the tokens its N, padded to 16, 32, 64 or 128 instead of 256;
// a CTA has a tile, and two CTAs on an SM keep 200 KB of weights in flight.
// Where tiles are fewer than half the SMs a cluster of 2, 4 or 8 CTAs shares a
// tile's K and the first adds up the others' parts, which they write to its
// shared memory (1 token, 1952 x 728: 10.8 us alone, 9 us with eight; with as
// many tiles as SMs parts only take the loads of a row apart: 24 tokens,
// 2560 x 10240: 36 us with two).
// A lane of tensor memory is a column of g (0..63) or u (64..127): they meet
// through shared memory.
// 24 tokens, 2560 x 10240: 22.8 us for 105 MB of weights, 4.6 TB/s (69 % of a
// copy's rate); memory is read 128 bytes of a row at a time, and the ring's
// first fill and the last epilogue have nothing to run under.
constexpr int kFewTokens = 128, kFewRows = 64, kFewThreads = 256, kFewStages = 8;

struct FewArgs {
    CUtensorMap x, w[2];
    int32_t tokens, columns, stages, k_steps;        // columns: the padded tokens
    int32_t parts;                   // CTAs to a tile
    int64_t d_ff;
    uint16_t* h;
    int64_t h_stride;
    float* save;
    int32_t act;
    int32_t* fault;
};

constexpr int kFewSmem = 112 * 1024;                 // two CTAs on an SM

int few_stage_bytes(int columns) { return kOperandBytes + columns * kStepK * 2; }

__global__ void __launch_bounds__(kFewThreads) few_kernel(const __grid_constant__ FewArgs args)
{
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_bar[2 * kFewStages + 1];
    __shared__ uint32_t s_tmem;
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    const uint32_t stage_bytes = kOperandBytes + args.columns * kStepK * 2;
    const auto full = [&](int s) { return smem_addr(&s_bar[s]); };
    const auto empty = [&](int s) { return smem_addr(&s_bar[kFewStages + s]); };
    const uint32_t done = smem_addr(&s_bar[2 * kFewStages]);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = static_cast<int>(cluster_rank());
    const int f0 = blockIdx.x / args.parts * kFewRows;
    const int k0 = args.k_steps * part / args.parts, k1 = args.k_steps * (part + 1) / args.parts;
    const uint32_t tmem_columns = max(32, args.columns);

    if (warp == 0 && elect()) {
        for (int s = 0; s < kFewStages; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        bar_init(done, 1);
        bar_init_fence();
    }
    if (warp == 1) tmem_alloc_single(smem_addr(&s_tmem), tmem_columns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    bool ok = true;
    if (warp == 0 && elect()) {
        int s = 0;
        uint32_t phase = 1;
        for (int k = k0; k < k1; ++k) {
            if (!(ok = bar_wait(empty(s), phase))) break;
            bar_expect(full(s), stage_bytes);
            const uint32_t sa = base + s * stage_bytes;
            tma_load_single(sa, &args.w[0], k * kStepK, f0, full(s));
            tma_load_single(sa + kOperandBytes / 2, &args.w[1], k * kStepK, f0, full(s));
            tma_load_single(sa + kOperandBytes, &args.x, k * kStepK, 0, full(s));
            if (++s == args.stages) s = 0, phase ^= 1;
        }
        // every load's stage has been given back before the CTA ends
        for (int i = 0; i < args.stages; ++i) {
            ok = bar_wait(empty(s), phase) && ok;
            if (++s == args.stages) s = 0, phase ^= 1;
        }
    } else if (warp == 1 && elect()) {
        const uint32_t desc = mma_desc(false, false, 128, args.columns);
        int s = 0;
        uint32_t phase = 0;
        for (int k = k0; k < k1; ++k) {
            if (!(ok = bar_wait(full(s), phase))) break;
            tc_fence_after();
            const uint32_t sa = base + s * stage_bytes, sb = sa + kOperandBytes;
#pragma unroll
            for (int j = 0; j < kStepK / 16; ++j)
                mma_single(tmem, smem_desc(sa + j * 32, 16, 1024), smem_desc(sb + j * 32, 16, 1024), desc, k > k0 || j > 0);
            mma_commit_single(empty(s));
            if (++s == args.stages) s = 0, phase ^= 1;
        }
        mma_commit_single(done);
    }
    __syncwarp();
    ok = __all_sync(0xFFFFFFFFu, bar_wait(done, 0)) && ok;
    tc_fence_after();

    // lane l < 64: column f0 + l of g; lane 64 + l: the same of u.  Warps 0..3 and
    // 4..7 take every other 16 tokens.
    const int quad = warp & 3, l = (quad & 1) * 32 + lane, side = quad >> 1;
    const int64_t f = static_cast<int64_t>(f0) + l;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // over the stages, which nobody reads any more: the other CTAs' parts
    // [parts - 1][columns][128], then what the warps of g and those of u give one
    // another, [columns][64]
    float* s_part = reinterpret_cast<float*>(raw + (base - smem_addr(raw)));
    float* s_other = s_part + (args.parts - 1) * args.columns * 128;
    const int c_first = (warp >> 2) * 16;
    float v[16];
    if (args.parts > 1) {
        cluster_sync();                              // all have read their stages
        if (part > 0) {
            const uint32_t to = peer_addr(smem_addr(s_part + (part - 1) * args.columns * 128 + quad * 32 + lane), 0);
            for (int c = c_first; c < args.columns; c += 32) {
                tmem_load16(lanes + c, v);
                tmem_load_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + (c + j) * 512), "f"(v[j]) : "memory");
            }
        }
        cluster_sync();
    } else {
        __syncthreads();
    }
    // the warps of g make h for the first half of the tokens, those of u for the
    // second; each gives the other its values of the other's half first
    for (int pass = 0; pass < 2 && part == 0; ++pass) {
        for (int c = c_first; c < args.columns; c += 32) {
            if (((2 * c >= args.columns) == (side == 1)) != (pass == 1)) continue;
            tmem_load16(lanes + c, v);
            tmem_load_wait();
            for (int p = 0; p < args.parts - 1; ++p)
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += s_part[(p * args.columns + c + j) * 128 + quad * 32 + lane];
            float* other = s_other + c * kFewRows + l;
            const int n = f < args.d_ff ? args.tokens - c : 0;       // of the 16 that exist
            if (args.save) {
                float* save = args.save + (static_cast<int64_t>(side) * args.tokens + c) * args.d_ff + f;
#pragma unroll
                for (int j = 0; j < 16; ++j, save += args.d_ff)
                    if (j < n) *save = v[j];
            }
            if (pass == 0) {
#pragma unroll
                for (int j = 0; j < 16; ++j) other[j * kFewRows] = v[j];
            } else {
                uint16_t* h = args.h + c * args.h_stride + f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float o = other[j * kFewRows];
                    v[j] = act_value(side ? o : v[j], args.act) * (side ? v[j] : o);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j, h += args.h_stride)
                    if (j < n) *h = float_to_bf16(v[j]);
            }
        }
        __syncthreads();
    }
    if (!ok) atomicExch_system(args.fault, 1);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_free_single(tmem, tmem_columns);
}

// out = the sum of the splits' parts, in their order: rows to blockIdx.x, four
// columns to a thread, a result to blockIdx.y.
struct Join {
    const float* partial;
    uint16_t* out;
    int64_t M, N, out_stride;
    int32_t splits;
};
struct JoinArgs {
    Join join[3];
};

__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs args)
{
    const Join& a = args.join[blockIdx.y];
    const int64_t part = a.M * a.N;
    const bool whole = (a.N & 3) == 0 && (a.out_stride & 3) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const float* p = a.partial + m * a.N;
        uint16_t* out = a.out + m * a.out_stride;
        for (int64_t n = 4 * threadIdx.x; n < a.N; n += 4 * 256) {
            if (whole) {
                float4 s = *reinterpret_cast<const float4*>(p + n);
                for (int k = 1; k < a.splits; ++k) {
                    const float4 q = *reinterpret_cast<const float4*>(p + k * part + n);
                    s.x += q.x;
                    s.y += q.y;
                    s.z += q.z;
                    s.w += q.w;
                }
                *reinterpret_cast<uint2*>(out + n) = make_uint2(pack2(s.x, s.y), pack2(s.z, s.w));
            } else {
                for (int64_t j = n; j < n + 4 && j < a.N; ++j) {
                    float s = p[j];
                    for (int k = 1; k < a.splits; ++k) s += p[k * part + j];
                    out[j] = float_to_bf16(s);
                }
            }
        }
    }
}

// dg and du from the saved g and u: eight columns of a row to a thread.  g and u
// are saved in 32 bits: dg and du are rounded once, as the products' operands,
// and dx and dw are then 1.4 times as far from float64 as a float32 evaluation
// (256 and 512 tokens, SiLU); with g and u rounded to 16 bits too, 1.8 times.
// Bytes bound it where d_ff is large (14 an element, 8 of them the saved ones).
__global__ void __launch_bounds__(256) gates_kernel(const float* save, const uint16_t* dh, int64_t dh_stride, int64_t M,
                                                    int64_t N, int act, uint16_t* dg, uint16_t* du, int64_t stride)
{
    const int64_t groups = (N + 7) / 8, n = M * groups;
    const bool whole = (N & 7) == 0 && ((reinterpret_cast<uintptr_t>(save) & 15) == 0) &&
                       ((reinterpret_cast<uintptr_t>(dh) & 15) == 0) && (dh_stride & 7) == 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t m = i / groups, c = (i - m * groups) * 8;
        const float *g = save + m * N + c, *u = g + M * N;
        const uint16_t* d = dh + m * dh_stride + c;
        float gv[8], uv[8], dv[8];
        if (whole) {
            *reinterpret_cast<float4*>(gv) = __ldcs(reinterpret_cast<const float4*>(g));
            *reinterpret_cast<float4*>(gv + 4) = __ldcs(reinterpret_cast<const float4*>(g) + 1);
            *reinterpret_cast<float4*>(uv) = __ldcs(reinterpret_cast<const float4*>(u));
            *reinterpret_cast<float4*>(uv + 4) = __ldcs(reinterpret_cast<const float4*>(u) + 1);
            const uint4 q = __ldcs(reinterpret_cast<const uint4*>(d));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dv[2 * j] = __uint_as_float(w[j] << 16);
                dv[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = c + j < N;
                gv[j] = in ? g[j] : 0.0f;
                uv[j] = in ? u[j] : 0.0f;
                dv[j] = in ? bf16_to_float(d[j]) : 0.0f;
            }
        }
        uint32_t a[4], b[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = act_both(gv[j], act);
            gv[j] = dv[j] * uv[j] * f.y;
            uv[j] = dv[j] * f.x;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = pack2(gv[2 * j], gv[2 * j + 1]);
            b[j] = pack2(uv[2 * j], uv[2 * j + 1]);
        }
        // the rows' stride is a multiple of 16: the last group's padding is there to be written
        *reinterpret_cast<uint4*>(dg + m * stride + c) = make_uint4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<uint4*>(du + m * stride + c) = make_uint4(b[0], b[1], b[2], b[3]);
    }
}

// Copies whose rows start on 16 bytes, for TMA: rows to blocks, eight columns to
// a thread, a matrix to blockIdx.y.
struct Align {
    const uint16_t* in;
    uint16_t* out;
    int64_t rows, in_stride;
};
struct AlignArgs {
    Align align[3];
    int64_t cols, out_stride;
};

__global__ void __launch_bounds__(256) align_kernel(const __grid_constant__ AlignArgs args)
{
    const Align& a = args.align[blockIdx.y];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const uint16_t* p = a.in + r * a.in_stride;
        for (int64_t c = 8 * threadIdx.x; c < args.cols; c += 8 * 256) {
            uint32_t w[4] = {};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < args.cols) w[j / 2] |= static_cast<uint32_t>(p[c + j]) << (16 * (j & 1));
            *reinterpret_cast<uint4*>(a.out + r * args.out_stride + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ------------------------------------------------------------------------- host

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// A bf16 matrix as TMA may read it.
struct Matrix {
    const uint16_t* p;
    int64_t rows, cols, stride;
};

bool tma_ready(const void* p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; }

// The workspace: aligned copies of x and the weights where TMA cannot read
// them in place, and for the backward call dg, du and the partial sums.
struct Layout {
    int64_t x = -1, w_gate = -1, w_up = -1, dg = -1, du = -1, input = -1, weight = -1, bytes = 0;   // the last two: parts
    int64_t d_stride, f_stride;              // row strides of the copies, and of dg and du
};

struct Device : DeviceInfo {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
};

// What a unit of n stages costs a pair, in stages: reading a tile out of tensor
// memory and storing it takes as long as some six stages, under the next tile's
// products where these are longer.
double cost_of(double n) { return n + 6.0; }

// The products of the backward call.  K is cut into parts where a tile alone
// would take longer than the pairs' even share of all the work, at least eight
// stages to a part (what fills the ring).
struct Shape {
    int64_t m_tiles, n_tiles, k_steps, segments;
    int splits;
};

struct Shapes {
    Shape input, weight;
};

Shapes shapes_of(const q8_gated_ff& f, int pairs)
{
    Shapes s{{ceil_div(f.tokens, kPairM), ceil_div(f.d_model, kPairN), ceil_div(f.d_ff, kStepK), 2, 1},
             {ceil_div(f.d_ff, kPairM), ceil_div(f.d_model, kPairN), ceil_div(f.tokens, kStepK), 1, 1}};
    const double all = static_cast<double>(s.input.m_tiles) * s.input.n_tiles * cost_of(2.0 * s.input.k_steps) +
                       2.0 * s.weight.m_tiles * s.weight.n_tiles * cost_of(static_cast<double>(s.weight.k_steps));
    const int64_t share = std::max<int64_t>(1, static_cast<int64_t>(all / pairs));
    for (Shape* j : {&s.input, &s.weight}) {
        const int64_t steps = j->k_steps * j->segments;
        j->splits = static_cast<int>(std::max<int64_t>(1, std::min(ceil_div(steps, share), steps / 8)));
    }
    return s;
}

std::mutex g_lock;
std::map<int, Device> g_devices;

cudaError_t device(Device* out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_lock);
    Device& d = g_devices[dev];
    if (!d.encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if ((e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found)) != cudaSuccess)
            return e;
        if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        if ((e = device_info(&d)) != cudaSuccess) return e;
        const void* kernels[] = {
            reinterpret_cast<const void*>(tile_kernel<kForward>), reinterpret_cast<const void*>(tile_kernel<kGates>),
            reinterpret_cast<const void*>(tile_kernel<kProducts>)};
        for (const void* k : kernels)
            if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem)) != cudaSuccess) return e;
        if ((e = cudaFuncSetAttribute(few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem)) != cudaSuccess) return e;
        d.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    *out = d;
    return cudaSuccess;
}

int pairs_of(int sms) { return std::max(1, std::min(sms / 2, kMostPairs)); }
int pairs_of(const Device& d) { return pairs_of(d.sms); }

// Two-dimensional map of m, boxes of box_cols x box_rows with the 128-byte
// swizzle; what lies outside reads as zeros.
cudaError_t encode(const Device& d, CUtensorMap* map, const Matrix& m, int box_cols, int box_rows)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(m.cols), static_cast<cuuint64_t>(m.rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(m.stride) * 2};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r = d.encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(m.p), dims, strides, box,
                                steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

Layout layout(const q8_gated_ff& f, bool backward, int pairs)
{
    Layout l;
    l.d_stride = round_up(f.d_model, 8);
    l.f_stride = round_up(f.d_ff, 16);
    auto take = [&](int64_t bytes) {
        const int64_t at = l.bytes;
        l.bytes += round_up(bytes, 256);
        return at;
    };
    if (f.tokens == 0) return l;
    if (!tma_ready(f.x, f.x_stride)) l.x = take(f.tokens * l.d_stride * 2);
    if (!tma_ready(f.w_gate, f.d_model)) l.w_gate = take(f.d_ff * l.d_stride * 2);
    if (!tma_ready(f.w_up, f.d_model)) l.w_up = take(f.d_ff * l.d_stride * 2);
    if (backward) {
        l.dg = take(f.tokens * l.f_stride * 2);
        l.du = take(f.tokens * l.f_stride * 2);
        const Shapes s = shapes_of(f, pairs);
        if (s.input.splits > 1) l.input = take(s.input.splits * f.tokens * f.d_model * 4);
        if (s.weight.splits > 1) l.weight = take(2 * s.weight.splits * f.d_ff * f.d_model * 4);
    }
    return l;
}

unsigned blocks_for(int64_t n, const Device& d)
{
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(n, 256), d.sms * int64_t(8))));
}

unsigned rows_for(int64_t rows, const Device& d) { return static_cast<unsigned>(std::min<int64_t>(rows, d.sms * int64_t(16))); }

// x and the weights as TMA may read them.
cudaError_t operands(const q8_gated_ff& f, const Layout& l, const Device& d, cudaStream_t st, Matrix m[3])
{
    m[0] = Matrix{f.x, f.tokens, f.d_model, f.x_stride};
    m[1] = Matrix{f.w_gate, f.d_ff, f.d_model, f.d_model};
    m[2] = Matrix{f.w_up, f.d_ff, f.d_model, f.d_model};
    const int64_t at[3] = {l.x, l.w_gate, l.w_up};
    AlignArgs a{};
    a.cols = f.d_model;
    a.out_stride = l.d_stride;
    unsigned count = 0;
    int64_t rows = 0;
    for (int i = 0; i < 3; ++i) {
        if (at[i] < 0) continue;
        uint16_t* copy = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(f.workspace) + at[i]);
        a.align[count++] = Align{m[i].p, copy, m[i].rows, m[i].stride};
        rows = std::max(rows, m[i].rows);
        m[i].p = copy;
        m[i].stride = l.d_stride;
    }
    if (count) align_kernel<<<dim3(rows_for(rows, d), count), 256, 0, st>>>(a);
    return cudaGetLastError();
}

template <int MODE>
cudaError_t run_tiles(TileArgs& a, const Device& d, cudaStream_t st)
{
    const int pairs = pairs_of(d);
    int64_t units[2];
    for (int i = 0; i < 2; ++i) {
        units[i] = a.job[i].units();
        if (units[i] >= (int64_t(1) << 31) - 2 * pairs) return cudaErrorInvalidValue;
    }
    // the second job's units go to the pairs so that all have about the same
    // work, counting that of the first job
    const auto steps = [&](int i) {
        const Job& j = a.job[i];
        return units[i] ? cost_of(static_cast<double>(j.k_steps) * j.segments / j.splits) : 0.0;
    };
    const int64_t ahead = units[0] % pairs;                  // pairs that have one more unit of the first job
    a.late = static_cast<int32_t>(pairs - ahead);
    if (units[1]) {
        const double share = (units[0] * steps(0) + units[1] * steps(1)) / pairs;
        const double left = share - (units[0] / pairs + (ahead > 0)) * steps(0);
        a.rounds = static_cast<int32_t>(std::min<double>(std::floor(std::max(0.0, left) / steps(1) + 0.5), static_cast<double>(units[1])));
        if (static_cast<int64_t>(a.rounds) * pairs > units[1]) a.rounds = static_cast<int32_t>(ceil_div(units[1], pairs));
    }
    const int64_t grid = units[1] ? pairs : std::min<int64_t>(units[0], pairs);
    a.fault = d.fault;
    tile_kernel<MODE><<<static_cast<unsigned>(2 * grid), kTileThreads, kTileSmem, st>>>(a);
    return cudaGetLastError();
}

// Where the product of x with both weights goes: kForward and kGates.
cudaError_t dual_args(const q8_gated_ff& f, const Device& d, const Matrix m[3], TileArgs* a)
{
    Job& j = a->job[0];
    j.m_tiles = static_cast<int32_t>(ceil_div(f.tokens, kPairM));
    j.n_tiles = static_cast<int32_t>(ceil_div(f.d_ff, kHalf));
    j.batches = j.splits = j.segments = 1;
    j.k_steps = static_cast<int32_t>(ceil_div(f.d_model, kStepK));
    j.M = f.tokens;
    j.N = f.d_ff;
    a->act = f.act;
    cudaError_t e = encode(d, &j.a[0], m[0], kStepK, kHalf);
    if (e == cudaSuccess) e = encode(d, &j.b[0], m[1], kStepK, kHalf);
    if (e == cudaSuccess) e = encode(d, &j.b[1], m[2], kStepK, kHalf);
    return e;
}

void set_shape(Job* j, const Shape& s, int64_t M, int64_t N)
{
    j->m_tiles = static_cast<int32_t>(s.m_tiles);
    j->n_tiles = static_cast<int32_t>(s.n_tiles);
    j->splits = s.splits;
    j->k_steps = static_cast<int32_t>(s.k_steps);
    j->segments = static_cast<int32_t>(s.segments);
    j->M = M;
    j->N = N;
}

}  // namespace

cudaError_t prepare_ff()
{
    Device d;
    return device(&d);
}

int64_t ff_workspace(const q8_gated_ff& f, bool backward)
{
    int dev = 0, sms = 0;                                    // sizes do not need a GPU: 152 SMs where there is none
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        sms = 152;
    }
    return layout(f, backward, pairs_of(sms)).bytes;
}

cudaError_t launch_ff_forward(const q8_gated_ff& f, uint16_t* h, int64_t h_stride, float* saved, cudaStream_t st)
{
    Device d;
    cudaError_t e = device(&d);
    if (e == cudaSuccess) e = earlier_fault(d.fault);
    if (e != cudaSuccess) return e;
    const Layout l = layout(f, false, pairs_of(d));
    Matrix m[3];
    if ((e = operands(f, l, d, st, m)) != cudaSuccess) return e;
    if (f.tokens <= kFewTokens) {
        FewArgs a{};
        a.tokens = static_cast<int32_t>(f.tokens);
        a.columns = 16;
        while (a.columns < a.tokens) a.columns *= 2;
        a.stages = std::min(kFewStages, (kFewSmem - 1024) / few_stage_bytes(a.columns));
        a.k_steps = static_cast<int32_t>(ceil_div(f.d_model, kStepK));
        a.d_ff = f.d_ff;
        a.h = h;
        a.h_stride = h_stride;
        a.save = saved;
        a.act = f.act;
        a.fault = d.fault;
        e = encode(d, &a.x, m[0], kStepK, a.columns);
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) e = encode(d, &a.w[i], m[1 + i], kStepK, kFewRows);
        if (e != cudaSuccess) return e;
        const int64_t tiles = ceil_div(f.d_ff, kFewRows);
        a.parts = 1;
        // at least four stages to a part, and the parts fit where the stages were
        while (a.parts < 8 && tiles * a.parts * 2 <= d.sms && a.k_steps >= 8 * a.parts &&
               (2 * a.parts - 1) * a.columns * 512 + a.columns * kFewRows * 4 <= a.stages * few_stage_bytes(a.columns))
            a.parts *= 2;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim = {static_cast<unsigned>(a.parts), 1, 1};
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.parts));
        cfg.blockDim = dim3(kFewThreads);
        cfg.dynamicSmemBytes = static_cast<size_t>(1024 + a.stages * few_stage_bytes(a.columns));
        cfg.stream = st;
        cfg.attrs = &attr;
        cfg.numAttrs = a.parts > 1;
        return cudaLaunchKernelEx(&cfg, few_kernel, a);
    }
    TileArgs a{};
    if ((e = dual_args(f, d, m, &a)) != cudaSuccess) return e;
    a.job[0].out[0] = h;
    a.job[0].out_stride = h_stride;
    a.save = saved;
    return run_tiles<kForward>(a, d, st);
}

cudaError_t launch_ff_backward(const q8_gated_ff& f, const FfBackward& b, cudaStream_t st)
{
    Device d;
    cudaError_t e = device(&d);
    if (e == cudaSuccess) e = earlier_fault(d.fault);
    if (e != cudaSuccess) return e;
    const Layout l = layout(f, true, pairs_of(d));
    uint8_t* ws = static_cast<uint8_t*>(f.workspace);
    uint16_t *dg = reinterpret_cast<uint16_t*>(ws + l.dg), *du = reinterpret_cast<uint16_t*>(ws + l.du);
    Matrix m[3];
    if ((e = operands(f, l, d, st, m)) != cudaSuccess) return e;
    if (b.saved) {
        gates_kernel<<<blocks_for(f.tokens * ceil_div(f.d_ff, 8), d), 256, 0, st>>>(
            b.saved, b.dh, b.dh_stride, f.tokens, f.d_ff, f.act, dg, du, l.f_stride);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    } else {
        TileArgs a{};
        if ((e = dual_args(f, d, m, &a)) != cudaSuccess) return e;
        a.job[0].out[0] = dg;
        a.job[0].out[1] = du;
        a.job[0].out_stride = l.f_stride;
        a.dh = b.dh;
        a.dh_stride = b.dh_stride;
        if ((e = run_tiles<kGates>(a, d, st)) != cudaSuccess) return e;
    }
    const Matrix grad[2] = {{dg, f.tokens, f.d_ff, l.f_stride}, {du, f.tokens, f.d_ff, l.f_stride}};
    const Shapes s = shapes_of(f, pairs_of(d));
    TileArgs a{};
    if (b.dx) {
        Job& j = a.job[kInput];
        set_shape(&j, s.input, f.tokens, f.d_model);
        j.batches = 1;
        j.out[0] = b.dx;
        j.out_stride = b.dx_stride;
        j.partial = reinterpret_cast<float*>(ws + l.input);
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
            e = encode(d, &j.a[i], grad[i], kStepK, kHalf);
            if (e == cudaSuccess) e = encode(d, &j.b[i], m[1 + i], 64, kStepK);
        }
    }
    uint16_t* dw[2] = {b.dw_gate, b.dw_up};
    if (dw[0] || dw[1]) {
        Job& j = a.job[kWeight];
        set_shape(&j, s.weight, f.d_ff, f.d_model);
        j.out_stride = f.d_model;
        j.partial = reinterpret_cast<float*>(ws + l.weight);
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
            if (!dw[i]) continue;
            j.out[j.batches] = dw[i];
            e = encode(d, &j.a[j.batches++], grad[i], 64, kStepK);
        }
        if (e == cudaSuccess) e = encode(d, &j.b[0], m[0], 64, kStepK);
    }
    // Both jobs in one launch fill the last rounds of one with the other's tiles
    // (1023 tokens, 1600 x 6400, backward with forward: 141 us apart, 127 us
    // together); with many rounds there is little to fill, and tiles of two jobs
    // at a time share less of L2 (8192 tokens, 4096 x 16384: 1 % slower together).
    const int64_t units = a.job[0].units() + a.job[1].units();
    if (units <= 16 * pairs_of(d)) {
        if (e == cudaSuccess) e = run_tiles<kProducts>(a, d, st);
    } else {
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
            TileArgs one = a;
            one.job[1 - i].batches = 0;
            if (one.job[i].batches) e = run_tiles<kProducts>(one, d, st);
        }
    }
    JoinArgs joins{};
    unsigned count = 0;
    int64_t rows = 0;
    for (const Job& j : a.job)
        for (int i = 0; i < j.batches && j.splits > 1; ++i) {
            joins.join[count++] = Join{j.partial + static_cast<int64_t>(i) * j.splits * j.M * j.N, j.out[i], j.M, j.N, j.out_stride,
                                       j.splits};
            rows = std::max(rows, j.M);
        }
    if (e == cudaSuccess && count) {
        join_kernel<<<dim3(rows_for(rows, d), count), 256, 0, st>>>(joins);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace q8
