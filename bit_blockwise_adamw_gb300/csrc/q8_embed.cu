// q8_embed.cu -- the token embedding: out[t] = scale * W[ids[t]], and the
// gradient of its table, dW[v] = scale * sum of dout[t] over the t with
// ids[t] = v (include/q8train.h).
//
// Neither does arithmetic worth counting: both are bound by the bytes of the
// rows that they move.
//
// The gradient takes three launches.
//  1. order_kernel.  One cluster of eight CTAs sorts the tokens by their id
//     (stable, so that a row's tokens keep their order: least significant digit
//     first, up to nine bits a pass, counts exchanged through the cluster's
//     shared memory), while all other CTAs write the zeros of the table's rows
//     that no token has.
//  2. sum_kernel.  The sorted tokens are cut into pieces of kPiece; a group of
//     warps adds up a piece's rows for its columns, in fp32 registers, and
//     writes a table row whenever the id changes.  An id of at most kPiece
//     tokens belongs to the piece that it begins in; longer ones (padding,
//     frequent words) are split at the pieces' ends, their parts left in the
//     workspace in fp32.
//  3. join_kernel adds up these parts, in their order.
// No result depends on which CTA comes first.
#include <algorithm>
#include <map>
#include <mutex>

#include "q8_device.cuh"
#include "q8_internal.h"
#include "q8_tc.cuh"
#include "q8_train.h"

namespace q8 {

namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = float_to_bf16(x); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// Eight elements of a row.
struct Eight {
    float2 x[4];
};

__device__ __forceinline__ uint32_t bf16_pair(float2 x)
{
    return static_cast<uint32_t>(float_to_bf16(x.x)) | static_cast<uint32_t>(float_to_bf16(x.y)) << 16;
}

__device__ __forceinline__ void write8(uint16_t* p, const Eight& v)
{
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v.x[0]), bf16_pair(v.x[1]), bf16_pair(v.x[2]), bf16_pair(v.x[3]));
}

__device__ __forceinline__ void write8(float* p, const Eight& v)
{
    reinterpret_cast<float4*>(p)[0] = make_float4(v.x[0].x, v.x[0].y, v.x[1].x, v.x[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(v.x[2].x, v.x[2].y, v.x[3].x, v.x[3].y);
}

// ----------------------------------------------------------------------- lookup

constexpr int kTile = 4;                       // vectors of a thread, all in flight

// Rows of whole 16-byte vectors: the output as one run of vectors, kTile *
// kRowThreads of them to a CTA at a time.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) lookup_kernel(q8_embedding e, const uint16_t* table, T* out, int64_t out_stride)
{
    const uint32_t width = static_cast<uint32_t>(e.dim / 8);
    const int64_t total = e.tokens * width;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kTile * kRowThreads); first < total;
         first += static_cast<int64_t>(gridDim.x) * (kTile * kRowThreads)) {
        const int64_t row0 = first / width;
        const uint32_t at = static_cast<uint32_t>(first - row0 * width) + threadIdx.x;
        uint4 w[kTile];
        T* to[kTile];
#pragma unroll
        for (int j = 0; j < kTile; ++j) {
            const uint32_t i = at + j * kRowThreads, r = i / width, c = (i - r * width) * 8;
            const int64_t t = row0 + r;
            to[j] = nullptr;
            w[j] = make_uint4(0, 0, 0, 0);
            if (t < e.tokens) {
                const int64_t id = e.ids[t];
                to[j] = out + t * out_stride + c;
                if (id >= 0 && id < e.vocab) w[j] = *reinterpret_cast<const uint4*>(table + id * e.dim + c);
            }
        }
#pragma unroll
        for (int j = 0; j < kTile; ++j) {
            if (!to[j]) continue;
            Eight v{{bf16x2(w[j].x), bf16x2(w[j].y), bf16x2(w[j].z), bf16x2(w[j].w)}};
#pragma unroll
            for (int k = 0; k < 4; ++k) v.x[k] = __fmul2_rn(v.x[k], splat(e.scale));
            write8(to[j], v);
        }
    }
}

// Other rows, element by element: a warp for 256 columns of one row.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) lookup_odd_kernel(q8_embedding e, const uint16_t* table, T* out, int64_t out_stride)
{
    const int lane = threadIdx.x % 32;
    const int64_t parts = (e.dim + 255) / 256, total = e.tokens * parts;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + threadIdx.x / 32; i < total;
         i += static_cast<int64_t>(gridDim.x) * (kRowThreads / 32)) {
        const int64_t t = i / parts, id = e.ids[t];
        const bool known = id >= 0 && id < e.vocab;
        const int64_t c0 = (i - t * parts) * 256 + lane;
        const uint16_t* row = table + (known ? id : 0) * e.dim;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = known && c0 + j * 32 < e.dim ? load1(row + c0 + j * 32) : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c0 + j * 32 < e.dim) store1(out + t * out_stride + c0 + j * 32, known ? __fmul_rn(e.scale, x[j]) : 0.0f);
    }
}

// ---------------------------------------------------------------------- gradient

constexpr int kPiece = 32;
constexpr int kCluster = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kItems = 8;                      // tokens of a thread in one tile of the sort
constexpr int kSortShared = kSortWarps * kBins * 4;
constexpr int kMapBits = kSortShared * 8;      // rows that a filling CTA's bitmap holds

// The workspace.
struct Room {
    uint64_t* sorted;          // [tokens]: id << 32 | token, ids outside the table as vocab
    uint64_t* other;           // the sort's second buffer
    int32_t* count;            // ids whose parts are to be joined
    int32_t* list;             // [pieces]: the piece that each of them begins in
    float* parts;              // [pieces][2][columns]: of an id from before the piece; of one that goes on behind it
    int64_t columns;           // dim, to whole vectors
    int64_t bytes;
};

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

Room room_of(const q8_embedding& e, void* workspace)
{
    const int64_t pieces = round_up(e.tokens, kPiece) / kPiece;
    char* p = static_cast<char*>(workspace);
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        char* q = p + at;
        at += round_up(bytes, 256);
        return q;
    };
    Room r{};
    r.columns = round_up(e.dim, 8);
    r.sorted = reinterpret_cast<uint64_t*>(take(e.tokens * 8));
    r.other = reinterpret_cast<uint64_t*>(take(e.tokens * 8));
    r.count = reinterpret_cast<int32_t*>(take(4));
    r.list = reinterpret_cast<int32_t*>(take(pieces * 4));
    r.parts = reinterpret_cast<float*>(take(pieces * 2 * r.columns * 4));
    r.bytes = at;
    return r;
}

struct OrderArgs {
    q8_embedding e;
    Room r;
    uint16_t* dtable;
    int32_t passes, digit;     // of the sort: passes, bits of each
    int32_t fill;              // 0: nothing; 1: all rows; 2: rows that no token has
};

__device__ __forceinline__ uint32_t cluster_read(const uint32_t* p, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(smem_addr(p), rank)) : "memory");
    return v;
}

// One CTA's part of the sort: the tokens [lo, hi) of each pass's order.
__device__ void sort_tokens(const OrderArgs& a, uint32_t (*counts)[kBins])
{
    __shared__ uint32_t hist[kBins], base[kBins], sums[kSortWarps];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const uint32_t rank = cluster_rank();
    const int64_t T = a.e.tokens;
    const int64_t lo = T * rank / kCluster, hi = T * (rank + 1) / kCluster;
    const int items = static_cast<int>(max(int64_t(1), min(int64_t(kItems), (hi - lo + kSortThreads - 1) / kSortThreads)));
    const int bins = 1 << a.digit;
    if (rank == 0 && tid == 0) *a.r.count = 0;
    for (int pass = 0; pass < a.passes; ++pass) {
        const uint64_t* from = (a.passes - pass) % 2 ? a.r.other : a.r.sorted;
        uint64_t* to = (a.passes - pass) % 2 ? a.r.sorted : a.r.other;
        const int shift = 32 + pass * a.digit;
        const auto token = [&](int64_t i) {
            if (pass > 0) return __ldcg(reinterpret_cast<const unsigned long long*>(from) + i);
            const int64_t id = a.e.ids[i];
            const uint32_t key = static_cast<uint32_t>(id >= 0 && id < a.e.vocab ? id : a.e.vocab);
            return static_cast<unsigned long long>(key) << 32 | static_cast<uint32_t>(i);
        };
        for (int d = tid; d < bins; d += kSortThreads) hist[d] = 0;
        __syncthreads();
        for (int64_t i0 = lo + warp * 32; i0 < hi; i0 += kSortThreads) {
            const bool on = i0 + lane < hi;
            const uint32_t d = on ? static_cast<uint32_t>(token(i0 + lane) >> shift) & (bins - 1) : ~0u;
            const uint32_t same = __match_any_sync(~0u, d);
            if (on && lane == __ffs(same) - 1) atomicAdd(&hist[d], __popc(same));
        }
        cluster_sync();
        // a digit's first place: all smaller digits, and its own in the CTAs before
        uint32_t all = 0, before = 0;
        if (tid < bins)
            for (uint32_t c = 0; c < kCluster; ++c) {
                const uint32_t h = cluster_read(&hist[tid], c);
                all += h;
                before += c < rank ? h : 0;
            }
        uint32_t sum = all;
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t s = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += s;
        }
        if (lane == 31) sums[warp] = sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) sum += sums[w];
        if (tid < bins) base[tid] = sum - all + before;
        for (int64_t tile = lo; tile < hi; tile += kSortThreads * items) {
            __syncwarp();                      // its lanes have read their places of the tile before
            for (int d = lane; d < bins; d += 32) counts[warp][d] = 0;
            __syncwarp();
            uint64_t x[kItems];
            uint32_t place[kItems];
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                const int64_t i = tile + (warp * items + j) * 32 + lane;
                x[j] = j < items && i < hi ? token(i) : ~uint64_t(0);
            }
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                if (j >= items) break;
                const bool on = tile + (warp * items + j) * 32 + lane < hi;
                const uint32_t d = on ? static_cast<uint32_t>(x[j] >> shift) & (bins - 1) : ~0u;
                const uint32_t same = __match_any_sync(~0u, d);
                const uint32_t seen = on ? counts[warp][d] : 0;
                place[j] = seen + __popc(same & ((1u << lane) - 1));
                __syncwarp();
                if (on && lane == __ffs(same) - 1) counts[warp][d] = seen + __popc(same);
                __syncwarp();
            }
            __syncthreads();
            if (tid < bins) {
                uint32_t at = base[tid];
                for (int w = 0; w < kSortWarps; ++w) {
                    const uint32_t n = counts[w][tid];
                    counts[w][tid] = at;
                    at += n;
                }
                base[tid] = at;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                if (j >= items) break;
                if (tile + (warp * items + j) * 32 + lane < hi)
                    to[counts[warp][static_cast<uint32_t>(x[j] >> shift) & (bins - 1)] + place[j]] = x[j];
            }
        }
        cluster_sync();                        // what all CTAs wrote is there, and their counts are read
    }
}

// Zeros, one warp: any 2-byte aligned range.
__device__ __forceinline__ void zero_run(uint16_t* p, int64_t n, int lane)
{
    const int64_t lead = min(n, static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / 2));
    const int64_t vecs = (n - lead) / 8;
    if (lane < lead) p[lane] = 0;
    uint4* q = reinterpret_cast<uint4*>(p + lead);
#pragma unroll 4
    for (int64_t i = lane; i < vecs; i += 32) q[i] = make_uint4(0, 0, 0, 0);
    if (lead + vecs * 8 + lane < n) p[lead + vecs * 8 + lane] = 0;
}

// One CTA's part of the zeros.
__device__ void fill_rows(const OrderArgs& a, uint32_t* map, int64_t cta, int64_t ctas)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t begin = a.e.vocab * cta / ctas, end = a.e.vocab * (cta + 1) / ctas;
    if (a.fill == 1) {                         // in runs of 8192 elements, a warp each
        const int64_t n = (end - begin) * a.e.dim;
        for (int64_t i = warp * int64_t(8192); i < n; i += kSortWarps * int64_t(8192))
            zero_run(a.dtable + begin * a.e.dim + i, min(int64_t(8192), n - i), lane);
        return;
    }
    for (int64_t first = begin; first < end; first += kMapBits) {
        const int64_t rows = min(int64_t(kMapBits), end - first);
        for (int64_t i = threadIdx.x; i < (rows + 31) / 32; i += kSortThreads) map[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int64_t t = threadIdx.x; t < a.e.tokens; t += kSortThreads) {
            const uint64_t r = static_cast<uint64_t>(a.e.ids[t]) - static_cast<uint64_t>(first);
            if (r < static_cast<uint64_t>(rows)) atomicOr(&map[r / 32], 1u << (r % 32));
        }
        __syncthreads();
        for (int64_t r = warp; r < rows; r += kSortWarps)
            if (!(map[r / 32] >> (r % 32) & 1)) zero_run(a.dtable + (first + r) * a.e.dim, a.e.dim, lane);
        __syncthreads();
    }
}

__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__global__ void __launch_bounds__(kSortThreads) order_kernel(const __grid_constant__ OrderArgs a)
{
    extern __shared__ __align__(16) uint32_t shared[];
    let_next_start();
    if (blockIdx.x < kCluster) sort_tokens(a, reinterpret_cast<uint32_t(*)[kBins]>(shared));
    else fill_rows(a, shared, blockIdx.x - kCluster, gridDim.x - kCluster);
}

struct SumArgs {
    q8_embedding e;
    Room r;
    const void* dout;
    int64_t stride;
    uint16_t* dtable;
    int32_t accumulate;
    int32_t group;             // threads that share a piece's columns
};

__device__ __forceinline__ uint32_t key_of(uint64_t x) { return static_cast<uint32_t>(x >> 32); }

// How an id lies across the start p of a piece (p is not the first): `before`
// of its tokens come before p and `from` from p on, each counted to kPiece.
struct Cut {
    uint32_t key;
    int before, from;

    __device__ __forceinline__ bool crosses() const { return before > 0; }
    __device__ __forceinline__ bool is_long() const { return before + from > kPiece; }
};

__device__ __forceinline__ Cut cut_at(const uint64_t* sorted, int64_t T, int64_t p, int lane)
{
    static_assert(kPiece == 32, "a lane for each token");
    Cut c;
    c.key = key_of(__ldcg(reinterpret_cast<const unsigned long long*>(sorted) + p));
    const uint32_t back = p - 1 - lane >= 0 ? key_of(__ldcg(reinterpret_cast<const unsigned long long*>(sorted) + p - 1 - lane)) : ~0u;
    const uint32_t forth = p + lane < T ? key_of(__ldcg(reinterpret_cast<const unsigned long long*>(sorted) + p + lane)) : ~0u;
    const uint32_t b = ~__ballot_sync(~0u, back == c.key), f = ~__ballot_sync(~0u, forth == c.key);
    c.before = b ? __ffs(b) - 1 : 32;
    c.from = f ? __ffs(f) - 1 : 32;
    return c;
}

// A thread's eight columns: VEC, contiguous; else every step-th.  What was read
// of a row stays as it lies in memory until it is added.
template <bool VEC>
struct Columns {
    int64_t first, dim;
    int step;

    template <typename T>
    struct Raw {
        uint4 w[VEC ? sizeof(T) / 2 : 1];
        T x[VEC ? 1 : 8];
    };

    template <typename T>
    __device__ __forceinline__ void read(Raw<T>& r, const T* row) const
    {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(row + first)[i];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r.x[j] = first + j * step < dim ? row[first + j * step] : T(0);
        }
    }
    template <typename T>
    __device__ __forceinline__ static float2 pair(const Raw<T>& r, int k)
    {
        if constexpr (!VEC) {
            return make_float2(load1(&r.x[2 * k]), load1(&r.x[2 * k + 1]));
        } else if constexpr (sizeof(T) == 2) {
            return bf16x2(k == 0 ? r.w[0].x : k == 1 ? r.w[0].y : k == 2 ? r.w[0].z : r.w[0].w);
        } else {
            const uint4& v = r.w[k / 2];
            return k % 2 ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w)) : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        }
    }
    template <typename T>
    __device__ __forceinline__ void write(T* row, const Eight& v) const
    {
        if constexpr (VEC) {
            write8(row + first, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (first + j * step < dim) store1(row + first + j * step, j % 2 ? v.x[j / 2].y : v.x[j / 2].x);
        }
    }
};

// scale * sum, or with accumulate that added to what the row holds.
template <bool VEC>
__device__ __forceinline__ void write_row(const Columns<VEC>& c, uint16_t* row, Eight sum, float scale, bool accumulate)
{
    if (accumulate) {
        typename Columns<VEC>::template Raw<uint16_t> old;
        c.read(old, static_cast<const uint16_t*>(row));
#pragma unroll
        for (int k = 0; k < 4; ++k) sum.x[k] = __ffma2_rn(sum.x[k], splat(scale), c.pair(old, k));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) sum.x[k] = __fmul2_rn(sum.x[k], splat(scale));
    }
    c.write(row, sum);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) sum_kernel(const __grid_constant__ SumArgs a)
{
    constexpr int kAhead = sizeof(T) == 2 && VEC ? 8 : 4;  // rows in flight: 32 registers
    let_next_start();
    wait_for_previous();
    const int lane = threadIdx.x % 32;
    const int64_t N = a.e.tokens, pieces = (N + kPiece - 1) / kPiece;
    const int64_t piece = static_cast<int64_t>(blockIdx.x) * (kRowThreads / a.group) + threadIdx.x / a.group;
    if (piece >= pieces) return;
    const uint64_t* sorted = a.r.sorted;
    const int64_t p0 = piece * kPiece, p1 = min(N, p0 + kPiece);
    int64_t begin = p0, end = p1;
    bool from_before = false, goes_on = false;             // parts of a long id
    if (p0 > 0) {
        const Cut c = cut_at(sorted, N, p0, lane);
        from_before = c.crosses() && c.is_long();
        if (c.crosses() && !from_before) begin += c.from;
    }
    if (p1 < N) {
        const Cut c = cut_at(sorted, N, p1, lane);
        goes_on = c.crosses() && c.is_long() && c.key < a.e.vocab;
        if (c.crosses() && !c.is_long()) end += c.from;
    }
    // the piece's tokens (at most 63), one or two to a lane
    const uint64_t none = static_cast<uint64_t>(a.e.vocab) << 32;
    const uint64_t e0 = begin + lane < end ? __ldcg(reinterpret_cast<const unsigned long long*>(sorted) + begin + lane) : none;
    const uint64_t e1 = begin + 32 + lane < end ? __ldcg(reinterpret_cast<const unsigned long long*>(sorted) + begin + 32 + lane) : none;
    const uint32_t vocab = static_cast<uint32_t>(a.e.vocab);
    const int count = __popc(__ballot_sync(~0u, key_of(e0) < vocab)) + __popc(__ballot_sync(~0u, key_of(e1) < vocab));
    if (count == 0) return;                                // tokens outside the table come last
    const auto entry = [&](int i) { return __shfl_sync(~0u, i < 32 ? e0 : e1, i % 32); };
    const uint32_t first_key = key_of(entry(0)), last_key = key_of(entry(count - 1));
    const T* dout = static_cast<const T*>(a.dout);
    const int64_t width = 8 * static_cast<int64_t>(a.group);
    for (int64_t c0 = blockIdx.y * width; c0 < a.e.dim; c0 += gridDim.y * width) {
        const int tid = threadIdx.x % a.group;
        const Columns<VEC> cols{VEC ? c0 + tid * 8 : c0 + tid, a.e.dim, a.group};
        const bool on = cols.first < a.e.dim;
        Eight sum{};
        uint32_t key = first_key;
        const auto finish = [&](bool last) {               // the sum of `key` is complete, as far as this piece goes
            if (!on) return;
            if (key == first_key && from_before) cols.write(a.r.parts + (piece * 2) * a.r.columns, sum);
            else if (last && key == last_key && goes_on) cols.write(a.r.parts + (piece * 2 + 1) * a.r.columns, sum);
            else write_row(cols, a.dtable + static_cast<int64_t>(key) * a.e.dim, sum, a.e.scale, a.accumulate);
        };
        for (int i = 0; i < count; i += kAhead) {
            typename Columns<VEC>::template Raw<T> v[kAhead];
            uint32_t keys[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const uint64_t x = entry(min(i + j, count - 1));
                keys[j] = key_of(x);
                if (on && i + j < count) cols.read(v[j], dout + static_cast<int64_t>(static_cast<uint32_t>(x)) * a.stride);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (i + j >= count) break;
                if (keys[j] != key) {
                    finish(false);
                    key = keys[j];
                    sum = Eight{};
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) sum.x[k] = __fadd2_rn(sum.x[k], cols.pair(v[j], k));
            }
        }
        finish(true);
    }
    if (goes_on && !(first_key == last_key && from_before) && blockIdx.y == 0 && threadIdx.x % a.group == 0)
        a.r.list[atomicAdd(a.r.count, 1)] = static_cast<int32_t>(piece);
}

// A CTA for 128 columns of one id: warps take its parts in turn.
constexpr int kJoinColumns = 128;

__global__ void __launch_bounds__(kRowThreads) join_kernel(const __grid_constant__ SumArgs a)
{
    constexpr int kWarps = kRowThreads / 32;
    __shared__ float4 sums[kWarps][kJoinColumns / 4];
    wait_for_previous();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t N = a.e.tokens, pieces = (N + kPiece - 1) / kPiece;
    const int64_t tiles = (a.e.dim + kJoinColumns - 1) / kJoinColumns, total = *a.r.count * tiles;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int64_t piece = a.r.list[i / tiles];
        const int64_t c0 = (i % tiles) * kJoinColumns;
        const uint32_t key = key_of(a.r.sorted[(piece + 1) * kPiece]);
        // the first piece behind it that does not begin with the id: 32 places at a time
        int64_t lo = piece + 2, hi = pieces;
        while (lo < hi) {
            const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
            const uint32_t less = __ballot_sync(~0u, at < hi && key_of(a.r.sorted[at * kPiece]) == key);
            const int n = __popc(less);                    // ones, then zeros
            if (n == 0) break;
            hi = min(hi, lo + n * step);
            lo += (n - 1) * step + 1;
        }
        const int64_t parts = lo - piece;                  // its own, and one of each piece behind it
        const int64_t c = c0 + lane * 4;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < a.r.columns) {
#pragma unroll 4
            for (int64_t q = warp; q < parts; q += kWarps) {
                const float4 x = *reinterpret_cast<const float4*>(a.r.parts + ((piece + q) * 2 + (q == 0)) * a.r.columns + c);
                sum = make_float4(__fadd_rn(sum.x, x.x), __fadd_rn(sum.y, x.y), __fadd_rn(sum.z, x.z), __fadd_rn(sum.w, x.w));
            }
        }
        sums[warp][lane] = sum;
        __syncthreads();
        if (threadIdx.x < kJoinColumns && c0 + threadIdx.x < a.e.dim) {
            float x = 0.0f;
            for (int w = 0; w < kWarps; ++w) x = __fadd_rn(x, reinterpret_cast<const float*>(sums[w])[threadIdx.x]);
            uint16_t* to = a.dtable + static_cast<int64_t>(key) * a.e.dim + c0 + threadIdx.x;
            store1(to, a.accumulate ? __fmaf_rn(a.e.scale, x, load1(to)) : __fmul_rn(a.e.scale, x));
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------- host

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T>
cudaError_t lookup(const q8_embedding& e, const uint16_t* table, void* out, int64_t out_stride, cudaStream_t st)
{
    constexpr int64_t kMost = 1 << 20;
    if (e.dim % 8 == 0 && on16(table) && on16(out) && (e.tokens == 1 || out_stride * sizeof(T) % 16 == 0)) {
        const int64_t tiles = (e.tokens * (e.dim / 8) + kTile * kRowThreads - 1) / (kTile * kRowThreads);
        lookup_kernel<T><<<static_cast<int>(std::min(kMost, tiles)), kRowThreads, 0, st>>>(e, table, static_cast<T*>(out), out_stride);
    } else {
        const int64_t warps = e.tokens * ((e.dim + 255) / 256);
        lookup_odd_kernel<T><<<static_cast<int>(std::min(kMost, (warps + 7) / 8)), kRowThreads, 0, st>>>(e, table, static_cast<T*>(out), out_stride);
    }
    return cudaGetLastError();
}

cudaLaunchConfig_t order_config(cudaLaunchAttribute* attr, int ctas, cudaStream_t st)
{
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim = {kCluster, 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortShared;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

std::mutex g_lock;
std::map<int, int> g_clusters;                 // clusters of order_kernel that a device runs at once

cudaError_t clusters_at_once(int* out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_lock);
    int& n = g_clusters[dev];
    if (n == 0) {
        cudaLaunchAttribute attr{};
        const cudaLaunchConfig_t cfg = order_config(&attr, kCluster, nullptr);
        const void* k = reinterpret_cast<const void*>(order_kernel);
        int found = 0;
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortShared)) != cudaSuccess) return e;
        if ((e = cudaOccupancyMaxActiveClusters(&found, k, &cfg)) != cudaSuccess) return e;
        if (found <= 0) return cudaErrorInvalidConfiguration;
        n = found;
    }
    *out = n;
    return cudaSuccess;
}

// The kernel after another one of the same call (wait_for_previous).
cudaError_t launch_after(void (*kernel)(SumArgs), dim3 grid, cudaStream_t st, const SumArgs& a)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t prepare_embed()
{
    int n = 0;
    cudaError_t e = clusters_at_once(&n);
    return e == cudaSuccess ? persistent_grid(reinterpret_cast<const void*>(join_kernel), kRowThreads, 0, &n) : e;
}

cudaError_t launch_embed_forward(const q8_embedding& e, const uint16_t* table, void* out, int64_t out_stride, cudaStream_t st)
{
    return e.dtype == Q8_F32 ? lookup<float>(e, table, out, out_stride, st) : lookup<uint16_t>(e, table, out, out_stride, st);
}

int64_t embed_workspace(const q8_embedding& e) { return e.tokens == 0 ? 0 : room_of(e, nullptr).bytes; }

cudaError_t launch_embed_backward(const q8_embedding& e, const void* dout, int64_t dout_stride, uint16_t* dtable,
                                  bool accumulate, void* workspace, cudaStream_t st)
{
    int clusters = 0, joins = 0;
    cudaError_t err = clusters_at_once(&clusters);
    if (err == cudaSuccess) err = persistent_grid(reinterpret_cast<const void*>(join_kernel), kRowThreads, 0, &joins);
    if (err != cudaSuccess) return err;
    const Room room = room_of(e, workspace);

    OrderArgs o{};
    o.e = e;
    o.r = room;
    o.dtable = dtable;
    int bits = 1;
    while (e.vocab >> bits) ++bits;            // vocab itself is the key of ids outside the table
    o.passes = (bits + kDigitBits - 1) / kDigitBits;
    o.digit = (bits + o.passes - 1) / o.passes;
    o.fill = accumulate ? 0 : 2;
    const int ctas = accumulate ? kCluster : std::max(2, clusters) * kCluster;
    cudaLaunchAttribute attr{};
    const cudaLaunchConfig_t cfg = order_config(&attr, ctas, st);
    if ((err = cudaLaunchKernelEx(&cfg, order_kernel, o)) != cudaSuccess) return err;

    SumArgs s{};
    s.e = e;
    s.r = room;
    s.dout = dout;
    s.stride = dout_stride;
    s.dtable = dtable;
    s.accumulate = accumulate;
    s.group = 32;
    while (s.group < kRowThreads && s.group * 8 < e.dim) s.group *= 2;
    const int size = e.dtype == Q8_F32 ? 4 : 2;
    const bool vec = e.dim % 8 == 0 && on16(dtable) && on16(dout) && (e.tokens == 1 || dout_stride * size % 16 == 0);
    const int64_t pieces = (e.tokens + kPiece - 1) / kPiece, each = kRowThreads / s.group;
    const dim3 grid(static_cast<unsigned>((pieces + each - 1) / each),
                    static_cast<unsigned>(std::min<int64_t>((e.dim + s.group * 8 - 1) / (s.group * 8), 65535)));
    const auto sum = size == 4 ? (vec ? sum_kernel<float, true> : sum_kernel<float, false>)
                               : (vec ? sum_kernel<uint16_t, true> : sum_kernel<uint16_t, false>);
    if ((err = launch_after(sum, grid, st, s)) != cudaSuccess) return err;
    return launch_after(join_kernel, dim3(static_cast<unsigned>(joins)), st, s);
}

}  // namespace q8
