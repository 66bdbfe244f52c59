// q8_embed.cu -- the token embedding: out[t] = scale * W[ids[t]], and the
// gradient of its table, dW[v] = scale * sum of dout[t] over the t with
// ids[t] = v (include/q8train.h).
//
// Neither does arithmetic worth counting: both are bound by the bytes of the
// rows that they move.
//
// Up to 256 tokens take one launch (few_kernel).  More take three.
//  1. rank_kernel, up to 4096 tokens and 64 MB of zeros: each token's place is the
//     number of those before it by id and order, counted by comparing it with all
//     of them; other CTAs write the zeros of the table's rows that no token has.
//     Elsewhere, order_kernel.  One cluster of eight CTAs sorts the tokens by their id
//     (stable, so that a row's tokens keep their order: least significant digit
//     first, up to nine bits a pass, counts exchanged through the cluster's
//     shared memory), the other CTAs writing zeros.
//  2. sum_kernel.  The sorted tokens are cut into pieces of 8 or 32; a group of
//     warps adds up a piece's rows for its columns, in fp32 registers, and
//     writes a table row whenever the id changes.  An id of no more tokens than
//     a piece has belongs to the piece that it begins in; longer ones (padding,
//     frequent words) are split at the pieces' ends, their parts left in the
//     workspace in fp32.  Further CTAs write the other zeros.
//  3. join_kernel adds up these parts, in their order.
// More than 32768 tokens are sorted by all SMs, in two launches a pass
// (count_kernel, place_kernel), and the zeros are then written behind the joins, by
// CTAs of their launch that start as those that join come to their end.
// No result depends on which CTA comes first.
//
// Measured, bf16, a vocabulary of 50257, tokens as frequent as words are: lookup
// of 16384 x 4096 32 us (5.8 TB/s), of one row 1.8 us.  Gradient of 16384 x 4096
// 94 us (546 MB that it cannot do without: 5.8 TB/s), of 262144 x 1024 of which
// half are padding 150 us (sort 27, sums 100, joins 23), of 24 x 2560 38.3 us (all
// of it the table's zeros: 6.7 TB/s).
#include <algorithm>
#include <limits>
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

__device__ __forceinline__ uint4 vector_of(const Eight& v)
{
    return make_uint4(bf16_pair(v.x[0]), bf16_pair(v.x[1]), bf16_pair(v.x[2]), bf16_pair(v.x[3]));
}

__device__ __forceinline__ void write8(uint16_t* p, const Eight& v) { *reinterpret_cast<uint4*>(p) = vector_of(v); }

__device__ __forceinline__ void write8(float* p, const Eight& v)
{
    reinterpret_cast<float4*>(p)[0] = make_float4(v.x[0].x, v.x[0].y, v.x[1].x, v.x[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(v.x[2].x, v.x[2].y, v.x[3].x, v.x[3].y);
}

// The same, of which L2 need not keep anything.
__device__ __forceinline__ void stream8(uint16_t* p, const Eight& v) { __stcs(reinterpret_cast<uint4*>(p), vector_of(v)); }

__device__ __forceinline__ void stream8(float* p, const Eight& v)
{
    __stcs(reinterpret_cast<float4*>(p), make_float4(v.x[0].x, v.x[0].y, v.x[1].x, v.x[1].y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v.x[2].x, v.x[2].y, v.x[3].x, v.x[3].y));
}

// ----------------------------------------------------------------------- lookup

constexpr int64_t kStreamBytes = 64 << 20;     // half of L2
constexpr int kTile = 4;                       // vectors of a thread, all in flight

// Rows of whole 16-byte vectors: the output as one run of vectors, kTile *
// kRowThreads of them to a CTA at a time.  STREAM: an output that L2 would not
// hold for its reader leaves L2 to the table's rows (16384 x 4096: 31.9 us,
// else 34.3).
template <typename T, bool STREAM>
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
            if (STREAM) stream8(to[j], v);
            else write8(to[j], v);
        }
    }
}

// Eight bf16 elements, `off` bytes into two 16-byte vectors.
__device__ __forceinline__ Eight values_across(uint4 a, uint4 b, uint32_t off)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8)
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    if (off & 4)
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    if (off & 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __byte_perm(w[i], w[i + 1], 0x5432);
    return Eight{{bf16x2(w[0]), bf16x2(w[1]), bf16x2(w[2]), bf16x2(w[3])}};
}

// Other rows: `group` threads for each, in vectors that start on 16 bytes of the
// output and lie in two of the table's; a row's first and last elements one by
// one.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) lookup_odd_kernel(q8_embedding e, const uint16_t* table, T* out, int64_t out_stride, int group)
{
    constexpr int kPair = 2;                   // vectors of a thread in flight
    const int x = threadIdx.x % group, rows = kRowThreads / group;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / group; t < e.tokens; t += static_cast<int64_t>(gridDim.x) * rows) {
        const int64_t id = e.ids[t];
        const bool known = id >= 0 && id < e.vocab;
        const bool inside = id > 0 && id < e.vocab - 1;    // neighbours on both sides: whole vectors may be read
        T* to = out + t * out_stride;
        const uint16_t* row = table + (known ? id : 0) * e.dim;
        const int64_t lead = min(e.dim, static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(to) % 16) % 16 / sizeof(T)));
        const int64_t vectors = (e.dim - lead) / 8, tail = lead + vectors * 8 + x;
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + lead) % 16);
        const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row + lead) - off);
        for (int64_t v0 = x; v0 < vectors; v0 += kPair * group) {
            uint4 a[kPair], b[kPair];
#pragma unroll
            for (int j = 0; j < kPair; ++j) {
                const int64_t v = v0 + j * group;
                a[j] = b[j] = make_uint4(0, 0, 0, 0);
                if (v < vectors && inside) {
                    a[j] = from[v];
                    if (off) b[j] = from[v + 1];
                } else if (v < vectors && known) {
                    uint16_t w[16] = {};
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[k] = row[lead + v * 8 + k];
                    a[j] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
                }
            }
#pragma unroll
            for (int j = 0; j < kPair; ++j) {
                const int64_t v = v0 + j * group;
                if (v >= vectors) break;
                Eight y = values_across(a[j], b[j], inside ? off : 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) y.x[k] = __fmul2_rn(y.x[k], splat(e.scale));
                write8(to + lead + v * 8, y);
            }
        }
        if (x < lead) store1(to + x, known ? __fmul_rn(e.scale, load1(row + x)) : 0.0f);
        if (tail < e.dim) store1(to + tail, known ? __fmul_rn(e.scale, load1(row + tail)) : 0.0f);
    }
}

// ---------------------------------------------------------------------- gradient

constexpr int kFewParts = 32;                  // (8: 262144 x 1024 178 us instead of 164)
// Sorted by one cluster, at most (a cluster / all SMs, with rows of 256: 16384
// tokens 24 / 31 us, 32768 31 / 33, 49152 40 / 36, 65536 50 / 38).
constexpr int64_t kClusterTokens = 32768;
constexpr int kMaxSorters = 128;               // CTAs that sort more of them (152 or 96: 2 us more at 262144)
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
    int32_t* count;            // [2]: ids whose parts are to be joined, of few parts and of many
    uint8_t* present;          // [vocab]: 1 where a token has the row
    uint32_t* digits;          // [SMs][kBins]: the sort's counts, of more than kClusterTokens
    int2* list;                // [2][pieces]: the piece that each of them begins in, and its parts
    float* parts;              // [pieces][2][columns]: of an id from before the piece; of one that goes on behind it
    int64_t columns;           // dim, to whole vectors
    int64_t pieces;
    int32_t piece;             // tokens of one
    int64_t bytes;
};

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Threads that share a piece's columns, eight columns each.
int group_of(const q8_embedding& e)
{
    int group = 32;
    while (group < kRowThreads && group * int64_t(8) < e.dim) group *= 2;
    return group;
}

// Pieces of 32, or of 8 where 32 would leave half of the GPU's 152 SMs with
// less than four groups of 256 threads: a piece's rows are added one after the
// other, and few tokens then wait for that (added to their rows, 8 / 32: 1024 x
// 1024 17 / 28 us, 8192 x 1024 25 / 30, 4096 x 4096 28 / 32, 8192 x 4096 48 / 45,
// 16384 x 4096 80 / 74).
constexpr int64_t kFewThreads = 152 / 2 * 4 * 256;

Room room_of(const q8_embedding& e, void* workspace)
{
    const int64_t group = group_of(e), threads = round_up(e.tokens, 32) / 32 * group * ((e.dim + group * 8 - 1) / (group * 8));
    const int piece = threads < kFewThreads ? 8 : 32;
    const int64_t pieces = round_up(e.tokens, piece) / piece;
    char* p = static_cast<char*>(workspace);
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        char* q = p + at;
        at += round_up(bytes, 256);
        return q;
    };
    Room r{};
    r.piece = piece;
    r.pieces = pieces;
    r.columns = round_up(e.dim, 8);
    r.sorted = reinterpret_cast<uint64_t*>(take(e.tokens * 8));
    r.other = reinterpret_cast<uint64_t*>(take(e.tokens * 8));
    r.count = reinterpret_cast<int32_t*>(take(8));
    r.present = reinterpret_cast<uint8_t*>(take(e.vocab));
    if (e.tokens > kClusterTokens) r.digits = reinterpret_cast<uint32_t*>(take(kMaxSorters * kBins * 4));
    r.list = reinterpret_cast<int2*>(take(2 * pieces * 8));
    r.parts = reinterpret_cast<float*>(take(pieces * 2 * r.columns * 4));
    r.bytes = at;
    return r;
}

struct OrderArgs {
    q8_embedding e;
    Room r;
    uint16_t* dtable;
    int32_t passes, digit;     // of the sort: passes, bits of each
    int32_t pass;              // count_kernel, place_kernel: the one at hand
    int32_t clear, note;       // r.present is cleared; the sort notes there what it meets
    int64_t fill;              // the table's rows [0, fill) get their zeros here
    int64_t fill_rows;         // rank_kernel: so many to a CTA
};

__device__ __forceinline__ uint32_t cluster_read(const uint32_t* p, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(smem_addr(p), rank)) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t key_of(uint64_t x) { return static_cast<uint32_t>(x >> 32); }

// The warp's lanes that have this lane's digit (of `bits` bits), among those that
// are on: a ballot for each bit.  __match_any_sync took four times as long.
__device__ __forceinline__ uint32_t same_digit(uint32_t d, bool on, int bits)
{
    uint32_t same = __ballot_sync(~0u, on);
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
        if (b >= bits) break;
        const uint32_t set = __ballot_sync(~0u, d >> b & 1);
        same &= d >> b & 1 ? set : ~set;
    }
    return same;
}

// One pass of the sort, as one CTA sees it: it owns the tokens [lo, hi) of the
// order that the pass before left (before the first, that of the ids), takes
// them in tiles, a warp `items` times 32 consecutive ones, and puts each behind
// those of its digit that came before.
struct Pass {
    uint8_t* present;          // of the first pass: the rows that it meets are noted here
    const int64_t* ids;        // of the first pass
    const uint64_t* from;      // of the others
    uint64_t* to;
    int64_t vocab, lo, hi;
    int shift, bits, items;
    uint64_t x[kItems];
    uint32_t place[kItems];

    __device__ __forceinline__ int64_t tile() const { return static_cast<int64_t>(kSortThreads) * items; }

    __device__ __forceinline__ void load(int64_t at)
    {
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int64_t i = at + (threadIdx.x / 32 * items + j) * 32 + threadIdx.x % 32;
            if (j >= items || i >= hi) continue;
            if (!ids) {
                x[j] = __ldcg(reinterpret_cast<const unsigned long long*>(from) + i);
            } else {
                const int64_t id = ids[i];
                const uint32_t key = static_cast<uint32_t>(id >= 0 && id < vocab ? id : vocab);
                x[j] = static_cast<uint64_t>(key) << 32 | static_cast<uint32_t>(i);
            }
        }
    }
    __device__ __forceinline__ uint32_t digit(int64_t at, int j) const
    {
        const int64_t i = at + (threadIdx.x / 32 * items + j) * 32 + threadIdx.x % 32;
        return i < hi ? static_cast<uint32_t>(x[j] >> shift) & ((1u << bits) - 1) : ~0u;
    }
    // Each token's place among its warp's of the same digit, and the warp's counts.
    __device__ __forceinline__ void rank(int64_t at, uint32_t (*counts)[kBins])
    {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        __syncwarp();                          // its lanes have read their places of the tile before
        for (int d = lane; d < 1 << bits; d += 32) counts[warp][d] = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            if (j >= items) break;
            const uint32_t d = digit(at, j), same = same_digit(d, d != ~0u, bits);
            const uint32_t seen = d != ~0u ? counts[warp][d] : 0;
            place[j] = seen + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (d != ~0u && lane == __ffs(same) - 1) counts[warp][d] = seen + __popc(same);
            __syncwarp();
        }
        __syncthreads();
    }
    // The CTA's counts, to thread d < 2^bits those of digit d; its tokens, if
    // they are one tile, ranked.
    __device__ __forceinline__ uint32_t count(uint32_t (*counts)[kBins], uint32_t* hist)
    {
        const int tid = threadIdx.x, bins = 1 << bits;
        if (hi - lo <= tile()) {
            load(lo);
            rank(lo, counts);
            uint32_t n = 0;
            if (tid < bins) {
#pragma unroll 8
                for (int w = 0; w < kSortWarps; ++w) n += counts[w][tid];
            }
            return n;
        }
        for (int d = tid; d < bins; d += kSortThreads) hist[d] = 0;
        __syncthreads();
        for (int64_t at = lo; at < hi; at += tile()) {
            load(at);
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                if (j >= items) break;
                const uint32_t d = digit(at, j), same = same_digit(d, d != ~0u, bits);
                if (d != ~0u && tid % 32 == __ffs(same) - 1) atomicAdd(&hist[d], __popc(same));
            }
        }
        __syncthreads();
        return tid < bins ? hist[tid] : 0;
    }
    // Puts the tokens in their places; base: to thread d the first one of digit d
    // in this CTA.  ranked: they are one tile, and count() has just ranked it.
    __device__ __forceinline__ void scatter(uint32_t (*counts)[kBins], uint32_t base, bool ranked)
    {
        for (int64_t at = lo; at < hi; at += tile()) {
            if (!ranked) {
                load(at);
                rank(at, counts);
            }
            if (threadIdx.x < 1 << bits) {
#pragma unroll 8
                for (int w = 0; w < kSortWarps; ++w) {
                    const uint32_t n = counts[w][threadIdx.x];
                    counts[w][threadIdx.x] = base;
                    base += n;
                }
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                if (j >= items) break;
                const uint32_t d = digit(at, j);
                if (d == ~0u) continue;
                to[counts[threadIdx.x / 32][d] + place[j]] = x[j];
                if (present && key_of(x[j]) < vocab) present[key_of(x[j])] = 1;
            }
        }
    }
};

// Pass `pass`, of which CTA `cta` of `ctas` has its share.
__device__ __forceinline__ Pass pass_of(const OrderArgs& a, int pass, int64_t cta, int64_t ctas)
{
    Pass p;
    p.ids = pass == 0 ? a.e.ids : nullptr;
    p.present = pass == 0 && a.note ? a.r.present : nullptr;
    p.from = (a.passes - pass) % 2 ? a.r.other : a.r.sorted;
    p.to = (a.passes - pass) % 2 ? a.r.sorted : a.r.other;
    p.vocab = a.e.vocab;
    p.lo = a.e.tokens * cta / ctas;
    p.hi = a.e.tokens * (cta + 1) / ctas;
    p.shift = 32 + pass * a.digit;
    p.bits = a.digit;
    p.items = static_cast<int>(max(int64_t(1), min(int64_t(kItems), (p.hi - p.lo + kSortThreads - 1) / kSortThreads)));
    return p;
}

// The sum of `x` over the threads before this one.
__device__ __forceinline__ uint32_t sum_before(uint32_t x, uint32_t* sums)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t sum = x;
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t s = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += s;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    if (threadIdx.x < kBins)
        for (int w = 0; w < warp; ++w) sum += sums[w];
    __syncthreads();
    return sum - x;
}

__device__ __forceinline__ void clear_present(const OrderArgs& a, int64_t cta, int64_t ctas)
{
    if (!a.clear) return;
    uint4* p = reinterpret_cast<uint4*>(a.r.present);        // up to its last, whole vector
    const int64_t n = (a.e.vocab + 15) / 16;
    for (int64_t i = cta * kSortThreads + threadIdx.x; i < n; i += ctas * kSortThreads) p[i] = make_uint4(0, 0, 0, 0);
}

// The sort by one cluster.
__device__ void sort_tokens(const OrderArgs& a, uint32_t (*counts)[kBins])
{
    __shared__ uint32_t hist[kBins], sums[kSortWarps];
    const int tid = threadIdx.x, bins = 1 << a.digit;
    const uint32_t rank = cluster_rank();
    if (rank == 0 && tid < 2) a.r.count[tid] = 0;
    clear_present(a, rank, kCluster);          // set after a barrier of the cluster
    for (int pass = 0; pass < a.passes; ++pass) {
        Pass p = pass_of(a, pass, rank, kCluster);
        const uint32_t n = p.count(counts, hist);
        if (tid < bins) hist[tid] = n;
        cluster_sync();
        // a digit's first place: all smaller digits, and its own in the CTAs before
        uint32_t all = 0, before = 0;
        if (tid < bins) {
#pragma unroll
            for (uint32_t c = 0; c < kCluster; ++c) {
                const uint32_t h = cluster_read(&hist[tid], c);
                all += h;
                before += c < rank ? h : 0;
            }
        }
        p.scatter(counts, sum_before(all, sums) + before, p.hi - p.lo <= p.tile());
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

// Zeros into those of the table's rows first + [begin, end) that have no bit in
// the map: run by run, one warp.
__device__ __forceinline__ void zero_absent(uint16_t* table, int64_t dim, int64_t first, int begin, int end, const uint32_t* map, int lane)
{
    for (int r = begin; r < end;) {
        if (map[r / 32] >> (r % 32) & 1) {
            ++r;
            continue;
        }
        int stop = r;                          // the next bit
        while (stop < end) {
            const uint32_t w = map[stop / 32] >> (stop % 32);
            if (w) {
                stop += __ffs(w) - 1;
                break;
            }
            stop = (stop / 32 + 1) * 32;
        }
        stop = min(stop, end);
        zero_run(table + (first + r) * dim, (stop - r) * dim, lane);
        r = stop;
    }
}

// One CTA's part of the zeros: the table's rows [begin, end) that no token has.
// kMapBits of them at a time.
__device__ void fill_rows(const OrderArgs& a, uint32_t* map, int64_t cta, int64_t ctas)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t begin = a.fill * cta / ctas, end = a.fill * (cta + 1) / ctas;
    for (int64_t first = begin; first < end; first += kMapBits) {
        const int64_t rows = min(int64_t(kMapBits), end - first);
        for (int64_t i = threadIdx.x; i < (rows + 31) / 32; i += kSortThreads) map[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int64_t t = threadIdx.x; t < a.e.tokens; t += kSortThreads) {
            const uint64_t r = static_cast<uint64_t>(a.e.ids[t]) - static_cast<uint64_t>(first);
            // seen before by most tokens of a frequent id: they would wait for one another's atomics
            if (r < static_cast<uint64_t>(rows) && !(static_cast<volatile uint32_t*>(map)[r / 32] >> (r % 32) & 1)) atomicOr(&map[r / 32], 1u << (r % 32));
        }
        __syncthreads();
        zero_absent(a.dtable, a.e.dim, first, static_cast<int>(rows * warp / kSortWarps), static_cast<int>(rows * (warp + 1) / kSortWarps),
                    map, lane);
        __syncthreads();
    }
}

__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Each token's place: the tokens of smaller ids, and those of its own before it.
// A CTA for 32 tokens, eight lanes for each, all ids in shared memory (added to
// their rows of 1024, 1024 / 4096 / 8192 tokens 11 / 16 / 30 us, by way of the
// cluster's sort 17 / 20 / 25).  The zeros of a large table are better written
// beside the sums, too (1024 x 752 rows of 4336 13 us, by the cluster 18; 385 x
// 10594 of 3704 26 and 27; 1024 x 50257 of 1024 30 and 27).
constexpr int kRankTokens = 4096;
constexpr int64_t kRankZeros = 64 << 20;
constexpr int kRanked = kRowThreads / 8;       // tokens of a CTA
constexpr int kRankRows = 512;                 // of the table, of a CTA that writes zeros, at most

__global__ void __launch_bounds__(kRowThreads) rank_kernel(const __grid_constant__ OrderArgs a)
{
    extern __shared__ __align__(16) uint32_t shared[];
    let_next_start();
    const int tid = threadIdx.x, tokens = static_cast<int>(a.e.tokens);
    const int ctas = (tokens + kRanked - 1) / kRanked;
    if (static_cast<int>(blockIdx.x) >= ctas) {
        constexpr int kWarps = kRowThreads / 32;
        const int64_t first = (static_cast<int64_t>(blockIdx.x) - ctas) * a.fill_rows;
        const int rows = static_cast<int>(min(a.fill_rows, a.fill - first)), warp = tid / 32;
        for (int i = tid; i < (rows + 31) / 32; i += kRowThreads) shared[i] = 0;
        __syncthreads();
#pragma unroll 8
        for (int t = tid; t < tokens; t += kRowThreads) {
            const uint64_t r = static_cast<uint64_t>(a.e.ids[t]) - static_cast<uint64_t>(first);
            if (r < static_cast<uint64_t>(rows) && !(static_cast<volatile uint32_t*>(shared)[r / 32] >> (r % 32) & 1)) atomicOr(&shared[r / 32], 1u << (r % 32));
        }
        __syncthreads();
        zero_absent(a.dtable, a.e.dim, first, rows * warp / kWarps, rows * (warp + 1) / kWarps, shared, tid % 32);
        return;
    }
    if (blockIdx.x == 0 && tid < 2) a.r.count[tid] = 0;
    const int vectors = (tokens + 3) / 4;
#pragma unroll 8
    for (int t = tid; t < vectors * 4; t += kRowThreads) {
        const int64_t id = t < tokens ? a.e.ids[t] : -1;
        shared[t] = t >= tokens ? ~0u : static_cast<uint32_t>(id >= 0 && id < a.e.vocab ? id : a.e.vocab);
    }
    __syncthreads();
    const int t = blockIdx.x * kRanked + tid / 8;
    const uint32_t mine = t < tokens ? shared[t] : 0;
    uint32_t place = 0;
#pragma unroll 8
    for (int v = tid % 8; v < vectors; v += 8) {
        const uint4 x = reinterpret_cast<const uint4*>(shared)[v];
        const uint32_t below = mine + (v < t / 4);         // equal ones count before this token's own four
        place += (x.x < below) + (x.y < below) + (x.z < below) + (x.w < below);
    }
    if (tid % 8 < t % 4 && t < tokens) place += shared[t / 4 * 4 + tid % 8] == mine;
    for (int o = 1; o < 8; o *= 2) place += __shfl_xor_sync(~0u, place, o);
    if (tid % 8 == 0 && t < tokens) a.r.sorted[place] = static_cast<uint64_t>(mine) << 32 | static_cast<uint32_t>(t);
}

__global__ void __launch_bounds__(kSortThreads) order_kernel(const __grid_constant__ OrderArgs a)
{
    extern __shared__ __align__(16) uint32_t shared[];
    let_next_start();
    if (blockIdx.x < kCluster) sort_tokens(a, reinterpret_cast<uint32_t(*)[kBins]>(shared));
    else fill_rows(a, shared, blockIdx.x - kCluster, gridDim.x - kCluster);
}

// The same sort of more tokens, by all SMs: two launches a pass, the first of
// which leaves the CTAs' counts in the workspace.
__global__ void __launch_bounds__(kSortThreads) count_kernel(const __grid_constant__ OrderArgs a)
{
    extern __shared__ __align__(16) uint32_t shared[];
    __shared__ uint32_t hist[kBins];
    let_next_start();
    wait_for_previous();
    if (blockIdx.x == 0 && threadIdx.x < 2) a.r.count[threadIdx.x] = 0;
    if (a.pass == 0) clear_present(a, blockIdx.x, gridDim.x);
    Pass p = pass_of(a, a.pass, blockIdx.x, gridDim.x);
    const uint32_t n = p.count(reinterpret_cast<uint32_t(*)[kBins]>(shared), hist);
    if (threadIdx.x < 1 << a.digit) a.r.digits[blockIdx.x * kBins + threadIdx.x] = n;
}

__global__ void __launch_bounds__(kSortThreads) place_kernel(const __grid_constant__ OrderArgs a)
{
    extern __shared__ __align__(16) uint32_t shared[];
    __shared__ uint32_t sums[kSortWarps];
    uint32_t(*counts)[kBins] = reinterpret_cast<uint32_t(*)[kBins]>(shared);
    let_next_start();
    wait_for_previous();
    Pass p = pass_of(a, a.pass, blockIdx.x, gridDim.x);
    const bool single = p.hi - p.lo <= p.tile();
    if (single) p.load(p.lo);
    // each digit's counts of all CTAs, and of those before: a share of the CTAs
    // for each of kSortThreads / bins threads
    const int bins = 1 << a.digit, shares = kSortThreads / bins, d = threadIdx.x % bins, share = threadIdx.x / bins;
    uint32_t all = 0, before = 0;
#pragma unroll 32
    for (int c = share; c < static_cast<int>(gridDim.x); c += shares) {
        const uint32_t n = __ldcg(a.r.digits + c * kBins + d);
        all += n;
        before += c < static_cast<int>(blockIdx.x) ? n : 0;
    }
    shared[threadIdx.x] = all;
    shared[kSortThreads + threadIdx.x] = before;
    __syncthreads();
    all = before = 0;
    if (threadIdx.x < bins)
        for (int i = 0; i < shares; ++i) {
            all += shared[i * bins + d];
            before += shared[kSortThreads + i * bins + d];
        }
    const uint32_t base = sum_before(all, sums) + before;
    if (single) p.rank(p.lo, counts);
    p.scatter(counts, base, single);
}

struct SumArgs {
    q8_embedding e;
    Room r;
    const void* dout;
    int64_t stride;
    uint16_t* dtable;
    int64_t filled, fill_rows; // the table's rows from `filled` on get their zeros here, so many to a CTA
    // CTAs that add up, and that join; those behind them write zeros (mixed
    // evenly, reads beside writes from the start: 16384 x 4096 106 us, not 94)
    int64_t sums, joins;
    int32_t late;              // the zeros are written behind the joins: sum_kernel notes the rows that it meets
    int32_t accumulate;
    int32_t group, tiles;      // threads that share a piece's columns, and tiles of 8 * group columns
};

// A thread's eight columns: VEC, contiguous; else every step-th, of bf16 in
// pairs.  Rows on their way wait in the thread's own slots of shared memory (no
// other thread reads them), which hold more of them in flight than registers
// would.
template <typename T, bool VEC>
struct Columns {
    static constexpr int kBytes = VEC ? 8 * sizeof(T) : 32;        // of a slot
    int64_t first, dim;
    int step;

    __device__ __forceinline__ int64_t column(int j) const
    {
        if constexpr (VEC) return first + j;
        else if constexpr (sizeof(T) == 4) return first + static_cast<int64_t>(j) * step;
        else return first + static_cast<int64_t>(j / 2) * 2 * step + j % 2;
    }
    static __device__ __forceinline__ uint32_t word(uint4* slot, int j)
    {
        return smem_addr(reinterpret_cast<uint32_t*>(slot) + (j / 4) * (kRowThreads * 4) + j % 4);
    }
    static __device__ __forceinline__ bool off4(const T* row) { return reinterpret_cast<uintptr_t>(row) % 4 != 0; }

    // slot: this thread's, kRowThreads vectors apart.  edge: the row is the first
    // or one of the last two of its matrix, and the words that its pairs lie in
    // may reach past it.
    __device__ __forceinline__ void fetch(uint4* slot, const T* row, bool edge) const
    {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(slot + i * kRowThreads)),
                             "l"(reinterpret_cast<const uint4*>(row + first) + i) : "memory");
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (column(j) < dim)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(word(slot, j)), "l"(row + column(j)) : "memory");
        } else if (edge) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t c = column(2 * k);
                x[k] = (c < dim ? row[c] : 0) | static_cast<uint32_t>(c + 1 < dim ? row[c + 1] : 0) << 16;
            }
            const bool off = off4(row);        // as copies would have brought it
            slot[0] = off ? make_uint4(x[0] << 16, x[1] << 16, x[2] << 16, x[3] << 16) : make_uint4(x[0], x[1], x[2], x[3]);
            if (off) slot[kRowThreads] = make_uint4(x[0] >> 16, x[1] >> 16, x[2] >> 16, x[3] >> 16);
        } else {
            // a pair off 4 bytes lies in two words
            const uint32_t* words = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(row) & ~uintptr_t(3));
            const bool off = off4(row);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (column(2 * k) < dim) {
                    const uint32_t* p = words + column(2 * k) / 2;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(word(slot, k)), "l"(p) : "memory");
                    if (off) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(word(slot, 4 + k)), "l"(p + 1) : "memory");
                }
        }
    }
    // What was fetched, added to sum.
    __device__ __forceinline__ void add(Eight& sum, const uint4* slot, const T* row) const
    {
        const uint4 u = slot[0];
        if constexpr (sizeof(T) == 2) {
            uint32_t x[4] = {u.x, u.y, u.z, u.w};
            if constexpr (!VEC) {
                if (off4(row)) {
                    const uint4 w = slot[kRowThreads];
                    const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = __byte_perm(x[k], y[k], 0x5432);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) sum.x[k] = __fadd2_rn(sum.x[k], bf16x2(x[k]));
        } else {
            const uint4 w = slot[kRowThreads];
            const uint32_t x[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sum.x[k] = __fadd2_rn(sum.x[k], make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])));
        }
    }
    template <typename U>
    __device__ __forceinline__ Eight read(const U* row) const
    {
        if constexpr (VEC && sizeof(U) == 2) {
            const uint4 w = *reinterpret_cast<const uint4*>(row + first);
            return Eight{{bf16x2(w.x), bf16x2(w.y), bf16x2(w.z), bf16x2(w.w)}};
        } else if constexpr (VEC) {
            const float4 u = reinterpret_cast<const float4*>(row + first)[0], w = reinterpret_cast<const float4*>(row + first)[1];
            return Eight{{make_float2(u.x, u.y), make_float2(u.z, u.w), make_float2(w.x, w.y), make_float2(w.z, w.w)}};
        } else {
            Eight v;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v.x[k] = make_float2(column(2 * k) < dim ? load1(row + column(2 * k)) : 0.0f,
                                     column(2 * k + 1) < dim ? load1(row + column(2 * k + 1)) : 0.0f);
            return v;
        }
    }
    template <typename U>
    __device__ __forceinline__ void write(U* row, const Eight& v) const
    {
        if constexpr (VEC) {
            write8(row + first, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (column(j) < dim) store1(row + column(j), j % 2 ? v.x[j / 2].y : v.x[j / 2].x);
        }
    }
    // scale * sum, or with accumulate that added to what the row holds.
    __device__ __forceinline__ void write_scaled(uint16_t* row, Eight sum, float scale, bool accumulate) const
    {
        if (accumulate) {
            const Eight old = read(row);
#pragma unroll
            for (int k = 0; k < 4; ++k) sum.x[k] = __ffma2_rn(sum.x[k], splat(scale), old.x[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) sum.x[k] = __fmul2_rn(sum.x[k], splat(scale));
        }
        write(row, sum);
    }
};

// Rows of a thread in flight: 32 or 64 KB a CTA, of which four or three run on an
// SM (16 rows of bf16 and three CTAs: 262144 x 1024 154 us instead of 150; a ring
// that goes on into the next piece, in CTAs that stay, took more).
constexpr int kAhead = 8;
template <typename T, bool VEC>
constexpr int kSumShared = kAhead * Columns<T, VEC>::kBytes * kRowThreads;

__device__ __forceinline__ uint64_t entry_at(const uint64_t* sorted, int64_t i, int64_t n, uint64_t none)
{
    return i >= 0 && i < n ? __ldcg(reinterpret_cast<const unsigned long long*>(sorted) + i) : none;
}

// Zeros of one CTA's rows [begin, end), a thread for each at most: those that no
// token has.
__device__ void fill_absent(const SumArgs& a, int64_t begin, int64_t end)
{
    constexpr int kWarps = kRowThreads / 32;
    __shared__ uint32_t present[kWarps];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t some = __ballot_sync(~0u, begin + threadIdx.x < end && a.r.present[begin + threadIdx.x]);
    if (lane == 0) present[warp] = some;
    __syncthreads();
    const int rows = static_cast<int>(end - begin);
    zero_absent(a.dtable, a.e.dim, begin, rows * warp / kWarps, rows * (warp + 1) / kWarps, present, lane);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads, 3) sum_kernel(const __grid_constant__ SumArgs a)
{
    constexpr int kRing = kAhead;
    constexpr int kVecs = Columns<T, VEC>::kBytes / 16;
    constexpr int kStep = 4;                               // rows that are waited for together
    static_assert(kRing % kStep == 0, "the ring holds whole steps");
    extern __shared__ __align__(16) uint4 ring[];          // [kRing][kVecs][kRowThreads]
    let_next_start();
    wait_for_previous();
    if (blockIdx.x >= a.sums) {
        const int64_t begin = a.filled + (blockIdx.x - a.sums) * a.fill_rows;
        fill_absent(a, begin, min(a.e.vocab, begin + a.fill_rows));
        return;
    }
    const int lane = threadIdx.x % 32;
    const int64_t N = a.e.tokens;
    const int P = a.r.piece;
    const int64_t piece = static_cast<int64_t>(blockIdx.x / a.tiles) * (kRowThreads / a.group) + threadIdx.x / a.group;
    if (piece >= a.r.pieces) return;
    // the piece's tokens, those behind it (an id goes on for at most P - 1 of
    // them) and the ids before it, one to a lane
    const uint32_t vocab = static_cast<uint32_t>(a.e.vocab);
    const uint64_t none = ~uint64_t(0);
    const int64_t p0 = piece * P;
    const uint64_t here = entry_at(a.r.sorted, lane < P ? p0 + lane : N, N, none);
    const uint64_t behind = entry_at(a.r.sorted, lane < P ? p0 + P + lane : N, N, none);
    const uint32_t before = key_of(entry_at(a.r.sorted, lane < P ? p0 - 1 - lane : N, N, none));
    const uint32_t first_here = __shfl_sync(~0u, key_of(here), 0), first_behind = __shfl_sync(~0u, key_of(behind), 0);
    // an id across the piece's start or end: its tokens on either side, each counted to P
    const auto ones = [](uint32_t m) { return ~m ? __ffs(~m) - 1 : 32; };
    const int back0 = ones(__ballot_sync(~0u, before == first_here)), on0 = ones(__ballot_sync(~0u, key_of(here) == first_here));
    const int back1 = __clz(~(__ballot_sync(~0u, key_of(here) == first_behind) << (32 - P)));
    const int on1 = ones(__ballot_sync(~0u, key_of(behind) == first_behind));
    const bool from_before = back0 > 0 && back0 + on0 > P;                             // parts of a long id
    const bool goes_on = first_behind < vocab && back1 > 0 && back1 + on1 > P;
    const int skip = back0 > 0 && !from_before ? on0 : 0;
    const int stop = first_behind < vocab && back1 > 0 && !goes_on ? P + on1 : P;
    const int known = __popc(__ballot_sync(~0u, key_of(here) < vocab)) + __popc(__ballot_sync(~0u, key_of(behind) < vocab));
    const int count = min(stop, known) - skip;             // ids outside the table come last
    if (count <= 0) return;
    // from here on the tokens in the order in which they are added: 0 to 31 and
    // 32 to 63 of them, one to a lane
    const auto in_order = [&](uint32_t here_, uint32_t behind_, int i) {
        const uint32_t x = __shfl_sync(~0u, here_, i & 31), y = __shfl_sync(~0u, behind_, (i - P) & 31);
        return i < P ? x : y;
    };
    const uint32_t key0 = in_order(key_of(here), key_of(behind), lane + skip), key1 = in_order(key_of(here), key_of(behind), lane + skip + 32);
    const uint32_t token0 = in_order(static_cast<uint32_t>(here), static_cast<uint32_t>(behind), lane + skip);
    const uint32_t token1 = in_order(static_cast<uint32_t>(here), static_cast<uint32_t>(behind), lane + skip + 32);
    const auto key_at = [&](int i) { return __shfl_sync(~0u, i < 32 ? key0 : key1, i & 31); };
    // bit i: the id of token i ends with it, or the piece does
    const uint32_t next0 = __shfl_down_sync(~0u, key0, 1), next1 = __shfl_down_sync(~0u, key1, 1), start1 = __shfl_sync(~0u, key1, 0);
    const uint32_t ends0 = __ballot_sync(~0u, lane == count - 1 || key0 != (lane == 31 ? start1 : next0));
    const uint32_t ends1 = __ballot_sync(~0u, lane + 32 == count - 1 || key1 != next1);
    const uint32_t first_key = key_at(0), last_key = key_at(count - 1);
    const T* dout = static_cast<const T*>(a.dout);
    uint4* mine = ring + threadIdx.x;
    const int tid = threadIdx.x % a.group;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x % a.tiles) * 8 * a.group;
    const Columns<T, VEC> cols{c0 + tid * (VEC ? 8 : sizeof(T) == 2 ? 2 : 1), a.e.dim, a.group};
    const bool on = cols.first < a.e.dim;
    const auto fetch = [&](int i) {                        // kStep rows from i on, one group of copies, be it empty
        const uint32_t tokens = i < 32 ? token0 : token1;
        uint4* slot = mine + i % kRing * (kVecs * kRowThreads);
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
            const uint32_t t = __shfl_sync(~0u, tokens, (i + j) & 31);
            // a row's words reach up to two elements past it, which are the next two rows where rows are single elements
            if (on && i + j < count) cols.fetch(slot + j * (kVecs * kRowThreads), dout + static_cast<int64_t>(t) * a.stride, t == 0 || t + 2 >= N);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kRing; i += kStep) fetch(i);
    Eight sum{};
#pragma unroll 1
    for (int i = 0; i < count; i += kStep) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing / kStep - 1) : "memory");
        const uint4* slot = mine + i % kRing * (kVecs * kRowThreads);
        const uint32_t ends = (i < 32 ? ends0 : ends1) >> (i & 31), tokens = i < 32 ? token0 : token1;
        const auto add = [&](int j) {
            const T* row = dout;                           // its alignment is all that counts
            if constexpr (!VEC && sizeof(T) == 2) row += static_cast<int64_t>(__shfl_sync(~0u, tokens, (i + j) & 31)) * a.stride;
            if (on) cols.add(sum, slot + j * (kVecs * kRowThreads), row);
        };
        if (!(ends & ((1u << kStep) - 1))) {               // all of one id, which goes on
#pragma unroll
            for (int j = 0; j < kStep; ++j) add(j);
        } else {
#pragma unroll 1
            for (int j = 0; j < kStep && i + j < count; ++j) {
                add(j);
                if (!(ends >> j & 1)) continue;
                const uint32_t key = key_at(i + j);
                if (on) {
                    if (key == first_key && from_before) {
                        cols.write(a.r.parts + (piece * 2) * a.r.columns, sum);
                    } else {
                        if (a.late && blockIdx.x % a.tiles == 0 && tid == 0) a.r.present[key] = 1;
                        if (i + j == count - 1 && goes_on) cols.write(a.r.parts + (piece * 2 + 1) * a.r.columns, sum);
                        else cols.write_scaled(a.dtable + static_cast<int64_t>(key) * a.e.dim, sum, a.e.scale, a.accumulate);
                    }
                }
                sum = Eight{};
            }
        }
        fetch(i + kRing);
    }
    if (goes_on && !(first_key == last_key && from_before) && blockIdx.x % a.tiles == 0 && tid < 32) {
        // a long id begins here: the first piece behind it that does not begin with it, 32 places at a time
        int64_t lo = piece + 2, hi = a.r.pieces;
        while (lo < hi) {
            const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
            const int n = __popc(__ballot_sync(~0u, at < hi && key_of(entry_at(a.r.sorted, at * P, N, none)) == last_key));
            if (n == 0) break;
            hi = min(hi, lo + n * step);
            lo += (n - 1) * step + 1;
        }
        const int parts = static_cast<int>(lo - piece);
        const int many = parts > kFewParts;
        if (lane == 0) a.r.list[many * a.r.pieces + atomicAdd(a.r.count + many, 1)] = make_int2(static_cast<int>(piece), parts);
    }
}

__device__ __forceinline__ float4 part_of(const SumArgs& a, int64_t piece, int q, int64_t c)
{
    // its own part, then one of each piece behind it
    return *reinterpret_cast<const float4*>(a.r.parts + ((piece + q) * 2 + (q == 0)) * a.r.columns + c);
}

__device__ __forceinline__ float4 add4(float4 x, float4 y)
{
    return make_float4(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y), __fadd_rn(x.z, y.z), __fadd_rn(x.w, y.w));
}

__device__ __forceinline__ void write_joined(const SumArgs& a, uint32_t key, int64_t c, float x)
{
    if (c >= a.e.dim) return;
    uint16_t* to = a.dtable + static_cast<int64_t>(key) * a.e.dim + c;
    store1(to, a.accumulate ? __fmaf_rn(a.e.scale, x, load1(to)) : __fmul_rn(a.e.scale, x));
}

// Ids of many parts: a CTA for eight columns (a sector of 32 bytes) of one of
// them; its 128 pairs of threads take the parts in turn.  Ids of few: a warp for
// 32 columns, its four groups of lanes take the parts in turn.
__global__ void __launch_bounds__(kRowThreads) join_kernel(const __grid_constant__ SumArgs a)
{
    constexpr int kPairs = kRowThreads / 2, kSums = kRowThreads / 8;
    __shared__ __align__(16) float sums[kPairs * 8];
    __shared__ float last[kSums * 8];
    wait_for_previous();
    if (blockIdx.x >= a.joins) {
        const int64_t begin = a.filled + (blockIdx.x - a.joins) * a.fill_rows;
        fill_absent(a, begin, min(a.e.vocab, begin + a.fill_rows));
        return;
    }
    const int tid = threadIdx.x, lane = tid % 32;
    const int64_t ctas = a.joins;
    const int64_t wide = (a.e.dim + 31) / 32, narrow = (a.e.dim + 7) / 8;
    const int64_t many = a.r.count[1] * narrow, few = a.r.count[0] * wide;
    for (int64_t i = blockIdx.x; i < many; i += ctas) {
        const int2 what = a.r.list[a.r.pieces + i / narrow];
        const uint32_t key = key_of(a.r.sorted[(static_cast<int64_t>(what.x) + 1) * a.r.piece]);
        const int64_t c0 = i % narrow * 8;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int q = tid / 2; q < what.y; q += kPairs) sum = add4(sum, part_of(a, what.x, q, c0 + tid % 2 * 4));
        reinterpret_cast<float4*>(sums)[tid] = sum;
        __syncthreads();
        float x = 0.0f;
#pragma unroll
        for (int r = 0; r < kPairs / kSums; ++r) x = __fadd_rn(x, sums[(tid / 8 * (kPairs / kSums) + r) * 8 + tid % 8]);
        last[tid] = x;
        __syncthreads();
        if (tid < 8) {
            x = 0.0f;
#pragma unroll
            for (int r = 0; r < kSums; ++r) x = __fadd_rn(x, last[r * 8 + tid]);
            write_joined(a, key, c0 + tid, x);
        }
    }
    // begun with the CTAs that had one id of many parts less
    const int64_t cta = (blockIdx.x + ctas - many % ctas) % ctas;
    for (int64_t i = cta * (kRowThreads / 32) + tid / 32; i < few; i += ctas * (kRowThreads / 32)) {
        const int2 what = a.r.list[i / wide];
        const uint32_t key = key_of(a.r.sorted[(static_cast<int64_t>(what.x) + 1) * a.r.piece]);
        const int64_t c0 = i % wide * 32, c = min(c0 + lane % 8 * 4, a.r.columns - 4);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int q = lane / 8; q < what.y; q += 4) sum = add4(sum, part_of(a, what.x, q, c));
        for (int o = 8; o < 32; o *= 2)
            sum = add4(sum, make_float4(__shfl_xor_sync(~0u, sum.x, o), __shfl_xor_sync(~0u, sum.y, o),
                                        __shfl_xor_sync(~0u, sum.z, o), __shfl_xor_sync(~0u, sum.w, o)));
        const int k = lane / 8;                            // each lane writes one of its four columns
        write_joined(a, key, c0 + lane % 8 * 4 + k, k == 0 ? sum.x : k == 1 ? sum.y : k == 2 ? sum.z : sum.w);
    }
}

// ----------------------------------------------------- gradient of a few tokens

// At most kFewTokens of them, one launch, no sort: the ids are compared with one
// another (added to their rows: one token of 64 2.5 us, 256 of 1024 4.3, all of one
// id 8.3; by way of the sort 10 to 17).  A CTA for each token and 256 columns: unless its id came before, the
// CTA's warps take the rows of that id in turn, and their sums are added.
// Further CTAs write the zeros.
constexpr int kFewTokens = kRowThreads;        // a thread for each
constexpr int kFewColumns = 256;
constexpr int kFewRows = 512;                  // of the table, of a CTA that writes zeros, at most

struct FewArgs {
    q8_embedding e;
    const void* dout;
    int64_t stride;
    uint16_t* dtable;
    int64_t sums, fill_rows;
    int32_t tiles, accumulate;
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) few_kernel(const __grid_constant__ FewArgs a)
{
    constexpr int kWarps = kRowThreads / 32;
    __shared__ __align__(16) float sums[kWarps][kFewColumns];
    __shared__ uint32_t map[kFewRows / 32], same[kWarps];
    __shared__ int list[kFewTokens];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int64_t id = tid < a.e.tokens ? a.e.ids[tid] : -1;
    if (id >= a.e.vocab) id = -1;
    if (blockIdx.x >= a.sums) {
        const int64_t first = (blockIdx.x - a.sums) * a.fill_rows;
        const int rows = static_cast<int>(min(a.fill_rows, a.e.vocab - first));
        for (int i = tid; i < (rows + 31) / 32; i += kRowThreads) map[i] = 0;
        __syncthreads();
        if (id >= first && id < first + rows) atomicOr(&map[(id - first) / 32], 1u << ((id - first) % 32));
        __syncthreads();
        zero_absent(a.dtable, a.e.dim, first, rows * warp / kWarps, rows * (warp + 1) / kWarps, map, lane);
        return;
    }
    const int token = static_cast<int>(blockIdx.x / a.tiles);
    const int64_t c0 = static_cast<int64_t>(blockIdx.x % a.tiles) * kFewColumns, mine = a.e.ids[token];
    if (mine < 0 || mine >= a.e.vocab) return;
    const uint32_t m = __ballot_sync(~0u, id == mine);
    if (lane == 0) same[warp] = m;
    __syncthreads();
    int before = 0, count = 0;                 // tokens of this id in the warps before this one, and in all
    bool first = true;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? __popc(same[w]) : 0;
        count += __popc(same[w]);
        first = first && !(w < token / 32 ? same[w] : w == token / 32 ? same[w] & ((1u << (token % 32)) - 1) : 0);
    }
    if (!first) return;
    if (id == mine) list[before + __popc(m & ((1u << lane) - 1))] = tid;
    __syncthreads();
    const Columns<T, VEC> cols{c0 + lane * (VEC ? 8 : sizeof(T) == 2 ? 2 : 1), a.e.dim, 32};
    Eight sum{};
    if (cols.first < a.e.dim) {
#pragma unroll 4
        for (int i = warp; i < count; i += kWarps) {
            const Eight x = cols.read(static_cast<const T*>(a.dout) + list[i] * a.stride);
#pragma unroll
            for (int k = 0; k < 4; ++k) sum.x[k] = __fadd2_rn(sum.x[k], x.x[k]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[warp][cols.column(j) - c0] = j % 2 ? sum.x[j / 2].y : sum.x[j / 2].x;
    __syncthreads();
    const int64_t c = c0 + tid;
    if (c >= a.e.dim) return;
    float x = 0.0f;
    for (int w = 0; w < min(kWarps, count); ++w) x = __fadd_rn(x, sums[w][tid]);
    uint16_t* to = a.dtable + mine * a.e.dim + c;
    store1(to, a.accumulate ? __fmaf_rn(a.e.scale, x, load1(to)) : __fmul_rn(a.e.scale, x));
}

// ------------------------------------------------------------------------- host

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T>
cudaError_t lookup(const q8_embedding& e, const uint16_t* table, void* out, int64_t out_stride, cudaStream_t st)
{
    constexpr int64_t kMost = 1 << 20;
    if (e.dim % 8 == 0 && on16(table) && on16(out) && (e.tokens == 1 || out_stride * sizeof(T) % 16 == 0)) {
        const int64_t tiles = (e.tokens * (e.dim / 8) + kTile * kRowThreads - 1) / (kTile * kRowThreads);
        const auto k = e.tokens * e.dim * int64_t(sizeof(T)) > kStreamBytes ? lookup_kernel<T, true> : lookup_kernel<T, false>;
        k<<<static_cast<int>(std::min(kMost, tiles)), kRowThreads, 0, st>>>(e, table, static_cast<T*>(out), out_stride);
    } else {
        int group = 8;                         // the first and last elements of a row: seven at most
        while (group < kRowThreads && group * 16 < e.dim) group *= 2;
        const int64_t rows = kRowThreads / group;
        lookup_odd_kernel<T><<<static_cast<int>(std::min(kMost, (e.tokens + rows - 1) / rows)), kRowThreads, 0, st>>>(e, table, static_cast<T*>(out), out_stride, group);
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
template <typename Args>
cudaError_t launch_after(void (*kernel)(Args), int64_t grid, int threads, int shared, cudaStream_t st, const Args& a)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = shared;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// What the sort takes in one cluster, and what the other SMs write meanwhile (16384 x 4096
// with 14 us: 95 us, with 8 us: 98 us, on one GPU).
constexpr double kSortUs = 14.0, kSortTokenUs = 2.0e-4, kFillBytesUs = 5.5e6;
constexpr int64_t kFillBytes = 1 << 17;        // of a CTA of sum_kernel

using SumKernel = void (*)(SumArgs);
struct SumShape {
    SumKernel kernel;
    int shared;
};

template <typename T, bool VEC>
SumShape sum_shape() { return {sum_kernel<T, VEC>, kSumShared<T, VEC>}; }

SumShape sum_shape(bool f32, bool vec)
{
    return f32 ? (vec ? sum_shape<float, true>() : sum_shape<float, false>())
               : (vec ? sum_shape<uint16_t, true>() : sum_shape<uint16_t, false>());
}

using FewKernel = void (*)(FewArgs);

FewKernel few_kernel_of(bool f32, bool vec)
{
    return f32 ? (vec ? few_kernel<float, true> : few_kernel<float, false>)
               : (vec ? few_kernel<uint16_t, true> : few_kernel<uint16_t, false>);
}

cudaError_t launch_few(const q8_embedding& e, const void* dout, int64_t dout_stride, uint16_t* dtable, bool accumulate, bool vec,
                       cudaStream_t st)
{
    FewArgs a{};
    a.e = e;
    a.dout = dout;
    a.stride = dout_stride;
    a.dtable = dtable;
    a.accumulate = accumulate;
    const int64_t tiles = (e.dim + kFewColumns - 1) / kFewColumns;
    a.tiles = static_cast<int32_t>(tiles);
    a.sums = e.tokens * tiles;
    a.fill_rows = std::max<int64_t>(1, std::min<int64_t>(kFewRows, kFillBytes / 2 / e.dim));
    const int64_t grid = a.sums + (accumulate ? 0 : (e.vocab + a.fill_rows - 1) / a.fill_rows);
    if (grid > std::numeric_limits<int32_t>::max()) return cudaErrorInvalidConfiguration;
    few_kernel_of(e.dtype == Q8_F32, vec)<<<static_cast<unsigned>(grid), kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_embed()
{
    int n = 0;
    cudaError_t e = clusters_at_once(&n);
    if (e == cudaSuccess) e = persistent_grid(reinterpret_cast<const void*>(rank_kernel), kRowThreads, 0, &n);
    for (const void* k : {reinterpret_cast<const void*>(count_kernel), reinterpret_cast<const void*>(place_kernel)})
        if (e == cudaSuccess) e = persistent_grid(k, kSortThreads, kSortShared, &n);
    for (const void* k : {reinterpret_cast<const void*>(lookup_kernel<uint16_t, false>), reinterpret_cast<const void*>(lookup_kernel<uint16_t, true>),
                          reinterpret_cast<const void*>(lookup_kernel<float, false>), reinterpret_cast<const void*>(lookup_kernel<float, true>),
                          reinterpret_cast<const void*>(lookup_odd_kernel<uint16_t>), reinterpret_cast<const void*>(lookup_odd_kernel<float>)})
        if (e == cudaSuccess) e = persistent_grid(k, kRowThreads, 0, &n);
    for (bool f32 : {false, true})
        for (bool vec : {false, true}) {
            const SumShape s = sum_shape(f32, vec);
            if (e == cudaSuccess) e = persistent_grid(reinterpret_cast<const void*>(few_kernel_of(f32, vec)), kRowThreads, 0, &n);
            if (e == cudaSuccess) e = persistent_grid(reinterpret_cast<const void*>(s.kernel), kRowThreads, s.shared, &n);
        }
    return e == cudaSuccess ? persistent_grid(reinterpret_cast<const void*>(join_kernel), kRowThreads, 0, &n) : e;
}

cudaError_t launch_embed_forward(const q8_embedding& e, const uint16_t* table, void* out, int64_t out_stride, cudaStream_t st)
{
    return e.dtype == Q8_F32 ? lookup<float>(e, table, out, out_stride, st) : lookup<uint16_t>(e, table, out, out_stride, st);
}

int64_t embed_workspace(const q8_embedding& e) { return e.tokens <= kFewTokens ? 0 : room_of(e, nullptr).bytes; }

cudaError_t launch_embed_backward(const q8_embedding& e, const void* dout, int64_t dout_stride, uint16_t* dtable,
                                  bool accumulate, void* workspace, cudaStream_t st)
{
    const int size = e.dtype == Q8_F32 ? 4 : 2;
    const bool vec = e.dim % 8 == 0 && on16(dtable) && on16(dout) && (e.tokens == 1 || dout_stride * size % 16 == 0);
    if (e.tokens <= kFewTokens) return launch_few(e, dout, dout_stride, dtable, accumulate, vec, st);
    const SumShape sum = sum_shape(size == 4, vec);
    int clusters = 0, sorters = 0, joins = 0;
    cudaError_t err = clusters_at_once(&clusters);
    for (const void* k : {reinterpret_cast<const void*>(count_kernel), reinterpret_cast<const void*>(place_kernel)})
        if (err == cudaSuccess) err = persistent_grid(k, kSortThreads, kSortShared, &sorters);
    if (err == cudaSuccess) err = persistent_grid(reinterpret_cast<const void*>(sum.kernel), kRowThreads, sum.shared, &joins);
    if (err == cudaSuccess) err = persistent_grid(reinterpret_cast<const void*>(join_kernel), kRowThreads, 0, &joins);
    if (err != cudaSuccess) return err;
    const Room room = room_of(e, workspace);

    SumArgs s{};
    s.e = e;
    s.r = room;
    s.dout = dout;
    s.stride = dout_stride;
    s.dtable = dtable;
    s.accumulate = accumulate;
    s.group = group_of(e);
    s.tiles = static_cast<int>((e.dim + s.group * 8 - 1) / (s.group * 8));
    const int64_t each = kRowThreads / s.group;
    s.sums = (room.pieces + each - 1) / each * s.tiles;
    s.joins = joins;
    s.late = !accumulate && e.tokens > kClusterTokens;
    s.fill_rows = std::max<int64_t>(1, std::min<int64_t>(kRowThreads, kFillBytes / 2 / e.dim));
    // before the first launch: a refused call leaves the table as it was
    if (std::max(s.sums, s.joins) + e.vocab / s.fill_rows >= std::numeric_limits<int32_t>::max()) return cudaErrorInvalidConfiguration;

    OrderArgs o{};
    o.e = e;
    o.r = room;
    o.dtable = dtable;
    o.note = !accumulate && e.tokens <= kClusterTokens;
    o.clear = !accumulate;
    int bits = 1;
    while (e.vocab >> bits) ++bits;            // vocab itself is the key of ids outside the table
    o.passes = (bits + kDigitBits - 1) / kDigitBits;
    o.digit = (bits + o.passes - 1) / o.passes;
    if (e.tokens <= kRankTokens && (accumulate || 2 * e.vocab * e.dim <= kRankZeros)) {
        o.note = 0;
        o.fill = accumulate ? 0 : e.vocab;
        o.fill_rows = std::max<int64_t>(1, std::min<int64_t>(kRankRows, kFillBytes / 2 / e.dim));
        const int64_t grid = (e.tokens + kRanked - 1) / kRanked + (o.fill + o.fill_rows - 1) / o.fill_rows;
        const int shared = std::max<int>(static_cast<int>(e.tokens + 3) / 4 * 16, kRankRows / 8);
        rank_kernel<<<static_cast<unsigned>(grid), kRowThreads, shared, st>>>(o);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    } else if (e.tokens <= kClusterTokens) {
        // as many rows as are written while the tokens are sorted
        const double sort_us = kSortUs + kSortTokenUs * static_cast<double>(e.tokens);
        const int64_t rows = static_cast<int64_t>(sort_us * kFillBytesUs / (2.0 * static_cast<double>(e.dim)));
        o.fill = accumulate ? 0 : std::min(e.vocab, rows);
        const int ctas = accumulate ? kCluster : std::max(2, clusters) * kCluster;
        cudaLaunchAttribute attr{};
        const cudaLaunchConfig_t cfg = order_config(&attr, ctas, st);
        if ((err = cudaLaunchKernelEx(&cfg, order_kernel, o)) != cudaSuccess) return err;
    } else {
        sorters = std::min(sorters, kMaxSorters);
        for (o.pass = 0; o.pass < o.passes; ++o.pass) {
            if (o.pass == 0) {
                count_kernel<<<sorters, kSortThreads, kSortShared, st>>>(o);
                err = cudaGetLastError();
            } else {
                err = launch_after(count_kernel, sorters, kSortThreads, kSortShared, st, o);
            }
            if (err == cudaSuccess) err = launch_after(place_kernel, sorters, kSortThreads, kSortShared, st, o);
            if (err != cudaSuccess) return err;
        }
    }

    // Behind the sums: zeros before them took 45 instead of 42 us (3001 x 1601), 101 instead of 94 us (16384 x 4096).
    s.filled = o.fill;
    const int64_t fills = accumulate ? 0 : (e.vocab - o.fill + s.fill_rows - 1) / s.fill_rows;
    if ((err = launch_after(sum.kernel, s.sums + (s.late ? 0 : fills), kRowThreads, sum.shared, st, s)) != cudaSuccess) return err;
    return launch_after(join_kernel, joins + (s.late ? fills : 0), kRowThreads, 0, st, s);
}

}  // namespace q8
