// q8_distill_plan.h -- the shape of a launch of q8_distill.cu's row kernel: a
// function of sizes, types and the SM count alone, without CUDA, so that a test
// can walk it over the documented ranges on any machine.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "q8train.h"

#ifdef __CUDACC__
#define Q8_BOTH __host__ __device__
#else
#define Q8_BOTH
#endif

namespace q8 {
namespace distill {

enum Mode { kForward, kTrain, kStream };

constexpr int kMaxSlots = 16;
constexpr int kTeachers = 3;         // rows whose teacher is held: one in pass 2, one in pass 1, one being prepared
constexpr int kOwn = 64;             // threads beside those of the passes

// The shapes of a CTA: threads of the passes, CTAs that fit on an SM, 16-byte
// vectors of a chunk to a thread.  A row costs each warp some 300 instructions
// beside its elements, so that a row has no more warps than it needs.
enum Shape { kFifth, kHalf, kWhole };
Q8_BOTH constexpr int threads_of(int shape) { return shape == kFifth ? 128 : 512; }
Q8_BOTH constexpr int ctas_per_sm(int shape) { return shape == kFifth ? 5 : shape == kHalf ? 2 : 1; }
Q8_BOTH constexpr int chunk_vectors(int shape, int elem) { return shape == kWhole ? 3 : elem == 2 ? 4 : 2; }

// The kernel that a CTA of that shape runs: loss and gradient from one call have
// one for an SM to itself; otherwise such a CTA, which many entries leave no
// half of an SM, runs that of the half.
constexpr int kernel_shape(int mode, int shape) { return shape == kWhole && mode != kTrain ? kHalf : shape; }

constexpr int kMaxCluster = 8;

// Shared memory of an SM and the most of a CTA; 1 KB to each CTA is kept by the
// system, 1.5 KB at most are static.
constexpr int64_t kSm = 228 * 1024, kOfCta = 1024 + 1536;

struct Config {
    int mode = kForward;
    int ctas = 1, shape = kHalf;     // CTAs to a row
    int slots = 0, chunk = 0, seen = 0;
    size_t smem = 0;
    bool usable = false;             // the ring takes what the mode needs of it
};

inline Config configure(const q8_distill_topk& d, bool grad, bool first_pass, int sms)
{
    const int64_t elem = d.logits_dtype == Q8_F32 ? 4 : 2;
    const int64_t vecs = std::max<int64_t>(1, d.vocab * elem / 16);
    Config c;
    c.mode = !grad ? kForward : first_pass ? kTrain : kStream;
    c.seen = 4;
    while (c.seen < 2 * d.k) c.seen *= 2;
    const int64_t teacher = (kTeachers * 16 + 24) * ((d.k + 4) & ~int64_t(3)) + 4 * c.seen;
    const auto set = [&](int ctas, int shape) {
        const int64_t share = (vecs + ctas - 1) / ctas;
        const int64_t most = chunk_vectors(kernel_shape(c.mode, shape), static_cast<int>(elem)) * threads_of(shape);
        c.ctas = ctas;
        c.shape = shape;
        c.chunk = static_cast<int>(std::min(share, most));
        const int64_t chunks = (share + c.chunk - 1) / c.chunk;
        const int64_t room = kSm / ctas_per_sm(shape) - kOfCta - teacher;
        c.slots = static_cast<int>(std::min<int64_t>(kMaxSlots, room / (c.chunk * 16)));
        c.smem = static_cast<size_t>(c.slots) * c.chunk * 16 + static_cast<size_t>(teacher);
        // kTrain: all of a slice, one chunk more when the next row's has one more,
        // and two ahead
        return c.slots >= (c.mode == kTrain ? chunks + 3 : 2);
    };
    // Rows up to 16 KB: small CTAs, many of them on an SM.  kTrain: otherwise the
    // smallest CTAs whose ring holds the row, and then more of them to a row.
    bool fits = (vecs <= 1024 && set(1, kFifth)) || set(1, kHalf);
    for (int n = 1; n <= kMaxCluster && !fits; n *= 2) fits = set(n, kWhole);
    if (!fits) {
        // a row too wide for any ring goes through it twice; where many entries
        // leave half an SM no two chunks, a CTA has the SM to itself
        c.mode = kStream;
        fits = set(1, kHalf) || set(1, kWhole);
    }
    // few rows: more CTAs to each, while a slice stays at least 8 KB
    int n = c.ctas;
    while (n < kMaxCluster && d.rows * n * 2 <= sms && vecs / (2 * n) >= 512) n *= 2;
    if (n > c.ctas) fits = set(n, c.shape);
    c.usable = fits;
    return c;
}

}  // namespace distill
}  // namespace q8
