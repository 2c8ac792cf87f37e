// Host-only exercise of calls at the vocabulary matrix that the header allows, for
// a build with AddressSanitizer and UndefinedBehaviorSanitizer on the host code
// (tests/test_vocab_calls_host.py). As in vocab_driver.cpp, the current device is
// answered here, the plan has a stand-in for its device table, and the launchers
// only record what they were asked for.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <random>
#include <vector>

#include "checks.h"
#include "kernels.h"
#include "vocab.h"
#include "zdo_vocab.h"

extern "C" hipError_t hipGetDevice(int *d) {
    *d = 0;
    return hipSuccess;
}

namespace zdo {
static long launches = 0;
static CeArgs ce;
hipError_t launch_reduce(const ReduceArgs &, int, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_step(const StepArgs &, int, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_writeback(const WritebackArgs &, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_copy(void *, const void *, int64_t, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_norm(const NormArgs &, double *, int, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_clip(const double *, int32_t, float, float *, double *, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_gather(const GatherArgs &, int, hipStream_t) { return hipErrorNoDevice; }
hipError_t no_alloc_scratch(void **out) { *out = nullptr; return hipErrorNoDevice; }
hipError_t launch_probe(const ProbeArgs &, int, int, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_lookup(const LookupArgs &, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_rows(const RowsArgs &, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_ce(const CeArgs &a, hipStream_t) { ++launches; ce = a; return hipSuccess; }
hipError_t launch_ce_grad(const CeArgs &a, hipStream_t) { ++launches; ce = a; return hipSuccess; }
}  // namespace zdo

#define WANT(code, call)                                                                     \
    do {                                                                                     \
        const int got_ = (call);                                                             \
        if (got_ != (code)) {                                                                \
            std::printf("line %d: %s gave %d, not %d (%s)\n", __LINE__, #call, got_, (code), \
                        zdo_last_error());                                                   \
            return 1;                                                                        \
        }                                                                                    \
    } while (0)
#define TRUE(what)                                                \
    do {                                                          \
        if (!(what)) {                                            \
            std::printf("line %d: not %s\n", __LINE__, #what);    \
            return 1;                                             \
        }                                                         \
    } while (0)

// Addresses that overlap only where a test means them to.
template <typename T>
T *at(uint64_t slot, uint64_t byte = 0) {
    return reinterpret_cast<T *>((slot << 44) + byte + (1u << 20));
}

static zdo_plan *make(const std::vector<int64_t> &sizes) {
    zdo_plan *p = nullptr;
    if (build_range_map(sizes.data(), int32_t(sizes.size()), 1 << 20, 4, 1, &p) != ZDO_OK)
        return nullptr;
    p->d_table = &zdo::launches;   // a stand-in: taken back before the plan is destroyed
    p->device = 0;
    return p;
}
static void drop(zdo_plan *p) {
    p->d_table = nullptr;
    zdo_plan_destroy(p);
}

// With no tokens every token array may be NULL, grad_hidden among them: a call for
// the gradient by hidden alone is then a call with nothing to do.
static int no_tokens() {
    zdo_plan *p = make({24, 50 * 16 + 3, 7});
    auto grad = [&](int64_t n, void *gh, uint16_t *grads) {
        const bool any = n > 0;
        return linear_cross_entropy_grad(p, 1, 50, 16, at<uint16_t>(1), any ? at<uint16_t>(2) : nullptr, 16,
                                         any ? at<int64_t>(3) : nullptr, n, any ? at<float>(4) : nullptr,
                                         any ? at<float>(5) : nullptr, gh, ZDO_BF16, 16, 0, grads, at<void>(8), nullptr);
    };
    WANT(ZDO_OK, grad(0, nullptr, nullptr));
    TRUE(zdo::ce.n == 0 && !zdo::ce.grad_hidden && !zdo::ce.grads);
    WANT(ZDO_OK, grad(0, nullptr, at<uint16_t>(7)));
    WANT(ZDO_OK, grad(0, at<void>(6), nullptr));
    WANT(ZDO_EINVAL, grad(1, nullptr, nullptr));
    drop(p);
    return 0;
}

// What the header says of the workspace's parts: a piece's d (both parts of it) and
// its copy of W take at most 256 MB each, or 256 rows of a piece for each token and
// column; the sums of splits at most 128 MB for each gradient.
static int documented_sizes() {
    using namespace zdo;
    std::mt19937_64 rng(5);
    auto some = [&](double most) { return int64_t(std::pow(most, double(rng() % 100001) / 1e5)); };
    constexpr int64_t kMB = 1 << 20, kRound = 256;   // parts are rounded up to 256 bytes
    for (int t = 0; t < 4000; ++t) {
        const int64_t n = t % 2 ? 1 + int64_t(rng() % 130) : some(double(kCeMaxN));
        const int64_t vocab = some(double(kVocabMaxRows)), any = some(double(kVocabMaxDim));
        const int64_t dim = t % 3 ? round_up(any, kDepth) : any;
        const bool in_place = dim % kDepth == 0 && rng() % 2;
        const CeLayout l = ce_layout(n, vocab, dim, in_place);
        TRUE(l.rest - l.d <= std::max(256 * kMB, 512 * l.parts * l.npad) + kRound);
        TRUE(in_place || l.d - l.w <= std::max(256 * kMB, 512 * l.kdim) + kRound);
        TRUE(l.splits == 1 || l.row_sum - l.sum <= 128 * kMB + kRound);
        TRUE(l.row_splits == 1 || 4 * l.row_splits * l.piece * l.kdim <= 128 * kMB);
    }
    return 0;
}

// Rows at a stride leave room between them: arrays whose rows lie in one another's
// gaps share no element, and are refused only where they do, or where their strides
// differ.
static int between_rows() {
    zdo_plan *p = make({24, 50 * 16 + 3, 7});
    const int64_t n = 10, d = 16, N = zdo_plan_buffer_numel(p);
    char *two = at<char>(6);   // rows of 32 or more bf16
    auto grad = [&](const void *h, int64_t hs, void *gh, int32_t type, int64_t ghs, const float *lse = at<float>(4),
                    int64_t rows = 10) {
        return linear_cross_entropy_grad(p, 1, 50, d, at<uint16_t>(1), static_cast<const uint16_t *>(h), hs,
                                         at<int64_t>(3), rows, lse, at<float>(5), gh, type, ghs, 0, at<uint16_t>(7),
                                         at<void>(8), nullptr);
    };
    // halves of one buffer, either way round, with room and without
    WANT(ZDO_OK, grad(two, 32, two + 32, ZDO_BF16, 32));
    WANT(ZDO_OK, grad(two + 32, 32, two, ZDO_BF16, 32));
    WANT(ZDO_OK, grad(two + 4, 40, two + 40, ZDO_BF16, 40));
    WANT(ZDO_OK, grad(two, 64, two + 64, ZDO_F32, 32));      // strides are equal in bytes
    WANT(ZDO_OK, grad(two, 32, two + 32 + 64 * 4, ZDO_BF16, 32));   // rows further on
    WANT(ZDO_OK, grad(two + 64 * 20, 32, two + 32, ZDO_BF16, 32));
    // one element shared
    WANT(ZDO_EALIAS, grad(two, 32, two + 30, ZDO_BF16, 32));
    WANT(ZDO_EALIAS, grad(two, 32, two + 34, ZDO_BF16, 32));
    WANT(ZDO_EALIAS, grad(two + 30, 32, two, ZDO_BF16, 32));
    WANT(ZDO_EALIAS, grad(two + 34, 32, two, ZDO_BF16, 32));
    WANT(ZDO_EALIAS, grad(two, 32, two, ZDO_BF16, 32));
    WANT(ZDO_EALIAS, grad(two, 32, two + 64 * 3, ZDO_BF16, 32));
    WANT(ZDO_EALIAS, grad(two, 31, two + 32, ZDO_BF16, 31));
    WANT(ZDO_EALIAS, grad(two, 32, two + 32, ZDO_F32, 16));
    WANT(ZDO_EALIAS, grad(two, 32, two + 32, ZDO_BF16, 48));   // strides that differ: by their whole extents
    WANT(ZDO_EALIAS, grad(two, 32, two + 32, ZDO_BF16, 64));
    // the last row ends the extent, and what lies behind it is free
    WANT(ZDO_OK, grad(two, 32, two + 64 * (n - 1) + 32, ZDO_BF16, 64));
    WANT(ZDO_EALIAS, grad(two, 32, two + 64 * (n - 1) + 30, ZDO_BF16, 64));
    // an array without gaps between two rows, or across one
    WANT(ZDO_OK, grad(at<char>(2), 16, two + 0, ZDO_BF16, 64, reinterpret_cast<float *>(two + 32)));
    WANT(ZDO_OK, grad(at<char>(2), 16, two + 64, ZDO_BF16, 64, reinterpret_cast<float *>(two + 64 * 3 - 40)));
    WANT(ZDO_EALIAS, grad(at<char>(2), 16, two + 64, ZDO_BF16, 64, reinterpret_cast<float *>(two + 64 * 3 - 36)));
    WANT(ZDO_OK, grad(at<char>(2), 16, two + 64, ZDO_BF16, 64, reinterpret_cast<float *>(two + 64 + 32 + 128 * 4)));
    WANT(ZDO_EALIAS, grad(at<char>(2), 16, two, ZDO_BF16, 64, reinterpret_cast<float *>(two + 28)));
    WANT(ZDO_EALIAS, grad(at<char>(2), 16, two, ZDO_BF16, 32, reinterpret_cast<float *>(two + 32)));   // longer than a gap
    // one row: its stride says nothing
    WANT(ZDO_OK, grad(two, 1, two + 32, ZDO_BF16, -5, at<float>(4), 1));
    WANT(ZDO_EALIAS, grad(two, 32, two + 30, ZDO_BF16, 32, at<float>(4), 1));

    // out between the parameters' elements is never free; tokens between out's rows are
    WANT(ZDO_EALIAS, embedding_lookup(p, 1, 50, d, at<uint16_t>(1), at<int64_t>(2), n, 1.0f, at<uint16_t>(1) + N - 16 * 2,
                                      ZDO_BF16, 32, nullptr));
    WANT(ZDO_OK, embedding_lookup(p, 1, 50, d, at<uint16_t>(1), at<int64_t>(6, 32), 4, 1.0f, two, ZDO_BF16, 32, nullptr));
    // against every pair of elements, small sizes
    std::mt19937_64 rng(3);
    long apart = 0, shared = 0;
    for (int t = 0; t < 200000; ++t) {
        const int64_t ra = 1 + int64_t(rng() % 4), rb = 1 + int64_t(rng() % 4), da = 1 + int64_t(rng() % 5), db = 1 + int64_t(rng() % 5);
        const int64_t sa = da + int64_t(rng() % 8), sb = rng() % 2 ? std::max(sa, db) : db + int64_t(rng() % 8);
        const uintptr_t pa = 1000 + rng() % 40, pb = 1000 + rng() % 40;
        auto rows = [](uintptr_t at, int64_t n, int64_t dim, int64_t stride) {
            return zdo::span_of_rows(reinterpret_cast<void *>(at), n, dim, stride, 1);
        };
        bool share = false;
        for (int64_t i = 0; i < ra * da; ++i)
            for (int64_t k = 0; k < rb * db; ++k)
                share |= pa + uintptr_t(i / da * sa + i % da) == pb + uintptr_t(k / db * sb + k % db);
        const bool said = zdo::overlap(rows(pa, ra, da, sa), rows(pb, rb, db, sb));
        TRUE(!share || said);   // what is shared is refused
        // and the rest is let through where the strides are equal, or an array has no gaps and fits in one
        const bool gaps_a = ra > 1 && sa > da, gaps_b = rb > 1 && sb > db;
        if (!share && gaps_a && gaps_b && sa == sb)
            TRUE(!said);
        apart += !said;
        shared += share;
    }
    TRUE(apart > 10000 && shared > 10000);
    drop(p);
    return 0;
}

int main() {
    if (no_tokens() || documented_sizes() || between_rows())
        return 1;
    std::printf("ok: calls that the header allows\n");
    return 0;
}
