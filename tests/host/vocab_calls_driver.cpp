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

int main() {
    if (no_tokens() || documented_sizes())
        return 1;
    std::printf("ok: calls that the header allows\n");
    return 0;
}
