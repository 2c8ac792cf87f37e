// Host-only exercise of the vocabulary calls' argument checks and workspace
// layouts, for a build with AddressSanitizer and UndefinedBehaviorSanitizer on
// the host code (tests/test_vocab_host.py). The current device is answered here
// and the plans are given a stand-in for their device table, so that the checks
// behind the plan's own are reached; the launchers are stand-ins that record
// what they were asked for. No device is used, and no pointer that is passed is
// ever followed.
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
static LookupArgs lookup;
static RowsArgs rows;
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
hipError_t launch_lookup(const LookupArgs &a, hipStream_t) { ++launches; lookup = a; return hipSuccess; }
hipError_t launch_rows(const RowsArgs &a, hipStream_t) { ++launches; rows = a; return hipSuccess; }
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

static zdo_plan *make(const std::vector<int64_t> &sizes, int64_t bucket, int32_t D, int32_t rank) {
    zdo_plan *p = nullptr;
    if (build_range_map(sizes.data(), int32_t(sizes.size()), bucket, D, rank, &p) != ZDO_OK)
        return nullptr;
    p->d_table = &zdo::launches;   // a stand-in: taken back before the plan is destroyed
    p->device = 0;
    return p;
}
static void drop(zdo_plan *p) {
    p->d_table = nullptr;
    zdo_plan_destroy(p);
}

// Where every parameter starts, against the layout's rule written out.
static int starts() {
    std::mt19937_64 rng(7);
    for (int t = 0; t < 300; ++t) {
        const int32_t n = 1 + int32_t(rng() % 40), D = 1 + int32_t(rng() % 64);
        std::vector<int64_t> sizes;
        for (int32_t i = 0; i < n; ++i)
            sizes.push_back(1 + int64_t(rng() % 300));
        const int64_t bucket = 1 + int64_t(rng() % 900);
        zdo_plan *p = make(sizes, bucket, D, int32_t(rng() % D));
        int64_t offset = 0, filled = 0;
        for (int32_t i = 0; i < n; ++i) {
            WANT(ZDO_OK, embedding_lookup(p, i, 1, sizes[size_t(i)], at<uint16_t>(1), at<int64_t>(2), 3, 1.0f, at<void>(3),
                                          ZDO_BF16, sizes[size_t(i)], nullptr));
            TRUE(zdo::lookup.w == at<uint16_t>(1) + offset + filled);
            filled += sizes[size_t(i)];
            if (filled >= bucket || i == n - 1) {
                offset += (filled + D - 1) / D * D;
                filled = 0;
            }
        }
        TRUE(offset == zdo_plan_buffer_numel(p));
        drop(p);
    }
    return 0;
}

// The layouts' parts lie one behind the other within the bytes that are asked
// for, and what the kernels assume of them holds.
static int layouts() {
    using namespace zdo;
    std::mt19937_64 rng(11);
    auto some = [&](double most) { return int64_t(std::pow(most, double(rng() % 100001) / 1e5)); };
    for (int t = 0; t < 3000; ++t) {
        const int64_t n = t % 50 == 0 ? 0 : some(double(kCeMaxN)), vocab = some(double(kVocabMaxRows));
        const int64_t any = some(double(kVocabMaxDim)), dim = rng() % 2 ? any : round_up(any, kDepth);
        const bool in_place = dim % kDepth == 0 && rng() % 2;
        const CeLayout l = ce_layout(n, vocab, dim, in_place);
        TRUE(l.kdim >= dim && l.kdim % kDepth == 0 && l.npad >= n && l.npad % kDepth == 0);
        TRUE(l.piece >= 1 && l.piece <= vocab && (l.piece == vocab || l.piece % 256 == 0));
        TRUE(l.vpad >= l.piece && l.vpad % kDepth == 0 && l.vpad < (int64_t(1) << 28));
        TRUE(l.splits >= 1 && l.splits <= 1 + l.piece / 256);
        TRUE(l.parts == (n <= kTwoPartTokens ? 2 : 1));
        // a tile's rows of d and hidden within 32 bits of bytes
        TRUE(256 * 2 * l.vpad < (int64_t(1) << 32) && 256 * 2 * l.kdim < (int64_t(1) << 32));
        TRUE(l.w - l.hidden >= 2 * l.parts * l.npad * l.kdim && (in_place || l.d - l.w >= 2 * l.piece * l.kdim));
        TRUE(l.rest - l.d >= 2 * l.parts * l.npad * l.vpad && l.sum - l.rest >= 4 * n);
        TRUE(l.row_sum - l.sum >= 4 * l.splits * n * l.kdim);
        TRUE(l.row_splits >= 1 && l.row_splits <= 1 + l.npad / 256);
        TRUE(l.row_splits == 1 || l.bytes - l.row_sum >= 4 * l.row_splits * l.piece * l.kdim);
        // the loss's partial results: every launch's tiles, whatever their size
        int64_t tiles = 0;
        for (int64_t row = 0; row < vocab && tiles < 400000; row += l.piece)
            tiles += ceil_div(std::min(l.piece, vocab - row), tile_rows(std::min(l.piece, vocab - row), std::max<int64_t>(n, 1)));
        TRUE(l.part >= l.w + (in_place ? 0 : 2 * l.piece * l.kdim) && l.pick - l.part >= 8 * n * std::min<int64_t>(tiles, 400000));
        const int64_t whole = std::max(l.piece, (int64_t(1) << 36) / l.npad / 256 * 256);
        tiles = 0;
        for (int64_t row = 0; row < vocab; row += whole)
            tiles += ceil_div(std::min(whole, vocab - row), tile_rows(std::min(whole, vocab - row), std::max<int64_t>(n, 1)));
        TRUE(l.pick - l.part >= 8 * n * tiles);
        if (n <= kThinTokens && !in_place)
            TRUE(l.pick - l.part >= 8 * n * ceil_div(vocab, kThinRows));
        TRUE(l.bytes - l.pick >= 4 * n);
        TRUE(l.bytes <= zdo_linear_cross_entropy_workspace_bytes(n, vocab, dim));
        // products are numbered in 32 bits
        TRUE(ceil_div(dim, 128) * ceil_div(std::max<int64_t>(n, 1), 128) * l.splits <= (int64_t(1) << 30));
        TRUE(ceil_div(l.piece, 128) * ceil_div(std::max<int64_t>(n, 1), 128) <= (int64_t(1) << 30));
        TRUE(ceil_div(dim, 128) * ceil_div(l.piece, 128) * l.row_splits <= (int64_t(1) << 30));

        const int64_t m = t % 50 == 0 ? 0 : some(double(kVocabMaxN));
        const RowsLayout r = rows_layout(m, dim);
        TRUE(r.pos[0] - r.key[0] >= 4 * m && r.key[1] - r.pos[0] >= 4 * m && r.pos[1] - r.key[1] >= 4 * m && r.hist - r.pos[1] >= 4 * m);
        TRUE(r.chunk >= 1 && r.chunk <= 64 && r.chunks * r.chunk >= m && r.blocks * r.items >= m && r.items % 256 == 0);
        TRUE(m <= kRankMax || r.part - r.hist >= 4 * kSortBins * (r.blocks + 1));
        TRUE(r.bytes - r.part >= 8 * r.chunks * dim && r.bytes == zdo_embedding_grad_workspace_bytes(m, dim));
    }
    for (int64_t bad : {int64_t(-1), kVocabMaxN + 1})
        TRUE(zdo_embedding_grad_workspace_bytes(bad, 8) == -1);
    for (int64_t bad : {int64_t(0), int64_t(-5), kVocabMaxDim + 1}) {
        TRUE(zdo_embedding_grad_workspace_bytes(8, bad) == -1);
        TRUE(zdo_linear_cross_entropy_workspace_bytes(8, 8, bad) == -1);
    }
    TRUE(zdo_linear_cross_entropy_workspace_bytes(kCeMaxN + 1, 8, 8) == -1);
    TRUE(zdo_linear_cross_entropy_workspace_bytes(-1, 8, 8) == -1);
    TRUE(zdo_linear_cross_entropy_workspace_bytes(8, 0, 8) == -1);
    TRUE(zdo_linear_cross_entropy_workspace_bytes(8, kVocabMaxRows + 1, 8) == -1);
    return 0;
}

static int refusals() {
    zdo_plan *p = make({24, 50 * 16 + 3, 7}, 1 << 20, 4, 1);
    const int64_t N = zdo_plan_buffer_numel(p), V = 50, d = 16, n = 10;
    uint16_t *params = at<uint16_t>(1), *grads = at<uint16_t>(2), *h = at<uint16_t>(3), *gh = at<uint16_t>(4);
    int64_t *t = at<int64_t>(5);
    float *loss = at<float>(6), *lse = at<float>(7), *w = at<float>(8);
    void *ws = at<void>(9);
    const int64_t rb = zdo_embedding_grad_workspace_bytes(n, d), cb = zdo_linear_cross_entropy_workspace_bytes(n, V, d);
    const long before = zdo::launches;

    auto look = [&](zdo_plan *pl, int32_t i, int64_t v, int64_t dim, const uint16_t *pa, const int64_t *tk, int64_t c, void *o, int32_t ty, int64_t st) {
        return embedding_lookup(pl, i, v, dim, pa, tk, c, 1.0f, o, ty, st, nullptr);
    };
    WANT(ZDO_EINVAL, look(nullptr, 1, V, d, params, t, n, h, 0, d));
    for (int32_t i : {-1, 3, 1 << 30})
        WANT(ZDO_EINVAL, look(p, i, V, d, params, t, n, h, 0, d));
    for (int64_t v : {int64_t(0), int64_t(-1), V + 1, zdo::kVocabMaxRows, zdo::kVocabMaxRows + 1, INT64_MAX})
        WANT(ZDO_EINVAL, look(p, 1, v, d, params, t, n, h, 0, d));
    for (int64_t dim : {int64_t(0), int64_t(-1), d + 1, zdo::kVocabMaxDim, zdo::kVocabMaxDim + 1, INT64_MAX})
        WANT(ZDO_EINVAL, look(p, 1, V, dim, params, t, n, h, 0, dim));
    for (int64_t c : {int64_t(-1), zdo::kVocabMaxN + 1, INT64_MAX})
        WANT(ZDO_EINVAL, look(p, 1, V, d, params, t, c, h, 0, d));
    WANT(ZDO_EINVAL, look(p, 1, V, d, nullptr, t, n, h, 0, d));
    WANT(ZDO_EALIGN, look(p, 1, V, d, at<uint16_t>(1, 8), t, n, h, 0, d));
    WANT(ZDO_EINVAL, look(p, 1, V, d, params, nullptr, n, h, 0, d));
    WANT(ZDO_EALIGN, look(p, 1, V, d, params, at<int64_t>(5, 4), n, h, 0, d));
    WANT(ZDO_EINVAL, look(p, 1, V, d, params, t, n, nullptr, 0, d));
    WANT(ZDO_EALIGN, look(p, 1, V, d, params, t, n, at<void>(3, 1), 0, d));
    WANT(ZDO_EALIGN, look(p, 1, V, d, params, t, n, at<void>(3, 2), 1, d));
    for (int32_t ty : {-1, 2})
        WANT(ZDO_EINVAL, look(p, 1, V, d, params, t, n, h, ty, d));
    for (int64_t st : {int64_t(0), d - 1, int64_t(-16), zdo::kVocabMaxStride + 1, INT64_MAX})
        WANT(ZDO_EINVAL, look(p, 1, V, d, params, t, n, h, 0, st));
    WANT(ZDO_EALIAS, look(p, 1, V, d, params, t, n, params + N - 1, 0, d));
    WANT(ZDO_EALIAS, look(p, 1, V, d, params, t, n, t + n - 1, 0, d));
    TRUE(zdo::launches == before);
    WANT(ZDO_OK, look(p, 1, V, d, params, t, n, params + N, 0, d));
    WANT(ZDO_OK, look(p, 1, V, d, params, t, 1, at<void>(3, 2), 0, -7));   // one row: the stride is not used
    WANT(ZDO_OK, look(p, 1, V, d, params, nullptr, 0, nullptr, 1, 0));
    TRUE(zdo::launches == before + 3);

    auto grad = [&](int64_t v, const int64_t *tk, int64_t c, const void *x, int32_t ty, int64_t st, uint16_t *g, void *s) {
        return embedding_grad(p, 1, v, d, tk, c, x, ty, st, 1.0f, 0, g, s, nullptr);
    };
    WANT(ZDO_EINVAL, grad(V + 1, t, n, h, 0, d, grads, ws));
    WANT(ZDO_EINVAL, grad(V, nullptr, n, h, 0, d, grads, ws));
    WANT(ZDO_EINVAL, grad(V, t, -1, h, 0, d, grads, ws));
    WANT(ZDO_EINVAL, grad(V, t, n, nullptr, 0, d, grads, ws));
    WANT(ZDO_EINVAL, grad(V, t, n, h, 3, d, grads, ws));
    WANT(ZDO_EINVAL, grad(V, t, n, h, 0, d - 1, grads, ws));
    WANT(ZDO_EINVAL, grad(V, t, n, h, 0, d, nullptr, ws));
    WANT(ZDO_EINVAL, grad(V, t, n, h, 0, d, grads, nullptr));
    WANT(ZDO_EALIGN, grad(V, t, n, h, 0, d, at<uint16_t>(2, 2), ws));
    WANT(ZDO_EALIGN, grad(V, t, n, h, 0, d, grads, at<void>(9, 8)));
    WANT(ZDO_EALIAS, grad(V, t, n, h, 0, d, grads, at<void>(2, 16)));
    WANT(ZDO_EALIAS, grad(V, t, n, h, 0, d, at<uint16_t>(9, uint64_t(rb) - 16), ws));
    WANT(ZDO_EALIAS, grad(V, t, n, grads + N - 1, 0, d, grads, ws));
    WANT(ZDO_EALIAS, grad(V, at<int64_t>(9, 64), n, h, 0, d, grads, ws));
    WANT(ZDO_OK, grad(V, t, n, h, 0, d, at<uint16_t>(9, uint64_t(rb)), ws));
    TRUE(zdo::launches == before + 4 && zdo::rows.g == at<uint16_t>(9, uint64_t(rb)) + 24 && zdo::rows.numel == 50 * 16 + 3);

    auto ce = [&](const uint16_t *x, int64_t st, const int64_t *tk, int64_t c, float *a, float *b, void *s) {
        return linear_cross_entropy(p, 1, V, d, params, x, st, tk, c, a, b, s, nullptr);
    };
    WANT(ZDO_EINVAL, ce(nullptr, d, t, n, loss, lse, ws));
    WANT(ZDO_EINVAL, ce(h, d - 1, t, n, loss, lse, ws));
    WANT(ZDO_EINVAL, ce(h, d, nullptr, n, loss, lse, ws));
    WANT(ZDO_EINVAL, ce(h, d, t, zdo::kCeMaxN + 1, loss, lse, ws));
    WANT(ZDO_EINVAL, ce(h, d, t, n, nullptr, lse, ws));
    WANT(ZDO_EINVAL, ce(h, d, t, n, loss, nullptr, ws));
    WANT(ZDO_EINVAL, ce(h, d, t, n, loss, lse, nullptr));
    WANT(ZDO_EALIGN, ce(h, d, t, n, at<float>(6, 2), lse, ws));
    WANT(ZDO_EALIGN, ce(h, d, t, n, loss, lse, at<void>(9, 4)));
    WANT(ZDO_EALIGN, ce(at<uint16_t>(3, 1), d, t, n, loss, lse, ws));
    WANT(ZDO_EALIAS, ce(h, d, t, n, loss, loss + n - 1, ws));
    WANT(ZDO_EALIAS, ce(h, d, t, n, loss, at<float>(9, uint64_t(cb) - 4), ws));
    WANT(ZDO_EALIAS, ce(at<uint16_t>(9, 2), d, t, n, loss, lse, ws));
    WANT(ZDO_EALIAS, ce(h, d, t, n, reinterpret_cast<float *>(params + 2), lse, ws));
    WANT(ZDO_OK, ce(at<uint16_t>(3, 2), d + 5, t, n, at<float>(6, 4), loss + 1 + n, ws));
    WANT(ZDO_OK, ce(nullptr, 0, nullptr, 0, nullptr, nullptr, ws));
    TRUE(zdo::launches == before + 6);

    auto ceg = [&](const float *l, const float *x, void *g, int32_t ty, int64_t st, uint16_t *gr, void *s) {
        return linear_cross_entropy_grad(p, 1, V, d, params, h, d, t, n, l, x, g, ty, st, 1, gr, s, nullptr);
    };
    WANT(ZDO_EINVAL, ceg(nullptr, w, gh, 0, d, grads, ws));
    WANT(ZDO_EINVAL, ceg(lse, nullptr, gh, 0, d, grads, ws));
    WANT(ZDO_EINVAL, ceg(lse, w, nullptr, 0, d, nullptr, ws));
    WANT(ZDO_EINVAL, ceg(lse, w, gh, 2, d, grads, ws));
    WANT(ZDO_EINVAL, ceg(lse, w, gh, 0, d - 1, grads, ws));
    WANT(ZDO_EINVAL, ceg(lse, w, gh, 0, d, grads, nullptr));
    WANT(ZDO_EALIGN, ceg(lse, w, at<void>(4, 2), 1, d, grads, ws));
    WANT(ZDO_EALIGN, ceg(at<float>(7, 1), w, gh, 0, d, grads, ws));
    WANT(ZDO_EALIGN, ceg(lse, w, gh, 0, d, at<uint16_t>(2, 2), ws));
    WANT(ZDO_EALIAS, ceg(lse, w, h, 0, d, grads, ws));
    WANT(ZDO_EALIAS, ceg(lse, w, gh, 0, d, params, ws));
    WANT(ZDO_EALIAS, ceg(lse, w, grads + N - 2, 1, d, grads, ws));
    WANT(ZDO_EALIAS, ceg(lse, w, gh, 0, d, grads, at<void>(2, 32)));
    WANT(ZDO_EALIAS, ceg(at<float>(9, 4), w, gh, 0, d, grads, ws));
    TRUE(zdo::launches == before + 6);
    WANT(ZDO_OK, ceg(lse, w, gh, 7, -1, nullptr, ws) == ZDO_EINVAL ? ZDO_OK : 1);   // the type of a grad_hidden that is there
    WANT(ZDO_OK, ceg(lse, w, nullptr, 7, -1, grads, ws));
    TRUE(!zdo::ce.grad_hidden && zdo::ce.grads == grads + 24 && zdo::ce.accumulate == 1);
    WANT(ZDO_OK, ceg(lse, w, gh, 1, d, nullptr, ws));
    TRUE(zdo::ce.grad_hidden == gh && !zdo::ce.grads && zdo::ce.f32 == 1);
    p->device = 1;
    WANT(ZDO_EINVAL, ceg(lse, w, gh, 1, d, nullptr, ws));
    p->device = 0;
    p->d_table = nullptr;
    WANT(ZDO_EHIP, ceg(lse, w, gh, 1, d, nullptr, ws));
    p->d_table = &zdo::launches;
    drop(p);
    return 0;
}

int main() {
    if (starts() || layouts() || refusals())
        return 1;
    std::printf("ok: starts, layouts, refusals\n");
    return 0;
}
