// Launch arguments, workspace layouts and launchers of the vocabulary
// matrix's kernels (vocab_kernels.hip, vocab_gemm.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "zdo_internal.h"

namespace zdo {

constexpr int64_t kVocabMaxN = int64_t(1) << 30;
constexpr int64_t kCeMaxN = int64_t(1) << 22;  // so that tiles are numbered in 32 bits
constexpr int64_t kVocabMaxRows = int64_t(1) << 30;
constexpr int64_t kVocabMaxDim = int64_t(1) << 20;
constexpr int64_t kVocabMaxStride = int64_t(1) << 30;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// ---- embedding -------------------------------------------------------------------

struct LookupArgs {
    const uint16_t *w;  // row 0
    int64_t vocab, dim;
    const int64_t *tokens;
    int64_t n;
    float scale;
    void *out;
    int32_t f32;
    int64_t stride;
};

// Sorted positions that a wave sums (see runs_kernel): at most its 64 lanes;
// with few positions fewer each, so that the chip has waves enough (8,192
// tokens of GPT-2 small: 8.4 us by 8, 11.6 by 16, 19 by 32; 131,072: the sums
// take the same at 16 and 64, and joining the parts 39 us at 16, 13 at 64). Rows of
// more columns make more waves, which the rule does not look at: 8,192 tokens of
// Llama-3-8B spend 19 of 233 us in joining, most workgroups finding nothing to join.
inline int rows_chunk(int64_t n) { return n >= 65536 ? 64 : n >= 32768 ? 32 : n >= 16384 ? 16 : 8; }

struct RowsArgs {
    uint16_t *g;  // the parameter's first element
    int64_t numel, vocab, dim;
    const int64_t *tokens;
    int64_t n;
    const void *x;
    int32_t f32;
    int64_t stride;
    float scale;
    int32_t accumulate;
    void *workspace;
};

// Up to this many positions are not sorted at all (see few_kernel; GPT-2 small, 400
// tokens 14.4 us, sorted 21.0; 1,024 tokens 20.4 and 22.2, but 32.4 and 25.8 where
// all of them are the same token, which one workgroup a column sums).
constexpr int64_t kFewTokens = 512;

// Up to this many positions are sorted by counting, in one launch (see
// rank_kernel, which holds as many keys in 32 KB of LDS); more by digits (GPT-2 small:
// 8,192 tokens 33 us, by digits 50; 16,384 by digits 52, by counting 56, so that they
// would cross a little below that).
constexpr int64_t kRankMax = 8192;
// Sorting by digits: positions a workgroup takes (few, so that there are
// workgroups enough; more where the scan of a digit's counts would weigh: of 50,257
// rows, 2^20 tokens of 64 columns 207 us by 1024, 251 by 8192; 2^26 of 4 columns
// 10.2 and 9.9 ms), and most bins of a digit.
inline int sort_items(int64_t n) { return n <= (int64_t(1) << 20) ? 1024 : 8192; }
constexpr int kSortBins = 512;

// The workspace of embedding_grad. Keys and positions lie in two sets, from
// one to the other a pass.
struct RowsLayout {
    int64_t blocks, chunks;
    int32_t chunk, items;
    int64_t key[2], pos[2], hist, part, bytes;
};

inline RowsLayout rows_layout(int64_t n, int64_t dim) {
    RowsLayout l{};
    l.items = sort_items(n);
    l.blocks = ceil_div(n, l.items);
    l.chunk = rows_chunk(n);
    l.chunks = ceil_div(n, l.chunk);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    for (int i = 0; i < 2; ++i) {
        l.key[i] = take(4 * n);
        l.pos[i] = take(4 * n);
    }
    l.hist = take(n > kRankMax ? 4 * kSortBins * (l.blocks + 1) : 0);
    l.part = take(4 * 2 * l.chunks * dim);
    l.bytes = std::max<int64_t>(at, 256);
    return l;
}

// ---- cross entropy -----------------------------------------------------------------

// C[m][n] = sum over k of A[m][k] B[n][k], in tiles (vocab_gemm.hip). A and B
// are bf16, rows of k (long) or, for each k, a row of m or n (wide), 16-byte
// aligned, strides of a multiple of 8 elements; long rows have a multiple of
// kDepth elements, wide ones at least m or n up to a multiple of 8. Which is
// which, and what becomes of C, is the epilogue's:
//   kScore, kDiff: A and B long; kSum: A wide, B long (k of it up to a multiple
//   of kDepth: zeros); kRows, kParts: A wide (with zero rows from k on, up to a
//   multiple of kDepth), B wide (finite ones).
constexpr int kDepth = 64;

enum Epilogue : int { kScore, kDiff, kSum, kRows, kParts };

struct GemmArgs {
    const uint16_t *a, *b;
    int64_t lda, ldb;
    int64_t m, n, k;
    int32_t splits;  // of k, each with an output of its own (kSum, kParts)

    // kScore, kDiff: m are a piece's rows of W, n tokens
    const int64_t *targets;
    int64_t row0;  // the piece's first row
    int64_t vocab;
    // kScore: per tile of rows and token the largest logit and the sum of
    // exp(logit - it), and the target's logit
    float2 *part;
    int64_t tile0;  // the piece's first tile
    float *pick;
    // kDiff: d in bf16, [n][m], zero up to the next multiple of kDepth of both; if
    // not NULL, low: what that rounding left, in bf16; rest: of the target's d, what
    // the rounding left
    const float *lse, *weight;
    uint16_t *d, *low;
    int64_t ldd;
    float *rest;

    // kSum, kParts: fp32 [split][n][lds], added to what is there unless `first`
    float *sum;
    int64_t lds;
    int32_t first;

    // kRows: bf16 rows n of m elements
    uint16_t *rows;
    int32_t accumulate;
};

// Tiles are 256 x 256, one workgroup a compute unit, or 128 x 128, two; the partial
// results of kScore are laid out for the smaller ones. Which of them, how many
// splits and pieces: by the time that rounds of tiles over the chip's 256 compute
// units take, kRoundK for each k of a round of large tiles (1.3 PFLOP/s) and
// kRoundOwn of its own for each round, in us. A round of 512 small tiles has half
// the work and takes 0.62 of a large one's time, of 256 and fewer 0.4 (loss of
// 128 tokens of Llama-3-8B by small tiles 197 us, by large ones 234; 8,192 tokens
// of GPT-2 small 653 and 540; loss and gradients of those with this choice 2.44 ms,
// at 0.5 and 0.3 2.63, at 1.1 and 0.9 2.51; of 16,384 tokens 5.04, 5.49 and 5.04).
constexpr int kTileRowsMin = 128;
constexpr double kRoundK = 0.026, kRoundOwn = 5.0;
inline double wide_rounds(int64_t m, int64_t n, int64_t splits) {
    return double(ceil_div(ceil_div(m, 256) * ceil_div(n, 256) * splits, 256));
}
inline double small_rounds(int64_t m, int64_t n, int64_t splits) {
    const int64_t tiles = ceil_div(m, 128) * ceil_div(n, 128) * splits;
    return 0.62 * double(tiles / 512) + (tiles % 512 > 256 ? 0.62 : tiles % 512 ? 0.4 : 0.0);
}
inline bool wide_tiles(int64_t m, int64_t n, int64_t splits) {
    return wide_rounds(m, n, splits) <= small_rounds(m, n, splits);
}
inline int64_t tile_rows(int64_t m, int64_t n) { return wide_tiles(m, n, 1) ? 256 : kTileRowsMin; }
inline double product_us(int64_t m, int64_t n, int64_t k, int64_t splits) {
    return std::min(wide_rounds(m, n, splits), small_rounds(m, n, splits)) *
           (kRoundOwn + kRoundK * double(ceil_div(k, splits)));
}

// The splits of a product's k, of at least 256 and with at most 2^25 sums in all,
// and the time with them: a sum and an addition take 8 bytes at 5 TB/s, and more
// than one split `join` us. (A training pass whose W's gradient is split so, and in
// one: 8,192 tokens of 256 rows of 768 77 us, 143; 16,384 of 300 rows of 512 86 and
// 224; of GPT-2 small's 50,257, in smaller pieces, 5.00 ms and 5.52.)
constexpr double kJoin = 4.0;
struct Splits {
    int64_t splits = 1;
    double us = 0.0;
};
inline Splits splits_of(int64_t m, int64_t n, int64_t k, double join) {
    Splits best{1, product_us(m, n, k, 1)};
    const double each = join > 0.0 ? 0.0 : double(n * m) * 8 / 5e6;
    best.us += each;
    for (int64_t s = 2; s <= k / 256 && s * n * round_up(m, kDepth) <= int64_t(1) << 25; s += s < 4 ? 1 : s / 2) {
        const double us = product_us(m, n, k, s) + join + double(s * n * m) * 8 / 5e6;
        if (us < best.us)
            best = {s, us};
    }
    return best;
}

// The loss of up to kThinTokens tokens may go by thin_score_kernel, kThinRows rows
// of W a tile.
constexpr int64_t kThinTokens = 32;
constexpr int kThinRows = 64;

// W's gradient of up to this many tokens takes d in two parts, the bf16 number
// nearest to it and what is left: its sums are then too short for the roundings to
// cancel, and its time is that of writing the gradient.
constexpr int64_t kTwoPartTokens = 128;

// Whether the products can read W where it lies: its rows are whole steps and
// 16-byte aligned. Else they take a copy, piece by piece.
inline bool rows_in_place(const void *w, int64_t dim) {
    return dim % kDepth == 0 && (reinterpret_cast<uintptr_t>(w) & 15) == 0;
}

// A call's workspace. The vocabulary is taken in pieces of `piece` rows: at most
// 2^27 elements of d, all its parts together (256 MB, the size of the Infinity
// Cache that they go through to the two products that read them), but at least 256
// rows, and, unless W is read in place, at most 2^27 elements of its copy
// (Llama-3-8B in place, by the smaller pieces: a training pass of 64 tokens 1.17 ms,
// 1.35; of 1,024 3.94 and 4.12).
struct CeLayout {
    int64_t kdim, npad, piece, vpad;  // dim, n and piece up to a multiple of kDepth
    int64_t splits;                   // of grad_hidden's sum
    int64_t row_splits;               // of W's gradient's
    int64_t parts;                    // of d: 2 for few tokens
    int64_t hidden, w, d, rest, sum, row_sum, part, pick, bytes;
};

inline CeLayout ce_layout(int64_t n, int64_t vocab, int64_t dim, bool in_place) {
    CeLayout l{};
    const int64_t some = std::max<int64_t>(n, 1);
    l.kdim = round_up(dim, kDepth);
    l.npad = round_up(some, kDepth);
    l.parts = n <= kTwoPartTokens ? 2 : 1;
    int64_t most = (int64_t(1) << 27) / (in_place ? l.parts * l.npad : std::max(l.parts * l.npad, l.kdim));
    most = std::max<int64_t>(256, most / 256 * 256);
    // the number of pieces, at least this many (few tokens: no more, their tiles
    // fill whole rounds anyway), and of splits of grad_hidden's sum over the
    // vocabulary (each adds to an fp32 sum of its own at 5 TB/s) and of W's gradient's
    // over the tokens (which takes another launch to add them)
    const int64_t least = ceil_div(vocab, most), tries = n <= 512 ? 1 : 4;
    double best = 0.0;
    for (int64_t p = least; p < least + tries && p <= vocab; ++p) {
        const int64_t piece = std::min(vocab, round_up(ceil_div(vocab, p), 256));
        const Splits sum = splits_of(dim, some, piece, 0.0), rows = splits_of(dim, piece, some, kJoin);
        const double us = double(ceil_div(vocab, piece)) * (product_us(piece, some, dim, 1) + sum.us + rows.us);
        if (best == 0.0 || us < best) {
            best = us;
            l.piece = piece;
            l.splits = sum.splits;
            l.row_splits = rows.splits;
        }
    }
    l.vpad = round_up(l.piece, kDepth);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    l.hidden = take(2 * l.parts * l.npad * l.kdim);
    l.w = take(in_place ? 0 : 2 * l.piece * l.kdim);
    const int64_t both = at;
    // the loss
    const int64_t tiles = ceil_div(vocab, l.piece) * ceil_div(l.piece, kTileRowsMin);
    l.part = take(8 * n * (n <= kThinTokens && !in_place ? std::max(tiles, ceil_div(vocab, kThinRows)) : tiles));
    l.pick = take(4 * n);
    const int64_t loss = at;
    // its gradient
    at = both;
    l.d = take(2 * l.parts * l.npad * l.vpad);
    l.rest = take(4 * n);
    l.sum = take(4 * l.splits * n * l.kdim);
    l.row_sum = take(l.row_splits > 1 ? 4 * l.row_splits * l.piece * l.kdim : 0);
    l.bytes = std::max<int64_t>(std::max(at, loss), 256);
    return l;
}

// What a caller provides, whether or not W will be read in place.
inline int64_t ce_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
    const int64_t copied = ce_layout(n, vocab, dim, false).bytes;
    return dim % kDepth ? copied : std::max(copied, ce_layout(n, vocab, dim, true).bytes);
}

struct CeArgs {
    const uint16_t *w;  // row 0
    int64_t vocab, dim;
    bool in_place;
    CeLayout layout;
    const uint16_t *hidden;
    int64_t hidden_stride;
    const int64_t *targets;
    int64_t n;
    float *loss;     // the loss: written
    float *lse;      // the loss: written; the gradient: read
    // the gradient
    const float *grad_loss;
    void *grad_hidden;  // may be NULL
    int32_t f32;
    int64_t grad_hidden_stride;
    uint16_t *grads;  // the parameter's first element; may be NULL
    int64_t numel;    // the parameter's
    int32_t accumulate;
    char *workspace;
};

hipError_t launch_lookup(const LookupArgs &a, hipStream_t stream);
hipError_t launch_rows(const RowsArgs &a, hipStream_t stream);
hipError_t launch_ce(const CeArgs &a, hipStream_t stream);
hipError_t launch_ce_grad(const CeArgs &a, hipStream_t stream);
hipError_t launch_thin_score(const GemmArgs &a, hipStream_t stream);
hipError_t launch_gemm(Epilogue e, const GemmArgs &a, hipStream_t stream);

// Elements [0, n) to zero.
hipError_t launch_zero(uint16_t *p, int64_t n, hipStream_t stream);

}  // namespace zdo
