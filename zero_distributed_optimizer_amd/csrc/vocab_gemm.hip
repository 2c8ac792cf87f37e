// The matrix products of the cross entropy over the vocabulary (zdo_vocab.h)
// for gfx950: the logits of a piece of the vocabulary with the softmax's
// statistics or its gradient as epilogue, and the two gradients' products.
//
// One kernel: C[m][n] = sum over k of A[m][k] B[n][k] on
// v_mfma_f32_16x16x32_bf16. An operand lies in memory either "long", rows of k
// (W and hidden for the logits), or "wide", rows of m or n, one for each k (W
// for grad_hidden, hidden and d for W's gradient): gfx950's transposing LDS
// read gives the instruction its 8 consecutive k of a lane from either, so that
// no product needs a transposed copy. A workgroup takes a tile of C and steps
// over k by kDepth; a step's part of both operands comes to LDS straight from
// memory (long rows by whole cache lines), one step ahead, and from there to
// registers half a step ahead of the products.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device.h"
#include "vocab.h"
#include "vocab_device.h"

#pragma clang fp contract(off)

namespace zdo {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// 16 bytes a lane from base + its offset to LDS, lane after lane from `to` (the
// same for the whole wave) on. Written as an instruction, because the compiler
// would wait for all such copies before every LDS read (it cannot tell the slots
// apart); the waits are wait_and_meet's. It has no result in registers. m0, which
// holds the place in LDS, is named as overwritten, so that no value of the
// compiler's own is expected in it afterwards; the compiler warns that it would not
// save the register, which is not asked of it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16_to_lds(const char *base, uint32_t offset, const uint16_t *to) {
    const uint32_t lds = __builtin_amdgcn_readfirstlane(
        uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint16_t *)to)));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// Where a target's row lies among `count` rows from the piece's row `from` on; -1
// if it is none of them.
__device__ __forceinline__ int row_of_target(const GemmArgs &g, int64_t target, int64_t from, int count) {
    const int64_t r = target - g.row0 - from;
    return target >= 0 && target < g.vocab && r >= 0 && r < count ? int(r) : -1;
}

// One operand's part of a step in LDS, R rows or columns of C.
//
// Long: R rows of kDepth elements (128 bytes). The 16-byte chunk c of row r lies
// at c ^ spread(r), so that the rows that a fragment's read takes at one chunk
// are in different banks. The read gives lane l the 8 elements of k from (l / 16)
// * 8 of row l % 16.
//
// Wide: kDepth rows of R elements. A transposing read takes, in each 16 lanes, 4
// rows of 16 elements, a row's four 8-byte parts from 4 lanes, and gives lane i
// the 4 rows' element i; two of them are a fragment. The 32-byte unit u of row r
// lies at u ^ spread(r), so that the 8 rows that 32 lanes read are in different
// banks.
template <int R, int kWaves, bool kWide>
struct Operand {
    static constexpr int kLoads = R * kDepth * 2 / 1024 / kWaves;  // of 1 KB, a wave
    static constexpr int kRowBytes = kWide ? R * 2 : kDepth * 2, kChunks = kRowBytes / 16;
    const char *base, *from;
    uint32_t off[kLoads];
    int64_t step;   // bytes from one step's part to the next
    uint32_t ld2;   // bytes from row to row
    int left;       // wide: rows of k that there are from base on
    int lane, load0, last_chunk;

    static __device__ __forceinline__ int spread(int r) {
        return kWide ? (r & 3) | ((r >> 3) & 1) << 2 : r & 7;
    }
    __device__ __forceinline__ int row_of(int i) const { return (load0 + i) * (64 / kChunks) + lane / kChunks; }
    // The chunk of its row that lane's 16 bytes of load i come from.
    __device__ __forceinline__ int chunk_of(int i) const {
        const int r = row_of(i), p = lane % kChunks;
        if constexpr (kWide) {
            const int c = ((p >> 1) ^ spread(r)) * 2 + (p & 1);
            return c < last_chunk ? c : last_chunk;
        } else {
            return p ^ spread(r);
        }
    }

    // Rows or columns [x0, x0 + R) of `count`, k from k0 on of `have`. What lies
    // behind the last is read as the last: it is not kept (m and n), or meets
    // zeros of the other operand (k).
    __device__ __forceinline__ void start(const uint16_t *p, int64_t ld, int64_t x0, int64_t count, int64_t k0,
                                          int64_t have, int wave, int l) {
        lane = l;
        load0 = wave * kLoads;
        ld2 = uint32_t(ld * 2);
        if constexpr (kWide) {
            base = reinterpret_cast<const char *>(p + k0 * ld + x0);
            step = ld * 2 * kDepth;
            left = int(have - k0 < (1 << 30) ? have - k0 : 1 << 30);
            const int64_t chunks = (count - x0 + 7) / 8;   // rows are padded to 8 elements
            last_chunk = chunks < kChunks ? int(chunks) - 1 : kChunks - 1;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                off[i] = uint32_t(row_of(i)) * ld2 + uint32_t(chunk_of(i)) * 16;
        } else {
            base = reinterpret_cast<const char *>(p + x0 * ld + k0);
            step = kDepth * 2;
            const int last = int(count - x0 < R ? count - x0 : R) - 1;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = row_of(i);
                off[i] = uint32_t(r < last ? r : last) * ld2 + uint32_t(chunk_of(i)) * 16;
            }
        }
    }
    // A step's copies: first next(), then each of them once.
    __device__ __forceinline__ void next() {
        if (kWide && left < kDepth) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = row_of(i);
                off[i] = uint32_t(r < left ? r : left - 1) * ld2 + uint32_t(chunk_of(i)) * 16;
            }
        }
        from = base;
        base += step;
        if (kWide)
            left -= kDepth;
    }
    __device__ __forceinline__ void copy(int i, uint16_t *stage) const {
        copy16_to_lds(from, off[i], stage + (load0 + i) * 512);
    }
};

// A wave's fragments of an operand: T of 16 rows or columns from x.
template <int R, int T, bool kWide>
struct Fragments {
    int at[kWide ? T : 2];

    __device__ __forceinline__ Fragments(int x, int lane) {
        if constexpr (kWide) {
            const int r = (lane >> 4) * 8 + ((lane & 15) >> 2), spread = Operand<R, 1, true>::spread(r);
#pragma unroll
            for (int i = 0; i < T; ++i)
                at[i] = r * R + (((x >> 4) + i) ^ spread) * 16 + (lane & 3) * 4;
        } else {
#pragma unroll
            for (int half = 0; half < 2; ++half)
                at[half] = (x + (lane & 15)) * kDepth +
                           ((half * 4 + (lane >> 4)) ^ Operand<R, 1, false>::spread(lane & 15)) * 8;
        }
    }
    // Of k, the first or the second half.
    __device__ __forceinline__ bf16x8 read(const uint16_t *stage, int i, int half) const {
        if constexpr (kWide) {
            const uint16_t *p = stage + at[i] + half * (kDepth / 2) * R;
            const bf16x4 lo = transposed(p), hi = transposed(p + 4 * R);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            return *reinterpret_cast<const bf16x8 *>(stage + at[half] + i * 16 * kDepth);
        }
    }
    static __device__ __forceinline__ bf16x4 transposed(const uint16_t *p) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) bf16x4 *)p);
    }
};

// Waits until at most `kLeft` of this wave's copies to LDS are still on their
// way and its LDS reads are done, then for the other waves to get here.
template <int kLeft>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
}

// Bound by the matrix cores and the power they draw (busy in 62 to 75% of the cycles,
// at 1.85 to 1.9 of 2.4 GHz): Llama-3-8B, 4,096 tokens, the logits 2.91 ms (1,480
// TFLOP/s), d 3.11, grad_hidden's sum 3.00, W's gradient 3.28 ms (medians; a call's
// first passes are up to 15% longer, until the clock has settled). With few steps a
// tile the epilogues weigh, the cores idle meanwhile: GPT-2 small's 12, 8,192 tokens,
// the logits 0.56 ms (1,130 TFLOP/s). Tiles of 256 x 256 read each operand from the caches
// half as often as those of 128 x 128, of which two share a compute unit.
template <int BM, int BN, int WM, int WN, int E>
__global__ __launch_bounds__(WM *WN * 64, 2) void gemm_kernel(GemmArgs g) {
    constexpr int kWaves = WM * WN;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;   // 16 x 16 tiles a wave
    constexpr bool kWideB = E == kRows || E == kParts, kWideA = E == kSum || kWideB;
    __shared__ __align__(1024) uint16_t stage[2][(BM + BN) * kDepth];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave / WN, wn = wave % WN;
    const int tiles_m = int((g.m + BM - 1) / BM), tiles_n = int((g.n + BN - 1) / BN);
    const int tiles = tiles_m * tiles_n * g.splits;
    const Fragments<BM, TM, kWideA> frag_a(wm * (BM / WM), lane);
    const Fragments<BN, TN, kWideB> frag_b(wn * (BN / WN), lane);

    for (int id = blockIdx.x; id < tiles; id += gridDim.x) {
        // The tiles of an XCD (workgroups go to the 8 of them in turn) follow
        // each other; in that order, 4 tiles along m at each n.
        const int each = tiles / 8, more = tiles % 8, x = id % 8;
        int t = x * each + (x < more ? x : more) + id / 8;
        const int split = t / (tiles_m * tiles_n);
        t -= split * tiles_m * tiles_n;
        const int band = t / (4 * tiles_n), wide = tiles_m - band * 4 < 4 ? tiles_m - band * 4 : 4;
        const int tm = band * 4 + (t - band * 4 * tiles_n) % wide, tn = (t - band * 4 * tiles_n) / wide;
        const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN;

        const int steps_all = int((g.k + kDepth - 1) / kDepth);
        const int first = int(int64_t(steps_all) * split / g.splits);
        const int steps = int(int64_t(steps_all) * (split + 1) / g.splits) - first;

        Operand<BM, kWaves, kWideA> a;
        Operand<BN, kWaves, kWideB> b;
        a.start(g.a, g.lda, m0, g.m, int64_t(first) * kDepth, g.k, wave, lane);
        b.start(g.b, g.ldb, n0, g.n, int64_t(first) * kDepth, g.k, wave, lane);

        f32x4 acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = f32x4{0, 0, 0, 0};

        constexpr int kCopies = a.kLoads + b.kLoads;   // a wave's, of a step
        auto next = [&] {
            a.next();
            b.next();
        };
        auto copy = [&](int i, int s) {
            if (i < a.kLoads)
                a.copy(i, stage[s]);
            else
                b.copy(i - a.kLoads, stage[s] + BM * kDepth);
        };
        bf16x8 fa[TM], fb[2][TN];
        // The products of half a step, whose fragments are in registers (fb[half]),
        // and meanwhile, where a fragment of A has been used, the next half's
        // from stage s and, if any, the copies to the other stage.
        auto products = [&](auto half, int s, auto copies) {
            constexpr int h = decltype(half)::value;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if constexpr (decltype(copies)::value)
#pragma unroll
                    for (int c = i * kCopies / TM; c < (i + 1) * kCopies / TM; ++c)
                        copy(c, s ^ 1);
#pragma unroll
                for (int j = i * TN / TM; j < (i + 1) * TN / TM; ++j)
                    fb[h ^ 1][j] = frag_b.read(stage[s] + BM * kDepth, j, h ^ 1);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[h][j], acc[i][j], 0, 0, 0);
                fa[i] = frag_a.read(stage[s], i, h ^ 1);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        constexpr std::integral_constant<int, 0> first_half;
        constexpr std::integral_constant<int, 1> second_half;
        constexpr std::true_type copies_yes;
        constexpr std::false_type copies_no;
        __syncthreads();   // the LDS is free
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (s < steps) {
                next();
#pragma unroll
                for (int c = 0; c < kCopies; ++c)
                    copy(c, s);
            }
        if (steps >= 2)
            wait_and_meet<kCopies>();
        else
            wait_and_meet<0>();
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[i] = frag_a.read(stage[0], i, 0);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[0][j] = frag_b.read(stage[0] + BM * kDepth, j, 0);
        int k = 0;
        for (; k + 2 < steps; ++k) {
            products(first_half, k & 1, copies_no);
            // step k is in registers in all waves, step k + 1 in LDS
            wait_and_meet<0>();
            next();
            products(second_half, (k + 1) & 1, copies_yes);
        }
        for (; k < steps; ++k) {
            products(first_half, k & 1, copies_no);
            wait_and_meet<0>();
            // (behind the last step the reads get whatever is there: unused)
            products(second_half, (k + 1) & 1, copies_no);
        }
        __syncthreads();   // LDS serves the epilogue

        // acc[i][j][r] is C[m][n] with, from the tile's corner,
        //   m = wm * BM / WM + i * 16 + (lane / 16) * 4 + r, n = wn * BN / WN + j * 16 + lane % 16
        // (as numbers that the compiler does not know from before: it would
        // compute the epilogue's addresses ahead of the tiles and spill them)
        int epi_lane = lane, epi_wave = wave;
        asm volatile("" : "+v"(epi_lane), "+s"(epi_wave));
        const int wave_m = epi_wave / WN * (BM / WM), wave_n = epi_wave % WN * (BN / WN);
        const int lane_m = (epi_lane >> 4) * 4, lane_n = epi_lane & 15;
        const int rows_in = int(g.m - m0 < BM ? g.m - m0 : BM), cols_in = int(g.n - n0 < BN ? g.n - n0 : BN);

        // all rows of the tile are there: then no element is asked for its row
        const bool whole = rows_in == BM;
        if constexpr (E == kScore) {
            float2 *red = reinterpret_cast<float2 *>(stage);   // [WM][BN]
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = wave_n + j * 16 + lane_n;
                // the target's row, from this wave's first, if it is one of its rows
                const int target = row_of_target(g, n < cols_in ? g.targets[n0 + n] : -1, m0 + wave_m, BM / WM);
                if (__any(target >= 0))
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (target == i * 16 + lane_m + r)
                                g.pick[n0 + n] = acc[i][j][r];
                if (!whole)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (wave_m + i * 16 + lane_m + r >= rows_in)
                                acc[i][j][r] = -INFINITY;
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        top = fmaxf(top, acc[i][j][r]);
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float base = base_of(top);
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        sum += __expf(acc[i][j][r] - base);
                sum += __shfl_xor(sum, 16);
                sum += __shfl_xor(sum, 32);
                if (epi_lane < 16)
                    red[epi_wave / WN * BN + n] = {top, sum};
            }
            __syncthreads();
            const int n = epi_wave * 64 + epi_lane;
            if (n < cols_in) {
                float2 all = red[n];
#pragma unroll
                for (int w = 1; w < WM; ++w)
                    all = join_softmax(all, red[w * BN + n]);
                g.part[(g.tile0 + tm) * g.n + n0 + n] = all;
            }
        } else if constexpr (E == kDiff) {
            // this wave's part of the tile, [n][m]
            constexpr int PM = BM / WM, PN = BN / WN;
            // calls for d in two parts have one small tile along n (in large ones the
            // second part's registers spill: 8,192 tokens of GPT-2 small 759 us, 724
            // without it)
            constexpr bool kLow = BM == kTileRowsMin;
            uint16_t *mine = reinterpret_cast<uint16_t *>(stage) + epi_wave * (PM * PN);
            uint32_t packed[4];
            // loads first (8,192 tokens of GPT-2 small 705 us, 693 so)
            int64_t named_row[TN];
            float lses[TN], weights[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = wave_n + j * 16 + lane_n;
                const bool in = n < cols_in;
                named_row[j] = in ? g.targets[n0 + n] : -1;
                lses[j] = in ? g.lse[n0 + n] : 0.0f;
                weights[j] = in ? g.weight[n0 + n] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = wave_n + j * 16 + lane_n;
                const bool named = named_row[j] >= 0 && named_row[j] < g.vocab;
                const int target = row_of_target(g, named_row[j], m0 + wave_m, PM);
                const float lse = named ? lses[j] : 0.0f, weight = named ? weights[j] : 0.0f;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][j][r] = __expf(acc[i][j][r] - lse);
                if (__any(target >= 0))
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (target == i * 16 + lane_m + r) {
                                acc[i][j][r] -= 1.0f;
                                const float d = acc[i][j][r] * weight;
                                g.rest[n0 + n] = d - lo_f32(to_bf16x2(d, 0.0f));
                            }
                if (!whole)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (wave_m + i * 16 + lane_m + r >= rows_in)
                                acc[i][j][r] = 0.0f;
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    // four bf16, and what their rounding left as four more, in the
                    // registers of the logits
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float x = acc[i][j][2 * h] * weight, y = acc[i][j][2 * h + 1] * weight;
                        const uint32_t high = to_bf16x2(x, y);
                        packed[h] = named ? high : 0u;
                        if constexpr (kLow) {
                            const uint32_t low = to_bf16x2(x - lo_f32(high), y - hi_f32(high));
                            packed[2 + h] = named ? low : 0u;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < (kLow ? 4 : 2); ++r)
                        acc[i][j][r] = __uint_as_float(packed[r]);
                }
            }
            // Chunks of 8 elements are moved within their row by the row's
            // number, so that neither the writes nor the reads meet in a bank.
            constexpr int CM = PM / 8;
            const int pad_m = (rows_in + kDepth - 1) / kDepth * kDepth;
            const int pad_n = (cols_in + kDepth - 1) / kDepth * kDepth;
            for (int part = 0; part < (kLow && g.low ? 2 : 1); ++part) {
                uint16_t *out = part ? g.low : g.d;
                if (part)
                    __syncthreads();
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int i = 0; i < TM; ++i) {
                        const int n = j * 16 + lane_n, c = i * 2 + (epi_lane >> 5);
                        *reinterpret_cast<u32x2 *>(
                            &mine[n * PM + (c ^ (n & (CM - 1))) * 8 + ((epi_lane >> 4) & 1) * 4]) =
                            part ? u32x2{__float_as_uint(acc[i][j][2]), __float_as_uint(acc[i][j][3])}
                                 : u32x2{__float_as_uint(acc[i][j][0]), __float_as_uint(acc[i][j][1])};
                    }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < PN * CM / 64; ++i) {
                    const int n = i * (64 / CM) + epi_lane / CM, c = epi_lane % CM;
                    if (wave_n + n < pad_n && wave_m + c * 8 < pad_m)
                        *reinterpret_cast<u32x4 *>(&out[(n0 + wave_n + n) * g.ldd + m0 + wave_m + c * 8]) =
                            *reinterpret_cast<const u32x4 *>(&mine[n * PM + (c ^ (n & (CM - 1))) * 8]);
                }
            }
        } else if constexpr (E == kSum || E == kParts) {
            // rows of the sum are padded to kDepth, so quads never pass their end
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = wave_n + j * 16 + lane_n;
                float *row = g.sum + ((int64_t(split) * g.n + n0 + n) * g.lds + m0);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int m = wave_m + i * 16 + lane_m;
                    if (n < cols_in && m < rows_in) {
                        f32x4 v = acc[i][j];
                        if (!g.first)
                            v += ldf4(row + m);
                        stf4(row + m, v);
                    }
                }
            }
        } else {
            // through LDS, in fp32, a wave's part [n][m] in as many passes as it
            // takes, so that rows are written by 16 bytes a lane and 256 or 128
            // bytes on end (Llama-3-8B's matrix from 64 tokens 443 us, 511 straight from
            // registers by 8 bytes; from 4,096 3.47 and 3.62 ms). Quads are moved within
            // their row by the row's number, so that the writes do not meet in a bank.
            constexpr int PM = BM / WM, PN = BN / WN, CM = PM / 8;
            constexpr int kPasses = BM * BN * 4 / int(sizeof(stage)), JN = TN / kPasses;
            float *mine = reinterpret_cast<float *>(stage) + epi_wave * (PM * PN / kPasses);
#pragma unroll
            for (int pass = 0; pass < kPasses; ++pass) {
                if (pass)
                    __syncthreads();
#pragma unroll
                for (int j = 0; j < JN; ++j)
#pragma unroll
                    for (int i = 0; i < TM; ++i) {
                        const int n = j * 16 + lane_n, q = i * 4 + (epi_lane >> 4);
                        *reinterpret_cast<f32x4 *>(&mine[n * PM + (q ^ (n & 15)) * 4]) = acc[i][pass * JN + j];
                    }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < JN * 16 * CM / 64; ++i) {
                    const int n = i * (64 / CM) + epi_lane / CM, c = epi_lane % CM;
                    const int at_n = wave_n + pass * JN * 16 + n, at_m = wave_m + c * 8;
                    if (at_n >= cols_in || at_m >= rows_in)
                        continue;
                    const f32x4 lo = *reinterpret_cast<const f32x4 *>(&mine[n * PM + (2 * c ^ (n & 15)) * 4]);
                    const f32x4 hi = *reinterpret_cast<const f32x4 *>(&mine[n * PM + ((2 * c + 1) ^ (n & 15)) * 4]);
                    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    uint16_t *row = g.rows + (n0 + at_n) * g.m + m0 + at_m;
                    if (at_m + 8 <= rows_in) {
                        loose_u32x4 *to = reinterpret_cast<loose_u32x4 *>(row);
                        if (g.accumulate) {
                            const u32x4 old = *to;
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                v[2 * r] += lo_f32(old[r]);
                                v[2 * r + 1] += hi_f32(old[r]);
                            }
                        }
                        // non-temporally: W, hidden and d stay in the caches
                        __builtin_nontemporal_store(u32x4{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]),
                                                          to_bf16x2(v[4], v[5]), to_bf16x2(v[6], v[7])},
                                                    to);
                    } else {
#pragma unroll
                        for (int r = 0; r < 7; ++r)
                            if (at_m + r < rows_in)
                                row[r] = uint16_t(to_bf16x2(g.accumulate ? v[r] + h_f32(row[r]) : v[r], 0.0f));
                    }
                }
            }
        }
    }
}

// The logits' statistics for few tokens, where reading W is all there is to do: a
// workgroup takes kThinRows rows of W, each of its 4 waves a quarter of k, and
// reads W from memory to registers as the instruction takes it (lane l: 16 bytes
// of row l % 16), the next 64 k while it multiplies these. Rows start anywhere
// and have any length; hidden comes out of the caches. The quarters are added
// through LDS. Bound by the L1 caches' address units, busy in 84% of the cycles: a lane's
// 16 bytes off their alignment count as 3.5 accesses of the cache on average (16 tokens of
// Llama-3-8B, off by an element: 1.05 GB in 482 us and 287 M accesses, where W in place
// takes 182 us and 33 M by copies of aligned 16 bytes).
template <int TN>
__global__ __launch_bounds__(256, 2) void thin_score_kernel(GemmArgs g) {
    constexpr int TM = kThinRows / 16;
    __shared__ f32x4 quarter[4][TM * TN][64];
    __shared__ float2 red[TM][TN * 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = int((g.m + kThinRows - 1) / kThinRows);
    const int64_t steps = g.k / 64, first = steps * wave / 4, last = steps * (wave + 1) / 4;   // and the rest of k

    // 8 elements from c on of a row of g.k, zeros behind its end: the row's last 8,
    // moved down
    auto load8 = [&](const uint16_t *row, int64_t c) {
        const int64_t past = c + 8 - g.k;   // of the 8
        u32x4 x = {0, 0, 0, 0};
        if (past >= 8)
            return x;
        if (g.k < 8) {
            for (int i = 0; i < 7; ++i)
                if (c + i < g.k)
                    x[i >> 1] |= uint32_t(row[c + i]) << (i & 1) * 16;
            return x;
        }
        x = *reinterpret_cast<const loose_u32x4 *>(row + (past > 0 ? g.k - 8 : c));
        if (past > 0) {
            uint64_t lo = uint64_t(x.y) << 32 | x.x, hi = uint64_t(x.w) << 32 | x.z;
            const int s = int(past) * 16;
            lo = s >= 64 ? hi >> (s - 64) : lo >> s | hi << (64 - s);
            hi = s >= 64 ? 0 : hi >> s;
            x = u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
        }
        return x;
    };
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t m0 = int64_t(tile) * kThinRows;
        const int rows_in = int(g.m - m0 < kThinRows ? g.m - m0 : kThinRows);
        // what lies behind the last row or token is read as the last, and not kept
        const uint16_t *a[TM], *b[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = i * 16 + (lane & 15);
            a[i] = g.a + (m0 + (r < rows_in ? r : rows_in - 1)) * g.lda;
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t n = j * 16 + (lane & 15);
            b[j] = g.b + (n < g.n ? n : g.n - 1) * g.ldb;
        }
        f32x4 acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = f32x4{0, 0, 0, 0};
        u32x4 fa[2][2][TM], fb[2][2][TN];
        auto load = [&](int set, int64_t step) {
            const int64_t c = step * 64 + (lane >> 4) * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    fa[set][h][i] = *reinterpret_cast<const loose_u32x4 *>(a[i] + c + h * 8);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    fb[set][h][j] = *reinterpret_cast<const loose_u32x4 *>(b[j] + c + h * 8);
            }
        };
        auto products = [&](int set) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, fa[set][h][i]), __builtin_bit_cast(bf16x8, fb[set][h][j]),
                            acc[i][j], 0, 0, 0);
        };
        if (first < last)
            load(0, first);
        for (int64_t k = first; k < last; k += 2) {
            if (k + 1 < last)
                load(1, k + 1);
            products(0);
            if (k + 1 >= last)
                break;
            if (k + 2 < last)
                load(0, k + 2);
            products(1);
        }
        if (wave == 3 && g.k % 64) {
            const int64_t c = g.k / 64 * 64 + (lane >> 4) * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    fa[0][h][i] = load8(a[i], c + h * 8);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    fb[0][h][j] = load8(b[j], c + h * 8);
            }
            products(0);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                quarter[wave][i * TN + j][lane] = acc[i][j];
        __syncthreads();
        // wave i: rows i * 16 + lane / 16 * 4 + r
        static_assert(TM == 4, "a wave for each 16 rows");
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            f32x4 z = quarter[0][wave * TN + j][lane];
            for (int w = 1; w < 4; ++w)
                z += quarter[w][wave * TN + j][lane];
            const int n = j * 16 + (lane & 15), m = wave * 16 + (lane >> 4) * 4;
            const int target = row_of_target(g, n < g.n ? g.targets[n] : -1, m0, kThinRows);
            float top = -INFINITY;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (m + r >= rows_in)
                    z[r] = -INFINITY;
                else if (m + r == target)
                    g.pick[n] = z[r];
                top = fmaxf(top, z[r]);
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                sum += __expf(z[r] - base_of(top));
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (lane < 16)
                red[wave][n] = {top, sum};
        }
        __syncthreads();
        const int n = threadIdx.x;
        if (n < g.n) {
            float2 all = red[0][n];
            for (int w = 1; w < TM; ++w)
                all = join_softmax(all, red[w][n]);
            g.part[(g.tile0 + tile) * g.n + n] = all;
        }
        __syncthreads();
    }
}

// Workgroups of a launch: one a tile, up to a number whose threads fit 32
// bits; more tiles are taken in turn. For the logits and d in large tiles, one a
// compute unit (8,192 tokens of GPT-2 small 588 and 700 us, 616 and 724 by one a
// tile; sums and rows take the same or, of few tokens, 5% more).
template <int BM, int BN, int WM, int WN, int E>
hipError_t launch(const GemmArgs &g, hipStream_t stream) {
    const int64_t tiles = ceil_div(g.m, BM) * ceil_div(g.n, BN) * g.splits;
    constexpr bool kStay = BM == 256 && (E == kScore || E == kDiff);
    const int64_t cap = std::min<int64_t>(kMaxGrid, kStay ? 256 : 1 << 21);
    gemm_kernel<BM, BN, WM, WN, E><<<unsigned(std::min(tiles, cap)), WM * WN * 64, 0, stream>>>(g);
    return hipGetLastError();
}

template <int E>
hipError_t launch_sized(const GemmArgs &g, hipStream_t stream) {
    const bool two_parts = E == kDiff && g.low;   // of few tokens: small tiles make them
    if (!two_parts && wide_tiles(g.m, g.n, g.splits))
        return launch<256, 256, 2, 4, E>(g, stream);
    return launch<128, 128, 2, 2, E>(g, stream);
}

}  // namespace

hipError_t launch_thin_score(const GemmArgs &g, hipStream_t stream) {
    const unsigned grid = unsigned(std::min<int64_t>(ceil_div(g.m, kThinRows), std::min<int64_t>(kMaxGrid, 1 << 21)));
    if (g.n <= 16)
        thin_score_kernel<1><<<grid, 256, 0, stream>>>(g);
    else
        thin_score_kernel<2><<<grid, 256, 0, stream>>>(g);
    return hipGetLastError();
}

hipError_t launch_gemm(Epilogue e, const GemmArgs &g, hipStream_t stream) {
    if (g.m <= 0 || g.n <= 0)
        return hipSuccess;
    if (ceil_div(g.m, kTileRowsMin) * ceil_div(g.n, kTileRowsMin) * g.splits > (int64_t(1) << 30))
        return hipErrorInvalidValue;   // tiles are numbered in 32 bits
    switch (e) {
    case kScore:
        return launch_sized<kScore>(g, stream);
    case kDiff:
        return launch_sized<kDiff>(g, stream);
    case kSum:
        return launch_sized<kSum>(g, stream);
    case kParts:
        return launch_sized<kParts>(g, stream);
    default:
        return launch_sized<kRows>(g, stream);
    }
}

}  // namespace zdo
