// The matrix products of the cross entropy over the vocabulary (zdo_vocab.h)
// for gfx950: the logits of a piece of the vocabulary with the softmax's
// statistics or its gradient as epilogue, and the two gradients' products.
//
// One kernel: C[m][n] = sum over k of A[m][k] B[n][k], both operands with k
// contiguous, on v_mfma_f32_16x16x32_bf16. A workgroup takes a tile of C; it
// stages kDepth columns of both operands at a time in LDS, straight from
// memory (16 bytes a lane), one step ahead of the products.
#include <hip/hip_runtime.h>

#include "device.h"
#include "vocab.h"

#pragma clang fp contract(off)

namespace zdo {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 or 16 bytes at any address that is aligned to an element.
template <typename V>
struct __attribute__((packed, aligned(2))) Loose {
    V v;
};

__device__ __forceinline__ void copy16_to_lds(const char *base, uint32_t offset, uint16_t *to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(base + offset),
                                     (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}

// exp(x - top) that is 1 at the top, whatever the top is (both infinite: the
// difference would be NaN).
__device__ __forceinline__ float exp_below(float x, float top) { return x == top ? 1.0f : __expf(x - top); }

template <int BM, int BN, int WM, int WN, int E>
__global__ __launch_bounds__(WM *WN * 64, 2) void gemm_kernel(GemmArgs g) {
    constexpr int kWaves = WM * WN;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;   // 16 x 16 tiles a wave
    constexpr int RA = BM / 8 / kWaves, RB = BN / 8 / kWaves;  // loads of 8 rows a wave
    // A step's rows of kDepth elements (128 bytes), A's then B's. The 16-byte
    // chunk c of row r lies at c ^ (r & 7), so that the 16 rows that a
    // fragment read takes at one chunk lie in different banks.
    __shared__ __align__(1024) uint16_t stage[2][(BM + BN) * kDepth];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave / WN, wn = wave % WN;
    const int tiles_m = int((g.m + BM - 1) / BM), tiles_n = int((g.n + BN - 1) / BN);
    const int tiles = tiles_m * tiles_n * g.splits;
    const int read_a = (wm * (BM / WM) + (lane & 15)) * kDepth;
    const int read_b = (BM + wn * (BN / WN) + (lane & 15)) * kDepth;
    const int chunk[2] = {((lane >> 4) ^ (lane & 7)) * 8, ((4 + (lane >> 4)) ^ (lane & 7)) * 8};

    for (int id = blockIdx.x; id < tiles; id += gridDim.x) {
        // The tiles of an XCD (workgroups go to the 8 of them in turn) follow
        // each other; in that order, 8 tiles along m at each n.
        const int each = tiles / 8, more = tiles % 8, x = id % 8;
        int t = x * each + (x < more ? x : more) + id / 8;
        const int split = t / (tiles_m * tiles_n);
        t -= split * tiles_m * tiles_n;
        const int band = t / (8 * tiles_n), wide = tiles_m - band * 8 < 8 ? tiles_m - band * 8 : 8;
        const int tm = band * 8 + (t - band * 8 * tiles_n) % wide, tn = (t - band * 8 * tiles_n) / wide;
        const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN;

        const int steps_all = int(g.k / kDepth);
        const int first = int(int64_t(steps_all) * split / g.splits);
        const int steps = int(int64_t(steps_all) * (split + 1) / g.splits) - first;

        // rows behind the last are read as the last: what they give is not kept
        uint32_t off_a[RA], off_b[RB];
        const int last_a = int(g.m - m0 < BM ? g.m - m0 : BM) - 1, last_b = int(g.n - n0 < BN ? g.n - n0 : BN) - 1;
#pragma unroll
        for (int i = 0; i < RA; ++i) {
            const int r = (wave * RA + i) * 8 + (lane >> 3);
            off_a[i] = uint32_t(r < last_a ? r : last_a) * uint32_t(g.lda * 2) + uint32_t((lane & 7) ^ (lane >> 3)) * 16;
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int r = (wave * RB + i) * 8 + (lane >> 3);
            off_b[i] = uint32_t(r < last_b ? r : last_b) * uint32_t(g.ldb * 2) + uint32_t((lane & 7) ^ (lane >> 3)) * 16;
        }
        const char *pa = reinterpret_cast<const char *>(g.a + m0 * g.lda + int64_t(first) * kDepth);
        const char *pb = reinterpret_cast<const char *>(g.b + n0 * g.ldb + int64_t(first) * kDepth);
        auto load = [&](int s) {
#pragma unroll
            for (int i = 0; i < RA; ++i)
                copy16_to_lds(pa, off_a[i], &stage[s][(wave * RA + i) * 8 * kDepth]);
#pragma unroll
            for (int i = 0; i < RB; ++i)
                copy16_to_lds(pb, off_b[i], &stage[s][(BM + (wave * RB + i) * 8) * kDepth]);
            pa += kDepth * 2;
            pb += kDepth * 2;
        };

        f32x4 acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = f32x4{0, 0, 0, 0};

        __syncthreads();   // the LDS is free
        if (steps > 0)
            load(0);
        __syncthreads();
        for (int k = 0; k < steps; ++k) {
            const uint16_t *in = stage[k & 1];
            if (k + 1 < steps)
                load((k + 1) & 1);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                bf16x8 a[TM], b[TN];
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    a[i] = *reinterpret_cast<const bf16x8 *>(&in[read_a + i * 16 * kDepth + chunk[half]]);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    b[j] = *reinterpret_cast<const bf16x8 *>(&in[read_b + j * 16 * kDepth + chunk[half]]);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
            }
            __syncthreads();   // the next step's loads have come, and this step's reads are done
        }

        // acc[i][j][r] is C[m][n] with, from the tile's corner,
        //   m = wm * BM / WM + i * 16 + (lane / 16) * 4 + r, n = wn * BN / WN + j * 16 + lane % 16
        const int wave_m = wm * (BM / WM), wave_n = wn * (BN / WN), lane_m = (lane >> 4) * 4, lane_n = lane & 15;
        const int rows_in = int(g.m - m0 < BM ? g.m - m0 : BM), cols_in = int(g.n - n0 < BN ? g.n - n0 : BN);

        if constexpr (E == kScore) {
            float2 *red = reinterpret_cast<float2 *>(stage);   // [WM][BN]
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = wave_n + j * 16 + lane_n;
                // the target's row in this tile, if it is in it
                int64_t target = n < cols_in ? g.targets[n0 + n] : -1;
                target = target >= 0 && target < g.vocab ? target - g.row0 - m0 : -1;
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int m = wave_m + i * 16 + lane_m + r;
                        if (m < rows_in) {
                            top = fmaxf(top, acc[i][j][r]);
                            if (m == target)
                                g.pick[n0 + n] = acc[i][j][r];
                        }
                    }
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (wave_m + i * 16 + lane_m + r < rows_in)
                            sum += exp_below(acc[i][j][r], top);
                sum += __shfl_xor(sum, 16);
                sum += __shfl_xor(sum, 32);
                if (lane < 16)
                    red[wm * BN + n] = {top, sum};
            }
            __syncthreads();
            const int n = threadIdx.x;
            if (n < cols_in) {
                float2 all = red[n];
#pragma unroll
                for (int w = 1; w < WM; ++w) {
                    const float2 one = red[w * BN + n];
                    const float top = fmaxf(all.x, one.x);
                    all = {top, all.y * exp_below(all.x, top) + one.y * exp_below(one.x, top)};
                }
                g.part[(g.tile0 + tm) * g.n + n0 + n] = all;
            }
        } else if constexpr (E == kDiff) {
            // this wave's part of the tile, [n][m], then [m][n]
            constexpr int PM = BM / WM, PN = BN / WN;
            uint16_t *mine = reinterpret_cast<uint16_t *>(stage) + wave * (PM * PN);
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = wave_n + j * 16 + lane_n;
                int64_t target = n < cols_in ? g.targets[n0 + n] : -1;
                const bool named = target >= 0 && target < g.vocab;
                target = named ? target - g.row0 - m0 : -1;
                const float lse = named ? g.lse[n0 + n] : 0.0f, weight = named ? g.weight[n0 + n] : 0.0f;
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int m = wave_m + i * 16 + lane_m + r;
                        const float p = __expf(acc[i][j][r] - lse);
                        v[r] = named && m < rows_in ? (m == target ? p - 1.0f : p) * weight : 0.0f;
                    }
                    // four bf16, in the registers of the logits
                    acc[i][j][0] = __uint_as_float(to_bf16x2(v[0], v[1]));
                    acc[i][j][1] = __uint_as_float(to_bf16x2(v[2], v[3]));
                }
            }
            // Chunks of 8 elements are moved within their row by the row's
            // number, so that neither the writes nor the reads meet in a bank.
            constexpr int CM = PM / 8, CN = PN / 8;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int n = j * 16 + lane_n, c = i * 2 + (lane >> 5);
                    *reinterpret_cast<u32x2 *>(&mine[n * PM + (c ^ (n & (CM - 1))) * 8 + ((lane >> 4) & 1) * 4]) =
                        u32x2{__float_as_uint(acc[i][j][0]), __float_as_uint(acc[i][j][1])};
                }
            __syncthreads();
            const int pad_m = (rows_in + kDepth - 1) / kDepth * kDepth;
            const int pad_n = (cols_in + kDepth - 1) / kDepth * kDepth;
#pragma unroll
            for (int i = 0; i < PN * CM / 64; ++i) {
                const int n = i * (64 / CM) + lane / CM, c = lane % CM;
                if (wave_n + n < cols_in && wave_m + c * 8 < pad_m)
                    *reinterpret_cast<u32x4 *>(&g.d[(n0 + wave_n + n) * g.ldd + m0 + wave_m + c * 8]) =
                        *reinterpret_cast<const u32x4 *>(&mine[n * PM + (c ^ (n & (CM - 1))) * 8]);
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int m = i * 16 + lane_m + r, c = j * 2 + ((lane >> 3) & 1);
                        mine[m * PN + (c ^ ((m >> 2) & (CN - 1))) * 8 + (lane & 7)] =
                            uint16_t(__float_as_uint(acc[i][j][r >> 1]) >> (r & 1) * 16);
                    }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PM * CN / 64; ++i) {
                const int m = i * (64 / CN) + lane / CN, c = lane % CN;
                if (wave_m + m < rows_in && wave_n + c * 8 < pad_n)
                    *reinterpret_cast<u32x4 *>(&g.dt[(m0 + wave_m + m) * g.lddt + n0 + wave_n + c * 8]) =
                        *reinterpret_cast<const u32x4 *>(&mine[m * PN + (c ^ ((m >> 2) & (CN - 1))) * 8]);
            }
        } else if constexpr (E == kSum) {
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
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = wave_n + j * 16 + lane_n;
                uint16_t *row = g.rows + (n0 + n) * g.m + m0;
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int m = wave_m + i * 16 + lane_m;
                    if (n >= cols_in || m >= rows_in)
                        continue;
                    f32x4 v = acc[i][j];
                    if (m + 4 <= rows_in) {
                        Loose<u32x2> *at = reinterpret_cast<Loose<u32x2> *>(row + m);
                        if (g.accumulate) {
                            const u32x2 old = at->v;
                            v += f32x4{lo_f32(old.x), hi_f32(old.x), lo_f32(old.y), hi_f32(old.y)};
                        }
                        at->v = u32x2{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3])};
                    } else {
                        for (int r = 0; r < rows_in - m; ++r) {
                            const float x = r == 0 ? v[0] : r == 1 ? v[1] : v[2];
                            row[m + r] = uint16_t(to_bf16x2(g.accumulate ? x + h_f32(row[m + r]) : x, 0.0f));
                        }
                    }
                }
            }
        }
    }
}

// Workgroups of a launch: one a tile, up to a number whose threads fit 32
// bits; more tiles are taken in turn.
template <int BM, int BN, int WM, int WN, int E>
hipError_t launch(const GemmArgs &g, hipStream_t stream) {
    const int64_t tiles = ceil_div(g.m, BM) * ceil_div(g.n, BN) * g.splits;
    const int64_t cap = std::min<int64_t>(kMaxGrid, int64_t(1) << 21);
    gemm_kernel<BM, BN, WM, WN, E><<<unsigned(std::min(tiles, cap)), WM * WN * 64, 0, stream>>>(g);
    return hipGetLastError();
}

template <int E>
hipError_t launch_sized(const GemmArgs &g, hipStream_t stream) {
    if (wide_tiles(g.m, g.n, g.splits))
        return launch<256, 256, 2, 4, E>(g, stream);
    return launch<128, 128, 2, 2, E>(g, stream);
}

}  // namespace

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
    default:
        return launch_sized<kRows>(g, stream);
    }
}

}  // namespace zdo
