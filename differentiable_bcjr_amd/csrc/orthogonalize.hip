// orthogonalize.hip -- an update of a weight matrix, orthogonalized by Newton-Schulz products:
//   X = G / (|G|_F + eps);  steps times:  A = X X^T,  B = b A + c A A,  X <- a X + B X
// (on G^T when G has more rows than columns, so A is the smaller square).
//
// X is m x n with m <= n.  It is held scaled by 2^10 as the sum of two halves (hi + lo, 22 bits of mantissa), row-major
// and transposed, so that every product reads both operands along their rows; A and B are symmetric and held scaled by
// 2^8.  The scales keep the entries of a normalised matrix (rms (m n)^-1/2) far from the halves' subnormal range and
// leave room for |X| < 64 and |A|, |B| < 256.  The products run on the 16-bit matrix instructions with float32 sums.
// For a bfloat16 result of more than 256 rows they take the hi halves alone: each product then rounds its operands to 11
// bits, while X itself keeps its 22 through a X, which carries the small singular values (rounding X to 11 bits in every
// step loses them: on a rank-16 matrix with 1% noise the result is 4e-2 off; with X kept it is 4e-4, below the 1.7e-3 of
// rounding the result to bfloat16).  The last step, whose errors no other step follows, takes (a + mu) X + (B - mu I) X
// with mu = b + c, B's diagonal where the rows of X are orthonormal: what is rounded is then mostly small (1.4e-3 to
// 1.1e-3 at 512 x 512).  Fewer rows take little more than their launches either way and are hurt most (2.7e-3 at 16 x
// 300), so they and float32 and float16 results take hi hi + hi lo + lo hi, three times the work, and come as near the
// exact result as float32 products do.
#include "bcjr.h"

#include <algorithm>

#include "layer_args.hpp"
#include "layer_types.hpp"
#include "mfma_tile.hpp"

namespace bcjr {
namespace {

constexpr float kXScale = 1024.0f;
constexpr float kAScale = 256.0f;
constexpr int kPad = 64;        // rows and columns of X are padded with zeros to multiples of it
constexpr int kSplitRows = 256; // up to so many rows of X every product is of both halves
constexpr int kPartials = 256;  // partial sums of |G|^2 per matrix

__host__ __device__ inline int64_t pad_up(int64_t v) { return (v + kPad - 1) / kPad * kPad; }
inline size_t area(size_t bytes) { return (bytes + 255) & ~(size_t)255; }

struct Cut;
inline Cut cut_product(int64_t batch, int64_t rows, int64_t cols, int64_t k, bool symmetric, int slab_cols);

struct Layout {
    int64_t m, n, mp, np;   // m <= n, and padded
    bool tall, split;
    size_t partials, x, x_lo, xt[2], a, b, sums, total;   // offsets in the workspace
};

Layout make_layout(int64_t batch, int64_t rows, int64_t cols, int32_t out_type);

// ---------------------------------------------------------------- the norm
//
// Squares are summed in 64 bits: no float32 entry overflows or vanishes, and the order is fixed.

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

constexpr int kSumAhead = 4;   // loads of eight elements that a thread has in flight

template <class T>
__global__ __launch_bounds__(256) void square_sum_kernel(const T* g, int rows, int cols, int64_t ld,
                                                         int64_t batch_stride, double* partials) {
    __shared__ double lds[4];
    const T* p = g + (int64_t)blockIdx.y * batch_stride;
    const uint32_t across = (uint32_t)(cols + 7) / 8, count = across * (uint32_t)rows, step = gridDim.x * 256;
    double sum = 0.0;
    for (uint32_t at = blockIdx.x * 256 + threadIdx.x; at < count; at += step * kSumAhead) {
        Eight<T> v[kSumAhead];
#pragma unroll
        for (int u = 0; u < kSumAhead; ++u) {
            const uint32_t i = at + u * step;
            const int col = i < count ? (int)(i % across) * 8 : cols;
            v[u].load(p + (int64_t)(i / across) * ld + col, cols - col);
        }
#pragma unroll
        for (int u = 0; u < kSumAhead; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double x = (double)v[u].at(j);
                sum = fma(x, x, sum);
            }
    }
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) partials[(int64_t)blockIdx.y * kPartials + blockIdx.x] = sum;
}

__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
    hi = (_Float16)v;
    lo = (_Float16)(v - (float)hi);
}

// G's tile of 64 x 64, normalised and scaled: as it lies into `direct`, transposed into `turned`, each in the layout of
// the products' operands.  lo: X's lo halves where they lie apart, on the side that X is (kSplit: unused).
template <class T, bool kSplit>
__global__ __launch_bounds__(256) void normalize_kernel(const T* g, int64_t rows, int64_t cols, int64_t ld,
                                                        int64_t batch_stride, const double* partials, int parts,
                                                        float eps, _Float16* direct, _Float16* turned,
                                                        _Float16* lo_out, int tall, int64_t rows_p, int64_t cols_p) {
    __shared__ double lds[4];
    __shared__ uint32_t tile[64][65];   // hi | lo << 16
    const int t = threadIdx.x;
    const int64_t item = blockIdx.z;
    const double total = block_sum(t < parts ? partials[item * kPartials + t] : 0.0, lds);
    // in 64 bits, as the norm of entries near float32's largest is beyond it and that of subnormal ones has no reciprocal
    const double scale = (double)kXScale / (sqrt(total) + (double)eps);
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const T* p = g + item * batch_stride;
    const int64_t base = item * rows_p * cols_p;
    // 16 neighbours of a row of the result, from column 16 q of the tile on
    const auto put = [&](_Float16* to, int64_t row, int64_t row_length, int64_t col, const uint32_t (&w)[16], bool lo_here) {
        v4i hi[2], lo[2];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            hi[j / 4][j % 4] = (int)((w[2 * j] & 0xffffu) | (w[2 * j + 1] << 16));
            lo[j / 4][j % 4] = (int)((w[2 * j] >> 16) | (w[2 * j + 1] & 0xffff0000u));
        }
        const int64_t at = kSplit ? 2 * (base + row * row_length) + (col >> 5) * 64 + (col & 31)
                                  : base + row * row_length + col;
        *(v4i*)(to + at) = hi[0];
        *(v4i*)(to + at + 8) = hi[1];
        if (kSplit || lo_here) {
            _Float16* to_lo = kSplit ? to + 32 : lo_out;
            *(v4i*)(to_lo + at) = lo[0];
            *(v4i*)(to_lo + at + 8) = lo[1];
        }
    };
    const int line = t >> 2, q = (t & 3) * 16;
    uint32_t w[16];
    const int64_t left = r0 + line < rows ? cols - (c0 + q) : 0;
    Eight<T> v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) v[h].load(p + (r0 + line) * ld + c0 + q + h * 8, left - h * 8);
#pragma unroll
    for (int j = 0; j < 16; ++j) {   // what lies outside G stays 0, also where the norm is 0 or NaN
        _Float16 hi, lo;
        split(j < left ? (float)((double)v[j / 8].at(j % 8) * scale) : 0.0f, hi, lo);
        w[j] = (uint32_t)__builtin_bit_cast(uint16_t, hi) | ((uint32_t)__builtin_bit_cast(uint16_t, lo) << 16);
    }
    put(direct, r0 + line, cols_p, c0 + q, w, !tall);
#pragma unroll
    for (int j = 0; j < 16; ++j) tile[line][q + j] = w[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = tile[q + j][line];
    put(turned, c0 + line, rows_p, r0 + q, w, tall);
}

// ---------------------------------------------------------------- the products
//
// What bounds them, 8192 x 2048 with a float32 result: a X + B X (206 GFLOP in its three products) takes 185 to 205 us, of
// which about 40 us are the 200 MB that its ending reads and writes (X, and X again and X^T), exposed because one
// workgroup fills a compute unit; X X^T 104 + 17 us for 116 GFLOP (75 us of the 104 without any
// load from memory).  The card holds 2.1 GHz under them.  Tiles of 128, two workgroups to a compute unit, would overlap endings with products but read
// the operands twice as often: 228 us against 208.
//
// Operands: with kSplit a row holds, for each 32 columns, the 32 hi halves and then the 32 lo halves, so one slab brings
// both halves of 32 columns and its three products are formed from the same two fragments; without, a row holds the hi
// halves alone (and X's lo halves lie in an array of their own).  The symmetric products compute the tiles on and below
// the diagonal and write each twice.

enum Mode { kGram, kPoly, kStep };

template <bool kSplit>
struct Halves2 {
    static constexpr int kPer = kSplit ? 2 : 1;         // halves stored for a column
    static constexpr int kSlabCols = kSplit ? 32 : 64;  // columns of a slab
    // where the hi half of column `col` lies in a row; its lo half lies 32 behind (kSplit)
    static __host__ __device__ __forceinline__ int64_t at(int64_t col) {
        return kSplit ? (col >> 5) * 64 + (col & 31) : col;
    }
};

struct ProdArgs {
    const _Float16 *p, *q;        // [rows][k] and [cols][k]
    int64_t p_batch, q_batch;     // halves from one matrix of the batch to the next
    int32_t rows, cols, k;        // multiples of kPad
    const _Float16 *old, *old_lo; // kPoly: A; kStep: X (old_lo: X's lo halves where they lie apart)
    _Float16 *o, *o_lo;           // the result [rows][cols]
    _Float16* t;                  // its transpose [cols][rows]: the same array where it is symmetric
    int64_t o_batch, lo_batch;
    float alpha, beta;            // kGram: alpha acc; kPoly, kStep: alpha old + beta acc
    float shift;                  // kPoly: subtracted on the diagonal
    void* out;                    // kStep, last: the result in its own type, m x n or (tall) n x m
    int32_t m, n, tall;
    int64_t out_batch;
    float* partial;               // more than one part: float32 sums [part][tile][wave][fragment][lane]
    int32_t parts;                // parts of the k loop
};

struct TilePlace {
    int bm, bn;
};

template <Mode kMode>
__device__ __forceinline__ TilePlace tile_place(int id, int tiles_m, int tiles_n) {
    TilePlace p;
    if constexpr (kMode == kStep) {
        banded_tile(id, tiles_m, tiles_n, 8, p.bm, p.bn);
    } else {   // row by row
        p.bm = (int)((sqrtf(8.0f * (float)id + 1.0f) - 1.0f) * 0.5f);
        while (p.bm * (p.bm + 1) / 2 > id) --p.bm;
        while ((p.bm + 1) * (p.bm + 2) / 2 <= id) ++p.bm;
        p.bn = id - p.bm * (p.bm + 1) / 2;
    }
    return p;
}

// A wave's block of TM x TN fragments whose first element is (row0, col0): the result and its transpose from the sums,
// through this wave's LDS.  A lane's four sums are neighbours along a row.
template <Mode kMode, bool kSplit, class T, int TM, int TN>
__device__ __forceinline__ void finish(const ProdArgs& a, v4f (&acc)[TM][TN], int row0, int col0, int64_t item,
                                       bool mirror, uint8_t* lds, int lane) {
    using H = Halves2<kSplit>;
    int r16 = lane & 15, g = lane >> 4;
    // Places in LDS are computed anew in each pass below: kept from one to the next they take more registers than there
    // are next to the sums.
    const auto forget = [&] { asm volatile("" : "+v"(r16), "+v"(g), "+v"(lane)); };
    forget();
    const int64_t o = item * a.o_batch;
    const int64_t ld = (int64_t)a.cols * H::kPer, ld_t = (int64_t)a.rows * H::kPer;
    constexpr int R = TM * 16, C = TN * 16;
    static_assert(kPad % R == 0 && kPad % C == 0, "a block lies wholly inside the padded result or outside");
    if (row0 >= a.rows || col0 >= a.cols) return;
    if constexpr (kMode == kGram) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] *= a.alpha;
    } else {
        v4h hi[TM][TN], lo[TM][TN];   // all loads, then their uses
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t row = row0 + i * 16 + r16;
            const _Float16* old = a.old + o + row * ld + (int64_t)col0 * H::kPer + g * 4;
            const _Float16* old_lo = old + 32;
            if constexpr (!kSplit && kMode == kStep) old_lo = a.old_lo + item * a.lo_batch + row * a.cols + col0 + g * 4;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int at = (int)H::at(j * 16);
                hi[i][j] = *(const v4h*)(old + at);
                if constexpr (kSplit || kMode == kStep) lo[i][j] = *(const v4h*)(old_lo + at);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = (float)hi[i][j][e];
                    if constexpr (kSplit || kMode == kStep) x += (float)lo[i][j][e];
                    acc[i][j][e] = fmaf(a.alpha, x, a.beta * acc[i][j][e]);
                    if constexpr (kMode == kPoly)
                        if (row0 + i * 16 + r16 == col0 + j * 16 + g * 4 + e) acc[i][j][e] -= a.shift;
                }
    }
    forget();
    if (kMode == kStep && a.out) {
        T* out = (T*)a.out + item * a.out_batch;
        if (a.tall) {
            using Tile = WaveTile<T, C, R>;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        Tile::put1(lds, j * 16 + g * 4 + e, i * 16 + r16, from_f32<T>(acc[i][j][e] * (1.0f / kXScale)));
            wave_fence();
            const bool wide = (uintptr_t)out % 16 == 0 && ((int64_t)a.m * sizeof(T)) % 16 == 0;
            Tile::store(lds, out + (int64_t)col0 * a.m + row0, a.m, a.n - col0, a.m - row0, wide, lane);
        } else {
            using Tile = WaveTile<T, R, C>;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    T v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = from_f32<T>(acc[i][j][e] * (1.0f / kXScale));
                    Tile::put(lds, i * 16 + r16, j * 16 + g * 4, v);
                }
            wave_fence();
            const bool wide = (uintptr_t)out % 16 == 0 && ((int64_t)a.n * sizeof(T)) % 16 == 0;
            Tile::store(lds, out + (int64_t)row0 * a.n + col0, a.n, a.m - row0, a.n - col0, wide, lane);
        }
        return;
    }

    {
        using Tile = WaveTile<_Float16, R, C * H::kPer>;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                _Float16 hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split(acc[i][j][e], hi[e], lo[e]);
                const int col = (int)H::at(j * 16 + g * 4);
                Tile::put(lds, i * 16 + r16, col, hi);
                if constexpr (kSplit) Tile::put(lds, i * 16 + r16, col + 32, lo);
            }
        wave_fence();
        Tile::store(lds, a.o + o + row0 * ld + (int64_t)col0 * H::kPer, ld, R, C * H::kPer, true, lane);
        wave_fence();
        if constexpr (!kSplit && kMode == kStep) {   // X's lo halves
            forget();
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    _Float16 hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split(acc[i][j][e], hi[e], lo[e]);
                    Tile::put(lds, i * 16 + r16, j * 16 + g * 4, lo);
                }
            wave_fence();
            Tile::store(lds, a.o_lo + item * a.lo_batch + (int64_t)row0 * a.cols + col0, a.cols, R, C, true, lane);
            wave_fence();
        }
    }
    if (mirror) {
        forget();
        using Tile = WaveTile<_Float16, C, R * H::kPer>;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    _Float16 hi, lo;
                    split(acc[i][j][e], hi, lo);
                    const int at = (int)H::at(i * 16 + r16);
                    Tile::put1(lds, j * 16 + g * 4 + e, at, hi);
                    if constexpr (kSplit) Tile::put1(lds, j * 16 + g * 4 + e, at + 32, lo);
                }
        wave_fence();
        Tile::store(lds, a.t + o + col0 * ld_t + (int64_t)row0 * H::kPer, ld_t, C, R * H::kPer, true, lane);
        wave_fence();
    }
}

// The first or second four registers of a fragment: halves of columns, or with kSplit the hi and lo halves.
__device__ __forceinline__ v8h half_slab(v8i v, int h) {
    return __builtin_bit_cast(v8h, h == 0 ? __builtin_shufflevector(v, v, 0, 1, 2, 3)
                                          : __builtin_shufflevector(v, v, 4, 5, 6, 7));
}

__device__ __forceinline__ v4f multiply(v8h a, v8h b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

constexpr int kFinishRows = 4;   // rows of fragments that `finish` takes at a time: its LDS is 16 KB a wave

template <Mode kMode, bool kSplit, class T, int BM, int WAVES_M, int WAVES_N, int kStages, int kGroups>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N * kGroups, 2) void ortho_product_kernel(ProdArgs a, int tiles_m,
                                                                                            int tiles_n) {
    constexpr int kWaves = WAVES_M * WAVES_N;
    constexpr int TM = BM / WAVES_M / 16, TN = BM / WAVES_N / 16;
    constexpr int TF = TM < kFinishRows ? TM : kFinishRows;
    constexpr int kStageBytes = 2 * BM * kSlab;
    constexpr int kFinishBytes = TF * 16 * TN * 16 * 4;
    constexpr int kJoinAt = kWaves * kFinishBytes, kJoinBytes = (kGroups - 1) * kWaves * TM * TN * 1024;
    __shared__ __align__(1024) uint8_t all_lds[kGroups * kStages * kStageBytes];
    static_assert(kJoinAt + kJoinBytes <= (int)sizeof(all_lds), "every wave's results and the groups' sums fit in LDS");
    const int t = threadIdx.x, lane = t & 63;
    const int any_wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int group = any_wave / kWaves, wave = any_wave % kWaves;
    uint8_t* const lds = all_lds + group * (kStages * kStageBytes);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int r16 = lane & 15, g = lane >> 4;
    const int tiles = gridDim.x / a.parts;
    const int id = xcd_order(blockIdx.x, gridDim.x);
    const int part = id / tiles, tile = id - part * tiles;
    const TilePlace at = tile_place<kMode>(tile, tiles_m, tiles_n);
    const int m0 = at.bm * BM, n0 = at.bn * BM;
    const int64_t item = blockIdx.z;
    const uint32_t ld = (uint32_t)a.k * Halves2<kSplit>::kPer * 2;
    const int slabs = a.k / Halves2<kSplit>::kSlabCols;
    const int first = (int)((int64_t)slabs * part / a.parts), last = (int)((int64_t)slabs * (part + 1) / a.parts);

    using Source = SlabSource<BM, kWaves>;
    Source src_p, src_q;
    src_p.set((const uint8_t*)(a.p + item * a.p_batch) + (int64_t)m0 * ld, ld, a.rows - m0, wave, lane);
    src_q.set((const uint8_t*)(a.q + item * a.q_batch) + (int64_t)n0 * ld, ld, a.cols - n0, wave, lane);

    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int wm0 = wm * TM * 16, wn0 = wn * TN * 16;

    // group i takes slabs first + i, first + i + kGroups, ...
    const auto issue = [&](int s, int slot) {
        uint8_t* stage = lds + slot * kStageBytes;
        const uint32_t at = (uint32_t)min(first + s * kGroups + group, last - 1) * kSlab;
        src_p.fetch(at, stage, wave);
        src_q.fetch(at, stage + BM * kSlab, wave);
    };
    const int total = (last - first + kGroups - 1) / kGroups;
    pipeline_ahead<kStages>(total, issue);
    pipelined<kStages, 2 * Source::kLoads>(
        total, (last - first - group + kGroups - 1) / kGroups, issue,
        [&](int slot) {
            const uint8_t* lp = lds + slot * kStageBytes;
            const uint8_t* lq = lp + BM * kSlab;
            v8i fq[TN], fp[2];
#pragma unroll
            for (int j = 0; j < TN; ++j) fq[j] = read_slab(lq, wn0 + j * 16 + r16, g);
            fp[0] = read_slab(lp, wm0 + r16, g);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if (i + 1 < TM) fp[(i + 1) & 1] = read_slab(lp, wm0 + (i + 1) * 16 + r16, g);
                const v8h p0 = half_slab(fp[i & 1], 0), p1 = half_slab(fp[i & 1], 1);
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = multiply(half_slab(fq[j], 0), p0, acc[i][j]);
                if constexpr (kSplit) {
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] = multiply(half_slab(fq[j], 0), p1, acc[i][j]);
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] = multiply(half_slab(fq[j], 1), p0, acc[i][j]);
                } else {
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] = multiply(half_slab(fq[j], 1), p1, acc[i][j]);
                }
                if (i + 1 < TM) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x8, (kSplit ? 3 : 2) * TN, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        });

    if (a.parts > 1) {
        const int64_t block = ((item * a.parts + part) * tiles + tile) * kWaves + wave;
        v4f* to = (v4f*)a.partial + block * (TM * TN * 64) + lane;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) to[(i * TN + j) * 64] = acc[i][j];
        return;
    }
    meet();   // nobody reads the operands any more
    join_groups<kGroups, kWaves>(acc, group, wave, lane, all_lds + kJoinAt);
    if (group > 0) return;
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += TF) {
        v4f some[TF][TN];
#pragma unroll
        for (int i = 0; i < TF; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) some[i][j] = acc[i0 + i][j];
        __builtin_amdgcn_sched_barrier(0);
        finish<kMode, kSplit, T, TF, TN>(a, some, m0 + wm0 + i0 * 16, n0 + wn0, item, kMode == kStep || at.bm != at.bn,
                                         all_lds + wave * kFinishBytes, lane);
    }
}

constexpr int kJoinRows = 2;

// The parts' sums, added in their order, and the result from them: one wave for each kJoinRows rows of fragments.
template <Mode kMode, bool kSplit, class T, int BM, int WAVES_M, int WAVES_N>
__global__ __launch_bounds__(64) void ortho_join_kernel(ProdArgs a, int tiles_m, int tiles_n) {
    constexpr int kWaves = WAVES_M * WAVES_N;
    constexpr int TM = BM / WAVES_M / 16, TN = BM / WAVES_N / 16;
    constexpr int TF = kJoinRows, kPieces = TM / TF;
    __shared__ __align__(1024) uint8_t lds[TF * 16 * TN * 16 * 4];
    const int lane = threadIdx.x;
    const int tiles = gridDim.x / (kWaves * kPieces);
    const int piece = blockIdx.x % kPieces, wave = blockIdx.x / kPieces % kWaves, tile = blockIdx.x / (kPieces * kWaves);
    const int64_t item = blockIdx.z;
    const TilePlace at = tile_place<kMode>(tile, tiles_m, tiles_n);
    const int row0 = at.bm * BM + (wave / WAVES_N) * TM * 16 + piece * TF * 16;
    const int col0 = at.bn * BM + (wave % WAVES_N) * TN * 16;
    v4f acc[TF][TN];
#pragma unroll 4
    for (int part = 0; part < a.parts; ++part) {
        const int64_t block = ((item * a.parts + part) * tiles + tile) * kWaves + wave;
        const v4f* from = (const v4f*)a.partial + block * (TM * TN * 64) + piece * (TF * TN * 64) + lane;
#pragma unroll
        for (int i = 0; i < TF; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const v4f v = from[(i * TN + j) * 64];
                acc[i][j] = part ? acc[i][j] + v : v;
            }
    }
    finish<kMode, kSplit, T, TF, TN>(a, acc, row0, col0, item, kMode == kStep || at.bm != at.bn, lds, lane);
}

template <Mode kMode, bool kSplit, class T, int BM, int WAVES_M, int WAVES_N, int kStages, int kGroups>
void launch_tiles(ProdArgs a, int64_t batch, int parts, hipStream_t st) {
    const int tm = (a.rows + BM - 1) / BM, tn = (a.cols + BM - 1) / BM;
    const unsigned tiles = kMode == kStep ? (unsigned)tm * tn : (unsigned)tm * (tm + 1) / 2;
    a.parts = parts;
    ortho_product_kernel<kMode, kSplit, T, BM, WAVES_M, WAVES_N, kStages, kGroups>
        <<<dim3(tiles * parts, 1, (unsigned)batch), 64 * WAVES_M * WAVES_N * kGroups, 0, st>>>(a, tm, tn);
    if (parts > 1) {
        constexpr int kPieces = BM / WAVES_M / 16 / kJoinRows;
        ortho_join_kernel<kMode, kSplit, T, BM, WAVES_M, WAVES_N>
            <<<dim3(tiles * WAVES_M * WAVES_N * kPieces, 1, (unsigned)batch), 64, 0, st>>>(a, tm, tn);
    }
}

// How a product over k is cut: tiles of 256, of 128 or of 64, as large as leave most of the card busy; the k loop of a
// tile shared by `groups` groups of waves, which meet in LDS; and a symmetric product's k loop in `parts` parts, which
// meet in a second kernel.  Parts pay where few tiles stand against a long k: 2048 x 2048 over k = 8192 for a float32
// result takes 104 + 17 us in 7 parts of 36 tiles of 256 and 167 us in 136 tiles of 128, over k = 2048 37 + 19 us and
// 54 us, and with the hi halves alone 22 + 11 us and 26 us.
struct Cut {
    int tile, parts, groups;
};

inline Cut cut_product(int64_t batch, int64_t rows, int64_t cols, int64_t k, bool symmetric, int slab_cols) {
    const auto tiles = [&](int64_t size) {
        const int64_t tm = (rows + size - 1) / size, tn = (cols + size - 1) / size;
        return batch * (symmetric ? tm * (tm + 1) / 2 : tm * tn);
    };
    constexpr int64_t kCus = 256;
    const int64_t slabs = k / slab_cols;
    // whether what tiles hold beyond the edges makes them not much more work than tiles of 64 (260 matrices of 64 x 64 in
    // float32 take 99 us, in tiles of 256, which they would fill the card with, 307 us)
    const auto fits = [&](int64_t size) { return tiles(size) * size * size * 2 <= tiles(64) * 64 * 64 * 3; };
    if (fits(256)) {
        if (tiles(256) >= kCus * 3 / 4) return {256, 1, 1};
        if (symmetric && tiles(256) >= 24 && slabs >= 64) return {256, (int)std::max<int64_t>(1, kCus / tiles(256)), 1};
    }
    if (fits(128)) {
        if (tiles(128) > kCus) return {128, 1, 1};
        if (tiles(128) >= kCus / 2 && slabs >= 4) return {128, 1, 2};
    }
    if (symmetric && tiles(64) <= kCus / 4 && slabs >= 64)
        return {64, (int)std::min(kCus / tiles(64), slabs / 16), 1};
    return {64, 1, tiles(64) <= kCus && slabs >= 4 ? 2 : 1};
}

template <Mode kMode, bool kSplit, class T>
void launch_product(const ProdArgs& a, int64_t batch, hipStream_t st) {
    const Cut c = cut_product(batch, a.rows, a.cols, a.k, kMode != kStep, Halves2<kSplit>::kSlabCols);
    if (c.tile == 256)
        launch_tiles<kMode, kSplit, T, 256, 2, 4, 2, 1>(a, batch, c.parts, st);
    else if (c.tile == 128 && c.groups == 1)
        launch_tiles<kMode, kSplit, T, 128, 2, 2, 2, 1>(a, batch, 1, st);
    else if (c.tile == 128)
        launch_tiles<kMode, kSplit, T, 128, 2, 2, 2, 2>(a, batch, 1, st);
    else if (c.groups == 2)
        launch_tiles<kMode, kSplit, T, 64, 2, 2, 4, 2>(a, batch, 1, st);
    else
        launch_tiles<kMode, kSplit, T, 64, 2, 2, 4, 1>(a, batch, c.parts, st);
}

template <bool kSplit, class Out>
hipError_t iterate(const OrthoArgs& o, const Layout& l, hipStream_t st) {
    unsigned char* ws = o.ws;
    auto at = [&](size_t off) { return (_Float16*)(ws + off); };
    constexpr int64_t kPer = Halves2<kSplit>::kPer;
    const int64_t x_batch = l.mp * l.np * kPer, s_batch = l.mp * l.mp * kPer;
    for (int s = 0; s < o.steps; ++s) {
        const int cur = s & 1, next = cur ^ 1;
        ProdArgs gram{};
        gram.p = gram.q = at(l.x);
        gram.p_batch = gram.q_batch = x_batch;
        gram.rows = gram.cols = (int32_t)l.mp;
        gram.k = (int32_t)l.np;
        gram.o = gram.t = at(l.a);
        gram.o_batch = s_batch;
        gram.alpha = kAScale / (kXScale * kXScale);
        gram.partial = (float*)(ws + l.sums);
        launch_product<kGram, kSplit, float>(gram, o.batch, st);

        ProdArgs poly{};
        poly.p = poly.q = poly.old = at(l.a);
        poly.p_batch = poly.q_batch = s_batch;
        poly.rows = poly.cols = poly.k = (int32_t)l.mp;
        poly.o = poly.t = at(l.b);
        poly.o_batch = s_batch;
        poly.alpha = o.b;
        poly.beta = o.c / kAScale;
        const float mu = !kSplit && s + 1 == o.steps ? o.b + o.c : 0.0f;
        poly.shift = mu * kAScale;
        poly.partial = (float*)(ws + l.sums);
        launch_product<kPoly, kSplit, float>(poly, o.batch, st);

        ProdArgs step{};
        step.p = at(l.b);
        step.p_batch = s_batch;
        step.q = at(l.xt[cur]);
        step.q_batch = x_batch;
        step.rows = (int32_t)l.mp;
        step.cols = (int32_t)l.np;
        step.k = (int32_t)l.mp;
        step.old = step.o = at(l.x);
        step.old_lo = step.o_lo = at(l.x_lo);
        step.lo_batch = l.mp * l.np;
        step.t = at(l.xt[next]);
        step.o_batch = x_batch;
        step.alpha = o.a + mu;
        step.beta = 1.0f / kAScale;
        step.m = (int32_t)l.m;
        step.n = (int32_t)l.n;
        step.tall = l.tall;
        step.out = s + 1 == o.steps ? o.out : nullptr;
        step.out_batch = l.m * l.n;
        launch_product<kStep, kSplit, Out>(step, o.batch, st);
    }
    return hipGetLastError();
}

template <class In>
hipError_t orthogonalize_from(const OrthoArgs& o, hipStream_t st) {
    const Layout l = make_layout(o.batch, o.rows, o.cols, o.out_type);
    double* partials = (double*)(o.ws + l.partials);
    const int64_t chunks = o.rows * ((o.cols + 7) / 8);
    const int parts = (int)std::min<int64_t>(kPartials, (chunks + 255) / 256);
    square_sum_kernel<In><<<dim3((unsigned)parts, (unsigned)o.batch), 256, 0, st>>>(
        (const In*)o.g, (int)o.rows, (int)o.cols, o.ld_g, o.batch_g, partials);
    auto at = [&](size_t off) { return (_Float16*)(o.ws + off); };
    const int64_t rp = pad_up(o.rows), cp = pad_up(o.cols);
    const dim3 grid((unsigned)(cp / 64), (unsigned)(rp / 64), (unsigned)o.batch);
    _Float16 *direct = at(l.tall ? l.xt[0] : l.x), *turned = at(l.tall ? l.x : l.xt[0]);
    if (l.split)
        normalize_kernel<In, true><<<grid, 256, 0, st>>>((const In*)o.g, o.rows, o.cols, o.ld_g, o.batch_g, partials,
                                                         parts, o.eps, direct, turned, nullptr, l.tall, rp, cp);
    else
        normalize_kernel<In, false><<<grid, 256, 0, st>>>((const In*)o.g, o.rows, o.cols, o.ld_g, o.batch_g, partials,
                                                          parts, o.eps, direct, turned, at(l.x_lo), l.tall, rp, cp);
    switch (o.out_type) {
        case BCJR_TYPE_F32: return iterate<true, float>(o, l, st);
        case BCJR_TYPE_BF16:
            return l.split ? iterate<true, __hip_bfloat16>(o, l, st) : iterate<false, __hip_bfloat16>(o, l, st);
        default: return iterate<true, _Float16>(o, l, st);
    }
}

}  // namespace

namespace {

Layout make_layout(int64_t batch, int64_t rows, int64_t cols, int32_t out_type) {
    Layout l{};
    l.tall = rows > cols;
    l.m = l.tall ? cols : rows;
    l.n = l.tall ? rows : cols;
    l.mp = pad_up(l.m);
    l.np = pad_up(l.n);
    l.split = out_type != BCJR_TYPE_BF16 || l.mp <= kSplitRows;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += area(bytes);
        return here;
    };
    const size_t per = l.split ? 4 : 2;   // bytes of an element of a product's operand
    const size_t x = (size_t)batch * l.mp * l.np, s = (size_t)batch * l.mp * l.mp;
    l.partials = take((size_t)batch * kPartials * 8);
    l.x = take(x * per);
    l.x_lo = l.split ? l.x : take(x * 2);
    l.xt[0] = take(x * per);
    l.xt[1] = take(x * per);
    l.a = take(s * per);
    l.b = take(s * per);
    size_t sums = 0;   // the symmetric products' partial sums
    for (const int64_t k : {l.np, l.mp}) {
        const Cut c = cut_product(batch, l.mp, l.mp, k, true, l.split ? 32 : 64);
        const size_t tm = (size_t)((l.mp + c.tile - 1) / c.tile);
        const size_t need = c.parts > 1 ? (size_t)batch * c.parts * (tm * (tm + 1) / 2) * c.tile * c.tile * 4 : 0;
        sums = need > sums ? need : sums;
    }
    l.sums = take(sums);
    l.total = at;
    return l;
}

}  // namespace

size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols, int32_t out_type) {
    return make_layout(batch, rows, cols, out_type).total;
}

hipError_t launch_orthogonalize(const OrthoArgs& o, hipStream_t st) {
    switch (o.type) {
        case BCJR_TYPE_F32: return orthogonalize_from<float>(o, st);
        case BCJR_TYPE_BF16: return orthogonalize_from<__hip_bfloat16>(o, st);
        default: return orthogonalize_from<_Float16>(o, st);
    }
}

}  // namespace bcjr
