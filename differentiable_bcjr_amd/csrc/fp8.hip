// fp8.hip -- 8-bit block quantization (e4m3 codes, one float32 scale per block of 128) and the product of two
// matrices held that way.
#include "bcjr.h"

#include <type_traits>

#include "layer_args.hpp"
#include "layer_types.hpp"
#include "mfma_tile.hpp"

namespace bcjr {
namespace {

// ------------------------------------------------------------------------------------------------ quantization
//
// A block's scale is s = max(amax / 448, 2^-126) and its codes are e4m3(x / s), with both divisions as multiplications
// by float32 constants (fl(1/448) and fl(1/s)), each product rounded to float32 before the rounding to e4m3 (to the
// nearest, ties to even): elementary float32 operations in a fixed order, so any implementation of them gives the same
// codes.  The floor 2^-126 keeps 1/s finite; it also makes a block of zeros quantize to zeros.  amax is taken on the
// bit patterns of |x|, where Inf and NaN sort above every number: they reach the scale and so the block's results.

constexpr float kInvMax = 1.0f / 448.0f;   // 448: the largest e4m3 number
constexpr float kMinScale = 1.17549435e-38f;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <class T>
__device__ __forceinline__ uint32_t max8(const Eight<T>& v) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v.at(j)));
    return m;
}

__device__ __forceinline__ float block_scale(uint32_t amax) {
    const float s = __uint_as_float(amax) * kInvMax;
    return s < kMinScale ? kMinScale : s;   // NaN stays
}

// Four codes in the bytes of one word.  |x r| is at most 448 (1 + 2^-23) unless it is NaN, and the instruction rounds
// that to 448.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

template <class T>
__device__ __forceinline__ uint2 codes8(const Eight<T>& v, float r) {
    return make_uint2(codes4(v.at(0) * r, v.at(1) * r, v.at(2) * r, v.at(3) * r),
                      codes4(v.at(4) * r, v.at(5) * r, v.at(6) * r, v.at(7) * r));
}

__device__ __forceinline__ void store8(uint8_t* p, int count, uint2 w) {
    if (count >= 8) {
        *(uint2*)p = w;
    } else {
        for (int j = 0; j < count; ++j) p[j] = (uint8_t)((j < 4 ? w.x >> (8 * j) : w.y >> (8 * (j - 4))) & 0xff);
    }
}

// Rows alone: 16 lanes hold one row's block of 128, eight elements each.  Bound by memory: 8192 x 2048 in bfloat16 take
// 10 us, 50 MB at 5.0 TB/s (a large copy moves 5.1).
constexpr int kRowsPerGroup = 16;

template <class T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantizeArgs a, int col_blocks) {
    const int t = threadIdx.x;
    const int cb = blockIdx.x % col_blocks;
    const int64_t row = (int64_t)(blockIdx.x / col_blocks) * kRowsPerGroup + (t >> 4);
    const int64_t col = (int64_t)cb * 128 + (t & 15) * 8;
    const bool have = row < a.rows;
    const int64_t left = have ? a.cols - col : 0;
    Eight<T> v;
    v.load((const T*)a.x + row * a.ld_x + col, left);
    const float s = block_scale(max16(max8(v)));
    if (left > 0) store8(a.q + row * a.ld_q + col, (int)min(left, (int64_t)8), codes8(v, 1.0f / s));
    if (have && (t & 15) == 0) a.scale[(int64_t)cb * a.rows + row] = s;
}

// A tile of 128 x 128: square blocks, and any quantization that also writes the transpose.  Thread t holds eight
// columns of eight consecutive rows, so both orientations leave it as words of eight codes; the transposed codes pass
// through LDS to be written in whole 128-byte lines.  The tile stays in registers as it lies in memory and is converted
// at each use, which halves its registers in 16-bit types.  8192 x 8192 in bfloat16, both orientations, take 48 us (268 MB
// at 5.6 TB/s), 8192 x 2048 in float32 with square blocks 16 us (101 MB at 6.3 TB/s, part of it from cache).
template <class T, bool kSquare, bool kTransposed>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantizeArgs a, int col_blocks, int row_blocks) {
    __shared__ uint32_t col_max[4][128];
    __shared__ __align__(16) uint8_t codes_t[kTransposed ? 128 * 128 : 16];
    const int t = threadIdx.x;
    const int i = t & 15, band = t >> 4;   // columns 8 i .. 8 i + 7, rows 8 band .. 8 band + 7 of the tile
    const int cb = blockIdx.x % col_blocks, rb = blockIdx.x / col_blocks;
    const int64_t row0 = (int64_t)rb * 128, col0 = (int64_t)cb * 128;
    const int64_t col = col0 + i * 8;
    const int64_t rows_left = a.rows - (row0 + band * 8);
    const int64_t cols_left = a.cols - col;
    Eight<T> v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p)
        v[p].load((const T*)a.x + (row0 + band * 8 + p) * a.ld_x + col, p < rows_left ? cols_left : 0);

    float inv_square = 0.0f;
    if constexpr (kSquare) {
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) m = max(m, max8(v[p]));
        m = max16(m);
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if ((t & 63) == 0) col_max[t >> 6][0] = m;
        __syncthreads();
        m = max(max(col_max[0][0], col_max[1][0]), max(col_max[2][0], col_max[3][0]));
        const float s = block_scale(m);
        inv_square = 1.0f / s;
        if (t == 0) {
            a.scale[(int64_t)cb * row_blocks + rb] = s;
            if constexpr (kTransposed) a.scale_t[(int64_t)rb * col_blocks + cb] = s;
        }
    }

#pragma unroll
    for (int p = 0; p < 8; ++p) {
        float r = inv_square;
        if constexpr (!kSquare) {
            const float s = block_scale(max16(max8(v[p])));
            r = 1.0f / s;
            if (i == 0 && p < rows_left) a.scale[(int64_t)cb * a.rows + row0 + band * 8 + p] = s;
        }
        if (p < rows_left && cols_left > 0)
            store8(a.q + (row0 + band * 8 + p) * a.ld_q + col, (int)min(cols_left, (int64_t)8), codes8(v[p], r));
    }

    if constexpr (kTransposed) {
        float inv[8];
        if constexpr (kSquare) {
#pragma unroll
            for (int j = 0; j < 8; ++j) inv[j] = inv_square;
        } else {
            uint32_t m[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m[j] = 0;
#pragma unroll
                for (int p = 0; p < 8; ++p) m[j] = max(m[j], abs_bits(v[p].at(j)));
                m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 16));
                m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 32));
            }
            if ((t & 63) < 16) {
#pragma unroll
                for (int j = 0; j < 8; ++j) col_max[t >> 6][i * 8 + j] = m[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = i * 8 + j;
                const float s = block_scale(max(max(col_max[0][c], col_max[1][c]), max(col_max[2][c], col_max[3][c])));
                inv[j] = 1.0f / s;
                if (band == 0 && j < cols_left) a.scale_t[(int64_t)rb * a.cols + col + j] = s;
            }
        }
        // column c's codes are 16 words of 8 rows; word `band` lies at band ^ (c / 8), which spreads the 16 columns
        // that a step writes over the banks
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float r = inv[j];
            const uint2 w = make_uint2(codes4(v[0].at(j) * r, v[1].at(j) * r, v[2].at(j) * r, v[3].at(j) * r),
                                       codes4(v[4].at(j) * r, v[5].at(j) * r, v[6].at(j) * r, v[7].at(j) * r));
            *(uint2*)(codes_t + (i * 8 + j) * 128 + ((band ^ i) * 8)) = w;
        }
        __syncthreads();
        const int64_t rows_tile = a.rows - row0;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int c = p * 32 + (t >> 3);
            const int w = (t & 7) * 2;
            if (col0 + c >= a.cols) continue;
            const uint2 lo = *(const uint2*)(codes_t + c * 128 + ((w ^ (c >> 3)) * 8));
            const uint2 hi = *(const uint2*)(codes_t + c * 128 + (((w + 1) ^ (c >> 3)) * 8));
            uint8_t* out = a.q_t + (col0 + c) * a.ld_qt + row0 + w * 8;
            const int64_t left = rows_tile - w * 8;
            if (left >= 16) {
                *(uint4*)out = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else if (left > 0) {
                store8(out, (int)min(left, (int64_t)8), lo);
                if (left > 8) store8(out + 8, (int)(left - 8), hi);
            }
        }
    }
}

template <class T>
hipError_t quantize(const QuantizeArgs& a, hipStream_t st) {
    const int cb = (int)((a.cols + 127) / 128), rb = (int)((a.rows + 127) / 128);
    if (a.block_rows == 1 && !a.q_t) {
        const unsigned grid = (unsigned)cb * (unsigned)((a.rows + kRowsPerGroup - 1) / kRowsPerGroup);
        quantize_rows_kernel<T><<<grid, 256, 0, st>>>(a, cb);
    } else {
        const unsigned grid = (unsigned)cb * (unsigned)rb;
        if (a.block_rows == 1)
            quantize_tile_kernel<T, false, true><<<grid, 256, 0, st>>>(a, cb, rb);
        else if (a.q_t)
            quantize_tile_kernel<T, true, true><<<grid, 256, 0, st>>>(a, cb, rb);
        else
            quantize_tile_kernel<T, true, false><<<grid, 256, 0, st>>>(a, cb, rb);
    }
    return hipGetLastError();
}

// ------------------------------------------------------------------------------------------------ product
//
// out[i][j] = sum over blocks B of sa[i][B] sb[j][B] sum over k in B of a[i][k] b[j][k].  A slab is one block, so each
// MFMA (or four of the 16-bit kind) sums one block of one 16 x 16 tile from zero, and a float32 fused multiply-add with
// the two scales' product moves it into the running sum.  The MFMA's row operand is b, so a lane holds four neighbouring
// outputs of one row of a: one scale of a for each 16 rows, and a vector store.  Against square blocks of b the two scales
// are multiplied first: blocks whose scales' product is below 2^-126 (x near 1e-31 and w near 1e-3) lose bits of it.
//
// The 8-bit instruction aligns the products of eight neighbouring k to the largest of them and drops what lies more than
// 13 bits below its leading bit (measured: 2^16 + 2^2 gives 2^16 within such a group, and a full float32 sum across
// groups).  That is far below the rounding of a 16-bit result but not of a float32 one, so a float32 result is computed
// with the 16-bit instruction on codes widened to halves, which hold every e4m3 number: exact products, float32 sums,
// at half the rate.

// The 32 codes of a fragment as 32 halves, for four 16x16x32 MFMAs.
struct Halves {
    v8h h[4];
};

__device__ __forceinline__ Halves widen(v8i codes) {
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    Halves out;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const v2h lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes[i], 1.0f, false);
        const v2h hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes[i], 1.0f, true);
        out.h[i / 2][i % 2 * 4 + 0] = lo[0];
        out.h[i / 2][i % 2 * 4 + 1] = lo[1];
        out.h[i / 2][i % 2 * 4 + 2] = hi[0];
        out.h[i / 2][i % 2 * 4 + 3] = hi[1];
    }
    return out;
}

__device__ __forceinline__ v4f block_product(v8i a, v8i b) {
    const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

// The block products of one fragment of a with each of b's.
template <int TN>
__device__ __forceinline__ void block_products(const v8i (&b)[TN], v8i a, v4f (&p)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j) p[j] = block_product(b[j], a);
}

template <int TN>
__device__ __forceinline__ void block_products(const Halves (&b)[TN], const Halves& a, v4f (&p)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j) p[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int j = 0; j < TN; ++j) p[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[j].h[h], a.h[h], p[j], 0, 0, 0);
}

// Every fragment of a with every one of b.
template <int TM, int TN, int N>
__device__ __forceinline__ void tile_products(const v8i (&b)[TN], const v8i (&a)[TM], v4f (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = block_product(b[i % TN], a[i / TN]);
}

template <int TM, int TN, int N>
__device__ __forceinline__ void tile_products(const Halves (&b)[TN], const Halves (&a)[TM], v4f (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int i = 0; i < N; ++i)
            p[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[i % TN].h[h], a[i / TN].h[h], p[i], 0, 0, 0);
}

__device__ __forceinline__ void take(v8i codes, v8i& out) { out = codes; }
__device__ __forceinline__ void take(v8i codes, Halves& out) { out = widen(codes); }

// A stage of the k loop in LDS: the slabs of BM rows of a and BN rows of b, and the scales of those rows' blocks (b's
// once for each row, also where a block is 128 rows).
template <class T, int BM, int BN, int WAVES_M, int WAVES_N, int kStages, int kGroups, bool kRowScales>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N * kGroups, 2) void product_kernel(ProductArgs a, int tiles_m,
                                                                                      int tiles_n) {
    constexpr int kWaves = WAVES_M * WAVES_N;
    constexpr bool kWide = sizeof(T) == 4;
    constexpr int TM = BM / WAVES_M / 16, TN = BN / WAVES_N / 16;
    constexpr int kScalesAt = (BM + BN) * kSlab, kStageBytes = kScalesAt + (BM + BN) * 4;
    constexpr int kScaleLoads = (BM + BN) / 64;                          // of 64 scales each, shared by the waves;
    constexpr int kScalePer = (kScaleLoads + kWaves - 1) / kWaves;       // where they do not come out even, some twice
    static_assert(kRowScales || 128 % (BN / WAVES_N) == 0, "a wave's columns lie in one block of b");
    using Frag = std::conditional_t<kWide, Halves, v8i>;
    __shared__ __align__(1024) uint8_t all_lds[kGroups * kStages * kStageBytes];
    const int t = threadIdx.x, lane = t & 63;
    const int any_wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int group = any_wave / kWaves, wave = any_wave % kWaves;
    uint8_t* const lds = all_lds + group * (kStages * kStageBytes);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    int bm, bn;
    banded_tile(xcd_order(blockIdx.x, gridDim.x), tiles_m, tiles_n, 8, bm, bn);
    const int m0 = bm * BM, n0 = bn * BN;
    const uint8_t* pa = a.a + (int64_t)m0 * a.ld_a;
    const uint8_t* pb = a.b + (int64_t)n0 * a.ld_b;
    const int rows_a = a.m - m0, rows_b = a.n - n0;
    const int r16 = lane & 15, g = lane >> 4;
    const int wm0 = wm * TM * 16, wn0 = wn * TN * 16;

    using SourceA = SlabSource<BM, kWaves>;
    using SourceB = SlabSource<BN, kWaves>;
    SourceA src_a;
    SourceB src_b;
    src_a.set(pa, (uint32_t)a.ld_a, rows_a, wave, lane);
    src_b.set(pb, (uint32_t)a.ld_b, rows_b, wave, lane);

    // this wave's scales of a stage, 64 a load
    const float* scales[kScalePer];
    uint32_t scale_step[kScalePer], scale_lane[kScalePer];
    int part[kScalePer];
#pragma unroll
    for (int x = 0; x < kScalePer; ++x) {
        part[x] = (wave + x * kWaves) % kScaleLoads;
        if (part[x] < BM / 64) {
            scales[x] = a.a_scale;
            scale_step[x] = (uint32_t)a.m;
            scale_lane[x] = (uint32_t)min(m0 + part[x] * 64 + lane, a.m - 1) * 4;
        } else {
            const int n = min(n0 + (part[x] - BM / 64) * 64 + lane, a.n - 1);
            scales[x] = a.b_scale;
            scale_step[x] = kRowScales ? (uint32_t)a.n : (uint32_t)((a.n + 127) / 128);
            scale_lane[x] = (uint32_t)(kRowScales ? n : n / 128) * 4;
        }
    }

    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // One slab: the fragments of b stay in registers, those of a pass through one ahead of their use, and a row of
    // tiles' sums are scaled and added while the next row's MFMAs run (a lone MFMA followed by the use of its result
    // would leave the matrix core idle for its latency).  The order is prescribed: left to itself the compiler puts
    // each use right behind its MFMA.
    auto multiply = [&](const uint8_t* la) {
        const uint8_t* lb = la + BM * kSlab;
        const float* ls = (const float*)(la + kScalesAt);
        Frag fb[TN], fa[2];
        float sa[TM];
        v4f sb[kRowScales ? TN : 1];
#pragma unroll
        for (int j = 0; j < TN; ++j) take(read_slab(lb, wn0 + j * 16 + r16, g), fb[j]);
        take(read_slab(la, wm0 + r16, g), fa[0]);
        v8i raw;   // codes that are yet to be widened
        if constexpr (kWide && TM * TN > 4) raw = read_slab(la, wm0 + 16 + r16, g);
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = ls[wm0 + i * 16 + r16];
        if constexpr (kRowScales) {
#pragma unroll
            for (int j = 0; j < TN; ++j) sb[j] = *(const v4f*)(ls + BM + wn0 + j * 16 + g * 4);
        } else {
            const float b = ls[BM + wn0];
#pragma unroll
            for (int i = 0; i < TM; ++i) sa[i] *= b;
        }
        if constexpr (TM * TN <= 4) {   // all at once: it takes every tile's MFMAs to cover one's latency
#pragma unroll
            for (int i = 1; i < TM; ++i) take(read_slab(la, wm0 + i * 16 + r16, g), fa[i]);
            v4f p[TM * TN];
            tile_products(fb, fa, p);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = kRowScales ? p[i * TN + j][e] * sb[kRowScales ? j : 0][e] : p[i * TN + j][e];
                        acc[i][j][e] = fmaf(v, sa[i], acc[i][j][e]);
                    }
            return;
        }
        v4f p[2][TN];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i <= TM; ++i) {
            if constexpr (kWide) {
                if (i + 1 < TM) take(raw, fa[(i + 1) & 1]);
                if (i + 2 < TM) raw = read_slab(la, wm0 + (i + 2) * 16 + r16, g);
            } else {
                if (i + 1 < TM) take(read_slab(la, wm0 + (i + 1) * 16 + r16, g), fa[(i + 1) & 1]);
            }
            if (i < TM) block_products(fb, fa[i & 1], p[i & 1]);
            if (i > 0) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = p[(i - 1) & 1][j][e];
                        if constexpr (kRowScales)
                            acc[i - 1][j][e] = fmaf(v * sb[j][e], sa[i - 1], acc[i - 1][j][e]);
                        else
                            acc[i - 1][j][e] = fmaf(v, sa[i - 1], acc[i - 1][j][e]);
                    }
            }
            // the next fragment's reads, then MFMAs with an even share of the multiply-adds (and widenings) after each
            constexpr int kMfma = kWide ? 4 * TN : TN;
            constexpr int kScale = (kRowScales ? 8 : 4) * TN, kWiden = kWide ? 16 : 0;
            const int valu = (i > 0 ? kScale : 0) + (i + 1 < TM ? kWiden : 0);
            if (!kWide && i + 1 < TM) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            if (i < TM) {
#pragma unroll
                for (int x = 0; x < kMfma; ++x) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    if (valu == kScale + kWiden) __builtin_amdgcn_sched_group_barrier(0x2, (kScale + kWiden) / kMfma, 0);
                    else if (valu == kScale) __builtin_amdgcn_sched_group_barrier(0x2, kScale / kMfma, 0);
                    else if (valu == kWiden && kWiden) __builtin_amdgcn_sched_group_barrier(0x2, kWiden ? kWiden / kMfma : 1, 0);
                }
            }
            if (kWide && i + 2 < TM) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // Group i takes the whole slabs i, i + kGroups, ...; the last group takes the cut one first, from the slot that the
    // stages ahead leave free, so that its loads wait along with theirs.
    const int full = a.k / kSlab, tail = a.k % kSlab;
    const auto issue = [&](int s, int slot) {
        uint8_t* stage = lds + slot * kStageBytes;
        const int slab = min(s * kGroups + group, full - 1);
        src_a.fetch((uint32_t)slab * kSlab, stage, wave);
        src_b.fetch((uint32_t)slab * kSlab, stage + BM * kSlab, wave);
#pragma unroll
        for (int x = 0; x < kScalePer; ++x) {
            uint32_t at = scale_lane[x];
            asm("" : "+v"(at));
            load4_to_lds((const uint8_t*)(scales[x] + (int64_t)slab * scale_step[x]) + at,
                         stage + kScalesAt + part[x] * 256);
        }
    };
    const int total = (full + kGroups - 1) / kGroups;
    if (tail && group == kGroups - 1) {
        TailSlab<BM, kWaves> tail_a;
        TailSlab<BN, kWaves> tail_b;
        tail_a.load(pa, (uint32_t)a.ld_a, rows_a, full * kSlab, a.k, wave, lane);
        tail_b.load(pb, (uint32_t)a.ld_b, rows_b, full * kSlab, a.k, wave, lane);
        float scale[kScalePer];
#pragma unroll
        for (int x = 0; x < kScalePer; ++x)
            scale[x] = *(const float*)((const uint8_t*)(scales[x] + (int64_t)full * scale_step[x]) + scale_lane[x]);
        uint8_t* stage = lds + (kStages - 1) * kStageBytes;
        pipeline_ahead<kStages>(total, issue);
        tail_a.put(stage, wave, lane);
        tail_b.put(stage + BM * kSlab, wave, lane);
#pragma unroll
        for (int x = 0; x < kScalePer; ++x) *(float*)(stage + kScalesAt + part[x] * 256 + lane * 4) = scale[x];
    } else {
        pipeline_ahead<kStages>(total, issue);
    }
    pipelined_after<kStages, SourceA::kLoads + SourceB::kLoads + kScalePer>(
        tail != 0, group == kGroups - 1, total, (full - group + kGroups - 1) / kGroups, issue,
        [&](int slot) { multiply(lds + slot * kStageBytes); });

    using Tile = WaveTile<T, TM * 16, TN * 16>;
    constexpr int kJoinAt = kWaves * Tile::kBytes, kJoinBytes = (kGroups - 1) * kWaves * TM * TN * 1024;
    static_assert(kJoinAt + kJoinBytes <= (int)sizeof(all_lds), "every wave's results and the groups' sums fit in LDS");
    meet();   // nobody reads the operands any more
    join_groups<kGroups, kWaves>(acc, group, wave, lane, all_lds + kJoinAt);
    if (group > 0) return;
    uint8_t* mine_lds = all_lds + wave * Tile::kBytes;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            T e[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) e[x] = from_f32<T>(acc[i][j][x]);
            Tile::put(mine_lds, i * 16 + r16, j * 16 + g * 4, e);
        }
    wave_fence();
    const bool wide = (uintptr_t)a.out % 16 == 0 && (a.ld_out * sizeof(T)) % 16 == 0;
    Tile::store(mine_lds, (T*)a.out + (int64_t)(m0 + wm0) * a.ld_out + n0 + wn0, a.ld_out, rows_a - wm0, rows_b - wn0, wide,
                lane);
}

// ---- few rows
//
// With few rows of a the product is bound by reading b, once, and by latency.  A wave takes 16 rows of b straight from
// memory into the MFMA's operand (lane l: the 16-byte chunks l >> 4 and (l >> 4) + 4 of row l & 15, so one load covers
// whole 64-byte sectors), the workgroup's waves share the slabs of those rows among them, and their sums meet in LDS in
// a fixed order.  All loads of the slabs that a wave takes at a time are issued before the first is used.  a (up to 16
// rows for each of kTiles fragments) comes as codes; or, where it is small, as numbers, which every workgroup quantizes
// into its LDS while its first rows of b are on their way.  One token against 8192 x 2048: 5.2 us either way (16.8 MB at
// 3.2 TB/s, about 2.5 us of it a launch's own time), where quantizing first would be a second launch of 2.7 us.

__device__ __forceinline__ v8i load_slab(const uint8_t* row, int at, int g, int k) {
    return __builtin_shufflevector(load_chunk(row, at + g * 16, k), load_chunk(row, at + 64 + g * 16, k), 0, 1, 2, 3, 4,
                                   5, 6, 7);
}

// A whole slab's chunks.
__device__ __forceinline__ v8i load_full_slab(const uint8_t* row, int at, int g) {
    const v4i lo = *(const v4i*)(row + at + g * 16), hi = *(const v4i*)(row + at + 64 + g * 16);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Rows that are quantized on the way, and their numbers (rows rounded up to whole blocks): 16 tokens against 2048 x 2048
// take 8.9 us with their launch, quantized first 13.8 us, 16 against 8192 x 2048 12.2 and 13.7; with twice the numbers 16
// against 8192 x 4096 would take 22.3 us, quantized first 13.3 us.
constexpr int kFewRows = 16;
constexpr int kFewNumbers = 32768;
constexpr int kFewCodedRows = 32;    // rows of codes

// X: the type of a's numbers, or uint8_t for codes.
template <class T, class X, int kTiles, bool kRowScales>
__global__ __launch_bounds__(1024) void few_rows_kernel(ProductArgs a) {
    constexpr bool kWide = sizeof(T) == 4, kCodes = sizeof(X) == 1;
    constexpr int kAhead = kTiles == 1 ? 4 : 2;   // slabs a wave takes at a time
    using Frag = std::conditional_t<kWide, Halves, v8i>;
    __shared__ float sums[16][256 * kTiles];
    __shared__ __align__(16) uint8_t own_codes[kCodes ? 16 : kFewNumbers];   // [row][slab]
    __shared__ float own_scales[kCodes ? 1 : kFewNumbers / kSlab];
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int full = a.k / kSlab, tail = a.k % kSlab, slabs = full + (tail ? 1 : 0);
    const uint8_t* b_row = a.b + (int64_t)min(n0 + r16, a.n - 1) * a.ld_b;
    int row[kTiles];   // rows behind the last repeat it; their results are not stored
#pragma unroll
    for (int i = 0; i < kTiles; ++i) row[i] = min(i * 16 + r16, a.m - 1);
    const int sb_len = kRowScales ? a.n : (a.n + 127) / 128;
    int sb_at[kRowScales ? 4 : 1];
#pragma unroll
    for (int e = 0; e < (kRowScales ? 4 : 1); ++e) sb_at[e] = kRowScales ? min(n0 + g * 4 + e, a.n - 1) : n0 / 128;

    v4f acc[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    struct Slab {
        v8i b, a[kCodes ? kTiles : 1];
        float sb[kRowScales ? 4 : 1], sa[kCodes ? kTiles : 1];
    };
    auto fetch = [&](int s, Slab& slab, auto whole) {
        constexpr bool kFull = decltype(whole)::value;
        slab.b = kFull ? load_full_slab(b_row, s * kSlab, g) : load_slab(b_row, s * kSlab, g, a.k);
#pragma unroll
        for (int e = 0; e < (kRowScales ? 4 : 1); ++e) slab.sb[e] = a.b_scale[(int64_t)s * sb_len + sb_at[e]];
        if constexpr (kCodes) {
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const uint8_t* a_row = a.a + (int64_t)row[i] * a.ld_a;
                slab.a[i] = kFull ? load_full_slab(a_row, s * kSlab, g) : load_slab(a_row, s * kSlab, g, a.k);
                slab.sa[i] = a.a_scale[(int64_t)s * a.m + row[i]];
            }
        }
    };
    auto use = [&](int s, const Slab& slab) {
        Frag fb[1];
        take(slab.b, fb[0]);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            float sa;
            Frag fa;
            if constexpr (kCodes) {
                sa = slab.sa[i];
                take(slab.a[i], fa);
            } else {
                sa = own_scales[row[i] * slabs + s];
                take(load_full_slab(own_codes, (row[i] * slabs + s) * kSlab, g), fa);
            }
            v4f p[1];
            block_products(fb, fa, p);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (kRowScales)
                    acc[i][e] = fmaf(p[0][e] * slab.sb[e], sa, acc[i][e]);
                else
                    acc[i][e] = fmaf(p[0][e], sa * slab.sb[0], acc[i][e]);
            }
        }
    };

    // Slab s belongs to wave s mod waves: kAhead at a time, then one at a time, then the cut one.
    Slab some[kAhead];
    int s = wave;
    bool ahead = s + (kAhead - 1) * waves < full;
    auto fetch_some = [&] {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) fetch(s + u * waves, some[u], std::true_type{});
        __builtin_amdgcn_sched_barrier(0);   // all of the loads, then their uses
    };
    if (ahead) fetch_some();
    if constexpr (!kCodes) {   // 16 lanes a block, as in quantize_rows_kernel
        for (int i = threadIdx.x >> 4; i < a.m * slabs; i += blockDim.x >> 4) {
            const int r = i / slabs, col = (i - r * slabs) * kSlab + (lane & 15) * 8;
            Eight<X> v;
            v.load((const X*)a.a + (int64_t)r * a.ld_a + col, a.k - col);
            const float scale = block_scale(max16(max8(v)));
            *(uint2*)(own_codes + i * kSlab + (lane & 15) * 8) = codes8(v, 1.0f / scale);
            if ((lane & 15) == 0) own_scales[i] = scale;
        }
        meet();
    }
    while (ahead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) use(s + u * waves, some[u]);
        s += kAhead * waves;
        ahead = s + (kAhead - 1) * waves < full;
        if (ahead) fetch_some();
    }
    for (; s < full; s += waves) {
        fetch(s, some[0], std::true_type{});
        use(s, some[0]);
    }
    if (s == full && tail) {
        fetch(s, some[0], std::false_type{});
        use(s, some[0]);
    }

    // sums[wave][row of a][column]
#pragma unroll
    for (int i = 0; i < kTiles; ++i) *(v4f*)&sums[wave][(i * 16 + r16) * 16 + g * 4] = acc[i];
    __syncthreads();
    for (int o = threadIdx.x; o < a.m * 16; o += blockDim.x) {
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) v += sums[w][o];
        if (n0 + (o & 15) < a.n) ((T*)a.out)[(int64_t)(o >> 4) * a.ld_out + n0 + (o & 15)] = from_f32<T>(v);
    }
}

template <class T, class X, int kTiles>
void few_rows(const ProductArgs& a, hipStream_t st) {
    const int slabs = (a.k + kSlab - 1) / kSlab;
    const unsigned grid = (unsigned)((a.n + 15) / 16);
    // Waves so that each takes about four slabs, all of whose loads it issues at once: one token against 8192 x 2048
    // 5.2 us, with a slab a wave 6.7 us.  A wave quantizes four blocks at a time; more waves so that they do it twice at
    // most, and four times where that takes 16 (16 tokens against 2048 x 2048 10.4 to 6.7 us, 4 against 8192 x 2048 7.4
    // to 6.3; 8 against 8192 x 2048 7.7 us in 8 waves and 9.6 in 16).
    const int blocks = sizeof(X) > 1 ? a.m * slabs : 0;
    int waves = 1;
    while (waves < 16 && (waves * 4 < slabs || waves * (waves < 8 ? 8 : 16) < blocks)) waves *= 2;
    if (a.b_rows == 1)
        few_rows_kernel<T, X, kTiles, true><<<grid, waves * 64, 0, st>>>(a);
    else
        few_rows_kernel<T, X, kTiles, false><<<grid, waves * 64, 0, st>>>(a);
}

template <class T, int BM, int BN, int WAVES_M, int WAVES_N, int kStages, int kGroups, bool kRows = true>
void product_tiles(const ProductArgs& a, hipStream_t st) {
    const int tm = (a.m + BM - 1) / BM, tn = (a.n + BN - 1) / BN;
    const unsigned grid = (unsigned)tm * (unsigned)tn;
    constexpr int kThreads = 64 * WAVES_M * WAVES_N * kGroups;
    if constexpr (kRows) {
        if (a.b_rows == 1) {
            product_kernel<T, BM, BN, WAVES_M, WAVES_N, kStages, kGroups, true><<<grid, kThreads, 0, st>>>(a, tm, tn);
            return;
        }
    }
    product_kernel<T, BM, BN, WAVES_M, WAVES_N, kStages, kGroups, false><<<grid, kThreads, 0, st>>>(a, tm, tn);
}

// Few rows: 16 against 2048 x 8192 take 10 us here and 18 us in tiles of 64, 32 take 12 and 18 us, 40 would take 20 and
// 18 us.  Otherwise the largest tiles that leave no compute unit idle; in microseconds, for a 16-bit result with square
// blocks (8-bit MFMAs) and a float32 one with a scale for each row of both (16-bit MFMAs):
//                              256 x 256   256 x 128   128 x 128   64 x 64
//   8192 x 8192 x 2048, 16-bit       146         173         157       303
//   4096 x 2048 x 2048, 16-bit        37          25          25        40
//   2048 x 2048 x 2048, 16-bit        34          22          18        21
//   8192 x 2048 x 8192, float32        -         343         362       478
//   2048 x 2048 x 2048, float32        -          40          30        34
// (256 x 256 holds no float32 kernel's widened operands, nor a scale for each of its columns, in registers.)  Where
// tiles of 64 do not fill the card, two groups of waves share a tile's k loop: 1000 x 512 x 2048 8.9 to 7.5 us, 100 x
// 512 x 8192 25 to 18 us.
//
// 8192 x 8192 x 2048 runs at 1.9 PFLOP/s; hipBLASLt reaches 2.45 with one scale for the whole matrix.  At 2.1 GHz (the
// clock that the power limit leaves) the matrix cores are busy 43% of it and the vector unit, with the scaling
// multiply-adds, 32%; without its loads the kernel takes 137 us, without the first fragments' LDS reads 141 us.  The
// float32 product is bound by the vector unit, which widens each code for two fragments' MFMAs.
template <class T>
hipError_t product(const ProductArgs& a, hipStream_t st) {
    constexpr bool kFloat = sizeof(T) == 4;
    constexpr int64_t kCus = 256;
    const auto tiles = [&](int64_t bm, int64_t bn) { return ((a.m + bm - 1) / bm) * ((a.n + bn - 1) / bn); };
    // Whether tiles fill the card and, with what they hold beyond the edges, are not much more work than smaller ones: a
    // quarter at most (300 x 65536 x 512 24 us, in tiles of 256 27 us), half where the smaller ones are of 64 (130 x
    // 16384 x 2048 18 us, in tiles of 64 21 us).
    const auto large = [&](int64_t bm, int64_t bn, int64_t small) {
        return tiles(bm, bn) >= kCus &&
               tiles(bm, bn) * bm * bn * 4 <= tiles(small, small) * small * small * (small == 64 ? 6 : 5);
    };
    if (a.m <= 16) {
        few_rows<T, uint8_t, 1>(a, st);
    } else if (a.m <= kFewCodedRows) {
        few_rows<T, uint8_t, 2>(a, st);
    } else if (kFloat ? large(256, 128, 128) : a.b_rows == 128 && large(256, 256, 128)) {
        if constexpr (kFloat)
            product_tiles<T, 256, 128, 4, 2, 3, 1>(a, st);
        else
            product_tiles<T, 256, 256, 2, 4, 2, 1, false>(a, st);
    } else if (large(128, 128, 64)) {
        product_tiles<T, 128, 128, 2, 2, 2, 1>(a, st);
    } else if (tiles(64, 64) <= kCus && a.k >= 8 * kSlab) {
        product_tiles<T, 64, 64, 2, 2, 4, 2>(a, st);
    } else {
        product_tiles<T, 64, 64, 2, 2, 4, 1>(a, st);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quantize(const QuantizeArgs& a, hipStream_t st) {
    switch (a.type) {
        case BCJR_TYPE_F32: return quantize<float>(a, st);
        case BCJR_TYPE_BF16: return quantize<__hip_bfloat16>(a, st);
        default: return quantize<_Float16>(a, st);
    }
}

bool fp8_few_rows(int64_t m, int64_t k) { return m <= kFewRows && m * ((k + 127) / 128 * 128) <= kFewNumbers; }

hipError_t launch_fp8_linear_few_rows(const ProductArgs& a, hipStream_t st) {
    switch (a.out_type) {
        case BCJR_TYPE_F32: few_rows<float, float, 1>(a, st); break;
        case BCJR_TYPE_BF16: few_rows<__hip_bfloat16, __hip_bfloat16, 1>(a, st); break;
        default: few_rows<_Float16, _Float16, 1>(a, st); break;
    }
    return hipGetLastError();
}

hipError_t launch_fp8_product(const ProductArgs& a, hipStream_t st) {
    switch (a.out_type) {
        case BCJR_TYPE_F32: return product<float>(a, st);
        case BCJR_TYPE_BF16: return product<__hip_bfloat16>(a, st);
        default: return product<_Float16>(a, st);
    }
}

}  // namespace bcjr
