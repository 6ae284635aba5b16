// orthogonalize.hip -- an update of a weight matrix, orthogonalized by Newton-Schulz products:
//   X = G / (|G|_F + eps);  steps times:  A = X X^T,  B = b A + c A A,  X <- a X + B X
// (on G^T when G has more rows than columns, so A is the smaller square).
//
// X is m x n with m <= n.  It is held scaled by 2^10 as the sum of two halves (hi + lo, 22 bits of mantissa), row-major
// and transposed, so that every product reads both operands along their rows; A and B are symmetric and held scaled by
// 2^8.  The scales keep the entries of a normalised matrix (rms (m n)^-1/2) far from the halves' subnormal range and
// leave room for |X| < 64 and |A|, |B| < 256.  The products run on the 16-bit matrix instructions with float32 sums.
// For a bfloat16 result they take the hi halves alone: each product then rounds its operands to 11 bits, while X itself
// keeps its 22 through a X, which carries the small singular values (rounding X to 11 bits in every step loses them:
// on a rank-16 matrix with 1% noise the result is 4e-2 off; with X kept it is 4e-4, below the 1.7e-3 of rounding the
// result to bfloat16).  For a float32 or float16 result each product is hi hi + hi lo + lo hi, three times the work,
// and the result is as near the exact one as that of float32 products.
#include "bcjr.h"

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "layer_args.hpp"
#include "mfma_tile.hpp"

namespace bcjr {
namespace {

constexpr float kXScale = 1024.0f;
constexpr float kAScale = 256.0f;
constexpr int kPad = 64;        // rows and columns of X are padded with zeros to multiples of it
constexpr int kPartials = 256;  // partial sums of |G|^2 per matrix

__host__ __device__ inline int64_t pad_up(int64_t v) { return (v + kPad - 1) / kPad * kPad; }
inline size_t area(size_t bytes) { return (bytes + 255) & ~(size_t)255; }

struct Layout {
    int64_t m, n, mp, np;   // m <= n, and padded
    bool tall, split;
    size_t partials, x_hi, x_lo, xt_hi[2], xt_lo[2], a_hi, a_lo, b_hi, b_lo, total;
};

Layout make_layout(int64_t batch, int64_t rows, int64_t cols, int32_t out_type) {
    Layout l{};
    l.tall = rows > cols;
    l.m = l.tall ? cols : rows;
    l.n = l.tall ? rows : cols;
    l.mp = pad_up(l.m);
    l.np = pad_up(l.n);
    l.split = out_type != BCJR_TYPE_BF16;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += area(bytes);
        return here;
    };
    const size_t x = (size_t)batch * l.mp * l.np * 2, s = (size_t)batch * l.mp * l.mp * 2;
    l.partials = take((size_t)batch * kPartials * 8);
    l.x_hi = take(x);
    l.x_lo = take(x);
    for (int i = 0; i < 2; ++i) {
        l.xt_hi[i] = take(x);
        l.xt_lo[i] = l.split ? take(x) : 0;
    }
    l.a_hi = take(s);
    l.a_lo = l.split ? take(s) : 0;
    l.b_hi = take(s);
    l.b_lo = l.split ? take(s) : 0;
    l.total = at;
    return l;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__hip_bfloat16 x) {
    return __uint_as_float((uint32_t)__builtin_bit_cast(uint16_t, x) << 16);
}
__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ _Float16 from_f32<_Float16>(float x) { return (_Float16)x; }
template <>
__device__ __forceinline__ __hip_bfloat16 from_f32<__hip_bfloat16>(float x) { return __float2bfloat16(x); }

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

template <class T>
__global__ __launch_bounds__(256) void square_sum_kernel(const T* g, int64_t rows, int64_t cols, int64_t ld,
                                                         int64_t batch_stride, double* partials) {
    __shared__ double lds[4];
    const T* p = g + (int64_t)blockIdx.y * batch_stride;
    double sum = 0.0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            const double v = (double)to_f32(p[r * ld + c]);
            sum += v * v;
        }
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) partials[(int64_t)blockIdx.y * kPartials + blockIdx.x] = sum;
}

__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
    hi = (_Float16)v;
    lo = (_Float16)(v - (float)hi);
}

// G's tile of 64 x 64, normalised and scaled: as it lies into `direct`, transposed into `turned`.
template <class T>
__global__ __launch_bounds__(256) void normalize_kernel(const T* g, int64_t rows, int64_t cols, int64_t ld,
                                                        int64_t batch_stride, const double* partials, int parts,
                                                        float eps, _Float16* direct_hi, _Float16* direct_lo,
                                                        _Float16* turned_hi, _Float16* turned_lo, int64_t rows_p,
                                                        int64_t cols_p) {
    __shared__ double lds[4];
    __shared__ uint32_t tile[64][65];
    const int t = threadIdx.x;
    const int64_t item = blockIdx.z;
    const double total = block_sum(t < parts ? partials[item * kPartials + t] : 0.0, lds);
    const float norm = (float)(sqrt(total) + (double)eps);
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const T* p = g + item * batch_stride;
    const int64_t base = item * rows_p * cols_p;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = i * 4 + (t >> 6), c = t & 63;
        float v = 0.0f;
        if (r0 + r < rows && c0 + c < cols) v = to_f32(p[(r0 + r) * ld + c0 + c]) / norm * kXScale;
        _Float16 hi, lo;
        split(v, hi, lo);
        if (direct_hi) direct_hi[base + (r0 + r) * cols_p + c0 + c] = hi;
        if (direct_lo) direct_lo[base + (r0 + r) * cols_p + c0 + c] = lo;
        tile[r][c] = (uint32_t)__builtin_bit_cast(uint16_t, hi) | ((uint32_t)__builtin_bit_cast(uint16_t, lo) << 16);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int c = i * 4 + (t >> 6), r = t & 63;
        const uint32_t w = tile[r][c];
        if (turned_hi) turned_hi[base + (c0 + c) * rows_p + r0 + r] = __builtin_bit_cast(_Float16, (uint16_t)(w & 0xffff));
        if (turned_lo) turned_lo[base + (c0 + c) * rows_p + r0 + r] = __builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
    }
}

// ---------------------------------------------------------------- the products

enum Mode { kGram, kPoly, kStep };

struct ProdArgs {
    const _Float16 *p_hi, *p_lo;   // [rows][k]
    const _Float16 *q_hi, *q_lo;   // [cols][k]
    int64_t p_batch, q_batch;      // elements from one matrix of the batch to the next
    int32_t rows, cols, k;         // multiples of kPad
    _Float16 *o_hi, *o_lo;         // [rows][cols]; kPoly reads A from a_hi, a_lo, kStep reads X here
    const _Float16 *a_hi, *a_lo;
    _Float16 *t_hi, *t_lo;         // kStep: the transpose [cols][rows]
    int64_t o_batch;
    float alpha, beta;             // kGram: alpha acc; kPoly: alpha A + beta acc; kStep: alpha X + beta acc
    void* out;                     // kStep, last: the result
    int32_t m, n, tall;
    int64_t out_batch;
};

// The first or second 32 halves of a slab.
__device__ __forceinline__ v8h half_slab(v8i v, int h) {
    return __builtin_bit_cast(v8h, h == 0 ? __builtin_shufflevector(v, v, 0, 1, 2, 3)
                                          : __builtin_shufflevector(v, v, 4, 5, 6, 7));
}

__device__ __forceinline__ v4f multiply(v8h a, v8h b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

template <Mode kMode, bool kSplit, class T, int BM, int BN, int WAVES_M, int WAVES_N>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N) void ortho_product_kernel(ProdArgs a, int tiles_m, int tiles_n) {
    constexpr int kWaves = WAVES_M * WAVES_N;
    constexpr int TM = BM / WAVES_M / 16, TN = BN / WAVES_N / 16;
    constexpr bool kSymmetric = kMode != kStep;
    __shared__ __align__(1024) uint8_t lds[2][(BM + BN) * kSlab];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int r16 = lane & 15, g = lane >> 4;
    int bm, bn;
    const int id = xcd_order(blockIdx.x, gridDim.x);
    if constexpr (kSymmetric) {   // the tiles on and below the diagonal, row by row
        bm = (int)((sqrtf(8.0f * (float)id + 1.0f) - 1.0f) * 0.5f);
        while (bm * (bm + 1) / 2 > id) --bm;
        while ((bm + 1) * (bm + 2) / 2 <= id) ++bm;
        bn = id - bm * (bm + 1) / 2;
    } else {
        banded_tile(id, tiles_m, tiles_n, 8, bm, bn);
    }
    const int m0 = bm * BM, n0 = bn * BN;
    const int64_t item = blockIdx.z;
    const uint32_t ld = (uint32_t)a.k * 2;
    const int per = a.k / 64;
    const int slabs = kSplit ? 3 * per : per;
    const uint8_t* p_hi = (const uint8_t*)(a.p_hi + item * a.p_batch + (int64_t)m0 * a.k);
    const uint8_t* q_hi = (const uint8_t*)(a.q_hi + item * a.q_batch + (int64_t)n0 * a.k);
    const uint8_t* p_lo = kSplit ? (const uint8_t*)(a.p_lo + item * a.p_batch + (int64_t)m0 * a.k) : nullptr;
    const uint8_t* q_lo = kSplit ? (const uint8_t*)(a.q_lo + item * a.q_batch + (int64_t)n0 * a.k) : nullptr;

    SlabSource<BM, kWaves> src_p;
    SlabSource<BN, kWaves> src_q;
    src_p.set(p_hi, ld, a.rows - m0, wave, lane);
    src_q.set(q_hi, ld, a.cols - n0, wave, lane);
    auto fetch = [&](int s, uint8_t* to) {
        const int part = kSplit ? s / per : 0;   // hi hi, hi lo, lo hi
        const uint32_t at = (uint32_t)(s - part * per) * kSlab;
        src_p.base = kSplit && part == 2 ? p_lo : p_hi;
        src_q.base = kSplit && part == 1 ? q_lo : q_hi;
        src_p.fetch(at, to, wave);
        src_q.fetch(at, to + BM * kSlab, wave);
    };

    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int wm0 = wm * TM * 16, wn0 = wn * TN * 16;

    fetch(0, lds[0]);
    for (int s = 0; s < slabs; ++s) {
        wait_loads();
        __syncthreads();   // slab s is in LDS, and nobody reads the other buffer any more
        if (s + 1 < slabs) fetch(s + 1, lds[(s + 1) & 1]);
        const uint8_t* lp = lds[s & 1];
        const uint8_t* lq = lp + BM * kSlab;
        v8i fq[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) fq[j] = read_slab(lq, wn0 + j * 16 + r16, g);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const v8i fp = read_slab(lp, wm0 + i * 16 + r16, g);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = multiply(half_slab(fq[j], h), half_slab(fp, h), acc[i][j]);
        }
    }

    // A lane's four sums are neighbours along a row of the result.
    const int64_t o = item * a.o_batch;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int row = m0 + wm0 + i * 16 + r16;
        if (row >= a.rows) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int col = n0 + wn0 + j * 16 + g * 4;
            if (col >= a.cols) continue;
            const int64_t at = o + (int64_t)row * a.cols + col;
            float v[4];
            if constexpr (kMode == kGram) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = a.alpha * acc[i][j][e];
            } else {
                const v4h hi = *(const v4h*)((kMode == kPoly ? a.a_hi : a.o_hi) + at);
                v4h lo = {0, 0, 0, 0};
                if (kMode == kStep || kSplit) lo = *(const v4h*)((kMode == kPoly ? a.a_lo : a.o_lo) + at);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = fmaf(a.alpha, (float)hi[e] + (float)lo[e], a.beta * acc[i][j][e]);
            }
            if (kMode == kStep && a.out) {
                T* out = (T*)a.out + item * a.out_batch;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (row < a.m && col + e < a.n)
                        out[a.tall ? (int64_t)(col + e) * a.m + row : (int64_t)row * a.n + col + e] =
                            from_f32<T>(v[e] * (1.0f / kXScale));
                continue;
            }
            v4h hi, lo;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                _Float16 h, l;
                split(v[e], h, l);
                hi[e] = h;
                lo[e] = l;
            }
            *(v4h*)(a.o_hi + at) = hi;
            if (kMode == kStep || kSplit) *(v4h*)(a.o_lo + at) = lo;
            if (kMode == kStep || bm != bn) {   // the mirror image, or the transpose
                _Float16* t_hi = (kMode == kStep ? a.t_hi : a.o_hi) + o + (int64_t)col * a.rows + row;
                _Float16* t_lo = kSplit ? (kMode == kStep ? a.t_lo : a.o_lo) + o + (int64_t)col * a.rows + row : nullptr;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    t_hi[(int64_t)e * a.rows] = hi[e];
                    if (kSplit) t_lo[(int64_t)e * a.rows] = lo[e];
                }
            }
        }
    }
}

template <Mode kMode, bool kSplit, class T, int BM, int WAVES_M, int WAVES_N>
void launch_tiles(const ProdArgs& a, int64_t batch, hipStream_t st) {
    const int tm = (a.rows + BM - 1) / BM, tn = (a.cols + BM - 1) / BM;
    const unsigned tiles = kMode == kStep ? (unsigned)tm * tn : (unsigned)tm * (tm + 1) / 2;
    ortho_product_kernel<kMode, kSplit, T, BM, BM, WAVES_M, WAVES_N>
        <<<dim3(tiles, 1, (unsigned)batch), 64 * WAVES_M * WAVES_N, 0, st>>>(a, tm, tn);
}

template <Mode kMode, bool kSplit, class T>
void launch_product(const ProdArgs& a, int64_t batch, hipStream_t st) {
    const auto tiles = [&](int64_t size) {
        const int64_t tm = (a.rows + size - 1) / size, tn = (a.cols + size - 1) / size;
        return batch * (kMode == kStep ? tm * tn : tm * (tm + 1) / 2);
    };
    if (tiles(256) >= 192)
        launch_tiles<kMode, kSplit, T, 256, 2, 4>(a, batch, st);
    else if (tiles(128) >= 192)
        launch_tiles<kMode, kSplit, T, 128, 2, 2>(a, batch, st);
    else
        launch_tiles<kMode, kSplit, T, 64, 2, 2>(a, batch, st);
}

template <bool kSplit, class Out>
hipError_t iterate(const OrthoArgs& o, const Layout& l, hipStream_t st) {
    unsigned char* ws = o.ws;
    auto at = [&](size_t off) { return (_Float16*)(ws + off); };
    const int64_t x_batch = l.mp * l.np, s_batch = l.mp * l.mp;
    for (int s = 0; s < o.steps; ++s) {
        const int cur = s & 1, next = cur ^ 1;
        ProdArgs gram{};
        gram.p_hi = gram.q_hi = at(l.x_hi);
        gram.p_lo = gram.q_lo = at(l.x_lo);
        gram.p_batch = gram.q_batch = x_batch;
        gram.rows = gram.cols = (int32_t)l.mp;
        gram.k = (int32_t)l.np;
        gram.o_hi = at(l.a_hi);
        gram.o_lo = at(l.a_lo);
        gram.o_batch = s_batch;
        gram.alpha = kAScale / (kXScale * kXScale);
        launch_product<kGram, kSplit, float>(gram, o.batch, st);

        ProdArgs poly{};
        poly.p_hi = poly.q_hi = poly.a_hi = at(l.a_hi);
        poly.p_lo = poly.q_lo = poly.a_lo = at(l.a_lo);
        poly.p_batch = poly.q_batch = s_batch;
        poly.rows = poly.cols = poly.k = (int32_t)l.mp;
        poly.o_hi = at(l.b_hi);
        poly.o_lo = at(l.b_lo);
        poly.o_batch = s_batch;
        poly.alpha = o.b;
        poly.beta = o.c / kAScale;
        launch_product<kPoly, kSplit, float>(poly, o.batch, st);

        ProdArgs step{};
        step.p_hi = at(l.b_hi);
        step.p_lo = at(l.b_lo);
        step.p_batch = s_batch;
        step.q_hi = at(l.xt_hi[cur]);
        step.q_lo = at(l.xt_lo[cur]);
        step.q_batch = x_batch;
        step.rows = (int32_t)l.mp;
        step.cols = (int32_t)l.np;
        step.k = (int32_t)l.mp;
        step.o_hi = at(l.x_hi);
        step.o_lo = at(l.x_lo);
        step.t_hi = at(l.xt_hi[next]);
        step.t_lo = at(l.xt_lo[next]);
        step.o_batch = x_batch;
        step.alpha = o.a;
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
    const int parts = (int)(o.rows < kPartials ? o.rows : kPartials);
    square_sum_kernel<In><<<dim3((unsigned)parts, (unsigned)o.batch), 256, 0, st>>>((const In*)o.g, o.rows, o.cols,
                                                                                   o.ld_g, o.batch_g, partials);
    auto at = [&](size_t off) { return (_Float16*)(o.ws + off); };
    _Float16 *x_hi = at(l.x_hi), *x_lo = at(l.x_lo), *xt_hi = at(l.xt_hi[0]);
    _Float16* xt_lo = l.split ? at(l.xt_lo[0]) : nullptr;
    const int64_t rp = pad_up(o.rows), cp = pad_up(o.cols);
    normalize_kernel<In><<<dim3((unsigned)(cp / 64), (unsigned)(rp / 64), (unsigned)o.batch), 256, 0, st>>>(
        (const In*)o.g, o.rows, o.cols, o.ld_g, o.batch_g, partials, parts, o.eps, l.tall ? xt_hi : x_hi,
        l.tall ? xt_lo : x_lo, l.tall ? x_hi : xt_hi, l.tall ? x_lo : xt_lo, rp, cp);
    switch (o.out_type) {
        case BCJR_TYPE_F32: return iterate<true, float>(o, l, st);
        case BCJR_TYPE_BF16: return iterate<false, __hip_bfloat16>(o, l, st);
        default: return iterate<true, _Float16>(o, l, st);
    }
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
