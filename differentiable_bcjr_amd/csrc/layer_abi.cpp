// layer_abi.cpp -- the C-ABI of the quantized layer and the orthogonalized update (declared in include/bcjr.h):
// argument checks and dispatch.  Every check runs on the host before any HIP call.
#include "bcjr.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "layer_args.hpp"

namespace {

using namespace bcjr;

constexpr int64_t kMaxDim = (int64_t)1 << 23;       // rows, columns and reduction lengths of the 8-bit operators
constexpr int64_t kMaxDistance = (int64_t)1 << 23;  // bytes between the rows of 8-bit operands: a tile's 256 rows within 2^31
// Grids stay under 2^32 threads: a product's results in tiles of 16 x 16 (the kernels' tiles are 128 to 256 times as
// large, with 512 threads), a quantization's blocks of 256 threads for 16 x 128 numbers.
constexpr int64_t kMaxTiles = (int64_t)1 << 29;
constexpr int64_t kMaxQuantizeBlocks = (int64_t)1 << 23;
constexpr int64_t kMaxUpdateDim = 65536;
constexpr int64_t kMaxBatch = 65535;                // a grid's third dimension
constexpr int32_t kMaxSteps = 1000;

int hip_status(hipError_t e) { return e == hipSuccess ? BCJR_OK : BCJR_ERR_HIP; }

bool known_type(int32_t t) { return t == BCJR_TYPE_F32 || t == BCJR_TYPE_BF16 || t == BCJR_TYPE_F16; }

bool dim(int64_t v) { return v >= 0 && v <= kMaxDim; }

int64_t blocks(int64_t v, int64_t of) { return (v + of - 1) / of; }

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// An 8-bit matrix: 16-byte boundaries throughout, rows no closer than their length.
bool rows16(const void* p, int64_t ld, int64_t cols) {
    return ((uintptr_t)p & 15u) == 0 && ld % 16 == 0 && ld >= cols && ld <= kMaxDistance;
}

// Room for the codes and scales of a matrix in a caller's buffer, each part on a 256-byte boundary.
struct Coded {
    int64_t ld;
    size_t scale_at, total;
    uint8_t* q;
    float* scale;

    Coded at(void* base) const {
        Coded c = *this;
        c.q = total ? (uint8_t*)base : nullptr;
        c.scale = total ? (float*)((uint8_t*)base + scale_at) : nullptr;
        return c;
    }
};

Coded coded(int64_t rows, int64_t cols, int64_t block_rows) {
    Coded c{};
    c.ld = blocks(cols, 16) * 16;
    c.scale_at = align256((size_t)rows * (size_t)c.ld);
    c.total = c.scale_at + align256((size_t)blocks(rows, block_rows) * (size_t)blocks(cols, 128) * sizeof(float));
    return c;
}

// What a linear layer's backward needs of its forward: x^T for the weights' gradient, w^T for x's.
struct SavedPlan {
    Coded x_t, w_t;
    size_t total;
};

SavedPlan saved_plan(int64_t m, int64_t n, int64_t k, int32_t grads) {
    SavedPlan p{};
    if (grads & BCJR_GRAD_W) p.x_t = coded(k, m, 1);
    if (grads & BCJR_GRAD_X) p.w_t = coded(k, n, 128);
    p.total = p.x_t.total + p.w_t.total;
    return p;
}

// Sizes for which every product of the layer and its gradients is within one grid.
bool linear_dims(int64_t m, int64_t n, int64_t k) {
    if (!dim(m) || !dim(n) || !dim(k)) return false;
    const auto fits = [](int64_t rows, int64_t cols) {
        return blocks(rows, 16) * blocks(cols, 16) <= kMaxTiles &&
               blocks(rows, 16) * blocks(cols, 128) <= kMaxQuantizeBlocks;
    };
    return fits(m, n) && fits(m, k) && fits(n, k);
}

bool scratch(const void* p, size_t bytes, size_t need) {
    return need == 0 || (p && ((uintptr_t)p & 255u) == 0 && bytes >= need);
}

QuantizeArgs quantize_args(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ld, int32_t block_rows,
                           const Coded& c, const Coded& c_t) {
    return QuantizeArgs{x, type, block_rows, rows, cols, ld, c.q, c.ld, c.scale, c_t.q, c_t.ld, c_t.scale};
}

ProductArgs product_args(const Coded& a, const Coded& b, int32_t b_rows, int64_t m, int64_t n, int64_t k, void* out,
                         int32_t type, int64_t ld) {
    return ProductArgs{a.q, a.scale, b.q, b.scale, a.ld, b.ld, (int32_t)m, (int32_t)n, (int32_t)k, b_rows, out, ld,
                       type};
}

bool update_shape(int64_t batch, int64_t rows, int64_t cols, int32_t out_type) {
    return batch >= 1 && batch <= kMaxBatch && rows >= 1 && rows <= kMaxUpdateDim && cols >= 1 &&
           cols <= kMaxUpdateDim && known_type(out_type);
}

}  // namespace

extern "C" {

int fp8_block_quantize(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ld_x, int32_t block_rows,
                       void* q, int64_t ld_q, float* scale, void* q_t, int64_t ld_qt, float* scale_t, void* stream) {
    if (!known_type(type) || (block_rows != 1 && block_rows != 128) || !dim(rows) || !dim(cols)) return BCJR_ERR_SIZE;
    if (rows == 0 || cols == 0) return BCJR_OK;
    if (!x || !q || !scale || (q_t == nullptr) != (scale_t == nullptr)) return BCJR_ERR_NULL;
    if (ld_x < cols || !rows16(q, ld_q, cols) || (q_t && !rows16(q_t, ld_qt, rows))) return BCJR_ERR_LAYOUT;
    if (blocks(rows, 16) * blocks(cols, 128) > kMaxQuantizeBlocks) return BCJR_ERR_SIZE;
    const QuantizeArgs a{x, type, block_rows, rows, cols, ld_x, (uint8_t*)q, ld_q, scale, (uint8_t*)q_t, ld_qt, scale_t};
    return hip_status(launch_fp8_quantize(a, (hipStream_t)stream));
}

int fp8_block_matmul(const void* a, int64_t ld_a, const float* a_scale, const void* b, int64_t ld_b,
                     const float* b_scale, int32_t b_block_rows, int64_t m, int64_t n, int64_t k, void* out,
                     int32_t out_type, int64_t ld_out, void* stream) {
    if (!known_type(out_type) || (b_block_rows != 1 && b_block_rows != 128) || !dim(m) || !dim(n) || !dim(k))
        return BCJR_ERR_SIZE;
    if (m == 0 || n == 0) return BCJR_OK;
    if (!out || (k > 0 && (!a || !a_scale || !b || !b_scale))) return BCJR_ERR_NULL;
    if (ld_out < n || (k > 0 && (!rows16(a, ld_a, k) || !rows16(b, ld_b, k)))) return BCJR_ERR_LAYOUT;
    if (blocks(m, 16) * blocks(n, 16) > kMaxTiles) return BCJR_ERR_SIZE;
    const ProductArgs p{(const uint8_t*)a, a_scale, (const uint8_t*)b, b_scale, ld_a, ld_b, (int32_t)m, (int32_t)n,
                        (int32_t)k, b_block_rows, out, ld_out, out_type};
    return hip_status(launch_fp8_product(p, (hipStream_t)stream));
}

size_t fp8_linear_saved_bytes(int64_t m, int64_t n, int64_t k, int32_t grads) {
    return linear_dims(m, n, k) ? saved_plan(m, n, k, grads).total : 0;
}

size_t fp8_linear_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (!linear_dims(m, n, k)) return 0;
    const size_t forward = coded(m, k, 1).total + coded(n, k, 128).total;
    const size_t backward = coded(m, n, 1).total + coded(n, m, 1).total;
    return forward > backward ? forward : backward;
}

int fp8_linear_forward(const void* x, int32_t type, int64_t m, int64_t ld_x, const void* w, int32_t w_type, int64_t n,
                       int64_t ld_w, int64_t k, int32_t grads, void* out, int64_t ld_out, void* saved,
                       size_t saved_bytes, void* workspace, size_t workspace_bytes, void* stream) {
    if (!known_type(type) || !known_type(w_type) || !linear_dims(m, n, k) || grads < 0 || grads > 3) return BCJR_ERR_SIZE;
    const bool have_x = m > 0 && k > 0, have_w = n > 0 && k > 0, have_out = m > 0 && n > 0;
    if ((have_x && !x) || (have_w && !w) || (have_out && !out)) return BCJR_ERR_NULL;
    if ((have_x && ld_x < k) || (have_w && ld_w < k) || (have_out && ld_out < n)) return BCJR_ERR_LAYOUT;
    const SavedPlan keep = saved_plan(m, n, k, grads);
    if (!scratch(saved, saved_bytes, keep.total) ||
        !scratch(workspace, workspace_bytes, fp8_linear_workspace_bytes(m, n, k)))
        return BCJR_ERR_WORKSPACE;
    const Coded xc = coded(m, k, 1).at(workspace), wc = coded(n, k, 128).at((uint8_t*)workspace + coded(m, k, 1).total);
    Coded x_t{}, w_t{};
    if (grads & BCJR_GRAD_W) x_t = keep.x_t.at(saved);
    if (grads & BCJR_GRAD_X) w_t = keep.w_t.at((uint8_t*)saved + keep.x_t.total);
    const hipStream_t st = (hipStream_t)stream;
    hipError_t e = hipSuccess;
    if (have_x) e = launch_fp8_quantize(quantize_args(x, type, m, k, ld_x, 1, xc, x_t), st);
    if (e == hipSuccess && have_w) e = launch_fp8_quantize(quantize_args(w, w_type, n, k, ld_w, 128, wc, w_t), st);
    if (e == hipSuccess && have_out) e = launch_fp8_product(product_args(xc, wc, 128, m, n, k, out, type, ld_out), st);
    return hip_status(e);
}

int fp8_linear_backward(const void* dy, int32_t type, int64_t m, int64_t ld_dy, int64_t n, int64_t k, int32_t grads,
                        const void* saved, size_t saved_bytes, void* dx, int64_t ld_dx, void* dw, int32_t dw_type,
                        int64_t ld_dw, void* workspace, size_t workspace_bytes, void* stream) {
    if (!known_type(type) || !known_type(dw_type) || !linear_dims(m, n, k) || grads < 0 || grads > 3)
        return BCJR_ERR_SIZE;
    const bool have_dy = m > 0 && n > 0, have_dx = (grads & BCJR_GRAD_X) && m > 0 && k > 0,
               have_dw = (grads & BCJR_GRAD_W) && n > 0 && k > 0;
    if ((have_dy && !dy) || (have_dx && !dx) || (have_dw && !dw)) return BCJR_ERR_NULL;
    if ((have_dy && ld_dy < n) || (have_dx && ld_dx < k) || (have_dw && ld_dw < k)) return BCJR_ERR_LAYOUT;
    const SavedPlan keep = saved_plan(m, n, k, grads);
    if (!scratch(saved, saved_bytes, keep.total) ||
        !scratch(workspace, workspace_bytes, fp8_linear_workspace_bytes(m, n, k)))
        return BCJR_ERR_WORKSPACE;
    const Coded dc = coded(m, n, 1).at(workspace);
    Coded dc_t{};
    if (grads & BCJR_GRAD_W) dc_t = coded(n, m, 1).at((uint8_t*)workspace + coded(m, n, 1).total);
    const hipStream_t st = (hipStream_t)stream;
    hipError_t e = hipSuccess;
    if (have_dy && grads) e = launch_fp8_quantize(quantize_args(dy, type, m, n, ld_dy, 1, dc, dc_t), st);
    if (e == hipSuccess && have_dx) {
        const Coded w_t = keep.w_t.at((uint8_t*)const_cast<void*>(saved) + keep.x_t.total);
        e = launch_fp8_product(product_args(dc, w_t, 128, m, k, n, dx, type, ld_dx), st);
    }
    if (e == hipSuccess && have_dw) {
        const Coded x_t = keep.x_t.at(const_cast<void*>(saved));
        e = launch_fp8_product(product_args(dc_t, x_t, 1, n, k, m, dw, dw_type, ld_dw), st);
    }
    return hip_status(e);
}

size_t fp8_linear_quantized_workspace_bytes(int64_t m, int64_t k) {
    if (!dim(m) || !dim(k) || m == 0 || k == 0 || fp8_few_rows(m, k)) return 0;
    return coded(m, k, 1).total;
}

int fp8_linear_quantized(const void* x, int32_t type, int64_t m, int64_t ld_x, const void* w, int64_t ld_w,
                         const float* w_scale, int32_t w_block_rows, int64_t n, int64_t k, void* out, int64_t ld_out,
                         void* workspace, size_t workspace_bytes, void* stream) {
    if (!known_type(type) || (w_block_rows != 1 && w_block_rows != 128) || !linear_dims(m, n, k)) return BCJR_ERR_SIZE;
    if (m == 0 || n == 0) return BCJR_OK;
    if (!out || (k > 0 && (!x || !w || !w_scale))) return BCJR_ERR_NULL;
    if (ld_out < n || (k > 0 && (ld_x < k || !rows16(w, ld_w, k)))) return BCJR_ERR_LAYOUT;
    const size_t need = fp8_linear_quantized_workspace_bytes(m, k);
    if (!scratch(workspace, workspace_bytes, need)) return BCJR_ERR_WORKSPACE;
    const hipStream_t st = (hipStream_t)stream;
    ProductArgs p{(const uint8_t*)x, nullptr, (const uint8_t*)w, w_scale, ld_x, ld_w, (int32_t)m, (int32_t)n,
                  (int32_t)k, w_block_rows, out, ld_out, type};
    if (fp8_few_rows(m, k)) return hip_status(launch_fp8_linear_few_rows(p, st));
    if (need > 0) {
        const Coded c = coded(m, k, 1).at(workspace);
        const hipError_t e = launch_fp8_quantize(quantize_args(x, type, m, k, ld_x, 1, c, Coded{}), st);
        if (e != hipSuccess) return BCJR_ERR_HIP;
        p.a = c.q;
        p.a_scale = c.scale;
        p.ld_a = c.ld;
    }
    return hip_status(launch_fp8_product(p, st));
}

size_t orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, int32_t out_type) {
    return update_shape(batch, rows, cols, out_type) ? ortho_workspace(batch, rows, cols, out_type) : 0;
}

int orthogonalize(const void* g, int32_t type, int64_t batch, int64_t rows, int64_t cols, int64_t ld_g, int64_t batch_g,
                  int32_t steps, float a, float b, float c, float eps, void* out, int32_t out_type, void* workspace,
                  size_t workspace_bytes, void* stream) {
    if (!known_type(type) || !update_shape(batch, rows, cols, out_type) || steps < 1 || steps > kMaxSteps ||
        !std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !std::isfinite(eps) || eps < 0.0f)
        return BCJR_ERR_SIZE;
    if (!g || !out) return BCJR_ERR_NULL;
    if (ld_g < cols || (batch > 1 && batch_g < 0)) return BCJR_ERR_LAYOUT;
    if (!workspace || ((uintptr_t)workspace & 255u) != 0 ||
        workspace_bytes < ortho_workspace(batch, rows, cols, out_type))
        return BCJR_ERR_WORKSPACE;
    const OrthoArgs o{g, type, batch, rows, cols, ld_g, batch_g, steps, a, b, c, eps, out, out_type,
                      (unsigned char*)workspace};
    return hip_status(launch_orthogonalize(o, (hipStream_t)stream));
}

}  // extern "C"
