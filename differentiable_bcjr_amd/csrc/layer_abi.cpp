// layer_abi.cpp -- the C-ABI of the quantized layer and the orthogonalized update (declared in include/bcjr.h):
// argument checks and dispatch.  Every check runs on the host before any HIP call.
#include "bcjr.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "layer_args.hpp"

namespace {

using namespace bcjr;

constexpr int64_t kMaxDim = (int64_t)1 << 30;       // rows, columns and reduction lengths of the 8-bit operators
constexpr int64_t kMaxTiles = ((int64_t)1 << 31) - 1;
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
    return ((uintptr_t)p & 15u) == 0 && ld % 16 == 0 && ld >= cols && ld < kMaxTiles;
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
    if (blocks(rows, 16) * blocks(cols, 128) > kMaxTiles) return BCJR_ERR_SIZE;
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

size_t fp8_linear_quantized_workspace_bytes(int64_t m, int64_t k) {
    if (!dim(m) || !dim(k) || m == 0 || k == 0 || fp8_few_rows(m)) return 0;
    return align256((size_t)m * (size_t)blocks(k, 16) * 16) + (size_t)m * (size_t)blocks(k, 128) * sizeof(float);
}

int fp8_linear_quantized(const void* x, int32_t type, int64_t m, int64_t ld_x, const void* w, int64_t ld_w,
                         const float* w_scale, int32_t w_block_rows, int64_t n, int64_t k, void* out, int64_t ld_out,
                         void* workspace, size_t workspace_bytes, void* stream) {
    if (!known_type(type) || (w_block_rows != 1 && w_block_rows != 128) || !dim(m) || !dim(n) || !dim(k))
        return BCJR_ERR_SIZE;
    if (m == 0 || n == 0) return BCJR_OK;
    if (!out || (k > 0 && (!x || !w || !w_scale))) return BCJR_ERR_NULL;
    if (ld_out < n || (k > 0 && (ld_x < k || !rows16(w, ld_w, k)))) return BCJR_ERR_LAYOUT;
    if (blocks(m, 16) * blocks(n, 16) > kMaxTiles || blocks(m, 16) * blocks(k, 128) > kMaxTiles) return BCJR_ERR_SIZE;
    const size_t need = fp8_linear_quantized_workspace_bytes(m, k);
    if (need > 0 && (!workspace || ((uintptr_t)workspace & 255u) != 0 || workspace_bytes < need))
        return BCJR_ERR_WORKSPACE;
    ProductArgs p{(const uint8_t*)x, nullptr, (const uint8_t*)w, w_scale, ld_x, ld_w, (int32_t)m, (int32_t)n,
                  (int32_t)k, w_block_rows, out, ld_out, type};
    if (fp8_few_rows(m)) return hip_status(launch_fp8_linear_few_rows(p, (hipStream_t)stream));
    if (need > 0) {
        const int64_t ld = blocks(k, 16) * 16;
        uint8_t* q = (uint8_t*)workspace;
        float* scale = (float*)(q + align256((size_t)m * (size_t)ld));
        const QuantizeArgs a{x, type, 1, m, k, ld_x, q, ld, scale, nullptr, 0, nullptr};
        const hipError_t e = launch_fp8_quantize(a, (hipStream_t)stream);
        if (e != hipSuccess) return BCJR_ERR_HIP;
        p.a = q;
        p.a_scale = scale;
        p.ld_a = ld;
    }
    return hip_status(launch_fp8_product(p, (hipStream_t)stream));
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
