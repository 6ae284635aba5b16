// layer_args.hpp -- argument blocks passed by value from the C-ABI to the kernels of a quantized layer (8-bit block
// quantization and its product) and of the orthogonalized update.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bcjr {

struct QuantizeArgs {
    const void* x;        // [rows, cols], rows ld_x elements apart
    int32_t type;         // BCJR_TYPE_*
    int32_t block_rows;   // 1 or 128
    int64_t rows;
    int64_t cols;
    int64_t ld_x;
    uint8_t* q;           // [rows, cols], rows ld_q bytes apart
    int64_t ld_q;
    float* scale;         // [ceil(cols / 128)][ceil(rows / block_rows)]
    uint8_t* q_t;         // [cols, rows], rows ld_qt bytes apart, or nullptr
    int64_t ld_qt;
    float* scale_t;       // [ceil(rows / 128)][ceil(cols / block_rows)]
};

struct ProductArgs {
    const uint8_t* a;     // [m, k] e4m3, rows ld_a bytes apart
    const float* a_scale; // [ceil(k / 128)][m]
    const uint8_t* b;     // [n, k] e4m3, rows ld_b bytes apart
    const float* b_scale; // [ceil(k / 128)][ceil(n / b_rows)]
    int64_t ld_a, ld_b;
    int32_t m, n, k;
    int32_t b_rows;       // 1 or 128
    void* out;            // [m, n], rows ld_out elements apart
    int64_t ld_out;
    int32_t out_type;     // BCJR_TYPE_*
};

struct OrthoArgs {
    const void* g;        // [batch][rows, cols]
    int32_t type;
    int64_t batch, rows, cols, ld_g, batch_g;
    int32_t steps;
    float a, b, c, eps;
    void* out;            // [batch][rows, cols], contiguous
    int32_t out_type;
    unsigned char* ws;
};

hipError_t launch_fp8_quantize(const QuantizeArgs& a, hipStream_t st);
bool fp8_few_rows(int64_t m, int64_t k);   // whether a product of m rows quantizes them on the way
hipError_t launch_fp8_linear_few_rows(const ProductArgs& a, hipStream_t st);   // a: numbers of out_type, ld_a elements
hipError_t launch_fp8_product(const ProductArgs& a, hipStream_t st);
size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols, int32_t out_type);
hipError_t launch_orthogonalize(const OrthoArgs& a, hipStream_t st);

}  // namespace bcjr
