// mfma_tile.hpp -- what the matrix-product kernels share: operand tiles in LDS as rows of 128-byte slabs, their
// fragments for the 16x16 MFMA instructions, and the order in which workgroups take output tiles.
//
// Both products here are "row times row": out[i][j] = sum_k a[i][k] b[j][k], so both operands are read along their
// rows.  A slab is the 128 bytes of a row that one step of the k loop consumes: 128 e4m3 codes (one 16x16x128 MFMA)
// or 64 halves (two 16x16x32 MFMAs).  In either type lane l of a wave feeds row l & 15 with the two 16-byte chunks
// g = l >> 4 and g + 4 of that row's slab.  Which k a chunk stands for does not matter as long as both operands agree.
//
// LDS layout: row r's slab lies at 128 r, its chunk c at position c ^ ((r >> 1) & 7).  LDS has 64 banks of 4 bytes, so
// two neighbouring rows fill them once; the 16 rows that 16 lanes read at one chunk index then touch every bank once.
// The permutation is applied to the global address (a wave's direct load writes LDS in lane order).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bcjr {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));

constexpr int kSlab = 128;    // bytes of a row per k step
constexpr int kXcds = 8;      // each with its own L2; workgroup i runs on XCD i mod 8

__device__ __forceinline__ uint32_t slab_chunk(int row, int pos) { return (uint32_t)(pos ^ ((row >> 1) & 7)); }

// 16 bytes per lane from global memory straight to LDS: lane l's land at lds + 16 l (lds is wave-uniform).
__device__ __forceinline__ void load_to_lds(const void* g, void* lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                     (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

// Every load this wave has issued is complete (those to LDS too, which a barrier alone does not wait for).
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// ROWS rows of one slab into LDS by NW waves; rows from `rows` on repeat the last one (their results are not stored).
template <int ROWS, int NW>
__device__ __forceinline__ void fetch_slab(const uint8_t* base, uint32_t ld, int rows, uint32_t kbyte, uint8_t* lds,
                                           int wave, int lane) {
    static_assert(ROWS % (8 * NW) == 0, "whole instructions for every wave");
#pragma unroll
    for (int i = 0; i < ROWS / (8 * NW); ++i) {
        const int part = i * NW + wave;
        const int row = part * 8 + (lane >> 3);
        const int r = row < rows ? row : rows - 1;
        load_to_lds(base + ((size_t)((uint32_t)r * (uint64_t)ld) + kbyte + slab_chunk(row, lane & 7) * 16),
                    lds + part * 1024);
    }
}

// The last slab of a row length that is no multiple of 128: `valid` bytes are there, the rest is written as zeros.
template <int ROWS, int NW>
__device__ __forceinline__ void fetch_tail(const uint8_t* base, uint32_t ld, int rows, uint32_t kbyte, int valid,
                                           uint8_t* lds, int wave, int lane) {
#pragma unroll 1
    for (int i = 0; i < ROWS / (8 * NW); ++i) {
        const int part = i * NW + wave;
        const int row = part * 8 + (lane >> 3);
        const int r = row < rows ? row : rows - 1;
        const int at = (int)slab_chunk(row, lane & 7) * 16;
        const uint8_t* p = base + ((size_t)((uint32_t)r * (uint64_t)ld) + kbyte + at);
        v4i v = {0, 0, 0, 0};
        if (at + 16 <= valid) {
            v = *(const v4i*)p;
        } else if (at < valid) {
            uint32_t w[4] = {0, 0, 0, 0};
            for (int b = 0; b < valid - at; ++b) w[b >> 2] |= (uint32_t)p[b] << ((b & 3) * 8);
            v = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
        }
        *(v4i*)(lds + part * 1024 + lane * 16) = v;
    }
}

// Chunks g and g + 4 of row `row`.
__device__ __forceinline__ v8i read_slab(const uint8_t* lds, int row, int g) {
    const uint32_t pos = slab_chunk(row, g) * 16;
    const v4i lo = *(const v4i*)(lds + row * kSlab + pos);
    const v4i hi = *(const v4i*)(lds + row * kSlab + (pos ^ 64));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Position of workgroup `id` of `count` in an order that gives each XCD one contiguous run of tiles, so that the
// workgroups that share an L2 share operand rows.
__device__ __forceinline__ int xcd_order(int id, int count) {
    const int per = count / kXcds, extra = count % kXcds;
    const int x = id % kXcds, i = id / kXcds;
    return x * per + (x < extra ? x : extra) + i;
}

// Tile (row, col) number t of a rows x cols grid, in bands of `band` tile rows walked column by column.
__device__ __forceinline__ void banded_tile(int t, int rows, int cols, int band, int& row, int& col) {
    const int b = t / (band * cols);
    const int first = b * band;
    const int height = min(band, rows - first);
    const int in = t - b * band * cols;
    row = first + in % height;
    col = in / height;
}

}  // namespace bcjr
