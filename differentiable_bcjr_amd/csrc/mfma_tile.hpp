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

// 4 bytes per lane, the same way.
__device__ __forceinline__ void load4_to_lds(const void* g, void* lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                     (__attribute__((address_space(3))) void*)lds, 4, 0, 0);
}

// All but the last `kPending` loads this wave has issued are complete (loads to LDS too, which a barrier alone does not
// wait for; loads complete in order).
template <int kPending>
__device__ __forceinline__ void wait_loads() {
    static_assert(kPending >= 0 && kPending < 64, "a 6-bit count");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kPending) : "memory");
}

// The workgroup's waves meet; none of what comes after is moved ahead of it, nor what came before behind it.
__device__ __forceinline__ void meet() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The k loop: stage s of `total` is loaded into LDS slot s mod kStages, kStages - 1 stages ahead of its use.  `issue`
// issues kLoads loads in every wave and no others are in flight; `use` reads the slot.  One meeting a stage: behind it
// the stage is there for all waves (each has waited for its own loads), and the slot that is loaded next is no longer
// read (it was used in the step before).  Waves that have fewer stages of their own (`mine`) load along, so that every
// wave's loads can be counted alike, and do not use what they load: `issue` takes any stage below `total` and keeps
// within the operands by itself.
//
// The first kStages - 1 stages' loads go out in pipeline_ahead(); slot kStages - 1 is free until pipelined() begins.
template <int kStages, class Issue>
__device__ __forceinline__ void pipeline_ahead(int total, Issue issue) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s)
        if (s < total) issue(s, s);
}

template <int kStages, int kLoads, class Issue, class Use>
__device__ __forceinline__ void pipelined(int total, int mine, Issue issue, Use use) {
    int slot = 0;
#pragma unroll 1
    for (int s = 0; s < total; ++s) {
        if (s + kStages - 1 <= total)
            wait_loads<kLoads*(kStages - 2)>();
        else
            wait_loads<0>();
        meet();
        if (s + kStages - 1 < total) issue(s + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
        if (s < mine) use(slot);
        slot = slot + 1 == kStages ? 0 : slot + 1;
    }
}

// pipelined() with a stage before the first where `lead` says so: slot kStages - 1 as it was written in between, used by
// the waves with `mine_lead`.  (The loop starts one stage early; a second copy of `use` would cost the small products,
// which run most of their code once from a cold instruction cache.)
template <int kStages, int kLoads, class Issue, class Use>
__device__ __forceinline__ void pipelined_after(bool lead, bool mine_lead, int total, int mine, Issue issue, Use use) {
    int slot = lead ? kStages - 1 : 0;
#pragma unroll 1
    for (int s = lead ? -1 : 0; s < total; ++s) {
        if (s + kStages - 1 <= total)
            wait_loads<kLoads*(kStages - 2)>();
        else
            wait_loads<0>();
        meet();
        if (s >= 0 && s + kStages - 1 < total) issue(s + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
        if (s < 0 ? mine_lead : s < mine) use(slot);
        slot = slot + 1 == kStages ? 0 : slot + 1;
    }
}

// Adds up the sums of kGroups groups of waves that each took a share of the k loop, in their order; the first group's
// waves leave with the total.  `wave`: within the group; `at`: a part of LDS that is otherwise unused from here on.
template <int kGroups, int kWaves, int TM, int TN>
__device__ __forceinline__ void join_groups(v4f (&acc)[TM][TN], int group, int wave, int lane, uint8_t* at) {
    if constexpr (kGroups > 1) {
        if (group > 0) {
            v4f* to = (v4f*)at + ((group - 1) * kWaves + wave) * (TM * TN * 64) + lane;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) to[(i * TN + j) * 64] = acc[i][j];
        }
        meet();
        if (group > 0) return;
#pragma unroll
        for (int other = 1; other < kGroups; ++other) {
            const v4f* from = (const v4f*)at + ((other - 1) * kWaves + wave) * (TM * TN * 64) + lane;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] += from[(i * TN + j) * 64];
        }
    }
}

// ROWS rows of an operand, of which NW waves fetch one slab after the other: lane l of a wave's i-th instruction brings
// 16 bytes of row 8 (i NW + wave) + l / 8.  Rows from `rows` on repeat the last one (their results are not stored).  The
// lanes' offsets stay in registers; what changes from slab to slab is the uniform base.
template <int ROWS, int NW>
struct SlabSource {
    static_assert(ROWS % (8 * NW) == 0, "whole instructions for every wave");
    static constexpr int kLoads = ROWS / (8 * NW);
    const uint8_t* base;
    uint32_t offset[kLoads];

    __device__ __forceinline__ void set(const uint8_t* first_row, uint32_t ld, int rows, int wave, int lane) {
        base = first_row;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int row = (i * NW + wave) * 8 + (lane >> 3);
            offset[i] = (uint32_t)min(row, rows - 1) * ld + slab_chunk(row, lane & 7) * 16;
        }
    }

    __device__ __forceinline__ void fetch(uint32_t kbyte, uint8_t* lds, int wave) const {
        const uint8_t* from = base + kbyte;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            uint32_t at = offset[i];
            asm("" : "+v"(at));   // widened here and not ahead of the loop: a register, not two, and a scalar base
            load_to_lds(from + at, lds + (i * NW + wave) * 1024);
        }
    }
};

// Bytes at .. at + 15 of a row of `length` bytes that starts at `row`, zeros behind its end.  The row starts on a
// 16-byte boundary; nothing behind its end is read: where the end cuts the chunk, the row's last 16 bytes are, and moved
// into place.
__device__ __forceinline__ v4i load_chunk(const uint8_t* row, int at, int length) {
    typedef v4i v4i_byte __attribute__((aligned(1)));
    v4i v = {0, 0, 0, 0};
    if (at + 16 <= length) {
        v = *(const v4i*)(row + at);
    } else if (at < length) {
        if (length >= 16) {
            unsigned __int128 w = __builtin_bit_cast(unsigned __int128, (v4i)*(const v4i_byte*)(row + length - 16));
            v = __builtin_bit_cast(v4i, w >> ((at + 16 - length) * 8));
        } else {
            for (int b = 0; b < length; ++b) v[b >> 2] |= (int)row[b] << ((b & 3) * 8);   // at is 0
        }
    }
    return v;
}

// The slab behind the last whole one of rows of `length` bytes (kbyte: where it begins), through registers.
template <int ROWS, int NW>
struct TailSlab {
    static constexpr int kLoads = ROWS / (8 * NW);
    v4i v[kLoads];

    __device__ __forceinline__ void load(const uint8_t* base, uint32_t ld, int rows, int kbyte, int length, int wave,
                                         int lane) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int row = (i * NW + wave) * 8 + (lane >> 3);
            v[i] = load_chunk(base + (size_t)((uint32_t)min(row, rows - 1) * ld),
                              kbyte + (int)slab_chunk(row, lane & 7) * 16, length);
        }
    }
    __device__ __forceinline__ void put(uint8_t* lds, int wave, int lane) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) *(v4i*)(lds + (i * NW + wave) * 1024 + lane * 16) = v[i];
    }
};

// Chunks g and g + 4 of row `row`.
__device__ __forceinline__ v8i read_slab(const uint8_t* lds, int row, int g) {
    const uint32_t pos = slab_chunk(row, g) * 16;
    const v4i lo = *(const v4i*)(lds + row * kSlab + pos);
    const v4i hi = *(const v4i*)(lds + row * kSlab + (pos ^ 64));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// What this wave wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A wave's tile of ROWS x COLS results on their way to memory: each lane of an MFMA holds four neighbours of one row, so
// stored directly the 16 rows of an instruction get 32 bytes each.  They pass through LDS instead and leave as whole
// rows of the tile.  LDS holds 16-byte chunks, permuted within a row so that neither side's accesses collide: rows r and
// r + R share banks (R = 256 bytes / row), so the permutation changes every R rows.
template <class T, int ROWS, int COLS>
struct WaveTile {
    static constexpr int kRowBytes = COLS * (int)sizeof(T);
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kBytes = ROWS * kRowBytes;
    static constexpr int kPeriod = kRowBytes >= 256 ? 1 : 256 / kRowBytes;
    static constexpr int kPer = 16 / (int)sizeof(T);   // elements of a chunk
    static_assert((kChunks & (kChunks - 1)) == 0 && kChunks <= 64, "");

    static __device__ __forceinline__ uint32_t at(int row, int chunk) {
        return (uint32_t)(row * kRowBytes + (chunk ^ ((row / kPeriod) & (kChunks - 1))) * 16);
    }
    // v[0..3] at row `row`, columns col .. col + 3 (col a multiple of 4)
    static __device__ __forceinline__ void put(uint8_t* lds, int row, int col, const T (&v)[4]) {
        __builtin_memcpy(__builtin_assume_aligned(lds + at(row, col / kPer) + (col % kPer) * sizeof(T), 4 * sizeof(T)),
                         v, sizeof(v));
    }
    // element at (row, col)
    static __device__ __forceinline__ void put1(uint8_t* lds, int row, int col, T v) {
        *(T*)(lds + at(row, col / kPer) + (col % kPer) * sizeof(T)) = v;
    }
    // The tile's rows to out (its first element's place; ld elements a row), the first `rows` rows and `cols` columns of
    // it.  `wide`: out and ld are on 16-byte boundaries.
    static __device__ __forceinline__ void store(const uint8_t* lds, T* out, int64_t ld, int rows, int cols, bool wide,
                                                 int lane) {
        constexpr int kRowsPer = 64 / kChunks;   // rows of one instruction
#pragma unroll 4
        for (int i = 0; i < ROWS / kRowsPer; ++i) {
            const int row = i * kRowsPer + lane / kChunks, chunk = lane % kChunks;
            const v4i w = *(const v4i*)(lds + at(row, chunk));
            const int left = cols - chunk * kPer;
            if (row >= rows || left <= 0) continue;
            T* to = out + (int64_t)row * ld + chunk * kPer;
            if (wide && left >= kPer) {
                *(v4i*)to = w;
            } else {
                T e[kPer];
                __builtin_memcpy(e, &w, 16);
#pragma unroll
                for (int x = 0; x < kPer; ++x)
                    if (x < left) to[x] = e[x];
            }
        }
    }
};

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
