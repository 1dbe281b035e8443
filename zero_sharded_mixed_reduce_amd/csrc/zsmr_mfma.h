// What the matrix products of this library share on the device: the matrix
// instruction, operands in memory, the transposing LDS read, waits and
// scheduling.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zsmr_dev.h"

namespace zsmr {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == ZSMR_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// A matrix in memory as an operand of a product: `rows` of `cols` elements,
// ld elements apart.
struct Mat {
    const uint16_t* p;
    int64_t ld, rows, cols;
};

// The transposing LDS read of four 16-bit elements.  __restrict__ tells the
// compiler that no load in flight writes what it reads (the waits of the main
// loops see to that); without it, it waits for all of them before each read.
template <typename = void>
__device__ __forceinline__ u32x2 read_transposed(const char* __restrict__ p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p)));
}

// The same for 16 bytes as they lie there.
template <typename = void>
__device__ __forceinline__ u32x4 read_lds16(const char* __restrict__ p) {
    return *reinterpret_cast<const u32x4*>(p);
}

// Spread a block's LDS reads and loads evenly among its matrix instructions.
template <int READS, int LOADS, int MFMA>
__device__ __forceinline__ void interleave() {
    constexpr int kOps = READS + LOADS, kEach = kOps < MFMA ? MFMA / kOps : 1;
    constexpr int kRounds = kOps < MFMA ? kOps : MFMA;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        if (i < LOADS) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);      // vector memory read
        else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                // LDS read
        __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);                 // matrix
    }
}

// vmcnt(n) and lgkmcnt(0)
#define ZSMR_WAIT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | 0x70 | ((n) >> 4 << 14))

}  // namespace zsmr
