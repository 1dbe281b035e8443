// Device helpers of the operators around the shard step: 16-bit formats,
// vectors at any element alignment, sums over a workgroup.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zsmr_ops.h"

namespace zsmr {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
// The same at the alignment of their elements: the hardware loads and stores
// 16 bytes at any address, so tensors that start anywhere take the same path.
typedef u16x8 u16x8_any __attribute__((aligned(2)));
typedef u16x4 u16x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <int DT>
__device__ __forceinline__ float widen16(uint16_t h) {
    if constexpr (DT == ZSMR_BF16) return __uint_as_float((uint32_t)h << 16);
    return static_cast<float>(__builtin_bit_cast(_Float16, h));
}
// round to nearest even (v_cvt_pk_bf16_f32 and v_cvt_f16_f32)
template <int DT>
__device__ __forceinline__ uint16_t narrow16(float x) {
    if constexpr (DT == ZSMR_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

// 16 bytes of any format as fp32 (kVec elements).  KEEP: through the caches,
// else past them.
template <int DT>
constexpr int kVec = DT == ZSMR_FP32 ? 4 : 8;
template <int DT>
struct Vec {
    float f[kVec<DT>];
};
template <int DT, bool KEEP>
__device__ __forceinline__ Vec<DT> load16(const void* p, int64_t e) {
    Vec<DT> v;
    if constexpr (DT == ZSMR_FP32) {
        const f32x4_any* q = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + e);
        const f32x4 x = KEEP ? *q : __builtin_nontemporal_load(q);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.f[i] = x[i];
    } else {
        const u16x8_any* q = reinterpret_cast<const u16x8_any*>(static_cast<const uint16_t*>(p) + e);
        const u16x8 x = KEEP ? *q : __builtin_nontemporal_load(q);
#pragma unroll
        for (int i = 0; i < 8; ++i) v.f[i] = widen16<DT>(x[i]);
    }
    return v;
}

// Eight elements of any format as fp32, and back.
template <int DT>
__device__ __forceinline__ f32x8 load8(const void* p, int64_t e) {
    f32x8 f;
    if constexpr (DT == ZSMR_FP32) {
        const f32x4 a = *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + e);
        const f32x4 b = *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + e + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    } else {
        const u16x8 h = *reinterpret_cast<const u16x8_any*>(static_cast<const uint16_t*>(p) + e);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = widen16<DT>(h[i]);
    }
    return f;
}
template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t e, f32x8 f) {
    if constexpr (DT == ZSMR_FP32) {
        f32x4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = f[i];
            b[i] = f[4 + i];
        }
        *reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + e) = a;
        *reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + e + 4) = b;
    } else {
        u16x8 h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = narrow16<DT>(f[i]);
        *reinterpret_cast<u16x8_any*>(static_cast<uint16_t*>(p) + e) = h;
    }
}
// store8 past the caches
template <int DT>
__device__ __forceinline__ void stream8(void* p, int64_t e, f32x8 f) {
    if constexpr (DT == ZSMR_FP32) {
        f32x4_any* q = reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + e);
        __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, q);
        __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]}, q + 1);
    } else {
        u16x8 h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = narrow16<DT>(f[i]);
        __builtin_nontemporal_store(h, reinterpret_cast<u16x8_any*>(static_cast<uint16_t*>(p) + e));
    }
}
template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t e) {
    if constexpr (DT == ZSMR_FP32) return static_cast<const float*>(p)[e];
    else return widen16<DT>(static_cast<const uint16_t*>(p)[e]);
}
template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t e, float f) {
    if constexpr (DT == ZSMR_FP32) static_cast<float*>(p)[e] = f;
    else static_cast<uint16_t*>(p)[e] = narrow16<DT>(f);
}

// Token ids of 4 or 8 bytes as an index below n, or -1 for padding.
__device__ __forceinline__ int32_t token_at(const void* ids, int id_bytes, int64_t t, int64_t n) {
    const int64_t id = id_bytes == 8 ? static_cast<const int64_t*>(ids)[t]
                                     : (int64_t) static_cast<const int32_t*>(ids)[t];
    return id >= 0 && id < n ? (int32_t)id : -1;
}

// Sum over a workgroup of THREADS in a fixed order; the result is valid in
// thread 0.
template <int THREADS>
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[THREADS / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < THREADS / 64; ++i) x += part[i];
    }
    return x;
}

}  // namespace zsmr
