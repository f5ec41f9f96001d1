// decode_device.h -- device helpers of the decode-step operators: element
// types, their conversions, and the exact division by a host-known divisor.
#ifndef DETFOLD_DECODE_DEVICE_H
#define DETFOLD_DECODE_DEVICE_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "decode.h"

namespace detfold_impl {

typedef __bf16 bf16;
typedef _Float16 f16;
struct e4m3 {  // 8-bit float, 4 exponent and 3 mantissa bits, no infinity
    uint8_t bits;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(f16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(e4m3 x) { return __builtin_amdgcn_cvt_f32_fp8((int)x.bits, 0); }

template <typename T> __device__ __forceinline__ T from_f32(float x) { return (T)x; }  // nearest, ties to even
// Clamped first, since the conversion itself has no infinity to go to; a NaN stays one.
template <> __device__ __forceinline__ e4m3 from_f32<e4m3>(float x)
{
    x = x > kE4m3Max ? kE4m3Max : x < -kE4m3Max ? -kE4m3Max : x;
    return {(uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false)};
}

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ uint32_t divide(uint32_t x, const Divider &d)
{
    return (uint32_t)(((uint64_t)x * d.magic) >> d.shift);
}

// A value of lane l.
__device__ __forceinline__ int64_t from_lane(int64_t x, int l)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * l, (int)x), hi = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * l, (int)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

}  // namespace detfold_impl

#endif  // DETFOLD_DECODE_DEVICE_H
