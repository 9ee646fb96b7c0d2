// Rows on their way into a cache: loads of eight input values as float, the
// amax of a CTA, and the codes of the 1-byte cache formats.
#pragma once

#include "device_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace dev {

// 8 consecutive input values as float, from f16 / bf16 / f32 storage.
template <int IN>
__device__ __forceinline__ void load8(const void* base, size_t idx, float (&x)[8]) {
  if constexpr (IN == PA_DTYPE_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + idx);
    const float4 a = p[0], b = p[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + idx);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (IN == PA_DTYPE_F16)
        f = unpack2<__half>(w[i]);
      else
        f = unpack2<__nv_bfloat16>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// Maximum of x over the CTA (at most 32 warps); `red`: 33 floats of shared
// memory, free for reuse after the next __syncthreads().
__device__ __forceinline__ float block_max(float x, float* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  if (l == 0) red[w] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    float y = threadIdx.x < (blockDim.x >> 5) ? red[threadIdx.x] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, off));
    if (threadIdx.x == 0) red[32] = y;
  }
  __syncthreads();
  return red[32];
}

// One code of a quantised cache from a float already divided by the scale:
// E4M3 round-to-nearest-even saturating to finite, or INT8 round-to-nearest-
// even (the scale makes |x| <= 127 up to its own rounding; clamped).
template <bool INT8>
__device__ __forceinline__ uint32_t encode_q8(float x) {
  if constexpr (INT8)
    return static_cast<uint32_t>(static_cast<uint8_t>(static_cast<int8_t>(max(-127, min(127, __float2int_rn(x))))));
  else
    return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

}  // namespace dev
}  // namespace pa
