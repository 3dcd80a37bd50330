// Loads and stores of fp32 and bf16 values, eight or one at a time.
#pragma once
#include "muon_b200.h"
#include "ptx.cuh"

namespace muon {

template <bool kBf16>
__device__ __forceinline__ void load8t(const void* base, long long i, float (&x)[8]) {
  if (kBf16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      x[2 * h] = bf16_lo_f(ww[h]);
      x[2 * h + 1] = bf16_hi_f(ww[h]);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = f[0], b = f[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

template <bool kBf16>
__device__ __forceinline__ void store8t(void* base, long long i, const float (&x)[8]) {
  if (kBf16) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    f[0] = make_float4(x[0], x[1], x[2], x[3]);
    f[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

template <bool kBf16>
__device__ __forceinline__ float load1t(const void* base, long long i) {
  return kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i])
               : static_cast<const float*>(base)[i];
}

template <bool kBf16>
__device__ __forceinline__ void store1t(void* base, long long i, float x) {
  if (kBf16)
    static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(x);
  else
    static_cast<float*>(base)[i] = x;
}

}  // namespace muon
