// Shared helpers of the language-model operators (det_logprobs.cu,
// det_relbias.cu, det_attention.cu): the 16-bit types, and exponentials.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/det_model.h"
#include "det_common.cuh"

namespace det {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// 2^x by the hardware's approximation: exact at 0, relative error at most
// 2^-22, +0 for -inf.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// e^x, for a difference of scores x <= 0.
__device__ __forceinline__ float exp_approx(float x) { return exp2_approx(__fmul_rn(x, kLog2e)); }
// The larger of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A 32-bit key in the order of the values: -0 and +0 are equal, NaN is above
// +inf.
__device__ __forceinline__ unsigned order_key(float v) {
  if (isnan(v)) return 0xffffffffu;
  const unsigned b = __float_as_uint(v + 0.0f);   // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The value at p of one of the three types.
__device__ __forceinline__ float load_as_f32(const void* p, long long i, int dtype) {
  if (dtype == DET_F32) return static_cast<const float*>(p)[i];
  if (dtype == DET_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_from_f32(void* p, long long i, float v, int dtype) {
  if (dtype == DET_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == DET_BF16) static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
  else static_cast<__half*>(p)[i] = from_f32<__half>(v);
}

inline bool valid_model_dtype(int dtype) { return dtype == DET_F32 || dtype == DET_BF16 || dtype == DET_F16; }
inline int model_elem_size(int dtype) { return dtype == DET_F32 ? 4 : 2; }

}  // namespace det
