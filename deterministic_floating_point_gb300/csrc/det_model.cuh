// Shared helpers of the language-model operators (det_logprobs.cu,
// det_relbias.cu, det_attention.cu, det_embedding.cu, det_layernorm.cu,
// det_recurrence.cu): the 16-bit types, exponentials, and eights of elements.
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

// Two 32-bit lanes in a 64-bit register.
__device__ __forceinline__ unsigned long long pack_f32x2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

// Two values worked on by one packed instruction.
using Two = float2;
__device__ __forceinline__ Two two(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ Two twice(float a) { return make_float2(a, a); }
__device__ __forceinline__ Two add(Two a, Two b) { return __fadd2_rn(a, b); }
// Rounded by itself, whatever is done with it.
__device__ __forceinline__ Two mul(Two a, Two b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack_f32x2(a.x, a.y)), "l"(pack_f32x2(b.x, b.y)));
  return unpack_f32x2(r);
}
// For a factor or an addend of fma() and for a result: the compiler may join it and an add() that takes it into one
// instruction, in one variant of a kernel and not in another.  (mul() in its place took the norms' registers: the gradient of
// 1,048,576 x 64 in bf16 250 us against 234, 4,096 x 16,384 forward 53 against 52.)
__device__ __forceinline__ Two factor(Two a, Two b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ Two fma(Two a, Two b, Two c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ Two minus(Two a, Two b) { return __ffma2_rn(b, twice(-1.0f), a); }

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

// Eight consecutive elements as they lie in memory: one 16-byte vector in 16
// bits, two in 32.
template <typename T> struct Eight { uint4 q; };
template <> struct Eight<float> { uint4 q, r; };

// n of the eight elements at p (the others 0).  VEC: p is 16-byte aligned and n is
// 0 or 8 in 16 bits, 0, 4 or 8 in 32.
template <bool VEC, typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* p, int n) {
  Eight<T> e;
  e.q = make_uint4(0, 0, 0, 0);
  if constexpr (VEC) {
    if (n > 0) e.q = *reinterpret_cast<const uint4*>(p);
  } else {
    unsigned w[4] = {0, 0, 0, 0};
    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 1] |= (unsigned)h[i] << (16 * (i & 1));
    e.q = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return e;
}
template <bool VEC>
__device__ __forceinline__ Eight<float> load_eight(const float* p, int n) {
  Eight<float> e;
  e.q = e.r = make_uint4(0, 0, 0, 0);
  if constexpr (VEC) {
    if (n > 0) e.q = *reinterpret_cast<const uint4*>(p);
    if (n > 4) e.r = *reinterpret_cast<const uint4*>(p + 4);
  } else {
    unsigned w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? reinterpret_cast<const unsigned*>(p)[i] : 0u;
    e.q = make_uint4(w[0], w[1], w[2], w[3]);
    e.r = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return e;
}
__device__ __forceinline__ void unpack_eight(const Eight<float>& e, float (&v)[8]) {
  v[0] = __uint_as_float(e.q.x), v[1] = __uint_as_float(e.q.y), v[2] = __uint_as_float(e.q.z), v[3] = __uint_as_float(e.q.w);
  v[4] = __uint_as_float(e.r.x), v[5] = __uint_as_float(e.r.y), v[6] = __uint_as_float(e.r.z), v[7] = __uint_as_float(e.r.w);
}
__device__ __forceinline__ void unpack_two(unsigned w, float& a, float& b, __nv_bfloat16) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack_two(unsigned w, float& a, float& b, __half) {
  a = __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
  b = __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}
template <typename T>
__device__ __forceinline__ void unpack_eight(const Eight<T>& e, float (&v)[8]) {
  unpack_two(e.q.x, v[0], v[1], T());
  unpack_two(e.q.y, v[2], v[3], T());
  unpack_two(e.q.z, v[4], v[5], T());
  unpack_two(e.q.w, v[6], v[7], T());
}
// Two values rounded to 16 bits each, a in the lower half.
template <typename T> __device__ __forceinline__ unsigned pack_two(float a, float b);
template <> __device__ __forceinline__ unsigned pack_two<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const unsigned*>(&v);
}
template <> __device__ __forceinline__ unsigned pack_two<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const unsigned*>(&v);
}
template <typename T>
__device__ __forceinline__ void store_eight(T* p, const float (&v)[8], int n) {
  if (n > 0)
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_two<T>(v[0], v[1]), pack_two<T>(v[2], v[3]), pack_two<T>(v[4], v[5]), pack_two<T>(v[6], v[7]));
}
__device__ __forceinline__ void store_eight(float* p, const float (&v)[8], int n) {
  if (n > 0) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  if (n > 4) *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

inline bool valid_model_dtype(int dtype) { return dtype == DET_F32 || dtype == DET_BF16 || dtype == DET_F16; }
inline int model_elem_size(int dtype) { return dtype == DET_F32 ? 4 : 2; }

}  // namespace det
