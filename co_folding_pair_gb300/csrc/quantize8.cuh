// quantize8.cuh -- bf16 numbers to e4m3 codes with a power of two (linear8.h).
#pragma once

#include <cuda_fp8.h>

#include "pair_ops.cuh"

namespace trimul {

// The larger ones of two pairs of bf16 magnitudes; NaN where one is (the packed whole-number maximum takes several instructions).
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The scale's byte for a largest magnitude, its fp32 bits (finite): 0.875 2^(e + 9) is the last value that 2^e covers.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return static_cast<uint32_t>(e > 1 ? e : 1);
}
__device__ __forceinline__ float over_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) { return codes2(a, b) | codes2(c, d) << 16; }

// Magnitudes of two bf16 numbers, zero for those that are not finite.
__device__ __forceinline__ uint32_t finite16x2(uint32_t w) {
  const uint32_t a = w & 0x7fff7fffu;
  return ((a & 0xffffu) >= 0x7f80u ? 0u : a & 0xffffu) | (a >= 0x7f800000u ? 0u : a & 0xffff0000u);
}
// Infinity as NaN.
__device__ __forceinline__ float no_infinity(float v) { return fmaf(v, 0.f, v); }

// Two numbers, a register of bf16, as codes: times `inv`, one for each.
__device__ __forceinline__ uint32_t codes_of(uint32_t w, f2 inv, bool all_finite) {
  f2 v = unpack_bf162(w);
  if (!all_finite) v = fma2(v, both(0.f), v);  // infinity as NaN
  const float2 f = split2(mul2(v, inv));
  return codes2(f.x, f.y);
}
__device__ __forceinline__ uint2 codes_of(const uint4& v, const f2 (&inv)[4], bool all_finite) {
  return make_uint2(codes_of(v.x, inv[0], all_finite) | codes_of(v.y, inv[1], all_finite) << 16,
                    codes_of(v.z, inv[2], all_finite) | codes_of(v.w, inv[3], all_finite) << 16);
}
__device__ __forceinline__ uint2 codes_of(const uint4& v, float inv, bool all_finite) {
  const f2 i = both(inv);
  const f2 four[4] = {i, i, i, i};
  return codes_of(v, four, all_finite);
}

__device__ __forceinline__ uint32_t max_of(const uint4& v) { return max16x2(max16x2(v.x, v.y), max16x2(v.z, v.w)); }
// The largest magnitudes of two registers, of four and of eight; the signs are left to be taken off once, at the end.
__device__ __forceinline__ uint32_t max_signed(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_signed(const uint4& v) { return max_signed(max_signed(v.x, v.y), max_signed(v.z, v.w)); }
__device__ __forceinline__ uint32_t max_magnitude(const uint4& a, const uint4& b) { return max_signed(max_signed(a), max_signed(b)) & 0x7fff7fffu; }
__device__ __forceinline__ uint4 magnitudes(const uint4& v) {
  return make_uint4(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
}
__device__ __forceinline__ uint4 finite(const uint4& v) {
  return make_uint4(finite16x2(v.x), finite16x2(v.y), finite16x2(v.z), finite16x2(v.w));
}

// Adds a row's eight numbers to the sums of their columns.
__device__ __forceinline__ void add_row(f2 (&sums)[4], const uint4& v) {
  sums[0] = add2(sums[0], unpack_bf162(v.x)), sums[1] = add2(sums[1], unpack_bf162(v.y));
  sums[2] = add2(sums[2], unpack_bf162(v.z)), sums[3] = add2(sums[3], unpack_bf162(v.w));
}
// Their sums over the sixteen lanes that have the same columns (all of a lane's bits but 8), written by one of them.
__device__ __forceinline__ void join_columns(const f2 (&sums)[4], float* to, bool any) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 two = split2(sums[e]);
    v[2 * e] = two.x, v[2 * e + 1] = two.y;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], k < 3 ? 1 << k : 16);
  if (any && (threadIdx.x & 0x17) == 0) {
    reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// The larger half of what kLanes neighbouring lanes have.
template <int kLanes>
__device__ __forceinline__ uint32_t over_lanes(uint32_t m) {
  m = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

}  // namespace trimul
