// pair_ops.cuh -- device helpers shared by the operators around the layer.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pair_ops.h"
#include "sm103_ptx.cuh"

namespace trimul {

// The two ends of an early launch (launch_early).
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Eight bf16 elements, 16 bytes, as fp32 and back.
__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = bf16_lo(w[e]);
    f[2 * e + 1] = bf16_hi(w[e]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf162(f[0], f[1]), pack_bf162(f[2], f[3]), pack_bf162(f[4], f[5]), pack_bf162(f[6], f[7]));
}
// Two fp32 numbers in a register pair: the packed instructions do both with one
// issue, which is what the row-wise kernels run short of.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 both(float v) { return pair2(v, v); }
__device__ __forceinline__ float2 split2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Eight numbers, as pairs.
struct F8 {
  f2 v[4];
};
__device__ __forceinline__ f2 unpack_bf162(uint32_t w) { return pair2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t pack_bf162(f2 v) {
  const float2 f = split2(v);
  return pack_bf162(f.x, f.y);
}
__device__ __forceinline__ float sum_of(const F8& a) {
  const float2 t = split2(add2(add2(a.v[0], a.v[1]), add2(a.v[2], a.v[3])));
  return t.x + t.y;
}
__device__ __forceinline__ float dot_of(const F8& a, const F8& b) {
  const float2 t = split2(fma2(a.v[3], b.v[3], fma2(a.v[2], b.v[2], fma2(a.v[1], b.v[1], mul2(a.v[0], b.v[0])))));
  return t.x + t.y;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// What the bucket of a pair is worked out from: loaded first, and looked at later.
struct RelposPair {
  int q, k, gq, gk;
  __device__ __forceinline__ void load(const RelposArgs& a, uint32_t qi, uint32_t kj) {
    q = a.q_pos[qi], k = a.k_pos[kj], gq = gk = 0;
    if (a.q_group) gq = a.q_group[qi], gk = a.k_group[kj];
  }
  __device__ __forceinline__ void none() { q = k = 0, gq = gk = -1; }
  // The table row; -1 for padding, and for none.
  __device__ __forceinline__ int bucket(const RelposArgs& a) const {
    const long long far = static_cast<long long>(q) - k;
    const int d = static_cast<int>(far < a.lo ? a.lo : far > a.M ? a.M : far) - a.lo;
    const int row = a.lut ? a.lut[d] : d;
    return (gq | gk) < 0 ? -1 : gq != gk ? a.rows - 1 : row;
  }
};

}  // namespace trimul
