// k10_adamw.cu -- one AdamW step over many tensors.
//
//   g = c grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p - lr wd p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// with c = min(1, max_norm / (norm + 1e-6)) where the gradients' norm is given:
// the factor is applied here, so that clipping needs no pass of its own.  A
// norm that is not finite makes the step nothing at all.
//
// One pass: every element of p, grad, m and v is read once and p, m, v and the
// copy are written once.  Bound by memory.  A thread has four neighbours, a
// warp 128: the 8-bit states' blocks, whose largest magnitudes two warp-wide
// reductions give.
//
// 8-bit states hold m and r = sqrt(v) as e4m3 with an fp32 scale for each
// block.  r and not v, because eight bits of e4m3 span 2^17 and a block's
// gradients, squared, would not fit.  At b2 = 0.999 a step changes r by less
// than a thousandth, and a code is an eighth: rounded to nearest, r would keep
// its code until |g| is some eleven times r.  Rounded at random, it moves as
// far as it should on average.
//
// A code is one of two neighbours, and an ulp in what is rounded can decide
// which.  So all that leads to a code is rounded operation by operation (the _rn
// intrinsics are not fused): the states are those of plain fp32 arithmetic, bit
// for bit.  What leads to the parameter alone may be approximate.
//
// The random bits are a hash of the seed, the step, the tensor's number and
// the element's, the PCG hash of Jarzynski and Olano, "Hash Functions for GPU
// Rendering" (2020): nothing is kept for them, and a step can be repeated.
#include <algorithm>
#include <cmath>

#include <cuda_fp8.h>

#include "pair_ops.cuh"
#include "step_ops.h"

namespace trimul {

namespace {

constexpr int kThreads = 256;
constexpr int kEach = 4;                    // neighbours of a thread
constexpr int kPart = kThreads * kEach;     // elements that a block takes at once
// What a kernel is for: states in 32 bits, or in 8 with one or two blocks of them a warp's turn, and the next turn's numbers on their
// way while one is worked on.
enum Form { F32_STATES, ONE_BLOCK, TWO_BLOCKS, TWO_AHEAD };
constexpr int parts(Form form) { return form == TWO_BLOCKS || form == TWO_AHEAD ? 2 : 1; }  // of a chunk, which is a thread block's turn
constexpr int blocks_per_sm(Form form) { return form == TWO_AHEAD ? 2 : 3; }                // what the registers allow
constexpr int kMostBlocks = 1024;
constexpr int kTableSmall = 64, kTableMax = 384;  // tensors of one launch
static_assert(32 * kEach == TRIMUL_STATE_BLOCK, "a warp has one block of the 8-bit states");

enum : uint8_t { PARAM_BF16 = 1, GRAD_SHIFT = 1, COPY_SHIFT = 3, WIDE = 32 };  // of Table::kind

constexpr int kF32 = TRIMUL_F32 << GRAD_SHIFT | WIDE, kF32Copy = kF32 | 1 << COPY_SHIFT;  // fp32 with fp32 gradients, and a bf16 copy
constexpr int kBf16 = PARAM_BF16 | TRIMUL_BF16 << GRAD_SHIFT | WIDE;

// The tensors of a launch, in its parameters.
template <int N>
struct Table {
  int n;
  uint32_t chunks;
  void* param[N];
  void* copy[N];
  const void* grad[N];
  void* m[N];
  void* v[N];
  float* m_scale[N];
  float* v_scale[N];
  long long numel[N];
  float decay[N];
  uint32_t index[N];                // the tensor's number in the call
  uint32_t chunk[N + 1];            // each tensor's first chunk, and the number of all
  uint16_t begin[kMostBlocks + 1];  // the tensor of each run's first chunk
  uint8_t kind[N];
};

struct Hyper {
  float b1, not_b1, b2, not_b2, log_b1, log_b2, eps, lr;
  const float* lr_device;
  const float* norm;
  float max_norm;
  uint32_t seed;
  int stochastic;
};
static_assert(sizeof(Table<kTableMax>) + sizeof(Hyper) + 64 <= 32764, "the table and the other arguments fit a launch's parameters");

struct Entry {
  void *param, *copy;
  const void* grad;
  void *m, *v;
  float *m_scale, *v_scale;
  long long numel;
  float decay;
  uint32_t chunk, index;
  int kind;
};

__device__ __forceinline__ uint32_t hash(uint32_t x) {
  x = x * 747796405u + 2891336453u;
  x = ((x >> ((x >> 28) + 4)) ^ x) * 277803737u;
  return (x >> 22) ^ x;
}

// ------------------------------------------------------------------ four neighbours
// Elements i .. i + 3 of a tensor of n as they lie there, 16 bytes or 8; `wide`: in one access, all of them there.  Nothing
// is made of them yet: the loads of all tensors are to be on their way together.
__device__ __forceinline__ uint4 load4(const void* p, int type, long long i, long long n, bool wide) {
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if (type == TRIMUL_F32) {
    const uint32_t* const q = static_cast<const uint32_t*>(p) + i;
    if (wide) return *reinterpret_cast<const uint4*>(q);
    if (i < n) r.x = q[0];
    if (i + 1 < n) r.y = q[1];
    if (i + 2 < n) r.z = q[2];
    if (i + 3 < n) r.w = q[3];
  } else {
    const uint16_t* const q = static_cast<const uint16_t*>(p) + i;
    if (wide) {
      const uint2 w = *reinterpret_cast<const uint2*>(q);
      r.x = w.x, r.y = w.y;
      return r;
    }
    if (i < n) r.x = q[0];
    if (i + 1 < n) r.x |= static_cast<uint32_t>(q[1]) << 16;
    if (i + 2 < n) r.y = q[2];
    if (i + 3 < n) r.y |= static_cast<uint32_t>(q[3]) << 16;
  }
  return r;
}
__device__ __forceinline__ void unpack4(const uint4& r, int type, float (&f)[4]) {
  if (type == TRIMUL_F32) {
    f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y), f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
  } else if (type == TRIMUL_BF16) {
    f[0] = bf16_lo(r.x), f[1] = bf16_hi(r.x), f[2] = bf16_lo(r.y), f[3] = bf16_hi(r.y);
  } else {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&r.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  }
}
__device__ __forceinline__ void store4(void* p, int type, long long i, long long n, bool wide, const float (&f)[4]) {
  if (wide) {
    if (type == TRIMUL_F32)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
          type == TRIMUL_BF16 ? make_uint2(pack_bf162(f[0], f[1]), pack_bf162(f[2], f[3]))
                              : make_uint2(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (i + e >= n) continue;
    if (type == TRIMUL_F32)
      static_cast<float*>(p)[i + e] = f[e];
    else if (type == TRIMUL_BF16)
      static_cast<__nv_bfloat16*>(p)[i + e] = __float2bfloat16_rn(f[e]);
    else
      static_cast<__half*>(p)[i + e] = __float2half_rn(f[e]);
  }
}
// The same for codes, four bytes.
__device__ __forceinline__ uint32_t load_codes(const void* p, long long i, long long n, bool whole) {
  if (whole) return *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p) + i);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) w |= static_cast<uint32_t>(static_cast<const uint8_t*>(p)[i + e]) << (8 * e);
  return w;
}
__device__ __forceinline__ void store_codes(void* p, long long i, long long n, bool whole, uint32_t w) {
  if (whole) {
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p) + i) = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) static_cast<uint8_t*>(p)[i + e] = static_cast<uint8_t>(w >> (8 * e));
}

// ------------------------------------------------------------------ roots and reciprocals
__device__ __forceinline__ float root_approx(float x) {  // within 2 ulp
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {  // of a normal number, within 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The root of x in [2^-60, inf), rounded to nearest: Newton's step from an approximation, with the remainder x - r^2
// exact in the fused product (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).  The
// tests compare a million of them, of all sizes, with the correctly rounded root.
__device__ __forceinline__ float root(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  const float r = x * y;
  return fmaf(fmaf(-r, r, x), 0.5f * y, r);
}
// 1 / x for x in [2^-100, 2^100], rounded to nearest: likewise.
__device__ __forceinline__ float reciprocal_rn(float x) {
  const float y = reciprocal(x);
  return fmaf(fmaf(-x, y, 1.f), y, y);
}
// ------------------------------------------------------------------ 8-bit states
__device__ __forceinline__ void unpack_codes(uint32_t w, float scale, float (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * e)), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * e] = __fmul_rn(v.x, scale), f[2 * e + 1] = __fmul_rn(v.y, scale);
  }
}
__device__ __forceinline__ uint32_t pack_codes(const float (&f)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

__device__ __forceinline__ float least_of(const float (&f)[4]) { return fminf(fminf(fabsf(f[0]), fabsf(f[1])), fminf(fabsf(f[2]), fabsf(f[3]))); }

__device__ __forceinline__ float larger(float a, float b) {  // NaN if one is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The largest magnitude of a warp's 128 numbers (a NaN's bits are above infinity's).
__device__ __forceinline__ float warp_largest(const float (&f)[4]) {
  const float top = larger(larger(fabsf(f[0]), fabsf(f[1])), larger(fabsf(f[2]), fabsf(f[3])));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
}

// x / scale as a number that e4m3 has: one of the two neighbours, the upper one
// with the probability of x's place between them (`bits`: 16, times 2^4).  From
// 2^-6 on the sum's carry out of what is cut off decides (past 448 the
// conversion saturates); below, where the codes are evenly spaced, they are as
// far apart as just above, so 2^-6 is added for the rounding.
__device__ __forceinline__ float at_random(float x, uint32_t bits) { return __uint_as_float((__float_as_uint(x) + bits) & 0xfff00000u); }
__device__ __forceinline__ float at_random_low(float x, uint32_t bits) {
  const float a = fabsf(x), base = a < 0x1p-6f ? 0x1p-6f : 0.f;
  return copysignf(at_random(a + base, bits) - base, x);
}

// A warp's blocks as codes with their scales; the first kParts are of m, the others of roots: none negative, the random bits from
// the hashes' upper halves, and what is above zero keeps a code above zero.  Few blocks have what takes longer (numbers below the evenly
// spaced codes, scales past the reciprocal's range), so it is asked once for all.  A lane that is not `inside` is not asked.
// A block with a number that is not finite gets such a scale, whatever its codes: they all stand for NaN.
template <int kParts>
__device__ __forceinline__ void quantize(const float (&f)[2 * kParts][4], const bool (&inside)[kParts], const uint32_t (&hashes)[kParts][4], bool stochastic,
                                         float (&scale)[2 * kParts], uint32_t (&codes)[2 * kParts]) {
  float inv[2 * kParts];
  bool normal = true, low = false;
#pragma unroll
  for (int k = 0; k < 2 * kParts; ++k) {
    scale[k] = __fmul_rn(larger(warp_largest(f[k]), 0x1p-90f), 1.f / 448.f);
    inv[k] = reciprocal_rn(scale[k]);
    normal = normal && scale[k] < 0x1p100f;
  }
  if (!normal) {
#pragma unroll
    for (int k = 0; k < 2 * kParts; ++k) inv[k] = __frcp_rn(scale[k]);
  }
#pragma unroll
  for (int k = 0; k < 2 * kParts; ++k) low = low || (inside[k % kParts] && !(__fmul_rn(least_of(f[k]), inv[k]) >= 0x1p-6f));
  low = __any_sync(0xffffffffu, low);
  auto bits = [&](int k, int e) {
    const uint32_t h = hashes[k % kParts][e];
    return k < kParts ? h << 4 & 0xffff0u : h >> 12 & 0xffff0u;
  };
  if (!low) {
#pragma unroll
    for (int k = 0; k < 2 * kParts; ++k) {
      float q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[e] = __fmul_rn(f[k][e], inv[k]);
        if (stochastic) q[e] = at_random(q[e], bits(k, e));
      }
      codes[k] = pack_codes(q);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2 * kParts; ++k) {
      float q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[e] = __fmul_rn(f[k][e], inv[k]);
        if (stochastic) q[e] = at_random_low(q[e], bits(k, e));
        if (k >= kParts && f[k][e] > 0.f) q[e] = fmaxf(q[e], 0x1p-9f);
      }
      codes[k] = pack_codes(q);
    }
  }
}

// ------------------------------------------------------------------ the step
template <int kParts>
__device__ __forceinline__ void roots(const float (&x)[kParts][4], float (&r)[2 * kParts][4]) {  // to r[kParts] ..
  bool usual = true;
#pragma unroll
  for (int u = 0; u < kParts; ++u) usual = usual && least_of(x[u]) >= 0x1p-60f && x[u][0] + x[u][1] + (x[u][2] + x[u][3]) < INFINITY;
  if (__all_sync(0xffffffffu, usual)) {
#pragma unroll
    for (int u = 0; u < kParts; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) r[kParts + u][e] = root(x[u][e]);
  } else {  // few blocks: the remainder would fall below fp32's range
#pragma unroll
    for (int u = 0; u < kParts; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) r[kParts + u][e] = __fsqrt_rn(x[u][e]);
  }
}

// What all elements of a step have in common.
struct Step {
  bool run;
  float clip, lr, rate, over_root_c2;  // rate: lr / (1 - b1^t)
  uint32_t key;
};
__device__ __forceinline__ Step step_of(const Hyper& h, int count) {
  Step s;
  s.run = true, s.clip = 1.f;
  if (h.norm) {
    const float norm = *h.norm, share = __fmul_rn(h.max_norm, __frcp_rn(__fadd_rn(norm, 1e-6f)));
    s.run = norm - norm == 0.f;
    s.clip = share < 1.f ? share : 1.f;
  }
  const float t = static_cast<float>(count + 1);
  s.lr = h.lr_device ? *h.lr_device : h.lr;
  // 1 - b^t without the cancellation of early steps
  s.rate = s.lr / -expm1f(t * h.log_b1);
  s.over_root_c2 = 1.f / sqrtf(-expm1f(t * h.log_b2));
  s.key = hash(static_cast<uint32_t>(count + 1) + hash(h.seed));
  return s;
}

template <int N>
__device__ __forceinline__ Entry entry(const Table<N>& tab, int k) {
  return Entry{tab.param[k],   tab.copy[k],  tab.grad[k],  tab.m[k],     tab.v[k],
               tab.m_scale[k], tab.v_scale[k], tab.numel[k], tab.decay[k], tab.chunk[k],
               tab.index[k],   tab.kind[k]};
}

// A thread's numbers of a chunk as they lie in memory; of 8-bit states m.x and v.x are codes, m.y and v.y scales.
struct Raw {
  uint4 p, g, m, v;
};
// The first of them: a warp has whole blocks, `parts` beside one another, so that at a tensor's end few warps have less to do.
template <Form kForm>
__device__ __forceinline__ long long place(const Entry& t, uint32_t chunk) {
  return static_cast<long long>(chunk - t.chunk) * (kPart * parts(kForm)) + threadIdx.x / 32 * (TRIMUL_STATE_BLOCK * parts(kForm)) + threadIdx.x % 32 * kEach;
}

// kKind: the tensor's kind, or -1 for one that is known only here.  sure: all four are the tensor's, and aligned.
template <bool k8, int kKind>
__device__ __forceinline__ void load_part(const Entry& t, long long i, bool sure, Raw& x) {
  const int kind = kKind < 0 ? t.kind : kKind;
  const bool whole = sure || i + 4 <= t.numel, wide = sure || (whole && kind & WIDE);
  x.p = load4(t.param, kind & PARAM_BF16 ? TRIMUL_BF16 : TRIMUL_F32, i, t.numel, wide);
  x.g = load4(t.grad, kind >> GRAD_SHIFT & 3, i, t.numel, wide);
  if (k8) {
    const long long block = i / TRIMUL_STATE_BLOCK;  // the same for a warp
    const bool any = sure || block * TRIMUL_STATE_BLOCK < t.numel;
    x.m.x = load_codes(t.m, i, t.numel, whole), x.v.x = load_codes(t.v, i, t.numel, whole);
    x.m.y = any ? __float_as_uint(t.m_scale[block]) : 0u, x.v.y = any ? __float_as_uint(t.v_scale[block]) : 0u;
  } else {
    x.m = load4(t.m, TRIMUL_F32, i, t.numel, whole), x.v = load4(t.v, TRIMUL_F32, i, t.numel, whole);
  }
}

// p after the step, from the new m and the root of the new v.
__device__ __forceinline__ float stepped(float p, float m, float r, float keep, const Hyper& h, const Step& s) {
  return fmaf(-(s.rate * m), reciprocal(fmaf(r, s.over_root_c2, h.eps)), p * keep);
}
__device__ __forceinline__ void moments(float g, float& m, float& v, const Hyper& h, const Step& s) {
  const float ge = __fmul_rn(g, s.clip);
  m = __fadd_rn(__fmul_rn(h.b1, m), __fmul_rn(h.not_b1, ge));
  v = __fadd_rn(__fmul_rn(h.b2, v), __fmul_rn(__fmul_rn(h.not_b2, ge), ge));
}
// The random bits of four neighbours, the first of them i.
__device__ __forceinline__ void random_bits(uint32_t tensor_key, long long i, uint32_t (&hashes)[4]) {
  const uint32_t key = hash(tensor_key + static_cast<uint32_t>(i >> 32)) ^ static_cast<uint32_t>(i);
#pragma unroll
  for (int e = 0; e < 4; ++e) hashes[e] = hash(key ^ e);  // (i is a multiple of four)
}
__device__ __forceinline__ void round_param(float (&p)[4], const uint32_t (&hashes)[4]) {  // to bf16
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (fabsf(p[e]) < INFINITY) p[e] = __uint_as_float((__float_as_uint(p[e]) + (hash(hashes[e]) & 0xffffu)) & 0xffff0000u);
}

template <int kKind>
__device__ __forceinline__ void step_f32(const Entry& t, long long i, const Raw& x, const Hyper& h, const Step& s) {
  const int kind = kKind < 0 ? t.kind : kKind;
  const int ptype = kind & PARAM_BF16 ? TRIMUL_BF16 : TRIMUL_F32, gtype = kind >> GRAD_SHIFT & 3, copy = kind >> COPY_SHIFT & 3;
  const bool whole = i + 4 <= t.numel, wide = whole && kind & WIDE;
  if (i >= t.numel) return;
  float p[4], g[4], m[4], v[4];
  unpack4(x.p, ptype, p), unpack4(x.g, gtype, g), unpack4(x.m, TRIMUL_F32, m), unpack4(x.v, TRIMUL_F32, v);
  const float keep = 1.f - s.lr * t.decay;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    moments(g[e], m[e], v[e], h, s);
    p[e] = stepped(p[e], m[e], root_approx(v[e]), keep, h, s);
  }
  if (copy) store4(t.copy, copy == 1 ? TRIMUL_BF16 : TRIMUL_F16, i, t.numel, wide, p);
  if (ptype == TRIMUL_BF16 && h.stochastic) {
    uint32_t hashes[4];
    random_bits(hash(t.index + s.key), i, hashes);
    round_param(p, hashes);
  }
  store4(t.param, ptype, i, t.numel, wide, p);
  store4(t.m, TRIMUL_F32, i, t.numel, whole, m);
  store4(t.v, TRIMUL_F32, i, t.numel, whole, v);
}

// What most programs have gets code without questions about types.
#define TRIMUL_BY_KIND(kind, f)      \
  do {                               \
    if ((kind) == kF32Copy)          \
      f(kF32Copy);                   \
    else if ((kind) == kF32)         \
      f(kF32);                       \
    else if ((kind) == kBf16)        \
      f(kBf16);                      \
    else                             \
      f(-1);                         \
  } while (0)

// fp32 states: a chunk is on its way while the one before is worked on (179 us for the 96 layers' tensors where
// loading two fours of a chunk together and then working on them takes 185).
template <int N>
__device__ __forceinline__ Step run_f32(const Table<N>& tab, const Hyper& h, const int* count, uint32_t c0, uint32_t c1) {
  int k = tab.begin[blockIdx.x];
  Entry t = entry(tab, k);
  uint32_t end = tab.chunk[k + 1];
  Raw x;
  auto load = [&](const Entry& t, uint32_t chunk) {
#define TRIMUL_LOAD(kKind) load_part<false, kKind>(t, place<F32_STATES>(t, chunk), false, x)
    TRIMUL_BY_KIND(t.kind, TRIMUL_LOAD);
#undef TRIMUL_LOAD
  };
  if (c0 < c1) load(t, c0);
  const Step s = step_of(h, *const_cast<const volatile int*>(count));  // behind the loads: it is made of what lies in memory as well
  for (uint32_t chunk = c0; chunk < c1 && s.run; ++chunk) {
    const Raw y = x;
    const bool other = chunk + 1 >= end;  // the next chunk is another tensor's
    if (chunk + 1 < c1) {
      if (other)
        load(entry(tab, k + 1), chunk + 1);
      else
        load(t, chunk + 1);
    }
#define TRIMUL_STEP(kKind) step_f32<kKind>(t, place<F32_STATES>(t, chunk), y, h, s)
    TRIMUL_BY_KIND(t.kind, TRIMUL_STEP);
#undef TRIMUL_STEP
    if (other && chunk + 1 < c1) {
      t = entry(tab, ++k);
      end = tab.chunk[k + 1];
    }
  }
  return s;
}

// 8-bit states: two fours of a thread are on their way together, and are worked on together.  The arithmetic is what takes the
// time, by its latency as much as by its instructions: one four after the other takes 185 us for the 96 layers' tensors, together 162, and
// with the next ones on their way (TWO_AHEAD) 150.
template <Form kForm>
struct Raws {
  Raw x[parts(kForm)];
};
template <Form kForm, int kKind>
__device__ __forceinline__ void load_8bit(const Entry& t, uint32_t chunk, Raws<kForm>& r) {
  constexpr int kParts = parts(kForm);
  const int kind = kKind < 0 ? t.kind : kKind;
  const long long i = place<kForm>(t, chunk);
  const bool all = i + (kParts - 1) * TRIMUL_STATE_BLOCK + 4 <= t.numel && kind & WIDE;
  if (all) {
#pragma unroll
    for (int u = 0; u < kParts; ++u) load_part<true, kKind>(t, i + u * TRIMUL_STATE_BLOCK, true, r.x[u]);
  } else {
#pragma unroll
    for (int u = 0; u < kParts; ++u) load_part<true, kKind>(t, i + u * TRIMUL_STATE_BLOCK, false, r.x[u]);
  }
}
template <Form kForm, int kKind>
__device__ __forceinline__ void step_8bit(const Entry& t, uint32_t chunk, const Raws<kForm>& raws, const Hyper& h, const Step& s) {
  const Raw (&x)[parts(kForm)] = raws.x;
  constexpr int kParts = parts(kForm);
  const int kind = kKind < 0 ? t.kind : kKind;
  const int ptype = kind & PARAM_BF16 ? TRIMUL_BF16 : TRIMUL_F32, gtype = kind >> GRAD_SHIFT & 3, copy = kind >> COPY_SHIFT & 3;
  const long long i = place<kForm>(t, chunk);
  const bool all = i + (kParts - 1) * TRIMUL_STATE_BLOCK + 4 <= t.numel && kind & WIDE;
  if (i / TRIMUL_STATE_BLOCK * TRIMUL_STATE_BLOCK >= t.numel) return;  // the same for a warp
  float p[kParts][4], v[kParts][4], f[2 * kParts][4];  // f: m, then roots
#pragma unroll
  for (int u = 0; u < kParts; ++u) {
    float g[4];
    unpack4(x[u].p, ptype, p[u]), unpack4(x[u].g, gtype, g);
    unpack_codes(x[u].m.x, __uint_as_float(x[u].m.y), f[u]), unpack_codes(x[u].v.x, __uint_as_float(x[u].v.y), v[u]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[u][e] = __fmul_rn(v[u][e], v[u][e]);
      moments(g[e], f[u][e], v[u][e], h, s);
    }
  }
  // lanes past the tensor's end have zeros, which would send their warp the longer ways: their v is one until the root is taken
  bool inside[kParts];
#pragma unroll
  for (int u = 0; u < kParts; ++u) inside[u] = all || i + u * TRIMUL_STATE_BLOCK < t.numel;
  if (!all) {
#pragma unroll
    for (int u = 0; u < kParts; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[u][e] = inside[u] ? v[u][e] : 1.f;
  }
  roots<kParts>(v, f);
  if (!all) {
#pragma unroll
    for (int u = 0; u < kParts; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) f[kParts + u][e] = inside[u] ? f[kParts + u][e] : 0.f;
  }
  const float keep = 1.f - s.lr * t.decay;
  const uint32_t tensor_key = hash(t.index + s.key);
  uint32_t hashes[kParts][4];
#pragma unroll
  for (int u = 0; u < kParts; ++u) {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[u][e] = stepped(p[u][e], f[u][e], f[kParts + u][e], keep, h, s);
    random_bits(tensor_key, i + u * TRIMUL_STATE_BLOCK, hashes[u]);
  }
  auto put_params = [&](bool sure) {
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
      const long long j = i + u * TRIMUL_STATE_BLOCK;
      const bool wide = sure || (j + 4 <= t.numel && kind & WIDE);
      if (copy) store4(t.copy, copy == 1 ? TRIMUL_BF16 : TRIMUL_F16, j, t.numel, wide, p[u]);
      if (ptype == TRIMUL_BF16 && h.stochastic) round_param(p[u], hashes[u]);
      store4(t.param, ptype, j, t.numel, wide, p[u]);
    }
  };
  if (all)
    put_params(true);
  else
    put_params(false);
  float scale[2 * kParts];
  uint32_t codes[2 * kParts];
  quantize<kParts>(f, inside, hashes, h.stochastic, scale, codes);
  auto put_states = [&](bool sure) {
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
      const long long j = i + u * TRIMUL_STATE_BLOCK, block = j / TRIMUL_STATE_BLOCK;
      const bool whole = sure || j + 4 <= t.numel;
      store_codes(t.m, j, t.numel, whole, codes[u]), store_codes(t.v, j, t.numel, whole, codes[kParts + u]);
      if (threadIdx.x % 32 == 0 && (sure || j < t.numel)) t.m_scale[block] = scale[u], t.v_scale[block] = scale[kParts + u];
    }
  };
  if (all)
    put_states(true);
  else
    put_states(false);
}
template <Form kForm, int N>
__device__ __forceinline__ Step run_8bit(const Table<N>& tab, const Hyper& h, const int* count, uint32_t c0, uint32_t c1) {
  Step s;
  if (c0 >= c1) return step_of(h, *const_cast<const volatile int*>(count));
  int k = tab.begin[blockIdx.x];
  Entry t = entry(tab, k);
  uint32_t end = tab.chunk[k + 1];
  Raws<kForm> x;
  if constexpr (kForm == TWO_AHEAD) {
    auto load = [&](const Entry& t, uint32_t chunk) {
#define TRIMUL_LOAD(kKind) load_8bit<kForm, kKind>(t, chunk, x)
      TRIMUL_BY_KIND(t.kind, TRIMUL_LOAD);
#undef TRIMUL_LOAD
    };
    load(t, c0);
    s = step_of(h, *const_cast<const volatile int*>(count));
    for (uint32_t chunk = c0; chunk < c1 && s.run; ++chunk) {
      const Raws<kForm> y = x;
      const bool other = chunk + 1 >= end;
      if (chunk + 1 < c1) {
        if (other)
          load(entry(tab, k + 1), chunk + 1);
        else
          load(t, chunk + 1);
      }
#define TRIMUL_STEP(kKind) step_8bit<kForm, kKind>(t, chunk, y, h, s)
      TRIMUL_BY_KIND(t.kind, TRIMUL_STEP);
#undef TRIMUL_STEP
      if (other && chunk + 1 < c1) {
        t = entry(tab, ++k);
        end = tab.chunk[k + 1];
      }
    }
  } else {
    bool known = false;
    for (uint32_t chunk = c0; chunk < c1; ++chunk) {
      if (chunk >= end) {
        t = entry(tab, ++k);
        end = tab.chunk[k + 1];
      }
#define TRIMUL_STEP(kKind)                                                                       \
  do {                                                                                           \
    load_8bit<kForm, kKind>(t, chunk, x);                                                        \
    if (!known) s = step_of(h, *const_cast<const volatile int*>(count)), known = true;           \
    if (s.run) step_8bit<kForm, kKind>(t, chunk, x, h, s);                                       \
  } while (0)
      TRIMUL_BY_KIND(t.kind, TRIMUL_STEP);
#undef TRIMUL_STEP
      if (!s.run) break;
    }
  }
  return s;
}
#undef TRIMUL_BY_KIND

__host__ __device__ __forceinline__ uint32_t run_begin(uint32_t chunks, uint32_t block, uint32_t blocks) {
  return static_cast<uint32_t>(static_cast<unsigned long long>(chunks) * block / blocks);
}

// count: {steps taken, blocks of the last launch that are done}.  Every block
// reads the steps before it says that it is done, and the last one of the last
// launch counts the step.  The launches of a step begin early, each in what room the
// one before leaves (their tensors are others), and wait for it before they end, so that what
// comes behind the last one comes behind all.
template <Form kForm, int N>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(kForm))
    k10_adamw(const __grid_constant__ Table<N> tab, const __grid_constant__ Hyper h, int* count, int last_launch) {
  let_next_begin();
  const uint32_t c0 = run_begin(tab.chunks, blockIdx.x, gridDim.x), c1 = run_begin(tab.chunks, blockIdx.x + 1, gridDim.x);
  Step s;
  if constexpr (kForm != F32_STATES)
    s = run_8bit<kForm>(tab, h, count, c0, c1);
  else
    s = run_f32(tab, h, count, c0, c1);
  after_previous();
  if (!last_launch) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    if (atomicAdd(count + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      count[1] = 0;
      if (s.run) count[0] += 1;
    }
  }
}

// ------------------------------------------------------------------ launches
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <Form kForm, int N>
int fill(Table<N>& tab, const trimul_adamw_tensor* t, const trimul_grad_tensor* g, int n, int& k, int blocks) {
  tab.n = 0;
  tab.chunks = 0;
  for (; k < n && tab.n < N; ++k) {
    if (t[k].numel == 0) continue;
    const int q = tab.n++;
    tab.param[q] = t[k].param;
    tab.copy[q] = t[k].copy;
    tab.grad[q] = g[k].data;
    tab.m[q] = t[k].m;
    tab.v[q] = t[k].v;
    tab.m_scale[q] = t[k].m_scale;
    tab.v_scale[q] = t[k].v_scale;
    tab.numel[q] = t[k].numel;
    tab.decay[q] = t[k].weight_decay;
    tab.index[q] = static_cast<uint32_t>(k);
    const int copy = !t[k].copy ? 0 : t[k].copy_type == TRIMUL_BF16 ? 1 : 2;
    const bool wide = aligned_to(t[k].param, t[k].param_type == TRIMUL_F32 ? 16 : 8) &&
                      aligned_to(g[k].data, g[k].type == TRIMUL_F32 ? 16 : 8) && (!copy || aligned_to(t[k].copy, 8));
    tab.kind[q] = static_cast<uint8_t>((t[k].param_type == TRIMUL_BF16 ? PARAM_BF16 : 0) | g[k].type << GRAD_SHIFT |
                                       copy << COPY_SHIFT | (wide ? WIDE : 0));
    tab.chunk[q] = tab.chunks;
    constexpr int kChunk = kPart * parts(kForm);
    tab.chunks += static_cast<uint32_t>((t[k].numel + kChunk - 1) / kChunk);
  }
  tab.chunk[tab.n] = tab.chunks;
  const int most = std::min(kMostBlocks, blocks);
  const int grid = static_cast<int>(std::max<long long>(1, std::min<long long>(tab.chunks, most)));
  int at = 0;
  for (int block = 0; block <= grid; ++block) {
    const uint32_t first = run_begin(tab.chunks, block, grid);
    while (at + 1 < tab.n && tab.chunk[at + 1] <= first) ++at;
    tab.begin[block] = static_cast<uint16_t>(at);
  }
  return grid;
}

template <Form kForm, int N>
cudaError_t run(const Hyper& h, const trimul_adamw_tensor* t, const trimul_grad_tensor* g, int n, int32_t* count, int num_sms, cudaStream_t s) {
  Table<N> tab;
  int k = 0;
  for (bool first = true; first || k < n; first = false) {
    const int grid = fill<kForm>(tab, t, g, n, k, blocks_per_sm(kForm) * num_sms);
    cudaError_t e = cudaSuccess;
    if (first) {  // behind all that was before the call
      k10_adamw<kForm, N><<<grid, kThreads, 0, s>>>(tab, h, count, k >= n);
      e = cudaGetLastError();
    } else {
      e = launch_early(k10_adamw<kForm, N>, dim3(grid), kThreads, s, tab, h, count, k >= n);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_adamw(const trimul_adamw_params& p, const trimul_adamw_tensor* t, const trimul_grad_tensor* g, int n, int32_t* count,
                         int num_sms, cudaStream_t s) {
  Hyper h{};
  h.b1 = static_cast<float>(p.beta1), h.not_b1 = static_cast<float>(1.0 - p.beta1);
  h.b2 = static_cast<float>(p.beta2), h.not_b2 = static_cast<float>(1.0 - p.beta2);
  h.log_b1 = static_cast<float>(std::log(p.beta1)), h.log_b2 = static_cast<float>(std::log(p.beta2));
  h.eps = p.eps, h.lr = p.lr, h.lr_device = p.lr_device;
  h.norm = p.norm, h.max_norm = p.max_norm;
  h.seed = p.seed, h.stochastic = p.rounding == TRIMUL_ROUND_STOCHASTIC;
  if (p.states != TRIMUL_STATES_E4M3)
    return n <= kTableSmall ? run<F32_STATES, kTableSmall>(h, t, g, n, count, num_sms, s) : run<F32_STATES, kTableMax>(h, t, g, n, count, num_sms, s);
  // us, 152 SMs:                                       one block   two   two, ahead
  //   a layer's 98k numbers                                 5.3     6.1
  //   460k (as many turns of one block as thread blocks)    5.1     5.1
  //   3.7M bf16 numbers in 240 tensors                     27      22.5    24.7
  //   37.8M in 960 tensors                                198     162     150
  long long turns = 0;
  for (int k = 0; k < n; ++k) turns += (t[k].numel + kPart - 1) / kPart;
  const bool small = n <= kTableSmall;
  if (turns > 32ll * num_sms)
    return small ? run<TWO_AHEAD, kTableSmall>(h, t, g, n, count, num_sms, s) : run<TWO_AHEAD, kTableMax>(h, t, g, n, count, num_sms, s);
  if (small && turns <= blocks_per_sm(ONE_BLOCK) * num_sms) return run<ONE_BLOCK, kTableSmall>(h, t, g, n, count, num_sms, s);
  return small ? run<TWO_BLOCKS, kTableSmall>(h, t, g, n, count, num_sms, s) : run<TWO_BLOCKS, kTableMax>(h, t, g, n, count, num_sms, s);
}

}  // namespace trimul
