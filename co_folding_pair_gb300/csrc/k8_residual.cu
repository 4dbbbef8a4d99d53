// k8_residual.cu -- the residual step, forward and backward.
//
//   y = Norm_post(u),  w = scale mask channel G(gate),  X = x + w y,  n = Norm_pre(X)
//
// Forward writes X and n.  Backward takes dX' = dout (+ dout2) and dn, computes
// y, X and both norms' statistics again from x and u (so nothing is kept from
// the forward, and X before its rounding is what the gradient is taken of), and
//
//   dX = dX' + Norm_pre'(dn),    dx = dX,   dy = w dX,   du = Norm_post'(dy),
//   dgate = scale mask channel y dX G'(gate),   dchannel = sum scale mask G y dX,
//   dgamma = sum (norm's gradient) (normalised value),   dbeta = sum (norm's gradient)
//
// with, for v^ = (v - mean) r normalised and t = dv' gamma,
//   Norm'(dv') = r (t - mean(t) - v^ mean(t v^))     (RMS: without the means of v and t).
//
// Each is one pass over the rows: 8 (forward) to 14 (backward) bytes an element
// in bf16 against some 20 to 60 operations, so both are bound by memory.
// Rounding: each output is rounded once, from fp32.
#include <algorithm>

#include "pair_ops.cuh"

namespace trimul {

namespace {

constexpr int kThreads = 256;

// Sum over the G lanes that share a row.
template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// v -> its normalised value; returns r.  Lanes past D hold and keep zeros.
// The mean is a true division: a row of one value has that value as its mean
// exactly, and the product with 1 / D, off by half an ulp of the mean, would be
// scaled by 1 / sqrt(eps) there.
template <int G>
__device__ __forceinline__ float normalise(F8& v, int kind, float d, float inv_d, float eps, bool live) {
  if (kind == TRIMUL_NORM_LAYER) {
    const float mean = row_sum<G>(sum_of(v)) / d;
    const f2 shift = both(live ? -mean : 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) v.v[e] = add2(v.v[e], shift);
  }
  const float r = rsqrtf(row_sum<G>(dot_of(v, v)) * inv_d + eps);
#pragma unroll
  for (int e = 0; e < 4; ++e) v.v[e] = mul2(v.v[e], both(r));
  return r;
}

// t (the gradient at the normalised value) -> the gradient at the norm's input.
template <int G>
__device__ __forceinline__ void normalise_grad(F8& t, const F8& hat, float r, int kind, float inv_d) {
  const float m2 = row_sum<G>(dot_of(t, hat)) * (-r * inv_d);
  const float m1 = kind == TRIMUL_NORM_LAYER ? row_sum<G>(sum_of(t)) * (-r * inv_d) : 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) t.v[e] = fma2(t.v[e], both(r), fma2(hat.v[e], both(m2), both(m1)));
}

// Eight of a parameter's values, or the value it has where it is absent.
__device__ __forceinline__ void param8(const float* p, int c, bool live, float absent, F8& f) {
  if (p && live) {
    const float4 a = reinterpret_cast<const float4*>(p + c)[0], b = reinterpret_cast<const float4*>(p + c)[1];
    f.v[0] = pair2(a.x, a.y), f.v[1] = pair2(a.z, a.w), f.v[2] = pair2(b.x, b.y), f.v[3] = pair2(b.z, b.w);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = both(absent);
  }
}

// The rows of the next turns are on their way while one is worked on: every
// thread copies its own 16 bytes of each tensor into a ring of its own in
// shared memory and reads them back itself, so the ring needs no barrier, only
// the thread's wait for its oldest copies.  Depth, not registers, sets the
// bytes in flight.
constexpr int kDepth = 4;

__device__ __forceinline__ void copy16(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // until at most N groups are on their way
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's eight elements of T at ring slots [k], [k + 1] (fp32 only), kThreads apart.
__device__ __forceinline__ void copy8(uint4* to, const __nv_bfloat16* from) { copy16(to, from); }
__device__ __forceinline__ void copy8(uint4* to, const float* from) {
  copy16(to, from);
  copy16(to + kThreads, from + 4);
}
__device__ __forceinline__ F8 widen8(const uint4 v) {
  return F8{{unpack_bf162(v.x), unpack_bf162(v.y), unpack_bf162(v.z), unpack_bf162(v.w)}};
}
__device__ __forceinline__ F8 take8(const uint4* from, bool on, __nv_bfloat16) {
  return widen8(on ? from[0] : make_uint4(0u, 0u, 0u, 0u));
}
__device__ __forceinline__ F8 take8(const uint4* from, bool on, float) {
  const ulonglong2 z = make_ulonglong2(0, 0);
  const ulonglong2 a = on ? reinterpret_cast<const ulonglong2*>(from)[0] : z;
  const ulonglong2 b = on ? reinterpret_cast<const ulonglong2*>(from)[kThreads] : z;
  return F8{{a.x, a.y, b.x, b.y}};
}
// Streaming stores: what is written is not read again here.
__device__ __forceinline__ void put8(__nv_bfloat16* p, const F8& f) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(pack_bf162(f.v[0]), pack_bf162(f.v[1]), pack_bf162(f.v[2]), pack_bf162(f.v[3])));
}
__device__ __forceinline__ void put8(float* p, const F8& f) {
  const float2 a = split2(f.v[0]), b = split2(f.v[1]), c = split2(f.v[2]), d = split2(f.v[3]);
  __stcs(reinterpret_cast<float4*>(p), make_float4(a.x, a.y, b.x, b.y));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(c.x, c.y, d.x, d.y));
}

// 1 / x for x in [1, 2], to 1 ulp (the approximate instruction).
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// sigmoid(x) and 1 - sigmoid(x), each to fp32's relative precision (the
// exponential's argument is never positive, so nothing overflows either).
__device__ __forceinline__ float2 sigmoid2(float x) {
  const float e = __expf(-fabsf(x)), big = reciprocal(1.0f + e), small = e * big;
  return x >= 0.f ? make_float2(big, small) : make_float2(small, big);
}
// The gate's values, in place; returns their derivatives.
__device__ __forceinline__ F8 sigmoid8(F8& g) {
  F8 d;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = split2(g.v[e]), a = sigmoid2(x.x), b = sigmoid2(x.y);
    g.v[e] = pair2(a.x, b.x);
    d.v[e] = pair2(a.x * a.y, b.x * b.y);
  }
  return d;
}

// The gate's eight values of a row (pair), as they are.
__device__ __forceinline__ const uint16_t* gate_row(const ResidualArgs& a, uint32_t pair) {
  if (a.p.gate == TRIMUL_GATE_PAIR) return a.gate + static_cast<size_t>(pair) * a.p.D;
  uint32_t row, j;
  a.by_J.divmod(pair, row, j);
  const size_t at = a.p.gate == TRIMUL_GATE_COL ? row : static_cast<size_t>(a.by_I.div(row)) * a.J + j;
  return a.gate + at * a.p.D;
}

using bf = __nv_bfloat16;

__device__ __forceinline__ float mask_of(const ResidualArgs& a, uint32_t pair) {
  return a.mask ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.mask)[pair]) : 1.f;
}

template <typename T>
constexpr int kSlots = sizeof(T) / 2;  // ring slots of eight elements

// Ring slots of a stage.
template <typename T>
__host__ __device__ constexpr int forward_slots(bool gate) {
  return kSlots<T> + 1 + (gate ? 1 : 0);
}
template <typename T>
__host__ __device__ constexpr int backward_slots(bool gate, bool second, bool pre) {
  return kSlots<T> * (second ? 3 : 2) + 1 + (gate ? 1 : 0) + (pre ? 1 : 0);
}

// G lanes share a row, eight channels each.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads, 3) k8_residual_fwd(ResidualArgs a, uint32_t rows) {
  extern __shared__ uint4 ring[];
  constexpr uint32_t kRows = kThreads / G;
  const int c = (threadIdx.x % G) * 8;
  const bool live = c < a.p.D;
  const float d_f = static_cast<float>(a.p.D), inv_d = 1.0f / d_f;
  // scale channel (gamma y^ + beta) = A y^ + B
  F8 A, B, ng, nb;
  {
    F8 ch;
    param8(a.p.post_gamma, c, live, 1.f, A);
    param8(a.p.post_beta, c, live, 0.f, B);
    param8(a.p.channel, c, live, 1.f, ch);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ch.v[e] = mul2(ch.v[e], both(a.p.scale));
      A.v[e] = mul2(A.v[e], ch.v[e]);
      B.v[e] = mul2(B.v[e], ch.v[e]);
    }
  }
  param8(a.p.pre_gamma, c, live, 1.f, ng);
  param8(a.p.pre_beta, c, live, 0.f, nb);
  const int slots = forward_slots<T>(a.gate);
  const uint32_t step = gridDim.x * kRows, mine = blockIdx.x * kRows + threadIdx.x / G;
  uint4* const own = ring + threadIdx.x;
  // row `row` into stage `stage`; rows past the end close an empty group
  auto fetch = [&](unsigned long long row, int stage) {
    if (live && row < rows) {
      const size_t at = static_cast<size_t>(row) * a.p.D + c;
      uint4* const to = own + stage * slots * kThreads;
      copy8(to, static_cast<const T*>(a.x) + at);
      copy16(to + kSlots<T> * kThreads, a.u + at);
      if (a.gate) copy16(to + (kSlots<T> + 1) * kThreads, gate_row(a, static_cast<uint32_t>(row)) + c);
    }
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) fetch(mine + static_cast<unsigned long long>(k) * step, k);
  int stage = 0;
  float m_next = (a.mask && mine < rows) ? mask_of(a, mine) : 1.f;
  // every lane of a warp takes the same number of turns, for the shuffles
  for (unsigned long long base = blockIdx.x * kRows; base < rows; base += step) {
    const unsigned long long row = base + threadIdx.x / G;
    const bool on = live && row < rows;
    const size_t at = static_cast<size_t>(row) * a.p.D + c;
    const float m = m_next;
    if (a.mask && row + step < rows) m_next = mask_of(a, static_cast<uint32_t>(row + step));
    fetch(row + (kDepth - 1ull) * step, (stage + kDepth - 1) % kDepth);
    copies_wait<kDepth - 1>();
    const uint4* const from = own + stage * slots * kThreads;
    stage = (stage + 1) % kDepth;
    F8 x = take8(from, on, T()), y = take8(from + kSlots<T> * kThreads, on, bf());
    if (a.p.post_norm != TRIMUL_NORM_NONE) normalise<G>(y, a.p.post_norm, d_f, inv_d, a.p.eps, live);
#pragma unroll
    for (int e = 0; e < 4; ++e) y.v[e] = fma2(y.v[e], A.v[e], B.v[e]);
    if (a.gate) {
      F8 g = take8(from + (kSlots<T> + 1) * kThreads, on, bf());
      if (a.p.gate_sigmoid) sigmoid8(g);
#pragma unroll
      for (int e = 0; e < 4; ++e) y.v[e] = mul2(y.v[e], g.v[e]);
    }
    if (m != 0.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x.v[e] = fma2(y.v[e], both(m), x.v[e]);
    }
    if (on) put8(static_cast<T*>(a.out) + at, x);
    if (a.normed) {
      normalise<G>(x, a.p.pre_norm, d_f, inv_d, a.p.eps, live);
      if (m != 0.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x.v[e] = fma2(x.v[e], ng.v[e], nb.v[e]);
      } else {
        x = F8{};
      }
      if (on) put8(reinterpret_cast<bf*>(a.normed) + at, x);
    }
  }
}

// Depth of the backward's ring: it has up to six tensors to read.
constexpr int kBackDepth = 2;

template <typename T, int G>
__global__ void __launch_bounds__(kThreads, 2) k8_residual_bwd(ResidualArgs a, uint32_t rows) {
  extern __shared__ uint4 ring[];
  // post_gamma, post_beta, pre_gamma, channel: the low and the high four of each lane's eight
  __shared__ float4 par4[4][2][32];
  constexpr uint32_t kRows = kThreads / G;
  const int c = (threadIdx.x % G) * 8;
  const bool live = c < a.p.D;
  const float d_f = static_cast<float>(a.p.D), inv_d = 1.0f / d_f;
  const bool post = a.p.post_norm != TRIMUL_NORM_NONE, pre = a.p.pre_norm != TRIMUL_NORM_NONE;
  {
    const float* const from[4] = {a.p.post_gamma, a.p.post_beta, a.p.pre_gamma, a.p.channel};
    for (int n = threadIdx.x; n < 4 * 256; n += kThreads) {
      const int q = n / 256, e = n % 256;
      reinterpret_cast<float*>(&par4[q][e / 4 % 2][e / 8])[e % 4] = e < a.p.D && from[q] ? from[q][e] : q == 1 ? 0.f : 1.f;
    }
    __syncthreads();
  }
  auto par = [&](int q) {
    const ulonglong2 lo = reinterpret_cast<const ulonglong2&>(par4[q][0][c / 8]);
    const ulonglong2 hi = reinterpret_cast<const ulonglong2&>(par4[q][1][c / 8]);
    return F8{{lo.x, lo.y, hi.x, hi.y}};
  };
  const int slots = backward_slots<T>(a.gate, a.dout2, pre);
  const int at_u = kSlots<T> * (a.dout2 ? 3 : 2), at_g = at_u + 1, at_n = at_g + (a.gate ? 1 : 0);
  const uint32_t step = gridDim.x * kRows, mine = blockIdx.x * kRows + threadIdx.x / G;
  uint4* const own = ring + threadIdx.x;
  auto fetch = [&](unsigned long long row, int stage) {
    if (live && row < rows) {
      const size_t at = static_cast<size_t>(row) * a.p.D + c;
      uint4* const to = own + stage * slots * kThreads;
      copy8(to, static_cast<const T*>(a.dout) + at);
      if (pre) copy8(to + kSlots<T> * kThreads, static_cast<const T*>(a.x) + at);  // only X's statistics need x
      if (a.dout2) copy8(to + 2 * kSlots<T> * kThreads, static_cast<const T*>(a.dout2) + at);
      copy16(to + at_u * kThreads, a.u + at);
      if (a.gate) copy16(to + at_g * kThreads, gate_row(a, static_cast<uint32_t>(row)) + c);
      if (pre) copy16(to + at_n * kThreads, a.dnormed + at);
    }
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < kBackDepth - 1; ++k) fetch(mine + static_cast<unsigned long long>(k) * step, k);
  F8 sums[RESIDUAL_SUMS] = {};
  int stage = 0;
  float m_next = mine < rows ? mask_of(a, mine) : 0.f;
  for (unsigned long long base = blockIdx.x * kRows; base < rows; base += step) {
    const unsigned long long row = base + threadIdx.x / G;
    const bool on = live && row < rows;
    const size_t at = static_cast<size_t>(row) * a.p.D + c;
    const float m = on ? m_next : 0.f;
    if (row + step < rows) m_next = mask_of(a, static_cast<uint32_t>(row + step));
    fetch(row + (kBackDepth - 1ull) * step, (stage + kBackDepth - 1) % kBackDepth);
    copies_wait<kBackDepth - 1>();
    const uint4* const from = own + stage * slots * kThreads;
    stage = (stage + 1) % kBackDepth;
    const bool real = on && m != 0.f;  // padding: zeros, whatever the tensors hold
    F8 d = take8(from, on, T());
    if (a.dout2) {
      const F8 t = take8(from + 2 * kSlots<T> * kThreads, on, T());
#pragma unroll
      for (int e = 0; e < 4; ++e) d.v[e] = add2(d.v[e], t.v[e]);
    }
    F8 yh = take8(from + at_u * kThreads, real, bf());
    float pr = 0.f;
    if (post) pr = normalise<G>(yh, a.p.post_norm, d_f, inv_d, a.p.eps, live);
    F8 gv, gd;  // scale mask times the gate's value, and times its derivative
    const f2 k = both(a.p.scale * m);
    if (a.gate) {
      gv = take8(from + at_g * kThreads, real, bf());
      if (a.p.gate_sigmoid) {
        gd = sigmoid8(gv);
#pragma unroll
        for (int e = 0; e < 4; ++e) gd.v[e] = mul2(gd.v[e], k);
      } else {
        gd = F8{{k, k, k, k}};
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) gv.v[e] = mul2(gv.v[e], k);
    } else {
      gv = F8{{k, k, k, k}};
    }
    if (pre) {
      F8 x = take8(from + kSlots<T> * kThreads, real, T());
      const F8 pg = par(0), pb = par(1), ch = par(3), ng = par(2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 y = post ? fma2(yh.v[e], pg.v[e], pb.v[e]) : yh.v[e];
        x.v[e] = fma2(mul2(gv.v[e], ch.v[e]), y, x.v[e]);
      }
      const float nr = normalise<G>(x, a.p.pre_norm, d_f, inv_d, a.p.eps, live);
      F8 dn = take8(from + at_n * kThreads, real, bf());
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sums[2].v[e] = fma2(dn.v[e], x.v[e], sums[2].v[e]);
        sums[3].v[e] = add2(dn.v[e], sums[3].v[e]);
        dn.v[e] = mul2(dn.v[e], ng.v[e]);
      }
      normalise_grad<G>(dn, x, nr, a.p.pre_norm, inv_d);
#pragma unroll
      for (int e = 0; e < 4; ++e) d.v[e] = add2(d.v[e], dn.v[e]);
    }
    if (on) put8(static_cast<T*>(a.dx) + at, d);
    if (!real) d = F8{};  // a padding pair passes nothing on to what follows
    const F8 pg = par(0), ch = par(3);
    if (a.dgate || a.g.channel) {
      const F8 pb = par(1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 y = post ? fma2(yh.v[e], pg.v[e], pb.v[e]) : yh.v[e];
        const f2 dy = mul2(d.v[e], y);
        sums[4].v[e] = fma2(dy, gv.v[e], sums[4].v[e]);
        if (a.dgate) gd.v[e] = mul2(gd.v[e], mul2(dy, ch.v[e]));
      }
      if (on && a.dgate) put8(reinterpret_cast<bf*>(a.dgate) + at, gd);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) d.v[e] = mul2(d.v[e], mul2(gv.v[e], ch.v[e]));
    if (post) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sums[0].v[e] = fma2(d.v[e], yh.v[e], sums[0].v[e]);
        sums[1].v[e] = add2(d.v[e], sums[1].v[e]);
        d.v[e] = mul2(d.v[e], pg.v[e]);
      }
      normalise_grad<G>(d, yh, pr, a.p.post_norm, inv_d);
    }
    if (on) put8(reinterpret_cast<bf*>(a.du) + at, d);
  }
  // the block's column sums, its rows added in order
  __shared__ float s[kRows][G * 8 + 1];
#pragma unroll
  for (int q = 0; q < RESIDUAL_SUMS; ++q) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = split2(sums[q].v[e]);
      s[threadIdx.x / G][c + 2 * e] = t.x, s[threadIdx.x / G][c + 2 * e + 1] = t.y;
    }
    __syncthreads();
    for (int n = threadIdx.x; n < a.p.D; n += kThreads) {
      float t = 0.f;
      for (int r = 0; r < static_cast<int>(kRows); ++r) t += s[r][n];
      a.part[(static_cast<size_t>(blockIdx.x) * RESIDUAL_SUMS + q) * a.p.D + n] = t;
    }
  }
}

// The blocks' column sums: 32 columns a block, eight groups of parts side by side.
__global__ void __launch_bounds__(256)
    k8_residual_sum(const float* __restrict__ part, trimul_residual_grads g, int D, int blocks) {
  __shared__ float s[8][32];
  const int n = blockIdx.x * 32 + threadIdx.x % 32, k0 = threadIdx.x / 32;
  float t = 0.f;
  if (n < RESIDUAL_SUMS * D) {
#pragma unroll 8
    for (int k = k0; k < blocks; k += 8) t += part[static_cast<size_t>(k) * RESIDUAL_SUMS * D + n];
  }
  s[k0][threadIdx.x % 32] = t;
  __syncthreads();
  float* const out[RESIDUAL_SUMS] = {g.post_gamma, g.post_beta, g.pre_gamma, g.pre_beta, g.channel};
  if (k0 != 0 || n >= RESIDUAL_SUMS * D || !out[n / D]) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) t += s[k][threadIdx.x];
  out[n / D][n % D] = t;
}

int lanes_of(int D) {
  int g = 1;
  while (g * 8 < D) g *= 2;
  return g;
}

int blocks_for(int D, long long rows, int num_sms, int per_sm) {
  const int per_block = kThreads / lanes_of(D);
  return static_cast<int>(std::min<long long>((rows + per_block - 1) / per_block, static_cast<long long>(per_sm) * num_sms));
}

template <typename K>
cudaError_t launch(K kernel, const ResidualArgs& a, uint32_t rows, int grid, int smem, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, smem, s>>>(a, rows);
  return cudaGetLastError();
}
template <typename T, int G>
cudaError_t forward(const ResidualArgs& a, uint32_t rows, int num_sms, cudaStream_t s) {
  return launch(k8_residual_fwd<T, G>, a, rows, blocks_for(a.p.D, rows, num_sms, 3),
                kDepth * forward_slots<T>(a.gate) * kThreads * 16, s);
}
template <typename T, int G>
cudaError_t backward(const ResidualArgs& a, uint32_t rows, int num_sms, cudaStream_t s) {
  return launch(k8_residual_bwd<T, G>, a, rows, blocks_for(a.p.D, rows, num_sms, 2),
                kBackDepth * backward_slots<T>(a.gate, a.dout2, a.p.pre_norm != TRIMUL_NORM_NONE) * kThreads * 16, s);
}

#define BY_LANES(FN, T)                                                  \
  switch (lanes_of(a.p.D)) {                                             \
    case 1: e = FN<T, 1>(a, rows, num_sms, s); break;                        \
    case 2: e = FN<T, 2>(a, rows, num_sms, s); break;                        \
    case 4: e = FN<T, 4>(a, rows, num_sms, s); break;                        \
    case 8: e = FN<T, 8>(a, rows, num_sms, s); break;                        \
    case 16: e = FN<T, 16>(a, rows, num_sms, s); break;                      \
    default: e = FN<T, 32>(a, rows, num_sms, s); break;                      \
  }

}  // namespace

cudaError_t launch_residual_forward(const ResidualArgs& a, int num_sms, cudaStream_t s) {
  const uint32_t rows = static_cast<uint32_t>(a.B) * a.I * a.J;
  cudaError_t e = cudaSuccess;
  if (a.p.stream_type == TRIMUL_F32) {
    BY_LANES(forward, float)
  } else {
    BY_LANES(forward, bf)
  }
  return e;
}

size_t residual_backward_workspace(int D, long long rows, int num_sms) {
  return static_cast<size_t>(blocks_for(D, rows, num_sms, 2)) * RESIDUAL_SUMS * D * sizeof(float);
}

cudaError_t launch_residual_backward(const ResidualArgs& a, int num_sms, cudaStream_t s) {
  const uint32_t rows = static_cast<uint32_t>(a.B) * a.I * a.J;
  cudaError_t e = cudaSuccess;
  if (a.p.stream_type == TRIMUL_F32) {
    BY_LANES(backward, float)
  } else {
    BY_LANES(backward, bf)
  }
  if (e != cudaSuccess) return e;
  const int n = RESIDUAL_SUMS * a.p.D;
  k8_residual_sum<<<(n + 31) / 32, 256, 0, s>>>(a.part, a.g, a.p.D, blocks_for(a.p.D, rows, num_sms, 2));
  return cudaGetLastError();
}

}  // namespace trimul
