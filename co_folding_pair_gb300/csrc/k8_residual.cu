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

__device__ __forceinline__ float sum8(const float (&v)[8]) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// v -> its normalised value; returns r.  Lanes past D hold and keep zeros.
// The mean is a true division: a row of one value has that value as its mean
// exactly, and the product with 1 / D, off by half an ulp of the mean, would be
// scaled by 1 / sqrt(eps) there.
template <int G>
__device__ __forceinline__ float normalise(float (&v)[8], int kind, float d, float inv_d, float eps, bool live) {
  if (kind == TRIMUL_NORM_LAYER) {
    const float mean = row_sum<G>(sum8(v)) / d;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = live ? v[e] - mean : 0.f;
  }
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = v[e] * v[e];
  const float r = rsqrtf(row_sum<G>(sum8(q)) * inv_d + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= r;
  return r;
}

// t (the gradient at the normalised value) -> the gradient at the norm's input.
template <int G>
__device__ __forceinline__ void normalise_grad(float (&t)[8], const float (&hat)[8], float r, int kind, float inv_d) {
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = t[e] * hat[e];
  const float m2 = row_sum<G>(sum8(q)) * inv_d;
  const float m1 = kind == TRIMUL_NORM_LAYER ? row_sum<G>(sum8(t)) * inv_d : 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = r * (t[e] - m1 - hat[e] * m2);
}

// Eight of a parameter's values, or the value it has where it is absent.
__device__ __forceinline__ void param8(const float* p, int c, bool live, float absent, float (&f)[8]) {
  if (p && live) {
    load8(p + c, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = absent;
  }
}

// sigmoid(x) and 1 - sigmoid(x), each to fp32's relative precision (the
// exponential's argument is never positive, so nothing overflows either).
__device__ __forceinline__ float2 sigmoid2(float x) {
  const float e = __expf(-fabsf(x)), big = __frcp_rn(1.0f + e);
  return x >= 0.f ? make_float2(big, e * big) : make_float2(e * big, big);
}

// The gate's eight values of a row (pair), as they are.
__device__ __forceinline__ const uint16_t* gate_row(const ResidualArgs& a, uint32_t pair) {
  if (a.p.gate == TRIMUL_GATE_PAIR) return a.gate + static_cast<size_t>(pair) * a.p.D;
  uint32_t row, j;
  a.by_J.divmod(pair, row, j);
  const size_t at = a.p.gate == TRIMUL_GATE_COL ? row : static_cast<size_t>(a.by_I.div(row)) * a.J + j;
  return a.gate + at * a.p.D;
}

__device__ __forceinline__ float mask_of(const ResidualArgs& a, uint32_t pair) {
  return a.mask ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.mask)[pair]) : 1.f;
}

__device__ __forceinline__ void zero8(float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = 0.f;
}

using bf = __nv_bfloat16;

// G lanes share a row, eight channels each.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads) k8_residual_fwd(ResidualArgs a, uint32_t rows) {
  const int c = (threadIdx.x % G) * 8;
  const bool live = c < a.p.D;
  const float d_f = static_cast<float>(a.p.D), inv_d = 1.0f / d_f;
  float pg[8], pb[8], ng[8], nb[8], ch[8];
  param8(a.p.post_gamma, c, live, 1.f, pg);
  param8(a.p.post_beta, c, live, 0.f, pb);
  param8(a.p.pre_gamma, c, live, 1.f, ng);
  param8(a.p.pre_beta, c, live, 0.f, nb);
  param8(a.p.channel, c, live, 1.f, ch);
  constexpr uint32_t kRows = kThreads / G;
  // every lane of a warp takes the same number of turns, for the shuffles
  for (uint32_t base = blockIdx.x * kRows; base < rows; base += gridDim.x * kRows) {
    const uint32_t row = base + threadIdx.x / G;
    const bool on = live && row < rows;
    const size_t at = static_cast<size_t>(row) * a.p.D + c;
    float x[8], y[8], g[8];
    zero8(x), zero8(y), zero8(g);
    float m = 1.f;
    if (on) {
      load8(static_cast<const T*>(a.x) + at, x);
      load8(reinterpret_cast<const bf*>(a.u) + at, y);
      if (a.gate) load8(reinterpret_cast<const bf*>(gate_row(a, row)) + c, g);
      m = mask_of(a, row);
    }
    if (a.p.post_norm != TRIMUL_NORM_NONE) normalise<G>(y, a.p.post_norm, d_f, inv_d, a.p.eps, live);
    const float k = a.p.scale * m;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float w = k * ch[e];
      if (a.gate) w *= a.p.gate_sigmoid ? sigmoid2(g[e]).x : g[e];
      if (m != 0.f) x[e] += w * (a.p.post_norm != TRIMUL_NORM_NONE ? y[e] * pg[e] + pb[e] : y[e]);
    }
    if (on) store8(static_cast<T*>(a.out) + at, x);
    if (a.normed) {
      if (!live) zero8(x);
      normalise<G>(x, a.p.pre_norm, d_f, inv_d, a.p.eps, live);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = m != 0.f ? x[e] * ng[e] + nb[e] : 0.f;
      if (on) store8(reinterpret_cast<bf*>(a.normed) + at, x);
    }
  }
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads) k8_residual_bwd(ResidualArgs a, uint32_t rows) {
  const int c = (threadIdx.x % G) * 8;
  const bool live = c < a.p.D;
  const float d_f = static_cast<float>(a.p.D), inv_d = 1.0f / d_f;
  const bool post = a.p.post_norm != TRIMUL_NORM_NONE, pre = a.p.pre_norm != TRIMUL_NORM_NONE;
  float pg[8], pb[8], ng[8], ch[8];
  param8(a.p.post_gamma, c, live, 1.f, pg);
  param8(a.p.post_beta, c, live, 0.f, pb);
  param8(a.p.pre_gamma, c, live, 1.f, ng);
  param8(a.p.channel, c, live, 1.f, ch);
  float sums[RESIDUAL_SUMS][8] = {};
  constexpr uint32_t kRows = kThreads / G;
  for (uint32_t base = blockIdx.x * kRows; base < rows; base += gridDim.x * kRows) {
    const uint32_t row = base + threadIdx.x / G;
    const bool on = live && row < rows;
    const size_t at = static_cast<size_t>(row) * a.p.D + c;
    float x[8], yh[8], g[8], d[8], dn[8];
    zero8(x), zero8(yh), zero8(g), zero8(d), zero8(dn);
    float m = 0.f;
    if (on) {
      m = mask_of(a, row);
      load8(static_cast<const T*>(a.dout) + at, d);
      if (a.dout2) {
        load8(static_cast<const T*>(a.dout2) + at, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] += x[e];
      }
      zero8(x);
      if (m != 0.f) {  // padding: zeros, whatever these hold
        load8(static_cast<const T*>(a.x) + at, x);
        load8(reinterpret_cast<const bf*>(a.u) + at, yh);
        if (a.gate) load8(reinterpret_cast<const bf*>(gate_row(a, row)) + c, g);
        if (pre) load8(reinterpret_cast<const bf*>(a.dnormed) + at, dn);
      }
    }
    float pr = 0.f;
    if (post) pr = normalise<G>(yh, a.p.post_norm, d_f, inv_d, a.p.eps, live);
    const float k = a.p.scale * m;
    float y[8], gv[8], gd[8];  // the gate's value and its derivative
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = post ? yh[e] * pg[e] + pb[e] : yh[e];
      const float2 sg = sigmoid2(g[e]);
      gv[e] = !a.gate ? 1.f : a.p.gate_sigmoid ? sg.x : g[e];
      gd[e] = a.p.gate_sigmoid ? sg.x * sg.y : 1.f;
    }
    if (pre) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += k * ch[e] * gv[e] * y[e];
      if (!live) zero8(x);
      const float nr = normalise<G>(x, a.p.pre_norm, d_f, inv_d, a.p.eps, live);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sums[2][e] += dn[e] * x[e];
        sums[3][e] += dn[e];
        dn[e] *= ng[e];
      }
      normalise_grad<G>(dn, x, nr, a.p.pre_norm, inv_d);
      if (live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] += dn[e];
      }
    }
    if (on) store8(static_cast<T*>(a.dx) + at, d);
    // from here on d is w dX, and a padding pair's is 0
    float dg[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float kd = m != 0.f ? k * d[e] : 0.f;
      const float ky = kd * y[e];
      sums[4][e] += ky * gv[e];
      dg[e] = ky * ch[e] * gd[e];
      d[e] = kd * ch[e] * gv[e];
      sums[0][e] += d[e] * yh[e];
      sums[1][e] += d[e];
    }
    if (on && a.dgate) store8(reinterpret_cast<bf*>(a.dgate) + at, dg);
    if (post) {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] *= pg[e];
      normalise_grad<G>(d, yh, pr, a.p.post_norm, inv_d);
    }
    if (on) store8(reinterpret_cast<bf*>(a.du) + at, d);
  }
  // the block's column sums, its rows added in order
  __shared__ float s[kRows][G * 8 + 1];
  for (int q = 0; q < RESIDUAL_SUMS; ++q) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) s[threadIdx.x / G][c + e] = sums[q][e];
    __syncthreads();
    for (int n = threadIdx.x; n < a.p.D; n += kThreads) {
      float t = 0.f;
      for (int r = 0; r < static_cast<int>(kRows); ++r) t += s[r][n];
      a.part[(static_cast<size_t>(blockIdx.x) * RESIDUAL_SUMS + q) * a.p.D + n] = t;
    }
  }
}

// The blocks' column sums added in order.
__global__ void __launch_bounds__(256)
    k8_residual_sum(const float* __restrict__ part, trimul_residual_grads g, int D, int blocks) {
  float* const out[RESIDUAL_SUMS] = {g.post_gamma, g.post_beta, g.pre_gamma, g.pre_beta, g.channel};
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= RESIDUAL_SUMS * D || !out[n / D]) return;
  float t = 0.f;
  for (int k = 0; k < blocks; ++k) t += part[static_cast<size_t>(k) * RESIDUAL_SUMS * D + n];
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

template <typename T, int G>
void forward(const ResidualArgs& a, uint32_t rows, int num_sms, cudaStream_t s) {
  k8_residual_fwd<T, G><<<blocks_for(a.p.D, rows, num_sms, 4), kThreads, 0, s>>>(a, rows);
}
template <typename T, int G>
void backward(const ResidualArgs& a, uint32_t rows, int num_sms, cudaStream_t s) {
  k8_residual_bwd<T, G><<<blocks_for(a.p.D, rows, num_sms, 2), kThreads, 0, s>>>(a, rows);
}

#define BY_LANES(FN, T)                                                  \
  switch (lanes_of(a.p.D)) {                                             \
    case 1: FN<T, 1>(a, rows, num_sms, s); break;                        \
    case 2: FN<T, 2>(a, rows, num_sms, s); break;                        \
    case 4: FN<T, 4>(a, rows, num_sms, s); break;                        \
    case 8: FN<T, 8>(a, rows, num_sms, s); break;                        \
    case 16: FN<T, 16>(a, rows, num_sms, s); break;                      \
    default: FN<T, 32>(a, rows, num_sms, s); break;                      \
  }

}  // namespace

cudaError_t launch_residual_forward(const ResidualArgs& a, int num_sms, cudaStream_t s) {
  const uint32_t rows = static_cast<uint32_t>(a.B) * a.I * a.J;
  if (a.p.stream_type == TRIMUL_F32) {
    BY_LANES(forward, float)
  } else {
    BY_LANES(forward, bf)
  }
  return cudaGetLastError();
}

size_t residual_backward_workspace(int D, long long rows, int num_sms) {
  return static_cast<size_t>(blocks_for(D, rows, num_sms, 2)) * RESIDUAL_SUMS * D * sizeof(float);
}

cudaError_t launch_residual_backward(const ResidualArgs& a, int num_sms, cudaStream_t s) {
  const uint32_t rows = static_cast<uint32_t>(a.B) * a.I * a.J;
  if (a.p.stream_type == TRIMUL_F32) {
    BY_LANES(backward, float)
  } else {
    BY_LANES(backward, bf)
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int n = RESIDUAL_SUMS * a.p.D;
  k8_residual_sum<<<(n + 255) / 256, 256, 0, s>>>(a.part, a.g, a.p.D, blocks_for(a.p.D, rows, num_sms, 2));
  return cudaGetLastError();
}

}  // namespace trimul
