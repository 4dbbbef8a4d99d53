// k8_residual.cu -- the residual step, forward and backward.
//
//   y = Norm_post(u),  w = scale mask channel G(gate),  X = x + w y,  n = Norm_pre(X)
//
// Forward writes X and n.  Backward takes dX' = dout (+ dout2) and dn, computes
// y, X and both norms' statistics again from x and u (so nothing is kept from
// the forward, and X before its rounding is what the gradient is taken of), and
//
//   dX = dX' + Norm_pre'(dn),    dx = dX,    q = scale mask G(gate) dX,
//   du = Norm_post'(q channel),    dgate = scale mask G'(gate) dX (channel y),
//   of the pre-norm: dgamma = sum dn X^, dbeta = sum dn, and of the rest, from
//   S0 = sum q u^ and S1 = sum q alone,  dgamma = channel S0,  dbeta = channel S1,
//   dchannel = gamma S0 + beta S1
//
// with, for v^ = (v - mean) r normalised and t = dv' gamma,
//   Norm'(dv') = r (t - mean(t) - v^ mean(t v^))     (RMS: without the means of v and t).
//
// Each is one pass over the rows: 8 (forward) to 14 (backward) bytes an element
// in bf16 against some 20 to 60 operations, so both should be bound by memory.
// The forward is (2048^2 x 256 bf16, both norms, a gate a row: 1.42 ms, 6.0
// TB/s), and the backward with an fp32 stream (1024^2 x 256, both norms, a gate a
// pair: 0.87 ms, 6.8 TB/s).  In bf16 with two layer norms the backward is bound
// by its instructions and their latency (1024^2 x 128: 0.28 ms, 0.85 of the
// floor, with a gate a row and a channel scale 0.33 ms, 0.72; with RMS norms
// 0.25 ms, 0.96).  Widths a little above a power of two
// leave lanes idle (136: 15 of 32), and that much of the rate.
// Rounding: each output is rounded once, from fp32.
#include <algorithm>
#include <type_traits>

#include "pair_ops.cuh"

namespace trimul {

namespace {

// Sums over the G lanes that share a row: of one number, or of two at once.  In the
// first step each half of the lanes takes over one of the numbers, and hands
// its sum back in the last: log2 G + 1 shuffles for both instead of 2 log2 G.
template <int G>
__device__ __forceinline__ void row_sums(float (&v)[1]) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
}
template <int G>
__device__ __forceinline__ void row_sums(float (&v)[2]) {
  if constexpr (G > 1) {
    const bool up = threadIdx.x & (G / 2);
    float keep = up ? v[1] : v[0];
    keep += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], G / 2);
#pragma unroll
    for (int o = G / 4; o > 0; o >>= 1) keep += __shfl_xor_sync(0xffffffffu, keep, o);
    const float other = __shfl_xor_sync(0xffffffffu, keep, G / 2);
    v[0] = up ? other : keep;
    v[1] = up ? keep : other;
  }
}
// 1 / sqrt(x) for x of normal size (eps keeps it from 0), to 2 ulp (the approximate instruction).
__device__ __forceinline__ float inverse_root(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Each row of v -> its normalised value; scale[r] its factor.  Lanes past D hold
// and keep zeros.  The mean has to be the sum over D exactly rounded: a row of
// one value has that value as its mean, and half an ulp of the mean more would
// be scaled by 1 / sqrt(eps) there.  So it is a division, unless 1 / D is a
// number itself.
template <int G, int R>
__device__ __forceinline__ void normalise(F8 (&v)[R], float (&scale)[R], int kind, float d, float inv_d, float eps,
                                          bool live) {
  float t[R];
  if (kind == TRIMUL_NORM_LAYER) {
#pragma unroll
    for (int r = 0; r < R; ++r) t[r] = sum_of(v[r]);
    row_sums<G>(t);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float mean = (__float_as_uint(d) & 0x7fffffu) ? t[r] / d : t[r] * inv_d;
      const f2 shift = both(live ? -mean : 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[r].v[e] = add2(v[r].v[e], shift);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) t[r] = dot_of(v[r], v[r]);
  row_sums<G>(t);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    scale[r] = inverse_root(t[r] * inv_d + eps);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[r].v[e] = mul2(v[r].v[e], both(scale[r]));
  }
}

// t (the gradient at the normalised value) -> the gradient at the norm's input.
// Lanes past D hold and keep zeros here too: the mean of t is not for them, as
// the next norm's gradient would sum it.
template <int G>
__device__ __forceinline__ void normalise_grad(F8& t, const F8& hat, float scale, int kind, float inv_d, bool live) {
  const float k = -scale * inv_d;
  float m[2] = {dot_of(t, hat), 0.f};
  if (kind == TRIMUL_NORM_LAYER) {
    m[1] = sum_of(t);
    row_sums<G>(m);
    if (!live) m[1] = 0.f;
  } else {
    float one[1] = {m[0]};
    row_sums<G>(one);
    m[0] = one[0];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) t.v[e] = fma2(t.v[e], both(scale), fma2(hat.v[e], both(m[0] * k), both(m[1] * k)));
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

// The rows of the next turns are on their way while some are worked on: every
// thread copies its own 16 bytes of each tensor into a ring of its own in
// shared memory and reads them back itself, so the ring needs no barrier, only
// the thread's wait for its oldest copies.  Depth, not registers, sets the
// bytes in flight.  (The backward has up to six tensors to read.)
constexpr int kForwardThreads = 256, kForwardBlocks = 2, kForwardDepth = 3;
constexpr int kBackwardThreads = 256, kBackwardBlocks = 2, kBackwardDepth = 2;

__device__ __forceinline__ void copy16(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // until at most N groups are on their way
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight elements a lane of a row of D, in ring slots kThreads apart: one slot
// (bf16), which the lane copies and reads itself, or two (fp32).  There, the
// lanes of a row copy its 16-byte groups in order, the first G of them to the
// first slot and the others to the second, so that every instruction reads
// whole sectors; a lane's two groups are copied by others, and the warp has to
// meet before they are read, and before they are written again (meet).
template <int kThreads, int G>
__device__ __forceinline__ void copy8(uint4* to, const __nv_bfloat16* row, int D) {
  const int i = threadIdx.x % G;
  copy16(to, row + i * 8);
}
template <int kThreads, int G>
__device__ __forceinline__ void copy8(uint4* to, const float* row, int D) {
  const int i = threadIdx.x % G;
  if (i * 4 < D) copy16(to, row + i * 4);
  if ((G + i) * 4 < D) copy16(to + kThreads, row + (G + i) * 4);
}
template <typename T>
__device__ __forceinline__ void meet() {
  if (sizeof(T) == 4) __syncwarp();
}
__device__ __forceinline__ F8 widen8(const uint4 v) {
  return F8{{unpack_bf162(v.x), unpack_bf162(v.y), unpack_bf162(v.z), unpack_bf162(v.w)}};
}
// The turns over whole blocks of rows without a mask need not look whether a
// row is there; the others (kAsk) read zeros where it is not.
template <bool kAsk, int kThreads, int G>
__device__ __forceinline__ F8 take8(const uint4* from, bool on, __nv_bfloat16) {
  return widen8(!kAsk || on ? from[0] : make_uint4(0u, 0u, 0u, 0u));
}
template <bool kAsk, int kThreads, int G>
__device__ __forceinline__ F8 take8(const uint4* from, bool on, float) {
  const int i = threadIdx.x % G;
  auto group = [&](int p) { return reinterpret_cast<const ulonglong2*>(from - i + p % G + p / G * kThreads)[0]; };
  const ulonglong2 z = make_ulonglong2(0, 0);
  const ulonglong2 a = !kAsk || on ? group(2 * i) : z;
  const ulonglong2 b = !kAsk || on ? group(2 * i + 1) : z;
  return F8{{a.x, a.y, b.x, b.y}};
}

// Slots that nothing is copied to hold zeros.
__device__ __forceinline__ void clear_slots(uint4* own, int n, int threads) {
  for (int k = 0; k < n; ++k) own[k * threads] = make_uint4(0u, 0u, 0u, 0u);
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
// A gate is kept as its value or, of a sigmoid, as one number that gives both
// the value and its derivative: with e = exp(-|x|) (which cannot overflow) and
// small = e / (1 + e), the lesser of sigmoid(x) and 1 - sigmoid(x), it is small
// for x < 0 and -small for x >= 0.  The fast exponential is off by up to 2 +
// 1.173 |x| ulp, and small with it, by some 3 more: 2^-18 of it at x = -20, when
// it is 2e-9 itself.  Below the least normal number (x < -87.3) it is 0.  1 -
// small, the value for x >= 0, has fp32's precision.
__device__ __forceinline__ float sigmoid_code(float x) {
  const float e = __expf(-fabsf(x)), small = e * reciprocal(1.0f + e);
  return x >= 0.f ? -small : small;
}
__device__ __forceinline__ void sigmoid_codes(F8& g) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = split2(g.v[e]);
    g.v[e] = pair2(sigmoid_code(x.x), sigmoid_code(x.y));
  }
}
__device__ __forceinline__ float sigmoid_value(float code) { return __float_as_int(code) < 0 ? 1.0f + code : code; }
// The gate's values, and their derivatives (1 of a gate without sigmoid).
__device__ __forceinline__ F8 gate_values(const F8& code, bool sigmoid) {
  F8 v = code;
  if (sigmoid) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = split2(code.v[e]);
      v.v[e] = pair2(sigmoid_value(x.x), sigmoid_value(x.y));
    }
  }
  return v;
}
__device__ __forceinline__ F8 gate_slopes(const F8& code) {
  F8 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = split2(code.v[e]);
    v.v[e] = pair2(fmaf(-fabsf(x.x), fabsf(x.x), fabsf(x.x)), fmaf(-fabsf(x.y), fabsf(x.y), fabsf(x.y)));
  }
  return v;
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

// A pair's mask, as its bits: they are loaded a turn early, and not looked at before they are needed.
constexpr uint32_t kOne = 0x3f80;
__device__ __forceinline__ uint32_t mask_of(const ResidualArgs& a, uint32_t pair, uint32_t rows) {
  return a.mask && pair < rows ? a.mask[pair] : kOne;
}

constexpr int kForwardRows = 2;  // R

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

// G lanes share a row, eight channels each.  A thread works on R rows at a
// time: their chains of operations, shuffles above all, run side by side, and
// their sums are reduced together.
template <typename T, int G>
__global__ void __launch_bounds__(kForwardThreads, kForwardBlocks) k8_residual_fwd(ResidualArgs a, uint32_t rows) {
  extern __shared__ uint4 ring[];
  constexpr int kThreads = kForwardThreads, kDepth = kForwardDepth, R = kForwardRows;
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
  const uint32_t step = gridDim.x * kRows * R;
  uint4* const own = ring + threadIdx.x;
  if (!live || sizeof(T) == 4) clear_slots(own, kDepth * R * slots, kThreads);
  // rows are below 2^31 and steps below 2^20: sums of a few stay within 32 bits
  uint32_t row = blockIdx.x * kRows * R + threadIdx.x / G;
  size_t at = static_cast<size_t>(row) * a.p.D + c;
  const size_t stride = static_cast<size_t>(step) * a.p.D, next = static_cast<size_t>(kRows) * a.p.D;
  // the rows from `row`, at element `at`, on into stage `stage`; rows past the end are left out
  auto fetch = [&](uint32_t row, size_t at, int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r, row += kRows, at += next) {
      if (row < rows) {
        uint4* const to = own + (stage * R + r) * slots * kThreads;
        if (live || sizeof(T) == 4) copy8<kThreads, G>(to, static_cast<const T*>(a.x) + (at - c), a.p.D);
        if (live) {
          copy16(to + kSlots<T> * kThreads, a.u + at);
          if (a.gate) copy16(to + (kSlots<T> + 1) * kThreads, gate_row(a, row) + c);
        }
      }
    }
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) fetch(row + k * step, at + k * stride, k);
  int stage = 0;
  uint32_t m_next[R];
#pragma unroll
  for (int r = 0; r < R; ++r) m_next[r] = mask_of(a, row + r * kRows, rows);
  auto turn = [&](auto ask) {
    constexpr bool kAsk = decltype(ask)::value;
    bool on[R];
    float m[R], unused[R];
    F8 x[R], y[R];
    meet<T>();
    fetch(row + (kDepth - 1) * step, at + (kDepth - 1) * stride, (stage + kDepth - 1) % kDepth);
    copies_wait<kDepth - 1>();
    meet<T>();
    const uint4* const from = own + stage * R * slots * kThreads;
    stage = (stage + 1) % kDepth;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t mine = row + r * kRows;
      on[r] = live && (!kAsk || mine < rows);
      m[r] = kAsk ? bf16_lo(m_next[r]) : 1.f;
      if (kAsk) m_next[r] = mask_of(a, mine + step, rows);
      x[r] = take8<kAsk, kThreads, G>(from + r * slots * kThreads, on[r], T());
      y[r] = take8<kAsk, kThreads, G>(from + (r * slots + kSlots<T>) * kThreads, on[r], bf());
    }
    if (a.p.post_norm != TRIMUL_NORM_NONE) normalise<G>(y, unused, a.p.post_norm, d_f, inv_d, a.p.eps, live);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[r].v[e] = fma2(y[r].v[e], A.v[e], B.v[e]);
      F8 g = {{both(m[r]), both(m[r]), both(m[r]), both(m[r])}};
      if (a.gate) {
        g = take8<kAsk, kThreads, G>(from + (r * slots + kSlots<T> + 1) * kThreads, on[r], bf());
        if (a.p.gate_sigmoid) {
          sigmoid_codes(g);
          g = gate_values(g, true);
        }
        if (kAsk) {
#pragma unroll
          for (int e = 0; e < 4; ++e) g.v[e] = mul2(g.v[e], both(m[r]));
        }
      }
      if (!kAsk || m[r] != 0.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[r].v[e] = fma2(y[r].v[e], g.v[e], x[r].v[e]);
      }
      if (on[r]) put8(static_cast<T*>(a.out) + at + r * next, x[r]);
    }
    if (a.normed) {
      normalise<G>(x, unused, a.p.pre_norm, d_f, inv_d, a.p.eps, live);
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[r].v[e] = fma2(x[r].v[e], ng.v[e], nb.v[e]);
        if (kAsk && m[r] == 0.f) x[r] = F8{};
        if (on[r]) put8(reinterpret_cast<bf*>(a.normed) + at + r * next, x[r]);
      }
    }
    row += step;
    at += stride;
  };
  // every lane of a warp takes the same number of turns, for the shuffles
  for (uint32_t base = blockIdx.x * kRows * R; base < rows; base += step) {
    if (a.mask || base + kRows * R > rows)
      turn(std::true_type());
    else
      turn(std::false_type());
  }
}

// One row at a time here: the sums take the registers that a second one would need.
template <typename T, int G>
__global__ void __launch_bounds__(kBackwardThreads, kBackwardBlocks) k8_residual_bwd(ResidualArgs a, uint32_t rows) {
  extern __shared__ uint4 ring[];
  // channel post_gamma, channel post_beta, pre_gamma: the low and the high four of each lane's eight
  __shared__ float4 par4[3][2][32];
  let_next_begin();
  constexpr int kThreads = kBackwardThreads, kDepth = kBackwardDepth;
  constexpr uint32_t kRows = kThreads / G;
  const int c = (threadIdx.x % G) * 8;
  const bool live = c < a.p.D;
  const float d_f = static_cast<float>(a.p.D), inv_d = 1.0f / d_f;
  const bool post = a.p.post_norm != TRIMUL_NORM_NONE, pre = a.p.pre_norm != TRIMUL_NORM_NONE;
  for (int n = threadIdx.x; n < 256; n += kThreads) {
    const bool in = n < a.p.D;
    const float ch = in && a.p.channel ? a.p.channel[n] : 1.f;
    const float v[3] = {ch * (in && a.p.post_gamma ? a.p.post_gamma[n] : 1.f),
                        ch * (in && a.p.post_beta ? a.p.post_beta[n] : 0.f), in && a.p.pre_gamma ? a.p.pre_gamma[n] : 1.f};
#pragma unroll
    for (int q = 0; q < 3; ++q) reinterpret_cast<float*>(&par4[q][n / 4 % 2][n / 8])[n % 4] = v[q];
  }
  __syncthreads();
  auto par = [&](int q) {
    const ulonglong2 lo = reinterpret_cast<const ulonglong2&>(par4[q][0][c / 8]);
    const ulonglong2 hi = reinterpret_cast<const ulonglong2&>(par4[q][1][c / 8]);
    return F8{{lo.x, lo.y, hi.x, hi.y}};
  };
  const int slots = backward_slots<T>(a.gate, a.dout2, pre);
  const int at_u = kSlots<T> * (a.dout2 ? 3 : 2), at_g = at_u + 1, at_n = at_g + (a.gate ? 1 : 0);
  const uint32_t step = gridDim.x * kRows;
  uint4* const own = ring + threadIdx.x;
  if (!live || sizeof(T) == 4) clear_slots(own, kDepth * slots, kThreads);
  uint32_t row = blockIdx.x * kRows + threadIdx.x / G;
  size_t at = static_cast<size_t>(row) * a.p.D + c;
  const size_t stride = static_cast<size_t>(step) * a.p.D;
  auto fetch = [&](uint32_t row, size_t at, int stage) {
    if (row < rows) {
      uint4* const to = own + stage * slots * kThreads;
      if (live || sizeof(T) == 4) {
        const size_t first = at - c;
        copy8<kThreads, G>(to, static_cast<const T*>(a.dout) + first, a.p.D);
        // only X's statistics need x
        if (pre) copy8<kThreads, G>(to + kSlots<T> * kThreads, static_cast<const T*>(a.x) + first, a.p.D);
        if (a.dout2) copy8<kThreads, G>(to + 2 * kSlots<T> * kThreads, static_cast<const T*>(a.dout2) + first, a.p.D);
      }
      if (live) {
        copy16(to + at_u * kThreads, a.u + at);
        if (a.gate) copy16(to + at_g * kThreads, gate_row(a, row) + c);
        if (pre) copy16(to + at_n * kThreads, a.dnormed + at);
      }
    }
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) fetch(row + k * step, at + k * stride, k);
  F8 sums[RESIDUAL_SUMS] = {};
  int stage = 0;
  uint32_t m_next = mask_of(a, row, rows);
  auto turn = [&](auto ask) {
    constexpr bool kAsk = decltype(ask)::value;
    const bool on = live && (!kAsk || row < rows);
    const float m = !kAsk ? 1.f : on ? bf16_lo(m_next) : 0.f;
    if (kAsk) m_next = mask_of(a, row + step, rows);
    const bool real = on && m != 0.f;  // padding: zeros, whatever the tensors hold
    const f2 k = both(a.p.scale * m);
    meet<T>();
    fetch(row + (kDepth - 1) * step, at + (kDepth - 1) * stride, (stage + kDepth - 1) % kDepth);
    copies_wait<kDepth - 1>();
    meet<T>();
    const uint4* const from = own + stage * slots * kThreads;
    stage = (stage + 1) % kDepth;
    auto slot = [&](int n) { return from + n * kThreads; };
    F8 yh[1] = {take8<kAsk, kThreads, G>(slot(at_u), real, bf())}, gate;
    float post_r[1], pre_r[1];
    if (post) normalise<G>(yh, post_r, a.p.post_norm, d_f, inv_d, a.p.eps, live);
    if (a.gate) {
      gate = take8<kAsk, kThreads, G>(slot(at_g), real, bf());
      if (a.p.gate_sigmoid) sigmoid_codes(gate);
    }
    F8 d = {};
    if (pre) {
      F8 x[1] = {take8<kAsk, kThreads, G>(slot(kSlots<T>), real, T())};
      {
        const F8 pg = par(0), pb = par(1);
        F8 w = {{k, k, k, k}};
        if (a.gate) {
          w = gate_values(gate, a.p.gate_sigmoid);
#pragma unroll
          for (int e = 0; e < 4; ++e) w.v[e] = mul2(w.v[e], k);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[0].v[e] = fma2(w.v[e], fma2(yh[0].v[e], pg.v[e], pb.v[e]), x[0].v[e]);
      }
      normalise<G>(x, pre_r, a.p.pre_norm, d_f, inv_d, a.p.eps, live);
      const F8 ng = par(2);
      d = take8<kAsk, kThreads, G>(slot(at_n), real, bf());
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sums[2].v[e] = fma2(d.v[e], x[0].v[e], sums[2].v[e]);
        sums[3].v[e] = add2(d.v[e], sums[3].v[e]);
        d.v[e] = mul2(d.v[e], ng.v[e]);
      }
      normalise_grad<G>(d, x[0], pre_r[0], a.p.pre_norm, inv_d, live);
    }
    {
      const F8 t = take8<kAsk, kThreads, G>(slot(0), on, T());
#pragma unroll
      for (int e = 0; e < 4; ++e) d.v[e] = add2(t.v[e], d.v[e]);
    }
    if (a.dout2) {
      const F8 t = take8<kAsk, kThreads, G>(slot(2 * kSlots<T>), on, T());
#pragma unroll
      for (int e = 0; e < 4; ++e) d.v[e] = add2(t.v[e], d.v[e]);
    }
    if (on) put8(static_cast<T*>(a.dx) + at, d);
    if (kAsk && !real) d = F8{};  // a padding pair passes nothing on to what follows
#pragma unroll
    for (int e = 0; e < 4; ++e) d.v[e] = mul2(d.v[e], k);
    const F8 pg = par(0);
    if (a.dgate) {
      const F8 pb = par(1);
      F8 t;
#pragma unroll
      for (int e = 0; e < 4; ++e) t.v[e] = mul2(d.v[e], fma2(yh[0].v[e], pg.v[e], pb.v[e]));
      if (a.p.gate_sigmoid) {
        const F8 slope = gate_slopes(gate);
#pragma unroll
        for (int e = 0; e < 4; ++e) t.v[e] = mul2(t.v[e], slope.v[e]);
      }
      if (on) put8(reinterpret_cast<bf*>(a.dgate) + at, t);
    }
    if (a.gate) {
      const F8 w = gate_values(gate, a.p.gate_sigmoid);
#pragma unroll
      for (int e = 0; e < 4; ++e) d.v[e] = mul2(d.v[e], w.v[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sums[0].v[e] = fma2(d.v[e], yh[0].v[e], sums[0].v[e]);
      sums[1].v[e] = add2(d.v[e], sums[1].v[e]);
      d.v[e] = mul2(d.v[e], pg.v[e]);
    }
    if (post) normalise_grad<G>(d, yh[0], post_r[0], a.p.post_norm, inv_d, live);
    if (on) put8(reinterpret_cast<bf*>(a.du) + at, d);
    row += step;
    at += stride;
  };
  for (uint32_t base = blockIdx.x * kRows; base < rows; base += step) {
    if (a.mask || base + kRows > rows)
      turn(std::true_type());
    else
      turn(std::false_type());
  }
  if (!a.part) return;  // no parameter's gradient is wanted
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

// The parameters' gradients from the blocks' column sums: 32 channels a block,
// 32 groups of parts side by side; blockIdx.y 0 for S0 and S1, 1 for the
// pre-norm's two.
__global__ void __launch_bounds__(1024) k8_residual_sum(ResidualArgs a, int blocks) {
  __shared__ float2 s[32][33];
  const int lane = threadIdx.x % 32, group = threadIdx.x / 32, D = a.p.D;
  int n = blockIdx.x * 32 + lane;
  float2 t = make_float2(0.f, 0.f);
  after_previous();
  if (n < D) {
#pragma unroll 4
    for (int k = group; k < blocks; k += 32) {
      const float* const p = a.part + (static_cast<size_t>(k) * RESIDUAL_SUMS + 2 * blockIdx.y) * D + n;
      t.x += p[0];
      t.y += p[D];
    }
  }
  s[group][lane] = t;
  __syncthreads();
  // a warp a channel from here on
  t = s[lane][group];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
    t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
  }
  n = blockIdx.x * 32 + group;
  if (lane != 0 || n >= D) return;
  if (blockIdx.y == 1) {
    if (a.g.pre_gamma) a.g.pre_gamma[n] = t.x;
    if (a.g.pre_beta) a.g.pre_beta[n] = t.y;
    return;
  }
  const float ch = a.p.channel ? a.p.channel[n] : 1.f;
  if (a.g.post_gamma) a.g.post_gamma[n] = ch * t.x;
  if (a.g.post_beta) a.g.post_beta[n] = ch * t.y;
  if (a.g.channel) a.g.channel[n] = (a.p.post_gamma ? a.p.post_gamma[n] : 1.f) * t.x + (a.p.post_beta ? a.p.post_beta[n] : 0.f) * t.y;
}

bool any_sum(const trimul_residual_grads& g) {
  return g.post_gamma || g.post_beta || g.pre_gamma || g.pre_beta || g.channel;
}

int lanes_of(int D) {
  int g = 1;
  while (g * 8 < D) g *= 2;
  return g;
}

// Blocks of a launch over `rows` rows.
int blocks_for(int D, long long rows, int threads, int R, int blocks) {
  const int per_block = threads / lanes_of(D) * R;
  return static_cast<int>(std::min<long long>((rows + per_block - 1) / per_block, blocks));
}

template <typename T, int G>
cudaError_t forward(const ResidualArgs& a, uint32_t rows, int num_sms, cudaStream_t s) {
  constexpr int kStage = kForwardDepth * kForwardRows * kForwardThreads * 16;
  cudaError_t e = allow_smem<k8_residual_fwd<T, G>>(forward_slots<T>(true) * kStage);
  if (e != cudaSuccess) return e;
  const int grid = blocks_for(a.p.D, rows, kForwardThreads, kForwardRows, kForwardBlocks * num_sms);
  k8_residual_fwd<T, G><<<grid, kForwardThreads, forward_slots<T>(a.gate) * kStage, s>>>(a, rows);
  return cudaGetLastError();
}
template <typename T, int G>
cudaError_t backward(const ResidualArgs& a, uint32_t rows, int num_sms, cudaStream_t s) {
  constexpr int kStage = kBackwardDepth * kBackwardThreads * 16;
  ResidualArgs b = a;
  if (!any_sum(a.g)) b.part = nullptr;
  cudaError_t e = allow_smem<k8_residual_bwd<T, G>>(backward_slots<T>(true, true, true) * kStage);
  if (e != cudaSuccess) return e;
  const int grid = blocks_for(a.p.D, rows, kBackwardThreads, 1, kBackwardBlocks * num_sms);
  const int slots = backward_slots<T>(a.gate, a.dout2, a.p.pre_norm != TRIMUL_NORM_NONE);
  k8_residual_bwd<T, G><<<grid, kBackwardThreads, slots * kStage, s>>>(b, rows);
  return cudaGetLastError();
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
  return static_cast<size_t>(blocks_for(D, rows, kBackwardThreads, 1, kBackwardBlocks * num_sms)) * RESIDUAL_SUMS * D * sizeof(float);
}

cudaError_t launch_residual_backward(const ResidualArgs& a, int num_sms, cudaStream_t s) {
  const uint32_t rows = static_cast<uint32_t>(a.B) * a.I * a.J;
  cudaError_t e = cudaSuccess;
  if (a.p.stream_type == TRIMUL_F32) {
    BY_LANES(backward, float)
  } else {
    BY_LANES(backward, bf)
  }
  if (e != cudaSuccess || !any_sum(a.g)) return e;
  return launch_early(k8_residual_sum, dim3((a.p.D + 31) / 32, 2), 1024, s, a,
                      blocks_for(a.p.D, rows, kBackwardThreads, 1, kBackwardBlocks * num_sms));
}

}  // namespace trimul
