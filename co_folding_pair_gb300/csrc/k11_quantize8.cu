// k11_quantize8.cu -- bf16 (and weights) to e4m3 with a power of two for each
// block of 128 (linear8.h).
//
// The scale is the least 2^e, e >= -126, with max |v| <= 448 2^e, taken from
// the largest number's bits; v 2^-e is exact, so each code is v's own rounding
// to nearest.  A group with numbers that are not finite takes its scale from
// the others, and those become NaN.
//
// Bound by memory: bf16 is read once; the codes are half of it, and where both
// forms of a gradient are wanted (rows for dx, columns for dW) one read makes
// both.
#include <cuda_fp8.h>

#include <algorithm>

#include "linear8.h"
#include "pair_ops.cuh"

namespace trimul {

namespace {

constexpr int kThreads = 256;

// The larger ones of two pairs of 16-bit numbers.
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

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

// Eight numbers as codes.
__device__ __forceinline__ uint2 codes8(const uint4& v, float inv, bool all_finite) {
  float f[8];
  unpack8(v, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = (all_finite ? f[e] : no_infinity(f[e])) * inv;
  return make_uint2(codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7]));
}

// The largest magnitude, bf16 bits, of the eight numbers of each of 16 lanes, of all of these; where one is not
// finite, `all_finite` is false and the largest is of the others.
__device__ __forceinline__ uint32_t largest_of_16(const uint4& v, bool& all_finite) {
  auto over_lanes = [](uint32_t m) {
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  };
  const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
  uint32_t m = over_lanes(max16x2(max16x2(w[0], w[1]), max16x2(w[2], w[3])));
  all_finite = m < 0x7f80u;
  if (__any_sync(0xffffffffu, !all_finite))  // rare
    m = over_lanes(max16x2(max16x2(finite16x2(w[0]), finite16x2(w[1])), max16x2(finite16x2(w[2]), finite16x2(w[3]))));
  return m;
}

// ------------------------------------------------------------------ rows
// Sixteen lanes have a block of 128 in one 16-byte load each; their turns run along the rows.
constexpr int kTurns = 4;  // loads of a thread that are on their way together
__global__ void __launch_bounds__(kThreads) k11_rows(const uint16_t* __restrict__ x, Operand8 o, long long items, uint32_t per_row,
                                                      uint8_t* __restrict__ out, int* status) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  uint8_t* const scales = out + o.scales_at();
  const int lane = threadIdx.x % 16;
  const long long step = static_cast<long long>(gridDim.x) * (kThreads / 16);
  const long long first = static_cast<long long>(blockIdx.x) * (kThreads / 16) + threadIdx.x / 16;
  // (a warp's two halves go through the turns together: the shuffles need all lanes)
  const long long turns = (items + step * kTurns - 1) / (step * kTurns);
  for (long long t = 0; t < turns; ++t) {
    uint4 v[kTurns];
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const long long item = first + (t * kTurns + u) * step;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (item < items) {
        const long long row = item / per_row, col = (item - row * per_row) * L8_BLOCK + lane * 8;
        if (col < o.depth) v[u] = __ldcs(reinterpret_cast<const uint4*>(x + row * o.depth + col));
      }
    }
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const long long item = first + (t * kTurns + u) * step;
      bool fine;
      const uint32_t byte = scale_byte(largest_of_16(v[u], fine) << 16);
      if (item >= items) continue;
      const long long row = item / per_row, block = item - row * per_row, col = block * L8_BLOCK + lane * 8;
      if (col < o.depth) *reinterpret_cast<uint2*>(out + row * o.ld() + col) = codes8(v[u], over_scale(byte), fine);
      if (lane == 0) scales[o.scale_at(row, block)] = static_cast<uint8_t>(byte);
    }
  }
}

// ------------------------------------------------------------------ columns
// A block takes 128 x 128 tiles below one another.  Rows come in as above (and
// leave as row-wise codes); the tile waits in shared memory, rows 272 bytes
// apart so that a warp's 32 words of one row, and its eight 16-byte stores, lie
// in different banks.  A thread then has two columns of 32 rows: 32 codes a
// column are a whole sector of the transposed output.
constexpr int kSide = 128;
constexpr int kRowBytes = kSide * 2 + 16;

template <bool kRows, bool kSums>
__global__ void __launch_bounds__(kThreads)
    k11_columns(const uint16_t* __restrict__ x, long long rows, int cols, uint8_t* __restrict__ out,
                uint8_t* __restrict__ by_rows, float* __restrict__ part, int parts, int* status) {
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && status) *status = 0;
  __shared__ alignas(16) uint8_t tile[kSide * kRowBytes];
  __shared__ uint32_t tops[4][kSide / 2];
  const Operand8 oc{cols, rows}, orow{rows, cols};
  uint8_t* const scales = out + oc.scales_at();
  uint8_t* const row_scales = kRows ? by_rows + orow.scales_at() : nullptr;
  const int c0 = blockIdx.x * kSide, lane16 = threadIdx.x % 16;
  const int word = threadIdx.x % 64, quarter = threadIdx.x / 64;  // columns 2 word and 2 word + 1, rows 32 quarter ..
  const long long tiles = l8_blocks(rows);
  float sum[2] = {0.f, 0.f};
  for (long long rt = blockIdx.y; rt < tiles; rt += parts) {
    const long long r0 = rt * kSide;
    const int col = c0 + lane16 * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = (h * 4 + u) * 16 + threadIdx.x / 16;
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r0 + r < rows && col < cols) v[u] = __ldcs(reinterpret_cast<const uint4*>(x + (r0 + r) * cols + col));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = (h * 4 + u) * 16 + threadIdx.x / 16;
        *reinterpret_cast<uint4*>(tile + r * kRowBytes + lane16 * 16) = v[u];
        if (kRows) {
          bool fine;
          const uint32_t byte = scale_byte(largest_of_16(v[u], fine) << 16);
          if (r0 + r < rows) {
            if (col < cols) *reinterpret_cast<uint2*>(by_rows + (r0 + r) * orow.ld() + col) = codes8(v[u], over_scale(byte), fine);
            if (lane16 == 0) row_scales[orow.scale_at(r0 + r, blockIdx.x)] = static_cast<uint8_t>(byte);
          }
        }
      }
    }
    __syncthreads();
    uint32_t w[32];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      w[r] = *reinterpret_cast<const uint32_t*>(tile + (quarter * 32 + r) * kRowBytes + word * 4);
      top = max16x2(top, w[r] & 0x7fff7fffu);
    }
    const bool fine = (top & 0xffffu) < 0x7f80u && top < 0x7f800000u;
    if (!fine) {  // rare
      top = 0;
#pragma unroll
      for (int r = 0; r < 32; ++r) top = max16x2(top, finite16x2(w[r]));
    }
    if (kSums) {
#pragma unroll
      for (int r = 0; r < 32; ++r) sum[0] += bf16_lo(w[r]), sum[1] += bf16_hi(w[r]);
    }
    tops[quarter][word] = top;
    __syncthreads();
    top = max16x2(max16x2(tops[0][word], tops[1][word]), max16x2(tops[2][word], tops[3][word]));
    const uint32_t byte[2] = {scale_byte(top << 16), scale_byte(top & 0xffff0000u)};
    const long long rq = r0 + quarter * 32;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = c0 + 2 * word + e;
      if (c >= cols) continue;
      const float inv = over_scale(byte[e]);
      uint32_t q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i] = e ? bf16_hi(w[4 * k + i]) : bf16_lo(w[4 * k + i]);
          f[i] = (fine ? f[i] : no_infinity(f[i])) * inv;
        }
        q[k] = codes4(f[0], f[1], f[2], f[3]);
      }
      uint8_t* const to = out + c * oc.ld() + rq;
      if (rq + 32 <= oc.ld()) {  // (zeros behind the last row)
        reinterpret_cast<uint4*>(to)[0] = make_uint4(q[0], q[1], q[2], q[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(q[4], q[5], q[6], q[7]);
      } else if (rq + 16 <= oc.ld()) {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(q[0], q[1], q[2], q[3]);
      }
      if (quarter == 0) scales[oc.scale_at(c, rt)] = static_cast<uint8_t>(byte[e]);
    }
    // the next tile's rows come where this one's have been read (before the second meeting), its largest ones after its own first meeting
  }
  if (kSums) {
    __syncthreads();
    float2* const s = reinterpret_cast<float2*>(tile);
    s[quarter * 64 + word] = make_float2(sum[0], sum[1]);
    __syncthreads();
    if (quarter == 0 && c0 + 2 * word < cols) {
      const float2 a = s[word], b = s[64 + word], c = s[128 + word], d = s[192 + word];
      *reinterpret_cast<float2*>(part + static_cast<size_t>(blockIdx.y) * cols + c0 + 2 * word) =
          make_float2((a.x + b.x) + (c.x + d.x), (a.y + b.y) + (c.y + d.y));
    }
  }
}

// ------------------------------------------------------------------ weights
// One 128 x 128 block of W a thread block, as the operands [N][K] and [K][N].
template <typename T>
__global__ void __launch_bounds__(kThreads) k11_weight(const T* __restrict__ w, int N, int K, uint8_t* __restrict__ out, uint8_t* __restrict__ out_t) {
  __shared__ uint8_t tile[kSide][kSide + 4];
  __shared__ uint32_t tops[kThreads / 32];
  const Operand8 o{N, K}, ot{K, N};
  const int n0 = blockIdx.y * kSide, k0 = blockIdx.x * kSide;
  const int k = k0 + threadIdx.x % 128, half = threadIdx.x / 128;
  float v[64];
  uint32_t top = 0;
#pragma unroll
  for (int r = 0; r < 64; ++r) {
    const int n = n0 + half * 64 + r;
    v[r] = n < N && k < K ? to_f32(w[static_cast<size_t>(n) * K + k]) : 0.f;
    const uint32_t bits = __float_as_uint(v[r]) & 0x7fffffffu;
    if (bits < 0x7f800000u) top = max(top, bits);
    v[r] = no_infinity(v[r]);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
  for (int q = 0; q < kThreads / 32; ++q) top = max(top, tops[q]);
  const uint32_t byte = scale_byte(top);
  const float inv = over_scale(byte);
#pragma unroll
  for (int r = 0; r < 64; ++r)
    tile[half * 64 + r][threadIdx.x % 128] = static_cast<uint8_t>(__nv_cvt_float_to_fp8(v[r] * inv, __NV_SATFINITE, __NV_E4M3));
  __syncthreads();
  for (int i = threadIdx.x; i < kSide * kSide; i += kThreads) {
    const int a = i / kSide, b = i % kSide;
    if (n0 + a < N && k0 + b < K) out[static_cast<size_t>(n0 + a) * o.ld() + k0 + b] = tile[a][b];
    if (k0 + a < K && n0 + b < N) out_t[static_cast<size_t>(k0 + a) * ot.ld() + n0 + b] = tile[b][a];
  }
  if (threadIdx.x < kSide) {
    const int n = n0 + threadIdx.x, kk = k0 + threadIdx.x;
    if (n < N) out[o.scales_at() + o.scale_at(n, blockIdx.x)] = static_cast<uint8_t>(byte);
    if (kk < K) out_t[ot.scales_at() + ot.scale_at(kk, blockIdx.y)] = static_cast<uint8_t>(byte);
  }
}

// ------------------------------------------------------------------ sums of slices
__global__ void __launch_bounds__(kThreads) k11_join(const float* __restrict__ part, int n_z, long long n, float* __restrict__ out) {
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
  for (int z = 0; z < n_z; ++z) s += part[z * n + i];
  out[i] = s;
}

}  // namespace

cudaError_t launch_quantize_rows(const uint16_t* x, long long rows, int depth, uint8_t* out, int* status, int num_sms, cudaStream_t s) {
  const Operand8 o{rows, depth};
  const uint32_t per_row = static_cast<uint32_t>(l8_blocks(depth));
  const long long items = rows * per_row, per_block = kThreads / 16 * kTurns;
  const int grid = static_cast<int>(std::max<long long>(1, std::min<long long>((items + per_block - 1) / per_block, 8ll * num_sms)));
  k11_rows<<<grid, kThreads, 0, s>>>(x, o, items, per_row, out, status);
  return cudaGetLastError();
}

int quantize_columns_parts(long long rows, int cols, int num_sms) {
  const long long across = l8_blocks(cols);
  return static_cast<int>(std::max<long long>(1, std::min<long long>(l8_blocks(rows), 4ll * num_sms / across)));
}

cudaError_t launch_quantize_columns(const uint16_t* x, long long rows, int cols, uint8_t* out, uint8_t* by_rows,
                                    float* column_sums, float* part, int* status, int num_sms, cudaStream_t s) {
  const int parts = quantize_columns_parts(rows, cols, num_sms);
  const dim3 grid(static_cast<unsigned>(l8_blocks(cols)), parts);
  auto kernel = by_rows ? (column_sums ? k11_columns<true, true> : k11_columns<true, false>)
                        : (column_sums ? k11_columns<false, true> : k11_columns<false, false>);
  kernel<<<grid, kThreads, 0, s>>>(x, rows, cols, out, by_rows, part, parts, status);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess && column_sums ? launch_join(part, parts, cols, column_sums, s) : e;
}

cudaError_t launch_quantize_weight(const void* w, bool f32, int N, int K, uint8_t* out, uint8_t* out_t, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(l8_blocks(K)), static_cast<unsigned>(l8_blocks(N)));
  if (f32)
    k11_weight<<<grid, kThreads, 0, s>>>(static_cast<const float*>(w), N, K, out, out_t);
  else
    k11_weight<<<grid, kThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(w), N, K, out, out_t);
  return cudaGetLastError();
}

cudaError_t launch_join(const float* part, int n_z, long long n, float* out, cudaStream_t s) {
  k11_join<<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(part, n_z, n, out);
  return cudaGetLastError();
}

}  // namespace trimul
