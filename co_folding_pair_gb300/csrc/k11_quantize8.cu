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
#include <algorithm>

#include "linear8.h"
#include "quantize8.cuh"

namespace trimul {

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ rows
// Eight lanes have a block of 128: two 16-byte loads each, 64 columns apart.  A
// thread block has whole rows, so that the place of a block among them is a
// 32-bit division.
constexpr int kGroup = 8;                       // lanes of a block of 128
constexpr int kPerTurn = kThreads / kGroup;
constexpr int kTurns = 2;                       // blocks of a thread that are on their way together
__global__ void __launch_bounds__(kThreads, 6)
    k11_rows(const uint16_t* __restrict__ x, long long rows, int depth, uint32_t ld, uint32_t groups, FastDiv per_row,
             uint8_t* __restrict__ out, uint8_t* __restrict__ scales, int* status) {
  let_next_begin();
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  const long long r0 = rows * blockIdx.x / gridDim.x, r1 = rows * (blockIdx.x + 1) / gridDim.x;
  const uint32_t items = static_cast<uint32_t>(r1 - r0) * per_row.d;
  const uint16_t* const from = x + r0 * depth;
  uint8_t* const to = out + r0 * ld;
  const int lane = threadIdx.x % kGroup;
  for (uint32_t at = 0; at < items; at += kPerTurn * kTurns) {  // (all lanes of a warp: the shuffles need them)
    uint4 v[kTurns][2];
    uint32_t row[kTurns], block[kTurns];
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const uint32_t item = at + u * kPerTurn + threadIdx.x / kGroup;
      per_row.divmod(item, row[u], block[u]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t col = block[u] * L8_BLOCK + h * 64 + lane * 8;
        v[u][h] = make_uint4(0u, 0u, 0u, 0u);
        if (item < items && col < depth) v[u][h] = __ldcs(reinterpret_cast<const uint4*>(from + static_cast<size_t>(row[u]) * depth + col));
      }
    }
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      uint32_t top = over_lanes<kGroup>(max_magnitude(v[u][0], v[u][1]));
      const bool fine = top < 0x7f80u;
      if (__any_sync(0xffffffffu, !fine))  // rare
        top = over_lanes<kGroup>(max16x2(max_of(finite(v[u][0])), max_of(finite(v[u][1]))));
      const uint32_t byte = scale_byte(top << 16);
      if (at + u * kPerTurn + threadIdx.x / kGroup >= items) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t col = block[u] * L8_BLOCK + h * 64 + lane * 8;
        if (col < depth) *reinterpret_cast<uint2*>(to + static_cast<size_t>(row[u]) * ld + col) = codes_of(v[u][h], over_scale(byte), fine);
      }
      if (lane == 0) scales[l8_scale_at(r0 + row[u], block[u], groups)] = static_cast<uint8_t>(byte);
    }
  }
}

// ------------------------------------------------------------------ columns
// A thread block takes 128 x 128 tiles below one another.  Sixteen lanes have a
// row's 128 columns, eight each, and sixteen groups of lanes have eight rows
// each: a thread keeps its 8 x 8 numbers in registers, the columns' largest
// magnitudes are taken over its rows, over the warp's two groups and, through
// shared memory, over the warps; then the codes leave the way the numbers came.
constexpr int kSide = 128;
constexpr int kWarps = kThreads / 32;

template <bool kRows, bool kSums>
__global__ void __launch_bounds__(kThreads, kRows && kSums ? 2 : 3)
    k11_columns(const uint16_t* __restrict__ x, long long rows, int cols, uint32_t ld, uint32_t groups, uint8_t* __restrict__ out,
                uint8_t* __restrict__ scales, uint32_t row_groups, uint8_t* __restrict__ by_rows, uint8_t* __restrict__ row_scales,
                float* __restrict__ part, int parts, int* status) {
  let_next_begin();
  after_previous();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && status) *status = 0;
  __shared__ uint4 tops[2][kWarps][16];
  __shared__ float sums[kSums ? kWarps : 1][kSums ? kSide : 1];
  const int lane16 = threadIdx.x % 16, warp = threadIdx.x / 32, group = threadIdx.x / 16;
  const int col = blockIdx.x * kSide + lane16 * 8;
  const bool inside = col < cols;  // of a multiple of eight: all eight or none
  const long long tiles = l8_blocks(rows);
  // a thread's sums wait in shared memory: in registers, two blocks an SM, 2^20 rows of 256 columns take 206 us for 162
  __shared__ ulonglong2 own[kSums ? 2 : 1][kSums ? kThreads : 1];
  if (kSums) own[0][threadIdx.x] = own[1][threadIdx.x] = make_ulonglong2(0, 0);
  int turn = 0;
  for (long long rt = blockIdx.y; rt < tiles; rt += parts, turn ^= 1) {
    const long long r0 = rt * kSide + group;  // rows 16 apart
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (inside && r0 + u * 16 < rows) v[u] = __ldcs(reinterpret_cast<const uint4*>(x + (r0 + u * 16) * cols + col));
    }
    uint4 top = v[0];
    auto join = [](uint4& a, const uint4& b) {
      a.x = max16x2(a.x, b.x), a.y = max16x2(a.y, b.y), a.z = max16x2(a.z, b.z), a.w = max16x2(a.w, b.w);
    };
#pragma unroll
    for (int u = 1; u < 8; ++u)
      top = make_uint4(max_signed(top.x, v[u].x), max_signed(top.y, v[u].y), max_signed(top.z, v[u].z), max_signed(top.w, v[u].w));
    top = magnitudes(top);
    const uint32_t all = max_of(top);
    const bool fine = (all & 0xffffu) < 0x7f80u && all < 0x7f800000u;
    if (!fine) {  // rare
      top = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int u = 0; u < 8; ++u) join(top, finite(v[u]));
    }
    join(top, make_uint4(__shfl_xor_sync(0xffffffffu, top.x, 16), __shfl_xor_sync(0xffffffffu, top.y, 16),
                         __shfl_xor_sync(0xffffffffu, top.z, 16), __shfl_xor_sync(0xffffffffu, top.w, 16)));
    if (threadIdx.x % 32 < 16) tops[turn][warp][lane16] = top;
    if (kSums) {
      const ulonglong2 a = own[0][threadIdx.x], b = own[1][threadIdx.x];
      f2 sum[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
      for (int u = 0; u < 8; ++u) add_row(sum, v[u]);
      own[0][threadIdx.x] = make_ulonglong2(sum[0], sum[1]), own[1][threadIdx.x] = make_ulonglong2(sum[2], sum[3]);
    }
    if (kRows) {
#pragma unroll
      for (int u = 0; u < 8; u += 2) {  // two rows' largest in a register
        auto over_rows = [&](uint32_t a, uint32_t b) {
          uint32_t two = max16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) two = max16x2(two, __shfl_xor_sync(0xffffffffu, two, o));
          return two;
        };
        uint32_t two = over_rows(max_signed(v[u]) & 0x7fff7fffu, max_signed(v[u + 1]) & 0x7fff7fffu);
        const bool row_fine[2] = {(two & 0xffffu) < 0x7f80u, two < 0x7f800000u};
        if (__any_sync(0xffffffffu, !(row_fine[0] && row_fine[1]))) two = over_rows(max_of(finite(v[u])), max_of(finite(v[u + 1])));  // rare
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t byte = scale_byte(h ? two & 0xffff0000u : two << 16);
          const long long r = r0 + (u + h) * 16;
          if (r < rows) {
            if (inside) *reinterpret_cast<uint2*>(by_rows + r * ld + col) = codes_of(v[u + h], over_scale(byte), row_fine[h]);
            if (lane16 == 0) row_scales[l8_scale_at(r, blockIdx.x, row_groups)] = static_cast<uint8_t>(byte);
          }
        }
      }
    }
    __syncthreads();  // (the other half of `tops` is written next: one meeting a tile is enough)
#pragma unroll
    for (int q = 0; q < kWarps; ++q) join(top, tops[turn][q][lane16]);
    const uint32_t word[4] = {top.x, top.y, top.z, top.w};
    f2 inv[4];
    uint32_t byte[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      byte[2 * e] = scale_byte(word[e] << 16), byte[2 * e + 1] = scale_byte(word[e] & 0xffff0000u);
      inv[e] = pair2(over_scale(byte[2 * e]), over_scale(byte[2 * e + 1]));
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (inside && r0 + u * 16 < rows) *reinterpret_cast<uint2*>(out + (r0 + u * 16) * ld + col) = codes_of(v[u], inv, fine);
    if (group < 8 && inside) {  // group g stores column g's byte of the lane's eight
      uint32_t mine = byte[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) mine = group == e ? byte[e] : mine;
      scales[l8_scale_at(col + group, rt, groups)] = static_cast<uint8_t>(mine);
    }
  }
  if (kSums) {  // in a fixed order: a thread's rows, the warp's two groups, the warps, then the blocks (k11_join)
    const ulonglong2 a = own[0][threadIdx.x], b = own[1][threadIdx.x];
    const f2 sum[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = split2(sum[e]);
      const float lo = f.x + __shfl_xor_sync(0xffffffffu, f.x, 16), hi = f.y + __shfl_xor_sync(0xffffffffu, f.y, 16);
      if (threadIdx.x % 32 < 16) sums[warp][lane16 * 8 + 2 * e] = lo, sums[warp][lane16 * 8 + 2 * e + 1] = hi;
    }
    __syncthreads();
    if (threadIdx.x < kSide && blockIdx.x * kSide + threadIdx.x < cols) {
      float t = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) t += sums[q][threadIdx.x];
      part[static_cast<size_t>(blockIdx.y) * cols + blockIdx.x * kSide + threadIdx.x] = t;
    }
  }
}

// ------------------------------------------------------------------ weights
// One 128 x 128 block of W a thread block, 8 x 8 numbers a thread as above.
__device__ __forceinline__ void load8(const float* p, bool wide, float (&f)[8]) {
  if (wide) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = p[e];
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, bool wide, float (&f)[8]) {
  if (wide) {
    unpack8(*reinterpret_cast<const uint4*>(p), f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __bfloat162float(p[e]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k11_weight(const T* __restrict__ w, int N, int K, uint32_t ld, uint32_t groups, uint32_t groups_mn,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                        uint8_t* __restrict__ scales_mn) {
  __shared__ uint32_t tops[kWarps];
  const int lane16 = threadIdx.x % 16, group = threadIdx.x / 16;
  const int k = blockIdx.x * kSide + lane16 * 8, n0 = blockIdx.y * kSide + group;
  const bool wide = reinterpret_cast<uintptr_t>(w) % 16 == 0;
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] = 0.f;
    if (n0 + u * 16 < N && k < K) load8(w + static_cast<size_t>(n0 + u * 16) * K + k, wide, v[u]);
  }
#pragma unroll
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t bits = __float_as_uint(v[u][e]) & 0x7fffffffu;
      top = max(top, bits < 0x7f800000u ? bits : 0u);
    }
  top = __reduce_max_sync(0xffffffffu, top);
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kWarps; ++q) top = max(top, tops[q]);
  const uint32_t byte = scale_byte(top);
  const float inv = over_scale(byte);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = no_infinity(v[u][e]) * inv;
    if (n0 + u * 16 < N && k < K)
      *reinterpret_cast<uint2*>(codes + static_cast<size_t>(n0 + u * 16) * ld + k) = make_uint2(codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7]));
  }
  if (threadIdx.x < kSide) {
    const int n = blockIdx.y * kSide + threadIdx.x, kk = blockIdx.x * kSide + threadIdx.x;
    if (n < N) scales[l8_scale_at(n, blockIdx.x, groups)] = static_cast<uint8_t>(byte);
    if (kk < K) scales_mn[l8_scale_at(kk, blockIdx.y, groups_mn)] = static_cast<uint8_t>(byte);
  }
}

// ------------------------------------------------------------------ sums of slices
// kEach threads a sum: each adds every kEach-th slice, and they are added in order.
// Few sums of many slices take eight (with one, the loads of a hundred slices come one after the other: 13 us for
// 512 sums, 5.4 with eight); many take one (262144 sums of 76 slices: 8 us, with eight 18.6).
template <int kEach>
__device__ __forceinline__ void join(const Join8& a, long long block, float* sums) {
  constexpr int kSums = kThreads / kEach;
  const int lane = threadIdx.x % kSums, q = threadIdx.x / kSums;
  const long long i = block * kSums + lane;
  float s = 0.f;
  if (i < a.n) {
#pragma unroll 8
    for (int z = q; z < a.n_z; z += kEach) s += a.part[z * a.n + i];
  }
  if (kEach > 1) {
    sums[q * kSums + lane] = s;
    __syncthreads();
    if (q != 0) return;
#pragma unroll
    for (int k = 1; k < kEach; ++k) s += sums[k * kSums + lane];
  }
  if (i < a.n) a.out[a.cols ? i % a.cols * (a.n / a.cols) + i / a.cols : i] = s;
}
template <int kEach>
__global__ void __launch_bounds__(kThreads) k11_join(const Join8 a, const Join8 few, unsigned blocks_a) {
  __shared__ float sums[kThreads];
  after_previous();
  if (blockIdx.x < blocks_a)
    join<kEach>(a, blockIdx.x, sums);
  else
    join<8>(few, blockIdx.x - blocks_a, sums);
}

// ------------------------------------------------------------------ sums of columns, as k13_fused8.cu takes them
// There a lane adds, of every other block of a slice, rows r, r + 16 .. of 128, and the lanes of r = 0 .. 15 are joined in pairs, by the bits
// of r from the lowest on.  Here a thread has one r and two columns, and a thread block all r of 128 columns.
constexpr int kSumThreads = 1024, kPairs = kSide / 2;
__global__ void __launch_bounds__(kSumThreads) k11_sums(const uint16_t* __restrict__ t, long long rows, int cols, int per_z,
                                                        float* __restrict__ out, int* __restrict__ status) {
  let_next_begin();
  after_previous();
  if (status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  __shared__ float2 sums[16][kPairs];
  const int z = blockIdx.y / 2, odd = blockIdx.y % 2, pair = threadIdx.x % kPairs, r = threadIdx.x / kPairs;
  const int c = blockIdx.x * kSide + 2 * pair;
  const long long blocks = l8_blocks(rows), end = min(static_cast<long long>(z + 1) * per_z, blocks);
  float2 s = make_float2(0.f, 0.f);
#pragma unroll 2
  for (long long b = static_cast<long long>(z) * per_z + odd; b < end; b += 2) {
    uint32_t v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const long long row = b * kSide + r + 16 * u;
      v[u] = row < rows && c < cols ? *reinterpret_cast<const uint32_t*>(t + row * cols + c) : 0u;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) s.x += bf16_lo(v[u]), s.y += bf16_hi(v[u]);
  }
  sums[r][pair] = s;
  __syncthreads();
  if (r != 0 || c >= cols) return;
  float2 all[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) all[k] = sums[k][pair];
#pragma unroll
  for (int n = 8; n > 0; n >>= 1)
#pragma unroll
    for (int k = 0; k < n; ++k) all[k] = make_float2(all[2 * k].x + all[2 * k + 1].x, all[2 * k].y + all[2 * k + 1].y);
  *reinterpret_cast<float2*>(out + static_cast<long long>(blockIdx.y) * cols + c) = all[0];
}

}  // namespace

cudaError_t launch_quantize_rows(const uint16_t* x, long long rows, int depth, uint8_t* out, int* status, int num_sms, cudaStream_t s) {
  const Operand8 o{rows, depth, false};
  const uint32_t per_row = static_cast<uint32_t>(l8_blocks(depth));
  const long long turns = (rows * per_row + kPerTurn * kTurns - 1) / (kPerTurn * kTurns);
  const int grid = static_cast<int>(std::min<long long>(rows, std::min<long long>(turns, 6ll * num_sms)));
  k11_rows<<<grid, kThreads, 0, s>>>(x, rows, depth, static_cast<uint32_t>(o.ld()), static_cast<uint32_t>(o.groups()), FastDiv(per_row), out,
                                     out + o.scales_at(), status);
  return cudaGetLastError();
}

int quantize_columns_parts(long long rows, int cols, int num_sms) {
  const long long across = l8_blocks(cols);
  return static_cast<int>(std::max<long long>(1, std::min<long long>(l8_blocks(rows), 3ll * num_sms / across)));
}

cudaError_t launch_quantize_columns(const uint16_t* x, long long rows, int cols, uint8_t* out, uint8_t* by_rows,
                                    float* column_sums, float* part, int* status, int num_sms, cudaStream_t s) {
  const Operand8 c{cols, rows, true}, r{rows, cols, false};
  const int parts = quantize_columns_parts(rows, cols, num_sms);
  const dim3 grid(static_cast<unsigned>(l8_blocks(cols)), parts);
  auto kernel = by_rows ? (column_sums ? k11_columns<true, true> : k11_columns<true, false>)
                        : (column_sums ? k11_columns<false, true> : k11_columns<false, false>);
  const cudaError_t e = launch8(kernel, grid, kThreads, 0, status == nullptr, s, x, rows, cols, static_cast<uint32_t>(c.ld()),
                                static_cast<uint32_t>(c.groups()), out, out + c.scales_at(), static_cast<uint32_t>(r.groups()), by_rows,
                                by_rows ? by_rows + r.scales_at() : nullptr, part, parts, status);
  return e == cudaSuccess && column_sums ? launch_join(Join8{}, Join8{part, parts, cols, 0, column_sums}, s) : e;
}

cudaError_t launch_quantize_weight(const void* w, bool f32, int N, int K, uint8_t* codes, uint8_t* scales, uint8_t* scales_mn,
                                   cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(l8_blocks(K)), static_cast<unsigned>(l8_blocks(N)));
  const Operand8 o{N, K, false}, t{K, N, true};
  const uint32_t ld = static_cast<uint32_t>(o.ld()), g = static_cast<uint32_t>(o.groups()), gt = static_cast<uint32_t>(t.groups());
  if (f32)
    k11_weight<<<grid, kThreads, 0, s>>>(static_cast<const float*>(w), N, K, ld, g, gt, codes, scales, scales_mn);
  else
    k11_weight<<<grid, kThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(w), N, K, ld, g, gt, codes, scales, scales_mn);
  return cudaGetLastError();
}

cudaError_t launch_join(const Join8& a, const Join8& few, cudaStream_t s) {
  const unsigned blocks_few = static_cast<unsigned>((few.n + 31) / 32);
  const bool short_one = a.n < 16384;
  const unsigned blocks = static_cast<unsigned>(short_one ? (a.n + 31) / 32 : (a.n + kThreads - 1) / kThreads);
  return launch8(short_one ? k11_join<8> : k11_join<1>, blocks + blocks_few, kThreads, 0, true, s, a, few, blocks);
}

cudaError_t launch_column_sums(const uint16_t* t, long long rows, int cols, int per_z, int n_z, float* sums, int* status, cudaStream_t s) {
  return launch8(k11_sums, dim3(static_cast<unsigned>(l8_blocks(cols)), 2 * n_z), kSumThreads, 0, status == nullptr, s, t, rows, cols, per_z,
                 sums, status);
}

}  // namespace trimul
