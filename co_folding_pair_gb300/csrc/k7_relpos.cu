// k7_relpos.cu -- relative position bias by buckets, and its table's gradient.
//
//   out[b,i,j,:] = base[b,i,j,:] + table[bucket(q_pos[b,i] - k_pos[b,j])]
//   dtable[n,:]  = sum of dout[b,i,j,:] over the pairs of bucket n
//
// The bucket of every distance within [-M, M] is a table of 16-bit numbers
// made when the plan is made; farther distances have the bucket of -M or M.
// Both directions are one pass over B I J D elements (the forward writes them,
// and reads them if there is a base; the gradient reads them), so both are
// bound by memory.
#include <algorithm>

#include "pair_ops.cuh"

namespace trimul {

namespace {

// One thread per eight channels of a pair, over all pairs.
template <typename T, typename Tab>
__global__ void __launch_bounds__(256)
    k7_relpos_pair(RelposArgs a, const Tab* __restrict__ table, const T* base, T* out, long long chunks, int per_pair) {
  for (long long n = blockIdx.x * 256ll + threadIdx.x; n < chunks; n += gridDim.x * 256ll) {
    const uint32_t pair = static_cast<uint32_t>(n / per_pair), c = static_cast<uint32_t>(n % per_pair);
    uint32_t row, j;
    a.by_J.divmod(pair, row, j);
    const int k = relpos_bucket(a, row, a.by_I.div(row) * a.J + j);
    float v[8] = {}, z[8];
    if (k >= 0) load8(table + static_cast<size_t>(k) * a.D + c * 8, v);
    if (base) {
      load8(base + n * 8, z);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += z[e];
    }
    store8(out + n * 8, v);
  }
}

// One thread per element of [B][H][I][J].
template <typename T, typename Tab>
__global__ void __launch_bounds__(256)
    k7_relpos_heads(RelposArgs a, const Tab* __restrict__ table, const T* base, T* out, long long n_out, FastDiv by_H) {
  for (long long n = blockIdx.x * 256ll + threadIdx.x; n < n_out; n += gridDim.x * 256ll) {
    const long long line = n / a.J;  // (b H + h) I + i
    const uint32_t j = static_cast<uint32_t>(n - line * a.J);
    const long long bh = line / a.I;
    const uint32_t i = static_cast<uint32_t>(line - bh * a.I);
    uint32_t b, h;
    by_H.divmod(static_cast<uint32_t>(bh), b, h);
    const int k = relpos_bucket(a, b * a.I + i, b * a.J + j);
    float v = k >= 0 ? to_f32(table[static_cast<size_t>(k) * a.D + h]) : 0.f;
    if (base) v += to_f32(base[n]);
    out[n] = from_f32<T>(v);
  }
}

// ------------------------------------------------------------------ gradient
// Each block adds up a range of pairs in shared memory, [rows][channels of the
// block], and writes its sums; k7_relpos_sum adds the blocks' sums in order.
constexpr int kSumBytes = 200 * 1024;  // shared memory for the sums

// One thread per channel; a block takes a slice of the channels and a range of pairs.
template <typename T>
__global__ void k7_relpos_grad_pair(RelposArgs a, const T* __restrict__ dout, float* part, uint32_t pairs) {
  extern __shared__ float sums[];
  const int W = blockDim.x, c = blockIdx.y * W + threadIdx.x;
  for (int r = 0; r < a.rows; ++r) sums[r * W + threadIdx.x] = 0.f;
  const uint32_t p0 = static_cast<uint32_t>(static_cast<unsigned long long>(pairs) * blockIdx.x / gridDim.x);
  const uint32_t p1 = static_cast<uint32_t>(static_cast<unsigned long long>(pairs) * (blockIdx.x + 1) / gridDim.x);
  if (c >= a.D) return;
  int at = -1;
  float run = 0.f;
  for (uint32_t p = p0; p < p1; ++p) {
    uint32_t row, j;
    a.by_J.divmod(p, row, j);
    const int k = relpos_bucket(a, row, a.by_I.div(row) * a.J + j);
    if (k < 0) continue;
    if (k != at) {
      if (at >= 0) sums[at * W + threadIdx.x] += run;
      at = k;
      run = 0.f;
    }
    run += to_f32(dout[static_cast<size_t>(p) * a.D + c]);
  }
  if (at >= 0) sums[at * W + threadIdx.x] += run;
  for (int r = 0; r < a.rows; ++r)
    part[(static_cast<size_t>(blockIdx.x) * a.rows + r) * a.D + c] = sums[r * W + threadIdx.x];
}

// One warp per head and range of pairs; every lane has its own column of sums.
template <typename T>
__global__ void __launch_bounds__(32)
    k7_relpos_grad_heads(RelposArgs a, const T* __restrict__ dout, float* part, uint32_t pairs, FastDiv by_plane) {
  extern __shared__ float sums[];
  const int lane = threadIdx.x, h = blockIdx.y;
  for (int r = 0; r < a.rows; ++r) sums[r * 32 + lane] = 0.f;
  const uint32_t p0 = static_cast<uint32_t>(static_cast<unsigned long long>(pairs) * blockIdx.x / gridDim.x);
  const uint32_t p1 = static_cast<uint32_t>(static_cast<unsigned long long>(pairs) * (blockIdx.x + 1) / gridDim.x);
  for (uint32_t p = p0 + lane; p < p1; p += 32) {
    uint32_t b, at, row, j;
    by_plane.divmod(p, b, at);
    a.by_J.divmod(p, row, j);
    const int k = relpos_bucket(a, row, b * a.J + j);
    if (k < 0) continue;
    sums[k * 32 + lane] += to_f32(dout[(static_cast<size_t>(b) * a.D + h) * by_plane.d + at]);
  }
  __syncwarp();
  for (int r = lane; r < a.rows; r += 32) {
    float t = 0.f;
    for (int l = 0; l < 32; ++l) t += sums[r * 32 + ((l + lane) & 31)];
    part[(static_cast<size_t>(blockIdx.x) * a.rows + r) * a.D + h] = t;
  }
}

__global__ void __launch_bounds__(256)
    k7_relpos_sum(const float* __restrict__ part, float* dtable, int n, int parts, int accumulate) {
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  float t = 0.f;
  for (int k = 0; k < parts; ++k) t += part[static_cast<size_t>(k) * n + e];
  dtable[e] = accumulate ? dtable[e] + t : t;
}

// Ranges of pairs (blocks) of a gradient, and the channels of a block.
void grad_split(int rows, int B, int I, int J, int D, trimul_layout layout, int num_sms, int* ranges, int* width) {
  const long long pairs = static_cast<long long>(B) * I * J;
  *width = layout == TRIMUL_LAYOUT_HEADS ? 1 : std::min(D, std::max(1, kSumBytes / (rows * 4)));
  const int slices = (D + *width - 1) / *width;
  *ranges = static_cast<int>(std::max<long long>(1, std::min<long long>(pairs / 64, std::max(1, 4 * num_sms / slices))));
}

template <typename T, typename Tab>
cudaError_t forward(const RelposArgs& a, const void* table, const void* base, void* out, trimul_layout layout,
                    int num_sms, cudaStream_t s) {
  const long long elems = static_cast<long long>(a.B) * a.I * a.J * a.D;
  const long long work = layout == TRIMUL_LAYOUT_PAIR ? elems / 8 : elems;
  const int grid = static_cast<int>(std::min<long long>((work + 255) / 256, 8ll * num_sms));
  if (layout == TRIMUL_LAYOUT_PAIR)
    k7_relpos_pair<T, Tab><<<grid, 256, 0, s>>>(a, static_cast<const Tab*>(table), static_cast<const T*>(base),
                                                static_cast<T*>(out), work, a.D / 8);
  else
    k7_relpos_heads<T, Tab><<<grid, 256, 0, s>>>(a, static_cast<const Tab*>(table), static_cast<const T*>(base),
                                                 static_cast<T*>(out), work, FastDiv(a.D));
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const RelposArgs& a, const void* dout, trimul_layout layout, float* dtable, bool accumulate,
                     float* ws, int num_sms, cudaStream_t s) {
  int ranges, width;
  grad_split(a.rows, a.B, a.I, a.J, a.D, layout, num_sms, &ranges, &width);
  const uint32_t pairs = static_cast<uint32_t>(a.B) * a.I * a.J;
  const dim3 grid(ranges, (a.D + width - 1) / width);
  if (layout == TRIMUL_LAYOUT_PAIR) {
    const int smem = a.rows * width * 4;
    cudaError_t e = cudaFuncSetAttribute(k7_relpos_grad_pair<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSumBytes);
    if (e != cudaSuccess) return e;
    k7_relpos_grad_pair<T><<<grid, width, smem, s>>>(a, static_cast<const T*>(dout), ws, pairs);
  } else {
    const int smem = a.rows * 32 * 4;
    cudaError_t e = cudaFuncSetAttribute(k7_relpos_grad_heads<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kRelposMaxRows * 32 * 4);
    if (e != cudaSuccess) return e;
    k7_relpos_grad_heads<T><<<grid, 32, smem, s>>>(a, static_cast<const T*>(dout), ws, pairs,
                                                   FastDiv(static_cast<uint32_t>(a.I) * a.J));
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int n = a.rows * a.D;
  k7_relpos_sum<<<(n + 255) / 256, 256, 0, s>>>(ws, dtable, n, ranges, accumulate ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_relpos_forward(const RelposArgs& a, const void* table, bool table_f32, const void* base, void* out,
                                  bool f32, trimul_layout layout, int num_sms, cudaStream_t s) {
  if (f32)
    return table_f32 ? forward<float, float>(a, table, base, out, layout, num_sms, s)
                     : forward<float, __nv_bfloat16>(a, table, base, out, layout, num_sms, s);
  return table_f32 ? forward<__nv_bfloat16, float>(a, table, base, out, layout, num_sms, s)
                   : forward<__nv_bfloat16, __nv_bfloat16>(a, table, base, out, layout, num_sms, s);
}

size_t relpos_backward_workspace(int rows, int B, int I, int J, int D, trimul_layout layout, bool f32, int num_sms) {
  int ranges, width;
  grad_split(rows, B, I, J, D, layout, num_sms, &ranges, &width);
  return static_cast<size_t>(ranges) * rows * D * sizeof(float);
}

cudaError_t launch_relpos_backward(const RelposArgs& a, const void* dout, bool f32, trimul_layout layout,
                                   float* dtable, bool accumulate, float* ws, int num_sms, cudaStream_t s) {
  return f32 ? backward<float>(a, dout, layout, dtable, accumulate, ws, num_sms, s)
             : backward<__nv_bfloat16>(a, dout, layout, dtable, accumulate, ws, num_sms, s);
}

}  // namespace trimul
