// k9_grad_clip.cu -- the norm over many tensors, and clipping by it.
//
//   norm = sqrt(sum g^2) or max |g|,   out = g min(1, max_norm / (norm + 1e-6))
//
// Two kernels: the first reads every element and leaves one number a block;
// every block of the second adds these up in the same order and scales its
// part of the tensors.  The tensors are cut into chunks of kChunk elements; a
// table of them travels in the launch's parameters, so nothing is copied to
// the device and a captured launch keeps its own table.  Bound by memory: one
// read for the norm, a read and a write to scale.
#include <algorithm>

#include "pair_ops.cuh"

namespace trimul {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;
constexpr int kTableMax = 1000;  // tensors of one launch: 32 bytes each of the 32764 bytes of parameters

struct Entry {
  const void* data;
  void* out;
  long long numel;
  uint32_t chunk;  // the tensor's first chunk of the launch
  int type;
};
struct Table {
  int n;
  uint32_t chunks;
  Entry t[kTableMax];
};
static_assert(sizeof(Table) + 64 <= 32764, "the table and the other arguments fit a launch's parameters");

// The entry that holds a chunk: the last with t[k].chunk <= chunk (tensors without elements have no chunk).
__device__ __forceinline__ int entry_of(const Table& tab, uint32_t chunk) {
  int lo = 0, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (tab.t[mid].chunk <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// A square that is summed in fp32 must neither overflow nor vanish: elements
// outside [2^-40, 2^60] are squared in fp64.
template <typename T>
__device__ __forceinline__ void take(const T* p, long long i, int kind, float& f, double& w, unsigned& top) {
  const float v = fabsf(to_f32(p[i]));
  if (kind == TRIMUL_NORM_INF)
    top = max(top, __float_as_uint(v));  // the bits of a NaN are above infinity's
  else if (v <= 0x1p60f && v >= 0x1p-40f)
    f += v * v;
  else
    w += static_cast<double>(v) * v;
}

__global__ void __launch_bounds__(kThreads) k9_norm(const __grid_constant__ Table tab, int kind, double* part) {
  double w = 0.0;
  unsigned top = 0;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    const Entry& t = tab.t[entry_of(tab, chunk)];
    const long long i0 = static_cast<long long>(chunk - t.chunk) * kChunk;
    const long long i1 = min(t.numel, i0 + kChunk);
    float f = 0.f;
    for (long long i = i0 + threadIdx.x; i < i1; i += kThreads) {
      if (t.type == TRIMUL_F32)
        take(static_cast<const float*>(t.data), i, kind, f, w, top);
      else if (t.type == TRIMUL_BF16)
        take(static_cast<const __nv_bfloat16*>(t.data), i, kind, f, w, top);
      else
        take(static_cast<const __half*>(t.data), i, kind, f, w, top);
    }
    w += f;
  }
  __shared__ double s[kThreads];
  s[threadIdx.x] = kind == TRIMUL_NORM_INF ? static_cast<double>(__uint_as_float(top)) : w;
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < o) {
      const double u = s[threadIdx.x], v = s[threadIdx.x + o];
      s[threadIdx.x] = kind != TRIMUL_NORM_INF ? u + v : (u != u || u > v) ? u : v;
    }
  }
  if (threadIdx.x == 0) part[blockIdx.x] = s[0];
}

// The norm from the blocks' numbers, the same in every block.
__device__ __forceinline__ double total_norm(const double* part, int parts, int kind) {
  __shared__ double s[kThreads];
  double w = 0.0;
  for (int k = threadIdx.x; k < parts; k += kThreads) {
    const double v = part[k];
    w = kind != TRIMUL_NORM_INF ? w + v : (w != w || w > v) ? w : v;
  }
  s[threadIdx.x] = w;
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < o) {
      const double u = s[threadIdx.x], v = s[threadIdx.x + o];
      s[threadIdx.x] = kind != TRIMUL_NORM_INF ? u + v : (u != u || u > v) ? u : v;
    }
  }
  __syncthreads();
  return kind == TRIMUL_NORM_INF ? s[0] : sqrt(s[0]);
}

template <typename T>
__device__ __forceinline__ void scale(const Entry& t, long long i0, long long i1, float coef) {
  for (long long i = i0 + threadIdx.x; i < i1; i += kThreads) {
    const T v = static_cast<const T*>(t.data)[i];
    static_cast<T*>(t.out)[i] = coef == 1.0f ? v : from_f32<T>(to_f32(v) * coef);
  }
}

__global__ void __launch_bounds__(kThreads)
    k9_scale(const __grid_constant__ Table tab, int kind, const double* part, int parts, float max_norm, float* norm,
             int write) {
  const double n = total_norm(part, parts, kind);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(n);
  if (!write) return;
  const double share = static_cast<double>(max_norm) / (n + 1e-6);
  // a norm that is not finite (inf - inf and NaN - NaN are NaN) scales nothing
  const float coef = (n - n == 0.0 && share < 1.0) ? static_cast<float>(share) : 1.0f;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    const Entry& t = tab.t[entry_of(tab, chunk)];
    if (coef == 1.0f && t.data == t.out) continue;
    const long long i0 = static_cast<long long>(chunk - t.chunk) * kChunk;
    const long long i1 = min(t.numel, i0 + kChunk);
    if (t.type == TRIMUL_F32)
      scale<float>(t, i0, i1, coef);
    else if (t.type == TRIMUL_BF16)
      scale<__nv_bfloat16>(t, i0, i1, coef);
    else
      scale<__half>(t, i0, i1, coef);
  }
}

constexpr int kBlocksPerSm = 4;

}  // namespace

size_t grad_workspace(int n, int num_sms) {
  const size_t launches = std::max(1, (n + kTableMax - 1) / kTableMax);
  return launches * kBlocksPerSm * num_sms * sizeof(double);
}

cudaError_t launch_grad_norm(const trimul_grad_tensor* t, int n, trimul_norm_kind kind, float* norm, void* ws,
                             bool clip, float max_norm, int num_sms, cudaStream_t s) {
  double* const part = static_cast<double*>(ws);
  int parts = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int k = 0;
    do {
      Table tab;
      tab.n = 0;
      tab.chunks = 0;
      for (; k < n && tab.n < kTableMax; ++k) {
        if (t[k].numel == 0) continue;
        tab.t[tab.n++] = Entry{t[k].data, t[k].out, static_cast<long long>(t[k].numel), tab.chunks, t[k].type};
        tab.chunks += static_cast<uint32_t>((t[k].numel + kChunk - 1) / kChunk);
      }
      const int grid = static_cast<int>(std::max<long long>(1, std::min<long long>(tab.chunks, kBlocksPerSm * num_sms)));
      if (pass == 0) {
        k9_norm<<<grid, kThreads, 0, s>>>(tab, kind, part + parts);
        parts += grid;
      } else {
        k9_scale<<<clip ? grid : 1, kThreads, 0, s>>>(tab, kind, part, parts, max_norm, norm, clip ? 1 : 0);
      }
      cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    } while (k < n && (pass == 0 || clip));
  }
  return cudaSuccess;
}

}  // namespace trimul
