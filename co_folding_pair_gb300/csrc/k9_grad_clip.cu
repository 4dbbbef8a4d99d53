// k9_grad_clip.cu -- the norm over many tensors, and clipping by it.
//
//   norm = sqrt(sum g^2) or max |g|,   out = g min(1, max_norm / (norm + 1e-6))
//
// Two kernels: the first reads every element and leaves one number a block;
// every block of the second adds these up in the same order and scales its
// part of the tensors.  The tensors are cut into chunks of kGroups 16-byte
// groups, and every block has a run of neighbouring chunks; a table of the
// tensors travels in the launch's parameters, so nothing is copied to the
// device and a captured launch keeps its own table.
//
// Bound by memory: one read for the norm, a read and a write to scale.  The
// second kernel goes through each block's run backwards, so that it begins
// with what the first one read last and L2 still holds.
#include <algorithm>

#include "pair_ops.cuh"

namespace trimul {

namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 4;                   // 16-byte loads of a thread that are on their way together
constexpr int kGroups = kThreads * kLoads;  // 16 KB a chunk
constexpr int kBlocksPerSm = 5;
constexpr int kTableSmall = 64, kTableMax = 1000;  // tensors of one launch: 32 bytes each of the 32764 bytes of parameters

struct Entry {
  const void* data;
  void* out;
  long long numel;
  uint32_t chunk;  // the tensor's first chunk of the launch
  int type;
};
template <int N>
struct Table {
  int n;
  uint32_t chunks;
  Entry t[N];
};
static_assert(sizeof(Table<kTableMax>) + 64 <= 32764, "the table and the other arguments fit a launch's parameters");

// The entry that holds a chunk: the last with t[k].chunk <= chunk (only tensors with elements are in the table).
template <int N>
__device__ __forceinline__ int entry_of(const Table<N>& tab, uint32_t chunk) {
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

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 v, float (&f)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ void unpack16<float>(const uint4 v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4 v, float (&f)[8]) {
  unpack8(v, f);
}
template <>
__device__ __forceinline__ void unpack16<__half>(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
    f[2 * e] = p.x, f[2 * e + 1] = p.y;
  }
}
__device__ __forceinline__ uint4 pack16(const float (&f)[4], float) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&f)[8], __nv_bfloat16) { return pack8(f); }
__device__ __forceinline__ uint4 pack16(const float (&f)[8], __half) {
  return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}

// A tensor's elements in 16-byte groups of the address space: group 0 begins
// `skip` elements before the first, and the ends may be less than whole groups.
template <typename T>
struct Groups {
  static constexpr int V = 16 / sizeof(T);
  const T* data;
  long long numel;
  int skip;
  __device__ __forceinline__ explicit Groups(const Entry& t)
      : data(static_cast<const T*>(t.data)), numel(t.numel),
        skip(static_cast<int>(reinterpret_cast<uintptr_t>(t.data) % 16 / sizeof(T))) {}
  __device__ __forceinline__ long long first(long long group) const { return group * V - skip; }
  __device__ __forceinline__ bool whole(long long i) const { return i >= 0 && i + V <= numel; }
  // the group at element i; zeros where it goes past the tensor
  __device__ __forceinline__ uint4 load(long long i) const {
    if (whole(i)) return *reinterpret_cast<const uint4*>(data + i);
    alignas(16) T v[V] = {};
    for (int e = 0; e < V; ++e)
      if (i + e >= 0 && i + e < numel) v[e] = data[i + e];
    return *reinterpret_cast<const uint4*>(v);
  }
};

// ------------------------------------------------------------------ norm
// Squares are summed in fp32 within a thread's part of a chunk (16 or 32
// numbers) and in fp64 from there on.  If an fp32 sum is not finite or below
// 2^-60, elements too large or too small for it may be among them (one whose
// square fp32 loses is below 2^-63, which 2^-60 hides for 32 numbers), and the
// part is summed again in fp64.
template <typename T>
__device__ __forceinline__ void add_chunk(const Entry& t, uint32_t chunk, int kind, double& w, unsigned& top) {
  constexpr int V = 16 / sizeof(T);
  const Groups<T> g(t);
  const long long first = static_cast<long long>(chunk - t.chunk) * kGroups + threadIdx.x;
  uint4 v[kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const long long i = g.first(first + k * kThreads);
    v[k] = i < g.numel ? g.load(i) : make_uint4(0u, 0u, 0u, 0u);
  }
  float f[V];
  if (kind == TRIMUL_NORM_INF) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      unpack16<T>(v[k], f);
#pragma unroll
      for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(fabsf(f[e])));  // a NaN's bits are above infinity's
    }
    return;
  }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    unpack16<T>(v[k], f);
    float q = f[0] * f[0];
#pragma unroll
    for (int e = 1; e < V; ++e) q += f[e] * f[e];
    s += q;
  }
  if (s >= 0x1p-60f && s <= 0x1p126f) {
    w += s;
    return;
  }
  double d = 0.0;
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    if ((v[k].x | v[k].y | v[k].z | v[k].w) == 0u) continue;
    unpack16<T>(v[k], f);
#pragma unroll
    for (int e = 0; e < V; ++e) d += static_cast<double>(f[e]) * f[e];
  }
  w += d;
}

// The block's s[] to s[0]: a sum, or the largest (NaN, if there is one).
__device__ __forceinline__ void block_total(double* s, int kind) {
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < o) {
      const double u = s[threadIdx.x], v = s[threadIdx.x + o];
      s[threadIdx.x] = kind != TRIMUL_NORM_INF ? u + v : (u != u || u > v) ? u : v;
    }
  }
  __syncthreads();
}

// The run of chunks of a block.
__device__ __forceinline__ uint32_t run_begin(uint32_t chunks, uint32_t block) {
  return static_cast<uint32_t>(static_cast<unsigned long long>(chunks) * block / gridDim.x);
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    k9_norm(const __grid_constant__ Table<N> tab, int kind, double* part) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  double w = 0.0;
  unsigned top = 0;
  const uint32_t c0 = run_begin(tab.chunks, blockIdx.x), c1 = run_begin(tab.chunks, blockIdx.x + 1);
  if (c0 < c1) {
    int k = entry_of(tab, c0);
    for (uint32_t chunk = c0; chunk < c1; ++chunk) {
      if (k + 1 < tab.n && tab.t[k + 1].chunk <= chunk) ++k;
      const Entry& t = tab.t[k];
      if (t.type == TRIMUL_F32)
        add_chunk<float>(t, chunk, kind, w, top);
      else if (t.type == TRIMUL_BF16)
        add_chunk<__nv_bfloat16>(t, chunk, kind, w, top);
      else
        add_chunk<__half>(t, chunk, kind, w, top);
    }
  }
  __shared__ double s[kThreads];
  s[threadIdx.x] = kind == TRIMUL_NORM_INF ? static_cast<double>(__uint_as_float(top)) : w;
  block_total(s, kind);
  if (threadIdx.x == 0) part[blockIdx.x] = s[0];
}

// ------------------------------------------------------------------ scale
template <typename T>
__device__ __forceinline__ void scale_chunk(const Entry& t, uint32_t chunk, float coef) {
  constexpr int V = 16 / sizeof(T);
  const Groups<T> g(t);
  T* const out = static_cast<T*>(t.out);
  const long long first = static_cast<long long>(chunk - t.chunk) * kGroups + threadIdx.x;
  const bool alike = reinterpret_cast<uintptr_t>(t.out) % 16 == reinterpret_cast<uintptr_t>(t.data) % 16;
  uint4 v[kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const long long i = g.first(first + k * kThreads);
    v[k] = i < g.numel ? g.load(i) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const long long i = g.first(first + k * kThreads);
    if (i >= g.numel) continue;
    uint4 r = v[k];
    if (coef != 1.0f) {
      float f[V];
      unpack16<T>(r, f);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] *= coef;
      r = pack16(f, T());
    }
    if (alike && g.whole(i)) {
      __stcs(reinterpret_cast<uint4*>(out + i), r);
    } else {
      alignas(16) T one[V];
      *reinterpret_cast<uint4*>(one) = r;
      for (int e = 0; e < V; ++e)
        if (i + e >= 0 && i + e < g.numel) out[i + e] = one[e];
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    k9_scale(const __grid_constant__ Table<N> tab, int kind, const double* part, int parts, float max_norm, float* norm,
             int write) {
  __shared__ double s[kThreads];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double w = 0.0;
  for (int k = threadIdx.x; k < parts; k += kThreads) {
    const double v = part[k];
    w = kind != TRIMUL_NORM_INF ? w + v : (w != w || w > v) ? w : v;
  }
  s[threadIdx.x] = w;
  block_total(s, kind);
  const double n = kind == TRIMUL_NORM_INF ? s[0] : sqrt(s[0]);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(n);
  if (!write) return;
  const double share = static_cast<double>(max_norm) / (n + 1e-6);
  // a norm that is not finite (inf - inf and NaN - NaN are NaN) scales nothing
  const float coef = (n - n == 0.0 && share < 1.0) ? static_cast<float>(share) : 1.0f;
  const uint32_t c0 = run_begin(tab.chunks, blockIdx.x), c1 = run_begin(tab.chunks, blockIdx.x + 1);
  if (c0 >= c1) return;
  int k = entry_of(tab, c1 - 1);
  for (uint32_t chunk = c1; chunk-- > c0;) {
    if (tab.t[k].chunk > chunk) --k;
    const Entry& t = tab.t[k];
    if (coef == 1.0f && t.data == t.out) continue;
    if (t.type == TRIMUL_F32)
      scale_chunk<float>(t, chunk, coef);
    else if (t.type == TRIMUL_BF16)
      scale_chunk<__nv_bfloat16>(t, chunk, coef);
    else
      scale_chunk<__half>(t, chunk, coef);
  }
}

uint32_t chunks_of(const trimul_grad_tensor& t) {
  const long long v = t.type == TRIMUL_F32 ? 4 : 8;
  const long long skip = static_cast<long long>(reinterpret_cast<uintptr_t>(t.data) % 16) * v / 16;
  const long long groups = (t.numel + skip + v - 1) / v;
  return static_cast<uint32_t>((groups + kGroups - 1) / kGroups);
}

int grid_of(uint32_t chunks, int num_sms) {
  return static_cast<int>(std::max<long long>(1, std::min<long long>(chunks, kBlocksPerSm * num_sms)));
}

// Fills a table from t[k] on; k moves past the tensors that are in it.
template <int N>
void fill(Table<N>& tab, const trimul_grad_tensor* t, int n, int& k) {
  tab.n = 0;
  tab.chunks = 0;
  for (; k < n && tab.n < N; ++k) {
    if (t[k].numel == 0) continue;
    tab.t[tab.n++] = Entry{t[k].data, t[k].out, static_cast<long long>(t[k].numel), tab.chunks, t[k].type};
    tab.chunks += chunks_of(t[k]);
  }
}

template <int N>
cudaError_t run(const trimul_grad_tensor* t, int n, trimul_norm_kind kind, float* norm, double* part, bool clip,
                float max_norm, int num_sms, cudaStream_t s) {
  Table<N> tab;
  int parts = 0, k = 0;
  do {
    fill(tab, t, n, k);
    const int grid = grid_of(tab.chunks, num_sms);
    k9_norm<N><<<grid, kThreads, 0, s>>>(tab, kind, part + parts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    parts += grid;
  } while (k < n);
  // the scaling kernel's blocks may be set up while the last norm kernel
  // runs; they wait for its end before they read anything
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  k = 0;
  bool first = true;
  do {
    if (n > N) fill(tab, t, n, k);  // else it is what the norm kernel had
    else k = n;
    cudaLaunchConfig_t c{};
    c.gridDim = clip ? grid_of(tab.chunks, num_sms) : 1;
    c.blockDim = kThreads;
    c.stream = s;
    c.attrs = &early;
    c.numAttrs = first ? 1 : 0;
    first = false;
    cudaError_t e = cudaLaunchKernelEx(&c, k9_scale<N>, tab, static_cast<int>(kind), static_cast<const double*>(part),
                                       parts, max_norm, norm, clip ? 1 : 0);
    if (e != cudaSuccess) return e;
  } while (k < n && clip);
  return cudaSuccess;
}

}  // namespace

size_t grad_workspace(int n, int num_sms) {
  const size_t launches = std::max(1, (n + kTableMax - 1) / kTableMax);
  return launches * kBlocksPerSm * num_sms * sizeof(double);
}

cudaError_t launch_grad_norm(const trimul_grad_tensor* t, int n, trimul_norm_kind kind, float* norm, void* ws,
                             bool clip, float max_norm, int num_sms, cudaStream_t s) {
  double* const part = static_cast<double*>(ws);
  return n <= kTableSmall ? run<kTableSmall>(t, n, kind, norm, part, clip, max_norm, num_sms, s)
                          : run<kTableMax>(t, n, kind, norm, part, clip, max_norm, num_sms, s);
}

}  // namespace trimul
