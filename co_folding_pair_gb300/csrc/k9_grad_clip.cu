// k9_grad_clip.cu -- the norm over many tensors, and clipping by it.
//
//   norm = sqrt(sum g^2) or max |g|,   out = g min(1, max_norm / (norm + 1e-6))
//
// The tensors are cut into chunks of kGroups 16-byte groups; a table of the
// tensors travels in the launch's parameters, so nothing is copied to the
// device and a captured launch keeps its own table.
//
// Two kernels: the first reads every element and leaves one sum a block; every
// block of the second adds these up in the same order and scales its run of
// neighbouring chunks, backwards, so that it begins with what the first one
// read last and asked L2 to keep (out of place, 151 MB: 73.4 us with 64 MB kept
// so, 77.5 with 32, 73.4 with 96, 76.3 with none).  Bound by memory: one read
// for the norm, a read and a write to scale.  (One cluster of eight blocks that keeps a small set in registers
// between the two took as long for ten tensors of 98k values: 5.2 us to 5.3.)
#include <algorithm>

#include "pair_ops.cuh"

namespace trimul {

namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 4;                   // 16-byte loads of a thread that are on their way together
constexpr int kGroups = kThreads * kLoads;  // 16 KB a chunk
constexpr uint32_t kKeep = 4096;            // chunks (64 MB) that the first kernel asks L2 to keep for the second
constexpr int kBlocksPerSm = 5, kMostBlocks = 1024;
constexpr int kTableSmall = 64, kTableMax = 1000;  // tensors of one launch

// The tensors of a launch.  Blocks find their first one in `begin`, not by a
// search: constant memory that nobody has read yet answers slowly.
template <int N>
struct Table {
  int n;
  uint32_t chunks;
  const void* data[N];
  void* out[N];
  long long numel[N];
  uint32_t chunk[N + 1];            // each tensor's first chunk, and the number of all
  uint16_t begin[kMostBlocks + 1];  // the tensor of each run's first chunk
  uint8_t type[N];
};
static_assert(sizeof(Table<kTableMax>) + 64 <= 32764, "the table and the other arguments fit a launch's parameters");

struct Entry {
  const void* data;
  void* out;
  long long numel;
  uint32_t chunk;
  int type;
};
template <int N>
__device__ __forceinline__ Entry entry(const Table<N>& tab, int k) {
  return Entry{tab.data[k], tab.out[k], tab.numel[k], tab.chunk[k], tab.type[k]};
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

// A tensor in 16-byte groups of the address space: group 0 begins up to 15
// bytes before the tensor, and the ends may be less than whole groups.
struct Groups {
  const char* data;
  long long bytes;
  int skip;
  __device__ __forceinline__ explicit Groups(const Entry& t)
      : data(static_cast<const char*>(t.data)), bytes(t.numel * (t.type == TRIMUL_F32 ? 4 : 2)),
        skip(static_cast<int>(reinterpret_cast<uintptr_t>(t.data) % 16)) {}
  // where a thread's groups of a chunk begin; they are kThreads groups apart
  __device__ __forceinline__ long long first(uint32_t chunk) const {
    return (static_cast<long long>(chunk) * kGroups + threadIdx.x) * 16 - skip;
  }
  __device__ __forceinline__ bool whole(long long i) const { return i >= 0 && i + 16 <= bytes; }
};

// Groups at a tensor's ends, two bytes at a time (out of line: they are few,
// and their code would cost the others registers).
__device__ __noinline__ uint4 load_part(const char* data, long long i, long long bytes) {
  alignas(16) uint16_t part[8] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + 2 * e >= 0 && i + 2 * e < bytes) part[e] = *reinterpret_cast<const uint16_t*>(data + i + 2 * e);
  return *reinterpret_cast<const uint4*>(part);
}
__device__ __noinline__ void store_part(char* out, long long i, long long bytes, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + 2 * e >= 0 && i + 2 * e < bytes)
      *reinterpret_cast<uint16_t*>(out + i + 2 * e) = static_cast<uint16_t>(w[e / 2] >> (e % 2 * 16));
}

// How L2 is to hold what a load brings: not for long, or longer than others.
__device__ __forceinline__ uint64_t policy_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_last() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint4 load16(const void* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy)
               : "memory");
  return v;
}

// A thread's groups of a chunk; zeros where they go past the tensor.
__device__ __forceinline__ void load_chunk(const Entry& t, uint32_t chunk, uint64_t policy, uint4 (&v)[kLoads]) {
  const Groups g(t);
  const long long first = g.first(chunk - t.chunk);
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const long long i = first + k * (kThreads * 16);
    v[k] = make_uint4(0u, 0u, 0u, 0u);
    if (g.whole(i))
      v[k] = load16(g.data + i, policy);
    else if (i < g.bytes)
      v[k] = load_part(g.data, i, g.bytes);
  }
}

// ------------------------------------------------------------------ norm
// Squares are summed in fp32 within a thread's part of a chunk (16 or 32
// numbers), and from there on as pairs of fp32 numbers, the sum and what its
// roundings lost: fp64 runs at about a sixtieth of fp32's rate here, and the
// fifty fp64 operations a thread of an fp64 reduction took longer than the
// reading.  Parts
// whose sum is outside [2^-60, 2^80] may hold elements whose squares fp32
// loses (within a part whose sum is not, those are too small to matter: below
// 2^-63, which 2^-60 hides for 32 numbers).  They are scaled and summed again,
// and go to a sum in fp64 of their own.
// What has been seen: hi + lo + wide is a sum of squares; of a maximum, hi's
// bits are the largest magnitude's (a NaN's are above infinity's).
struct Seen {
  float hi = 0.f, lo = 0.f;
  double wide = 0.0;
  __device__ __forceinline__ void add(float v) {  // the rounding error of a sum, as in Knuth's TwoSum
    const float t = hi + v, b = t - hi;
    lo += (hi - (t - b)) + (v - b);
    hi = t;
  }
  __device__ __forceinline__ void join(float h, float l, int kind) {
    if (kind == TRIMUL_NORM_INF) {
      hi = __uint_as_float(max(__float_as_uint(hi), __float_as_uint(h)));
    } else {
      add(h);
      lo += l;
    }
  }
  __device__ __forceinline__ bool any_wide() const { return __double_as_longlong(wide) != 0; }
  // (of a sum that fp32 holds well, the root of that; its error is 2 ulp)
  __device__ __forceinline__ float norm(int kind) const {
    if (kind == TRIMUL_NORM_INF) return hi;
    if (!any_wide()) return sqrtf(hi + lo);
    return static_cast<float>(sqrt(wide + (static_cast<double>(hi) + lo)));
  }
};

template <typename T>
__device__ __forceinline__ float square(const uint4 v, float scale) {
  constexpr int V = 16 / sizeof(T);
  float f[V];
  unpack16<T>(v, f);
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] *= scale;
  float q = f[0] * f[0];
#pragma unroll
  for (int e = 1; e < V; ++e) q += f[e] * f[e];
  return q;
}
template <typename T>
__device__ __forceinline__ float largest(const uint4 v) {
  constexpr int V = 16 / sizeof(T);
  float f[V];
  unpack16<T>(v, f);
  unsigned top = __float_as_uint(fabsf(f[0]));
#pragma unroll
  for (int e = 1; e < V; ++e) top = max(top, __float_as_uint(fabsf(f[e])));
  return __uint_as_float(top);
}
__device__ __forceinline__ float square(const uint4 v, int type, float scale) {
  return type == TRIMUL_F32 ? square<float>(v, scale) : type == TRIMUL_BF16 ? square<__nv_bfloat16>(v, scale) : square<__half>(v, scale);
}
__device__ __forceinline__ float largest(const uint4 v, int type) {
  return type == TRIMUL_F32 ? largest<float>(v) : type == TRIMUL_BF16 ? largest<__nv_bfloat16>(v) : largest<__half>(v);
}

// The sum of squares of a part that fp32 did not hold (out of line, as it is rare); low: it came out too small.
__device__ __noinline__ double wide_squares(uint4 a, uint4 b, uint4 c, uint4 d, int type, bool low) {
  static_assert(kLoads == 4, "one argument a load");
  const float scale = low ? 0x1p90f : 0x1p-80f;  // low: elements below 2^-30, the smallest 2^-149
  const float s = (square(a, type, scale) + square(b, type, scale)) + (square(c, type, scale) + square(d, type, scale));
  return static_cast<double>(s) * (low ? 0x1p-180 : 0x1p160);
}

__device__ __forceinline__ void add_chunk(const uint4 (&v)[kLoads], int type, int kind, Seen& seen) {
  if (kind == TRIMUL_NORM_INF) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) seen.join(largest(v[k], type), 0.f, kind);
    return;
  }
  float s;
  if (type == TRIMUL_F32)
    s = (square<float>(v[0], 1.f) + square<float>(v[1], 1.f)) + (square<float>(v[2], 1.f) + square<float>(v[3], 1.f));
  else if (type == TRIMUL_BF16)
    s = (square<__nv_bfloat16>(v[0], 1.f) + square<__nv_bfloat16>(v[1], 1.f)) + (square<__nv_bfloat16>(v[2], 1.f) + square<__nv_bfloat16>(v[3], 1.f));
  else
    s = (square<__half>(v[0], 1.f) + square<__half>(v[1], 1.f)) + (square<__half>(v[2], 1.f) + square<__half>(v[3], 1.f));
  if (s >= 0x1p-60f && s <= 0x1p80f) {
    seen.add(s);
    return;
  }
  const bool low = s < 0x1p-60f;  // else too large, infinite or NaN
  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < kLoads; ++k) bits |= v[k].x | v[k].y | v[k].z | v[k].w;
  if (bits != 0) seen.wide += wide_squares(v[0], v[1], v[2], v[3], type, low);
}

// All threads' numbers as one, in a fixed order; every thread gets it.
constexpr int kWarps = kThreads / 32;
struct Shared {
  float hi[kWarps], lo[kWarps];
  double wide[kWarps];
};
__device__ __forceinline__ Seen block_total(Seen v, Shared& s, int kind) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v.join(__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o), kind);
  const int warp = threadIdx.x / 32;
  if (threadIdx.x % 32 == 0) s.hi[warp] = v.hi, s.lo[warp] = v.lo;
  const bool any = __syncthreads_or(v.any_wide());
  if (any) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v.wide += __shfl_xor_sync(0xffffffffu, v.wide, o);
    if (threadIdx.x % 32 == 0) s.wide[warp] = v.wide;
    __syncthreads();
  }
  Seen t;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    t.join(s.hi[k], s.lo[k], kind);
    if (any) t.wide += s.wide[k];
  }
  return t;
}

// The run of chunks of a block.
__host__ __device__ __forceinline__ uint32_t run_begin(uint32_t chunks, uint32_t block, uint32_t blocks) {
  return static_cast<uint32_t>(static_cast<unsigned long long>(chunks) * block / blocks);
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    k9_norm(const __grid_constant__ Table<N> tab, int kind, Seen* part, uint32_t keep) {
  let_next_begin();
  __shared__ Shared s;
  Seen seen;
  const uint32_t c0 = run_begin(tab.chunks, blockIdx.x, gridDim.x), c1 = run_begin(tab.chunks, blockIdx.x + 1, gridDim.x);
  int k = tab.begin[blockIdx.x];
  Entry t = entry(tab, k);
  uint32_t end = tab.chunk[k + 1];  // of tensor k's chunks
  const uint64_t first = policy_first(), last = policy_last();
  const uint32_t kept = c1 - min(c1 - c0, keep);  // the run's last ones
  for (uint32_t chunk = c0; chunk < c1; ++chunk) {
    if (chunk >= end) {
      t = entry(tab, ++k);
      end = tab.chunk[k + 1];
    }
    uint4 v[kLoads];
    load_chunk(t, chunk, chunk < kept ? first : last, v);
    const int type = t.type;
    add_chunk(v, type, kind, seen);
  }
  const Seen all = block_total(seen, s, kind);
  if (threadIdx.x == 0) part[blockIdx.x] = all;
}

// ------------------------------------------------------------------ scale
// The factor for a norm.  One that is not finite (inf - inf and NaN - NaN are NaN) scales nothing.
__device__ __forceinline__ float factor(float norm, float max_norm) {
  const float share = max_norm / (norm + 1e-6f);
  return (norm - norm == 0.f && share < 1.0f) ? share : 1.0f;
}

template <typename T>
__device__ __forceinline__ uint4 scaled(const uint4 v, float coef) {
  float f[16 / sizeof(T)];
  unpack16<T>(v, f);
#pragma unroll
  for (int e = 0; e < static_cast<int>(16 / sizeof(T)); ++e) f[e] *= coef;
  return pack16(f, T());
}

__device__ __forceinline__ void scale_chunk(const Entry& t, uint32_t chunk, uint4 (&v)[kLoads], float coef) {
  const Groups g(t);
  char* const out = static_cast<char*>(t.out);
  const long long first = g.first(chunk - t.chunk);
  const bool alike = reinterpret_cast<uintptr_t>(t.out) % 16 == reinterpret_cast<uintptr_t>(t.data) % 16;
  if (coef != 1.0f) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      v[k] = t.type == TRIMUL_F32    ? scaled<float>(v[k], coef)
             : t.type == TRIMUL_BF16 ? scaled<__nv_bfloat16>(v[k], coef)
                                     : scaled<__half>(v[k], coef);
  }
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const long long i = first + k * (kThreads * 16);
    if (alike && g.whole(i)) {
      __stcs(reinterpret_cast<uint4*>(out + i), v[k]);
    } else if (i < g.bytes) {
      store_part(out, i, g.bytes, v[k]);
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    k9_scale(const __grid_constant__ Table<N> tab, int kind, const Seen* part, int parts, float max_norm, float* norm,
             int write, int in_place) {
  __shared__ Shared s;
  const uint32_t c0 = run_begin(tab.chunks, blockIdx.x, gridDim.x), c1 = run_begin(tab.chunks, blockIdx.x + 1, gridDim.x);
  int k = c0 < c1 ? tab.begin[blockIdx.x + 1] : 0;
  if (k > 0 && tab.chunk[k] >= c1) --k;  // the tensor of the run's last chunk
  Entry t = entry(tab, k);
  after_previous();
  Seen seen;
  for (int q = threadIdx.x; q < parts; q += kThreads) {
    const Seen v = part[q];
    seen.join(v.hi, v.lo, kind);
    if (v.any_wide()) seen.wide += v.wide;
  }
  const float n = block_total(seen, s, kind).norm(kind);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  if (!write) return;
  const float coef = factor(n, max_norm);
  if (coef == 1.0f && in_place) return;
  const uint64_t once = policy_first();
  for (uint32_t chunk = c1; chunk-- > c0;) {
    if (chunk < t.chunk) t = entry(tab, --k);
    if (coef == 1.0f && t.data == t.out) continue;
    uint4 v[kLoads];
    load_chunk(t, chunk, once, v);
    scale_chunk(t, chunk, v, coef);
  }
}

// ------------------------------------------------------------------ launches
uint32_t chunks_of(const trimul_grad_tensor& t) {
  const long long v = t.type == TRIMUL_F32 ? 4 : 8;
  const long long skip = static_cast<long long>(reinterpret_cast<uintptr_t>(t.data) % 16) * v / 16;
  const long long groups = (t.numel + skip + v - 1) / v;
  return static_cast<uint32_t>((groups + kGroups - 1) / kGroups);
}

// Fills a table from t[k] on; k moves past the tensors that are in it.  Returns the launch's blocks.
template <int N>
int fill(Table<N>& tab, const trimul_grad_tensor* t, int n, int& k, int num_sms) {
  tab.n = 0;
  tab.chunks = 0;
  for (; k < n && tab.n < N; ++k) {
    if (t[k].numel == 0) continue;
    const int q = tab.n++;
    tab.data[q] = t[k].data;
    tab.out[q] = t[k].out;
    tab.numel[q] = t[k].numel;
    tab.type[q] = static_cast<uint8_t>(t[k].type);
    tab.chunk[q] = tab.chunks;
    tab.chunks += chunks_of(t[k]);
  }
  tab.chunk[tab.n] = tab.chunks;
  const int most = std::min(kMostBlocks, kBlocksPerSm * num_sms);
  const int grid = static_cast<int>(std::max<long long>(1, std::min<long long>(tab.chunks, most)));
  int at = 0;
  for (int block = 0; block <= grid; ++block) {
    const uint32_t first = run_begin(tab.chunks, block, grid);
    while (at + 1 < tab.n && tab.chunk[at + 1] <= first) ++at;
    tab.begin[block] = static_cast<uint16_t>(at);
  }
  return grid;
}

template <int N>
cudaError_t run(const trimul_grad_tensor* t, int n, trimul_norm_kind kind, float* norm, Seen* part, bool clip,
                float max_norm, int num_sms, cudaStream_t s) {
  Table<N> tab;
  int parts = 0, k = 0, grid = 0;
  bool in_place = true;  // all of them: nothing to do where the factor is 1
  for (int q = 0; q < n; ++q) in_place = in_place && t[q].data == t[q].out;
  do {
    grid = fill(tab, t, n, k, num_sms);
    k9_norm<N><<<grid, kThreads, 0, s>>>(tab, kind, part + parts, clip ? kKeep / grid : 0);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    parts += grid;
  } while (k < n);
  k = 0;
  for (bool first = true; first || (k < n && clip); first = false) {
    if (n > N)
      grid = fill(tab, t, n, k, num_sms);
    else  // the table is what the norm kernel had
      k = n;
    const dim3 blocks(clip ? grid : 1);
    cudaError_t e = cudaSuccess;
    if (first) {
      e = launch_early(k9_scale<N>, blocks, kThreads, s, tab, kind, part, parts, max_norm, norm, clip, in_place);
    } else {
      k9_scale<N><<<blocks, kThreads, 0, s>>>(tab, kind, part, parts, max_norm, norm, 1, in_place);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_workspace(int n, int num_sms) {
  const size_t launches = std::max(1, (n + kTableMax - 1) / kTableMax);
  return launches * std::min(kMostBlocks, kBlocksPerSm * num_sms) * sizeof(Seen);
}

cudaError_t launch_grad_norm(const trimul_grad_tensor* t, int n, trimul_norm_kind kind, float* norm, void* ws,
                             bool clip, float max_norm, int num_sms, cudaStream_t s) {
  Seen* const part = static_cast<Seen*>(ws);
  return n <= kTableSmall ? run<kTableSmall>(t, n, kind, norm, part, clip, max_norm, num_sms, s)
                          : run<kTableMax>(t, n, kind, norm, part, clip, max_norm, num_sms, s);
}

}  // namespace trimul
