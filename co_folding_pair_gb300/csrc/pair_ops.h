// pair_ops.h -- argument blocks and launchers of the operators around the layer (internal):
// relative position bias, residual step, gradient norm and clipping.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "trimul.h"

namespace trimul {

// Division of n < 2^31 by a fixed d in [1, 2^31): q = (umulhi(n, m) + n) >> s
// with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1, the round-up
// method of Granlund and Montgomery ("Division by Invariant Integers using
// Multiplication"); n < 2^31 keeps the sum within 32 bits.
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
  __device__ __forceinline__ void divmod(uint32_t n, uint32_t& q, uint32_t& r) const {
    q = div(n);
    r = n - q * d;
  }
#endif
};

// Lets a kernel have `most` bytes of dynamic shared memory; asked for once a device.
template <auto kKernel>
cudaError_t allow_smem(int most) {
  static std::atomic<uint64_t> done{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess || (device < 64 && (done.load() >> device & 1))) return e;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess && device < 64) done.fetch_or(1ull << device);
  return e;
}

// Launches a kernel whose blocks may be set up while the one before it in the
// stream still runs (programmatic dependent launch).  The kernel waits
// (after_previous) before it reads what that one writes; that one says with
// let_next_begin that all its blocks have begun.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t s, Args... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = threads;
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<Params>(args)...);
}

// ---------------------------------------------------------------- relative position bias
constexpr int kRelposMaxDistance = 32768;
constexpr int kRelposMaxRows = 1024;

struct RelposArgs {
  const int16_t* lut;  // [M - lo + 1]: the bucket of distance d, lo <= d <= M, at d - lo; null: d - lo itself
  int lo, M, rows;     // distances below lo have lo's bucket; rows: of the table, the one for different groups (the last) among them
  const int32_t *q_pos, *k_pos, *q_group, *k_group;  // groups: both null, or neither
  int B, I, J, D;
  FastDiv by_I, by_J;
};

// HEADS layout [B][H][n]: head h's plane of batch b, as groups of V elements (16
// bytes) on the tensor's 16-byte boundaries.  A group takes in what lies before
// and behind the plane, other planes, but nothing past the tensor: behind small
// planes that is soon.
struct HeadPlane {
  long long at;         // the boundary at or before the plane's first element
  uint32_t early;       // elements from there to it
  uint32_t end, whole;  // from `at` on: past the plane's last element; a group at k < end is all in the tensor if k + V <= whole
  __host__ __device__ HeadPlane(uint32_t b, int h, int B, int H, uint32_t n, int V) {
    const long long begin = (static_cast<long long>(b) * H + h) * n;
    early = static_cast<uint32_t>(begin % V);
    at = begin - early;
    end = early + n;
    // elements behind the plane, where they are less than the V - 1 that a group may reach past it
    const uint32_t most = V - 1, batches = B - 1 - b;
    const uint32_t planes = (batches < most ? batches : most) * H + (H - 1 - h);
    const uint32_t behind = (planes < most ? planes : most) * (n < most ? n : most);
    whole = end + (behind < most ? behind : most);
  }
};

cudaError_t launch_relpos_forward(const RelposArgs& a, const void* table, bool table_f32, const void* base, void* out,
                                  bool f32, trimul_layout layout, int num_sms, cudaStream_t s);
size_t relpos_backward_workspace(int rows, int B, int I, int J, int D, trimul_layout layout, bool f32, int num_sms);
cudaError_t launch_relpos_backward(const RelposArgs& a, const void* dout, bool f32, trimul_layout layout,
                                   float* dtable, bool accumulate, float* ws, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------- residual step
struct ResidualArgs {
  trimul_residual_params p;
  const void* x;
  const uint16_t *u, *gate, *mask;
  int B, I, J;
  FastDiv by_I, by_J;
  void* out;          // forward
  uint16_t* normed;
  const void *dout, *dout2;  // backward
  const uint16_t* dnormed;
  void* dx;
  uint16_t *du, *dgate;
  trimul_residual_grads g;
  float* part;        // [blocks][RESIDUAL_SUMS][D] column sums
};
constexpr int RESIDUAL_SUMS = 4;  // S0 and S1 (k8_residual.cu), and the gradients of pre_gamma and pre_beta

cudaError_t launch_residual_forward(const ResidualArgs& a, int num_sms, cudaStream_t s);
size_t residual_backward_workspace(int D, long long rows, int num_sms);
cudaError_t launch_residual_backward(const ResidualArgs& a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------- gradient norm and clipping
size_t grad_workspace(int n, int num_sms);
cudaError_t launch_grad_norm(const trimul_grad_tensor* t, int n, trimul_norm_kind kind, float* norm, void* ws,
                             bool clip, float max_norm, int num_sms, cudaStream_t s);

}  // namespace trimul
