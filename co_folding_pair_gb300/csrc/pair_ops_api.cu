// pair_ops_api.cu -- the C ABI's entry points of the operators around the layer
// (include/trimul.h): argument checks, the relpos plan, and the launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "trimul.h"
#include "api_status.h"
#include "pair_ops.h"

using namespace trimul;

struct trimul_relpos_s {
  int device = 0;
  int lo = 0, M = 0, rows = 0;  // as in RelposArgs
  bool groups = false;
  int num_sms = 0;
  int16_t* lut = nullptr;
};

namespace {

// Makes `device` current for a call, and the caller's device again after it.
class DeviceScope {
 public:
  trimul_status enter(int device) {
    TRY_CUDA(cudaGetDevice(&before_), "cudaGetDevice");
    if (before_ == device) return TRIMUL_OK;
    TRY_CUDA(cudaSetDevice(device), "cudaSetDevice");
    changed_ = true;
    return TRIMUL_OK;
  }
  ~DeviceScope() {
    if (changed_) cudaSetDevice(before_);
  }

 private:
  int before_ = 0;
  bool changed_ = false;
};

// Checks the device (compute capability 10.3) and gives its SM count; both are
// asked for once a device.
trimul_status device_sms(int device, int* sms) {
  constexpr int kMost = 64;
  static std::atomic<int> known[kMost];
  int ndev = 0;
  if (device >= 0 && device < kMost && (*sms = known[device].load()) > 0) return TRIMUL_OK;
  TRY_CUDA(cudaGetDeviceCount(&ndev), "cudaGetDeviceCount");
  if (device < 0 || device >= ndev) return fail(TRIMUL_ERR_INVALID_ARG, "device %d out of range (%d devices)", device, ndev);
  int major = 0, minor = 0;
  TRY_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device), "cudaDeviceGetAttribute");
  TRY_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device), "cudaDeviceGetAttribute");
  if (major != 10 || minor != 3)
    return fail(TRIMUL_ERR_UNSUPPORTED_ARCH, "TriMul kernels are built for sm_103 (GB300); got sm_%d%d", major, minor);
  TRY_CUDA(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device), "cudaDeviceGetAttribute");
  if (device < kMost) known[device].store(*sms);
  return TRIMUL_OK;
}

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

bool overlap(const void* p, size_t pn, const void* q, size_t qn) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + qn && b < a + pn;
}

trimul_status check_pairs(int B, int I, int J) {
  if (B < 1 || I < 1 || J < 1) return fail(TRIMUL_ERR_SHAPE, "B (%d), I (%d) and J (%d) must be >= 1", B, I, J);
  const long long rows = static_cast<long long>(B) * I;
  if (rows > INT32_MAX || rows * J > INT32_MAX || static_cast<long long>(B) * J > INT32_MAX)
    return fail(TRIMUL_ERR_SHAPE, "B=%d I=%d J=%d: 2^31 pairs or more", B, I, J);
  return TRIMUL_OK;
}

trimul_status check_width(int D) {
  if (D < 8 || D > 256 || D % 8 != 0) return fail(TRIMUL_ERR_SHAPE, "D (%d) must be a multiple of 8 in [8, 256]", D);
  return TRIMUL_OK;
}

trimul_status check_flags(unsigned flags, unsigned known) {
  if (flags & ~known) return fail(TRIMUL_ERR_INVALID_ARG, "flags 0x%x are not taken by this entry point", flags & ~known);
  return TRIMUL_OK;
}

trimul_status check_workspace(const void* ws, size_t have, size_t need, size_t align) {
  if (have < need || !ws) return fail(TRIMUL_ERR_INVALID_ARG, "the workspace holds %zu bytes, %zu are needed", ws ? have : 0, need);
  if (!aligned(ws, align)) return fail(TRIMUL_ERR_INVALID_ARG, "the workspace must be %zu-byte aligned", align);
  return TRIMUL_OK;
}

trimul_status finish(cudaError_t launched, cudaStream_t s, unsigned flags, const char* what) {
  TRY_CUDA(launched, what);
  if (flags & TRIMUL_FLAG_CHECK) TRY_CUDA(cudaStreamSynchronize(s), "stream synchronize");
  return TRIMUL_OK;
}

#define TRY(expr)                            \
  do {                                       \
    const trimul_status s_ = (expr);         \
    if (s_ != TRIMUL_OK) return s_;          \
  } while (0)

// ------------------------------------------------------------------ relpos
// n^p as little-endian 32-bit digits times m^q: what the borders of the LOG
// buckets are compared in.
using Digits = std::vector<uint32_t>;
void multiply(Digits& x, uint32_t by) {
  uint64_t carry = 0;
  for (uint32_t& d : x) {
    carry += static_cast<uint64_t>(d) * by;
    d = static_cast<uint32_t>(carry);
    carry >>= 32;
  }
  if (carry) x.push_back(static_cast<uint32_t>(carry));
}
Digits powers(uint32_t n, int p, uint32_t m, int q) {
  Digits x{1};
  for (int k = 0; k < p; ++k) multiply(x, n);
  for (int k = 0; k < q; ++k) multiply(x, m);
  return x;
}
bool less(const Digits& a, const Digits& b) {
  if (a.size() != b.size()) return a.size() < b.size();
  for (size_t k = a.size(); k-- > 0;)
    if (a[k] != b[k]) return a[k] < b[k];
  return false;
}

// The LOG bucket of n in [0, M] for K buckets.  Bucket E + k begins at the
// least n with log(n / E) / log(M / E) (K - E) >= k, that is
// n^(K - E) E^k >= M^k E^(K - E), decided in whole numbers.
std::vector<int16_t> log_buckets(int K, int M) {
  const int E = K / 2, steps = K - E;
  std::vector<int16_t> b(M + 1);
  int n = 0;
  for (; n < E; ++n) b[n] = static_cast<int16_t>(n);
  for (int k = 1; k < steps; ++k) {
    const Digits right = powers(M, k, E, steps);
    // from the floating-point estimate to the border itself; at M every k < steps holds
    int lo = static_cast<int>(std::lround(E * std::pow(static_cast<double>(M) / E, static_cast<double>(k) / steps)));
    lo = lo < n ? n : lo > M ? M : lo;
    while (lo < M && less(powers(lo, steps, E, k), right)) ++lo;
    while (lo > n && !less(powers(lo - 1, steps, E, k), right)) --lo;
    for (; n < lo; ++n) b[n] = static_cast<int16_t>(E + k - 1);
  }
  for (; n <= M; ++n) b[n] = static_cast<int16_t>(K - 1);
  return b;
}

trimul_status check_relpos(trimul_relpos r, const int32_t* q_pos, const int32_t* k_pos, const int32_t* q_group,
                           const int32_t* k_group, int B, int I, int J, int D, trimul_layout layout,
                           trimul_dtype type) {
  if (!r) return fail(TRIMUL_ERR_INVALID_ARG, "null plan");
  TRY(check_pairs(B, I, J));
  if (layout == TRIMUL_LAYOUT_PAIR) {
    TRY(check_width(D));
  } else if (layout == TRIMUL_LAYOUT_HEADS) {
    if (D < 1 || D > 256) return fail(TRIMUL_ERR_SHAPE, "D (%d heads) must be in [1, 256]", D);
  } else {
    return fail(TRIMUL_ERR_INVALID_ARG, "unknown layout %d", static_cast<int>(layout));
  }
  if (type != TRIMUL_BF16 && type != TRIMUL_F32) return fail(TRIMUL_ERR_INVALID_ARG, "type must be BF16 or F32");
  if (!q_pos || !k_pos) return fail(TRIMUL_ERR_INVALID_ARG, "positions are null");
  if (!q_group != !k_group) return fail(TRIMUL_ERR_INVALID_ARG, "give both groups or neither");
  if (q_group && !r->groups) return fail(TRIMUL_ERR_INVALID_ARG, "the plan was made without groups");
  for (const int32_t* p : {q_pos, k_pos, q_group, k_group})
    if (!aligned(p, 4)) return fail(TRIMUL_ERR_INVALID_ARG, "positions and groups must be 4-byte aligned");
  return TRIMUL_OK;
}

RelposArgs relpos_args(trimul_relpos r, const int32_t* q_pos, const int32_t* k_pos, const int32_t* q_group,
                       const int32_t* k_group, int B, int I, int J, int D) {
  RelposArgs a{};
  a.lut = r->lut;
  a.lo = r->lo;
  a.M = r->M;
  a.rows = r->rows;
  a.q_pos = q_pos, a.k_pos = k_pos, a.q_group = q_group, a.k_group = k_group;
  a.B = B, a.I = I, a.J = J, a.D = D;
  a.by_I = FastDiv(I), a.by_J = FastDiv(J);
  return a;
}

// ------------------------------------------------------------------ residual
trimul_status check_residual(const trimul_residual_params* p, const uint16_t* gate, const uint16_t* mask, int B, int I,
                             int J) {
  if (!p) return fail(TRIMUL_ERR_INVALID_ARG, "params is null");
  TRY(check_width(p->D));
  TRY(check_pairs(B, I, J));
  if (p->stream_type != TRIMUL_BF16 && p->stream_type != TRIMUL_F32)
    return fail(TRIMUL_ERR_INVALID_ARG, "stream_type must be BF16 or F32");
  if (!std::isnormal(p->eps) || p->eps < 0.0f) return fail(TRIMUL_ERR_INVALID_ARG, "eps must be a normal number > 0");
  if (!std::isfinite(p->scale)) return fail(TRIMUL_ERR_INVALID_ARG, "scale must be finite");
  const struct {
    trimul_norm kind;
    const float *gamma, *beta;
    const char* name;
  } norms[] = {{p->post_norm, p->post_gamma, p->post_beta, "post_norm"}, {p->pre_norm, p->pre_gamma, p->pre_beta, "pre_norm"}};
  for (const auto& n : norms) {
    if (n.kind != TRIMUL_NORM_NONE && n.kind != TRIMUL_NORM_LAYER && n.kind != TRIMUL_NORM_RMS)
      return fail(TRIMUL_ERR_INVALID_ARG, "unknown %s %d", n.name, static_cast<int>(n.kind));
    if (n.kind == TRIMUL_NORM_NONE && n.gamma) return fail(TRIMUL_ERR_INVALID_ARG, "%s is NONE, but has a gamma", n.name);
    if (n.kind != TRIMUL_NORM_LAYER && n.beta) return fail(TRIMUL_ERR_INVALID_ARG, "%s is not LAYER, but has a beta", n.name);
  }
  if (p->gate < TRIMUL_GATE_NONE || p->gate > TRIMUL_GATE_COL)
    return fail(TRIMUL_ERR_INVALID_ARG, "unknown gate %d", static_cast<int>(p->gate));
  if ((p->gate == TRIMUL_GATE_NONE) != !gate) return fail(TRIMUL_ERR_INVALID_ARG, "the gate and params->gate do not agree");
  for (const void* q : {(const void*)p->post_gamma, (const void*)p->post_beta, (const void*)p->pre_gamma,
                        (const void*)p->pre_beta, (const void*)p->channel, (const void*)gate})
    if (!aligned(q, 16)) return fail(TRIMUL_ERR_INVALID_ARG, "parameters and gate must be 16-byte aligned");
  if (!aligned(mask, 2)) return fail(TRIMUL_ERR_INVALID_ARG, "the mask must be 2-byte aligned");
  return TRIMUL_OK;
}

size_t gate_elems(const trimul_residual_params* p, int B, int I, int J) {
  const size_t b = static_cast<size_t>(B) * p->D;
  return p->gate == TRIMUL_GATE_PAIR ? b * I * J : p->gate == TRIMUL_GATE_ROW ? b * J : p->gate == TRIMUL_GATE_COL ? b * I : 0;
}

struct Buffer {
  const void* p;
  size_t bytes;
  const char* name;
};

// Every output apart from every input and from the other outputs; output 0 may be input 0 itself.
trimul_status check_apart(const Buffer* in, int n_in, const Buffer* out, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int k = 0; k < n_in; ++k)
      if (overlap(out[i].p, out[i].bytes, in[k].p, in[k].bytes) && !(i == 0 && k == 0 && out[0].p == in[0].p))
        return fail(TRIMUL_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[k].name);
    for (int k = 0; k < i; ++k)
      if (overlap(out[i].p, out[i].bytes, out[k].p, out[k].bytes))
        return fail(TRIMUL_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[k].name);
  }
  return TRIMUL_OK;
}

ResidualArgs residual_args(const trimul_residual_params* p, const void* x, const uint16_t* u, const uint16_t* gate,
                           const uint16_t* mask, int B, int I, int J) {
  ResidualArgs a{};
  a.p = *p;
  a.x = x, a.u = u, a.gate = gate, a.mask = mask;
  a.B = B, a.I = I, a.J = J;
  a.by_I = FastDiv(I), a.by_J = FastDiv(J);
  return a;
}

// ------------------------------------------------------------------ gradients
size_t type_bytes(trimul_dtype t) { return t == TRIMUL_F32 ? 4 : 2; }

trimul_status check_tensors(const trimul_grad_tensor* t, int n, trimul_norm_kind kind, const float* norm,
                            const void* ws, size_t ws_bytes, bool out) {
  if (n < 0) return fail(TRIMUL_ERR_INVALID_ARG, "n (%d) must be >= 0", n);
  if (n > 0 && !t) return fail(TRIMUL_ERR_INVALID_ARG, "tensors is null");
  if (kind != TRIMUL_NORM_L2 && kind != TRIMUL_NORM_INF) return fail(TRIMUL_ERR_INVALID_ARG, "unknown norm %d", static_cast<int>(kind));
  if (!norm || !aligned(norm, 4)) return fail(TRIMUL_ERR_INVALID_ARG, "norm is null or not 4-byte aligned");
  if (overlap(norm, 4, ws, ws_bytes)) return fail(TRIMUL_ERR_INVALID_ARG, "norm overlaps the workspace");
  for (int k = 0; k < n; ++k) {
    if (t[k].numel < 0) return fail(TRIMUL_ERR_SHAPE, "tensor %d: numel (%lld) must be >= 0", k, static_cast<long long>(t[k].numel));
    if (t[k].numel >= (1ll << 42)) return fail(TRIMUL_ERR_SHAPE, "tensor %d: numel (%lld) is too large", k, static_cast<long long>(t[k].numel));
    if (t[k].type != TRIMUL_BF16 && t[k].type != TRIMUL_F32 && t[k].type != TRIMUL_F16)
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: unknown type %d", k, static_cast<int>(t[k].type));
    if (t[k].numel == 0) continue;
    const size_t w = type_bytes(t[k].type);
    if (!t[k].data || !aligned(t[k].data, w)) return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: data is null or not aligned to its type", k);
    for (const void* q : {t[k].data, out ? static_cast<const void*>(t[k].out) : nullptr})
      if (overlap(norm, 4, q, t[k].numel * w) || overlap(ws, ws_bytes, q, t[k].numel * w))
        return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d overlaps norm or the workspace", k);
    if (!out) continue;
    if (!t[k].out || !aligned(t[k].out, w)) return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: out is null or not aligned to its type", k);
    if (t[k].out != t[k].data && overlap(t[k].out, t[k].numel * w, t[k].data, t[k].numel * w))
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: out overlaps data, but is not data", k);
  }
  return TRIMUL_OK;
}

}  // namespace

extern "C" {

trimul_status trimul_relpos_create(trimul_relpos* out, const trimul_relpos_params* p, int device) {
  if (!out) return fail(TRIMUL_ERR_INVALID_ARG, "out is null");
  *out = nullptr;
  if (!p) return fail(TRIMUL_ERR_INVALID_ARG, "params is null");
  const int M = p->max_distance;
  if (M < 1 || M > kRelposMaxDistance)
    return fail(TRIMUL_ERR_SHAPE, "max_distance (%d) must be in [1, %d]", M, kRelposMaxDistance);
  int buckets = 0;
  if (p->kind == TRIMUL_BUCKETS_LINEAR) {
    buckets = p->bidirectional ? 2 * M + 1 : M + 1;
    if (p->num_buckets != 0 && p->num_buckets != buckets)
      return fail(TRIMUL_ERR_SHAPE, "num_buckets (%d) of linear buckets must be 0 or %d", p->num_buckets, buckets);
  } else if (p->kind == TRIMUL_BUCKETS_LOG) {
    buckets = p->num_buckets;
    if (p->bidirectional && buckets % 2 != 0)
      return fail(TRIMUL_ERR_SHAPE, "num_buckets (%d) of two-sided log buckets must be even", buckets);
  } else {
    return fail(TRIMUL_ERR_INVALID_ARG, "unknown bucket kind %d", static_cast<int>(p->kind));
  }
  const int rows = buckets + (p->groups ? 1 : 0);
  if (buckets < 2 || rows > kRelposMaxRows)
    return fail(TRIMUL_ERR_SHAPE, "%d buckets: 2 to %d are taken, the one for groups among them", buckets, kRelposMaxRows);
  const int K = p->bidirectional ? buckets / 2 : buckets;
  if (p->kind == TRIMUL_BUCKETS_LOG && (K < 2 || M <= K / 2))
    return fail(TRIMUL_ERR_SHAPE, "log buckets: %d a side need max_distance > %d, and at least 2", K, K / 2);

  int sms = 0;
  TRY(device_sms(device, &sms));
  trimul_relpos r = nullptr;
  try {
    const int lo = p->bidirectional ? -M : 0;
    std::vector<int16_t> lut;
    if (p->kind == TRIMUL_BUCKETS_LOG) {
      const std::vector<int16_t> b = log_buckets(K, M);
      lut.resize(M - lo + 1);
      for (int d = lo; d <= M; ++d) lut[d - lo] = d >= 0 ? b[d] : static_cast<int16_t>(K + b[-d]);
    }
    r = new trimul_relpos_s;
    r->device = device;
    r->lo = lo;
    r->M = M;
    r->rows = rows;
    r->groups = p->groups != 0;
    r->num_sms = sms;
    DeviceScope scope;
    trimul_status st = scope.enter(device);
    if (st == TRIMUL_OK && !lut.empty()) {
      cudaError_t e = cudaMalloc(&r->lut, lut.size() * sizeof(int16_t));
      if (e == cudaSuccess) e = cudaMemcpy(r->lut, lut.data(), lut.size() * sizeof(int16_t), cudaMemcpyHostToDevice);
      // a copy from pageable memory may return before it is done, and streams that do not block on stream 0 would not wait
      if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
      if (e != cudaSuccess) {
        cudaGetLastError();
        st = cuda_fail(e, "relpos plan");
      }
    }
    if (st != TRIMUL_OK) {
      cudaFree(r->lut);
      delete r;
      return st;
    }
  } catch (const std::bad_alloc&) {
    delete r;
    return fail(TRIMUL_ERR_OOM, "out of host memory");
  }
  *out = r;
  return TRIMUL_OK;
}

int trimul_relpos_rows(trimul_relpos r) {
  if (!r) {
    fail(TRIMUL_ERR_INVALID_ARG, "null plan");
    return -1;
  }
  return r->rows;
}

trimul_status trimul_relpos_forward(trimul_relpos r, const void* table, trimul_dtype table_type, const int32_t* q_pos,
                                    const int32_t* k_pos, const int32_t* q_group, const int32_t* k_group,
                                    const void* base, int B, int I, int J, int D, trimul_layout layout, void* out,
                                    trimul_dtype type, void* stream, unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK));
  TRY(check_relpos(r, q_pos, k_pos, q_group, k_group, B, I, J, D, layout, type));
  if (table_type != TRIMUL_BF16 && table_type != TRIMUL_F32) return fail(TRIMUL_ERR_INVALID_ARG, "table_type must be BF16 or F32");
  if (!table || !out) return fail(TRIMUL_ERR_INVALID_ARG, "table or out is null");
  if (!aligned(base, 16) || !aligned(out, 16)) return fail(TRIMUL_ERR_INVALID_ARG, "base and out must be 16-byte aligned");
  // PAIR reads the table's rows 16 bytes at a time, HEADS its elements one by one
  const size_t at = layout == TRIMUL_LAYOUT_PAIR ? 16 : type_bytes(table_type);
  if (!aligned(table, at)) return fail(TRIMUL_ERR_INVALID_ARG, "table must be %zu-byte aligned", at);
  const size_t bytes = static_cast<size_t>(B) * I * J * D * type_bytes(type);
  const size_t nq = static_cast<size_t>(B) * I * 4, nk = static_cast<size_t>(B) * J * 4;
  const Buffer in[] = {{base, bytes, "base"}, {table, r->rows * static_cast<size_t>(D) * type_bytes(table_type), "table"},
                       {q_pos, nq, "q_pos"}, {k_pos, nk, "k_pos"}, {q_group, nq, "q_group"}, {k_group, nk, "k_group"}};
  const Buffer to[] = {{out, bytes, "out"}};
  TRY(check_apart(in, 6, to, 1));
  DeviceScope scope;
  TRY(scope.enter(r->device));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return finish(launch_relpos_forward(relpos_args(r, q_pos, k_pos, q_group, k_group, B, I, J, D), table,
                                      table_type == TRIMUL_F32, base, out, type == TRIMUL_F32, layout, r->num_sms, s),
                s, flags, "relpos forward launch");
}

size_t trimul_relpos_backward_workspace_bytes(trimul_relpos r, int B, int I, int J, int D, trimul_layout layout,
                                              trimul_dtype type) {
  static const int32_t some = 0;  // stands for the positions, which the sizes do not depend on
  if (check_relpos(r, &some, &some, nullptr, nullptr, B, I, J, D, layout, type) != TRIMUL_OK) return 0;
  return relpos_backward_workspace(r->rows, B, I, J, D, layout, type == TRIMUL_F32, r->num_sms);
}

trimul_status trimul_relpos_backward(trimul_relpos r, const void* dout, trimul_dtype type, const int32_t* q_pos,
                                     const int32_t* k_pos, const int32_t* q_group, const int32_t* k_group, int B,
                                     int I, int J, int D, trimul_layout layout, float* dtable, void* workspace,
                                     size_t workspace_bytes, void* stream, unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK | TRIMUL_FLAG_ACCUMULATE));
  TRY(check_relpos(r, q_pos, k_pos, q_group, k_group, B, I, J, D, layout, type));
  if (!dout || !dtable) return fail(TRIMUL_ERR_INVALID_ARG, "dout or dtable is null");
  if (!aligned(dout, 16)) return fail(TRIMUL_ERR_INVALID_ARG, "dout must be 16-byte aligned");
  if (!aligned(dtable, 4)) return fail(TRIMUL_ERR_INVALID_ARG, "dtable must be 4-byte aligned");
  const size_t need = relpos_backward_workspace(r->rows, B, I, J, D, layout, type == TRIMUL_F32, r->num_sms);
  TRY(check_workspace(workspace, workspace_bytes, need, 16));
  const size_t nq = static_cast<size_t>(B) * I * 4, nk = static_cast<size_t>(B) * J * 4;
  const Buffer in[] = {{nullptr, 0, ""}, {dout, static_cast<size_t>(B) * I * J * D * type_bytes(type), "dout"},
                       {q_pos, nq, "q_pos"}, {k_pos, nk, "k_pos"}, {q_group, nq, "q_group"}, {k_group, nk, "k_group"}};
  const Buffer to[] = {{dtable, r->rows * static_cast<size_t>(D) * 4, "dtable"}, {workspace, need, "workspace"}};
  TRY(check_apart(in, 6, to, 2));
  DeviceScope scope;
  TRY(scope.enter(r->device));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return finish(launch_relpos_backward(relpos_args(r, q_pos, k_pos, q_group, k_group, B, I, J, D), dout,
                                       type == TRIMUL_F32, layout, dtable, flags & TRIMUL_FLAG_ACCUMULATE,
                                       static_cast<float*>(workspace), r->num_sms, s),
                s, flags, "relpos backward launch");
}

trimul_status trimul_relpos_destroy(trimul_relpos r) {
  if (!r) return TRIMUL_OK;
  if (r->lut) {
    DeviceScope scope;
    TRY(scope.enter(r->device));
    cudaDeviceSynchronize();
    cudaFree(r->lut);
  }
  delete r;
  return TRIMUL_OK;
}

trimul_status trimul_residual_forward(const trimul_residual_params* p, const void* x, const uint16_t* u,
                                      const uint16_t* gate, const uint16_t* mask, int B, int I, int J, void* out,
                                      uint16_t* normed, int device, void* stream, unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK));
  TRY(check_residual(p, gate, mask, B, I, J));
  if (!x || !u || !out) return fail(TRIMUL_ERR_INVALID_ARG, "x, u or out is null");
  if ((p->pre_norm == TRIMUL_NORM_NONE) != !normed) return fail(TRIMUL_ERR_INVALID_ARG, "normed and pre_norm do not agree");
  if (!aligned(x, 16) || !aligned(u, 16) || !aligned(out, 16) || !aligned(normed, 16))
    return fail(TRIMUL_ERR_INVALID_ARG, "x, u, out and normed must be 16-byte aligned");
  const size_t n = static_cast<size_t>(B) * I * J * p->D, w = n * type_bytes(p->stream_type);
  const size_t wd = p->D * 4;
  const Buffer in[] = {{x, w, "x"}, {u, n * 2, "u"}, {gate, gate_elems(p, B, I, J) * 2, "gate"}, {mask, n / p->D * 2, "mask"},
                       {p->post_gamma, wd, "post_gamma"}, {p->post_beta, wd, "post_beta"}, {p->pre_gamma, wd, "pre_gamma"},
                       {p->pre_beta, wd, "pre_beta"}, {p->channel, wd, "channel"}};
  const Buffer to[] = {{out, w, "out"}, {normed, n * 2, "normed"}};
  TRY(check_apart(in, 9, to, 2));
  int sms = 0;
  TRY(device_sms(device, &sms));
  DeviceScope scope;
  TRY(scope.enter(device));
  ResidualArgs a = residual_args(p, x, u, gate, mask, B, I, J);
  a.out = out;
  a.normed = normed;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return finish(launch_residual_forward(a, sms, s), s, flags, "residual forward launch");
}

size_t trimul_residual_backward_workspace_bytes(const trimul_residual_params* p, int B, int I, int J) {
  if (!p || check_width(p->D) != TRIMUL_OK || check_pairs(B, I, J) != TRIMUL_OK) return 0;
  // for any device: as many blocks as the largest launch has on 256 SMs
  return residual_backward_workspace(p->D, static_cast<long long>(B) * I * J, 256);
}

trimul_status trimul_residual_backward(const trimul_residual_params* p, const void* x, const uint16_t* u,
                                       const uint16_t* gate, const uint16_t* mask, const void* dout,
                                       const void* dout2, const uint16_t* dnormed, int B, int I, int J, void* dx,
                                       uint16_t* du, uint16_t* dgate, const trimul_residual_grads* grads,
                                       void* workspace, size_t workspace_bytes, int device, void* stream,
                                       unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK));
  TRY(check_residual(p, gate, mask, B, I, J));
  if (!x || !u || !dout || !dx || !du || !grads) return fail(TRIMUL_ERR_INVALID_ARG, "x, u, dout, dx, du or grads is null");
  if ((p->pre_norm == TRIMUL_NORM_NONE) != !dnormed) return fail(TRIMUL_ERR_INVALID_ARG, "dnormed and pre_norm do not agree");
  if (dgate && p->gate != TRIMUL_GATE_PAIR)
    return fail(TRIMUL_ERR_INVALID_ARG, "dgate: only a gate of every pair has a gradient");
  for (const void* q : {x, (const void*)u, dout, dout2, (const void*)dnormed, (const void*)dx, (const void*)du, (const void*)dgate})
    if (!aligned(q, 16)) return fail(TRIMUL_ERR_INVALID_ARG, "x, u, dout, dout2, dnormed, dx, du and dgate must be 16-byte aligned");
  const struct {
    float* to;
    bool has;
    const char* name;
  } gs[] = {{grads->post_gamma, p->post_norm != TRIMUL_NORM_NONE, "post_gamma"},
            {grads->post_beta, p->post_norm == TRIMUL_NORM_LAYER, "post_beta"},
            {grads->pre_gamma, p->pre_norm != TRIMUL_NORM_NONE, "pre_gamma"},
            {grads->pre_beta, p->pre_norm == TRIMUL_NORM_LAYER, "pre_beta"},
            {grads->channel, true, "channel"}};
  const size_t n = static_cast<size_t>(B) * I * J * p->D, w = n * type_bytes(p->stream_type), wd = p->D * 4;
  const size_t need = trimul_residual_backward_workspace_bytes(p, B, I, J);
  for (const auto& g : gs) {
    if (g.to && !g.has) return fail(TRIMUL_ERR_INVALID_ARG, "there is no %s to give a gradient of", g.name);
    if (!aligned(g.to, 4)) return fail(TRIMUL_ERR_INVALID_ARG, "the gradient of %s must be 4-byte aligned", g.name);
  }
  TRY(check_workspace(workspace, workspace_bytes, need, 16));
  const Buffer in[] = {{dout, w, "dout"}, {dout2, w, "dout2"}, {x, w, "x"}, {u, n * 2, "u"},
                       {gate, gate_elems(p, B, I, J) * 2, "gate"}, {mask, n / p->D * 2, "mask"}, {dnormed, n * 2, "dnormed"},
                       {p->post_gamma, wd, "post_gamma"}, {p->post_beta, wd, "post_beta"}, {p->pre_gamma, wd, "pre_gamma"},
                       {p->pre_beta, wd, "pre_beta"}, {p->channel, wd, "channel"}};
  const Buffer to[] = {{dx, w, "dx"}, {du, n * 2, "du"}, {dgate, n * 2, "dgate"}, {gs[0].to, wd, "the gradient of post_gamma"},
                       {gs[1].to, wd, "the gradient of post_beta"}, {gs[2].to, wd, "the gradient of pre_gamma"},
                       {gs[3].to, wd, "the gradient of pre_beta"}, {gs[4].to, wd, "the gradient of channel"},
                       {workspace, need, "workspace"}};
  TRY(check_apart(in, 12, to, 9));
  int sms = 0;
  TRY(device_sms(device, &sms));
  DeviceScope scope;
  TRY(scope.enter(device));
  ResidualArgs a = residual_args(p, x, u, gate, mask, B, I, J);
  a.dout = dout, a.dout2 = dout2, a.dnormed = dnormed;
  a.dx = dx, a.du = du, a.dgate = dgate;
  a.g = *grads;
  a.part = static_cast<float*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return finish(launch_residual_backward(a, sms, s), s, flags, "residual backward launch");
}

size_t trimul_grad_workspace_bytes(int n) { return n < 0 ? 0 : grad_workspace(n, 256); }

trimul_status trimul_grad_norm(const trimul_grad_tensor* tensors, int n, trimul_norm_kind kind, float* norm,
                               void* workspace, size_t workspace_bytes, int device, void* stream, unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK));
  const size_t need = trimul_grad_workspace_bytes(n);
  TRY(check_tensors(tensors, n, kind, norm, workspace, need, false));
  TRY(check_workspace(workspace, workspace_bytes, need, 16));
  int sms = 0;
  TRY(device_sms(device, &sms));
  DeviceScope scope;
  TRY(scope.enter(device));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return finish(launch_grad_norm(tensors, n, kind, norm, workspace, false, INFINITY, sms, s), s, flags, "gradient norm launch");
}

trimul_status trimul_grad_clip(const trimul_grad_tensor* tensors, int n, float max_norm, trimul_norm_kind kind,
                               float* norm, void* workspace, size_t workspace_bytes, int device, void* stream,
                               unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK));
  if (!(max_norm >= 0.0f)) return fail(TRIMUL_ERR_INVALID_ARG, "max_norm must be >= 0");
  const size_t need = trimul_grad_workspace_bytes(n);
  TRY(check_tensors(tensors, n, kind, norm, workspace, need, true));
  TRY(check_workspace(workspace, workspace_bytes, need, 16));
  int sms = 0;
  TRY(device_sms(device, &sms));
  DeviceScope scope;
  TRY(scope.enter(device));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return finish(launch_grad_norm(tensors, n, kind, norm, workspace, true, max_norm, sms, s), s, flags, "gradient clip launch");
}

}  // extern "C"
