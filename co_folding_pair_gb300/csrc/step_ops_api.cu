// step_ops_api.cu -- the C ABI's entry point of AdamW (include/trimul.h): argument
// checks and the launch.  Those of the linear layer in 8 bits are in linear8_api.cu.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "trimul.h"
#include "api_checks.h"
#include "api_status.h"
#include "step_ops.h"

using namespace trimul;

namespace {

// ------------------------------------------------------------------ AdamW
trimul_status check_adamw(const trimul_adamw_params* p, int n, const trimul_adamw_tensor* t, const trimul_grad_tensor* g,
                          const int32_t* count) {
  if (!p) return fail(TRIMUL_ERR_INVALID_ARG, "params is null");
  if (n < 0) return fail(TRIMUL_ERR_INVALID_ARG, "n (%d) must be >= 0", n);
  if (n > 0 && (!t || !g)) return fail(TRIMUL_ERR_INVALID_ARG, "tensors or grads is null");
  if (!(p->beta1 >= 0.0 && p->beta1 < 1.0) || !(p->beta2 >= 0.0 && p->beta2 < 1.0))
    return fail(TRIMUL_ERR_INVALID_ARG, "beta1 (%g) and beta2 (%g) must be in [0, 1)", p->beta1, p->beta2);
  if (!std::isnormal(p->eps) || p->eps < 0.0f) return fail(TRIMUL_ERR_INVALID_ARG, "eps must be a normal number > 0");
  if (!p->lr_device && !std::isfinite(p->lr)) return fail(TRIMUL_ERR_INVALID_ARG, "lr must be finite");
  if (p->norm && !(p->max_norm >= 0.0f)) return fail(TRIMUL_ERR_INVALID_ARG, "max_norm must be >= 0");
  if (p->states != TRIMUL_STATES_F32 && p->states != TRIMUL_STATES_E4M3)
    return fail(TRIMUL_ERR_INVALID_ARG, "unknown states %d", static_cast<int>(p->states));
  if (p->rounding != TRIMUL_ROUND_NEAREST && p->rounding != TRIMUL_ROUND_STOCHASTIC)
    return fail(TRIMUL_ERR_INVALID_ARG, "unknown rounding %d", static_cast<int>(p->rounding));
  if (!count || !aligned(count, 4)) return fail(TRIMUL_ERR_INVALID_ARG, "count is null or not 4-byte aligned");
  if (!aligned(p->lr_device, 4) || !aligned(p->norm, 4)) return fail(TRIMUL_ERR_INVALID_ARG, "lr_device and norm must be 4-byte aligned");
  if (overlap(count, 8, p->lr_device, 4) || overlap(count, 8, p->norm, 4))
    return fail(TRIMUL_ERR_INVALID_ARG, "count overlaps lr_device or norm");
  const bool codes = p->states == TRIMUL_STATES_E4M3;
  int64_t all = 0;
  for (int k = 0; k < n; ++k) {
    const trimul_adamw_tensor& a = t[k];
    if (a.numel < 0) return fail(TRIMUL_ERR_SHAPE, "tensor %d: numel (%lld) must be >= 0", k, static_cast<long long>(a.numel));
    if (a.numel >= (1ll << 40) || (all += a.numel) >= (1ll << 41))
      return fail(TRIMUL_ERR_SHAPE, "tensor %d: numel (%lld) is too large", k, static_cast<long long>(a.numel));
    if (a.param_type != TRIMUL_F32 && a.param_type != TRIMUL_BF16)
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: param_type must be BF16 or F32", k);
    if (g[k].numel != a.numel)
      return fail(TRIMUL_ERR_SHAPE, "tensor %d: its gradient has %lld elements, not %lld", k, static_cast<long long>(g[k].numel), static_cast<long long>(a.numel));
    if (g[k].type != TRIMUL_F32 && g[k].type != TRIMUL_BF16 && g[k].type != TRIMUL_F16)
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: unknown type %d of its gradient", k, static_cast<int>(g[k].type));
    if (a.copy && a.copy_type != TRIMUL_BF16 && a.copy_type != TRIMUL_F16)
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: copy_type must be BF16 or F16", k);
    if (!std::isfinite(a.weight_decay) || a.weight_decay < 0.0f)
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: weight_decay must be finite and >= 0", k);
    if (a.numel == 0) continue;
    const size_t num = static_cast<size_t>(a.numel), state = num * (codes ? 1 : 4);
    const size_t scales = codes ? (num + TRIMUL_STATE_BLOCK - 1) / TRIMUL_STATE_BLOCK * 4 : 0;
    if (!a.param || !aligned(a.param, type_bytes(a.param_type)))
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: param is null or not aligned to its type", k);
    if (!g[k].data || !aligned(g[k].data, type_bytes(g[k].type)))
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: grad is null or not aligned to its type", k);
    if (!aligned(a.copy, 2)) return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: copy is not aligned to its type", k);
    if (!a.m || !a.v || !aligned(a.m, 16) || !aligned(a.v, 16))
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: m or v is null or not 16-byte aligned", k);
    if (codes && (!a.m_scale || !a.v_scale || !aligned(a.m_scale, 4) || !aligned(a.v_scale, 4)))
      return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: m_scale or v_scale is null or not 4-byte aligned", k);
    const Buffer all_of[] = {{a.param, num * type_bytes(a.param_type), "param"}, {a.copy, num * 2, "copy"},
                             {a.m, state, "m"}, {a.v, state, "v"}, {codes ? a.m_scale : nullptr, scales, "m_scale"},
                             {codes ? a.v_scale : nullptr, scales, "v_scale"}, {count, 8, "count"},
                             {g[k].data, num * type_bytes(g[k].type), "grad"}, {p->norm, 4, "norm"}, {p->lr_device, 4, "lr_device"}};
    constexpr int kOutputs = 6;  // of these; what comes behind is read (count: seen to above)
    for (int x = 0; x < kOutputs; ++x)
      for (int y = x + 1; y < 10; ++y)
        if (overlap(all_of[x].p, all_of[x].bytes, all_of[y].p, all_of[y].bytes))
          return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: %s overlaps %s", k, all_of[x].name, all_of[y].name);
    if (overlap(count, 8, g[k].data, num * type_bytes(g[k].type))) return fail(TRIMUL_ERR_INVALID_ARG, "tensor %d: count overlaps grad", k);
  }
  return TRIMUL_OK;
}

}  // namespace

extern "C" {

trimul_status trimul_adamw_step(const trimul_adamw_params* p, const trimul_adamw_tensor* tensors, const trimul_grad_tensor* grads,
                                int n, int32_t* count, int device, void* stream, unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK));
  TRY(check_adamw(p, n, tensors, grads, count));
  int sms = 0;
  TRY(device_sms(device, &sms));
  DeviceScope scope;
  TRY(scope.enter(device));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return finish(launch_adamw(*p, tensors, grads, n, count, sms, s), s, flags, "AdamW launch");
}

}  // extern "C"
