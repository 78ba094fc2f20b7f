// learn_api.cu -- the C ABI (include/moe_zc.h) of the operators with which the
// router and the weights learn: argument checks and launches.  They keep no
// state and no workspace of the library's own, so calls on different streams
// (or captured into different graphs) are independent.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <vector>

#include "../../include/moe_zc.h"
#include "learn.cuh"

namespace {

using namespace moezc;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int status_of(cudaError_t e) {
  if (e == cudaSuccess) return MOE_ZC_OK;
  cudaGetLastError();
  return MOE_ZC_ERR_CUDA;
}

// Sizes that the balance loss and the logits' gradient share.
int check_rows(int64_t T, int32_t S, int32_t E, int32_t K) {
  if (T < 0 || S < 0 || E < 1 || K < 1 || K > E) return MOE_ZC_ERR_INVALID_ARG;
  if (K > MOE_ZC_MAX_K || E > MOE_ZC_MAX_E) return MOE_ZC_ERR_UNSUPPORTED;
  if (T > 0x7fffffffLL - S) return MOE_ZC_ERR_UNSUPPORTED;   // (offsets are int32)
  if (S > (1 << 27)) return MOE_ZC_ERR_UNSUPPORTED;           // (8 CTAs each)
  return MOE_ZC_OK;
}

}  // namespace

extern "C" {

int moe_zc_balance_workspace(int64_t T, int32_t S, int32_t E, int64_t* bytes) {
  if (!bytes) return MOE_ZC_ERR_INVALID_ARG;
  const int s = check_rows(T, S, E, 1);
  if (s != MOE_ZC_OK) return s;
  *bytes = static_cast<int64_t>(balance_plan(T, S, E).bytes);
  return MOE_ZC_OK;
}

int moe_zc_balance_loss(const float* logits, const float* logit_offset, const int32_t* idx,
                        const uint8_t* mask, const int32_t* seq_start, const float* weight,
                        int64_t T, int32_t S, int32_t E, int32_t K, float* loss, int32_t* counts,
                        float* prob, float* coef, void* workspace, int64_t workspace_bytes,
                        void* stream) {
  const int s = check_rows(T, S, E, K);
  if (s != MOE_ZC_OK) return s;
  if (T > 0 && (!logits || !idx)) return MOE_ZC_ERR_INVALID_ARG;
  if (!seq_start && S != 1) return MOE_ZC_ERR_INVALID_ARG;
  if (S > 0 && (!loss || !counts || !prob || !coef || !workspace)) return MOE_ZC_ERR_INVALID_ARG;
  if (S > 0 && workspace_bytes < static_cast<int64_t>(balance_plan(T, S, E).bytes))
    return MOE_ZC_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(logit_offset, 16) || !aligned(coef, 16) ||
      !aligned(workspace, 16) || !aligned(idx, 4) || !aligned(seq_start, 4) ||
      !aligned(weight, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(prob, 4))
    return MOE_ZC_ERR_UNSUPPORTED;
  return status_of(launch_balance_loss(logits, logit_offset, idx, mask, seq_start, weight, T, S, E,
                                       K, loss, counts, prob, coef, workspace,
                                       static_cast<cudaStream_t>(stream)));
}

int moe_zc_route_backward(const float* logits, const float* logit_offset, const int32_t* idx,
                          const float* dgate, const uint8_t* mask, const int32_t* seq_start,
                          const float* coef, const float* dloss, int64_t T, int32_t S, int32_t E,
                          int32_t K, void* dlogits, int32_t dtype, void* stream) {
  const int s = check_rows(T, S, E, K);
  if (s != MOE_ZC_OK) return s;
  if (dtype != MOE_ZC_F32 && dtype != MOE_ZC_BF16) return MOE_ZC_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !dlogits)) return MOE_ZC_ERR_INVALID_ARG;
  if (T > 0 && dgate && !idx) return MOE_ZC_ERR_INVALID_ARG;
  if (coef && (!dloss || (!seq_start && S != 1))) return MOE_ZC_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(logit_offset, 16) || !aligned(coef, 16) ||
      !aligned(dlogits, 16) || !aligned(idx, 4) || !aligned(dgate, 4) || !aligned(seq_start, 4) ||
      !aligned(dloss, 4))
    return MOE_ZC_ERR_UNSUPPORTED;
  return status_of(launch_route_backward(logits, logit_offset, idx, dgate, mask, seq_start, coef,
                                         dloss, T, S, E, K, dlogits, dtype == MOE_ZC_BF16,
                                         static_cast<cudaStream_t>(stream)));
}

int moe_zc_combine_backward(const void* dout, const void* x, const void* y_rows,
                            const int32_t* slot, const float* gate, int64_t T, int32_t d,
                            int32_t K, int64_t rows, float* dgate, void* dy_rows, void* stream) {
  if (T < 0 || K < 1 || d <= 0 || rows < 0) return MOE_ZC_ERR_INVALID_ARG;
  if (K > MOE_ZC_MAX_K) return MOE_ZC_ERR_UNSUPPORTED;
  if (T > 0 && (!dout || !x || !slot || !dgate)) return MOE_ZC_ERR_INVALID_ARG;
  if (T > 0 && rows > 0 && (!y_rows || (dy_rows && !gate))) return MOE_ZC_ERR_INVALID_ARG;
  if (d % 8 != 0 || T > 0x7fffffffLL) return MOE_ZC_ERR_UNSUPPORTED;
  if (!aligned(dout, 16) || !aligned(x, 16) || !aligned(y_rows, 16) || !aligned(dy_rows, 16) ||
      !aligned(slot, 4) || !aligned(gate, 4) || !aligned(dgate, 4))
    return MOE_ZC_ERR_UNSUPPORTED;
  return status_of(launch_combine_backward(
      static_cast<const __nv_bfloat16*>(dout), static_cast<const __nv_bfloat16*>(x),
      static_cast<const __nv_bfloat16*>(y_rows), slot, gate, T, d, K, rows, dgate,
      static_cast<__nv_bfloat16*>(rows > 0 ? dy_rows : nullptr),
      static_cast<cudaStream_t>(stream)));
}

int moe_zc_adamw(const moe_zc_adamw_tensor* tensors, int32_t n_tensors,
                 const moe_zc_adamw_args* args, int32_t* step, const float* lr_scale,
                 const float* grad_scale, void* stream) {
  if (n_tensors < 0 || !args || !step || (n_tensors > 0 && !tensors)) return MOE_ZC_ERR_INVALID_ARG;
  const moe_zc_adamw_args& a = *args;
  if ((a.param_type != MOE_ZC_F32 && a.param_type != MOE_ZC_BF16) ||
      (a.grad_type != MOE_ZC_F32 && a.grad_type != MOE_ZC_BF16) ||
      (a.state_bits != 32 && a.state_bits != 8) || (a.master != 0 && a.master != 1) ||
      (a.master && a.param_type != MOE_ZC_BF16))
    return MOE_ZC_ERR_INVALID_ARG;
  // (written so that a NaN fails)
  if (!(a.beta1 >= 0.0 && a.beta1 < 1.0) || !(a.beta2 >= 0.0 && a.beta2 < 1.0) ||
      !(static_cast<float>(a.eps) >= 0x1p-126f) || !std::isfinite(a.eps) || !std::isfinite(a.lr) ||
      !std::isfinite(a.weight_decay))
    return MOE_ZC_ERR_INVALID_ARG;
  if (!aligned(step, 4) || !aligned(lr_scale, 4) || !aligned(grad_scale, 4))
    return MOE_ZC_ERR_UNSUPPORTED;
  if (n_tensors == 0) return MOE_ZC_OK;
  const bool bits8 = a.state_bits == 8;
  static_assert(sizeof(AdamTensor) == sizeof(moe_zc_adamw_tensor), "one layout");
  for (int32_t i = 0; i < n_tensors; ++i) {
    const moe_zc_adamw_tensor& t = tensors[i];
    if (t.n < 0) return MOE_ZC_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || (a.master && !t.master) ||
        (bits8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
      return MOE_ZC_ERR_INVALID_ARG;
    if (t.n > (1LL << 40)) return MOE_ZC_ERR_UNSUPPORTED;
    if (!aligned(t.param, 16) || !aligned(t.grad, 16) || !aligned(t.exp_avg, 16) ||
        !aligned(t.exp_avg_sq, 16) || (a.master && !aligned(t.master, 16)) ||
        (bits8 && (!aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4))))
      return MOE_ZC_ERR_UNSUPPORTED;
  }
  const AdamHyper h{a.lr, a.beta1, a.beta2, a.eps, a.weight_decay};
  return status_of(launch_adamw(reinterpret_cast<const AdamTensor*>(tensors), n_tensors,
                                a.param_type == MOE_ZC_BF16, a.grad_type == MOE_ZC_BF16,
                                a.master != 0, bits8, h, step, lr_scale, grad_scale,
                                static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
