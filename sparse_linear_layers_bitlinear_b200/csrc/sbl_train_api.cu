// C ABI of the operators around the products (norm, AdamW, linear cross
// entropy): argument checks and dispatch.  See include/sbl.h for the contract.
#include <algorithm>
#include <cmath>
#include <functional>
#include <vector>

#include "sbl_kernels.h"

using namespace sbl;

namespace {

constexpr uint32_t kNormFwdFlags = SBL_NORM_X_F32 | SBL_NORM_STREAM_F32 | SBL_NORM_W_F32;
constexpr uint32_t kNormBwdFlags = SBL_NORM_STREAM_F32 | SBL_NORM_W_F32 | SBL_NORM_DY_F32;
constexpr uint32_t kAdamFlags = SBL_ADAMW_GRAD_F32 | SBL_ADAMW_STATE_8BIT | SBL_ADAMW_NO_DECAY;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kCeMaxRows = int64_t(1) << 22, kCeMaxD = 131072;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool all_aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 16)) return false;
  return true;
}

sbl_status code(cudaError_t e) { return e == cudaSuccess ? SBL_OK : SBL_ERR_CUDA; }

bool norm_shape(int64_t t, int64_t k) {
  return t >= 0 && t <= kMaxRows && k >= 8 && k % 8 == 0 && k <= SBL_NORM_MAX_K;
}

bool ce_shape(int64_t t, int64_t v, int64_t d) {
  return t >= 0 && t <= kCeMaxRows && v >= 1 && v <= kCeMaxRows && d >= 8 && d % 8 == 0 && d <= kCeMaxD;
}

bool factor(double x) { return std::isfinite(x) && x >= 0.0; }

}  // namespace

extern "C" {

sbl_status sbl_rmsnorm_forward(const sbl_rmsnorm_args* args, sbl_stream_t stream) {
  if (args == nullptr) return SBL_ERR_INVALID_ARG;
  const sbl_rmsnorm_args& a = *args;
  if ((a.flags & ~kNormFwdFlags) != 0u || a.reserved != 0u) return SBL_ERR_INVALID_ARG;
  if (!norm_shape(a.t, a.k)) return SBL_ERR_SHAPE;
  if (!(a.eps >= 1e-12 && a.eps <= 1.0)) return SBL_ERR_INVALID_ARG;
  if (a.t == 0) return SBL_OK;
  if (a.x == nullptr) return SBL_ERR_INVALID_ARG;
  if (!a.h_out && !a.xn_out && !a.xhat_out && !a.xq_out && !a.xscale_out && !a.rstd_out) return SBL_ERR_INVALID_ARG;
  if (!all_aligned16({a.x, a.residual, a.weight, a.h_out, a.xn_out, a.xhat_out, a.xq_out, a.xscale_out, a.rstd_out}) ||
      !aligned(a.status_dev, 4))
    return SBL_ERR_ALIGN;
  int sms = 0;
  const sbl_status st = current_device(&sms);
  if (st != SBL_OK) return st;
  return code(launch_rmsnorm(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t sbl_rmsnorm_backward_workspace_bytes(int64_t t, int64_t k) {
  if (!norm_shape(t, k) || t == 0) return 0;
  return size_t(rmsnorm_bwd_max_blocks(t)) * size_t(k) * 4;
}

sbl_status sbl_rmsnorm_backward(const sbl_rmsnorm_backward_args* args, sbl_stream_t stream) {
  if (args == nullptr) return SBL_ERR_INVALID_ARG;
  const sbl_rmsnorm_backward_args& a = *args;
  if ((a.flags & ~kNormBwdFlags) != 0u || a.dy_count < 1 || a.dy_count > 3) return SBL_ERR_INVALID_ARG;
  if (!norm_shape(a.t, a.k)) return SBL_ERR_SHAPE;
  if (!aligned(a.dw, 16)) return SBL_ERR_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  if (a.t == 0) {
    if (a.dw == nullptr) return SBL_OK;
    const sbl_status st = current_device(&sms);
    if (st != SBL_OK) return st;
    return code(cudaMemsetAsync(a.dw, 0, size_t(a.k) * 4, s));
  }
  if (a.h == nullptr || a.rstd == nullptr || a.dh == nullptr) return SBL_ERR_INVALID_ARG;
  for (int i = 0; i < a.dy_count; ++i) {
    if (a.dys[i] == nullptr) return SBL_ERR_INVALID_ARG;
    if (!aligned(a.dys[i], 16)) return SBL_ERR_ALIGN;
  }
  if (a.dw != nullptr && a.workspace == nullptr) return SBL_ERR_INVALID_ARG;
  if (!all_aligned16({a.h, a.weight, a.dres, a.dh, a.dx, a.workspace}) || !aligned(a.rstd, 4)) return SBL_ERR_ALIGN;
  const sbl_status st = current_device(&sms);
  if (st != SBL_OK) return st;
  return code(launch_rmsnorm_bwd(a, sms, s));
}

sbl_status sbl_adamw_step(const sbl_adamw_tensor* tensors, int32_t count, const sbl_adamw_params* params,
                          uint32_t* status_dev, sbl_stream_t stream) {
  if (count < 0 || params == nullptr || (count > 0 && tensors == nullptr)) return SBL_ERR_INVALID_ARG;
  const sbl_adamw_params& q = *params;
  if (!(q.beta1 >= 0.0 && q.beta1 < 1.0 && q.beta2 >= 0.0 && q.beta2 < 1.0)) return SBL_ERR_INVALID_ARG;
  if (!factor(q.lr) || !factor(q.eps) || !factor(q.weight_decay)) return SBL_ERR_INVALID_ARG;
  if (q.step_dev == nullptr && q.step < 1) return SBL_ERR_INVALID_ARG;
  if (!aligned(q.lr_dev, 4) || !aligned(q.step_dev, 8) || !aligned(q.grad_scale_dev, 4) || !aligned(status_dev, 4))
    return SBL_ERR_ALIGN;
  try {
    std::vector<const void*> ws;
    ws.reserve(static_cast<size_t>(count));
    for (int32_t i = 0; i < count; ++i) {
      const sbl_adamw_tensor& t = tensors[i];
      if ((t.flags & ~kAdamFlags) != 0u || t.reserved != 0u) return SBL_ERR_INVALID_ARG;
      if (t.numel < 0 || t.numel > (int64_t(1) << 40)) return SBL_ERR_SHAPE;
      if (t.numel == 0) continue;
      if (t.w == nullptr || t.grad == nullptr || t.m == nullptr || t.v == nullptr) return SBL_ERR_INVALID_ARG;
      if ((t.flags & SBL_ADAMW_STATE_8BIT) && (t.m_scale == nullptr || t.v_scale == nullptr))
        return SBL_ERR_INVALID_ARG;
      if (!all_aligned16({t.w, t.master, t.grad, t.m, t.v}) || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
        return SBL_ERR_ALIGN;
      // one array in two places of an entry (between entries only w is looked at: a call is short)
      if ((t.m == t.v) | (t.m == t.w) | (t.v == t.w) | (t.grad == t.w) | (t.grad == t.m) | (t.grad == t.v) |
          (t.master == t.w) | (t.master == t.m) | (t.master == t.v) | (t.master == t.grad))
        return SBL_ERR_INVALID_ARG;
      if (t.flags & SBL_ADAMW_STATE_8BIT)
        for (const void* scale : {t.m_scale, t.v_scale})
          if (t.m_scale == t.v_scale || scale == t.w || scale == t.master || scale == t.grad || scale == t.m ||
              scale == t.v)
            return SBL_ERR_INVALID_ARG;
      ws.push_back(t.w);
    }
    if (ws.empty()) return SBL_OK;
    // ascending addresses, as an allocator gives them, need no sorting
    if (std::adjacent_find(ws.begin(), ws.end(), std::greater_equal<const void*>()) != ws.end())
      std::sort(ws.begin(), ws.end());
    if (std::adjacent_find(ws.begin(), ws.end()) != ws.end()) return SBL_ERR_INVALID_ARG;  // the same tensor twice
    int sms = 0;
    const sbl_status st = current_device(&sms);
    if (st != SBL_OK) return st;
    // up to kAdamMaxTensors of one kind of states a launch, empty ones left out
    for (const uint32_t kind : {0u, uint32_t(SBL_ADAMW_STATE_8BIT)}) {
      sbl_adamw_tensor batch[kAdamMaxTensors];
      int n = 0;
      uint64_t elements = 0;
      auto launch = [&] {
        const int count = n;
        n = 0;
        elements = 0;
        return count == 0 || launch_adamw(batch, count, q, status_dev, reinterpret_cast<cudaStream_t>(stream)) ==
                                 cudaSuccess;
      };
      for (int32_t i = 0; i < count; ++i) {
        const sbl_adamw_tensor& t = tensors[i];
        if (t.numel == 0 || (t.flags & SBL_ADAMW_STATE_8BIT) != kind) continue;
        if ((n == kAdamMaxTensors || elements + uint64_t(t.numel) > (uint64_t(1) << 40)) && !launch())
          return SBL_ERR_CUDA;
        batch[n++] = t;
        elements += uint64_t(t.numel);
      }
      if (!launch()) return SBL_ERR_CUDA;
    }
    return SBL_OK;
  } catch (...) {
    return SBL_ERR_INVALID_ARG;  // a count the host cannot hold
  }
}

size_t sbl_linear_ce_workspace_bytes(int64_t t, int64_t v, int64_t d, int32_t backward) {
  if (!ce_shape(t, v, d) || t == 0) return 0;
  return static_cast<size_t>(linear_ce_workspace(t, v, d, backward != 0));
}

sbl_status sbl_linear_ce_forward(const sbl_linear_ce_args* args, sbl_stream_t stream) {
  if (args == nullptr) return SBL_ERR_INVALID_ARG;
  const sbl_linear_ce_args& a = *args;
  if (!ce_shape(a.t, a.v, a.d)) return SBL_ERR_SHAPE;
  if (a.t == 0) return SBL_OK;
  if (!a.h || !a.w || !a.targets || !a.loss || !a.lse || !a.workspace) return SBL_ERR_INVALID_ARG;
  if (!all_aligned16({a.h, a.w}) || !aligned(a.targets, 8) || !aligned(a.loss, 4) || !aligned(a.lse, 4) ||
      !aligned(a.workspace, 256) || !aligned(a.status_dev, 4))
    return SBL_ERR_ALIGN;
  int sms = 0;
  const sbl_status st = current_device(&sms);
  if (st != SBL_OK) return st;
  return code(launch_linear_ce(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

sbl_status sbl_linear_ce_backward(const sbl_linear_ce_backward_args* args, sbl_stream_t stream) {
  if (args == nullptr) return SBL_ERR_INVALID_ARG;
  const sbl_linear_ce_backward_args& a = *args;
  if (!ce_shape(a.t, a.v, a.d)) return SBL_ERR_SHAPE;
  if (a.dloss_stride != 0 && a.dloss_stride != 1) return SBL_ERR_INVALID_ARG;
  if (a.dw == nullptr) return SBL_ERR_INVALID_ARG;
  if (!aligned(a.dw, 16)) return SBL_ERR_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  sbl_status st;
  if (a.t == 0) {  // no rows: dh is empty and dw = 0
    if ((st = current_device(&sms)) != SBL_OK) return st;
    return code(cudaMemsetAsync(a.dw, 0, size_t(a.v) * size_t(a.d) * 2, s));
  }
  if (!a.h || !a.w || !a.targets || !a.lse || !a.dloss || !a.dh || !a.workspace) return SBL_ERR_INVALID_ARG;
  if (!all_aligned16({a.h, a.w, a.dh}) || !aligned(a.targets, 8) || !aligned(a.lse, 4) || !aligned(a.dloss, 4) ||
      !aligned(a.workspace, 256) || !aligned(a.status_dev, 4))
    return SBL_ERR_ALIGN;
  if ((st = current_device(&sms)) != SBL_OK) return st;
  try {
    return code(launch_linear_ce_bwd(a, sms, s));
  } catch (...) {
    return SBL_ERR_CUDA;  // no host memory for the tile schedule
  }
}

}  // extern "C"
