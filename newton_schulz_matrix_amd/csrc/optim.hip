// optim.hip - C entry point of the AdamW step (adamw.hpp), for the parameters
// that the Muon step leaves out.
#include <math.h>

#include <algorithm>

#include "adamw.hpp"
#include "host.hpp"

namespace {

using namespace nsk;

// Blocks of a launch: eight per compute unit, which walk the chunks.
constexpr int64_t kAdamwBlocks = 2048;

ns_status check_tensor(const ns_adamw_tensor& t) {
  if (t.numel < 0 || t.reserved != 0 || !isfinite(t.lr) || !isfinite(t.weight_decay)) return NS_ERR_INVALID_ARG;
  if (!known(t.param_dtype) || !known(t.grad_dtype) || (t.copy && !known(t.copy_dtype)))
    return NS_ERR_UNSUPPORTED_DTYPE;
  if (t.numel > 0 && (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq)) return NS_ERR_INVALID_ARG;
  // Chunks are counted in 32 bits.
  return t.numel <= int64_t(1) << 40 ? NS_OK : NS_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

ns_status ns_adamw_step(const ns_adamw_tensor* tensors, int64_t count, double beta1, double beta2, float eps,
                        int64_t step, const int32_t* d_step, const float* d_grad_scale, const float* d_lr_scale,
                        int32_t* d_status, ns_stream_t stream) {
  if (count < 0 || (count > 0 && !tensors)) return NS_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return NS_ERR_INVALID_ARG;
  if (!(eps >= 0.f && isfinite(eps)) || (!d_step && step < 1)) return NS_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    const ns_status s = check_tensor(tensors[i]);
    if (s != NS_OK) return s;
  }
  AdamwArgs a;
  a.b1 = (float)beta1;
  a.a1 = (float)(1.0 - beta1);
  a.b2 = (float)beta2;
  a.a2 = (float)(1.0 - beta2);
  a.eps = eps;
  a.c1 = a.c2 = 1.f;
  if (!d_step) {
    a.c1 = (float)(1.0 / (1.0 - pow(beta1, (double)step)));
    a.c2 = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
  }
  a.log_b1 = log(beta1);  // -inf for 0: 1 - 0^t is 1
  a.log_b2 = log(beta2);
  a.d_step = d_step;
  a.d_grad_scale = d_grad_scale;
  a.d_lr_scale = d_lr_scale;
  a.d_status = d_status;
  a.status_bits = (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  for (int64_t i = 0; i < count;) {
    a.count = 0;
    int64_t chunks = 0;
    for (; i < count && a.count < kAdamwItems; ++i) {
      const ns_adamw_tensor& t = tensors[i];
      if (t.numel == 0) continue;
      const int64_t more = (t.numel + kAdamwChunk - 1) / kAdamwChunk;
      if (chunks + more >= int64_t(1) << 31 && a.count > 0) break;
      a.types[a.count] = (int32_t)t.param_dtype | (int32_t)t.grad_dtype << 4 | (t.copy ? (int32_t)t.copy_dtype : 0) << 8;
      a.first[a.count] = (int32_t)chunks;
      AdamwItem& o = a.item[a.count++];
      o.p = t.param;
      o.g = t.grad;
      o.m = t.exp_avg;
      o.v = t.exp_avg_sq;
      o.scales = t.scales;
      o.copy = t.copy;
      o.n = t.numel;
      o.lr = t.lr;
      o.decay = t.weight_decay;
      chunks += more;
    }
    if (a.count == 0) break;
    a.chunks = (int)chunks;
    hipLaunchKernelGGL(k_adamw, dim3((unsigned)std::min(chunks, kAdamwBlocks)), dim3(kAdamwThreads), 0, st, a);
    const ns_status s = launched();
    if (s != NS_OK) return s;
  }
  return NS_OK;
}

}  // extern "C"
