// Gradient of the token log-probabilities and of the entropy with respect to
// the logits:
//   dz_i = (1/T) [ sum_g gl_g (1[i = t_g] - p_i) - gH p_i (log p_i + H) ]
// for legal i, 0 elsewhere, with log p_i = (z_i - m) / T - log S from the
// forward pass's row maximum and log sum.
//
// One thread per token; a token named by several slots gets their sum, added
// in slot order and rounded once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qs.h"
#include "qs_device.hpp"
#include "qs_score.hpp"

namespace qs {
namespace score {
namespace {

constexpr int kBlock = 256;

template <int DT>
__global__ void __launch_bounds__(kBlock) grad_kernel(GradArgs a) {
  const int r = blockIdx.x;
  const uint8_t* row = a.logits + (size_t)r * a.row_bytes;
  uint8_t* out = a.grad + (size_t)r * a.grad_bytes;
  const uint32_t* bm = a.bitmask ? a.bitmask + (size_t)r * a.bm_stride : nullptr;
  const int32_t* tokens = a.tokens + (size_t)r * a.G;
  const float* gl = a.g_lp + (size_t)r * a.G;
  const bool ok = a.status[r] == QS_ROW_OK;
  const float T = a.T ? a.T[r] : 1.0f;
  const float m = a.row_max[r], log_sum = a.log_sum[r];
  const float gH = a.g_ent ? a.g_ent[r] : 0.0f, H = a.g_ent ? a.entropy[r] : 0.0f;
  float gs = 0.0f;
  for (int g = 0; g < a.G; ++g)
    if (tokens[g] >= 0) gs += gl[g];
  for (int i = threadIdx.x; i < a.V; i += kBlock) {
    float v = 0.0f;
    if (ok && (bm == nullptr || ((bm[i >> 5] >> (i & 31)) & 1u))) {
      float z;
      if constexpr (DT == QS_F32) z = reinterpret_cast<const float*>(row)[i];
      else z = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
      const float lp = (z - m) / T - log_sum;
      const float p = __expf(lp);
      v = -p * gs;
      if (p > 0.0f) v -= gH * p * (lp + H);
      for (int g = 0; g < a.G; ++g)
        if (tokens[g] == i) v += gl[g];
      v /= T;
    }
    if constexpr (DT == QS_F32) reinterpret_cast<float*>(out)[i] = v;
    else reinterpret_cast<__bf16*>(out)[i] = (__bf16)v;
  }
}

}  // namespace

hipError_t launch_grad(const GradArgs& a, int dtype, int B, hipStream_t st) {
  if (dtype == QS_F32)
    hipLaunchKernelGGL(grad_kernel<QS_F32>, dim3((unsigned)B), dim3(kBlock), 0, st, a);
  else
    hipLaunchKernelGGL(grad_kernel<QS_BF16>, dim3((unsigned)B), dim3(kBlock), 0, st, a);
  return hipGetLastError();
}

}  // namespace score
}  // namespace qs
