// Output head with 4-bit weights: logits of hidden states,
//   y[b][v] = sum_g s[v][g] sum_{k in g} x[b][k] (q[v][k] - z[v][g]),
// q the codes 0..15, s a scale and z a zero point per row and group of k.
//
// One wave per vocabulary row and hidden row: each lane takes every 64th
// dword of the row's codes (8 columns, inside one group), and the wave adds
// the lanes' sums.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qs.h"
#include "qs_device.hpp"
#include "qs_head.hpp"

namespace qs {
namespace head {
namespace {

constexpr int kBlock = 256;

__global__ void __launch_bounds__(kBlock) head_kernel(Args a) {
  const int v = blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
  if (v >= a.V) return;
  const int lane = lane_id();
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes + (size_t)v * a.codes_stride);
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const uint16_t* x = a.hidden + (size_t)b * a.hidden_stride;
    float acc = 0.0f;
    for (int i = lane; i < a.K / 8; i += 64) {
      const uint32_t c = codes[i];
      const int g = i * 8 / a.group;
      const size_t gi = (size_t)v * a.scale_stride + g;
      const float s = a.scale_dtype == QS_F32
                          ? static_cast<const float*>(a.scales)[gi]
                          : __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.scales)[gi] << 16);
      const float zero = a.zeros ? (float)a.zeros[(size_t)v * a.zero_stride + g] : 8.0f;
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        t += __uint_as_float((uint32_t)x[i * 8 + j] << 16) * ((float)((c >> (4 * j)) & 15u) - zero);
      acc += s * t;
    }
    for (int off = 32; off > 0; off >>= 1) acc += __shfl_xor(acc, off, 64);
    if (lane == 0) {
      const size_t o = (size_t)b * a.row_stride + v;
      if (a.logits_dtype == QS_F32) static_cast<float*>(a.logits)[o] = acc;
      else static_cast<__bf16*>(a.logits)[o] = (__bf16)acc;
    }
  }
}

}  // namespace

hipError_t launch_head(const Args& a, hipStream_t st) {
  const unsigned gx = (unsigned)((a.V + kBlock / 64 - 1) / (kBlock / 64));
  const unsigned gy = (unsigned)(a.B < 64 ? a.B : 64);
  hipLaunchKernelGGL(head_kernel, dim3(gx, gy), dim3(kBlock), 0, st, a);
  return hipGetLastError();
}

}  // namespace head
}  // namespace qs
