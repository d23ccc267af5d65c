// Low-rank adapters of many requests beside a shared output projection: with a the
// adapter of row b,
//   y[b][v] = z[b][v] + scale[a] sum_r up[a][v][r] u[b][r],
//   u[b][r] = sum_k down[a][r][k] x[b][k].
// Two launches: the rows' low-rank coordinates u, in float32, then their product with
// the adapters' up factors on top of the logits. Products are exact in float32, sums
// are held in float32, and each logit is rounded once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qs.h"
#include "qs_adapters.hpp"
#include "qs_device.hpp"

namespace qs {
namespace adapters {
namespace {

constexpr int kBlock = 256;

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// One wave per row and rank.
__global__ void __launch_bounds__(kBlock) down_kernel(Args a) {
  const int lane = lane_id();
  const int64_t item = (int64_t)blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
  if (item >= (int64_t)a.B * a.rank) return;
  const int b = (int)(item / a.rank), q = (int)(item - (int64_t)b * a.rank);
  const int n = a.index[b];
  const bool valid = n >= -1 && n < a.count;
  if (q == 0 && lane == 0) a.status[b] = valid ? QS_ROW_OK : QS_ROW_BAD_PARAM;
  if (!valid || n < 0) return;
  const uint16_t* const x = a.hidden + (size_t)b * a.hidden_stride;
  const uint16_t* const w = a.down + (size_t)n * a.down_stride + (size_t)q * a.down_row_stride;
  float sum = 0.0f;
  for (int k = lane * 8; k < a.K; k += 512) {
    const uint4 xv = *reinterpret_cast<const uint4*>(x + k);
    const uint4 wv = *reinterpret_cast<const uint4*>(w + k);
    const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum = fmaf(lo(xs[e]), lo(ws[e]), sum);
      sum = fmaf(hi(xs[e]), hi(ws[e]), sum);
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if (lane == 0) a.low[item] = sum * (a.scale ? a.scale[n] : 1.0f);
}

// One thread per logit.
template <int DT>
__global__ void __launch_bounds__(kBlock) up_kernel(Args a, int chunks) {
  const int b = (int)(blockIdx.x / (unsigned)chunks);
  const int v = (int)(blockIdx.x - (unsigned)b * (unsigned)chunks) * kBlock + (int)threadIdx.x;
  if (v >= a.V) return;
  const int n = a.index[b];
  const bool adapted = n >= 0 && n < a.count;
  if (!adapted && a.out == a.logits) return;
  const uint8_t* const z = a.logits + (size_t)b * a.row_bytes;
  uint8_t* const out = a.out + (size_t)b * a.out_bytes;
  float sum = 0.0f;
  if (adapted) {
    const uint16_t* const w = a.up + (size_t)n * a.up_stride + (size_t)v * a.up_row_stride;
    const float* const u = a.low + (size_t)b * a.rank;
    for (int q = 0; q < a.rank; q += 8) {
      const uint4 wv = *reinterpret_cast<const uint4*>(w + q);
      const uint32_t ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum = fmaf(lo(ws[e]), u[q + 2 * e], sum);
        sum = fmaf(hi(ws[e]), u[q + 2 * e + 1], sum);
      }
    }
  }
  if constexpr (DT == QS_F32) {
    const float y = reinterpret_cast<const float*>(z)[v];
    reinterpret_cast<float*>(out)[v] = adapted ? y + sum : y;
  } else {
    const uint16_t y = reinterpret_cast<const uint16_t*>(z)[v];
    if (adapted)
      reinterpret_cast<__bf16*>(out)[v] = (__bf16)(__uint_as_float((uint32_t)y << 16) + sum);
    else
      reinterpret_cast<uint16_t*>(out)[v] = y;
  }
}

}  // namespace

size_t workspace_bytes(int64_t B, int64_t rank) {
  return ((size_t)B * (size_t)rank * sizeof(float) + 255) & ~(size_t)255;
}

bool grid_fits(int64_t B, int64_t V, int64_t rank) {
  const int64_t chunks = (V + kBlock - 1) / kBlock;
  return B * chunks * kBlock < (int64_t)1 << 32 && B * rank * 64 < (int64_t)1 << 32;
}

hipError_t launch_adapters(const Args& a, int dtype, hipStream_t st) {
  const int64_t items = (int64_t)a.B * a.rank;
  hipLaunchKernelGGL(down_kernel, dim3((unsigned)((items + 3) / 4)), dim3(kBlock), 0, st, a);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  const int chunks = (a.V + kBlock - 1) / kBlock;
  const dim3 grid((unsigned)a.B * (unsigned)chunks);
  if (dtype == QS_F32)
    hipLaunchKernelGGL((up_kernel<QS_F32>), grid, dim3(kBlock), 0, st, a, chunks);
  else
    hipLaunchKernelGGL((up_kernel<QS_BF16>), grid, dim3(kBlock), 0, st, a, chunks);
  return hipGetLastError();
}

}  // namespace adapters
}  // namespace qs
