// Log-probabilities of given tokens under the tempered, masked softmax of a
// row, with the row's entropy and its most probable tokens.
//
// With L the legal tokens, m = max_L z, d_i = (z_i - m) / T and
// S = sum_L exp d_i:
//   log p_t = d_t - log S,   H = log S - (1/S) sum_L exp(d_i) d_i.
// Both terms of H are non-negative, so nothing cancels. The top tokens are
// those of the largest z, ties by id.
//
// One workgroup per row: one pass for the maximum and the row's checks, one
// for the two sums, and one per top token (the largest key below the last).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qs.h"
#include "qs_device.hpp"
#include "qs_score.hpp"

namespace qs {
namespace score {
namespace {

constexpr int kBlock = 256;
constexpr int kBlockWaves = kBlock / 64;

template <int DT>
__device__ __forceinline__ float load_logit(const uint8_t* row, int i) {
  if constexpr (DT == QS_F32) return reinterpret_cast<const float*>(row)[i];
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
}

__device__ __forceinline__ bool is_legal(const uint32_t* bm, int i) {
  return bm == nullptr || ((bm[i >> 5] >> (i & 31)) & 1u);
}

template <int DT>
__global__ void __launch_bounds__(kBlock) score_kernel(Args a) {
  __shared__ uint64_t s_u64[kBlockWaves];
  __shared__ float s_f[2 * kBlockWaves];
  __shared__ uint32_t s_flags;
  const int r = blockIdx.x;
  const int tid = threadIdx.x;
  const int w = tid >> 6;
  const uint8_t* row = a.logits + (size_t)r * a.row_bytes;
  const uint32_t* bm = a.bitmask ? a.bitmask + (size_t)r * a.bm_stride : nullptr;
  const int32_t* tokens = a.tokens + (size_t)r * a.G;
  const float T = a.T ? a.T[r] : 1.0f;
  if (tid == 0) s_flags = 0u;
  __syncthreads();
  // bit 0: a legal token, bit 1: NaN or +inf at one, bit 2: a bad token id
  uint32_t flags = 0u;
  float m = -INFINITY;
  for (int i = tid; i < a.V; i += kBlock) {
    if (!is_legal(bm, i)) continue;
    const float z = load_logit<DT>(row, i);
    flags |= (z != z || z == INFINITY) ? 3u : 1u;
    m = fmaxf(m, z);
  }
  for (int g = tid; g < a.G; g += kBlock)
    if (tokens[g] < -1 || tokens[g] >= a.V) flags |= 4u;
  if (flags) atomicOr(&s_flags, flags);
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if (lane_id() == 0) s_f[w] = m;
  __syncthreads();
  flags = s_flags;
  m = s_f[0];
  for (int k = 1; k < kBlockWaves; ++k) m = fmaxf(m, s_f[k]);
  __syncthreads();
  int status = QS_ROW_OK;
  if (!(T > 0.0f) || T == INFINITY || (flags & 4u)) status = QS_ROW_BAD_PARAM;
  else if (!(flags & 1u)) status = QS_ROW_EMPTY;
  else if (flags & 2u) status = QS_ROW_NONFINITE;
  else if (m == -INFINITY) status = QS_ROW_ALL_NEG_INF;
  if (tid == 0) a.status[r] = status;
  if (status != QS_ROW_OK) {
    for (int g = tid; g < a.G; g += kBlock)
      a.logprobs[(size_t)r * a.G + g] = tokens[g] == -1 ? 0.0f : NAN;
    for (int j = tid; j < a.top_n; j += kBlock) {
      a.top_ids[(size_t)r * a.top_n + j] = -1;
      a.top_lp[(size_t)r * a.top_n + j] = -INFINITY;
    }
    if (tid == 0) {
      a.row_max[r] = NAN;
      a.log_sum[r] = NAN;
      if (a.entropy) a.entropy[r] = NAN;
    }
    return;
  }
  float S = 0.0f, E = 0.0f;
  for (int i = tid; i < a.V; i += kBlock) {
    if (!is_legal(bm, i)) continue;
    const float d = (load_logit<DT>(row, i) - m) / T;
    const float e = __expf(d);
    S += e;
    if (e > 0.0f) E += e * d;
  }
  for (int off = 32; off > 0; off >>= 1) {
    S += __shfl_xor(S, off, 64);
    E += __shfl_xor(E, off, 64);
  }
  if (lane_id() == 0) {
    s_f[2 * w] = S;
    s_f[2 * w + 1] = E;
  }
  __syncthreads();
  S = E = 0.0f;
  for (int k = 0; k < kBlockWaves; ++k) {
    S += s_f[2 * k];
    E += s_f[2 * k + 1];
  }
  const float log_sum = logf(S);
  if (tid == 0) {
    a.row_max[r] = m;
    a.log_sum[r] = log_sum;
    if (a.entropy) a.entropy[r] = log_sum - E / S;
  }
  for (int g = tid; g < a.G; g += kBlock) {
    const int t = tokens[g];
    float lp = 0.0f;
    if (t >= 0) lp = is_legal(bm, t) ? (load_logit<DT>(row, t) - m) / T - log_sum : -INFINITY;
    a.logprobs[(size_t)r * a.G + g] = lp;
  }
  uint64_t prev = ~0ull;
  for (int j = 0; j < a.top_n; ++j) {
    uint64_t best = 0u;
    for (int i = tid; i < a.V; i += kBlock) {
      const float z = load_logit<DT>(row, i);
      if (!is_legal(bm, i) || z == -INFINITY) continue;
      const uint64_t key =
          ((uint64_t)Keys<QS_F32>::of(__float_as_uint(z)) << 32) | (uint32_t)~i;
      if (key < prev && key > best) best = key;
    }
    for (int off = 32; off > 0; off >>= 1) {
      const uint64_t o = (uint64_t)__shfl_xor((long long)best, off, 64);
      best = o > best ? o : best;
    }
    if (lane_id() == 0) s_u64[w] = best;
    __syncthreads();
    for (int k = 0; k < kBlockWaves; ++k) best = s_u64[k] > best ? s_u64[k] : best;
    __syncthreads();
    if (tid == 0) {
      const float z = Keys<QS_F32>::value((uint32_t)(best >> 32));
      a.top_ids[(size_t)r * a.top_n + j] = best ? (int32_t)~(uint32_t)best : -1;
      a.top_lp[(size_t)r * a.top_n + j] = best ? (z - m) / T - log_sum : -INFINITY;
    }
    if (best) prev = best;
    else prev = 0u;  // no token left: the later slots stay empty
  }
}

}  // namespace

size_t workspace_bytes(int64_t B, int64_t V, int dtype, int64_t top_n) {
  (void)B; (void)V; (void)dtype; (void)top_n;
  return 0;
}

hipError_t launch_score(const Args& a, int dtype, int B, void* workspace, hipStream_t st) {
  (void)workspace;
  if (dtype == QS_F32)
    hipLaunchKernelGGL(score_kernel<QS_F32>, dim3((unsigned)B), dim3(kBlock), 0, st, a);
  else
    hipLaunchKernelGGL(score_kernel<QS_BF16>, dim3((unsigned)B), dim3(kBlock), 0, st, a);
  return hipGetLastError();
}

}  // namespace score
}  // namespace qs
