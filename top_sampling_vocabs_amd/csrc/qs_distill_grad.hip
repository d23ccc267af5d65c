// Gradient of the distillation loss with respect to the student's logits. With Q the
// teacher's mass in the loss (named tokens and rest), p the student's probabilities
// and w the softmax over the rest alone,
//   a named legal token:  dz_j = (g / T) (Q p_j - q_j)
//   every other legal one: dz_i = (g / T) (Q p_R - q_R) w_i
// and 0 at illegal tokens. The forward pass left Q p_R - q_R, formed without
// cancellation, and the rest's own maximum and log sum, so that a token of the rest
// costs one exponential and one product, and the kernel is bound by reading the
// logits and writing their gradient once.
//
// A workgroup takes kLoads 16-byte loads per lane of one row. Each thread holds up to
// kSlots of the row's slots; those that name a token of this workgroup are worked out
// in 64 bits as (Q - 1) + Q expm1(log p) - expm1(log q), which keeps its relative
// precision where teacher and student are almost certain of the same token, and
// written over the 16-byte stores at the end. Each element is rounded to 32 bits,
// then once to the logits' type.
//
// Measured: 2048 rows of 151936 bf16, 64 named tokens each, 231 us (5.4 TB/s read and
// written, where a large copy reaches 5.2); 333 masked rows of 128259 with 256 tokens,
// 31.4 us (5.6 TB/s); 8 rows of 32000 fp32, 4.0 us, the launch and one chain of loads.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qs.h"
#include "qs_device.hpp"
#include "qs_distill.hpp"
#include "qs_softmax.hpp"

namespace qs {
namespace distill {
namespace {

using namespace score;

constexpr int kBlock = 256;
constexpr int kLoads = 4;                     // 16-byte loads per lane
constexpr int kSlots = kSlotsMax / kBlock;    // slots per thread

template <int DT, bool MASK>
__global__ void __launch_bounds__(kBlock) distill_grad_kernel(GradArgs a, int chunks) {
  constexpr int P = kPer<DT>, kSpan = kBlock * kLoads * P;
  const int tid = threadIdx.x;
  const int r = (int)(blockIdx.x / (unsigned)chunks);
  const int begin = (int)(blockIdx.x - (unsigned)r * (unsigned)chunks) * kSpan;
  const uint8_t* const row = a.logits + (size_t)r * a.row_bytes;
  const uint32_t* const mask = MASK ? a.bitmask + (size_t)r * a.bm_stride : nullptr;
  uint8_t* const out = a.grad + (size_t)r * a.grad_bytes;
  const bool ok = a.status[r] == QS_ROW_OK;

  uint4 v[kLoads];
  uint32_t legal[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int d = (u * kBlock + tid) * P;
    v[u] = make_uint4(0u, 0u, 0u, 0u);
    legal[u] = 0u;
    if (d < a.V - begin && ok) {
      const int i = begin + d;
      v[u] = *reinterpret_cast<const uint4*>(row + (size_t)i * (16 / P));
      legal[u] = 0xFFu;
      if constexpr (MASK) {
        legal[u] = reinterpret_cast<const uint8_t*>(mask)[i >> 3];
        if constexpr (P == 4) legal[u] >>= i & 4;
      }
    }
  }
  // this thread's slots among the workgroup's tokens, and their logits, all read
  // before any element is written (the gradient may replace the logits)
  int place[kSlots];
  float z[kSlots], t[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = s * kBlock + tid;
    place[s] = -1;
    z[s] = t[s] = 0.0f;
    if (s * kBlock < a.K && j < a.K && ok) {
      const int id = a.ids[(size_t)r * a.K + j];
      if (id >= begin && id < a.V && id - begin < kSpan &&
          (!MASK || ((mask[id >> 5] >> (id & 31)) & 1u))) {
        place[s] = id;
        z[s] = logit_at<DT>(row, id);
        t[s] = a.values[(size_t)r * a.K + j];
      }
    }
  }
  const float* const state = a.state + (size_t)r * kState;
  const float T = a.T ? a.T[r] : 1.0f, g = a.g_loss[r];
  const float m = state[0], ls = state[1], mr = state[2], rest_grad = state[4], tmax = state[5],
              tls = state[6], over = state[7];
  const float c = scale_of(T), lsr2 = state[3] * kLog2e;
  // Differences from m_R at temperatures that weigh ones past float32's largest value are
  // taken as halves: the factor is exact, and 1 elsewhere, where it changes no bit.
  const bool far = c < 1e-30f;
  const float h = far ? 0.5f : 1.0f, mr_h = mr * h, c_h = far ? 2.0f * c : c;
  // finite where g is, so that a token of no weight gets 0: of a factor past the largest
  // value a power of two goes into the exponents, so that what has a small share of it
  // gets that; an infinite or NaN g goes through to every legal token
  const double factor = (double)g * (double)rest_grad / (double)T;
  float coef = (float)factor, bias = -lsr2;
  if (__builtin_expect(ballot(fabsf(coef) > 3e38f && fabsf(g) < INFINITY) != 0, 0)) {
    const int n = __builtin_amdgcn_frexp_exp(factor) - 127;  // coef from 2^126 up
    const double sum = n - (double)lsr2;
    bias = (float)sum;
    // the bias's rounding is taken back
    coef = (float)(ldexp(factor, -n) * (1.0 + 0.6931471805599453 * (sum - (double)bias)));
  }

#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if (place[s] < 0) continue;
    const double lp = ((double)z[s] - (double)m) / (double)T - (double)ls;
    const double lq = a.rest ? (double)t[s]
                             : ((double)t[s] - (double)tmax) / (double)T - (double)tls;
    const double e = (double)over + (1.0 + (double)over) * expm1(lp) - expm1(lq);
    z[s] = (float)((double)g * e / (double)T);
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int d0 = (u * kBlock + tid) * P;
    if (d0 >= a.V - begin) break;
    const int i = begin + d0;
    float x[P];
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const float l = fmaxf(fmaf(fmaf(token<DT>(v[u], e), h, -mr_h), c_h, bias), -200.0f);
      x[e] = exp2_hw(l) * coef;
    }
    uint32_t o[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if constexpr (DT == QS_F32) {
        o[d] = __float_as_uint(x[d]) & (uint32_t)__builtin_amdgcn_sbfe((int)legal[u], d, 1);
      } else {
        const f32x2 pair = {x[2 * d], x[2 * d + 1]};
        o[d] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, bf16x2));
        const uint32_t lo = (uint32_t)__builtin_amdgcn_sbfe((int)legal[u], 2 * d, 1);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_sbfe((int)legal[u], 2 * d + 1, 1);
        o[d] &= bfi(0xFFFFu, lo, hi);
      }
    }
    uint8_t* const at = out + (size_t)i * (16 / P);
    if (a.V - i >= P) {
      *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {  // the row's last tokens: what lies behind them stays
#pragma unroll
      for (int e = 0; e < P - 1; ++e) {
        if (i + e < a.V) {
          if constexpr (DT == QS_F32) reinterpret_cast<uint32_t*>(at)[e] = o[e];
          else reinterpret_cast<uint16_t*>(at)[e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if (place[s] < 0) continue;
    if constexpr (DT == QS_F32) reinterpret_cast<float*>(out)[place[s]] = z[s];
    else reinterpret_cast<__bf16*>(out)[place[s]] = (__bf16)z[s];
  }
}

int64_t chunks_for(int64_t V, int dtype) {
  const int64_t n = (int64_t)kBlock * kLoads * (dtype == QS_F32 ? 4 : 8);
  return (V + n - 1) / n;
}

}  // namespace

bool grad_grid_fits(int64_t B, int64_t V, int dtype) {
  return B * chunks_for(V, dtype) * kBlock < (int64_t)1 << 32;
}

hipError_t launch_grad(const GradArgs& a, int dtype, int B, hipStream_t st) {
  const int chunks = (int)chunks_for(a.V, dtype);
  const dim3 grid((unsigned)B * (unsigned)chunks), block(kBlock);
  const bool mask = a.bitmask != nullptr;
  if (dtype == QS_F32 && mask)
    hipLaunchKernelGGL((distill_grad_kernel<QS_F32, true>), grid, block, 0, st, a, chunks);
  else if (dtype == QS_F32)
    hipLaunchKernelGGL((distill_grad_kernel<QS_F32, false>), grid, block, 0, st, a, chunks);
  else if (mask)
    hipLaunchKernelGGL((distill_grad_kernel<QS_BF16, true>), grid, block, 0, st, a, chunks);
  else
    hipLaunchKernelGGL((distill_grad_kernel<QS_BF16, false>), grid, block, 0, st, a, chunks);
  return hipGetLastError();
}

}  // namespace distill
}  // namespace qs
