// Distillation from a teacher of which only the top tokens are known: per row the
// divergence of the student's tempered, masked softmax from the teacher.
//
// With L the legal tokens, m = max_L z, p_i = exp((z_i - m) / T) / S, the teacher's
// tokens j with probabilities q_j, and R the legal tokens that the teacher does not
// name (the rest), p_R their mass and q_R the mass the teacher leaves them,
//   loss = sum_j q_j (log q_j - log p_j) + q_R (log q_R - log p_R).
// The named tokens are kept out of the sum over the row, whose maximum m_R and sum
// S_R = sum_R exp((z - m_R) / T) are therefore the rest's own: p_R is never 1 less
// the others. What is left, a few values per teacher's token, is done in 64 bits:
// log p and log q are numbers around 10 whose differences may be far smaller.
//
// Which tokens are named: each workgroup marks the teacher's tokens among its own in
// a bitmap in LDS (a bit that is set already shows a token named twice), and a
// 16-byte load's byte of it joins the legal bits.

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

constexpr int kRowBlock = 1024;  // threads of a row's workgroup
constexpr int kRowLoads = 8;     // 16-byte loads per lane at a time
constexpr float kLowest = -3.402823466e38f;

// What a pass over (a part of) a row leaves.
struct Part {
  float m;        // largest legal token outside the list (kLowest: none is finite)
  float S;        // sum of 2^((z - m) c) over them; NaN if one is NaN or +inf
  uint32_t any;   // a legal token exists
  uint32_t dup;   // a token is named twice
};
static_assert(sizeof(Part) == 16, "one 16-byte store");

struct FinishShared {
  float zmax[kRowBlock / 64], tmax[kRowBlock / 64];
  uint32_t flags[kRowBlock / 64];
  double sum[5][kRowBlock / 64];
};

constexpr uint32_t kBadSlot = 1u, kNonfinite = 2u;

// Writes one row's outputs from the rest's statistics; called by every thread of a
// workgroup of THREADS, at most kSlotsMax slots.
template <int DT, int THREADS>
__device__ __forceinline__ void finish_row(const Args& a, int r, int tid, const Part& rest,
                                           FinishShared& s) {
  constexpr int kWavesHere = THREADS / 64;
  constexpr int kSlots = (kSlotsMax + THREADS - 1) / THREADS;
  const int lane = lane_id(), w = tid >> 6;
  const float Tf = a.T ? a.T[r] : 1.0f;
  const bool bad_T = !(Tf > 0.0f) || Tf == INFINITY;
  const double T = Tf;
  const uint8_t* const row = a.logits + (size_t)r * a.row_bytes;
  const uint32_t* const mask = a.bitmask ? a.bitmask + (size_t)r * a.bm_stride : nullptr;
  const float most = a.rest ? 1.0f : 3.402823466e38f;

  float z[kSlots], t[kSlots];
  bool live[kSlots];
  float zmax = -INFINITY, tmax = -INFINITY;
  uint32_t flags = 0u;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int j = i * THREADS + tid;
    live[i] = false;
    z[i] = t[i] = -INFINITY;
    if (j < a.K) {
      const int id = a.ids[(size_t)r * a.K + j];
      if (id < -1 || id >= a.V) flags |= kBadSlot;
      else if (id >= 0 && (!mask || ((mask[id >> 5] >> (id & 31)) & 1u))) {
        live[i] = true;
        t[i] = a.values[(size_t)r * a.K + j];
        z[i] = logit_at<DT>(row, id);
        if (!(t[i] <= most)) flags |= kBadSlot;
        if (!(z[i] < INFINITY)) flags |= kNonfinite;
        zmax = fmaxf(zmax, z[i]);
        tmax = fmaxf(tmax, t[i]);
      }
    }
  }
  zmax = wave_max_f32(zmax);
  tmax = wave_max_f32(tmax);
  flags = (ballot(flags & kBadSlot) ? kBadSlot : 0u) | (ballot(flags & kNonfinite) ? kNonfinite : 0u);
  if constexpr (kWavesHere > 1) {
    if (lane == 0) {
      s.zmax[w] = zmax;
      s.tmax[w] = tmax;
      s.flags[w] = flags;
    }
    __syncthreads();
    zmax = s.zmax[0], tmax = s.tmax[0], flags = s.flags[0];
#pragma unroll
    for (int k = 1; k < kWavesHere; ++k) {
      zmax = fmaxf(zmax, s.zmax[k]);
      tmax = fmaxf(tmax, s.tmax[k]);
      flags |= s.flags[k];
    }
  }
  const bool has = rest.S != 0.0f;  // the rest has a finite token (or is NaN)
  const float m = has ? fmaxf(rest.m, zmax) : zmax;
  int status = QS_ROW_OK;
  if (bad_T || rest.dup || (flags & kBadSlot)) status = QS_ROW_BAD_PARAM;
  else if (!rest.any) status = QS_ROW_EMPTY;
  else if ((flags & kNonfinite) || !(rest.S < INFINITY)) status = QS_ROW_NONFINITE;
  else if (m == -INFINITY) status = QS_ROW_ALL_NEG_INF;
  float* const state = a.state + (size_t)r * kState;
  if (status != QS_ROW_OK) {  // the same in every thread
    if (tid == 0) {
      a.status[r] = status;
      a.loss[r] = NAN;
    }
    if (tid < kState) state[tid] = NAN;
    return;
  }
  if (tmax == -INFINITY) tmax = 0.0f;  // no teacher's token has a weight

  // sums over the list: student's weights (below the maximum, and how many are at
  // it), teacher's weights likewise, and teacher's weight times log q - log p but
  // for the two normalisers
  double sum[5] = {0.0, 0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    if (!live[i]) continue;
    const double d = ((double)z[i] - (double)m) / T;
    const double tau = a.rest ? (double)t[i] : ((double)t[i] - (double)tmax) / T;
    const double wt = exp(tau);
    if (z[i] == m) sum[1] += 1.0;
    else sum[0] += exp(d);
    if (!a.rest && t[i] == tmax) sum[3] += 1.0;
    else sum[2] += wt;
    if (wt > 0.0) sum[4] += wt * (tau - d);
  }
#pragma unroll
  for (int k = 0; k < 5; ++k) sum[k] = wave_sum_f64(sum[k]);
  if constexpr (kWavesHere > 1) {
    if (lane < 5) s.sum[lane][w] = lane == 0 ? sum[0] : lane == 1 ? sum[1] : lane == 2 ? sum[2]
                                   : lane == 3 ? sum[3] : sum[4];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      sum[k] = s.sum[k][0];
#pragma unroll
      for (int v = 1; v < kWavesHere; ++v) sum[k] += s.sum[k][v];
    }
  }
  if (tid != 0) return;
  const double below = sum[0], at = sum[1], cross = sum[4];
  // the rest's weight against m; one maximum's own 1 is left out of the sum, so
  // that log S keeps its relative precision where one token is almost certain
  const double dr = has ? ((double)rest.m - (double)m) / T : 0.0;
  const double f = has ? exp(dr) * (double)rest.S : 0.0;
  const double others = at > 0.0 ? below + (at - 1.0) + f : below + (f - 1.0);
  const double ls = log1p(others);
  const double lsr = has ? log((double)rest.S) : 0.0;
  const double lpr = dr + lsr - ls;
  double loss, mass, q_list, q_rest = 0.0, tls = 0.0;
  if (a.rest) {
    q_list = sum[2];
    if (has) q_rest = fmax(1.0 - q_list, 0.0);
    loss = cross + ls * q_list;
    if (q_rest > 0.0) loss += q_rest * (log(q_rest) - lpr);
  } else {
    const double W = sum[2] + sum[3];
    q_list = W > 0.0 ? 1.0 : 0.0;
    if (W > 0.0) tls = log1p(sum[2] + (sum[3] - 1.0));
    loss = W > 0.0 ? cross / W - tls + ls : 0.0;
  }
  mass = q_list + q_rest;
  const double pr = exp(lpr);
  // Q p_R - q_R, from the smaller of the two halves
  const double rest_grad =
      !has ? 0.0 : pr < 0.5 ? mass * pr - q_rest : q_list - mass * (below + at) / (1.0 + others);
  a.status[r] = QS_ROW_OK;
  a.loss[r] = (float)loss;
  state[0] = m;
  state[1] = (float)ls;
  state[2] = has ? rest.m : 0.0f;
  state[3] = (float)lsr;
  state[4] = (float)rest_grad;
  state[5] = a.rest ? 0.0f : tmax;
  state[6] = (float)tls;
  state[7] = (float)(mass - 1.0);
}

// One workgroup per row, which walks it.
template <int DT, bool MASK>
__global__ void __launch_bounds__(kRowBlock) distill_row_kernel(Args a) {
  constexpr int P = kPer<DT>, kSpan = kRowBlock * kRowLoads * P;
  __shared__ uint32_t s_named[kSpan / 32];
  __shared__ FinishShared s_fin;
  __shared__ float s_m[kRowBlock / 64], s_S[kRowBlock / 64];
  const int tid = threadIdx.x, lane = lane_id(), w = tid >> 6;
  const int r = blockIdx.x;
  const uint8_t* const row = a.logits + (size_t)r * a.row_bytes;
  const uint8_t* const mask_row =
      reinterpret_cast<const uint8_t*>(a.bitmask + (size_t)r * a.bm_stride);
  const float c = scale_of(a.T ? a.T[r] : 1.0f);
  float m = kLowest, S = 0.0f;
  uint32_t any = 0u, dup = 0u;
  for (int64_t begin64 = 0; begin64 < a.V; begin64 += kSpan) {
    const int begin = (int)begin64;
    __syncthreads();  // the bitmap of the span before has been read
    for (int i = tid; i < kSpan / 32; i += kRowBlock) s_named[i] = 0u;
    __syncthreads();
    for (int j = tid; j < a.K; j += kRowBlock) {
      const int id = a.ids[(size_t)r * a.K + j], d = id - begin;
      if (id >= begin && id < a.V && d < kSpan) {
        const uint32_t bit = 1u << (d & 31);
        dup |= atomicOr(&s_named[d >> 5], bit) & bit;
      }
    }
    __syncthreads();
    uint4 v[kRowLoads];
    float top = m;
#pragma unroll
    for (int u = 0; u < kRowLoads; ++u) {
      const int d = (u * kRowBlock + tid) * P;
      uint32_t bits = 0u;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (d < a.V - begin) {
        const int i = begin + d;
        bits = 0xFFu;
        if constexpr (MASK) bits = mask_row[i >> 3];
        uint32_t named = reinterpret_cast<const uint8_t*>(s_named)[d >> 3];
        if constexpr (P == 4) {
          if (MASK) bits >>= i & 4;
          named >>= d & 4;
        }
        const int left = a.V - i;
        bits &= left >= P ? (1u << P) - 1u : (1u << left) - 1u;
        any |= bits;
        bits &= ~named;
        v[u] = *reinterpret_cast<const uint4*>(row + (size_t)i * (16 / P));
      }
      v[u] = blank<DT>(v[u], masks_of<DT>(bits));
#pragma unroll
      for (int e = 0; e < P; ++e) top = fmaxf(top, token<DT>(v[u], e));
    }
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kRowLoads; ++u) {
#pragma unroll
      for (int e = 0; e < P; ++e) sum += exp2_hw((token<DT>(v[u], e) - top) * c);
    }
    S = fmaf(S, exp2_hw((m - top) * c), sum);
    m = top;
  }
  const float wm = wave_max_f32(m);
  S = wave_sum_f32(S * exp2_hw((m - wm) * c));
  if (lane == 0) s_m[w] = wm, s_S[w] = S;
  any = __syncthreads_or(any != 0u);
  dup = __syncthreads_or(dup != 0u);
  Part p{s_m[0], 0.0f, any, dup};
#pragma unroll
  for (int k = 1; k < kRowBlock / 64; ++k) p.m = fmaxf(p.m, s_m[k]);
#pragma unroll
  for (int k = 0; k < kRowBlock / 64; ++k) p.S += s_S[k] * exp2_hw((s_m[k] - p.m) * c);
  finish_row<DT, kRowBlock>(a, r, tid, p, s_fin);
}

}  // namespace

size_t workspace_bytes(int64_t, int64_t, int) { return 0; }
bool grid_fits(int64_t B, int64_t, int) { return B * kRowBlock < (int64_t)1 << 32; }

hipError_t launch_loss(const Args& a, int dtype, int B, void*, hipStream_t st) {
  const dim3 grid((unsigned)B), block(kRowBlock);
  const bool mask = a.bitmask != nullptr;
  if (dtype == QS_F32 && mask)
    hipLaunchKernelGGL((distill_row_kernel<QS_F32, true>), grid, block, 0, st, a);
  else if (dtype == QS_F32)
    hipLaunchKernelGGL((distill_row_kernel<QS_F32, false>), grid, block, 0, st, a);
  else if (mask)
    hipLaunchKernelGGL((distill_row_kernel<QS_BF16, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((distill_row_kernel<QS_BF16, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace distill
}  // namespace qs
