// Gradient of the token log-probabilities and of the entropy with respect to
// the logits:
//   dz_i = (1/T) [ sum_g gl_g (1[i = t_g] - p_i) - gH p_i (log p_i + H) ]
// for legal i, 0 elsewhere, with log p_i = (z_i - m) / T - log S from the
// forward pass's row maximum and log sum. With a_i = log2 p_i, per row
//   dz_i = p_i (A + B a_i) + hit_i / T,
//   A = -(sum_g gl_g + gH H) / T,  B = -gH ln 2 / T,
// so a token costs one exponential and a few operations, and the kernel is
// bound by reading the logits and writing their gradient once.
//
// A workgroup takes kLoads 16-byte loads per lane of one row. The row's single
// token is compared directly. Of a list of tokens one wave keeps the slots that lie
// in this workgroup, in LDS; a thread to each works out its token's element from
// them, and the elements are written over the 16-byte stores at the end, so that
// the other 8191 know nothing of the list. (Every 16-byte chunk with a given token
// going through the list itself: 333 masked rows of 128259 with four tokens each
// 38.6 us against 35.2; 512 rows of 151936 with 64 tokens 189 against 53, with 1024
// tokens 7.4 ms against 90 us.) A token named by several slots gets their sum, in
// slot order, and each element is rounded once.
//
// At a given token the sum of its own slots enters as gl (1 - p) = -gl expm1(log p):
// where the token is almost certain, gl / T and p A would cancel to the rounding
// of either, and what the rest of the row gets would have no counterpart. The
// other slots' sum is added up without its own for the same reason.
//
// Measured: 2048 rows of 151936 bf16, one token each, 225 us (5.5 TB/s read and
// written, where a large copy reaches 4.8); the 333 rows 35.2 us (5.0 TB/s, the
// launch included).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qs.h"
#include "qs_device.hpp"
#include "qs_score.hpp"
#include "qs_softmax.hpp"

namespace qs {
namespace score {
namespace {

constexpr int kBlock = 256;
constexpr int kLoads = 4;  // 16-byte loads per lane

// x within +-most; as it is where `keep` is set (fmaxf would turn a NaN into -most)
__device__ __forceinline__ float clamp_to(float x, float most, bool keep) {
  return keep ? x : fminf(fmaxf(x, -most), most);
}

template <int DT, bool MASK, bool ONE>
__global__ void __launch_bounds__(kBlock) grad_kernel(GradArgs a, int chunks) {
  constexpr int P = kPer<DT>;
  __shared__ int2 s_slot[ONE ? 1 : kTokensMax];  // this block's slots: place, gradient's bits
  __shared__ float s_given[ONE ? 1 : kTokensMax];
  __shared__ int s_slots;
  __shared__ float s_sum[2];
  const int tid = threadIdx.x;
  const int r = (int)(blockIdx.x / (unsigned)chunks);
  const int begin = (int)(blockIdx.x - (unsigned)r * (unsigned)chunks) * (kBlock * kLoads * P);
  const uint8_t* row = a.logits + (size_t)r * a.row_bytes;
  uint8_t* out = a.grad + (size_t)r * a.grad_bytes;
  const int32_t* tokens = a.tokens + (size_t)r * a.G;
  const float* gl = a.g_lp + (size_t)r * a.G;
  const bool ok = a.status[r] == QS_ROW_OK;

  uint4 v[kLoads];
  uint32_t legal[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = begin + (u * kBlock + tid) * P;
    v[u] = make_uint4(0u, 0u, 0u, 0u);
    legal[u] = 0u;
    if (i < a.V && ok) {
      v[u] = *reinterpret_cast<const uint4*>(row + (size_t)i * (16 / P));
      legal[u] = 0xFFu;
      if constexpr (MASK) {
        legal[u] = reinterpret_cast<const uint8_t*>(a.bitmask + (size_t)r * a.bm_stride)[i >> 3];
        if constexpr (P == 4) legal[u] >>= i & 4;
      }
    }
  }

  const float T = a.T ? a.T[r] : 1.0f;
  const float c = scale_of(T);
  const float m = a.row_max[r];
  const float ls = a.log_sum[r], ls2 = ls * kLog2e;
  float gs = 0.0f;
  int only = -1;
  if constexpr (ONE) {
    only = tokens[0];
    if (only >= 0 && only < a.V) gs = gl[0];
  } else {
    // one wave reads the list: sums over the whole row, and the slots whose tokens
    // lie in this block, in slot order
    if (tid < 64) {
      float away = 0.0f;
      int n = 0;
      for (int g0 = 0; g0 < a.G; g0 += 64) {
        const int g = g0 + tid;
        int t = -1;
        float v = 0.0f;
        if (g < a.G) {
          t = tokens[g];
          v = gl[g];
        }
        if (t < 0 || t >= a.V) t = -1, v = 0.0f;
        const int d = t - begin;
        const bool here = t >= begin && d < kBlock * kLoads * P;
        const uint64_t lanes = ballot(here);
        if (here)
          s_slot[n + __popcll(lanes & ((1ull << tid) - 1ull))] =
              make_int2(d, (int)__float_as_uint(v));
        else
          away += v;
        gs += v;
        n += __popcll(lanes);
      }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        gs += __shfl_xor(gs, off, 64);
        away += __shfl_xor(away, off, 64);
      }
      if (tid == 0) {
        s_slots = ok ? n : 0;
        s_sum[0] = gs;
        s_sum[1] = away;
      }
    }
    __syncthreads();
    gs = s_sum[0];
  }
  const float gH = a.g_ent ? a.g_ent[r] : 0.0f, H = a.g_ent ? a.entropy[r] : 0.0f;
  // finite where the row's incoming sums are, so that a p of 0 gives 0; infinities
  // and NaN go through to every legal token
  const bool lost = !(fabsf(gs) < INFINITY && fabsf(gH) < INFINITY && fabsf(H) < INFINITY);
  const float A = clamp_to(-(gs + gH * H) / T, 3e38f, lost);
  const float Bc = clamp_to(-gH * kLn2 / T, 1e36f, lost);

  auto logit = [](const uint32_t* w, int e) {
    if constexpr (DT == QS_F32) return __uint_as_float(w[e]);
    return __uint_as_float((e & 1) ? (w[e >> 1] & 0xFFFF0000u) : (w[e >> 1] << 16));
  };
  // a given token's element, its slots' sum and that of the others apart
  auto given = [&](float z, float own, float others) {
    const float lp = fmaxf((z - m) / T - ls, -140.0f);
    const float p = __builtin_amdgcn_exp2f((z - m) * c - ls2);
    return -(own * expm1f(lp) + others * p + gH * (p * (lp + H))) / T;
  };

  // a thread to each of the block's slots: its token's element, written over the
  // others' 16 bytes at the end (slots of one token write the same bits)
  int slots = 0;
  if constexpr (!ONE) {
    slots = s_slots;
    for (int j = tid; j < slots; j += kBlock) {
      const int d = s_slot[j].x, i = begin + d;
      const float z = logit_at<DT>(row, i);
      bool is_legal = true;
      if constexpr (MASK)
        is_legal = (a.bitmask[(size_t)r * a.bm_stride + (i >> 5)] >> (i & 31)) & 1u;
      float own = 0.0f, others = s_sum[1];
      for (int q = 0; q < slots; ++q) {
        const int2 slot = s_slot[q];
        const float v = __uint_as_float((uint32_t)slot.y);
        own += slot.x == d ? v : 0.0f;
        others += slot.x == d ? 0.0f : v;
      }
      s_given[j] = is_legal ? given(z, own, others) : 0.0f;
    }
    if (slots > 0) __syncthreads();  // in place: no element changes before it is read here
  }

#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = begin + (u * kBlock + tid) * P;
    if (i >= a.V) break;
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    float x[P];
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const float l = fmaxf((logit(w, e) - m) * c - ls2, -200.0f);
      x[e] = __builtin_amdgcn_exp2f(l) * (A + Bc * l);
    }
    if constexpr (ONE) {
      const int at = only - i;
      if (at >= 0 && at < P) {
        float z = 0.0f;
#pragma unroll
        for (int e = 0; e < P; ++e) z = at == e ? logit(w, e) : z;
        const float y = given(z, gs, 0.0f);
#pragma unroll
        for (int e = 0; e < P; ++e) x[e] = at == e ? y : x[e];
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if constexpr (DT == QS_F32) {
        const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)legal[u], d, 1);
        o[d] = __float_as_uint(x[d]) & keep;
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
  if (slots > 0) {
    __syncthreads();
    for (int j = tid; j < slots; j += kBlock) {
      const int i = begin + s_slot[j].x;
      if constexpr (DT == QS_F32) reinterpret_cast<float*>(out)[i] = s_given[j];
      else reinterpret_cast<__bf16*>(out)[i] = (__bf16)s_given[j];
    }
  }
}

template <int DT>
void launch(const GradArgs& a, unsigned blocks, int chunks, hipStream_t st) {
  const dim3 grid(blocks), block(kBlock);
  const bool mask = a.bitmask != nullptr, one = a.G == 1;
  if (mask && one)
    hipLaunchKernelGGL((grad_kernel<DT, true, true>), grid, block, 0, st, a, chunks);
  else if (mask)
    hipLaunchKernelGGL((grad_kernel<DT, true, false>), grid, block, 0, st, a, chunks);
  else if (one)
    hipLaunchKernelGGL((grad_kernel<DT, false, true>), grid, block, 0, st, a, chunks);
  else
    hipLaunchKernelGGL((grad_kernel<DT, false, false>), grid, block, 0, st, a, chunks);
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
  const unsigned blocks = (unsigned)B * (unsigned)chunks;
  if (dtype == QS_F32) launch<QS_F32>(a, blocks, chunks, st);
  else launch<QS_BF16>(a, blocks, chunks, st);
  return hipGetLastError();
}

}  // namespace score
}  // namespace qs
