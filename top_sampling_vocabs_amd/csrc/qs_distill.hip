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
//
// The logits are read once, into registers, all requested before the first is used, so
// that the maximum comes first and every exponential is taken once. Rows of up to
// kRowLoads loads go to one workgroup and one launch; longer ones are split into parts,
// joined by a second launch.
//
// Measured: 2048 rows of 151936 bf16 with 64 named tokens each, 100 to 104 us (6.1 TB/s,
// where a large copy reaches 5.2: bound by the reads) and 9 for the join, 3 to 6 of which
// are the named tokens' 131072 cache lines; 64 rows of 128256 fp32, 7.2 us and 4.4; one
// row of 32000 fp32, 6.6 us, its latency (11.2 with all 16 waves finishing the row and its
// logarithms one after another); 37 masked rows of 32003 bf16, 7.5 us. One workgroup a row
// that walks it with a running maximum took 206 us for the 2048 rows.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/qs.h"
#include "qs_device.hpp"
#include "qs_distill.hpp"
#include "qs_softmax.hpp"

namespace qs {
namespace distill {
namespace {

using namespace score;

constexpr int kPartBlock = 256;   // threads of a part's workgroup
// 16-byte loads per lane of a part. Few parts are short, so that they fill the chip
// (1 row of 151936 bf16: 7.2 us with 4 loads, 8.3 with 8, 9.7 with 16; 32 rows 9.0, 9.6
// and 10.1); many unmasked bf16 rows are cut into long ones (2048 rows of 151936: 110 us
// with 16, 113 with 8, 117 with 4), whose exponentials are enough to hide their start;
// masked and fp32 ones are not (2048 masked rows of 100003: 80 with 8, 84 with 16).
constexpr int kShortLoads = 4, kPartLoads = 8, kLongLoads = 16;
constexpr int kRowLoads = 8192;   // 16-byte loads of a row that goes to one workgroup
constexpr int kRowBlock = 1024;   // threads of the largest workgroup
constexpr int kJoinSlots = 4;     // slots per thread of the join
constexpr float kLowest = -3.402823466e38f;

// What a part's workgroup leaves for the join.
struct Part {
  float m;        // largest legal token outside the list (kLowest: none is finite)
  float S;        // sum of 2^((z - m) c) over them; NaN if one is NaN or +inf
  uint32_t any;   // a legal token exists
  uint32_t dup;   // a token is named twice
};
static_assert(sizeof(Part) == 16, "one 16-byte store");

constexpr int64_t kFewParts = 2048, kManyParts = 4096;  // of kPartLoads loads
int64_t parts_of(int64_t V, int dtype, int loads) {
  const int64_t n = (int64_t)(dtype == QS_F32 ? 4 : 8) * kPartBlock * loads;
  return (V + n - 1) / n;
}
bool one_part(int64_t V, int dtype) {
  return V <= (int64_t)(dtype == QS_F32 ? 4 : 8) * kRowLoads;
}
int loads_for(int64_t B, int64_t V, int dtype, bool mask) {
  const int64_t n = B * parts_of(V, dtype, kPartLoads);
  return n <= kFewParts ? kShortLoads
         : n > kManyParts && dtype == QS_BF16 && !mask ? kLongLoads : kPartLoads;
}

constexpr uint32_t kBadSlot = 1u, kNonfinite = 2u;

// The exponent of a wave's or a part's sum against the row's. From halves: finite logits
// may lie further apart than float32's largest value, at temperatures where that is
// little. (A difference inside a wave that passes it is either taken by a multiply-add or
// an exponent past 2^24.)
__device__ __forceinline__ float apart(float m, float top, float c) {
  return fmaxf((0.5f * m - 0.5f * top) * c * 2.0f, -200.0f);
}

// A thread's slots j = i * THREADS + tid: the teacher's value and the student's logit
// of those that name a legal token.
template <int DT, int THREADS, int N>
struct Slots {
  int id[N];
  float z[N], t[N];
  uint32_t live, flags;

  __device__ __forceinline__ void load_ids(const Args& a, int r, int tid) {
    flags = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = i * THREADS + tid;
      id[i] = -1;
      if (j < a.K) id[i] = a.ids[(size_t)r * a.K + j];
      if (id[i] < -1 || id[i] >= a.V) {
        flags = kBadSlot;
        id[i] = -1;
      }
    }
  }
  // the teacher's values
  __device__ __forceinline__ void load_values(const Args& a, int r, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      t[i] = -INFINITY;
      if (id[i] >= 0) t[i] = a.values[(size_t)r * a.K + i * THREADS + tid];
    }
  }
  // the students' logits, and which tokens are legal
  __device__ __forceinline__ void load_logits(const Args& a, int r, int tid) {
    const uint8_t* const row = a.logits + (size_t)r * a.row_bytes;
    const uint32_t* const mask = a.bitmask ? a.bitmask + (size_t)r * a.bm_stride : nullptr;
    live = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      z[i] = -INFINITY;
      if (id[i] < 0) continue;
      z[i] = logit_at<DT>(row, id[i]);
      if (!mask || ((mask[id[i] >> 5] >> (id[i] & 31)) & 1u)) live |= 1u << i;
    }
  }
};

struct FinishShared {
  float zmax[kRowBlock / 64], tmax[kRowBlock / 64];
  uint32_t flags[kRowBlock / 64];
  double sum[5][kRowBlock / 64];
};

// Writes one row's outputs from the rest's statistics; called by every thread of a
// workgroup of THREADS with its slots.
template <int DT, int THREADS, int N>
__device__ __forceinline__ void finish_row(const Args& a, int r, int tid,
                                           Slots<DT, THREADS, N> s, const Part& rest,
                                           FinishShared& sh) {
  constexpr int kWavesHere = THREADS / 64;
  const int lane = lane_id(), w = tid >> 6;
  const float Tf = a.T ? a.T[r] : 1.0f;
  const bool bad_T = !(Tf > 0.0f) || Tf == INFINITY;
  const double T = Tf;
  const float most = a.rest ? 1.0f : 3.402823466e38f;

  float zmax = -INFINITY, tmax = -INFINITY;
  uint32_t flags = s.flags;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!((s.live >> i) & 1u)) continue;
    if (!(s.t[i] <= most)) flags |= kBadSlot;
    if (!(s.z[i] < INFINITY)) flags |= kNonfinite;
    zmax = fmaxf(zmax, s.z[i]);
    tmax = fmaxf(tmax, s.t[i]);
  }
  zmax = wave_max_f32(zmax);
  tmax = wave_max_f32(tmax);
  flags = (ballot(flags & kBadSlot) ? kBadSlot : 0u) | (ballot(flags & kNonfinite) ? kNonfinite : 0u);
  if constexpr (kWavesHere > 1) {
    if (lane == 0) {
      sh.zmax[w] = zmax;
      sh.tmax[w] = tmax;
      sh.flags[w] = flags;
    }
    __syncthreads();
    zmax = sh.zmax[0], tmax = sh.tmax[0], flags = sh.flags[0];
#pragma unroll
    for (int k = 1; k < kWavesHere; ++k) {
      zmax = fmaxf(zmax, sh.zmax[k]);
      tmax = fmaxf(tmax, sh.tmax[k]);
      flags |= sh.flags[k];
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
  const double inv_T = 1.0 / T;
  double sum[5] = {0.0, 0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i * THREADS >= a.K) continue;
    const bool live = (s.live >> i) & 1u;
    const bool at_m = live && s.z[i] == m, at_t = live && !a.rest && s.t[i] == tmax;
    // by all lanes, also those whose own slot is empty: each holds the counts
    sum[1] += __popcll(ballot(at_m));
    sum[3] += __popcll(ballot(at_t));
    if (live) {
      const double d = ((double)s.z[i] - (double)m) * inv_T;
      const double tau = a.rest ? (double)s.t[i] : ((double)s.t[i] - (double)tmax) * inv_T;
      const double wt = exp(tau);
      if (!at_m) sum[0] += exp(d);
      if (!at_t) sum[2] += wt;
      if (wt > 0.0) sum[4] += wt * (tau - d);
    }
  }
#pragma unroll
  for (int k = 0; k < 5; k += 2) sum[k] = wave_sum_f64(sum[k]);
  if constexpr (kWavesHere > 1) {
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < 5; ++k) sh.sum[k][w] = sum[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      sum[k] = sh.sum[k][0];
#pragma unroll
      for (int v = 1; v < kWavesHere; ++v) sum[k] += sh.sum[k][v];
    }
  }
  if (tid >= 64) return;
  // What is left is a handful of numbers. Four logarithms of the row stand side by
  // side in four lanes, as log1p of an argument that keeps their relative precision:
  // 0 the student's sum, one maximum's own 1 left out (so that log S keeps it where
  // one token is almost certain), 1 the rest's sum, 2 the teacher's sum likewise,
  // 3 q_R = 2^n (1 + x).
  const double below = sum[0], at = sum[1], cross = sum[4];
  const double dr = has ? ((double)rest.m - (double)m) * inv_T : 0.0;
  const double f = has ? exp(dr) * (double)rest.S : 0.0;
  const double others = at > 0.0 ? below + (at - 1.0) + f : below + (f - 1.0);
  const double W = sum[2] + sum[3];
  const double q_list = a.rest ? W : W > 0.0 ? 1.0 : 0.0;
  const double q_rest = a.rest && has ? fmax(1.0 - q_list, 0.0) : 0.0;
  int n = 0;
  const double x3 = q_rest > 0.5 ? q_rest - 1.0 : q_rest > 0.0 ? frexp(q_rest, &n) - 1.0 : 0.0;
  const double x = lane == 0 ? others : lane == 1 ? (has ? (double)rest.S - 1.0 : 0.0)
                   : lane == 2 ? (!a.rest && W > 0.0 ? sum[2] + (sum[3] - 1.0) : 0.0) : x3;
  const double y = log1p(x);
  const double ls = readlane_f64(y, 0), lsr = readlane_f64(y, 1), tls = readlane_f64(y, 2);
  const double lqr = readlane_f64(y, 3) + n * 0.69314718055994530942;
  const double lpr = dr + lsr - ls;
  double loss;
  if (a.rest) {
    loss = cross + ls * q_list;
    if (q_rest > 0.0) loss += q_rest * (lqr - lpr);
  } else {
    loss = W > 0.0 ? cross / W - tls + ls : 0.0;
  }
  const double mass = q_list + q_rest;
  const double pr = exp(lpr);
  // Q p_R - q_R, from the smaller of the two halves
  const double rest_grad =
      !has ? 0.0 : pr < 0.5 ? mass * pr - q_rest : q_list - mass * (below + at) / (1.0 + others);
  if (tid != 0) return;
  a.status[r] = QS_ROW_OK;
  a.loss[r] = (float)loss;
  float4* const out = reinterpret_cast<float4*>(state);
  out[0] = make_float4(m, (float)ls, has ? rest.m : 0.0f, (float)lsr);
  out[1] = make_float4((float)rest_grad, a.rest ? 0.0f : tmax, (float)tls, (float)(mass - 1.0));
}

// One workgroup per row (ROW: parts == 1, outputs written here) or per part. Of a whole
// row's workgroup one wave takes the slots and finishes the row, which needs no
// barrier, where its lanes hold them (FT == 64), and all waves longer lists.
template <int DT, int THREADS, int NL, bool MASK, bool ROW, int FT>
__global__ void __launch_bounds__(THREADS)
    distill_kernel(Args a, int parts, int part_loads, Part* ws_parts) {
  constexpr int kWavesHere = THREADS / 64;
  constexpr int P = kPer<DT>, kSpan = THREADS * NL * P;
  constexpr bool kTable = MASK && DT == QS_BF16;
  constexpr int N = FT == 64 ? kJoinSlots : kSlotsMax / FT;
  __shared__ uint32_t s_named[kSpan / 32];
  __shared__ uint4 s_masks[kTable ? 256 : 1];  // masks_of every byte of legal bits
  __shared__ FinishShared s_fin;
  __shared__ float s_m[kWavesHere], s_S[kWavesHere];
  __shared__ uint32_t s_any[kWavesHere], s_dup[kWavesHere];
  const int tid = threadIdx.x, lane = lane_id(), w = uni(tid >> 6);
  const int r = ROW ? (int)blockIdx.x : (int)(blockIdx.x / (unsigned)parts);
  const int part = ROW ? 0 : (int)(blockIdx.x - (unsigned)r * (unsigned)parts);
  const int span = part_loads * THREADS * P;
  const int begin = part * span;  // first token of this workgroup
  const uint8_t* const row = a.logits + (size_t)r * a.row_bytes;
  const uint8_t* const mask_row =
      reinterpret_cast<const uint8_t*>(a.bitmask + (size_t)r * a.bm_stride);
  const float c = scale_of(a.T ? a.T[r] : 1.0f);

  // requests: the slots, then 16 bytes per lane and load; loads that begin past the
  // row's end are left out (a 16-byte chunk that begins inside the row ends inside
  // its stride)
  Slots<DT, FT, N> slots;
  const bool finisher = FT == THREADS || w == 0;
  if (finisher) slots.load_ids(a, r, tid);
  uint4 v[NL];
  uint32_t legal[NL];
#pragma unroll
  for (int u = 0; u < NL; ++u) {
    const int i = begin + (u * THREADS + tid) * P;
    v[u] = make_uint4(0u, 0u, 0u, 0u);
    legal[u] = 0u;
    if (u < part_loads && i < a.V) {
      v[u] = *reinterpret_cast<const uint4*>(row + (size_t)i * (16 / P));
      legal[u] = 0xFFu;
      if constexpr (MASK) legal[u] = mask_row[i >> 3];
    }
  }
  // which tokens of this workgroup are named
  for (int i = tid; i < kSpan / 32; i += THREADS) s_named[i] = 0u;
  if constexpr (kTable) {
    for (int k = tid; k < 256; k += THREADS) s_masks[k] = masks_of<DT>((uint32_t)k);
  }
  __syncthreads();
  uint32_t dup = 0u;
  if (finisher) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int d = slots.id[i] - begin;
      if (slots.id[i] >= begin && d < span) {
        const uint32_t bit = 1u << (d & 31);
        dup |= atomicOr(&s_named[d >> 5], bit) & bit;
      }
    }
    if constexpr (ROW) slots.load_values(a, r, tid);
  }
  __syncthreads();

  // largest legal token of the lane that is not named; the others become -inf
  Largest<DT> largest;
  uint32_t any = 0u;
#pragma unroll
  for (int u = 0; u < NL; ++u) {
    const int d = (u * THREADS + tid) * P, left = a.V - begin - d;
    uint32_t bits = legal[u], named = reinterpret_cast<const uint8_t*>(s_named)[d >> 3];
    if constexpr (P == 4) {
      if (MASK) bits >>= d & 4;
      named >>= d & 4;
    }
    bits &= left >= P ? (1u << P) - 1u : left > 0 ? (1u << left) - 1u : 0u;
    any |= bits;
    bits &= ~named;
    if constexpr (kTable) v[u] = blank<DT>(v[u], s_masks[bits]);
    else if (MASK || bits != (1u << P) - 1u) v[u] = blank<DT>(v[u], masks_of<DT>(bits));
    largest.add(v[u]);
  }
  const float wave_max = wave_max_f32(fmaxf(largest.value(), kLowest));

  // the wave's sum against its own maximum: with 2^(z c - k), k = fl(m_w c), from one
  // multiply-add it is off by the factor 2^(m_w c - k) alone; past |k| = 2^24 the
  // difference comes first
  float S[2] = {0.0f, 0.0f};
  const float k = wave_max * c;
  if (fabsf(k) < kFused && c < 1e30f) {
#pragma unroll
    for (int u = 0; u < NL; ++u) {
      opaque(v[u]);
#pragma unroll
      for (int e = 0; e < P; ++e) S[e & 1] += exp2_hw(fmaf(token<DT>(v[u], e), c, -k));
    }
    const float f = exp2_hw(-fmaf(wave_max, c, -k));
    S[0] *= f;
    S[1] *= f;
  } else {
#pragma unroll
    for (int u = 0; u < NL; ++u) {
      opaque(v[u]);
#pragma unroll
      for (int e = 0; e < P; ++e) S[e & 1] += exp2_hw((token<DT>(v[u], e) - wave_max) * c);
    }
  }
  // the named tokens' logits, now that the row's cache lines are here (requested beside
  // them they are a line apiece more to fetch: 4096 rows of 32000 bf16 with 64 tokens
  // each 104 us against 99)
  if constexpr (ROW) {
    if (finisher) slots.load_logits(a, r, tid);
  }
  const float Sw = wave_sum_f32(S[0] + S[1]);
  const bool anyw = ballot(any != 0u) != 0, dupw = ballot(dup != 0u) != 0;
  if (lane == 0) {
    s_m[w] = wave_max;
    s_S[w] = Sw;
    s_any[w] = anyw;
    s_dup[w] = dupw;
  }
  __syncthreads();
  if (!finisher) return;
  Part p{s_m[0], 0.0f, s_any[0], s_dup[0]};
#pragma unroll
  for (int q = 1; q < kWavesHere; ++q) {
    p.m = fmaxf(p.m, s_m[q]);
    p.any |= s_any[q];
    p.dup |= s_dup[q];
  }
#pragma unroll
  for (int q = 0; q < kWavesHere; ++q) p.S += s_S[q] * exp2_hw(apart(s_m[q], p.m, c));
  if constexpr (ROW) {
    finish_row<DT, FT, N>(a, r, tid, slots, p, s_fin);
  } else {
    if (tid == 0) ws_parts[(size_t)r * parts + part] = p;
  }
}

// Joins the parts of each row: one workgroup per row.
template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS)
    distill_join_kernel(Args a, int parts, const Part* ws_parts) {
  __shared__ FinishShared s_fin;
  const int r = blockIdx.x, tid = threadIdx.x, lane = lane_id();
  const Part* const p = ws_parts + (size_t)r * parts;
  Slots<DT, THREADS, kJoinSlots> slots;
  slots.load_ids(a, r, tid);
  Part mine{kLowest, 0.0f, 0u, 0u};
  if (lane < parts) mine = p[lane];
  slots.load_values(a, r, tid);
  slots.load_logits(a, r, tid);
  const float c = scale_of(a.T ? a.T[r] : 1.0f);
  // every wave joins all parts (the same values in every thread)
  float m = mine.m;
  uint32_t any = mine.any, dup = mine.dup;
  for (int k = lane + 64; k < parts; k += 64) {
    m = fmaxf(m, p[k].m);
    any |= p[k].any;
    dup |= p[k].dup;
  }
  m = wave_max_f32(m);
  float S = mine.S * exp2_hw(apart(mine.m, m, c));
  for (int k = lane + 64; k < parts; k += 64) S += p[k].S * exp2_hw(apart(p[k].m, m, c));
  const Part rest{m, wave_sum_f32(S), ballot(any != 0u) != 0, ballot(dup != 0u) != 0};
  finish_row<DT, THREADS, kJoinSlots>(a, r, tid, slots, rest, s_fin);
}

template <int DT, int THREADS, int NL, bool ROW, int FT>
void launch(const Args& a, int blocks, int parts, int part_loads, Part* wp, hipStream_t st) {
  const dim3 grid((unsigned)blocks), block(THREADS);
  if (a.bitmask)
    hipLaunchKernelGGL((distill_kernel<DT, THREADS, NL, true, ROW, FT>), grid, block, 0, st, a,
                       parts, part_loads, wp);
  else
    hipLaunchKernelGGL((distill_kernel<DT, THREADS, NL, false, ROW, FT>), grid, block, 0, st, a,
                       parts, part_loads, wp);
}

template <int N> using Int = std::integral_constant<int, N>;

// A whole row's workgroup holds the row and little more, so that where rows are many
// others load while its one wave finishes it. (bf16, 32 named tokens, 1 and 4096 rows:
// 1000 tokens 4.6 and 9.4 us with 128 threads x 1 load, 5.3 and 19 with 256 x 4; 16000
// tokens 5.8 and 31 with 512 x 4, 8.8 and 96 with 1024 x 8; 32000 tokens 6.8 and 52 with
// 512 x 8, 8.8 and 97 with 1024 x 8; 3000 tokens 5.0 and 14.4 with 256 x 2, 5.3 and 12.1
// with 128 x 4; 65536 tokens 8.8 and 123 with 1024 x 8, 9.1 and 102 with 512 x 16.)
template <int DT>
hipError_t launch_dt(const Args& a, int B, Part* wp, hipStream_t st) {
  constexpr int P = kPer<DT>;
  const bool few = a.K <= 64 * kJoinSlots;  // slots that one wave holds
  if (one_part(a.V, DT)) {
    auto run = [&](auto threads, auto loads) {
      constexpr int TH = decltype(threads)::value, NL = decltype(loads)::value;
      const int each = (a.V + TH * P - 1) / (TH * P);
      if (few) launch<DT, TH, NL, true, 64>(a, B, 1, each, nullptr, st);
      else launch<DT, TH, NL, true, TH>(a, B, 1, each, nullptr, st);
    };
    const int n = (a.V + P - 1) / P;  // 16-byte loads of a row
    auto pick = [&](auto threads, auto loads) {
      if (n > decltype(threads)::value * decltype(loads)::value) return false;
      run(threads, loads);
      return true;
    };
    const bool done = pick(Int<128>(), Int<1>()) || pick(Int<128>(), Int<2>()) ||
                      (B <= 512 ? pick(Int<256>(), Int<2>()) : pick(Int<128>(), Int<4>())) ||
                      pick(Int<256>(), Int<4>()) || pick(Int<512>(), Int<4>()) ||
                      pick(Int<512>(), Int<8>()) ||
                      (B <= 256 ? pick(Int<1024>(), Int<8>()) : pick(Int<512>(), Int<16>()));
    return done ? hipGetLastError() : hipErrorInvalidValue;
  }
  // parts of equal length, in whole loads
  const int most = loads_for(B, a.V, DT, a.bitmask != nullptr);
  const int parts = (int)parts_of(a.V, DT, most);
  const int loads = (a.V + kPartBlock * P - 1) / (kPartBlock * P);
  const int each = (loads + parts - 1) / parts;
  auto run = [&](auto nl) {
    launch<DT, kPartBlock, decltype(nl)::value, false, kPartBlock>(a, B * parts, parts, each, wp,
                                                                  st);
  };
  if (most == kShortLoads) run(Int<kShortLoads>());
  else if (most == kPartLoads) run(Int<kPartLoads>());
  else run(Int<kLongLoads>());
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  if (few)
    hipLaunchKernelGGL((distill_join_kernel<DT, 64>), dim3((unsigned)B), dim3(64), 0, st, a, parts,
                       wp);
  else
    hipLaunchKernelGGL((distill_join_kernel<DT, 256>), dim3((unsigned)B), dim3(256), 0, st, a,
                       parts, wp);
  return hipGetLastError();
}

}  // namespace

// Enough for every batch of at most B rows: the largest of them whose parts are short
// has up to twice the parts of a somewhat larger one whose parts are longer.
size_t workspace_bytes(int64_t B, int64_t V, int dtype) {
  if (one_part(V, dtype)) return 0;
  const int64_t per_row = parts_of(V, dtype, kPartLoads);
  const int64_t few = kFewParts / per_row;  // rows of the last batch of short parts
  int64_t n = B * per_row, short_parts = (B < few ? B : few) * parts_of(V, dtype, kShortLoads);
  if (n < short_parts) n = short_parts;
  return ((size_t)n * sizeof(Part) + 255) & ~(size_t)255;
}

bool grid_fits(int64_t B, int64_t V, int dtype) {
  if (one_part(V, dtype)) return B * kRowBlock < (int64_t)1 << 32;
  return B * parts_of(V, dtype, kPartLoads) * kPartBlock < (int64_t)1 << 32;
}

hipError_t launch_loss(const Args& a, int dtype, int B, void* workspace, hipStream_t st) {
  Part* const wp = static_cast<Part*>(workspace);
  return dtype == QS_F32 ? launch_dt<QS_F32>(a, B, wp, st) : launch_dt<QS_BF16>(a, B, wp, st);
}

}  // namespace distill
}  // namespace qs
