// Log-probabilities of given tokens under the tempered, masked softmax of a
// row, with the row's entropy and its most probable tokens.
//
// With L the legal tokens, m = max_L z, d_i = (z_i - m) / T and
// S = sum_L exp d_i:
//   log p_t = d_t - log S,   H = log S - (1/S) sum_L exp(d_i) d_i.
// Both terms of H are non-negative, so nothing cancels. The top tokens are
// those of the largest z, ties by id.
//
// The logits are read once. A workgroup holds its share of a row in registers
// (NL 16-byte loads per lane, all requested before the first is used), so the
// maximum comes first and every exponential is taken once against it: no
// rescaling. Each wave uses its own maximum m_w and, for one operation per
// token, the rounded product k_w = fl(m_w c), c = log2(e) / T, as its reference:
// with 2^(z c - k_w) from one fused multiply-add the sums are off by the common
// factor 2^(m_w c - k_w) alone, which one more gives exactly. (Past |k_w| = 2^24,
// where that factor is no longer within 1/2 and 2 and soon leaves float32's range,
// the difference comes first.) The waves' (m, S, E) are joined as
//   S = sum_w S_w f_w,  E = sum_w f_w (E_w + S_w (m_w - m) c),
//   f_w = 2^((m_w - m) c).
// Weights and E are kept in units of log 2 (one hardware exponential each).
//
// One maximum's own weight, exactly 1, is left out of every sum: R = S - 1 is what
// a wave, a part and a row hold, and log S = log1p(R). The log-probability of a
// token that is almost certain then keeps float32's relative precision (added to
// 1, the other weights would keep 2^-24 absolutely). A wave whose S is 2.25 or
// more loses nothing by the subtraction; the others take the lane of their maximum,
// whose tokens are read again, a load to a lane, and weighed again without the
// one. (2048 rows of 151936 bf16: 112 us; 110 with the plain sum, 115 with the
// lane's registers kept for it, 119 if every wave did that.)
//
// Rows of up to kRowBlock * kRowLoads loads go to one workgroup and one launch:
// a second launch costs more than one compute unit needs for such a row. Longer
// rows are split into parts of kPartBlock * kPartLoads loads, several of which
// fit a compute unit at once, so that one part's loads run under another's
// exponentials; a second launch joins the parts of each row. Where that gives
// at most kFewParts parts they are halved, so that the chip fills evenly.
//
// Measured: 2048 rows of 151936 bf16, 110 us (5.6 TB/s, where a large copy
// reaches 4.8: bound by the reads); 256 such rows, 18.9 us and 3.9 for the join,
// with a mask 2 more, with 20 top tokens 5 and 2 more, with both 29.7 and 6.2 (each
// part searches for its own top tokens); one row of 32000 fp32, 8 us, its latency.
// A workgroup per row that walks the row in a loop, with one launch, was slower in
// every form tried (28 us against 24 + 5.6 for the 256 rows; 21 against 11 + 4.6 for
// 64 rows of 128256 fp32).
//
// Top tokens: with t the n-th largest of the maxima of 256 groups of lanes, n
// tokens (one of each of n groups) reach t, so the n largest tokens lie among
// those with z >= t. These are few (a little over n unless values repeat);
// the lanes whose maximum reaches t (again few) are noted, all threads search
// their tokens, read again from the caches, and what is found is ranked. Keys
// (z's order-preserving bits << 32 | ~id) are distinct. Where more than the
// list holds reach t (long runs of equal values) the workgroup takes its n
// largest keys one after another instead.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/qs.h"
#include "qs_device.hpp"
#include "qs_score.hpp"
#include "qs_softmax.hpp"

namespace qs {
namespace score {
namespace {

constexpr int kPartBlock = 256;   // threads of a part's workgroup
constexpr int kPartLoads = 16;    // 16-byte loads per lane
constexpr int kShortLoads = 8;    // the same where parts are few
constexpr int kRowBlock = 1024;   // threads of a whole row's workgroup
constexpr int kRowLoads = 8;
constexpr int kSmallBlock = 256;  // threads of a short row's workgroup
constexpr int kSmallLoads = 4;
constexpr int kListCap = 256;     // collected keys per workgroup
constexpr int kJoinCap = 1024;    // keys of all parts that reach the row's t
// S from which 1 may be subtracted: R's relative error is then at most 1.8 times
// S's, whose terms pass at most 73 additions in a wave
constexpr float kPlain = 2.25f;

// What a part's workgroup leaves for the join.
struct Part {
  float m;        // largest legal logit (-FLT_MAX if none is finite)
  float R;        // sum of 2^((z - m) c), c = log2(e) / T, without one z = m; NaN if a
                  // legal z is NaN or +inf
  float E;        // sum of 2^((z - m) c) (z - m) c
  uint32_t any;   // a legal token exists
  uint32_t t;     // threshold: order-preserving key of a lower bound of the n-th largest z
  int32_t count;  // keys in the part's list
  uint32_t has;   // a legal z = m exists
  uint32_t pad;
};
static_assert(sizeof(Part) == 32, "two 16-byte stores");

// Loads per lane of a part: the long parts' workgroups are more than kFewParts
// (eight per compute unit), or else the row is cut into twice as many.
constexpr int64_t kFewParts = 2048;
int64_t parts_of(int64_t V, int dtype, int loads) {
  const int64_t n = (int64_t)(dtype == QS_F32 ? 4 : 8) * kPartBlock * loads;
  return (V + n - 1) / n;
}
int loads_for(int64_t B, int64_t V, int dtype) {
  return B * parts_of(V, dtype, kPartLoads) > kFewParts ? kPartLoads : kShortLoads;
}
int64_t parts_for(int64_t B, int64_t V, int dtype) {
  if (V <= (int64_t)(dtype == QS_F32 ? 4 : 8) * kRowBlock * kRowLoads) return 1;
  return parts_of(V, dtype, loads_for(B, V, dtype));
}
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The order-preserving key of a logit and back (fp32 keys for both dtypes).
__device__ __forceinline__ uint32_t key_of(float z) { return Keys<QS_F32>::of(__float_as_uint(z)); }

// The n-th largest (n <= 64) of the wave's 4 * 64 keys, low 16 bits cleared.
__device__ __forceinline__ uint32_t wave_nth_high16(const uint4& key, int n) {
  uint32_t t = 0u;
#pragma unroll
  for (int b = 31; b >= 16; --b) {
    const uint32_t c = t | (1u << b);
    const int reach = __popcll(ballot(key.x >= c)) + __popcll(ballot(key.y >= c)) +
                      __popcll(ballot(key.z >= c)) + __popcll(ballot(key.w >= c));
    if (reach >= n) t = c;
  }
  return t;
}

constexpr int kGroups = 256;

struct Shared {
  uint64_t list[kListCap];
  uint4 group[kGroups / 4];  // keys of the groups' maxima
  float m[kRowBlock / 64], R[kRowBlock / 64], E[kRowBlock / 64];
  uint32_t any[kRowBlock / 64], has[kRowBlock / 64];
  uint64_t best[kRowBlock / 64];
  uint16_t lanes[kRowBlock];  // threads whose maximum reaches t
  int n_lanes;
  int count;
  uint32_t t;
};

// The given token of a slot, and its logit once the token is here.
struct Given {
  int token;
  float z;
  bool legal;
};
__device__ __forceinline__ int given_token(const Args& a, int r, int g) {
  return g < a.G ? a.tokens[(size_t)r * a.G + g] : -1;
}
template <int DT>
__device__ __forceinline__ Given load_given(const Args& a, int r, int token) {
  Given v{token, 0.0f, false};
  if (token >= 0 && token < a.V) {
    v.z = logit_at<DT>(a.logits + (size_t)r * a.row_bytes, token);
    v.legal = a.bitmask == nullptr ||
              ((a.bitmask[(size_t)r * a.bm_stride + (token >> 5)] >> (token & 31)) & 1u);
  }
  return v;
}

// Writes one row's outputs; called by every thread of a workgroup of `threads`,
// with the row's joined statistics (has: a finite maximum), the thread's slot, and
// (top_n > 0) `n_list` distinct keys in LDS that hold its top tokens.
template <int DT>
__device__ __forceinline__ void finish_row(const Args& a, int r, int tid, int threads, float m,
                                           float R, bool has, float E, bool any, float T,
                                           Given given, const uint64_t* list, int n_list) {
  float* const lps = a.logprobs + (size_t)r * a.G;
  int bad = given.token < -1 || given.token >= a.V;
  for (int g = tid + threads; g < a.G; g += threads) {
    const int t = a.tokens[(size_t)r * a.G + g];
    bad |= t < -1 || t >= a.V;
  }
  if (threads > 64) bad = __syncthreads_or(bad);
  else bad = ballot(bad) != 0;
  int status = QS_ROW_OK;
  if (bad || !(T > 0.0f) || T == INFINITY) status = QS_ROW_BAD_PARAM;
  else if (!any) status = QS_ROW_EMPTY;
  else if (!(R < INFINITY)) status = QS_ROW_NONFINITE;
  else if (!has) status = QS_ROW_ALL_NEG_INF;
  const bool ok = status == QS_ROW_OK;
  const float log_sum = ok ? log1pf(R) : NAN;
  if (tid == 0) {
    a.status[r] = status;
    a.row_max[r] = ok ? m : NAN;
    a.log_sum[r] = log_sum;
    if (a.entropy) a.entropy[r] = ok ? log_sum - kLn2 * (E / (1.0f + R)) : NAN;
  }
  for (int g = tid; g < a.G; g += threads) {
    if (g != tid) given = load_given<DT>(a, r, given_token(a, r, g));
    float lp = ok ? -INFINITY : NAN;
    if (given.token == -1) lp = 0.0f;
    else if (ok && given.legal) lp = (given.z - m) / T - log_sum;
    lps[g] = lp;
  }
  if (a.top_n == 0) return;
  int32_t* const ids = a.top_ids + (size_t)r * a.top_n;
  float* const tlp = a.top_lp + (size_t)r * a.top_n;
  if (!ok) n_list = 0;
  for (int i = tid; i < n_list; i += threads) {
    const uint64_t key = list[i];
    int rank = 0;
    int j = 0;
    for (; j + 8 <= n_list; j += 8) {  // eight LDS reads under way at a time
#pragma unroll
      for (int e = 0; e < 8; ++e) rank += list[j + e] > key;
    }
    for (; j < n_list; ++j) rank += list[j] > key;
    if (rank < a.top_n) {
      ids[rank] = (int32_t)~(uint32_t)key;
      tlp[rank] = (Keys<QS_F32>::value((uint32_t)(key >> 32)) - m) / T - log_sum;
    }
  }
  for (int j = n_list + tid; j < a.top_n; j += threads) {
    ids[j] = -1;
    tlp[j] = -INFINITY;
  }
}

// One workgroup per row (ROW: parts == 1, outputs written here) or per part.
template <int DT, int THREADS, int NL, bool MASK, bool TOP, bool ROW>
__global__ void __launch_bounds__(THREADS)
    score_kernel(Args a, int parts, int part_loads, Part* ws_parts, uint64_t* ws_list) {
  constexpr int kWavesHere = THREADS / 64;
  constexpr int P = kPer<DT>;
  constexpr bool kTable = MASK && DT == QS_BF16;
  __shared__ Shared s;
  __shared__ uint4 s_masks[kTable ? 256 : 1];  // masks_of every byte of legal bits
  const int tid = threadIdx.x;
  const int lane = lane_id();
  const int w = tid >> 6;
  const int r = ROW ? (int)blockIdx.x : (int)(blockIdx.x / (unsigned)parts);
  const int part = ROW ? 0 : (int)(blockIdx.x - (unsigned)r * (unsigned)parts);
  const int begin = part * part_loads * THREADS * P;  // first token of this workgroup
  const uint8_t* row = a.logits + (size_t)r * a.row_bytes;
  const uint8_t* mask_row = reinterpret_cast<const uint8_t*>(a.bitmask + (size_t)r * a.bm_stride);
  int given_id = -1;
  if constexpr (ROW) given_id = given_token(a, r, tid);
  const float T = a.T ? a.T[r] : 1.0f;
  const float c = scale_of(T);

  // requests: 16 bytes per lane and load; loads that begin past the row's end
  // are left out (a 16-byte chunk that begins inside the row ends inside its
  // stride)
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
  Given given{-1, 0.0f, false};
  if constexpr (ROW) given = load_given<DT>(a, r, given_id);
  // a load's legal bits: the bitmask's, none past the row's end
  auto bits_at = [&](int i, uint32_t bits) {
    if constexpr (P == 4) bits = MASK ? bits >> (i & 4) : bits;
    const int left = a.V - i;
    return bits & (left >= P ? (1u << P) - 1u : left > 0 ? (1u << left) - 1u : 0u);
  };
  if (TOP && tid == 0) s.count = s.n_lanes = 0;
  if constexpr (kTable) {
    for (int k = tid; k < 256; k += THREADS) s_masks[k] = masks_of<DT>((uint32_t)k);
    __syncthreads();
  }

  // largest legal token of the lane; illegal ones become -inf
  Largest<DT> largest;
  uint32_t any = 0u;
#pragma unroll
  for (int u = 0; u < NL; ++u) {
    const uint32_t bits = bits_at(begin + (u * THREADS + tid) * P, legal[u]);
    any |= bits;
    if constexpr (kTable) v[u] = blank<DT>(v[u], s_masks[bits]);
    else if (MASK || bits != (1u << P) - 1u) v[u] = blank<DT>(v[u], masks_of<DT>(bits));
    largest.add(v[u]);
  }
  const float lane_max = fmaxf(largest.value(), -3.402823466e38f);
  const float wave_max = wave_max_f32(lane_max);
  if constexpr (TOP) {
    static_assert(THREADS == kGroups || THREADS == 4 * kGroups, "groups of 1 or 4 lanes");
    uint32_t* const group = reinterpret_cast<uint32_t*>(s.group);
    if constexpr (THREADS == kGroups) {
      group[tid] = key_of(lane_max);
    } else {
      float g = fmaxf(lane_max, dpp_f32<kDppXor1>(lane_max));
      g = fmaxf(g, dpp_f32<kDppXor2>(g));
      if ((lane & 3) == 0) group[tid >> 2] = key_of(g);
    }
  }

  // the wave's sums against its own maximum
  float S[2] = {0.0f, 0.0f}, E[2] = {0.0f, 0.0f};
  const float k = wave_max * c;
  if (fabsf(k) < kFused && c < 1e30f) {
#pragma unroll
    for (int u = 0; u < NL; ++u) {
      opaque(v[u]);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float d = fmaf(token<DT>(v[u], e), c, -k);
        const float x = exp2_hw(d);
        S[e & 1] += x;
        E[e & 1] = fmaf(x, fmaxf(d, -200.0f), E[e & 1]);  // not 0 times -inf
      }
    }
    const float over = fmaf(wave_max, c, -k), f = exp2_hw(-over);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      E[e] = f * (E[e] - over * S[e]);
      S[e] *= f;
    }
  } else {
#pragma unroll
    for (int u = 0; u < NL; ++u) {
      opaque(v[u]);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float d = (token<DT>(v[u], e) - wave_max) * c;
        const float x = exp2_hw(d);
        S[e & 1] += x;
        E[e & 1] = fmaf(x, fmaxf(d, -200.0f), E[e & 1]);
      }
    }
  }
  float Rw = wave_sum_f32(S[0] + S[1]), Ew = wave_sum_f32(E[0] + E[1]);
  bool has = true;
  if (Rw >= kPlain || Rw != Rw) {
    Rw -= 1.0f;
  } else {
    // the maximum's lane again, a load to each of the first lanes, without the one
    const int peak = __builtin_ctzll(ballot(lane_max == wave_max));
    const int i = begin + (lane * THREADS + (tid & ~63) + peak) * P;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    uint32_t bits = 0u;
    if (lane < part_loads && i < a.V) {
      q = *reinterpret_cast<const uint4*>(row + (size_t)i * (16 / P));
      bits = bits_at(i, MASK ? mask_row[i >> 3] : 0xFFu);
    }
    q = blank<DT>(q, masks_of<DT>(bits));
    bool is_max = false;
#pragma unroll
    for (int e = 0; e < P; ++e) is_max |= token<DT>(q, e) == wave_max;
    const uint64_t holders = ballot(is_max);
    has = holders != 0u;
    bool out = !has || lane != __builtin_ctzll(holders);  // the one is not here
    float R = 0.0f, ER = 0.0f;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const float z = token<DT>(q, e), d = (z - wave_max) * c;
      const bool one = !out && z == wave_max;
      const float x = one ? 0.0f : exp2_hw(d);
      R += x;
      ER = fmaf(x, fmaxf(d, -200.0f), ER);
      out |= one;
    }
    Rw = wave_sum_f32(lane == peak ? R : R + (S[0] + S[1]));
    Ew = wave_sum_f32(lane == peak ? ER : ER + (E[0] + E[1]));
  }
  const bool anyw = ballot(any != 0u) != 0;
  if (lane == 0) {
    s.m[w] = wave_max;
    s.R[w] = Rw;
    s.E[w] = Ew;
    s.any[w] = anyw;
    s.has[w] = has;
  }
  __syncthreads();
  float top = s.m[0];
  bool any_all = s.any[0] != 0u, has_all = s.has[0] != 0u;
#pragma unroll
  for (int k = 1; k < kWavesHere; ++k) {
    top = fmaxf(top, s.m[k]);
    any_all |= s.any[k] != 0u;
    has_all |= s.has[k] != 0u;
  }
  float R_all = 0.0f, E_all = 0.0f;
  bool left_out = false;  // the one of the first wave that holds the top
#pragma unroll
  for (int k = 0; k < kWavesHere; ++k) {
    const float d = rel(s.m[k], top, c);
    const float fk = exp2_hw(d), one = s.has[k] ? 1.0f : 0.0f;
    const bool here = !left_out && s.has[k] && s.m[k] == top;
    R_all += fk * (here ? s.R[k] : s.R[k] + one);
    E_all += fk * (s.E[k] + d * (s.R[k] + one));
    left_out |= here;
  }

  int n_list = 0;
  uint32_t t = 0u;
  if constexpr (TOP) {
    // finite tokens only: keys above -inf's (groups without one hold the key of
    // -FLT_MAX, the lowest of those). One wave searches: in every wave the search
    // would cost as much as half a lane's exponentials.
    if (w == 0) {
      t = max(wave_nth_high16(s.group[lane], a.top_n), Keys<QS_F32>::kNegInf + 1u);
      if (lane == 0) s.t = t;
    }
    __syncthreads();
    t = s.t;
    if (key_of(lane_max) >= t) s.lanes[atomicAdd(&s.n_lanes, 1)] = (uint16_t)tid;
    __syncthreads();
    const float tz = Keys<QS_F32>::value(t);
    const int chunks = s.n_lanes * part_loads;
    for (int j = tid; j < chunks; j += THREADS) {
      const int l = (int)((unsigned)j / (unsigned)part_loads), u = j - l * part_loads;
      const int i = begin + (u * THREADS + s.lanes[l]) * P;
      if (i >= a.V) continue;
      const uint32_t bits = bits_at(i, MASK ? mask_row[i >> 3] : 0xFFu);
      const uint4 q = blank<DT>(*reinterpret_cast<const uint4*>(row + (size_t)i * (16 / P)),
                                masks_of<DT>(bits));
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float z = token<DT>(q, e);
        if (z >= tz) {
          const int at = atomicAdd(&s.count, 1);
          if (at < kListCap) s.list[at] = ((uint64_t)key_of(z) << 32) | (uint32_t)~(i + e);
        }
      }
    }
    __syncthreads();
    n_list = s.count;
    if (n_list > kListCap) {
      // too many at or above t: the n largest keys, each below the one before
      uint64_t prev = ~0ull;
      n_list = 0;
      for (int j = 0; j < a.top_n; ++j) {
        uint64_t best = 0u;
        const int end = min(a.V, begin + part_loads * THREADS * P);
        const uint32_t* bm = MASK ? a.bitmask + (size_t)r * a.bm_stride : nullptr;
        for (int i = begin + tid; i < end; i += THREADS) {
          const float z = logit_at<DT>(row, i);
          if ((MASK && !((bm[i >> 5] >> (i & 31)) & 1u)) || z == -INFINITY) continue;
          const uint64_t key = ((uint64_t)key_of(z) << 32) | (uint32_t)~i;
          if (key < prev && key > best) best = key;
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
          const uint64_t o = (uint64_t)__shfl_xor((long long)best, off, 64);
          best = o > best ? o : best;
        }
        if (lane == 0) s.best[w] = best;
        __syncthreads();
        for (int k = 0; k < kWavesHere; ++k) best = s.best[k] > best ? s.best[k] : best;
        __syncthreads();
        if (best == 0u) break;  // the same in every thread
        if (tid == 0) s.list[j] = best;
        prev = best;
        n_list = j + 1;
      }
      __syncthreads();
    }
  }
  if constexpr (ROW) {
    finish_row<DT>(a, r, tid, THREADS, top, R_all, has_all, E_all, any_all, T, given, s.list,
                   n_list);
  } else {
    const size_t p = (size_t)r * parts + part;
    if (tid == 0) {
      Part out;
      out.m = top;
      out.R = R_all;
      out.E = E_all;
      out.any = any_all;
      out.t = t;
      out.count = n_list;
      out.has = has_all;
      out.pad = 0u;
      ws_parts[p] = out;
    }
    if constexpr (TOP)
      for (int i = tid; i < n_list; i += THREADS) ws_list[p * kListCap + i] = s.list[i];
  }
}

// Joins the parts of each row: one workgroup per row (one wave without top
// tokens).
template <int DT, bool TOP>
__global__ void __launch_bounds__(TOP ? 256 : 64)
    join_kernel(Args a, int parts, const Part* ws_parts, const uint64_t* ws_list) {
  constexpr int kThreadsHere = TOP ? 256 : 64;
  __shared__ uint64_t s_list[TOP ? kJoinCap : 1];
  __shared__ uint64_t s_best[4];
  __shared__ int s_count;
  const int r = blockIdx.x;
  const int tid = threadIdx.x;
  const int lane = lane_id();
  const Part* p = ws_parts + (size_t)r * parts;
  // requests that need nothing else first: the thread's slot, a part per lane,
  // and the first 64 keys of 4 lists per wave whatever their counts
  const int given_id = given_token(a, r, tid);
  Part mine{-3.402823466e38f, 0.0f, 0.0f, 0u, 0u, 0, 0u, 0u};
  if (lane < parts) mine = p[lane];
  const uint64_t* const list = ws_list + (size_t)r * parts * kListCap;
  constexpr int kAhead = 4;
  uint64_t ahead[kAhead];
  if constexpr (TOP) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = (tid >> 6) + j * (kThreadsHere / 64);
      ahead[j] = k < parts ? list[(size_t)k * kListCap + lane] : 0u;
    }
  }
  const float T = a.T ? a.T[r] : 1.0f;
  const float c = scale_of(T);
  const Given given = load_given<DT>(a, r, given_id);
  // every wave joins all parts (the same values in every thread)
  float m = mine.m;
  uint32_t t = mine.t, any = mine.any;
  for (int k = lane + 64; k < parts; k += 64) {
    m = fmaxf(m, p[k].m);
    t = max(t, p[k].t);
    any |= p[k].any;
  }
  m = wave_max_f32(m);
  t = wave_reduce<OpMax>(t);
  const bool any_all = ballot(any != 0u) != 0;
  // a part's maximum counts 1, but for the first part's that holds the row's
  uint32_t first = mine.has && mine.m == m ? ~(uint32_t)lane : 0u;
  for (int k = lane + 64; k < parts; k += 64)
    if (p[k].has && p[k].m == m) first = max(first, ~(uint32_t)k);
  first = ~wave_reduce<OpMax>(first);
  const bool has_all = first != ~0u;
  const float d0 = rel(mine.m, m, c), f0 = exp2_hw(d0), one0 = mine.has ? 1.0f : 0.0f;
  float R = f0 * ((uint32_t)lane == first ? mine.R : mine.R + one0);
  float E = f0 * (mine.E + d0 * (mine.R + one0));
  for (int k = lane + 64; k < parts; k += 64) {
    const float d = rel(p[k].m, m, c);
    const float f = exp2_hw(d), one = p[k].has ? 1.0f : 0.0f;
    R += f * ((uint32_t)k == first ? p[k].R : p[k].R + one);
    E += f * (p[k].E + d * (p[k].R + one));
  }
  R = wave_sum_f32(R);
  E = wave_sum_f32(E);
  int n_list = 0;
  if constexpr (TOP) {
    // the row's n-th largest token is at or above every part's t
    if (tid == 0) s_count = 0;
    __syncthreads();
    auto add = [&](uint64_t key) {
      if ((uint32_t)(key >> 32) >= t) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kJoinCap) s_list[at] = key;
      }
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = (tid >> 6) + j * (kThreadsHere / 64);
      if (k < parts && lane < __shfl(mine.count, k, 64)) add(ahead[j]);
    }
    for (int j = 0, k = tid >> 6; k < parts; ++j, k += kThreadsHere / 64) {
      const int n = k < 64 ? __shfl(mine.count, k, 64) : p[k].count;
      for (int i = lane + (j < kAhead ? 64 : 0); i < n; i += 64) add(list[(size_t)k * kListCap + i]);
    }
    __syncthreads();
    n_list = s_count;
    if (n_list > kJoinCap) {
      // more than the list holds: the n largest keys, one after another
      uint64_t prev = ~0ull;
      n_list = 0;
      for (int j = 0; j < a.top_n; ++j) {
        uint64_t best = 0u;
        for (int k = tid >> 6; k < parts; k += kThreadsHere / 64) {
          const int n = p[k].count;
          for (int i = lane; i < n; i += 64) {
            const uint64_t key = list[(size_t)k * kListCap + i];
            if (key < prev && key > best) best = key;
          }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
          const uint64_t o = (uint64_t)__shfl_xor((long long)best, off, 64);
          best = o > best ? o : best;
        }
        if (lane == 0) s_best[tid >> 6] = best;
        __syncthreads();
        for (int k = 0; k < kThreadsHere / 64; ++k) best = s_best[k] > best ? s_best[k] : best;
        __syncthreads();
        if (best == 0u) break;
        if (tid == 0) s_list[j] = best;
        prev = best;
        n_list = j + 1;
      }
      __syncthreads();
    }
  }
  finish_row<DT>(a, r, tid, kThreadsHere, m, R, has_all, E, any_all, T, given, s_list, n_list);
}

template <int DT, int THREADS, int NL, bool ROW>
void launch(const Args& a, int blocks, int parts, int part_loads, Part* wp, uint64_t* wl,
            hipStream_t st) {
  const dim3 grid((unsigned)blocks), block(THREADS);
  const bool mask = a.bitmask != nullptr, top = a.top_n > 0;
  if (mask && top)
    hipLaunchKernelGGL((score_kernel<DT, THREADS, NL, true, true, ROW>), grid, block, 0, st, a,
                       parts, part_loads, wp, wl);
  else if (mask)
    hipLaunchKernelGGL((score_kernel<DT, THREADS, NL, true, false, ROW>), grid, block, 0, st, a,
                       parts, part_loads, wp, wl);
  else if (top)
    hipLaunchKernelGGL((score_kernel<DT, THREADS, NL, false, true, ROW>), grid, block, 0, st, a,
                       parts, part_loads, wp, wl);
  else
    hipLaunchKernelGGL((score_kernel<DT, THREADS, NL, false, false, ROW>), grid, block, 0, st, a,
                       parts, part_loads, wp, wl);
}

template <int DT>
hipError_t launch_dt(const Args& a, int B, int parts, uint8_t* ws, hipStream_t st) {
  constexpr int P = kPer<DT>;
  if (parts == 1) {
    if (a.V <= kSmallBlock * kSmallLoads * P)
      launch<DT, kSmallBlock, kSmallLoads, true>(
          a, B, 1, (a.V + kSmallBlock * P - 1) / (kSmallBlock * P), nullptr, nullptr, st);
    else
      launch<DT, kRowBlock, kRowLoads, true>(
          a, B, 1, (a.V + kRowBlock * P - 1) / (kRowBlock * P), nullptr, nullptr, st);
    return hipGetLastError();
  }
  Part* const wp = reinterpret_cast<Part*>(ws);
  uint64_t* const wl =
      reinterpret_cast<uint64_t*>(ws + align256((size_t)B * parts * sizeof(Part)));
  // parts of equal length, in whole loads
  const int loads = (a.V + kPartBlock * P - 1) / (kPartBlock * P);
  const int each = (loads + parts - 1) / parts;
  if (loads_for(B, a.V, DT) == kPartLoads)
    launch<DT, kPartBlock, kPartLoads, false>(a, B * parts, parts, each, wp, wl, st);
  else
    launch<DT, kPartBlock, kShortLoads, false>(a, B * parts, parts, each, wp, wl, st);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  if (a.top_n > 0)
    hipLaunchKernelGGL((join_kernel<DT, true>), dim3((unsigned)B), dim3(256), 0, st, a, parts, wp,
                       wl);
  else
    hipLaunchKernelGGL((join_kernel<DT, false>), dim3((unsigned)B), dim3(64), 0, st, a, parts, wp,
                       wl);
  return hipGetLastError();
}

}  // namespace

// Enough for every batch of at most B rows: the largest of them whose parts are
// short has up to twice the parts of a somewhat larger one whose parts are long.
size_t workspace_bytes(int64_t B, int64_t V, int dtype, int64_t top_n) {
  const int64_t parts = parts_for(B, V, dtype);
  if (parts == 1) return 0;
  const int64_t few = kFewParts / parts_of(V, dtype, kPartLoads);  // rows of the last such batch
  size_t n = (size_t)B * parts;
  if (B > few) n = std::max(n, (size_t)few * parts_of(V, dtype, kShortLoads));
  return align256(n * sizeof(Part)) + (top_n > 0 ? n * kListCap * sizeof(uint64_t) : 0);
}

bool grid_fits(int64_t B, int64_t V, int dtype) {
  return B * parts_for(B, V, dtype) * kPartBlock < (int64_t)1 << 32;
}

hipError_t launch_score(const Args& a, int dtype, int B, void* workspace, hipStream_t st) {
  const int parts = (int)parts_for(B, a.V, dtype);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  return dtype == QS_F32 ? launch_dt<QS_F32>(a, B, parts, ws, st)
                         : launch_dt<QS_BF16>(a, B, parts, ws, st);
}

}  // namespace score
}  // namespace qs
