// Low-rank adapters of many requests beside a shared output projection: with a the
// adapter of row b,
//   y[b][v] = z[b][v] + scale[a] sum_r up[a][v][r] u[b][r],
//   u[b][r] = sum_k down[a][r][k] x[b][k].
// Two launches: the rows' low-rank coordinates scale * u, then their product with the
// up factors on top of the logits. Every used adapter is read once per 64 rows,
// however they share it; what bounds the calls is reading the up factors, and the
// logits read and written.
//
// The second product runs on the matrix cores (16x16x32) with the factor's rows on one
// side and 16 rows of the batch on the other. A product's column depends on its own
// batch row alone, so an adapter is multiplied with all 16 and taken by the rows that
// are its own: no gathering of rows by adapter, and what another row holds (an
// infinity, uninitialised scratch) cannot reach a result. The coordinates are float32;
// each is cut into three bf16 numbers of 8 bits, whose sum is it, so that products are
// exact: three products cost nothing beside the factors' bytes (one rounded to bf16
// would cost the result 2^-8 of the adapter's share). Sums are held in float32, and each
// logit is rounded once.
//
// Measured (first and second launch): 64 rows of 151936 bf16 on adapters of their own of
// rank 32, 8192 columns, 11 and 118 us (5.6 TB/s in the second, where a large copy reaches
// 5.2); on three of rank 64, 4096 columns, 5.6 and 19.9 us (4.9 TB/s); 16 rows of 128256
// fp32, each its own of rank 32, 3.9 and 23.5 us (6.2 TB/s); 1 row of 151936, rank 16, 3.5
// and 3.9 us, two dependent loads each.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qs.h"
#include "qs_adapters.hpp"
#include "qs_device.hpp"

namespace qs {
namespace adapters {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 64;         // batch rows of a block
constexpr int kTerms = 3;         // bf16 numbers per coordinate
constexpr int kUpWaves = 4;
constexpr int kTiles = 2;         // tiles of 16 vocabulary rows per wave
constexpr int kWavesWanted = 4096;  // up to which a block's adapters are dealt out
constexpr int kAhead = 8;         // loads of 512 columns that a wave of the first product
                                  // requests at a time

// The workspace holds the coordinates as the second product takes them: per tile of
// 16 batch rows, step of 32 ranks and term the 64 lanes' 8 bf16 numbers, lane
// (row n, ranks 8 g to 8 g + 7) at 16 g + n.
constexpr int kStepBytes = kTerms * 64 * 16;

// The adapter of each of a block's rows in its lane; -1: none, or none that exists.
__device__ __forceinline__ int row_index(const Args& a, int row0, int lane) {
  const int b = row0 + lane;
  const int n = b < a.B ? a.index[b] : -1;
  return n >= 0 && n < a.count ? n : -1;
}

// The rows' coordinates, a wave to each row and rank: few rows spread over as many
// compute units as they have ranks, each wave requests up to 8 KiB of the factor before
// it uses any, and rows that share an adapter read it from the L2. (On the matrix cores,
// 16 ranks and the rows that share an adapter to a workgroup: 1 row of 4096 columns, rank
// 16, 6.5 us, one compute unit's loads, against 3.5; 64 rows of 8192 on adapters of their
// own, rank 32, 14.2 against 10.7; 64 on 3 of rank 64, 4096 columns, 7.9 against 6.1.
// Four ranks a wave, which reads the hidden state once for them, were up to 2 us slower.)
__global__ void __launch_bounds__(256) down_kernel(Args a, int steps) {
  const int lane = lane_id();
  const int item = uni((int)(blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6)));
  const int ranks = steps * 32;            // with zeros behind the last
  const int b = item / ranks, q = item - b * ranks;
  if (b >= a.B) return;
  const int n = a.index[b];
  const bool valid = n >= -1 && n < a.count;
  if (q == 0 && lane == 0) a.status[b] = valid ? QS_ROW_OK : QS_ROW_BAD_PARAM;
  if (!valid || n < 0) return;
  float u = 0.0f;
  if (q < a.rank) {
    const float scale = a.scale ? a.scale[n] : 1.0f;
    const uint16_t* const x = a.hidden + (size_t)b * a.hidden_stride;
    const uint16_t* const d =
        a.down + (size_t)n * a.down_stride + (size_t)q * a.down_row_stride;
    float sum[2] = {0.0f, 0.0f};
    for (int k0 = lane * 8; k0 < a.K; k0 += kAhead * 512) {
      uint4 dv[kAhead], xv[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        dv[j] = xv[j] = make_uint4(0u, 0u, 0u, 0u);
        if (k0 + j * 512 < a.K) {
          dv[j] = *reinterpret_cast<const uint4*>(d + k0 + j * 512);
          xv[j] = *reinterpret_cast<const uint4*>(x + k0 + j * 512);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint32_t ds[4] = {dv[j].x, dv[j].y, dv[j].z, dv[j].w};
        const uint32_t xs[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[0] = fmaf(__uint_as_float(ds[e] << 16), __uint_as_float(xs[e] << 16), sum[0]);
          sum[1] = fmaf(__uint_as_float(ds[e] & 0xFFFF0000u), __uint_as_float(xs[e] & 0xFFFF0000u),
                        sum[1]);
        }
      }
    }
    u = sum[0] + sum[1];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) u += __shfl_xor(u, off, 64);
    u *= scale;
  }
  if (lane == 0) {
    uint8_t* const out = a.low + ((size_t)(b / 16) * steps + (q >> 5)) * kStepBytes +
                         (((q & 31) >> 3) * 16 + (b & 15)) * 16 + (q & 7) * 2;
#pragma unroll
    for (int k = 0; k < kTerms; ++k) {
      const __bf16 part = (__bf16)u;
      *reinterpret_cast<__bf16*>(out + k * 1024) = part;
      u -= (float)part;
    }
  }
}

// The logits. A wave takes kTiles tiles of 16 vocabulary rows and up to RT tiles of 16
// batch rows: the logits are its accumulators, and it walks the block's adapters, A at a
// time (2 where their rows are so short, up to rank 16, that one's are too few bytes under
// way: 64 rows of 151936 on adapters of rank 16 of their own 69 us against 77; of rank 32
// 130 against 126, of 64 102 against 100). Two tiles leave room for more waves than four
// (64 rows on 16 adapters of rank 128: 147 us against 172; on 4 of rank 16, float32, 24.5
// against 33). The tiles' rows are dealt out so that a lane holds 4 kTiles consecutive
// logits of one batch row: product row 4 g + e of tile t is vocabulary row
// 4 (kTiles g + t) + e.
//
// A wave that walks many adapters waits for each one's factors, so where the vocabulary
// makes few waves a block's adapters are dealt out to up to 64 groups of workgroups, each
// with the rows of its own (64 rows on adapters of their own of rank 16: 1000 tokens 7.0
// us against 26.6, 8000 10.8 against 32, 32000 20.7 against 34, 64000 31 against 37; past
// kWavesWanted, 128256 in two groups, 62 against 57. 3 adapters of rank 64: 9.9 against
// 12.0, 10.1 against 12.1, 11.7 against 12.7, 15.3 against 15.8 and, past it, 24.5 against
// 21.0).
template <int DT, int KS, int RT, int A>
__global__ void __launch_bounds__(kUpWaves * 64)
    up_kernel(Args a, int tiles, int groups_log2, uint64_t every) {
  constexpr int kSpan = 16 * kTiles;      // vocabulary rows per wave
  constexpr int P = DT == QS_F32 ? 4 : 8; // logits per 16 bytes
  __shared__ uint4 s_low[RT * KS * kTerms * 64];
  const int tid = threadIdx.x, lane = lane_id(), w = uni(tid >> 6);
  const int n = lane & 15, kg = lane >> 4;
  const int group = (int)blockIdx.y & ((1 << groups_log2) - 1);
  const int row0 = ((int)blockIdx.y >> groups_log2) * kRows;
  const int tile = (int)blockIdx.x * kUpWaves + w;
  const int v0 = tile * kSpan, first = v0 + kg * 4 * kTiles;  // the lane's first logit
  const int mine = row_index(a, row0, lane);
  // this workgroup's adapters, by their first rows, and the rows they cover; the first
  // group copies the rows without an adapter
  const uint64_t none = ~ballot(mine >= 0);
  uint64_t leaders = ~none, rows = ~none;
  if (groups_log2 > 0) {
    leaders = rows = 0u;
    for (uint64_t left = ~none & every << group; left != 0u;) {
      const int l = __builtin_ctzll(left);
      const uint64_t members = ballot(mine == (int)readlane_u32((uint32_t)mine, l));
      left &= ~members;
      if (__builtin_ctzll(members) != l) continue;
      leaders |= 1ull << l;
      rows |= members;
    }
  }
  if (group == 0 && a.out != a.logits) rows |= none;
  if (rows == 0u) return;

  int own[RT];     // the adapter of this lane's batch row
  f32x4 y[kTiles][RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    own[t] = __shfl(mine, t * 16 + n, 64);
    const int b = row0 + t * 16 + n;
    const bool use = b < a.B && ((rows >> (t * 16 + n)) & 1u);
    const uint8_t* const z = a.logits + (size_t)(use ? b : 0) * a.row_bytes;
#pragma unroll
    for (int c = 0; c < 4 * kTiles / P; ++c) {
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (use && first + c * P < a.V)
        q = *reinterpret_cast<const uint4*>(z + (size_t)(first + c * P) * (16 / P));
      const uint32_t word[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const int i = c * P + e;
        if constexpr (DT == QS_F32) y[i >> 2][t][i & 3] = __uint_as_float(word[e]);
        else y[i >> 2][t][i & 3] =
            __uint_as_float((e & 1) ? word[e >> 1] & 0xFFFF0000u : word[e >> 1] << 16);
      }
    }
  }
  // their coordinates, as they lie
  const uint4* const low =
      reinterpret_cast<const uint4*>(a.low + (size_t)(row0 / 16) * KS * kStepBytes);
  for (int i = tid; i < RT * KS * kTerms * 64; i += kUpWaves * 64) {
    if ((rows & ~none) >> (i / (KS * kTerms * 64) * 16 + (i & 15)) & 1u) s_low[i] = low[i];
  }
  __syncthreads();
  if (tile >= tiles) return;

  for (uint64_t left = leaders; left != 0u;) {
    int d[A];
    uint64_t members[A];
    bf16x8 f[A][kTiles][KS];
#pragma unroll
    for (int j = 0; j < A; ++j) {
      d[j] = -1;
      members[j] = 0u;
      if (left == 0u) continue;
      d[j] = readlane_u32((uint32_t)mine, __builtin_ctzll(left));
      members[j] = ballot(mine == d[j]);
      left &= ~members[j];
      const uint16_t* const up = a.up + (size_t)d[j] * a.up_stride;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const int v = min(v0 + (n >> 2) * 4 * kTiles + i * 4 + (n & 3), a.V - 1);
        const uint16_t* const row = up + (size_t)v * a.up_row_stride;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint4 q = make_uint4(0u, 0u, 0u, 0u);
          if (s * 32 + kg * 8 < a.rank) q = *reinterpret_cast<const uint4*>(row + s * 32 + kg * 8);
          f[j][i][s] = __builtin_bit_cast(bf16x8, q);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < A; ++j) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if (((members[j] >> (t * 16)) & 0xFFFFu) == 0u) continue;
        f32x4 acc[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) acc[i] = y[i][t];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
#pragma unroll
          for (int k = 0; k < kTerms; ++k) {
            const bf16x8 u =
                __builtin_bit_cast(bf16x8, s_low[((t * KS + s) * kTerms + k) * 64 + lane]);
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
              acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[j][i][s], u, acc[i], 0, 0, 0);
          }
        }
        const bool take = own[t] == d[j];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[i][t][e] = take ? acc[i][e] : y[i][t][e];
        }
      }
    }
  }

#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int b = row0 + t * 16 + n;
    if (b >= a.B || !((rows >> (t * 16 + n)) & 1u)) continue;
    uint8_t* const out = a.out + (size_t)b * a.out_bytes;
#pragma unroll
    for (int c = 0; c < 4 * kTiles / P; ++c) {
      const int v = first + c * P;
      if (v >= a.V) break;
      uint32_t word[4];
      if constexpr (DT == QS_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) word[e] = __float_as_uint(y[c][t][e]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bf16x4 half = __builtin_convertvector(y[c * 2 + h][t], bf16x4);
          __builtin_memcpy(word + 2 * h, &half, 8);
        }
      }
      if (a.V - v >= P) {
        *reinterpret_cast<uint4*>(out + (size_t)v * (16 / P)) =
            make_uint4(word[0], word[1], word[2], word[3]);
      } else {  // the row's last logits: what lies behind them stays
#pragma unroll
        for (int e = 0; e < P - 1; ++e) {
          if (v + e < a.V) {
            if constexpr (DT == QS_F32) reinterpret_cast<uint32_t*>(out)[v + e] = word[e];
            else reinterpret_cast<uint16_t*>(out)[v + e] =
                (uint16_t)(word[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
    }
  }
}

template <int DT, int KS, int A>
void launch_up(const Args& a, hipStream_t st) {
  const int tiles = (a.V + 16 * kTiles - 1) / (16 * kTiles);
  const int64_t waves = (int64_t)tiles * ((a.B + kRows - 1) / kRows);
  int groups_log2 = 0;
  while (groups_log2 < 6 && 1 << groups_log2 < a.B && waves << (groups_log2 + 1) <= kWavesWanted)
    ++groups_log2;
  // a row in each group's turn: every 2^groups_log2-th bit
  const uint64_t every = ~0ull / (~0ull >> (64 - (1 << groups_log2)));
  const dim3 grid((unsigned)((tiles + kUpWaves - 1) / kUpWaves),
                  (unsigned)((a.B + kRows - 1) / kRows) << groups_log2);
  const dim3 block(kUpWaves * 64);
  auto run = [&](auto* kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, a, tiles, groups_log2, every); };
  if (a.B <= 16) run(up_kernel<DT, KS, 1, A>);
  else if (a.B <= 32) run(up_kernel<DT, KS, 2, A>);
  else run(up_kernel<DT, KS, 4, A>);
}

template <int DT>
void launch_rank(const Args& a, int steps, hipStream_t st) {
  if (a.rank <= 16) launch_up<DT, 1, 2>(a, st);
  else if (steps == 1) launch_up<DT, 1, 1>(a, st);
  else if (steps == 2) launch_up<DT, 2, 1>(a, st);
  else if (steps == 3) launch_up<DT, 3, 1>(a, st);
  else launch_up<DT, 4, 1>(a, st);
}

int steps_of(int64_t rank) { return (int)((rank + 31) / 32); }

}  // namespace

size_t workspace_bytes(int64_t B, int64_t rank) {
  return (size_t)((B + 15) / 16) * steps_of(rank) * kStepBytes;
}

hipError_t launch_adapters(const Args& a, int dtype, hipStream_t st) {
  const int steps = steps_of(a.rank);
  const int64_t items = (int64_t)a.B * steps * 32;
  // one wave a workgroup where that spreads few waves over more compute units
  const int waves = items > 1024 ? 4 : 1;
  hipLaunchKernelGGL(down_kernel, dim3((unsigned)((items + waves - 1) / waves)), dim3(waves * 64), 0,
                     st, a, steps);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  if (dtype == QS_F32) launch_rank<QS_F32>(a, steps, st);
  else launch_rank<QS_BF16>(a, steps, st);
  return hipGetLastError();
}

}  // namespace adapters
}  // namespace qs
