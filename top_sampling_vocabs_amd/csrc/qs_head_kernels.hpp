// Output head with 4-bit weights: logits of hidden states,
//   y[b][v] = sum_g s[v][g] sum_{k in g} x[b][k] (q[v][k] - z[v][g]),
// q the codes 0..15, s a scale and z a zero point per row and group of k.
//
// The codes are streamed once from memory in the checkpoint's own row order and
// meet the matrix cores without a table: a nibble shifted to bits 3..6 under
// the exponent of 16 is the bf16 number 16 + q, so one shift and one and-or
// make two factors, and
//   sum x (q - z) = sum x (16 + q) - (16 + z) sum x
// with exact products and float32 sums; sum x is added up once per launch or per
// chunk and starts the group's sum. The scale is applied to the float32 group
// sum, never to a factor, so no weight is rounded; the logit's own rounding to
// bf16, where that is asked for, is the only one to fewer bits.
//
// A 16x16x32 product takes 16 hidden rows (A) and 16 vocabulary rows (B), 8
// columns of k per lane on both sides. Which columns those are is free as long
// as both sides agree and a product stays inside one group: a lane takes 16, 8
// or 4 bytes of codes in a row (groups of 128, 64, 32) per 128-column step. The
// nibbles i and i + 4 of a dword share a register, so the hidden values are
// laid out in the order 0 4 1 5 2 6 3 7 beforehand.
//
// Two kernels. Few rows: the codes' bytes bound the call, and the hidden values
// stay in registers for the whole launch (head_split_kernel). More rows, or
// rows too long for the registers: making factors and multiplying costs as much
// as the bytes, and one set of factors meets up to 64 hidden rows, which pass
// through LDS (head_stream_kernel).

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qs.h"
#include "qs_device.hpp"
#include "qs_head.hpp"

namespace qs {
namespace head {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStepK = 128;                // columns per step
constexpr uint32_t kOnes = 0x3F803F80u;    // two bf16 ones

// Where an MFMA's 8 columns of lane group kg lie, in chunks of the step.
template <int G>
__device__ __forceinline__ int chunk_of(int j, int kg) {
  if constexpr (G == 128) return kg * 4 + j;
  if constexpr (G == 64) return (j >> 1) * 8 + kg * 2 + (j & 1);
  return j * 4 + kg;
}

// The two constants of a code's bf16 factor, in a scalar and a vector register so
// that and and or are one instruction.
struct Pattern {
  uint32_t mant, exp;
  __device__ __forceinline__ Pattern() : mant(0x00780078u), exp(0x41804180u) {
    asm("" : "+s"(mant));
    asm("" : "+v"(exp));
  }
};

// 8 codes as the bf16 numbers 16 + q, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 factors(uint32_t c, const Pattern& k) {
  u32x4 r;
  r.x = ((c << 3) & k.mant) | k.exp;
  r.y = ((c >> 1) & k.mant) | k.exp;
  r.z = ((c >> 5) & k.mant) | k.exp;
  r.w = ((c >> 9) & k.mant) | k.exp;
  return __builtin_bit_cast(bf16x8, r);
}

// 8 hidden values in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 ordered(const uint4& v) {
  return make_uint4(bfi(0xFFFFu, v.x, v.z << 16), bfi(0xFFFFu, v.x >> 16, v.z),
                    bfi(0xFFFFu, v.y, v.w << 16), bfi(0xFFFFu, v.y >> 16, v.w));
}

__device__ __forceinline__ void store_logit(const Args& a, int b, int v, float y) {
  const size_t o = (size_t)b * a.row_stride + v;
  if (a.logits_dtype == QS_F32) static_cast<float*>(a.logits)[o] = y;
  else static_cast<__bf16*>(a.logits)[o] = (__bf16)y;
}

// ---------------------------------------------------------------------------

constexpr int kThreads8 = 512;          // 8 waves
// waves per SIMD that the registers are held to
constexpr int occupancy(int P, int MT) { return P * MT <= 4 ? 4 : 2; }

// The hidden values of one slice of k stay in each wave's registers: the NW (8 or
// 16) waves of a workgroup are KS slices of k by NW / KS tiles of 16 vocabulary
// rows, a wave holds P steps of x (16 MT hidden rows; the grid's y counts blocks
// of as many), and the workgroup walks the tiles. A wave's codes of a tile are
// P * 64 consecutive bytes a row: they are read with consecutive lanes on
// consecutive bytes (lanes in the product's own order, 16 rows apart, cost four
// times the cache accesses), one tile ahead,
// and change lanes through the wave's own LDS. The slices' float32 sums meet in
// LDS (two buffers, one barrier a tile) and are added in slice order, so the
// result does not depend on which wave is first.
//
// Measured: 1 row, 151936 x 4096 in groups of 128, 59 us (5.5 TB/s of codes and
// scales, where a large copy reaches 4.8 and a large sum 4.0); the same with 8192
// columns, 115 us (5.5 TB/s); 1 row, 32000 x 2048, 11.3 us; 16 rows, 128256 x 4096
// in groups of 64 with zero points and float32 logits, 74 us (4.0 TB/s).
template <int NW, int P, int MT, int G, int SD, bool ZEROS>
__global__ void __launch_bounds__(NW * 64, occupancy(P, MT))
    head_split_kernel(Args a, int steps, int tiles, int ks_log2) {
  constexpr int kGroups = kStepK / G;      // groups per step
  constexpr int NG = P * kGroups;          // groups per slice
  constexpr int CL = 4 * P;                // lanes per row of a code load
  constexpr int kRows = 64 / CL;           // rows per code load
  constexpr int kCodeStride = P * 64 + 16; // bytes per row in LDS
  constexpr int kScaleStride = NG + 4;     // floats per row in LDS
  constexpr int SL = NG < 4 ? NG : 4;      // lanes per row of a scale load
  constexpr int EL = NG / SL;              // scales per lane
  __shared__ f32x4 s_part[2][NW][MT][64];
  __shared__ f32x4 s_sum[NW][NG][MT][4];    // sums of x over a slice's groups
  __shared__ __align__(16) uint8_t s_code[NW][16 * kCodeStride];
  __shared__ __align__(16) float s_scale[NW][16 * kScaleStride];
  __shared__ __align__(16) float s_off[ZEROS ? NW : 1][ZEROS ? 16 * kScaleStride : 1];
  const int tid = threadIdx.x;
  const int w = uni(tid >> 6);
  const int lane = lane_id();
  const int n = lane & 15, kg = lane >> 4;
  const int KS = 1 << ks_log2, TG = NW >> ks_log2;
  const int ks = w & (KS - 1), tg = w >> ks_log2;
  const int per = (steps + KS - 1) >> ks_log2;  // at most P
  const int s0 = ks * per;
  const int mine = max(0, min(per, steps - s0));
  const int k0 = s0 * kStepK;                    // the slice's first column
  const int cols = max(0, min(mine * kStepK, a.K - k0));
  const int batches = (tiles + TG - 1) / TG;
  const int row0 = (int)blockIdx.y * MT * 16;

  // a tile's codes, scales and zero points, lanes along the rows: a scalar base
  // per tile and a lane's offset from it, which only the last tile changes
  const int c_row = lane / CL, c_chunk = lane % CL;
  const int g_row = min(lane / SL, 15), g_part = (lane % SL) * EL;
  const bool c_in = c_chunk * 32 < cols;
  const int groups = cols / G;
  constexpr int kScaleSize = SD == QS_F32 ? 4 : 2;
  using Raw = std::conditional_t<SD == QS_F32, float, uint16_t>;
  u32x4 code[P];
  Raw scale[EL];
  uint8_t zero[EL];
  auto load_tile = [&](int tile) {
    const int last = min(15, a.V - 1 - tile * 16);  // below 0 past the last tile
    const int v0 = last < 0 ? a.V - 1 : tile * 16;
    const int rows = max(last, 0);
    const uint8_t* const pc = a.codes + (size_t)v0 * a.codes_stride + (k0 >> 1);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint32_t at = (uint32_t)min(i * kRows + c_row, rows) * (uint32_t)a.codes_stride +
                          (uint32_t)c_chunk * 16u;
      if (c_in) code[i] = *reinterpret_cast<const u32x4*>(pc + at);
    }
    const int g = k0 / G;
    const uint8_t* const ps = static_cast<const uint8_t*>(a.scales) +
                              ((size_t)v0 * a.scale_stride + g) * kScaleSize;
    const uint32_t row = (uint32_t)min(g_row, rows);
    const uint32_t at = (row * (uint32_t)a.scale_stride + (uint32_t)g_part) * kScaleSize;
    const uint8_t* const pz = ZEROS ? a.zeros + (size_t)v0 * a.zero_stride + g : nullptr;
    const uint32_t zat = row * (uint32_t)a.zero_stride + (uint32_t)g_part;
    if (groups == NG) {
      __builtin_memcpy(scale, ps + at, kScaleSize * EL);
      if constexpr (ZEROS) __builtin_memcpy(zero, pz + zat, EL);
    } else {
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        scale[e] = Raw(0);
        zero[e] = 0;
        if (g_part + e < groups) {
          scale[e] = reinterpret_cast<const Raw*>(ps + at)[e];
          if constexpr (ZEROS) zero[e] = pz[zat + e];
        }
      }
    }
  };
  int batch = blockIdx.x;
  load_tile(batch * TG + tg);

  bf16x8 x[P][4][MT];
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int k = k0 + p * kStepK + chunk_of<G>(j, kg) * 8;
        const int m = min(row0 + t * 16 + n, a.B - 1);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (p < mine && k < a.K)
          v = ordered(*reinterpret_cast<const uint4*>(a.hidden + (size_t)m * a.hidden_stride + k));
        x[p][j][t] = __builtin_bit_cast(bf16x8, v);
      }
    }
  }
  {
    const u32x4 one = {kOnes, kOnes, kOnes, kOnes};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, one);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int jj = 0; jj < G / 32; ++jj) {
          const int j = g * (G / 32) + jj;
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j / 4][j % 4][t], ones, sum, 0, 0, 0);
        }
        // every column holds the same sums: one lane per four rows writes them
        if (!ZEROS) sum *= -24.0f;
        if (n == 0) s_sum[w][g][t][kg] = sum;
      }
    }
  }
  const Pattern pattern;

  int buf = 0;
  for (; batch < batches; batch += gridDim.x) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      *reinterpret_cast<u32x4*>(&s_code[w][(i * kRows + c_row) * kCodeStride + c_chunk * 16]) =
          code[i];
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      float sc;
      if constexpr (SD == QS_F32) sc = scale[e];
      else sc = __uint_as_float((uint32_t)scale[e] << 16);
      s_scale[w][g_row * kScaleStride + g_part + e] = sc;
      if constexpr (ZEROS) s_off[w][g_row * kScaleStride + g_part + e] = -16.0f - (float)zero[e];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_sched_barrier(0);
    load_tile((batch + (int)gridDim.x) * TG + tg);
    __builtin_amdgcn_sched_barrier(0);

    f32x4 y[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) y[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint8_t* const row = &s_code[w][n * kCodeStride + p * 64];
      uint32_t q[4];
      if constexpr (G == 128) {
        *reinterpret_cast<u32x4*>(q) = *reinterpret_cast<const u32x4*>(row + kg * 16);
      } else if constexpr (G == 64) {
        *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(row + kg * 8);
        *reinterpret_cast<uint2*>(q + 2) = *reinterpret_cast<const uint2*>(row + 32 + kg * 8);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          q[j] = *reinterpret_cast<const uint32_t*>(row + j * 16 + kg * 4);
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        constexpr int J = G / 32;
        const float sc = s_scale[w][n * kScaleStride + p * kGroups + g];
        f32x4 acc[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          acc[t] = s_sum[w][p * kGroups + g][t][kg];
          if constexpr (ZEROS) acc[t] *= s_off[w][n * kScaleStride + p * kGroups + g];
        }
#pragma unroll
        for (int jj = 0; jj < J; ++jj) {
          const int j = g * J + jj;
          const bf16x8 f = factors(q[j], pattern);
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[p][j][t], f, acc[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[t][e] += sc * acc[t][e];
        }
      }
      // one step's LDS reads at a time: more in flight spill registers
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) s_part[buf][w][t][lane] = y[t];
    __syncthreads();
    for (int i = tid; i < TG * MT * 256; i += NW * 64) {
      const int q = i / (MT * 256), t = (i >> 8) % MT;
      const int m = (i >> 4) & 15, col = i & 15;
      const int v = (batch * TG + q) * 16 + col, b = row0 + t * 16 + m;
      if (v < a.V && b < a.B) {
        float sum = 0.0f;
        for (int k = 0; k < KS; ++k) sum += s_part[buf][q * KS + k][t][(m >> 2) * 16 + col][m & 3];
        store_logit(a, b, v, sum);
      }
    }
    buf ^= 1;
  }
}

template <int NW, int P, int MT, int G, int SD, bool ZEROS>
hipError_t launch_split(const Args& a, int steps, int ks_log2, hipStream_t st) {
  const int tiles = (a.V + 15) / 16;
  const int tg = NW >> ks_log2;
  const int full = 256 * occupancy(P, MT) * 4 / NW;  // workgroups that the chip holds
  const int grid = min(full, (tiles + tg - 1) / tg);
  const int blocks = (a.B + MT * 16 - 1) / (MT * 16);
  hipLaunchKernelGGL((head_split_kernel<NW, P, MT, G, SD, ZEROS>),
                     dim3((unsigned)grid, (unsigned)blocks), dim3(NW * 64), 0, st, a, steps,
                     tiles, ks_log2);
  return hipGetLastError();
}

template <int MT, int G, int SD, bool ZEROS>
hipError_t pick_steps(const Args& a, hipStream_t st) {
  const int steps = (a.K + kStepK - 1) / kStepK;
  // 16 waves where 8 slices would hold more than 4 steps each
  if constexpr (MT == 1) {
    if (steps > 32) return launch_split<16, 4, MT, G, SD, ZEROS>(a, steps, 4, st);
  }
  // the fewest slices that leave a wave at most 4 steps
  int ks_log2 = 0;
  while (ks_log2 < 3 && (steps + (1 << ks_log2) - 1) >> ks_log2 > 4) ++ks_log2;
  // few tiles: more slices of each, so that more workgroups share them (2
  // rows, 10000 x 2048: 8.7 us against 12.8 without; 1 row, 32000 x 2048, past
  // the rule's reach: 12.5 us)
  const int tiles = (a.V + 15) / 16;
  while (ks_log2 < 3 && (steps >> ks_log2) > 1 && tiles < (512 << (3 - ks_log2))) ++ks_log2;
  const int per = (steps + (1 << ks_log2) - 1) >> ks_log2;
  if (per <= 1) return launch_split<8, 1, MT, G, SD, ZEROS>(a, steps, ks_log2, st);
  if (per == 2) return launch_split<8, 2, MT, G, SD, ZEROS>(a, steps, ks_log2, st);
  return launch_split<8, 4, MT, G, SD, ZEROS>(a, steps, ks_log2, st);
}

// ---------------------------------------------------------------------------

constexpr int kChunkK = 2 * kStepK;      // columns per chunk: 128 bytes of codes a row
constexpr int kMaxRows = 64;             // hidden rows per workgroup
constexpr int kMaxTiles = 5;             // tiles a wave holds at once

// More hidden rows, or rows too long for the registers: x passes through LDS in
// steps of 128 columns (two steps a buffer where LDS has room; two buffers, one
// barrier each), already in the product's lane order, with the sums of its
// groups; every wave of the workgroup multiplies the same x with up to NT tiles
// of its own, whose sums stay in registers over all of k. x is read from L2 once
// per 8 NT tiles and from LDS once per NT, so NT is as large as the registers
// allow.
//
// What the weights' loads look like decides the rest. The workgroups of an XCD
// hold 8 NT * 16 rows each at a time, more cache lines than its L2, so a line
// read in pieces at different times comes from behind L2 each time: a row's
// codes are read 128 bytes at once (a chunk of 256 columns), its scales as many
// at a time as a lane can keep (4 lanes a row, 8 or 16 bytes each, for 2 to 8
// chunks). A chunk's codes are requested while the one before is multiplied, and
// pass through the wave's own LDS from lanes along a row to the product's.
//
// Measured: 64 rows, 151936 x 8192 in groups of 128, 235 us (680 TFLOP/s, 2.8
// TB/s; 288 with 3 tiles a wave and scales read per chunk); in groups of 32 with
// float32 scales, 287 us (317; the first calls after a pause up to 350); 48 rows,
// 100003 x 4096 in groups of 32 with zero points, 140 us (187). With all loads but
// the first taken out the products of
// the first two take 181 and 210 us (the factors and, at small groups, the
// scaling cost as many vector instructions as products); the loads alone 168 and
// 196. 8 waves a compute unit are all that the registers of 5 tiles by 64 rows
// allow, so the two overlap imperfectly. Fewer waves with more columns, or a
// chunk's columns split over the waves, were slower (355 and 328 us).
template <int MT, int NT, int G, bool ZEROS>
struct StreamLds {
  static constexpr int GC = kChunkK / G;           // groups per chunk
  // columns whose sum is scaled at once: half a group of 128 where the registers
  // of many tiles leave no room for more of x
  static constexpr int C = NT > 2 && G == 128 ? 64 : G;
  static constexpr int XS = NT > 3 ? 1 : 2;        // steps of x per buffer
  static constexpr int kCodeStride = kChunkK / 2 + 16;  // bytes per row
  static constexpr int kScaleStride = GC + 1;      // floats per row
  static constexpr int kZeroStride = GC < 4 ? 4 : GC + 4;  // bytes per row
  uint4 x[2][XS][4 * MT * 64];
  f32x4 sum[2][XS][kStepK / C][MT * 4];
  u32x4 code[8][NT][kCodeStride];                  // 16 rows each
  float scale[8][NT][16 * kScaleStride];
  uint8_t zero[ZEROS ? 8 : 1][ZEROS ? NT : 1][ZEROS ? 16 * kZeroStride : 1];
};

template <int MT, int NT, int G, int SD, bool ZEROS>
__global__ void __launch_bounds__(kThreads8, 2) head_stream_kernel(Args a, int chunks, int tiles) {
  using Lds = StreamLds<MT, NT, G, ZEROS>;
  __shared__ Lds lds;
  constexpr int GC = Lds::GC, XS = Lds::XS, C = Lds::C;
  constexpr int kCodeStride = Lds::kCodeStride, kScaleStride = Lds::kScaleStride;
  constexpr int kZeroStride = Lds::kZeroStride;
  constexpr int XI = (MT + 1) / 2;         // 16-byte items of x per thread and step
  constexpr int kScaleSize = SD == QS_F32 ? 4 : 2;
  constexpr int EL = (G == 32 ? 16 : 8) / kScaleSize;  // scales per lane: 4 lanes a row
  constexpr int R = 4 * EL / GC;           // chunks that a block of scales lasts
  constexpr int SW = EL * kScaleSize / 4, ZW = (EL + 3) / 4;  // their registers
  using Raw = std::conditional_t<SD == QS_F32, uint32_t, uint16_t>;
  const int tid = threadIdx.x;
  const int w = uni(tid >> 6);
  const int lane = lane_id();
  const int n = lane & 15, kg = lane >> 4;
  const int row0 = (int)blockIdx.y * kMaxRows;
  const int rows_x = min(a.B - row0, MT * 16);

  // x: 16 lanes along a row's step, 32 rows at a time
  const int xc = tid & 15, xm = tid >> 4;
  uint4 xv[XS][XI];
  auto load_x = [&](int step) {
#pragma unroll
    for (int s = 0; s < XS; ++s) {
      const int k = (step + s) * kStepK + xc * 8;
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int m = xm + 32 * i;
        xv[s][i] = make_uint4(0u, 0u, 0u, 0u);
        if (m < rows_x && k < a.K)
          xv[s][i] =
              *reinterpret_cast<const uint4*>(a.hidden + (size_t)(row0 + m) * a.hidden_stride + k);
      }
    }
  };
  // where item c (8 columns) of a step goes: product j, lane group g; within the
  // product's 64 places rows are turned by 4 g + j, so that neither these writes
  // nor the reads meet in a bank
  const int xj = C == 128 ? xc & 3 : C == 64 ? (xc >> 3) * 2 + (xc & 1) : xc >> 2;
  const int xg = C == 128 ? xc >> 2 : C == 64 ? (xc >> 1) & 3 : xc & 3;
  auto place = [](int j, int t, int g, int m) {
    return (j * MT + t) * 64 + g * 16 + ((m + 4 * g + j) & 15);
  };
  auto store_x = [&](int buf) {
#pragma unroll
    for (int s = 0; s < XS; ++s) {
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int m = xm + 32 * i;
        const uint32_t q[4] = {xv[s][i].x, xv[s][i].y, xv[s][i].z, xv[s][i].w};
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum += __uint_as_float(q[e] << 16) + __uint_as_float(q[e] & 0xFFFF0000u);
        sum += __uint_as_float(dpp_u32<kDppXor1>(__float_as_uint(sum)));
        sum += __uint_as_float(dpp_u32<kDppXor2>(__float_as_uint(sum)));
        if constexpr (C >= 64)
          sum += __uint_as_float(dpp_u32<kDppHalfMirror>(__float_as_uint(sum)));
        if constexpr (C == 128) sum += __uint_as_float(dpp_u32<kDppMirror>(__float_as_uint(sum)));
        if (MT > 1 || m < 16) {
          lds.x[buf][s][place(xj, m >> 4, xg, m & 15)] = ordered(xv[s][i]);
          if ((xc & (C / 8 - 1)) == 0)
            reinterpret_cast<float*>(lds.sum[buf][s][xc / (C / 8)])[m] =
                ZEROS ? sum : -24.0f * sum;
        }
      }
    }
  };

  // codes: 8 lanes along the 128 bytes of a row, 8 rows a load; scales and zero
  // points: 4 lanes a row
  const int c_row = lane >> 3, c_part = lane & 7;
  const int g_row = lane >> 2, g_part = (lane & 3) * EL;
  const Pattern pattern;
  int first = 0;
  u32x4 code[NT][2];
  uint32_t scale[NT][SW];
  uint32_t zero[NT][ZW];
  // past the last tile: the last row again, never stored
  auto load_codes = [&](int chunk) {
    // past the row's end: its last bytes again, against hidden values of 0
    const uint32_t col = (uint32_t)min(chunk * (kChunkK / 2) + c_part * 16, a.K / 2 - 16);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int v0 = min((first + i) * 16, a.V - 1), rows = min(15, a.V - 1 - v0);
      const uint8_t* const pc = a.codes + (size_t)v0 * a.codes_stride;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at =
            (uint32_t)min(h * 8 + c_row, rows) * (uint32_t)a.codes_stride + col;
        code[i][h] = *reinterpret_cast<const u32x4*>(pc + at);
      }
    }
  };
  int g_first = 0;  // the first group a lane holds
  auto load_scales = [&](int chunk) {
    const int groups = a.K / G;
    g_first = max(min(chunk * GC + g_part, groups - EL), 0);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int v0 = min((first + i) * 16, a.V - 1), rows = min(15, a.V - 1 - v0);
      const uint8_t* const ps =
          static_cast<const uint8_t*>(a.scales) + (size_t)v0 * a.scale_stride * kScaleSize;
      const uint32_t row = (uint32_t)min(g_row, rows);
      const uint32_t at = (row * (uint32_t)a.scale_stride + (uint32_t)g_first) * kScaleSize;
      const uint8_t* const pz = ZEROS ? a.zeros + (size_t)v0 * a.zero_stride : nullptr;
      const uint32_t zat = row * (uint32_t)a.zero_stride + (uint32_t)g_first;
      if (groups >= EL) {
        __builtin_memcpy(scale[i], ps + at, 4 * SW);
        if constexpr (ZEROS && EL == 2) {
          uint16_t z;
          __builtin_memcpy(&z, pz + zat, 2);
          zero[i][0] = z;
        } else if constexpr (ZEROS) {
          __builtin_memcpy(zero[i], pz + zat, EL);
        }
      } else {  // fewer groups than a lane holds: the last one again
#pragma unroll
        for (int k = 0; k < SW; ++k) scale[i][k] = 0u;
#pragma unroll
        for (int k = 0; k < ZW; ++k) zero[i][k] = 0u;
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          const int k = min(e, groups - 1);
          const uint32_t sc = *reinterpret_cast<const Raw*>(ps + k * kScaleSize + at);
          scale[i][e * kScaleSize / 4] |= SD == QS_F32 ? sc : sc << (16 * (e & 1));
          if constexpr (ZEROS) zero[i][e / 4] |= (uint32_t)*(pz + k + zat) << (8 * (e & 3));
        }
      }
    }
  };

  for (int base = (int)blockIdx.x * 8 * NT; base < tiles; base += (int)gridDim.x * 8 * NT) {
    first = base + w * NT;
    f32x4 y[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int t = 0; t < MT; ++t) y[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    load_x(0);
    load_scales(0);
    load_codes(0);
    __syncthreads();  // the round before has read its last step
    store_x(0);
    load_x(XS);
    for (int chunk = 0; chunk < chunks; ++chunk) {
      // this chunk's codes, scales and zero points through LDS: from lanes along a
      // row to the product's
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        uint8_t* const turn = reinterpret_cast<uint8_t*>(lds.code[w][i]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<u32x4*>(turn + (h * 8 + c_row) * kCodeStride + c_part * 16) =
              code[i][h];
      }
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        // groups of other chunks go to the row's spare place
        const uint32_t part = min((uint32_t)(g_first + e - chunk * GC), (uint32_t)GC);
        const uint32_t to = (uint32_t)g_row * kScaleStride + part;
        const uint32_t zto = (uint32_t)g_row * kZeroStride + part;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          uint32_t sc = scale[i][e * kScaleSize / 4];
          if constexpr (SD != QS_F32) sc = (e & 1) ? sc & 0xFFFF0000u : sc << 16;
          lds.scale[w][i][to] = __uint_as_float(sc);
          if constexpr (ZEROS) lds.zero[w][i][zto] = (uint8_t)(zero[i][e / 4] >> (8 * (e & 3)));
        }
      }
      const int left = a.K / G - chunk * GC;  // groups of the row's last chunk
      if (left < GC) {
        // a scale of 0 behind them: what LDS held could be an infinity, which would
        // make a NaN of the hidden values' 0
        int at = n * kScaleStride + left + kg;
        asm volatile("" : "+v"(at));  // worked out here, not kept over the loop
        for (int g = left + kg; g < GC; g += 4, at += 4) {
#pragma unroll
          for (int i = 0; i < NT; ++i) lds.scale[w][i][at] = 0.0f;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      load_codes(chunk + 1);
      if ((chunk + 1) % R == 0) load_scales(chunk + 1);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int buf = XS == 1 ? p : chunk & 1;
        if (p % XS == 0) {
          __syncthreads();  // x of this step is in place, the other buffer is free
          store_x(buf ^ 1);
          load_x(chunk * 2 + p + 2 * XS);
          __builtin_amdgcn_sched_barrier(0);
        }
        constexpr int J = C / 32;
        // a tile's codes of a group, its scale and its offset, one tile ahead
        uint32_t q[2][J];
        float sc[2], off[2];
        auto read = [&](int at, int g, int i) {
          const uint8_t* const row =
              reinterpret_cast<const uint8_t*>(lds.code[w][i]) + n * kCodeStride + p * 64;
          if constexpr (C == 128) {
            *reinterpret_cast<u32x4*>(q[at]) = *reinterpret_cast<const u32x4*>(row + kg * 16);
          } else if constexpr (C == 64) {
            *reinterpret_cast<uint2*>(q[at]) =
                *reinterpret_cast<const uint2*>(row + g * 32 + kg * 8);
          } else {
            q[at][0] = *reinterpret_cast<const uint32_t*>(row + g * 16 + kg * 4);
          }
          sc[at] = lds.scale[w][i][n * kScaleStride + (p * kStepK + g * C) / G];
          if constexpr (ZEROS)
            off[at] = -16.0f - (float)lds.zero[w][i][n * kZeroStride + (p * kStepK + g * C) / G];
        };
        read(0, 0, 0);
#pragma unroll
        for (int g = 0; g < kStepK / C; ++g) {
          bf16x8 x[J][MT];
          f32x4 sum[MT];
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            sum[t] = lds.sum[buf][p % XS][g][t * 4 + kg];
#pragma unroll
            for (int jj = 0; jj < J; ++jj)
              x[jj][t] =
                  __builtin_bit_cast(bf16x8, lds.x[buf][p % XS][place(g * J + jj, t, kg, n)]);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const int at = (g * NT + i) & 1;
            if (i + 1 < NT) read(at ^ 1, g, i + 1);
            else if (g + 1 < kStepK / C) read(at ^ 1, g + 1, 0);
            f32x4 acc[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              acc[t] = sum[t];
              if constexpr (ZEROS) acc[t] *= off[at];
            }
#pragma unroll
            for (int jj = 0; jj < J; ++jj) {
              const bf16x8 f = factors(q[at][jj], pattern);
#pragma unroll
              for (int t = 0; t < MT; ++t)
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[jj][t], f, acc[t], 0, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
#pragma unroll
              for (int e = 0; e < 4; ++e) y[i][t][e] += sc[at] * acc[t][e];
              asm volatile("" : "+v"(y[i][t]));  // added here, not when all products are done
            }
            if (MT * NT > 6) __builtin_amdgcn_sched_barrier(0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    int m0 = kg * 4;
    asm volatile("" : "+v"(m0));  // the rows' addresses are not kept over the loop
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = t * 16 + m0 + e;
        if (m < rows_x) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const int v = (first + i) * 16 + n;
            if (v < a.V) store_logit(a, row0 + m, v, y[i][t][e]);
          }
        }
      }
    }
  }
}

template <int MT, int G, int SD, bool ZEROS>
hipError_t launch_stream(const Args& a, hipStream_t st) {
  const int chunks = (a.K + kChunkK - 1) / kChunkK;
  const int tiles = (a.V + 15) / 16;
  const int blocks = (a.B + kMaxRows - 1) / kMaxRows;
  // tiles per wave: the fewest rounds of (at most) one workgroup per compute
  // unit, a round taking as long as its tiles and one more
  int nt = 1;
  auto rounds = [&](int t) { return (tiles + 256 * 8 * t - 1) / (256 * 8 * t); };
  for (int t = 2; t <= kMaxTiles; ++t)
    if (rounds(t) * (t + 1) < rounds(nt) * (nt + 1)) nt = t;
  const int grid = min(256, (tiles + 8 * nt - 1) / (8 * nt));
  auto run = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid, (unsigned)blocks), dim3(kThreads8), 0, st, a,
                       chunks, tiles);
    return hipGetLastError();
  };
  if (nt == 1) return run(head_stream_kernel<MT, 1, G, SD, ZEROS>);
  if (nt == 2) return run(head_stream_kernel<MT, 2, G, SD, ZEROS>);
  if (nt == 3) return run(head_stream_kernel<MT, 3, G, SD, ZEROS>);
  if (nt == 4) return run(head_stream_kernel<MT, 4, G, SD, ZEROS>);
  return run(head_stream_kernel<MT, 5, G, SD, ZEROS>);
}

template <int G, int SD, bool ZEROS>
hipError_t pick(const Args& a, hipStream_t st) {
  // Up to 16 rows: in registers, but for 6 rows and more where a wave of the
  // streaming kernel has one to three tiles and nearly all waves have one. There
  // the registers' way pays for x, read by every workgroup, over few tiles (16
  // rows, 65000 x 4096: 42 us against 33.5; 8 rows, 32000 x 2048: 15.8 against 12.1;
  // beside it 4 rows, 56000 x 4096: 28.3 against 29.0, 16 rows, 128256 x 4096 in
  // groups of 64: 79 against 83, 8 rows, 17000 x 4096: 16.2 against 19.1).
  // Past 4096 columns 16 slices of 4 steps have to be full (4 rows, 128256 x 8192:
  // 101 us against 134; x 6144, 48 steps: 91 against 95; x 5120: 90 against 84), and
  // in groups of 32 with zero points their scales and offsets outgrow the
  // registers (196 against 182).
  const int tiles = (a.V + 15) / 16, steps = (a.K + kStepK - 1) / kStepK;
  const bool few = a.B < 6 || tiles < 1280 || tiles > 3 * 2048;
  const bool full = steps > 48 || (few && steps > 40);
  const bool slices = steps <= 32 ? few : tiles < 1280 || (full && !(G == 32 && ZEROS));
  if (a.B <= 16 && a.K <= 8192 && slices) return pick_steps<1, G, SD, ZEROS>(a, st);
  if (a.B <= 16) return launch_stream<1, G, SD, ZEROS>(a, st);
  // More rows of small vocabularies: 16 at a time in registers, so that the blocks
  // of rows and the slices of k fill the chip (64 rows, 1000 x 8192: 16 us against
  // 63; 40 rows, 8000 x 8192: 53 against 78; 64 rows, 4000 x 8192: 57 against 63, of
  // 8000: 68 against 64; 24 rows, 2000 x 4096: 9 against 12, of 4000: 13 either way).
  const int blocks = (a.B + 15) / 16;
  const int most = a.B <= 32 && a.K <= 4096 ? 256 : 1536;
  if (a.B <= 64 && a.K <= 8192 && tiles * blocks <= most)
    return pick_steps<1, G, SD, ZEROS>(a, st);
  // 17 to 32 rows: in registers up to 4096 columns where tiles are few and the
  // slices of k fill the chip (32 rows, 5000 x 4096: 17 us against 21; 20 rows,
  // 12000 x 2048: 14 against 16). Large vocabularies are a draw or worse (151936 x
  // 4096: 97 us either way; in groups of 32 with zero points 162 against 139).
  if (a.B <= 32 && a.K <= 4096 && a.V < 16384) return pick_steps<2, G, SD, ZEROS>(a, st);
  if (a.B <= 32) return launch_stream<2, G, SD, ZEROS>(a, st);
  return launch_stream<4, G, SD, ZEROS>(a, st);
}

template <int G, int SD>
hipError_t pick_zeros(const Args& a, hipStream_t st) {
  return a.zeros ? pick<G, SD, true>(a, st) : pick<G, SD, false>(a, st);
}
template <int G>
hipError_t pick_scale(const Args& a, hipStream_t st) {
  return a.scale_dtype == QS_F32 ? pick_zeros<G, QS_F32>(a, st) : pick_zeros<G, QS_BF16>(a, st);
}

}  // namespace
}  // namespace head
}  // namespace qs
