// Low-rank adapters of many requests beside a shared output projection: with a the
// adapter of row b,
//   y[b][v] = z[b][v] + sum_r up[a][v][r] u[b][r],
//   u[b][r] = scale[a] sum_k down[a][r][k] x[b][k].
// Two launches: the rows' low-rank coordinates u, then their product with the up factors
// on top of the logits. Up to 64 rows read each used up factor once, wherever they stand;
// more are taken in the order of their adapters (4096 to an order), 64 at a time, and each
// 64 read the up factors of theirs once. Down factors are read for every row, from the L2
// where rows share them. What bounds the calls is reading the up factors, and the logits
// read and written.
//
// The second product runs on the matrix cores (16x16x32) with the factor's rows on one
// side and 16 rows of the batch on the other. A product's column depends on its own
// batch row alone, so an adapter is multiplied with all 16 and taken by the rows that
// are its own; what another row holds (an infinity, uninitialised scratch) cannot reach
// a result. The first launch also puts the rows in the order of their adapters, so that
// an adapter meets few blocks of 64 rows (512 rows of 151936 on 64 adapters of rank 16:
// 147 us against 498 with an order in each block alone; 320 rows 125 against 313; on 8 of
// them, whose factors the L2 held either way, 512 rows 121 against 111) and few tiles of 16
// (64 rows of 151936 bf16 on 8 adapters in turn, of rank 16 20.0 us against 26.7 in the
// batch's own order, of rank 8 17.7 against 26.4; on 16 of rank 32, fp32, 40 against 47).
// The coordinates are float32; each is cut into three bf16 numbers of 8 bits, whose sum is
// it (from 2^-110 up; below that bf16's least number, 2^-133, bounds what is left), so that
// products are exact: three products cost nothing beside the factors' bytes
// (one rounded to bf16 would cost the result 2^-8 of the adapter's share). Sums are held in
// float32, and each logit is rounded once.
//
// Measured (first and second launch): 64 rows of 151936 bf16 on adapters of their own of
// rank 32, 8192 columns, 10.5 and 116 us (5.7 TB/s in the second, where a large copy
// reaches 5.2); on three of rank 64, 4096 columns, 5.8 and 18.3 us (5.3 TB/s); 16 rows of
// 128256 fp32, each its own of rank 32, 4.0 and 22.6 us (6.4 TB/s); 1 row of 151936, rank
// 16, 3.4 and 3.8 us, two dependent loads each. Both together, 151936 bf16, 2048 columns:
// 512 rows on 8 and 64 adapters of rank 16 102 and 135 us, 2048 rows on one and 64 of them
// 295 and 361 (4.3 and 4.4 TB/s), on 4 of rank 64 434 (3.1 TB/s: the products and the
// coordinates' way to them).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/qs.h"
#include "qs_adapters.hpp"
#include "qs_device.hpp"

namespace qs {
namespace adapters {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 64;         // batch rows of a block
constexpr int kNone = 0x1FFF;     // in place of an adapter's number
constexpr int kRowBits = 18;      // of a row's number beside an adapter's
static_assert(kMaxB <= 1 << kRowBits && kNone < 1 << (31 - kRowBits), "in 31 bits");
constexpr int kTerms = 3;         // bf16 numbers per coordinate
constexpr int kUpWaves = 4;
constexpr int kTiles = 2;         // tiles of 16 vocabulary rows per wave
constexpr int kWavesWanted = 4096;  // up to which a block's adapters are dealt out
constexpr int kManyCoordinates = 4096;  // from which a wave of the first product takes two
constexpr int kAhead = 8;         // loads of 512 columns that a wave of the first product
                                  // requests at a time

// The workspace holds, per tile of 16 batch rows, the coordinates as the second
// product's operands: lane (row n, group g) of an operand has 8 bf16 numbers at 16 g + n.
// Past rank 16 there are kTerms operands per step of 32 ranks, one per term, group g
// with ranks 8 g to 8 g + 7. Shorter ranks leave groups free: of rank 16 the first
// operand holds the first two terms, the second the third; of rank 8 one holds all.
constexpr int kOperandBytes = 64 * 16;
int operands_of(int64_t rank) {
  return rank <= 8 ? 1 : rank <= 16 ? 2 : (int)((rank + 31) / 32) * kTerms;
}
// Coordinates per row, with the zeros behind the last.
int places_of(int64_t rank) {
  return rank <= 16 ? (int)rank : (int)((rank + 31) / 32) * 32;
}

// Behind them, for a batch of at most kRows rows, its plan: the rows in the order of
// their adapters (first come, first), those without one last, and the adapters (found
// again by every workgroup of the second launch, as for more rows, 0.3 to 0.6 us more).
struct Plan {
  int32_t row[kRows];      // the row's place in the block | its adapter's number << 16
                           // (kNone without one); -1 behind the last
  int32_t adapter[kRows];  // the adapters
  int32_t span[kRows];     // their first row | the one behind their last << 16; 0: no more
};

__device__ __forceinline__ void write_plan(const Args& a, Plan* plan) {
  const int lane = lane_id(), rows = a.B;
  const int asked = lane < rows ? a.index[lane] : -1;
  const bool adapted = asked >= 0 && asked < a.count;
  const int mine = adapted ? asked : -1;
  if (lane < rows) a.status[lane] = adapted || asked == -1 ? QS_ROW_OK : QS_ROW_BAD_PARAM;
  // the rows that share this lane's adapter: every row's is compared with every other's,
  // without a chain from one to the next (a walk from adapter to adapter took 6 us for 64)
  uint32_t same[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < kRows; ++j)
    same[j >> 5] |= mine == (int)readlane_u32((uint32_t)mine, j) ? 1u << (j & 31) : 0u;
  const uint64_t members = (uint64_t)same[1] << 32 | same[0], below = (1ull << lane) - 1ull;
  const int leader = __builtin_ctzll(members), size = __popcll(members);
  const bool leads = adapted && leader == lane;
  const uint64_t leaders = ballot(leads);
  const int adapters = __popcll(leaders), number = __popcll(leaders & below);
  const int end = (int)scan_incl_u32(leads ? (uint32_t)size : 0u), first = end - size;
  const int total = __popcll(ballot(adapted));
  const uint64_t none = ballot(!adapted && lane < rows);
  const int my_number = __shfl(number, leader, 64), my_first = __shfl(first, leader, 64);
  const int at = adapted ? my_first + __popcll(members & below)
                 : lane < rows ? total + __popcll(none & below) : lane;
  plan->row[at] = lane < rows ? lane | (adapted ? my_number : kNone) << 16 : -1;
  if (leads) {
    plan->adapter[number] = mine;
    plan->span[number] = first | end << 16;
  }
  if (lane >= adapters) {
    plan->adapter[lane] = -1;
    plan->span[lane] = 0;
  }
}

// For more rows the order of all of them by adapter, those without one last (of more than
// kOrdered rows each so many in an order of their own).
struct Place {
  int32_t row, adapter;  // adapter -1: none, or none that exists
};
constexpr int kOrdered = 4096;

// 64 rows' places: every row's key is compared with every other's; the four waves of a
// workgroup share the keys.
__device__ __forceinline__ void place_rows(const Args& a, int row0, Place* order) {
  __shared__ uint32_t s_count[256];
  const int lane = lane_id(), w = uni((int)(threadIdx.x >> 6));
  const int segment = row0 & ~(kOrdered - 1), end = min(segment + kOrdered, a.B);
  auto key_of = [&](int r, int n) {  // behind the last row: behind every key
    return r >= end ? 0xFFFFFFFFu : n >= 0 && n < a.count ? (uint32_t)n : 0x80000000u;
  };
  const int r = row0 + lane, asked = r < end ? a.index[r] : -1;
  const uint32_t mine = key_of(r, asked);
  uint32_t count = 0u;
  for (int j0 = segment + w * 64; j0 < end; j0 += 256) {
    const uint32_t keys = key_of(j0 + lane, j0 + lane < end ? a.index[j0 + lane] : -1);
    // among equals the row that comes first
    const uint32_t than = j0 < row0 ? mine + 1u : mine;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      const uint32_t k = readlane_u32(keys, j);
      count += k < than || (j0 == row0 && k == mine && j < lane) ? 1u : 0u;
    }
  }
  s_count[threadIdx.x] = count;
  __syncthreads();
  if (w != 0 || r >= end) return;
  for (int k = 1; k < 4; ++k) count += s_count[k * 64 + lane];
  a.status[r] = asked == -1 || mine != 0x80000000u ? QS_ROW_OK : QS_ROW_BAD_PARAM;
  order[segment + (int)count] = Place{r, mine == 0x80000000u ? -1 : asked};
}

// The sum over 16 neighbouring lanes, in each of them.
__device__ __forceinline__ float sum_of_16(float v) {
  auto add = [&](uint32_t other) { v += __uint_as_float(other); };
  add(dpp_u32<kDppXor1>(__float_as_uint(v)));
  add(dpp_u32<kDppXor2>(__float_as_uint(v)));
  add(dpp_u32<kDppHalfMirror>(__float_as_uint(v)));
  add(dpp_u32<kDppMirror>(__float_as_uint(v)));
  return v;
}

// The rows' coordinates, a wave to each row and rank or few ranks: few rows spread over as
// many compute units as they have ranks, each wave requests up to 8 KiB of the factor before
// it uses any, and rows that share an adapter read it from the L2. (On the matrix cores,
// 16 ranks and the rows that share an adapter to a workgroup: 1 row of 4096 columns, rank
// 16, 6.5 us, one compute unit's loads, against 3.5; 64 rows of 8192 on adapters of their
// own, rank 32, 14.2 against 10.7; 64 on 3 of rank 64, 4096 columns, 7.9 against 6.1.)
// A wave with R ranks reads the hidden state once for them. That leaves fewer waves to
// wait for memory, but from 4096 coordinates on the L2's rate bounds the kernel: both
// launches for 1000 tokens, 4096 columns, on 3 shared adapters, 64 rows of rank 32 7.6 us
// with one rank a wave, 7.8 with two, 8.5 with four; of rank 64 9.2, 8.7 and 9.3; of rank
// 128 12.2, 11.0 and 11.3; on 64 adapters of rank 32, 8192 columns, 13.5, 13.8 and 15.5.
// Past 64 rows four: 2048 rows of 151936 tokens, 2048 columns, on 4 adapters of rank 64 502
// us with one, 468 with two, 459 with four, 457 with eight.
template <bool WIDE, int R>
__global__ void __launch_bounds__(256)
    down_kernel(Args a, int places, int operands, int blocks, void* order) {
  const int lane = lane_id();
  if ((int)blockIdx.x < blocks) {  // the first workgroups put the rows in order
    if constexpr (WIDE) place_rows(a, (int)blockIdx.x * 64, static_cast<Place*>(order));
    else if (threadIdx.x < 64) write_plan(a, static_cast<Plan*>(order));
    return;
  }
  constexpr int kLoads = kAhead / R;
  const int item =
      uni((int)((blockIdx.x - blocks) * (blockDim.x >> 6) + (threadIdx.x >> 6)));
  const int b = item / (places / R), q0 = (item - b * (places / R)) * R;
  if (b >= a.B) return;
  const int n = a.index[b];
  if (n < 0 || n >= a.count) return;
  float u = 0.0f;
  int q = q0;  // the rank that u is of
  if (q0 < a.rank) {
    const float scale = a.scale ? a.scale[n] : 1.0f;
    const uint16_t* const x = a.hidden + (size_t)b * a.hidden_stride;
    const uint16_t* const d =
        a.down + (size_t)n * a.down_stride + (size_t)q0 * a.down_row_stride;
    float sum[R][2];
#pragma unroll
    for (int i = 0; i < R; ++i) sum[i][0] = sum[i][1] = 0.0f;
    for (int k0 = lane * 8; k0 < a.K; k0 += kLoads * 512) {
      uint4 dv[R][kLoads], xv[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        xv[j] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < R; ++i) dv[i][j] = make_uint4(0u, 0u, 0u, 0u);
        if (k0 + j * 512 < a.K) {
#pragma unroll
          for (int i = 0; i < R; ++i)
            dv[i][j] = *reinterpret_cast<const uint4*>(d + (size_t)i * a.down_row_stride + k0 +
                                                       j * 512);
          xv[j] = *reinterpret_cast<const uint4*>(x + k0 + j * 512);
        }
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const uint32_t xs[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const uint32_t ds[4] = {dv[i][j].x, dv[i][j].y, dv[i][j].z, dv[i][j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum[i][0] = fmaf(__uint_as_float(ds[e] << 16), __uint_as_float(xs[e] << 16), sum[i][0]);
            sum[i][1] = fmaf(__uint_as_float(ds[e] & 0xFFFF0000u),
                             __uint_as_float(xs[e] & 0xFFFF0000u), sum[i][1]);
          }
        }
      }
    }
    float v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = sum[i][0] + sum[i][1];
    // summed over the lanes, of several ranks each half of the lanes going on with half of
    // them; the same pairs for any R, so a row's bits are the same in any batch
    int off = 32;
#pragma unroll
    for (int left = R / 2; left > 0; left >>= 1, off >>= 1) {
      const bool upper = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < left; ++i) {
        const float other = __shfl_xor(upper ? v[i] : v[i + left], off, 64);
        v[i] = (upper ? v[i + left] : v[i]) + other;
      }
      q += upper ? left : 0;
    }
    u = v[0];
#pragma unroll
    for (int o = 32 / R; o >= 16; o >>= 1) u += __shfl_xor(u, o, 64);
    u = sum_of_16(u) * scale;
  } else {
    q += lane / (64 / R);
  }
  if ((lane & (64 / R - 1)) != 0) return;
  uint8_t* const out =
      a.low + (size_t)(b / 16) * operands * kOperandBytes + (b & 15) * 16 + (q & 7) * 2;
  // the group (of all operands' groups) that holds the coordinate's term k
  const int g = q >> 3;
#pragma unroll
  for (int k = 0; k < kTerms; ++k) {
    const int to = operands == 1 ? k
                   : operands == 2 ? 2 * k + g
                                   : (g >> 2) * 4 * kTerms + 4 * k + (g & 3);
    // the upper half of the bits: rounded it could pass the largest number
    const uint32_t part = __float_as_uint(u) & 0xFFFF0000u;
    *reinterpret_cast<uint16_t*>(out + to * 256) = (uint16_t)(part >> 16);
    // an infinity's (or NaN's) other terms are 0, so that its products are the formula's
    u = fabsf(u) < INFINITY ? u - __uint_as_float(part) : 0.0f;
  }
  // the groups that short ranks leave free
  if (operands <= 2) *reinterpret_cast<uint16_t*>(out + (operands == 1 ? 3 : 6 + g) * 256) = 0;
}

// The logits. A wave takes kTiles tiles of 16 vocabulary rows and up to RT tiles of 16
// batch rows: the logits are its accumulators, and it walks the block's adapters, A at a
// time (2 where their rows are so short, up to rank 16, that one's are too few bytes under
// way: 64 rows of 151936 on adapters of rank 16 of their own 70 us, 77 with one at a time,
// 86 with four; of rank 32 126 with one, 131 with two). Two tiles leave room for more
// waves than four (64 rows on 16 adapters of rank 128: 147 us against 172; on 4 of rank
// 16, fp32, 24.5 against 33). The tiles' rows are dealt out so that a lane holds 4 kTiles
// consecutive logits of one batch row: product row 4 g + e of tile t is vocabulary row
// 4 (kTiles g + t) + e.
//
// A wave that walks many adapters waits for each one's factors, so where the vocabulary
// makes few waves a block's adapters are dealt out to up to 64 groups of workgroups, each
// with the rows of its own (64 rows on adapters of their own of rank 16: 1000 tokens 7.1
// us against 26.6 in one group, 8000 10.1 against 32, 32000 18.8 against 34, 64000 28.4
// against 37). Past kWavesWanted that costs more than it gives (64000 tokens in four
// groups 30.6, 128256 in two 57.0 against 55.7).
//
// A workgroup requests the coordinates, and then its logits, all at once: one after
// another, as a loop over them came out, they were a chain of up to 12 loads (64 rows on 3
// adapters of rank 64: 24.9 us against 23.4 for both launches; on 64 of rank 16, 128256
// tokens, 55.5 against 52.9).
template <int DT, int KS, int OPS, int RT, int A, bool WIDE>
__global__ void __launch_bounds__(kUpWaves * 64)
    up_kernel(Args a, int tiles, int turns, int groups_log2, const void* order) {
  constexpr int kSpan = 16 * kTiles;      // vocabulary rows per wave
  constexpr int P = DT == QS_F32 ? 4 : 8; // logits per 16 bytes
  constexpr int kLow = RT * OPS * 64, kParts = (kLow + kUpWaves * 64 - 1) / (kUpWaves * 64);
  __shared__ uint4 s_low[kLow];
  uint4 part_low[kParts];  // this thread's share of the coordinates on their way there
  const int tid = threadIdx.x, lane = lane_id(), w = uni(tid >> 6);
  const int n = lane & 15, kg = lane >> 4;
  const int part = (int)blockIdx.y;
  const int group = part & ((1 << groups_log2) - 1), row0 = (part >> groups_log2) * kRows;
  int tile = (int)blockIdx.x * turns * kUpWaves + w;
  const int rows = min(a.B - row0, kRows);
  const uint4* const low = reinterpret_cast<const uint4*>(a.low);
  const bool copies = group == 0 && a.out != a.logits;  // the rows without an adapter
  auto row_of = [](int mine) { return mine & ((1 << kRowBits) - 1); };
  auto of_group = [&](int number) { return (number & ((1 << groups_log2) - 1)) == group; };
  // the lane's place in the order: its row and its adapter's number in the block (-1: not
  // this workgroup's row, kNone: no adapter); the lane's adapter and the places it has
  int mine_row, mine_number, adapter, span, adapters;
  if constexpr (!WIDE) {
    const Plan* const plan = static_cast<const Plan*>(order);
    const int p = plan->row[lane];
    adapter = plan->adapter[lane];
    span = plan->span[lane];
    // the coordinates as they lie
    const int items = (rows + 15) / 16 * OPS * 64;
#pragma unroll
    for (int k = 0; k < kParts; ++k) part_low[k] = low[min(k * kUpWaves * 64 + tid, items - 1)];
    adapters = __popcll(ballot(span != 0));
    mine_row = p < 0 ? 0 : p & 0xFFFF;
    mine_number = p >> 16;
  } else {
    Place p{0, -1};
    if (lane < rows) p = static_cast<const Place*>(order)[row0 + lane];
    const int before = __shfl_up(p.adapter, 1, 64);
    const uint64_t starts = ballot(p.adapter >= 0 && (lane == 0 || before != p.adapter));
    const int number = __popcll(starts & (~0ull >> (63 - lane))) - 1;
    const int total = __popcll(ballot(p.adapter >= 0));
    adapters = __popcll(starts);
    mine_row = p.row;
    mine_number = lane >= rows ? -1 : p.adapter < 0 ? kNone : number;
    __shared__ int s_adapter[64], s_span[64];
    if (w == 0 && ((starts >> lane) & 1u)) {
      const uint64_t later = starts & (~1ull << lane);
      const int end = later != 0u ? __builtin_ctzll(later) : total;
      s_adapter[number] = p.adapter;
      s_span[number] = lane | end << 16;
    }
    __syncthreads();
    adapter = s_adapter[lane];
    span = s_span[lane];
  }
  if (mine_number == kNone ? !copies : !of_group(mine_number)) mine_number = -1;
  if constexpr (WIDE) {  // the coordinates from where they lie
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const int i = k * kUpWaves * 64 + tid, o = (i >> 6) % OPS;
      const int r = __shfl(mine_row, i / (OPS * 64) * 16 + (i & 15), 64);
      part_low[k] = low[((size_t)(r >> 4) * OPS + o) * 64 + (lane & 48) + (r & 15)];
    }
    static_assert(RT == 4, "whole turns");
  }

  // this lane's batch rows, in that order, and their logits
  int mine[RT], place[RT];  // row | adapter's number in the block << kRowBits
  f32x4 y[kTiles][RT];
  int v0, first;  // the tile's and the lane's first logit
  auto load_logits = [&](auto start) {
    v0 = tile * kSpan;
    first = v0 + kg * 4 * kTiles;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      if constexpr (start) {
        mine[t] = __shfl(mine_row | mine_number << kRowBits, t * 16 + n, 64);
        place[t] = WIDE ? t * OPS * 64 + lane  // of its coordinates
                        : (row_of(mine[t]) >> 4) * OPS * 64 + kg * 16 + (mine[t] & 15);
      } else {
        // worked out again in every turn: the rows' addresses held from one to the next
        // cost a wave of five
        asm volatile("" : "+v"(mine[t]));
      }
      // lanes without a row keep what their registers hold (never stored): a value of their
      // own would make the requests wait for one another
      u32x4 q[4 * kTiles / P];
#pragma unroll
      for (int c = 0; c < 4 * kTiles / P; ++c) q[c] = __builtin_nondeterministic_value(q[c]);
      if (mine[t] >= 0) {
        const uint8_t* const z = a.logits + (size_t)row_of(mine[t]) * a.row_bytes;
#pragma unroll
        for (int c = 0; c < 4 * kTiles / P; ++c) {
          const int v = first + c * P < a.V ? first + c * P : 0;
          q[c] = *reinterpret_cast<const u32x4*>(z + (size_t)v * (16 / P));
        }
      }
#pragma unroll
      for (int c = 0; c < 4 * kTiles / P; ++c) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const int i = c * P + e;
          if constexpr (DT == QS_F32) y[i >> 2][t][i & 3] = __uint_as_float(q[c][e]);
          else y[i >> 2][t][i & 3] =
              __uint_as_float((e & 1) ? q[c][e >> 1] & 0xFFFF0000u : q[c][e >> 1] << 16);
        }
      }
    }
  };
  load_logits(std::true_type{});
  // not earlier: this workgroup's loads would wait for the answer
  if (group >= adapters && !copies) return;
#pragma unroll
  for (int k = 0; k < kParts; ++k) {
    const int i = k * kUpWaves * 64 + tid;
    if (kLow % (kUpWaves * 64) == 0 || i < kLow) s_low[i] = part_low[k];
  }
  __syncthreads();
  for (;;) {
    if (tile >= tiles) return;
    for (int i0 = group; i0 < adapters; i0 += A << groups_log2) {
      int at[A], end[A];
      bf16x8 f[A][kTiles][KS];
#pragma unroll
      for (int j = 0; j < A; ++j) {
        const int i = i0 + (j << groups_log2);
        at[j] = end[j] = 0;
        if (i >= adapters) continue;
        const int where = (int)readlane_u32((uint32_t)span, i);
        at[j] = where & 0xFFFF;
        end[j] = where >> 16;
        const uint16_t* const up = a.up + (size_t)readlane_u32((uint32_t)adapter, i) * a.up_stride;
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
          const int v = min(v0 + (n >> 2) * 4 * kTiles + k * 4 + (n & 3), a.V - 1);
          const uint16_t* const r = up + (size_t)v * a.up_row_stride;
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            // groups beside the terms' or past the rank read others' ranks again: their
            // coordinates are 0
            const int at_rank = OPS == 1 ? 0 : OPS == 2 ? (kg & 1) * 8 : s * 32 + kg * 8;
            const uint4 q = *reinterpret_cast<const uint4*>(r + (at_rank < a.rank ? at_rank : 0));
            f[j][k][s] = __builtin_bit_cast(bf16x8, q);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < A; ++j) {
        const int i = i0 + (j << groups_log2);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          if (t * 16 >= end[j] || t * 16 + 16 <= at[j]) continue;
          f32x4 acc[kTiles];
#pragma unroll
          for (int k = 0; k < kTiles; ++k) acc[k] = y[k][t];
#pragma unroll
          for (int o = 0; o < OPS; ++o) {
            const bf16x8 u = __builtin_bit_cast(bf16x8, s_low[place[t] + o * 64]);
#pragma unroll
            for (int k = 0; k < kTiles; ++k)
              acc[k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  f[j][k][OPS <= 2 ? 0 : o / kTerms], u, acc[k], 0, 0, 0);
          }
          const bool take = mine[t] >> kRowBits == i;
#pragma unroll
          for (int k = 0; k < kTiles; ++k) {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[k][t][e] = take ? acc[k][e] : y[k][t][e];
          }
        }
      }
    }

#pragma unroll
    for (int t = 0; t < RT; ++t) {
      if (mine[t] < 0) continue;
      uint8_t* const out = a.out + (size_t)row_of(mine[t]) * a.out_bytes;
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
    if (!WIDE || --turns == 0) return;
    tile += kUpWaves;
    load_logits(std::false_type{});
  }
}

template <int DT, int KS, int OPS, int A>
void launch_up(const Args& a, const void* order, hipStream_t st) {
  const int tiles = (a.V + 16 * kTiles - 1) / (16 * kTiles);
  const int blocks = (a.B + kRows - 1) / kRows;
  int groups_log2 = 0;
  while (groups_log2 < 6 && 1 << groups_log2 < a.B &&
         (int64_t)tiles * blocks << (groups_log2 + 1) <= kWavesWanted)
    ++groups_log2;
  // Of many rows a workgroup takes several tiles per wave one after another, so that the
  // order and the coordinates (rank 64: 24 KiB for 16 KiB of bf16 logits) are fetched once
  // for them, as long as enough workgroups are left. (2048 rows of 151936 on 4 adapters of
  // rank 64, 38000 workgroups: 487 us with 1 tile, 459 with 2, 438 with 4; on 64 of rank 16
  // 421, 392, 396; 256 rows of 32000 on 8 of rank 128, 1000 workgroups, 40, 34, 35; 128 rows
  // of 151936 on 64 of rank 16, 2374 workgroups, 83, 87, 104.)
  int turns = 1;
  if (a.B > kRows) {
    const int64_t workgroups = (int64_t)((tiles + kUpWaves - 1) / kUpWaves) * blocks;
    if (a.rank > 32) turns = workgroups >= 4000 ? 4 : workgroups >= 1000 ? 2 : 1;
    else turns = workgroups >= 4000 ? 2 : 1;
  }
  const int each = kUpWaves * turns;
  const dim3 grid((unsigned)((tiles + each - 1) / each), (unsigned)blocks << groups_log2);
  const dim3 block(kUpWaves * 64);
  auto run = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, st, a, tiles, turns, groups_log2, order);
  };
  if (a.B <= 16) run(up_kernel<DT, KS, OPS, 1, A, false>);
  else if (a.B <= 32) run(up_kernel<DT, KS, OPS, 2, A, false>);
  else if (a.B <= kRows) run(up_kernel<DT, KS, OPS, 4, A, false>);
  else run(up_kernel<DT, KS, OPS, 4, A, true>);
}

template <int DT>
void launch_rank(const Args& a, const void* order, hipStream_t st) {
  if (a.rank <= 8) launch_up<DT, 1, 1, 2>(a, order, st);
  else if (a.rank <= 16) launch_up<DT, 1, 2, 2>(a, order, st);
  else if (a.rank <= 32) launch_up<DT, 1, kTerms, 1>(a, order, st);
  else if (a.rank <= 64) launch_up<DT, 2, 2 * kTerms, 1>(a, order, st);
  else if (a.rank <= 96) launch_up<DT, 3, 3 * kTerms, 1>(a, order, st);
  else launch_up<DT, 4, 4 * kTerms, 1>(a, order, st);
}

size_t low_bytes(int64_t B, int64_t rank) {
  return (size_t)((B + 15) / 16) * operands_of(rank) * kOperandBytes;
}

}  // namespace

size_t workspace_bytes(int64_t B, int64_t rank) {
  // a plan is larger than the order of 64 rows; sizes grow with B
  return low_bytes(B, rank) + sizeof(Plan) + (B > kRows ? (size_t)B * sizeof(Place) : 0);
}

bool grid_fits(int64_t B, int64_t V) {
  const int64_t parts = (V + 16 * kTiles * kUpWaves - 1) / (16 * kTiles * kUpWaves);
  return parts * ((B + kRows - 1) / kRows) * kUpWaves * 64 < (int64_t)1 << 32;
}

hipError_t launch_adapters(const Args& a, int dtype, hipStream_t st) {
  void* const order = a.low + low_bytes(a.B, a.rank);
  const int places = places_of(a.rank), blocks = (a.B + kRows - 1) / kRows;
  auto run = [&](auto* kernel, int ranks) {
    const int64_t items = (int64_t)a.B * places / ranks;
    // one wave a workgroup where that spreads few waves over more compute units
    const int waves = items > 1024 || a.B > kRows ? 4 : 1;
    const dim3 grid((unsigned)(blocks + (items + waves - 1) / waves)), block(waves * 64);
    hipLaunchKernelGGL(kernel, grid, block, 0, st, a, places, operands_of(a.rank), blocks, order);
  };
  if (a.B > kRows) run(down_kernel<true, 4>, 4);
  else if (a.B * a.rank >= kManyCoordinates) run(down_kernel<false, 2>, 2);
  else run(down_kernel<false, 1>, 1);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  if (dtype == QS_F32) launch_rank<QS_F32>(a, order, st);
  else launch_rank<QS_BF16>(a, order, st);
  return hipGetLastError();
}

}  // namespace adapters
}  // namespace qs
