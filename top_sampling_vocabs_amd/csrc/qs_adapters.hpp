// Argument block and launchers of low-rank adapters beside the output projection.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qs {
namespace adapters {

constexpr int64_t kMaxB = (int64_t)1 << 18;  // a row's number stands beside its adapter's in 31 bits
constexpr int64_t kMaxV = (int64_t)1 << 24;
constexpr int64_t kMaxK = 65536;
constexpr int64_t kMaxRank = 128;

struct Args {
  const uint8_t* logits;     // [B][row_bytes]
  int64_t row_bytes;
  uint8_t* out;              // may be logits
  int64_t out_bytes;
  int B, V, K, rank;
  int64_t count;             // adapters held
  const uint16_t* hidden;    // [B][hidden_stride] bf16
  int64_t hidden_stride;
  const uint16_t* down;      // [count][rank][K] bf16
  int64_t down_stride, down_row_stride;
  const uint16_t* up;        // [count][V][rank] bf16
  int64_t up_stride, up_row_stride;
  const int32_t* index;      // [B]; -1: none
  const float* scale;        // [count], optional (NULL: 1)
  int32_t* status;           // [B]
  uint8_t* low;              // workspace: the rows' low-rank coordinates and order
};

size_t workspace_bytes(int64_t B, int64_t rank);
// whether one workgroup per tiles and block of rows fits one launch grid (batches past
// that, 2^37 logits, are larger than the memory)
bool grid_fits(int64_t B, int64_t V);
hipError_t launch_adapters(const Args& a, int dtype, hipStream_t st);

}  // namespace adapters
}  // namespace qs
