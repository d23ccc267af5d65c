// Argument block and launcher of the output head with 4-bit weights.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qs {
namespace head {

constexpr int64_t kMaxB = (int64_t)1 << 20;  // 64 rows a block of the grid's y
constexpr int64_t kMaxV = (int64_t)1 << 24;
constexpr int64_t kMaxK = 65536;
// 15 rows of codes, scales (4 bytes) or zero points are reached with a lane's
// unsigned 32-bit offset from the first of 16
constexpr int64_t kMaxWeightStride = (int64_t)1 << 26;

struct Args {
  const uint16_t* hidden;    // [B][hidden_stride] bf16
  int64_t hidden_stride;
  int B;
  int V;
  int K;
  int group;                 // 32, 64 or 128; K is a multiple of it
  const uint8_t* codes;      // [V][codes_stride] bytes, two codes each
  int64_t codes_stride;
  const void* scales;        // [V][scale_stride] bf16 or fp32
  int scale_dtype;
  int64_t scale_stride;
  const uint8_t* zeros;      // [V][zero_stride], optional (NULL: 8)
  int64_t zero_stride;
  void* logits;              // [B][row_stride]
  int logits_dtype;
  int64_t row_stride;
};

// one translation unit per group size
hipError_t launch_g32(const Args& a, hipStream_t st);
hipError_t launch_g64(const Args& a, hipStream_t st);
hipError_t launch_g128(const Args& a, hipStream_t st);

inline hipError_t launch_head(const Args& a, hipStream_t st) {
  return a.group == 128 ? launch_g128(a, st) : a.group == 64 ? launch_g64(a, st) : launch_g32(a, st);
}

}  // namespace head
}  // namespace qs
