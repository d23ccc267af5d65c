// Argument blocks and launchers of the scoring kernels: log-probabilities of
// given tokens with entropy and top tokens, and their gradient.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qs {
namespace score {

constexpr int kTopMax = 64;       // top tokens per row
constexpr int kTokensMax = 1024;  // given tokens per row

struct Args {
  const uint8_t* logits;
  int64_t row_bytes;
  int V;
  const float* T;            // optional (NULL: 1)
  const uint32_t* bitmask;   // optional
  int64_t bm_stride;
  const int32_t* tokens;     // [B][G]; -1: empty slot
  int G;
  float* logprobs;           // [B][G]
  float* row_max;            // [B]
  float* log_sum;            // [B]
  float* entropy;            // [B], optional
  int top_n;
  int32_t* top_ids;          // [B][top_n]
  float* top_lp;
  int32_t* status;
};

struct GradArgs {
  const uint8_t* logits;
  int64_t row_bytes;
  int V;
  const float* T;
  const uint32_t* bitmask;
  int64_t bm_stride;
  const int32_t* tokens;
  int G;
  const float* row_max;
  const float* log_sum;
  const int32_t* status;
  const float* g_lp;         // [B][G]
  const float* entropy;      // [B] with g_ent, or both NULL
  const float* g_ent;
  uint8_t* grad;             // logits' dtype; may be logits itself
  int64_t grad_bytes;
};

size_t workspace_bytes(int64_t B, int64_t V, int dtype, int64_t top_n);
// whether one workgroup per part of every row fits one launch grid (batches
// past that, over 2^24 parts, are larger than the memory)
bool grid_fits(int64_t B, int64_t V, int dtype);
bool grad_grid_fits(int64_t B, int64_t V, int dtype);
hipError_t launch_score(const Args& a, int dtype, int B, void* workspace, hipStream_t st);
hipError_t launch_grad(const GradArgs& a, int dtype, int B, hipStream_t st);

}  // namespace score
}  // namespace qs
