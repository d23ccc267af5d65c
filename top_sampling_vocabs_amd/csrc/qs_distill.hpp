// Argument blocks and launchers of distillation from a teacher's top tokens: the
// loss of each row and its gradient.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qs {
namespace distill {

constexpr int kSlotsMax = 1024;  // teacher's tokens per row
constexpr int kState = 8;        // floats per row left for the gradient

struct Args {
  const uint8_t* logits;
  int64_t row_bytes;
  int V;
  const float* T;            // optional (NULL: 1)
  const uint32_t* bitmask;   // optional
  int64_t bm_stride;
  const int32_t* ids;        // [B][K]; -1: empty slot
  const float* values;       // [B][K]
  int K;
  int rest;                  // values are log-probabilities, the missing mass counts
  float* loss;               // [B]
  float* state;              // [B][kState]
  int32_t* status;           // [B]
};

struct GradArgs {
  const uint8_t* logits;
  int64_t row_bytes;
  int V;
  const float* T;
  const uint32_t* bitmask;
  int64_t bm_stride;
  const int32_t* ids;
  const float* values;
  int K;
  int rest;
  const float* state;
  const int32_t* status;
  const float* g_loss;       // [B]
  uint8_t* grad;             // logits' dtype; may be logits itself
  int64_t grad_bytes;
};

size_t workspace_bytes(int64_t B, int64_t V, int dtype);
// whether one workgroup per part of every row fits one launch grid
bool grid_fits(int64_t B, int64_t V, int dtype);
bool grad_grid_fits(int64_t B, int64_t V, int dtype);
hipError_t launch_loss(const Args& a, int dtype, int B, void* workspace, hipStream_t st);
hipError_t launch_grad(const GradArgs& a, int dtype, int B, hipStream_t st);

}  // namespace distill
}  // namespace qs
