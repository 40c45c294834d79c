// logits.h -- internal interface of the logits processing kernel (kernel_logits.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace rwo {

constexpr int kMaxBias = 1024;             // bias entries of a row
constexpr int64_t kMaxHistory = 1 << 20;   // tokens of a row, less one

// One call.  Device pointers; null where a part is not used.
struct LogitsProblem {
  const void* x = nullptr;
  void* y = nullptr;
  float* lse = nullptr;
  int64_t M = 0, N = 0, x_pitch = 0, y_pitch = 0;  // pitches in elements
  int dtype = 0, out = 0;                          // out: 0 logits, 1 softmax, 2 log softmax
  const int32_t* tokens = nullptr;                 // [M][token_pitch]: prompt, then output
  int64_t token_pitch = 0;                         // tokens a row has room for
  const int32_t* prompt_lens = nullptr;
  const int32_t* token_lens = nullptr;
  const float* repetition = nullptr;
  const float* frequency = nullptr;
  const float* presence = nullptr;
  const int32_t* bias_ids = nullptr;               // [M][bias_count], negative: none
  const float* bias_values = nullptr;
  int bias_count = 0;
  const uint32_t* mask = nullptr;                  // [M][mask_pitch] words, bit set: allowed
  int64_t mask_pitch = 0;
  const float* scale = nullptr;
  cudaStream_t stream = nullptr;
};

cudaError_t launch_logits(const LogitsProblem& p, const DeviceInfo& dev);

}  // namespace rwo
