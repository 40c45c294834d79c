// train.h -- internal interface of the training-step kernels: loss gradient (kernel_loss_grad.cu), root-mean-square norm
// (kernel_rms_norm.cu), embedding (kernel_embedding.cu), gradient norm (kernel_grad_norm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/softmax_rows.h"
#include "launch.h"

namespace rwo {

// Device pointers throughout; null where a part is not used.  Pitches in elements.

struct LossGrad {
  const void* x = nullptr;
  void* grad = nullptr;
  int64_t x_pitch = 0, g_pitch = 0, M = 0, N = 0;
  const int64_t* labels = nullptr;
  const float* upstream = nullptr;
  float* loss = nullptr;
  float* lse = nullptr;
  float grad_scale = 1.f, smoothing = 0.f, z = 0.f;
  int dtype = 0;
  cudaStream_t stream = nullptr;
};
cudaError_t launch_loss_grad(const LossGrad& p, const DeviceInfo& dev);

struct RmsNorm {
  rms_norm_args a{};  // pitches filled in
  int64_t M = 0, N = 0;
  int dtype = 0, out = 0;
  cudaStream_t stream = nullptr;
};
cudaError_t launch_rms_norm(const RmsNorm& p, const DeviceInfo& dev);

struct RmsNormGrad {
  rms_norm_grad_args a{};  // pitches filled in
  int64_t M = 0, N = 0;
  int dtype = 0;
  float* parts = nullptr;  // rms_norm_grad_parts() rows of N
  cudaStream_t stream = nullptr;
};
int64_t rms_norm_grad_parts(int64_t M, int64_t N, const DeviceInfo& dev);
cudaError_t launch_rms_norm_grad(const RmsNormGrad& p, const DeviceInfo& dev);

struct Embedding {
  const void* table = nullptr;
  void* y = nullptr;
  int64_t table_pitch = 0, y_pitch = 0, T = 0, V = 0, D = 0;
  const void* tokens = nullptr;
  int token_bytes = 8, dtype = 0;
  float scale = 1.f;
  cudaStream_t stream = nullptr;
};
cudaError_t launch_embedding(const Embedding& p, const DeviceInfo& dev);

struct EmbeddingGrad {
  const void* dy = nullptr;
  void* grad = nullptr;
  int64_t dy_pitch = 0, g_pitch = 0, T = 0, V = 0, D = 0;
  const void* tokens = nullptr;
  int token_bytes = 8, dtype = 0, grad_dtype = 0;
  float scale = 1.f;
  bool accumulate = false;
  void* workspace = nullptr;
  cudaStream_t stream = nullptr;
};
size_t embedding_grad_scratch(int64_t T, int64_t V, int64_t D);
cudaError_t launch_embedding_grad(const EmbeddingGrad& p, const DeviceInfo& dev);

struct GradNorm {
  const grad_tensor* tensors = nullptr;  // host
  int64_t count = 0;
  float scale = 1.f;
  double max_norm = 0.0;  // 0: the norm alone
  float* norm = nullptr;
  double* parts = nullptr;
  cudaStream_t stream = nullptr;
};
size_t grad_norm_scratch(int64_t count, const DeviceInfo& dev);
cudaError_t launch_grad_norm(const GradNorm& p, const DeviceInfo& dev);

}  // namespace rwo
