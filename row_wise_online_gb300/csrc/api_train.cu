// api_train.cu -- the C ABI of the training-step operators: loss gradient, root-mean-square norm, embedding, gradient
// norm.  Host side only: argument checks and launches.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "train.h"

namespace rwo {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMaxLength = (int64_t(1) << 31) - 256;  // a row's length is 32-bit in the kernels
constexpr int64_t kMaxDim = int64_t(1) << 30;  // of an embedding: vectors behind a row's end are counted in 32 bits too
constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxVocab = (int64_t(1) << 31) - 2;
constexpr int64_t kMaxTensors = int64_t(1) << 20;
constexpr int64_t kMaxElements = int64_t(1) << 42;  // of all gradients: their chunks are counted in 32 bits

int check_dtype(int dtype) {
  return dtype == SOFTMAX_F32 || dtype == SOFTMAX_BF16 || dtype == SOFTMAX_F16 ? SOFTMAX_OK : SOFTMAX_ERR_INVALID_ARG;
}

// M rows of N elements of a type, M >= 0.
int check_sizes(int64_t M, int64_t N, int dtype) {
  if (check_dtype(dtype) != SOFTMAX_OK || M < 0 || N < 1) return SOFTMAX_ERR_INVALID_ARG;
  return N > kMaxLength ? SOFTMAX_ERR_UNSUPPORTED : SOFTMAX_OK;
}

// A matrix of M rows of N elements of `bytes` each at a pitch (0: N), filled in.
int check_matrix(const void* p, int64_t* ld, int64_t M, int64_t N, int64_t bytes) {
  if (*ld == 0) *ld = N;
  if (*ld < N || (M > 0 && *ld > INT64_MAX / bytes / M)) return SOFTMAX_ERR_INVALID_ARG;
  if (M == 0) return SOFTMAX_OK;
  if (!p) return SOFTMAX_ERR_INVALID_ARG;
  return aligned(p, uintptr_t(bytes)) ? SOFTMAX_OK : SOFTMAX_ERR_MISALIGNED;
}

// Whether two matrices that share their first element also share their pitch, as a call in place needs it.
bool alike(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t M) { return a != b || lda == ldb || M < 2; }

bool finite(float v) { return std::isfinite(v); }

// Whether what a list of checked tensors has written meets what it has read or written elsewhere: a CTA might scale what another has
// yet to read, or has scaled.  A tensor in place is one range that is written.
int check_overlaps(const grad_tensor* t, int64_t count) {
  struct Range {
    uintptr_t begin, end;
    bool written;
  };
  constexpr int64_t kOnStack = 128;
  Range few[kOnStack];
  std::unique_ptr<Range[]> many;
  Range* r = few;
  if (2 * count > kOnStack) {
    many.reset(new (std::nothrow) Range[size_t(2 * count)]);
    if (!many) return cuda_failure(cudaErrorMemoryAllocation);
    r = many.get();
  }
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const uintptr_t g = reinterpret_cast<uintptr_t>(t[i].grad), out = reinterpret_cast<uintptr_t>(t[i].out);
    if (out != g) r[n++] = Range{g, g + uintptr_t(t[i].n * elem_bytes(t[i].dtype)), false};
    r[n++] = Range{out, out + uintptr_t(t[i].n * elem_bytes(t[i].out_dtype)), true};
  }
  std::sort(r, r + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t read = 0, written = 0;  // where those before end
  for (int64_t i = 0; i < n; ++i) {
    if (r[i].begin < written || (r[i].written && r[i].begin < read)) return SOFTMAX_ERR_INVALID_ARG;
    uintptr_t& end = r[i].written ? written : read;
    end = std::max(end, r[i].end);
  }
  return SOFTMAX_OK;
}

int done(cudaError_t err) { return err == cudaSuccess ? SOFTMAX_OK : cuda_failure(err); }

}  // namespace
}  // namespace rwo

using namespace rwo;

extern "C" {

int cross_entropy_rows_grad(const void* x, int64_t ldx, const int64_t* labels, const float* upstream, float grad_scale,
                            float label_smoothing, float z_loss, void* grad, int64_t ldg, float* loss, float* lse_out,
                            int64_t M, int64_t N, int dtype, void* stream) {
  int st = check_sizes(M, N, dtype);
  if (st != SOFTMAX_OK) return st;
  if (!finite(grad_scale) || !(label_smoothing >= 0.f && label_smoothing < 1.f) || !finite(z_loss) || z_loss < 0.f)
    return SOFTMAX_ERR_INVALID_ARG;
  const int64_t s = elem_bytes(dtype);
  if ((st = check_matrix(x, &ldx, M, N, s)) != SOFTMAX_OK || (st = check_matrix(grad, &ldg, M, N, s)) != SOFTMAX_OK) return st;
  if (M == 0) return SOFTMAX_OK;
  if (!labels || !loss) return SOFTMAX_ERR_INVALID_ARG;
  if (!alike(x, ldx, grad, ldg, M)) return SOFTMAX_ERR_INVALID_ARG;
  if (!aligned(labels, 8) || !aligned(upstream, 4) || !aligned(loss, 4) || !aligned(lse_out, 4)) return SOFTMAX_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != SOFTMAX_OK) return st;
  LossGrad p;
  p.x = x;
  p.grad = grad;
  p.x_pitch = ldx;
  p.g_pitch = ldg;
  p.M = M;
  p.N = N;
  p.labels = labels;
  p.upstream = upstream;
  p.loss = loss;
  p.lse = lse_out;
  p.grad_scale = grad_scale;
  p.smoothing = label_smoothing;
  p.z = z_loss;
  p.dtype = dtype;
  p.stream = static_cast<cudaStream_t>(stream);
  return done(launch_loss_grad(p, *dev));
}

int rms_norm_rows(const rms_norm_args* args, int64_t M, int64_t N, int dtype, int out, void* stream) {
  if (!args) return SOFTMAX_ERR_INVALID_ARG;
  int st = check_sizes(M, N, dtype);
  if (st != SOFTMAX_OK) return st;
  if (out != RMS_NORM_OUT_SAME && out != RMS_NORM_OUT_E4M3) return SOFTMAX_ERR_INVALID_ARG;
  RmsNorm p;
  p.a = *args;
  rms_norm_args& a = p.a;
  if (!finite(a.eps) || a.eps < 0.f || !finite(a.offset)) return SOFTMAX_ERR_INVALID_ARG;
  if (a.weight_f32 != 0 && a.weight_f32 != 1) return SOFTMAX_ERR_INVALID_ARG;
  const bool e4m3 = out == RMS_NORM_OUT_E4M3;
  if (a.group != 0 && (!e4m3 || a.group < 0)) return SOFTMAX_ERR_INVALID_ARG;
  if (a.group != 0 && a.group != 128) return SOFTMAX_ERR_UNSUPPORTED;
  if ((a.residual == nullptr) != (a.sum_out == nullptr)) return SOFTMAX_ERR_INVALID_ARG;
  const int64_t s = elem_bytes(dtype);
  if ((st = check_matrix(a.x, &a.ldx, M, N, s)) != SOFTMAX_OK) return st;
  if (a.residual && ((st = check_matrix(a.residual, &a.ld_residual, M, N, s)) != SOFTMAX_OK ||
                     (st = check_matrix(a.sum_out, &a.ld_sum, M, N, s)) != SOFTMAX_OK))
    return st;
  if ((st = check_matrix(a.y, &a.ldy, M, N, e4m3 ? 1 : s)) != SOFTMAX_OK) return st;
  if (M == 0) return SOFTMAX_OK;
  if (e4m3 && !a.scales) return SOFTMAX_ERR_INVALID_ARG;
  if (a.residual && a.y == a.sum_out) return SOFTMAX_ERR_INVALID_ARG;
  if (e4m3 && (a.y == a.x || a.y == a.residual)) return SOFTMAX_ERR_INVALID_ARG;  // elements of another size
  if (!alike(a.x, a.ldx, a.y, a.ldy, M) ||
      (a.residual && (!alike(a.x, a.ldx, a.sum_out, a.ld_sum, M) || !alike(a.residual, a.ld_residual, a.sum_out, a.ld_sum, M) ||
                      !alike(a.residual, a.ld_residual, a.y, a.ldy, M))))
    return SOFTMAX_ERR_INVALID_ARG;
  if (!aligned(a.weight, a.weight_f32 ? 4 : uintptr_t(s)) || !aligned(a.scales, 4) || !aligned(a.rstd_out, 4)) return SOFTMAX_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != SOFTMAX_OK) return st;
  p.M = M;
  p.N = N;
  p.dtype = dtype;
  p.out = out;
  p.stream = static_cast<cudaStream_t>(stream);
  return done(launch_rms_norm(p, *dev));
}

int64_t rms_norm_backward_workspace(int64_t M, int64_t N, int dtype) {
  if (check_sizes(M, N, dtype) != SOFTMAX_OK) return -1;
  const DeviceInfo* dev = nullptr;
  if (current_device(&dev) != SOFTMAX_OK) return -1;
  return rms_norm_grad_parts(M, N, *dev) * N * 4;
}

int rms_norm_rows_backward(const rms_norm_grad_args* args, int64_t M, int64_t N, int dtype, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  if (!args) return SOFTMAX_ERR_INVALID_ARG;
  int st = check_sizes(M, N, dtype);
  if (st != SOFTMAX_OK) return st;
  RmsNormGrad p;
  p.a = *args;
  rms_norm_grad_args& a = p.a;
  if (!finite(a.offset) || (a.weight_f32 != 0 && a.weight_f32 != 1) || (a.accumulate != 0 && a.accumulate != 1)) return SOFTMAX_ERR_INVALID_ARG;
  const int64_t s = elem_bytes(dtype);
  if ((st = check_matrix(a.dy, &a.ld_dy, M, N, s)) != SOFTMAX_OK || (st = check_matrix(a.h, &a.ldh, M, N, s)) != SOFTMAX_OK ||
      (a.sum_grad && (st = check_matrix(a.sum_grad, &a.ld_sum_grad, M, N, s)) != SOFTMAX_OK) ||
      (st = check_matrix(a.dx, &a.ld_dx, M, N, s)) != SOFTMAX_OK)
    return st;
  if (M == 0 && (!a.dweight || a.accumulate)) return SOFTMAX_OK;
  if (M > 0 && !a.rstd) return SOFTMAX_ERR_INVALID_ARG;
  if (!alike(a.dy, a.ld_dy, a.dx, a.ld_dx, M) || !alike(a.h, a.ldh, a.dx, a.ld_dx, M) || (a.sum_grad && !alike(a.sum_grad, a.ld_sum_grad, a.dx, a.ld_dx, M)))
    return SOFTMAX_ERR_INVALID_ARG;
  if (!aligned(a.weight, a.weight_f32 ? 4 : uintptr_t(s)) || !aligned(a.rstd, 4) || !aligned(a.dweight, 4)) return SOFTMAX_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != SOFTMAX_OK) return st;
  const int64_t need = a.dweight ? rms_norm_grad_parts(M, N, *dev) * N * 4 : 0;
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return SOFTMAX_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return SOFTMAX_ERR_MISALIGNED;
  }
  p.M = M;
  p.N = N;
  p.dtype = dtype;
  p.parts = static_cast<float*>(workspace);
  p.stream = static_cast<cudaStream_t>(stream);
  return done(launch_rms_norm_grad(p, *dev));
}

static int check_tokens(const void* tokens, int token_bytes, int64_t T, int64_t V) {
  if ((token_bytes != 4 && token_bytes != 8) || T < 0 || V < 1) return SOFTMAX_ERR_INVALID_ARG;
  if (T > 0 && !tokens) return SOFTMAX_ERR_INVALID_ARG;
  return aligned(tokens, uintptr_t(token_bytes)) ? SOFTMAX_OK : SOFTMAX_ERR_MISALIGNED;
}

int embedding_rows(const void* table, int64_t ld_table, const void* tokens, int token_bytes, void* y, int64_t ldy, int64_t T,
                   int64_t V, int64_t D, float scale, int dtype, void* stream) {
  int st = check_sizes(T, D, dtype);
  if (st == SOFTMAX_OK) st = check_tokens(tokens, token_bytes, T, V);
  if (st != SOFTMAX_OK) return st;
  if (!finite(scale)) return SOFTMAX_ERR_INVALID_ARG;
  if (D > kMaxDim) return SOFTMAX_ERR_UNSUPPORTED;
  const int64_t s = elem_bytes(dtype);
  if ((st = check_matrix(table, &ld_table, T > 0 ? V : 0, D, s)) != SOFTMAX_OK || (st = check_matrix(y, &ldy, T, D, s)) != SOFTMAX_OK) return st;
  if (T == 0) return SOFTMAX_OK;
  const DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != SOFTMAX_OK) return st;
  Embedding p;
  p.table = table;
  p.y = y;
  p.table_pitch = ld_table;
  p.y_pitch = ldy;
  p.T = T;
  p.V = V;
  p.D = D;
  p.tokens = tokens;
  p.token_bytes = token_bytes;
  p.dtype = dtype;
  p.scale = scale;
  p.stream = static_cast<cudaStream_t>(stream);
  return done(launch_embedding(p, *dev));
}

static int check_embedding_grad(int64_t T, int64_t V, int64_t D) {
  if (T < 0 || V < 1 || D < 1) return SOFTMAX_ERR_INVALID_ARG;
  return T > kMaxTokens || V > kMaxVocab || D > kMaxDim || (T > 0 && D > INT64_MAX / 16 / T) ? SOFTMAX_ERR_UNSUPPORTED : SOFTMAX_OK;
}

int64_t embedding_backward_workspace(int64_t T, int64_t V, int64_t D) {
  if (check_embedding_grad(T, V, D) != SOFTMAX_OK) return -1;
  return int64_t(embedding_grad_scratch(T, V, D));
}

int embedding_rows_backward(const void* dy, int64_t ld_dy, const void* tokens, int token_bytes, void* grad, int64_t ld_grad,
                            int64_t T, int64_t V, int64_t D, float scale, int accumulate, int dtype, int grad_dtype,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_sizes(T, D, dtype);
  if (st == SOFTMAX_OK) st = check_tokens(tokens, token_bytes, T, V);
  if (st == SOFTMAX_OK) st = check_embedding_grad(T, V, D);
  if (st != SOFTMAX_OK) return st;
  if (check_dtype(grad_dtype) != SOFTMAX_OK || !finite(scale) || (accumulate != 0 && accumulate != 1)) return SOFTMAX_ERR_INVALID_ARG;
  if (grad_dtype != dtype && grad_dtype != SOFTMAX_F32) return SOFTMAX_ERR_UNSUPPORTED;
  if ((st = check_matrix(dy, &ld_dy, T, D, elem_bytes(dtype))) != SOFTMAX_OK ||
      (st = check_matrix(grad, &ld_grad, T == 0 && accumulate ? 0 : V, D, elem_bytes(grad_dtype))) != SOFTMAX_OK)
    return st;
  if (T == 0 && accumulate) return SOFTMAX_OK;
  if (!workspace || workspace_bytes < int64_t(embedding_grad_scratch(T, V, D))) return SOFTMAX_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return SOFTMAX_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != SOFTMAX_OK) return st;
  EmbeddingGrad p;
  p.dy = dy;
  p.grad = grad;
  p.dy_pitch = ld_dy;
  p.g_pitch = ld_grad;
  p.T = T;
  p.V = V;
  p.D = D;
  p.tokens = tokens;
  p.token_bytes = token_bytes;
  p.dtype = dtype;
  p.grad_dtype = grad_dtype;
  p.scale = scale;
  p.accumulate = accumulate != 0;
  p.workspace = workspace;
  p.stream = static_cast<cudaStream_t>(stream);
  return done(launch_embedding_grad(p, *dev));
}

int64_t grad_norm_workspace(int64_t count) {
  if (count < 0 || count > kMaxTensors) return -1;
  const DeviceInfo* dev = nullptr;
  if (current_device(&dev) != SOFTMAX_OK) return -1;
  return int64_t(grad_norm_scratch(count, *dev));
}

static int run_grad_norm(const grad_tensor* t, int64_t count, float scale, double max_norm, float* norm_out, void* workspace,
                         int64_t workspace_bytes, void* stream) {
  if (count < 0 || (count > 0 && !t) || !finite(scale) || !norm_out) return SOFTMAX_ERR_INVALID_ARG;
  if (count > kMaxTensors) return SOFTMAX_ERR_UNSUPPORTED;
  if (!aligned(norm_out, 4)) return SOFTMAX_ERR_MISALIGNED;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (check_dtype(t[i].dtype) != SOFTMAX_OK || t[i].n < 0) return SOFTMAX_ERR_INVALID_ARG;
    if (t[i].n > kMaxElements || (total += t[i].n) > kMaxElements) return SOFTMAX_ERR_UNSUPPORTED;
    if (t[i].n > 0 && !t[i].grad) return SOFTMAX_ERR_INVALID_ARG;
    if (!aligned(t[i].grad, uintptr_t(elem_bytes(t[i].dtype)))) return SOFTMAX_ERR_MISALIGNED;
    if (max_norm == 0.0) continue;
    if (check_dtype(t[i].out_dtype) != SOFTMAX_OK || (t[i].n > 0 && !t[i].out)) return SOFTMAX_ERR_INVALID_ARG;
    if (t[i].out_dtype != t[i].dtype && t[i].out_dtype != SOFTMAX_F32) return SOFTMAX_ERR_UNSUPPORTED;
    if (t[i].out == t[i].grad && t[i].out_dtype != t[i].dtype && t[i].n > 0) return SOFTMAX_ERR_INVALID_ARG;
    if (!aligned(t[i].out, uintptr_t(elem_bytes(t[i].out_dtype)))) return SOFTMAX_ERR_MISALIGNED;
  }
  int st = max_norm == 0.0 ? SOFTMAX_OK : check_overlaps(t, count);
  if (st != SOFTMAX_OK) return st;
  const DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != SOFTMAX_OK) return st;
  if (!workspace || workspace_bytes < int64_t(grad_norm_scratch(count, *dev))) return SOFTMAX_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return SOFTMAX_ERR_MISALIGNED;
  GradNorm p;
  p.tensors = t;
  p.count = count;
  p.scale = scale;
  p.max_norm = max_norm;
  p.norm = norm_out;
  p.parts = static_cast<double*>(workspace);
  p.stream = static_cast<cudaStream_t>(stream);
  return done(launch_grad_norm(p, *dev));
}

int grad_norm(const grad_tensor* tensors, int64_t count, float scale, float* norm_out, void* workspace, int64_t workspace_bytes,
              void* stream) {
  return run_grad_norm(tensors, count, scale, 0.0, norm_out, workspace, workspace_bytes, stream);
}

int clip_grad_norm(const grad_tensor* tensors, int64_t count, float scale, double max_norm, float* norm_out, void* workspace,
                   int64_t workspace_bytes, void* stream) {
  if (!std::isfinite(max_norm) || !(max_norm > 0.0)) return SOFTMAX_ERR_INVALID_ARG;
  return run_grad_norm(tensors, count, scale, max_norm, norm_out, workspace, workspace_bytes, stream);
}

}  // extern "C"
