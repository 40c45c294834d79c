// kernel_rms_norm.cu -- root-mean-square norm of rows, with the residual's addition and an output in 8 bits, and its
// backward pass.
//
//     h = x + residual (rounded to the element type),  rstd = (mean_j h_j^2 + eps)^-1/2,  y_j = h_j rstd (w_j + offset)
//     backward, with xhat = h rstd and g = dy (w + offset):
//     dx_j = rstd (g_j - xhat_j mean_i(g_i xhat_i)) + sum_grad_j,   dw_j = sum over rows of dy_j xhat_j
#include "train.cuh"
#include "train.h"

namespace rwo {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 0x1p-126f;
constexpr int kGroup = 128;

struct NormArgs {
  const unsigned char* x;
  const unsigned char* r;
  unsigned char* h;
  const void* w;
  unsigned char* y;
  float* scales;
  float* rstd;
  int64_t M, N;
  int64_t x_pitch, r_pitch, h_pitch, y_pitch;  // bytes
  int64_t groups;                              // scales of a row
  float eps, offset;
  bool w_f32;
};

struct GradArgs {
  const unsigned char* dy;
  const unsigned char* h;
  const unsigned char* sg;
  const float* rstd;
  const void* w;
  unsigned char* dx;
  float* dw;
  float* parts;
  int64_t M, N;
  int64_t dy_pitch, h_pitch, sg_pitch, dx_pitch;  // bytes
  int64_t rows_per_part;
  int parts_n;
  float offset;
  bool w_f32, accumulate;
};

template <class D, class A>
__device__ __forceinline__ float weight1(const A& a, int64_t i) {
  if (!a.w) return 1.f;
  return (a.w_f32 ? __ldg(static_cast<const float*>(a.w) + i) : D::load1(a.w, i)) + a.offset;
}

// Two values -> two e4m3 codes (lo in the low byte), to the nearest, limited to +-448.
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int WARPS>
__device__ __forceinline__ float block_sum(float v, float* slots) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();
  if (lane == 0) slots[warp] = v;
  __syncthreads();
  v = lane < WARPS ? slots[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

template <int WARPS>
__device__ __forceinline__ float block_max(float v, float* slots) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  __syncthreads();
  if (lane == 0) slots[warp] = v;
  __syncthreads();
  v = lane < WARPS ? slots[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}

// ---- rows of any length and alignment: a CTA a row, read anew for each pass -----------------------------------------

constexpr int kThreads = 256;

template <class D, bool E4M3>
__global__ void __launch_bounds__(kThreads) k_rms_norm_loop(NormArgs a) {
  __shared__ float slots[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const unsigned char* xr = a.x + row * a.x_pitch;
    const unsigned char* hr = xr;
    float sum = 0.f;
    if (a.r) {
      const unsigned char* rr = a.r + row * a.r_pitch;
      unsigned char* to = a.h + row * a.h_pitch;
      hr = to;
      for (int64_t i = threadIdx.x; i < a.N; i += kThreads) {
        const float h = rounded<D>(load1c<D>(xr, i) + load1c<D>(rr, i));
        D::store1(to, i, h);
        sum = __fmaf_rn(h, h, sum);
      }
    } else {
      for (int64_t i = threadIdx.x; i < a.N; i += kThreads) {
        const float h = load1c<D>(xr, i);
        sum = __fmaf_rn(h, h, sum);
      }
    }
    sum = block_sum<kThreads / 32>(sum, slots);  // its barriers also order h's stores before the loads below
    const float rstd = 1.f / sqrtf(sum / float(a.N) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    unsigned char* yr = a.y + row * a.y_pitch;
    if constexpr (!E4M3) {
      for (int64_t i = threadIdx.x; i < a.N; i += kThreads) D::store1(yr, i, load1c<D>(hr, i) * rstd * weight1<D>(a, i));
    } else if (a.groups == 1 && a.N > kGroup) {
      float top = 0.f;
      for (int64_t i = threadIdx.x; i < a.N; i += kThreads) top = fmaxf(top, fabsf(load1c<D>(hr, i) * rstd * weight1<D>(a, i)));
      top = block_max<kThreads / 32>(top, slots);
      const float scale = fmaxf(top / kE4m3Max, kScaleMin), inv = 1.f / scale;
      if (threadIdx.x == 0) a.scales[row] = scale;
      for (int64_t i = threadIdx.x; i < a.N; i += kThreads)
        yr[i] = (unsigned char)(pack_e4m3x2(load1c<D>(hr, i) * rstd * weight1<D>(a, i) * inv, 0.f) & 0xff);
    } else {
      for (int64_t g = warp; g < a.groups; g += kThreads / 32) {
        float v[kGroup / 32], top = 0.f;
#pragma unroll
        for (int k = 0; k < kGroup / 32; ++k) {
          const int64_t i = g * kGroup + k * 32 + lane;
          v[k] = i < a.N ? load1c<D>(hr, i) * rstd * weight1<D>(a, i) : 0.f;
          top = fmaxf(top, fabsf(v[k]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const float scale = fmaxf(top / kE4m3Max, kScaleMin), inv = 1.f / scale;
        if (lane == 0) a.scales[row * a.groups + g] = scale;
#pragma unroll
        for (int k = 0; k < kGroup / 32; ++k) {
          const int64_t i = g * kGroup + k * 32 + lane;
          if (i < a.N) yr[i] = (unsigned char)(pack_e4m3x2(v[k] * inv, 0.f) & 0xff);
        }
      }
    }
  }
}

// dx alone, two reads of the row.
template <class D>
__global__ void __launch_bounds__(kThreads) k_rms_grad_loop(GradArgs a) {
  __shared__ float slots[32];
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const unsigned char* dr = a.dy + row * a.dy_pitch;
    const unsigned char* hr = a.h + row * a.h_pitch;
    const unsigned char* sr = a.sg + row * a.sg_pitch;
    unsigned char* to = a.dx + row * a.dx_pitch;
    const float rstd = a.rstd[row];
    float sum = 0.f;
    for (int64_t i = threadIdx.x; i < a.N; i += kThreads) sum = __fmaf_rn(load1c<D>(dr, i) * weight1<D>(a, i), load1c<D>(hr, i) * rstd, sum);
    const float mean = block_sum<kThreads / 32>(sum, slots) / float(a.N);
    for (int64_t i = threadIdx.x; i < a.N; i += kThreads) {
      float v = rstd * __fmaf_rn(-(load1c<D>(hr, i) * rstd), mean, load1c<D>(dr, i) * weight1<D>(a, i));
      if (a.sg) v += load1c<D>(sr, i);
      D::store1(to, i, v);
    }
  }
}

// Part blockIdx.y of dw's columns blockIdx.x * kThreads ..: a run of rows.
template <class D>
__global__ void __launch_bounds__(kThreads) k_rms_weight_grad(GradArgs a) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= a.N) return;
  const int64_t r0 = blockIdx.y * a.rows_per_part, r1 = r0 + a.rows_per_part < a.M ? r0 + a.rows_per_part : a.M;
  float sum = 0.f;
  for (int64_t row = r0; row < r1; ++row)
    sum = __fmaf_rn(D::load1(a.dy + row * a.dy_pitch, i), D::load1(a.h + row * a.h_pitch, i) * a.rstd[row], sum);
  a.parts[blockIdx.y * a.N + i] = sum;
}

// dw = the parts added up in their order.
__global__ void __launch_bounds__(kThreads) k_rms_weight_sum(GradArgs a) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= a.N) return;
  float sum = 0.f;
  for (int k = 0; k < a.parts_n; ++k) sum += a.parts[k * a.N + i];
  a.dw[i] = a.accumulate ? a.dw[i] + sum : sum;
}

unsigned row_grid(int64_t M, const DeviceInfo& dev) {
  const int64_t slots = int64_t(dev.sm_count) * (dev.max_threads_per_sm / kThreads);
  return unsigned(M < slots ? M : slots);
}

template <class D>
cudaError_t launch_norm_type(const RmsNorm& p, const NormArgs& a, const DeviceInfo& dev) {
  if (p.out == RMS_NORM_OUT_E4M3) k_rms_norm_loop<D, true><<<row_grid(p.M, dev), kThreads, 0, p.stream>>>(a);
  else k_rms_norm_loop<D, false><<<row_grid(p.M, dev), kThreads, 0, p.stream>>>(a);
  return cudaGetLastError();
}

template <class D>
cudaError_t launch_grad_type(const RmsNormGrad& p, const GradArgs& a, const DeviceInfo& dev) {
  const unsigned columns = unsigned((p.N + kThreads - 1) / kThreads);
  // the weight's gradient first: dx may be written where dy or h are
  if (a.dw) {
    if (p.M > 0) {
      k_rms_weight_grad<D><<<dim3(columns, a.parts_n), kThreads, 0, p.stream>>>(a);
      if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
    k_rms_weight_sum<<<columns, kThreads, 0, p.stream>>>(a);
    if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  }
  if (p.M > 0) k_rms_grad_loop<D><<<row_grid(p.M, dev), kThreads, 0, p.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNorm& p, const DeviceInfo& dev) {
  const int64_t s = elem_bytes(p.dtype);
  NormArgs a;
  a.x = static_cast<const unsigned char*>(p.a.x);
  a.r = static_cast<const unsigned char*>(p.a.residual);
  a.h = static_cast<unsigned char*>(p.a.sum_out);
  a.w = p.a.weight;
  a.y = static_cast<unsigned char*>(p.a.y);
  a.scales = p.a.scales;
  a.rstd = p.a.rstd_out;
  a.M = p.M;
  a.N = p.N;
  a.x_pitch = p.a.ldx * s;
  a.r_pitch = p.a.ld_residual * s;
  a.h_pitch = p.a.ld_sum * s;
  a.y_pitch = p.a.ldy * (p.out == RMS_NORM_OUT_E4M3 ? 1 : s);
  a.groups = p.a.group ? (p.N + kGroup - 1) / kGroup : 1;
  a.eps = p.a.eps;
  a.offset = p.a.offset;
  a.w_f32 = p.a.weight_f32 != 0;
  return p.dtype == SOFTMAX_F32 ? launch_norm_type<F32>(p, a, dev) : p.dtype == SOFTMAX_BF16 ? launch_norm_type<BF16>(p, a, dev) : launch_norm_type<F16>(p, a, dev);
}

int64_t rms_norm_grad_parts(int64_t M, int64_t N, const DeviceInfo& dev) {
  const int64_t most = int64_t(dev.sm_count) * 8, parts = (M + 31) / 32;
  return parts < most ? parts : most;
}

cudaError_t launch_rms_norm_grad(const RmsNormGrad& p, const DeviceInfo& dev) {
  const int64_t s = elem_bytes(p.dtype);
  GradArgs a;
  a.dy = static_cast<const unsigned char*>(p.a.dy);
  a.h = static_cast<const unsigned char*>(p.a.h);
  a.sg = static_cast<const unsigned char*>(p.a.sum_grad);
  a.rstd = p.a.rstd;
  a.w = p.a.weight;
  a.dx = static_cast<unsigned char*>(p.a.dx);
  a.dw = p.a.dweight;
  a.parts = p.parts;
  a.M = p.M;
  a.N = p.N;
  a.dy_pitch = p.a.ld_dy * s;
  a.h_pitch = p.a.ldh * s;
  a.sg_pitch = p.a.ld_sum_grad * s;
  a.dx_pitch = p.a.ld_dx * s;
  a.parts_n = int(rms_norm_grad_parts(p.M, p.N, dev));
  a.rows_per_part = a.parts_n ? (p.M + a.parts_n - 1) / a.parts_n : 0;
  a.offset = p.a.offset;
  a.w_f32 = p.a.weight_f32 != 0;
  a.accumulate = p.a.accumulate != 0;
  return p.dtype == SOFTMAX_F32 ? launch_grad_type<F32>(p, a, dev) : p.dtype == SOFTMAX_BF16 ? launch_grad_type<BF16>(p, a, dev) : launch_grad_type<F16>(p, a, dev);
}

}  // namespace rwo
