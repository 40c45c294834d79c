// kernel_rms_norm.cu -- root-mean-square norm of rows, with the residual's addition and an output in 8 bits, and its
// backward pass.
//
//     h = x + residual (rounded to the element type),  rstd = (mean_j h_j^2 + eps)^-1/2,  y_j = h_j rstd (w_j + offset)
//     backward, with xhat = h rstd and g = dy (w + offset):
//     dx_j = rstd (g_j - xhat_j mean_i(g_i xhat_i)) + sum_grad_j,   dw_j = sum over rows of dy_j xhat_j
#include <initializer_list>

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

// ---- rows in registers ------------------------------------------------------------------------------------------------
//
// W warps own a row.  VEC: thread t of the group has the 16-byte vectors t, t + 32 W, ...; else its warp has runs of 128
// elements (run w, w + W, ...), a lane every 32nd of one.  Either way the 128 elements that share a scale in 8 bits lie in
// one warp.

template <class D, int W, bool VEC>
struct Place {
  static constexpr int E = VEC ? D::kVec : 1;
  // Unit k of a thread: a vector, or an element.
  __device__ static __forceinline__ int unit(int t, int k) {
    return VEC ? t + k * (W * 32) : ((t >> 5) + (k >> 2) * W) * kGroup + (k & 3) * 32 + (t & 31);
  }
};

// The sum of v over the W warps of a group, the same in all threads.  slots: W floats of the group, another set for the next call.
template <int W>
__device__ __forceinline__ float group_sum(float v, float* slots, int group, int t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if constexpr (W > 1) {
    if ((t & 31) == 0) slots[t >> 5] = v;
    named_barrier_sync(1 + group, W * 32);
    v = slots[t & (W - 1)];
#pragma unroll
    for (int o = W >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  }
  return v;
}
template <int W>
__device__ __forceinline__ float group_max(float v, float* slots, int group, int t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  if constexpr (W > 1) {
    if ((t & 31) == 0) slots[t >> 5] = v;
    named_barrier_sync(1 + group, W * 32);
    v = slots[t & (W - 1)];
#pragma unroll
    for (int o = W >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  }
  return v;
}

// The factors weight + offset of unit u.
template <class D, bool VEC, class A>
__device__ __forceinline__ void weights(const A& a, int u, float (&w)[VEC ? D::kVec : 1]) {
  constexpr int E = VEC ? D::kVec : 1;
  if (!a.w) {
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = 1.f;
    return;
  }
  if constexpr (VEC) {
    if (a.w_f32 && D::kBytes == 2) {
      const float4* p = static_cast<const float4*>(a.w) + 2 * u;
      const float4 lo = __ldg(p), hi = __ldg(p + 1);
      w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
      w[E - 4] = hi.x, w[E - 3] = hi.y, w[E - 2] = hi.z, w[E - 1] = hi.w;
    } else {
      D::unpack(__ldg(static_cast<const uint4*>(a.w) + u), w);
    }
  } else {
    w[0] = a.w_f32 ? __ldg(static_cast<const float*>(a.w) + u) : D::load1(a.w, u);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] += a.offset;
}

// What a thread holds of a unit: packed elements, or one in 32 bits.
template <class D, bool VEC>
struct Held {
  static constexpr int E = VEC ? D::kVec : 1;
  uint4 q;
  __device__ __forceinline__ void load(const unsigned char* row, int u) { q = ld_stream16(row + int64_t(u) * 16); }
  __device__ __forceinline__ void clear() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[E]) const { D::unpack(q, v); }
  __device__ __forceinline__ void set(const float (&v)[E]) { q = D::pack(v); }
  __device__ __forceinline__ void store(unsigned char* row, int u) const { st_stream16(row + int64_t(u) * 16, q); }
};
template <class D>
struct Held<D, false> {
  float q;
  __device__ __forceinline__ void load(const unsigned char* row, int u) { q = D::load1(row, u); }
  __device__ __forceinline__ void clear() { q = 0.f; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = q; }
  __device__ __forceinline__ void set(const float (&v)[1]) { q = rounded<D>(v[0]); }
  __device__ __forceinline__ void store(unsigned char* row, int u) const { D::store1(row, u, q); }
};

// E codes of unit u.
template <int E>
__device__ __forceinline__ void store_codes(unsigned char* row, int u, const float (&v)[E], float inv) {
  if constexpr (E == 8) {
    uint2 c;
    c.x = uint32_t(pack_e4m3x2(v[0] * inv, v[1] * inv)) | uint32_t(pack_e4m3x2(v[2] * inv, v[3] * inv)) << 16;
    c.y = uint32_t(pack_e4m3x2(v[4] * inv, v[5] * inv)) | uint32_t(pack_e4m3x2(v[6] * inv, v[7] * inv)) << 16;
    *reinterpret_cast<uint2*>(row + int64_t(u) * 8) = c;
  } else if constexpr (E == 4) {
    *reinterpret_cast<uint32_t*>(row + int64_t(u) * 4) =
        uint32_t(pack_e4m3x2(v[0] * inv, v[1] * inv)) | uint32_t(pack_e4m3x2(v[2] * inv, v[3] * inv)) << 16;
  } else {
    row[u] = (unsigned char)(pack_e4m3x2(v[0] * inv, 0.f) & 0xff);
  }
}

__host__ __device__ constexpr int reg_threads(int warps) { return warps * 32 > 256 ? warps * 32 : 256; }

template <class D, int K, int W, bool VEC, bool E4M3>
__global__ void __launch_bounds__(reg_threads(W)) k_rms_norm(NormArgs a) {
  using P = Place<D, W, VEC>;
  constexpr int E = P::E, GT = W * 32, G = reg_threads(W) / GT;
  __shared__ float sums[2][reg_threads(W) / 32], tops[2][reg_threads(W) / 32];
  const int group = threadIdx.x / GT, t = threadIdx.x % GT, lane = t & 31;
  const int units = int(a.N / E);
  int it = 0;
  for (int64_t row = int64_t(blockIdx.x) * G + group; row < a.M; row += int64_t(gridDim.x) * G, it ^= 1) {
    const unsigned char* xr = a.x + row * a.x_pitch;
    Held<D, VEC> h[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = P::unit(t, k);
      if (u < units) h[k].load(xr, u);
      else h[k].clear();
    }
    if (a.r) {
      const unsigned char* rr = a.r + row * a.r_pitch;
      unsigned char* to = a.h + row * a.h_pitch;
      Held<D, VEC> r[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = P::unit(t, k);
        if (u < units) r[k].load(rr, u);
        else r[k].clear();
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = P::unit(t, k);
        float v[E], w[E];
        h[k].get(v);
        r[k].get(w);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] += w[e];
        h[k].set(v);
        if (u < units) h[k].store(to, u);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[E];
      h[k].get(v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum = __fmaf_rn(v[e], v[e], sum);
    }
    sum = group_sum<W>(sum, sums[it] + group * W, group, t);
    const float rstd = 1.f / sqrtf(sum / float(a.N) + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    unsigned char* yr = a.y + row * a.y_pitch;
    if constexpr (!E4M3) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = P::unit(t, k);
        if (u >= units) continue;
        float v[E], w[E];
        h[k].get(v);
        weights<D, VEC>(a, u, w);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = v[e] * rstd * w[e];
        h[k].set(v);
        h[k].store(yr, u);
      }
    } else {
      const auto value = [&](int k, float(&v)[E]) {  // y in 32 bits, 0 behind the row's end
        const int u = P::unit(t, k);
        float w[E];
        h[k].get(v);
        if (u < units) weights<D, VEC>(a, u, w);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = u < units ? v[e] * rstd * w[e] : 0.f;
      };
      const auto top_of = [&](const float(&v)[E]) {
        float m = fabsf(v[0]);
#pragma unroll
        for (int e = 1; e < E; ++e) m = fmaxf(m, fabsf(v[e]));
        return m;
      };
      if (a.groups == 1 && a.N > kGroup) {
        float y[K][E], top = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          value(k, y[k]);
          top = fmaxf(top, top_of(y[k]));
        }
        top = group_max<W>(top, tops[it] + group * W, group, t);
        const float scale = fmaxf(top / kE4m3Max, kScaleMin), inv = 1.f / scale;
        if (t == 0) a.scales[row] = scale;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int u = P::unit(t, k);
          if (u < units) store_codes<E>(yr, u, y[k], inv);
        }
      } else {
        constexpr int step = VEC ? 1 : 4, lanes = VEC ? kGroup / E : 32;  // units of a group in a lane; lanes of a group
#pragma unroll
        for (int k = 0; k < K; k += step) {
          float y[step][E], top = 0.f;
#pragma unroll
          for (int j = 0; j < step; ++j) {
            value(k + j, y[j]);
            top = fmaxf(top, top_of(y[j]));
          }
#pragma unroll
          for (int o = lanes >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
          const float scale = fmaxf(top / kE4m3Max, kScaleMin), inv = 1.f / scale;
          const int u = P::unit(t, k);
          if (u < units && (lane & (lanes - 1)) == 0) a.scales[row * a.groups + u * E / kGroup] = scale;
#pragma unroll
          for (int j = 0; j < step; ++j)
            if (P::unit(t, k + j) < units) store_codes<E>(yr, P::unit(t, k + j), y[j], inv);
        }
      }
    }
  }
}

// Backward: every CTA walks its rows with the columns' sums of dw in registers, and leaves them as one part.
template <class D, int K, int W, bool VEC>
__global__ void __launch_bounds__(reg_threads(W)) k_rms_grad(GradArgs a) {
  using P = Place<D, W, VEC>;
  constexpr int E = P::E, GT = W * 32, G = reg_threads(W) / GT;
  __shared__ float sums[2][reg_threads(W) / 32];
  __shared__ float columns[G > 1 ? K * E * GT : 1];
  const int group = threadIdx.x / GT, t = threadIdx.x % GT;
  const int units = int(a.N / E);
  const int64_t step = int64_t(gridDim.x) * G;
  float dw[K][E] = {};
  Held<D, VEC> dy[K], h[K], sg[K];
  float rstd = 0.f;
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = P::unit(t, k);
      if (u < units) {
        dy[k].load(a.dy + row * a.dy_pitch, u);
        h[k].load(a.h + row * a.h_pitch, u);
        if (a.sg) sg[k].load(a.sg + row * a.sg_pitch, u);
      }
    }
    rstd = a.rstd[row];
  };
#pragma unroll
  for (int k = 0; k < K; ++k) dy[k].clear(), h[k].clear(), sg[k].clear();
  int64_t row = int64_t(blockIdx.x) * G + group;
  if (row < a.M) fetch(row);
  int it = 0;
  for (; row < a.M; row += step, it ^= 1) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = P::unit(t, k);
      if (u >= units) continue;
      float d[E], x[E], w[E];
      dy[k].get(d);
      h[k].get(x);
      weights<D, VEC>(a, u, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float p = d[e] * (x[e] * rstd);
        sum = __fmaf_rn(p, w[e], sum);
        dw[k][e] += p;
      }
    }
    const float mean = group_sum<W>(sum, sums[it] + group * W, group, t) / float(a.N);
    unsigned char* to = a.dx + row * a.dx_pitch;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = P::unit(t, k);
      if (u >= units) continue;
      float d[E], x[E], w[E], s[E];
      dy[k].get(d);
      h[k].get(x);
      sg[k].get(s);
      weights<D, VEC>(a, u, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float v = rstd * __fmaf_rn(-(x[e] * rstd), mean, d[e] * w[e]);
        d[e] = a.sg ? v + s[e] : v;
      }
      Held<D, VEC> out;
      out.set(d);
      out.store(to, u);
    }
    if (row + step < a.M) fetch(row + step);
  }
  if (!a.dw) return;
  float* part = a.parts + blockIdx.x * a.N;
  if constexpr (G == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = P::unit(t, k);
      if (u >= units) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) part[u * E + e] = dw[k][e];
    }
  } else {
    // the groups' sums one after the other
    for (int g = 0; g < G; ++g) {
      if (group == g) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float* c = columns + (k * E + e) * GT + t;
            *c = g ? *c + dw[k][e] : dw[k][e];
          }
      }
      __syncthreads();
    }
    if (group == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = P::unit(t, k);
        if (u >= units) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) part[u * E + e] = columns[(k * E + e) * GT + t];
      }
    }
  }
}

// dw = the parts added up: 32 columns a CTA, eight warps every eighth part.
__global__ void __launch_bounds__(kThreads) k_rms_weight_join(GradArgs a) {
  __shared__ float sums[kThreads / 32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = int64_t(blockIdx.x) * 32 + lane;
  float sum = 0.f;
  if (i < a.N) {
#pragma unroll 8
    for (int k = warp; k < a.parts_n; k += kThreads / 32) sum += a.parts[k * a.N + i];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && i < a.N) {
    float all = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) all += sums[w][lane];
    a.dw[i] = a.accumulate ? a.dw[i] + all : all;
  }
}

struct NormConfig {
  int warps, units;            // warps a row, units they hold
  void (*fn[2])(NormArgs);     // [e4m3]
};
template <class D, int K, int W, bool VEC>
constexpr NormConfig norm_cfg() {
  return NormConfig{W, 32 * W * K, {k_rms_norm<D, K, W, VEC, false>, k_rms_norm<D, K, W, VEC, true>}};
}
struct GradConfig {
  int warps, units;
  void (*fn)(GradArgs);
};
template <class D, int K, int W, bool VEC>
constexpr GradConfig grad_cfg() {
  return GradConfig{W, 32 * W * K, k_rms_grad<D, K, W, VEC>};
}

// The first configuration that holds a row.
template <class C, int n>
const C* pick(const C (&table)[n], int64_t units) {
  for (const C& c : table)
    if (units <= c.units) return &c;
  return nullptr;
}

unsigned row_grid(int64_t M, const DeviceInfo& dev) {
  const int64_t slots = int64_t(dev.sm_count) * (dev.max_threads_per_sm / kThreads);
  return unsigned(M < slots ? M : slots);
}

bool on16(std::initializer_list<uintptr_t> v) {
  uintptr_t all = 0;
  for (const uintptr_t x : v) all |= x;
  return (all & 15) == 0;
}
template <class T>
uintptr_t bits(const T* p) {
  return reinterpret_cast<uintptr_t>(p);
}

template <class D>
cudaError_t launch_norm_type(const RmsNorm& p, const NormArgs& a, const DeviceInfo& dev) {
  // at most 64 elements a thread
  static const NormConfig vectors[] = {norm_cfg<D, 1, 1, true>(), norm_cfg<D, 2, 1, true>(), norm_cfg<D, 4, 1, true>(), norm_cfg<D, 4, 2, true>(),
                                       norm_cfg<D, 4, 4, true>(), norm_cfg<D, 4, 8, true>(), norm_cfg<D, 4, 16, true>(), norm_cfg<D, 8, 16, true>()};
  static const NormConfig elements[] = {norm_cfg<D, 4, 1, false>(), norm_cfg<D, 16, 1, false>(), norm_cfg<D, 16, 4, false>(), norm_cfg<D, 32, 4, false>(),
                                        norm_cfg<D, 32, 8, false>(), norm_cfg<D, 32, 16, false>()};
  const bool e4m3 = p.out == RMS_NORM_OUT_E4M3;
  // codes of a vector are 8 or 4 bytes: half or a quarter of what the element types need
  const uintptr_t code = e4m3 ? 16 / D::kVec : 1;
  const bool vec = on16({bits(a.x), bits(a.r), bits(a.h), bits(a.y) * code, bits(static_cast<const char*>(a.w)), uintptr_t(a.x_pitch),
                         a.r ? uintptr_t(a.r_pitch | a.h_pitch) : 0, uintptr_t(a.y_pitch) * code, uintptr_t(p.N * D::kBytes)});
  const NormConfig* c = vec ? pick(vectors, p.N / D::kVec) : pick(elements, p.N);
  if (c) {
    const int threads = reg_threads(c->warps), groups = threads / 32 / c->warps;
    const int64_t ctas = (p.M + groups - 1) / groups, most = int64_t(dev.sm_count) * (dev.max_threads_per_sm / threads) * 4;
    c->fn[e4m3]<<<unsigned(ctas < most ? ctas : most), threads, 0, p.stream>>>(a);
  } else if (e4m3) {
    k_rms_norm_loop<D, true><<<row_grid(p.M, dev), kThreads, 0, p.stream>>>(a);
  } else {
    k_rms_norm_loop<D, false><<<row_grid(p.M, dev), kThreads, 0, p.stream>>>(a);
  }
  return cudaGetLastError();
}

constexpr int kGradCtas = 4;  // parts of dw for each SM at most

template <class D>
cudaError_t launch_grad_type(const RmsNormGrad& p, GradArgs a, const DeviceInfo& dev) {
  // at most 32 elements a thread, whose sums of dw stay in registers
  constexpr int F = D::kBytes / 2;  // fp32 vectors have half the elements
  static const GradConfig vectors[] = {grad_cfg<D, F, 1, true>(), grad_cfg<D, 2 * F, 1, true>(), grad_cfg<D, 4 * F, 1, true>(), grad_cfg<D, 4 * F, 2, true>(),
                                       grad_cfg<D, 2 * F, 8, true>(), grad_cfg<D, 4 * F, 8, true>(), grad_cfg<D, 4 * F, 16, true>()};
  static const GradConfig elements[] = {grad_cfg<D, 4, 1, false>(), grad_cfg<D, 16, 1, false>(), grad_cfg<D, 16, 4, false>(), grad_cfg<D, 16, 8, false>(),
                                        grad_cfg<D, 32, 8, false>(), grad_cfg<D, 32, 16, false>()};
  const bool vec = on16({bits(a.dy), bits(a.h), bits(a.sg), bits(a.dx), bits(static_cast<const char*>(a.w)), uintptr_t(a.dy_pitch), uintptr_t(a.h_pitch),
                         a.sg ? uintptr_t(a.sg_pitch) : 0, uintptr_t(a.dx_pitch), uintptr_t(p.N * D::kBytes)});
  const GradConfig* c = vec ? pick(vectors, p.N / D::kVec) : pick(elements, p.N);
  const unsigned joins = unsigned((p.N + 31) / 32);
  if (p.M == 0) {
    a.parts_n = 0;
  } else if (c) {
    const int threads = reg_threads(c->warps), groups = threads / 32 / c->warps;
    const int64_t ctas = (p.M + groups - 1) / groups;
    const int64_t per_sm = threads > 256 ? 2 : kGradCtas;
    a.parts_n = int(ctas < dev.sm_count * per_sm ? ctas : dev.sm_count * per_sm);
    c->fn<<<unsigned(a.parts_n), threads, 0, p.stream>>>(a);
    if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  } else if (a.dw) {
    // the weight's gradient first: dx may be written where dy or h are
    a.rows_per_part = (p.M + a.parts_n - 1) / a.parts_n;
    k_rms_weight_grad<D><<<dim3(unsigned((p.N + kThreads - 1) / kThreads), a.parts_n), kThreads, 0, p.stream>>>(a);
    if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  }
  if (a.dw) {
    k_rms_weight_join<<<joins, kThreads, 0, p.stream>>>(a);
    if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  }
  if (p.M > 0 && !c) k_rms_grad_loop<D><<<row_grid(p.M, dev), kThreads, 0, p.stream>>>(a);
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

int64_t rms_norm_grad_parts(int64_t M, int64_t, const DeviceInfo& dev) {
  const int64_t most = int64_t(dev.sm_count) * kGradCtas;
  return M < most ? M : most;
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
  a.rows_per_part = 0;
  a.offset = p.a.offset;
  a.w_f32 = p.a.weight_f32 != 0;
  a.accumulate = p.a.accumulate != 0;
  return p.dtype == SOFTMAX_F32 ? launch_grad_type<F32>(p, a, dev) : p.dtype == SOFTMAX_BF16 ? launch_grad_type<BF16>(p, a, dev) : launch_grad_type<F16>(p, a, dev);
}

}  // namespace rwo
