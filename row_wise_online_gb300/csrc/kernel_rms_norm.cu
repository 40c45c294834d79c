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
  bool w_f32, w_vec;  // w_vec: on a 16-byte boundary
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
  bool w_f32, w_vec, accumulate;
};

// What a factor weight + offset is multiplied by on its way into 8 bits (Codes).
constexpr float kSeven = 3.5f;

// A weight as it lies, to a factor; into 8 bits kSeven times it.
template <bool E4M3, class A>
__device__ __forceinline__ float factor(const A& a, float w) {
  return E4M3 ? __fmaf_rn(w, kSeven, kSeven * a.offset) : w + a.offset;
}
template <class D, bool E4M3 = false, class A>
__device__ __forceinline__ float weight1(const A& a, int64_t i) {
  if (!a.w) return E4M3 ? kSeven : 1.f;
  return factor<E4M3>(a, a.w_f32 ? __ldg(static_cast<const float*>(a.w) + i) : D::load1(a.w, i));
}

// Codes in 8 bits: the nearest to y / scale, scale = max |y| / 448 over a group.  rstd is in both, so of rstd = two * rest, two a power of
// 2, the kernels take two alone and work with
//     v = h two (7/2) (weight + offset) = (7/2) y / rest,    scale = (2/7) rest t,    y / scale = v / t,    t = max |v| / 448.
// Of bf16 elements and weights v is exact (7 times a product of 16 bits), and so is t.  One value in 2500 lies in the middle between two
// codes there; roundings of y, scale and 1 / scale put it on either side, by the order in which a row's squares are added up.  So the
// quotient's remainder against t takes up what v * (1 / t) rounded: the code is that of the exact quotient, ties to even, in every kernel.
struct Codes {
  float t, inv;
};
struct Parts {
  float two, back, least;  // back: (2/7) rest; least: the t of the least scale
};
__device__ __forceinline__ Parts parts_of(float rstd) {
  const uint32_t b = __float_as_uint(rstd);
  const bool number = rstd <= 3.4028234663852886e38f;
  Parts p;
  p.two = number ? __uint_as_float(b & 0x7f800000u) : rstd;
  p.back = (number ? __uint_as_float((b & 0x007fffffu) | 0x3f800000u) : 1.f) * (1.f / kSeven);
  p.least = __fdividef(kScaleMin, p.back);
  return p;
}
// Of a group whose largest |v| is top; its scale.
__device__ __forceinline__ Codes codes_of(float top, const Parts& p, float* scale) {
  float t = top * (1.f / kE4m3Max);
  if (top <= 3.4028234663852886e38f) t = __fmaf_rn(__fmaf_rn(-t, kE4m3Max, top), 1.f / kE4m3Max, t);
  *scale = fmaxf(t * p.back, kScaleMin);
  t = fmaxf(t, p.least);
  return Codes{t, __fdividef(1.f, t)};
}
__device__ __forceinline__ float quotient(float v, const Codes& c) {
  const float q = v * c.inv;
  return __fmaf_rn(__fmaf_rn(-q, c.t, v), c.inv, q);
}
__device__ __forceinline__ float2 quotient2(const float2& v, const Codes& c) {
  const float2 inv = make_float2(c.inv, c.inv), q = __fmul2_rn(v, inv);
  return __ffma2_rn(__ffma2_rn(q, make_float2(-c.t, -c.t), v), inv, q);
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
// A thread's elements are loaded kBatch at a time, and kPlain of them added up before they go to its long sum (all of them plainly, 2^22
// equal squares are off by 2e-4).
// Eight CTAs an SM, as many as row_grid() counts on (at 40 registers a thread some of them make a second round: 4096 x 40960 fp32 forward
// 961 us instead of 738).
constexpr int kBatch = 4, kPlain = 64;

// Elements i, i + kThreads, ... of a row of n, 0 behind its end.
template <class D>
__device__ __forceinline__ void load_batch(const unsigned char* row, int64_t i, int64_t n, float (&v)[kBatch]) {
#pragma unroll
  for (int k = 0; k < kBatch; ++k) v[k] = i + k * kThreads < n ? load1c<D>(row, i + k * kThreads) : 0.f;
}

template <class D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 8) k_rms_norm_loop(NormArgs a) {
  __shared__ float slots[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const unsigned char* xr = a.x + row * a.x_pitch;
    const unsigned char* hr = xr;
    LongSum squares;
    if (a.r) {
      const unsigned char* rr = a.r + row * a.r_pitch;
      unsigned char* to = a.h + row * a.h_pitch;
      hr = to;
      for (int64_t i = threadIdx.x; i < a.N;) {
        float part = 0.f;
        for (int j = 0; j < kPlain / kBatch && i < a.N; ++j, i += kBatch * kThreads) {
          float h[kBatch], r[kBatch];
          load_batch<D>(xr, i, a.N, h);
          load_batch<D>(rr, i, a.N, r);
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            h[k] = rounded<D>(h[k] + r[k]);
            if (i + k * kThreads < a.N) D::store1(to, i + k * kThreads, h[k]);
            part = __fmaf_rn(h[k], h[k], part);
          }
        }
        squares.add(part);
      }
    } else {
      for (int64_t i = threadIdx.x; i < a.N;) {
        float part = 0.f;
        for (int j = 0; j < kPlain / kBatch && i < a.N; ++j, i += kBatch * kThreads) {
          float h[kBatch];
          load_batch<D>(xr, i, a.N, h);
#pragma unroll
          for (int k = 0; k < kBatch; ++k) part = __fmaf_rn(h[k], h[k], part);
        }
        squares.add(part);
      }
    }
    const float sum = block_sum<kThreads / 32>(squares.s, slots);  // its barriers also order h's stores before the loads below
    const float rstd = 1.f / sqrtf(sum / float(a.N) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    unsigned char* yr = a.y + row * a.y_pitch;
    if constexpr (!E4M3) {
      for (int64_t i = threadIdx.x; i < a.N; i += kThreads) D::store1(yr, i, load1c<D>(hr, i) * rstd * weight1<D>(a, i));
    } else if (a.groups == 1 && a.N > kGroup) {
      const Parts p = parts_of(rstd);
      float top = 0.f;
      for (int64_t i = threadIdx.x; i < a.N; i += kThreads) top = fmaxf(top, fabsf(load1c<D>(hr, i) * p.two * weight1<D, true>(a, i)));
      top = block_max<kThreads / 32>(top, slots);
      float scale;
      const Codes c = codes_of(top, p, &scale);
      if (threadIdx.x == 0) a.scales[row] = scale;
      for (int64_t i = threadIdx.x; i < a.N; i += kThreads)
        yr[i] = (unsigned char)(pack_e4m3x2(quotient(load1c<D>(hr, i) * p.two * weight1<D, true>(a, i), c), 0.f) & 0xff);
    } else {
      const Parts p = parts_of(rstd);
      for (int64_t g = warp; g < a.groups; g += kThreads / 32) {
        float v[kGroup / 32], top = 0.f;
#pragma unroll
        for (int k = 0; k < kGroup / 32; ++k) {
          const int64_t i = g * kGroup + k * 32 + lane;
          v[k] = i < a.N ? load1c<D>(hr, i) * p.two * weight1<D, true>(a, i) : 0.f;
          top = fmaxf(top, fabsf(v[k]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        float scale;
        const Codes c = codes_of(top, p, &scale);
        if (lane == 0) a.scales[row * a.groups + g] = scale;
#pragma unroll
        for (int k = 0; k < kGroup / 32; ++k) {
          const int64_t i = g * kGroup + k * 32 + lane;
          if (i < a.N) yr[i] = (unsigned char)(pack_e4m3x2(quotient(v[k], c), 0.f) & 0xff);
        }
      }
    }
  }
}

// dx alone, two reads of the row.
template <class D>
__global__ void __launch_bounds__(kThreads, 8) k_rms_grad_loop(GradArgs a) {
  __shared__ float slots[32];
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const unsigned char* dr = a.dy + row * a.dy_pitch;
    const unsigned char* hr = a.h + row * a.h_pitch;
    const unsigned char* sr = a.sg + row * a.sg_pitch;
    unsigned char* to = a.dx + row * a.dx_pitch;
    const float rstd = a.rstd[row];
    LongSum sum;
    for (int64_t i = threadIdx.x; i < a.N;) {
      float part = 0.f;
      for (int j = 0; j < kPlain / kBatch && i < a.N; ++j, i += kBatch * kThreads) {
        float d[kBatch], h[kBatch];
        load_batch<D>(dr, i, a.N, d);
        load_batch<D>(hr, i, a.N, h);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i + k * kThreads < a.N) part = __fmaf_rn(d[k] * weight1<D>(a, i + k * kThreads), h[k] * rstd, part);
      }
      sum.add(part);
    }
    const float mean = block_sum<kThreads / 32>(sum.s, slots) / float(a.N);
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
// W warps own a row, K vectors a thread; a warp's 32 K vectors lie together.  SHIFT: rows that start anywhere, of any length
// (load_vectors, store_vectors); without, rows are on 16-byte boundaries.  The 128 elements that share a scale in 8 bits lie in
// one warp.

template <int K>
__device__ __forceinline__ int unit_of(int t, int k) {
  return (t >> 5) * (32 * K) + k * 32 + (t & 31);
}
template <class D, int K, bool SHIFT>
__device__ __forceinline__ void take(const RowAt& r, int t, int units, uint4 (&q)[K]) {
  if constexpr (SHIFT) {
    load_vectors<D>(r, unit_of<K>(t, 0), q);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = unit_of<K>(t, k);
      q[k] = u < units ? ld_stream16(r.row + int64_t(u) * 16) : make_uint4(0, 0, 0, 0);
    }
  }
}
template <class D, int K, bool SHIFT>
__device__ __forceinline__ void put(unsigned char* row, int t, int units, int n, const uint4 (&q)[K]) {
  if constexpr (SHIFT) {
    store_vectors<D>(row, unit_of<K>(t, 0), n, q);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = unit_of<K>(t, k);
      if (u < units) st_stream16(row + int64_t(u) * 16, q[k]);
    }
  }
}

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

// The factors weight + offset of vector u (into 8 bits, kSeven times them), 0 behind the row's end.
template <class D, bool SHIFT, bool E4M3 = false, class A>
__device__ __forceinline__ void weights(const A& a, int u, float (&w)[D::kVec]) {
  constexpr int E = D::kVec;
  const int left = SHIFT ? int(a.N) - u * E : E;
  if (!a.w) {
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = e < left ? (E4M3 ? kSeven : 1.f) : 0.f;
    return;
  }
  if (SHIFT && (left < E || !a.w_vec)) {
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = e < left ? weight1<D, E4M3>(a, int64_t(u) * E + e) : 0.f;
    return;
  }
  if (a.w_f32 && D::kBytes == 2) {
    const float4* p = static_cast<const float4*>(a.w) + 2 * u;
    const float4 lo = __ldg(p), hi = __ldg(p + 1);
    w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
    w[E - 4] = hi.x, w[E - 3] = hi.y, w[E - 2] = hi.z, w[E - 1] = hi.w;
  } else {
    D::unpack(__ldg(static_cast<const uint4*>(a.w) + u), w);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = factor<E4M3>(a, w[e]);
}

// The codes of vector u, left elements of it.
template <int E, bool SHIFT>
__device__ __forceinline__ void store_codes(unsigned char* row, int u, int left, const float2 (&v)[E / 2], const Codes& codes) {
  uint16_t c[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    const float2 q = quotient2(v[e], codes);
    c[e] = pack_e4m3x2(q.x, q.y);
  }
  unsigned char* p = row + int64_t(u) * E;
  if (SHIFT && (left < E || (reinterpret_cast<uintptr_t>(p) & (E - 1)))) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < left) p[e] = (unsigned char)(c[e / 2] >> (e & 1) * 8);
  } else if constexpr (E == 8) {
    asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(c[0] | uint32_t(c[1]) << 16), "r"(c[2] | uint32_t(c[3]) << 16) : "memory");
  } else {
    *reinterpret_cast<uint32_t*>(p) = c[0] | uint32_t(c[1]) << 16;
  }
}

__host__ __device__ constexpr int reg_threads(int warps) { return warps * 32 > 256 ? warps * 32 : 256; }

// CTAs of 256 threads an SM: in 8 bits three for 16-bit rows (16384 x 4096 bf16 with a residual 75 us; when it took 74, two 101, four 97), else
// four (16384 x 8192 bf16 86 us; when it took 84, three 93, six 91).
template <class D, int K, int W, bool SHIFT, bool E4M3>
__global__ void __launch_bounds__(reg_threads(W), (K > 4 ? 2 : E4M3 && D::kBytes == 2 ? 3 : 4) * 256 / reg_threads(W)) k_rms_norm(NormArgs a) {
  constexpr int E = D::kVec, GT = W * 32, G = reg_threads(W) / GT;
  __shared__ float sums[2][reg_threads(W) / 32], tops[2][reg_threads(W) / 32];
  const int group = threadIdx.x / GT, t = threadIdx.x % GT, lane = t & 31;
  const int n = int(a.N), units = (n + E - 1) / E;
  const int64_t bytes = a.N * D::kBytes;
  const Bytes xm = bytes_of(a.x, a.M, a.x_pitch, bytes), rm = bytes_of(a.r, a.M, a.r_pitch, bytes);
  constexpr bool PACKED = !SHIFT && E4M3;
  const bool packed = a.w && !(a.w_f32 && D::kBytes == 2);
  int it = 0;
  for (int64_t row = int64_t(blockIdx.x) * G + group; row < a.M; row += int64_t(gridDim.x) * G, it ^= 1) {
    const RowAt xr = row_at<D>(a.x + row * a.x_pitch, n, xm);
    uint4 h[K];
    take<D, K, SHIFT>(xr, t, units, h);
    if (a.r) {
      const RowAt rr = row_at<D>(a.r + row * a.r_pitch, n, rm);
      unsigned char* to = a.h + row * a.h_pitch;
      uint4 r[K];
      take<D, K, SHIFT>(rr, t, units, r);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float v[E], w[E];
        D::unpack(h[k], v);
        D::unpack(r[k], w);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] += w[e];
        h[k] = D::pack(v);
      }
      put<D, K, SHIFT>(to, t, units, n, h);
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[E];
      D::unpack(h[k], v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum = __fmaf_rn(v[e], v[e], sum);
    }
    uint4 wq[K];  // the weights as they are, under way while the sum is joined (in 8 bits: 164 us against 198)
    if (PACKED && packed) {
#pragma unroll
      for (int k = 0; k < K; ++k) wq[k] = __ldg(static_cast<const uint4*>(a.w) + min(unit_of<K>(t, k), units - 1));
    }
    sum = group_sum<W>(sum, sums[it] + group * W, group, t);
    const float rstd = 1.f / sqrtf(sum / float(a.N) + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    unsigned char* yr = a.y + row * a.y_pitch;
    if constexpr (!E4M3) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float v[E], w[E];
        D::unpack(h[k], v);
        weights<D, SHIFT>(a, min(unit_of<K>(t, k), units - 1), w);  // h is 0 behind the end
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = v[e] * rstd * w[e];
        h[k] = D::pack(v);
      }
      put<D, K, SHIFT>(yr, t, units, n, h);
    } else {
      const Parts p = parts_of(rstd);
      const float2 two = make_float2(p.two, p.two), seven = make_float2(kSeven, kSeven), offset = make_float2(kSeven * a.offset, kSeven * a.offset);
      const auto value = [&](int k, float2(&v)[E / 2]) {  // v of Codes, 0 behind the row's end
        float2 w[E / 2];
        if (PACKED && packed) {
          D::unpack2(wq[k], w);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) w[e] = __ffma2_rn(w[e], seven, offset);
        } else {
          float f[E];
          weights<D, SHIFT, true>(a, min(unit_of<K>(t, k), units - 1), f);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) w[e] = make_float2(f[2 * e], f[2 * e + 1]);
        }
        D::unpack2(h[k], v);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) v[e] = __fmul2_rn(__fmul2_rn(v[e], two), w[e]);
      };
      const auto top_of = [&](const float2(&v)[E / 2]) {
        float m = fmaxf(fabsf(v[0].x), fabsf(v[0].y));
#pragma unroll
        for (int e = 1; e < E / 2; ++e) m = fmaxf(m, fmaxf(fabsf(v[e].x), fabsf(v[e].y)));
        return m;
      };
      const auto store = [&](int k, const float2(&v)[E / 2], const Codes& c) {
        const int u = unit_of<K>(t, k);
        if (u < units) store_codes<E, SHIFT>(yr, u, n - u * E, v, c);
      };
      if (a.groups == 1 && a.N > kGroup) {
        float2 y[K][E / 2];
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          value(k, y[k]);
          top = fmaxf(top, top_of(y[k]));
        }
        top = group_max<W>(top, tops[it] + group * W, group, t);
        float scale;
        const Codes c = codes_of(top, p, &scale);
        if (t == 0) a.scales[row] = scale;
#pragma unroll
        for (int k = 0; k < K; ++k) store(k, y[k], c);
      } else {
        constexpr int lanes = kGroup / E, per = 32 / lanes;  // of a group; groups of a warp's 32 vectors
        float mine = 0.f;  // lane i: scale i of the warp's
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float2 y[E / 2];
          value(k, y);
          float top = top_of(y);
#pragma unroll
          for (int o = lanes >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
          float scale;
          const Codes c = codes_of(top, p, &scale);
          const float theirs = __shfl_sync(~0u, scale, (lane & (per - 1)) * lanes);
          if (lane / per == k) mine = theirs;
          store(k, y, c);
        }
        // one store for the warp's groups, which lie together: by twos, as they came, 16384 x 8192 took 163 us instead of 144
        const int g = unit_of<K>(t - lane, 0) / lanes + lane;
        if (lane < K * per && g < a.groups) a.scales[row * a.groups + g] = mine;
      }
    }
  }
}

// Forward into the element type for rows of x on no boundary (and a residual that starts at the same place of its 16-byte lines).  As
// that place comes again after 16 bytes' worth of rows, and a CTA's turns are a multiple of those apart, it is one for all rows of a group: lines
// are worked on where they are, and the weights lie moved in shared memory, each thread's for itself.  Taken by what is read alone:
// a call in place gives the bits of one that is not.  16384 x 5003 bf16 with a residual 130 us (lines shifted in registers, for single rows, 243), 65536 x 333 fp32 71.
template <class D, int K>
constexpr int lines_shared(int threads) { return threads * K * D::kVec * 4; }
constexpr int lines_ctas(int K, int threads) { return (K > 4 ? 2 : 4) * 256 / threads; }

template <class D, int K, int W>
__global__ void __launch_bounds__(reg_threads(W), lines_ctas(K, reg_threads(W))) k_rms_norm_lines(NormArgs a) {
  constexpr int E = D::kVec, GT = W * 32, T = reg_threads(W), G = T / GT;
  extern __shared__ float4 held[];  // [K][E / 4][T]
  __shared__ float sums[2][T / 32];
  const int group = threadIdx.x / GT, t = threadIdx.x % GT, n = int(a.N);
  const int64_t bytes = a.N * D::kBytes;
  const Bytes xm = bytes_of(a.x, a.M, a.x_pitch, bytes), rm = bytes_of(a.r, a.M, a.r_pitch, bytes);
  int64_t row = int64_t(blockIdx.x) * G + group;
  const int from = int(reinterpret_cast<uintptr_t>(a.x + row * a.x_pitch) & 15) / D::kBytes, end = from + n, units = (end + E - 1) / E;
  const auto whole = [&](int u) { return u * E >= from && u * E + E <= end; };
  const auto load = [&](const RowAt& r, uint4 (&q)[K]) {
    const unsigned char* p = r.row - r.delta;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = t + k * GT;
      q[k] = make_uint4(0, 0, 0, 0);
      if (u < units) q[k] = whole(u) || r.inside ? ld_stream16(p + int64_t(u) * 16) : load_elements<D>(p + int64_t(u) * 16, r.row, r.end);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = t + k * GT;
      if (u < units && !whole(u)) q[k] = keep<D>(q[k], from - u * E, end - u * E, 0);
    }
  };
  const auto store = [&](unsigned char* to, int k, const uint4& q) {
    const int u = t + k * GT, lane = t & 31, u0 = u - lane;
    unsigned char* p = to - from * D::kBytes + int64_t(u) * 16;
    if (reinterpret_cast<uintptr_t>(p) & 15 && u0 * E >= from && (u0 + 32) * E <= end) {  // an output that starts elsewhere: a warp's vectors
      const uint4 one[1] = {q};
      store_vectors<D>(p - lane * 16, lane, 32 * E, one);
    } else if (u < units) {
      if (!(reinterpret_cast<uintptr_t>(p) & 15) && whole(u)) st_stream16(p, q);
      else store_elements<D>(p, q, from - u * E, end - u * E);
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int b = (t + k * GT) * E;
    float w[E];
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = b + e >= from && b + e < end ? weight1<D>(a, b + e - from) : 0.f;
#pragma unroll
    for (int i = 0; i < E / 4; ++i) held[(k * (E / 4) + i) * T + threadIdx.x] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  int it = 0;
  for (; row < a.M; row += int64_t(gridDim.x) * G, it ^= 1) {
    uint4 h[K];
    load(row_at<D>(a.x + row * a.x_pitch, n, xm), h);
    if (a.r) {
      uint4 r[K];
      load(row_at<D>(a.r + row * a.r_pitch, n, rm), r);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float v[E], w[E];
        D::unpack(h[k], v);
        D::unpack(r[k], w);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] += w[e];
        h[k] = D::pack(v);
        store(a.h + row * a.h_pitch, k, h[k]);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[E];
      D::unpack(h[k], v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum = __fmaf_rn(v[e], v[e], sum);
    }
    sum = group_sum<W>(sum, sums[it] + group * W, group, t);
    const float rstd = 1.f / sqrtf(sum / float(a.N) + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[E];
      D::unpack(h[k], v);
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 w = held[(k * (E / 4) + i) * T + threadIdx.x];
        v[4 * i] = v[4 * i] * rstd * w.x, v[4 * i + 1] = v[4 * i + 1] * rstd * w.y;
        v[4 * i + 2] = v[4 * i + 2] * rstd * w.z, v[4 * i + 3] = v[4 * i + 3] * rstd * w.w;
      }
      store(a.y + row * a.y_pitch, k, D::pack(v));
    }
  }
}

// Backward: every CTA walks its rows with the columns' sums of dw in registers, and leaves them as one part.  h is multiplied by rstd before
// dy meets it, and rstd stands before no power of itself: h dy and rstd^3 leave fp32's range long before xhat dy and rstd do (of
// rows of magnitude 1e15 rstd^3 is 0, and dx would lose all of its second term).
template <class D, int K, int W, bool SHIFT>
__global__ void __launch_bounds__(reg_threads(W)) k_rms_grad(GradArgs a) {
  constexpr int E = D::kVec, GT = W * 32, G = reg_threads(W) / GT;
  __shared__ float sums[2][reg_threads(W) / 32];
  __shared__ float columns[G > 1 ? K * E * GT : 1];
  const int group = threadIdx.x / GT, t = threadIdx.x % GT;
  const int n = int(a.N), units = (n + E - 1) / E;
  const int64_t step = int64_t(gridDim.x) * G, bytes = a.N * D::kBytes;
  const Bytes dm = bytes_of(a.dy, a.M, a.dy_pitch, bytes), hm = bytes_of(a.h, a.M, a.h_pitch, bytes), gm = bytes_of(a.sg, a.M, a.sg_pitch, bytes);
  float dw[K][E] = {};
  int it = 0;
  for (int64_t row = int64_t(blockIdx.x) * G + group; row < a.M; row += step, it ^= 1) {
    uint4 dy[K], h[K], sg[K];
    const RowAt dr = row_at<D>(a.dy + row * a.dy_pitch, n, dm), hr = row_at<D>(a.h + row * a.h_pitch, n, hm), gr = row_at<D>(a.sg + row * a.sg_pitch, n, gm);
    take<D, K, SHIFT>(dr, t, units, dy);
    take<D, K, SHIFT>(hr, t, units, h);
    if (a.sg) {
      take<D, K, SHIFT>(gr, t, units, sg);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) sg[k] = make_uint4(0, 0, 0, 0);
    }
    const float rstd = a.rstd[row];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = unit_of<K>(t, k);
      if (u >= units) continue;
      float d[E], x[E], w[E];
      D::unpack(dy[k], d);
      D::unpack(h[k], x);
      weights<D, SHIFT>(a, u, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float p = d[e] * (x[e] * rstd);
        sum = __fmaf_rn(p, w[e], sum);
        dw[k][e] += p;
      }
    }
    sum = group_sum<W>(sum, sums[it] + group * W, group, t);  // and every load of the row is done
    const float slope = -rstd * (sum / float(a.N));
    unsigned char* to = a.dx + row * a.dx_pitch;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = unit_of<K>(t, k);
      float d[E], x[E], w[E] = {}, s[E];
      D::unpack(dy[k], d);
      D::unpack(h[k], x);
      D::unpack(sg[k], s);
      if (u < units) weights<D, SHIFT>(a, u, w);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = __fmaf_rn(rstd, __fmaf_rn(slope, x[e], d[e] * w[e]), s[e]);
      dy[k] = D::pack(d);
    }
    put<D, K, SHIFT>(to, t, units, n, dy);
  }
  griddep_launch();
  if (!a.dw) return;
  float* part = a.parts + blockIdx.x * a.N;
  for (int g = 0; g < G; ++g) {  // the groups' sums one after the other
    if (group == g) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = unit_of<K>(t, k);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float* c = columns + (G > 1 ? (k * E + e) * GT + t : 0);
          const float v = g ? *c + dw[k][e] : dw[k][e];
          if (g < G - 1) *c = v;
          else if (u * E + e < n) part[u * E + e] = v;
        }
      }
    }
    __syncthreads();
  }
}

// The same with the rows on their way in shared memory: a slot has the G rows of dy, h and sum_grad that the CTA's groups take
// next, copied by cp.async.bulk, and is read twice.  The copies of up to kMostSlots turns are under way while one is worked on,
// whatever the registers leave of the SM's warps: 16384 x 4096 bf16 takes 85 us; when it took 88, with the rows in registers 103 (at the best
// number of CTAs an SM).  Arithmetic in pairs of fp32: with single operations, 104 us.
// LINES: rows on no boundary, which start at the same place of their 16-byte lines in all matrices.  That place comes again
// after 16 bytes' worth of rows, and a CTA's turns are a multiple of those apart: it is one for all rows of a group, so lines are
// worked on where they are, with the weights and the sums of dw moved instead (16384 x 5003 bf16 151 us; vectors shifted out of the
// slots' lines 237, out of lines in registers 384).
constexpr int kMostSlots = 4;
constexpr int kStaticShared = 1024;  // more than these kernels have

struct RingArgs {
  GradArgs g;
  int slots;  // at least 2
  uint32_t row_bytes, slot_row, slot_bytes;  // slot_row: from row to row of a slot
  unsigned* status;
  uint64_t wait_ns;
};

// A lane's row with LINES: the 16-byte lines that it has a part in, to their places from `to` on.  Where not all of them lie inside
// the matrix, the first and the last one's elements are read by themselves.  Returns the bytes to copy, and what from.
template <class D>
__device__ __forceinline__ uint32_t edges(const RowAt& r, uint32_t& to, const unsigned char*& from) {
  const unsigned char* end = r.end + (-reinterpret_cast<uintptr_t>(r.end) & 15);
  from = r.row - r.delta;
  if (!r.inside) {
    sts16(to, load_elements<D>(from, r.row, r.end));
    if (end - from > 16) sts16(to + uint32_t(end - from) - 16, load_elements<D>(end - 16, r.row, r.end));
    from += 16, to += 16, end -= 16;
  }
  return end > from ? uint32_t(end - from) : 0;
}

// Vector u of a row in a slot, whose elements are the from-th to the end-th of its lines; 0 around them.
template <class D, bool LINES>
__device__ __forceinline__ uint4 slot_vector(uint32_t row, int u, int from, int end) {
  const uint4 q = lds16(row + u * 16);
  if constexpr (!LINES) return q;
  const int b = u * D::kVec;
  return b < from || b + D::kVec > end ? keep<D>(q, from - b, end - b, 0) : q;
}

template <class D, int K, int W, bool LINES>
__global__ void __launch_bounds__(reg_threads(W), 512 / reg_threads(W)) k_rms_grad_ring(RingArgs r) {
  constexpr int E = D::kVec, GT = W * 32, G = reg_threads(W) / GT;
  extern __shared__ __align__(128) unsigned char shared[];
  __shared__ uint64_t full[kMostSlots];
  __shared__ float sums[2][reg_threads(W) / 32];
  const GradArgs& a = r.g;
  const int tid = threadIdx.x, group = tid / GT, t = tid % GT;
  const int n = int(a.N);
  int64_t row = int64_t(blockIdx.x) * G + group;
  const int from = LINES ? int(reinterpret_cast<uintptr_t>(a.dy + row * a.dy_pitch) & 15) / D::kBytes : 0, end = from + n, units = (end + E - 1) / E;
  const Bytes dm = bytes_of(a.dy, a.M, a.dy_pitch, r.row_bytes), hm = bytes_of(a.h, a.M, a.h_pitch, r.row_bytes), gm = bytes_of(a.sg, a.M, a.sg_pitch, r.row_bytes);
  const int64_t turns = (a.M + G - 1) / G, mine = turns > blockIdx.x ? (turns - 1 - blockIdx.x) / gridDim.x + 1 : 0;
  const uint64_t policy = policy_evict_first();
  bool timed_out = false;

  const auto fetch = [&](int64_t i) {  // turn i of this CTA, by warp 0
    const int s = int(i % r.slots), arrays = a.sg ? 3 : 2;
    const int64_t row0 = (blockIdx.x + i * gridDim.x) * G;
    const int rows = int(a.M - row0 < G ? a.M - row0 : G);
    const uint32_t bar = smem_addr(&full[s]), slot = smem_addr(shared) + s * r.slot_bytes;
    const int which = tid / rows, row = tid % rows;
    const unsigned char* at = which == 0   ? a.dy + (row0 + row) * a.dy_pitch
                              : which == 1 ? a.h + (row0 + row) * a.h_pitch
                                           : a.sg + (row0 + row) * a.sg_pitch;
    uint32_t to = slot + uint32_t(which * G + row) * r.slot_row, bytes = r.row_bytes, all = uint32_t(rows * arrays) * r.row_bytes;
    if constexpr (LINES) {
      bytes = 0;
      if (tid < rows * arrays) bytes = edges<D>(row_at<D>(at, n, which == 0 ? dm : which == 1 ? hm : gm), to, at);
      all = __reduce_add_sync(~0u, bytes);
      fence_proxy_async_smem();  // elements stored here, now or in an earlier turn, before what is copied over them
      __syncwarp();              // and before the arrival
    }
    if (tid == 0) mbar_arrive_expect_tx(bar, all);
    __syncwarp();
    if (tid < rows * arrays && bytes > 0) bulk_g2s(to, at, bytes, bar, policy);
  };
  if (tid == 0) {
    for (int s = 0; s < r.slots; ++s) mbar_init(smem_addr(&full[s]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (tid < 32)
    for (int64_t i = 0; i < r.slots && i < mine; ++i) fetch(i);
  float2 w[K][E / 2], dw[K][E / 2];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float f[E] = {};
    const int u = t + k * GT;
    if constexpr (LINES) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = u * E + e >= from && u * E + e < end ? weight1<D>(a, u * E + e - from) : 0.f;
    } else {
      if (u < units) weights<D, false>(a, u, f);
    }
#pragma unroll
    for (int e = 0; e < E / 2; ++e) w[k][e] = make_float2(f[2 * e], f[2 * e + 1]), dw[k][e] = make_float2(0.f, 0.f);
  }
  const int64_t step = int64_t(gridDim.x) * G;
  float next_rstd = row < a.M ? a.rstd[row] : 0.f;
  int s = 0;
  uint32_t parity = 0;
  for (int64_t i = 0; i < mine; ++i, row += step) {
    const float rstd = next_rstd;
    if (row + step < a.M) next_rstd = a.rstd[row + step];
    const uint32_t dys = smem_addr(shared) + s * r.slot_bytes + group * r.slot_row, hs = dys + G * r.slot_row, sgs = hs + G * r.slot_row;
    const bool on = row < a.M;
    if (!mbar_wait(smem_addr(&full[s]), parity, r.wait_ns)) timed_out = true;
    const float2 rstd2 = make_float2(rstd, rstd);
    float2 sum2 = make_float2(0.f, 0.f);  // of g xhat
    if (on) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = t + k * GT;
        if (u >= units) continue;
        float2 d[E / 2], x[E / 2];
        D::unpack2(slot_vector<D, LINES>(dys, u, from, end), d);
        D::unpack2(slot_vector<D, LINES>(hs, u, from, end), x);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float2 p = __fmul2_rn(d[e], __fmul2_rn(x[e], rstd2));
          sum2 = __ffma2_rn(p, w[k][e], sum2);
          dw[k][e] = __fadd2_rn(dw[k][e], p);
        }
      }
    }
    float sum = sum2.x + sum2.y;
    // the barrier here also says that every thread is done with the turn before: its slot is refilled
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    float* const slots = sums[i & 1] + group * W;
    if ((t & 31) == 0) slots[t >> 5] = sum;
    __syncthreads();
    if (tid < 32 && i > 0 && i - 1 + r.slots < mine) fetch(i - 1 + r.slots);
    if constexpr (W > 1) {
      sum = slots[t & (W - 1)];
#pragma unroll
      for (int o = W >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    }
    if (on) {
      const float slope = -rstd * (sum / float(a.N));  // dx = rstd (g + slope h) + sum_grad
      const float2 slope2 = make_float2(slope, slope);
      unsigned char* to = a.dx + row * a.dx_pitch - from * D::kBytes;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = t + k * GT;
        if (u >= units) continue;
        float2 d[E / 2], x[E / 2], g[E / 2] = {};
        D::unpack2(slot_vector<D, LINES>(dys, u, from, end), d);
        D::unpack2(slot_vector<D, LINES>(hs, u, from, end), x);
        if (a.sg) D::unpack2(slot_vector<D, LINES>(sgs, u, from, end), g);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) d[e] = __ffma2_rn(__ffma2_rn(x[e], slope2, __fmul2_rn(d[e], w[k][e])), rstd2, g[e]);
        const int first = from - u * E, last = end - u * E;
        if (LINES && (first > 0 || last < E)) store_elements<D>(to + int64_t(u) * 16, D::pack2(d), first, last);
        else st_stream16(to + int64_t(u) * 16, D::pack2(d));
      }
    }
    if (++s == r.slots) {
      s = 0;
      parity ^= 1;
    }
  }
  if (timed_out) atomicOr(r.status, kStatusTimeout);
  griddep_launch();
  if (!a.dw) return;
  float* part = a.parts + blockIdx.x * a.N;
  // the groups' sums one after the other, where the slots were
  __syncthreads();
  float* columns = reinterpret_cast<float*>(shared);
  for (int g = 0; g < G; ++g) {
    if (group == g) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = t + k * GT;
        if (u >= units) continue;
        if constexpr (LINES) {  // the groups' rows start elsewhere in their lines
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int i = u * E + e - from;
            if (i < 0 || i >= n) continue;
            const float v = (e & 1 ? dw[k][e / 2].y : dw[k][e / 2].x) + (g ? columns[i] : 0.f);
            (g == G - 1 ? part : columns)[i] = v;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            float4 v = make_float4(dw[k][e / 2].x, dw[k][e / 2].y, dw[k][e / 2 + 1].x, dw[k][e / 2 + 1].y);
            float4* c = reinterpret_cast<float4*>(columns + u * E + e);
            if (g) v.x += c->x, v.y += c->y, v.z += c->z, v.w += c->w;
            *(g == G - 1 ? reinterpret_cast<float4*>(part + u * E + e) : c) = v;
          }
        }
      }
    }
    if constexpr (G > 1) __syncthreads();
  }
}

// dw = the parts added up: 32 columns a CTA, its warps every 32nd part.
constexpr int kJoinThreads = 1024, kAtOnce = 10;  // parts that a warp has under way: all of 304
__global__ void __launch_bounds__(kJoinThreads) k_rms_weight_join(GradArgs a) {
  __shared__ float sums[kJoinThreads / 32][33];
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = int64_t(blockIdx.x) * 32 + lane;
  float sum = 0.f;
  if (i < a.N) {
    for (int k0 = warp; k0 < a.parts_n; k0 += kAtOnce * (kJoinThreads / 32)) {
      float v[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int k = k0 + j * (kJoinThreads / 32);
        v[j] = k < a.parts_n ? a.parts[k * a.N + i] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) sum += v[j];
    }
  }
  sums[warp][lane] = sum;
  __syncthreads();
  // warp w: column w's sums over the warps
  sum = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  const int64_t c = int64_t(blockIdx.x) * 32 + warp;
  if (lane == 0 && c < a.N) a.dw[c] = a.accumulate ? a.dw[c] + sum : sum;
}

struct NormConfig {
  int warps, units;            // warps a row, units they hold
  void (*fn[2])(NormArgs);     // [e4m3]
};
template <class D, int K, int W, bool SHIFT>
constexpr NormConfig norm_cfg() {
  return NormConfig{W, 32 * W * K, {k_rms_norm<D, K, W, SHIFT, false>, k_rms_norm<D, K, W, SHIFT, true>}};
}
struct GradConfig {
  int warps, units;
  void (*fn)(GradArgs);
};
template <class D, int K, int W, bool SHIFT>
constexpr GradConfig grad_cfg() {
  return GradConfig{W, 32 * W * K, k_rms_grad<D, K, W, SHIFT>};
}
struct RingConfig {
  int warps, units;
  void (*fn)(RingArgs);
};
template <class D, int K, int W, bool LINES>
constexpr RingConfig ring_cfg() {
  return RingConfig{W, 32 * W * K, k_rms_grad_ring<D, K, W, LINES>};
}

struct LinesConfig {
  int warps, units, shared, ctas;
  void (*fn)(NormArgs);
};
template <class D, int K, int W>
constexpr LinesConfig lines_cfg() {
  return LinesConfig{W, 32 * W * K, lines_shared<D, K>(reg_threads(W)), lines_ctas(K, reg_threads(W)), k_rms_norm_lines<D, K, W>};
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
  static const NormConfig aligned[] = {norm_cfg<D, 1, 1, false>(), norm_cfg<D, 2, 1, false>(), norm_cfg<D, 4, 1, false>(), norm_cfg<D, 4, 2, false>(),
                                       norm_cfg<D, 3, 4, false>(), norm_cfg<D, 4, 4, false>(), norm_cfg<D, 3, 8, false>(), norm_cfg<D, 4, 8, false>(), norm_cfg<D, 4, 16, false>(), norm_cfg<D, 8, 16, false>()};
  static const NormConfig anywhere[] = {norm_cfg<D, 1, 1, true>(), norm_cfg<D, 4, 1, true>(), norm_cfg<D, 4, 4, true>(), norm_cfg<D, 4, 8, true>(),
                                        norm_cfg<D, 4, 16, true>(), norm_cfg<D, 8, 16, true>()};
  static const LinesConfig lined[] = {lines_cfg<D, 1, 1>(), lines_cfg<D, 2, 1>(), lines_cfg<D, 4, 1>(), lines_cfg<D, 4, 2>(), lines_cfg<D, 4, 4>(),
                                      lines_cfg<D, 3, 8>(), lines_cfg<D, 4, 8>(), lines_cfg<D, 4, 16>(), lines_cfg<D, 8, 16>()};
  const bool e4m3 = p.out == RMS_NORM_OUT_E4M3;
  // codes of a vector are 8 or 4 bytes: half or a quarter of what the element types need
  const uintptr_t code = e4m3 ? 16 / D::kVec : 1;
  const bool vec = on16({bits(a.x), bits(a.r), bits(a.h), bits(a.y) * code, bits(static_cast<const char*>(a.w)), uintptr_t(a.x_pitch),
                         a.r ? uintptr_t(a.r_pitch | a.h_pitch) : 0, uintptr_t(a.y_pitch) * code, uintptr_t(p.N * D::kBytes)});
  const int64_t units = (p.N + D::kVec - 1) / D::kVec;
  const NormConfig* c = vec ? pick(aligned, units) : pick(anywhere, units);
  const bool lines = !e4m3 && !on16({bits(a.x), uintptr_t(a.x_pitch)}) && (!a.r || !(((bits(a.r) ^ bits(a.x)) | uintptr_t(a.r_pitch ^ a.x_pitch)) & 15));
  if (const LinesConfig* l = lines ? pick(lined, (p.N + 2 * D::kVec - 2) / D::kVec) : nullptr) {
    const int threads = reg_threads(l->warps), groups = threads / 32 / l->warps;
    const int64_t ctas = (p.M + groups - 1) / groups, most = int64_t(dev.sm_count) * l->ctas / D::kVec * D::kVec;
    const cudaError_t e = allow_shared((const void*)l->fn, dev, kStaticShared);
    if (e != cudaSuccess) return e;
    l->fn<<<unsigned(ctas < most ? ctas : most), threads, size_t(l->shared), p.stream>>>(a);
  } else if (c) {
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
  static const RingConfig rings[] = {ring_cfg<D, F, 1, false>(), ring_cfg<D, 2 * F, 1, false>(), ring_cfg<D, 4 * F, 1, false>(), ring_cfg<D, 4 * F, 2, false>(),
                                     ring_cfg<D, 2 * F, 8, false>(), ring_cfg<D, 4 * F, 8, false>(), ring_cfg<D, 4 * F, 16, false>()};
  static const RingConfig lined[] = {ring_cfg<D, F, 1, true>(), ring_cfg<D, 2 * F, 1, true>(), ring_cfg<D, 4 * F, 1, true>(), ring_cfg<D, 4 * F, 2, true>(),
                                      ring_cfg<D, 2 * F, 8, true>(), ring_cfg<D, 4 * F, 8, true>(), ring_cfg<D, 4 * F, 16, true>()};
  static const GradConfig aligned[] = {grad_cfg<D, 4 * F, 16, false>()};  // two slots of such rows may not fit an SM
  static const GradConfig anywhere[] = {grad_cfg<D, F, 1, true>(), grad_cfg<D, 2 * F, 2, true>(), grad_cfg<D, 2 * F, 8, true>(), grad_cfg<D, 4 * F, 8, true>(),
                                        grad_cfg<D, 4 * F, 16, true>()};
  const bool vec = on16({bits(a.dy), bits(a.h), bits(a.sg), bits(a.dx), bits(static_cast<const char*>(a.w)), uintptr_t(a.dy_pitch), uintptr_t(a.h_pitch),
                         a.sg ? uintptr_t(a.sg_pitch) : 0, uintptr_t(a.dx_pitch), uintptr_t(p.N * D::kBytes)});
  const int64_t units = (p.N + D::kVec - 1) / D::kVec;
  // all rows of a number start at the same place of their 16-byte lines
  const auto same = [&](const unsigned char* q, int64_t pitch) { return ((bits(q) ^ bits(a.dy)) & 15) == 0 && ((pitch ^ a.dy_pitch) & 15) == 0; };
  const bool lines = same(a.h, a.h_pitch) && (!a.sg || same(a.sg, a.sg_pitch)) && same(a.dx, a.dx_pitch);
  const RingConfig* ring = vec ? pick(rings, units) : lines ? pick(lined, (p.N + 2 * D::kVec - 2) / D::kVec) : nullptr;
  RingArgs r;
  int ring_ctas = 0, shared = 0;  // of an SM
  if (ring) {
    const int threads = reg_threads(ring->warps), groups = threads / 32 / ring->warps, arrays = a.sg ? 3 : 2;
    r.row_bytes = uint32_t(p.N * D::kBytes);
    r.slot_row = vec ? r.row_bytes : (r.row_bytes + 15) / 16 * 16 + 16;  // lines that a row has parts in
    r.slot_bytes = r.slot_row * uint32_t(groups * arrays);
    const auto slots = [&](int ctas) { return (dev.max_smem_per_sm / ctas - 1024 - kStaticShared) / int(r.slot_bytes); };
    for (ring_ctas = 512 / threads; ring_ctas > 1 && slots(ring_ctas) < 2;) --ring_ctas;
    r.slots = slots(ring_ctas) < kMostSlots ? slots(ring_ctas) : kMostSlots;
    shared = r.slots * int(r.slot_bytes);
    if (r.slots < 2) ring = nullptr;
  }
  const GradConfig* c = ring ? nullptr : vec ? pick(aligned, units) : pick(anywhere, units);
  const unsigned joins = unsigned((p.N + 31) / 32);
  if (p.M == 0) {
    a.parts_n = 0;
  } else if (ring) {
    const int threads = reg_threads(ring->warps), groups = threads / 32 / ring->warps;
    const int64_t turns = (p.M + groups - 1) / groups, most = int64_t(dev.sm_count) * ring_ctas / D::kVec * D::kVec;  // LINES' rows
    a.parts_n = int(turns < most ? turns : most);
    r.g = a;
    r.status = dev.status;
    r.wait_ns = local_wait_limit_ns();
    cudaError_t e = allow_shared((const void*)ring->fn, dev, kStaticShared);
    if (e != cudaSuccess) return e;
    ring->fn<<<unsigned(a.parts_n), threads, size_t(shared), p.stream>>>(r);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  } else if (c) {
    const int threads = reg_threads(c->warps), groups = threads / 32 / c->warps;
    const int64_t ctas = (p.M + groups - 1) / groups;
    const int64_t per_sm = threads > 256 ? 1 : 2;  // what the registers allow
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
    if (const cudaError_t e = launch_after(k_rms_weight_join, joins, kJoinThreads, p.stream, a); e != cudaSuccess) return e;
  }
  if (p.M > 0 && !c && !ring) k_rms_grad_loop<D><<<row_grid(p.M, dev), kThreads, 0, p.stream>>>(a);
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
  a.w_vec = (reinterpret_cast<uintptr_t>(a.w) & 15) == 0;
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
  a.w_vec = (reinterpret_cast<uintptr_t>(a.w) & 15) == 0;
  a.accumulate = p.a.accumulate != 0;
  return p.dtype == SOFTMAX_F32 ? launch_grad_type<F32>(p, a, dev) : p.dtype == SOFTMAX_BF16 ? launch_grad_type<BF16>(p, a, dev) : launch_grad_type<F16>(p, a, dev);
}

}  // namespace rwo
