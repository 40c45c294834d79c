// kernel_loss_grad.cu -- the cross-entropy loss of a row of logits and its gradient.
//
// With the row's online state (m, d), S = sum_j (m - x_j), label t, e = label smoothing, z the weight of LSE^2 and
// w = grad_scale * upstream:
//     LSE  = m + ln d
//     loss = (1 - e) (m - x_t) + e S / N + ln d + z LSE^2
//     grad_j = w (1 + 2 z LSE) / d * e^(x_j - m) - w e / N - [j = t] w (1 - e)
// so once (m, d, S) are known an element needs one exponential and one multiply-add.  S is taken relative to the
// maximum, as d is: m - x_j loses nothing where |m| is large.
#include "train.cuh"
#include "train.h"

namespace rwo {
namespace {

struct Args {
  const unsigned char* x;
  unsigned char* g;
  const int64_t* labels;
  const float* upstream;
  float* loss;
  float* lse;
  int64_t M, N;
  int64_t x_pitch, g_pitch;  // bytes
  float grad_scale, smoothing, z;
  unsigned* status;
};

// Part of a row: (m, d) of softmax, s = sum of (m - x) and n, how many elements (s and n with smoothing only).
struct Fold {
  float m, d, s, n;
};
__device__ __forceinline__ Fold empty_fold() { return Fold{-INFINITY, 0.f, 0.f, 0.f}; }

// s of a part, relative to a maximum mx >= its own.  Entries of -inf make s +inf; a part of nothing stays 0.
__device__ __forceinline__ float moved(const Fold& f, float mx) {
  return f.n > 0.f ? __fmaf_rn(f.n, mx - safe_max(f.m), f.s) : 0.f;
}

__device__ __forceinline__ Fold merge(const Fold& a, const Fold& b) {
  const State t = merge(State{a.m, a.d}, State{b.m, b.d});
  const float ms = safe_max(t.m);
  return Fold{t.m, t.d, __fadd_rn(moved(a, ms), moved(b, ms)), a.n + b.n};
}

template <bool SMOOTH>
__device__ __forceinline__ Fold warp_fold(Fold f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Fold t{__shfl_xor_sync(~0u, f.m, o), __shfl_xor_sync(~0u, f.d, o), 0.f, 0.f};
    if constexpr (SMOOTH) {
      t.s = __shfl_xor_sync(~0u, f.s, o);
      t.n = __shfl_xor_sync(~0u, f.n, o);
    }
    f = merge(f, t);
  }
  return f;
}

// What the elements of a row need once its state is known.
struct Slope {
  float ms;     // the maximum (0 for an empty row)
  float a;      // factor of e^(x - m)
  float b;      // subtracted from every element
  float c;      // and from the labelled one
  int64_t label;
  bool live;    // false: every element is 0
};

// One thread of a row passes write = true: it stores the loss and LSE and records a bad label.
__device__ __forceinline__ Slope slope_of(const Args& a, int64_t row, const Fold& f, int64_t label, float x_label, bool write) {
  Slope s;
  const float lnd = logf(f.d), lse = f.m + lnd;  // an empty row: -inf; NaN among -inf: NaN
  const bool bad = label >= a.N;
  const float w = a.grad_scale * (a.upstream ? a.upstream[row] : 1.f);
  s.ms = safe_max(f.m);
  s.a = bad ? __int_as_float(0x7fc00000) : w * (1.f + 2.f * a.z * lse) / f.d;
  s.b = w * (a.smoothing / float(a.N));
  s.c = w * (1.f - a.smoothing);
  s.label = label;
  s.live = label >= 0;
  if (write) {
    float l = 0.f;
    if (bad) {
      l = __int_as_float(0x7fc00000);
      atomicOr(a.status, kStatusBadLabel);
    } else if (label >= 0) {
      if (f.m == -INFINITY) {
        l = __int_as_float(0x7fc00000);
      } else {
        l = __fmaf_rn(1.f - a.smoothing, f.m - x_label, lnd);
        if (a.smoothing > 0.f) l = __fmaf_rn(a.smoothing, f.s / float(a.N), l);
        if (a.z > 0.f) l = __fmaf_rn(a.z * lse, lse, l);
      }
    }
    a.loss[row] = l;
    if (a.lse) a.lse[row] = lse;
  }
  return s;
}

__device__ __forceinline__ float grad_of(const Slope& s, float x) { return s.live ? __fmaf_rn(exp_diff(x, s.ms), s.a, -s.b) : 0.f; }

// ---- two passes, rows of any length and alignment ------------------------------------------------------------------

constexpr int kThreads = 512;

// A CTA a row: the fold, then the gradient from a second read.  VEC: 16-byte units, else single elements.
template <class D, bool VEC, bool SMOOTH>
__global__ void __launch_bounds__(kThreads) k_loss_grad_twopass(Args a) {
  constexpr int E = VEC ? D::kVec : 1;
  __shared__ Fold parts[2][kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t units = a.N / E;
  int it = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, it ^= 1) {
    const unsigned char* xr = a.x + row * a.x_pitch;
    unsigned char* gr = a.g + row * a.g_pitch;
    const int64_t label = a.labels[row];
    // read before any element is overwritten: the gradient may go where the logits are
    const float x_label = label >= 0 && label < a.N ? load1c<D>(xr, label) : 0.f;
    Fold f = empty_fold();
    float lost = 0.f;  // what the additions to f.d rounded away (long runs of a thread)
    for (int64_t u = threadIdx.x; u < units; u += kThreads) {
      float v[E];
      if constexpr (VEC) D::unpack(ld16(xr + u * 16), v);
      else v[0] = D::load1(xr, u);
      float mx = v[0];
#pragma unroll
      for (int e = 1; e < E; ++e) mx = fmaxf(mx, v[e]);
      if (mx > f.m) {
        const float k = exp_diff(f.m, mx);
        f.d *= k;
        lost *= k;
        if constexpr (SMOOTH) f.s = moved(f, mx);
        f.m = mx;
      }
      const float ms = safe_max(f.m);
      float t = 0.f, r = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        t += exp_diff(v[e], ms);
        if constexpr (SMOOTH) r += ms - v[e];
      }
      const float want = t - lost, sum = __fadd_rn(f.d, want);
      lost = __fsub_rn(__fsub_rn(sum, f.d), want);
      f.d = sum;
      if constexpr (SMOOTH) {
        f.s += r;
        f.n += float(E);
      }
    }
    f = warp_fold<SMOOTH>(f);
    if (lane == 0) parts[it][warp] = f;
    __syncthreads();
    f = warp_fold<SMOOTH>(lane < kThreads / 32 ? parts[it][lane] : empty_fold());
    const Slope s = slope_of(a, row, f, label, x_label, threadIdx.x == 0);
    for (int64_t u = threadIdx.x; u < units; u += kThreads) {
      float v[E];
      if constexpr (VEC) D::unpack(ld16(xr + u * 16), v);
      else v[0] = D::load1(xr, u);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[e] = grad_of(s, v[e]);
        if (s.live && u * E + e == s.label) v[e] -= s.c;
      }
      if constexpr (VEC) st_stream16(gr + u * 16, D::pack(v));
      else D::store1(gr, u, v[0]);
    }
  }
}

using Kernel = void (*)(Args);

template <class D>
cudaError_t launch_type(const LossGrad& p, Args a, const DeviceInfo& dev) {
  const bool smooth = p.smoothing > 0.f;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.g) | uintptr_t(a.x_pitch) | uintptr_t(a.g_pitch) |
                     uintptr_t(p.N * D::kBytes)) & 15) == 0;
  const Kernel k = vec ? (smooth ? k_loss_grad_twopass<D, true, true> : k_loss_grad_twopass<D, true, false>)
                       : (smooth ? k_loss_grad_twopass<D, false, true> : k_loss_grad_twopass<D, false, false>);
  const int64_t slots = int64_t(dev.sm_count) * (dev.max_threads_per_sm / kThreads);
  k<<<unsigned(p.M < slots ? p.M : slots), kThreads, 0, p.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_loss_grad(const LossGrad& p, const DeviceInfo& dev) {
  Args a;
  const int64_t s = elem_bytes(p.dtype);
  a.x = static_cast<const unsigned char*>(p.x);
  a.g = static_cast<unsigned char*>(p.grad);
  a.labels = p.labels;
  a.upstream = p.upstream;
  a.loss = p.loss;
  a.lse = p.lse;
  a.M = p.M;
  a.N = p.N;
  a.x_pitch = p.x_pitch * s;
  a.g_pitch = p.g_pitch * s;
  a.grad_scale = p.grad_scale;
  a.smoothing = p.smoothing;
  a.z = p.z;
  a.status = dev.status;
  return p.dtype == SOFTMAX_F32 ? launch_type<F32>(p, a, dev) : p.dtype == SOFTMAX_BF16 ? launch_type<BF16>(p, a, dev) : launch_type<F16>(p, a, dev);
}

}  // namespace rwo
