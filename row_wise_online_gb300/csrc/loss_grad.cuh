// loss_grad.cuh -- the cross-entropy loss of a row of logits and its gradient: what the kernels share.
//
// With the row's online state (m, d), S = sum_j (m - x_j), label t, e = label smoothing, z the weight of LSE^2 and
// w = grad_scale * upstream:
//     LSE  = m + ln d
//     loss = (1 - e) (m - x_t) + e S / N + ln d + z LSE^2
//     grad_j = w (1 + 2 z LSE) / d * e^(x_j - m) - w e / N - [j = t] w (1 - e)
// so once (m, d, S) are known an element needs one exponential and one multiply-add.  S is taken relative to the
// maximum, as d is: m - x_j loses nothing where |m| is large.
#pragma once

#include "train.cuh"
#include "train.h"

namespace rwo {

struct LossArgs {
  const unsigned char* x;
  unsigned char* g;
  const int64_t* labels;
  const float* upstream;
  float* loss;
  float* lse;
  int64_t M, N;
  int64_t x_pitch, g_pitch;  // bytes
  float grad_scale, smoothing, z;
  float smoothing_each;  // smoothing / N
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

// The parts that lanes 0 .. width - 1 hold (and every run of as many lanes alike), width a power of two: the maximum
// first, then one rescaling a lane and sums by butterfly.  Every lane returns the same bits.
template <bool SMOOTH>
__device__ __forceinline__ Fold fold_lanes(Fold f, int width) {
  float m = f.m;
  for (int o = width >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const float ms = safe_max(m);
  Fold r{m, __fmul_rn(f.d, exp_diff(f.m, ms)), SMOOTH ? moved(f, ms) : 0.f, f.n};
  for (int o = width >> 1; o > 0; o >>= 1) {
    r.d = __fadd_rn(r.d, __shfl_xor_sync(~0u, r.d, o));
    if constexpr (SMOOTH) {
      r.s = __fadd_rn(r.s, __shfl_xor_sync(~0u, r.s, o));
      r.n += __shfl_xor_sync(~0u, r.n, o);
    }
  }
  return r;
}

// Packed 16-byte vectors of a thread, elements that are not the row's set to -inf: their state.  whole: bit k for a vector k that
// is all the row's; s and n are of those alone.
template <class D, int K, bool SMOOTH>
__device__ __forceinline__ Fold fold_vectors(const uint4 (&q)[K], uint32_t whole) {
  constexpr int E = D::kVec;
  Fold f;
  f.m = D::vmax_all(q);
  f.n = float(E * __popc(whole));
  f.s = 0.f;
  const float ms = safe_max(f.m);
  float2 d = make_float2(0.f, 0.f);
  const float2 ms2 = make_float2(ms, ms), minus = make_float2(-1.f, -1.f);
  const auto sum = [&](auto&& term) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 v[E / 2], s = make_float2(0.f, 0.f);
      D::unpack2(q[k], v);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        d = __fadd2_rn(d, term(v[e]));
        if constexpr (SMOOTH) s = __fadd2_rn(s, __ffma2_rn(v[e], minus, ms2));
      }
      if constexpr (SMOOTH) f.s += whole >> k & 1 ? __fadd_rn(s.x, s.y) : 0.f;
    }
  };
  if (exp_shift_ok(ms)) {
    const ExpShift sh = exp_shift(ms);
    sum([&](float2 v) { return exp_shifted2(v, sh); });
    f.d = __fmul_rn(__fadd_rn(d.x, d.y), sh.unscale);
  } else {
    sum([&](float2 v) { return exp_diff2(v, make_float2(-ms, -ms)); });
    f.d = __fadd_rn(d.x, d.y);
  }
  return f;
}

// What the elements of a row need once its state is known.
struct Slope {
  float ms;     // the maximum (0 for an empty row)
  float a;      // factor of e^(x - m)
  float b;      // subtracted from every element
  float c;      // and from the labelled one
  bool live;    // false: every element is 0
};

// One thread of a row passes write = true: it stores the loss and LSE and records a bad label.
__device__ __forceinline__ Slope slope_of(const LossArgs& a, int64_t row, const Fold& f, int64_t label, float x_label, bool write) {
  Slope s;
  const float w = a.grad_scale * (a.upstream ? a.upstream[row] : 1.f);
  const bool bad = label >= a.N;
  s.ms = safe_max(f.m);
  s.a = __fmul_rn(w, __frcp_rn(f.d));
  s.b = w * a.smoothing_each;
  s.c = w * (1.f - a.smoothing);
  s.live = label >= 0;
  if (a.z > 0.f || write) {
    const float lnd = logf(f.d), lse = f.m + lnd;  // an empty row: -inf; NaN among -inf: NaN
    if (a.z > 0.f) s.a *= __fmaf_rn(2.f * a.z, lse, 1.f);
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
  }
  if (bad) s.a = __int_as_float(0x7fc00000);
  return s;
}

__device__ __forceinline__ float grad_of(const Slope& s, float x) { return s.live ? __fmaf_rn(exp_diff(x, s.ms), s.a, -s.b) : 0.f; }

// The gradients of a thread's vectors: put(k, values) for each k that holds(k) says is the thread's.  at(k): the labelled
// element counted from vector k's first.  The row's cases are told apart once, not for each vector: 8192 x 131072 bf16
// rows are bound by the instructions of this and of fold_vectors.
template <class D, int K, class Holds, class At, class Put>
__device__ __forceinline__ void grad_vectors(const Slope& s, const uint4 (&q)[K], Holds&& holds, At&& at, Put&& put) {
  constexpr int E = D::kVec;
  const auto all = [&](auto&& term) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!holds(k)) continue;
      float2 v[E / 2];
      D::unpack2(q[k], v);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) v[e] = term(v[e]);
      const int l = at(k);
      if (unsigned(l) < unsigned(E)) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          if (l == 2 * e) v[e].x -= s.c;
          if (l == 2 * e + 1) v[e].y -= s.c;
        }
      }
      put(k, v);
    }
  };
  const float2 b = make_float2(-s.b, -s.b);
  if (!s.live) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 v[E / 2] = {};
      if (holds(k)) put(k, v);
    }
  } else if (exp_shift_ok(s.ms)) {
    const ExpShift sh = exp_shift(s.ms);
    const float f = s.a * sh.unscale;
    const float2 a = make_float2(f, f);
    all([&](float2 v) { return __ffma2_rn(exp_shifted2(v, sh), a, b); });
  } else {
    const float2 a = make_float2(s.a, s.a), m = make_float2(-s.ms, -s.ms);
    all([&](float2 v) { return __ffma2_rn(exp_diff2(v, m), a, b); });
  }
}

// Rows that a cluster of at most 16 CTAs holds on chip (kernel_loss_grad_cluster.cu).
bool loss_grad_cluster_fits(const LossGrad& p);
cudaError_t launch_loss_grad_cluster(const LossGrad& p, const LossArgs& a, const DeviceInfo& dev);

}  // namespace rwo
