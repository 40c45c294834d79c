// train.cuh -- device helpers of the training-step kernels.
#pragma once

#include "device_common.cuh"

namespace rwo {

// One element, by a load that is not moved and sees this kernel's own stores.
template <class D>
__device__ __forceinline__ float load1c(const void* p, int64_t i) {
  if constexpr (D::kBytes == 4) {
    return static_cast<const volatile float*>(p)[i];
  } else {
    const uint32_t b = static_cast<const volatile uint16_t*>(p)[i];
    if constexpr (D::kNegInfWord == BF16::kNegInfWord) return bf16_lo(b);
    else return f16_lo(b);
  }
}

// A long sum of a thread: lost is what the additions to s rounded away, which the next one takes up.  An infinite sum stays one.
struct LongSum {
  float s = 0.f, lost = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float want = __fsub_rn(v, lost), t = __fadd_rn(s, want);
    lost = fabsf(t) < INFINITY ? __fsub_rn(__fsub_rn(t, s), want) : 0.f;
    s = t;
  }
};

// A value as the element type holds it.
template <class D>
__device__ __forceinline__ float rounded(float v) {
  if constexpr (D::kBytes == 4) return v;
  else if constexpr (D::kNegInfWord == BF16::kNegInfWord) return bf16_lo(pack_bf16x2(v, 0.f));
  else return f16_lo(pack_f16x2(v, 0.f));
}

// A kernel started by launch_after() may begin while the one before it in the stream still runs: griddep_wait() waits
// until that has ended and its writes are seen.  griddep_launch() in the one before: from here on the next may be started.
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- vectors of rows that start anywhere ---------------------------------------------------------------------------------
//
// Vector u of a row are its elements u E .. u E + E - 1, 16 bytes.  Where rows are not on 16-byte boundaries a warp whose
// lanes have consecutive vectors moves whole 16-byte lines of memory and shifts them over its lanes: each lane loads the
// line that its vector begins in and has the rest from the next lane, and stores the line that begins in its vector; only
// the ends of what a warp has are stored by single elements.  (By single
// elements the backward norm of 777 rows of 5003 fp16 elements took 74 us; so it takes 24, with a dx that starts elsewhere in its lines.)

// The bytes of a matrix: whole lines are loaded only inside them.
struct Bytes {
  const unsigned char* lo;
  const unsigned char* hi;
};
__device__ __forceinline__ Bytes bytes_of(const unsigned char* p, int64_t rows, int64_t pitch, int64_t row_bytes) {
  return Bytes{p, p + (rows - 1) * pitch + row_bytes};
}

// Bytes delta .. delta + 15 of a and b one after the other, delta even and the same in all lanes.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int delta) {
  const uint32_t bits = (delta & 3) * 8;
  const auto from = [&](uint32_t v, uint32_t w, uint32_t x, uint32_t y, uint32_t z) {
    return make_uint4(__funnelshift_r(v, w, bits), __funnelshift_r(w, x, bits), __funnelshift_r(x, y, bits), __funnelshift_r(y, z, bits));
  };
  switch (delta >> 2) {
    case 0: return from(a.x, a.y, a.z, a.w, b.x);
    case 1: return from(a.y, a.z, a.w, b.x, b.y);
    case 2: return from(a.z, a.w, b.x, b.y, b.z);
    default: return from(a.w, b.x, b.y, b.z, b.w);
  }
}

// Elements [from, to) of a vector, the others fill (a word).
template <class D>
__device__ __forceinline__ uint4 keep(uint4 q, int from, int to, uint32_t fill) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (D::kBytes == 4) {
      if (i < from || i >= to) w[i] = fill;
    } else {
      if (2 * i < from || 2 * i >= to) w[i] = (w[i] & 0xffff0000u) | (fill & 0xffffu);
      if (2 * i + 1 < from || 2 * i + 1 >= to) w[i] = (w[i] & 0xffffu) | (fill & 0xffff0000u);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The next lane's q; for lane 31 lane 0's first.
__device__ __forceinline__ uint4 next_lane(const uint4& q, const uint4& first) {
  const int lane = threadIdx.x & 31, from = (lane + 1) & 31;
  return make_uint4(__shfl_sync(~0u, lane ? q.x : first.x, from), __shfl_sync(~0u, lane ? q.y : first.y, from),
                    __shfl_sync(~0u, lane ? q.z : first.z, from), __shfl_sync(~0u, lane ? q.w : first.w, from));
}

// The line at a, elements of the row [row, end) only: for the few lines that are not all inside the matrix.
template <class D>
__device__ __noinline__ uint4 load_elements(const unsigned char* a, const unsigned char* row, const unsigned char* end) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < D::kVec; ++e) {
    const unsigned char* p = a + e * D::kBytes;
    if (p < row || p >= end) continue;
    if constexpr (D::kBytes == 4) w[e] = *reinterpret_cast<const volatile uint32_t*>(p);
    else w[e / 2] |= uint32_t(*reinterpret_cast<const volatile uint16_t*>(p)) << (e & 1) * 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row of n elements; inside: all lines that it has a part in are.
struct RowAt {
  const unsigned char* row;
  const unsigned char* end;
  int n, delta;  // delta: bytes from a line's start to a vector's
  bool inside;
};
template <class D>
__device__ __forceinline__ RowAt row_at(const unsigned char* row, int n, const Bytes& m) {
  RowAt r{row, row + int64_t(n) * D::kBytes, n, int(reinterpret_cast<uintptr_t>(row) & 15), true};
  r.inside = row - r.delta >= m.lo && r.end + (-reinterpret_cast<uintptr_t>(r.end) & 15) <= m.hi;
  return r;
}

// Vectors u, u + 32, ... u + 32 (K - 1) of a row, 0 behind its end.  All lanes of a warp, with consecutive u.
template <class D, int K>
__device__ __forceinline__ void load_vectors(const RowAt& r, int u, uint4 (&q)[K]) {
  const unsigned char* p = r.row + int64_t(u) * 16 - r.delta;
  const auto line = [&](const unsigned char* a) {
    if (a >= r.end) return make_uint4(0, 0, 0, 0);
    return r.inside ? ld_stream16(a) : load_elements<D>(a, r.row, r.end);
  };
#pragma unroll
  for (int k = 0; k < K; ++k) q[k] = line(p + k * 512);
  if (r.delta) {
    uint4 last = make_uint4(0, 0, 0, 0);  // lane 0: the line behind the warp's vectors
    if ((threadIdx.x & 31) == 0) last = line(p + K * 512);
#pragma unroll
    for (int k = 0; k < K; ++k) q[k] = shifted(q[k], next_lane(q[k], k + 1 < K ? q[k + 1] : last), r.delta);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int left = r.n - (u + k * 32) * D::kVec;
    if (left < D::kVec) q[k] = keep<D>(q[k], 0, left, 0);
  }
}

// Elements [from, to) of a vector, to their places from p on.
template <class D>
__device__ __noinline__ void store_elements(unsigned char* p, uint4 q, int from, int to) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int e = 0; e < D::kVec; ++e) {
    if (e < from || e >= to) continue;
    if constexpr (D::kBytes == 4) reinterpret_cast<uint32_t*>(p)[e] = w[e];
    else reinterpret_cast<uint16_t*>(p)[e] = uint16_t(w[e / 2] >> (e & 1) * 16);
  }
}

// Stores what load_vectors reads.
template <class D, int K>
__device__ __forceinline__ void store_vectors(unsigned char* row, int u, int n, const uint4 (&q)[K]) {
  const int delta = int(reinterpret_cast<uintptr_t>(row) & 15), lane = threadIdx.x & 31;
  // elements before the line that begins in a vector; the lane before stores them where its line is whole
  const int head = delta ? (16 - delta) / D::kBytes : 0;
  unsigned char* p = row + int64_t(u) * 16;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int left = n - (u + k * 32) * D::kVec;
    uint4 line = q[k];
    if (delta) line = shifted(line, next_lane(line, q[k + 1 < K ? k + 1 : k]), 16 - delta);
    const bool whole = left >= D::kVec + head && (lane < 31 || k + 1 < K || !delta), first = delta && ((lane == 0 && k == 0) || left < head);
    if (whole) st_stream16(p + k * 512 + (delta ? 16 - delta : 0), line);
    if ((first || !whole) && left > 0) store_elements<D>(p + k * 512, q[k], first ? 0 : head, whole ? min(head, left) : min(D::kVec, left));
  }
}

}  // namespace rwo
