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
// line that its vector begins in and has the rest from the next lane, and stores the line that begins in its vector.  (By single
// elements the backward norm of 777 rows of 5003 fp16 elements took 74 us; so it takes 25.)

// The bytes of a matrix: whole lines are loaded only inside them.
struct Bytes {
  const unsigned char* lo;
  const unsigned char* hi;
};
__device__ __forceinline__ Bytes bytes_of(const unsigned char* p, int64_t rows, int64_t pitch, int64_t row_bytes) {
  return Bytes{p, p + (rows - 1) * pitch + row_bytes};
}

// Bytes delta .. delta + 15 of a and b one after the other, delta even.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int delta) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int words = delta >> 2;
  if (words & 2) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (words & 1) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const uint32_t bits = (delta & 3) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
  return make_uint4(w[0], w[1], w[2], w[3]);
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

__device__ __forceinline__ uint4 next_lane(uint4 q) {
  return make_uint4(__shfl_down_sync(~0u, q.x, 1), __shfl_down_sync(~0u, q.y, 1), __shfl_down_sync(~0u, q.z, 1), __shfl_down_sync(~0u, q.w, 1));
}

// The line at a: of the row's elements where it is not all inside the matrix.
template <class D>
__device__ __forceinline__ uint4 load_line(const unsigned char* a, const unsigned char* row, const unsigned char* end, const Bytes& m) {
  if (a >= end || a + 16 <= row) return make_uint4(0, 0, 0, 0);
  if (a >= m.lo && a + 16 <= m.hi) return ld_stream16(a);
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

// Vector u of a row of n elements, 0 behind its end.  All lanes of a warp, with consecutive u.
template <class D>
__device__ __forceinline__ uint4 load_vector(const unsigned char* row, int u, int n, const Bytes& m) {
  const unsigned char* p = row + int64_t(u) * 16;
  const unsigned char* end = row + int64_t(n) * D::kBytes;
  const int delta = int(reinterpret_cast<uintptr_t>(p) & 15);
  uint4 q = load_line<D>(p - delta, row, end, m);
  if (delta) {
    uint4 b = next_lane(q);
    if ((threadIdx.x & 31) == 31) b = load_line<D>(p - delta + 16, row, end, m);
    q = shifted(q, b, delta);
  }
  const int left = n - u * D::kVec;
  return left >= D::kVec ? q : keep<D>(q, 0, left, 0);
}

template <class D>
__device__ __forceinline__ void store_elements(unsigned char* p, const uint4& q, int from, int to) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int e = 0; e < D::kVec; ++e) {
    if (e < from || e >= to) continue;
    if constexpr (D::kBytes == 4) reinterpret_cast<uint32_t*>(p)[e] = w[e];
    else reinterpret_cast<uint16_t*>(p)[e] = uint16_t(w[e / 2] >> (e & 1) * 16);
  }
}

// Stores what load_vector reads.
template <class D>
__device__ __forceinline__ void store_vector(unsigned char* row, int u, int n, const uint4& q) {
  unsigned char* p = row + int64_t(u) * 16;
  const int delta = int(reinterpret_cast<uintptr_t>(p) & 15), left = n - u * D::kVec, lane = threadIdx.x & 31;
  if (!delta) {
    if (left >= D::kVec) st_stream16(p, q);
    else store_elements<D>(p, q, 0, left);
    return;
  }
  // elements before the line that begins in this vector; the lane before stores them where its line is whole
  const int head = (16 - delta) / D::kBytes;
  const uint4 b = next_lane(q);
  if (lane == 0 || left < head) store_elements<D>(p, q, 0, min(head, left));
  if (lane < 31 && left >= D::kVec + head) st_stream16(p + 16 - delta, shifted(q, b, 16 - delta));
  else store_elements<D>(p, q, head, min(D::kVec, left));
}

}  // namespace rwo
