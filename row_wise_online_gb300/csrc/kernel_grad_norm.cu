// kernel_grad_norm.cu -- the global norm of many gradients, and clipping.
//
//     norm = |scale| sqrt(sum g^2),   out = g * scale * min(1, max_norm / norm)
//
// The list of tensors travels in the kernel's parameters, so a call needs no copy to the device and can be captured.
// Every tensor is cut into chunks; chunk c belongs to CTA c mod grid.  k_squares leaves one sum a CTA in fp64; each
// CTA of k_scale adds those up for itself, all in one order, and so needs nobody to wait for.
#include <cmath>

#include "train.cuh"
#include "train.h"

namespace rwo {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunkVecs = 4;  // 16-byte vectors of a thread in a chunk
constexpr int kSmall = 64, kLarge = 512;

template <int K>
struct Table {
  const unsigned char* g[K];
  unsigned char* out[K];
  int64_t n[K];
  uint32_t first[K + 1];  // chunk that a tensor begins with
  unsigned char type[K], out_type[K];
  int count;
};

struct Params {
  double* parts;  // [parts_n]
  float* norm;
  int parts_n, part0;
  float scale, max_norm;
};

__host__ __device__ constexpr int chunk_elems(int type) { return kThreads * kChunkVecs * (type == 0 ? 4 : 8); }

// The tensor of a chunk.
template <int K>
__device__ __forceinline__ int tensor_of(const Table<K>& t, uint32_t chunk) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Elements before a tensor's first 16-byte boundary.
__host__ __device__ inline int64_t lead_of(const void* g, int64_t n, int bytes) {
  const int64_t lead = int64_t((16 - (reinterpret_cast<uintptr_t>(g) & 15)) & 15) / bytes;
  return lead < n ? lead : n;
}

// Elements of a chunk: whole 16-byte vectors from the tensor's first aligned element on; the first chunk also has the
// elements before it, the last one the rest.
struct Span {
  int64_t begin;   // first element of the first vector
  int vecs;        // whole vectors
  int64_t loose0;  // single elements [loose0, loose1) and [begin + vecs * E, tail1)
  int64_t loose1;
  int64_t tail1;
};
template <class D>
__device__ __forceinline__ Span span_of(const unsigned char* g, int64_t n, uint32_t index, bool last) {
  constexpr int E = D::kVec;
  const int64_t lead = lead_of(g, n, D::kBytes);
  Span s;
  s.begin = lead + int64_t(index) * (kThreads * kChunkVecs * E);
  int64_t v = (n - s.begin) / E;
  if (v < 0) v = 0;
  s.vecs = int(v < kThreads * kChunkVecs ? v : kThreads * kChunkVecs);
  s.loose0 = 0;
  s.loose1 = index == 0 ? lead : 0;
  s.tail1 = last ? n : 0;
  return s;
}

__device__ __forceinline__ double block_sum(double v, double* slots) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if (lane == 0) slots[warp] = v;
  __syncthreads();
  v = lane < kWarps ? slots[lane] : 0.0;
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return __shfl_sync(~0u, v, 0);
}

// This thread's part of a chunk's sum of squares.  A thread adds up at most some 40 squares in fp32.  Where their sum may
// have run over, or may have lost squares below fp32's range to it, they are taken again in fp64.
template <class D>
__device__ __forceinline__ double squares(const unsigned char* g, const Span& s) {
  constexpr int E = D::kVec;
  uint4 q[kChunkVecs];
#pragma unroll
  for (int k = 0; k < kChunkVecs; ++k) {
    const int i = threadIdx.x + k * kThreads;
    q[k] = i < s.vecs ? ld_stream16(g + (s.begin + int64_t(i) * E) * D::kBytes) : make_uint4(0, 0, 0, 0);
  }
  float loose[2] = {0.f, 0.f};
  if (s.loose0 + threadIdx.x < s.loose1) loose[0] = D::load1(g, s.loose0 + threadIdx.x);
  const int64_t rest = s.begin + int64_t(s.vecs) * E + threadIdx.x;
  if (rest < s.tail1) loose[1] = D::load1(g, rest);
  float2 a = make_float2(loose[0] * loose[0], loose[1] * loose[1]);
  uint32_t any = __float_as_uint(loose[0]) | __float_as_uint(loose[1]);
#pragma unroll
  for (int k = 0; k < kChunkVecs; ++k) {
    float2 f[E / 2];
    D::unpack2(q[k], f);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) a = __ffma2_rn(f[e], f[e], a);
    any |= q[k].x | q[k].y | q[k].z | q[k].w;
  }
  const float sum = a.x + a.y;
  if constexpr (D::kBytes == 2 && D::kNegInfWord == F16::kNegInfWord) {
    return sum;  // squares of 2^-48 .. 2^32
  } else {
    if ((sum >= 0x1p-90f && sum <= 0x1p120f) || !(any & (D::kBytes == 2 ? 0x7fff7fffu : 0x7fffffffu))) return sum;
    double d = double(loose[0]) * loose[0] + double(loose[1]) * loose[1];
#pragma unroll
    for (int k = 0; k < kChunkVecs; ++k) {
      float f[E];
      D::unpack(q[k], f);
#pragma unroll
      for (int e = 0; e < E; ++e) d = fma(double(f[e]), double(f[e]), d);
    }
    return d;
  }
}

template <int K>
__global__ void __launch_bounds__(kThreads) k_squares(const __grid_constant__ Table<K> t, Params p) {
  __shared__ double slots[kWarps];
  double sum = 0.0;
  const uint32_t chunks = t.first[t.count];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const bool last = c + 1 == t.first[i + 1];
    const uint32_t index = c - t.first[i];
    if (t.type[i] == SOFTMAX_F32) sum += squares<F32>(t.g[i], span_of<F32>(t.g[i], t.n[i], index, last));
    else if (t.type[i] == SOFTMAX_BF16) sum += squares<BF16>(t.g[i], span_of<BF16>(t.g[i], t.n[i], index, last));
    else sum += squares<F16>(t.g[i], span_of<F16>(t.g[i], t.n[i], index, last));
  }
  sum = block_sum(sum, slots);
  if (threadIdx.x == 0) p.parts[p.part0 + blockIdx.x] = sum;
}

// The norm, the same in every thread of every CTA.
__device__ __forceinline__ double norm_of(const Params& p, double* slots) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < p.parts_n; i += kThreads) sum += p.parts[i];
  return fabs(double(p.scale)) * sqrt(block_sum(sum, slots));
}

__global__ void __launch_bounds__(kThreads) k_norm(Params p) {
  __shared__ double slots[kWarps];
  const double norm = norm_of(p, slots);
  if (threadIdx.x == 0) *p.norm = float(norm);
}

// O: the output's type.
template <class D, class O>
__device__ __forceinline__ void scaled(const unsigned char* g, unsigned char* out, const Span& s, float k) {
  constexpr int E = D::kVec;
  if (s.loose0 + threadIdx.x < s.loose1) O::store1(out, s.loose0 + threadIdx.x, k * D::load1(g, s.loose0 + threadIdx.x));
  const int64_t rest = s.begin + int64_t(s.vecs) * E + threadIdx.x;
  if (rest < s.tail1) O::store1(out, rest, k * D::load1(g, rest));
  const bool wide = (reinterpret_cast<uintptr_t>(out + s.begin * O::kBytes) & 15) == 0;
  uint4 q[kChunkVecs];
#pragma unroll
  for (int j = 0; j < kChunkVecs; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < s.vecs) q[j] = ld_stream16(g + (s.begin + int64_t(i) * E) * D::kBytes);
  }
#pragma unroll
  for (int j = 0; j < kChunkVecs; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i >= s.vecs) continue;
    float f[E];
    D::unpack(q[j], f);
    unsigned char* at = out + (s.begin + int64_t(i) * E) * O::kBytes;
    if (wide) {
#pragma unroll
      for (int b = 0; b < E / O::kVec; ++b) {
        float y[O::kVec];
#pragma unroll
        for (int e = 0; e < O::kVec; ++e) y[e] = k * f[b * O::kVec + e];
        st_stream16(at + b * 16, O::pack(y));
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) O::store1(at, e, k * f[e]);
    }
  }
}

template <int K>
__global__ void __launch_bounds__(kThreads) k_scale(const __grid_constant__ Table<K> t, Params p) {
  __shared__ double slots[kWarps];
  const double norm = norm_of(p, slots);
  if (p.part0 == 0 && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = float(norm);
  const bool limited = norm > double(p.max_norm) && float(norm) <= 3.4028234663852886e38f;
  const float k = limited ? float(double(p.scale) * (double(p.max_norm) / norm)) : p.scale;
  const uint32_t chunks = t.first[t.count];
  for (uint32_t b = blockIdx.x; b < chunks; b += gridDim.x) {
    const uint32_t c = chunks - 1 - b;  // last chunks first: they are the likeliest to be in L2 still
    const int i = tensor_of(t, c);
    if (k == 1.f && t.out[i] == t.g[i]) continue;
    const bool last = c + 1 == t.first[i + 1];
    const uint32_t index = c - t.first[i];
    if (t.type[i] == SOFTMAX_F32) {
      scaled<F32, F32>(t.g[i], t.out[i], span_of<F32>(t.g[i], t.n[i], index, last), k);
    } else if (t.type[i] == SOFTMAX_BF16) {
      const Span s = span_of<BF16>(t.g[i], t.n[i], index, last);
      if (t.out_type[i] == SOFTMAX_F32) scaled<BF16, F32>(t.g[i], t.out[i], s, k);
      else scaled<BF16, BF16>(t.g[i], t.out[i], s, k);
    } else {
      const Span s = span_of<F16>(t.g[i], t.n[i], index, last);
      if (t.out_type[i] == SOFTMAX_F32) scaled<F16, F32>(t.g[i], t.out[i], s, k);
      else scaled<F16, F16>(t.g[i], t.out[i], s, k);
    }
  }
}

int64_t grid_most(const DeviceInfo& dev) { return int64_t(dev.sm_count) * (dev.max_threads_per_sm / kThreads); }

// Tensors from `from` on that fit a table; returns the first one after them.
template <int K>
int64_t fill(Table<K>& t, const GradNorm& p, int64_t from) {
  t.count = 0;
  t.first[0] = 0;
  int64_t i = from;
  for (; i < p.count && t.count < K; ++i) {
    const grad_tensor& g = p.tensors[i];
    if (g.n == 0) continue;
    const int64_t c = chunk_elems(g.dtype), chunks = (g.n - lead_of(g.grad, g.n, elem_bytes(g.dtype)) + c - 1) / c;
    t.g[t.count] = static_cast<const unsigned char*>(g.grad);
    t.out[t.count] = static_cast<unsigned char*>(g.out);
    t.n[t.count] = g.n;
    t.type[t.count] = (unsigned char)g.dtype;
    t.out_type[t.count] = (unsigned char)g.out_dtype;
    t.first[t.count + 1] = t.first[t.count] + uint32_t(chunks > 1 ? chunks : 1);
    ++t.count;
  }
  return i;
}

template <int K>
cudaError_t run(const GradNorm& p, const DeviceInfo& dev) {
  Params a;
  a.parts = p.parts;
  a.norm = p.norm;
  a.parts_n = 0;
  a.part0 = 0;
  a.scale = p.scale;
  a.max_norm = p.max_norm;
  Table<K> t;
  cudaError_t e;
  for (int64_t from = 0; from < p.count;) {
    from = fill(t, p, from);
    if (t.count == 0) continue;
    const int64_t chunks = t.first[t.count], most = grid_most(dev);
    const unsigned grid = unsigned(chunks < most ? chunks : most);
    a.part0 = a.parts_n;
    k_squares<K><<<grid, kThreads, 0, p.stream>>>(t, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    a.parts_n += int(grid);
  }
  if (p.max_norm == 0.f || a.parts_n == 0) {
    k_norm<<<1, kThreads, 0, p.stream>>>(a);
    return cudaGetLastError();
  }
  a.part0 = 0;
  for (int64_t from = 0; from < p.count;) {
    from = fill(t, p, from);
    if (t.count == 0) continue;
    const int64_t chunks = t.first[t.count], most = grid_most(dev);
    k_scale<K><<<unsigned(chunks < most ? chunks : most), kThreads, 0, p.stream>>>(t, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    a.part0 = 1;  // the norm is written
  }
  return cudaSuccess;
}

}  // namespace

// A sum in fp64 of each CTA of each launch.
size_t grad_norm_scratch(int64_t count, const DeviceInfo& dev) {
  const int64_t launches = (count + kLarge - 1) / kLarge + 1;
  return size_t(launches * grid_most(dev) * 8);
}

cudaError_t launch_grad_norm(const GradNorm& p, const DeviceInfo& dev) {
  return p.count <= kSmall ? run<kSmall>(p, dev) : run<kLarge>(p, dev);
}

}  // namespace rwo
