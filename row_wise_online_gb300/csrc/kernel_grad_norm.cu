// kernel_grad_norm.cu -- the global norm of many gradients, and clipping.
//
//     norm = |scale| sqrt(sum g^2),   out = g * scale * min(1, max_norm / norm)
//
// The list of tensors travels in the kernel's parameters, so a call needs no copy to the device and can be captured.
// Every tensor is cut into chunks; chunk c belongs to CTA c mod grid.  k_squares leaves one sum a CTA in fp64; each
// CTA of k_scale adds those up for itself, all in one order, and so needs nobody to wait for.  The memory's rate bounds both: the
// norm of 1.07e9 bf16 elements in 160 tensors takes 336 us (6.4 TB/s), scaling them into fp32 1044 us (6.2 TB/s), where a tensor is read again unless
// L2 still has it.
#include <cmath>

#include "train.cuh"
#include "train.h"

namespace rwo {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunkVecs = 8;  // 16-byte vectors of a thread in a chunk
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
  float scale;
  double max_norm;  // 0: the norm alone
  bool in_place;  // every tensor of the table
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

// A chunk: whole 16-byte vectors from the tensor's first aligned element on; the first chunk also has the elements before
// it, the last one the rest.
struct Chunk {
  const unsigned char* g;
  unsigned char* out;
  int64_t begin;  // first element of the first vector
  int64_t tail;   // the rest ends here (0: none)
  int vecs;       // whole vectors
  int lead;       // single elements from the tensor's first on
  int type, out_type;
};
template <int K>
__device__ __forceinline__ Chunk chunk_of(const Table<K>& t, uint32_t c) {
  const int i = tensor_of(t, c);
  const uint32_t index = c - t.first[i];
  Chunk s;
  s.g = t.g[i];
  s.out = t.out[i];
  s.type = t.type[i];
  s.out_type = t.out_type[i];
  const int bytes = s.type == SOFTMAX_F32 ? 4 : 2, per = 16 / bytes;
  const int64_t n = t.n[i], lead = lead_of(s.g, n, bytes);
  s.begin = lead + int64_t(index) * (kThreads * kChunkVecs * per);
  const int64_t v = n > s.begin ? (n - s.begin) / per : 0;
  s.vecs = int(v < kThreads * kChunkVecs ? v : kThreads * kChunkVecs);
  s.lead = index == 0 ? int(lead) : 0;
  s.tail = c + 1 == t.first[i + 1] ? n : 0;
  return s;
}

// This thread's vectors of a chunk, 0 where it has none.
__device__ __forceinline__ void load(const Chunk& s, uint4 (&q)[kChunkVecs]) {
  const unsigned char* p = s.g + s.begin * (s.type == SOFTMAX_F32 ? 4 : 2) + threadIdx.x * 16;
#pragma unroll
  for (int k = 0; k < kChunkVecs; ++k)
    q[k] = int(threadIdx.x) + k * kThreads < s.vecs ? ld_stream16(p + k * (kThreads * 16)) : make_uint4(0, 0, 0, 0);
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

// This thread's part of a chunk's sum of squares.  A thread adds up at most 66 squares in fp32.  Where their sum may
// have run over, or may have lost squares below fp32's range to it, they are taken again in fp64.
template <class D>
__device__ __forceinline__ double squares(const Chunk& s, const uint4 (&q)[kChunkVecs]) {
  constexpr int E = D::kVec;
  float loose[2] = {0.f, 0.f};
  if (int(threadIdx.x) < s.lead) loose[0] = D::load1(s.g, threadIdx.x);
  const int64_t rest = s.begin + int64_t(s.vecs) * E + threadIdx.x;
  if (rest < s.tail) loose[1] = D::load1(s.g, rest);
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

// Chunks first, first + step, ... of a table: the next one's vectors are under way while one is worked on.
template <int K, class Work>
__device__ __forceinline__ void each_chunk(const Table<K>& t, bool backwards, Work&& work) {
  const uint32_t chunks = t.first[t.count];
  const auto nth = [&](uint32_t i) { return chunk_of(t, backwards ? chunks - 1 - i : i); };
  uint32_t i = blockIdx.x;
  if (i >= chunks) return;
  Chunk s = nth(i);
  uint4 q[kChunkVecs];
  load(s, q);
  while (true) {
    i += gridDim.x;
    Chunk next;
    uint4 p[kChunkVecs];
    if (i < chunks) {
      next = nth(i);
      load(next, p);
    }
    work(s, q);
    if (i >= chunks) return;
    s = next;
#pragma unroll
    for (int k = 0; k < kChunkVecs; ++k) q[k] = p[k];
  }
}

// CTAs of an SM.  Two with eight vectors a thread under way and eight worked on: the norm of 2^30 bf16 elements took 349 us; four with four
// and four 402, six 671.
constexpr int kCtas = 2;

template <int K>
__global__ void __launch_bounds__(kThreads, kCtas) k_squares(const __grid_constant__ Table<K> t, Params p) {
  __shared__ double slots[kWarps];
  griddep_launch();
  double sum = 0.0;
  each_chunk(t, false, [&](const Chunk& s, const uint4(&q)[kChunkVecs]) {
    sum += s.type == SOFTMAX_F32 ? squares<F32>(s, q) : s.type == SOFTMAX_BF16 ? squares<BF16>(s, q) : squares<F16>(s, q);
  });
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
  griddep_wait();
  const double norm = norm_of(p, slots);
  if (threadIdx.x == 0) *p.norm = float(norm);
}

// Eight fp32 values a lane, 32 bytes at p: two lanes write 32 bytes of one together, then of the other, so that every store fills
// whole sectors (2^30 elements, bf16 into fp32, when it was done: 1082 us against 1322).  All lanes of a warp.
__device__ __forceinline__ void pair_store(unsigned char* p, const float2 (&f)[4]) {
  const bool odd = threadIdx.x & 1;
  float2 a = odd ? f[0] : f[2], b = odd ? f[1] : f[3];  // what the other lane stores
  a = make_float2(__shfl_xor_sync(~0u, a.x, 1), __shfl_xor_sync(~0u, a.y, 1));
  b = make_float2(__shfl_xor_sync(~0u, b.x, 1), __shfl_xor_sync(~0u, b.y, 1));
  // the even lane's 32 bytes, its own first half and the odd lane's copy of the second; then the odd lane's
  const float2 lo[2] = {odd ? a : f[0], odd ? b : f[1]}, hi[2] = {odd ? f[2] : a, odd ? f[3] : b};
  unsigned char* even = p - (odd ? 32 : 0) + (odd ? 16 : 0);
  st_stream16(even, F32::pack2(lo));
  st_stream16(even + 32, F32::pack2(hi));
}

// What gradients are multiplied by.  Where they are limited, scale * max_norm / norm to 48 bits, hi + lo, so that a product is rounded once
// (2^30 bf16 elements, norm and scaling into fp32: 1410 us a call, 1407 with hi alone); a factor below 2^-90 as pre, a power of 2, and the rest: hi alone would
// be below fp32's normal values where a norm of 1e38 is limited to 1.  Else the scale as it is, which keeps infinities.
struct Factor {
  float hi, lo, pre;
};
__device__ __forceinline__ Factor factor_of(double k) {
  Factor f;
  f.pre = 1.f;
  if (fabs(k) < 0x1p-90 && k != 0.0) {
    const int e = max(ilogb(k) + 30, -126);
    f.pre = ldexpf(1.f, e);
    k = ldexp(k, -e);
  }
  f.hi = float(k);
  f.lo = float(k - double(f.hi));
  return f;
}
template <bool LIMITED>
__device__ __forceinline__ float times(float g, const Factor& f) {
  if constexpr (!LIMITED) return g * f.hi;
  g *= f.pre;
  return __fmaf_rn(g, f.hi, g * f.lo);
}
template <bool LIMITED>
__device__ __forceinline__ float2 times2(float2 g, const Factor& f) {
  const float2 hi = make_float2(f.hi, f.hi);
  if constexpr (!LIMITED) return __fmul2_rn(g, hi);
  if (f.pre != 1.f) g = __fmul2_rn(g, make_float2(f.pre, f.pre));
  return __ffma2_rn(g, hi, __fmul2_rn(g, make_float2(f.lo, f.lo)));
}

// O: the output's type.
template <class D, class O, bool LIMITED>
__device__ __forceinline__ void scaled(const Chunk& s, const uint4 (&q)[kChunkVecs], const Factor& k) {
  constexpr int E = D::kVec;
  if (int(threadIdx.x) < s.lead) O::store1(s.out, threadIdx.x, times<LIMITED>(D::load1(s.g, threadIdx.x), k));
  const int64_t rest = s.begin + int64_t(s.vecs) * E + threadIdx.x;
  if (rest < s.tail) O::store1(s.out, rest, times<LIMITED>(D::load1(s.g, rest), k));
  unsigned char* out = s.out + s.begin * O::kBytes + threadIdx.x * (E * O::kBytes);
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  const bool paired = s.vecs == kThreads * kChunkVecs;
#pragma unroll
  for (int j = 0; j < kChunkVecs; ++j) {
    if (int(threadIdx.x) + j * kThreads >= s.vecs) continue;
    float2 f[E / 2];
    D::unpack2(q[j], f);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) f[e] = times2<LIMITED>(f[e], k);
    unsigned char* at = out + j * (kThreads * E * O::kBytes);
    if (wide) {
      if constexpr (E == O::kVec) st_stream16(at, O::pack2(f));
      else if (paired) pair_store(at, f);
      else st_stream16(at, O::pack2({f[0], f[1]})), st_stream16(at + 16, O::pack2({f[2], f[3]}));
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) O::store1(at, e, e & 1 ? f[e / 2].y : f[e / 2].x);
    }
  }
}

// A table's tensors scaled.
template <int K, bool LIMITED>
__device__ __forceinline__ void scale_table(const Table<K>& t, const Factor& k) {
  // last chunks first: they are the likeliest to be in L2 still
  each_chunk(t, true, [&](const Chunk& s, const uint4(&q)[kChunkVecs]) {
    if (!LIMITED && k.hi == 1.f && s.out == s.g) return;
    if (s.type == SOFTMAX_F32) {
      scaled<F32, F32, LIMITED>(s, q, k);
    } else if (s.type == SOFTMAX_BF16) {
      if (s.out_type == SOFTMAX_F32) scaled<BF16, F32, LIMITED>(s, q, k);
      else scaled<BF16, BF16, LIMITED>(s, q, k);
    } else {
      if (s.out_type == SOFTMAX_F32) scaled<F16, F32, LIMITED>(s, q, k);
      else scaled<F16, F16, LIMITED>(s, q, k);
    }
  });
}

// The norm written by one CTA, and a table's tensors scaled.
template <int K>
__device__ __forceinline__ void scale_all(const Table<K>& t, const Params& p, double norm, bool writes) {
  if (writes && threadIdx.x == 0) *p.norm = float(norm);
  if (p.max_norm == 0.0) return;  // the norm alone
  if (norm > p.max_norm && float(norm) <= 3.4028234663852886e38f) {
    scale_table<K, true>(t, factor_of(double(p.scale) * (p.max_norm / norm)));
  } else if (p.scale != 1.f || !p.in_place) {
    scale_table<K, false>(t, Factor{p.scale, 0.f, 1.f});
  }
}

template <int K>
__global__ void __launch_bounds__(kThreads, kCtas) k_scale(const __grid_constant__ Table<K> t, Params p) {
  __shared__ double slots[kWarps];
  griddep_wait();
  scale_all(t, p, norm_of(p, slots), p.part0 == 0 && blockIdx.x == 0);
}

// A few chunks: one launch of one cluster for the norm and the scaling both.  Its CTAs' sums go to all of them over distributed
// shared memory, to be added up in their order.  (30 small tensors: 7.4 us on the GPU; two launches, 4 us more a call.)
constexpr int kFew = 16, kFewChunks = 4 * kFew;

__global__ void __launch_bounds__(kThreads, kCtas) k_few(const __grid_constant__ Table<kSmall> t, Params p) {
  __shared__ double slots[kWarps], sums[kFew];
  cluster_sync();  // every CTA is there before another writes into it
  double sum = 0.0;
  each_chunk(t, false, [&](const Chunk& s, const uint4(&q)[kChunkVecs]) {
    sum += s.type == SOFTMAX_F32 ? squares<F32>(s, q) : s.type == SOFTMAX_BF16 ? squares<BF16>(s, q) : squares<F16>(s, q);
  });
  sum = block_sum(sum, slots);
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x < kFew)
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(map_to_rank(smem_addr(sums + rank), threadIdx.x)), "d"(sum) : "memory");
  cluster_sync();
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < kFew; ++i) sum += sums[i];
  scale_all(t, p, fabs(double(p.scale)) * sqrt(sum), rank == 0);
}

int64_t grid_most(const DeviceInfo& dev) { return int64_t(dev.sm_count) * kCtas; }

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
bool every_in_place(const Table<K>& t) {
  for (int i = 0; i < t.count; ++i)
    if (t.out[i] != t.g[i]) return false;
  return true;
}

cudaError_t launch_few(const Table<kSmall>& t, const Params& a, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute((const void*)k_few, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kFew);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kFew;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_few, t, a);
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
  a.in_place = false;
  Table<K> t;
  cudaError_t e;
  if constexpr (K == kSmall) {
    if (p.count > 0 && fill(t, p, 0) == p.count && t.first[t.count] <= kFewChunks) {
      a.in_place = every_in_place(t);
      return launch_few(t, a, p.stream);
    }
  }
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
  if (p.max_norm == 0.0 || a.parts_n == 0) {
    return launch_after(k_norm, dim3(1), kThreads, p.stream, a);
  }
  a.part0 = 0;
  for (int64_t from = 0; from < p.count;) {
    from = fill(t, p, from);
    if (t.count == 0) continue;
    const int64_t chunks = t.first[t.count], most = grid_most(dev);
    a.in_place = every_in_place(t);
    if ((e = launch_after(k_scale<K>, dim3(unsigned(chunks < most ? chunks : most)), kThreads, p.stream, t, a)) != cudaSuccess) return e;
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
