// kernel_embedding.cu -- embedding lookup and its gradient.
//
// Lookup: y_t = scale * table[token_t], a copy of rows.
//
// Gradient: grad_v = scale * sum of dy_t over the t with token_t = v.  The tokens are sorted with their positions
// (k_sort_tokens: a stable radix sort by one thread-block cluster), so that the rows of a token are one run of the
// sorted list.  The list is cut into chunks of kChunk tokens, whatever the runs: a CTA takes a chunk's columns and adds
// up the runs in it (k_embedding_rows).  A run inside a chunk is written at once; one that goes on into the next chunk
// leaves partial sums, which k_embedding_join adds up in their order.  So a frequent token is spread over the GPU as
// others are, no atomics touch the sums, and their order is a function of the tokens alone.  Rows without a token
// are zeroed by the same launch, from a bit map that the sort leaves.
#include "train.cuh"
#include "train.h"

namespace rwo {
namespace {

constexpr int kChunk = 32;
constexpr int kSortThreads = 1024, kSortWarps = 32, kSortCtas = 8;
constexpr int kDigitBits = 10;

__device__ __forceinline__ int64_t token_at(const void* tokens, int bytes, int64_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(tokens)[i] : int64_t(static_cast<const int32_t*>(tokens)[i]);
}

// ---- lookup ---------------------------------------------------------------------------------------------------------

struct LookupArgs {
  const unsigned char* table;
  unsigned char* y;
  const void* tokens;
  int64_t T, V;
  int64_t table_pitch, y_pitch;  // bytes
  uint32_t units;                // of a row
  int token_bytes;
  float scale;
  unsigned* status;
};

constexpr int kLookupThreads = 256, kLookupPer = 4;

// Units (16-byte vectors, or elements) of all rows in one line; a thread takes kLookupPer of them.
template <class D, bool VEC>
__global__ void __launch_bounds__(kLookupThreads) k_embedding(LookupArgs a) {
  constexpr int E = VEC ? D::kVec : 1;
  const int64_t base = int64_t(blockIdx.x) * (kLookupThreads * kLookupPer);
  const int64_t t0 = base / a.units;
  const uint32_t first = uint32_t(base - t0 * a.units);
  float v[kLookupPer][E];
  int64_t at[kLookupPer];
#pragma unroll
  for (int k = 0; k < kLookupPer; ++k) {
    const uint64_t o = uint64_t(first) + threadIdx.x + k * kLookupThreads;
    const uint64_t dt = o >> 32 ? o / a.units : uint32_t(o) / a.units;
    const int64_t t = t0 + int64_t(dt);
    const uint32_t u = uint32_t(o - dt * a.units);
    at[k] = -1;
    if (t >= a.T) continue;
    const int64_t token = token_at(a.tokens, a.token_bytes, t);
    at[k] = t * a.y_pitch + int64_t(u) * (E * D::kBytes);
    if (token >= 0 && token < a.V) {
      const unsigned char* row = a.table + token * a.table_pitch;
      if constexpr (VEC) D::unpack(ld_stream16(row + int64_t(u) * 16), v[k]);
      else v[k][0] = D::load1(row, u);
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] *= a.scale;
    } else {
      if (token >= 0 && u == 0) atomicOr(a.status, kStatusBadIndex);
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = token < 0 ? 0.f : __int_as_float(0x7fc00000);
    }
  }
#pragma unroll
  for (int k = 0; k < kLookupPer; ++k)
    if (at[k] >= 0) {
      if constexpr (VEC) st_stream16(a.y + at[k], D::pack(v[k]));
      else D::store1(a.y + at[k], 0, v[k][0]);
    }
}

template <class D>
cudaError_t launch_lookup(const Embedding& p, const DeviceInfo& dev) {
  LookupArgs a;
  a.table = static_cast<const unsigned char*>(p.table);
  a.y = static_cast<unsigned char*>(p.y);
  a.tokens = p.tokens;
  a.T = p.T;
  a.V = p.V;
  a.table_pitch = p.table_pitch * D::kBytes;
  a.y_pitch = p.y_pitch * D::kBytes;
  a.token_bytes = p.token_bytes;
  a.scale = p.scale;
  a.status = dev.status;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.table) | reinterpret_cast<uintptr_t>(a.y) | uintptr_t(a.table_pitch) | uintptr_t(a.y_pitch) |
                     uintptr_t(p.D * D::kBytes)) & 15) == 0;
  a.units = uint32_t(vec ? p.D / D::kVec : p.D);
  const int64_t per = kLookupThreads * kLookupPer;
  // the grid's limit of 2^31 - 1 CTAs: more rows than that take further launches
  const int64_t rows = (int64_t(1) << 30) * per / a.units;
  for (int64_t t = 0; t < p.T; t += rows) {
    LookupArgs b = a;
    b.T = p.T - t < rows ? p.T - t : rows;
    b.tokens = static_cast<const unsigned char*>(p.tokens) + t * p.token_bytes;
    b.y = a.y + t * a.y_pitch;
    const unsigned grid = unsigned((b.T * a.units + per - 1) / per);
    if (vec) k_embedding<D, true><<<grid, kLookupThreads, 0, p.stream>>>(b);
    else k_embedding<D, false><<<grid, kLookupThreads, 0, p.stream>>>(b);
    if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// ---- gradient: the sort ---------------------------------------------------------------------------------------------

struct GradArgs {
  const unsigned char* dy;
  unsigned char* g;
  const void* tokens;
  uint32_t* keys[2];
  uint32_t* pos[2];
  const uint32_t* sorted_keys;
  const uint32_t* sorted_pos;
  uint32_t* bits;  // rows that a token names
  float* parts;    // [chunk][2][part_pitch]: sums of the run that came from the chunk before, of the one that goes on
  int64_t T, V, D;
  int64_t dy_pitch, g_pitch;  // bytes
  int64_t part_pitch;         // floats
  int64_t chunks;
  uint32_t units;             // of a row
  int slices;                 // CTAs of a chunk
  int64_t fill_rows;          // rows of a zeroing CTA
  int token_bytes, passes, digit_bits;
  float scale;
  bool accumulate, fill_vec;
  unsigned* status;
};

// Least significant digit first, digits of digit_bits.  A warp owns a run of the list and a column of counts; ranks
// within 32 tokens come from a vote (lanes of the same digit), so equal tokens keep their order.  Tokens outside the
// table get the key V and end up last.
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) k_sort_tokens(GradArgs a) {
  extern __shared__ uint32_t shared[];
  const int bins = 1 << a.digit_bits, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* total = shared;                             // [bins], read by the cluster's other CTAs
  uint32_t* base = total + bins;                        // [bins]
  uint32_t* counts = base + bins;                       // [bins][33]: a warp's counts, then where they start
  __shared__ uint32_t sums[kSortWarps];
  const uint32_t cta = cluster_ctarank();
  const int64_t per = ((a.T + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) / 32 * 32;
  const int64_t i0 = (int64_t(cta) * kSortWarps + warp) * per;
  const int64_t i1 = i0 + per < a.T ? i0 + per : a.T;
  const uint32_t below = (1u << lane) - 1;

  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.digit_bits;
    const uint32_t* from_keys = a.keys[(pass + 1) & 1];
    const uint32_t* from_pos = a.pos[(pass + 1) & 1];
    uint32_t* to_keys = a.keys[pass & 1];
    uint32_t* to_pos = a.pos[pass & 1];
    auto key_at = [&](int64_t i) -> uint32_t {
      if (pass) return __ldcg(from_keys + i);
      const int64_t t = token_at(a.tokens, a.token_bytes, i);
      return t >= 0 && t < a.V ? uint32_t(t) : uint32_t(a.V);
    };
    for (int b = tid; b < bins * 33; b += kSortThreads) counts[b] = 0;
    __syncthreads();
    for (int64_t i = i0; i < i1; i += 32) {
      const bool on = i + lane < i1;
      const uint32_t d = on ? key_at(i + lane) >> shift & (bins - 1) : 0xffffffffu;
      if (!pass && on && token_at(a.tokens, a.token_bytes, i + lane) >= a.V) atomicOr(a.status, kStatusBadIndex);
      const uint32_t same = __match_any_sync(~0u, d);
      if (on && !(same & below)) counts[d * 33 + warp] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // bin b's counts to starts within this CTA's part of the bin
    if (tid < bins) {
      uint32_t run = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = counts[tid * 33 + w];
        counts[tid * 33 + w] = run;
        run += c;
      }
      total[tid] = run;
    }
    cluster_sync();
    uint32_t all = 0, before = 0;
    if (tid < bins)
      for (uint32_t c = 0; c < kSortCtas; ++c) {
        uint32_t n;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(n) : "r"(map_to_rank(smem_addr(total + tid), c)) : "memory");
        all += n;
        before += c < cta ? n : 0;
      }
    // exclusive sum over the bins
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    uint32_t w = lane < warp ? sums[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(~0u, w, o);
    if (tid < bins) base[tid] = w + incl - all + before;
    __syncthreads();
    for (int64_t i = i0; i < i1; i += 32) {
      const bool on = i + lane < i1;
      const uint32_t key = on ? key_at(i + lane) : 0, d = on ? key >> shift & (bins - 1) : 0xffffffffu;
      const uint32_t same = __match_any_sync(~0u, d);
      if (on) {
        const uint32_t to = base[d] + counts[d * 33 + warp] + __popc(same & below);
        to_keys[to] = key;
        to_pos[to] = pass ? __ldcg(from_pos + i + lane) : uint32_t(i + lane);
      }
      __syncwarp();
      if (on && !(same & below)) counts[d * 33 + warp] += __popc(same);
      __syncwarp();
    }
    cluster_sync();
  }
  if (a.accumulate) return;
  const int64_t words = (a.V + 31) / 32;
  for (int64_t i = int64_t(cta) * kSortThreads + tid; i < words; i += kSortCtas * kSortThreads) a.bits[i] = 0;
  cluster_sync();
  for (int64_t i = int64_t(cta) * kSortThreads + tid; i < a.T; i += kSortCtas * kSortThreads) {
    const uint32_t key = __ldcg(a.sorted_keys + i);
    if (key < a.V && (i == 0 || __ldcg(a.sorted_keys + i - 1) != key)) atomicOr(a.bits + key / 32, 1u << key % 32);
  }
}

// ---- gradient: the sums ---------------------------------------------------------------------------------------------

// E sums to elements u * E .. of row v of the gradient.
template <class G, bool VEC, int E>
__device__ __forceinline__ void write_grad(const GradArgs& a, uint32_t v, int64_t u, const float (&sum)[E]) {
  unsigned char* at = a.g + int64_t(v) * a.g_pitch + u * (E * G::kBytes);
  float y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = sum[e] * a.scale;
  if constexpr (VEC) {
    constexpr int n = E / G::kVec;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      float part[G::kVec];
      if (a.accumulate) {
        float old[G::kVec];
        G::unpack(ld16(at + k * 16), old);
#pragma unroll
        for (int e = 0; e < G::kVec; ++e) part[e] = __fmaf_rn(sum[k * G::kVec + e], a.scale, old[e]);
      } else {
#pragma unroll
        for (int e = 0; e < G::kVec; ++e) part[e] = y[k * G::kVec + e];
      }
      st_stream16(at + k * 16, G::pack(part));
    }
  } else {
    if (a.accumulate) y[0] = __fmaf_rn(sum[0], a.scale, G::load1(at, 0));
    G::store1(at, 0, y[0]);
  }
}

constexpr int kRowThreads = 128, kAhead = 8;

template <class D, class G, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_embedding_rows(GradArgs a) {
  constexpr int E = VEC ? D::kVec : 1;
  const int64_t chunk_ctas = a.chunks * a.slices;
  if (blockIdx.x >= chunk_ctas) {
    // rows without a token
    const int64_t v0 = (blockIdx.x - chunk_ctas) * a.fill_rows, v1 = v0 + a.fill_rows < a.V ? v0 + a.fill_rows : a.V;
    for (int64_t v = v0; v < v1; ++v) {
      if (a.bits[v / 32] >> (v % 32) & 1) continue;
      unsigned char* row = a.g + v * a.g_pitch;
      if (a.fill_vec)
        for (int64_t o = threadIdx.x * 16; o < a.D * G::kBytes; o += kRowThreads * 16) st_stream16(row + o, make_uint4(0, 0, 0, 0));
      else
        for (int64_t i = threadIdx.x; i < a.D; i += kRowThreads) G::store1(row, i, 0.f);
    }
    return;
  }
  __shared__ uint32_t keys[kChunk + 2], pos[kChunk];
  const int64_t chunk = blockIdx.x / a.slices, first = chunk * kChunk;
  const int64_t u = (blockIdx.x - chunk * a.slices) * int64_t(kRowThreads) + threadIdx.x;
  if (threadIdx.x < kChunk + 2) {
    const int64_t i = first + int(threadIdx.x) - 1;
    keys[threadIdx.x] = i >= 0 && i < a.T ? a.sorted_keys[i] : 0xffffffffu;
    if (threadIdx.x >= 1 && threadIdx.x <= kChunk && i < a.T) pos[threadIdx.x - 1] = a.sorted_pos[i];
  }
  __syncthreads();
  if (u >= a.units) return;
  const unsigned char* column = a.dy + u * (E * D::kBytes);
  float sum[E] = {};
  bool head = keys[0] == keys[1];  // the run came from the chunk before
  for (int i = 0; i < kChunk && keys[i + 1] < a.V; i += kAhead) {
    uint4 q[kAhead];
    float s[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (keys[i + j + 1] < a.V) {
        const unsigned char* at = column + int64_t(pos[i + j]) * a.dy_pitch;
        if constexpr (VEC) q[j] = ld_stream16(at);
        else s[j] = D::load1(at, 0);
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t key = keys[i + j + 1], next = keys[i + j + 2];
      if (key >= a.V) break;
      if constexpr (VEC) {
        float f[E];
        D::unpack(q[j], f);
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] += f[e];
      } else {
        sum[0] += s[j];
      }
      const bool last = i + j + 1 == kChunk;
      if (next == key && !last) continue;
      if (head || (last && next == key)) {
        float* part = a.parts + (chunk * 2 + (head ? 0 : 1)) * a.part_pitch + u * E;
#pragma unroll
        for (int e = 0; e < E; ++e) part[e] = sum[e];
      } else {
        write_grad<G, VEC, E>(a, key, u, sum);
      }
      head = false;
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] = 0.f;
    }
  }
}

// Runs that go over the end of the chunk they begin in: a CTA takes 32 columns of one, eight warps every eighth partial sum.
constexpr int kJoinWarps = 8;

template <class G>
__global__ void __launch_bounds__(kJoinWarps * 32) k_embedding_join(GradArgs a) {
  const int64_t chunk = blockIdx.x, end = (chunk + 1) * kChunk;
  if (end >= a.T) return;
  const uint32_t key = a.sorted_keys[end];
  if (key >= a.V || a.sorted_keys[end - 1] != key) return;
  if (chunk > 0 && a.sorted_keys[chunk * kChunk] == key && a.sorted_keys[chunk * kChunk - 1] == key) return;  // began earlier
  // the last chunk that the run reaches: its first token is the run's
  int64_t lo = chunk + 1, step = 1;
  while (lo + step < a.chunks && a.sorted_keys[(lo + step) * kChunk] == key) {
    lo += step;
    step *= 2;
  }
  int64_t hi = lo + step < a.chunks ? lo + step : a.chunks;  // lo is the run's, hi is not
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (a.sorted_keys[mid * kChunk] == key) lo = mid;
    else hi = mid;
  }
  const int64_t n = lo - chunk + 1;  // parts: the chunk's second, then the first of each that follows
  __shared__ float sums[kJoinWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t c0 = int64_t(blockIdx.y) * 32; c0 < a.D; c0 += int64_t(gridDim.y) * 32) {
    const int64_t c = c0 + lane;
    float sum = 0.f;
    if (c < a.D)
      for (int64_t k = warp; k < n; k += kJoinWarps) sum += a.parts[((chunk + k) * 2 + (k == 0)) * a.part_pitch + c];
    __syncthreads();
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < a.D) {
      float one[1] = {0.f};
      for (int w = 0; w < kJoinWarps; ++w) one[0] += sums[w][lane];
      write_grad<G, false, 1>(a, key, c, one);
    }
  }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace: keys and positions twice, the bit map, the partial sums.
struct Scratch {
  size_t list, bits, parts, bytes;
  int64_t part_pitch, chunks;
};
Scratch scratch_of(int64_t T, int64_t V, int64_t D) {
  Scratch s;
  s.list = up256(size_t(T) * 4);
  s.bits = up256(size_t((V + 31) / 32) * 4);
  s.part_pitch = (D + 7) / 8 * 8;
  s.chunks = (T + kChunk - 1) / kChunk;
  s.parts = up256(size_t(s.chunks) * 2 * size_t(s.part_pitch) * 4);
  s.bytes = 4 * s.list + s.bits + s.parts + 256;
  return s;
}

template <class D, class G>
cudaError_t launch_grad(const EmbeddingGrad& p, const DeviceInfo& dev) {
  const Scratch s = scratch_of(p.T, p.V, p.D);
  GradArgs a{};
  a.dy = static_cast<const unsigned char*>(p.dy);
  a.g = static_cast<unsigned char*>(p.grad);
  a.tokens = p.tokens;
  unsigned char* w = static_cast<unsigned char*>(p.workspace);
  for (int k = 0; k < 2; ++k) {
    a.keys[k] = reinterpret_cast<uint32_t*>(w + 2 * k * s.list);
    a.pos[k] = reinterpret_cast<uint32_t*>(w + (2 * k + 1) * s.list);
  }
  a.bits = reinterpret_cast<uint32_t*>(w + 4 * s.list);
  a.parts = reinterpret_cast<float*>(w + 4 * s.list + s.bits);
  a.T = p.T;
  a.V = p.V;
  a.D = p.D;
  a.dy_pitch = p.dy_pitch * D::kBytes;
  a.g_pitch = p.g_pitch * G::kBytes;
  a.part_pitch = s.part_pitch;
  a.chunks = s.chunks;
  a.token_bytes = p.token_bytes;
  int bits = 1;
  while (p.V >> bits) ++bits;  // keys 0 .. V
  a.passes = (bits + kDigitBits - 1) / kDigitBits;
  a.digit_bits = (bits + a.passes - 1) / a.passes;
  a.sorted_keys = a.keys[(a.passes - 1) & 1];
  a.sorted_pos = a.pos[(a.passes - 1) & 1];
  a.scale = p.scale;
  a.accumulate = p.accumulate;
  a.status = dev.status;
  const bool grad16 = ((reinterpret_cast<uintptr_t>(a.g) | uintptr_t(a.g_pitch) | uintptr_t(p.D * G::kBytes)) & 15) == 0;
  const bool vec = grad16 && ((reinterpret_cast<uintptr_t>(a.dy) | uintptr_t(a.dy_pitch) | uintptr_t(p.D * D::kBytes)) & 15) == 0;
  a.fill_vec = grad16;
  a.units = uint32_t(vec ? p.D / D::kVec : p.D);
  a.slices = int((a.units + kRowThreads - 1) / kRowThreads);
  a.fill_rows = (65536 + p.D * G::kBytes - 1) / (p.D * G::kBytes);
  const int64_t fill = p.accumulate ? 0 : (p.V + a.fill_rows - 1) / a.fill_rows;
  cudaError_t e;
  const size_t shared = (size_t(1) << a.digit_bits) * 35 * 4;
  if ((e = cudaFuncSetAttribute(k_sort_tokens, cudaFuncAttributeMaxDynamicSharedMemorySize, int(shared))) != cudaSuccess) return e;
  k_sort_tokens<<<kSortCtas, kSortThreads, shared, p.stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t ctas = a.chunks * a.slices + fill;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (ctas > 0) {
    if (vec) k_embedding_rows<D, G, true><<<unsigned(ctas), kRowThreads, 0, p.stream>>>(a);
    else k_embedding_rows<D, G, false><<<unsigned(ctas), kRowThreads, 0, p.stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (a.chunks > 1) {
    const int64_t columns = (p.D + 31) / 32;
    k_embedding_join<G><<<dim3(unsigned(a.chunks), unsigned(columns < 1024 ? columns : 1024)), kJoinWarps * 32, 0, p.stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embedding(const Embedding& p, const DeviceInfo& dev) {
  return p.dtype == SOFTMAX_F32 ? launch_lookup<F32>(p, dev) : p.dtype == SOFTMAX_BF16 ? launch_lookup<BF16>(p, dev) : launch_lookup<F16>(p, dev);
}

size_t embedding_grad_scratch(int64_t T, int64_t V, int64_t D) { return scratch_of(T, V, D).bytes; }

cudaError_t launch_embedding_grad(const EmbeddingGrad& p, const DeviceInfo& dev) {
  if (p.dtype == SOFTMAX_F32) return launch_grad<F32, F32>(p, dev);
  if (p.dtype == SOFTMAX_BF16) return p.grad_dtype == SOFTMAX_F32 ? launch_grad<BF16, F32>(p, dev) : launch_grad<BF16, BF16>(p, dev);
  return p.grad_dtype == SOFTMAX_F32 ? launch_grad<F16, F32>(p, dev) : launch_grad<F16, F16>(p, dev);
}

}  // namespace rwo
