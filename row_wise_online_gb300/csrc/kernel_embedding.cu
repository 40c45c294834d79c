// kernel_embedding.cu -- embedding lookup and its gradient.
//
// Lookup: y_t = scale * table[token_t], a copy of rows.
//
// Gradient: grad_v = scale * sum of dy_t over the t with token_t = v.  The tokens are sorted with their positions
// (k_rank_tokens: few tokens, each counts those that come before it; k_sort_tokens: a stable radix sort by one thread-block
// cluster), so that the rows of a token are one run of the sorted list.  The list is cut into chunks of some tokens, whatever
// the runs: a CTA takes a chunk's columns and adds up the runs in it (k_embedding_rows).  A run inside a chunk is written at
// once; one that goes on into the next chunk leaves partial sums, which k_embedding_join adds up in their order.  So a frequent
// token is spread over the GPU as others are, no atomics touch the sums, and their order is a function of the tokens alone.
// Rows without a token are zeroed by the same launch, from a bit map that the sort leaves.
#include <initializer_list>

#include "train.cuh"
#include "train.h"

namespace rwo {
namespace {

constexpr int kMostChunk = 32;  // tokens of a chunk at most

// Tokens of a chunk: 32, fewer where that would leave SMs without one (1500 tokens of 512 elements: 8).
int chunk_of(int64_t T, int64_t D) {
  int c = kMostChunk;
  while (c > 8 && (T + c - 1) / c * ((D + 1023) / 1024) < 512) c /= 2;
  return c;
}

constexpr int kStaticShared = 1024;  // more than the sort has
constexpr int kSortThreads = 1024, kSortWarps = 32, kSortCtas = 16;
constexpr int kDigitBits = 10;

__device__ __forceinline__ int64_t token_at(const void* tokens, int bytes, int64_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(tokens)[i] : int64_t(static_cast<const int32_t*>(tokens)[i]);
}

// ---- lookup ---------------------------------------------------------------------------------------------------------

struct LookupArgs {
  const unsigned char* table;
  unsigned char* y;
  const void* tokens;
  int64_t T, V, D;
  int64_t table_pitch, y_pitch;  // bytes
  int64_t pieces;                // of a row
  int units;                     // vectors of a row
  int token_bytes;
  float scale;
  unsigned* status;
};

constexpr int kLookupThreads = 256;

// The value of an element of a row that no table row gives: 0 for padding, else NaN.
template <class D>
__device__ __forceinline__ uint4 no_row(int64_t token) {
  const float f = token < 0 ? 0.f : __int_as_float(0x7fc00000);
  float2 v[D::kVec / 2];
#pragma unroll
  for (int e = 0; e < D::kVec / 2; ++e) v[e] = make_float2(f, f);
  return D::pack2(v);
}
template <class D>
__device__ __forceinline__ uint4 times(const uint4& q, float scale) {
  const float2 s = make_float2(scale, scale);
  float2 v[D::kVec / 2];
  D::unpack2(q, v);
#pragma unroll
  for (int e = 0; e < D::kVec / 2; ++e) v[e] = __fmul2_rn(v[e], s);
  return D::pack2(v);
}

// Short rows on 16-byte boundaries: 2^shift lanes a row, kLookupRows rows a lane at a time (200000 rows of 64 bf16 elements: 12 to 14 us,
// a warp a row 43).
constexpr int kLookupRows = 4;

template <class D>
__global__ void __launch_bounds__(kLookupThreads) k_embedding_short(LookupArgs a, int shift) {
  const int64_t step = int64_t(gridDim.x) * kLookupThreads >> shift, thread = int64_t(blockIdx.x) * kLookupThreads + threadIdx.x;
  const int u = int(thread & ((1 << shift) - 1));
  if (u >= a.units) return;
  for (int64_t t0 = thread >> shift; t0 < a.T; t0 += step * kLookupRows) {
    int64_t token[kLookupRows];
    uint4 q[kLookupRows];
#pragma unroll
    for (int k = 0; k < kLookupRows; ++k) token[k] = t0 + k * step < a.T ? token_at(a.tokens, a.token_bytes, t0 + k * step) : -1;
#pragma unroll
    for (int k = 0; k < kLookupRows; ++k) {
      if (token[k] >= 0 && token[k] < a.V) {
        q[k] = times<D>(ld_stream16(a.table + token[k] * a.table_pitch + u * 16), a.scale);
      } else {
        if (token[k] >= 0 && u == 0) atomicOr(a.status, kStatusBadIndex);
        q[k] = no_row<D>(token[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kLookupRows; ++k)
      if (t0 + k * step < a.T) st_stream16(a.y + (t0 + k * step) * a.y_pitch + u * 16, q[k]);
  }
}

// A warp moves pieces of rows: kLookupPer vectors a lane, all loaded before the first is stored, and the next piece's token is
// under way meanwhile.
template <class D, bool SHIFT, int kLookupPer>
__global__ void __launch_bounds__(kLookupThreads, kLookupPer == 8 ? 4 : kLookupPer == 4 ? 5 : 6) k_embedding(LookupArgs a) {
  const int lane = threadIdx.x & 31, n = int(a.D);
  const int64_t warps = int64_t(gridDim.x) * (kLookupThreads / 32), items = a.T * a.pieces;
  const Bytes table = bytes_of(a.table, a.V, a.table_pitch, a.D * D::kBytes);
  int64_t item = int64_t(blockIdx.x) * (kLookupThreads / 32) + (threadIdx.x >> 5);
  if (item >= items) return;
  int64_t t = item / a.pieces;
  int64_t next = token_at(a.tokens, a.token_bytes, t);
  while (true) {
    const int64_t token = next;
    const int u0 = int(item - t * a.pieces) * (kLookupPer * 32) + lane;
    unsigned char* to = a.y + t * a.y_pitch;
    item += warps;
    t = item / a.pieces;
    if (item < items) next = token_at(a.tokens, a.token_bytes, t);
    uint4 q[kLookupPer];
    const bool real = token >= 0 && token < a.V;
    if (real) {
      const RowAt r = row_at<D>(a.table + token * a.table_pitch, n, table);
      if constexpr (SHIFT) {
        load_vectors<D>(r, u0, q);
      } else {
#pragma unroll
        for (int k = 0; k < kLookupPer; ++k)
          if (u0 + k * 32 < a.units) q[k] = ld_stream16(r.row + int64_t(u0 + k * 32) * 16);
      }
      if (a.scale != 1.f) {
#pragma unroll
        for (int k = 0; k < kLookupPer; ++k) q[k] = times<D>(q[k], a.scale);
      }
    } else {
      if (token >= 0 && u0 == 0) atomicOr(a.status, kStatusBadIndex);
#pragma unroll
      for (int k = 0; k < kLookupPer; ++k) q[k] = no_row<D>(token);
    }
    if constexpr (SHIFT) {
      store_vectors<D>(to, u0, n, q);
    } else {
#pragma unroll
      for (int k = 0; k < kLookupPer; ++k)
        if (u0 + k * 32 < a.units) st_stream16(to + int64_t(u0 + k * 32) * 16, q[k]);
    }
    if (item >= items) return;
  }
}

bool on16(std::initializer_list<uintptr_t> v) {
  uintptr_t all = 0;
  for (const uintptr_t x : v) all |= x;
  return (all & 15) == 0;
}

template <class D>
cudaError_t launch_lookup(const Embedding& p, const DeviceInfo& dev) {
  LookupArgs a;
  a.table = static_cast<const unsigned char*>(p.table);
  a.y = static_cast<unsigned char*>(p.y);
  a.tokens = p.tokens;
  a.T = p.T;
  a.V = p.V;
  a.D = p.D;
  a.table_pitch = p.table_pitch * D::kBytes;
  a.y_pitch = p.y_pitch * D::kBytes;
  a.token_bytes = p.token_bytes;
  a.scale = p.scale;
  a.status = dev.status;
  const bool vec = on16({reinterpret_cast<uintptr_t>(a.table), reinterpret_cast<uintptr_t>(a.y), uintptr_t(a.table_pitch), uintptr_t(a.y_pitch),
                         uintptr_t(p.D * D::kBytes)});
  a.units = int((p.D + D::kVec - 1) / D::kVec);
  if (vec && a.units <= 16) {
    int shift = 0;
    while (1 << shift < a.units) ++shift;
    const int64_t per = int64_t(kLookupThreads >> shift) * kLookupRows, most = int64_t(dev.sm_count) * (dev.max_threads_per_sm / kLookupThreads);
    const int64_t ctas = (p.T + per - 1) / per;
    k_embedding_short<D><<<unsigned(ctas < most ? ctas : most), kLookupThreads, 0, p.stream>>>(a, shift);
    return cudaGetLastError();
  }
  const int held = a.units <= 64 ? 2 : a.units <= 128 ? 4 : 8;  // vectors of a lane
  a.pieces = (a.units + held * 32 - 1) / (held * 32);
  const int64_t per = kLookupThreads / 32, most = int64_t(dev.sm_count) * (held == 8 ? 4 : held == 4 ? 5 : 6);
  const int64_t ctas = p.T > most * per ? most : (p.T * a.pieces + per - 1) / per;
  const unsigned grid = unsigned(ctas < most ? ctas : most);
  const auto fn = vec ? (held == 8 ? k_embedding<D, false, 8> : held == 4 ? k_embedding<D, false, 4> : k_embedding<D, false, 2>)
                      : (held == 8 ? k_embedding<D, true, 8> : held == 4 ? k_embedding<D, true, 4> : k_embedding<D, true, 2>);
  fn<<<grid, kLookupThreads, 0, p.stream>>>(a);
  return cudaGetLastError();
}

// ---- gradient: the sort ---------------------------------------------------------------------------------------------

// A run of equal tokens over many chunks: where it begins, and its partial sums.
struct LongRun {
  int64_t chunk, parts;
};

struct GradArgs {
  const unsigned char* dy;
  unsigned char* g;
  const void* tokens;
  uint32_t* keys[2];
  uint32_t* pos[2];
  const uint32_t* sorted_keys;
  const uint32_t* sorted_pos;
  uint32_t* bits;  // rows that a token names
  uint32_t* long_count;
  LongRun* long_runs;
  float* parts;    // [chunk][2][part_pitch]: sums of the run that came from the chunk before, of the one that goes on
  int64_t T, V, D;
  int64_t dy_pitch, g_pitch;  // bytes
  int64_t part_pitch;         // floats
  int64_t chunks;
  int64_t groups;             // of chunks that a CTA has
  int chunk;                  // tokens of one
  bool small;                 // rows of at most 32 vectors: a warp a chunk
  int units;                  // vectors of a row of dy
  int slices;                 // CTAs of a chunk
  int64_t fill_rows;          // rows of a zeroing CTA
  int token_bytes, passes, digit_bits;
  float scale;
  bool accumulate, fill_vec;
  unsigned* status;
};

// The token's key: its row, or V where it names none; such keys end up last.
__device__ __forceinline__ uint32_t key_of(const GradArgs& a, int64_t i) {
  const int64_t t = token_at(a.tokens, a.token_bytes, i);
  if (t >= a.V) atomicOr(a.status, kStatusBadIndex);
  return t >= 0 && t < a.V ? uint32_t(t) : uint32_t(a.V);
}

// Few tokens: a warp a token counts the keys before its own (smaller, or equal and earlier), which is the token's place.  Every
// CTA also makes its part of the bit map.  1500 tokens take 7 us, the radix sort's two passes 13.
constexpr int kRankTokens = 4096, kRankWords = 8192;

__global__ void __launch_bounds__(kSortThreads) k_rank_tokens(GradArgs a) {
  __shared__ uint32_t keys[kRankTokens];
  __shared__ uint32_t bits[kRankWords];
  griddep_launch();
  const int n = int(a.T), tid = threadIdx.x, lane = tid & 31;
  const int64_t words = (a.V + 31) / 32, mine = (words + gridDim.x - 1) / gridDim.x;
  const int64_t w0 = blockIdx.x * mine < words ? blockIdx.x * mine : words, w1 = w0 + mine < words ? w0 + mine : words;
  if (blockIdx.x == 0 && tid == 0) *a.long_count = 0;
  for (int i = tid; i < n; i += kSortThreads) keys[i] = key_of(a, i);
  for (int w = tid; w < int(w1 - w0); w += kSortThreads) bits[w] = 0;
  __syncthreads();
  if (!a.accumulate) {
    for (int i = tid; i < n; i += kSortThreads) {
      const int64_t w = int64_t(keys[i] / 32) - w0;
      if (keys[i] < a.V && w >= 0 && w < w1 - w0) atomicOr(bits + w, 1u << keys[i] % 32);
    }
    __syncthreads();
    for (int w = tid; w < int(w1 - w0); w += kSortThreads) a.bits[w0 + w] = bits[w];
  }
  for (int i = int(blockIdx.x) * kSortWarps + (tid >> 5); i < n; i += int(gridDim.x) * kSortWarps) {
    const uint32_t key = keys[i];
    int before = 0;
    for (int j = lane; j < n; j += 32) before += keys[j] < key || (keys[j] == key && j < i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(~0u, before, o);
    if (lane == 0) {
      a.keys[0][before] = key;
      a.pos[0][before] = uint32_t(i);
    }
  }
}

// Least significant digit first, digits of digit_bits.  A warp owns a run of the list and a column of counts; ranks
// within 32 tokens come from a vote (lanes of the same digit), so equal tokens keep their order.  A run is loaded kRun tokens a
// lane at a time, and stays in registers between counting and moving where that is all of it.
constexpr int kRun = 8;

// The lanes whose digit is this lane's, of those that have one.  A vote for each bit (32768 tokens over 8 CTAs: 31 us;
// with __match_any_sync 33; over 16 CTAs 25).
__device__ __forceinline__ uint32_t alike(uint32_t digit, bool on, int bits) {
  uint32_t same = __ballot_sync(~0u, on);
#pragma unroll
  for (int b = 0; b < kDigitBits; ++b) {
    if (b >= bits) break;
    const uint32_t ones = __ballot_sync(~0u, digit >> b & 1);
    same &= digit >> b & 1 ? ones : ~ones;
  }
  return same;
}

__global__ void __launch_bounds__(kSortThreads) k_sort_tokens(GradArgs a) {
  extern __shared__ uint32_t shared[];
  const int bins = 1 << a.digit_bits, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* total = shared;                             // [bins], read by the cluster's other CTAs
  uint32_t* base = total + bins;                        // [bins]
  uint32_t* counts = base + bins;                       // [bins][33]: a warp's counts, then where they start
  __shared__ uint32_t sums[kSortWarps];
  griddep_launch();
  const uint32_t cta = cluster_ctarank();
  const int64_t per = ((a.T + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) / 32 * 32;
  const int64_t i0 = (int64_t(cta) * kSortWarps + warp) * per < a.T ? (int64_t(cta) * kSortWarps + warp) * per : a.T;
  const int64_t i1 = i0 + per < a.T ? i0 + per : a.T;
  const uint32_t below = (1u << lane) - 1;
  const bool whole = per <= kRun * 32;

  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.digit_bits;
    const uint32_t* from_keys = a.keys[(pass + 1) & 1];
    const uint32_t* from_pos = a.pos[(pass + 1) & 1];
    uint32_t* to_keys = a.keys[pass & 1];
    uint32_t* to_pos = a.pos[pass & 1];
    uint32_t key[kRun], pos[kRun];
    const auto load = [&](int64_t i, bool positions) {
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const int64_t at = i + k * 32 + lane;
        key[k] = pos[k] = 0;
        if (at >= i1) continue;
        key[k] = pass ? __ldcg(from_keys + at) : key_of(a, at);
        if (positions) pos[k] = pass ? __ldcg(from_pos + at) : uint32_t(at);
      }
    };
    if (whole) load(i0, true);
    for (int b = tid; b < bins * 33; b += kSortThreads) counts[b] = 0;
    __syncthreads();
    for (int64_t i = i0; i < i1; i += kRun * 32) {
      if (!whole) load(i, false);
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        if (i + k * 32 >= i1) break;
        const bool on = i + k * 32 + lane < i1;
        const uint32_t d = key[k] >> shift & (bins - 1);
        const uint32_t same = alike(d, on, a.digit_bits);
        if (on && !(same & below)) counts[d * 33 + warp] += __popc(same);
        __syncwarp();
      }
    }
    __syncthreads();
    // bin b's counts to starts within this CTA's part of the bin
    if (tid < bins) {
      uint32_t run = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = counts[tid * 33 + w];
        counts[tid * 33 + w] = run;
        run += c;
      }
      total[tid] = run;
    }
    cluster_sync();
    uint32_t all = 0, before = 0;
    if (tid < bins) {
      uint32_t n[kSortCtas];
#pragma unroll
      for (uint32_t c = 0; c < kSortCtas; ++c)
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(n[c]) : "r"(map_to_rank(smem_addr(total + tid), c)) : "memory");
#pragma unroll
      for (uint32_t c = 0; c < kSortCtas; ++c) {
        all += n[c];
        before += c < cta ? n[c] : 0;
      }
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
    for (int64_t i = i0; i < i1; i += kRun * 32) {
      if (!whole) load(i, true);
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        if (i + k * 32 >= i1) break;
        const bool on = i + k * 32 + lane < i1;
        const uint32_t d = key[k] >> shift & (bins - 1);
        const uint32_t same = alike(d, on, a.digit_bits);
        if (on) {
          const uint32_t to = base[d] + counts[d * 33 + warp] + __popc(same & below);
          to_keys[to] = key[k];
          to_pos[to] = pos[k];
        }
        __syncwarp();
        if (on && !(same & below)) counts[d * 33 + warp] += __popc(same);
        __syncwarp();
      }
    }
    cluster_sync();
  }
  if (cta == 0 && tid == 0) *a.long_count = 0;
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

// A vector's sums, times scale, into vector u of a row of the gradient (or added to it), of the gradient's type.
template <class G, bool SHIFT>
__device__ __forceinline__ void write_vector(const GradArgs& a, unsigned char* row, int u, const float (&sum)[G::kVec], const Bytes& m) {
  const int n = int(a.D);
  float y[G::kVec];
  if (a.accumulate) {
    uint4 old[1] = {};
    if constexpr (SHIFT) load_vectors<G>(row_at<G>(row, n, m), u, old);
    else if (u * G::kVec < n) old[0] = ld16(row + int64_t(u) * 16);
    G::unpack(old[0], y);
#pragma unroll
    for (int e = 0; e < G::kVec; ++e) y[e] = __fmaf_rn(sum[e], a.scale, y[e]);
  } else {
#pragma unroll
    for (int e = 0; e < G::kVec; ++e) y[e] = sum[e] * a.scale;
  }
  const uint4 q[1] = {G::pack(y)};
  if constexpr (SHIFT) store_vectors<G>(row, u, n, q);
  else if (u * G::kVec < n) st_stream16(row + int64_t(u) * 16, q[0]);
}

// E sums a lane, of elements u * E .. of row v; all lanes of a warp, with consecutive u.
template <class G, bool SHIFT, int E>
__device__ __forceinline__ void write_grad(const GradArgs& a, uint32_t v, int u, const float (&sum)[E], const Bytes& m) {
  unsigned char* row = a.g + int64_t(v) * a.g_pitch;
  if constexpr (E == G::kVec) {
    write_vector<G, SHIFT>(a, row, u, sum, m);
  } else {
    // sixteen bits into 32: a lane's elements are two vectors.  Each half of the warp's elements is dealt out, a vector a lane.
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float part[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = __shfl_sync(~0u, sum[e], half * 16 + lane / 2), hi = __shfl_sync(~0u, sum[e + 4], half * 16 + lane / 2);
        part[e] = lane & 1 ? hi : lo;
      }
      write_vector<G, SHIFT>(a, row, (u - lane) * 2 + half * 32 + lane, part, m);
    }
  }
}

constexpr int kRowThreads = 128, kAhead = 8;

template <class D, class G, bool SHIFT>
__global__ void __launch_bounds__(kRowThreads) k_embedding_rows(GradArgs a) {
  constexpr int E = D::kVec;
  griddep_wait();
  griddep_launch();
  const int64_t chunk_ctas = a.groups * a.slices;
  if (blockIdx.x >= chunk_ctas) {
    // rows without a token
    const int64_t v0 = (blockIdx.x - chunk_ctas) * a.fill_rows, v1 = v0 + a.fill_rows < a.V ? v0 + a.fill_rows : a.V;
    const uint32_t per = uint32_t(a.fill_vec ? a.D * G::kBytes / 16 : a.D), rows = uint32_t(v1 - v0);
    uint32_t row = threadIdx.x / per, at = threadIdx.x - row * per;  // vectors, or elements, of the rows in one line
    const uint32_t rows_on = kRowThreads / per, at_on = kRowThreads - rows_on * per;
    while (row < rows) {
      const int64_t v = v0 + row;
      if (!(a.bits[v / 32] >> (v % 32) & 1)) {
        unsigned char* to = a.g + v * a.g_pitch;
        if (a.fill_vec) st_stream16(to + int64_t(at) * 16, make_uint4(0, 0, 0, 0));
        else G::store1(to, at, 0.f);
      }
      row += rows_on;
      at += at_on;
      if (at >= per) {
        at -= per;
        ++row;
      }
    }
    return;
  }
  // a CTA has a chunk's columns, or, of short rows, a warp has a chunk
  __shared__ uint32_t all_keys[kRowThreads / 32][kMostChunk + 2], all_pos[kRowThreads / 32][kMostChunk];
  const int part = a.small ? int(threadIdx.x) >> 5 : 0, t = a.small ? int(threadIdx.x) & 31 : int(threadIdx.x);
  const int64_t group = blockIdx.x / a.slices, chunk = a.small ? group * (kRowThreads / 32) + part : group, first = chunk * a.chunk;
  const int u = int(blockIdx.x - group * a.slices) * kRowThreads + t;
  uint32_t* keys = all_keys[part];
  uint32_t* pos = all_pos[part];
  for (int k = t; k < a.chunk + 2; k += a.small ? 32 : kRowThreads) {
    const int64_t i = first + k - 1;
    keys[k] = i >= 0 && i < a.T ? a.sorted_keys[i] : 0xffffffffu;
    if (k >= 1 && k <= a.chunk && i < a.T) pos[k - 1] = a.sorted_pos[i];
  }
  __syncthreads();
  if ((u & ~31) >= a.units || chunk >= a.chunks) return;  // warps stay whole
  const int n = int(a.D);
  const Bytes dm = bytes_of(a.dy, a.T, a.dy_pitch, a.D * D::kBytes), gm = bytes_of(a.g, a.V, a.g_pitch, a.D * G::kBytes);
  float sum[E] = {};
  bool head = keys[0] == keys[1];  // the run came from the chunk before
  for (int i = 0; i < a.chunk && keys[i + 1] < a.V; i += kAhead) {
    uint4 q[kAhead][1];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (keys[i + j + 1] >= a.V) continue;
      const unsigned char* row = a.dy + int64_t(pos[i + j]) * a.dy_pitch;
      if constexpr (SHIFT) load_vectors<D>(row_at<D>(row, n, dm), u, q[j]);
      else q[j][0] = u < a.units ? ld_stream16(row + int64_t(u) * 16) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t key = keys[i + j + 1], next = keys[i + j + 2];
      if (key >= a.V) break;
      float f[E];
      D::unpack(q[j][0], f);
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += f[e];
      const bool last = i + j + 1 == a.chunk;
      if (next == key && !last) continue;
      if (head || (last && next == key)) {
        float* part = a.parts + (chunk * 2 + (head ? 0 : 1)) * a.part_pitch + int64_t(u) * E;
        if (u < a.units) {
#pragma unroll
          for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(part + e) = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
        }
      } else {
        write_grad<G, SHIFT, E>(a, key, u, sum, gm);
      }
      head = false;
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] = 0.f;
    }
  }
}

// Runs that go over the end of the chunk they begin in: a warp looks at one chunk for its run, and adds up the partial sums.  Runs
// of many parts it puts on a list for k_embedding_long, where 32 warps share one's (262144 tokens of which 43000 are one: 510 us
// with the CTA's eight warps here).
constexpr int kJoinWarps = 8, kJoinColumns = 128;  // columns of a warp at a time, four a lane
constexpr int kLongWarps = 32, kLongCtas = 32;
constexpr int kAlone = 16;          // parts of a run that one warp adds up ...
constexpr int64_t kFewChunks = 256;  // ... or all of them, where no run can have more parts than this

template <class G>
__device__ __forceinline__ void write_four(const GradArgs& a, uint32_t key, int64_t c, const float4& sum) {
  unsigned char* row = a.g + int64_t(key) * a.g_pitch;
  const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < a.D) G::store1(row, c + e, a.accumulate ? __fmaf_rn(v[e], a.scale, load1c<G>(row, c + e)) : v[e] * a.scale);
}
__device__ __forceinline__ void add(float4& a, const float4& b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }

// Four columns' sums of part k of the run that begins in chunk `first`: that chunk's second, then the first of each that follows.
__device__ __forceinline__ float4 part_of(const GradArgs& a, int64_t first, int64_t k, int64_t c) {
  return *reinterpret_cast<const float4*>(a.parts + ((first + k) * 2 + (k == 0)) * a.part_pitch + c);
}

template <class G>
__global__ void __launch_bounds__(kJoinWarps * 32) k_embedding_join(GradArgs a) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const uint32_t* keys = a.sorted_keys;
  const int64_t C = a.chunk, chunk = int64_t(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5), end = (chunk + 1) * C;
  if (end >= a.T) return;
  const uint32_t key = keys[end];
  if (key >= a.V || keys[end - 1] != key || (chunk > 0 && keys[chunk * C] == key && keys[chunk * C - 1] == key)) return;  // none begins here
  // the last chunk that the run reaches: its first token is the run's
  int64_t lo = chunk + 1, step = 1;
  while (lo + step < a.chunks && keys[(lo + step) * C] == key) {
    lo += step;
    step *= 2;
  }
  int64_t hi = lo + step < a.chunks ? lo + step : a.chunks;  // lo is the run's, hi is not
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (keys[mid * C] == key) lo = mid;
    else hi = mid;
  }
  const int64_t n = lo - chunk + 1;
  if (n > kAlone && a.chunks > kFewChunks) {
    if (blockIdx.y == 0 && lane == 0) a.long_runs[atomicAdd(a.long_count, 1u)] = LongRun{chunk, n};
    return;
  }
  for (int64_t c = int64_t(blockIdx.y) * kJoinColumns + lane * 4; c < a.D; c += int64_t(gridDim.y) * kJoinColumns) {
    float4 sum = make_float4(0, 0, 0, 0);
#pragma unroll 8
    for (int64_t k = 0; k < n; ++k) add(sum, part_of(a, chunk, k, c));
    write_four<G>(a, key, c, sum);
  }
}

template <class G>
__global__ void __launch_bounds__(kLongWarps * 32) k_embedding_long(GradArgs a) {
  __shared__ float4 sums[kLongWarps][32];
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t count = *a.long_count;
  for (uint32_t i = blockIdx.x; i < count; i += gridDim.x) {
    const LongRun run = a.long_runs[i];
    const uint32_t key = a.sorted_keys[(run.chunk + 1) * a.chunk];
    for (int64_t c0 = int64_t(blockIdx.y) * kJoinColumns; c0 < a.D; c0 += int64_t(gridDim.y) * kJoinColumns) {
      const int64_t c = c0 + lane * 4;
      float4 sum = make_float4(0, 0, 0, 0);
      if (c < a.D) {
#pragma unroll 8
        for (int64_t k = warp; k < run.parts; k += kLongWarps) add(sum, part_of(a, run.chunk, k, c));
      }
      __syncthreads();
      sums[warp][lane] = sum;
      __syncthreads();
      if (warp == 0 && c < a.D) {
        for (int w = 1; w < kLongWarps; ++w) add(sum, sums[w][lane]);
        write_four<G>(a, key, c, sum);
      }
    }
  }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace: keys and positions twice, the bit map, the partial sums.
struct Scratch {
  size_t list, bits, runs, parts, bytes;
  int64_t part_pitch, chunks;
  int chunk;
};
Scratch scratch_of(int64_t T, int64_t V, int64_t D) {
  Scratch s;
  s.list = up256(size_t(T) * 4);
  s.bits = up256(size_t((V + 31) / 32) * 4);
  s.part_pitch = (D + 7) / 8 * 8;
  s.chunk = chunk_of(T, D);
  s.chunks = (T + s.chunk - 1) / s.chunk;
  s.parts = up256(size_t(s.chunks) * 2 * size_t(s.part_pitch) * 4);
  s.runs = up256(size_t(s.chunks / kAlone + 1) * sizeof(LongRun));
  s.bytes = 4 * s.list + s.bits + s.parts + s.runs + 256;
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
  a.long_runs = reinterpret_cast<LongRun*>(w + 4 * s.list + s.bits + s.parts);
  a.long_count = reinterpret_cast<uint32_t*>(w + 4 * s.list + s.bits + s.parts + s.runs);
  a.T = p.T;
  a.V = p.V;
  a.D = p.D;
  a.dy_pitch = p.dy_pitch * D::kBytes;
  a.g_pitch = p.g_pitch * G::kBytes;
  a.part_pitch = s.part_pitch;
  a.chunks = s.chunks;
  a.chunk = s.chunk;
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
  a.fill_vec = on16({reinterpret_cast<uintptr_t>(a.g), uintptr_t(a.g_pitch), uintptr_t(p.D * G::kBytes)});
  const bool vec = a.fill_vec && on16({reinterpret_cast<uintptr_t>(a.dy), uintptr_t(a.dy_pitch), uintptr_t(p.D * D::kBytes)});
  a.units = int((p.D + D::kVec - 1) / D::kVec);
  a.slices = (a.units + kRowThreads - 1) / kRowThreads;
  a.small = a.units <= 32;
  a.groups = a.small ? (a.chunks + kRowThreads / 32 - 1) / (kRowThreads / 32) : a.chunks;
  a.fill_rows = (65536 + p.D * G::kBytes - 1) / (p.D * G::kBytes);
  const int64_t fill = p.accumulate ? 0 : (p.V + a.fill_rows - 1) / a.fill_rows;
  cudaError_t e;
  if (p.T <= kRankTokens && (p.V + 31) / 32 <= int64_t(kRankWords) * dev.sm_count) {
    a.sorted_keys = a.keys[0];
    a.sorted_pos = a.pos[0];
    k_rank_tokens<<<unsigned(dev.sm_count), kSortThreads, 0, p.stream>>>(a);
  } else {
    const size_t shared = (size_t(1) << a.digit_bits) * 35 * 4;
    if ((e = allow_shared((const void*)k_sort_tokens, dev, kStaticShared)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(k_sort_tokens, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortCtas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = p.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSortCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, k_sort_tokens, a)) != cudaSuccess) return e;
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t ctas = a.groups * a.slices + fill;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (ctas > 0 && (e = launch_after(vec ? k_embedding_rows<D, G, false> : k_embedding_rows<D, G, true>, dim3(unsigned(ctas)), kRowThreads, p.stream, a)) != cudaSuccess)
    return e;
  if (a.chunks > 1) {
    const int64_t columns = (p.D + kJoinColumns - 1) / kJoinColumns, across = (a.chunks + kJoinWarps - 1) / kJoinWarps;
    int64_t down = (int64_t(dev.sm_count) * 8 + across - 1) / across;  // a CTA's columns are as few as one round of CTAs allows
    if (down > columns) down = columns;
    if ((e = launch_after(k_embedding_join<G>, dim3(unsigned(across), unsigned(down)), kJoinWarps * 32, p.stream, a)) != cudaSuccess) return e;
    if (a.chunks > kFewChunks)
      return launch_after(k_embedding_long<G>, dim3(kLongCtas, unsigned(columns < 64 ? columns : 64)), kLongWarps * 32, p.stream, a);
  }
  return cudaSuccess;
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
