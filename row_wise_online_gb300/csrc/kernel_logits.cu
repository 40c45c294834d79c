// kernel_logits.cu -- penalties, biases and masks on logits, fused with the softmax that follows.
//
// For token j of row r, with c the times it was generated and "seen" whether it is in the prompt or was generated:
//     l = x;  seen: l = l > 0 ? l / repetition : l repetition;
//     c > 0: l -= frequency c + presence;  l += biases;  l *= scale;  mask bit clear: l = -inf
// and y = l, softmax(l) or log softmax(l) with the row's online (m, d) state.
//
// What bounds it: x is read once from HBM and y written once.  A thread-block cluster owns a row (one CTA where there are
// rows enough), each CTA a part of it; the part is streamed twice, once for the state and once for the output, the
// second time from L2, where the rows in work (a few hundred of up to half a MB) stay.  Holding the part on chip between
// the two (registers, 16384 elements a CTA, eight CTAs a row) cost more in barriers between CTAs than the second
// reading: 256 rows of 131072 bf16 logits took 156 us that way.
//
// The few tokens that occur in the row's lists are dealt with before the streaming.  A bit map over the part's elements
// says which they are, a running count over its words numbers them, and each has a word in shared memory that becomes
//     bits 20-30: bias_count - index of its first bias (integer maximum);  bit 31: in the prompt;  bits 0-19: c
// (integer sums: the order of the atomics does not matter) and then the masked l before scale, worked out once, one token
// a thread.  Streaming treats listed tokens as masked; their values join the state from the list, and their outputs are
// written over the streamed ones at the end.  So a streamed element costs a mask bit and nothing else: 256 rows of 131072
// bf16 logits with 8192 tokens of history, 64 biases and a mask take 57 us (11 more when each vector is looked up in the
// map, in both passes).  The lists are 17 of these and the mask 10; the bytes alone would be 22.  Latency bounds it:
// 256 rows are one wave, in which every CTA works on its lists at the same time and streams at the same time, and a batch of
// vectors is loaded when the last one has been worked.  (Fetching the part into L2 while the lists are looked through: 2
// more; the streaming then waits for the same bytes.)
// The scale is folded into the exponent.  Biases of one token add up in the order of the list.
// Where the listed tokens of a part may be more than shared memory holds, the part is taken in chunks.
#include <atomic>

#include "device_common.cuh"
#include "logits.h"

namespace rwo {
namespace {

constexpr int kMostThreads = 512;
constexpr uint32_t kSeen = 1u << 31;
constexpr uint32_t kCount = (1u << 20) - 1;
constexpr uint32_t kField = 2047u << 20;
constexpr int kMaxCluster = 16;
constexpr int kMaxListed = 16384;     // words of a chunk's listed tokens
constexpr int kMaxChunk = 1 << 18;    // elements of a chunk: bit map and running count are 6 bytes for 32 elements

struct Args {
  LogitsProblem p;
  unsigned* status;
  int log2_ranks;
  int chunk;      // vectors of a chunk
  int chunks;     // chunks of a part
  int listed;     // words of listed tokens, 0 where no tokens and biases are given
  int map_words;  // words of the bit map
  int mask_words;  // words of the mask for a chunk
};

struct Smem {
  State warp[kMostThreads / 32];
  State ranks[kMaxCluster];
  int sums[kMostThreads / 32];
  int twice;  // some token has several biases
  int pad[3];
};

// Dynamic shared memory behind Smem: words and ids of the listed tokens, bit map, mask, ids and values of the biases,
// running count.
__host__ __device__ inline size_t smem_bytes(int listed, int map_words, int mask_words, int bias_count) {
  return sizeof(Smem) + size_t(listed) * 8 + size_t(map_words) * 6 + size_t(mask_words) * 4 + size_t(bias_count) * 8;
}

// A vector's elements where bit i of `bits` is set, -inf elsewhere: on the packed words, before they are widened.
template <class D>
__device__ __forceinline__ uint4 only(uint4 v, uint32_t bits) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (D::kBytes == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(bits & (1u << i))) w[i] = D::kNegInfWord;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      // bit k of four becomes the top bit of byte k, and a byte permutation spreads top bits over two bytes each
      const uint32_t tops = ((bits >> (2 * i)) & 15u) * 0x10204080u;
      uint32_t k0, k1;
      asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(k0) : "r"(tops));
      asm("prmt.b32 %0, %1, 0, 0xbbaa;" : "=r"(k1) : "r"(tops));
      w[i] = (w[i] & k0) | (D::kNegInfWord & ~k0);
      w[i + 1] = (w[i + 1] & k1) | (D::kNegInfWord & ~k1);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

enum { kLogits = 0, kSoftmax = 1, kLogSoftmax = 2 };

template <class D, int OUT, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) k_logits(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  constexpr int V = D::kVec;
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const LogitsProblem& p = a.p;
  uint32_t* words = reinterpret_cast<uint32_t*>(smem_raw + sizeof(Smem));
  int* ids = reinterpret_cast<int*>(words + a.listed);
  uint32_t* map = words + 2 * a.listed;
  uint32_t* allowed = map + a.map_words;
  int* bias_id = reinterpret_cast<int*>(allowed + a.mask_words);
  float* bias_value = reinterpret_cast<float*>(bias_id + p.bias_count);
  uint16_t* below = reinterpret_cast<uint16_t*>(bias_value + p.bias_count);  // listed tokens in the map's words before
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = int(p.N);
  const int rank = int(cluster_ctarank()), ranks = 1 << a.log2_ranks;
  const int64_t r = cluster_id_x();
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  const unsigned char* x = static_cast<const unsigned char*>(p.x) + r * p.x_pitch * D::kBytes;
  unsigned char* y = static_cast<unsigned char*>(p.y) + r * p.y_pitch * D::kBytes;
  const uint32_t* mask = p.mask ? p.mask + r * p.mask_pitch : nullptr;
  const int32_t* toks = p.tokens ? p.tokens + r * p.token_pitch : nullptr;
  // The row as whole 16-byte vectors, with the few elements before its first boundary (rank 0) and behind its last (the
  // last rank), which threads 0 .. and 32 .. of those CTAs take one each.
  const int off = int((reinterpret_cast<uintptr_t>(x) & 15u) / D::kBytes), front = off ? min(V - off, N) : 0;
  const int vecs = (N - front) / V, back = N - front - vecs * V, per = (vecs + ranks - 1) >> a.log2_ranks;
  const int v0 = min(per * rank, vecs), v1 = min(v0 + per, vecs);
  const bool whole = ((reinterpret_cast<uintptr_t>(y) ^ reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
  const float scale = p.scale ? __ldg(p.scale + r) : 1.f, slope = __fmul_rn(scale, kLog2e);
  const bool masked = a.mask_words > 0;

  int n_tokens = 0, n_prompt = 0;
  if (toks) {
    n_tokens = __ldg(p.token_lens + r);
    n_prompt = p.prompt_lens ? __ldg(p.prompt_lens + r) : 0;
  }
  int listed = 0, base = 0, e0 = 0, e1 = 0;  // tokens on the chunk's list; element of place 0; the chunk's elements
  // f(i, id) for this thread's tokens i, id = -1 behind the last.  Some are loaded at once: sixteen and no branches where rows
  // are many (256 rows: 57.7 us against 58.3 with them), four where they are few and a launch fetches its instructions anew
  // (one row: 8.6 us against 9.0 with sixteen).
  auto each_token = [&](auto f) {
    constexpr bool kMany = kThreads == kMostThreads;
    constexpr int kAhead = kMany ? 16 : 4;
    for (int i0 = tid; i0 < n_tokens; i0 += kAhead * kThreads) {
      int ahead[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) ahead[k] = i0 + k * kThreads < n_tokens ? __ldg(toks + i0 + k * kThreads) : -1;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (!kMany && i0 + k * kThreads >= n_tokens) break;
        f(i0 + k * kThreads, ahead[k]);
      }
    }
  };
  auto number = [&](int at) { return int(below[at >> 5]) + __popc(map[at >> 5] & ((1u << (at & 31)) - 1u)); };
  // The listed tokens among vectors [c0, c0 + n) and this part's single elements.  Place of element id in the map: 32 for
  // the first vector's first, the elements before it below that.
  auto lists = [&](int c0, int n) {
    if (n_tokens < 0 || n_tokens > p.token_pitch || n_prompt < 0 || n_prompt > n_tokens) {
      if (tid == 0) atomicOr(a.status, kStatusBadIndex);
      n_tokens = n_tokens < 0 ? 0 : n_tokens > p.token_pitch ? int(p.token_pitch) : n_tokens;
    }
    base = front + c0 * V - 32;
    e0 = rank == 0 && c0 == v0 ? 0 : base + 32;
    e1 = rank == ranks - 1 && c0 + n == v1 ? N : base + 32 + n * V;
    const int used = (n * V + 32 + V + 31) / 32;  // of the map's words
    __syncthreads();  // the last chunk's have been read
    for (int i = tid; i < used; i += kThreads) map[i] = 0u;
    for (int i = tid; i < a.listed; i += kThreads) words[i] = 0u;
    if (tid == 0) sm.twice = 0;
    __syncthreads();
    auto set = [&](int at) {
      const uint32_t bit = 1u << (at & 31);
      if (!(map[at >> 5] & bit)) atomicOr(&map[at >> 5], bit);
    };
    for (int i = tid; i < p.bias_count; i += kThreads) {
      const int id = __ldg(p.bias_ids + r * p.bias_count + i);
      const bool here = id >= e0 && id < e1 && id < N;
      bias_id[i] = here ? id : -1;
      bias_value[i] = __ldg(p.bias_values + r * p.bias_count + i);
      if (here) set(id - base);
      if (id >= N) atomicOr(a.status, kStatusBadIndex);
    }
    each_token([&](int, int id) {
      if (id >= e0 && id < e1) set(id - base);
      else if (id >= N) atomicOr(a.status, kStatusBadIndex);
    });
    __syncthreads();
    // the running count: every thread a run of words
    const int each = (used + kThreads - 1) / kThreads, w0 = min(tid * each, used), w1 = min(w0 + each, used);
    int sum = 0;
    for (int w = w0; w < w1; ++w) sum += __popc(map[w]);
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int s = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += s;
    }
    if (lane == 31) sm.sums[warp] = upto;
    __syncthreads();
    int before = upto - sum;
    listed = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sm.sums[w];
      listed += sm.sums[w];
    }
    for (int w = w0; w < w1; ++w) {
      below[w] = uint16_t(before);
      before += __popc(map[w]);
    }
    __syncthreads();
  };
  // Their counts, and from these their values.
  auto values = [&] {
    if (p.bias_count) {
      for (int i = tid; i < p.bias_count; i += kThreads)
        if (bias_id[i] >= 0) {
          const int k = number(bias_id[i] - base);
          ids[k] = bias_id[i];
          atomicMax(&words[k], uint32_t(p.bias_count - i) << 20);
        }
      __syncthreads();
      for (int i = tid; i < p.bias_count; i += kThreads)
        if (bias_id[i] >= 0 && int((words[number(bias_id[i] - base)] & kField) >> 20) != p.bias_count - i) sm.twice = 1;
      // (counts, added from here on, leave that field alone)
    }
    each_token([&](int i, int id) {
      if (id < e0 || id >= e1) return;
      const int k = number(id - base);
      ids[k] = id;
      if (i < n_prompt) atomicOr(&words[k], kSeen);
      else atomicAdd(&words[k], 1u);
    });
    const float rep = p.repetition ? __ldg(p.repetition + r) : 1.f;
    const float freq = p.frequency ? __ldg(p.frequency + r) : 0.f, pres = p.presence ? __ldg(p.presence + r) : 0.f;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < listed; i += kThreads) {
      const int id = ids[i];
      const uint32_t w = words[i], c = w & kCount;
      float l = D::load1(x, id);
      if ((w & kSeen) || c) l = l > 0.f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
      if (c) l = __fsub_rn(l, __fadd_rn(__fmul_rn(freq, float(c)), pres));
      if (const int field = int((w & kField) >> 20)) {
        const int first = p.bias_count - field;
        float add = bias_value[first];
        if (sm.twice)
          for (int k = first + 1; k < p.bias_count; ++k)
            if (bias_id[k] == id) add = __fadd_rn(add, bias_value[k]);
        l = __fadd_rn(l, add);
      }
      words[i] = __float_as_uint(mask && !((__ldg(mask + (id >> 5)) >> (id & 31)) & 1u) ? -INFINITY : l);
    }
    __syncthreads();
  };
  // The elements of vectors [c0, c0 + n) that are streamed, bit by bit from the word of the first one's index on: allowed
  // by the mask, and not listed.
  auto masks = [&](int c0, int n) {
    const int e0 = front + c0 * V, w0 = e0 >> 5, w1 = n ? (e0 + n * V - 1) >> 5 : w0 - 1, sh = e0 & 31;
    if (!a.listed) __syncthreads();  // the last chunk's have been read (lists() waits too)
    for (int i = tid; i <= w1 - w0; i += kThreads) {
      uint32_t bits = mask ? __ldg(mask + w0 + i) : 0xffffffffu;
      // bit k of word i is element 32 (w0 + i) + k, at place 32 i + k + 32 - sh of the map
      if (a.listed) bits &= ~(sh ? __funnelshift_r(map[i], i < (n * V + 32 + V - 1) / 32 ? map[i + 1] : 0u, 32 - sh) : map[i + 1]);
      allowed[i] = bits;
    }
    __syncthreads();
  };
  // The single element id (in the map at place `at`), masked.
  auto single = [&](int id, int at) {
    if (a.listed && ((map[at >> 5] >> (at & 31)) & 1u)) return -INFINITY;
    return mask && !((__ldg(mask + (id >> 5)) >> (id & 31)) & 1u) ? -INFINITY : D::load1(x, id);
  };
  // Streams chunk [c0, c0 + n), masked and before scale: f(values, vector) for each vector, g(value, element) for this
  // thread's single element.
  auto stream = [&](int c0, int n, auto f, auto g) {
    constexpr int kAhead = 4;
    const unsigned char* from = x + (int64_t(c0) * V + front) * D::kBytes;
    for (int i0 = tid; i0 < n; i0 += kAhead * kThreads) {
      uint4 raw[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k * kThreads < n) raw[k] = ld16(from + int64_t(i0 + k * kThreads) * 16);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * kThreads;
        if (i >= n) break;
        if (masked) {
          const int e = ((front + c0 * V) & 31) + i * V, sh = e & 31;
          uint32_t bits = allowed[e >> 5] >> sh;
          if (front && sh + V > 32) bits |= allowed[(e >> 5) + 1] << (32 - sh);
          raw[k] = only<D>(raw[k], bits);
        }
        float l[V];
        D::unpack(raw[k], l);
        f(l, c0 + i);
      }
    }
    if (rank == 0 && c0 == v0 && tid < front) g(single(tid, 32 - front + tid), tid);
    if (rank == ranks - 1 && c0 + n == v1 && tid >= 32 && tid - 32 < back) g(single(N - back + tid - 32, 32 + n * V + tid - 32), N - back + tid - 32);
  };
  auto put = [&](const float (&o)[V], int v) {
    unsigned char* to = y + (int64_t(v) * V + front) * D::kBytes;
    if (whole) {
      st_stream16(to, D::pack(o));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) D::store1(to, i, o[i]);
    }
  };

  // Outputs of the listed tokens, over what was streamed there.
  auto put_listed = [&](auto g) {
    if (!a.listed) return;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < listed; i += kThreads) D::store1(y, ids[i], g(__uint_as_float(words[i])));
  };

  State s = empty_state();  // of l before scale
  const bool state = OUT != kLogits || p.lse;
  for (int c = 0; c < a.chunks; ++c) {
    const int c0 = min(v0 + c * a.chunk, v1), n = min(a.chunk, v1 - c0);
    if (c > 0 && n == 0) break;
    if (a.listed) {
      lists(c0, n);
      values();
    }
    if (masked) masks(c0, n);
    auto one = [&](float l) { s = merge(s, State{l, l == -INFINITY ? 0.f : 1.f}, slope); };
    stream(
        c0, n,
        [&](float (&l)[V], int v) {
          if (state) {
            float m = l[0];
#pragma unroll
            for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
            m = fmaxf(m, s.m);
            const float ms = safe_max(m);
            float2 d = make_float2(__fmul_rn(s.d, exp_diff(s.m, ms, slope)), 0.f);
#pragma unroll
            for (int i = 0; i < V; i += 2) d = __fadd2_rn(d, exp_diff2(make_float2(l[i], l[i + 1]), make_float2(-ms, -ms), slope));
            s = State{m, d.x + d.y};
          }
          if (OUT == kLogits) {
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = __fmul_rn(l[i], scale);
            put(l, v);
          }
        },
        [&](float l, int id) {
          if (OUT == kLogits) D::store1(y, id, __fmul_rn(l, scale));
          one(l);
        });
    if (a.listed && state)
      for (int i = tid; i < listed; i += kThreads) one(__uint_as_float(words[i]));
    if (OUT == kLogits) put_listed([&](float l) { return __fmul_rn(l, scale); });
  }
  if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster runs
  if (!state) return;
  s = group_merge_nary(s, sm.warp, kThreads / 32, warp, lane, [] { __syncthreads(); }, slope);
  if (ranks > 1) {
    if (tid < ranks) st_cluster_f32x2(map_to_rank(smem_addr(&sm.ranks[rank]), uint32_t(tid)), s.m, s.d);
    cluster_sync();
    s = sm.ranks[0];
    for (int k = 1; k < ranks; ++k) s = merge(s, sm.ranks[k], slope);
  }
  if (rank == 0 && tid == 0 && p.lse) p.lse[r] = lse_of(scaled_state(s, scale));
  if (OUT == kLogits) return;
  const float ms = safe_max(s.m), inv = safe_inv(s.d);
  const LogNorm ln = log_norm(s);
  auto output = [&](float l) { return OUT == kSoftmax ? __fmul_rn(exp_diff(l, ms, slope), inv) : log_prob(l, ln, scale); };
  for (int c = 0; c < a.chunks; ++c) {
    const int c0 = min(v0 + c * a.chunk, v1), n = min(a.chunk, v1 - c0);
    if (c > 0 && n == 0) break;
    if (a.listed && a.chunks > 1) {
      lists(c0, n);
      values();
    }
    if (masked && a.chunks > 1) masks(c0, n);
    stream(
        c0, n,
        [&](float (&l)[V], int v) {
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            if (OUT == kSoftmax) {
              const float2 e = __fmul2_rn(exp_diff2(make_float2(l[i], l[i + 1]), make_float2(-ms, -ms), slope), make_float2(inv, inv));
              l[i] = e.x;
              l[i + 1] = e.y;
            } else {
              l[i] = output(l[i]);
              l[i + 1] = output(l[i + 1]);
            }
          }
          put(l, v);
        },
        [&](float l, int id) { D::store1(y, id, output(l)); });
    put_listed(output);
  }
}

template <class D>
cudaError_t launch_for(const LogitsProblem& p, const DeviceInfo& dev) {
  // One CTA a row where that gives every SM one; else more while a CTA's part is above 2048 elements.  (256 rows of 131072
  // bf16 logits: one CTA a row 57 us, two 70: a row's lists are looked through by each of its CTAs.)
  const int64_t vecs = (p.N + D::kVec - 1) / D::kVec;
  int log2 = 0;
  while ((1 << log2) < kMaxCluster && (p.M << log2) < dev.sm_count && (p.N >> log2) > 4096) ++log2;
  Args a;
  a.p = p;
  a.status = dev.status;
  const bool counted = p.tokens || p.bias_count;
  // a part is one chunk, unless its listed tokens or its map may not fit
  const int64_t entries = (p.tokens ? p.token_pitch : 0) + p.bias_count;
  int64_t most = !counted || entries <= kMaxListed ? kMaxChunk : kMaxListed - 16;
  while ((1 << log2) < kMaxCluster && (counted || p.mask) && (((vecs - 1) >> log2) + 1) * D::kVec > most) ++log2;
  const int64_t per = ((vecs - 1) >> log2) + 1, room = counted || p.mask ? most / D::kVec : per;
  a.log2_ranks = log2;
  a.chunk = int(per < room ? per : room);
  a.chunks = int((per + a.chunk - 1) / a.chunk);
  const int64_t elements = int64_t(a.chunk) * D::kVec + 16;
  a.listed = counted ? int((entries < elements ? entries : elements) + 3) / 4 * 4 : 0;
  a.map_words = counted ? (a.chunk * D::kVec + 32 + D::kVec + 31) / 32 : 0;
  a.mask_words = p.mask || counted ? a.chunk * D::kVec / 32 + 3 : 0;
  using Kern = void (*)(Args);
  // Clusters of four and more take CTAs of 256 threads, of which more clusters are resident at once (37 rows of 131072 bf16
  // logits over clusters of 8: 14 us against 22 with 512 threads); fewer, larger parts are better served by 512 (100 rows over
  // clusters of 2: 25 against 26; 256 rows, one CTA each: 44 against 58, with 1000 tokens of history).
  const bool few = log2 >= 2;
  const Kern kern = few ? (p.out == kLogits    ? (Kern)k_logits<D, kLogits, 256>
                           : p.out == kSoftmax ? (Kern)k_logits<D, kSoftmax, 256>
                                               : (Kern)k_logits<D, kLogSoftmax, 256>)
                        : (p.out == kLogits    ? (Kern)k_logits<D, kLogits, 512>
                           : p.out == kSoftmax ? (Kern)k_logits<D, kSoftmax, 512>
                                               : (Kern)k_logits<D, kLogSoftmax, 512>);
  // the kernel's limits are set once per device
  constexpr int kDevices = 64;
  static std::atomic<bool> ready[kDevices][6];
  std::atomic<bool>& done = ready[dev.device % kDevices][p.out * 2 + (few ? 1 : 0)];
  if (!done.load(std::memory_order_acquire)) {
    cudaError_t err = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           int(smem_bytes(kMaxListed, kMaxChunk / 32 + 4, kMaxChunk / 32 + 3, kMaxBias)));
    if (err == cudaSuccess) err = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err != cudaSuccess) return err;
    done.store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.M << log2));
  cfg.blockDim = dim3(few ? 256 : 512);
  cfg.dynamicSmemBytes = smem_bytes(a.listed, a.map_words, a.mask_words, p.bias_count);
  cfg.stream = p.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1u << log2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_logits(const LogitsProblem& p, const DeviceInfo& dev) {
  return p.dtype == 0 ? launch_for<F32>(p, dev) : p.dtype == 1 ? launch_for<BF16>(p, dev) : launch_for<F16>(p, dev);
}

}  // namespace rwo
