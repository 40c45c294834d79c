// kernel_logits.cu -- penalties, biases and masks on logits, fused with the softmax that follows.
//
// For token j of row r, with c the times it was generated and "seen" whether it is in the prompt or was generated:
//     l = x;  seen: l = l > 0 ? l / repetition : l repetition;  c > 0: l -= frequency c + presence;  l += biases;
//     l *= scale;  mask bit clear: l = -inf
// and y = l, softmax(l) or log softmax(l) with the row's online (m, d) state.
//
// What bounds it: x is read once and y written once.  A thread-block cluster owns a row; a CTA holds its part of it in
// registers from the read to the write.  The few tokens that occur in the row's lists are dealt with apart from the
// many that do not: each has a word in shared memory, set to zero, then
//     bits 20-30: bias_count - index of its first bias (integer maximum);  bit 31: in the prompt;  bits 0-19: c
// (integer sums: the order of the atomics does not matter), then replaced by l before scale and mask, worked out once,
// by the first thread that takes the token's bit.  A second bit map tells the pass over all elements which of them to
// take from there, so that pass looks at one bit an element.  Biases of one token add up in the order of the list.
// CTA states are merged over distributed shared memory in the order of the ranks.  Rows longer than a cluster holds are
// taken in chunks, read twice and their lists looked at twice.
#include "device_common.cuh"
#include "logits.h"

namespace rwo {
namespace {

constexpr int kThreads = 512;
constexpr int kChunk = 16384;  // elements of a CTA's part that are held (32 a thread)
constexpr int kVals = kChunk / kThreads;
constexpr uint32_t kSeen = 1u << 31;
constexpr uint32_t kCount = (1u << 20) - 1;
constexpr int kMaxCluster = 16;

struct Args {
  LogitsProblem p;
  unsigned* status;
  int chunks;   // chunks of a CTA's part
  int counted;  // tokens or biases are given
};

struct Smem {
  State warp[kThreads / 32];
  State ranks[kMaxCluster];
  int twice;                       // some token has several biases
  int pad[3];
  uint32_t listed[kChunk / 32];    // elements whose value is in `words`
  uint32_t taken[kChunk / 32];     // elements that a thread has taken on itself
  int bias_id[kMaxBias];
  float bias_value[kMaxBias];
};
constexpr int kSmemWords = (sizeof(Smem) + 127) / 128 * 128;

enum { kLogits = 0, kSoftmax = 1, kLogSoftmax = 2 };

template <class D, int OUT>
__global__ void __launch_bounds__(kThreads, 2) k_logits(Args a) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  uint32_t* words = reinterpret_cast<uint32_t*>(smem_raw + kSmemWords);
  constexpr int V = D::kVec, K = kVals / V;  // vectors a thread holds
  const LogitsProblem& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  uint32_t ranks;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int64_t r = cluster_id_x();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const unsigned char* xr = static_cast<const unsigned char*>(p.x) + r * p.x_pitch * D::kBytes;
  unsigned char* yr = static_cast<unsigned char*>(p.y) + r * p.y_pitch * D::kBytes;
  // places count from the 16-byte boundary at or below the row's start: element j is place j + off
  const int N = int(p.N), off = int((reinterpret_cast<uintptr_t>(xr) & 15u) / D::kBytes);
  const bool same = ((reinterpret_cast<uintptr_t>(yr) ^ reinterpret_cast<uintptr_t>(xr)) & 15u) == 0;
  const int vecs = (N + off + V - 1) / V, per = (vecs + int(ranks) - 1) / int(ranks);
  const int v0 = min(per * int(rank), vecs), v1 = min(v0 + per, vecs);

  const float scale = p.scale ? __ldg(p.scale + r) : 1.f;
  int n_tokens = 0, n_prompt = 0;
  if (p.tokens) {
    n_tokens = __ldg(p.token_lens + r);
    n_prompt = p.prompt_lens ? __ldg(p.prompt_lens + r) : 0;
    if (n_tokens < 0 || n_tokens > p.token_pitch || n_prompt < 0 || n_prompt > n_tokens) {
      if (tid == 0) atomicOr(a.status, kStatusBadIndex);
      n_tokens = n_tokens < 0 ? 0 : n_tokens > p.token_pitch ? int(p.token_pitch) : n_tokens;
    }
  }
  const int32_t* toks = p.tokens ? p.tokens + r * p.token_pitch : nullptr;
  const uint32_t* mask = p.mask ? p.mask + r * p.mask_pitch : nullptr;

  // The listed tokens of elements [j0, j0 + n): their values before scale and mask into `words`, their bits into `listed`.
  // j0 may be negative (places before the row); ids are not.
  auto lists = [&](int j0, int n) {
    __syncthreads();  // the last chunk's words have been read
    for (int i = tid; i < kChunk / 32; i += kThreads) sm.listed[i] = sm.taken[i] = 0u;
    if (tid == 0) sm.twice = 0;
    for (int i = tid; i < p.bias_count; i += kThreads) {
      const int id = __ldg(p.bias_ids + r * p.bias_count + i);
      sm.bias_id[i] = id < N ? id : -1;
      sm.bias_value[i] = __ldg(p.bias_values + r * p.bias_count + i);
      if (id >= N) atomicOr(a.status, kStatusBadIndex);
      else if (id >= 0 && uint32_t(id - j0) < uint32_t(n)) words[id - j0] = 0u;
    }
    auto each_token = [&](auto f) {
#pragma unroll 4
      for (int i = tid; i < n_tokens; i += kThreads) {
        const int id = __ldg(toks + i);
        if (id >= 0 && id < N && uint32_t(id - j0) < uint32_t(n)) f(id - j0, i, id);
      }
    };
#pragma unroll 4
    for (int i = tid; i < n_tokens; i += kThreads) {
      const int id = __ldg(toks + i);
      if (id >= N) atomicOr(a.status, kStatusBadIndex);
      else if (id >= 0 && uint32_t(id - j0) < uint32_t(n)) words[id - j0] = 0u;
    }
    __syncthreads();
    if (p.bias_count) {
      for (int i = tid; i < p.bias_count; i += kThreads) {
        const int id = sm.bias_id[i];
        if (id >= 0 && uint32_t(id - j0) < uint32_t(n)) atomicMax(&words[id - j0], uint32_t(p.bias_count - i) << 20);
      }
      __syncthreads();
    }
    each_token([&](int at, int i, int) {
      if (i < n_prompt) atomicOr(&words[at], kSeen);
      else atomicAdd(&words[at], 1u);
    });
    for (int i = tid; i < p.bias_count; i += kThreads) {
      const int id = sm.bias_id[i];
      if (id >= 0 && uint32_t(id - j0) < uint32_t(n) && int((words[id - j0] >> 20) & 2047u) != p.bias_count - i) sm.twice = 1;
    }
    __syncthreads();
    const float rep = p.repetition ? __ldg(p.repetition + r) : 1.f;
    const float freq = p.frequency ? __ldg(p.frequency + r) : 0.f, pres = p.presence ? __ldg(p.presence + r) : 0.f;
    auto settle = [&](int at, int id) {
      const uint32_t bit = 1u << (at & 31);
      if (sm.taken[at >> 5] & bit) return;
      if (atomicOr(&sm.taken[at >> 5], bit) & bit) return;
      const uint32_t w = words[at], c = w & kCount;
      float l = D::load1(xr, id);
      if ((w & kSeen) || c) l = l > 0.f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
      if (c) l = __fsub_rn(l, __fadd_rn(__fmul_rn(freq, float(c)), pres));
      if (const int field = int((w >> 20) & 2047u)) {
        const int first = p.bias_count - field;
        float sum = sm.bias_value[first];
        if (sm.twice)
          for (int k = first + 1; k < p.bias_count; ++k)
            if (sm.bias_id[k] == id) sum = __fadd_rn(sum, sm.bias_value[k]);
        l = __fadd_rn(l, sum);
      }
      words[at] = __float_as_uint(l);
      atomicOr(&sm.listed[at >> 5], bit);
    };
    each_token([&](int at, int, int id) { settle(at, id); });
    for (int i = tid; i < p.bias_count; i += kThreads) {
      const int id = sm.bias_id[i];
      if (id >= 0 && uint32_t(id - j0) < uint32_t(n)) settle(id - j0, id);
    }
    __syncthreads();
  };

  float val[kVals];
  // Loads vectors c0 .. of the part, up to kChunk elements, and processes them.
  auto process = [&](int c0) {
    const int c1 = min(c0 + kChunk / V, v1);
    uint4 raw[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = c0 + tid + k * kThreads, j = v * V - off;
      if (v < c1 && j >= 0 && j + V <= N) raw[k] = ld16(xr + int64_t(j) * D::kBytes);
    }
    if (a.counted) lists(c0 * V - off, (c1 - c0) * V);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = c0 + tid + k * kThreads, j = v * V - off;
      float f[V];
      if (v < c1 && j >= 0 && j + V <= N) {
        D::unpack(raw[k], f);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = v < c1 && j + i >= 0 && j + i < N ? D::load1(xr, j + i) : -INFINITY;
      }
      if (a.counted) {
        const int at = (tid + k * kThreads) * V;  // v - c0
        const uint32_t bits = sm.listed[at >> 5] >> (at & 31);
        if (bits & ((1u << V) - 1u)) {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if ((bits >> i) & 1u) f[i] = __uint_as_float(words[at + i]);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = __fmul_rn(f[i], scale);
      if (mask && v < c1) {
        const int lo = max(j, 0), w0 = lo >> 5, sh = lo & 31;
        const uint32_t a0 = __ldg(mask + w0), a1 = sh + V > 32 && w0 < ((N - 1) >> 5) ? __ldg(mask + w0 + 1) : 0u;
        const uint32_t bits = __funnelshift_r(a0, a1, uint32_t(sh)) << (lo - j);  // bit i: element j + i
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (!((bits >> i) & 1u)) f[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) val[k * V + i] = f[i];
    }
  };
  // Writes the values held, those of the vectors from c0 on; f maps a processed value to the output.
  auto write = [&](int c0, auto f) {
    const int c1 = min(c0 + kChunk / V, v1);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = c0 + tid + k * kThreads, j = v * V - off;
      if (v >= c1) continue;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = f(val[k * V + i]);
      if (same && j >= 0 && j + V <= N) {
        st_stream16(yr + int64_t(j) * D::kBytes, D::pack(o));
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (j + i >= 0 && j + i < N) D::store1(yr, j + i, o[i]);
      }
    }
  };
  auto chunk_at = [&](int c) { return min(v0 + c * (kChunk / V), v1); };

  // The row's state.  A softmax's values become e^(l - m) of this thread's own maximum m: one exponential an element.
  State s = empty_state();
  float mine = 0.f;
  const bool state = OUT != kLogits || p.lse;
  for (int c = 0; c < a.chunks; ++c) {
    process(chunk_at(c));
    if (OUT == kLogits) write(chunk_at(c), [](float v) { return v; });
    if (!state) continue;
    float m = val[0];
#pragma unroll
    for (int i = 1; i < kVals; ++i) m = fmaxf(m, val[i]);
    mine = safe_max(m);
    float2 d = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kVals; i += 2) {
      const float2 e = exp_diff2(make_float2(val[i], val[i + 1]), make_float2(-mine, -mine));
      d = __fadd2_rn(d, e);
      if (OUT == kSoftmax) {
        val[i] = e.x;
        val[i + 1] = e.y;
      }
    }
    s = merge(s, State{m, d.x + d.y});
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA of the cluster runs
  if (!state) return;
  s = group_merge_nary(s, sm.warp, kThreads / 32, warp, lane, [] { __syncthreads(); });
  if (tid < int(ranks)) st_cluster_f32x2(map_to_rank(smem_addr(&sm.ranks[rank]), uint32_t(tid)), s.m, s.d);
  cluster_sync();
  s = sm.ranks[0];
  for (uint32_t k = 1; k < ranks; ++k) s = merge(s, sm.ranks[k]);
  if (rank == 0 && tid == 0 && p.lse) p.lse[r] = lse_of(s);
  if (OUT == kLogits) return;
  const float ms = safe_max(s.m), inv = safe_inv(s.d);
  const LogNorm ln = log_norm(s);
  if (OUT == kSoftmax && a.chunks == 1) {
    const float fix = __fmul_rn(exp_diff(mine, ms), inv);
    write(v0, [&](float e) { return __fmul_rn(e, fix); });
    return;
  }
  for (int c = 0; c < a.chunks; ++c) {
    if (a.chunks > 1) process(chunk_at(c));
    if (OUT == kSoftmax) write(chunk_at(c), [&](float v) { return __fmul_rn(exp_diff(v, ms), inv); });
    else write(chunk_at(c), [&](float v) { return log_prob(v, ln); });
  }
}

template <class D>
cudaError_t launch_for(const LogitsProblem& p, const DeviceInfo& dev) {
  // The smallest cluster whose CTAs hold their parts; larger ones while SMs would stay idle and a part is above 2048
  // elements.  A part is a whole number of 16-byte vectors; rows that do not begin on one may need one more.
  const bool even = (reinterpret_cast<uintptr_t>(p.x) & 15u) == 0 && (p.M == 1 || p.x_pitch % D::kVec == 0);
  const int64_t vecs = (p.N + (even ? D::kVec - 1 : 2 * D::kVec - 2)) / D::kVec;
  int ranks = 1;
  while (ranks < kMaxCluster && (vecs + ranks - 1) / ranks * D::kVec > kChunk) ranks *= 2;
  while (ranks < kMaxCluster && p.M * ranks < dev.sm_count && p.N / ranks > 4096) ranks *= 2;
  const int64_t per = (vecs + ranks - 1) / ranks;
  Args a;
  a.p = p;
  a.status = dev.status;
  a.chunks = int((per * D::kVec + kChunk - 1) / kChunk);
  a.counted = p.tokens || p.bias_count ? 1 : 0;
  using Kern = void (*)(Args);
  const Kern kern = p.out == kLogits ? (Kern)k_logits<D, kLogits> : p.out == kSoftmax ? (Kern)k_logits<D, kSoftmax> : (Kern)k_logits<D, kLogSoftmax>;
  cudaError_t err = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemWords + kChunk * 4);
  if (err == cudaSuccess) err = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.M * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(kSmemWords + (a.counted ? kChunk * 4 : 0));
  cfg.stream = p.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ranks);
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
