// kernel_logits.cu -- penalties, biases and masks on logits, fused with the softmax that follows.
//
// For token j of row r, with c the times it was generated and "seen" whether it is in the prompt or was generated:
//     l = x;  seen: l = l > 0 ? l / repetition : l repetition;  l -= frequency c + presence [c > 0];  l += biases;
//     l *= scale;  mask bit clear: l = -inf
// and y = l, softmax(l) or log softmax(l) with the row's online (m, d) state.
//
// What bounds it: x is read once and y written once.  A thread-block cluster owns a row; a CTA holds its part of it in
// registers from the read to the write.  The counts of a CTA's part are 32-bit words in shared memory, filled by a scan
// of the row's tokens with integer atomics (sums of integers: the order does not matter):
//     bit 31: in the prompt;  bits 20-30: index + 1 of its bias;  bits 0-19: c.
// Biases of one token add up in the order of the list: the first entry of a token sums its later ones.
// CTA states are merged over distributed shared memory in the order of the ranks.  Rows longer than a cluster holds are
// taken in chunks, read twice and their counts made twice.
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
  int chunks;  // chunks of a CTA's part
  int counted; // tokens or biases are given
};

struct Smem {
  State warp[kThreads / 32];
  State ranks[kMaxCluster];
  int bias_id[kMaxBias];
  float bias_sum[kMaxBias];
};
constexpr int kSmemCounts = (sizeof(Smem) + 127) / 128 * 128;

template <class D>
__global__ void __launch_bounds__(kThreads, 2) k_logits(Args a) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  uint32_t* counts = reinterpret_cast<uint32_t*>(smem_raw + kSmemCounts);
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
  const int off = int((reinterpret_cast<uintptr_t>(xr) & 15u) / D::kBytes);
  const bool same = ((reinterpret_cast<uintptr_t>(yr) ^ reinterpret_cast<uintptr_t>(xr)) & 15u) == 0;
  const int64_t vecs = (p.N + off + V - 1) / V, per = (vecs + ranks - 1) / ranks;
  const int64_t v0 = per * rank < vecs ? per * rank : vecs, v1 = v0 + per < vecs ? v0 + per : vecs;

  const float rep = p.repetition ? __ldg(p.repetition + r) : 1.f;
  const float freq = p.frequency ? __ldg(p.frequency + r) : 0.f, pres = p.presence ? __ldg(p.presence + r) : 0.f;
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

  float val[kVals];
  // Loads vectors [c0, c0 + kChunk / V) of the part, makes their counts and the processed values.
  auto process = [&](int64_t c0) {
    const int64_t c1 = c0 + kChunk / V < v1 ? c0 + kChunk / V : v1;
    const int64_t j0 = c0 * V - off, j1 = c1 * V - off;  // elements [j0, j1) of the row (its ends may lie inside)
    uint4 raw[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t v = c0 + tid + int64_t(k) * kThreads, j = v * V - off;
      if (v < c1 && j >= 0 && j + V <= p.N) raw[k] = ld16(xr + j * D::kBytes);
    }
    if (a.counted) {
      __syncthreads();  // the last chunk's counts have been read
      for (int i = tid; i < kChunk / 4; i += kThreads) reinterpret_cast<uint4*>(counts)[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int i = tid; i < p.bias_count; i += kThreads) sm.bias_id[i] = __ldg(p.bias_ids + r * p.bias_count + i);
      __syncthreads();
      for (int i = tid; i < n_tokens; i += kThreads) {
        const int64_t id = __ldg(toks + i);
        if (id >= p.N) {
          atomicOr(a.status, kStatusBadIndex);
        } else if (id >= 0 && id >= j0 && id < j1) {
          if (i < n_prompt) atomicOr(&counts[id - j0], kSeen);
          else atomicAdd(&counts[id - j0], 1u);
        }
      }
      for (int i = tid; i < p.bias_count; i += kThreads) {
        const int id = sm.bias_id[i];
        if (id >= p.N) atomicOr(a.status, kStatusBadIndex);
        if (id < 0 || id < j0 || id >= j1 || id >= p.N) continue;
        const float* values = p.bias_values + r * p.bias_count;
        int before = 0;
        while (before < i && sm.bias_id[before] != id) ++before;
        if (before < i) continue;
        float sum = __ldg(values + i);
        for (int k = i + 1; k < p.bias_count; ++k)
          if (sm.bias_id[k] == id) sum += __ldg(values + k);
        sm.bias_sum[i] = sum;
        atomicOr(&counts[id - j0], uint32_t(i + 1) << 20);
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t v = c0 + tid + int64_t(k) * kThreads, j = v * V - off;
      const bool inside = v < c1 && j >= 0 && j + V <= p.N;
      float f[V];
      if (inside) {
        D::unpack(raw[k], f);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = v < c1 && j + i >= 0 && j + i < p.N ? D::load1(xr, j + i) : -INFINITY;
      }
      if (a.counted && v < c1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const uint32_t w = counts[(v - c0) * V + i];
          if (w) {
            const uint32_t c = w & kCount;
            float l = f[i];
            if ((w & kSeen) || c) l = l > 0.f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
            if (c) l = __fsub_rn(l, __fadd_rn(__fmul_rn(freq, float(c)), pres));
            if (w & ~(kSeen | kCount)) l = __fadd_rn(l, sm.bias_sum[((w & ~kSeen) >> 20) - 1]);
            f[i] = l;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = __fmul_rn(f[i], scale);
      if (mask && v < c1) {
        const int64_t lo = j < 0 ? 0 : j, w0 = lo >> 5;
        const int64_t last = (p.N - 1) >> 5;
        const uint32_t a0 = __ldg(mask + w0), a1 = w0 < last ? __ldg(mask + w0 + 1) : 0u;
        const uint32_t bits = __funnelshift_r(a0, a1, uint32_t(lo & 31));  // bit i: element lo + i
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (!((bits >> ((j + i - lo) & 31)) & 1u)) f[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) val[k * V + i] = f[i];
    }
  };

  // Writes the values held, those of the vectors from c0 on; f maps a processed value to the output.
  auto write = [&](int64_t c0, auto f) {
    const int64_t c1 = c0 + kChunk / V < v1 ? c0 + kChunk / V : v1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t v = c0 + tid + int64_t(k) * kThreads, j = v * V - off;
      if (v >= c1) continue;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = f(val[k * V + i]);
      if (same && j >= 0 && j + V <= p.N) {
        st_stream16(yr + j * D::kBytes, D::pack(o));
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (j + i >= 0 && j + i < p.N) D::store1(yr, j + i, o[i]);
      }
    }
  };
  auto chunk_at = [&](int64_t c) {
    const int64_t c0 = v0 + c * (kChunk / V);
    return c0 < v1 ? c0 : v1;
  };

  State s = empty_state();
  const bool state = p.lse || p.out != 0;
  for (int64_t c = 0; c < a.chunks; ++c) {
    process(chunk_at(c));
    if (p.out == 0) write(chunk_at(c), [](float v) { return v; });
    if (!state) continue;
    float m = val[0];
#pragma unroll
    for (int i = 1; i < kVals; ++i) m = fmaxf(m, val[i]);
    const float ms = safe_max(m);
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) d += exp_diff(val[i], ms);
    s = merge(s, State{m, d});
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA of the cluster runs
  if (!state) return;
  s = group_merge_nary(s, sm.warp, kThreads / 32, warp, lane, [] { __syncthreads(); });
  if (tid < int(ranks)) st_cluster_f32x2(map_to_rank(smem_addr(&sm.ranks[rank]), uint32_t(tid)), s.m, s.d);
  cluster_sync();
  s = sm.ranks[0];
  for (uint32_t k = 1; k < ranks; ++k) s = merge(s, sm.ranks[k]);
  if (rank == 0 && tid == 0 && p.lse) p.lse[r] = lse_of(s);
  if (p.out == 0) return;
  const float ms = safe_max(s.m), inv = safe_inv(s.d);
  const LogNorm ln = log_norm(s);
  for (int64_t c = 0; c < a.chunks; ++c) {
    if (a.chunks > 1) process(chunk_at(c));
    if (p.out == 1) write(chunk_at(c), [&](float v) { return __fmul_rn(exp_diff(v, ms), inv); });
    else write(chunk_at(c), [&](float v) { return log_prob(v, ln); });
  }
}

template <class D>
cudaError_t launch_for(const LogitsProblem& p, const DeviceInfo& dev) {
  // The smallest cluster whose CTAs hold their parts; larger ones while SMs would stay idle and a part is above 2048
  // elements.  A part is a whole number of 16-byte vectors, and a row may begin inside one.
  const int64_t vecs = (p.N + 2 * D::kVec - 2) / D::kVec;
  int ranks = 1;
  while (ranks < kMaxCluster && (vecs + ranks - 1) / ranks * D::kVec > kChunk) ranks *= 2;
  while (ranks < kMaxCluster && p.M * ranks < dev.sm_count && p.N / ranks > 4096) ranks *= 2;
  const int64_t per = (vecs + ranks - 1) / ranks;
  Args a;
  a.p = p;
  a.status = dev.status;
  a.chunks = int((per * D::kVec + kChunk - 1) / kChunk);
  a.counted = p.tokens || p.bias_count ? 1 : 0;
  const int smem = kSmemCounts + (a.counted ? kChunk * 4 : 0);
  auto kern = k_logits<D>;
  cudaError_t err = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemCounts + kChunk * 4);
  if (err == cudaSuccess) err = cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.M * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(smem);
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
