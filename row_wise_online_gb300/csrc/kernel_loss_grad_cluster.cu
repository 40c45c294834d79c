// kernel_loss_grad_cluster.cu -- the cross-entropy loss and its gradient (loss_grad.cuh) of long rows, each read once.
//
// What bounds it is the memory's rate, one read and one write of every element: 8192 rows of 131072 bf16 entries take 664 us, 6.46
// TB/s; 1023 rows of 50021 fp32 entries on no boundary, with smoothing, 79 us, 5.2 TB/s.
//
// A thread-block cluster of 1 .. 16 CTAs holds a row: every CTA has a run of its 16-byte vectors, copied to shared memory by
// cp.async.bulk, and takes them into registers as they are (a slot is refilled with the next row's run as soon as it has been
// read, so a row is on its way while another is worked on).  The CTAs' states are merged over distributed shared memory;
// then each thread forms the gradient from its registers.
//
// Rows start anywhere: the vectors are those of the gradient's 16-byte grid, so that whole vectors are stored; the copy takes
// whole 16-byte lines of x, the few elements around them are copied one by one, and where x lies otherwise than the gradient
// (SHIFT) a vector is put together from two of shared memory.
#include <mutex>

#include "loss_grad.cuh"

namespace rwo {
namespace {

constexpr int kMaxSlots = 4;
constexpr int kMaxCluster = 16;

struct Args {
  LossArgs p;
  int cluster;
  int lanes;       // the power of two >= cluster
  int run;         // vectors of a CTA
  int slots;
  int slot_bytes;
  bool edges;      // rows do not all begin and end on 16-byte boundaries
  uint64_t wait_ns;
};

// A CTA's part of a row: vectors [j0, j1) of the gradient's grid, elements [e0, e1).
struct Part {
  const unsigned char* x;    // the row
  uintptr_t base;            // the 16-byte line that shared memory's part begins with
  int lead;                  // elements of the grid before the row
  int delta;                 // where in its line of x a vector begins
  int j0, j1, e0, e1;
  int w0, w1;                // vectors [w0, w1) of the grid are all the row's
};

template <class D>
__device__ __forceinline__ Part part_of(const Args& a, int64_t row, int rank) {
  constexpr int E = D::kVec, S = D::kBytes;
  Part p;
  p.x = a.p.x + row * a.p.x_pitch;
  p.lead = a.edges ? int((reinterpret_cast<uintptr_t>(a.p.g) + row * a.p.g_pitch) & 15) / S : 0;
  const int n = int(a.p.N), vectors = (n + p.lead + E - 1) / E;
  p.w0 = p.lead ? 1 : 0;
  p.w1 = (n + p.lead) / E;
  p.j0 = min(rank * a.run, vectors);
  p.j1 = min(p.j0 + a.run, vectors);
  p.e0 = max(0, p.j0 * E - p.lead);
  p.e1 = max(p.e0, min(n, p.j1 * E - p.lead));
  const uintptr_t first = reinterpret_cast<uintptr_t>(p.x) + (int64_t(p.j0) * E - p.lead) * S;
  p.base = first & ~uintptr_t(15);
  p.delta = int(first & 15);
  return p;
}

// Copies a part to its slot: one thread the 16-byte lines inside it ...
template <class D>
__device__ __forceinline__ void copy_lines(const Part& p, uint32_t slot, uint32_t bar, uint64_t policy) {
  constexpr int S = D::kBytes;
  const uintptr_t x = reinterpret_cast<uintptr_t>(p.x);
  const uintptr_t lo = (x + int64_t(p.e0) * S + 15) & ~uintptr_t(15), hi = (x + int64_t(p.e1) * S) & ~uintptr_t(15);
  const uint32_t bytes = hi > lo ? uint32_t(hi - lo) : 0;
  mbar_arrive_expect_tx(bar, bytes);
  if (bytes) bulk_g2s(slot + uint32_t(lo - p.base), reinterpret_cast<const void*>(lo), bytes, bar, policy);
}

// ... and 16 lanes what lies before and behind them.
template <class D>
__device__ __forceinline__ void copy_edges(const Part& p, uint32_t slot, int lane) {
  constexpr int S = D::kBytes, E = D::kVec;
  const uintptr_t x = reinterpret_cast<uintptr_t>(p.x);
  const uintptr_t lo = (x + int64_t(p.e0) * S + 15) & ~uintptr_t(15), hi = (x + int64_t(p.e1) * S) & ~uintptr_t(15);
  int e, end;
  if (lane < E) {
    e = p.e0 + lane;
    end = min(p.e1, int((lo - x) / S));
  } else {
    e = int(((hi > lo ? hi : lo) - x) / S) + lane - E;
    end = p.e1;
  }
  if (lane < 2 * E && e < end) {
    const uint32_t to = slot + uint32_t(x + int64_t(e) * S - p.base);
    if constexpr (S == 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(reinterpret_cast<const volatile uint32_t*>(p.x)[e]) : "memory");
    else asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(reinterpret_cast<const volatile uint16_t*>(p.x)[e]) : "memory");
  }
}

// 16 bytes of shared memory from byte delta (a multiple of 2, below 16) of an aligned address on.
__device__ __forceinline__ uint4 lds16_shifted(uint32_t at, int delta) { return shifted(lds16(at), lds16(at + 16), delta); }

// s and n of elements [from, to) of a vector.
template <class D>
__device__ __forceinline__ void add_part(Fold& f, const uint4& q, int from, int to) {
  float v[D::kVec];
  D::unpack(q, v);
#pragma unroll
  for (int e = 0; e < D::kVec; ++e)
    if (e >= from && e < to) f.s += safe_max(f.m) - v[e];
  f.n += float(to - from);
}

template <class D, int T, int K, bool SMOOTH, bool SHIFT>
__global__ void __launch_bounds__(T, 8192 / (T * K)) k_loss_grad_cluster(Args a) {
  constexpr int E = D::kVec, W = T / 32;
  extern __shared__ __align__(128) unsigned char slots[];
  __shared__ uint64_t full[kMaxSlots];
  __shared__ Fold warps[2][W];
  __shared__ float4 states[2][kMaxCluster];  // of the cluster's CTAs: m, d, s, x_label
  __shared__ uint64_t arrived[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = int(cluster_ctarank());
  const int64_t first = blockIdx.x / a.cluster, step = gridDim.x / a.cluster;
  const uint64_t policy = policy_evict_first();
  bool timed_out = false;

  if (tid == 0) {
    for (int s = 0; s < a.slots; ++s) mbar_init(smem_addr(&full[s]), 1);
    for (int i = 0; i < 2; ++i) mbar_init(smem_addr(&arrived[i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  for (int s = 0; s < a.slots; ++s) {
    const int64_t row = first + s * step;
    if (row >= a.p.M) break;
    if (warp == 0) {
      const Part p = part_of<D>(a, row, rank);
      const uint32_t slot = smem_addr(slots) + s * a.slot_bytes;
      if (a.edges) copy_edges<D>(p, slot, lane);
      if (lane == 0) copy_lines<D>(p, slot, smem_addr(&full[s]), policy);
    }
  }
  if (a.cluster > 1) cluster_sync();  // every CTA is there before another writes into it
  else __syncthreads();

  int s = 0, it = 0;
  uint32_t parity = 0, exchange = 0;
  for (int64_t row = first; row < a.p.M; row += step, it ^= 1) {
    const Part p = part_of<D>(a, row, rank);
    const uint32_t slot = smem_addr(slots) + s * a.slot_bytes;
    const int64_t label = a.p.labels[row];
    if (!mbar_wait(smem_addr(&full[s]), parity, a.wait_ns)) timed_out = true;
    float x_label = 0.f;
    if (tid == 0 && label >= p.e0 && label < p.e1)
      x_label = D::lds1(slot + uint32_t(reinterpret_cast<uintptr_t>(p.x) + label * D::kBytes - p.base), 0);
    uint4 q[K];
    uint32_t whole = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = tid + k * T, j = p.j0 + i;
      q[k] = make_uint4(D::kNegInfWord, D::kNegInfWord, D::kNegInfWord, D::kNegInfWord);
      if (j < p.j1) {
        q[k] = SHIFT ? lds16_shifted(slot + i * 16, p.delta) : lds16(slot + i * 16);
        if (j >= p.w0 && j < p.w1) whole |= 1u << k;
        else q[k] = keep<D>(q[k], max(0, p.lead - j * E), min(E, int(a.p.N) + p.lead - j * E), D::kNegInfWord);
      }
    }
    const auto refill = [&] {  // every thread has read the slot
      const int64_t next = row + a.slots * step;
      if (warp == 0 && next < a.p.M) {
        const Part n = part_of<D>(a, next, rank);
        if (a.edges) copy_edges<D>(n, slot, lane);
        if (lane == 0) {
          fence_proxy_async_smem();
          copy_lines<D>(n, slot, smem_addr(&full[s]), policy);
        }
      }
    };
    if (a.slots == 1) {
      __syncthreads();
      refill();
    }
    Fold f = fold_vectors<D, K, SMOOTH>(q, whole);
    if (SMOOTH && a.edges) {  // the row's first and last vector may be its in part
      const int mine = p.j0 + tid;
      if (p.w0 && mine == 0 && p.w1 > 0) add_part<D>(f, q[0], p.lead, E);
      if (p.w1 < p.j1 && p.w1 >= mine && (p.w1 - mine) % T == 0) {
        uint4 last = q[0];
#pragma unroll
        for (int k = 1; k < K; ++k)
          if (mine + k * T == p.w1) last = q[k];
        add_part<D>(f, last, p.w1 == 0 ? p.lead : 0, int(a.p.N) + p.lead - p.w1 * E);
      }
    }
    f = fold_lanes<SMOOTH>(f, 32);
    if (lane == 0) warps[it][warp] = f;
    __syncthreads();
    if (a.slots > 1) refill();
    f = fold_lanes<SMOOTH>(warps[it][lane & (W - 1)], W);
    if (a.cluster > 1) {
      // Each CTA's state to all of them, counted in on their barriers.  (A cluster barrier in its place has to
      // release this CTA's stores, those of the row before among them, and waited for them: 8192 x 131072 bf16 took
      // 968 us instead of 873.)  A CTA writes to states[it] again when all have sent the row in between, and so have read this one.
      const uint32_t bar = smem_addr(&arrived[it]);
      if (warp == 0) {
        x_label = __shfl_sync(~0u, x_label, 0);
        if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(a.cluster) * 16);
        if (lane < a.cluster)
          asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                           map_to_rank(smem_addr(&states[it][rank]), lane)),
                       "f"(f.m), "f"(f.d), "f"(f.s), "f"(x_label), "r"(map_to_rank(bar, lane))
                       : "memory");
      }
      if (!mbar_wait_cluster(bar, exchange, a.wait_ns)) timed_out = true;
      if (it) exchange ^= 1;
      const int other = lane & (a.lanes - 1);
      f = empty_fold();
      if (other < a.cluster) {
        const float4 o = states[it][other];
        f = Fold{o.x, o.y, o.z, 0.f};
        if constexpr (SMOOTH) {
          const Part q = part_of<D>(a, row, other);
          f.n = float(q.e1 - q.e0);
        }
      }
      f = fold_lanes<SMOOTH>(f, a.lanes);
      if (label >= 0 && label < a.p.N) x_label = states[it][(int(label) + p.lead) / E / a.run].w;
    }
    const Slope sl = slope_of(a.p, row, f, label, x_label, rank == 0 && tid == 0);
    unsigned char* gr = a.p.g + row * a.p.g_pitch - p.lead * D::kBytes;  // the grid's first vector
    const int mine = p.j0 + tid, at = (label >= 0 && label < a.p.N ? int(label) + p.lead : -1) - mine * E;
    gr += int64_t(mine) * 16;
    grad_vectors<D, K>(sl, q, [&](int k) { return mine + k * T < p.j1; }, [&](int k) { return at - k * T * E; },
                       [&](int k, const float2(&y)[E / 2]) {
                         if (whole >> k & 1) {
                           st_stream16(gr + k * T * 16, D::pack2(y));
                         } else {
                           const int j = mine + k * T, from = max(0, p.lead - j * E), to = min(E, int(a.p.N) + p.lead - j * E);
#pragma unroll
                           for (int e = 0; e < E; ++e)
                             if (e >= from && e < to) D::store1(gr + k * T * 16, e, e & 1 ? y[e / 2].y : y[e / 2].x);
                         }
                       });
    if (++s == a.slots) {
      s = 0;
      parity ^= 1;
    }
  }
  if (timed_out) atomicOr(a.p.status, kStatusTimeout);
}

using Kernel = void (*)(Args);

// T threads a CTA, K vectors a thread.
template <class D, int T, int K>
Kernel pick(bool smooth, bool shift) {
  return smooth ? (shift ? k_loss_grad_cluster<D, T, K, true, true> : k_loss_grad_cluster<D, T, K, true, false>)
                : (shift ? k_loss_grad_cluster<D, T, K, false, true> : k_loss_grad_cluster<D, T, K, false, false>);
}
template <class D>
Kernel pick(int threads, bool smooth, bool shift) {
  return threads == 512 ? pick<D, 512, 8>(smooth, shift) : pick<D, 256, 8>(smooth, shift);
}

// Clusters of a launch that the device holds at once, asked once for each configuration (each time, it would be half of a call's time
// on the host).
cudaError_t resident_clusters(Kernel fn, const cudaLaunchConfig_t& cfg, int cluster, const DeviceInfo& dev, int* out) {
  struct Known {
    int device;
    Kernel fn;
    int cluster;
    size_t shared;
    int clusters;
  };
  constexpr int kMost = 256;
  static std::mutex mutex;
  static Known known[kMost];  // nothing is allocated, and so nothing thrown, behind the C calls
  static int held = 0;
  std::lock_guard<std::mutex> lock(mutex);
  for (int i = 0; i < held; ++i) {
    const Known& k = known[i];
    if (k.device == dev.device && k.fn == fn && k.cluster == cluster && k.shared == cfg.dynamicSmemBytes) {
      *out = k.clusters;
      return cudaSuccess;
    }
  }
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, (const void*)fn);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.max_smem_per_block_optin - int(attr.sharedSizeBytes));
  if (e == cudaSuccess) e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(out, (const void*)fn, &cfg);
  if (e == cudaSuccess) {
    if (held == kMost) held = 0;
    known[held++] = Known{dev.device, fn, cluster, cfg.dynamicSmemBytes, *out};
  }
  return e;
}

int64_t vectors_of(const LossGrad& p) { return (p.N + (16 / elem_bytes(p.dtype)) - 1) / (16 / elem_bytes(p.dtype)) + 1; }

constexpr int kHeld = 2048;  // vectors of a CTA of 256 threads
constexpr int64_t kMostVectors = int64_t(kMaxCluster) * 2 * kHeld;

}  // namespace

bool loss_grad_cluster_fits(const LossGrad& p) { return vectors_of(p) <= kMostVectors; }

cudaError_t launch_loss_grad_cluster(const LossGrad& p, const LossArgs& args, const DeviceInfo& dev) {
  Args a;
  a.p = args;
  const uintptr_t x = reinterpret_cast<uintptr_t>(args.x), g = reinterpret_cast<uintptr_t>(args.g);
  a.edges = ((x | g | uintptr_t(args.x_pitch) | uintptr_t(args.g_pitch) | uintptr_t(p.N * elem_bytes(p.dtype))) & 15) != 0;
  const bool shift = (((x - g) | uintptr_t(args.x_pitch - args.g_pitch)) & 15) != 0;
  const int64_t vectors = vectors_of(p) - (a.edges ? 0 : 1);
  // Eight CTAs of 256 threads hold a row of 256 KiB, four CTAs an SM; longer rows take 512 threads (4096 rows of 262144 bf16 entries:
  // 721 us; sixteen CTAs of 256 threads, 766).  As few CTAs as hold a row, whatever their number: 1023 x 50021 fp32 over seven
  // takes 69 us, over eight 75 (without smoothing).
  const int threads = vectors > 8 * kHeld ? 512 : 256;
  const int64_t held = int64_t(kHeld) * (threads / 256);
  a.cluster = int((vectors + held - 1) / held);
  // few rows: over more SMs (16 unaligned rows of 64 KiB 5.6 us against 6.8)
  while (a.cluster <= 4 && p.M * a.cluster * 2 <= dev.sm_count && vectors / (a.cluster * 2) >= 256) a.cluster *= 2;
  a.run = int((vectors + a.cluster - 1) / a.cluster);
  a.lanes = 1;
  while (a.lanes < a.cluster) a.lanes *= 2;
  a.slot_bytes = (a.run * 16 + 32 + 127) / 128 * 128;
  const int resident = threads == 512 ? 2 : 4;
  const int room = (dev.max_smem_per_sm / resident - 4096) / a.slot_bytes;
  a.slots = room < 1 ? 1 : room > kMaxSlots ? kMaxSlots : room;
  a.wait_ns = local_wait_limit_ns();
  const bool smooth = p.smoothing > 0.f;
  const Kernel fn = p.dtype == SOFTMAX_F32    ? pick<F32>(threads, smooth, shift)
                    : p.dtype == SOFTMAX_BF16 ? pick<BF16>(threads, smooth, shift)
                                              : pick<F16>(threads, smooth, shift);
  const int shared = a.slots * a.slot_bytes;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(a.cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = size_t(shared);
  cfg.stream = p.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(unsigned(a.cluster));
  int clusters = 0;
  if (const cudaError_t e = resident_clusters(fn, cfg, a.cluster, dev, &clusters); e != cudaSuccess) return e;
  if (clusters < 1) return cudaErrorLaunchOutOfResources;
  const int64_t n = p.M < clusters ? p.M : clusters;
  cfg.gridDim = dim3(unsigned(n * a.cluster));
  return cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace rwo
