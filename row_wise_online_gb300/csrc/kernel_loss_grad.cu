// kernel_loss_grad.cu -- the cross-entropy loss and its gradient (loss_grad.cuh): rows of up to 64 KiB in registers, two passes
// for rows that are too long for a cluster, and the choice.
#include "loss_grad.cuh"

namespace rwo {
namespace {

// ---- rows of up to 64 KiB: W warps a row, the row in registers --------------------------------------------------------
//
// Loaded once as packed vectors, 64 registers a thread, CTAs beside each other hide the waits.  Measured (bf16; in clusters with the next
// row's copy under way): rows of 16 KiB 324 us a 2 GiB launch (468), of 32 KiB 157 us a GiB (181), of 64 KiB 318 us (328), and 4.1
// us for 16 rows of 64 KiB (5.6).

__host__ __device__ constexpr int reg_threads(int warps) { return warps * 32 > 256 ? warps * 32 : 256; }

// VEC: 16-byte vectors, K a thread; else K single elements.
template <class D, int K, int W, bool VEC, bool SMOOTH>
__global__ void __launch_bounds__(reg_threads(W), 1024 / reg_threads(W)) k_loss_grad_reg(LossArgs a) {
  constexpr int E = VEC ? D::kVec : 1, GT = W * 32, G = reg_threads(W) / GT;
  __shared__ Fold parts[2][reg_threads(W) / 32];
  const int group = threadIdx.x / GT, t = threadIdx.x % GT, lane = threadIdx.x & 31, warp = t >> 5;
  const int units = int(a.N / E);
  int it = 0;
  for (int64_t row = int64_t(blockIdx.x) * G + group; row < a.M; row += int64_t(gridDim.x) * G, it ^= 1) {
    const unsigned char* xr = a.x + row * a.x_pitch;
    unsigned char* gr = a.g + row * a.g_pitch;
    const int64_t label = a.labels[row];
    const float x_label = t == 0 && label >= 0 && label < a.N ? load1c<D>(xr, label) : 0.f;
    Fold f;
    uint4 q[VEC ? K : 1];
    float v[VEC ? 1 : K];
    if constexpr (VEC) {
      uint32_t whole = 0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = t + k * GT;
        if (u < units) whole |= 1u << k;
        q[k] = u < units ? ld_stream16(xr + u * 16) : make_uint4(D::kNegInfWord, D::kNegInfWord, D::kNegInfWord, D::kNegInfWord);
      }
      f = fold_vectors<D, K, SMOOTH>(q, whole);
    } else {
      f = empty_fold();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = t + k * GT;
        v[k] = u < units ? D::load1(xr, u) : -INFINITY;
        f.m = fmaxf(f.m, v[k]);
      }
      const float ms = safe_max(f.m);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        f.d += exp_diff(v[k], ms);
        if (SMOOTH && t + k * GT < units) {
          f.s += ms - v[k];
          f.n += 1.f;
        }
      }
    }
    f = fold_lanes<SMOOTH>(f, 32);
    if constexpr (W > 1) {
      Fold* mine = parts[it] + group * W;
      if (lane == 0) mine[warp] = f;
      named_barrier_sync(1 + group, GT);
      f = fold_lanes<SMOOTH>(mine[lane & (W - 1)], W);
    } else {
      __syncwarp();  // x_label is read before the row is overwritten
    }
    const Slope s = slope_of(a, row, f, label, x_label, t == 0);
    if constexpr (VEC) {
      const int at = label >= 0 && label < a.N ? int(label) - t * E : -1 - t * E;
      grad_vectors<D, K>(s, q, [&](int k) { return t + k * GT < units; }, [&](int k) { return at - k * GT * E; },
                         [&](int k, const float2(&y)[E / 2]) { st_stream16(gr + (t + k * GT) * 16, D::pack2(y)); });
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int u = t + k * GT;
        if (u >= units) continue;
        float y = grad_of(s, v[k]);
        if (s.live && u == label) y -= s.c;
        D::store1(gr, u, y);
      }
    }
  }
}

// ---- two passes, rows of any length and alignment ------------------------------------------------------------------

constexpr int kThreads = 512;

// A thread's sums are relative to a reference that rises to the maximum only when that is kRise above it, not to the maximum itself: each time
// they are rescaled they take on the exponential's error, and entries that rise along a row of millions did so 8192 times (1.5e-5 of
// the sum).  e^kRise times 2^31 terms is far from fp32's range.
constexpr float kRise = 8.f;
constexpr int kBatch = 4;

// A CTA a row: the fold, then the gradient from a second read.  VEC: 16-byte units, else single elements, kBatch of them under way.
// Four CTAs an SM, as many as the grid counts on (2000 rows of 600001 bf16 1839 us; single elements one by one, 2972), but for vectors without
// smoothing, which gain nothing by it (8 x 4194304 bf16 854 us, held to 32 registers 999).
template <class D, bool VEC, bool SMOOTH>
__global__ void __launch_bounds__(kThreads, VEC && !SMOOTH ? 0 : 4) k_loss_grad_twopass(LossArgs a) {
  constexpr int E = VEC ? D::kVec : 1, B = VEC ? E : kBatch;
  __shared__ Fold parts[2][kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t units = a.N / E;
  int it = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, it ^= 1) {
    const unsigned char* xr = a.x + row * a.x_pitch;
    unsigned char* gr = a.g + row * a.g_pitch;
    const int64_t label = a.labels[row];
    // read before any element is overwritten: the gradient may go where the logits are
    const float x_label = label >= 0 && label < a.N ? load1c<D>(xr, label) : 0.f;
    Fold f = empty_fold();  // f.m: the reference
    float top = -INFINITY;
    float lost = 0.f;  // what the additions to f.d rounded away (long runs of a thread)
    LongSum far;       // f.s, alike (added up plainly, 2^22 equal distances are off by 8e-5)
    uint4 q;  // VEC: with smoothing the next vector is under way meanwhile
    if (VEC && SMOOTH) q = ld16(xr + (threadIdx.x < units ? threadIdx.x : 0) * 16);
    for (int64_t u = threadIdx.x; u < units; u += kThreads * (VEC ? 1 : B)) {
      float v[B];
      if constexpr (VEC) {
        if (!SMOOTH) q = ld16(xr + u * 16);
        D::unpack(q, v);
        if (SMOOTH && u + kThreads < units) q = ld16(xr + (u + kThreads) * 16);
      } else {
#pragma unroll
        for (int e = 0; e < B; ++e) v[e] = u + e * kThreads < units ? D::load1(xr, u + e * kThreads) : -INFINITY;
      }
      float mx = v[0];
#pragma unroll
      for (int e = 1; e < B; ++e) mx = fmaxf(mx, v[e]);
      top = fmaxf(top, mx);
      if (mx > f.m + kRise) {
        const float k = exp_diff(f.m, mx);
        f.d *= k;
        lost *= k;
        if constexpr (SMOOTH) {
          if (f.n > 0.f) {
            const float by = mx - safe_max(f.m), move = f.n * by;
            far.add(move);
            far.add(__fmaf_rn(f.n, by, -move));
          }
        }
        f.m = mx;
      }
      const float ms = safe_max(f.m);
      float t = 0.f, r = 0.f;
#pragma unroll
      for (int e = 0; e < B; ++e) {
        t += exp_diff(v[e], ms);
        if constexpr (SMOOTH) {
          if (VEC || u + e * kThreads < units) {
            r += ms - v[e];
            f.n += 1.f;
          }
        }
      }
      const float want = t - lost, sum = __fadd_rn(f.d, want);
      lost = __fsub_rn(__fsub_rn(sum, f.d), want);
      f.d = sum;
      if constexpr (SMOOTH) far.add(r);
    }
    f.s = far.s;
    f.d *= exp_diff(f.m, safe_max(top));
    if constexpr (SMOOTH) f.s = moved(f, safe_max(top));
    f.m = top;
    f = fold_lanes<SMOOTH>(f, 32);
    if (lane == 0) parts[it][warp] = f;
    __syncthreads();
    f = fold_lanes<SMOOTH>(parts[it][lane & (kThreads / 32 - 1)], kThreads / 32);
    const Slope s = slope_of(a, row, f, label, x_label, threadIdx.x == 0);
    for (int64_t u = threadIdx.x; u < units; u += kThreads) {
      float v[E];
      if constexpr (VEC) D::unpack(ld16(xr + u * 16), v);
      else v[0] = D::load1(xr, u);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[e] = grad_of(s, v[e]);
        if (s.live && u * E + e == label) v[e] -= s.c;
      }
      if constexpr (VEC) st_stream16(gr + u * 16, D::pack(v));
      else D::store1(gr, u, v[0]);
    }
  }
}

using Kernel = void (*)(LossArgs);

struct RegConfig {
  int warps, units;  // warps a row, units they hold
  Kernel fn[2];      // [smoothing]
};
template <class D, int K, int W, bool VEC>
constexpr RegConfig reg() {
  return RegConfig{W, 32 * W * K, {k_loss_grad_reg<D, K, W, VEC, false>, k_loss_grad_reg<D, K, W, VEC, true>}};
}

template <class D>
cudaError_t launch_type(const LossGrad& p, const LossArgs& a, const DeviceInfo& dev) {
  static const RegConfig vectors[] = {reg<D, 1, 1, true>(), reg<D, 2, 1, true>(), reg<D, 4, 1, true>(), reg<D, 4, 2, true>(), reg<D, 4, 4, true>(), reg<D, 4, 8, true>(), reg<D, 8, 8, true>(), reg<D, 8, 16, true>()};
  static const RegConfig elements[] = {reg<D, 2, 1, false>(), reg<D, 8, 1, false>(), reg<D, 8, 4, false>(), reg<D, 16, 4, false>(), reg<D, 16, 8, false>(), reg<D, 32, 8, false>()};
  const bool smooth = p.smoothing > 0.f;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.g) | uintptr_t(a.x_pitch) | uintptr_t(a.g_pitch) |
                     uintptr_t(p.N * D::kBytes)) & 15) == 0;
  const int64_t units = vec ? p.N / D::kVec : p.N;
  const RegConfig* tab = vec ? vectors : elements;
  // rows on no boundary by single elements: up to 4096, in 32 bits 8192 (clusters in their place: 20000 rows of 3001 bf16 139 us
  // against 111, 10000 of 7999 fp32 109 against 98; but 10000 of 8001 bf16 82 against 117)
  for (int i = 0; i < (vec ? 8 : D::kBytes == 4 ? 6 : 5); ++i) {
    if (units > tab[i].units) continue;
    const int threads = reg_threads(tab[i].warps);
    const int64_t groups = threads / 32 / tab[i].warps, ctas = (p.M + groups - 1) / groups;
    const int64_t slots = int64_t(dev.sm_count) * (dev.max_threads_per_sm / threads) * 4;
    tab[i].fn[smooth]<<<unsigned(ctas < slots ? ctas : slots), threads, 0, p.stream>>>(a);
    return cudaGetLastError();
  }
  if (loss_grad_cluster_fits(p)) return launch_loss_grad_cluster(p, a, dev);
  const Kernel k = vec ? (smooth ? k_loss_grad_twopass<D, true, true> : k_loss_grad_twopass<D, true, false>)
                       : (smooth ? k_loss_grad_twopass<D, false, true> : k_loss_grad_twopass<D, false, false>);
  const int64_t slots = int64_t(dev.sm_count) * (dev.max_threads_per_sm / kThreads);
  k<<<unsigned(p.M < slots ? p.M : slots), kThreads, 0, p.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_loss_grad(const LossGrad& p, const DeviceInfo& dev) {
  LossArgs a;
  const int64_t s = elem_bytes(p.dtype);
  a.x = static_cast<const unsigned char*>(p.x);
  a.g = static_cast<unsigned char*>(p.grad);
  a.labels = p.labels;
  a.upstream = p.upstream;
  a.loss = p.loss;
  a.lse = p.lse;
  a.M = p.M;
  a.N = p.N;
  a.x_pitch = p.x_pitch * s;
  a.g_pitch = p.g_pitch * s;
  a.grad_scale = p.grad_scale;
  a.smoothing = p.smoothing;
  a.z = p.z;
  a.smoothing_each = p.smoothing / float(p.N);
  a.status = dev.status;
  return p.dtype == SOFTMAX_F32 ? launch_type<F32>(p, a, dev) : p.dtype == SOFTMAX_BF16 ? launch_type<BF16>(p, a, dev) : launch_type<F16>(p, a, dev);
}

}  // namespace rwo
