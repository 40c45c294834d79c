// kernel_kv4_cache.cu -- tokens into and out of the 4-bit paged key/value cache.
//
// k_kv4_append: for each new token and head, rotate the key (and the queries) by the token's position, then for each
// group of 32 elements x of a key or value
//     z = f16(min x),  s = f16((max x - min x) / 15),  c = clamp(rint((x - z) / s), 0, 15)  (c = 0 where s = 0)
// in fp32, every operation rounded on its own and half-way quotients to the even code, so that the stored bytes can be
// reproduced on a host bit for bit.  x is limited to fp16's range first.
// k_kv4_gather: s c + z of the same tokens, rounded once to bf16 or fp16.
//
// A row (one head of one token) is d / 4 lanes of 4 elements; a group is 8 lanes, its minimum and maximum three
// shuffles.  Both are bound by the bytes that they move.
#include "kv4.cuh"

namespace rwo {
namespace {

constexpr int kCacheThreads = 256;

template <class D>
__device__ __forceinline__ float4 load4(const void* p, int64_t at) {
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(p) + at * 2);
  if constexpr (D::kNegInfWord == F16::kNegInfWord) return make_float4(f16_lo(w.x), f16_hi(w.x), f16_lo(w.y), f16_hi(w.y));
  else return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
template <class D>
__device__ __forceinline__ void store4(void* p, int64_t at, float4 v) {
  uint2 w;
  if constexpr (D::kNegInfWord == F16::kNegInfWord) w = make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w));
  else w = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  *reinterpret_cast<uint2*>(static_cast<unsigned char*>(p) + at * 2) = w;
}

// Offsets and lengths are looked at once for each call, by its first block: a row's own sequence may look right where
// another's offsets are wrong.
__device__ __forceinline__ void check_sequences(const Kv4View& c) {
  if (blockIdx.x) return;
  bool bad = false;
  for (int b = threadIdx.x; b < c.batch; b += kCacheThreads) kv4_seq(c, b, bad);
  if (bad) kv4_bad(c);
}

struct AppendArgs {
  Kv4View c;
  Kv4Rows k, v, q, q_out;
  const float* cos_sin;  // [positions][rot]: cosines, then sines; null: no rotation
  int64_t positions;
  int q_heads, rot, neighbours;
};

// Elements e .. e + 3 of a row, rotated by the position's angles.
template <class D>
__device__ __forceinline__ float4 rotated4(const void* p, int64_t row, int e, const float* cs, int rot, bool neighbours) {
  const float4 x = load4<D>(p, row + e);
  if (e >= rot) return x;
  const int half = rot >> 1;
  if (neighbours) {  // pairs (2 i, 2 i + 1)
    const float2 c = __ldg(reinterpret_cast<const float2*>(cs + (e >> 1)));
    const float2 s = __ldg(reinterpret_cast<const float2*>(cs + half + (e >> 1)));
    return make_float4(__fsub_rn(__fmul_rn(x.x, c.x), __fmul_rn(x.y, s.x)), __fadd_rn(__fmul_rn(x.y, c.x), __fmul_rn(x.x, s.x)),
                       __fsub_rn(__fmul_rn(x.z, c.y), __fmul_rn(x.w, s.y)), __fadd_rn(__fmul_rn(x.w, c.y), __fmul_rn(x.z, s.y)));
  }
  const bool first = e < half;  // pairs (i, i + rot / 2)
  const int i = first ? e : e - half;
  const float4 o = load4<D>(p, row + (first ? e + half : i));
  const float4 c = __ldg(reinterpret_cast<const float4*>(cs + i));
  float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + i));
  if (first) s = make_float4(-s.x, -s.y, -s.z, -s.w);
  return make_float4(__fadd_rn(__fmul_rn(x.x, c.x), __fmul_rn(o.x, s.x)), __fadd_rn(__fmul_rn(x.y, c.y), __fmul_rn(o.y, s.y)),
                     __fadd_rn(__fmul_rn(x.z, c.z), __fmul_rn(o.z, s.z)), __fadd_rn(__fmul_rn(x.w, c.w), __fmul_rn(o.w, s.w)));
}

__device__ __forceinline__ float limited(float x) { return fminf(fmaxf(x, -65504.f), 65504.f); }

// rint((x - z) / s) within 0 .. 15.  The reciprocal's quotient is off by less than 2^-18, so the division itself is
// needed only next to a half-way point.
__device__ __forceinline__ uint32_t code_of(float x, float z, float s, float inv) {
  const float t = __fsub_rn(x, z);
  float u = __fmul_rn(t, inv), c = rintf(u);
  if (fabsf(u - c) > 0.4999f) c = rintf(__fdiv_rn(t, s));
  return uint32_t(fminf(fmaxf(c, 0.f), 15.f));
}

template <class D, int DH>
__global__ void __launch_bounds__(kCacheThreads) k_kv4_append(AppendArgs a) {
  using B = Kv4Block<DH>;
  constexpr int kLanes = DH / 4, kRows = 32 / kLanes;
  const Kv4View& c = a.c;
  check_sequences(c);
  const int lane = threadIdx.x & 31, sub = lane / kLanes, e = (lane % kLanes) * 4;
  const int rows = 2 * c.heads + a.q_heads, units = (rows + kRows - 1) / kRows;
  const int64_t total = c.tokens * units;
  for (int64_t u = (int64_t(blockIdx.x) * kCacheThreads + threadIdx.x) >> 5; u < total; u += int64_t(gridDim.x) * (kCacheThreads / 32)) {
    const int64_t i = u / units;
    const int row = int(u - i * units) * kRows + sub;
    const int b = kv4_seq_of(c, i);
    if (b < 0) continue;  // uniform over the warp, as all below that depends on the token alone
    bool bad = false;
    const Kv4Seq s = kv4_seq(c, b, bad);
    const int pos = s.len - (s.start + s.n - int(i));
    int64_t at = -1;
    if (!bad && pos >= 0 && !(a.cos_sin && pos >= a.positions)) at = kv4_block_at(c, b, pos, B::kBytes);
    if (at < 0) {
      if (lane == 0) kv4_bad(c);
      continue;
    }
    const float* cs = a.cos_sin ? a.cos_sin + int64_t(pos) * a.rot : nullptr;
    const int rot = a.cos_sin ? a.rot : 0;
    const bool is_k = row < c.heads, is_v = !is_k && row < 2 * c.heads, is_q = !is_k && !is_v && row < rows;
    const int h = is_k ? row : is_v ? row - c.heads : row - 2 * c.heads;
    const Kv4Rows& src = is_k ? a.k : is_v ? a.v : a.q;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (is_k || is_v || is_q) x = rotated4<D>(src.p, i * src.token + h * src.head, e, cs, is_v ? 0 : rot, a.neighbours);
    __syncwarp();  // q may be rotated in place: every lane has its partner's elements
    if (is_q) store4<D>(const_cast<void*>(a.q_out.p), i * a.q_out.token + h * a.q_out.head + e, x);
    x = make_float4(limited(x.x), limited(x.y), limited(x.z), limited(x.w));
    float lo = fminf(fminf(x.x, x.y), fminf(x.z, x.w)), hi = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
    }
    const __half zh = __float2half_rn(lo), sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float z = __half2float(zh), sc = __half2float(sh);
    uint32_t four = 0;
    if (sc > 0.f) {
      const float inv = __frcp_rn(sc);
      four = code_of(x.x, z, sc, inv) | code_of(x.y, z, sc, inv) << 4 | code_of(x.z, z, sc, inv) << 8 | code_of(x.w, z, sc, inv) << 12;
    }
    if (!is_k && !is_v) continue;  // (no shuffles below)
    const int r = pos % kKv4Block, m = e >> 2, j = m >> 3, g = m & 7;
    unsigned char* blk = c.data + at + int64_t(h) * c.page_blocks * B::kBytes;
    uint16_t* hw = reinterpret_cast<uint16_t*>(blk);
    if (is_k) {
      hw[r * (DH / 4) + ((g >> 1) * B::G + j) * 2 + (g & 1)] = uint16_t(four);
      if (g == 0) {
        reinterpret_cast<__half*>(blk + B::kKScale)[r * B::G + j] = sh;
        reinterpret_cast<__half*>(blk + B::kKZero)[r * B::G + j] = zh;
      }
    } else {
      const int f = r >> 3, t = (r & 7) >> 1, ee = r & 1;
      hw[B::kV / 2 + (((f * 8 + g) * 4 + t) * B::G + j) * 2 + ee] = uint16_t(four);
      if (g == 0) {
        reinterpret_cast<__half*>(blk + B::kVScale)[((r >> 1) * B::G + j) * 2 + ee] = sh;
        reinterpret_cast<__half*>(blk + B::kVZero)[((r >> 1) * B::G + j) * 2 + ee] = zh;
      }
    }
  }
}

struct GatherArgs {
  Kv4View c;
  Kv4Rows k, v;
};

__device__ __forceinline__ float4 decoded4(uint32_t four, float s, float z) {
  return make_float4(__fmaf_rn(float(four & 15u), s, z), __fmaf_rn(float((four >> 4) & 15u), s, z),
                     __fmaf_rn(float((four >> 8) & 15u), s, z), __fmaf_rn(float((four >> 12) & 15u), s, z));
}

template <class D, int DH>
__global__ void __launch_bounds__(kCacheThreads) k_kv4_gather(GatherArgs a) {
  using B = Kv4Block<DH>;
  constexpr int kLanes = DH / 4, kRows = 32 / kLanes;
  const Kv4View& c = a.c;
  check_sequences(c);
  const int lane = threadIdx.x & 31, sub = lane / kLanes, m = lane % kLanes;
  const int units = (c.heads + kRows - 1) / kRows;
  const int64_t total = c.tokens * units;
  const int j = m >> 3, g = m & 7;
  for (int64_t u = (int64_t(blockIdx.x) * kCacheThreads + threadIdx.x) >> 5; u < total; u += int64_t(gridDim.x) * (kCacheThreads / 32)) {
    const int64_t i = u / units;
    const int h = int(u - i * units) * kRows + sub;
    const int b = kv4_seq_of(c, i);
    if (b < 0 || h >= c.heads) continue;
    bool bad = false;
    const Kv4Seq s = kv4_seq(c, b, bad);
    const int pos = s.len - (s.start + s.n - int(i));
    const int64_t at = !bad && pos >= 0 ? kv4_block_at(c, b, pos, B::kBytes) : -1;
    if (at < 0) {
      if (m == 0) kv4_bad(c);
      continue;
    }
    const int r = pos % kKv4Block, f = r >> 3, t = (r & 7) >> 1, ee = r & 1;
    const unsigned char* blk = c.data + at + int64_t(h) * c.page_blocks * B::kBytes;
    const uint16_t* hw = reinterpret_cast<const uint16_t*>(blk);
    const __half* sz = reinterpret_cast<const __half*>(blk + B::kKScale);
    const int ks = r * B::G + j, vs = ((r >> 1) * B::G + j) * 2 + ee;
    const float4 k = decoded4(hw[r * (DH / 4) + ((g >> 1) * B::G + j) * 2 + (g & 1)], __half2float(sz[ks]), __half2float(sz[16 * B::G + ks]));
    const float4 v = decoded4(hw[B::kV / 2 + (((f * 8 + g) * 4 + t) * B::G + j) * 2 + ee], __half2float(sz[32 * B::G + vs]),
                              __half2float(sz[48 * B::G + vs]));
    store4<D>(const_cast<void*>(a.k.p), i * a.k.token + h * a.k.head + 4 * m, k);
    store4<D>(const_cast<void*>(a.v.p), i * a.v.token + h * a.v.head + 4 * m, v);
  }
}

int grid_for(int64_t warps, const DeviceInfo& dev) {
  const int64_t blocks = (warps + kCacheThreads / 32 - 1) / (kCacheThreads / 32), most = int64_t(dev.sm_count) * 32;
  return int(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4View& c, const Kv4Rows& k, const Kv4Rows& v, const Kv4Rows& q, const Kv4Rows& q_out,
                              int q_heads, const float* cos_sin, int64_t positions, int rot, bool neighbours, int dtype,
                              cudaStream_t stream, const DeviceInfo& dev) {
  const AppendArgs a{c, k, v, q, q_out, cos_sin, positions, q_heads, rot, neighbours ? 1 : 0};
  const int per = c.d == 64 ? 2 : 1, rows = 2 * c.heads + q_heads;
  const int grid = grid_for(c.tokens * ((rows + per - 1) / per), dev);
  using Kern = void (*)(AppendArgs);
  const Kern kern = dtype == 2 ? (c.d == 64 ? (Kern)k_kv4_append<F16, 64> : (Kern)k_kv4_append<F16, 128>)
                               : (c.d == 64 ? (Kern)k_kv4_append<BF16, 64> : (Kern)k_kv4_append<BF16, 128>);
  kern<<<grid, kCacheThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const Kv4View& c, const Kv4Rows& k, const Kv4Rows& v, int dtype, cudaStream_t stream,
                              const DeviceInfo& dev) {
  const GatherArgs a{c, k, v};
  const int per = c.d == 64 ? 2 : 1;
  const int grid = grid_for(c.tokens * ((c.heads + per - 1) / per), dev);
  using Kern = void (*)(GatherArgs);
  const Kern kern = dtype == 2 ? (c.d == 64 ? (Kern)k_kv4_gather<F16, 64> : (Kern)k_kv4_gather<F16, 128>)
                               : (c.d == 64 ? (Kern)k_kv4_gather<BF16, 64> : (Kern)k_kv4_gather<BF16, 128>);
  kern<<<grid, kCacheThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace rwo
