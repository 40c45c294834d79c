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
// shuffles.  Few tokens are taken row by row, where latency bounds (128 rows: 4.7 us in, 2.2 back); longer runs a block of 16
// tokens at a time, so that the cache is touched in whole blocks.  Reading back is bound by bytes: 154480 tokens of 8 heads of
// 128 take 131 us (floor 123).  Writing is bound by latency: 15714 tokens of 8 heads of 128 with 32 rotated query heads take
// 85 us (the bytes alone 52); half as many (ncu) keep issue 53% and DRAM 39% busy with 41% of the warps resident, which
// wait for rows from memory more than for anything else.
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

// ---- runs of tokens -------------------------------------------------------------------------------------------
//
// Where sequences bring many tokens (prompts, prefixes read back), a warp takes a block of 16 tokens of one head: the
// lookups are made once for the block and whole words move.  The blocks that the call's tokens touch form one list over
// the sequences, cut into equal parts, one a CTA; each CTA finds its part by a scan over the sequences.

// The blocks of sequence b's new tokens: positions [len - n, len).  Tokens before the sequence's start have none, nor has
// a sequence whose length or offsets are out of range.
struct RunSeq {
  Kv4Seq s;
  int first, blocks;  // first block, how many
};
__device__ __forceinline__ RunSeq run_seq(const Kv4View& c, int b, bool& bad) {
  RunSeq r;
  bool wrong = false;
  r.s = kv4_seq(c, b, wrong);
  const int p0 = r.s.len - r.s.n;
  bad |= wrong || p0 < 0;
  r.first = max(p0, 0) / kKv4Block;
  r.blocks = !wrong && r.s.n > 0 && r.s.len > 0 ? (r.s.len - 1) / kKv4Block - r.first + 1 : 0;
  return r;
}

// Calls f(sequence, block of it, sub-task) for the units of this warp, `subs` a block; this CTA is number `part` of `parts`.
template <class F>
__device__ __forceinline__ void for_units(const Kv4View& c, int subs, int part, int parts, F f) {
  __shared__ int64_t scan[kCacheThreads / 32];
  __shared__ int where[2];  // sequence, first unit of it
  __shared__ int taken;     // units of this CTA's part that warps have taken: they take turns, as units differ in work
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (c.batch + kCacheThreads - 1) / kCacheThreads, b0 = min(tid * per, c.batch), b1 = min(b0 + per, c.batch);
  bool bad = false;
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += int64_t(run_seq(c, b, bad).blocks) * subs;
  int64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) scan[warp] = upto;
  if (tid == 0) taken = kCacheThreads / 32;
  __syncthreads();
  int64_t all = 0, below = upto - sum;
  for (int w = 0; w < kCacheThreads / 32; ++w) {
    if (w < warp) below += scan[w];
    all += scan[w];
  }
  // Offsets that ascend give fewer units than 2^31 (the host saw to that); where some descend, sequences overlap and may not.
  const bool many = all >= (int64_t(1) << 31);
  if ((bad || many) && part == 0) kv4_bad(c);
  if (many) return;
  const int total = int(all), before = int(below), mine = int(sum);
  const int u0 = int(int64_t(total) * part / parts), u1 = int(int64_t(total) * (part + 1) / parts);
  if (u0 >= u1) return;
  if (u0 >= before && u0 < before + mine) {
    int at = before;
    for (int b = b0; b < b1; ++b) {
      const int n = run_seq(c, b, bad).blocks * subs;
      if (u0 < at + n) {
        where[0] = b;
        where[1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  int b = where[0];
  int at = where[1];
  RunSeq r = run_seq(c, b, bad);
  for (int u = u0 + warp; u < u1;) {
    while (u >= at + r.blocks * subs) {
      at += r.blocks * subs;
      r = run_seq(c, ++b, bad);
    }
    const int x = (u - at) / subs;
    f(b, r, r.first + x, u - at - x * subs);
    int next = 0;
    if (lane == 0) next = atomicAdd(&taken, 1);
    u = u0 + __shfl_sync(kFull, next, 0);
  }
}

template <class D>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(static_cast<unsigned char*>(p) + at * 2) = D::pack(f);
}

// a b + c d, products and sum each rounded.  (The additions are scalar: a packed product and a packed addition after it
// come out of the compiler as one fused operation, .rn or not, which rounds once.)
__device__ __forceinline__ float2 sum_of_products(float2 a, float2 b, float2 c, float2 d) {
  const float2 x = __fmul2_rn(a, b), y = __fmul2_rn(c, d);
  return make_float2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

// Angles of elements e .. e + 7 at a position, as pairs (neighbours: one angle a pair, in x and y of c alone).
struct Turn {
  float2 c[4], s[4];
};
__device__ __forceinline__ Turn turn_at(const float* cs, int rot, int e, bool neighbours) {
  Turn t;
  const int half = rot >> 1;
  if (neighbours) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + (e >> 1))), s = __ldg(reinterpret_cast<const float4*>(cs + half + (e >> 1)));
    t.c[0] = make_float2(c.x, c.x);
    t.c[1] = make_float2(c.y, c.y);
    t.c[2] = make_float2(c.z, c.z);
    t.c[3] = make_float2(c.w, c.w);
    t.s[0] = make_float2(s.x, s.x);
    t.s[1] = make_float2(s.y, s.y);
    t.s[2] = make_float2(s.z, s.z);
    t.s[3] = make_float2(s.w, s.w);
    return t;
  }
  const float* p = cs + (e < half ? e : e - half);
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(p + 2 * i)), s = __ldg(reinterpret_cast<const float4*>(p + half + 2 * i));
    t.c[i] = make_float2(c.x, c.y);
    t.c[i + 1] = make_float2(c.z, c.w);
    t.s[i] = make_float2(s.x, s.y);
    t.s[i + 1] = make_float2(s.z, s.w);
  }
  return t;
}

// Eight elements (packed in x) of a row rotated: y = x cos + o sin with o the partner, negated for the first of a pair.
// Without neighbours the partners are the elements of lane `from` (rot / 2 is a multiple of 8 here); flip: their signs'
// bits where they are second.  All lanes take part.
template <class D>
__device__ __forceinline__ void turned(float2 (&f)[4], uint4 x, bool on, bool neighbours, int from, uint32_t flip, const Turn& t) {
  uint4 w;
  if (neighbours) {
    w = make_uint4(__funnelshift_l(x.x, x.x, 16) ^ 0x8000u, __funnelshift_l(x.y, x.y, 16) ^ 0x8000u,
                   __funnelshift_l(x.z, x.z, 16) ^ 0x8000u, __funnelshift_l(x.w, x.w, 16) ^ 0x8000u);
  } else {
    w = make_uint4(__shfl_sync(kFull, x.x, from) ^ flip, __shfl_sync(kFull, x.y, from) ^ flip, __shfl_sync(kFull, x.z, from) ^ flip,
                   __shfl_sync(kFull, x.w, from) ^ flip);
  }
  D::unpack2(x, f);
  if (on) {
    float2 o[4];
    D::unpack2(w, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = sum_of_products(f[i], t.c[i], o[i], t.s[i]);
  }
}

__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// c << 8 | b << 4 | a with a and b limited to 0 .. 15.
__device__ __forceinline__ uint32_t pack_codes(uint32_t c, int b, int a) {
  uint32_t d;
  asm("cvt.pack.sat.u4.s32.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(b), "r"(a), "r"(c));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Codes of eight elements of a group that four lanes hold (nibble i: element i), its scale and zero.
__device__ __forceinline__ uint32_t quantised8(float2 (&x)[4], __half& sh, __half& zh) {
  float lo = fminf(min3(x[0].x, x[0].y, x[1].x), min3(x[1].y, x[2].x, x[2].y)), hi = fmaxf(max3(x[0].x, x[0].y, x[1].x), max3(x[1].y, x[2].x, x[2].y));
  lo = min3(lo, x[3].x, x[3].y);
  hi = max3(hi, x[3].x, x[3].y);
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
  }
  if (!(lo >= -65504.f && hi <= 65504.f)) {  // (a group of NaN alone too: scales and zeros are finite, whatever comes in)
    lo = limited(lo);
    hi = limited(hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(limited(x[i].x), limited(x[i].y));
  }
  zh = __float2half_rn(lo);
  sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
  const float z = __half2float(zh), s = __half2float(sh);
  if (!(s > 0.f)) return 0u;
  // Adding 1.5 2^23 rounds a quotient to the nearest integer, ties to even, in the sum's low bits.  (A quotient lies in
  // [0, 15] but for the roundings of z and s, which can take it no further than 2^18.)
  constexpr float kRound = 12582912.f;
  float i1;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i1) : "f"(s));
  const float2 inv = both(i1);
  uint32_t eight = 0;
  float edge = 0.f;  // largest distance from the integer
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const float2 u = __fmul2_rn(__fadd2_rn(x[i], both(-z)), inv);
    const float2 r = __fadd2_rn(u, both(kRound)), c = __fadd2_rn(r, both(-kRound));
    const float2 d = __fadd2_rn(u, make_float2(-c.x, -c.y));
    edge = max3(edge, fabsf(d.x), fabsf(d.y));
    eight = pack_codes(eight, __float_as_int(r.y) - 0x4b400000, __float_as_int(r.x) - 0x4b400000);
  }
  if (edge > 0.4999f) {  // next to a half-way point the division itself is needed (the quotients above are off by 2^-17 at most)
    eight = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i)
      eight = eight << 8 | code_of(x[i].y, z, s, i1) << 4 | code_of(x[i].x, z, s, i1);
  }
  return eight;
}

constexpr int kAppendCtas = 4;  // resident on an SM: 64 registers a thread (15714 prompt tokens: 85 us; with three, 96)
constexpr int kDepth = 2;       // rows that a lane loads ahead (1: 87 us, 3: 93)
constexpr int kQHeads = 32;  // query heads of a warp: a token's angles are loaded once for them

// CTAs that write the cache and CTAs that rotate queries take turns in the grid, so that the ones' arithmetic runs beside
// the others' traffic.
template <class D, int DH>
__global__ void __launch_bounds__(kCacheThreads, kAppendCtas) k_kv4_append_runs(AppendArgs a, int kv_ctas) {
  using B = Kv4Block<DH>;
  constexpr int kLanes = DH / 8, kRows = 32 / kLanes;  // lanes a row; rows a warp moves at once
  const Kv4View& c = a.c;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, e = (lane % kLanes) * 8;
  const int rot = a.cos_sin ? a.rot : 0;
  const bool neighbours = a.neighbours, second = e >= (rot >> 1);
  const int partner = second ? lane - rot / 16 : lane + rot / 16;
  const uint32_t flip = second ? 0u : 0x80008000u;
  const int q_ctas = int(gridDim.x) - kv_ctas, mixed = 2 * min(q_ctas, kv_ctas), id = int(blockIdx.x);
  const bool q_turn = id < mixed ? id & 1 : q_ctas > kv_ctas;
  const int part = id < mixed ? id >> 1 : id - mixed / 2;
  // Pointers are made once and stepped from row to row: 64-bit products for every row had been half of the instructions.
  if (q_turn) {  // a warp takes kQHeads heads of a token, kRows at once
    const int chunks = (a.q_heads + kQHeads - 1) / kQHeads;
    const int64_t w = int64_t(part) * (kCacheThreads / 32) + (threadIdx.x >> 5), i = w / chunks;
    if (i >= c.tokens) return;
    const int b = kv4_seq_of(c, i);
    if (b < 0) return;
    bool bad = false;
    const Kv4Seq s = kv4_seq(c, b, bad);
    const int pos = s.len - (s.start + s.n - int(i));
    if (bad || pos < 0 || (rot && pos >= a.positions)) return;  // (the CTAs that write the cache report these)
    if (kv4_block_at(c, b, pos, B::kBytes) < 0) return;
    Turn t;
    if (e < rot) t = turn_at(a.cos_sin + int64_t(pos) * rot, rot, e, neighbours);
    int h = int(w - i * chunks) * kQHeads + sub;
    const int h1 = min(int(w - i * chunks) * kQHeads + kQHeads, a.q_heads);
    const unsigned char* from = static_cast<const unsigned char*>(a.q.p) + (i * a.q.token + h * a.q.head + e) * 2;
    unsigned char* to = const_cast<unsigned char*>(static_cast<const unsigned char*>(a.q_out.p)) + (i * a.q_out.token + h * a.q_out.head + e) * 2;
    const int64_t step = a.q.head * (2 * kRows), step_out = a.q_out.head * (2 * kRows);
    uint4 next[kDepth];  // rows on their way while earlier ones are turned
#pragma unroll
    for (int m = 0; m < kDepth; ++m)
      if (h + m * kRows < h1) next[m] = *reinterpret_cast<const uint4*>(from + m * step);
#pragma unroll 1
    while (__any_sync(kFull, h < h1)) {
      uint4 x = next[0];
#pragma unroll
      for (int m = 1; m < kDepth; ++m) next[m - 1] = next[m];
      if (h + kDepth * kRows < h1) next[kDepth - 1] = *reinterpret_cast<const uint4*>(from + kDepth * step);
      from += step;
      if (rot) {
        float2 f[4];
        turned<D>(f, x, e < rot, neighbours, partner, flip, t);  // (shuffles: a row's lanes have its elements before one is written)
        x = D::pack2(f);
      }
      if (h < h1) *reinterpret_cast<uint4*>(to) = x;
      to += step_out;
      h += kRows;
    }
    return;
  }
  const int kv_units = c.heads;
  for_units(c, 2 * c.heads, part, kv_ctas, [&](int b, const RunSeq& rs, int blk, int what) {
    const int64_t at = kv4_block_at(c, b, blk * kKv4Block, B::kBytes);
    const int p0 = max(rs.s.len - rs.s.n, blk * kKv4Block), p1 = min(rs.s.len, (blk + 1) * kKv4Block);
    const int last = a.cos_sin && p1 > a.positions ? int(a.positions) : p1;  // positions [p0, last) are handled
    if (at < 0 || last < p1) {
      if (lane == 0) kv4_bad(c);
      if (at < 0) return;
    }
    const int64_t row0 = int64_t(rs.s.start) + rs.s.n - rs.s.len;  // row of position 0
    const bool is_v = what >= kv_units;
    const int h = is_v ? what - c.heads : what;
    const Kv4Rows& src = is_v ? a.v : a.k;
    const int turn = is_v ? 0 : rot, j = e >> 5, t8 = (e & 31) >> 3;
    unsigned char* out = c.data + at + int64_t(h) * c.page_blocks * B::kBytes;
    const int first = blk * kKv4Block + sub;  // this lane's first position
    const unsigned char* from = static_cast<const unsigned char*>(src.p) + ((row0 + first) * src.token + h * src.head + e) * 2;
    const float* cs = a.cos_sin + int64_t(first) * rot;
    const int64_t step = src.token * (2 * kRows);
    uint4 next[kDepth];  // rows on their way while earlier ones are quantised
#pragma unroll
    for (int m = 0; m < kDepth; ++m) {
      next[m] = make_uint4(0u, 0u, 0u, 0u);
      if (first + m * kRows >= p0 && first + m * kRows < last) next[m] = *reinterpret_cast<const uint4*>(from + m * step);
    }
#pragma unroll 1
    for (int r = sub; r < kKv4Block; r += kRows) {  // kRows tokens of the block
      const int p = blk * kKv4Block + r, then = p + kDepth * kRows;
      const bool on = p >= p0 && p < last;
      const uint4 x = next[0];
#pragma unroll
      for (int m = 1; m < kDepth; ++m) next[m - 1] = next[m];
      if (r + kDepth * kRows < kKv4Block && then >= p0 && then < last) next[kDepth - 1] = *reinterpret_cast<const uint4*>(from + kDepth * step);
      from += step;
      if (__any_sync(kFull, on)) {
        float2 f[4];
        if (turn) {
          Turn t;
          if (on && e < turn) t = turn_at(cs, rot, e, neighbours);
          turned<D>(f, x, on && e < turn, neighbours, partner, flip, t);
        } else {
          D::unpack2(x, f);
        }
        __half sh, zh;
        const uint32_t eight = quantised8(f, sh, zh);
        if (!is_v) {
          if (on) {
            reinterpret_cast<uint32_t*>(out)[r * (DH / 8) + B::G * t8 + j] = eight;
            if (t8 == 0) {
              reinterpret_cast<__half*>(out + B::kKScale)[r * B::G + j] = sh;
              reinterpret_cast<__half*>(out + B::kKZero)[r * B::G + j] = zh;
            }
          }
        } else {  // a word holds four elements of two tokens: the lanes of an even and an odd token make one each
          const uint32_t other = __shfl_xor_sync(kFull, eight, kLanes);
          const bool odd = r & 1;
          const bool pair = __shfl_xor_sync(kFull, on ? 1 : 0, kLanes) && on;
          const int fh = r >> 3, tt = (r & 7) >> 1;
          uint32_t* w = reinterpret_cast<uint32_t*>(out + B::kV) + ((fh * 8 + 2 * t8) * 4 + tt) * B::G + j;  // g = 2 t8; g + 1 is 4 G further
          if (pair) {
            w[odd ? 4 * B::G : 0] = odd ? (other >> 16) | (eight & 0xffff0000u) : (eight & 0xffffu) | (other << 16);
          } else if (on) {
            reinterpret_cast<uint16_t*>(w)[odd] = uint16_t(eight);
            reinterpret_cast<uint16_t*>(w + 4 * B::G)[odd] = uint16_t(eight >> 16);
          }
          if (on && t8 == 0) {
            reinterpret_cast<__half*>(out + B::kVScale)[((r >> 1) * B::G + j) * 2 + odd] = sh;
            reinterpret_cast<__half*>(out + B::kVZero)[((r >> 1) * B::G + j) * 2 + odd] = zh;
          }
        }
      }
      cs += kRows * rot;
    }
  });
}

template <int n>
__device__ __forceinline__ void load_words(uint32_t (&w)[n], const uint32_t* p) {
  if constexpr (n == 4) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x;
    w[1] = v.y;
  }
}

constexpr int kGatherCtas = 4;  // resident on an SM; 154480 tokens of 8 heads: 131 us, 143 with 3, 163 with 5 (two waves)

template <class D, int DH>
__global__ void __launch_bounds__(kCacheThreads) k_kv4_gather_runs(GatherArgs a) {
  using B = Kv4Block<DH>;
  constexpr int G = B::G;
  const Kv4View& c = a.c;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  for_units(c, c.heads, int(blockIdx.x), int(gridDim.x), [&](int b, const RunSeq& rs, int blk, int h) {
    int64_t at = kv4_block_at(c, b, blk * kKv4Block, B::kBytes);
    if (at < 0) {
      if (lane == 0) kv4_bad(c);
      return;
    }
    const unsigned char* from = c.data + at + int64_t(h) * c.page_blocks * B::kBytes;
    const int p0 = max(rs.s.len - rs.s.n, 0);
    const int64_t row0 = int64_t(rs.s.start) + rs.s.n - rs.s.len;
    // keys: lane (g, t) has words G t .. of token g, then of token g + 8
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i, p = blk * kKv4Block + r;
      if (p < p0 || p >= rs.s.len) continue;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(from) + r * (DH / 8) + G * t;
      const __half* s = reinterpret_cast<const __half*>(from + B::kKScale) + r * G;
      uint32_t x[G];
      load_words<G>(x, w);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const float4 lo = decoded4(x[j] & 0xffffu, __half2float(s[j]), __half2float(s[16 * G + j]));
        const float4 hi = decoded4(x[j] >> 16, __half2float(s[j]), __half2float(s[16 * G + j]));
        const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        store8<D>(const_cast<void*>(a.k.p), (row0 + p) * a.k.token + h * a.k.head + 32 * j + 8 * t, f);
      }
    }
    // values: lane (g, t) has words of tokens 8 f + 2 t and the next
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(from + B::kV) + ((f * 8 + g) * 4 + t) * G;
      const uint32_t* s = reinterpret_cast<const uint32_t*>(from + B::kVScale) + (4 * f + t) * G;
      uint32_t xs[G], ss[G], zs[G];
      load_words<G>(xs, w);
      load_words<G>(ss, s);
      load_words<G>(zs, s + 8 * G);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const uint32_t x = xs[j], sc = ss[j], z = zs[j];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int p = blk * kKv4Block + 8 * f + 2 * t + k;
          if (p < p0 || p >= rs.s.len) continue;
          const float4 v = decoded4(k ? x >> 16 : x & 0xffffu, k ? f16_hi(sc) : f16_lo(sc), k ? f16_hi(z) : f16_lo(z));
          store4<D>(const_cast<void*>(a.v.p), (row0 + p) * a.v.token + h * a.v.head + 32 * j + 4 * g, v);
        }
      }
    }
  });
}

int grid_for(int64_t warps, const DeviceInfo& dev) {
  const int64_t blocks = (warps + kCacheThreads / 32 - 1) / (kCacheThreads / 32), most = int64_t(dev.sm_count) * 32;
  return int(blocks < most ? blocks : most);
}

// Runs of at least 4 tokens a sequence on average go by blocks of 16, fewer by single rows: a block's lookups and the scan
// are shared by its tokens.  (128 sequences of 1 token: 2.2 us read back by rows; 154480 tokens in 4 sequences: 375 by rows,
// 131 by blocks.)  Units are counted in 32 bits.
int64_t run_units(const Kv4View& c, int subs) { return (c.tokens / kKv4Block + 2 * int64_t(c.batch)) * subs; }
bool in_runs(const Kv4View& c, int subs) { return c.cu && c.tokens >= 4 * int64_t(c.batch) && run_units(c, subs) < (int64_t(1) << 31); }
// There a lane's eight elements have their partners in one other lane: rot / 2 is a multiple of 8, or pairs are neighbours.
bool whole_lanes(const float* cos_sin, int rot, bool neighbours) { return !cos_sin || neighbours || rot % 16 == 0; }
// As many CTAs as are resident at once (`per_sm`), fewer where there is not a unit a warp.
int grid_for_runs(const Kv4View& c, int subs, int per_sm, const DeviceInfo& dev) {
  const int64_t few = (run_units(c, subs) + 7) / 8, most = int64_t(dev.sm_count) * per_sm;
  return int(few < most ? few : most);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4View& c, const Kv4Rows& k, const Kv4Rows& v, const Kv4Rows& q, const Kv4Rows& q_out,
                              int q_heads, const float* cos_sin, int64_t positions, int rot, bool neighbours, int dtype,
                              cudaStream_t stream, const DeviceInfo& dev) {
  const AppendArgs a{c, k, v, q, q_out, cos_sin, positions, q_heads, rot, neighbours ? 1 : 0};
  const int64_t q_ctas = (c.tokens * ((q_heads + kQHeads - 1) / kQHeads) + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
  if (in_runs(c, 2 * c.heads) && whole_lanes(cos_sin, rot, neighbours)) {
    using Kern = void (*)(AppendArgs, int);
    const Kern kern = dtype == 2 ? (c.d == 64 ? (Kern)k_kv4_append_runs<F16, 64> : (Kern)k_kv4_append_runs<F16, 128>)
                                 : (c.d == 64 ? (Kern)k_kv4_append_runs<BF16, 64> : (Kern)k_kv4_append_runs<BF16, 128>);
    const int kv_ctas = grid_for_runs(c, 2 * c.heads, 3, dev);
    kern<<<unsigned(kv_ctas + q_ctas), kCacheThreads, 0, stream>>>(a, kv_ctas);
    return cudaGetLastError();
  }
  using Kern = void (*)(AppendArgs);
  const int per = c.d == 64 ? 2 : 1, rows = 2 * c.heads + q_heads;
  const int grid = grid_for(c.tokens * ((rows + per - 1) / per), dev);
  const Kern kern = dtype == 2 ? (c.d == 64 ? (Kern)k_kv4_append<F16, 64> : (Kern)k_kv4_append<F16, 128>)
                               : (c.d == 64 ? (Kern)k_kv4_append<BF16, 64> : (Kern)k_kv4_append<BF16, 128>);
  kern<<<grid, kCacheThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const Kv4View& c, const Kv4Rows& k, const Kv4Rows& v, int dtype, cudaStream_t stream,
                              const DeviceInfo& dev) {
  const GatherArgs a{c, k, v};
  using Kern = void (*)(GatherArgs);
  if (in_runs(c, c.heads)) {
    const Kern kern = dtype == 2 ? (c.d == 64 ? (Kern)k_kv4_gather_runs<F16, 64> : (Kern)k_kv4_gather_runs<F16, 128>)
                                 : (c.d == 64 ? (Kern)k_kv4_gather_runs<BF16, 64> : (Kern)k_kv4_gather_runs<BF16, 128>);
    kern<<<grid_for_runs(c, c.heads, kGatherCtas, dev), kCacheThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const int per = c.d == 64 ? 2 : 1;
  const int grid = grid_for(c.tokens * ((c.heads + per - 1) / per), dev);
  const Kern kern = dtype == 2 ? (c.d == 64 ? (Kern)k_kv4_gather<F16, 64> : (Kern)k_kv4_gather<F16, 128>)
                               : (c.d == 64 ? (Kern)k_kv4_gather<BF16, 64> : (Kern)k_kv4_gather<BF16, 128>);
  kern<<<grid, kCacheThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace rwo
