// kernel_kv4_attention.cu -- attention of a few query tokens per sequence over the 4-bit paged cache.
//
// For every query row (one head of one token) o = sum_j p_j v_j / l with p_j = 2^(c q.k_j - m), l = sum p_j, over the keys
// j that the token sees, k_j = s c + z and v_j = s c + z per group of 32 elements; LSE = m ln 2 + ln l.
//
// What bounds it: the cache is read once (1.25 d bytes a token and head), every query head of a key/value head shares
// the read, so HBM bandwidth is the floor; the work per byte (two products, 4-bit codes) has to stay below it.  Measured:
// one token each, d = 128: 2 x 262144 keys with 8 query heads a key/value head 108 us (floor 99), 64 x 9000 keys on average
// with 4 121 (110): 0.90-0.92 of the copy rate.  With more work a byte latency bounds it: d = 64 with 8 rows a head 73 us (64
// sequences, floor 55); 16 sequences of 8191 keys and 4 drafted tokens, 32 rows: d = 64 60 us, floor 12, d = 128 89, floor 25.
// There (ncu, 8 of the 16, d = 64) instructions issue in 44% of the cycles and the matrix pipe is 29% busy: 12 consumer warps an
// SM, each with one chain of product, scales, exponent, conversion and product, and 120 to 148 bytes of registers spilled
// by tiles of 16 rows.
//
// * The products take codes, not values.  A code at bit 0 or 4 of a half word is the fp16 subnormal c 2^-24 or c 2^-20
//   (exact), so A operands are made with one AND each, and the powers of two go into the other operand or the
//   end: S = sum_g s_g (sum_{e in g} q_e c_e) + sum_g z_g (sum_{e in g} q_e).  q is scaled by a power of two per row into
//   fp16's range and then exact there (bf16 has 8 significant bits); the second sum is one product of the zeros with the
//   group sums of q, split into two fp16 parts, so that scores have fp32 accuracy.
// * S^T = K Q^T (m16n8k16: 16 keys by 8 query rows) and O^T = V^T P^T: with the keys as M a tile of 8 query rows wastes
//   nothing, as it would with queries as M = 16.  P changes from accumulator to operand layout with movmatrix.
// * Per group, P is multiplied by the values' scales (8 packed multiplications per 16 keys) instead of 512 values per
//   16 keys being multiplied by them; the zeros are one more product, with P alone.  A row of ones beside the zeros gives
//   the sum of the rounded weights, by which the result is divided, so that what rounding does to all weights alike
//   cancels; l, for the LSE, sums the weights before rounding, in fp32.
// * A weight is p = 2^(score + mb), fp16 for the product: mb puts the running maximum at 2^(9 - e) and moves only when a
//   score exceeds it by 2^6, or a scale of V exceeds 2^e (e = 0 at first, so V up to 15 in magnitude), so that p s stays
//   below 2^15.  One vote per 32 or 64 keys replaces a maximum over lanes; then each row moves by its own keys.  fp16's
//   rounding is 2^-11 of a weight (bf16 would be 2^-8); weights down to 2^-(33 - e) of the largest still count.
// * A CTA is 4 consumer warps and a producer warp, which keeps a ring of stages (cp.async.bulk of one to four blocks per
//   consumer warp) ahead of them.  The tiles of all sequences and heads form one list, cut into equal runs, one per
//   resident CTA: long and short sequences mix without imbalance (an item's own start and end count as two tiles).  A
//   run that ends inside a (sequence, head) leaves its state (m, l, O) in the workspace; a second kernel merges such
//   states in the order of the runs.
// Every wait is bounded; a wait that runs out sets the status word.
#include <atomic>

#include "kv4.cuh"

namespace rwo {
namespace {

constexpr int kWarps = 4;                     // consumer warps (the scan and the merges below are written for four)
constexpr int kThreads = (kWarps + 1) * 32;
constexpr float kBase = 9.f, kSlack = 6.f;    // log2 of the maximum's weight, and by how much a score may exceed it
constexpr float kUnseen = 1e30f;              // mb of a row that has seen no key

struct AttnArgs {
  Kv4View c;
  Kv4Rows q;
  unsigned char* o;  // [tokens][q_heads][d]
  float* lse;        // [tokens][q_heads] or null
  int q_heads, group;
  float scale;
  int64_t* prefix;   // [batch + 1]: first place of each sequence in the list (workspace)
  float4* part_l;    // [2 grid][rows]: mb, l, sum of the rounded weights
  float* part_o;     // [2 grid][rows][d]
  int runs;          // CTAs of the main kernel
  int lead;          // places before an item's tiles in the list
  uint64_t wait_ns;
};

// D = A B + C, 16 x 8 x 16 and 16 x 8 x 8, fp16 in, fp32 out.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma8_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %7, %7, %7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
// An 8 x 8 matrix of 16-bit elements: lane (g, t) gives row g, columns 2 t and 2 t + 1 and gets column g, rows 2 t, 2 t + 1.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// a b + c, rounded once.
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Two fp32 operations an instruction, on neighbours of an accumulator: what does not go through the matrix pipe is short of
// issue slots (16 rows a head, d = 128: 214 -> 211 us; one token, 8 rows: 126.4 -> 124.6).
__device__ __forceinline__ void fma2(float& x0, float& x1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\tfma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float& x0, float& x1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(float& x0, float& x1, float a0, float a1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a0), "f"(a1));
}

// n consecutive 32-bit words.
template <int n>
__device__ __forceinline__ void words_at(uint32_t (&w)[n], const unsigned char* p) {
  if constexpr (n == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (n == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ uint32_t word_at(const unsigned char* p) { return *reinterpret_cast<const uint32_t*>(p); }

// Tiles of a sequence in the list: every head and block of query rows takes all of its keys.
struct SeqWork {
  Kv4Seq s;
  int row_blocks, tiles;
};
template <int R, int KEYS>
__device__ __forceinline__ SeqWork seq_work(const Kv4View& c, int b, int group, bool& bad) {
  SeqWork w;
  w.s = kv4_seq(c, b, bad);
  w.row_blocks = (w.s.n * group + R - 1) / R;
  w.tiles = int((unsigned(w.s.len) + KEYS - 1) / KEYS);
  if (w.tiles < 1) w.tiles = 1;
  return w;
}
// The list has `lead` places before each (sequence, head, block of rows)'s tiles, for the time that its start and its end take
// (queries, merge): runs of equal length then take equal time.
__device__ __forceinline__ int64_t seq_places(const SeqWork& w, int heads, int lead) { return int64_t(heads) * w.row_blocks * (w.tiles + lead); }

// The list of W places is cut into `n` runs: run i is [first(i), first(i + 1)).
struct Runs {
  int64_t W;
  int n;
  __device__ __forceinline__ int64_t first(int i) const { return W * i / n; }
  __device__ __forceinline__ int of(int64_t place) const { return int(((place + 1) * n - 1) / W); }
};
__device__ __forceinline__ Runs runs_of(int64_t W, int runs) { return Runs{W, int(W < 1 ? 1 : W < runs ? W : runs)}; }

// A place in the list: one (sequence, head, block of rows) and a range of its tiles.
struct Cursor {
  int b, h, rb, tile;
  SeqWork w;
};
// To the next (sequence, head, block of rows).
template <int R, int KEYS>
__device__ __forceinline__ void next_item(Cursor& k, const Kv4View& c, int group) {
  k.tile = 0;
  if (++k.rb < k.w.row_blocks) return;
  k.rb = 0;
  if (++k.h < c.heads) return;
  k.h = 0;
  bool bad = false;
  do {
    if (++k.b >= c.batch) return;
    k.w = seq_work<R, KEYS>(c, k.b, group, bad);
  } while (k.w.row_blocks == 0);
}

template <int DH, int NT, int KB>
struct Smem {
  using B = Kv4Block<DH>;
  static constexpr int kStages = DH == 64 ? 3 : 2;
  static constexpr int kCtas = NT == 2 ? (DH == 64 ? 3 : 2) : 3;  // resident on an SM: bounds the registers
  static constexpr int kBlocks = kWarps * KB;            // of a stage
  static constexpr int kKeys = kBlocks * kKv4Block;
  static constexpr int R = 8 * NT;                       // query rows of a tile
  static constexpr int kStage = kBlocks * B::kBytes;
  static constexpr int kPad = DH + 8;
  static constexpr int kOffQ = kStages * kStage;         // fragments: [NT][2 G][32 lanes][2 words]
  static constexpr int kOffQz = kOffQ + NT * 2 * B::G * 256;   // [NT][32 lanes] words
  static constexpr int kOffRow = kOffQz + NT * 128;      // [R] score factors
  static constexpr int kOffMl = kOffRow + R * 4;         // [4 warps][R] x 3
  static constexpr int kOffO = kOffMl + kWarps * R * 16;  // [4 warps][8 rows][kPad]
  static constexpr int kOffBar = kOffO + kWarps * 8 * kPad * 4;
  static constexpr int kOffScan = kOffBar + 2 * kStages * 8;  // [4 warps] + start
  static constexpr int kBytes = kOffScan + 64;
};

template <bool H>
__device__ __forceinline__ float elem_to_f32(uint32_t w, int half) {
  if constexpr (H) return half ? f16_hi(w) : f16_lo(w);
  else return half ? bf16_hi(w) : bf16_lo(w);
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

// One finished row: O over the sum of its weights in the element type, LSE = ln l - mb ln 2.  A row that saw no key gives
// 0 and -inf.  s: mb, l, sum of the rounded weights.
template <bool H, int DH>
__device__ __forceinline__ void write_row(const AttnArgs& a, int64_t out, int lane, const float (&x)[DH / 32], float4 s) {
  constexpr int E = DH / 32;
  const float inv = safe_inv(s.z);
  uint32_t w[E / 2];
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float lo = __fmul_rn(x[e], inv), hi = __fmul_rn(x[e + 1], inv);
    w[e / 2] = H ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
  }
  unsigned char* o = a.o + out * DH * 2 + lane * E * 2;
  if constexpr (E == 4) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(o) = w[0];
  if (lane == 0 && a.lse) a.lse[out] = s.y > 0.f ? __fmaf_rn(s.x, -0.6931471805599453f, logf(s.y)) : -INFINITY;
}

// H: fp16 elements (else bf16); DH: head dimension; NT: tiles of 8 query rows; KB: blocks of 16 keys a warp takes at once.
template <bool H, int DH, int NT, int KB>
__global__ void __launch_bounds__(kThreads, Smem<DH, NT, KB>::kCtas) k_attention_kv4(AttnArgs a) {
  using B = Kv4Block<DH>;
  using SM = Smem<DH, NT, KB>;
  constexpr int G = B::G, R = SM::R, kKeys = SM::kKeys, kStages = SM::kStages;
  constexpr bool kQInSmem = NT * DH > 128;  // Q's fragments are read again for every stage: their 32 registers are short
  extern __shared__ __align__(128) unsigned char smem[];
  const Kv4View& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_addr(smem);
  auto full = [&](int s) { return sbase + uint32_t(SM::kOffBar + s * 8); };
  auto empty = [&](int s) { return sbase + uint32_t(SM::kOffBar + (kStages + s) * 8); };

  // ---- where this CTA's run starts: a scan over the sequences ----
  int64_t* scan = reinterpret_cast<int64_t*>(smem + SM::kOffScan);   // [4]
  int* start = reinterpret_cast<int*>(smem + SM::kOffScan + 32);     // b, h, rb, tile
  const int per = (c.batch + 127) / 128, b0 = tid < 128 ? min(tid * per, c.batch) : c.batch, b1 = tid < 128 ? min(b0 + per, c.batch) : c.batch;
  bool bad = false;
  int64_t mine = 0;
  bool down = false;
  for (int b = b0; b < b1; ++b) {
    const SeqWork w = seq_work<R, kKeys>(c, b, a.group, bad);
    mine += seq_places(w, c.heads, a.lead);
    down |= w.s.down;
  }
  // Where offsets descend, sequences claim the same rows, up to batch times the work of the call: more places than a call has
  // are taken off, the sum is negative, and no row is worked on.
  if (down) mine = -(int64_t(1) << 55);
  if (bad && blockIdx.x == 0) kv4_bad(c);
  int64_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(kFull, before, o);
    if (lane >= o) before += x;
  }
  if (warp < 4 && lane == 31) scan[warp] = before;
  if (tid == 128) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  before -= mine;
  for (int w = 0; w < 4 && w < warp; ++w) before += scan[w];
  const int64_t W = scan[0] + scan[1] + scan[2] + scan[3];
  if (blockIdx.x == 0) {  // for the merging kernel
    int64_t p = before;
    for (int b = b0; b < b1; ++b) {
      a.prefix[b] = p;
      p += seq_places(seq_work<R, kKeys>(c, b, a.group, bad), c.heads, a.lead);
    }
    if (tid == 0) a.prefix[c.batch] = W;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Runs runs = runs_of(W, a.runs);
  if (W <= 0 || int(blockIdx.x) >= runs.n) return;
  const int64_t run0 = runs.first(blockIdx.x), run1 = runs.first(blockIdx.x + 1);
  if (tid < 128 && run0 >= before && run0 < before + mine) {
    int64_t p = before;
    for (int b = b0; b < b1; ++b) {
      const SeqWork w = seq_work<R, kKeys>(c, b, a.group, bad);
      const int64_t n = seq_places(w, c.heads, a.lead);
      if (run0 < p + n) {
        const int64_t x = run0 - p, item = x / (w.tiles + a.lead);
        start[0] = b;
        start[1] = int(item / w.row_blocks);
        start[2] = int(item % w.row_blocks);
        start[3] = int(x - item * (w.tiles + a.lead)) - a.lead;
        break;
      }
      p += n;
    }
  }
  __syncthreads();
  Cursor at;
  at.b = start[0];
  at.h = start[1];
  at.rb = start[2];
  at.tile = max(start[3], 0);
  at.w = seq_work<R, kKeys>(c, at.b, a.group, bad);
  int64_t left = run1 - run0 + min(start[3], 0);  // of the run: tiles of this item, and the places behind it
  if (left <= 0) return;
  bool timed_out = false;

  if (warp == kWarps) {
    // ---- producer: a copy for each run of blocks that lie together in a page, by the lane of the run's first block; the
    // next stage's pages are looked up while a slot is waited for ----
    const uint64_t policy = policy_evict_first();
    uint32_t bytes = 0;                   // of this lane's next copy
    auto block_of = [&]() -> int64_t {    // and where it starts; -1: this lane has none
      const int blk = at.tile * SM::kBlocks + lane, in_page = blk % c.page_blocks;
      const int n = min(min(SM::kBlocks - lane, (at.w.s.len + kKv4Block - 1) / kKv4Block - blk), c.page_blocks - in_page);
      if (n <= 0 || (lane && in_page)) return -1;
      bytes = uint32_t(n * B::kBytes);
      int64_t off = kv4_block_at(c, at.b, blk * kKv4Block, B::kBytes);
      if (off < 0) {  // no page: the status says so, and page 0 stands in
        kv4_bad(c);
        off = int64_t(in_page) * B::kBytes;
      }
      return off + int64_t(at.h) * c.page_blocks * B::kBytes;
    };
    int slot = 0;
    uint32_t lap = 0;
    int64_t issued = 0, off = block_of();
    while (left > 0) {
      const int64_t now = off;
      const uint32_t size = now >= 0 ? bytes : 0u;
      // whole blocks of the tile that hold a key
      const int blocks = max(0, min(SM::kBlocks, (at.w.s.len + kKv4Block - 1) / kKv4Block - at.tile * SM::kBlocks));
      if (--left > 0) {
        if (++at.tile == at.w.tiles && (left -= a.lead) > 0) next_item<R, kKeys>(at, c, a.group);
        if (left > 0) off = block_of();
      }
      if (issued >= kStages && !mbar_wait(empty(slot), lap ^ 1u, a.wait_ns)) timed_out = true;
      if (lane == 0) {
        if (blocks) mbar_arrive_expect_tx(full(slot), uint32_t(blocks * B::kBytes));
        else mbar_arrive(full(slot));
      }
      __syncwarp();
      if (size) bulk_g2s(sbase + uint32_t(slot * SM::kStage + lane * B::kBytes), c.data + now, size, full(slot), policy);
      ++issued;
      if (++slot == kStages) {
        slot = 0;
        lap ^= 1u;
      }
    }
    // no copy may be in flight into this CTA when it exits: the last phase of every stage
    for (int s = 0; s < kStages && s < issued; ++s) {
      const int64_t uses = (issued - 1 - s) / kStages;
      if (!mbar_wait(full(s), uint32_t(uses & 1), a.wait_ns)) timed_out = true;
    }
    if (timed_out && lane == 0) atomicOr(c.status, kStatusTimeout);
    return;
  }

  // ---- consumers ----
  const int g = lane >> 2, t = lane & 3;
  int slot = 0;
  uint32_t lap = 0;
  bool first = true;
  constexpr int E = DH / 32;  // elements of a row a lane, E lane .. E lane + E - 1
  while (left > 0) {
    const int here = int(left < at.w.tiles - at.tile ? left : at.w.tiles - at.tile);
    const int n = at.w.s.n, len = at.w.s.len, row0 = at.rb * R;
    // Q rows of the item as operand fragments; row r is head h G + r % G of token r / G
    // (A warp's rows are loaded at once: 16 rows a head 210 -> 206 us, d = 64 82 -> 79; at d = 128 with 8 rows one by one,
    // where more registers cost the loop over the keys 1%.)
    constexpr int kOnce = NT == 1 && DH == 128 ? 1 : R / kWarps;
#pragma unroll 1
    for (int r0 = warp; r0 < R; r0 += kOnce * kWarps) {
      uint32_t rows[kOnce][E / 2];
#pragma unroll
      for (int k = 0; k < kOnce; ++k) {
        const int rr = row0 + r0 + k * kWarps, tok = rr / a.group, hd = at.h * a.group + rr - tok * a.group;
        const unsigned char* p = static_cast<const unsigned char*>(a.q.p) + (int64_t(at.w.s.start + tok) * a.q.token + int64_t(hd) * a.q.head) * 2;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) rows[k][e] = tok < n ? __ldg(reinterpret_cast<const uint32_t*>(p) + lane * (E / 2) + e) : 0u;
      }
#pragma unroll
      for (int k = 0; k < kOnce; ++k) {
        const int r = r0 + k * kWarps;
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = elem_to_f32<H>(rows[k][e / 2], e & 1);
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) mx = fmaxf(mx, fabsf(x[i]));
        // the row's power of two: the largest element lands in [2^5, 2^6)
        const uint32_t top = __reduce_max_sync(kFull, __float_as_uint(mx));
        int ex = int(top >> 23) - 127;
        ex = ex < -122 ? -122 : ex;
        const float to = pow2(5 - ex);
        // (neither 0 nor infinite, so that -inf, where a key is hidden, stays -inf, and 0, where q is, 0)
        const float factor = a.scale * pow2(ex) * (kLog2e * 0x1p19f);
        if (lane == 0) reinterpret_cast<float*>(smem + SM::kOffRow)[r] = fminf(fmaxf(factor, 0x1p-126f), 0x1.fffffep127f);
        float sum = 0.f;
        __half* qf = reinterpret_cast<__half*>(smem + SM::kOffQ);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int e = lane * E + i, j = e >> 5, w = e & 31, tt = w >> 3, nn = w & 7;
          const __half hv = __float2half_rn(x[i] * to * ((nn & 1) ? 0.0625f : 1.f));
          qf[(((((r >> 3) * 2 * G + 2 * j + ((nn & 3) >> 1)) * 32 + (r & 7) * 4 + tt) * 2 + (nn & 1)) * 2) + (nn >> 2)] = hv;
          sum += __half2float(hv) * ((nn & 1) ? 16.f : 1.f);
        }
#pragma unroll
        for (int o = 1; o < 32 / G; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (lane % (32 / G) == 0) {
          const int j = lane / (32 / G);
          const __half hi = __float2half_rn(sum), lo = __float2half_rn(sum - __half2float(hi));
          __half* qz = reinterpret_cast<__half*>(smem + SM::kOffQz) + ((r >> 3) * 32 + (r & 7) * 4) * 2;
          qz[j] = hi;
          qz[G + j] = lo;
          if (G == 2) qz[4 + j] = qz[6 + j] = __ushort_as_half(0);
        }
      }
    }
    named_barrier_sync(1, kWarps * 32);
    uint32_t qf[NT][2 * G][2], qz[NT];
    auto load_q = [&] {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int s = 0; s < 2 * G; ++s) words_at<2>(qf[i][s], smem + SM::kOffQ + ((i * 2 * G + s) * 32 + lane) * 8);
    };
    if (!kQInSmem) load_q();
    float ch[NT][2], mb[NT][2], l[NT][2], O[NT][2 * G][4], Z[NT][4];
    int seen[NT][2];  // keys that the row of column 2 t, 2 t + 1 sees
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int s = 0; s < 2 * G; ++s) {
#pragma unroll
        for (int k = 0; k < 4; ++k) O[i][s][k] = 0.f;
      }
      qz[i] = word_at(smem + SM::kOffQz + (i * 32 + lane) * 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) Z[i][k] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = i * 8 + 2 * t + k;
        ch[i][k] = reinterpret_cast<const float*>(smem + SM::kOffRow)[r];
        mb[i][k] = kUnseen;
        l[i][k] = 0.f;
        const int tok = (row0 + r) / a.group;
        seen[i][k] = tok < n ? len - n + tok + 1 : 0;
      }
    }
    const int all_see = len - n + row0 / a.group + 1;  // keys that every row sees
    int es = 0;                                        // V's scales have been at most 2^es
    float most = kBase + kSlack;                       // weights stay at or below 2^most, most = base + slack - es
    uint32_t over = 0x7fff7fffu - 0x3c003c00u;         // added to two scales' bits, sets bit 15 of one above 2^es

    for (int k = 0; k < here; ++k) {
      if (!mbar_wait(full(slot), lap, a.wait_ns)) timed_out = true;
      const int key0 = (at.tile + k) * kKeys + warp * KB * kKv4Block;
      if (key0 < len) {
        const unsigned char* blk0 = smem + slot * SM::kStage + warp * KB * B::kBytes;
        // S^T = K Q^T
        if (kQInSmem) load_q();
        float S[KB][NT][4];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const unsigned char* blk = blk0 + kb * B::kBytes;
          uint32_t wa[G], wb[G], ksa[G / 2], ksb[G / 2];
          words_at<G>(wa, blk + g * (DH / 2) + t * G * 4);
          words_at<G>(wb, blk + (g + 8) * (DH / 2) + t * G * 4);
          words_at<G / 2>(ksa, blk + B::kKScale + g * G * 2);
          words_at<G / 2>(ksb, blk + B::kKScale + (g + 8) * G * 2);
          const uint32_t kza = word_at(blk + B::kKZero + g * G * 2 + (t % (G / 2)) * 4);
          const uint32_t kzb = word_at(blk + B::kKZero + (g + 8) * G * 2 + (t % (G / 2)) * 4);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            float z[4];
            mma8_first(z, kza, kzb, qz[i]);
#pragma unroll
            for (int q = 0; q < 4; q += 2) mul2(S[kb][i][q], S[kb][i][q + 1], z[q], z[q + 1], 0x1p-24f, 0x1p-24f);
          }
#pragma unroll
          for (int j = 0; j < G; ++j) {
            const uint32_t ua = wa[j] >> 8, ub = wb[j] >> 8;
            const float sa = (j & 1) ? f16_hi(ksa[j / 2]) : f16_lo(ksa[j / 2]), sb = (j & 1) ? f16_hi(ksb[j / 2]) : f16_lo(ksb[j / 2]);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              float d[4];
              mma16_first(d, wa[j] & 0x000f000fu, wb[j] & 0x000f000fu, wa[j] & 0x00f000f0u, wb[j] & 0x00f000f0u, qf[i][2 * j][0], qf[i][2 * j][1]);
              mma16(d, ua & 0x000f000fu, ub & 0x000f000fu, ua & 0x00f000f0u, ub & 0x00f000f0u, qf[i][2 * j + 1][0], qf[i][2 * j + 1][1]);
              fma2(S[kb][i][0], S[kb][i][1], sa, sa, d[0], d[1], S[kb][i][0], S[kb][i][1]);
              fma2(S[kb][i][2], S[kb][i][3], sb, sb, d[2], d[3], S[kb][i][2], S[kb][i][3]);
            }
          }
        }
        const bool tail = key0 + KB * kKv4Block > all_see;  // some row does not see all of these keys
        if (tail) {
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (key0 + kb * kKv4Block + g + (q & 2) * 4 >= seen[i][q & 1]) S[kb][i][q] = -INFINITY;
        }
        // a vote: is a weight, or a scale of V, above its bound?  (lane (g, t) looks at the scales of one word, of a slot
        // that holds no token too: a vote for those alone moves nothing)
        bool move = false;
        float p[KB][NT][4], ptop = -INFINITY;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const int f = (g / G) & 1, j = g % G;
          move |= ((word_at(blk0 + kb * B::kBytes + B::kVScale + ((4 * f + t) * G + j) * 4) + over) & 0x80008000u) != 0u;
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
              fma2(p[kb][i][q], p[kb][i][q + 1], S[kb][i][q], S[kb][i][q + 1], ch[i][0], ch[i][1], mb[i][0], mb[i][1]);
              ptop = fmaxf(ptop, fmaxf(p[kb][i][q], p[kb][i][q + 1]));
            }
        }
        if (__any_sync(kFull, move || ptop > most)) {  // a new maximum, or larger scales: rescale what is summed so far
          // Each row moves by what it sees itself, so that its bits are the same whatever later tokens, other rows and slots that
          // hold no token hold.  (A row that does not see the last of these keys sees none after them: es need not be its own.)
          // Rows that share their moves make fewer (4 drafted tokens a sequence, d = 128: 88 us against 89).
          int er[NT][2], e = es;
#pragma unroll
          for (int i = 0; i < NT; ++i) er[i][0] = er[i][1] = es;
          if (__any_sync(kFull, move)) {
            float vs[KB][2];  // largest scales of tokens g and g + 8
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t w[G];
                words_at<G>(w, blk0 + kb * B::kBytes + B::kVScale + (g / 2 + 4 * h) * G * 4);
#pragma unroll
                for (int j = 1; j < G; ++j) w[0] = hmax2(w[0], w[j]);
                vs[kb][h] = (g & 1) ? f16_hi(w[0]) : f16_lo(w[0]);
              }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float top = 0.f;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                  for (int h = 0; h < 2; ++h) top = fmaxf(top, S[kb][i][q + 2 * h] == -INFINITY ? 0.f : vs[kb][h]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
                const int x = int((__float_as_uint(top) + 0x7fffffu) >> 23) - 127;  // the smallest power of two not below
                er[i][q] = x < es ? es : x > 16 ? 16 : x;
                e = e < er[i][q] ? er[i][q] : e;
              }
            e = __reduce_max_sync(kFull, e);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            float al[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float mx = fmaxf(S[0][i][q], S[0][i][q + 2]);
#pragma unroll
              for (int kb = 1; kb < KB; ++kb) mx = fmaxf(mx, fmaxf(S[kb][i][q], S[kb][i][q + 2]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
              const float to = fmaf(mx, ch[i][q], mb[i][q]) > most ? kBase - float(er[i][q]) - mx * ch[i][q] : mb[i][q] - float(er[i][q] - es);
              al[q] = ex2(to - mb[i][q]);
              mb[i][q] = to;
              l[i][q] *= al[q];
              Z[i][q] *= al[q];
            }
#pragma unroll
            for (int s = 0; s < 2 * G; ++s)
#pragma unroll
              for (int q = 0; q < 4; ++q) O[i][s][q] *= al[q & 1];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int q = 0; q < 4; ++q) p[kb][i][q] = fmaf(S[kb][i][q], ch[i][q & 1], mb[i][q & 1]);
          }
          es = e;
          most = kBase + kSlack - float(e);
          over = 0x7fff7fffu - 0x3c003c00u - uint32_t(e) * 0x04000400u;
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const unsigned char* blk = blk0 + kb * B::kBytes;
          uint32_t pb[NT][2];
#pragma unroll
          for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q) p[kb][i][q] = ex2(p[kb][i][q]);
            add2(l[i][0], l[i][1], p[kb][i][0], p[kb][i][1]);
            add2(l[i][0], l[i][1], p[kb][i][2], p[kb][i][3]);
            pb[i][0] = transposed(pack_f16x2(p[kb][i][0], p[kb][i][1]));
            pb[i][1] = transposed(pack_f16x2(p[kb][i][2], p[kb][i][3]));
          }
          // O^T += V^T P^T; Z^T: rows g < G for the zeros, row G for ones
          uint32_t vs[2][G], vz[2], va[G], vb[G];
          words_at<G>(va, blk + B::kV + (g * 4 + t) * G * 4);
          words_at<G>(vb, blk + B::kV + ((8 + g) * 4 + t) * G * 4);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            words_at<G>(vs[f], blk + B::kVScale + (4 * f + t) * G * 4);
            vz[f] = word_at(blk + B::kVZero + ((4 * f + t) * G + g % G) * 4);
            if (g >= G) vz[f] = g == G ? 0x3c003c00u : 0u;
          }
          uint32_t takes[NT];  // halves whose second token has a weight
#pragma unroll
          for (int i = 0; i < NT; ++i) takes[i] = kFull;
          if (H && tail) {  // (0 times the code of an unseen token is 0: a remainder times it would not be)
#pragma unroll
            for (int i = 0; i < NT; ++i) takes[i] = (pb[i][1] & 0xffffu ? 0xffffu : 0u) | (pb[i][1] >> 16 ? 0xffff0000u : 0u);
          }
          if (tail) {  // a slot that holds no token counts with zero
            const int live = len - key0 - kb * kKv4Block;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const uint32_t keep = (8 * f + 2 * t < live ? 0xffffu : 0u) | (8 * f + 2 * t + 1 < live ? 0xffff0000u : 0u);
              vz[f] &= keep;
#pragma unroll
              for (int j = 0; j < G; ++j) vs[f][j] &= keep;
            }
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) mma16(Z[i], vz[0], 0u, vz[1], 0u, pb[i][0], pb[i][1]);
#pragma unroll
          for (int j = 0; j < G; ++j) {
            const uint32_t ua = va[j] >> 8, ub = vb[j] >> 8;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const uint32_t p0 = hmul2(pb[i][0], vs[0][j]);
              // fp16 results show these roundings: what one loses, the next takes up, if the row sees its token
              const uint32_t p1 = H ? hfma2(pb[i][1], vs[1][j], hfma2(pb[i][0] & takes[i], vs[0][j], (p0 ^ 0x80008000u) & takes[i]))
                                    : hmul2(pb[i][1], vs[1][j]);
              mma16(O[i][2 * j], va[j] & 0x000f000fu, va[j] & 0x00f000f0u, vb[j] & 0x000f000fu, vb[j] & 0x00f000f0u, p0, p1);
              mma16(O[i][2 * j + 1], ua & 0x000f000fu, ua & 0x00f000f0u, ub & 0x000f000fu, ub & 0x00f000f0u, p0, p1);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(slot));
      if (++slot == kStages) {
        slot = 0;
        lap ^= 1u;
      }
    }

    // ---- the four warps' states merged, then written: the rows themselves, or a part of them ----
    const bool whole = at.tile == 0 && here == at.w.tiles;
    const int part = 2 * int(blockIdx.x) + (first ? 0 : 1);
    float4* ml = reinterpret_cast<float4*>(smem + SM::kOffMl);
    float* ob = reinterpret_cast<float*>(smem + SM::kOffO);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[i][q] += __shfl_xor_sync(kFull, l[i][q], o);
        const float ones = __shfl_sync(kFull, Z[i][q], G * 4 + t);
        if (g == 0) ml[warp * R + i * 8 + 2 * t + q] = make_float4(mb[i][q], l[i][q], ones, 0.f);
      }
      if (i > 0) named_barrier_sync(1, kWarps * 32);  // the buffer has been read
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const float z0 = __shfl_sync(kFull, Z[i][0], j * 4 + t), z1 = __shfl_sync(kFull, Z[i][1], j * 4 + t);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float (&o)[4] = O[i][2 * j + h];
          float* d0 = ob + (warp * 8 + 2 * t) * SM::kPad + 32 * j + 4 * g + 2 * h;
          *reinterpret_cast<float2*>(d0) = make_float2(fmaf(o[0], 0x1p24f, z0), fmaf(o[2], 0x1p20f, z0));
          *reinterpret_cast<float2*>(d0 + SM::kPad) = make_float2(fmaf(o[1], 0x1p24f, z1), fmaf(o[3], 0x1p20f, z1));
        }
      }
      named_barrier_sync(1, kWarps * 32);
      // warp w: rows w, w + 4 of the tile
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int r = warp + 4 * rr, row = row0 + i * 8 + r;
        float4 s[kWarps], sum = make_float4(kUnseen, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          s[w] = ml[w * R + i * 8 + r];
          sum.x = fminf(sum.x, s[w].x);
        }
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float fix = ex2(sum.x - s[w].x);
          sum.y = fmaf(fix, s[w].y, sum.y);
          sum.z = fmaf(fix, s[w].z, sum.z);
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = fmaf(fix, ob[(w * 8 + r) * SM::kPad + lane * E + e], x[e]);
        }
        if (row < n * a.group) {
          if (whole) {
            const int tok = row / a.group, hd = at.h * a.group + row - tok * a.group;
            write_row<H, DH>(a, int64_t(at.w.s.start + tok) * a.q_heads + hd, lane, x, sum);
          } else {
            float* po = a.part_o + (int64_t(part) * R + i * 8 + r) * DH + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) po[e] = x[e];
            if (lane == 0) a.part_l[int64_t(part) * R + i * 8 + r] = sum;
          }
        }
      }
    }
    first = false;
    left -= here;
    if (left > 0) left -= a.lead;
    if (left > 0) next_item<R, kKeys>(at, c, a.group);
    named_barrier_sync(1, kWarps * 32);  // Q and the merge buffers are free
  }
  if (timed_out && lane == 0) atomicOr(c.status, kStatusTimeout);
}

// Merges the parts of rows whose keys were spread over several runs, in the order of the runs: eight warps a row, a CTA each,
// where rows are few and their parts many (one sequence of 16384 keys, 57 parts a row: 15.2 us with four warps, 13.8 with
// eight; sixteen 13.3, but short sequences lose 0.4), else one, four rows a CTA.
constexpr int kMergeWarps = 8;
constexpr int kMergeAhead = 4;  // parts that a warp loads at once
template <bool H, int DH, int NT, int KB>
__global__ void __launch_bounds__(kMergeWarps * 32) k_attention_kv4_merge(AttnArgs a, int split) {
  constexpr int E = DH / 32, R = 8 * NT, kKeys = Smem<DH, NT, KB>::kKeys;
  const Kv4View& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t x = split > 1 ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 4 + warp, i = x / a.q_heads;
  const int hq = int(x - i * a.q_heads), share = split > 1 ? warp : 0;
  // what the main kernel does not write is read before it is waited for
  const int b = i < c.tokens ? kv4_seq_of(c, i) : -1;
  bool bad = false;
  SeqWork w;
  w.s.n = 0;
  if (b >= 0) w = seq_work<R, kKeys>(c, b, a.group, bad);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (b < 0 || i < w.s.start || i >= w.s.start + w.s.n) return;
  const int64_t W = a.prefix[c.batch], p0 = a.prefix[b];
  if (W <= 0) return;
  const int h = hq / a.group, rr = int(i - w.s.start) * a.group + hq - h * a.group, rb = rr / R, r = rr - rb * R;
  const Runs runs = runs_of(W, a.runs);
  const int64_t t0 = p0 + (int64_t(h) * w.row_blocks + rb) * (w.tiles + a.lead);
  const int c0 = runs.of(t0 + a.lead), c1 = runs.of(t0 + a.lead + w.tiles - 1);
  if (c0 == c1) return;  // one run held all of its keys and wrote the row
  const int late = t0 > runs.first(c0) ? 1 : 0;  // the part in run c0 is not that run's first
  float4 s = make_float4(kUnseen, 0.f, 0.f, 0.f);
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int k0 = c0 + share; k0 <= c1; k0 += kMergeAhead * split) {
    float4 v[kMergeAhead];
    float x[kMergeAhead][E];
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k) {  // absent parts weigh nothing
      const int run = k0 + k * split;
      const int64_t part = int64_t(2 * run + (run == c0 ? late : 0)) * R + r;
      v[k] = make_float4(kUnseen, 0.f, 0.f, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) x[k][e] = 0.f;
      if (run <= c1) {
        v[k] = a.part_l[part];
#pragma unroll
        for (int e = 0; e < E; ++e) x[k][e] = a.part_o[part * DH + lane * E + e];
      }
    }
    float mb = s.x;
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k) mb = fminf(mb, v[k].x);
    const float old = ex2(mb - s.x);
    s = make_float4(mb, s.y * old, s.z * old, 0.f);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= old;
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k) {
      const float fix = ex2(mb - v[k].x);
      s.y = fmaf(fix, v[k].y, s.y);
      s.z = fmaf(fix, v[k].z, s.z);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(fix, x[k][e], o[e]);
    }
  }
  if (split > 1) {
    __shared__ float4 sm[kMergeWarps];
    __shared__ float so[kMergeWarps][DH];
    if (lane == 0) sm[warp] = s;
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    __syncthreads();
    if (warp) return;
    float mb = kUnseen;
    for (int k = 0; k < split; ++k) mb = fminf(mb, sm[k].x);
    s = make_float4(mb, 0.f, 0.f, 0.f);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int k = 0; k < split; ++k) {
      const float fix = ex2(mb - sm[k].x);
      s.y = fmaf(fix, sm[k].y, s.y);
      s.z = fmaf(fix, sm[k].z, s.z);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(fix, so[k][lane * E + e], o[e]);
    }
  }
  write_row<H, DH>(a, i * a.q_heads + hq, lane, o, s);
}

struct Plan {
  void (*main)(AttnArgs);
  void (*merge)(AttnArgs, int);
  int smem, rows;
};
template <bool H, int DH, int NT, int KB>
Plan plan_as() {
  return Plan{k_attention_kv4<H, DH, NT, KB>, k_attention_kv4_merge<H, DH, NT, KB>, Smem<DH, NT, KB>::kBytes, 8 * NT};
}
template <bool H, int DH>
Plan plan_of(bool wide) {
  return wide ? plan_as<H, DH, 2, 2>() : plan_as<H, DH, 1, 256 / DH>();
}
// Tiles of 8 query rows, or of 16 where a sequence has more rows to a key/value head than 8 on average: a tile's rows share
// what a code costs (32 rows a head, d = 64: 62 us with tiles of 16, 83 with 8; d = 128: 91 against 113; tiles of 32 run out
// of registers, 85).  A warp takes 32 keys at once; at d = 64 with 8 rows, 64, in three CTAs an SM (then 82 us against 95 with 32
// keys in four or five).  CTAs without a producer, each warp copying its own blocks, make room for a fourth, which
// is slower: what the registers spill no longer stays in L1 (d = 64, 16 rows: 62 -> 96 us).
Plan plan_for(int64_t batch, int64_t tokens, int q_heads, int heads, int d, int dtype) {
  const bool wide = tokens * (q_heads / heads) > 8 * batch;
  if (d == 64) return dtype == 2 ? plan_of<true, 64>(wide) : plan_of<false, 64>(wide);
  return dtype == 2 ? plan_of<true, 128>(wide) : plan_of<false, 128>(wide);
}

constexpr int kMaxCtasPerSm = 4;

// CTAs of the main kernel that an SM holds: asked once per device and kernel (the answer is the kernel's own).
cudaError_t resident_ctas(const Plan& p, bool d64, bool f16, const DeviceInfo& dev, int* out) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][8];
  std::atomic<int>& slot = known[dev.device % kDevices][(d64 ? 4 : 0) + (f16 ? 2 : 0) + (p.rows == 16 ? 1 : 0)];
  int n = slot.load(std::memory_order_acquire);
  if (n == 0) {
    cudaError_t err = cudaFuncSetAttribute((const void*)p.main, cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem);
    if (err == cudaSuccess) err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, (const void*)p.main, kThreads, size_t(p.smem));
    if (err != cudaSuccess) return err;
    if (n < 1) return cudaErrorInvalidConfiguration;
    if (n > kMaxCtasPerSm) n = kMaxCtasPerSm;
    slot.store(n, std::memory_order_release);
  }
  *out = n;
  return cudaSuccess;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

size_t attention_kv4_scratch(int64_t batch, int64_t tokens, int q_heads, int heads, int d, const DeviceInfo& dev) {
  const Plan p = plan_for(batch, tokens, q_heads, heads, d, 1);
  const size_t parts = size_t(2) * kMaxCtasPerSm * dev.sm_count * p.rows;
  return up256(size_t(batch + 1) * 8) + up256(parts * 16) + parts * size_t(d) * 4;
}

cudaError_t launch_attention_kv4(const Kv4View& c, const Kv4Rows& q, void* o, float* lse, int q_heads, float scale, int dtype,
                                 void* scratch, cudaStream_t stream, const DeviceInfo& dev) {
  const Plan p = plan_for(c.batch, c.tokens, q_heads, c.heads, c.d, dtype);
  int per_sm = 0;
  cudaError_t err = resident_ctas(p, c.d == 64, dtype == 2, dev, &per_sm);
  if (err != cudaSuccess) return err;
  AttnArgs a;
  a.c = c;
  a.q = q;
  a.o = static_cast<unsigned char*>(o);
  a.lse = lse;
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  a.scale = scale;
  a.runs = per_sm * dev.sm_count;
  a.wait_ns = exchange_wait_limit_ns();
  // Two places where a run is likely to hold several (sequence, head, block of rows)s (64 ragged sequences of 8 heads: 126 -> 121 us,
  // d = 64 79 -> 72; 128 of at most 700 keys 29 -> 23; 16 rows a head 203 -> 187, with one place 194); none where it is one or
  // two of a few (one sequence of 16384 keys: 13.8 us, with two 14.4).
  const int64_t items = c.heads * (c.batch > c.tokens * a.group / p.rows ? int64_t(c.batch) : c.tokens * a.group / p.rows);
  a.lead = 2 * items >= a.runs ? 2 : 0;
  unsigned char* w = static_cast<unsigned char*>(scratch);
  const size_t parts = size_t(2) * a.runs * p.rows;
  a.prefix = reinterpret_cast<int64_t*>(w);
  w += up256(size_t(c.batch + 1) * 8);
  a.part_l = reinterpret_cast<float4*>(w);
  w += up256(parts * 16);
  a.part_o = reinterpret_cast<float*>(w);
  p.main<<<a.runs, kThreads, p.smem, stream>>>(a);
  if ((err = cudaGetLastError()) != cudaSuccess) return err;
  // the merge is launched while the last runs finish, and waits for them itself
  cudaLaunchConfig_t cfg = {};
  const int64_t rows = c.tokens * q_heads;
  const int split = rows <= 4 * int64_t(dev.sm_count) ? kMergeWarps : 1;
  cfg.gridDim = dim3(unsigned(split > 1 ? rows : (rows + 3) / 4));
  cfg.blockDim = dim3(split > 1 ? kMergeWarps * 32 : 128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.merge, a, split);
}

}  // namespace rwo
