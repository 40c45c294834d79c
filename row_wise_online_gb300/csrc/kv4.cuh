// kv4.cuh -- layout of the 4-bit paged key/value cache and the device code that its kernels share.
//
// A block holds 16 tokens of one head, 20 d bytes (G = d / 32 groups of 32 elements a token):
//   [0, 8 d)        key codes.    Word r d/8 + G t + j (token r, t < 4): nibble n is element 32 j + 8 t + n.
//   [8 d, 16 d)     value codes.  Word ((8 f + g) 4 + t) G + j (f < 2, g < 8, t < 4): the low half belongs to token
//                   8 f + 2 t, the high half to the next one; nibble n of a half is element 32 j + 4 g + n.
//   16 d            key scales, then key zeros: fp16 [16 tokens][G] each.
//   16 d + 64 G     value scales, then value zeros: fp16 [8 token pairs][G][2] each.
// An element is scale * code + zero.
//
// The order is that of the matrix instruction's fragments (m16n8k16): in the products with the keys, lane (g, t)
// needs, for tokens g and g + 8, the same 8 elements of each group -- G consecutive words; in the products with the
// values it needs element pairs of two tokens -- the two halves of a word.  A nibble at bit 0 or 4 of a half, the rest
// masked off, is the fp16 subnormal code * 2^-24 or code * 2^-20, so a word of 8 codes becomes four operand registers
// with four ANDs and one shift, and no conversion.  No byte is shared by two tokens: tokens can be written apart.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"
#include "kv4.h"

namespace rwo {

constexpr unsigned kFull = 0xffffffffu;

template <int DH>
struct Kv4Block {
  static_assert(DH == 64 || DH == 128, "head dimension 64 or 128");
  static constexpr int G = DH / kKv4Group;
  static constexpr int kBytes = 20 * DH;
  static constexpr int kV = 8 * DH;             // value codes
  static constexpr int kKScale = 16 * DH;       // fp16 [16][G]
  static constexpr int kKZero = kKScale + 32 * G;
  static constexpr int kVScale = kKZero + 32 * G;  // fp16 [8][G][2]
  static constexpr int kVZero = kVScale + 32 * G;
};

// New tokens of sequence b: rows [start, start + n) of the call.  Offsets outside the call's rows give n = 0 (and
// `bad`): nothing is read or written for them.
struct Kv4Seq {
  int start, n, len;
  bool down;  // the next offset is smaller
};
__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4View& c, int b, bool& bad) {
  Kv4Seq s;
  s.len = __ldg(c.lens + b);
  s.down = false;
  if (c.cu) {
    const int lo = __ldg(c.cu + b), hi = __ldg(c.cu + b + 1);
    s.start = lo;
    s.n = hi - lo;
    s.down = hi < lo;
    if (lo < 0 || hi < lo || hi > c.tokens) {
      bad = true;
      s.start = s.n = 0;
    }
  } else {
    s.start = b;
    s.n = 1;
  }
  const int64_t room = c.width * c.page_blocks * kKv4Block;
  if (s.len < 0 || s.len > room) {
    bad = true;
    s.len = s.len < 0 ? 0 : int(room);
  }
  return s;
}

// Sequence of row i of the call (-1: a row behind the last sequence).
__device__ __forceinline__ int kv4_seq_of(const Kv4View& c, int64_t i) {
  if (!c.cu) return i < c.batch ? int(i) : -1;
  int lo = 0, hi = c.batch;  // the last b with cu[b] <= i, among [0, batch)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(c.cu + mid) <= i) lo = mid;
    else hi = mid;
  }
  return i >= __ldg(c.cu + lo) && i < __ldg(c.cu + lo + 1) ? lo : -1;
}

// Byte offset of the block of head 0 that holds position pos of sequence b; -1 where the table's entry is no page.
__device__ __forceinline__ int64_t kv4_block_at(const Kv4View& c, int b, int pos, int64_t block_bytes) {
  const int blk = pos / kKv4Block;
  const int page = __ldg(c.table + int64_t(b) * c.width + blk / c.page_blocks);
  if (page < 0 || page >= c.num_pages) return -1;
  return (int64_t(page) * c.heads * c.page_blocks + blk % c.page_blocks) * block_bytes;
}

__device__ __forceinline__ void kv4_bad(const Kv4View& c) { atomicOr(c.status, kStatusBadIndex); }

}  // namespace rwo
