// kv4.h -- internal interface of the 4-bit paged key/value cache: append, read back, attention.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace rwo {

constexpr int kKv4Group = 32;  // elements that share a scale and a zero
constexpr int kKv4Block = 16;  // tokens of a head that lie together

// The cache and the sequences of one call (device pointers; sizes checked by the caller).
struct Kv4View {
  unsigned char* data = nullptr;     // [num_pages][heads][page_size / 16][20 d] bytes
  const int32_t* table = nullptr;    // [batch][width]
  const int32_t* lens = nullptr;     // [batch]: tokens in the cache, this call's included
  const int32_t* cu = nullptr;       // [batch + 1] offsets into the call's tokens, or null: one token each
  int64_t num_pages = 0, width = 0;  // width: pages a row of the table has room for
  int64_t tokens = 0;                // rows of q, k, v, o
  int batch = 0, heads = 0, d = 0;
  int page_blocks = 0;               // page_size / 16
  unsigned* status = nullptr;
};

// Rows [tokens][heads][d] at token and head strides in elements.
struct Kv4Rows {
  const void* p = nullptr;
  int64_t token = 0, head = 0;
};

cudaError_t launch_kv4_append(const Kv4View& c, const Kv4Rows& k, const Kv4Rows& v, const Kv4Rows& q, const Kv4Rows& q_out,
                              int q_heads, const float* cos_sin, int64_t positions, int rot, bool neighbours, int dtype,
                              cudaStream_t stream, const DeviceInfo& dev);

cudaError_t launch_kv4_gather(const Kv4View& c, const Kv4Rows& k, const Kv4Rows& v, int dtype, cudaStream_t stream,
                              const DeviceInfo& dev);

// Workspace of the attention, and the attention itself.
size_t attention_kv4_scratch(int64_t batch, int64_t tokens, int q_heads, int heads, int d, const DeviceInfo& dev);
cudaError_t launch_attention_kv4(const Kv4View& c, const Kv4Rows& q, void* o, float* lse, int q_heads, float scale, int dtype,
                                 void* scratch, cudaStream_t stream, const DeviceInfo& dev);

}  // namespace rwo
