// Internal launcher interface of the attention-side operators (rotary
// positions, the 8-bit paged KV cache and attention over it) between the C
// ABI (api_attention.cu) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace nvfp4 {

// ------------------------------------------------------------------ rope
constexpr int kMaxRopeTensors = 8;
constexpr int kMaxRopePairs = 256;  // head_dim <= 512

struct RopeTensor {
  const void* x;
  void* out;
  int64_t x_token, x_head, out_token, out_head;  // strides in elements
  int32_t heads;
  // filled by the launch: a thread's step in tokens and heads, 65536 / heads + 1
  int32_t step_tokens, step_heads, heads_inv;
};

struct RopeArgs {
  RopeTensor t[kMaxRopeTensors];
  int32_t n;
  int64_t tokens;
  int32_t dim;         // head_dim
  int32_t pairs;       // rotated pairs, the rest of a head is copied
  const int32_t* pos;  // [tokens, pos_stride]
  int64_t pos_stride;
  double turns[kMaxRopePairs];   // turns per position of pair i, signed by the direction
  uint8_t axis[kMaxRopePairs];
};
cudaError_t launch_rope(RopeArgs& a, bool bf16, bool interleaved, cudaStream_t s);

// --------------------------------------------------------------- kv cache
constexpr int kKv8MinExp = -40, kKv8MaxExp = 40;  // exponents of the cache's scales

struct Kv8Cache {
  uint8_t* codes[2];  // K, V: [pages, heads, page_tokens, dim]
  float* scales[2];   // K, V: [pages, heads]
  int64_t pages;
  int32_t heads, page_tokens, dim;
};

struct Kv8Batch {
  const int32_t* table;  // [n, table_stride], table_pages entries used
  int64_t table_stride;
  const int32_t* lens;   // [n]
  const int32_t* starts; // [n + 1] first packed row of each sequence
  int64_t rows;          // rows of the packed tensors
  int32_t table_pages, n, max_rows;
};

struct Kv8Rows {  // packed rows of K and V, written from or read into
  void* x[2];
  int64_t token[2], head[2];  // strides in elements
};
cudaError_t launch_kv8_write(const Kv8Cache& c, const Kv8Batch& b, const Kv8Rows& r, bool bf16,
                             uint32_t* err, cudaStream_t s);
cudaError_t launch_kv8_read(const Kv8Cache& c, const Kv8Batch& b, const Kv8Rows& r, bool bf16,
                            uint32_t* err, cudaStream_t s);

// -------------------------------------------------------------- attention
struct Kv8Attention {
  Kv8Cache c;
  Kv8Batch b;
  const void* q;  // bf16
  void* out;      // bf16
  float* lse;     // [rows, q_heads] or null
  int64_t q_token, q_head, out_token, out_head;
  int32_t q_heads, group;  // group = q_heads / c.heads
  float scale_log2;        // softmax scale * log2(e)
  int32_t causal, window, sink;
  uint32_t* err;
  float* part;  // partial results of split tiles (workspace)
  uint64_t wait_limit_ns;
  // test hook (nvfp4_set_test_stall), 0 or 1: an arrival that the first copies'
  // barrier of a CTA waits for in vain
  int32_t stall;
};
// Bytes of partial results the launch of these sizes uses.
size_t kv8_attention_partial_bytes(int32_t heads, int32_t dim, int32_t group, int32_t n,
                                   int32_t max_rows, int64_t max_len);
cudaError_t launch_kv8_attention(const Kv8Attention& a, cudaStream_t s);
// The kernel for many query rows (kv8_attention_tiles.cu), chosen by the two above.
size_t attend_tiles_partial_bytes(int32_t heads, int32_t dim, int32_t group, int32_t n,
                                  int32_t max_rows, int64_t max_len);
cudaError_t launch_attend_tiles(const Kv8Attention& a, cudaStream_t s);

}  // namespace nvfp4
