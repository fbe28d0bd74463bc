// C ABI of the attention-side operators (declared in include/nvfp4.h):
// argument validation on the host, workspace carve-up, kernel launches.
#include <climits>
#include <cmath>
#include <cstring>

#include "../../include/nvfp4.h"
#include "attention.h"
#include "kernels.h"

using namespace nvfp4;

namespace {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool aligned(int64_t stride, int64_t a) { return stride % a == 0; }
inline int64_t elem_bytes(int32_t dt) { return dt == NVFP4_BF16 ? 2 : 4; }
inline bool dtype_ok(int32_t dt) { return dt == NVFP4_F32 || dt == NVFP4_BF16; }
inline cudaStream_t S(void* s) { return static_cast<cudaStream_t>(s); }
nvfp4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// Whether the rows of `dim` elements that a call writes at i s0 + j s1, i < n0 and
// j < n1, lie apart: one stride steps over a row, the other over all rows of the
// first.  (An expanded output would get what CTAs store in any order.)
bool rows_apart(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t dim) {
  if (n0 <= 1) return n1 <= 1 || s1 >= dim;
  if (n1 <= 1) return s0 >= dim;
  if (s0 < s1) return rows_apart(n1, s1, n0, s0, dim);
  return s1 >= dim && (s0 - dim) / s1 >= n1 - 1;
}

// Partial results follow the error word in the workspace.
constexpr size_t kPartOffset = 256;

nvfp4_status check_cache(const nvfp4_kv8_cache* c) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return NVFP4_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return NVFP4_ERR_SHAPE;
  if (c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128) return NVFP4_ERR_SHAPE;
  // heads (times K and V) are a grid dimension
  if (c->heads < 1 || c->heads > 32767 || c->pages < 1 || c->pages > INT32_MAX)
    return NVFP4_ERR_SHAPE;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) ||
      !aligned(c->v_scales, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

nvfp4_status check_batch(const nvfp4_kv8_batch* b, int32_t page_tokens) {
  if (!b) return NVFP4_ERR_INVALID_ARG;
  // (arrays of no sequences have no address)
  if (b->n != 0 && (!b->page_table || !b->lens || !b->starts)) return NVFP4_ERR_INVALID_ARG;
  // sequences are a grid dimension; token positions are 32-bit
  if (b->n < 0 || b->n > 65535 || b->rows < 0 || b->max_rows < 0 || b->table_pages < 1 ||
      b->table_stride < b->table_pages)
    return NVFP4_ERR_SHAPE;
  if (b->max_rows > (1 << 30) || (int64_t)b->table_pages * page_tokens > (1 << 30))
    return NVFP4_ERR_SHAPE;
  if (!aligned(b->page_table, 4) || !aligned(b->lens, 4) || !aligned(b->starts, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

Kv8Cache cache_of(const nvfp4_kv8_cache* c) {
  return Kv8Cache{{c->k_codes, c->v_codes}, {c->k_scales, c->v_scales}, c->pages, c->heads,
                  c->page_tokens, c->head_dim};
}
Kv8Batch batch_of(const nvfp4_kv8_batch* b) {
  return Kv8Batch{b->page_table, b->table_stride, b->lens, b->starts, b->rows,
                  b->table_pages, b->n, b->max_rows};
}

nvfp4_status write_or_read(bool write, const nvfp4_kv8_cache* cache, const nvfp4_kv8_batch* batch,
                           int32_t dtype, void* k, void* v, const int64_t strides[4], void* ws,
                           size_t ws_bytes, void* stream) {
  nvfp4_status st = check_cache(cache);
  if (st != NVFP4_OK) return st;
  st = check_batch(batch, cache->page_tokens);
  if (st != NVFP4_OK) return st;
  if (!dtype_ok(dtype)) return NVFP4_ERR_INVALID_ARG;
  if (batch->n == 0 || batch->rows == 0 || batch->max_rows == 0) return NVFP4_OK;
  if (!k || !v) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return NVFP4_ERR_ALIGN;
  for (int i = 0; i < 4; ++i) {
    if (strides[i] < 0) return NVFP4_ERR_SHAPE;
    if (!aligned(strides[i] * elem_bytes(dtype), 16)) return NVFP4_ERR_ALIGN;
  }
  for (int i = 0; i < 4 && !write; i += 2)
    if (!rows_apart(batch->rows, strides[i], cache->heads, strides[i + 1], cache->head_dim))
      return NVFP4_ERR_SHAPE;
  if (!ws || ws_bytes < nvfp4_workspace_bytes(0)) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 4)) return NVFP4_ERR_ALIGN;  // the error word
  if (!write && k == v) return NVFP4_ERR_INVALID_ARG;
  // one CTA per page that a sequence may touch, head, K and V: a grid dimension
  if (((int64_t)batch->max_rows / cache->page_tokens + 2) * cache->heads * 2 > INT32_MAX)
    return NVFP4_ERR_SHAPE;
  const Kv8Rows r{{k, v}, {strides[0], strides[2]}, {strides[1], strides[3]}};
  uint32_t* err = static_cast<uint32_t*>(ws);
  const bool bf16 = dtype == NVFP4_BF16;
  return cuda_status(write ? launch_kv8_write(cache_of(cache), batch_of(batch), r, bf16, err, S(stream))
                           : launch_kv8_read(cache_of(cache), batch_of(batch), r, bf16, err, S(stream)));
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_rope(const nvfp4_rope_tensor* tensors, int32_t n, int32_t dtype, int64_t tokens,
                        int32_t head_dim, const int32_t* positions, int64_t positions_stride,
                        const nvfp4_rope_params* rp, void* stream) {
  if (!tensors || !rp || n < 0 || !dtype_ok(dtype)) return NVFP4_ERR_INVALID_ARG;
  if (n > kMaxRopeTensors) return NVFP4_ERR_SHAPE;
  if (rp->axes < 1 || rp->axes > 4 || !(rp->theta > 0.0) || !std::isfinite(rp->theta))
    return NVFP4_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > INT32_MAX || head_dim < 2 || head_dim > 2 * kMaxRopePairs ||
      head_dim % 2 || positions_stride < rp->axes)
    return NVFP4_ERR_SHAPE;
  RopeArgs a;
  a.n = 0;
  a.tokens = tokens;
  a.dim = head_dim;
  a.pos = positions;
  a.pos_stride = positions_stride;
  a.pairs = 0;
  for (int i = 0; i < rp->axes; ++i) {
    if (rp->sections[i] < 0 || rp->sections[i] > head_dim / 2) return NVFP4_ERR_SHAPE;
    a.pairs += rp->sections[i];
  }
  if (a.pairs > head_dim / 2) return NVFP4_ERR_SHAPE;
  const int64_t eb = elem_bytes(dtype);
  for (int32_t i = 0; i < n; ++i) {
    const nvfp4_rope_tensor& t = tensors[i];
    if (t.heads < 0 || t.heads > 65535) return NVFP4_ERR_SHAPE;
    if (t.heads == 0) continue;
    if (tokens > 0 && (!t.x || !t.out)) return NVFP4_ERR_INVALID_ARG;
    const int64_t strides[4] = {t.x_token_stride, t.x_head_stride, t.out_token_stride,
                                t.out_head_stride};
    for (int64_t s : strides) {
      if (s < 0) return NVFP4_ERR_SHAPE;
      if (s % 2) return NVFP4_ERR_ALIGN;  // pairs of elements
    }
    if (!aligned(t.x, 2 * eb) || !aligned(t.out, 2 * eb)) return NVFP4_ERR_ALIGN;
    if (!rows_apart(tokens, t.out_token_stride, t.heads, t.out_head_stride, head_dim))
      return NVFP4_ERR_SHAPE;
    a.t[a.n++] = RopeTensor{t.x, t.out, t.x_token_stride, t.x_head_stride, t.out_token_stride,
                            t.out_head_stride, (int32_t)t.heads, 0, 0, 0};
  }
  if (tokens == 0 || a.n == 0) return NVFP4_OK;
  // an output may take the place of its own input, element by element, and of
  // nothing else that the call reads or writes
  for (int i = 0; i < a.n; ++i) {
    const RopeTensor& t = a.t[i];
    if (t.out == t.x && ((tokens > 1 && t.out_token != t.x_token) ||
                         (t.heads > 1 && t.out_head != t.x_head)))
      return NVFP4_ERR_INVALID_ARG;
    for (int j = 0; j < a.n; ++j)
      if (j != i && (t.out == a.t[j].out || t.out == a.t[j].x)) return NVFP4_ERR_INVALID_ARG;
  }
  if (!positions) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return NVFP4_ERR_ALIGN;
  // turns per position: theta^-(j / pairs of the axis) or theta^-(i / all pairs),
  // over 2 pi; one power per axis, the rest by repeated products (relative
  // error below 256 * 2^-52)
  const double turn = (rp->inverse ? -1.0 : 1.0) / 6.283185307179586476925286766559;
  double step = rp->per_axis || a.pairs == 0 ? 1.0 : std::pow(rp->theta, -1.0 / a.pairs);
  double rate = turn;
  for (int i = 0, at = 0; i < rp->axes; ++i) {
    if (rp->per_axis && rp->sections[i] > 0) {
      step = std::pow(rp->theta, -1.0 / rp->sections[i]);
      rate = turn;
    }
    for (int j = 0; j < rp->sections[i]; ++j, ++at) {
      a.turns[at] = rate;
      a.axis[at] = (uint8_t)i;
      rate *= step;
    }
  }
  return cuda_status(launch_rope(a, dtype == NVFP4_BF16, rp->interleaved != 0, S(stream)));
}

nvfp4_status nvfp4_kv8_write(const nvfp4_kv8_cache* cache, const nvfp4_kv8_batch* batch,
                             int32_t dtype, const void* k, int64_t k_token_stride,
                             int64_t k_head_stride, const void* v, int64_t v_token_stride,
                             int64_t v_head_stride, void* ws, size_t ws_bytes, void* stream) {
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  return write_or_read(true, cache, batch, dtype, const_cast<void*>(k), const_cast<void*>(v),
                       strides, ws, ws_bytes, stream);
}

nvfp4_status nvfp4_kv8_read(const nvfp4_kv8_cache* cache, const nvfp4_kv8_batch* batch,
                            int32_t dtype, void* k, int64_t k_token_stride, int64_t k_head_stride,
                            void* v, int64_t v_token_stride, int64_t v_head_stride, void* ws,
                            size_t ws_bytes, void* stream) {
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  return write_or_read(false, cache, batch, dtype, k, v, strides, ws, ws_bytes, stream);
}

namespace {
// Tiles of query rows over all sequences and KV heads, each a CTA or several:
// at most 2^30.  Of up to three tiles of 16 rows, tiles and heads are a grid
// dimension.
inline bool tiles_ok(int64_t heads, int64_t group, int64_t n, int64_t max_rows) {
  const int64_t rows = max_rows * group;
  return rows <= (1 << 30) && (rows + 255) / 256 * heads * n <= (1 << 30) &&
         (rows > 48 || (rows + 15) / 16 * heads <= 65535);
}
}  // namespace

size_t nvfp4_kv8_attention_workspace_bytes(int32_t heads, int32_t head_dim, int32_t page_tokens,
                                           int32_t q_heads, int32_t n, int32_t max_rows,
                                           int32_t table_pages) {
  if (heads < 1 || q_heads < heads || q_heads % heads || n < 1 || max_rows < 1 || table_pages < 1 ||
      page_tokens < 1 || (head_dim != 64 && head_dim != 128) || !tiles_ok(heads, q_heads / heads, n, max_rows))
    return kPartOffset;
  return kPartOffset + kv8_attention_partial_bytes(heads, head_dim, q_heads / heads, n, max_rows,
                                                   (int64_t)table_pages * page_tokens);
}

nvfp4_status nvfp4_kv8_attention(const nvfp4_kv8_cache* cache, const nvfp4_kv8_batch* batch,
                                 const nvfp4_kv8_query* qp, void* ws, size_t ws_bytes,
                                 void* stream) {
  nvfp4_status st = check_cache(cache);
  if (st != NVFP4_OK) return st;
  st = check_batch(batch, cache->page_tokens);
  if (st != NVFP4_OK) return st;
  if (!qp) return NVFP4_ERR_INVALID_ARG;
  if (!(qp->scale > 0.0f) || !std::isfinite(qp->scale)) return NVFP4_ERR_INVALID_ARG;
  if ((qp->causal != 0 && qp->causal != 1) || qp->window < -1 || qp->sink < 0)
    return NVFP4_ERR_INVALID_ARG;
  if (qp->q_heads < cache->heads || qp->q_heads % cache->heads) return NVFP4_ERR_SHAPE;
  const int64_t group = qp->q_heads / cache->heads;
  if (!tiles_ok(cache->heads, group, batch->n, batch->max_rows)) return NVFP4_ERR_SHAPE;
  if (batch->n == 0 || batch->rows == 0 || batch->max_rows == 0) return NVFP4_OK;
  if (!qp->q || !qp->out) return NVFP4_ERR_INVALID_ARG;
  const int64_t strides[4] = {qp->q_token_stride, qp->q_head_stride, qp->out_token_stride,
                              qp->out_head_stride};
  for (int64_t s : strides) {
    if (s < 0) return NVFP4_ERR_SHAPE;
    if (s % 8) return NVFP4_ERR_ALIGN;  // 16 bytes of bf16
  }
  if (!aligned(qp->q, 16) || !aligned(qp->out, 16) || (qp->lse && !aligned(qp->lse, 4)))
    return NVFP4_ERR_ALIGN;
  if (!rows_apart(batch->rows, qp->out_token_stride, qp->q_heads, qp->out_head_stride,
                  cache->head_dim))
    return NVFP4_ERR_SHAPE;
  // a tile reads its rows of q before it writes any of them
  if (qp->out == qp->q && ((batch->rows > 1 && qp->out_token_stride != qp->q_token_stride) ||
                           (qp->q_heads > 1 && qp->out_head_stride != qp->q_head_stride)))
    return NVFP4_ERR_INVALID_ARG;
  Kv8Attention a;
  std::memset(&a, 0, sizeof(a));
  a.c = cache_of(cache);
  a.b = batch_of(batch);
  a.q = qp->q;
  a.out = qp->out;
  a.lse = qp->lse;
  a.q_token = qp->q_token_stride;
  a.q_head = qp->q_head_stride;
  a.out_token = qp->out_token_stride;
  a.out_head = qp->out_head_stride;
  a.q_heads = qp->q_heads;
  a.group = (int32_t)group;
  a.scale_log2 = (float)((double)qp->scale * 1.4426950408889634074);
  a.causal = qp->causal;
  // places in a sequence are in -2^30 .. 2^30: a window of 2^30 hides nothing,
  // and what the kernels subtract from a place stays in 32 bits
  a.window = qp->window < (1 << 30) ? qp->window : (1 << 30);
  a.sink = qp->sink;
  const size_t need = nvfp4_kv8_attention_workspace_bytes(
      cache->heads, cache->head_dim, cache->page_tokens, qp->q_heads, batch->n, batch->max_rows,
      batch->table_pages);
  if (!ws || ws_bytes < need) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
  a.err = static_cast<uint32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kPartOffset);
  a.wait_limit_ns = gemm_wait_limit_ns();
  a.stall = gemm_test_stall();
  return cuda_status(launch_kv8_attention(a, S(stream)));
}

}  // extern "C"
