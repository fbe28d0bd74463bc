// What the two attention kernels over the 8-bit cache share: bounded mbarrier
// waits, bulk copies, the ranges of keys a tile of query rows sees, and the
// layout of partial results.
//
// The arithmetic of both, per query row i (t in units of log2):
//
//   t_ij = c_i (q_i . kcode_j) ks_j + log2(vs_j),   m_i = max_j t_ij
//   w_ij = 2^(t_ij - m_i)                           (<= 2^kLazy)
//   o_i  = sum_j w_ij vcode_j / sum_j w_ij / vs_j
//
// ks_j, vs_j are the scales of j's page and head.  With V's scale inside the
// exponent the value codes enter the matrix product as they are, at no
// operation per element; log2(vs) is a whole number.  The row sum divides a
// page's sum of weights by vs once.  With |log2 vs| <= 40 a weight that underflows
// fp32 (2^-126) belongs to a probability below 2^-46 of the row's largest.
//
// The weights are rounded to fp16 for the product with V, the one rounding below
// 32 bits: the tensor cores take both operands in 16 bits at full rate, the codes
// are exact in fp16, and its half step of 2^-11 stays well under that of the bf16
// output (2^-8): the error against 64 bits is 1.66e-3 of the output in either case
// (a bf16 weight's own half step would be 2^-8 too).  No weight overflows
// (kLazy, kJump).  One below 2^-25 becomes 0 in the product, while the row sum,
// in fp32, still counts it: what such a key adds, at most 448 * 2^-25 value codes
// of the row's largest s_v exp(score), is lost.  That is 2^-7 of the smallest
// code's step for each; it only shows where many keys' s_v is smaller than that
// by 2^10 and more.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attention.h"
#include "device_common.cuh"

namespace nvfp4 {

constexpr uint32_t kDevErrShape = 2u;  // NVFP4_ERR_SHAPE
// A row's maximum is replaced only when a new one is larger by more than this
// (in log2): rescaling the accumulators is rare, and weights stay <= 2^8, far
// inside fp16.
constexpr float kLazy = 8.0f;
// Where a maximum is found too late for that, weights may grow to 2^15.
constexpr float kJump = 15.0f;
constexpr float kNegInf = -INFINITY;

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait: false when it ran out or another role gave up.  The clock and
// the flag are only looked at every 32 tries: most waits are short, and what
// follows them waits for their latency.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up,
                                         uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (bar_try(bar, parity)) return true;
    if ((i & 31) == 0) {
      if (gave_up && *gave_up) return false;
      const uint64_t t = global_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > limit_ns) return false;
    }
  }
}
// The same for a whole warp, with one answer for all of its lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* gave_up,
                                          uint64_t limit_ns) {
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, gave_up, limit_ns));
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two E4M3 codes -> two fp16 values (exact), the low code in the low half.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t pair) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)pair));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------------ sequences
struct QuerySeq {
  int64_t first;  // first packed query row
  int len, n;     // cached tokens, queries
};
__device__ __forceinline__ bool load_query_seq(const Kv8Batch& b, int page_tokens, int s,
                                               QuerySeq& q) {
  const int64_t r0 = b.starts[s], r1 = b.starts[s + 1];
  q.first = r0;
  q.len = b.lens[s];
  q.n = (int)(r1 - r0);
  return r0 >= 0 && r1 >= r0 && r1 <= b.rows && r1 - r0 <= b.max_rows && q.len >= 0 &&
         q.len <= (int64_t)b.table_pages * page_tokens;
}

// Keys that a query sees: [lo, hi) and [0, sink).  `at`: the query's place in
// its sequence of `len` cached tokens, negative before the cache's start, at least
// -2^30, as a window is at most 2^30.
struct Seen {
  int lo, hi, sink;
};
__device__ __forceinline__ Seen seen_at(const Kv8Attention& a, int len, int at) {
  Seen s;
  s.hi = a.causal ? max(0, min(len, at + 1)) : len;
  s.lo = a.window >= 0 ? max(0, min(at, len) - a.window) : 0;
  s.sink = a.window >= 0 ? min(a.sink, s.hi) : 0;
  return s;
}
// Query i of a sequence.
__device__ __forceinline__ Seen seen_by(const Kv8Attention& a, const QuerySeq& q, int i) {
  return seen_at(a, q.len, q.len - q.n + i);
}
// Whether some query sees one of keys [key, end), of queries whose first and last
// see these.  (From query to query the limits only move up, by one.)
__device__ __forceinline__ bool any_seen(const Seen& first, const Seen& last, int key, int end) {
  return (key < last.hi && end > first.lo) || key < last.sink;
}
// Steps of kKeys keys that queries [i0, i1] of a sequence need: `head` steps
// from 0 (the sink) and then those from `from` on, `total` in all.
struct Steps {
  int head, from, total;
};
template <int kKeys>
__device__ __forceinline__ Steps steps_of(const Kv8Attention& a, const QuerySeq& q, int i0,
                                          int i1) {
  const Seen first = seen_by(a, q, i0), last = seen_by(a, q, i1);
  Steps s;
  const int end = (last.hi + kKeys - 1) / kKeys;
  s.head = (last.sink + kKeys - 1) / kKeys;
  s.from = max(first.lo / kKeys, s.head);
  s.total = s.head + max(0, end - s.from);
  return s;
}
__device__ __forceinline__ int step_at(const Steps& s, int i) {
  return i < s.head ? i : s.from + (i - s.head);
}

// The power of two that brings a query row of largest magnitude amax into [1, 2), as
// an exponent.  In fp16 its values then keep all eight bits of bf16 down to 2^-17;
// smaller ones are rounded to whole 2^-24, an error of at most 2^-25 of the row's
// largest.
__device__ __forceinline__ int row_exponent(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23) - 127;
  return max(-126, min(126, e));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// ------------------------------------------------------- partial results
// Part `i` of `kRows` rows: kRows x dim fp32 sums of w v, then, after all
// parts, kRows pairs (m, l) each.  The sums of 8 or 16 rows lie row by row; of
// 256 rows, whose lanes hold a row each, as dim / 4 columns of kRows groups of 4.
template <int kRows>
__device__ __forceinline__ float* part_rows(const Kv8Attention& a, int64_t i) {
  return a.part + i * kRows * a.c.dim;
}
template <int kRows>
__device__ __forceinline__ float2* part_stats(const Kv8Attention& a, int64_t parts, int64_t i) {
  return reinterpret_cast<float2*>(a.part + parts * kRows * a.c.dim) + i * kRows;
}

// Joins the `splits` parts from part0 on of row r of a tile, in the order of
// the keys (so the result does not depend on which CTA finished first), and
// stores row `row` of the sequence's rows of a KV head: one warp.
template <int kRows>
__device__ __forceinline__ void join_row(const Kv8Attention& a, const QuerySeq& q, int64_t parts,
                                         int64_t part0, int splits, int r, int row, int head,
                                         int lane) {
  const int dim = a.c.dim;
  float top = kNegInf;
  for (int s = lane; s < splits; s += 32)
    top = fmaxf(top, part_stats<kRows>(a, parts, part0 + s)[r].x);
#pragma unroll
  for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
  float sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int d0 = lane * (dim / 32);
  for (int s0 = 0; s0 < splits; s0 += 32) {
    // each lane the factor of one part: 0 where nothing was seen (its rows are
    // not even read, they may be unwritten), NaN where its sum is NaN
    float f = 0.0f;
    if (s0 + lane < splits) {
      const float2 st = part_stats<kRows>(a, parts, part0 + s0 + lane)[r];
      if (!(st.x == kNegInf && st.y == 0.0f)) f = st.x == kNegInf ? 1.0f : exp2_approx(st.x - top);
      sum = fmaf(st.y, f, sum);
    }
    const int n = min(32, splits - s0);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
      const float g = __shfl_sync(0xFFFFFFFFu, f, s);
      if (g == 0.0f) continue;
      const float* src = part_rows<kRows>(a, part0 + s0 + s) +
                         (kRows <= 16 ? r * dim + d0 : (d0 / 4 * kRows + r) * 4 + d0 % 4);
      if (dim == 128) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(x.x, g, acc[0]), acc[1] = fmaf(x.y, g, acc[1]);
        acc[2] = fmaf(x.z, g, acc[2]), acc[3] = fmaf(x.w, g, acc[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(x.x, g, acc[0]), acc[1] = fmaf(x.y, g, acc[1]);
      }
    }
  }
#pragma unroll
  for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
  const int i = row / a.group, qh = head * a.group + row - i * a.group;
  // a row that sees nothing has sum 0: zeros (a NaN sum stays)
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(
      static_cast<__nv_bfloat16*>(a.out) + (q.first + i) * a.out_token + (int64_t)qh * a.out_head +
      d0);
  dst[0] = __floats2bfloat162_rn(acc[0] * f, acc[1] * f);
  if (dim == 128) dst[1] = __floats2bfloat162_rn(acc[2] * f, acc[3] * f);
  if (a.lse && lane == 0)
    a.lse[(q.first + i) * a.q_heads + qh] =
        sum == 0.0f ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace nvfp4
