// The 8-bit paged KV cache: quantizing tokens as they are written, and reading
// them back.
//
// A page holds page_tokens tokens of every head; the codes of one page and head
// are one contiguous [page_tokens, dim] block of E4M3 bytes with one scale.
//
//   write  scale = 2^e, e the smallest whole number (in [-40, 40]) with
//          amax <= 448 * 2^e over the finite values the page and head hold;
//          code = e4m3(x / scale), round to nearest even.
//   read   x = code * scale, rounded once to the output's type.
//
// A power-of-two scale costs a floating-point code nothing but up to one bit of
// its subnormal range (the largest code lies in (224, 448]), and it makes three
// things exact: x / scale; bringing a page's earlier codes to a scale that has
// grown with later tokens (an exponent shift; only codes that become subnormal
// round again); and the attention kernel's use of log2(scale).
//
// What bounds both: bytes.  Write reads 2 B (bf16) and writes 1 B per value,
// read the reverse.  One CTA owns the (page, head, K or V) block, so a page's
// maximum, its scale and its codes need one pass over the data held in
// registers (64 values per thread, as they were loaded), no atomics and no
// second launch; the result does not depend on the order of CTAs.  A token's
// heads lie next to each other in memory, so neighbouring CTAs take
// neighbouring heads of a page's tokens, and K's CTA has V's beside it.
//
// Measured (device time), 24 heads of 128, pages of 64: 12480 tokens written
// from bf16 39 us, 5.9 TB/s; 23400 read to bf16 68.7 us, 6.3 TB/s; one token of
// each of 32 sequences written 3.7 us.
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "device_common.cuh"

namespace nvfp4 {

namespace {

constexpr uint32_t kDevErrShape = 2u;  // NVFP4_ERR_SHAPE

// Rows of one sequence, checked against the packed tensor and the page table.
struct Seq {
  int64_t first;  // its first packed row
  int64_t len;    // tokens in the cache before the packed rows
  int n;          // packed rows
};
__device__ __forceinline__ bool load_seq(const Kv8Batch& b, int page_tokens, int s, Seq& q) {
  const int64_t r0 = b.starts[s], r1 = b.starts[s + 1];
  q.first = r0;
  q.len = b.lens[s];
  q.n = (int)(r1 - r0);
  return r0 >= 0 && r1 >= r0 && r1 <= b.rows && r1 - r0 <= b.max_rows && q.len >= 0 &&
         q.len + (r1 - r0) <= (int64_t)b.table_pages * page_tokens;
}

// The exponent of the scale of a block whose largest finite magnitude is amax.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int e = (int)(bits >> 23) - 127 - 8;               // amax = m 2^(e + 8), m in [1, 2)
  e += (bits & 0x7FFFFFu) > 0x600000u ? 1 : 0;       // m > 1.75: 448 2^e is too small
  return e < kKv8MinExp ? kKv8MinExp : (e > kKv8MaxExp ? kKv8MaxExp : e);
}

// |v| when finite, else 0, as fp32 bits (monotone as integers).
__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
  const uint32_t a = __float_as_uint(v) & 0x7FFFFFFFu;
  return a < 0x7F800000u ? a : 0u;
}

// 8 consecutive values of a packed row, as loaded and as fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void values(float v[8]) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void values(float v[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// Four fp32 values -> four E4M3 codes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Four E4M3 codes -> fp32 values (exact).
__device__ __forceinline__ void e4m3x4_values(uint32_t w, float v[4]) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(w & 0xFFFFu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// One CTA of kTokens * kDim / 64 threads per (page of the sequence, head, K or
// V): thread t holds the 8 values at column (t % (kDim / 8)) * 8 of rows
// t / (kDim / 8) + k * kRows.
template <typename T, int kDim, int kTokens>
__global__ void __launch_bounds__(kTokens * kDim / 64)
    kv8_write_kernel(const __grid_constant__ Kv8Cache c, const __grid_constant__ Kv8Batch b,
                     const __grid_constant__ Kv8Rows r, uint32_t* err) {
  constexpr int kThreads = kTokens * kDim / 64;
  constexpr int kCols = kDim / 8, kRows = kThreads / kCols, kSteps = 8;
  static_assert(kRows * kSteps == kTokens, "each thread holds 64 values");
  const int blocks = 2 * c.heads;  // of a page: K and V of each head
  const int slot0 = blockIdx.x / blocks, in_page = blockIdx.x - slot0 * blocks;
  const int which = in_page & 1, head = in_page >> 1, s = blockIdx.y;
  Seq q;
  if (!load_seq(b, kTokens, s, q)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, kDevErrShape);
    return;
  }
  const int64_t slot = q.len / kTokens + slot0;  // of the sequence's pages
  const int64_t base = slot * kTokens;
  if (q.n == 0 || base >= q.len + q.n) return;
  const int64_t page = b.table[s * b.table_stride + slot];  // checked below
  // rows [r0, r1) of the page are new; its rows before r0 hold earlier tokens
  const int r0 = (int)(q.len > base ? q.len - base : 0);
  const int r1 = (int)(q.len + q.n - base < kTokens ? q.len + q.n - base : kTokens);
  const int col = (threadIdx.x % kCols) * 8, row = threadIdx.x / kCols;
  const T* x = static_cast<const T*>(r.x[which]) + head * r.head[which] + col;
  Raw8<T> v[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int at = row + k * kRows;
    if (at >= r0 && at < r1)
      v[k].load(x + (q.first + (base + at - q.len)) * r.token[which]);
    else
      v[k].zero();
  }
  if (page < 0 || page >= c.pages) {
    if (in_page == 0 && threadIdx.x == 0) atomicOr(err, kDevErrShape);
    return;
  }
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    float f[8];
    v[k].values(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_abs_bits(f[i]));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if constexpr (kThreads > 32) {
    __shared__ uint32_t warp_max[kThreads / 32];
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, warp_max[w]);
  }
  const int e = scale_exponent(__uint_as_float(m));
  float scale = __uint_as_float((uint32_t)(e + 127) << 23);
  const int64_t block = page * c.heads + head;
  uint8_t* codes = c.codes[which] + block * (int64_t)(kTokens * kDim) + col;
  if (r0 > 0) {
    const float before = c.scales[which][block];
    if (before >= scale) {
      scale = before;
    } else {
      // earlier tokens at the smaller scale: their codes, brought to the new one
      const float ratio = before / scale;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int at = row + k * kRows;
        if (at >= r0) continue;
        uint2* w = reinterpret_cast<uint2*>(codes + at * kDim);
        const uint2 was = *w;
        float f[8];
        e4m3x4_values(was.x, f);
        e4m3x4_values(was.y, f + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= ratio;
        *w = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
      }
    }
    // every thread has read the scale before it changes
    __syncthreads();
  }
  const float inv = 1.0f / scale;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int at = row + k * kRows;
    if (at < r0 || at >= r1) continue;
    float f[8];
    v[k].values(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= inv;
    *reinterpret_cast<uint2*>(codes + at * kDim) =
        make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
  }
  if (threadIdx.x == 0) c.scales[which][block] = scale;
}

// 32 bytes, one store where the row is 32-byte aligned (whole sectors).
__device__ __forceinline__ void store32(uint8_t* p, const uint32_t h[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(h[0]),
                 "r"(h[1]), "r"(h[2]), "r"(h[3]), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(h[0], h[1], h[2], h[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

// One CTA per (page of the sequence, head, K or V): 16 codes per thread step.
template <typename T, int kDim, int kTokens>
__global__ void __launch_bounds__(kTokens * kDim / 64)
    kv8_read_kernel(const __grid_constant__ Kv8Cache c, const __grid_constant__ Kv8Batch b,
                    const __grid_constant__ Kv8Rows r, uint32_t* err) {
  constexpr int kThreads = kTokens * kDim / 64;
  constexpr int kCols = kDim / 16, kRows = kThreads / kCols, kSteps = 4;
  static_assert(kRows * kSteps == kTokens, "each thread holds 64 values");
  const int blocks = 2 * c.heads;  // of a page: K and V of each head
  const int slot0 = blockIdx.x / blocks, in_page = blockIdx.x - slot0 * blocks;
  const int which = in_page & 1, head = in_page >> 1, s = blockIdx.y;
  Seq q;
  if (!load_seq(b, kTokens, s, q)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, kDevErrShape);
    return;
  }
  const int64_t slot = q.len / kTokens + slot0;
  const int64_t base = slot * kTokens;
  if (q.n == 0 || base >= q.len + q.n) return;
  const int64_t page = b.table[s * b.table_stride + slot];  // checked below
  const int r0 = (int)(q.len > base ? q.len - base : 0);
  const int r1 = (int)(q.len + q.n - base < kTokens ? q.len + q.n - base : kTokens);
  const int col = (threadIdx.x % kCols) * 16, row = threadIdx.x / kCols;
  if (page < 0 || page >= c.pages) {
    if (in_page == 0 && threadIdx.x == 0) atomicOr(err, kDevErrShape);
    return;
  }
  const int64_t block = page * c.heads + head;
  const uint8_t* codes = c.codes[which] + block * (int64_t)(kTokens * kDim) + col;
  const float scale = c.scales[which][block];
  uint4 w[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int at = row + k * kRows;
    if (at >= r0 && at < r1) w[k] = __ldg(reinterpret_cast<const uint4*>(codes + at * kDim));
  }
  T* out = static_cast<T*>(r.x[which]) + head * r.head[which] + col;
  const bool wide =
      (((uintptr_t)r.x[which] | (uintptr_t)(r.head[which] * sizeof(T)) |
        (uintptr_t)(r.token[which] * sizeof(T))) & 31) == 0;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int at = row + k * kRows;
    if (at < r0 || at >= r1) continue;
    T* o = out + (q.first + (base + at - q.len)) * r.token[which];
    const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
    for (int i = 0; i < 4; i += 4 / (int)sizeof(T) * 2) {
      // 32 bytes of output: 16 values of bf16, 8 of fp32
      constexpr int kOut = 32 / (int)sizeof(T);
      float f[kOut];
#pragma unroll
      for (int j = 0; j < kOut / 4; ++j) e4m3x4_values(u[i + j], f + 4 * j);
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(T) == 2) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * j] * scale, f[2 * j + 1] * scale);
          h[j] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
          h[j] = __float_as_uint(f[j] * scale);
        }
      }
      store32(reinterpret_cast<uint8_t*>(o) + (i / (4 / (int)sizeof(T) * 2)) * 32, h, wide);
    }
  }
}

template <typename T, int kDim, int kTokens>
cudaError_t launch(bool write, const Kv8Cache& c, const Kv8Batch& b, const Kv8Rows& r,
                   uint32_t* err, cudaStream_t s) {
  // a sequence's rows touch at most this many pages
  const int64_t slots = ((int64_t)b.max_rows - 1 + kTokens - 1) / kTokens + 1;
  if (slots * c.heads * 2 > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(slots * c.heads * 2), (unsigned)b.n);
  constexpr int kThreads = kTokens * kDim / 64;
  if (write)
    kv8_write_kernel<T, kDim, kTokens><<<grid, kThreads, 0, s>>>(c, b, r, err);
  else
    kv8_read_kernel<T, kDim, kTokens><<<grid, kThreads, 0, s>>>(c, b, r, err);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick(bool write, const Kv8Cache& c, const Kv8Batch& b, const Kv8Rows& r,
                 uint32_t* err, cudaStream_t s) {
  if (c.dim == 128) {
    if (c.page_tokens == 32) return launch<T, 128, 32>(write, c, b, r, err, s);
    if (c.page_tokens == 64) return launch<T, 128, 64>(write, c, b, r, err, s);
    return launch<T, 128, 128>(write, c, b, r, err, s);
  }
  if (c.page_tokens == 32) return launch<T, 64, 32>(write, c, b, r, err, s);
  if (c.page_tokens == 64) return launch<T, 64, 64>(write, c, b, r, err, s);
  return launch<T, 64, 128>(write, c, b, r, err, s);
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8Cache& c, const Kv8Batch& b, const Kv8Rows& r, bool bf16,
                             uint32_t* err, cudaStream_t s) {
  return bf16 ? pick<__nv_bfloat16>(true, c, b, r, err, s) : pick<float>(true, c, b, r, err, s);
}

cudaError_t launch_kv8_read(const Kv8Cache& c, const Kv8Batch& b, const Kv8Rows& r, bool bf16,
                            uint32_t* err, cudaStream_t s) {
  return bf16 ? pick<__nv_bfloat16>(false, c, b, r, err, s) : pick<float>(false, c, b, r, err, s);
}

}  // namespace nvfp4
