// Rotary positions over several axes (time, height, width): each pair of a
// head's elements is turned by position[axis of the pair] * rate[pair].
//
//   out0 = x0 cos - x1 sin,  out1 = x0 sin + x1 cos      (fp32, one rounding)
//
// The gradient with respect to x is the same rotation by the negative angle.
//
// What bounds it: every element is read and written once, 4 B of bf16 against
// three operations.  The angles belong to a token, not to its heads, so a CTA
// computes the sine and cosine of its tokens' pairs once into shared memory --
// one of each per thread -- and its threads then stream the heads of one
// tensor past them with 16-byte loads; the first ones are on the way while the
// angles are computed.
//
// The angle in turns is a double product: position * rate reaches 10^4..10^5
// turns, where fp32 would keep 2^-8 of a turn.  Its fraction, exact, is
// rounded to fp32 once and goes through sincospif: 2^-26 of a turn, 9.4e-8 rad, no
// more than the rounding of the fp32 products that follow (fp32 gradient against
// 64 bits 4.1e-8 of its norm; with sine and cosine in 64 bits 3.75e-8).
//
// Measured (device time): q and k of 4680 tokens, 24 heads of 128, bf16: 23.3 us
// for 115 MB, 4.9 TB/s; the fp32 gradient of 2641 tokens, 20 heads of 128: 8.9
// us, 6.1 TB/s; one token 2.2 us.  With two heads in flight per thread 23.5 and
// 9.3 us, with four 25.3 and 11.0: fewer CTAs fit an SM.
#include <cuda_bf16.h>

#include "attention.h"

namespace nvfp4 {

namespace {

constexpr int kRopeThreads = 256;

// Elements 2 i, 2 i + 1 of a vector as fp32, and back (rounded once).
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* v) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(v);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 pair_of(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ void set_pair(__nv_bfloat16* v, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(v) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void set_pair(float* v, float a, float b) { v[0] = a, v[1] = b; }
__device__ __forceinline__ float one_of(const __nv_bfloat16* v) { return __bfloat162float(*v); }
__device__ __forceinline__ float one_of(const float* v) { return *v; }
__device__ __forceinline__ void set_one(__nv_bfloat16* v, float a) { *v = __float2bfloat16_rn(a); }
__device__ __forceinline__ void set_one(float* v, float a) { *v = a; }

// x / d for x < 256 and 1 <= d <= 256, inv = 65536 / d + 1: the product is off
// by x d / 65536 < 1 of a unit.
__device__ __forceinline__ int div256(int x, int inv) { return (x * inv) >> 16; }

template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Vec {
  T v[N];
};

struct RopeLaunch {
  int tokens;     // per CTA
  int cols_inv;   // 65536 / d + 1 of the pairs of a head,
  int units_inv;  // and of the threads of a head
};

// P pairs per thread step.  Interleaved: elements [2i, 2i + 2P), one vector;
// halves: elements [i, i + P) and [i + pairs, i + pairs + P), two vectors; past
// the rotated pairs both copy elements [2i, 2i + 2P).
template <typename T, bool kInterleaved, int P>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeArgs a, const RopeLaunch d) {
  constexpr int kN = kInterleaved ? 2 * P : P;  // elements per vector
  using V = Vec<T, kN>;
  __shared__ __align__(16) float2 cs[kRopeThreads];
  const RopeTensor& r = a.t[blockIdx.y];
  const int cols = a.dim / 2;  // table entries per token
  const int64_t t0 = (int64_t)blockIdx.x * d.tokens;
  const int n_tok = (int)(a.tokens - t0 < d.tokens ? a.tokens - t0 : d.tokens);
  // thread: unit u of the heads lane, lane + step, ... of the CTA's tokens,
  // counted token by token
  const int units = cols / P, step = div256(kRopeThreads - 1, d.units_inv) + (kRopeThreads % units == 0);
  const int lane = div256(threadIdx.x, d.units_inv), u = threadIdx.x - lane * units;
  const int i0 = u * P;
  const bool turned = kInterleaved || i0 < a.pairs;
  const int off0 = kInterleaved ? 2 * i0 : (turned ? i0 : 2 * i0);
  const int off1 = kInterleaved ? 0 : (turned ? i0 + a.pairs : 2 * i0 + P);
  const int heads = r.heads, next_tok = r.step_tokens, next_head = r.step_heads;
  int tok = heads < kRopeThreads ? div256(lane, r.heads_inv) : 0;
  int head = lane - tok * heads;
  if (lane >= step) tok = n_tok;  // threads left over
  const T* src = static_cast<const T*>(r.x) + t0 * r.x_token + off0;
  T* out = static_cast<T*>(r.out) + t0 * r.out_token + off0;
  const int second = off1 - off0;
  V x0, x1;
  auto load = [&]() {
    if (tok >= n_tok) return;
    const T* p = src + (tok * r.x_token + head * r.x_head);
    x0 = *reinterpret_cast<const V*>(p);
    if constexpr (!kInterleaved) x1 = *reinterpret_cast<const V*>(p + second);
  };
  load();
  if (threadIdx.x < n_tok * cols) {
    const int t = div256(threadIdx.x, d.cols_inv), pair = threadIdx.x - t * cols;
    float2 v = make_float2(1.0f, 0.0f);
    if (pair < a.pairs) {
      // one entry per lane: as generic loads (the constant cache would serve
      // the lanes one after the other)
      double rate;
      uint32_t axis;
      asm volatile("ld.f64 %0, [%1];" : "=d"(rate) : "l"(a.turns + pair));
      asm volatile("ld.u8 %0, [%1];" : "=r"(axis) : "l"(a.axis + pair));
      const double turns = (double)a.pos[(t0 + t) * a.pos_stride + axis] * rate;
      sincospif(2.0f * (float)(turns - rint(turns)), &v.y, &v.x);
    }
    cs[threadIdx.x] = v;
  }
  __syncthreads();
  // pairs that are not turned are stored as they were read: x * 1 - y * 0 is
  // not x when y is infinite
  const int n_turn = min(P, max(0, a.pairs - i0));
  while (tok < n_tok) {
    float2 c[P];
    const float2* table = cs + tok * cols + i0;
#pragma unroll
    for (int p = 0; p < P; ++p) c[p] = table[p];
    if constexpr (kInterleaved) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float2 f = pair_of(x0.v + 2 * p);
        if (p < n_turn)
          set_pair(x0.v + 2 * p, f.x * c[p].x - f.y * c[p].y, f.x * c[p].y + f.y * c[p].x);
      }
    } else if (turned) {
      if constexpr (P > 1) {
#pragma unroll
        for (int p = 0; p < P; p += 2) {
          const float2 f = pair_of(x0.v + p), g = pair_of(x1.v + p);
          set_pair(x0.v + p, f.x * c[p].x - g.x * c[p].y, f.y * c[p + 1].x - g.y * c[p + 1].y);
          set_pair(x1.v + p, f.x * c[p].y + g.x * c[p].x, f.y * c[p + 1].y + g.y * c[p + 1].x);
        }
      } else {
        const float f = one_of(x0.v), g = one_of(x1.v);
        set_one(x0.v, f * c[0].x - g * c[0].y);
        set_one(x1.v, f * c[0].y + g * c[0].x);
      }
    }
    T* p = out + (tok * r.out_token + head * r.out_head);
    *reinterpret_cast<V*>(p) = x0;
    if constexpr (!kInterleaved) *reinterpret_cast<V*>(p + second) = x1;
    tok += next_tok;
    head += next_head;
    if (head >= heads) head -= heads, ++tok;
    load();
  }
}

template <typename T, bool kInterleaved, int P>
cudaError_t launch(RopeArgs& a, cudaStream_t s) {
  // as many tokens per CTA as give each thread one sine and cosine
  const int cols = a.dim / 2, units = cols / P, step = kRopeThreads / units;
  const RopeLaunch d{kRopeThreads / cols, 65536 / cols + 1, 65536 / units + 1};
  for (int i = 0; i < a.n; ++i) {
    RopeTensor& t = a.t[i];
    t.step_tokens = step / t.heads;
    t.step_heads = step % t.heads;
    t.heads_inv = 65536 / t.heads + 1;
  }
  const int64_t gx = (a.tokens + d.tokens - 1) / d.tokens;
  rope_kernel<T, kInterleaved, P><<<dim3((unsigned)gx, (unsigned)a.n), kRopeThreads, 0, s>>>(a, d);
  return cudaGetLastError();
}

// Whether every pointer and stride lets vectors of `bytes` bytes at the
// offsets of P-pair units be aligned.
bool fits(const RopeArgs& a, size_t elem, bool interleaved, int P) {
  const int n = interleaved ? 2 * P : P;
  size_t bytes = elem * n;
  if (bytes > 16) bytes = 16;
  if (a.dim / 2 % P || a.dim / 2 / P > kRopeThreads) return false;
  if (!interleaved && a.pairs % P) return false;
  for (int i = 0; i < a.n; ++i) {
    const RopeTensor& t = a.t[i];
    const uintptr_t all = (uintptr_t)t.x | (uintptr_t)t.out | (uintptr_t)(t.x_token * elem) |
                          (uintptr_t)(t.x_head * elem) | (uintptr_t)(t.out_token * elem) |
                          (uintptr_t)(t.out_head * elem);
    if (all % bytes) return false;
  }
  return true;
}

template <typename T, bool kInterleaved>
cudaError_t pick(RopeArgs& a, cudaStream_t s) {
  constexpr int kWide = kInterleaved ? 8 / (int)sizeof(T) : 16 / (int)sizeof(T);  // 16 bytes
  if (fits(a, sizeof(T), kInterleaved, kWide)) return launch<T, kInterleaved, kWide>(a, s);
  if constexpr (kWide > 4) {
    if (fits(a, sizeof(T), kInterleaved, 4)) return launch<T, kInterleaved, 4>(a, s);
  }
  if (kInterleaved && !fits(a, sizeof(T), true, 1)) {
    // (the caller has checked the alignment of pairs)
    return cudaErrorMisalignedAddress;
  }
  return launch<T, kInterleaved, 1>(a, s);
}

}  // namespace

cudaError_t launch_rope(RopeArgs& a, bool bf16, bool interleaved, cudaStream_t s) {
  if (bf16)
    return interleaved ? pick<__nv_bfloat16, true>(a, s) : pick<__nv_bfloat16, false>(a, s);
  return interleaved ? pick<float, true>(a, s) : pick<float, false>(a, s);
}

}  // namespace nvfp4
