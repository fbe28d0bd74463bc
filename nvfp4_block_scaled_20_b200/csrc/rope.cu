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
// one of each per thread -- and its threads then stream the heads of all
// tensors past them with 16-byte loads, four heads in flight per thread.
//
// The angle in turns is a double product: position * rate reaches 10^4..10^5
// turns, where fp32 would keep 2^-8 of a turn.  Its fraction, exact, is
// rounded to fp32 once and goes through sincospif.
#include <cuda_bf16.h>

#include "attention.h"

namespace nvfp4 {

namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}

template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Vec {
  T v[N];
};

// P pairs per thread step.  Interleaved: elements [2i, 2i + 2P), one vector;
// halves: elements [i, i + P) and [i + pairs, i + pairs + P), two vectors; past
// the rotated pairs both copy elements [2i, 2i + 2P).
template <typename T, bool kInterleaved, int P>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeArgs a, int tokens_per_cta) {
  constexpr int kN = kInterleaved ? 2 * P : P;  // elements per vector
  constexpr int kHeads = 4;                     // heads in flight per thread
  using V = Vec<T, kN>;
  __shared__ float2 cs[kRopeThreads];
  const int cols = a.dim / 2;  // table entries per token
  const int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta;
  const int n_tok = (int)(a.tokens - t0 < tokens_per_cta ? a.tokens - t0 : tokens_per_cta);
  for (int i = threadIdx.x; i < n_tok * cols; i += kRopeThreads) {
    const int tok = i / cols, pair = i - tok * cols;
    float2 r = make_float2(1.0f, 0.0f);
    if (pair < a.pairs) {
      const double turns = (double)a.pos[(t0 + tok) * a.pos_stride + a.axis[pair]] * a.turns[pair];
      sincospif(2.0f * (float)(turns - rint(turns)), &r.y, &r.x);
    }
    cs[i] = r;
  }
  __syncthreads();
  const int units = cols / P, lanes = kRopeThreads / units;
  const int u = threadIdx.x % units, lane = threadIdx.x / units;
  if (lane >= lanes) return;
  const int i0 = u * P;
  const bool turned = kInterleaved || i0 < a.pairs;
  const int off0 = kInterleaved ? 2 * i0 : (turned ? i0 : 2 * i0);
  const int off1 = kInterleaved ? 0 : (turned ? i0 + a.pairs : 2 * i0 + P);
  for (int tok = 0; tok < n_tok; ++tok) {
    const int64_t t = t0 + tok;
    for (int h0 = blockIdx.y * lanes * kHeads; h0 < a.heads; h0 += gridDim.y * lanes * kHeads) {
      V x0[kHeads], x1[kHeads];
      T* dst[kHeads];
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        const int h = h0 + k * lanes + lane;
        dst[k] = nullptr;
        if (h >= a.heads) continue;
        int j = 0;
        while (h >= a.t[j].head_end) ++j;
        const RopeTensor& r = a.t[j];
        const int64_t hh = h - (j ? a.t[j - 1].head_end : 0);
        const T* src = static_cast<const T*>(r.x) + t * r.x_token + hh * r.x_head;
        dst[k] = static_cast<T*>(r.out) + t * r.out_token + hh * r.out_head;
        x0[k] = *reinterpret_cast<const V*>(src + off0);
        if constexpr (!kInterleaved) x1[k] = *reinterpret_cast<const V*>(src + off1);
      }
      const float2* c = cs + tok * cols + i0;
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        if (!dst[k]) continue;
        // pairs that are not turned are stored as they were read: x * 1 - y * 0
        // is not x when y is infinite
        if constexpr (kInterleaved) {
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const float f0 = to_f32(x0[k].v[2 * p]), f1 = to_f32(x0[k].v[2 * p + 1]);
            if (i0 + p < a.pairs) {
              x0[k].v[2 * p] = from_f32<T>(f0 * c[p].x - f1 * c[p].y);
              x0[k].v[2 * p + 1] = from_f32<T>(f0 * c[p].y + f1 * c[p].x);
            }
          }
        } else if (turned) {
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const float f0 = to_f32(x0[k].v[p]), f1 = to_f32(x1[k].v[p]);
            x0[k].v[p] = from_f32<T>(f0 * c[p].x - f1 * c[p].y);
            x1[k].v[p] = from_f32<T>(f0 * c[p].y + f1 * c[p].x);
          }
        }
        *reinterpret_cast<V*>(dst[k] + off0) = x0[k];
        if constexpr (!kInterleaved) *reinterpret_cast<V*>(dst[k] + off1) = x1[k];
      }
    }
  }
}

template <typename T, bool kInterleaved, int P>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  // as many tokens per CTA as give each thread one sine and cosine
  int tokens = kRopeThreads / (a.dim / 2);
  const int lanes = kRopeThreads / (a.dim / 2 / P);
  // few tokens: one each, and the heads over several CTAs
  unsigned gy = 1;
  if (a.tokens < 148 * tokens) {
    tokens = 1;
    gy = (unsigned)((a.heads + lanes * 4 - 1) / (lanes * 4));
    if (gy > 64) gy = 64;
  }
  const int64_t gx = (a.tokens + tokens - 1) / tokens;
  rope_kernel<T, kInterleaved, P><<<dim3((unsigned)gx, gy), kRopeThreads, 0, s>>>(a, tokens);
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
cudaError_t pick(const RopeArgs& a, cudaStream_t s) {
  constexpr int kWide = kInterleaved ? 8 / (int)sizeof(T) : 16 / (int)sizeof(T);  // 16 bytes
  if (fits(a, sizeof(T), kInterleaved, kWide)) return launch<T, kInterleaved, kWide>(a, s);
  if constexpr (kWide > 4) {
    if (fits(a, sizeof(T), kInterleaved, 4)) return launch<T, kInterleaved, 4>(a, s);
  }
  if (kInterleaved && !fits(a, sizeof(T), true, 1)) {
    // element-aligned pairs: the two halves of a pair through separate loads
    return cudaErrorMisalignedAddress;
  }
  return launch<T, kInterleaved, 1>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, bool interleaved, cudaStream_t s) {
  if (bf16)
    return interleaved ? pick<__nv_bfloat16, true>(a, s) : pick<__nv_bfloat16, false>(a, s);
  return interleaved ? pick<float, true>(a, s) : pick<float, false>(a, s);
}

}  // namespace nvfp4
