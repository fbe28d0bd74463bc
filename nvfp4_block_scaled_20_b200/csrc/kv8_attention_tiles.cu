// Attention of many query rows over the 8-bit paged cache on the
// 5th-generation tensor cores.
//
// One CTA takes 256 rows (queries of one sequence times the query heads of one
// KV head, in two halves of 128) and walks the keys in steps of 128:
//   warps 0..7    softmax, one thread per row (tensor-memory lane): warps 0..3
//                 the first half, 4..7 the second.  They first bring their q
//                 row to fp16 (a power of two out, exact) in shared memory.
//   warps 8..11   bring K and V: 16-byte loads from the pages, E4M3 to fp16
//                 (exact, one conversion per pair), into a ring of 128-key
//                 tiles in the 128-byte swizzle.  The next step's loads are in
//                 flight in registers, of K and of V apart.
//   warp 12       allocates tensor memory; one thread issues the MMAs
//                 (tcgen05.mma.cta_group::1.kind::f16): S = Q K^T from shared
//                 memory, O += P V with P read from tensor memory, where the
//                 softmax writes it in the place of S.
// The halves alternate: while one half's scores are in the softmax the tensor
// pipe works for the other.  K tiles are K-major operands; V tiles lie the
// same way in memory, [key][dim], and are read as an MN-major operand, so
// nothing is transposed.
//
// Tensor memory (columns): S / P of the halves at 0 and 128, O at 256 and 384.
#include <climits>

#include "attention_common.cuh"
#include "kernels.h"

namespace nvfp4 {

namespace {

constexpr int kKeys = 128;   // keys per step
constexpr int kHalf = 128;   // rows per half (tensor-memory lanes)
constexpr int kTileRows = 2 * kHalf;
constexpr int kSlots = 5;    // ring of K and V tiles
constexpr int kInfo = 4;     // ring of a step's scales
constexpr int kTileThreads = 512;
constexpr int kLoadWarp = 8, kMmaWarp = 12;
constexpr uint32_t kTmemCols = 512;
// One pair of weights in kPolyEvery takes its powers of two from the FMA pipe:
// the special-function unit's 4 results per clock and SM quarter would take as
// long for all of them as the tensor pipe takes for the products.
constexpr int kPolyEvery = 4;
constexpr float kPoly0 = 0x1.000002p+0f, kPoly1 = 0x1.62e430p-1f, kPoly2 = 0x1.ebf906p-3f,
                kPoly3 = 0x1.c6af6cp-5f, kPoly4 = 0x1.3d1070p-7f, kPoly5 = 0x1.5f0890p-10f;
// Tensor-memory columns of a half's scores (and weights) and sums.
__host__ __device__ constexpr uint32_t col_s(int h) { return 128u * h; }
__host__ __device__ constexpr uint32_t col_o(int h) { return 256u + 128u * h; }

struct TilesPlan {
  int row_tiles;    // 256-row tiles per sequence and KV head
  int tiles, full;  // all tiles; those run whole, the others in `splits` key ranges
  int splits;
};

struct TilesSmem {  // after the q tiles and the ring
  float4 info[kInfo][4];  // per 32 keys of a step: ks, log2 vs, 1 / vs
  uint64_t kv_full[kSlots], kv_empty[kSlots];
  uint64_t q_full, s_full[2], p_half[2], p_full[2], o_full[2], mma_done;
  uint32_t tmem;
  int gave_up;
};
template <int kDim>
__host__ __device__ constexpr int tile_bytes() { return kKeys * kDim * 2; }
template <int kDim>
constexpr int tiles_smem_bytes() {
  return (2 + kSlots) * tile_bytes<kDim>() + (int)sizeof(TilesSmem) + 1024;
}

// --------------------------------------------------------------- tcgen05
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Issued by the lane with `lead` set; the whole warp runs the code around, so
// that addresses and descriptors stay in uniform registers.
__device__ __forceinline__ void commit(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{ .reg .pred e; setp.ne.b32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar),
      "r"(lead)
      : "memory");
}
// Shared-memory operand of 128-byte rows in the 128-byte swizzle: 8-row groups
// 1024 bytes apart.  K-major: `lead` unused.  MN-major: the next 64 elements
// of the row dimension lie `lead` bytes on.
// The low word of the descriptor (address and `lead`, in 16 bytes); the high
// word is the same for all.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t lead) {
  return (addr >> 4) | ((lead >> 4) << 16);
}
constexpr uint32_t kOperandHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
// kind::f16, fp16 operands (format 0), fp32 accumulator; bit 16: B is MN-major.
__host__ __device__ constexpr uint32_t f16_instr(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t instr,
                                       uint32_t acc, uint32_t lead) {
  asm volatile(
      "{ .reg .pred p, e; .reg .b64 a, b; setp.ne.b32 p, %4, 0; setp.ne.b32 e, %6, 0;\n"
      "mov.b64 a, {%1, %5}; mov.b64 b, {%2, %5};\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(instr), "r"(acc), "r"(kOperandHigh), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t instr,
                                       uint32_t acc, uint32_t lead) {
  asm volatile(
      "{ .reg .pred p, e; .reg .b64 b; setp.ne.b32 p, %4, 0; setp.ne.b32 e, %6, 0;\n"
      "mov.b64 b, {%2, %5};\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(instr), "r"(acc), "r"(kOperandHigh), "r"(lead)
      : "memory");
}
// 1 in one lane of the warp.
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r;
}
#define NVFP4_R8(r, i) \
  "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
      "=r"(r[i + 6]), "=r"(r[i + 7])
#define NVFP4_I8(r, i) \
  "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
      "r"(r[i + 6]), "r"(r[i + 7])
// 32 consecutive columns of the warp's lanes; valid after ld_wait.
__device__ __forceinline__ void ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : NVFP4_R8(r, 0), NVFP4_R8(r, 8), NVFP4_R8(r, 16), NVFP4_R8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      NVFP4_I8(r, 0), NVFP4_I8(r, 8), NVFP4_I8(r, 16), NVFP4_I8(r, 24)
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      NVFP4_I8(r, 0), NVFP4_I8(r, 8)
      : "memory");
}
#undef NVFP4_R8
#undef NVFP4_I8
// Waits for this thread's tensor-memory loads; r passes through, so that no
// use of it is moved before the wait.
__device__ __forceinline__ void tie16(uint32_t* r) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                    "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                    "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
template <int kRegs>
__device__ __forceinline__ void ld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < kRegs; i += 16) tie16(r + i);
}
__device__ __forceinline__ void st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 16 bytes, or zeros: one predicated load, no branch (which would wait for the
// data before the next load is issued).
__device__ __forceinline__ uint4 load_if(const void* p, bool want) {
  uint4 v;
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %5, 0;\n"
      "mov.b32 %0, 0; mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0;\n"
      "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4]; }"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((int)want));
  return v;
}

// Where a 16-byte chunk of row `row` lies in a [128][64 fp16] block.
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
  return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void store_bf16x8(__nv_bfloat16* dst, const uint32_t* o, float f) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * f,
                                                   __uint_as_float(o[2 * j + 1]) * f);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// max(a, b, c), NaN when one of them is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two powers of two on the FMA pipe.  x = n + f, n whole, |f| <= 1/2 (adding
// 1.5 2^23 rounds to n and leaves it in the low bits); 2^f by the polynomial of
// degree 5 that interpolates it at the Chebyshev nodes of [-1/2, 1/2] (relative
// error below 2.5e-7); n goes into the exponent.  x is at most 2^6 here; below
// -125 it gives 2^-125, which no fp16 weight and no sum notices.
__device__ __forceinline__ uint64_t exp2_poly(uint64_t x) {
  float a, b;
  unpack2(x, a, b);
  x = pack2(fmaxf(a, -125.0f), fmaxf(b, -125.0f));
  const uint64_t r = add2(x, pack2(12582912.0f, 12582912.0f));
  const uint64_t f = sub2(x, sub2(r, pack2(12582912.0f, 12582912.0f)));
  uint64_t p = pack2(kPoly5, kPoly5);
  p = fma2(p, f, pack2(kPoly4, kPoly4));
  p = fma2(p, f, pack2(kPoly3, kPoly3));
  p = fma2(p, f, pack2(kPoly2, kPoly2));
  p = fma2(p, f, pack2(kPoly1, kPoly1));
  p = fma2(p, f, pack2(kPoly0, kPoly0));
  float r0, r1, p0, p1;
  unpack2(r, r0, r1);
  unpack2(p, p0, p1);
  // n 2^23 + p as integers; a multiply-add, on the FMA pipe too
  uint32_t b0, b1;
  asm("mad.lo.u32 %0, %1, 0x800000, %2;" : "=r"(b0) : "r"(__float_as_uint(r0)), "r"(__float_as_uint(p0)));
  asm("mad.lo.u32 %0, %1, 0x800000, %2;" : "=r"(b1) : "r"(__float_as_uint(r1)), "r"(__float_as_uint(p1)));
  return pack2(__uint_as_float(b0), __uint_as_float(b1));
}

// A work unit: a tile, its steps, and its part (-1: the whole tile).
struct Unit {
  int seq, head, tile, split;
  int64_t part;
};
__device__ __forceinline__ Unit unit_of(const Kv8Attention& a, const TilesPlan& p, int u) {
  Unit w;
  int t = u;
  w.split = 0;
  w.part = -1;
  if (u >= p.full && p.splits > 1) {
    const int v = u - p.full;
    t = p.full + v / p.splits;
    w.split = v - (t - p.full) * p.splits;
    w.part = v;
  }
  const int per_head = p.row_tiles;
  w.seq = t / (per_head * a.c.heads);
  const int rest = t - w.seq * per_head * a.c.heads;
  w.head = rest / per_head;
  // late rows see most keys when the mask is causal: longest tiles first
  w.tile = per_head - 1 - (rest - w.head * per_head);
  return w;
}

template <int kDim>
__global__ void __launch_bounds__(kTileThreads, 1)
    attend_tiles_kernel(const __grid_constant__ Kv8Attention a, const TilesPlan plan) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kTile = tile_bytes<kDim>();
  constexpr int kBlock = kKeys * 128;  // [128][64 fp16]
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = smem;              // two q tiles
  uint8_t* ring = smem + 2 * kTile;
  TilesSmem& sm = *reinterpret_cast<TilesSmem*>(ring + kSlots * kTile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pt = a.c.page_tokens;

  const Unit unit = unit_of(a, plan, blockIdx.x);
  QuerySeq q;
  if (!load_query_seq(a.b, pt, unit.seq, q)) {
    if (unit.head == 0 && unit.tile == 0 && unit.split == 0 && threadIdx.x == 0)
      atomicOr(a.err, kDevErrShape);
    return;
  }
  const int row0 = unit.tile * kTileRows, rows = q.n * a.group;
  if (row0 >= rows) return;
  const int live = min(kTileRows, rows - row0);
  const int halves = live > kHalf ? 2 : 1;
  const int i_first = row0 / a.group, i_last = (row0 + live - 1) / a.group;
  const Steps steps = steps_of<kKeys>(a, q, i_first, i_last);
  int s0 = 0, s1 = steps.total;
  if (unit.part >= 0) {
    s0 = (int)((int64_t)steps.total * unit.split / plan.splits);
    s1 = (int)((int64_t)steps.total * (unit.split + 1) / plan.splits);
  }
  const int n_steps = s1 - s0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      bar_init(smem_addr(&sm.kv_full[i]), 4);
      bar_init(smem_addr(&sm.kv_empty[i]), 1);
    }
    bar_init(smem_addr(&sm.q_full), 4 * halves);
    for (int h = 0; h < 2; ++h) {
      bar_init(smem_addr(&sm.s_full[h]), 1);
      bar_init(smem_addr(&sm.p_half[h]), 4);
      bar_init(smem_addr(&sm.p_full[h]), 4);
      bar_init(smem_addr(&sm.o_full[h]), 1);
    }
    bar_init(smem_addr(&sm.mma_done), 1);
    sm.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&sm.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  volatile int* gave_up = &sm.gave_up;

  if (warp < kLoadWarp) {
    // ---------------------------------------------------------------- softmax
    const int h = warp >> 2, r = threadIdx.x & (kHalf - 1);
    if (h < halves) {
      float crow;
      int at;  // place of the row's query in its sequence
      {
        // the row to fp16, a power of two out
        const int row = row0 + h * kHalf + r;
        const bool mine = row < rows;  // the others work on zeros and store nothing
        const int i = mine ? row / a.group : i_last;
        at = q.len - q.n + i;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(a.q) + (q.first + i) * a.q_token +
            (int64_t)(unit.head * a.group + (mine ? row - i * a.group : 0)) * a.q_head);
        uint32_t w[kDim / 2];
#pragma unroll
        for (int k = 0; k < kDim / 8; ++k) {
          const uint4 x = mine ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
          w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
        }
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kDim / 2; ++k)
          m = max(m, max((w[k] << 16) & 0x7FFFFFFFu, w[k] & 0x7FFF0000u));
        const int e = m ? row_exponent(__uint_as_float(m)) : 0;
        const float down = pow2(-e);
        crow = a.scale_log2 * pow2(e);
#pragma unroll
        for (int k = 0; k < kDim / 8; ++k) {
          uint32_t f[4];
#pragma unroll
          for (int t = 0; t < 4; ++t)
            f[t] = f16x2(__uint_as_float(w[4 * k + t] << 16) * down,
                         __uint_as_float(w[4 * k + t] & 0xFFFF0000u) * down);
          *reinterpret_cast<uint4*>(sq + h * kTile + (k >> 3) * kBlock + chunk_at(r, k & 7)) =
              make_uint4(f[0], f[1], f[2], f[3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&sm.q_full));
      }
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + lanes + col_s(h), to = tmem + lanes + col_o(h);
      // keys that every row of the warp sees
      const int all_lo = seen_at(a, q.len, __reduce_max_sync(0xFFFFFFFFu, at)).lo;
      const int all_hi = seen_at(a, q.len, __reduce_min_sync(0xFFFFFFFFu, at)).hi;
      float m = kNegInf, l = 0.0f;
      bool ok = true;
      for (int j = 0; j < n_steps; ++j) {
        const int key0 = step_at(steps, s0 + j) * kKeys;
        if (!warp_wait(smem_addr(&sm.s_full[h]), j & 1, gave_up, a.wait_limit_ns)) {
          ok = false;
          break;
        }
        fence_after();
        const bool masked = key0 < all_lo || key0 + kKeys > all_hi;
        const float4* info = sm.info[j % kInfo];
        // Two passes over the scores in tensor memory, 32 columns at a time in
        // two buffers, the next 32 on the way while these are worked on.  (All
        // 128 in registers, unrolled, overran the instruction cache.)
        uint32_t s0_[32], s1_[32];
        auto hide = [&](uint32_t* s, int key) {
          const Seen see = seen_at(a, q.len, at);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((key + k >= see.lo && key + k < see.hi) || key + k < see.sink))
              s[k] = __float_as_uint(kNegInf);
        };
        float top = kNegInf;
        auto maximum = [&](uint32_t* s, int c) {
          if (masked) hide(s, key0 + 32 * c);
          const float4 x = info[c];
          float t[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            t[k] = max3(__uint_as_float(s[8 * k]), __uint_as_float(s[8 * k + 1]),
                        __uint_as_float(s[8 * k + 2]));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            t[k] = max3(t[k], __uint_as_float(s[8 * k + 3]), __uint_as_float(s[8 * k + 4]));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            t[k] = max3(t[k], __uint_as_float(s[8 * k + 5]), __uint_as_float(s[8 * k + 6]));
          t[0] = max3(t[0], __uint_as_float(s[7]), __uint_as_float(s[15]));
          t[1] = max3(t[1], __uint_as_float(s[23]), __uint_as_float(s[31]));
          t[0] = max3(t[0], t[1], max3(t[2], t[2], t[3]));
          // the factor is never 0: masked scores (-inf) stay -inf
          top = max3(top, top, fmaf(t[0], fmaxf(crow * x.x, 1e-37f), x.y));
        };
        ld32(ts, s0_);
        ld_wait<32>(s0_);
#pragma unroll 1
        for (int c = 0; c < 4; c += 2) {
          ld32(ts + 32 * (c + 1), s1_);
          maximum(s0_, c);
          ld_wait<32>(s1_);
          ld32(ts + 32 * ((c + 2) & 3), s0_);  // at last the first for the second pass
          maximum(s1_, c + 1);
          ld_wait<32>(s0_);
        }
        // a NaN among the scores that a row sees makes its maximum, and with it
        // the whole row, NaN
        if (__any_sync(0xFFFFFFFFu, !(top <= m + kLazy))) {
          const float next = max3(m, m, top);
          const float g = m == kNegInf ? 0.0f : exp2_approx(m - next);
          m = next;
          l *= g;
          if (j > 0) {
            // the products of the steps before are complete: this step's
            // scores were issued after them
#pragma unroll 1
            for (int c = 0; c < kDim; c += 32) {
              ld32(to + c, s1_);
              ld_wait<32>(s1_);
#pragma unroll
              for (int k = 0; k < 32; ++k) s1_[k] = __float_as_uint(__uint_as_float(s1_[k]) * g);
              st32(to + c, s1_);
            }
          }
        }
        const float base = m == kNegInf ? 0.0f : m;
        // the weights of 32 columns, written over scores already read
        auto weights = [&](uint32_t* s, int c) {
          if (masked) hide(s, key0 + 32 * c);
          const float4 x = info[c];
          const float f = fmaxf(crow * x.x, 1e-37f);
          const uint64_t ff = pack2(f, f), bb = pack2(x.y - base, x.y - base);
          uint32_t p[16];
          uint64_t sum = pack2(0.0f, 0.0f);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            uint64_t t = fma2(pack2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), ff, bb);
            float x0, x1;
            if (k % kPolyEvery == kPolyEvery - 1) {
              t = exp2_poly(t);
              unpack2(t, x0, x1);
            } else {
              unpack2(t, x0, x1);
              x0 = exp2_approx(x0);
              x1 = exp2_approx(x1);
              t = pack2(x0, x1);
            }
            sum = add2(sum, t);
            p[k] = f16x2(x0, x1);
          }
          st16(ts + 16 * c, p);
          float a0, a1;
          unpack2(sum, a0, a1);
          l = fmaf(a0 + a1, x.z, l);
        };
#pragma unroll 1
        for (int c = 0; c < 4; c += 2) {
          ld32(ts + 32 * (c + 1), s1_);
          weights(s0_, c);
          ld_wait<32>(s1_);
          if (c == 0) ld32(ts + 64, s0_);
          weights(s1_, c + 1);
          if (c == 0) ld_wait<32>(s0_);
          // the product with V starts on the first half's weights
          st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(smem_addr(c == 0 ? &sm.p_half[h] : &sm.p_full[h]));
        }
      }
      // nothing seen: what the polynomial gave for masked keys is no weight
      if (m == kNegInf) l = 0.0f;
      if (ok && n_steps > 0 &&
          !warp_wait(smem_addr(&sm.o_full[h]), 0, gave_up, a.wait_limit_ns))
        ok = false;
      if (!ok) {
        *gave_up = 1;
        if (lane == 0) atomicOr(a.err, kDevErrTimeout);
      }
      fence_after();
      // the row's place again, so that it need not be kept in registers above
      int tid = threadIdx.x, block = blockIdx.x;
      asm volatile("" : "+r"(tid), "+r"(block)::"memory");
      const Unit u = unit_of(a, plan, block);
      QuerySeq qs;
      load_query_seq(a.b, pt, u.seq, qs);
      const int row = u.tile * kTileRows + tid;  // tid < 256: half and row
      const bool mine = row < qs.n * a.group;
      const int i = mine ? row / a.group : 0;
      const int qh = u.head * a.group + row - i * a.group;
      const float by = u.part >= 0 ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
      if (u.part >= 0 && mine) {
        const int64_t parts = (int64_t)(plan.tiles - plan.full) * plan.splits;
        part_stats<kTileRows>(a, parts, u.part)[tid] = make_float2(m, l);
      }
#pragma unroll 1
      for (int c = 0; c < kDim; c += 32) {
        uint32_t o[32];
        if (ok && n_steps > 0) {
          ld32(to + c, o);
          ld_wait<32>(o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (!mine) continue;
        if (u.part >= 0) {
          float4* dst = reinterpret_cast<float4*>(part_rows<kTileRows>(a, u.part) +
                                                  tid * kDim + c);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                 __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (qs.first + i) * a.out_token +
                               (int64_t)qh * a.out_head + c;
          // a row that sees nothing (sum 0) is zero; a NaN sum stays
          if (l == 0.0f) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) store_bf16x8(dst + 8 * k, o + 8 * k, by);
        }
      }
      if (a.lse && mine && u.part < 0)
        a.lse[(qs.first + i) * a.q_heads + qh] =
            l == 0.0f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
    }
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------------- loaders
    constexpr int kLanesRow = kDim / 16;             // lanes per key
    constexpr int kRowsLoad = 4 * 32 / kLanesRow;    // keys per load of the four warps
    constexpr int kLoads = kKeys / kRowsLoad;
    const int w = warp - kLoadWarp;
    // The eight lanes of a shared-memory store phase write eight different
    // 16-byte chunks of 128 (chunk 2 col, + 1, xor row): four columns of two
    // rows.  The lanes' columns 4..7 go to the upper half of the warp.
    const int row = w * (32 / kLanesRow) + (kDim == 128 ? (lane >> 2) & 3 : lane >> 2);
    const int col = (lane & 3) + (kDim == 128 ? (lane >> 4) * 4 : 0);
    const int pt_log = 31 - __clz(pt);            // 5, 6 or 7
    const int step_log = 7 - pt_log;              // pages per step, as a power of two
    const int group = 32 >> step_log;             // steps per look-up of pages
    const Seen first = seen_by(a, q, i_first), last = seen_by(a, q, i_last);
    int looked = 0;   // steps [looked, looked + group) are looked up:
    int block = -1;   // each lane's page of them, as its block of codes
    bool all_here = false;  // no page of the looked-up steps lies outside the cache
    float ks = 0.0f, vs = -1.0f;  // lanes 0..3: of the step's 32-key groups
    auto look_up = [&](int step) {
      looked = step;
      block = -1;
      bool bad = false;
      const int mine = step + (lane >> step_log);
      if (mine < s1) {
        const int key =
            step_at(steps, mine) * kKeys + ((lane & ((1 << step_log) - 1)) << pt_log);
        if (key < q.len) {
          const int page = a.b.table[unit.seq * a.b.table_stride + (key >> pt_log)];
          if (page < 0 || page >= a.c.pages) {
            atomicOr(a.err, kDevErrShape);
            bad = true;
          } else {
            block = page;
          }
        }
      }
      all_here = !__any_sync(0xFFFFFFFFu, bad);
    };
    // one tile's codes: 16 bytes of kLoads keys
    auto load = [&](uint4* raw, int step, int which) {
      const int key0 = step_at(steps, step) * kKeys;
      const bool whole = (key0 >= first.lo && key0 + kKeys <= last.hi) || key0 + kKeys <= last.sink;
      const uint8_t* from = nullptr;
      bool here = false;
      // the next page, every 32, 64 or 128 keys
      auto turn = [&](int k) {
        const int pg = __shfl_sync(0xFFFFFFFFu, block,
                                   ((step - looked) << step_log) + (k * kRowsLoad >> pt_log));
        here = pg >= 0;
        from = a.c.codes[which] + ((int64_t)pg * a.c.heads + unit.head) * (pt * kDim) + row * kDim +
               col * 16;
      };
      if (whole && all_here) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int in_page = (k * kRowsLoad) & (pt - 1);
          if (in_page == 0) turn(k);
          raw[k] = __ldg(reinterpret_cast<const uint4*>(from + in_page * kDim));
        }
        return;
      }
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int in_page = (k * kRowsLoad) & (pt - 1);
        if (in_page == 0) turn(k);
        const int key = key0 + k * kRowsLoad + row;
        // codes that no row of the tile sees may be anything, NaN among it
        const bool want =
            here && (whole || (key >= first.lo && key < last.hi) || key < last.sink);
        raw[k] = load_if(from + in_page * kDim, want);
      }
    };
    auto scales = [&](int step) {
      const int pg =
          __shfl_sync(0xFFFFFFFFu, block, ((step - looked) << step_log) + ((lane & 3) * 32 >> pt_log));
      ks = 0.0f;
      vs = -1.0f;
      if (w == 0 && lane < 4 && pg >= 0) {
        ks = a.c.scales[0][(int64_t)pg * a.c.heads + unit.head];
        vs = a.c.scales[1][(int64_t)pg * a.c.heads + unit.head];
      }
    };
    auto store = [&](const uint4* raw, int slot) {
      uint8_t* to = ring + slot * kTile + (col >> 2) * kBlock;
      const int chunk = (2 * col) & 7;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const uint32_t x[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
        uint32_t f[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          f[2 * t] = e4m3x2_f16x2(x[t] & 0xFFFFu);
          f[2 * t + 1] = e4m3x2_f16x2(x[t] >> 16);
        }
        const int at = k * kRowsLoad + row;
        *reinterpret_cast<uint4*>(to + chunk_at(at, chunk)) = make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(to + chunk_at(at, chunk + 1)) = make_uint4(f[4], f[5], f[6], f[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sm.kv_full[slot]));
    };
    auto wait_slot = [&](int n) {
      return warp_wait(smem_addr(&sm.kv_empty[n % kSlots]), ((n / kSlots) & 1) ^ 1, gave_up,
                       a.wait_limit_ns);
    };
    // K and V each have a tile's loads in flight: a step's time to arrive
    uint4 rk[kLoads], rv[kLoads];
    bool ok = true;
    if (n_steps > 0) {
      look_up(s0);
      scales(s0);
      load(rk, s0, 0);
      load(rv, s0, 1);
    }
    for (int j = 0; j < n_steps; ++j) {
      const int next = s0 + j + 1;
      if (!wait_slot(2 * j)) {
        ok = false;
        break;
      }
      if (w == 0 && lane < 4) {
        // an absent page: its keys' scores become -inf
        const float lv = vs < 0.0f ? kNegInf : (float)((int)(__float_as_uint(vs) >> 23) - 127);
        sm.info[j % kInfo][lane] = make_float4(ks, lv, vs < 0.0f ? 0.0f : 1.0f / vs, 0.0f);
      }
      store(rk, (2 * j) % kSlots);
      if (next < s1) {
        if (next >= looked + group) look_up(next);
        scales(next);
        load(rk, next, 0);
      }
      if (!wait_slot(2 * j + 1)) {
        ok = false;
        break;
      }
      store(rv, (2 * j + 1) % kSlots);
      if (next < s1) load(rv, next, 1);
    }
    if (!ok) {
      *gave_up = 1;
      if (lane == 0) atomicOr(a.err, kDevErrTimeout);
    }
  } else {
    // -------------------------------------------------------------------- MMA
    if (warp == kMmaWarp) {
      constexpr uint32_t kInstrS = f16_instr(kHalf, kKeys, false);
      constexpr uint32_t kInstrO = f16_instr(kHalf, kDim, true);
      const uint32_t lead = elect();
      const uint32_t ring_at = smem_addr(ring), q_at = smem_addr(sq);
      auto wait_tile = [&](int n) {
        return warp_wait(smem_addr(&sm.kv_full[n % kSlots]), (n / kSlots) & 1, gave_up,
                        a.wait_limit_ns);
      };
      auto scores = [&](int h, int n) {  // S of half h = Q K^T with the K tile n
        const uint32_t qa = operand(q_at + h * kTile, 16);
        const uint32_t kb = operand(ring_at + (n % kSlots) * kTile, 16);
#pragma unroll
        for (int k = 0; k < kDim / 16; ++k) {
          const uint32_t step = (uint32_t)((k >> 2) * (kBlock >> 4) + (k & 3) * 2);
          mma_ss(tmem + col_s(h), qa + step, kb + step, kInstrS, k > 0, lead);
        }
        commit(smem_addr(&sm.s_full[h]), lead);
      };
      // O of half h += P V over 64 keys of the V tile n
      auto output = [&](int h, int n, int part, bool first_step) {
        const uint32_t vb = operand(ring_at + (n % kSlots) * kTile, kBlock);
#pragma unroll
        for (int i = 0; i < kKeys / 32; ++i) {
          const int k = part * (kKeys / 32) + i;
          mma_ts(tmem + col_o(h), tmem + col_s(h) + 8 * k, vb + (uint32_t)(k * (2048 >> 4)), kInstrO,
                 !first_step || k > 0, lead);
        }
      };
      bool ok = true;
      if (n_steps > 0) {
        ok = warp_wait(smem_addr(&sm.q_full), 0, gave_up, a.wait_limit_ns) && wait_tile(0);
        if (ok) {
          fence_after();
          for (int h = 0; h < halves; ++h) scores(h, 0);
          commit(smem_addr(&sm.kv_empty[0]), lead);
        }
      }
      for (int j = 0; j < n_steps && ok; ++j) {
        const int nv = 2 * j + 1, nk = 2 * j + 2;
        const bool more = j + 1 < n_steps;
        for (int h = 0; h < halves && ok; ++h) {
          if ((h == 0 && !wait_tile(nv)) ||
              !warp_wait(smem_addr(&sm.p_half[h]), j & 1, gave_up, a.wait_limit_ns)) {
            ok = false;
            break;
          }
          fence_after();
          output(h, nv, 0, j == 0);
          if (!warp_wait(smem_addr(&sm.p_full[h]), j & 1, gave_up, a.wait_limit_ns)) {
            ok = false;
            break;
          }
          fence_after();
          output(h, nv, 1, false);
          if (h == halves - 1) commit(smem_addr(&sm.kv_empty[nv % kSlots]), lead);
          if (more) {
            if (h == 0 && !wait_tile(nk)) {
              ok = false;
              break;
            }
            fence_after();
            scores(h, nk);
            if (h == halves - 1) commit(smem_addr(&sm.kv_empty[nk % kSlots]), lead);
          } else {
            commit(smem_addr(&sm.o_full[h]), lead);
          }
        }
      }
      if (!ok) {
        *gave_up = 1;
        if (lane == 0) atomicOr(a.err, kDevErrTimeout);
      }
      // no MMA may still run when the tensor memory is freed
      commit(smem_addr(&sm.mma_done), lead);
      bar_wait(smem_addr(&sm.mma_done), 0, nullptr, 2000000000ull);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
  }
}

// Joins the key ranges of the split tiles in their order: one warp per row.
__global__ void __launch_bounds__(256)
    join_tiles_kernel(const __grid_constant__ Kv8Attention a, const TilesPlan plan) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int v0 = blockIdx.x / (kTileRows / 8) * plan.splits;
  const int r = (blockIdx.x % (kTileRows / 8)) * 8 + (threadIdx.x >> 5);
  const Unit unit = unit_of(a, plan, plan.full + v0);
  QuerySeq q;
  if (!load_query_seq(a.b, a.c.page_tokens, unit.seq, q)) return;
  const int row = unit.tile * kTileRows + r;
  if (row >= q.n * a.group) return;
  const int64_t parts = (int64_t)(plan.tiles - plan.full) * plan.splits;
  join_row<kTileRows>(a, q, parts, v0, plan.splits, r, row, unit.head, lane);
}

TilesPlan plan_tiles(int32_t heads, int32_t group, int32_t n, int32_t max_rows, int64_t max_len) {
  TilesPlan p;
  p.row_tiles = (int)(((int64_t)max_rows * group + kTileRows - 1) / kTileRows);
  p.tiles = p.row_tiles * heads * n;
  p.full = p.tiles;
  p.splits = 1;
  // The tiles of the last, partial round are cut along the keys for the SMs
  // that would idle; a range has at least four steps.
  const int sms = num_sms();
  const int rest = p.tiles % sms;
  int64_t splits = rest ? sms / rest : 1;
  const int64_t steps = (max_len + kKeys - 1) / kKeys;
  if (splits > steps / 4) splits = steps / 4;
  if (splits > 1) {
    p.full = p.tiles - rest;
    p.splits = (int)splits;
  }
  return p;
}

template <int kDim>
cudaError_t launch(const Kv8Attention& a, const TilesPlan& p, cudaStream_t s) {
  constexpr int kSmem = tiles_smem_bytes<kDim>();
  cudaError_t e = cudaFuncSetAttribute(attend_tiles_kernel<kDim>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const unsigned units = (unsigned)(p.full + (p.tiles - p.full) * p.splits);
  attend_tiles_kernel<kDim><<<units, kTileThreads, kSmem, s>>>(a, p);
  return cudaGetLastError();
}

}  // namespace

size_t attend_tiles_partial_bytes(int32_t heads, int32_t dim, int32_t group, int32_t n,
                                  int32_t max_rows, int64_t max_len) {
  const TilesPlan p = plan_tiles(heads, group, n, max_rows, max_len);
  return (size_t)(p.tiles - p.full) * p.splits * kTileRows * ((size_t)dim * 4 + 8);
}

cudaError_t launch_attend_tiles(const Kv8Attention& a, cudaStream_t s) {
  const TilesPlan p = plan_tiles(a.c.heads, a.group, a.b.n, a.b.max_rows,
                                 (int64_t)a.b.table_pages * a.c.page_tokens);
  cudaError_t e = a.c.dim == 128 ? launch<128>(a, p, s) : launch<64>(a, p, s);
  if (e != cudaSuccess || p.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.tiles - p.full) * (kTileRows / 8)));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_tiles_kernel, a, p);
}

}  // namespace nvfp4
