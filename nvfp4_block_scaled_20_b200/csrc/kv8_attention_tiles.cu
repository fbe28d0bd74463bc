// Attention of many query rows over the 8-bit paged cache on the
// 5th-generation tensor cores.
//
// One CTA takes 256 rows (queries of one sequence times the query heads of one
// KV head, in two halves of 128) and walks the keys in steps of 128:
//   warps 0..7    softmax, one thread per row (tensor-memory lane): warps 0..3
//                 the first half, 4..7 the second.  They first bring their q
//                 row to fp16 (a power of two out, exact) in shared memory.
//   warps 8, 9    bring the codes of a 128-key tile to fp16 (exact, one
//                 conversion per pair), in the 128-byte swizzle, into a ring of
//                 four tiles.
//   warp 10       allocates tensor memory and issues the MMAs
//                 (tcgen05.mma.cta_group::1.kind::f16): S = Q K^T from shared
//                 memory, O += P V with P read from tensor memory, where the
//                 softmax writes it in the place of S.
//   warp 11       looks pages up 32 at a time, one group ahead, and keeps two
//                 tiles of codes in flight with untiled bulk copies (a page and
//                 head is one contiguous block).
// The halves take turns: while one half's scores are in the softmax the tensor
// pipe works for the other.  K tiles are K-major operands; V tiles lie the
// same way in memory, [key][dim], and are read as an MN-major operand, so
// nothing is transposed.
//
// What bounds it: the turn of one half.  Scores ready -> maximum and weights of
// 96 keys -> their product under way while the last 32 are worked on -> the
// last product and the next scores, two hops through an mbarrier of about 200
// clocks each on the way: about 3600 clocks alone, 2048 of them the
// special-function unit's when both halves' exponentials are counted, and 2048
// the tensor pipe's for both.  Measured at 4680 x 32760 x 24 heads of 128
// (one GPU, us): scores in two passes, K and V through registers 1925; codes by
// bulk copies 1845 (loads of two paths that meet wait for their data at the
// join, and what a warp cannot keep in registers goes to an L1 cache that the
// shared memory has left almost nothing of: spills in a step cost more than the
// work they stand for); one pass, two turns of 64 keys 1784; 96 and 32 keys
// 1632 while the GPU is cool, 1700 to 1800 (1050 to 1110 TFLOP/s) in a loop that
// holds it at its power limit.  What a tile costs besides its steps, 4736 rows
// of 24 heads that see 128 keys: 57 with a thread on each row of q and out, 43
// with a warp on each row.  Measured and not kept: two
// softmax warps per row, an issuing thread per half (the halves fall into step
// and wait together, 2300), the softmax warps issuing their own products
// (2600), scores by 64 keys in two buffers per half (products of 64 columns
// take as long as of 128: 1900), a quarter of the exponentials as polynomials
// on the FMA pipe (packed fma: 3.6 clocks a warp; no change), CTAs that stay and
// take the next tile by cluster launch control (they hide a tile's set-up and
// look-ups, 0.5 us of 9, and cost registers in the steps: three prompts 439 beside
// 405 of the kernel at that time, a chunk 1820 beside 1720), counting the tiles of
// ragged sequences in the kernel to split the true last round (three prompts 399
// beside 405 at that time, one prompt 224 beside 217, 40 short ones 1122 beside
// 1095; today's three prompts take 399 without), and taking NaN codes out of V in
// steps that only some rows see, to set them in those rows at the end (the
// converters are at their rate: three prompts 426 beside 400).
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
constexpr int kSlots = 4;    // ring of K and V tiles in fp16
constexpr int kRaw = 2;      // ring of tiles as they lie in the pages
constexpr int kInfo = 4;     // ring of a step's scales
constexpr int kTileThreads = 12 * 32;
constexpr int kLoadWarp = 8, kLoadWarps = 2, kMmaWarp = 10, kCopyWarp = 11;
constexpr uint32_t kTmemCols = 512;
constexpr int kNoPage = INT_MIN;
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
  uint64_t kv_full[kSlots], kv_empty[kSlots], raw_full[kRaw], raw_empty[kRaw];
  int whole[kInfo];  // every key of the step is in the cache and seen by a row
  uint64_t q_full, s_full[2], p_part[2], p_full[2], pv_part[2], o_full[2], mma_done;
  uint32_t tmem;
  int gave_up;
};
template <int kDim>
__host__ __device__ constexpr int tile_bytes() { return kKeys * kDim * 2; }
template <int kDim>
constexpr int tiles_smem_bytes() {
  return (2 + kSlots) * tile_bytes<kDim>() + kRaw * tile_bytes<kDim>() / 2 + (int)sizeof(TilesSmem) + 1024;
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
// 1024 bytes apart.  MN-major: the next 64 elements of the row dimension lie
// `block` bytes on (K-major operands do not use it).  This is the low word of
// the descriptor (address and `block`, in units of 16 bytes); the high word is
// the same for all.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t block) {
  return (addr >> 4) | ((block >> 4) << 16);
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
__device__ __forceinline__ void ld8(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : NVFP4_R8(r, 0)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
               NVFP4_I8(r, 0)
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

// Where a 16-byte chunk of row `row` lies in a [128][64 fp16] block.
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
  return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// Eight sums times f as bf16.
__device__ __forceinline__ uint4 bf16x8(const uint32_t* o, float f) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * f,
                                                   __uint_as_float(o[2 * j + 1]) * f);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
}

// max(a, b, c), NaN when one of them is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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
  uint8_t* raw = ring + kSlots * kTile;  // kRaw tiles of codes
  TilesSmem& sm = *reinterpret_cast<TilesSmem*>(raw + kRaw * kTile / 2);
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
    for (int i = 0; i < kRaw; ++i) {
      bar_init(smem_addr(&sm.raw_full[i]), i == 0 ? 1 + a.stall : 1);
      bar_init(smem_addr(&sm.raw_empty[i]), kLoadWarps);
    }
    for (int i = 0; i < kSlots; ++i) {
      bar_init(smem_addr(&sm.kv_full[i]), kLoadWarps);
      bar_init(smem_addr(&sm.kv_empty[i]), 1);
    }
    bar_init(smem_addr(&sm.q_full), 4 * halves);
    for (int h = 0; h < 2; ++h) {
      bar_init(smem_addr(&sm.s_full[h]), 1);
      bar_init(smem_addr(&sm.p_part[h]), 4);
      bar_init(smem_addr(&sm.pv_part[h]), 1);
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
  // The copying warp's look-up: the page of each lane's piece of the steps from
  // `step` on.  The first is on the way while the others set up.
  const int pt_log = 31 - __clz(pt);  // 5, 6 or 7
  const int step_log = 7 - pt_log;    // pages per step, as a power of two
  const Seen first = seen_by(a, q, i_first), last = seen_by(a, q, i_last);
  auto fetch_page = [&](int step) {
    const int mine = step + (lane >> step_log);
    if (mine >= s1) return kNoPage;
    const int key = step_at(steps, mine) * kKeys + ((lane & ((1 << step_log) - 1)) << pt_log);
    // pages of keys that no row sees are not looked up: past the sequence's end, or
    // out of the window, they may be gone
    return any_seen(first, last, key, key + pt)
               ? a.b.table[unit.seq * a.b.table_stride + (key >> pt_log)]
               : kNoPage;
  };
  int next_page = kNoPage;
  if (warp == kCopyWarp) next_page = fetch_page(s0);
  if (threadIdx.x < kTileRows && row0 + (int)threadIdx.x < rows) {
    // and so are the rows of q, as far as the L2 cache (a tile of one step: 2 of
    // 46 us of four rounds)
    const int row = row0 + threadIdx.x, i = row / a.group;
    const char* src = reinterpret_cast<const char*>(
        static_cast<const __nv_bfloat16*>(a.q) + (q.first + i) * a.q_token +
        (int64_t)(unit.head * a.group + row - i * a.group) * a.q_head);
#pragma unroll
    for (int k = 0; k < kDim * 2; k += 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(src + k));
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
      float crow = 0.0f;
      int at;  // place of the row's query in its sequence
      // Rows of q and out go through a warp together, kRowLanes lanes on one
      // (16 bytes each): a thread on a row of its own would touch a line of
      // memory per lane.
      constexpr int kRowLanes = kDim / 8, kRowsAtOnce = 32 / kRowLanes;
      const int chunk = lane % kRowLanes;
      {
        // the rows to fp16, a power of two out
        const int row = row0 + h * kHalf + r;
        const bool mine = row < rows;  // the others work on zeros and store nothing
        const int i = mine ? row / a.group : i_last;
        at = q.len - q.n + i;
        const __nv_bfloat16* src =
            static_cast<const __nv_bfloat16*>(a.q) + (q.first + i) * a.q_token +
            (int64_t)(unit.head * a.group + (mine ? row - i * a.group : 0)) * a.q_head;
        constexpr int kAtOnce = 8;  // loads in flight; 16 spill: 416 us for 3 prompts, 394 so
#pragma unroll 1
        for (int t0 = 0; t0 < kRowLanes; t0 += kAtOnce) {
          uint4 x[kAtOnce];
#pragma unroll
          for (int t = 0; t < kAtOnce; ++t) {
            const int from = (t0 + t) * kRowsAtOnce + lane / kRowLanes;
            const uint64_t p = __shfl_sync(0xFFFFFFFFu, (uint64_t)src, from);
            const bool live = __shfl_sync(0xFFFFFFFFu, (int)mine, from);
            x[t] = live ? __ldg(reinterpret_cast<const uint4*>(p) + chunk) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int t = 0; t < kAtOnce; ++t) {
            const uint32_t w[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m = max(m, max((w[k] << 16) & 0x7FFFFFFFu, w[k] & 0x7FFF0000u));
#pragma unroll
            for (int k = 1; k < kRowLanes; k <<= 1)
              m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
            const int e = m ? row_exponent(__uint_as_float(m)) : 0;
            const float down = pow2(-e);
            uint32_t f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              f[k] = f16x2(__uint_as_float(w[k] << 16) * down,
                           __uint_as_float(w[k] & 0xFFFF0000u) * down);
            const int in = (warp & 3) * 32 + (t0 + t) * kRowsAtOnce + lane / kRowLanes;
            *reinterpret_cast<uint4*>(sq + h * kTile + (chunk >> 3) * kBlock +
                                      chunk_at(in, chunk & 7)) = make_uint4(f[0], f[1], f[2], f[3]);
            // each lane keeps its own row's
            const int own = __shfl_sync(0xFFFFFFFFu, e, lane % kRowsAtOnce * kRowLanes);
            if (lane / kRowsAtOnce == t0 + t) crow = a.scale_log2 * pow2(own);
          }
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
      float m = kNegInf, l = 0.0f, pending = kNegInf;
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
        // Scores of 32 columns, three at a time.  (Registers are what limits it:
        // spills are slow beside so much shared memory, which leaves little of
        // the L1 cache.)
        uint32_t s0_[32], s1_[32], s2_[32];
        auto hide = [&](uint32_t* s, int key) {
          // most groups of a masked step are seen whole by the warp's rows (three
          // prompts 404 us without this line, 394 with it)
          if ((key >= all_lo || key + 32 <= a.sink) && key + 32 <= all_hi) return;
          const Seen see = seen_at(a, q.len, at);
          const uint32_t bits = (below(see.hi - key) & ~below(see.lo - key)) | below(see.sink - key);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!(bits >> k & 1)) s[k] = __float_as_uint(kNegInf);
        };
        auto maximum = [&](const uint32_t* s, int c) {
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
          return fmaf(t[0], fmaxf(crow * x.x, 1e-37f), x.y);
        };
        float base = 0.0f;
        // the weights of 32 columns, written over scores already read
        auto weights = [&](const uint32_t* s, int c) {
          const float4 x = info[c];
          const float f = fmaxf(crow * x.x, 1e-37f);
          const uint64_t ff = pack2(f, f), bb = pack2(x.y - base, x.y - base);
          uint32_t p[16];
          uint64_t sum = pack2(0.0f, 0.0f);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float x0, x1;
            unpack2(fma2(pack2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), ff, bb), x0, x1);
            x0 = exp2_approx(x0);
            x1 = exp2_approx(x1);
            sum = add2(sum, pack2(x0, x1));
            p[k] = f16x2(x0, x1);  // (see attention_common.cuh; the sum is of the fp32 weights)
          }
          st16(ts + 16 * c, p);
          float a0, a1;
          unpack2(sum, a0, a1);
          l = fmaf(a0 + a1, x.z, l);
        };
        // Moves the row's maximum to at least `top` where it has to.  A NaN among
        // the scores that a row sees makes its maximum, and with it the whole
        // row, NaN.
        auto raise = [&](float top, float slack, bool late) {
          if (!__any_sync(0xFFFFFFFFu, !(top <= m + slack))) return;
          if (late) ok = warp_wait(smem_addr(&sm.pv_part[h]), j & 1, gave_up, a.wait_limit_ns);
          fence_after();
          const float next = max3(m, m, top);
          const float g = m == kNegInf ? 0.0f : exp2_approx(m - next);
          m = next;
          l *= g;
          if (j == 0 && !late) return;
          // the products issued so far are complete: this step's scores came
          // after those of the steps before
#pragma unroll 1
          for (int c = 0; c < kDim; c += 8) {
            uint32_t o[8];
            ld8(to + c, o);
            asm volatile("tcgen05.wait::ld.sync.aligned;"
                         : "+r"(o[0]), "+r"(o[1]), "+r"(o[2]), "+r"(o[3]), "+r"(o[4]), "+r"(o[5]),
                           "+r"(o[6]), "+r"(o[7])::"memory");
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * g);
            st8(to + c, o);
          }
        };
        auto hand_over = [&](uint64_t* bar) {
          st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(smem_addr(bar));
        };
        ld32(ts, s0_);
        ld32(ts + 32, s1_);
        ld32(ts + 64, s2_);
        ld_wait<32>(s0_);
        ld_wait<32>(s1_);
        ld_wait<32>(s2_);
        if (masked) {
          hide(s0_, key0);
          hide(s1_, key0 + 32);
          hide(s2_, key0 + 64);
        }
        // The first 96 keys' weights go to the tensor pipe while the last 32 are
        // worked on.  Their maximum only moves the row's own with the next
        // step's, unless fp16 weights could overflow: the product of the first
        // 96 is under way by then.
        raise(max3(pending, maximum(s0_, 0), max3(maximum(s1_, 1), maximum(s2_, 2), kNegInf)), kLazy,
              false);
        base = m == kNegInf ? 0.0f : m;
        weights(s0_, 0);
        ld32(ts + 96, s0_);
        weights(s1_, 1);
        weights(s2_, 2);
        hand_over(&sm.p_part[h]);
        ld_wait<32>(s0_);
        if (masked) hide(s0_, key0 + 96);
        pending = maximum(s0_, 3);
        raise(pending, kJump, true);
        if (!ok) break;
        base = m == kNegInf ? 0.0f : m;
        weights(s0_, 3);
        hand_over(&sm.p_full[h]);
      }
      // The q tile becomes the stage of out, and at head size 128 a warp's part of
      // it lies on q rows that other warps wrote: not before all have.  The last
      // product comes after that; without steps the q tile itself is waited for.
      if (ok && !warp_wait(smem_addr(n_steps > 0 ? &sm.o_full[h] : &sm.q_full), 0, gave_up,
                           a.wait_limit_ns))
        ok = false;
      if (!ok) {
        *gave_up = 1;
        if (lane == 0) atomicOr(a.err, kDevErrTimeout);
        st_wait();  // of the step that was left
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
      // The rows of out through the half's q tile, which its products are done
      // with; parts of split tiles lie so that lanes write next to each other.
      constexpr int kRowBytes = kDim * 2;
      uint8_t* stage = sq + h * kTile + (warp & 3) * 32 * kRowBytes;
#pragma unroll 1
      for (int c = 0; c < kDim; c += 32) {
        uint32_t o[32];
        if (ok && n_steps > 0) {
          ld32(to + c, o);
          ld_wait<32>(o);
        }
        // a row that sees nothing is zero; a NaN sum stays
        if (!ok || n_steps == 0 || l == 0.0f) {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (u.part >= 0) {
          if (!mine) continue;
          float4* dst = reinterpret_cast<float4*>(part_rows<kTileRows>(a, u.part)) + tid;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[(c / 4 + k) * kTileRows] =
                make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                            __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at_chunk = c / 8 + k;
            *reinterpret_cast<uint4*>(stage + lane * kRowBytes +
                                      ((at_chunk & ~7) | ((at_chunk ^ lane) & 7)) * 16) =
                bf16x8(o + 8 * k, by);
          }
        }
      }
      if (u.part < 0) {
        const __nv_bfloat16* dst = static_cast<const __nv_bfloat16*>(a.out) +
                                   (qs.first + i) * a.out_token + (int64_t)qh * a.out_head;
        __syncwarp();
#pragma unroll
        for (int t = 0; t < kRowLanes; ++t) {
          const int from = t * kRowsAtOnce + lane / kRowLanes;
          const uint64_t to_row = __shfl_sync(0xFFFFFFFFu, (uint64_t)dst, from);
          const bool live = __shfl_sync(0xFFFFFFFFu, (int)mine, from);
          if (live)
            reinterpret_cast<uint4*>(to_row)[chunk] = *reinterpret_cast<const uint4*>(
                stage + from * kRowBytes + ((chunk & ~7) | ((chunk ^ from) & 7)) * 16);
        }
      }
      if (a.lse && mine && u.part < 0)
        a.lse[(qs.first + i) * a.q_heads + qh] =
            l == 0.0f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------- converters
    constexpr int kLanesRow = kDim / 16;             // lanes per key
    constexpr int kRowsLoad = kLoadWarps * 32 / kLanesRow;  // keys per load of the warps
    constexpr int kLoads = kKeys / kRowsLoad;
    const int w = warp - kLoadWarp;
    // The eight lanes of a shared-memory store phase write eight different
    // 16-byte chunks of 128 (chunk 2 col, + 1, xor row): four columns of two
    // rows.  The lanes' columns 4..7 go to the upper half of the warp.
    const int row = w * (32 / kLanesRow) + (kDim == 128 ? (lane >> 2) & 3 : lane >> 2);
    const int col = (lane & 3) + (kDim == 128 ? (lane >> 4) * 4 : 0);
    bool ok = true;
    for (int n = 0; n < 2 * n_steps; ++n) {
      const int slot = n % kSlots, from = n % kRaw, j = n >> 1;
      ok = warp_wait(smem_addr(&sm.kv_empty[slot]), ((n / kSlots) & 1) ^ 1, gave_up, a.wait_limit_ns) &&
           warp_wait(smem_addr(&sm.raw_full[from]), (n / kRaw) & 1, gave_up, a.wait_limit_ns);
      if (!ok) break;
      const uint8_t* codes = raw + from * (kTile / 2) + row * kDim + col * 16;
      uint4 x[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        x[k] = *reinterpret_cast<const uint4*>(codes + k * kRowsLoad * kDim);
      if (!sm.whole[j % kInfo]) {
        // codes that no row of the tile sees, or that were not copied, may be
        // anything, NaN among it
        const int key0 = step_at(steps, s0 + j) * kKeys;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int in = k * kRowsLoad + row, key = key0 + in;
          const bool want = sm.info[j % kInfo][in >> 5].y != kNegInf &&
                            ((key >= first.lo && key < last.hi) || key < last.sink);
          if (!want) x[k] = make_uint4(0, 0, 0, 0);
        }
      }
      uint8_t* to = ring + slot * kTile + (col >> 2) * kBlock;
      const int chunk = (2 * col) & 7;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const uint32_t y[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        uint32_t f[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          f[2 * t] = e4m3x2_f16x2(y[t] & 0xFFFFu);
          f[2 * t + 1] = e4m3x2_f16x2(y[t] >> 16);
        }
        const int at = k * kRowsLoad + row;
        *reinterpret_cast<uint4*>(to + chunk_at(at, chunk)) = make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(to + chunk_at(at, chunk + 1)) = make_uint4(f[4], f[5], f[6], f[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(smem_addr(&sm.raw_empty[from]));
        bar_arrive(smem_addr(&sm.kv_full[slot]));
      }
    }
    if (!ok) {
      *gave_up = 1;
      if (lane == 0) atomicOr(a.err, kDevErrTimeout);
    }
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------------ copies
    const int pieces = 1 << step_log, group = 32 >> step_log;  // pages per step, steps per look-up
    const uint32_t piece_bytes = (uint32_t)pt * kDim;
    // Each lane holds one of the next 32 pages and its scales; the following
    // ones are on the way, the scales a step after the pages: a look-up is two
    // dependent loads from memory, longer than a step.
    int looked = s0, page = kNoPage;  // kNoPage: nothing to copy
    float ks = 0.0f, vs = -1.0f, next_ks = 0.0f, next_vs = -1.0f;
    auto check_page = [&]() {
      if (next_page != kNoPage && (next_page < 0 || next_page >= a.c.pages)) {
        atomicOr(a.err, kDevErrShape);
        next_page = kNoPage;
      }
    };
    auto fetch_scales = [&]() {
      check_page();
      next_ks = 0.0f;
      next_vs = -1.0f;
      if (next_page >= 0) {
        next_ks = a.c.scales[0][(int64_t)next_page * a.c.heads + unit.head];
        next_vs = a.c.scales[1][(int64_t)next_page * a.c.heads + unit.head];
      }
    };
    bool ok = true;
    int n = 0;
    for (int j = 0; j < n_steps && ok; ++j) {
      if (j == 0) {
        check_page();
        page = next_page;
      } else if (s0 + j == looked + group) {
        looked = s0 + j;
        page = next_page;
        ks = next_ks;
        vs = next_vs;
        next_page = fetch_page(looked + group);
      } else if (s0 + j == looked + 1) {
        fetch_scales();
      }
      const int base = (s0 + j - looked) << step_log;
      const bool mine = lane >= base && lane < base + pieces;
      const uint32_t here = __ballot_sync(0xFFFFFFFFu, mine && page >= 0);
      for (int which = 0; which < 2; ++which, ++n) {
        const int to = n % kRaw;
        ok = warp_wait(smem_addr(&sm.raw_empty[to]), ((n / kRaw) & 1) ^ 1, gave_up, a.wait_limit_ns);
        if (!ok) break;
        const uint32_t full = smem_addr(&sm.raw_full[to]);
        // (the bytes may be counted down before they are announced: the phase
        // ends with the arrival below at the earliest)
        if (mine && page >= 0)
          bulk_copy(smem_addr(raw) + to * (kTile / 2) + (lane - base) * piece_bytes,
                    a.c.codes[which] + ((int64_t)page * a.c.heads + unit.head) * piece_bytes,
                    piece_bytes, full);
        if (which == 0) {
          if (j == 0) {
            fetch_scales();
            ks = next_ks;
            vs = next_vs;
            next_page = fetch_page(looked + group);
          }
          // the scales of the step's four groups of 32 keys
          const int from = base + ((lane & 3) * 32 >> pt_log);
          const float k1 = __shfl_sync(0xFFFFFFFFu, ks, from), v1 = __shfl_sync(0xFFFFFFFFu, vs, from);
          if (lane < 4) {
            // an absent page: its keys' scores become -inf
            const float lv = v1 < 0.0f ? kNegInf : (float)((int)(__float_as_uint(v1) >> 23) - 127);
            sm.info[j % kInfo][lane] = make_float4(k1, lv, v1 < 0.0f ? 0.0f : 1.0f / v1, 0.0f);
          }
          if (lane == 0) {
            const int key0 = step_at(steps, s0 + j) * kKeys;
            sm.whole[j % kInfo] =
                __popc(here) == pieces &&
                ((key0 >= first.lo && key0 + kKeys <= last.hi) || key0 + kKeys <= last.sink);
          }
        }
        __syncwarp();
        if (lane == 0) bar_expect(full, __popc(here) * piece_bytes);
      }
    }
    if (!ok) {
      *gave_up = 1;
      if (lane == 0) atomicOr(a.err, kDevErrTimeout);
    }
    // no copy may land after the CTA is gone
    for (int i = max(0, n - kRaw); i < n; ++i)
      bar_wait(smem_addr(&sm.raw_full[i % kRaw]), (i / kRaw) & 1, nullptr, 200000000ull);
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
      // O of half h += P V over keys 16 k0 .. 16 k1 of the V tile n
      auto output = [&](int h, int n, int k0, int k1, bool first_step) {
        const uint32_t vb = operand(ring_at + (n % kSlots) * kTile, kBlock);
#pragma unroll
        for (int k = k0; k < k1; ++k)
          mma_ts(tmem + col_o(h), tmem + col_s(h) + 8 * k, vb + (uint32_t)(k * (2048 >> 4)), kInstrO,
                 !first_step || k > 0, lead);
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
              !warp_wait(smem_addr(&sm.p_part[h]), j & 1, gave_up, a.wait_limit_ns)) {
            ok = false;
            break;
          }
          fence_after();
          output(h, nv, 0, 6, j == 0);
          commit(smem_addr(&sm.pv_part[h]), lead);
          if (!warp_wait(smem_addr(&sm.p_full[h]), j & 1, gave_up, a.wait_limit_ns)) {
            ok = false;
            break;
          }
          fence_after();
          output(h, nv, 6, 8, false);
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

// (The caller has checked that the tiles of all sequences fit 30 bits.)
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
