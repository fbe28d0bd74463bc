// Attention of few query rows over the 8-bit paged cache, and the kernel that
// joins partial results.
//
// One CTA takes 8 or 16 rows (the queries of one sequence times the query heads
// of one KV head) and a run of steps of 16 KB of codes (64 keys of 128 elements,
// 128 of 64).  What bounds it: the cache's bytes, read once: 2 dim bytes per key
// and KV head.  So
//   * a producer warp keeps a ring of steps in flight with untiled bulk copies
//     -- the codes of a page and head are one contiguous block, so a step is
//     one or two copies each of K and V -- and looks 32 pages ahead in the
//     page table;
//   * four warps each take 16 or 32 keys of a step with their own running
//     maximum and sum and join once at the end;
//   * the products run on mma.sync m16n8k16 in fp16 with the keys, not the
//     queries, along the 16: S^T = K Q^T and O^T = V^T P^T.  Eight rows fill an
//     instruction's 8 columns, so one token's grouped heads waste little, and
//     the accumulators of 8 rows take 32 registers.  The weights turn from one
//     layout to the other with movmatrix.  The order of k inside a product is
//     free as long as both operands agree, so a thread takes its K fragment as
//     dim / 4 consecutive bytes of a key, and its V fragment as dim / 8
//     consecutive bytes of four keys: vector loads from shared memory and one
//     conversion per pair of codes, no transposition.  So few rows are far from
//     a tcgen05 tile of 128, and the tensor pipe is not what bounds it;
//   * a row's maximum is only looked for when a score exceeds the old one by
//     2^kLazy (one vote per step), its sum only added up at the end.
// The steps of a tile of rows are cut into runs, a CTA each.
//   * While all CTAs fit the GPU at once: even shares of what the tile sees, so
//     that wide page tables, windows and ragged batches still fill it.  At most
//     eight short runs are one cluster, which joins its sums through distributed
//     shared memory; more or longer ones are joined by a second kernel.  One
//     token of 24 heads of 128, us with the cluster / the kernel: 1561 tokens
//     8.8 / 11.3, 3000 10.1 / 12.3, 6000 15.2 / 16.6, 12000 (24 steps a run)
//     23.5 / 23.4.
//   * Beyond: runs of fixed length; those past a sequence's end return at once.
//     Even shares there start more CTAs for the same work (32 sequences, 8 heads
//     of 128: 193 us in shares of at least 16 steps, 184 in runs of 64).
// Measured (device time): 32 sequences of 800..32760 tokens, 8 KV heads of 128,
// 4 query heads each: 183 us, 6.0 TB/s.  8 sequences of 4100..8200 tokens, 4 KV
// heads of 64, 30 rows each: 19.7 us, of which the bytes are 4: a warp's chain
// of conversions, products and softmax, three CTAs an SM.  With 64 keys a step 3
// us more, with a branch per masked key or 32 rows a CTA (half the conversions,
// two CTAs an SM) 3 and 9 more.
#include "attention_common.cuh"
#include "kernels.h"

namespace nvfp4 {

namespace {

constexpr int kDepth = 4;     // steps in flight
constexpr int kWarps = 4;     // consumer warps
// Groups of 16 keys that a warp takes of a step, and keys of a step: 16 KB of
// codes at either head size.
__host__ __device__ constexpr int groups_of(int dim) { return 128 / dim; }
__host__ __device__ constexpr int step_keys(int dim) { return kWarps * 16 * groups_of(dim); }
// A CTA's start costs as much as several steps.
constexpr int kLeastRun = 2, kWaveRun = 32;  // of a CTA, in steps of 64 keys
constexpr int kMaxCluster = 8, kClusterRun = 12;  // CTAs; steps of each
constexpr int kRowThreads = (kWarps + 1) * 32;

struct RowsPlan {
  int rows;       // of a tile, 8 or 16
  int row_tiles;  // tiles per sequence and KV head
  int splits;     // runs of keys
  int run;        // steps per run; 0: the tile's steps in even shares
  int cluster;    // the runs of a tile are one cluster, which joins them itself
};

__device__ __forceinline__ void mma_f16(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements held two per lane.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Stores four elements of row `row` of a KV head's rows, and with the first
// four its log-sum-exp.
__device__ __forceinline__ void store_row4(const Kv8Attention& a, const QuerySeq& q, int row,
                                           int head, int d0, float4 acc, float top, float sum) {
  const int i = row / a.group, qh = head * a.group + row - i * a.group;
  // a row that sees nothing has sum 0: zeros (a NaN sum stays)
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * f, acc.y * f);
  const __nv_bfloat162 y = __floats2bfloat162_rn(acc.z * f, acc.w * f);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (q.first + i) * a.out_token +
                            (int64_t)qh * a.out_head + d0) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  if (a.lse && d0 == 0)
    a.lse[(q.first + i) * a.q_heads + qh] =
        sum == 0.0f ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
}

template <int kDim>
struct RowsSmem {
  uint8_t k[kDepth][step_keys(kDim) * kDim];
  uint8_t v[kDepth][step_keys(kDim) * kDim];
  float2 scale[kDepth][step_keys(kDim) / 32];  // (ks, vs) of each 32 keys; vs < 0: the page is absent
  uint64_t full[kDepth], empty[kDepth];
  float2 stats[kWarps][16];
  float2 joined[16];  // of the CTA's run
  int gave_up;
};

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same place in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t smem_of(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 load_of2(uint32_t addr) {
  float2 x;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ float4 load_of4(uint32_t addr) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}

// CTAs of an SM, by registers and shared memory.
__host__ __device__ constexpr int ctas_per_sm(int dim, int tiles) {
  return (tiles == 1 ? 3 : 2) + (dim == 64);
}

// Joins the runs of a tile of rows in the order of the keys, each CTA of the
// cluster a share of the rows' elements.  `sums` holds a run's [rows][dim].
template <int kDim, int kRowsCta>
__device__ __forceinline__ void join_cluster(const Kv8Attention& a, const QuerySeq& q, int splits,
                                             int rank, const float* sums, const float2* joined,
                                             int row0, int rows, int head) {
  const uint32_t from = smem_addr(sums), stats = smem_addr(joined);
  for (int u = rank * kWarps * 32 + threadIdx.x; u < kRowsCta * kDim / 4; u += splits * kWarps * 32) {
    const int r = u / (kDim / 4), d0 = u % (kDim / 4) * 4;
    if (row0 + r >= rows) break;
    float2 st[kMaxCluster];
    float4 x[kMaxCluster];
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      st[s] = make_float2(kNegInf, 0.0f);
      if (s >= splits) continue;
      st[s] = load_of2(smem_of(stats + r * 8, s));
      x[s] = load_of4(smem_of(from + u * 16, s));
    }
    float top = kNegInf;
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) top = fmaxf(top, st[s].x);
    float sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      // a run that saw nothing may not have written its sums; a NaN sum counts
      if (st[s].x == kNegInf && st[s].y == 0.0f) continue;
      const float f = st[s].x == kNegInf ? 1.0f : exp2_approx(st[s].x - top);
      sum = fmaf(st[s].y, f, sum);
      acc.x = fmaf(x[s].x, f, acc.x), acc.y = fmaf(x[s].y, f, acc.y);
      acc.z = fmaf(x[s].z, f, acc.z), acc.w = fmaf(x[s].w, f, acc.w);
    }
    store_row4(a, q, row0 + r, head, d0, acc, top, sum);
  }
}

// kTiles tiles of 8 rows.
template <int kDim, int kTiles>
__global__ void __launch_bounds__(kRowThreads, ctas_per_sm(kDim, kTiles))
    attend_rows_kernel(const __grid_constant__ Kv8Attention a, const RowsPlan plan) {
  constexpr int kRowsCta = 8 * kTiles;
  constexpr int kStepKeys = step_keys(kDim), kGroups = groups_of(kDim);
  extern __shared__ __align__(128) uint8_t smem_raw[];
  RowsSmem<kDim>& sm = *reinterpret_cast<RowsSmem<kDim>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, head = blockIdx.y / plan.row_tiles;
  const int tile = blockIdx.y - head * plan.row_tiles, seq = blockIdx.z;
  const int pt = a.c.page_tokens;

  QuerySeq q;
  if (!load_query_seq(a.b, pt, seq, q)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.err, kDevErrShape);
    return;
  }
  const int row0 = tile * kRowsCta, rows = q.n * a.group;
  if (row0 >= rows) return;
  const Steps steps = steps_of<kStepKeys>(a, q, row0 / a.group,
                                          (min(row0 + kRowsCta, rows) - 1) / a.group);
  const int run = plan.run ? plan.run
                           : max((steps.total + plan.splits - 1) / plan.splits, kLeastRun / kGroups);
  const int s0 = min(split * run, steps.total), s1 = min(s0 + run, steps.total);
  const int64_t parts = (int64_t)gridDim.x * gridDim.y * gridDim.z;
  const int64_t part = ((int64_t)seq * gridDim.y + blockIdx.y) * gridDim.x + split;
  if (s0 == s1 && plan.splits > 1) {
    // nothing in this run: what joins the runs skips it
    if (threadIdx.x < kRowsCta) {
      const float2 none = make_float2(kNegInf, 0.0f);
      if (plan.cluster) sm.joined[threadIdx.x] = none;
      else part_stats<kRowsCta>(a, parts, part)[threadIdx.x] = none;
    }
    if (plan.cluster) {
      if (warp == kWarps) return;
      cluster_sync();
      join_cluster<kDim, kRowsCta>(a, q, plan.splits, split, reinterpret_cast<float*>(smem_raw),
                                   sm.joined, row0, rows, head);
      cluster_sync();
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDepth; ++i) {
      bar_init(smem_addr(&sm.full[i]), i == 0 ? 1 + a.stall : 1);
      bar_init(smem_addr(&sm.empty[i]), kWarps);
    }
    sm.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------- producer
    const int pieces = pt < kStepKeys ? kStepKeys / pt : 1;  // copies per step
    const int piece_keys = kStepKeys / pieces;
    const uint32_t piece_bytes = piece_keys * kDim;
    const int per_piece = piece_keys / 32;
    const Seen first = seen_by(a, q, row0 / a.group);
    const Seen last = seen_by(a, q, (min(row0 + kRowsCta, rows) - 1) / a.group);
    bool ok = true;
    int issued = 0;
    for (int i0 = s0; i0 < s1 && ok; i0 += 32 / pieces) {
      // each lane: the page and scales of one coming piece
      const int mine = i0 + lane / pieces;
      int64_t page = -1;
      float ks = 0.0f, vs = -1.0f;
      if (mine < s1) {
        const int key = step_at(steps, mine) * kStepKeys + (lane % pieces) * piece_keys;
        // pages of keys that no row sees are not looked up: past the sequence's
        // end, or out of the window, they may be gone
        if (any_seen(first, last, key, key + piece_keys)) {
          page = a.b.table[seq * a.b.table_stride + key / pt];
          if (page < 0 || page >= a.c.pages) {
            atomicOr(a.err, kDevErrShape);
            page = -1;
          } else {
            ks = a.c.scales[0][page * a.c.heads + head];
            vs = a.c.scales[1][page * a.c.heads + head];
          }
        }
      }
      for (int i = i0; i < min(s1, i0 + 32 / pieces); ++i, ++issued) {
        const int st = issued % kDepth;
        if (lane == 0 && !bar_wait(smem_addr(&sm.empty[st]), ((issued / kDepth) & 1) ^ 1,
                                   &sm.gave_up, a.wait_limit_ns))
          ok = false;
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
        const int from = (i - i0) * pieces;
        const bool mine_now = lane >= from && lane < from + pieces;
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, mine_now && page >= 0);
        const uint32_t full = smem_addr(&sm.full[st]);
        if (mine_now) {
          const int p = lane - from;
          const float2 sc = make_float2(ks, vs);
          for (int k = 0; k < per_piece; ++k) sm.scale[st][p * per_piece + k] = sc;
        }
        __syncwarp();
        if (lane == 0) bar_expect(full, __popc(here) * 2 * piece_bytes);
        __syncwarp();
        if (mine_now && page >= 0) {
          const int p = lane - from;
          const int key = step_at(steps, i) * kStepKeys + p * piece_keys;
          const int64_t off = ((page * a.c.heads + head) * pt + key % pt) * kDim;
          bulk_copy(smem_addr(sm.k[st]) + p * piece_bytes, a.c.codes[0] + off, piece_bytes, full);
          bulk_copy(smem_addr(sm.v[st]) + p * piece_bytes, a.c.codes[1] + off, piece_bytes, full);
        }
        __syncwarp();
      }
    }
    if (!ok) {
      if (lane == 0) {
        *(volatile int*)&sm.gave_up = 1;
        atomicOr(a.err, kDevErrTimeout);
      }
    }
    // no copy may land after the CTA is gone
    for (int j = max(0, issued - kDepth); j < issued; ++j)
      bar_wait(smem_addr(&sm.full[j % kDepth]), (j / kDepth) & 1, nullptr, 200000000ull);
    return;
  }

  // --------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  constexpr int kPer = kDim / 4;  // elements of a row per thread
  // B fragments of row 8 n + g: k-step s holds elements c * kPer + 4 s + {0..3}
  uint32_t qf[kTiles][kDim / 16][2];
  // of rows 8 n + 2 c and + 1, as the scores lie
  float crow[kTiles][2], m[kTiles][2], l[kTiles][2];
  int at[kTiles][2];  // the query's place in its sequence
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
    const int r = row0 + 8 * n + g;
    const bool live = r < rows;
    const int i = live ? r / a.group : (rows - 1) / a.group;
    const __nv_bfloat16* src =
        static_cast<const __nv_bfloat16*>(a.q) + (q.first + i) * a.q_token +
        (int64_t)(head * a.group + (live ? r - i * a.group : 0)) * a.q_head + c * kPer;
    uint32_t w[kPer / 2];
#pragma unroll
    for (int j = 0; j < kPer / 8; ++j) {
      const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(src) + j) : make_uint4(0, 0, 0, 0);
      w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
    }
    uint32_t big = 0;
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j)
      big = max(big, max((w[j] << 16) & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
    big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
    big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
    const int e = big ? row_exponent(__uint_as_float(big)) : 0;
    const float down = pow2(-e), up = a.scale_log2 * pow2(e);
#pragma unroll
    for (int s = 0; s < kDim / 16; ++s)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t x = w[2 * s + p];
        qf[n][s][p] =
            f16x2(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xFFFF0000u) * down);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      crow[n][h] = __shfl_sync(0xFFFFFFFFu, up, (2 * c + h) * 4);
      at[n][h] = q.len - q.n + __shfl_sync(0xFFFFFFFFu, i, (2 * c + h) * 4);
      m[n][h] = kNegInf;
      l[n][h] = 0.0f;
    }
  }
  // O^T: fragment t holds elements g * kDim / 8 + 2 t (and + 1) of rows 2 c, 2 c + 1
  float o[kTiles][kDim / 16][4];
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int t = 0; t < kDim / 16; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][t][j] = 0.0f;
  // what any row of the tile sees, and what all do
  const Seen first = seen_by(a, q, row0 / a.group);
  const Seen last = seen_by(a, q, (min(row0 + kRowsCta, rows) - 1) / a.group);

  bool ok = true;
  for (int i = s0; i < s1; ++i) {
    const int st = (i - s0) % kDepth;
    if (!warp_wait(smem_addr(&sm.full[st]), ((i - s0) / kDepth) & 1, &sm.gave_up, a.wait_limit_ns)) {
      ok = false;
      break;
    }
    const int in0 = warp * 16 * kGroups;  // this warp's keys
    const int key0 = step_at(steps, i) * kStepKeys + in0;
    const float2 sc = sm.scale[st][in0 >> 5];
    const bool absent = sc.y < 0.0f;
    // scores of keys key0 + 16 u + g and + 8 for rows 2 c, 2 c + 1
    float s[kGroups][kTiles][4];
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.0f;
      const uint8_t* kr = sm.k[st] + (in0 + 16 * u + g) * kDim + c * kPer;
#pragma unroll
      for (int j = 0; j < kPer / 16; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(kr + 16 * j);
        const uint4 y = *reinterpret_cast<const uint4*>(kr + 8 * kDim + 16 * j);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w}, z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t af[4] = {e4m3x2_f16x2(w[k] & 0xFFFFu), e4m3x2_f16x2(z[k] & 0xFFFFu),
                                  e4m3x2_f16x2(w[k] >> 16), e4m3x2_f16x2(z[k] >> 16)};
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
            mma_f16(s[u][n], af, qf[n][4 * j + k][0], qf[n][4 * j + k][1]);
        }
      }
    }
    // V of keys 2 c, 2 c + 1 (and + 8), bytes g * kDim / 8 of each
    constexpr int kVWords = kDim / 32;
    uint32_t v[kGroups][4][kVWords];
    const int end = key0 + 16 * kGroups;
    const bool whole = !absent && ((key0 >= first.lo && end <= last.hi) || end <= last.sink);
#pragma unroll
    for (int u = 0; u < kGroups; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int in = 16 * u + 2 * c + (k & 1) + 8 * (k >> 1);
        const uint8_t* vr = sm.v[st] + (in0 + in) * kDim + g * (kDim / 8);
        if constexpr (kVWords == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(vr);
          v[u][k][0] = x.x, v[u][k][1] = x.y, v[u][k][2] = x.z, v[u][k][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(vr);
          v[u][k][0] = x.x, v[u][k][1] = x.y;
        }
      }
    // codes that no row sees, past the sequence's end above all, may be
    // anything, NaN among it, and 0 * NaN is not 0
    if (!whole) {
#pragma unroll
      for (int u = 0; u < kGroups; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = key0 + 16 * u + 2 * c + (k & 1) + 8 * (k >> 1);
          if (absent || !((key >= first.lo && key < last.hi) || key < last.sink)) {
#pragma unroll
            for (int w = 0; w < kVWords; ++w) v[u][k][w] = 0u;
          }
        }
    }
    // the step's bytes are in registers: its slot may refill
    __syncwarp();
    if (lane == 0) bar_arrive(smem_addr(&sm.empty[st]));

    const float lv = absent ? 0.0f : (float)((int)(__float_as_uint(sc.y) >> 23) - 127);
    const bool all_see = !absent && key0 >= last.lo && end <= first.hi;
    bool higher = false;
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f = crow[n][h] * sc.x;
#pragma unroll
        for (int u = 0; u < kGroups; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float& x = s[u][n][2 * j + h];
            x = fmaf(x, f, lv);
          }
      }
    if (!all_see) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const Seen see = seen_at(a, q.len, at[n][h]);
#pragma unroll
          for (int u = 0; u < kGroups; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int key = key0 + 16 * u + g + 8 * j;
              if (absent || !((key >= see.lo && key < see.hi) || key < see.sink))
                s[u][n][2 * j + h] = kNegInf;
            }
        }
    }
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = s[0][n][h];
#pragma unroll
        for (int u = 0; u < kGroups; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j) top = fmaxf(top, s[u][n][2 * j + h]);
        higher |= top > m[n][h] + kLazy;
      }
    if (__any_sync(0xFFFFFFFFu, higher)) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float next = m[n][h];
#pragma unroll
          for (int u = 0; u < kGroups; ++u) next = fmaxf(next, fmaxf(s[u][n][h], s[u][n][2 + h]));
          next = fmaxf(next, __shfl_xor_sync(0xFFFFFFFFu, next, 4));
          next = fmaxf(next, __shfl_xor_sync(0xFFFFFFFFu, next, 8));
          next = fmaxf(next, __shfl_xor_sync(0xFFFFFFFFu, next, 16));
          // a row that has seen nothing yet keeps -inf; nothing to rescale
          const float f = m[n][h] == kNegInf ? 0.0f : exp2_approx(m[n][h] - next);
          m[n][h] = next;
          l[n][h] *= f;
#pragma unroll
          for (int t = 0; t < kDim / 16; ++t) o[n][t][h] *= f, o[n][t][2 + h] *= f;
        }
    }
    const float inv = absent ? 0.0f : 1.0f / sc.y;
    uint32_t pf[kGroups][kTiles][2];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const float base[2] = {m[n][0] == kNegInf ? 0.0f : m[n][0],
                             m[n][1] == kNegInf ? 0.0f : m[n][1]};
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        float p[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          p[h] = exp2_approx(s[u][n][h] - base[h]);
          p[2 + h] = exp2_approx(s[u][n][2 + h] - base[h]);
          l[n][h] = fmaf(p[h] + p[2 + h], inv, l[n][h]);
        }
        // (to fp16: see attention_common.cuh; the sum above is of the fp32 weights)
        pf[u][n][0] = transposed(f16x2(p[0], p[1]));
        pf[u][n][1] = transposed(f16x2(p[2], p[3]));
      }
    }
#pragma unroll
    for (int u = 0; u < kGroups; ++u)
#pragma unroll
      for (int w = 0; w < kVWords; ++w) {
        const uint32_t a0 = __byte_perm(v[u][0][w], v[u][1][w], 0x5140);
        const uint32_t a1 = __byte_perm(v[u][0][w], v[u][1][w], 0x7362);
        const uint32_t b0 = __byte_perm(v[u][2][w], v[u][3][w], 0x5140);
        const uint32_t b1 = __byte_perm(v[u][2][w], v[u][3][w], 0x7362);
        const uint32_t f0[4] = {e4m3x2_f16x2(a0 & 0xFFFFu), e4m3x2_f16x2(a0 >> 16),
                                e4m3x2_f16x2(b0 & 0xFFFFu), e4m3x2_f16x2(b0 >> 16)};
        const uint32_t f1[4] = {e4m3x2_f16x2(a1 & 0xFFFFu), e4m3x2_f16x2(a1 >> 16),
                                e4m3x2_f16x2(b1 & 0xFFFFu), e4m3x2_f16x2(b1 >> 16)};
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          mma_f16(o[n][2 * w], f0, pf[u][n][0], pf[u][n][1]);
          mma_f16(o[n][2 * w + 1], f1, pf[u][n][0], pf[u][n][1]);
        }
      }
  }
  if (!ok && lane == 0) {
    *(volatile int*)&sm.gave_up = 1;
    atomicOr(a.err, kDevErrTimeout);
  }

  // ------------------------------------------------- join the four warps
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[n][h] += __shfl_xor_sync(0xFFFFFFFFu, l[n][h], 4);
      l[n][h] += __shfl_xor_sync(0xFFFFFFFFu, l[n][h], 8);
      l[n][h] += __shfl_xor_sync(0xFFFFFFFFu, l[n][h], 16);
      if (g == 0) sm.stats[warp][8 * n + 2 * c + h] = make_float2(m[n][h], l[n][h]);
    }
  // all consumer warps are done with the ring
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
  float* sums = reinterpret_cast<float*>(smem_raw);  // [kWarps][rows][kDim], in the ring's place
  static_assert(sizeof(float) * kWarps * kRowsCta * kDim <= sizeof(sm.k) + sizeof(sm.v), "fits");
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float* dst = sums + (warp * kRowsCta + 8 * n + 2 * c + h) * kDim + g * (kDim / 8);
#pragma unroll
      for (int t = 0; t < kDim / 16; t += 2)
        *reinterpret_cast<float4*>(dst + 2 * t) =
            make_float4(o[n][t][h], o[n][t][2 + h], o[n][t + 1][h], o[n][t + 1][2 + h]);
    }
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
  constexpr int kThreadsRow = 16 / kTiles, kOut = kDim / kThreadsRow;  // threads per row, elements each
  const int r = threadIdx.x / kThreadsRow, part_of = threadIdx.x % kThreadsRow, d0 = part_of * kOut;
  float top = kNegInf;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.stats[w][r].x);
  float sum = 0.0f, acc[kOut];
#pragma unroll
  for (int t = 0; t < kOut; ++t) acc[t] = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float2 st = sm.stats[w][r];
    const float f = st.x == kNegInf ? 0.0f : exp2_approx(st.x - top);
    sum = fmaf(st.y, f, sum);
    const float* src = sums + (w * kRowsCta + r) * kDim + d0;
#pragma unroll
    for (int t = 0; t < kOut; t += 4) {
      const float4 x = *reinterpret_cast<const float4*>(src + t);
      acc[t] = fmaf(x.x, f, acc[t]), acc[t + 1] = fmaf(x.y, f, acc[t + 1]);
      acc[t + 2] = fmaf(x.z, f, acc[t + 2]), acc[t + 3] = fmaf(x.w, f, acc[t + 3]);
    }
  }
  if (plan.splits > 1 && plan.cluster) {
    // in the place of the first warp's, which only this thread reads
    float* dst = sums + r * kDim + d0;
#pragma unroll
    for (int t = 0; t < kOut; t += 4)
      *reinterpret_cast<float4*>(dst + t) = make_float4(acc[t], acc[t + 1], acc[t + 2], acc[t + 3]);
    if (part_of == 0) sm.joined[r] = make_float2(top, sum);
    cluster_sync();
    join_cluster<kDim, kRowsCta>(a, q, plan.splits, split, sums, sm.joined, row0, rows, head);
    cluster_sync();  // no CTA leaves while others read its sums
    return;
  }
  if (row0 + r >= rows) return;
  if (plan.splits > 1) {
    float* dst = part_rows<kRowsCta>(a, part) + r * kDim + d0;
#pragma unroll
    for (int t = 0; t < kOut; t += 4)
      *reinterpret_cast<float4*>(dst + t) = make_float4(acc[t], acc[t + 1], acc[t + 2], acc[t + 3]);
    if (part_of == 0) part_stats<kRowsCta>(a, parts, part)[r] = make_float2(top, sum);
    return;
  }
#pragma unroll
  for (int t = 0; t < kOut; t += 4)
    store_row4(a, q, row0 + r, head, d0 + t,
               make_float4(acc[t], acc[t + 1], acc[t + 2], acc[t + 3]), top, sum);
}

// Joins the parts of the rows: one warp per row.
template <int kRows>
__global__ void __launch_bounds__(256)
    join_rows_kernel(const __grid_constant__ Kv8Attention a, const RowsPlan plan) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int seq = blockIdx.z, head = blockIdx.y;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  QuerySeq q;
  if (!load_query_seq(a.b, a.c.page_tokens, seq, q) || row >= q.n * a.group) return;
  const int64_t parts = (int64_t)plan.splits * plan.row_tiles * a.c.heads * gridDim.z;
  const int64_t part0 =
      ((int64_t)(seq * a.c.heads + head) * plan.row_tiles + row / kRows) * plan.splits;
  join_row<kRows>(a, q, parts, part0, plan.splits, row % kRows, row, head, threadIdx.x & 31);
}

RowsPlan plan_rows(int32_t heads, int32_t dim, int32_t group, int32_t n, int32_t max_rows,
                   int64_t max_len) {
  RowsPlan p;
  const int64_t rows = (int64_t)max_rows * group;
  p.rows = rows <= 8 ? 8 : 16;
  p.row_tiles = (int)((rows + p.rows - 1) / p.rows);
  const int64_t steps = (max_len + step_keys(dim) - 1) / step_keys(dim);
  const int64_t slots = (int64_t)ctas_per_sm(dim, p.rows / 8) * num_sms();
  const int64_t tiles = (int64_t)n * heads * p.row_tiles;
  const int64_t least = kLeastRun / groups_of(dim), wave = kWaveRun / groups_of(dim);
  int64_t splits = slots / tiles;
  if (splits * wave >= steps) {
    // all CTAs at once
    const int64_t most = (steps + least - 1) / least;
    if (splits > most) splits = most;
    p.cluster = kMaxCluster * kClusterRun >= steps;
    if (p.cluster && splits > kMaxCluster) splits = kMaxCluster;
    p.run = 0;
  } else {
    // about three waves at full length, since the sequences of a batch are
    // seldom all that long
    int64_t run = tiles * steps / (3 * slots);
    run = run < wave ? wave : (run > 2 * wave ? 2 * wave : run);
    splits = (steps + run - 1) / run;
    p.cluster = 0;
    p.run = (int)run;
  }
  p.splits = splits < 1 ? 1 : (int)splits;
  return p;
}

template <int kDim, int kTiles>
cudaError_t launch_rows(const Kv8Attention& a, const RowsPlan& p, cudaStream_t s) {
  constexpr int kSmem = (int)sizeof(RowsSmem<kDim>);
  cudaError_t e = cudaFuncSetAttribute(attend_rows_kernel<kDim, kTiles>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)p.splits, (unsigned)(a.c.heads * p.row_tiles), (unsigned)a.b.n);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster && p.splits > 1;
  e = cudaLaunchKernelEx(&cfg, attend_rows_kernel<kDim, kTiles>, a, p);
  if (e != cudaSuccess || p.splits == 1 || p.cluster) return e;
  cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)a.b.max_rows * a.group + 7) / 8), (unsigned)a.c.heads,
                     (unsigned)a.b.n);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_rows_kernel<8 * kTiles>, a, p);
}

}  // namespace

namespace {
// Whether tiles of 256 rows on the tensor pipe are faster than tiles of 16 rows
// that each read the cache.  Measured with rows of 6 heads (tiles of 256 / of 16
// rows, us): 8 sequences of 4100..8200 tokens and 4 KV heads, dim 64, 30 rows
// 38 / 20, 48 rows 38 / 28, 66 rows 38 / 46; dim 128, 30 rows 44 / 37, 48 rows
// 44 / 51.  32 sequences and 8 KV heads: dim 64, 48 rows 191 / 145, 66 rows 192
// / 221; dim 128, 30 rows 214 / 191, 48 rows 215 / 272.  So above three tiles of
// 16 rows at 64 and above two at 128.
inline bool many_rows(int32_t dim, int64_t max_rows, int32_t group) {
  return max_rows * group > 16 * (dim == 64 ? 3 : 2);
}
}  // namespace

size_t kv8_attention_partial_bytes(int32_t heads, int32_t dim, int32_t group, int32_t n,
                                   int32_t max_rows, int64_t max_len) {
  if (many_rows(dim, max_rows, group))
    return attend_tiles_partial_bytes(heads, dim, group, n, max_rows, max_len);
  const RowsPlan p = plan_rows(heads, dim, group, n, max_rows, max_len);
  if (p.splits == 1) return 0;
  return (size_t)n * heads * p.row_tiles * p.splits * p.rows * ((size_t)dim * 4 + 8);
}

cudaError_t launch_kv8_attention(const Kv8Attention& a, cudaStream_t s) {
  if (many_rows(a.c.dim, a.b.max_rows, a.group)) return launch_attend_tiles(a, s);
  const RowsPlan p = plan_rows(a.c.heads, a.c.dim, a.group, a.b.n, a.b.max_rows,
                               (int64_t)a.b.table_pages * a.c.page_tokens);
  if (a.c.dim == 128)
    return p.rows == 8 ? launch_rows<128, 1>(a, p, s) : launch_rows<128, 2>(a, p, s);
  return p.rows == 8 ? launch_rows<64, 1>(a, p, s) : launch_rows<64, 2>(a, p, s);
}

}  // namespace nvfp4
