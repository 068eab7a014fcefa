// Attention weights received by the cached tokens, accumulated over steps:
//   w[r][j] = decay * w[r][j] + sum over query rows (i, h) that see j of
//             exp(scale * q_{i,h} . C_j - lse_{i,h})
// with the lse that the decode returned.
//
// Why tokens are the rows of the product.  The sum runs over query rows, so
// S^T = C . Q^T puts a token on a TMEM lane and the rows on its columns: the
// thread that owns the lane adds up exp2(S^T * scale' - lse') over its columns
// in registers, and nothing is exchanged or normalised (the lse is known).
//
// Why a CTA pair.  One MMA covers 256 tokens x up to 256 rows over the two
// SMs of a cluster (cta_group::2): each SM holds its 128 tokens and half of
// the rows, so a tile of rows costs each SM's shared memory half of what it
// would alone (9 chunks x 128 rows x 128 bytes = 144 KB for 256 rows) and a
// page is loaded once per 256 rows.  The rows of a tile stay in shared memory
// while the pair's tokens pass through a ring of 16 KB stages (one 128-byte
// column box of 128 tokens each), as deep as the rows leave room for.
//
// Roles (both CTAs; 384 threads): warp 0 streams pages and rows by TMA,
// signalling the pair's first CTA; warp 1 of the first CTA issues the MMAs
// into one of two TMEM accumulators; two warpgroups drain them, each half of
// the columns: one fused multiply-add, one exp2 and one add a score.  (One
// warpgroup alone could not hide its own TMEM, exp2 and memory latencies;
// two that take units in turn hold each accumulator twice as long.)
//
// Split.  The work is (request, 256-token unit, tile of rows).  Every pair
// counts the units from the lengths and takes an equal share, in the order
// (request, group of tiles, unit).  The tiles form one group, and a unit's
// weights stay with one thread, unless there are fewer than 4 units a pair
// and more groups shorten the longest pair's work (us in 1, 2, 4, 8 groups,
// 128 heads: 16 queries of 16 x 4096 tokens 129, 123, 128, 132; of 1 x 4096
// 44, 33, 26, 28; 5 queries of 6 x 6000 36, 41, 38, 37).  The groups' sums
// then go through the workspace, and the last group to finish a unit adds
// them in their order: no order of sums depends on timing.
//
// FP8 cache: the e4m3 bytes go to the tensor core as they are (kind::f8f6f4)
// against a two-part e4m3 copy of the query (hi + lo with a power-of-two
// scale per row, which reproduces bf16), made by a small kernel before; the
// RoPE columns are a bf16 product with an accumulator of its own, since the
// token's scale multiplies the latent part alone.
//
// Every wait is bounded: a wait that runs out sets a status bit, both CTAs
// leave their loops, the copies in flight are given time to land, and TMEM
// is freed.
#include <cuda.h>

#include "decode_launch.cuh"
#include "kernel_util.cuh"
#include "sm100_ptx.cuh"

namespace mla {

namespace {

using namespace ptx;

constexpr int kWThreads = 384;
constexpr int kEpiThreads = 256;                 // warps 4-11
constexpr int kUnit = 256;                       // tokens of a unit: 128 on each CTA
constexpr int kHalf = kUnit / 2;
constexpr uint32_t kWBox = 8192;                 // 64 tokens x 128 bytes
constexpr uint32_t kWStage = 2 * kWBox;
constexpr int kWMaxStages = 12;
constexpr uint32_t kWHead = 3 * 1024;            // barriers and column constants
constexpr uint32_t kWSmem = 232448;
constexpr int kMaxGroups = 16;                   // groups of row tiles per unit
constexpr int kSplitBelow = 4;                   // units a pair below which the tiles may be grouped
constexpr uint64_t kWTimeoutNs = 2000000000ull;
constexpr uint32_t kEpiBar = 1;

// One stage per 128 bytes of a token's row.  BF16: 9 of 64 columns.  FP8: the
// RoPE columns, then 4 of 128 e4m3 bytes, each against a hi and a lo chunk.
template <bool kFp8>
struct W {
  static constexpr int stages = kFp8 ? 5 : 9;    // of a unit
  static constexpr int tile = kFp8 ? 128 : 256;  // most rows of a tile (FP8: two accumulators a buffer)
};

// BF16: the tensor core's fp32 accumulator drops what does not fit, always
// towards zero, and the scores of random values come out smaller by about
// 4e-7 of themselves.  The scale does not make up for that: the lse that
// belongs to a call is the decode's, whose scores went through the same 36
// steps, so in x - lse most of it is gone.  Mean (rms) error of a weight
// against attention in 64 bits, h=128, t=4096: 2.8e-7 (5.4e-7) with the
// decode's lse, -1.3e-6 (1.4e-6) with an exact one.  (A scale larger by 4e-7
// gave 1.5e-6 (1.5e-6) and -1.5e-7 (3.1e-7), and put scores whose sums are
// exact off by 4e-7 of the score.)  FP8's two shorter sums lose less.

struct WBars {
  uint64_t full[kWMaxStages], empty[kWMaxStages], q_full[9], q_free[9], d_full[2], d_empty[2], part_full[2], done;
  uint64_t never;   // test hook: nothing arrives on it (WArgs::test_stall)
  uint32_t tmem_base;
  int32_t abort;
  int32_t r0, base0;
};
// Behind the barriers: the units of each warp's requests (at the start), then
// per 32 columns the fewest and the most tokens one of them sees; per column
// -lse (FP8: and the row's scale) and what it sees; the second warpgroup's
// sums, [accumulator][token].
constexpr uint32_t kOffWarpSum = 448, kOffGmin = 448, kOffGmax = 480, kOffNlse = 512, kOffHid = 1536, kOffPart = 2048;
static_assert(sizeof(WBars) <= kOffGmin && kOffPart + 1024 <= kWHead, "head");
constexpr uint16_t kDead = 0xffff;   // a column that adds nothing

struct WArgs {
  const uint8_t* kv;
  const float* kv_scale;
  const int32_t* block_table;
  const int32_t* seqlens;
  const float* lse;
  const float* q_scale;      // FP8: 2^e of every row
  float* weights;
  char* ws;
  uint32_t* counters;        // [units][8]: one for each warp's 32 tokens of a unit
  float* partial;            // [groups][units][256]
  float sl2, decay;
  int batch, s_q, heads, rows, causal, max_pages, num_pages, max_units;
  int test_stall;            // 0 in every product call
};

// What every role derives from the lengths.
struct Plan {
  int r0, base0;             // first request with work for this pair, units before it
  int64_t c0, c1;            // this pair's share, in unit x tile steps
  int tile, tiles, groups;
};

struct Seg {
  int r, t, row0, nh, u0, u1, unit0, group;
  bool first_tile, first, last;   // of the request; of its group
};

__device__ __forceinline__ int w_len(const WArgs& a, int r) {
  return max(0, min(a.seqlens[r], a.max_pages * MLA_PAGE_SIZE));
}

// Calls f for every (request, tile of rows, run of units) of this pair, in
// order, until f returns false.
template <class F>
__device__ __forceinline__ bool each_seg(const WArgs& a, const Plan& p, F&& f) {
  int64_t base = p.base0;
  for (int r = p.r0; r < a.batch; ++r) {
    if (base * p.tiles >= p.c1) break;
    const int t = w_len(a, r), U = (t + kUnit - 1) / kUnit;
    for (int s = 0; s < p.groups; ++s) {
      const int ta = int(int64_t(s) * p.tiles / p.groups), tb = int(int64_t(s + 1) * p.tiles / p.groups), L = tb - ta;
      const int64_t cb = base * p.tiles + int64_t(U) * ta;
      const int u0 = p.c0 <= cb ? 0 : int(min(int64_t(U), (p.c0 - cb + L - 1) / L));
      const int u1 = p.c1 <= cb ? 0 : int(min(int64_t(U), (p.c1 - cb + L - 1) / L));
      if (u0 >= u1) continue;
      for (int q = ta; q < tb; ++q) {
        const int row0 = q * p.tile, left = min(p.tile, a.rows - row0);
        if (!f(Seg{r, t, row0, ((left + 63) / 64) * 32, u0, u1, int(base), s, q == 0, q == ta, q == tb - 1})) return false;
      }
    }
    base += U;
  }
  return true;
}

struct WCtl {
  volatile int32_t* abort;
  uint32_t peer_abort;
  char* ws;
};

__device__ __noinline__ void w_trip(const WCtl& c) {
  *c.abort = 1;
  st_cluster_u32(c.peer_abort, 1);
  flag_status(c.ws, kStatusTimeout);
}

// Bounded wait of a warp; false when the pair is aborting.  Every lane polls,
// without suspending, and the warp leaves together: the loop around it stays
// converged (its operands then stay in uniform registers), and waking up from
// a suspended wait cost the FP8 case 4 us in 77.  kCluster: the barrier's
// arrivals are threads of either CTA; the others are completed by copies and
// MMAs alone.
template <bool kCluster = false>
__device__ __forceinline__ bool w_warp_wait(const WCtl& c, uint32_t bar, uint32_t parity) {
  auto once = [&] { return kCluster ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity); };
  if (__all_sync(0xffffffffu, once())) return true;
  const bool lead = (threadIdx.x & 31) == 0;
  const uint64_t t0 = lead ? globaltimer() : 0ull;
  for (uint32_t n = 1;; ++n) {
    if (__all_sync(0xffffffffu, once())) return true;
    if ((n & 15) == 0) {
      const int stop = __shfl_sync(0xffffffffu, lead ? (*c.abort ? 1 : (globaltimer() - t0 > kWTimeoutNs ? 2 : 0)) : 0, 0);
      if (stop != 0) {
        if (stop == 2 && lead) w_trip(c);
        return false;
      }
    }
  }
}

__device__ __forceinline__ uint64_t w_desc(uint32_t addr) {
  return uint64_t((addr >> 4) & 0x3FFF) | (uint64_t(16 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}

// The pair's forms of the tensor core and copy instructions.  A load lands in
// this CTA's shared memory and completes on the barrier `bar` (an address in
// the cluster's window: the first CTA's).
__device__ __forceinline__ void tma2_3d(uint32_t dst, const void* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma2_2d(uint32_t dst, const void* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void mma2_f16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma2_f8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs so far are done.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(uint16_t(3))
      : "memory");
}

// Arrives on a barrier of the pair's first CTA.  What it orders are this
// warp's TMEM reads (complete, and fenced by tcgen05.fence), so the arrival
// needs no wider scope: a release at cluster scope would make the warp wait
// for its global loads and stores in flight.
__device__ __forceinline__ void arrive_first(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// kind::f16 (bf16 A and B) and kind::f8f6f4 (e4m3), fp32 D, K-major, M = 256.
__device__ __forceinline__ uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t(n) >> 3) << 17) | ((256u >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_e4m3(int n) {
  return (1u << 4) | ((uint32_t(n) >> 3) << 17) | ((256u >> 4) << 24);
}

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWThreads, 1)
attn_weights_kernel(const __grid_constant__ CUtensorMap pool_map, const __grid_constant__ CUtensorMap rope_map,
                    const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap q8_map, const WArgs a) {
  constexpr int kStages = W<kFp8>::stages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0) {   // the layout fills the SM: there is no room to align it
    if (threadIdx.x == 0) flag_status(a.ws, kStatusWorkspace);
    return;
  }
  WBars* bars = reinterpret_cast<WBars*>(smem);
  auto bar = [&](const uint64_t& b) { return smem_u32(&b); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int pairs = int(nclusters_x()), pair = int(cluster_id_x());

  if (tid == 0) {
    for (int s = 0; s < kWMaxStages; ++s) {
      mbar_init(bar(bars->full[s]), 1);
      mbar_init(bar(bars->empty[s]), 1);
    }
    for (int s = 0; s < 9; ++s) {
      mbar_init(bar(bars->q_full[s]), 1);
      mbar_init(bar(bars->q_free[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(bars->d_full[s]), 1);
      mbar_init(bar(bars->d_empty[s]), 16);     // 8 warps of each CTA
      mbar_init(bar(bars->part_full[s]), 4);    // the second warpgroup's warps
    }
    mbar_init(bar(bars->done), 1);
    mbar_init(bar(bars->never), 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&pool_map);
    tma_prefetch_desc(&q_map);
    if (kFp8) {
      tma_prefetch_desc(&rope_map);
      tma_prefetch_desc(&q8_map);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bars->tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }

  // the units of all requests, and this pair's first request
  Plan plan;
  {
    const int per = (a.batch + kWThreads - 1) / kWThreads;
    const int ra = min(a.batch, tid * per), rb = min(a.batch, ra + per);
    int mine = 0;
    bool bad = false;
    for (int r = ra; r < rb; ++r) {
      const int t = a.seqlens[r];
      bad |= t < 0 || t > a.max_pages * MLA_PAGE_SIZE;
      mine += (w_len(a, r) + kUnit - 1) / kUnit;
    }
    if (bad && blockIdx.x == 0) flag_status(a.ws, kStatusBadSeqlen);
    int inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += u;
    }
    int* warp_sum = reinterpret_cast<int*>(smem + kOffWarpSum);
    if (lane == 31) warp_sum[warp] = inc;
    if (tid == 0) bars->r0 = a.batch;
    __syncthreads();
    int before = inc - mine, total = 0;
#pragma unroll
    for (int k = 0; k < kWThreads / 32; ++k) {
      before += k < warp ? warp_sum[k] : 0;
      total += warp_sum[k];
    }
    plan.tile = min(W<kFp8>::tile, (a.rows + 63) / 64 * 64);
    plan.tiles = (a.rows + plan.tile - 1) / plan.tile;
    // groups of tiles: the number that makes the longest pair's time least, in
    // tenths of a step (a unit against a tile).  A pair takes `items` units of
    // a group of `len` tiles, or its even share and one item; each tile of a
    // run costs 0.6 steps to load its rows, each item of more than one group
    // 0.6 for the workspace.
    plan.groups = 1;
    if (total < kSplitBelow * pairs) {
      const int64_t share = (int64_t(total) * plan.tiles + pairs - 1) / pairs;
      int64_t least = 0;
      for (int g = 1; g <= min(plan.tiles, kMaxGroups); g *= 2) {
        const int64_t len = (plan.tiles + g - 1) / g, items = (int64_t(total) * g + pairs - 1) / pairs;
        const int64_t time = 10 * min(items * len, share + len) + 6 * len + (g > 1 ? 6 * items : 0);
        if (g == 1 || time < least) {
          least = time;
          plan.groups = g;
        }
      }
    }
    const int64_t cost = int64_t(total) * plan.tiles;
    plan.c0 = cost * pair / pairs;
    plan.c1 = cost * (pair + 1) / pairs;
    if (plan.c0 < plan.c1 && before * int64_t(plan.tiles) <= plan.c0 && plan.c0 < (before + mine) * int64_t(plan.tiles)) {
      int r = ra;
      for (; r < rb; ++r) {
        const int U = (w_len(a, r) + kUnit - 1) / kUnit;
        if (plan.c0 < int64_t(before + U) * plan.tiles) break;
        before += U;
      }
      bars->r0 = r;
      bars->base0 = before;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    plan.r0 = bars->r0;
    plan.base0 = plan.r0 < a.batch ? bars->base0 : 0;
  }
  cluster_sync();
  griddep_wait();   // FP8: the query's two parts

  const uint32_t tmem = bars->tmem_base;
  const uint32_t q_stride = uint32_t(plan.tile / 2) * 128u;     // one chunk of this CTA's half of the rows
  const uint32_t q_base = sbase + kWHead, ring = q_base + 9u * q_stride;
  const uint32_t nst = min(uint32_t(kWMaxStages), (kWSmem - kWHead - 9u * q_stride) / kWStage);
  WCtl ctl{&bars->abort, mapa(smem_u32(&bars->abort), rank ^ 1u), a.ws};

  if (warp == 0) {
    // ---- producer warp (one lane issues)
    {
      const bool leader = elect_one();
      const bool arm = leader && rank == 0;
      const uint32_t full0 = mapa(bar(bars->full[0]), 0), q_full0 = mapa(bar(bars->q_full[0]), 0);
      uint32_t slot = 0, ph = 0, segs = 0;
      const bool ok = each_seg(a, plan, [&](const Seg& sg) {
        const int pages = (sg.t + MLA_PAGE_SIZE - 1) / MLA_PAGE_SIZE;
        const int32_t* bt = a.block_table + size_t(sg.r) * a.max_pages;
        auto page_of = [&](int j) {   // -1: no such page; a bad id reads page 0, and its tokens receive nothing
          if (j >= pages) return -1;
          const int p = bt[j];
          return p < 0 || p >= a.num_pages ? 0 : p;
        };
        const int row0 = sg.r * a.rows + sg.row0 + int(rank) * sg.nh;
        int j = 4 * sg.u0 + 2 * int(rank);
        int pa = page_of(j), pb = page_of(j + 1);
        for (int u = sg.u0; u < sg.u1; ++u, j += 4) {
          const int na = u + 1 < sg.u1 ? page_of(j + 4) : -1, nb = u + 1 < sg.u1 ? page_of(j + 5) : -1;
          const uint32_t bytes = uint32_t(min(4, pages - 4 * u)) * kWBox;   // of both CTAs
#pragma unroll 1
          for (int st = 0; st < kStages; ++st) {
            if (u == sg.u0) {
              if (!w_warp_wait(ctl, bar(bars->q_free[st]), (segs & 1u) ^ 1u)) return false;
              const int chunks = kFp8 && st > 0 ? 2 : 1;
              if (arm) mbar_arrive_expect_tx(bar(bars->q_full[st]), uint32_t(chunks) * 2u * uint32_t(sg.nh) * 128u);
              const uint32_t qb = q_full0 + 8u * uint32_t(st);
              if (leader) {
                for (int y = 0; y < sg.nh; y += 32) {
                  const uint32_t dst = q_base + uint32_t(y) * 128u;
                  if (!kFp8) {
                    tma2_2d(dst + uint32_t(st) * q_stride, &q_map, 64 * st, row0 + y, qb);
                  } else if (st == 0) {
                    tma2_2d(dst, &q_map, MLA_D_V, row0 + y, qb);
                  } else {
                    tma2_2d(dst + uint32_t(st) * q_stride, &q8_map, 128 * (st - 1), row0 + y, qb);
                    tma2_2d(dst + uint32_t(st + 4) * q_stride, &q8_map, MLA_D_V + 128 * (st - 1), row0 + y, qb);
                  }
                }
              }
              __syncwarp();
            }
            if (!w_warp_wait(ctl, bar(bars->empty[slot]), ph ^ 1u)) return false;
            if (arm) mbar_arrive_expect_tx(bar(bars->full[slot]), bytes);
            const uint32_t dst = ring + slot * kWStage, fb = full0 + 8u * slot;
            const CUtensorMap* map = kFp8 && st == 0 ? &rope_map : &pool_map;
            const int col = kFp8 ? (st == 0 ? 0 : 128 * (st - 1)) : 64 * st;
            if (leader) {
              if (pa >= 0) tma2_3d(dst, map, col, 0, pa, fb);
              if (pb >= 0) tma2_3d(dst + kWBox, map, col, 0, pb, fb);
            }
            __syncwarp();
            if (++slot == nst) {
              slot = 0;
              ph ^= 1u;
            }
          }
          pa = na;
          pb = nb;
        }
        ++segs;
        return true;
      });
      if (!ok) {
        // the pair is aborting: give this CTA's copies (which may complete on
        // the other CTA's barrier) time to land before it leaves
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---- MMA issuer warp of the pair's first CTA (one lane issues)
    {
      const bool leader = elect_one();
      uint32_t slot = 0, ph = 0, segs = 0, units = 0;
      const uint64_t ad0 = w_desc(ring), bd0 = w_desc(q_base);
      const uint32_t qs = q_stride >> 4;
      each_seg(a, plan, [&](const Seg& sg) {
        if (a.test_stall && !w_warp_wait(ctl, bar(bars->never), 0)) return false;
        const uint32_t ib = idesc_bf16(2 * sg.nh), i8 = idesc_e4m3(2 * sg.nh);
        for (int u = sg.u0; u < sg.u1; ++u, ++units) {
          const uint32_t buf = units & 1u, d = tmem + 256u * buf;
          if (!w_warp_wait<true>(ctl, bar(bars->d_empty[buf]), ((units >> 1) & 1u) ^ 1u)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int st = 0; st < kStages; ++st) {
            if (u == sg.u0 && !w_warp_wait(ctl, bar(bars->q_full[st]), segs & 1u)) return false;
            if (!w_warp_wait(ctl, bar(bars->full[slot]), ph)) return false;
            tc_fence_after();
            const uint64_t ad = ad0 + uint64_t(slot * (kWStage >> 4)), bd = bd0 + uint64_t(uint32_t(st) * qs);
            if (leader) {
              if (!kFp8 || st == 0) {
                const uint32_t dd = kFp8 ? d + 128u : d;
                mma2_f16(dd, ad, bd, ib, st != 0 ? 1u : 0u);
#pragma unroll
                for (int k = 1; k < 4; ++k) mma2_f16(dd, ad + 2u * k, bd + 2u * k, ib, 1u);
              } else {
                const uint64_t bl = bd + uint64_t(4u * qs);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  mma2_f8(d, ad + 2u * k, bd + 2u * k, i8, st != 1 || k != 0 ? 1u : 0u);
                  mma2_f8(d, ad + 2u * k, bl + 2u * k, i8, 1u);
                }
              }
              commit2(bar(bars->empty[slot]));
              if (u == sg.u1 - 1) commit2(bar(bars->q_free[st]));
              if (st == kStages - 1) commit2(bar(bars->d_full[buf]));
            }
            __syncwarp();
            if (++slot == nst) {
              slot = 0;
              ph ^= 1u;
            }
          }
        }
        ++segs;
        return true;
      });
      if (leader) commit2(bar(bars->done));
      __syncwarp();
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait_cluster(bar(bars->done), 0) && globaltimer() - t0 < kWTimeoutNs) {
      }
    }
  } else if (warp >= 4) {
    // ---- epilogue: thread i of either warpgroup holds token i of this CTA's
    // half; the first adds up the even groups of 32 columns, the second the
    // odd ones
    const int i = (tid - 128) & 127, wg = warp >= 8 ? 1 : 0, wq = warp & 3;
    const uint32_t lane_off = uint32_t(wq * 32) << 16;
    const uint32_t d_empty0 = mapa(bar(bars->d_empty[0]), 0);
    float* nlse = reinterpret_cast<float*>(smem + kOffNlse);      // per column: -lse in log2 units
    float* cscale = nlse + 128;                                   // FP8: 2^e * scale
    uint16_t* hid = reinterpret_cast<uint16_t*>(smem + kOffHid);  // per column: the last tokens that it does not see
    int* gmin = reinterpret_cast<int*>(smem + kOffGmin);
    int* gmax = reinterpret_cast<int*>(smem + kOffGmax);
    float* part = reinterpret_cast<float*>(smem + kOffPart);
    const int cap = a.max_pages * MLA_PAGE_SIZE;
    uint32_t n = 0;   // units so far
    // A warp whose wait failed says so at the group's next barrier, where all
    // eight leave together.
    bool ok = true, met = true;
    each_seg(a, plan, [&](const Seg& sg) {
      if (!named_bar_and(kEpiBar, kEpiThreads, ok)) return met = false;   // everyone is done with the last columns
      const int c = tid - 128;
      if (c < 2 * sg.nh) {
        const int row = sg.row0 + c;
        int v = 0;
        uint16_t hd = kDead;
        float nl = 0.f, cs = 0.f;
        if (row < min(a.rows, sg.row0 + plan.tile)) {
          const float l = a.lse[size_t(sg.r) * a.rows + row];
          if (l != -INFINITY) {
            v = min(sg.t, visible_len(sg.t, a.s_q, row / a.heads, a.causal));
            hd = uint16_t(sg.t - v < kDead ? sg.t - v : kDead);   // (sees nothing, or hides fewer than s_q <= 65534)
            nl = -l * 1.4426950408889634f;
          }
          if (kFp8) cs = a.q_scale[size_t(sg.r) * a.rows + row] * a.sl2;
        }
        nlse[c] = nl;
        if (kFp8) cscale[c] = cs;
        hid[c] = v > 0 ? hd : kDead;
        const int lo = __reduce_min_sync(0xffffffffu, v), hi = __reduce_max_sync(0xffffffffu, v);
        if (lane == 0) {
          gmin[c >> 5] = lo;
          gmax[c >> 5] = hi;
        }
      }
      const int ngroups = 2 * sg.nh / 32;
      const int32_t* bt = a.block_table + size_t(sg.r) * a.max_pages;
      const bool direct = plan.groups == 1;
      const bool reads_old = wg == 0 && (direct ? !sg.first_tile || a.decay != 0.f : !sg.first);
      auto pos_of = [&](int u) { return u * kUnit + int(rank) * kHalf + i; };
      auto sum_at = [&](int u) {   // where the token's sum of unit u lives
        return direct ? a.weights + size_t(sg.r) * cap + pos_of(u)
                      : a.partial + (size_t(sg.group) * a.max_units + sg.unit0 + u) * kUnit + (pos_of(u) - u * kUnit);
      };
      // page id (-2: no token here), token scale and old sum of a unit; the
      // ids are read two units ahead, the rest one
      auto page_at = [&](int u) { return u < sg.u1 && pos_of(u) < sg.t ? bt[pos_of(u) / MLA_PAGE_SIZE] : -2; };
      auto scale_at = [&](int u, int page) {
        return kFp8 && page >= 0 && page < a.num_pages ? a.kv_scale[size_t(page) * MLA_PAGE_SIZE + pos_of(u) % MLA_PAGE_SIZE]
                                                       : 0.f;
      };
      auto old_at = [&](int u, int page) { return reads_old && page != -2 ? *sum_at(u) : 0.f; };
      int page = page_at(sg.u0), page1 = page_at(sg.u0 + 1);
      float stok = scale_at(sg.u0, page), old = old_at(sg.u0, page);
      if (!named_bar_and(kEpiBar, kEpiThreads, true)) return met = false;   // the columns are in place
      for (int u = sg.u0; u < sg.u1; ++u, ++n) {
        const int page2 = page_at(u + 2);
        const float stok1 = scale_at(u + 1, page1), old1 = old_at(u + 1, page1);
        const uint32_t buf = n & 1u, par = (n >> 1) & 1u, d = tmem + lane_off + 256u * buf;
        const int pos0 = u * kUnit + int(rank) * kHalf, pos = pos0 + i;
        const bool live = page != -2, good = page >= 0 && page < a.num_pages;
        const int top = min(sg.t, pos0 + kHalf) - 1;   // the half's last token
        if (!w_warp_wait(ctl, bar(bars->d_full[buf]), par)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
        if (top >= pos0) {
#pragma unroll 1
          for (int g = wg; g < ngroups; g += 2) {
            if (pos0 >= gmax[g]) continue;   // no column of the group sees a token of this half
            uint32_t x[32];
            tmem_ld32(d + 32u * uint32_t(g), x);
            float v[32];
            if constexpr (kFp8) {
              uint32_t y[32];
              tmem_ld32(d + 128u + 32u * uint32_t(g), y);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 nl = *reinterpret_cast<const float4*>(nlse + 32 * g + k);
                const float4 cs = *reinterpret_cast<const float4*>(cscale + 32 * g + k);
                v[k] = fmaf(__uint_as_float(x[k]), stok * cs.x, fmaf(__uint_as_float(y[k]), a.sl2, nl.x));
                v[k + 1] = fmaf(__uint_as_float(x[k + 1]), stok * cs.y, fmaf(__uint_as_float(y[k + 1]), a.sl2, nl.y));
                v[k + 2] = fmaf(__uint_as_float(x[k + 2]), stok * cs.z, fmaf(__uint_as_float(y[k + 2]), a.sl2, nl.z));
                v[k + 3] = fmaf(__uint_as_float(x[k + 3]), stok * cs.w, fmaf(__uint_as_float(y[k + 3]), a.sl2, nl.w));
              }
            } else {
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 nl = *reinterpret_cast<const float4*>(nlse + 32 * g + k);
                v[k] = fmaf(__uint_as_float(x[k]), a.sl2, nl.x);
                v[k + 1] = fmaf(__uint_as_float(x[k + 1]), a.sl2, nl.y);
                v[k + 2] = fmaf(__uint_as_float(x[k + 2]), a.sl2, nl.z);
                v[k + 3] = fmaf(__uint_as_float(x[k + 3]), a.sl2, nl.w);
              }
            }
            if (top < gmin[g]) {   // every column sees every token of this half
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                s0 += ex2(v[k]);
                s1 += ex2(v[k + 1]);
                s2 += ex2(v[k + 2]);
                s3 += ex2(v[k + 3]);
              }
            } else {
              const int behind = sg.t - pos;   // tokens from this one to the end (a column that hides fewer sees it)
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const ushort4 h = *reinterpret_cast<const ushort4*>(hid + 32 * g + k);
                s0 += h.x != kDead && int(h.x) < behind ? ex2(v[k]) : 0.f;
                s1 += h.y != kDead && int(h.y) < behind ? ex2(v[k + 1]) : 0.f;
                s2 += h.z != kDead && int(h.z) < behind ? ex2(v[k + 2]) : 0.f;
                s3 += h.w != kDead && int(h.w) < behind ? ex2(v[k + 3]) : 0.f;
              }
            }
          }
        }
        tc_fence_before();
        float sum = (s0 + s1) + (s2 + s3);
        if (wg == 1) {
          // hand the odd groups' sum over; the first warpgroup frees the
          // accumulator only once it has it, so this place is free again
          // before the accumulator's next unit
          part[128 * buf + i] = sum;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(bars->part_full[buf]));
            arrive_first(d_empty0 + 8u * buf);
          }
        } else {
          if (!w_warp_wait(ctl, bar(bars->part_full[buf]), par)) {
            ok = false;
            break;
          }
          sum += part[128 * buf + i];
          __syncwarp();
          if (lane == 0) arrive_first(d_empty0 + 8u * buf);
          if (!good) sum = 0.f;
          if (live) {
            if (!good) flag_status(a.ws, kStatusBadPage);
            *sum_at(u) = fmaf(direct && sg.first_tile ? a.decay : 1.f, old, sum);
          }
          if (!direct && sg.last) {
            // the group's sums of this unit are in: whichever warp is the
            // last of the groups to say so adds its 32 tokens' sums up, in
            // the groups' order
            __threadfence();
            __syncwarp();
            uint32_t* count = a.counters + 8 * size_t(sg.unit0 + u) + 4 * rank + wq;
            uint32_t done = 0;
            if (lane == 0) done = atomicAdd(count, 1u);
            done = __shfl_sync(0xffffffffu, done, 0);
            if (done == uint32_t(plan.groups - 1)) {
              __threadfence();
              if (lane == 0) *count = 0u;
              if (live) {
                float* w = a.weights + size_t(sg.r) * cap + pos;
                float s = a.decay != 0.f ? a.decay * *w : 0.f;
                const float* from = a.partial + size_t(sg.unit0 + u) * kUnit + (pos - u * kUnit);
                for (int k = 0; k < plan.groups; ++k) s += __ldcg(from + size_t(k) * a.max_units * kUnit);
                *w = s;
              }
            }
          }
        }
        page = page1;
        page1 = page2;
        stok = stok1;
        old = old1;
      }
      return true;
    });
    if (met) named_bar_and(kEpiBar, kEpiThreads, ok);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  cluster_sync();
}

// FP8: the query rows' latent columns as two e4m3 parts, [row][hi 512, lo
// 512], with a power-of-two scale per row.  One warp per row.
__global__ void __launch_bounds__(256) split_query_kernel(const uint16_t* __restrict__ q, int rows, uint8_t* __restrict__ q8,
                                                          float* __restrict__ q_scale) {
  griddep_launch_dependents();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= rows) return;
  const uint4* src = reinterpret_cast<const uint4*>(q + size_t(row) * MLA_D_QK) + 2 * lane;
  const uint4 x = src[0], y = src[1];
  float am = fmaxf(fmaxf(fmaxf(bf16_abs_max(x.x), bf16_abs_max(x.y)), fmaxf(bf16_abs_max(x.z), bf16_abs_max(x.w))),
                   fmaxf(fmaxf(bf16_abs_max(y.x), bf16_abs_max(y.y)), fmaxf(bf16_abs_max(y.z), bf16_abs_max(y.w))));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, off));
  const int e = pow2_scale_exp(am);
  const float inv = ldexpf(1.f, -e);
  uint4 hi, lo;
  split_e4m3x4(x.x, x.y, inv, &hi.x, &lo.x);
  split_e4m3x4(x.z, x.w, inv, &hi.y, &lo.y);
  split_e4m3x4(y.x, y.y, inv, &hi.z, &lo.z);
  split_e4m3x4(y.z, y.w, inv, &hi.w, &lo.w);
  uint4* dst = reinterpret_cast<uint4*>(q8 + size_t(row) * 1024);
  dst[lane] = hi;
  dst[32 + lane] = lo;
  if (lane == 0) q_scale[row] = ldexpf(1.f, e);
}

// Workspace: [status][counters][groups' sums][FP8: query parts, scales].
struct WLayout {
  size_t counters, partial, q8, q_scale, total;
  int max_units;
};

WLayout w_layout(const mla_shape_t* s, int num_sms) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  WLayout L;
  const size_t rows = size_t(s->batch) * s->s_q * s->num_heads;
  L.max_units = kSplitBelow * (num_sms >= 2 ? num_sms / 2 : 1);   // more units than this are never split
  L.counters = kStatusBytes;
  L.partial = up(L.counters + size_t(L.max_units) * 32);
  L.q8 = up(L.partial + size_t(kMaxGroups) * L.max_units * kUnit * 4);
  L.q_scale = L.total = L.q8;
  if (s->cache_dtype == MLA_CACHE_FP8_E4M3) {
    L.q_scale = up(L.q8 + rows * 1024);
    L.total = up(L.q_scale + rows * 4);
  }
  return L;
}

}  // namespace

size_t attn_weights_workspace_bytes(const mla_shape_t* shape, int num_sms) { return w_layout(shape, num_sms).total; }

int launch_attn_weights(const mla_shape_t* shape, const void* q, const void* kv, const float* kv_scale,
                        const int32_t* block_table, const int32_t* seqlens, const float* lse, float scale, float decay,
                        float* weights, void* ws, int num_sms, cudaStream_t stream, int test_stall) {
  const bool fp8 = shape->cache_dtype == MLA_CACHE_FP8_E4M3;
  const WLayout L = w_layout(shape, num_sms);
  char* w = static_cast<char*>(ws);
  const int rows = shape->s_q * shape->num_heads, q_rows = shape->batch * rows;
  CUtensorMap pool_map, rope_map, q_map, q8_map;
  if (!make_q_map(&q_map, q, q_rows, 32)) return MLA_ERR_CUDA;
  if (fp8) {
    if (!make_fp8_maps(&pool_map, &rope_map, kv, shape->num_pages)) return MLA_ERR_CUDA;
    if (!make_byte_map(&q8_map, w + L.q8, q_rows, 1024, 32)) return MLA_ERR_CUDA;
  } else {
    if (!make_pool_map(&pool_map, kv, shape->num_pages)) return MLA_ERR_CUDA;
    rope_map = pool_map;   // not read
    q8_map = q_map;
  }
  auto fn = fp8 ? &attn_weights_kernel<true> : &attn_weights_kernel<false>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(fn), int(kWSmem))) return MLA_ERR_CUDA;
  WArgs a{static_cast<const uint8_t*>(kv), kv_scale, block_table, seqlens, lse,
          reinterpret_cast<const float*>(w + L.q_scale), weights, w, reinterpret_cast<uint32_t*>(w + L.counters),
          reinterpret_cast<float*>(w + L.partial),
          float(double(scale) * 1.4426950408889634), decay, shape->batch, shape->s_q, shape->num_heads, rows,
          shape->causal, shape->max_pages_per_seq, shape->num_pages, L.max_units, test_stall};
  if (fp8) {
    split_query_kernel<<<(q_rows + 7) / 8, 256, 0, stream>>>(static_cast<const uint16_t*>(q), q_rows,
                                                              reinterpret_cast<uint8_t*>(w + L.q8),
                                                              reinterpret_cast<float*>(w + L.q_scale));
    if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(num_sms >= 2 ? num_sms / 2 * 2 : 2));
  cfg.blockDim = dim3(kWThreads);
  cfg.dynamicSmemBytes = kWSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = fp8 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, fn, pool_map, rope_map, q_map, q8_map, a) != cudaSuccess) return MLA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla
