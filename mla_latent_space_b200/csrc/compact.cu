// Cache rows moved to the front of their request's own pages, in place: the
// row at position src[r][k] goes to position base[r] + k (the tokens that an
// eviction kept, or the accepted path of a drafted tree behind its prefix).
// src ascends and never lies before its destination, so rows only move
// towards the front.
//
// The list is cut into groups of rows, dealt out in the list's order to the
// CTAs of a cooperative launch (all of them run at once).  A CTA holds a
// group's rows in registers, says that it has read them, and writes them once
// the groups whose sources lie at its destinations have been read: those are
// earlier groups or its own (src[k] >= base + k), two of them at most, and a
// search of the list names them.  A CTA takes its groups in order and waits
// only for earlier ones, so every wait ends; the waits are bounded all the
// same.  Each row is read once and written once, and what bounds it is how
// many rows are in flight: four CTAs an SM hold 36 KB each, and a CTA resolves
// its next group's pages and search while the current rows are on their way,
// but has none in flight while it waits and stores (DRAM at 52% of its peak,
// FP8's shorter lists 24%).  64 x 2048 of 4096 rows of BF16 (303 MB): 61 us on the device,
// 64 a call; with a CTA a group, handed out by a counter, 70 a call; waiting
// for all earlier groups instead of searching makes the CTAs queue behind
// each other: 94.
//
// Workspace: [status][finished CTAs][epoch] in the first 256 bytes, then a
// word a group: the epoch of the last call that read its rows.  Epochs only
// grow, so no call has to clear anything: the last CTA to leave steps it.  A
// list of one group needs none of this.
#include <cuda_runtime.h>

#include "kernel_util.cuh"

namespace mla {

namespace {

constexpr int kCompThreads = 256;
constexpr int kCompCtas = 4;   // per SM
constexpr uint64_t kCompTimeoutNs = 2000000000ull;
enum CtlWord { C_STATUS = 0, C_DONE, C_EPOCH };
constexpr int kFp8LatBytes = MLA_PAGE_SIZE * MLA_D_V;
constexpr int kFp8PageBytes = kFp8LatBytes + MLA_PAGE_SIZE * MLA_D_ROPE * 2;

template <bool kFp8>
constexpr int kChunks = kFp8 ? (MLA_D_V + 2 * MLA_D_ROPE) / 16 : 2 * MLA_D_QK / 16;   // 16-byte pieces of a row

template <bool kFp8>
constexpr int kCompRows = kFp8 ? 64 : 32;   // rows per group: 40 KB and 36 KB in registers

struct CompArgs {
  uint8_t* kv;
  float* kv_scale;
  const int32_t* block_table;
  const int32_t* src;
  const int32_t* src_lens;
  const int32_t* base;
  float* weights;
  uint32_t* ws;
  int batch, groups, max_rows, max_pages, num_pages;
  int test_stall;   // 0 in every product call; 1: nobody learns that a request's first group has been read
};

// Byte offset of piece `ch` of row `slot` (page * 64 + place) in the pool.
template <bool kFp8>
__device__ __forceinline__ size_t piece_offset(int64_t slot, int ch) {
  if constexpr (kFp8) {
    const size_t pg = size_t(slot >> 6) * kFp8PageBytes, row = size_t(slot & 63);
    return ch < MLA_D_V / 16 ? pg + row * MLA_D_V + 16 * ch
                             : pg + kFp8LatBytes + row * (2 * MLA_D_ROPE) + 16 * (ch - MLA_D_V / 16);
  } else {
    return size_t(slot) * (2 * MLA_D_QK) + 16 * size_t(ch);
  }
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Of the groups 0 .. n-1 of an ascending list, the last whose first entry is
// below x (0 if none), by one warp, 64 groups a step.
template <int kRows>
__device__ __forceinline__ int group_below(const int32_t* src, int n, int x) {
  const int lane = int(threadIdx.x & 31);
  int a = 0, b = n;   // the answer is in [a, b), or 0
  while (b - a > 1) {
    const int step = (b - a + 63) / 64;
    const int64_t i = int64_t(a) + int64_t(lane) * step, j = i + int64_t(32) * step;
    const int c = __popc(__ballot_sync(0xffffffffu, i < b && src[i * kRows] < x)) +
                  __popc(__ballot_sync(0xffffffffu, j < b && src[j * kRows] < x));
    if (c == 0) return a;
    b = int(min(int64_t(b), int64_t(a) + int64_t(c) * step));
    a = a + (c - 1) * step;
  }
  return a;
}

template <bool kFp8>
__global__ void __launch_bounds__(kCompThreads, kCompCtas) compact_kernel(const CompArgs a) {
  constexpr int kRows = kCompRows<kFp8>, kCh = kChunks<kFp8>, kPer = kRows * kCh / kCompThreads;
  static_assert(kRows * kCh % kCompThreads == 0 && kRows <= kCompThreads - 32, "pieces");
  // three buffers: a group's rows are still being written when the one after
  // the next is resolved
  __shared__ int64_t from[3][kRows], to[3][kRows];
  __shared__ int pos_from[3][kRows], pos_to[3][kRows];
  __shared__ int needs[3];        // the first of the groups whose sources may lie at its destinations; the group itself: none
  __shared__ int ready_sh[3];     // ... have been read already
  __shared__ uint32_t epoch_sh;
  const int tid = threadIdx.x;
  const bool solo = a.groups == 1;   // no other group's rows to wait for
  const uint32_t total = uint32_t(a.batch) * uint32_t(a.groups);
  const int cap = a.max_pages * MLA_PAGE_SIZE;
  bool bad = false;
  int r_known = -1, n = 0, base = 0;   // request, its list's length and base

  // Resolves the rows of group `item` into buffer b; true where this
  // thread's row moves.  exists: whether the request's list reaches the group.
  auto resolve = [&](uint32_t item, int b, bool* exists) -> bool {
    const int r = int(item % uint32_t(a.batch)), g = int(item / uint32_t(a.batch));
    if (r != r_known) {
      r_known = r;
      n = a.src_lens[r];
      base = a.base != nullptr ? a.base[r] : 0;
      if (g == 0 && (n < 0 || n > a.max_rows || base < 0)) bad = true;
      n = base < 0 ? 0 : max(0, min(n, a.max_rows));
    }
    const int k0 = g * kRows;
    const int32_t* src = a.src + size_t(r) * a.max_rows;
    *exists = k0 < n;
    if (tid >= kCompThreads - 32) {   // the last warp resolves no rows
      // (src[k] >= base + k, so an earlier entry whose source is not before
      // this group's destinations exists only where the last one's is not)
      const bool none = g == 0 || k0 >= n || int64_t(base) + k0 >= cap || src[k0 - 1] < base + k0;
      const int g0 = none ? g : group_below<kRows>(src, g, base + k0);
      if (tid == kCompThreads - 32) needs[b] = g0;
    }
    if (tid >= kRows) return false;
    const int k = k0 + tid;
    int64_t fr = -1;
    if (k < n) {
      const int p = src[k], before = k > 0 ? src[k - 1] : -1;
      const int64_t d = int64_t(base) + k;
      if (p < d || p >= cap || p <= before) {
        bad = true;
      } else if (p != d) {
        const int32_t* bt = a.block_table + size_t(r) * a.max_pages;
        const int pa = bt[p / MLA_PAGE_SIZE], pb = bt[d / MLA_PAGE_SIZE];
        if (pa < 0 || pa >= a.num_pages || pb < 0 || pb >= a.num_pages) {
          bad = true;
        } else {
          fr = int64_t(pa) * MLA_PAGE_SIZE + p % MLA_PAGE_SIZE;
          to[b][tid] = int64_t(pb) * MLA_PAGE_SIZE + d % MLA_PAGE_SIZE;
          pos_from[b][tid] = p;
          pos_to[b][tid] = int(d);
        }
      }
    }
    from[b][tid] = fr;
    return fr >= 0;
  };

  if (tid == 0) epoch_sh = solo ? 0u : *const_cast<volatile uint32_t*>(a.ws + C_EPOCH) + 1u;
  uint32_t item = blockIdx.x;   // group item / batch of request item % batch
  bool exists = false;
  bool moves = __syncthreads_or(resolve(item, 0, &exists));   // (the grid has no CTA without an item)
  const uint32_t epoch = epoch_sh;
  int b = 0;
  while (item < total) {   // (uniform in the CTA)
    const int r = int(item % uint32_t(a.batch)), g = int(item / uint32_t(a.batch));
    uint32_t* flags = a.ws + kStatusBytes / 4 + size_t(r) * a.groups;
    uint4 v[kPer];
    float sc = 0.f, w = 0.f;
    const bool mine = moves && tid < kRows && from[b][tid] >= 0;
    uint32_t seen = 0;
    if (moves) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int e = tid + kCompThreads * u, row = e / kCh;
        v[u] = make_uint4(0, 0, 0, 0);
        if (from[b][row] >= 0)
          v[u] = __ldcg(reinterpret_cast<const uint4*>(a.kv + piece_offset<kFp8>(from[b][row], e % kCh)));
      }
      if (mine) {
        if (kFp8) sc = __ldcg(a.kv_scale + from[b][tid]);
        if (a.weights != nullptr) w = __ldcg(a.weights + size_t(r) * cap + pos_from[b][tid]);
      }
    }
    // while they are on their way: whether the groups to wait for have been
    // read, and the next group
    const int g0 = needs[b], g1 = min(g0 + 1, g - 1);   // two at most: kRows places hold sources of kRows entries in a row
    const bool waits = moves && !solo && g0 < g;
    if (waits && tid < 2) {
      const bool ok = g0 + tid > g1 || ld_acquire(flags + g0 + tid) == epoch;
      const bool both = __all_sync(3u, ok);
      if (tid == 0) ready_sh[b] = both;
    }
    const uint32_t next = item + gridDim.x;   // (below 2^32: both are below 2^31)
    const int bn = b == 2 ? 0 : b + 1;
    bool next_exists = false, next_moves = false;
    if (next < total) next_moves = resolve(next, bn, &next_exists);
    // This thread's rows have been read once something has used them; `zero`
    // is a zero that the compiler does not know.  (A fence would also wait
    // for the last group's stores.)
    if (moves) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) seen |= v[u].x;
      seen |= __float_as_uint(sc) | __float_as_uint(w);
    }
    uint32_t zero = uint32_t(a.batch) >> 31;
    asm volatile("and.b32 %0, %0, %1;" : "+r"(zero) : "r"(seen));
    next_moves = __syncthreads_or(next_moves || zero != 0u) != 0;   // the CTA's rows have been read
    bool ok = true;
    if (exists && !solo) {
      if (tid == 0 && !(a.test_stall != 0 && g == 0)) st_release(flags + g, epoch);
      if (waits && !ready_sh[b]) {
        if (tid <= g1 - g0) {
          uint64_t t0, t1;
          asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
          while (ld_acquire(flags + g0 + tid) != epoch) {
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t1));
            if (t1 - t0 > kCompTimeoutNs) {
              ok = false;
              atomicOr(reinterpret_cast<int32_t*>(a.ws), kStatusTimeout);
              break;
            }
          }
        }
        ok = __syncthreads_and(ok);
      }
    }
    if (moves && ok) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int e = tid + kCompThreads * u, row = e / kCh;
        if (from[b][row] >= 0)
          *reinterpret_cast<uint4*>(a.kv + piece_offset<kFp8>(to[b][row], e % kCh)) = v[u];
      }
      if (mine) {
        if (kFp8) a.kv_scale[to[b][tid]] = sc;
        if (a.weights != nullptr) a.weights[size_t(r) * cap + pos_to[b][tid]] = w;
      }
    }
    item = next;
    exists = next_exists;
    moves = next_moves;
    b = bn;
  }
  if (bad) atomicOr(reinterpret_cast<int32_t*>(a.ws), kStatusBadInput);
  if (!solo && tid == 0 && atomicAdd(a.ws + C_DONE, 1u) == gridDim.x - 1) {
    a.ws[C_DONE] = 0u;
    a.ws[C_EPOCH] = epoch;
  }
}

int groups_for(bool fp8, int max_rows) {
  const int rows = fp8 ? kCompRows<true> : kCompRows<false>;
  return (max_rows + rows - 1) / rows;
}

}  // namespace

// 0: more groups than 31 bits count.
size_t compact_workspace_bytes(const mla_shape_t* shape, int max_rows) {
  const int64_t n = int64_t(shape->batch) * groups_for(shape->cache_dtype == MLA_CACHE_FP8_E4M3, max_rows);
  return n < (int64_t(1) << 31) ? kStatusBytes + size_t(n) * 4 : 0;
}

int launch_compact(const mla_shape_t* shape, void* kv, float* kv_scale, const int32_t* block_table, const int32_t* src,
                   const int32_t* src_lens, const int32_t* base, int max_rows, float* weights, void* ws, int num_sms,
                   cudaStream_t stream, int test_stall) {
  const bool fp8 = shape->cache_dtype == MLA_CACHE_FP8_E4M3;
  const int groups = groups_for(fp8, max_rows);
  CompArgs a{static_cast<uint8_t*>(kv), kv_scale, block_table, src, src_lens, base, weights, static_cast<uint32_t*>(ws),
             shape->batch, groups, max_rows, shape->max_pages_per_seq, shape->num_pages, test_stall};
  // As many CTAs as are resident; where no CTA waits for another, one each.
  // (A whole number of them a request, so that a CTA stays with one, leaves up
  // to half of the machine idle and gains nothing: us with all / with whole
  // rounds, BF16, 64 x 2048 rows 62 / 62, 200 x 512 49 / 53, 300 x 512 70 / 88,
  // 400 x 512 90 / 101; FP8, 300 x 1024 rows 86 / 106.)
  const int64_t total = int64_t(shape->batch) * groups;
  const int64_t resident = kCompCtas * int64_t(num_sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(groups == 1 || total < resident ? total : resident));
  cfg.blockDim = dim3(kCompThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = groups == 1 ? 0 : 1;
  if (cudaLaunchKernelEx(&cfg, fp8 ? &compact_kernel<true> : &compact_kernel<false>, a) != cudaSuccess) return MLA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla
