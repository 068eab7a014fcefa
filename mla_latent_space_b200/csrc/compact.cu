// Cache rows moved to the front of their request's own pages, in place: the
// row at position src[r][k] goes to position base[r] + k (the tokens that an
// eviction kept, or the accepted path of a drafted tree behind its prefix).
// src ascends and never lies before its destination, so rows only move
// towards the front.
//
// The list is cut into groups of rows.  A CTA takes the next group from a
// counter, holds its rows in registers (four CTAs of 36 KB keep an SM's share
// of the memory bandwidth in flight), says that it has read them, and writes
// them once nobody still needs what lies there: the rows at its destinations
// are the sources of earlier groups or of its own (src[k] >= base + k), and a
// search of the list names them.  Groups are handed out in the order of the
// list and a CTA waits only for reads of earlier ones, none of which wait for
// anything, so every wait ends; the waits are bounded all the same.  Each row
// is read once and written once: what bounds it is HBM.
//
// Workspace: [status][counter][finished CTAs][epoch] in the first 256 bytes,
// then one word a group, which holds the epoch of the last call that read the
// group's rows (plus one).  The last CTA of a call resets the counters and
// steps the epoch, so no call has to clear anything.
#include <cuda_runtime.h>

#include "kernel_util.cuh"

namespace mla {

namespace {

constexpr int kCompThreads = 256;
constexpr uint64_t kCompTimeoutNs = 2000000000ull;
enum CtlWord { C_STATUS = 0, C_TICKET, C_DONE, C_EPOCH };
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

// Index of the first of the ascending src[0..n) that is >= x (n if none): a
// search in steps of 256, by the whole CTA.
__device__ __forceinline__ int first_at_least(const int32_t* src, int n, int x) {
  int a = 0, b = n;
  while (a < b) {
    const int step = (b - a + kCompThreads - 1) / kCompThreads;
    const int64_t i = int64_t(a) + int64_t(threadIdx.x) * step;
    const int c = __syncthreads_count(i < b && src[i] < x);
    if (c == 0) return a;
    b = int(min(int64_t(b), int64_t(a) + int64_t(c) * step));
    a = a + (c - 1) * step + 1;
  }
  return a;
}

template <bool kFp8>
__global__ void __launch_bounds__(kCompThreads, 4) compact_kernel(const CompArgs a) {
  constexpr int kRows = kCompRows<kFp8>, kCh = kChunks<kFp8>, kPer = kRows * kCh / kCompThreads;
  static_assert(kRows * kCh % kCompThreads == 0, "pieces");
  __shared__ int64_t from[kRows], to[kRows];
  __shared__ int pos_from[kRows], pos_to[kRows];
  __shared__ uint32_t ticket_sh, epoch_sh;
  const int tid = threadIdx.x;
  if (tid == 0) {
    epoch_sh = *const_cast<volatile uint32_t*>(a.ws + C_EPOCH) + 1u;
    ticket_sh = atomicAdd(a.ws + C_TICKET, 1u);
  }
  __syncthreads();
  const int r = int(ticket_sh % uint32_t(a.batch)), g = int(ticket_sh / uint32_t(a.batch));
  const uint32_t epoch = epoch_sh;
  uint32_t* flags = a.ws + kStatusBytes / 4 + size_t(r) * a.groups;
  const int cap = a.max_pages * MLA_PAGE_SIZE;
  int n = a.src_lens[r];
  const int base = a.base != nullptr ? a.base[r] : 0;
  bool bad = g == 0 && (n < 0 || n > a.max_rows || base < 0);
  n = base < 0 ? 0 : max(0, min(n, a.max_rows));
  const int32_t* src = a.src + size_t(r) * a.max_rows;
  const int k0 = g * kRows;
  if (k0 < n) {   // (uniform in the CTA)
    bool moves = false;
    if (tid < kRows) {
      const int k = k0 + tid;
      int64_t fr = -1;
      if (k < n) {
        const int p = src[k];
        const int64_t d = int64_t(base) + k;
        if (p < d || p >= cap || (k > 0 && p <= src[k - 1])) {
          bad = true;
        } else if (p != d) {
          const int pa = a.block_table[size_t(r) * a.max_pages + p / MLA_PAGE_SIZE];
          const int pb = a.block_table[size_t(r) * a.max_pages + d / MLA_PAGE_SIZE];
          if (pa < 0 || pa >= a.num_pages || pb < 0 || pb >= a.num_pages) {
            bad = true;
          } else {
            fr = int64_t(pa) * MLA_PAGE_SIZE + p % MLA_PAGE_SIZE;
            to[tid] = int64_t(pb) * MLA_PAGE_SIZE + d % MLA_PAGE_SIZE;
            pos_from[tid] = p;
            pos_to[tid] = int(d);
            moves = true;
          }
        }
      }
      from[tid] = fr;
    }
    if (__syncthreads_or(moves)) {
      uint4 v[kPer];
      float sc = 0.f, w = 0.f;
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int e = tid + kCompThreads * u, row = e / kCh;
        if (from[row] >= 0) v[u] = __ldcg(reinterpret_cast<const uint4*>(a.kv + piece_offset<kFp8>(from[row], e % kCh)));
      }
      const bool mine = tid < kRows && from[tid] >= 0;
      if (mine) {
        if (kFp8) sc = __ldcg(a.kv_scale + from[tid]);
        if (a.weights != nullptr) w = __ldcg(a.weights + size_t(r) * cap + pos_from[tid]);
      }
      // while the rows are on their way: the earlier entries whose sources
      // are this group's destinations are [first, first + kRows) at most
      const int first = g == 0 || int64_t(base) + k0 >= cap ? k0 : first_at_least(src, k0, base + k0);
      __threadfence();   // this thread's rows have been read ...
      __syncthreads();
      if (tid == 0) st_release(flags + g, epoch);   // ... and the CTA's
      bool ok = true;
      if (first < k0) {
        const int g0 = first / kRows, g1 = (min(first + kRows, k0) - 1) / kRows;   // at most two groups, before g
        if (tid <= g1 - g0) {
          const uint32_t* f = flags + g0 + tid;
          if (ld_acquire(f) != epoch) {
            uint64_t t0, t1;
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
            while (ld_acquire(f) != epoch) {
              asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t1));
              if (t1 - t0 > kCompTimeoutNs) {
                ok = false;
                atomicOr(reinterpret_cast<int32_t*>(a.ws), kStatusTimeout);
                break;
              }
            }
          }
        }
        ok = __syncthreads_and(ok);
      }
      if (ok) {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          const int e = tid + kCompThreads * u, row = e / kCh;
          if (from[row] >= 0) *reinterpret_cast<uint4*>(a.kv + piece_offset<kFp8>(to[row], e % kCh)) = v[u];
        }
        if (mine) {
          if (kFp8) a.kv_scale[to[tid]] = sc;
          if (a.weights != nullptr) a.weights[size_t(r) * cap + pos_to[tid]] = w;
        }
      }
    } else if (tid == 0) {
      st_release(flags + g, epoch);   // rows that stay are nobody's destination
    }
  }
  if (bad) atomicOr(reinterpret_cast<int32_t*>(a.ws), kStatusBadInput);
  if (tid == 0 && atomicAdd(a.ws + C_DONE, 1u) == gridDim.x - 1) {
    a.ws[C_TICKET] = 0u;
    a.ws[C_DONE] = 0u;
    a.ws[C_EPOCH] = epoch;
  }
}

int groups_for(bool fp8, int max_rows) {
  const int rows = fp8 ? kCompRows<true> : kCompRows<false>;
  return (max_rows + rows - 1) / rows;
}

}  // namespace

// 0: more groups than one launch takes.
size_t compact_workspace_bytes(const mla_shape_t* shape, int max_rows) {
  const int64_t ctas = int64_t(shape->batch) * groups_for(shape->cache_dtype == MLA_CACHE_FP8_E4M3, max_rows);
  return ctas < (int64_t(1) << 31) ? kStatusBytes + size_t(ctas) * 4 : 0;
}

int launch_compact(const mla_shape_t* shape, void* kv, float* kv_scale, const int32_t* block_table, const int32_t* src,
                   const int32_t* src_lens, const int32_t* base, int max_rows, float* weights, void* ws,
                   cudaStream_t stream) {
  const bool fp8 = shape->cache_dtype == MLA_CACHE_FP8_E4M3;
  const int groups = groups_for(fp8, max_rows);
  CompArgs a{static_cast<uint8_t*>(kv), kv_scale, block_table, src, src_lens, base, weights, static_cast<uint32_t*>(ws),
             shape->batch, groups, max_rows, shape->max_pages_per_seq, shape->num_pages};
  const unsigned grid = unsigned(shape->batch) * unsigned(groups);
  if (fp8) compact_kernel<true><<<grid, kCompThreads, 0, stream>>>(a);
  else compact_kernel<false><<<grid, kCompThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla
