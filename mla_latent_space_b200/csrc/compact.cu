// Cache rows moved to the front of their request's own pages, in place: the
// row at position src[r][k] goes to position base[r] + k (the tokens that an
// eviction kept, or the accepted path of a drafted tree behind its prefix).
// src ascends and never lies before its destination, so rows only move
// towards the front.
//
// One CTA per request takes the list in order, 32 rows at a time: it holds a
// group of rows in registers before it writes any of them, so no row is
// overwritten before it has been read.
#include <cuda_runtime.h>

#include "kernel_util.cuh"

namespace mla {

namespace {

constexpr int kCompThreads = 256;
constexpr int kCompRows = 32;   // rows per group
constexpr int kFp8LatBytes = MLA_PAGE_SIZE * MLA_D_V;
constexpr int kFp8PageBytes = kFp8LatBytes + MLA_PAGE_SIZE * MLA_D_ROPE * 2;

template <bool kFp8>
constexpr int kChunks = kFp8 ? (MLA_D_V + 2 * MLA_D_ROPE) / 16 : 2 * MLA_D_QK / 16;   // 16-byte pieces of a row

struct CompArgs {
  uint8_t* kv;
  float* kv_scale;
  const int32_t* block_table;
  const int32_t* src;
  const int32_t* src_lens;
  const int32_t* base;
  float* weights;
  int32_t* status;
  int max_rows, max_pages, num_pages;
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

template <bool kFp8>
__global__ void __launch_bounds__(kCompThreads) compact_kernel(const CompArgs a) {
  constexpr int kCh = kChunks<kFp8>, kPer = kCompRows * kCh / kCompThreads;
  static_assert(kCompRows * kCh % kCompThreads == 0, "pieces");
  __shared__ int64_t from[kCompRows], to[kCompRows];
  __shared__ int pos_from[kCompRows], pos_to[kCompRows];
  const int r = blockIdx.x, tid = threadIdx.x;
  const int cap = a.max_pages * MLA_PAGE_SIZE;
  int n = a.src_lens[r], base = a.base != nullptr ? a.base[r] : 0;
  bool bad = n < 0 || n > a.max_rows || base < 0;
  n = base < 0 ? 0 : max(0, min(n, a.max_rows));
  const int32_t* src = a.src + size_t(r) * a.max_rows;
  for (int k0 = 0; k0 < n; k0 += kCompRows) {
    __syncthreads();
    if (tid < kCompRows) {
      const int k = k0 + tid;
      from[tid] = -1;
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
            from[tid] = int64_t(pa) * MLA_PAGE_SIZE + p % MLA_PAGE_SIZE;
            to[tid] = int64_t(pb) * MLA_PAGE_SIZE + d % MLA_PAGE_SIZE;
            pos_from[tid] = p;
            pos_to[tid] = int(d);
          }
        }
      }
    }
    __syncthreads();
    uint4 v[kPer];
    float sc = 0.f, w = 0.f;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int e = tid + kCompThreads * u, row = e / kCh;
      if (from[row] >= 0) v[u] = __ldcg(reinterpret_cast<const uint4*>(a.kv + piece_offset<kFp8>(from[row], e % kCh)));
    }
    if (tid < kCompRows && from[tid] >= 0) {
      if (kFp8) sc = __ldcg(a.kv_scale + from[tid]);
      if (a.weights != nullptr) w = __ldcg(a.weights + size_t(r) * cap + pos_from[tid]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int e = tid + kCompThreads * u, row = e / kCh;
      if (from[row] >= 0) *reinterpret_cast<uint4*>(a.kv + piece_offset<kFp8>(to[row], e % kCh)) = v[u];
    }
    if (tid < kCompRows && from[tid] >= 0) {
      if (kFp8) a.kv_scale[to[tid]] = sc;
      if (a.weights != nullptr) a.weights[size_t(r) * cap + pos_to[tid]] = w;
    }
  }
  if (bad) atomicOr(a.status, kStatusBadInput);
}

}  // namespace

size_t compact_workspace_bytes(int, int) { return kStatusBytes; }

int launch_compact(const mla_shape_t* shape, void* kv, float* kv_scale, const int32_t* block_table, const int32_t* src,
                   const int32_t* src_lens, const int32_t* base, int max_rows, float* weights, void* ws,
                   cudaStream_t stream) {
  const bool fp8 = shape->cache_dtype == MLA_CACHE_FP8_E4M3;
  CompArgs a{static_cast<uint8_t*>(kv), kv_scale, block_table, src, src_lens, base, weights, static_cast<int32_t*>(ws),
             max_rows, shape->max_pages_per_seq, shape->num_pages};
  if (fp8) compact_kernel<true><<<unsigned(shape->batch), kCompThreads, 0, stream>>>(a);
  else compact_kernel<false><<<unsigned(shape->batch), kCompThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla
