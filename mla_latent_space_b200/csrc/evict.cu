// Eviction from the cache by accumulated attention weight: which tokens of
// each request stay.  Of a request with more than `budget` tokens the first
// `sink`, the last `recent` and, between them, the budget - sink - recent of
// the largest weight stay; of equal weights the lowest positions.
//
// One CTA per request: a radix select (8 bits a pass, histogram in shared
// memory) finds the threshold weight and how many tokens of exactly that
// weight stay, then one ordered pass writes the kept positions.
#include <cuda_runtime.h>

#include "kernel_util.cuh"

namespace mla {

namespace {

constexpr int kSelThreads = 1024;

// Unsigned key in the order of the weights; NaN below everything, -0 = +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Exclusive block-wide scan of one value a thread; *total gets the sum.
__device__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int base = 0, sum = 0;
  for (int k = 0; k < kSelThreads / 32; ++k) {
    base += k < warp ? warp_sums[k] : 0;
    sum += warp_sums[k];
  }
  *total = sum;
  return base + inc - v;
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const float* __restrict__ weights, int64_t max_tokens, const int32_t* __restrict__ seqlens, int budget,
                    int sink, int recent, int32_t* __restrict__ kept, int32_t* __restrict__ kept_lens,
                    int32_t* __restrict__ status) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kSelThreads / 32];
  __shared__ uint32_t prefix_sh;
  __shared__ int need_sh;
  const int r = blockIdx.x, tid = threadIdx.x;
  int64_t t64 = seqlens[r];
  if (t64 < 0 || t64 > max_tokens) {
    if (tid == 0 && status != nullptr) atomicOr(status, kStatusBadSeqlen);
    t64 = t64 < 0 ? 0 : max_tokens;
  }
  const int t = int(t64);
  const float* w = weights + size_t(r) * size_t(max_tokens);
  int32_t* out = kept + size_t(r) * size_t(budget);
  if (tid == 0) kept_lens[r] = min(t, budget);
  if (t <= budget) {
    for (int k = tid; k < budget; k += kSelThreads) out[k] = k < t ? k : -1;
    return;
  }
  const int lo = sink, hi = t - recent;
  int need = budget - sink - recent;   // of the tokens in [lo, hi)
  uint32_t prefix = 0;
  for (int shift = 24; need > 0 && shift >= 0; shift -= 8) {
    for (int k = tid; k < 256; k += kSelThreads) hist[k] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const uint32_t k = weight_key(w[j]);
      if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int b = 255, n = need;
      while (b > 0 && hist[b] < n) n -= hist[b--];
      prefix_sh = prefix | (uint32_t(b) << shift);
      need_sh = n;
    }
    __syncthreads();
    prefix = prefix_sh;
    need = need_sh;
    __syncthreads();
  }
  const bool none = budget - sink - recent == 0;
  // keys above `prefix` stay, and the first `need` of those equal to it
  int done = 0, eq_done = 0;
  for (int j0 = 0; j0 < t; j0 += kSelThreads) {
    const int j = j0 + tid;
    const bool in = j < t, mid = in && j >= lo && j < hi;
    const uint32_t k = mid ? weight_key(w[j]) : 0u;
    const bool eq = mid && !none && k == prefix;
    int eq_total, total;
    const int eq_rank = eq_done + block_scan(eq ? 1 : 0, warp_sums, &eq_total);
    const bool keep = in && (!mid || (!none && (k > prefix || (eq && eq_rank < need))));
    const int at = done + block_scan(keep ? 1 : 0, warp_sums, &total);
    if (keep) out[at] = j;
    done += total;
    eq_done += eq_total;
  }
}

}  // namespace

cudaError_t launch_evict_select(const float* weights, int64_t max_tokens, const int32_t* seqlens, int batch, int budget,
                                int sink, int recent, int32_t* kept, int32_t* kept_lens, int32_t* status,
                                cudaStream_t stream) {
  evict_select_kernel<<<unsigned(batch), kSelThreads, 0, stream>>>(weights, max_tokens, seqlens, budget, sink, recent, kept,
                                                                    kept_lens, status);
  return cudaGetLastError();
}

}  // namespace mla
