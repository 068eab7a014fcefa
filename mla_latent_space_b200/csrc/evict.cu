// Eviction from the cache by accumulated attention weight: which tokens of
// each request stay.  Of a request with more than `budget` tokens the first
// `sink`, the last `recent` and, between them, the budget - sink - recent of
// the largest weight stay; of equal weights the lowest positions.
//
// Mathematics.  Every token gets an unsigned 32-bit key in the order of the
// weights (NaN 0, sink and recent tokens the largest key, which no weight
// has); what stays are the `budget` largest keys, ties by position.  A radix
// select finds the smallest kept key `thr` in at most three passes of 11, 11
// and 10 bits (a histogram of the keys that match the digits so far, the
// suffix sum that reaches what is still needed), and stops early when a
// bucket is needed whole.  One ordered pass then writes the positions with
// key > thr and the first `need` of those with key == thr.
//
// Layout.  The weights are read once: the keys stay in shared memory.  A row
// is one CTA's work, or it is cut into contiguous chunks over a cluster of 8
// CTAs, which add up each other's histograms and counts over distributed
// shared memory.  Rows too long even for that re-read the weights through L2
// in every pass.  The cluster pays for long rows as long as the clusters of
// all rows run at once, two CTAs an SM (us, one CTA / cluster; a row is full):
//
//   tokens   batch 2       8         16        32        33        37        64
//    4096    8 / 10      8 / 11    8 / 11    8 / 13    8 / 13    8 / 18    9 / 22
//   10000   11 / 11     11 / 12   11 / 13   11 / 15   11 / 15   11 / 20   11 / 24
//   16384   13 / 11     13 / 11   13 / 13   13 / 15   13 / 15   13 / 20   14 / 26
//   24576   15 / 11     15 / 11   18 / 14   18 / 16   18 / 17   17 / 22   18 / 28
//   32768   22 / 13     20 / 12   22 / 15   22 / 15   22 / 17   22 / 24   22 / 28
//   49152   26 / 12     28 / 13   28 / 16   28 / 20   28 / 19   28 / 25   28 / 32
//
// so a row is one CTA's up to 8192 tokens and 400 more for each row of the
// batch, or where the clusters would queue.  The host knows the rows' length,
// not the requests': 64 requests of 4096 tokens in rows of 131072, which only
// a cluster holds, take 22 us.  What bounds it is latency: of the 16 us of two
// rows of 131072 tokens, 3.5 are the trip to memory, 5 the digits' passes with
// their cluster barriers, 5 the ordered output.  (Adding up equal bins within a warp before the shared-memory adds,
// for the many weights that are zero, costs more than it saves: 30.7 us
// against 26.6 at that stage.)
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "kernel_util.cuh"

namespace cg = cooperative_groups;

namespace mla {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kPasses = 3;
constexpr int kCluster = 8;
constexpr int kWideTokens = 8192;            // up to here, and kWidePerRow more for each row, one CTA a row
constexpr int kWidePerRow = 400;
constexpr int kSmemKeys = 48 * 1024;         // keys per CTA that fit beside the histograms (192 KB)

struct alignas(16) SelShared {
  int hist[kPasses][kBins];
  int coarse[kPasses][kSelWarps];            // sums of 64 bins
  int warp_a[kSelWarps], warp_b[kSelWarps];
  int digit, need, count;                    // a pass's verdict
  int cta_gt, cta_eq;                        // this CTA's chunk: keys above thr, keys equal to it
};

// Unsigned key in the order of the weights; NaN below everything, -0 = +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Sum of v over the CTA's warps before this one, exclusive; all threads call.
__device__ __forceinline__ int warp_prefix(const int* sums, int warp, int lane) {
  int v = lane < warp ? sums[lane] : 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <int kCtas, bool kInSmem>
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const float* __restrict__ weights, int max_tokens, const int32_t* seqlens, int budget, int sink,
                    int recent, int32_t* __restrict__ kept, int32_t* kept_lens, int32_t* __restrict__ status) {
  extern __shared__ uint32_t keys[];
  __shared__ SelShared sh;
  const int r = blockIdx.x / kCtas, rank = blockIdx.x % kCtas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int t = seqlens[r];
  if (t < 0 || t > max_tokens) {
    if (rank == 0 && tid == 0 && status != nullptr) atomicOr(status, kStatusBadSeqlen);
    t = t < 0 ? 0 : max_tokens;
  }
  const float* w = weights + size_t(r) * size_t(max_tokens);
  int32_t* out = kept + size_t(r) * size_t(budget);
  // kept_lens may be seqlens: it is written where every thread has read the
  // length, or where what is written is the length
  if (t <= budget) {   // (every CTA of the cluster agrees)
    if (rank == 0 && tid == 0) kept_lens[r] = t;
    for (int k = rank * kSelThreads + tid; k < budget; k += kCtas * kSelThreads) out[k] = k < t ? k : -1;
    return;
  }
  for (int k = tid; k < kPasses * kBins; k += kSelThreads) (&sh.hist[0][0])[k] = 0;
  __syncthreads();

  // this CTA's chunk [lo, lo + n), a multiple of 32 tokens but for the last
  const int chunk = ((t + kCtas - 1) / kCtas + 31) & ~31;
  const int lo = min(t, rank * chunk), n = min(t - lo, chunk);
  const int n32 = (n + 31) & ~31;
  auto key_of = [&](int i, float x) -> uint32_t {
    const int j = lo + i;
    return j < sink || j >= t - recent ? 0xffffffffu : weight_key(x);
  };
  auto key_at = [&](int i) -> uint32_t { return kInSmem ? keys[i] : key_of(i, w[lo + i]); };

  uint32_t prefix = 0;
  int need = budget, shift = 21;
  uint32_t thr = 0;
  for (int pass = 0; pass < kPasses; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    const uint32_t fixed = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
    int* hist = sh.hist[pass];
    if (pass == 0) {
      // the only pass over memory: eight loads in flight a thread
      constexpr int kU = 8;
      for (int i0 = tid; i0 < n32; i0 += kU * kSelThreads) {
        float x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = i0 + u * kSelThreads;
          x[u] = i < n ? w[lo + i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = i0 + u * kSelThreads;
          if (i < n) {
            const uint32_t k = key_of(i, x[u]);
            if (kInSmem) keys[i] = k;
            atomicAdd(&hist[k >> 21], 1);
          }
        }
      }
    } else {
#pragma unroll 4
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t k = key_at(i);
        if ((k & fixed) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1);
      }
    }
    // sums of 64 bins, then one warp finds the 64 and, within them, the bin
    // that holds the last kept key, counting from the largest: of a cluster's
    // histograms it reads 32 + 64 words each, not 2048
    __syncthreads();
    {
      const int2 v = *reinterpret_cast<const int2*>(hist + 64 * warp + 2 * lane);
      const int sum = __reduce_add_sync(0xffffffffu, v.x + v.y);
      if (lane == 0) sh.coarse[pass][warp] = sum;
    }
    if constexpr (kCtas > 1) cg::this_cluster().sync();
    else __syncthreads();
    if (warp == 0) {
      // keys in the lanes above (larger bins), exclusive
      auto above_of = [&](int v) {
        int inc = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int u = __shfl_down_sync(0xffffffffu, inc, off);
          if (lane + off < 32) inc += u;
        }
        return inc - v;
      };
      int c = 0;
      if constexpr (kCtas > 1) {
#pragma unroll
        for (int q = 0; q < kCtas; ++q) c += cg::this_cluster().map_shared_rank(sh.coarse[pass], q)[lane];
      } else {
        c = sh.coarse[pass][lane];
      }
      int above = above_of(c);
      const int big = __ffs(int(__ballot_sync(0xffffffffu, above < need && need <= above + c))) - 1;
      above = __shfl_sync(0xffffffffu, above, big);
      int2 f = make_int2(0, 0);   // bins 64 big + 2 lane, + 1
      if constexpr (kCtas > 1) {
#pragma unroll
        for (int q = 0; q < kCtas; ++q) {
          const int2 v = *reinterpret_cast<const int2*>(cg::this_cluster().map_shared_rank(hist, q) + 64 * big + 2 * lane);
          f.x += v.x;
          f.y += v.y;
        }
      } else {
        f = *reinterpret_cast<const int2*>(hist + 64 * big + 2 * lane);
      }
      above += above_of(f.x + f.y);
      if (above < need && need <= above + f.x + f.y) {   // one lane
        const bool in_hi = need <= above + f.y;
        sh.digit = 64 * big + 2 * lane + (in_hi ? 1 : 0);
        sh.need = in_hi ? need - above : need - above - f.y;
        sh.count = in_hi ? f.y : f.x;
      }
    }
    __syncthreads();
    prefix |= uint32_t(sh.digit) << shift;
    need = sh.need;
    thr = prefix;
    if (need == sh.count) {   // the whole bucket stays (never the bucket of key 0: fewer stay than there are)
      thr = prefix - 1u;
      need = 0;
      break;
    }
    shift -= pass == 0 ? 11 : 10;
  }

  if (rank == 0 && tid == 0) kept_lens[r] = budget;   // (a pass has met all threads of the row)

  // ordered output: warp `warp` owns a contiguous run of the chunk
  const int run = (n32 / 32 + kSelWarps - 1) / kSelWarps * 32;
  const int b = min(n32, warp * run), e = min(n32, b + run);
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = b + lane; i < min(e, n); i += 32) {
    const uint32_t k = key_at(i);
    gt += k > thr;
    eq += k == thr;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    sh.warp_a[warp] = gt;
    sh.warp_b[warp] = eq;
  }
  __syncthreads();
  const int gt_before = warp_prefix(sh.warp_a, warp, lane), eq_before = warp_prefix(sh.warp_b, warp, lane);
  int at = gt_before, eq_rank = eq_before;
  if constexpr (kCtas > 1) {
    if (tid == kSelThreads - 1) {
      sh.cta_gt = gt_before + gt;
      sh.cta_eq = eq_before + eq;
    }
    cg::this_cluster().sync();
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
      if (c >= rank) break;
      at += *cg::this_cluster().map_shared_rank(&sh.cta_gt, c);
      eq_rank += *cg::this_cluster().map_shared_rank(&sh.cta_eq, c);
    }
  }
  at += min(eq_rank, need);
  const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
  for (int i = b + lane; i < e; i += 32) {
    const uint32_t k = i < n ? key_at(i) : 0u;
    const bool is_eq = i < n && k == thr;
    const unsigned eqs = __ballot_sync(0xffffffffu, is_eq);
    const bool keep = (i < n && k > thr) || (is_eq && eq_rank + __popc(eqs & below) < need);
    const unsigned keeps = __ballot_sync(0xffffffffu, keep);
    if (keep) out[at + __popc(keeps & below)] = lo + i;
    at += __popc(keeps);
    eq_rank += __popc(eqs);
  }
  if constexpr (kCtas > 1) cg::this_cluster().sync();   // no CTA leaves while another reads its counts
}

template <int kCtas, bool kInSmem>
cudaError_t launch(const float* weights, int max_tokens, const int32_t* seqlens, int batch, int budget, int sink, int recent,
                   int32_t* kept, int32_t* kept_lens, int32_t* status, cudaStream_t stream) {
  auto fn = &evict_select_kernel<kCtas, kInSmem>;
  const int chunk = ((max_tokens + kCtas - 1) / kCtas + 31) & ~31;
  const size_t smem = kInSmem ? size_t(chunk) * 4 : 0;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(fn), kInSmem ? kSmemKeys * 4 : 0))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(batch) * kCtas);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, weights, max_tokens, seqlens, budget, sink, recent, kept, kept_lens,
                                           status);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

namespace {

// Clusters that run at once on the current device, of rows of up to kSmemKeys
// tokens (an eighth of the keys and the histograms a CTA); 0 if unknown.
int resident_clusters() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  static std::mutex mu;
  static int cache[64] = {};   // + 1
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    auto fn = &evict_select_kernel<kCluster, true>;
    if (!ensure_smem_attr(reinterpret_cast<const void*>(fn), kSmemKeys * 4)) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = kSmemKeys / kCluster * 4;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    cache[dev] = n + 1;
  }
  return cache[dev] - 1;
}

}  // namespace

cudaError_t launch_evict_select(const float* weights, int max_tokens, const int32_t* seqlens, int batch, int budget,
                                int sink, int recent, int32_t* kept, int32_t* kept_lens, int32_t* status,
                                cudaStream_t stream) {
  const bool one = max_tokens <= kSmemKeys &&
                   (max_tokens <= kWideTokens + int64_t(kWidePerRow) * batch || batch > resident_clusters());
  const auto fn = one                                   ? &launch<1, true>
                  : max_tokens <= kCluster * kSmemKeys ? &launch<kCluster, true>
                                                         : &launch<kCluster, false>;
  return fn(weights, max_tokens, seqlens, batch, budget, sink, recent, kept, kept_lens, status, stream);
}

}  // namespace mla
