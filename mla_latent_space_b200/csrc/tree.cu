// Ancestor masks of drafted token trees.  Node i of a tree sees the drafted
// tokens on its path to the root: itself, parents[i], its parent, and so on
// until -1, where the path meets the committed prefix.
//
// Up to 8192 nodes one thread owns one 64-bit word of one node's row and walks
// that node's path, keeping the bits that fall into its word.  Parents come
// before their children, so every walk ends; a parent that does not is flagged
// and read as -1.  The parents of the request sit in shared memory, so a step
// of the walk costs one shared-memory latency; the kernel is bound by the
// deepest path (a few microseconds at most for a chain of 64 nodes).
//
// A walk costs nodes x words x depth, and where the parents do not fit shared
// memory eleven times as much for twice the nodes (chains of 16384 and 32768
// nodes: 15 and 171 ms; the limit of 2^20 would take hours).  Larger trees are
// swept instead: a warp owns one word of all rows and takes 32 nodes at a
// time; a row is its parent's row and the node's own bit, the parent's read
// back from the mask, or from a lane of the same 32 (pointer jumping, 5
// steps): 0.3, 0.7 and, at 131072 nodes, 3.9 ms, whatever the depth.  Walk
// and sweep of 1024 nodes x 16 requests, 4096 and 8192 nodes: 97 / 15, 253 /
// 76 and 1411 / 161 us of a chain, 4.3 / 17, 5.3 / 91 and 13 / 185 of a random
// tree, whose paths are short, as those of drafted trees are.
#include <cuda_runtime.h>

#include "kernel_util.cuh"

namespace mla {

namespace {

constexpr int kMaskThreads = 256;
constexpr int kMaskSmemNodes = 8192;   // trees up to this size are walked in shared memory, larger ones swept

__global__ void __launch_bounds__(kMaskThreads)
tree_mask_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ draft_lens, int s_q, int words,
                 int64_t* __restrict__ mask, int32_t* __restrict__ status) {
  extern __shared__ int32_t par_sm[];
  const int r = blockIdx.y;
  const int32_t* par_g = parents + size_t(r) * s_q;
  int n = draft_lens != nullptr ? draft_lens[r] : s_q;
  bool bad = n < 0 || n > s_q;
  n = max(0, min(n, s_q));
  for (int i = threadIdx.x; i < n; i += kMaskThreads) {
    const int p = par_g[i];
    bad |= p < -1 || p >= i;
    par_sm[i] = p < -1 || p >= i ? -1 : p;
  }
  __syncthreads();
  const int64_t cells = int64_t(s_q) * words;
  const int64_t stride = int64_t(gridDim.x) * kMaskThreads;
  for (int64_t c = int64_t(blockIdx.x) * kMaskThreads + threadIdx.x; c < cells; c += stride) {
    const int i = int(c / words), w = int(c % words);
    uint64_t bits = 0;
    for (int j = i < n ? i : -1; j >= 64 * w; j = par_sm[j])   // a path only descends: below the word, nothing is left
      if ((j >> 6) == w) bits |= 1ull << (j & 63);
    mask[size_t(r) * size_t(cells) + size_t(c)] = int64_t(bits);
  }
  if (bad && status != nullptr) atomicOr(status, kStatusBadInput);
}

// A warp owns word w of every row of a request.  (mask is read where the warp
// has written it.)
__global__ void __launch_bounds__(kMaskThreads)
tree_mask_sweep_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ draft_lens, int s_q, int words,
                       int64_t* mask, int32_t* __restrict__ status) {
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  const int w = int(blockIdx.x) * (kMaskThreads / 32) + int(threadIdx.x >> 5);
  if (w >= words) return;   // (a whole warp)
  const int32_t* par = parents + size_t(r) * s_q;
  int64_t* m = mask + size_t(r) * size_t(s_q) * words + w;
  int n = draft_lens != nullptr ? draft_lens[r] : s_q;
  bool bad = n < 0 || n > s_q;
  n = max(0, min(n, s_q));
  for (int i0 = 0; i0 < s_q; i0 += 32) {   // (s_q <= 2^20)
    const int i = i0 + lane;
    uint64_t bits = 0;
    int up = -1;   // the lane of this node's parent, if it is one of these 32
    if (i < n && (i0 >= 64 * w || w == 0)) {   // (rows above the word's own are zero; the first word's warp checks all)
      int p = par[i];
      if (p < -1 || p >= i) {
        bad = true;
        p = -1;
      }
      if ((i >> 6) == w) bits = 1ull << (i & 63);
      if (p >= i0) up = p - i0;
      else if (p >= 64 * w) bits |= uint64_t(m[size_t(p) * words]);
    }
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int from = up < 0 ? lane : up;
      const uint64_t b = __shfl_sync(0xffffffffu, bits, from);
      const int u = __shfl_sync(0xffffffffu, up, from);
      if (up >= 0) {
        bits |= b;
        up = u;
      }
    }
    if (i < s_q) m[size_t(i) * words] = int64_t(bits);
    __syncwarp();
  }
  if (bad && status != nullptr) atomicOr(status, kStatusBadInput);
}

}  // namespace

cudaError_t launch_tree_mask(const int32_t* parents, const int32_t* draft_lens, int batch, int s_q, int64_t* mask,
                             int32_t* status, cudaStream_t stream) {
  const int words = (s_q + 63) / 64;
  if (s_q <= kMaskSmemNodes) {
    const int64_t blocks = ceil_div64(int64_t(s_q) * words, kMaskThreads);
    tree_mask_kernel<<<dim3(unsigned(blocks < 1024 ? blocks : 1024), unsigned(batch)), kMaskThreads, size_t(s_q) * 4,
                       stream>>>(parents, draft_lens, s_q, words, mask, status);
  } else {
    const int per = kMaskThreads / 32;
    tree_mask_sweep_kernel<<<dim3(unsigned((words + per - 1) / per), unsigned(batch)), kMaskThreads, 0, stream>>>(
        parents, draft_lens, s_q, words, mask, status);
  }
  return cudaGetLastError();
}

}  // namespace mla
