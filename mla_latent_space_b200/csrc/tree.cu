// Ancestor masks of drafted token trees.  Node i of a tree sees the drafted
// tokens on its path to the root: itself, parents[i], its parent, and so on
// until -1, where the path meets the committed prefix.
//
// One thread owns one 64-bit word of one node's row and walks that node's
// path, keeping the bits that fall into its word.  Parents come before their
// children, so every walk ends; a parent that does not is flagged and read
// as -1.  The parents of the request sit in shared memory, so a step of the
// walk costs one shared-memory latency; the kernel is bound by the deepest
// path (a few microseconds at most for a chain of 64 nodes).
#include <cuda_runtime.h>

#include "kernel_util.cuh"

namespace mla {

namespace {

constexpr int kMaskThreads = 256;
constexpr int kMaskSmemNodes = 8192;   // trees up to this size are walked in shared memory

__global__ void __launch_bounds__(kMaskThreads)
tree_mask_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ draft_lens, int s_q, int words,
                 int64_t* __restrict__ mask, int32_t* __restrict__ status) {
  extern __shared__ int32_t par_sm[];
  const int r = blockIdx.y;
  const int32_t* par_g = parents + size_t(r) * s_q;
  int n = draft_lens != nullptr ? draft_lens[r] : s_q;
  bool bad = n < 0 || n > s_q;
  n = max(0, min(n, s_q));
  const bool in_smem = s_q <= kMaskSmemNodes;
  if (in_smem) {
    for (int i = threadIdx.x; i < n; i += kMaskThreads) {
      const int p = par_g[i];
      bad |= p < -1 || p >= i;
      par_sm[i] = p < -1 || p >= i ? -1 : p;
    }
    __syncthreads();
  }
  const int64_t cells = int64_t(s_q) * words;
  const int64_t stride = int64_t(gridDim.x) * kMaskThreads;
  for (int64_t c = int64_t(blockIdx.x) * kMaskThreads + threadIdx.x; c < cells; c += stride) {
    const int i = int(c / words), w = int(c % words);
    uint64_t bits = 0;
    for (int j = i < n ? i : -1; j >= 64 * w;) {   // a path only descends: below the word, nothing is left
      if ((j >> 6) == w) bits |= 1ull << (j & 63);
      int p;
      if (in_smem) {
        p = par_sm[j];
      } else {
        p = par_g[j];
        if (p < -1 || p >= j) {
          bad = true;
          p = -1;
        }
      }
      j = p;
    }
    mask[size_t(r) * size_t(cells) + size_t(c)] = int64_t(bits);
  }
  if (bad && status != nullptr) atomicOr(status, kStatusBadInput);
}

}  // namespace

cudaError_t launch_tree_mask(const int32_t* parents, const int32_t* draft_lens, int batch, int s_q, int64_t* mask,
                             int32_t* status, cudaStream_t stream) {
  const int words = (s_q + 63) / 64;
  const int64_t cells = int64_t(s_q) * words;
  const int64_t blocks = ceil_div64(cells, kMaskThreads);
  const size_t smem = s_q <= kMaskSmemNodes ? size_t(s_q) * 4 : 0;
  tree_mask_kernel<<<dim3(unsigned(blocks < 1024 ? blocks : 1024), unsigned(batch)), kMaskThreads, smem, stream>>>(
      parents, draft_lens, s_q, words, mask, status);
  return cudaGetLastError();
}

}  // namespace mla
