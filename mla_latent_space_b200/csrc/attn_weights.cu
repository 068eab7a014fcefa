// Attention weights received by the cached tokens, accumulated over steps:
//   w[r][j] = decay * w[r][j] + sum over query rows (i, h) that see j of
//             exp(scale * q_{i,h} . C_j - lse_{i,h})
// with the lse that the decode returned.
//
// One CTA per (page, request): the page's 64 rows sit in shared memory as
// fp32, the query rows pass through in groups, and every thread holds one
// token's scores against a quarter of a group.
#include <cuda_runtime.h>

#include "kernel_util.cuh"

namespace mla {

namespace {

constexpr int kWThreads = 256;
constexpr int kWGroup = 16;                     // query rows per pass
constexpr int kWRow = MLA_D_QK + 1;             // padded row of floats
constexpr size_t kWSmem = sizeof(float) * (size_t(MLA_PAGE_SIZE) * kWRow + size_t(kWGroup) * MLA_D_QK + 4 * MLA_PAGE_SIZE);

struct WArgs {
  const uint16_t* q;
  const uint8_t* kv;
  const float* kv_scale;
  const int32_t* block_table;
  const int32_t* seqlens;
  const float* lse;
  float* weights;
  void* ws;
  float scale, decay;
  int s_q, heads, causal, max_pages, num_pages;
};

template <bool kFp8>
__global__ void __launch_bounds__(kWThreads) attn_weights_kernel(const WArgs a) {
  extern __shared__ float sm[];
  float* c_sm = sm;
  float* q_sm = c_sm + MLA_PAGE_SIZE * kWRow;
  float* part = q_sm + kWGroup * MLA_D_QK;
  const int r = blockIdx.y, j = blockIdx.x, tid = threadIdx.x;
  int t = a.seqlens[r];
  const int cap = a.max_pages * MLA_PAGE_SIZE;
  if ((t < 0 || t > cap) && j == 0 && tid == 0) flag_status(a.ws, kStatusBadSeqlen);
  t = max(0, min(t, cap));
  if (j * MLA_PAGE_SIZE >= t) return;
  const int page = a.block_table[size_t(r) * a.max_pages + j];
  const bool ok = page >= 0 && page < a.num_pages;
  if (!ok && tid == 0) flag_status(a.ws, kStatusBadPage);
  if (ok) {
    for (int e = tid; e < MLA_PAGE_SIZE * MLA_D_QK; e += kWThreads) {
      const int row = e / MLA_D_QK, col = e % MLA_D_QK;
      float v;
      if constexpr (kFp8) {
        const uint8_t* pg = a.kv + size_t(page) * (MLA_PAGE_SIZE * (MLA_D_V + 2 * MLA_D_ROPE));
        v = col < MLA_D_V ? e4m3_to_float(pg[row * MLA_D_V + col]) * a.kv_scale[size_t(page) * MLA_PAGE_SIZE + row]
                          : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(pg + MLA_PAGE_SIZE * MLA_D_V)[row * MLA_D_ROPE + col - MLA_D_V]);
      } else {
        v = bf16_bits_to_float(reinterpret_cast<const uint16_t*>(a.kv)[(size_t(page) * MLA_PAGE_SIZE + row) * MLA_D_QK + col]);
      }
      c_sm[row * kWRow + col] = v;
    }
  }
  const int tok = tid % MLA_PAGE_SIZE, part_id = tid / MLA_PAGE_SIZE;   // 4 rows of a group per thread
  const int pos = j * MLA_PAGE_SIZE + tok;
  const int rows = a.s_q * a.heads;
  float acc = 0.f;
  for (int g = 0; ok && g < rows; g += kWGroup) {
    __syncthreads();
    for (int e = tid; e < kWGroup * MLA_D_QK; e += kWThreads) {
      const int rho = g + e / MLA_D_QK;
      q_sm[e] = rho < rows ? bf16_bits_to_float(a.q[(size_t(r) * rows + rho) * MLA_D_QK + e % MLA_D_QK]) : 0.f;
    }
    __syncthreads();
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int d = 0; d < MLA_D_QK; ++d) {
      const float c = c_sm[tok * kWRow + d];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = fmaf(q_sm[(part_id * 4 + k) * MLA_D_QK + d], c, s[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int rho = g + part_id * 4 + k;
      if (rho >= rows || pos >= visible_len(t, a.s_q, rho / a.heads, a.causal)) continue;
      const float l = a.lse[size_t(r) * rows + rho];
      if (l != -INFINITY) acc += expf(s[k] * a.scale - l);
    }
  }
  part[part_id * MLA_PAGE_SIZE + tok] = acc;
  __syncthreads();
  if (tid < MLA_PAGE_SIZE && pos < t) {
    const float sum = (part[tid] + part[MLA_PAGE_SIZE + tid]) + (part[2 * MLA_PAGE_SIZE + tid] + part[3 * MLA_PAGE_SIZE + tid]);
    float* w = a.weights + size_t(r) * cap + pos;
    *w = a.decay != 0.f ? fmaf(a.decay, *w, sum) : sum;
  }
}

}  // namespace

size_t attn_weights_workspace_bytes(const mla_shape_t*, int) { return kStatusBytes; }

int launch_attn_weights(const mla_shape_t* shape, const void* q, const void* kv, const float* kv_scale,
                        const int32_t* block_table, const int32_t* seqlens, const float* lse, float scale, float decay,
                        float* weights, void* ws, int, cudaStream_t stream) {
  const bool fp8 = shape->cache_dtype == MLA_CACHE_FP8_E4M3;
  auto fn = fp8 ? &attn_weights_kernel<true> : &attn_weights_kernel<false>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(fn), int(kWSmem))) return MLA_ERR_CUDA;
  WArgs a{static_cast<const uint16_t*>(q), static_cast<const uint8_t*>(kv), kv_scale, block_table, seqlens, lse, weights,
          ws, scale, decay, shape->s_q, shape->num_heads, shape->causal, shape->max_pages_per_seq, shape->num_pages};
  fn<<<dim3(unsigned(shape->max_pages_per_seq), unsigned(shape->batch)), kWThreads, kWSmem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla
