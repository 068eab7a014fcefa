// Device helpers shared by the decode and combine kernels: schedule walking,
// output / partial-slot addressing and element conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <mutex>

#include "common.cuh"

namespace mla {

// Raises a kernel's dynamic shared-memory limit on the CURRENT device, once
// per (kernel, device): the attribute is per device, so a process that
// launches on several GPUs sets it on each of them.  Returns false when the
// runtime refuses it.  Device ordinals at or above 64 are set on every call.
inline bool ensure_smem_attr(const void* fn, int bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
  constexpr int kFns = 16;
  static std::mutex mu;
  static const void* fns[kFns] = {};
  static uint64_t done[kFns] = {};
  std::lock_guard<std::mutex> lock(mu);
  int i = 0;
  while (i < kFns && fns[i] != nullptr && fns[i] != fn) ++i;
  if (i < kFns && fns[i] == fn && dev < 64 && ((done[i] >> dev) & 1u)) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (i < kFns && dev < 64) {
    fns[i] = fn;
    done[i] |= uint64_t(1) << dev;
  }
  return true;
}

struct SchedView {
  const int32_t* hdr;
  const int32_t* workers;
  const int32_t* tiles;
  int W, num_tiles, tiles_per_req, batch, s_q, heads, causal, max_pages;

  __device__ __forceinline__ explicit SchedView(const void* p) {
    hdr = static_cast<const int32_t*>(p);
    W = hdr[H_WORKERS];
    num_tiles = hdr[H_TILES];
    tiles_per_req = hdr[H_TILES_PER_REQ];
    batch = hdr[H_BATCH];
    s_q = hdr[H_SQ];
    heads = hdr[H_HEADS];
    causal = hdr[H_CAUSAL];
    max_pages = hdr[H_MAX_PAGES];
    workers = hdr + kHeaderInts;
    tiles = workers + size_t(W) * kWorkerInts;
  }
  __device__ __forceinline__ int tile_pages(int T) const { return tiles[size_t(T) * kTileInts + T_PAGES]; }
  __device__ __forceinline__ int tile_splits(int T) const { return tiles[size_t(T) * kTileInts + T_SPLITS]; }
  __device__ __forceinline__ int tile_slot_base(int T) const { return tiles[size_t(T) * kTileInts + T_SLOT_BASE]; }
};

// One piece of a worker's range: pages [p0, p1) of tile T, split index `split`.
struct Piece {
  int T, p0, p1, split;
};

// Iterates the pieces of worker w in order.  Usage:
//   PieceIter it(sv, w); Piece pc; while (it.next(&pc)) {...}
struct PieceIter {
  const SchedView& sv;
  int tb, pb, te, pe, fs, T;
  __device__ __forceinline__ PieceIter(const SchedView& s, int w) : sv(s) {
    const int32_t* wm = s.workers + size_t(w) * kWorkerInts;
    tb = wm[W_TILE_BEGIN]; pb = wm[W_PAGE_BEGIN];
    te = wm[W_TILE_END]; pe = wm[W_PAGE_END]; fs = wm[W_FIRST_SPLIT];
    T = tb;
  }
  __device__ __forceinline__ bool next(Piece* pc) {
    while (T <= te && T < sv.num_tiles) {
      int pages = sv.tile_pages(T);
      int p0 = T == tb ? pb : 0;
      int p1 = T == te ? pe : pages;
      if (p1 > pages) p1 = pages;
      int split = T == tb ? fs : 0;
      int cur = T++;
      if (p0 < p1) { *pc = Piece{cur, p0, p1, split}; return true; }
    }
    return false;
  }
};

// Partial-slot regions are laid out for `cap` slots, the capacity the host
// derives from the workspace size (so decode and combine agree on it).
__device__ __forceinline__ float* ws_partial_o(void* ws, int cap, int slot) {
  (void)cap;
  return reinterpret_cast<float*>(static_cast<char*>(ws) + kStatusBytes) + size_t(slot) * kSlotOFloats;
}
__device__ __forceinline__ float* ws_partial_lse(void* ws, int cap, int slot) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + kStatusBytes) + size_t(cap) * kSlotOFloats +
         size_t(slot) * MLA_TILE_ROWS;
}
__device__ __forceinline__ int32_t* ws_status(void* ws) { return static_cast<int32_t*>(ws); }

__device__ __forceinline__ void flag_status(void* ws, int32_t bits) { atomicOr(ws_status(ws), bits); }

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  __half_raw hr = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
  return __half2float(__half(hr));
}

__device__ __forceinline__ float bf16_bits_to_float(uint16_t b) {
  return __uint_as_float(uint32_t(b) << 16);
}

// Largest |value| of the two bf16 values of w.
__device__ __forceinline__ float bf16_abs_max(uint32_t w) {
  return fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xFFFF0000u)));
}

// e with am / 2^e <= 448 (e4m3's largest finite value), the smallest such
// but at least -126, so that 2^-e stays finite (a row that small loses
// nothing that matters: its values still land in e4m3's range); 0 for
// am = 0 or a non-finite am (its NaN or infinity then reaches S as is).
// frexpf gives the estimate; the loops correct it by at most a few steps
// (at most 126 for a subnormal am) and always end.
__device__ __forceinline__ int pow2_scale_exp(float am) {
  if (!(am > 0.f) || !(am <= 3.402823466e38f)) return 0;
  int e = 0;
  frexpf(am * (1.f / 448.f), &e);   // am / 448 = m 2^e, 0.5 <= m < 1
  while (ldexpf(am, -e) > 448.f) ++e;
  while (e > -126 && ldexpf(am, -(e - 1)) <= 448.f) --e;
  return e < -126 ? -126 : e;
}

// Four bf16 values (w01, w23, low half first) times `inv` (a power of two)
// as e4m3 hi = RNE(x) and lo = RNE(x - hi), four bytes each, value 4k+j in
// byte j.  x - hi is exact in fp32.
__device__ __forceinline__ void split_e4m3x4(uint32_t w01, uint32_t w23, float inv, uint32_t* hi, uint32_t* lo) {
  const float2 a = make_float2(__uint_as_float(w01 << 16) * inv, __uint_as_float(w01 & 0xFFFF0000u) * inv);
  const float2 b = make_float2(__uint_as_float(w23 << 16) * inv, __uint_as_float(w23 & 0xFFFF0000u) * inv);
  const __nv_fp8x2_storage_t ha = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hb = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
  const float2 fa = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(ha, __NV_E4M3)));
  const float2 fb = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(hb, __NV_E4M3)));
  const __nv_fp8x2_storage_t la = __nv_cvt_float2_to_fp8x2(make_float2(a.x - fa.x, a.y - fa.y), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t lb = __nv_cvt_float2_to_fp8x2(make_float2(b.x - fb.x, b.y - fb.y), __NV_SATFINITE, __NV_E4M3);
  *hi = uint32_t(ha) | (uint32_t(hb) << 16);
  *lo = uint32_t(la) | (uint32_t(lb) << 16);
}

}  // namespace mla
