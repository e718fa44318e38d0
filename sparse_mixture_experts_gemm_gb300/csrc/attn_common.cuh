// attn_common.cuh -- what the kernels of a full-attention layer share: the
// sequences of a packed call and the pages of a 4-bit key/value cache.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

constexpr int kPage = 64;   // tokens per page of the cache
constexpr int kGroup = 64;  // columns that share a scale and a bias

// scores are exponents of 2: scale times this, which has to be finite
constexpr float kLog2e = 1.4426950408889634f, kMostScale = 2.35e38f;

// rows lo .. hi of sequence i; offsets outside [0, total] or running backwards
// are clamped.  offsets null: n sequences of total / n rows.
__device__ __forceinline__ void seq_rows(const int *offsets, int n, long long total, int i, int &lo,
                                         int &hi) {
  if (offsets) {
    lo = static_cast<int>(min(max(static_cast<long long>(offsets[i]), 0LL), total));
    hi = static_cast<int>(min(max(static_cast<long long>(offsets[i + 1]), static_cast<long long>(lo)), total));
  } else {
    const int len = static_cast<int>(total / n);
    lo = i * len;
    hi = lo + len;
  }
}

// A key/value cache: codes [pages][2][heads][64][D / 2] (keys, then values; the
// even column in the low half of a byte), affine [pages][2][heads][64][D / 64][2]
// (bf16 scale, bias).  table [n_seq][width]: page numbers of each sequence.
struct CacheArgs {
  uint8_t *codes;
  uint32_t *affine;  // one (scale, bias) pair per word, the scale in the low half
  const int *table;
  long long n_pages;
  int width, H, D;
  int *status;
};

// the page of position `at` of sequence i, -1 where there is none
__device__ __forceinline__ int page_of(const CacheArgs &c, int i, long long at) {
  if (at < 0 || at >= static_cast<long long>(c.width) * kPage) return -1;
  const int p = c.table[static_cast<long long>(i) * c.width + at / kPage];
  return p >= 0 && p < c.n_pages ? p : -1;
}
// the row of a page's token: index into codes in rows of D / 2 bytes, into
// affine in rows of D / 64 words
__device__ __forceinline__ long long cache_row(const CacheArgs &c, int page, int which, int h, int place) {
  return ((static_cast<long long>(page) * 2 + which) * c.H + h) * kPage + place;
}

// two fp32 values side by side
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(uint64_t p, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// one launch as a programmatic dependent of the kernel before it
template <typename K, typename... Args>
cudaError_t launch_attn(K kern, dim3 grid, int threads, int smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

inline bool off_boundary(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) != 0; }

}  // namespace moe
