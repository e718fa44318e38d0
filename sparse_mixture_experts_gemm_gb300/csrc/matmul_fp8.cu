// matmul_fp8.cu -- matrix product of e4m3 codes with a scale per token and a
// scale per output channel (moe_matmul_fp8 in include/moe.h):
//     out[t][n] = x_scale[t] * w_scale[n] * sum_k x[t][k] * w[n][k]
// The scales do not depend on k, so the sum runs over the codes alone, in
// fp32, and each output is scaled and rounded to bf16 once.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"

namespace moe {

namespace {

constexpr int kTile = 64;  // tokens and channels of a block's tile
constexpr int kTileK = 16;

struct MatmulArgs {
  const uint8_t *x, *w;
  const float *xs, *ws;
  __nv_bfloat16 *out;
  int T, N, K;
  long long x_stride, w_stride, out_stride;
};

__device__ __forceinline__ float e4m3(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

}  // namespace

// 256 threads, 4 x 4 outputs each, codes widened to fp32 in shared memory.
__global__ void __launch_bounds__(256) matmul_fp8_kernel(const MatmulArgs a) {
  __shared__ float sx[kTileK][kTile + 1], sw[kTileK][kTile + 1];
  const int n0 = blockIdx.x * kTile, t0 = blockIdx.y * kTile;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kTileK) {
    for (int i = threadIdx.x; i < kTile * kTileK; i += 256) {
      const int r = i / kTileK, c = i % kTileK;
      sx[c][r] = t0 + r < a.T ? e4m3(a.x[(t0 + r) * a.x_stride + k0 + c]) : 0.0f;
      sw[c][r] = n0 + r < a.N ? e4m3(a.w[(n0 + r) * a.w_stride + k0 + c]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kTileK; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sx[c][ty + 16 * i], sw[c][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (t < a.T && n < a.N)
        a.out[t * a.out_stride + n] = __float2bfloat16_rn(acc[i][j] * a.xs[t] * a.ws[n]);
    }
}

}  // namespace moe

using namespace moe;

extern "C" int moe_matmul_fp8(const uint8_t *x, const float *x_scales, int T, long long x_stride,
                              const uint8_t *w, const float *w_scales, int N, int K,
                              long long w_stride, void *out, long long out_stride,
                              void *cuda_stream) {
  if (T < 0 || N <= 0 || K <= 0 || x_stride < K || w_stride < K || out_stride < N)
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !x_scales || !w || !w_scales || !out)) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || T > (1 << 22) || N > (1 << 20) || K > (1 << 17)) return MOE_ERR_UNSUPPORTED;
  auto misaligned = [](const void *p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) % n) != 0;
  };
  if (misaligned(x, 16) || misaligned(w, 16) || x_stride % 16 != 0 || w_stride % 16 != 0 ||
      misaligned(x_scales, 4) || misaligned(w_scales, 4) || misaligned(out, 2))
    return MOE_ERR_ALIGNMENT;
  if (T == 0) return MOE_OK;
  const MatmulArgs a = {x, w, x_scales, w_scales, static_cast<__nv_bfloat16 *>(out), T, N, K,
                        x_stride, w_stride, out_stride};
  matmul_fp8_kernel<<<dim3((N + kTile - 1) / kTile, (T + kTile - 1) / kTile), 256, 0,
                      static_cast<cudaStream_t>(cuda_stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
