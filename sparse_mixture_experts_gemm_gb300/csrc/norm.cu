// norm.cu -- root-mean-square norm with the residual's addition, kept in the
// row's type or quantised to e4m3 codes with one scale per row, and the same
// quantisation without the norm (the C ABI in include/moe.h).
//
// Per row:  s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s w r,
//           scale = max|y| / 448,  code = e4m3(y / scale).
// The order of the products is (s w) r, so that max|y| = max|s w| r (rounding
// is monotone) and y / scale = s w (448 / max|s w|): the mean square and the
// maximum come out of one reduction, and the row is read once and stays in
// registers.  Everything is computed in fp32 from the unrounded sum s; sum,
// out, codes and scales are each rounded once.  The maximum is taken over the
// bit patterns of |s w| as integers, where a NaN is larger than every number:
// a row that holds a NaN or an infinity gets NaN codes and a NaN scale.
//
// Bound by memory: 7 bytes per element with a bf16 residual and codes.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"

namespace moe {

namespace {

constexpr int kMaxNormD = 16384;

struct NormArgs {
  const void *x, *residual, *weight;  // residual, weight: null where there is none
  void *sum, *out;                    // null where not asked for
  uint8_t *codes;
  float *scales;
  long long rows, x_stride, r_stride;  // strides in elements
  int d;
  float eps;
  bool wide;  // every row of every tensor starts on a 16-byte boundary (codes: 8)
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[V], bool wide) {
  if constexpr (V == 1) {
    v[0] = static_cast<float>(*p);
  } else {
    alignas(16) T t[V];
    if (wide) {
      *reinterpret_cast<uint4 *>(t) = *reinterpret_cast<const uint4 *>(p);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) t[e] = p[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = static_cast<float>(t[e]);
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[V], bool wide) {
  if constexpr (V == 1) {
    *p = static_cast<T>(v[0]);
  } else {
    alignas(16) T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = static_cast<T>(v[e]);
    if (wide) {
      *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(t);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) p[e] = t[e];
    }
  }
}

__device__ __forceinline__ uint32_t code2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

template <int V>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&v)[V], bool wide) {
  if (V == 1 || !wide) {
#pragma unroll
    for (int e = 0; e < V; ++e) p[e] = __nv_cvt_float_to_fp8(v[e], __NV_SATFINITE, __NV_E4M3);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint32_t *>(p) = code2(v[0], v[1]) | code2(v[2], v[3]) << 16;
  } else {
    *reinterpret_cast<uint2 *>(p) = make_uint2(code2(v[0], v[1]) | code2(v[2], v[3]) << 16,
                                               code2(v[4], v[5]) | code2(v[6], v[7]) << 16);
  }
}

}  // namespace

// kTpr threads hold one row: thread i has the vectors i, i + kTpr, .. of V
// elements, kPer of them.  Blocks of max(kTpr, 128) threads.
template <typename T, int V, int kTpr, int kPer>
__global__ void __launch_bounds__(kTpr > 128 ? kTpr : 128) norm_kernel(const NormArgs a) {
  constexpr int kRows = kTpr >= 128 ? 1 : 128 / kTpr;
  constexpr int kW = kTpr / 32;  // warps per row
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / kTpr;
  if (row >= a.rows) return;  // (whole warps; whole blocks where kW > 1)
  const int t = threadIdx.x % kTpr;
  const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
  const T *w = static_cast<const T *>(a.weight);
  float v[kPer][V];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int c = (p * kTpr + t) * V;
    if (c < a.d)
      load_vec<T, V>(x + c, v[p], a.wide);
    else
#pragma unroll
      for (int e = 0; e < V; ++e) v[p][e] = 0.0f;
  }
  if (a.residual) {
    const T *r = static_cast<const T *>(a.residual) + row * a.r_stride;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int c = (p * kTpr + t) * V;
      if (c < a.d) {
        float u[V];
        load_vec<T, V>(r + c, u, a.wide);
#pragma unroll
        for (int e = 0; e < V; ++e) v[p][e] += u[e];
      }
    }
  }
  if (a.sum) {
    T *s = static_cast<T *>(a.sum) + row * a.d;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int c = (p * kTpr + t) * V;
      if (c < a.d) store_vec<T, V>(s + c, v[p], a.wide);
    }
  }
  // mean square, and max|s w| as a bit pattern
  float ss = 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int c = (p * kTpr + t) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) ss = fmaf(v[p][e], v[p][e], ss);
    if (w && c < a.d) {
      float u[V];
      load_vec<T, V>(w + c, u, a.wide);
#pragma unroll
      for (int e = 0; e < V; ++e) v[p][e] *= u[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(fabsf(v[p][e])));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if constexpr (kW > 1) {
    __shared__ float s_ss[kW];
    __shared__ uint32_t s_top[kW];
    if ((t & 31) == 0) {
      s_ss[t >> 5] = ss;
      s_top[t >> 5] = top;
    }
    __syncthreads();
    ss = 0.0f;
    top = 0;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      ss += s_ss[i];
      top = max(top, s_top[i]);
    }
  }
  const float r = w ? rsqrtf(ss / static_cast<float>(a.d) + a.eps) : 1.0f;
  if (a.out) {
    T *o = static_cast<T *>(a.out) + row * a.d;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int c = (p * kTpr + t) * V;
      if (c < a.d) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[p][e] *= r;
        store_vec<T, V>(o + c, v[p], a.wide);
      }
    }
  }
  if (a.codes) {
    const float m = __uint_as_float(top);
    const bool finite = top < 0x7f800000u;
    const float scale = finite ? m * r / 448.0f : __uint_as_float(0x7fffffffu);
    // rows of tiny values are lifted by an exact power of two first, so that
    // 448 / m stays finite
    const float lift = m < 0x1p-60f ? 0x1p80f : 1.0f;
    const float f = finite ? (scale == 0.0f ? 0.0f : 448.0f / (m * lift)) : scale;
    uint8_t *q = a.codes + row * a.d;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int c = (p * kTpr + t) * V;
      if (c < a.d) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[p][e] = v[p][e] * lift * f;
        store_codes<V>(q + c, v[p], a.wide);
      }
    }
    if (t == 0) a.scales[row] = scale;
  }
}

namespace {

template <typename T, int V, int kTpr, int kPer>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) {
  constexpr int kRows = kTpr >= 128 ? 1 : 128 / kTpr;
  const long long grid = (a.rows + kRows - 1) / kRows;
  norm_kernel<T, V, kTpr, kPer>
      <<<static_cast<unsigned>(grid), kTpr > 128 ? kTpr : 128, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick_norm(const NormArgs &a, cudaStream_t st) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  // The width alone decides which thread holds which elements, so a result
  // does not depend on where its tensors lie.
  if (a.d % V == 0) {
    const int n = a.d / V;
    if (n <= 128) return launch_norm<T, V, 32, 4>(a, st);
    if (n <= 256) return launch_norm<T, V, 256, 1>(a, st);
    if (n <= 512) return launch_norm<T, V, 256, 2>(a, st);
    if (n <= 1024) return launch_norm<T, V, 256, 4>(a, st);
    return launch_norm<T, V, 1024, 4>(a, st);
  }
  if (a.d <= 256) return launch_norm<T, 1, 32, 8>(a, st);
  if (a.d <= 1024) return launch_norm<T, 1, 256, 4>(a, st);
  if (a.d <= 2048) return launch_norm<T, 1, 256, 8>(a, st);
  return launch_norm<T, 1, 1024, 16>(a, st);
}

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) != 0; }

int run_norm(NormArgs a, moe_dtype dtype, cudaStream_t st) {
  const uintptr_t esz = dtype == MOE_BF16 ? 2 : 4;
  const void *ptrs[] = {a.x, a.residual, a.weight, a.sum, a.out};
  a.wide = a.d % static_cast<int>(16 / esz) == 0 && a.x_stride % static_cast<int>(16 / esz) == 0 &&
             (!a.residual || a.r_stride % static_cast<int>(16 / esz) == 0) && !misaligned(a.codes, 8);
  for (const void *p : ptrs) {
    if (misaligned(p, esz)) return MOE_ERR_ALIGNMENT;
    a.wide = a.wide && !misaligned(p, 16);
  }
  if (misaligned(a.scales, 4)) return MOE_ERR_ALIGNMENT;
  const cudaError_t e =
      dtype == MOE_BF16 ? pick_norm<__nv_bfloat16>(a, st) : pick_norm<float>(a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// the checks that the three entry points share; MOE_OK with rows == 0 is "nothing to do"
int check_norm(const void *x, moe_dtype dtype, long long rows, int d, long long x_stride) {
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (rows < 0 || d <= 0 || x_stride < d) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && !x) return MOE_ERR_INVALID_ARG;
  if (d > kMaxNormD || rows > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int add_rmsnorm(const void *x, const void *residual, const void *weight, moe_dtype dtype,
                long long rows, int d, long long x_stride, long long r_stride, float eps, void *sum,
                void *out, uint8_t *codes, float *scales, void *stream) {
  const int rc = check_norm(x, dtype, rows, d, x_stride);
  if (rc != MOE_OK) return rc;
  if (!(eps >= 0.0f) || (residual && r_stride < d)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!weight) return MOE_ERR_INVALID_ARG;
  const NormArgs a = {x, residual, weight, sum, out, codes, scales, rows, x_stride, r_stride, d, eps, false};
  return run_norm(a, dtype, static_cast<cudaStream_t>(stream));
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_add_rmsnorm(const void *x, const void *residual, const void *weight,
                               moe_dtype dtype, long long rows, int d, long long x_stride,
                               long long residual_stride, float eps, void *sum, void *out,
                               void *cuda_stream) {
  if (rows > 0 && !out) return MOE_ERR_INVALID_ARG;
  return add_rmsnorm(x, residual, weight, dtype, rows, d, x_stride, residual_stride, eps, sum, out,
                     nullptr, nullptr, cuda_stream);
}

extern "C" int moe_add_rmsnorm_fp8(const void *x, const void *residual, const void *weight,
                                   moe_dtype dtype, long long rows, int d, long long x_stride,
                                   long long residual_stride, float eps, void *sum, uint8_t *codes,
                                   float *scales, void *cuda_stream) {
  if (rows > 0 && (!codes || !scales)) return MOE_ERR_INVALID_ARG;
  return add_rmsnorm(x, residual, weight, dtype, rows, d, x_stride, residual_stride, eps, sum,
                     nullptr, codes, scales, cuda_stream);
}

extern "C" int moe_quantize_fp8(const void *w, moe_dtype dtype, long long rows, int cols,
                                long long stride, uint8_t *codes, float *scales, void *cuda_stream) {
  const int rc = check_norm(w, dtype, rows, cols, stride);
  if (rc != MOE_OK) return rc;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales) return MOE_ERR_INVALID_ARG;
  const NormArgs a = {w, nullptr, nullptr, nullptr, nullptr, codes, scales, rows, stride, 0, cols, 0.0f, false};
  return run_norm(a, dtype, static_cast<cudaStream_t>(cuda_stream));
}
