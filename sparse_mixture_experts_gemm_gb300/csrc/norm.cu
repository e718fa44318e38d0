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
// Bound by memory: 7 bytes per element with a bf16 residual and codes.  A block
// holds one row.  Rows of whole 16-byte vectors move as such; rows of another
// width one element per lane and load, neighbouring lanes on neighbouring
// elements (16,384 rows of 1,001: 29 us; cutting such rows into vectors with
// ragged ends took 32, because the weights lie differently in every row).  Odd
// widths past 4,096 leave that rate: codes of 16,384 x 4,097 take 292 us.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kMaxNormD = 16384;

// The sum of squares is taken again from elements times kDown or kUp where it
// exceeds fp32's range, or where it is below kTinySum and eps below kTinyEps
// (squares under 2^-126 lose bits, which an eps of normal size hides).  Scaled,
// 2^128 squares to 2^112 and 2^-149 to 2^-98, 16,384 of either add up in range.
constexpr float kMaxFloat = 3.402823466e38f, kTinySum = 0x1p-90f, kTinyEps = 0x1p-90f;
constexpr float kDown = 0x1p-72f, kUp = 0x1p100f;

struct NormArgs {
  const void *x, *residual, *weight;  // residual, weight: null where there is none
  void *sum, *out;                    // null where not asked for
  uint8_t *codes;
  float *scales;
  long long rows, x_stride, r_stride;  // strides in elements
  int d;
  float eps;
  bool wide;  // every row of every tensor starts on a 16-byte boundary (codes: 8 or 4)
};

// A thread's vectors of a row: columns c0 + p step .. + V - 1, p < kPer.
template <typename T, int V, int kPer>
__device__ __forceinline__ void load_row(const T *row, int c0, int step, int d, bool wide,
                                         float (&v)[kPer][V]) {
  if constexpr (V == 1) {
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int c = c0 + p * step;
      v[p][0] = c < d ? static_cast<float>(row[c]) : 0.0f;
    }
  } else if (wide) {
    uint4 u[kPer];
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      u[p] = make_uint4(0, 0, 0, 0);
      if (c0 + p * step < d) u[p] = *reinterpret_cast<const uint4 *>(row + c0 + p * step);
    }
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const uint32_t w[4] = {u[p].x, u[p].y, u[p].z, u[p].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (V == 8) {
          v[p][2 * i] = __uint_as_float(w[i] << 16);
          v[p][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
          v[p][i] = __uint_as_float(w[i]);
        }
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < kPer; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = c0 + p * step;
        v[p][e] = c < d ? static_cast<float>(row[c + e]) : 0.0f;
      }
  }
}

template <typename T, int V, int kPer>
__device__ __forceinline__ void store_row(T *row, int c0, int step, int d, bool wide,
                                          const float (&v)[kPer][V]) {
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int c = c0 + p * step;
    if (c >= d) continue;
    if (V == 1 || !wide) {
#pragma unroll
      for (int e = 0; e < V; ++e) row[c + e] = static_cast<T>(v[p][e]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (V == 8) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[p][2 * i], v[p][2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
          w[i] = __float_as_uint(v[p][i]);
        }
      }
      *reinterpret_cast<uint4 *>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

__device__ __forceinline__ uint32_t code2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

template <int V, int kPer>
__device__ __forceinline__ void store_codes(uint8_t *row, int c0, int step, int d, bool wide,
                                            const float (&v)[kPer][V]) {
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int c = c0 + p * step;
    if (c >= d) continue;
    if (V == 1 || !wide) {
#pragma unroll
      for (int e = 0; e < V; ++e) row[c + e] = __nv_cvt_float_to_fp8(v[p][e], __NV_SATFINITE, __NV_E4M3);
    } else {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        w[i] = code2(v[p][4 * i], v[p][4 * i + 1]) | code2(v[p][4 * i + 2], v[p][4 * i + 3]) << 16;
      if constexpr (V == 8)
        *reinterpret_cast<uint2 *>(row + c) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t *>(row + c) = w[0];
    }
  }
}

}  // namespace

// Thread i has the vectors i, i + kThreads, .. of V elements, kPer of them.
template <typename T, int V, int kThreads, int kPer>
__global__ void __launch_bounds__(kThreads) norm_kernel(const NormArgs a) {
  constexpr int kW = kThreads / 32;
  __shared__ float s_ss[kW];
  __shared__ uint32_t s_top[kW];
  const int t = threadIdx.x, d = a.d;
  pdl_wait();
  const long long row = blockIdx.x;
  const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
  const T *w = static_cast<const T *>(a.weight);
  const int c0 = t * V;
  constexpr int step = kThreads * V;
  float v[kPer][V];
  load_row<T, V, kPer>(x, c0, step, d, a.wide, v);
  if (a.residual) {
    float u[kPer][V];
    load_row<T, V, kPer>(static_cast<const T *>(a.residual) + row * a.r_stride, c0, step, d, a.wide, u);
#pragma unroll
    for (int p = 0; p < kPer; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) v[p][e] += u[p][e];
  }
  if (a.sum) store_row<T, V, kPer>(static_cast<T *>(a.sum) + row * d, c0, step, d, a.wide, v);
  // mean square, and max|s w| as a bit pattern
  float ss = 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < kPer; ++p)
#pragma unroll
    for (int e = 0; e < V; ++e) ss = fmaf(v[p][e], v[p][e], ss);
  // a thread whose own squares leave that range adds them up scaled, too
  const float part = ss;
  float scaled = 0.0f;
  if (part > kMaxFloat || (a.eps < kTinyEps && part < kTinySum)) {
    const float f = part > kMaxFloat ? kDown : kUp;
#pragma unroll
    for (int p = 0; p < kPer; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) scaled = fmaf(v[p][e] * f, v[p][e] * f, scaled);
  }
  if (w) {
    float u[kPer][V];
    load_row<T, V, kPer>(w, c0, step, d, a.wide, u);
#pragma unroll
    for (int p = 0; p < kPer; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) v[p][e] *= u[p][e];
  }
#pragma unroll
  for (int p = 0; p < kPer; ++p)
#pragma unroll
    for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(fabsf(v[p][e])));
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  top = __reduce_max_sync(0xffffffffu, top);
  if constexpr (kW > 1) {
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
  // the norm's factor is pre * r
  float r = 1.0f, pre = 1.0f;
  if (w) {
    const bool huge = ss > kMaxFloat, tiny = a.eps < kTinyEps && ss < kTinySum;
    if (huge || tiny) {  // (one answer in the whole block)
      // squares past fp32's range, or so small that they lose bits beside an
      // eps as small: the sum of the scaled elements' instead
      pre = huge ? kDown : kUp;
      float x = huge ? (part < kTinySum ? 0.0f : part <= kMaxFloat ? part * kDown * kDown : scaled) : scaled;
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if constexpr (kW > 1) {
        __syncthreads();
        if ((t & 31) == 0) s_ss[t >> 5] = x;
        __syncthreads();
        x = 0.0f;
        for (int i = 0; i < kW; ++i) x += s_ss[i];
      }
      ss = x;
    }
    r = rsqrtf(ss / static_cast<float>(d) + a.eps * pre * pre);
    // a row of zeros stays one where eps is 0 and r infinite
    if (top == 0) r = 0.0f;
  }
  if (a.out) {
#pragma unroll
    for (int p = 0; p < kPer; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) v[p][e] = v[p][e] * pre * r;
    store_row<T, V, kPer>(static_cast<T *>(a.out) + row * d, c0, step, d, a.wide, v);
  }
  if (a.codes) {
    const float m = __uint_as_float(top);
    const bool finite = top < 0x7f800000u;
    const float scale = finite ? m * pre * r / 448.0f : __uint_as_float(0x7fffffffu);
    // rows of tiny values are lifted by an exact power of two first, so that
    // 448 / m stays finite
    const float lift = m < 0x1p-60f ? 0x1p80f : 1.0f;
    float f = finite ? (scale == 0.0f ? 0.0f : 448.0f / (m * lift)) : scale;
    // a scale below 2^-126 is off by up to half of itself: the codes make up
    // for that, as y / scale does (the largest one may then be less than 448)
    if (finite && scale > 0.0f && scale < 0x1p-126f) f = pre * r / (scale * lift);
#pragma unroll
    for (int p = 0; p < kPer; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) v[p][e] = v[p][e] * lift * f;
    store_codes<V, kPer>(a.codes + row * d, c0, step, d, a.wide, v);
    if (t == 0) a.scales[row] = scale;
  }
}

namespace {

template <typename T, int V, int kThreads, int kPer>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_kernel<T, V, kThreads, kPer>, a);
}

// The width alone decides which thread holds which elements, so a row's result
// depends neither on where its tensors lie nor on how many rows there are.  Two
// to four vectors per thread (with a residual and codes, 16,384 rows of 2,048
// bf16 timed one call at a time: 42.4 us with 64 threads of 4, 42.6 with 128 of
// 2, 48.9 with 256 of 1; back to back 38.0 us, 6.2 TB/s; one row: 2.2 in a
// graph).  Rows off the 16-byte boundaries keep their elements' threads and are
// read element by element: codes of 16,384 x 4,096 from column 3 of a wider
// tensor 60 to 75 us, from column 0 46.
// Blocks that stay and take several rows, loading ahead, were slower (67 us).
template <typename T>
cudaError_t pick_norm(const NormArgs &a, cudaStream_t st) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  if (a.d % V != 0) {
    if (a.d <= 256) return launch_norm<T, 1, 64, 4>(a, st);
    if (a.d <= 1024) return launch_norm<T, 1, 128, 8>(a, st);
    if (a.d <= 2048) return launch_norm<T, 1, 256, 8>(a, st);
    if (a.d <= 4096) return launch_norm<T, 1, 512, 8>(a, st);
    return launch_norm<T, 1, 1024, 16>(a, st);
  }
  const int n = a.d / V;
  if (n <= 64) return launch_norm<T, V, 32, 2>(a, st);
  if (n <= 128) return launch_norm<T, V, 32, 4>(a, st);
  if (n <= 256) return launch_norm<T, V, 64, 4>(a, st);
  if (n <= 512) return launch_norm<T, V, 128, 4>(a, st);
  if (n <= 1024) return launch_norm<T, V, 256, 4>(a, st);
  if (n <= 2048) return launch_norm<T, V, 512, 4>(a, st);
  return launch_norm<T, V, 1024, 4>(a, st);
}

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) != 0; }

int run_norm(NormArgs a, moe_dtype dtype, cudaStream_t st) {
  const uintptr_t esz = dtype == MOE_BF16 ? 2 : 4;
  const int V = static_cast<int>(16 / esz);
  a.wide = a.x_stride % V == 0 && (!a.residual || a.r_stride % V == 0) && !misaligned(a.codes, V);
  const void *ptrs[] = {a.x, a.residual, a.weight, a.sum, a.out};
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
