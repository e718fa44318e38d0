// qk_rope.cu -- root-mean-square norm of every query and key head with the
// position rotation in the same pass (moe_qk_norm_rope in include/moe.h).
//
// Per head row of D columns:  y = x w / sqrt(mean(x^2) + eps);  the first R
// columns turn in pairs (i, i + R / 2) by a = position * inv_freq[i]:
//     out_i = y_i cos a - y_(i+R/2) sin a,  out_(i+R/2) = y_(i+R/2) cos a + y_i sin a
// Everything is fp32 from the bf16 inputs, rounded once.  The angle is not: a
// float32 of position 120,000 is off by up to 2^-8 turns of a radian, so the
// turns position * inv_freq / (2 pi) are formed in 64 bits, whole turns are
// dropped there, and sine and cosine see at most half a turn in fp32.
//
// Bound by memory, and by instructions on the way there.  A warp has one token and
// some of its rows, 16 columns of a row per lane: in the part that turns 8 and their 8
// partners, so that no value is exchanged (with 8 columns in one load and 8 shuffles
// a row 16,384 tokens of 18 heads of 256 took 67 us in place of 56, 5.4 TB/s).  The
// next row is on its way meanwhile; two rows ahead, or more warps by fewer registers
// (60 us at 72, 67 at 64), gained nothing.  The token's angles are made once, one
// frequency per lane, and handed round through shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "attn_common.cuh"

namespace moe {

namespace {

constexpr int kRopeWarps = 4;

struct RopeArgs {
  const __nv_bfloat16 *q, *k, *qw, *kw;
  __nv_bfloat16 *qo, *ko;
  const int *positions;
  const double *freq;
  long long tokens, qs, ks, qos, kos;  // strides in elements
  int Hq, Hk, rot;
  int split, per;  // warps of a token, rows of a warp
  float eps;
};

// squares past fp32's range, or so small that they lose bits beside an eps as
// small, are taken again from elements scaled by a power of two
constexpr float kMaxFloat = 3.402823466e38f, kTiny = 0x1p-90f, kDown = 0x1p-72f, kUp = 0x1p100f;

// 8 bf16 as pairs of fp32
__device__ __forceinline__ void unpack8(const uint4 &u, uint64_t (&v)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    split(v[i], a, b);
    w[i] = bf16x2_bits(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kRopeWarps * 32) qk_rope_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;  // lanes of a row, rows side by side
  __shared__ __align__(16) float s_cos[kRopeWarps][D / 2], s_sin[kRopeWarps][D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const long long unit = static_cast<long long>(blockIdx.x) * kRopeWarps + warp;
  const long long token = unit / a.split;
  if (token >= a.tokens) return;
  const int first = static_cast<int>(unit % a.split) * a.per, H = a.Hq + a.Hk, last = min(first + a.per, H);
  const int half = a.rot / 2, sub = lane / kLanes, l = lane % kLanes;
  const bool turned = 16 * l < a.rot;
  // this lane's columns: c0 .. c0 + 7, c1 .. c1 + 7
  const int c0 = turned ? 8 * l : a.rot + 8 * l - half, c1 = c0 + (turned ? half : (D - a.rot) / 2);

  uint4 next[2];
  auto fetch = [&](int r) {
    next[0] = next[1] = make_uint4(0, 0, 0, 0);
    if (r < last) {
      const __nv_bfloat16 *x = r < a.Hq ? a.q + token * a.qs + r * D : a.k + token * a.ks + (r - a.Hq) * D;
      next[0] = *reinterpret_cast<const uint4 *>(x + c0);
      next[1] = *reinterpret_cast<const uint4 *>(x + c1);
    }
  };
  fetch(first + sub);
  if (half) {
    const double p = static_cast<double>(a.positions[token]) * 0.15915494309189533577;  // 1 / (2 pi)
    for (int i = lane; i < half; i += 32) {
      const double t = p * a.freq[i];
      float sn, cs;
      sincospif(2.0f * static_cast<float>(t - rint(t)), &sn, &cs);
      s_cos[warp][i] = cs;
      s_sin[warp][i] = sn;
    }
    __syncwarp();
  }
  uint64_t cs[4] = {}, sn[4] = {};
  if (turned)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = *reinterpret_cast<const uint64_t *>(&s_cos[warp][8 * l + 2 * i]);
      sn[i] = *reinterpret_cast<const uint64_t *>(&s_sin[warp][8 * l + 2 * i]);
    }
  uint64_t w[2][4];  // the weights of the kind of rows at hand
  int kind = -1;

  for (int r0 = first; r0 < last; r0 += kRows) {
    const int r = r0 + sub;
    uint64_t v[2][4];
    unpack8(next[0], v[0]);
    unpack8(next[1], v[1]);
    fetch(r + kRows);
    if (kind != (r >= a.Hq)) {
      kind = r >= a.Hq;
      const __nv_bfloat16 *from = kind ? a.kw : a.qw;
      unpack8(*reinterpret_cast<const uint4 *>(from + c0), w[0]);
      unpack8(*reinterpret_cast<const uint4 *>(from + c1), w[1]);
    }
    auto squares = [&] {
      uint64_t two[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        two[0] = fma2(v[0][i], v[0][i], two[0]);
        two[1] = fma2(v[1][i], v[1][i], two[1]);
      }
      float x, y;
      split(add2(two[0], two[1]), x, y);
      x += y;
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      return x;
    };
    auto times = [&](float f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = mul2(v[i >> 2][i & 3], pair_of(f, f));
    };
    float ss = squares();
    const bool huge = ss > kMaxFloat, tiny = a.eps < kTiny && ss < kTiny;
    float pre = 1.0f;
    if (__any_sync(0xffffffffu, huge || tiny)) {
      if (huge || tiny) pre = huge ? kDown : kUp;
      times(pre);
      ss = squares();
    }
    // (a row of zeros stays one where eps is 0)
    times(ss == 0.0f ? 0.0f : rsqrtf(ss * (1.0f / D) + a.eps * pre * pre));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = mul2(v[i >> 2][i & 3], w[i >> 2][i & 3]);
    if (turned)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t x = v[0][i], y = v[1][i];
        v[0][i] = fma2(x, cs[i], mul2(y, sn[i]) ^ 0x8000000080000000ull);
        v[1][i] = fma2(y, cs[i], mul2(x, sn[i]));
      }
    if (r < last) {
      __nv_bfloat16 *o = kind ? a.ko + token * a.kos + (r - a.Hq) * D : a.qo + token * a.qos + r * D;
      *reinterpret_cast<uint4 *>(o + c0) = pack8(v[0]);
      *reinterpret_cast<uint4 *>(o + c1) = pack8(v[1]);
    }
  }
}

}  // namespace moe

using namespace moe;

extern "C" int moe_qk_norm_rope(const void *q, const void *k, const void *q_weight,
                                const void *k_weight, const int32_t *positions,
                                const double *inv_freq, long long n_tokens, int n_q_heads,
                                int n_k_heads, int head_dim, int rot_dim, long long q_stride,
                                long long k_stride, float eps, void *q_out, long long q_out_stride,
                                void *k_out, long long k_out_stride, void *cuda_stream) {
  if (n_tokens < 0 || n_q_heads <= 0 || n_k_heads <= 0 || rot_dim < 0 || rot_dim > head_dim || !(eps >= 0.0f))
    return MOE_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || rot_dim % 16 != 0 || n_q_heads > 4096 || n_k_heads > 4096 ||
      n_tokens > 0x7fffffffLL)
    return MOE_ERR_UNSUPPORTED;
  const long long qw = static_cast<long long>(n_q_heads) * head_dim, kw = static_cast<long long>(n_k_heads) * head_dim;
  if (q_stride < qw || q_out_stride < qw || k_stride < kw || k_out_stride < kw) return MOE_ERR_INVALID_ARG;
  const long long strides[] = {q_stride, k_stride, q_out_stride, k_out_stride};
  for (long long s : strides) {
    if (s >= (1LL << 39)) return MOE_ERR_UNSUPPORTED;
    if (s % 8 != 0) return MOE_ERR_ALIGNMENT;
  }
  if (n_tokens == 0) return MOE_OK;
  if (!q || !k || !q_weight || !k_weight || !q_out || !k_out || (rot_dim > 0 && (!positions || !inv_freq)))
    return MOE_ERR_INVALID_ARG;
  const void *ptrs[] = {q, k, q_weight, k_weight, q_out, k_out};
  for (const void *p : ptrs)
    if (off_boundary(p, 16)) return MOE_ERR_ALIGNMENT;
  if (off_boundary(positions, 4) || off_boundary(inv_freq, 8)) return MOE_ERR_ALIGNMENT;
  RopeArgs a = {};
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.qw = static_cast<const __nv_bfloat16 *>(q_weight);
  a.kw = static_cast<const __nv_bfloat16 *>(k_weight);
  a.qo = static_cast<__nv_bfloat16 *>(q_out);
  a.ko = static_cast<__nv_bfloat16 *>(k_out);
  a.positions = positions;
  a.freq = inv_freq;
  a.tokens = n_tokens;
  a.qs = q_stride;
  a.ks = k_stride;
  a.qos = q_out_stride;
  a.kos = k_out_stride;
  a.Hq = n_q_heads;
  a.Hk = n_k_heads;
  a.rot = rot_dim;
  a.eps = eps;
  const int H = n_q_heads + n_k_heads, least = 256 / head_dim;
  // a warp per token where that fills the GPU, else fewer rows per warp
  const long long want = 152 * 16;
  long long split = n_tokens >= want ? 1 : (want + n_tokens - 1) / n_tokens;
  a.per = static_cast<int>((H + split - 1) / split);
  if (a.per < least) a.per = least;
  a.split = (H + a.per - 1) / a.per;
  const long long units = n_tokens * a.split, blocks = (units + kRopeWarps - 1) / kRopeWarps;
  if (blocks > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = head_dim == 128 ? launch_attn(qk_rope_kernel<128>, grid, kRopeWarps * 32, 0, st, a)
                                        : launch_attn(qk_rope_kernel<256>, grid, kRopeWarps * 32, 0, st, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
