// decay.cu -- linear attention with one decay per value head (gdn_decay_scan
// in include/gdn.h).  With S the state [d_v][d_k] of a value head and lambda
// its decay:
//     S <- lambda S + v_t k_t^T,   o_t = S q_t
//
// The recurrent form (single tokens): rows of S are independent, so a warp
// holds a few of them in registers, a row spread over d_k / 4 lanes, for the
// whole call; each token costs one decay and write (2 operations an element)
// and one dot product per row.  One token per sequence reads and writes the
// state once and little else, so it is bound by memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/gdn.h"
#include "internal.h"

namespace moe {

namespace {

struct DecayArgs {
  const __nv_bfloat16 *q, *k, *v;
  const float *decay, *s_in;
  float *s_out;
  __nv_bfloat16 *o;
  const int *offsets;  // null: n_seq sequences of n_tokens / n_seq tokens
  long long n_tokens, q_stride, k_stride, v_stride;
  int n_seq, Hk, Hv, dv;
};

// first token and number of tokens of sequence i; offsets outside
// [0, n_tokens] or running backwards are clamped
__device__ __forceinline__ void seq_range(const DecayArgs &a, int i, long long &first,
                                          long long &len) {
  if (a.offsets) {
    const long long lo = min(max(static_cast<long long>(a.offsets[i]), 0LL), a.n_tokens);
    const long long hi = min(max(static_cast<long long>(a.offsets[i + 1]), lo), a.n_tokens);
    first = lo;
    len = hi - lo;
  } else {
    len = a.n_tokens / a.n_seq;
    first = len * i;
  }
}

__device__ __forceinline__ float4 ld_bf16x4(const __nv_bfloat16 *p) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

constexpr int kRecWarps = 4;

}  // namespace

// One CTA: kRecWarps * kR * (128 / kDk) rows of one (sequence, value head).
template <int kDk, int kR>
__global__ void __launch_bounds__(kRecWarps * 32) decay_recurrent_kernel(const DecayArgs a) {
  constexpr int kLpr = kDk / 4;          // lanes per row
  constexpr int kRpl = 32 / kLpr;        // rows per warp-wide load
  constexpr int kRowsWarp = kR * kRpl;   // rows of a warp
  constexpr int kRows = kRecWarps * kRowsWarp;
  const int tiles = (a.dv + kRows - 1) / kRows;
  const int tile = blockIdx.x % tiles;
  const int sh = blockIdx.x / tiles, h = sh % a.Hv, seq = sh / a.Hv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kLpr;
  const int j0 = tile * kRows + warp * kRowsWarp + lane / kLpr;  // this lane's rows: j0 + r kRpl
  if (j0 - lane / kLpr >= a.dv) return;
  long long first, len;
  seq_range(a, seq, first, len);
  const long long sbase = (static_cast<long long>(seq) * a.Hv + h) * a.dv * kDk + 4 * c;
  float4 S[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int j = j0 + r * kRpl;
    S[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.s_in && j < a.dv)
      S[r] = *reinterpret_cast<const float4 *>(a.s_in + sbase + static_cast<long long>(j) * kDk);
  }
  const float lam = a.decay[h];
  const int hk = h / (a.Hv / a.Hk);
  for (long long t = first; t < first + len; ++t) {
    const float4 q = ld_bf16x4(a.q + t * a.q_stride + hk * kDk + 4 * c);
    const float4 k = ld_bf16x4(a.k + t * a.k_stride + hk * kDk + 4 * c);
    float d[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int j = j0 + r * kRpl;
      const float v = j < a.dv ? __bfloat162float(a.v[t * a.v_stride + h * a.dv + j]) : 0.0f;
      S[r].x = fmaf(lam, S[r].x, v * k.x);
      S[r].y = fmaf(lam, S[r].y, v * k.y);
      S[r].z = fmaf(lam, S[r].z, v * k.z);
      S[r].w = fmaf(lam, S[r].w, v * k.w);
      d[r] = S[r].x * q.x + S[r].y * q.y + S[r].z * q.z + S[r].w * q.w;
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
#pragma unroll
      for (int m = kLpr / 2; m; m >>= 1) d[r] += __shfl_xor_sync(0xffffffffu, d[r], m);
      const int j = j0 + r * kRpl;
      if (c == 0 && j < a.dv)
        a.o[(t * a.Hv + h) * a.dv + j] = __float2bfloat16_rn(d[r]);
    }
  }
  if (a.s_out) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int j = j0 + r * kRpl;
      if (j < a.dv)
        *reinterpret_cast<float4 *>(a.s_out + sbase + static_cast<long long>(j) * kDk) = S[r];
    }
  }
}

namespace {

template <int kDk, int kR>
cudaError_t launch_recurrent(const DecayArgs &a, cudaStream_t st) {
  constexpr int kRows = kRecWarps * kR * (128 / kDk);
  const int tiles = (a.dv + kRows - 1) / kRows;
  decay_recurrent_kernel<kDk, kR><<<static_cast<unsigned>(a.n_seq) * a.Hv * tiles, kRecWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int gdn_decay_workspace(long long n_tokens, int n_seq, int n_v_heads, int d_k, int d_v,
                                   size_t *bytes) {
  if (!bytes || n_tokens < 0 || n_seq < 0 || n_v_heads <= 0 || d_k <= 0 || d_v <= 0)
    return MOE_ERR_INVALID_ARG;
  *bytes = 0;
  return MOE_OK;
}

extern "C" int gdn_decay_scan(const void *q, const void *k, const void *v, const float *decay,
                              const float *state_in, float *state_out, void *o, const int *offsets,
                              long long n_tokens, int n_seq, int n_k_heads, int n_v_heads, int d_k,
                              int d_v, long long q_stride, long long k_stride, long long v_stride,
                              void *workspace, size_t workspace_bytes, void *cuda_stream) {
  if (n_tokens < 0 || n_seq < 0 || n_k_heads <= 0 || n_v_heads <= 0 || d_k <= 0 || d_v <= 0)
    return MOE_ERR_INVALID_ARG;
  if (n_v_heads % n_k_heads != 0 || (n_seq == 0 && n_tokens > 0)) return MOE_ERR_INVALID_ARG;
  if (!offsets && n_seq > 0 && n_tokens % n_seq != 0) return MOE_ERR_INVALID_ARG;
  if (n_seq == 0) return MOE_OK;
  if (!decay || (n_tokens > 0 && (!q || !k || !v || !o))) return MOE_ERR_INVALID_ARG;
  if (q_stride < static_cast<long long>(n_k_heads) * d_k ||
      k_stride < static_cast<long long>(n_k_heads) * d_k ||
      v_stride < static_cast<long long>(n_v_heads) * d_v)
    return MOE_ERR_INVALID_ARG;
  if ((d_k != 64 && d_k != 128) || d_v % 16 != 0 || d_v > 1024 || n_v_heads > 4096 ||
      n_tokens > 0x7fffffffLL ||
      static_cast<long long>(n_seq) * n_v_heads * (d_v / 16) > 0x7fffffffLL)
    return MOE_ERR_UNSUPPORTED;
  auto misaligned = [](const void *p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) % n) != 0;
  };
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || misaligned(state_in, 16) ||
      misaligned(state_out, 16) || misaligned(decay, 4) || misaligned(offsets, 4) ||
      misaligned(workspace, 16))
    return MOE_ERR_ALIGNMENT;
  size_t need = 0;
  const int rc = gdn_decay_workspace(n_tokens, n_seq, n_v_heads, d_k, d_v, &need);
  if (rc != MOE_OK) return rc;
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  DecayArgs a;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.v = static_cast<const __nv_bfloat16 *>(v);
  a.decay = decay;
  a.s_in = state_in;
  a.s_out = state_out;
  a.o = static_cast<__nv_bfloat16 *>(o);
  a.offsets = offsets;
  a.n_tokens = n_tokens;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.n_seq = n_seq;
  a.Hk = n_k_heads;
  a.Hv = n_v_heads;
  a.dv = d_v;
  const cudaError_t e = d_k == 128 ? launch_recurrent<128, 8>(a, st) : launch_recurrent<64, 8>(a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
