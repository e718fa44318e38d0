// attn_prefill.cu -- causal attention of packed prompts, several query heads on
// one key/value head (moe_attention_prefill in include/moe.h):
//     o_i = sum_j softmax_j(scale q_i . k_j) v_j   over keys j <= i + (keys - queries)
// A warp has one query of one head; the running maximum and sum of the softmax
// are kept in fp32 and the output accumulated in registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "attn_common.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;

struct PrefillArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *out;
  const int *offsets, *k_offsets;
  long long n_q, n_k, qs, ks, vs;
  int n_seq, Hq, Hk;
  float scale;  // times log2(e)
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_prefill_kernel(const PrefillArgs a) {
  constexpr int kE = D / 32;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const long long t = unit / a.Hq;
  const int h = static_cast<int>(unit % a.Hq), hk = h / (a.Hq / a.Hk);
  if (t >= a.n_q) return;
  const int s = seq_of_row(a.offsets, a.n_seq, a.n_q, static_cast<int>(t));
  if (s < 0) return;
  int q0, q1, k0, k1;
  seq_rows(a.offsets, a.n_seq, a.n_q, s, q0, q1);
  seq_rows(a.k_offsets, a.n_seq, a.n_k, s, k0, k1);
  const int seen = min(k1 - k0, static_cast<int>(t) - q0 + 1 + (k1 - k0) - (q1 - q0));
  float q[kE], o[kE], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    q[e] = __bfloat162float(a.q[t * a.qs + h * D + e * 32 + lane]);
    o[e] = 0.0f;
  }
  for (int j = 0; j < seen; ++j) {
    const __nv_bfloat16 *k = a.k + (k0 + j) * a.ks + hk * D + lane, *v = a.v + (k0 + j) * a.vs + hk * D + lane;
    float x = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) x = fmaf(q[e], __bfloat162float(k[e * 32]), x);
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= a.scale;
    const float top = fmaxf(m, x), ref = top == -INFINITY ? 0.0f : top;
    const float f = exp2f(m - ref), p = exp2f(x - ref);
    m = top;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = o[e] * f + p * __bfloat162float(v[e * 32]);
  }
#pragma unroll
  for (int e = 0; e < kE; ++e)
    a.out[(t * a.Hq + h) * D + e * 32 + lane] = __float2bfloat16_rn(seen > 0 ? o[e] / l : 0.0f);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_attention_prefill(const void *q, const void *k, const void *v,
                                     const int32_t *offsets, const int32_t *k_offsets,
                                     long long n_q, long long n_k, int n_seq, int n_q_heads,
                                     int n_kv_heads, int head_dim, long long q_stride,
                                     long long k_stride, long long v_stride, float scale, void *out,
                                     void *cuda_stream) {
  if (n_q < 0 || n_k < 0 || n_seq < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0 ||
      !(scale > 0.0f) || scale > 3.0e38f)
    return MOE_ERR_INVALID_ARG;
  if (k_offsets && !offsets) return MOE_ERR_INVALID_ARG;
  if (offsets ? (!k_offsets && n_q != n_k) : (n_seq > 0 && (n_q % n_seq != 0 || n_k % n_seq != 0)))
    return MOE_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || n_q_heads / n_kv_heads > 64 || n_kv_heads > 4096 ||
      n_q > 0x7fffffffLL || n_k > 0x7fffffffLL)
    return MOE_ERR_UNSUPPORTED;
  const long long qw = static_cast<long long>(n_q_heads) * head_dim, kw = static_cast<long long>(n_kv_heads) * head_dim;
  if (q_stride < qw || k_stride < kw || v_stride < kw) return MOE_ERR_INVALID_ARG;
  const long long strides[] = {q_stride, k_stride, v_stride};
  for (long long s : strides) {
    if (s >= (1LL << 38)) return MOE_ERR_UNSUPPORTED;
    if (s % 8 != 0) return MOE_ERR_ALIGNMENT;
  }
  if (n_q == 0 || n_seq == 0) return MOE_OK;
  if (!q || !out || (n_k > 0 && (!k || !v))) return MOE_ERR_INVALID_ARG;
  if (off_boundary(q, 16) || off_boundary(k, 16) || off_boundary(v, 16) || off_boundary(out, 16) ||
      off_boundary(offsets, 4) || off_boundary(k_offsets, 4))
    return MOE_ERR_ALIGNMENT;
  PrefillArgs a = {};
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.v = static_cast<const __nv_bfloat16 *>(v);
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.offsets = offsets;
  a.k_offsets = k_offsets ? k_offsets : offsets;
  a.n_q = n_q;
  a.n_k = n_k;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.n_seq = n_seq;
  a.Hq = n_q_heads;
  a.Hk = n_kv_heads;
  a.scale = scale * 1.4426950408889634f;
  const long long blocks = (n_q * n_q_heads + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = head_dim == 128 ? launch_attn(attn_prefill_kernel<128>, grid, kWarps * 32, 0, st, a)
                                        : launch_attn(attn_prefill_kernel<256>, grid, kWarps * 32, 0, st, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
