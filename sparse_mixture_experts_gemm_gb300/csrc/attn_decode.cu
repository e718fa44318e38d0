// attn_decode.cu -- attention of one query token per sequence over a cache held
// in 4 bits (moe_attention_decode in include/moe.h):
//     o = sum_t softmax_t(scale q . k_t) v_t,   k_t, v_t = scale * code + bias
// A warp has one query head of a sequence; the running maximum and sum of the
// softmax are kept in fp32 and the output accumulated in registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "attn_common.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;

struct DecodeAttnArgs {
  CacheArgs c;
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  const int *lengths;
  long long qs;
  int n_seq, Hq;
  float scale;  // times log2(e)
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_decode_kernel(const DecodeAttnArgs a) {
  constexpr int kE = D / 32;  // columns of a lane: kE lane ..
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int s = static_cast<int>(unit / a.Hq), h = static_cast<int>(unit % a.Hq), hk = h / (a.Hq / a.c.H);
  if (s >= a.n_seq) return;
  int len = a.lengths[s];
  if (len > static_cast<long long>(a.c.width) * kPage) {
    len = a.c.width * kPage;
    if (lane == 0) report_error(a.c.status, MOE_ERR_DEVICE_BOUNDS, KID_ATTN_DECODE * 100 + SITE_INDEX);
  }
  float q[kE], o[kE], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    q[e] = __bfloat162float(a.q[s * a.qs + h * D + kE * lane + e]);
    o[e] = 0.0f;
  }
  bool any = false;
  for (int t = 0; t < len; ++t) {
    const int page = page_of(a.c, s, t);
    if (page < 0) {
      if (lane == 0) report_error(a.c.status, MOE_ERR_DEVICE_BOUNDS, KID_ATTN_DECODE * 100 + SITE_INDEX);
      continue;
    }
    any = true;
    float kv[2][kE];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const long long row = cache_row(a.c, page, w, hk, t % kPage);
      const uint32_t pair = a.c.affine[row * (D / kGroup) + kE * lane / kGroup];
      const float f = __uint_as_float(pair << 16), b = __uint_as_float(pair & 0xffff0000u);
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        const uint32_t c = a.c.codes[row * (D / 2) + (kE * lane + e) / 2];
        kv[w][e] = fmaf(f, static_cast<float>(c & 15u), b);
        kv[w][e + 1] = fmaf(f, static_cast<float>(c >> 4), b);
      }
    }
    float x = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) x = fmaf(q[e], kv[0][e], x);
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= a.scale;
    const float top = fmaxf(m, x), ref = top == -INFINITY ? 0.0f : top;
    const float f = exp2f(m - ref), p = exp2f(x - ref);
    m = top;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = o[e] * f + p * kv[1][e];
  }
#pragma unroll
  for (int e = 0; e < kE; ++e)
    a.out[(static_cast<long long>(s) * a.Hq + h) * D + kE * lane + e] = __float2bfloat16_rn(any ? o[e] / l : 0.0f);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_attention_decode_workspace(int n_seq, int table_width, int n_q_heads,
                                              int n_kv_heads, int head_dim, size_t *bytes) {
  if (!bytes || n_seq < 0 || table_width < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0)
    return MOE_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || n_q_heads > 65536 || table_width > (1 << 25)) return MOE_ERR_UNSUPPORTED;
  *bytes = 0;
  return MOE_OK;
}

extern "C" int moe_attention_decode(const void *q, long long q_stride, const uint8_t *codes,
                                    const uint16_t *affine, long long n_pages, const int32_t *pages,
                                    int table_width, const int32_t *lengths, int n_seq,
                                    int n_q_heads, int n_kv_heads, int head_dim, float scale,
                                    void *out, void *workspace, size_t workspace_bytes,
                                    void *cuda_stream) {
  size_t need = 0;
  const int rc = moe_attention_decode_workspace(n_seq, table_width, n_q_heads, n_kv_heads, head_dim, &need);
  if (rc != MOE_OK) return rc;
  if (n_pages < 0 || !(scale > 0.0f) || scale > 3.0e38f || q_stride < static_cast<long long>(n_q_heads) * head_dim)
    return MOE_ERR_INVALID_ARG;
  if (n_pages > 0x7fffffffLL || n_pages * 2 * n_kv_heads * kPage > 0x7fffffffLL || q_stride >= (1LL << 39)) return MOE_ERR_UNSUPPORTED;
  if (q_stride % 8 != 0) return MOE_ERR_ALIGNMENT;
  if (n_seq == 0) return MOE_OK;
  if (!q || !out || !lengths || (n_pages > 0 && (!codes || !affine)) || (table_width > 0 && !pages) ||
      (need > 0 && (!workspace || workspace_bytes < need)))
    return MOE_ERR_INVALID_ARG;
  if (off_boundary(q, 16) || off_boundary(out, 16) || off_boundary(codes, 16) || off_boundary(affine, 16) ||
      off_boundary(workspace, 16) || off_boundary(pages, 4) || off_boundary(lengths, 4))
    return MOE_ERR_ALIGNMENT;
  DecodeAttnArgs a = {};
  a.c = {const_cast<uint8_t *>(codes), reinterpret_cast<uint32_t *>(const_cast<uint16_t *>(affine)), pages,
         n_pages, table_width, n_kv_heads, head_dim, noalloc_status_word()};
  if (!a.c.status) return MOE_ERR_CUDA;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lengths = lengths;
  a.qs = q_stride;
  a.n_seq = n_seq;
  a.Hq = n_q_heads;
  a.scale = scale * 1.4426950408889634f;
  const long long blocks = (static_cast<long long>(n_seq) * n_q_heads + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = head_dim == 128 ? launch_attn(attn_decode_kernel<128>, grid, kWarps * 32, 0, st, a)
                                        : launch_attn(attn_decode_kernel<256>, grid, kWarps * 32, 0, st, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
