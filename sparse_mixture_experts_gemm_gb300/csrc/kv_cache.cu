// kv_cache.cu -- keys and values quantised to 4 bits as they are written into
// the pages of a cache, and read back (moe_kv_write, moe_kv_read in
// include/moe.h).
//
// Per 64 columns of a head's row, in fp32:
//     bias = bf16(min), scale = bf16((max - min) / 15), code = round((x - bias) / scale) in 0 .. 15
//     value = bf16(scale * code + bias)
// the format of moe_quantize_q4.  A range past fp32's largest number is formed
// from halves.  A group that holds a NaN or an infinity has scale and bias NaN
// and reads back as NaN.
//
// Bound by memory, 2.56 bytes moved per column.  8 columns per lane: one 16-byte
// vector of keys or values, one word of codes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/moe.h"
#include "attn_common.cuh"

namespace moe {

namespace {

constexpr int kKvWarps = 4;

struct KvArgs {
  CacheArgs c;
  const __nv_bfloat16 *k, *v;
  __nv_bfloat16 *ko, *vo;
  const int *starts, *offsets;
  long long n_tokens, ks, vs;
  int n_seq;
};

__device__ __forceinline__ void bad_page(const CacheArgs &c) {
  report_error(c.status, MOE_ERR_DEVICE_BOUNDS, KID_KV_CACHE * 100 + SITE_INDEX);
}

// page and place of token t (the whole warp); false: none
__device__ __forceinline__ bool slot_of(const KvArgs &a, int t, int &page, int &place) {
  const int i = seq_of_row(a.offsets, a.n_seq, a.n_tokens, t);
  if (i < 0) return false;
  int lo, hi;
  seq_rows(a.offsets, a.n_seq, a.n_tokens, i, lo, hi);
  const long long at = static_cast<long long>(a.starts ? a.starts[i] : 0) + t - lo;
  page = page_of(a.c, i, at);
  place = static_cast<int>(at & (kPage - 1));
  return true;
}

}  // namespace

// A warp per token: its 2 H rows of keys and values, 32 lanes over 256 columns.
template <int D>
__global__ void __launch_bounds__(kKvWarps * 32) kv_write_kernel(const KvArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const long long t = static_cast<long long>(blockIdx.x) * kKvWarps + warp;
  if (t >= a.n_tokens) return;
  int page, place;
  if (!slot_of(a, static_cast<int>(t), page, place)) return;
  if (page < 0) {
    if (lane == 0) bad_page(a.c);
    return;
  }
  const int sub = lane / kLanes, c = lane % kLanes * 8, H = a.c.H;
  for (int r0 = 0; r0 < 2 * H; r0 += kRows) {
    const int r = min(r0 + sub, 2 * H - 1), which = r >= H, h = r - which * H;
    const __nv_bfloat16 *src = (which ? a.v + t * a.vs : a.k + t * a.ks) + h * D + c;
    const uint4 u = *reinterpret_cast<const uint4 *>(src);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    float lo = x[0], hi = x[0];
    bool fin = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, x[e]);
      hi = fmaxf(hi, x[e]);
      fin = fin && fabsf(x[e]) <= 3.402823466e38f;
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const uint32_t all = __ballot_sync(0xffffffffu, fin);
    fin = ((all >> (lane & 24)) & 255u) == 255u;  // the group's eight lanes
    // halves where the range leaves fp32
    const float f = hi - lo > 3.402823466e38f ? 0.5f : 1.0f;
    __nv_bfloat16 bias = __float2bfloat16_rn(lo);
    __nv_bfloat16 scale = __float2bfloat16_rn(__fdiv_rn(hi * f - lo * f, 15.0f * f));
    const float s = __bfloat162float(scale), b = __bfloat162float(bias);
    uint32_t code = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = s == 0.0f ? 0.0f : rintf(__fdiv_rn(x[e] * f - b * f, s * f));
      code |= static_cast<uint32_t>(fminf(fmaxf(y, 0.0f), 15.0f)) << (4 * e);
    }
    uint32_t pair = static_cast<uint32_t>(__bfloat16_as_ushort(scale)) |
                    static_cast<uint32_t>(__bfloat16_as_ushort(bias)) << 16;
    if (!fin) {
      code = 0;
      pair = 0x7fff7fffu;
    }
    if (r0 + sub < 2 * H) {
      const long long row = cache_row(a.c, page, which, h, place);
      *reinterpret_cast<uint32_t *>(a.c.codes + row * (D / 2) + c / 2) = code;
      if ((lane & 7) == 0) a.c.affine[row * (D / kGroup) + c / kGroup] = pair;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kKvWarps * 32) kv_read_kernel(const KvArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const long long t = static_cast<long long>(blockIdx.x) * kKvWarps + warp;
  if (t >= a.n_tokens) return;
  int page, place;
  if (!slot_of(a, static_cast<int>(t), page, place)) return;
  if (page < 0 && lane == 0) bad_page(a.c);
  const int sub = lane / kLanes, c = lane % kLanes * 8, H = a.c.H;
  for (int r = sub; r < 2 * H; r += kRows) {
    const int which = r >= H, h = r - which * H;
    uint32_t code = 0, pair = 0;
    if (page >= 0) {
      const long long row = cache_row(a.c, page, which, h, place);
      code = *reinterpret_cast<const uint32_t *>(a.c.codes + row * (D / 2) + c / 2);
      pair = a.c.affine[row * (D / kGroup) + c / kGroup];
    }
    const float s = __uint_as_float(pair << 16), b = __uint_as_float(pair & 0xffff0000u);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(s, static_cast<float>(code >> (4 * e) & 15u), b);
    __nv_bfloat16 *o = (which ? a.vo : a.ko) + (t * H + h) * D + c;
    *reinterpret_cast<uint4 *>(o) = make_uint4(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]),
                                               bf16x2_bits(x[4], x[5]), bf16x2_bits(x[6], x[7]));
  }
}

namespace {

// the checks that write and read share; MOE_OK with n_tokens or n_seq 0 is "nothing to do"
int check_kv(const void *codes, const void *affine, long long n_pages, const int32_t *pages,
             int table_width, long long n_tokens, int n_seq, const int32_t *offsets, int H, int D) {
  if (n_tokens < 0 || n_seq < 0 || n_pages < 0 || table_width < 0 || H <= 0) return MOE_ERR_INVALID_ARG;
  if (!offsets && n_seq > 0 && n_tokens % n_seq != 0) return MOE_ERR_INVALID_ARG;
  if ((D != 128 && D != 256) || H > 4096 || n_tokens > 0x7fffffffLL || n_pages > 0x7fffffffLL ||
      table_width > (1 << 25))
    return MOE_ERR_UNSUPPORTED;
  // rows of codes are addressed by 32-bit coordinates
  if (n_pages * 2 * H * kPage > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if (n_tokens == 0 || n_seq == 0) return MOE_OK;
  if ((n_pages > 0 && (!codes || !affine)) || (table_width > 0 && !pages)) return MOE_ERR_INVALID_ARG;
  if (off_boundary(codes, 16) || off_boundary(affine, 16) || off_boundary(pages, 4) || off_boundary(offsets, 4))
    return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_kv_write(uint8_t *codes, uint16_t *affine, long long n_pages, const void *k,
                            const void *v, const int32_t *pages, int table_width,
                            const int32_t *starts, const int32_t *offsets, long long n_tokens,
                            int n_seq, int n_heads, int head_dim, long long k_stride,
                            long long v_stride, void *cuda_stream) {
  const int rc = check_kv(codes, affine, n_pages, pages, table_width, n_tokens, n_seq, offsets, n_heads, head_dim);
  if (rc != MOE_OK) return rc;
  const long long wide = static_cast<long long>(n_heads) * head_dim;
  if (k_stride < wide || v_stride < wide) return MOE_ERR_INVALID_ARG;
  if (k_stride >= (1LL << 39) || v_stride >= (1LL << 39)) return MOE_ERR_UNSUPPORTED;
  if (k_stride % 8 != 0 || v_stride % 8 != 0) return MOE_ERR_ALIGNMENT;
  if (n_tokens == 0 || n_seq == 0) return MOE_OK;
  if (!k || !v) return MOE_ERR_INVALID_ARG;
  if (off_boundary(k, 16) || off_boundary(v, 16) || off_boundary(starts, 4)) return MOE_ERR_ALIGNMENT;
  KvArgs a = {};
  a.c = {codes, reinterpret_cast<uint32_t *>(affine), pages, n_pages, table_width, n_heads, head_dim,
         noalloc_status_word()};
  if (!a.c.status) return MOE_ERR_CUDA;
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.v = static_cast<const __nv_bfloat16 *>(v);
  a.starts = starts;
  a.offsets = offsets;
  a.n_tokens = n_tokens;
  a.ks = k_stride;
  a.vs = v_stride;
  a.n_seq = n_seq;
  const dim3 grid(static_cast<unsigned>((n_tokens + kKvWarps - 1) / kKvWarps));
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = head_dim == 128 ? launch_attn(kv_write_kernel<128>, grid, kKvWarps * 32, 0, st, a)
                                        : launch_attn(kv_write_kernel<256>, grid, kKvWarps * 32, 0, st, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" int moe_kv_read(const uint8_t *codes, const uint16_t *affine, long long n_pages,
                           const int32_t *pages, int table_width, const int32_t *starts,
                           const int32_t *offsets, long long n_tokens, int n_seq, int n_heads,
                           int head_dim, void *k_out, void *v_out, void *cuda_stream) {
  const int rc = check_kv(codes, affine, n_pages, pages, table_width, n_tokens, n_seq, offsets, n_heads, head_dim);
  if (rc != MOE_OK || n_tokens == 0 || n_seq == 0) return rc;
  if (!k_out || !v_out) return MOE_ERR_INVALID_ARG;
  if (off_boundary(k_out, 16) || off_boundary(v_out, 16) || off_boundary(starts, 4)) return MOE_ERR_ALIGNMENT;
  KvArgs a = {};
  a.c = {const_cast<uint8_t *>(codes), reinterpret_cast<uint32_t *>(const_cast<uint16_t *>(affine)), pages,
         n_pages, table_width, n_heads, head_dim, noalloc_status_word()};
  if (!a.c.status) return MOE_ERR_CUDA;
  a.ko = static_cast<__nv_bfloat16 *>(k_out);
  a.vo = static_cast<__nv_bfloat16 *>(v_out);
  a.starts = starts;
  a.offsets = offsets;
  a.n_tokens = n_tokens;
  a.n_seq = n_seq;
  const dim3 grid(static_cast<unsigned>((n_tokens + kKvWarps - 1) / kKvWarps));
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = head_dim == 128 ? launch_attn(kv_read_kernel<128>, grid, kKvWarps * 32, 0, st, a)
                                        : launch_attn(kv_read_kernel<256>, grid, kKvWarps * 32, 0, st, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
