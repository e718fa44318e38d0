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
// Bound by memory, 2.56 bytes moved per column, and on the way there by instructions,
// those of the addresses as much as those of the columns: 16 columns per lane, a
// block of several tokens whose places its first warp looks up, one token per lane.
// 16,384 tokens of 2 heads of 256 are written in 14.4 us (3.0 TB/s) and read in 10
// (4.3 TB/s), four caches in turn; with a warp per token, a division per code and 8
// columns per lane both took 43 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "attn_common.cuh"

namespace moe {

namespace {

constexpr int kKvWarps = 4;
constexpr int kBatch = 2;  // rows of a lane in flight (4: 1.5 us more of those 14)
// the sum of 0x4b400000 << 4 e, the bits of 2^23 + 2^22, modulo 2^32
constexpr uint32_t kMagicBits = 0x3f400000u;

struct KvArgs {
  CacheArgs c;
  const __nv_bfloat16 *k, *v;
  __nv_bfloat16 *ko, *vo;
  const int *starts, *offsets;
  long long n_tokens, ks, vs;
  int n_seq, tokens;  // tokens: of a block, up to 32
  float per_rows;     // 1 / (2 H)
};

// row r of a block (below 2^21) is row x of token t
__device__ __forceinline__ void split_row(const KvArgs &a, int r, int &t, int &x) {
  t = static_cast<int>((static_cast<float>(r) + 0.5f) * a.per_rows);
  x = r - t * 2 * a.c.H;
}

__device__ __forceinline__ void bad_page(const CacheArgs &c) {
  report_error(c.status, MOE_ERR_DEVICE_BOUNDS, KID_KV_CACHE * 100 + SITE_INDEX);
}

// Where the tokens of a block are, by its first warp, one token per lane: page (-1:
// outside the cache, -2: a token of no sequence) and place.
__device__ __forceinline__ void find_slots(const KvArgs &a, long long t0, int (&page)[32], int (&place)[32]) {
  const int lane = threadIdx.x;
  if (lane >= 32) return;
  const long long t = t0 + lane;
  int pg = -2, pl = 0;
  if (lane < a.tokens && t < a.n_tokens) {
    int i = -1;
    if (a.offsets) {  // the last sequence that starts at or before t, unless it has ended
      int lo = 0, hi = a.n_seq;  // offsets[lo - 1] <= t < offsets[hi]
      while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (a.offsets[mid] <= t) {
          lo = mid + 1;
        } else {
          hi = mid;
        }
      }
      if (lo > 0 && a.offsets[lo] > t) i = lo - 1;
    } else {
      i = static_cast<int>(t) / static_cast<int>(a.n_tokens / a.n_seq);
    }
    if (i >= 0) {
      int q0, q1;
      seq_rows(a.offsets, a.n_seq, a.n_tokens, i, q0, q1);
      const long long at = static_cast<long long>(a.starts ? a.starts[i] : 0) + t - q0;
      pg = page_of(a.c, i, at);
      pl = static_cast<int>(at & (kPage - 1));
      if (pg < 0) bad_page(a.c);
    }
  }
  page[lane] = pg;
  place[lane] = pl;
}

}  // namespace

namespace {

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace

// A block has a.tokens tokens: 2 H rows of keys and values each, kBatch rows of a
// lane in flight, 16 columns per lane.
template <int D>
__global__ void __launch_bounds__(kKvWarps * 32) kv_write_kernel(const KvArgs a) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  __shared__ int s_page[32], s_place[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
  const int H = a.c.H, c = lane % kLanes * 16;
  const int rows = 2 * H * static_cast<int>(min(static_cast<long long>(a.tokens), a.n_tokens - t0));
  auto source = [&](int r) {
    int t, x;
    split_row(a, r, t, x);
    return c + (x >= H ? a.v + (t0 + t) * a.vs + (x - H) * D : a.k + (t0 + t) * a.ks + x * D);
  };
  uint4 u[kBatch][2];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = r0 + b * kRows;
      u[b][0] = u[b][1] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const uint4 *src = reinterpret_cast<const uint4 *>(source(r));
        u[b][0] = src[0];
        u[b][1] = src[1];
      }
    }
  };
  const int mine = warp * kBatch * kRows + lane / kLanes;  // this lane's first row
  fetch(mine);
  find_slots(a, t0, s_page, s_place);
  __syncthreads();
  // (all lanes stay in the loop: the rows of a warp are of one count)
  for (int r0 = mine; r0 - lane / kLanes < rows; r0 += kKvWarps * kBatch * kRows) {
    if (r0 != mine) fetch(r0);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = r0 + b * kRows;
      if (r - lane / kLanes >= rows) break;  // (the whole warp)
      const uint32_t w[8] = {u[b][0].x, u[b][0].y, u[b][0].z, u[b][0].w,
                             u[b][1].x, u[b][1].y, u[b][1].z, u[b][1].w};
      // smallest and largest of the group's 64 columns; a NaN among them stays
      uint32_t least = w[0], most = w[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        least = min2(least, w[i]);
        most = max2(most, w[i]);
      }
      // the two halves: (least, - most), whose least over the group's lanes is sought
      const uint32_t flip = most ^ 0x80008000u;
      uint32_t both = min2(__byte_perm(least, flip, 0x5410), __byte_perm(least, flip, 0x7632));
      both = min2(both, __shfl_xor_sync(0xffffffffu, both, 2));
      both = min2(both, __shfl_xor_sync(0xffffffffu, both, 1));
      const float lo = __uint_as_float(both << 16), hi = -__uint_as_float(both & 0xffff0000u);
      const bool finite = fabsf(lo) <= 3.402823466e38f && fabsf(hi) <= 3.402823466e38f;
      // halves where the range leaves fp32
      const float f = hi - lo > 3.402823466e38f ? 0.5f : 1.0f;
      const __nv_bfloat16 scale = __float2bfloat16_rn(__fdiv_rn(hi * f - lo * f, 15.0f * f));
      const float s = __bfloat162float(scale);
      // A code is the quotient (x - bias) / scale, rounded to even.  Two estimates of it,
      // a little more and a little less than the quotient, are rounded: by the sum with
      // 2^23 + 2^22, which leaves the code in the low bits.  Where they agree, that is
      // the code.  (1 / scale is within 2^-22 of itself, so that 2^-20 more and less
      // enclose the quotient as divided; where scale has no such reciprocal or the range
      // was halved, none is taken to agree.)  Else the quotient itself is formed:
      // one code in some hundreds, as values of 8 bits often fall between two codes.
      const float inv = __fdividef(1.0f, s), top = 15.0f * s;
      const uint64_t less = pair_of(-lo, -lo), magic = pair_of(12582912.0f, 12582912.0f);
      const float up = inv * (1.0f + 0x1p-20f), down = inv * (1.0f - 0x1p-20f);
      const uint64_t up2 = pair_of(up, up), down2 = pair_of(down, down);
      const bool plain = s > 0x1p-100f && s < 0x1p100f && f == 1.0f;
      uint32_t code[2] = {0, 0};
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        uint32_t low = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          const uint32_t v = w[z * 4 + i];
          float y0, y1, m0, m1;
          split(add2(pair_of(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)), less), y0, y1);
          const uint64_t y = pair_of(fminf(y0, top), fminf(y1, top));
          split(fma2(y, up2, magic), m0, m1);
          code[z] = (code[z] * 16 + __float_as_uint(m1)) * 16 + __float_as_uint(m0);
          split(fma2(y, down2, magic), m0, m1);
          low = (low * 16 + __float_as_uint(m1)) * 16 + __float_as_uint(m0);
        }
        code[z] -= kMagicBits;
        uint32_t open = plain ? code[z] ^ (low - kMagicBits) : 0xffffffffu;
        while (open) {
          const int e = (__ffs(open) - 1) / 4;
          const uint32_t v0 = e & 2 ? w[z * 4 + 1] : w[z * 4], v1 = e & 2 ? w[z * 4 + 3] : w[z * 4 + 2];
          const uint32_t v = e & 4 ? v1 : v0;
          const float x = __uint_as_float(e & 1 ? v & 0xffff0000u : v << 16) * f, from = lo * f, y = x - from;
          float quot = s == 0.0f ? 0.0f : __fdiv_rn(y, s * f);
          // Half way between two codes the exact quotient decides: what is left of y, which
          // a fused sum has exactly, else what x - bias lost when it was rounded to y.
          const float low = floorf(quot);
          if (quot - low == 0.5f) {
            const float left = fmaf(-(low + 0.5f), s * f, y), took = y - x;
            const float more = left != 0.0f ? left : (x - (y - took)) + (-from - took);
            if (more != 0.0f) quot = more > 0.0f ? low + 1.0f : low;
          }
          const uint32_t n = static_cast<uint32_t>(fminf(rintf(quot), 15.0f)), nibble = 15u << (4 * e);
          code[z] = (code[z] & ~nibble) | n << (4 * e);
          open &= ~nibble;
        }
      }
      uint32_t pair = static_cast<uint32_t>(__bfloat16_as_ushort(scale)) | both << 16;
      if (!finite) {
        code[0] = code[1] = 0;
        pair = 0x7fff7fffu;
      }
      if (r < rows) {
        int t, y;
        split_row(a, r, t, y);
        const int which = y >= H, page = s_page[t];
        if (page >= 0) {
          const long long row = cache_row(a.c, page, which, y - which * H, s_place[t]);
          *reinterpret_cast<uint2 *>(a.c.codes + row * (D / 2) + c / 2) = make_uint2(code[0], code[1]);
          if ((lane & 3) == 0) a.c.affine[row * (D / kGroup) + c / kGroup] = pair;
        }
      }
    }
  }
}

// 16 columns per lane, half of the row apart, so that the addresses are shared.
template <int D>
__global__ void __launch_bounds__(kKvWarps * 32) kv_read_kernel(const KvArgs a) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  __shared__ int s_page[32], s_place[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
  const int H = a.c.H, c = lane % kLanes * 8;
  const int rows = 2 * H * static_cast<int>(min(static_cast<long long>(a.tokens), a.n_tokens - t0));
  find_slots(a, t0, s_page, s_place);
  __syncthreads();
  for (int r0 = warp * kBatch * kRows + lane / kLanes; r0 < rows; r0 += kKvWarps * kBatch * kRows) {
    uint32_t code[kBatch][2], pair[kBatch][2];
    __nv_bfloat16 *to[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = r0 + b * kRows;
      code[b][0] = code[b][1] = pair[b][0] = pair[b][1] = 0;
      to[b] = nullptr;
      if (r < rows) {
        int t, y;
        split_row(a, r, t, y);
        const int which = y >= H, page = s_page[t];
        if (page != -2) to[b] = (which ? a.vo : a.ko) + ((t0 + t) * H + y - which * H) * D + c;
        if (page >= 0) {
          const long long row = cache_row(a.c, page, which, y - which * H, s_place[t]);
          const uint8_t *codes = a.c.codes + row * (D / 2) + c / 2;
          const uint32_t *affine = a.c.affine + row * (D / kGroup) + c / kGroup;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            code[b][z] = *reinterpret_cast<const uint32_t *>(codes + z * (D / 4));
            pair[b][z] = affine[z * (D / kGroup / 2)];
          }
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (!to[b]) continue;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float s = __uint_as_float(pair[b][z] << 16), bias = __uint_as_float(pair[b][z] & 0xffff0000u);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 2^23 + code, less 2^23: a conversion at the rate of sums
          const uint64_t two = pair_of(__uint_as_float((code[b][z] >> (8 * i) & 15u) | 0x4b000000u),
                                       __uint_as_float((code[b][z] >> (8 * i + 4) & 15u) | 0x4b000000u));
          float x, y;
          split(fma2(pair_of(s, s), add2(two, pair_of(-8388608.0f, -8388608.0f)), pair_of(bias, bias)), x, y);
          out[i] = bf16x2_bits(x, y);
        }
        *reinterpret_cast<uint4 *>(to[b] + z * (D / 2)) = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
  }
}

namespace {

// Tokens of a block: 16 rows of 256 columns, or twice that of 128, if that leaves two
// blocks per SM.  (Half as many tokens: 16.4 and 10.2 us in place of 14 and 8.5; twice
// as many: 14.4 and 9.)
int block_tokens(long long n_tokens, int H, int D) {
  const int rows = 16 * (256 / D), fit = rows / (2 * H);
  const long long spread = n_tokens / (2 * 152);
  long long t = fit < spread ? fit : spread;
  t = t < 1 ? 1 : t;
  return static_cast<int>(t > 32 ? 32 : t);
}

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
  a.tokens = block_tokens(n_tokens, n_heads, head_dim);
  a.per_rows = 1.0f / (2.0f * static_cast<float>(n_heads));
  const dim3 grid(static_cast<unsigned>((n_tokens + a.tokens - 1) / a.tokens));
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
  a.tokens = block_tokens(n_tokens, n_heads, head_dim);
  a.per_rows = 1.0f / (2.0f * static_cast<float>(n_heads));
  const dim3 grid(static_cast<unsigned>((n_tokens + a.tokens - 1) / a.tokens));
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = head_dim == 128 ? launch_attn(kv_read_kernel<128>, grid, kKvWarps * 32, 0, st, a)
                                        : launch_attn(kv_read_kernel<256>, grid, kKvWarps * 32, 0, st, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
