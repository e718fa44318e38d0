// attn_decode.cu -- attention of one query token per sequence over a cache held
// in 4 bits (moe_attention_decode in include/moe.h):
//     o = sum_t softmax_t(scale q . k_t) v_t,   k_t, v_t = scale_t * code + bias_t
//
// Bound by the cache's bytes, so every page is read once for the 8 query heads
// that share it, and the codes go to the tensor cores as they are:
//     q . k_t = sum_g [ s_tg (q_g . c_tg) + b_tg sum(q_g) ]       g: groups of 64 columns
//     o_g     = sum_t (p_t s'_tg) (c'_tg - 8) + sum_t p_t (b'_tg + 8 s'_tg)
// with products and sums in fp32.
//   * Keys: a code in the low bits of an fp16 is the number c 2^-24, four bits up c
//     2^-20: one AND makes two.  The queries become fp16 by a power of two per head
//     (the largest is in [2^12, 2^13): what is lost is below 2^-34 of it).
//   * Values: weights times scales need bf16's range, and 128 + c is one AND-OR away
//     from a nibble; a second product takes off 136 p_t s'_tg at once, so that the
//     sum stays centred and has no large part that cancels against the bias's.
//   * The biases' sums are products, too: bf16 biases with the sums of q in three bf16
//     parts, p in two with b' and s'.
// The only rounding before the result's is that of p_t s'_tg to bf16 (2^-8), which
// multiplies codes less 8 (and that of p to 2^-16 with the biases).
//
// Work split.  All (sequence, key/value head, 8 query heads) rows' pages lie on one
// line that is cut into equal shares, one per SM, whatever the lengths; a CTA
// finds its share from the lengths on the device.  Rows that are cut leave their
// parts (maximum, sum, output) in the workspace for a second kernel, which joins
// them in a fixed order.
//
// Roles: warp 12 copies pages by TMA (6 pages deep), warps 0-11 take 16 tokens of a
// page each, four warps per page, with a running softmax of their own; their parts
// are joined through shared memory at a row's end.  The codes are the A operand of
// both products (tokens x columns, columns x tokens), whose four registers the
// dequantisation fills as they are; P is turned in between, four 8 x 8 matrices.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <mutex>

#include "../../include/moe.h"
#include "attn_common.cuh"

namespace moe {

namespace {

constexpr int kConsumers = 12;
constexpr int kTeams = kConsumers / 4;  // of four warps, that take a page each
constexpr int kThreadsD = 32 * (kConsumers + 4);  // (whole warpgroups, for their shares of the registers)
// 128 registers a thread at launch: 16 warps x 32 x 128 = 12 x 32 x 152 + 4 x 32 x 40 + 2048
constexpr int kRegsConsumer = 152, kRegsProducer = 40;
constexpr int kHeads = 8;  // query heads of a row
constexpr int kPagesDeep = 6;
constexpr int kJoinThreads = 512;
static_assert(kPagesDeep % kTeams == 0, "a team's pages are in the same stages");
constexpr float kLateDecode = 8.0f;  // as in attn_prefill.cu
constexpr int kShares = 152;         // one per SM
static_assert(kShares <= kJoinThreads, "a thread per part");

struct DecodeAttnArgs {
  CacheArgs c;
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  const int *lengths;
  long long qs;
  int n_seq, Hq, group, blocks;  // blocks: rows of a key/value head, 8 query heads each
  float scale;                   // times log2(e)
  int4 *head;                    // [kShares]: what is to be joined
  float *part;                   // [2 kShares][8][D + 2]: output, maximum, sum
};

template <int D>
struct Page {
  static constexpr int kCodes = kPage * D / 2, kAffine = kPage * (D / kGroup) * 4;
  static constexpr int kBytes = 2 * (kCodes + kAffine);
  static constexpr int kPitch = D + 8;  // of the warps' outputs
  static constexpr int kOut = kConsumers * kHeads * kPitch * 4;
  static constexpr int kCtl = 12288;
  static constexpr int kTotal = kPagesDeep * kBytes + kOut + kCtl + 1024;
  static_assert(kTotal <= 227 * 1024 && kBytes % 1024 == 0, "shared memory");
};

struct DCtl {
  uint64_t full[kPagesDeep], empty[kPagesDeep];
  int ok[kPagesDeep];  // whether the stage holds a page
  int abort_flag, seq, at;  // at: the share's first unit within sequence seq's
  int warp_sum[kConsumers + 4];
  float m[kConsumers][kHeads], l[kConsumers][kHeads];
  alignas(16) float e[kConsumers][8][kHeads];  // sum of p b' of each group, then of p s'
  uint4 q[4][2][32];  // a row's queries as the first product's A: [group][8 columns][lane]
  float qsum[4][kHeads];
  alignas(16) float unit[kHeads][2];
  uint2 qbias[32];  // the sums of q as the A of the biases' product
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the first of a sum
__device__ __forceinline__ void mma0_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma0_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&v)[N]) {
  if constexpr (N == 4) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(a)
                 : "memory");
  } else {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a) : "memory");
  }
}
// nibbles 0 and 4 of w as bf16 128 + c
__device__ __forceinline__ uint32_t plus128(uint32_t w) { return (w & 0x000f000fu) | 0x43004300u; }
constexpr uint32_t kMinus136 = 0xc308c308u;  // bf16 -136, twice

// four 8 x 8 matrices of 16-bit values: lane l gets row l / 4, values 2 (l % 4), + 1
// of each; lanes 8 m .. 8 m + 7 the addresses of matrix m's rows
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// the same, transposed: rows 2 (l % 4), + 1 of value l / 4
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// an 8 x 8 matrix of 16-bit values (row l / 4, values 2 (l % 4), + 1 in lane l) transposed
__device__ __forceinline__ uint32_t turned(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// 16-byte piece of a row of codes in a stage, swizzled by TMA (128-byte or 64-byte
// pattern: the same piece of 8 rows lies in all banks); piece ^ p is that ^ 16 p
template <int D>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  return D == 256 ? row * 128 + (((piece ^ row) & 7) << 4) : row * 64 + (((piece ^ (row >> 1)) & 3) << 4);
}

// tokens of sequence i in the cache, its pages
__device__ __forceinline__ int pages_of(const DecodeAttnArgs &a, int i, int &len) {
  const long long most = static_cast<long long>(a.c.width) * kPage;
  len = max(a.lengths[i], 0);
  if (len > most) len = static_cast<int>(most);
  return len / kPage + (len % kPage != 0);
}

// where share s of `total` units starts: each of the first min(kShares, total)
// shares has a unit at least, so the parts of a row are in neighbouring ones
__device__ __forceinline__ int share_at(int total, int s) {
  return total >= kShares ? static_cast<int>(static_cast<long long>(total) * s / kShares) : min(s, total);
}

__device__ __forceinline__ bool poll_d(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < (1 << 21); ++i) {
    if (mbar_try_wait_sleep(bar, parity, 2000u)) return true;
    if (*abort_flag) return false;
  }
  return false;
}
// named barrier of the consumers that tells each whether any of them brought `bad`
__device__ __forceinline__ bool consumers_any(bool bad) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, 2, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(bad ? 1u : 0u), "n"(32 * kConsumers)
      : "memory");
  return r != 0;
}

}  // namespace

static_assert(offsetof(DCtl, e) % 16 == 0 && offsetof(DCtl, unit) % 16 == 0 && offsetof(DCtl, q) % 16 == 0 &&
                  offsetof(DCtl, qbias) % 8 == 0,
              "read and written as vectors");

// The queries as the first product's A: fp16 of q 2^-power, in the column order in
// which nibbles come out of a word (every other pair 4 bits up there, so 2^-4
// here), and their sums over the groups in the same unit as the products.
template <int D>
__device__ __forceinline__ void make_queries(const DecodeAttnArgs &a, DCtl &ctl, int seq, int head, int heads) {
  constexpr int kG = D / kGroup;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const __nv_bfloat16 *src = a.q + seq * a.qs + static_cast<long long>(head + (g < heads ? g : 0)) * D + 8 * c;
  uint4 v[kG][2];
  uint32_t most = 0;
#pragma unroll
  for (int x = 0; x < kG; ++x)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      v[x][t] = make_uint4(0, 0, 0, 0);
      if (g < heads) v[x][t] = *reinterpret_cast<const uint4 *>(src + 64 * x + 32 * t);
      const uint32_t w[4] = {v[x][t].x, v[x][t].y, v[x][t].z, v[x][t].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) most = max(most, max(w[i] << 16 & 0x7fff0000u, w[i] & 0x7fff0000u));
    }
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
  const int power = min(max(static_cast<int>(most >> 23) - 127 - 12, -126), 126);
  const float down = __uint_as_float(static_cast<uint32_t>(127 - power) << 23);
#pragma unroll
  for (int x = 0; x < kG; ++x) {
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t w[4] = {v[x][t].x, v[x][t].y, v[x][t].z, v[x][t].w};
      float f[8];
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16) * down;
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * down;
        sum += f[2 * i] + f[2 * i + 1];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float up = i & 1 ? 0x1p-4f : 1.0f;
        const __half2 z = __floats2half2_rn(f[i] * up, f[i + 4] * up);
        y[i] = *reinterpret_cast<const uint32_t *>(&z);
      }
      ctl.q[x][t][lane] = make_uint4(y[0], y[1], y[2], y[3]);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (c == 0) ctl.qsum[x][g] = sum * 0x1p-24f;
  }
  __syncwarp();
  {  // index k of the biases' product: group k % kG of part k / kG of the sums
    float part[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = 2 * c + j + 8 * i, which = k / kG;
        const float all = ctl.qsum[k % kG][g];
        const float hi = __bfloat162float(__float2bfloat16_rn(all));
        const float mid = __bfloat162float(__float2bfloat16_rn(all - hi));
        part[i][j] = which == 0 ? hi : which == 1 ? mid : which == 2 ? all - hi - mid : 0.0f;
      }
    ctl.qbias[lane] = make_uint2(bf16x2_bits(part[0][0], part[0][1]), bf16x2_bits(part[1][0], part[1][1]));
  }
  if (c == 0) {
    // scores come out in units of 2^(power + 24), taken off in two steps within range
    const int first = (power + 24) / 2;
    ctl.unit[g][0] = __uint_as_float(static_cast<uint32_t>(127 + first) << 23);
    ctl.unit[g][1] = a.scale * __uint_as_float(static_cast<uint32_t>(127 + power + 24 - first) << 23);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreadsD, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tm, const DecodeAttnArgs a) {
  using P = Page<D>;
  constexpr int kG = D / kGroup;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  float *obuf = reinterpret_cast<float *>(smem + kPagesDeep * P::kBytes);
  DCtl &ctl = *reinterpret_cast<DCtl *>(smem + kPagesDeep * P::kBytes + P::kOut);
  static_assert(sizeof(DCtl) <= P::kCtl, "control block");
  volatile int *abort_flag = &ctl.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = a.c.H * a.blocks, cta = blockIdx.x;
  if (tid == 0) {
    for (int s = 0; s < kPagesDeep; ++s) {
      mbar_init(smem_u32(&ctl.full[s]), 1);
      mbar_init(smem_u32(&ctl.empty[s]), 4);
    }
    ctl.abort_flag = 0;
    ctl.seq = 0;
    ctl.at = 0;
    fence_mbar_init();
    prefetch_tmap(&tm);
  }
  pdl_wait();
  pdl_launch_dependents();
  // pages before each thread's sequences, and the share's start
  const int per = (a.n_seq + kThreadsD - 1) / kThreadsD, i0 = min(tid * per, a.n_seq), i1 = min(i0 + per, a.n_seq);
  int sum = 0;
  bool over = false;
  for (int i = i0; i < i1; ++i) {
    int len;
    sum += pages_of(a, i, len);
    over = over || a.lengths[i] > len;
  }
  if (over && cta == 0) report_error(a.c.status, MOE_ERR_DEVICE_BOUNDS, KID_ATTN_DECODE * 100 + SITE_INDEX);
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) ctl.warp_sum[warp] = upto;
  __syncthreads();
  int before = upto - sum, total = 0;
  for (int w = 0; w < kThreadsD / 32; ++w) {
    if (w < warp) before += ctl.warp_sum[w];
    total += ctl.warp_sum[w];
  }
  total *= R;
  const int u0 = share_at(total, cta), u1 = share_at(total, cta + 1);
  if (u0 < u1 && u0 >= before * R && u0 < (before + sum) * R) {
    int at = u0 - before * R;
    for (int i = i0; i < i1; ++i) {
      int len;
      const int mine = pages_of(a, i, len) * R;
      if (at < mine) {
        ctl.seq = i;
        ctl.at = at;
        break;
      }
      at -= mine;
    }
  }
  if (tid == 0) a.head[cta] = make_int4(0, 0, 0, 0);
  __syncthreads();
  // sequences without tokens: zeros
  for (int i = cta; i < a.n_seq; i += kShares)
    if (a.lengths[i] <= 0 || a.c.width == 0)
      for (int x = tid; x < a.Hq * D / 8; x += kThreadsD)
        reinterpret_cast<uint4 *>(a.out + static_cast<long long>(i) * a.Hq * D)[x] = make_uint4(0, 0, 0, 0);

  int seq = ctl.seq, st = 0, len = 0;
  uint32_t phase = 0;
  int u = u0, at = ctl.at;
  int np = u0 < u1 ? pages_of(a, seq, len) : 0;
  bool ok = true;
  if (warp >= kConsumers) {
    // ------------------------------------------------------------ copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsProducer));
    if (warp > kConsumers) return;
    const uint64_t pol = policy_evict_first();
    while (ok && u < u1) {
      if (at >= np * R) {
        ++seq;
        at = 0;
        np = pages_of(a, seq, len);
        continue;
      }
      const int h = at / np / a.blocks, p0 = at % np, n = min(min(np - p0, 32), u1 - u);
      int page = -1;
      if (lane < n) {
        page = page_of(a.c, seq, static_cast<long long>(p0 + lane) * kPage);
        if (page < 0) report_error(a.c.status, MOE_ERR_DEVICE_BOUNDS, KID_ATTN_DECODE * 100 + SITE_INDEX);
      }
      for (int i = 0; i < n; ++i) {
        const int pg = __shfl_sync(0xffffffffu, page, i);
        ok = __all_sync(0xffffffffu, poll_d(smem_u32(&ctl.empty[st]), phase ^ 1, abort_flag));
        if (!ok) {
          if (lane == 0) {
            *abort_flag = 1;
            report_error(a.c.status, MOE_ERR_DEVICE_TIMEOUT, KID_ATTN_DECODE * 100 + SITE_PRODUCER_EMPTY);
          }
          break;
        }
        if (lane == 0) {
          ctl.ok[st] = pg >= 0;
          const uint32_t fb = smem_u32(&ctl.full[st]);
          uint8_t *dst = smem + st * P::kBytes;
          if (pg < 0) {
            mbar_arrive(fb);
          } else {
            mbar_arrive_expect_tx(fb, P::kBytes);
            for (int w = 0; w < 2; ++w) {
              const long long row = cache_row(a.c, pg, w, h, 0);
              tma_load_2d(smem_u32(dst) + w * P::kCodes, &tm, fb, 0, static_cast<int>(row), pol);
              bulk_g2s(dst + 2 * P::kCodes + w * P::kAffine, a.c.affine + row * kG, P::kAffine, &ctl.full[st]);
            }
          }
        }
        __syncwarp();
        if (++st == kPagesDeep) {
          st = 0;
          phase ^= 1;
        }
      }
      u += n;
      at += n;
    }
    if (!ok && lane == 0)  // copies in flight get time to land
      for (int i = 0; i < 200; ++i) __nanosleep(1000);
  } else {
    // ------------------------------------------------------------ tokens
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsConsumer));
    const int g = lane >> 2, c = lane & 3, tile = 16 * (warp & 3);
    // this lane's tokens: columns 2 c, 2 c + 1 of the two score tiles of 8
    const int key = tile + 2 * c;
    // rows of codes for the matrix loads: keys 8 (m & 1) + .. , pieces m >> 1 of matrix
    // m; values the same
    const int mrow = tile + 8 * ((lane >> 3) & 1) + (lane & 7);
    const uint32_t mat = piece_at<D>(mrow, lane >> 4);
    int mine = warp >> 2;
    st = mine;
    while (u < u1) {
      if (at >= np * R) {
        ++seq;
        at = 0;
        np = pages_of(a, seq, len);
        continue;
      }
      // a row, or the part of it that lies in this share
      const int rr = at / np, h = rr / a.blocks, head0 = rr % a.blocks * kHeads;
      const int heads = min(kHeads, a.group - head0), p0 = at % np;
      const int n = min(np - p0, u1 - u);
      const long long orow = static_cast<long long>(seq) * a.Hq + h * a.group + head0;
      // (all warps have left the row before)
      if (warp == 0) make_queries<D>(a, ctl, seq, h * a.group + head0, heads);
      named_bar_sync(1, 32 * kConsumers);
      const uint32_t sq = smem_u32(&ctl.q[0][0][lane]);
      const uint2 qb = ctl.qbias[lane];
      const float2 unit[2] = {*reinterpret_cast<const float2 *>(ctl.unit[2 * c]),
                              *reinterpret_cast<const float2 *>(ctl.unit[2 * c + 1])};
      // heads 2 c, 2 c + 1
      float o[kG][4][4] = {}, e[4] = {}, m[2] = {-INFINITY, -INFINITY}, ref[2] = {0.0f, 0.0f}, l[2] = {0.0f, 0.0f};
      // the pages of these four warps: mine pages on, and every kTeams-th
      int i = mine;
      for (; ok && i < n; i += kTeams) {
        const int now = st;
        const uint32_t ph = phase;
        if ((st += kTeams) >= kPagesDeep) {
          st -= kPagesDeep;
          phase ^= 1;
        }
        ok = __all_sync(0xffffffffu, poll_d(smem_u32(&ctl.full[now]), ph, abort_flag));
        if (!ok) {
          if (lane == 0) {
            *abort_flag = 1;
            report_error(a.c.status, MOE_ERR_DEVICE_TIMEOUT, KID_ATTN_DECODE * 100 + SITE_MMA_FULL);
          }
          break;
        }
        const int left = len - (p0 + i) * kPage;  // tokens of the sequence from this page on
        if (ctl.ok[now] && tile < left) {
          const uint32_t sk = smem_u32(smem) + now * P::kBytes, sv = sk + P::kCodes;
          const uint32_t fk = sv + P::kCodes, fv = fk + P::kAffine;
          // scores of 16 tokens (rows g, g + 8; heads 2 c, 2 c + 1): first the biases' part
          float s[4];
          {
            uint32_t bb[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint2 w = lds64(fk + (tile + g + 8 * y) * kG * 4 + (D == 256 ? 8 * (c & 1) : 0));
              bb[y] = __byte_perm(w.x, w.y, 0x7632);
            }
            mma0_bf16(s, bb[0], bb[1], bb[0], bb[1], qb.x, qb.y);
          }
          uint32_t ka[2][kG];
#pragma unroll
          for (int y = 0; y < 2; ++y) lds_words<kG>(fk + (tile + g + 8 * y) * kG * 4, ka[y]);
#pragma unroll
          for (int x = 0; x < kG; ++x) {
            const uint4 q0 = lds128(sq + x * 1024), q1 = lds128(sq + x * 1024 + 512);
            float acc[4];
            uint32_t w[4], u[4];  // 8 columns of the keys 0 .. 7, 8 .. 15, then 32 columns on
            ldsm4((sk + mat) ^ (32 * x), w);
#pragma unroll
            for (int y = 0; y < 4; ++y) u[y] = w[y] >> 8;
            mma0_f16(acc, w[0] & 0x000f000fu, w[1] & 0x000f000fu, w[0] & 0x00f000f0u, w[1] & 0x00f000f0u, q0.x, q0.y);
            mma_f16(acc, u[0] & 0x000f000fu, u[1] & 0x000f000fu, u[0] & 0x00f000f0u, u[1] & 0x00f000f0u, q0.z, q0.w);
            mma_f16(acc, w[2] & 0x000f000fu, w[3] & 0x000f000fu, w[2] & 0x00f000f0u, w[3] & 0x00f000f0u, q1.x, q1.y);
            mma_f16(acc, u[2] & 0x000f000fu, u[3] & 0x000f000fu, u[2] & 0x00f000f0u, u[3] & 0x00f000f0u, q1.z, q1.w);
#pragma unroll
            for (int y = 0; y < 4; ++y) s[y] = fmaf(__uint_as_float(ka[y >> 1][x] << 16), acc[y], s[y]);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) s[y] = s[y] * unit[y & 1].x * unit[y & 1].y;
          const bool end = left < tile + 16;  // the sequence ends in these tokens
          if (end) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (tile + g + 8 * (y >> 1) >= left) s[y] = -INFINITY;
          }
          float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
          if (__any_sync(0xffffffffu, top[0] > m[0] + kLateDecode || top[1] > m[1] + kLateDecode)) {
            float f[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
#pragma unroll
              for (int x = 4; x < 32; x *= 2) top[z] = fmaxf(top[z], __shfl_xor_sync(0xffffffffu, top[z], x));
              const float to = top[z] > m[z] + kLateDecode ? top[z] : m[z];
              f[z] = to == m[z] ? 1.0f : fast_exp2(m[z] - to);
              m[z] = to;
              ref[z] = to == -INFINITY ? 0.0f : to;
              l[z] *= f[z];
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              e[y] *= f[y & 1];
#pragma unroll
              for (int x = 0; x < kG; ++x)
#pragma unroll
                for (int t = 0; t < 4; ++t) o[x][t][y] *= f[y & 1];
            }
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            s[y] = fast_exp2(s[y] - ref[y & 1]);
            l[y & 1] += s[y];
          }
          // P turned (head g, tokens 2 c, 2 c + 1 of both halves), in two bf16 parts
          uint32_t h0 = bf16x2_bits(s[0], s[1]), h1 = bf16x2_bits(s[2], s[3]);
          uint32_t l0 = bf16x2_bits(s[0] - __uint_as_float(h0 << 16), s[1] - __uint_as_float(h0 & 0xffff0000u));
          uint32_t l1 = bf16x2_bits(s[2] - __uint_as_float(h1 << 16), s[3] - __uint_as_float(h1 & 0xffff0000u));
          h0 = turned(h0);
          h1 = turned(h1);
          l0 = turned(l0);
          l1 = turned(l1);
          const float pt[4] = {__uint_as_float(h0 << 16) + __uint_as_float(l0 << 16),
                               __uint_as_float(h0 & 0xffff0000u) + __uint_as_float(l0 & 0xffff0000u),
                               __uint_as_float(h1 << 16) + __uint_as_float(l1 << 16),
                               __uint_as_float(h1 & 0xffff0000u) + __uint_as_float(l1 & 0xffff0000u)};
          // scales of the values; of what is behind the end nothing may be seen (0 x NaN
          // is NaN)
          uint32_t va[4][kG], ve[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t at4 = fv + (key + 8 * (y >> 1) + (y & 1)) * kG * 4;
            ve[y] = lds32(at4 + (g & (kG - 1)) * 4);
            lds_words<kG>(at4, va[y]);
          }
          if (end) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (key + 8 * (y >> 1) + (y & 1) >= left) {
                ve[y] = 0u;
#pragma unroll
                for (int x = 0; x < kG; ++x) va[y][x] = 0u;
              }
          }
          {  // sums of p b' (rows g, group g % kG) and p s' (rows g + 8)
            const uint32_t a0 = __byte_perm(ve[0], ve[1], 0x7632), a1 = __byte_perm(ve[0], ve[1], 0x5410);
            const uint32_t a2 = __byte_perm(ve[2], ve[3], 0x7632), a3 = __byte_perm(ve[2], ve[3], 0x5410);
            mma_bf16(e, a0, a1, a2, a3, h0, h1);
            mma_bf16(e, a0, a1, a2, a3, l0, l1);
          }
          // the values: transposed, so that a word has four columns of two tokens
#pragma unroll
          for (int x = 0; x < kG; ++x) {
            float p[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) p[y] = pt[y] * __uint_as_float(va[y][x] << 16);
            const uint32_t b0 = bf16x2_bits(p[0], p[1]), b1 = bf16x2_bits(p[2], p[3]);
            uint32_t w[4];  // tokens 0 .. 7, 8 .. 15 of 32 columns, then 32 columns on
            ldsm4_t((sv + mat) ^ (32 * x), w);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t lo = w[t & 2] >> (8 * (t & 1)), hi = w[(t & 2) + 1] >> (8 * (t & 1));
              mma_bf16(o[x][t], plus128(lo), plus128(lo >> 4), plus128(hi), plus128(hi >> 4), b0, b1);
              mma_bf16(o[x][t], kMinus136, kMinus136, kMinus136, kMinus136, b0, b1);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.empty[now]));
      }
      mine = i - n;
      // join the warps' parts (also after an abort: all warps meet here)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[z] += __shfl_xor_sync(0xffffffffu, l[z], x);
        if (g == 0) {
          ctl.m[warp][2 * c + z] = m[z];
          ctl.l[warp][2 * c + z] = l[z];
        }
      }
      if (g < kG) {
        *reinterpret_cast<float2 *>(&ctl.e[warp][g][2 * c]) = make_float2(e[0], e[1]);
        *reinterpret_cast<float2 *>(&ctl.e[warp][4 + g][2 * c]) = make_float2(e[2], e[3]);
      }
#pragma unroll
      for (int x = 0; x < kG; ++x)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float *to = obuf + (warp * kHeads + 2 * c + z) * P::kPitch + 64 * x + 4 * g;
          *reinterpret_cast<float4 *>(to) = make_float4(o[x][0][z], o[x][0][2 + z], o[x][1][z], o[x][1][2 + z]);
          *reinterpret_cast<float4 *>(to + 32) = make_float4(o[x][2][z], o[x][2][2 + z], o[x][3][z], o[x][3][2 + z]);
        }
      named_bar_sync(1, 32 * kConsumers);
      if (warp < heads) {
        constexpr int kE = D / 32;  // columns per thread; the head is the warp's
        const int d0 = kE * lane;
        float M = -INFINITY, L = 0.0f, v[kE];
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, ctl.m[w][warp]);
#pragma unroll
        for (int i = 0; i < kE; ++i) v[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
          const float mw = ctl.m[w][warp], f = mw == M ? 1.0f : fast_exp2(mw - M);
          const float ew = fmaf(8.0f, ctl.e[w][4 + d0 / kGroup][warp], ctl.e[w][d0 / kGroup][warp]);
          L = fmaf(f, ctl.l[w][warp], L);
          const float *from = obuf + (w * kHeads + warp) * P::kPitch + d0;
#pragma unroll
          for (int i = 0; i < kE; ++i) v[i] = fmaf(f, from[i] + ew, v[i]);
        }
        if (n == np) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          __nv_bfloat16 *to = a.out + (orow + warp) * D + d0;
#pragma unroll
          for (int i = 0; i < kE; i += 2)
            *reinterpret_cast<uint32_t *>(to + i) = bf16x2_bits(v[i] * inv, v[i + 1] * inv);
        } else {
          const int slot = 2 * cta + (u == u0 ? 0 : 1);
          float *to = a.part + (static_cast<long long>(slot) * kHeads + warp) * (D + 2);
#pragma unroll
          for (int i = 0; i < kE; i += 2) *reinterpret_cast<float2 *>(to + d0 + i) = make_float2(v[i], v[i + 1]);
          if (lane == 0) *reinterpret_cast<float2 *>(to + D) = make_float2(M, L);
          if (p0 == 0 && tid == 0) {  // the row starts here: this share's entry says how it goes on
            const int last = u + np - 1;
            int end = static_cast<int>(min(((last + 1LL) * kShares - 1) / total, kShares - 1LL));
            while (share_at(total, end + 1) <= last) ++end;
            while (share_at(total, end) > last) --end;
            a.head[cta] = make_int4(end - cta + 1, slot, static_cast<int>(orow), heads);
          }
        }
      }
      if (consumers_any(!ok)) break;
      u += n;
      at += n;
    }
  }
}

// Joins the parts of the row that starts in share blockIdx.x and does not end
// there, for one of its heads: groups of D / 4 threads add up every so many parts,
// then their sums are added.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const DecodeAttnArgs a) {
  constexpr int kT = D / 4, kGroups = kJoinThreads / kT;
  __shared__ float s_f[kShares], s_red[kJoinThreads / 32], s_l[kJoinThreads / 32];
  __shared__ float4 s_o[kGroups][kT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hd = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  const int4 head = a.head[blockIdx.x];
  const int n = head.x;
  if (n <= 1 || hd >= head.w) return;
  auto part = [&](int i) {
    const int slot = i == 0 ? head.y : 2 * (static_cast<int>(blockIdx.x) + i);
    return a.part + (static_cast<long long>(slot) * kHeads + hd) * (D + 2);
  };
  float2 ml = make_float2(-INFINITY, 0.0f);
  if (tid < n) ml = *reinterpret_cast<const float2 *>(part(tid) + D);
  float M = ml.x;
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_red[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) M = fmaxf(M, s_red[w]);
  const float f = ml.x == M ? 1.0f : fast_exp2(ml.x - M);
  if (tid < n) s_f[tid] = f;
  float L = f * ml.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane == 0) s_l[warp] = L;
  __syncthreads();
  const int t = tid % kT, grp = tid / kT;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = grp; i < n; i += kGroups) {
    const float2 *p = reinterpret_cast<const float2 *>(part(i) + 4 * t);
    const float2 x = p[0], y = p[1];
    const float w = s_f[i];
    v.x = fmaf(w, x.x, v.x);
    v.y = fmaf(w, x.y, v.y);
    v.z = fmaf(w, y.x, v.z);
    v.w = fmaf(w, y.y, v.w);
  }
  s_o[grp][t] = v;
  __syncthreads();
  if (grp == 0) {
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) L += s_l[w];
#pragma unroll
    for (int x = 1; x < kGroups; ++x) {
      const float4 y = s_o[x][t];
      v.x += y.x;
      v.y += y.y;
      v.z += y.z;
      v.w += y.w;
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    uint32_t *to = reinterpret_cast<uint32_t *>(a.out + (static_cast<long long>(head.z) + hd) * D + 4 * t);
    to[0] = bf16x2_bits(v.x * inv, v.y * inv);
    to[1] = bf16x2_bits(v.z * inv, v.w * inv);
  }
}

namespace {

struct DecodeDevice {
  int *status = nullptr;
  int rc = MOE_ERR_CUDA;
};

const DecodeDevice &decode_device() {
  static DecodeDevice devs[64];
  static std::once_flag once[64];
  static const DecodeDevice none;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return none;
  std::call_once(once[dev], [dev] {
    DecodeDevice &d = devs[dev];
    d.status = noalloc_status_word();
    auto set = [](auto kern, int bytes) {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
    };
    if (d.status && set(attn_decode_kernel<128>, Page<128>::kTotal) && set(attn_decode_kernel<256>, Page<256>::kTotal))
      d.rc = MOE_OK;
  });
  return devs[dev];
}

template <int D>
cudaError_t launch_decode_attn(const CUtensorMap &tm, const DecodeAttnArgs &a, cudaStream_t st) {
  const cudaError_t e = launch_attn(attn_decode_kernel<D>, dim3(kShares), kThreadsD, Page<D>::kTotal, st, tm, a);
  if (e != cudaSuccess) return e;
  return launch_attn(attn_join_kernel<D>, dim3(kShares, a.group < kHeads ? a.group : kHeads), kJoinThreads, 0, st, a);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_attention_decode_workspace(int n_seq, int table_width, int n_q_heads,
                                              int n_kv_heads, int head_dim, size_t *bytes) {
  if (!bytes || n_seq < 0 || table_width < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0)
    return MOE_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || n_q_heads > 4096 || table_width > (1 << 25)) return MOE_ERR_UNSUPPORTED;
  *bytes = n_seq == 0 ? 0 : kShares * sizeof(int4) + 2 * kShares * sizeof(float) * kHeads * (head_dim + 2);
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
  if (n_pages > 0x7fffffffLL || n_pages * 2 * n_kv_heads * kPage > 0x7fffffffLL || q_stride >= (1LL << 39) ||
      static_cast<long long>(n_seq) * n_q_heads > 0x7fffffffLL ||
      static_cast<long long>(n_seq) * table_width >
          0x7fffffffLL / (n_kv_heads * ((n_q_heads / n_kv_heads + kHeads - 1) / kHeads)))
    return MOE_ERR_UNSUPPORTED;
  if (q_stride % 8 != 0) return MOE_ERR_ALIGNMENT;
  if (n_seq == 0) return MOE_OK;
  if (!q || !out || !lengths || (n_pages > 0 && (!codes || !affine)) || (table_width > 0 && !pages) || !workspace ||
      workspace_bytes < need)
    return MOE_ERR_INVALID_ARG;
  if (off_boundary(q, 16) || off_boundary(out, 16) || off_boundary(codes, 16) || off_boundary(affine, 16) ||
      off_boundary(workspace, 16) || off_boundary(pages, 4) || off_boundary(lengths, 4))
    return MOE_ERR_ALIGNMENT;
  const DecodeDevice &dev = decode_device();
  if (dev.rc != MOE_OK) return dev.rc;
  DecodeAttnArgs a = {};
  a.c = {const_cast<uint8_t *>(codes), reinterpret_cast<uint32_t *>(const_cast<uint16_t *>(affine)), pages,
         n_pages, table_width, n_kv_heads, head_dim, dev.status};
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lengths = lengths;
  a.qs = q_stride;
  a.n_seq = n_seq;
  a.Hq = n_q_heads;
  a.group = n_q_heads / n_kv_heads;
  a.blocks = (a.group + kHeads - 1) / kHeads;
  a.scale = scale * 1.4426950408889634f;
  a.head = static_cast<int4 *>(workspace);
  a.part = reinterpret_cast<float *>(a.head + kShares);
  // (without pages nothing is read: the map then stands over the queries)
  CUtensorMap tm;
  const uint64_t rows = n_pages > 0 ? n_pages * 2 * n_kv_heads * kPage : 1;
  if (!encode_map_2d(&tm, n_pages > 0 ? static_cast<const void *>(codes) : q, 1, rows, head_dim / 2, head_dim / 2,
                     kPage, head_dim == 256, 0, head_dim == 128))
    return MOE_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = head_dim == 128 ? launch_decode_attn<128>(tm, a, st) : launch_decode_attn<256>(tm, a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
