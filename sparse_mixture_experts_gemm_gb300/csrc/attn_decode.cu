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
//     (the largest is in [2^12, 2^13): what is lost is at most 2^-33 of it).
//   * Values: weights times scales need bf16's range, and 128 + c is one AND-OR away
//     from a nibble; a second product takes off 136 p_t s'_tg at once, so that the
//     sum stays centred and has no large part that cancels against the bias's.
//   * The biases' sums are products, too: bf16 biases with the sums of q in three bf16
//     parts, p in two with b' and s'.
// The only rounding before the result's is that of p_t s'_tg to bf16 (2^-8), which
// multiplies codes less 8 (and that of p to 2^-16 with the biases).
//
// Work split.  All (sequence, key/value head, 8 query heads) rows' pages lie on one
// line that is cut into equal shares, three per SM, whatever the lengths; a CTA
// finds its shares from the lengths on the device.  Rows that are cut leave their
// parts (output, maximum, sum) in the workspace for a second kernel, which joins
// them in a fixed order.
//
// Roles: three teams of four warps have a share each; a page's tokens go to the four
// warps by 16, with a running softmax of their own, and their parts are joined
// through shared memory at a row's end, while the other teams go on (with one share
// per SM and all warps on it, every row's end cost 5 us).  Warps 12-14 walk along the
// teams' rows and copy their pages by TMA, three ahead.  The codes are the A operand of
// both products (tokens x columns, columns x tokens), whose four registers the
// dequantisation fills as they are; P is turned in between, four 8 x 8 matrices.
//
// Measured, 16 query heads on 2 of 256: 64 sequences of 17 to 8,192 tokens 44 us (148 MB,
// 3.3 TB/s), one of 131,072 26.6 us, one of 4,097 9.2 us.  32 on 8 of 128: the same 64
// sequences 89 us (294 MB, 3.3 TB/s), one of 131,072 42 us; 16 on 2 of 128: 30, 17.4 us.
// No unit is at its limit (ALU 57 % busy, matrix instructions 32 %, issue 50 %, DRAM 45 %):
// three warps a scheduler have a long chain from codes to scores to weights to values
// to cover, with 5 ALU instructions per 8 codes of the keys and 7 of the values.  Scores of
// the next page between the products of this one (47 us) and shifts by high products on the
// other pipe (48) gained nothing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <mutex>

#include "../../include/moe.h"
#include "attn_common.cuh"

namespace moe {

namespace {

constexpr int kTeams = 3, kTeamWarps = 4;
constexpr int kConsumers = kTeams * kTeamWarps;
constexpr int kThreadsD = 32 * (kConsumers + 4);  // (whole warpgroups, for their shares of the registers)
// 128 registers a thread at launch: 16 x 32 x 128 = 12 x 32 x 152 + 4 x 32 x 48 + 1024
constexpr int kRegsConsumer = 152, kRegsProducer = 48;
constexpr int kHeads = 8;      // query heads of a row
constexpr int kPagesDeep = 3;  // of a team
constexpr int kRowsDeep = 4;   // more than kPagesDeep: that many rows can the copies be ahead
constexpr int kJoinThreads = 512;
constexpr float kLateDecode = 8.0f;  // as in attn_prefill.cu
constexpr float kLowest = -3.402823466e38f;
constexpr int kCtas = 152, kShares = kCtas * kTeams;  // one CTA per SM

struct DecodeAttnArgs {
  CacheArgs c;
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  const int *lengths;
  long long qs;
  int n_seq, Hq, group, blocks;  // blocks: rows of a key/value head, 8 query heads each
  float scale;                   // times log2(e)
  AttnWaits waits;
  int4 *head;                    // [kShares]: what is to be joined
  float *part;                   // [2 kShares][8][D + 4]: output, maximum, sum
};

// A row, or the part of it that lies in a share: what the roles walk along.
struct Row {
  int u, at, seq, np, len;  // unit, unit within the sequence's, the sequence, its pages and tokens
  int h, head0, heads;      // key/value head, first query head of the 8 in its group, how many
  int p0, n;                // first page, pages
};

struct Team {
  uint64_t full[kPagesDeep], empty[kPagesDeep], row[kRowsDeep];
  int ok[kPagesDeep];  // whether the stage holds a page
  int u0, u1, seq, at;  // the share; its first unit's sequence, unit within the sequence's
  // rows: pages (0: no more), tokens from the first on, heads, row of out, place of
  // the part or -1, sequence, query head.  Read until the row's end, when the copies
  // are at most kPagesDeep rows on.
  struct {
    int n, left, heads, out, slot, seq, head;
  } todo[2 * kRowsDeep];
  float m[kTeamWarps][kHeads], l[kTeamWarps][kHeads];
  uint32_t most[kTeamWarps][kHeads];
  float qsum[4][kHeads];
  alignas(16) uint4 q[4][2][32];  // a row's queries as the first product's B: [group][32 columns][lane]
};

struct DCtl {
  Team team[kTeams];
  int abort_flag, total;  // total: all units
  int warp_sum[4];
};

template <int D>
struct Page {
  static constexpr int kCodes = kPage * D / 2, kAffine = kPage * (D / kGroup) * 4;
  static constexpr int kBytes = 2 * (kCodes + kAffine);
  static constexpr int kOut = kHeads * D * 4;  // a warp's output
  static constexpr int kSlots = kTeams * 2;
  static constexpr int kTotal = kTeams * kPagesDeep * kBytes + kSlots * kOut + static_cast<int>(sizeof(DCtl)) + 1024;
  static_assert(kTotal <= 227 * 1024 && kBytes % 1024 == 0, "shared memory");
};
static_assert(offsetof(Team, q) % 16 == 0 && sizeof(Team) % 16 == 0, "read and written as vectors");

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

__device__ __forceinline__ bool poll_d(uint32_t bar, uint32_t parity, const volatile int *abort_flag, int polls) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < polls; ++i) {
    if (mbar_try_wait_sleep(bar, parity, 2000u)) return true;
    if (*abort_flag) return false;
  }
  return false;
}
}  // namespace

// the share's start; then to the next row, false: the share is done
__device__ __forceinline__ void start_row(Row &r, const DecodeAttnArgs &a, const Team &t) {
  r.u = t.u0;
  r.at = t.at;
  r.seq = t.seq;
  r.np = r.len = r.n = 0;
  if (t.u0 < t.u1) r.np = pages_of(a, r.seq, r.len);
}
__device__ __forceinline__ bool next_row(Row &r, const DecodeAttnArgs &a, const Team &t) {
  r.u += r.n;
  r.at += r.n;
  if (r.u >= t.u1) return false;
  while (r.at >= r.np * a.c.H * a.blocks) {
    ++r.seq;
    r.at = 0;
    r.np = pages_of(a, r.seq, r.len);
  }
  const int x = r.at / r.np;
  r.h = x / a.blocks;
  r.head0 = x % a.blocks * kHeads;
  r.heads = min(kHeads, a.group - r.head0);
  r.p0 = r.at % r.np;
  r.n = min(r.np - r.p0, t.u1 - r.u);
  return true;
}

// A row's queries as the first product's B, by a team's warps, which have a group of
// 64 columns each (lane (g, c): head g, columns 8 c .. of each 32): fp16 of q
// 2^-power, in the column order in which nibbles come out of a word (every other
// pair 4 bits up there, so 2^-4 here), and their sums in the same unit as the
// products, all of which each warp then takes as the B of the biases' product.
// unit: what scores of heads 2 c, 2 c + 1 are to be multiplied with, in two steps
// within range.
template <int D>
__device__ __forceinline__ void make_queries(const DecodeAttnArgs &a, Team &t, int tw, int sync, int seq, int head,
                                             int heads, uint2 &qbias, float2 (&unit)[2]) {
  constexpr int kG = D / kGroup;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint32_t w[2][4] = {};
  if (tw < kG && g < heads) {
    const __nv_bfloat16 *src = a.q + seq * a.qs + static_cast<long long>(head + g) * D + 64 * tw + 8 * c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = *reinterpret_cast<const uint4 *>(src + 32 * i);
      w[i][0] = v.x;
      w[i][1] = v.y;
      w[i][2] = v.z;
      w[i][3] = v.w;
    }
  }
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = w[i >> 2][i & 3];
    most = max(most, max(x << 16 & 0x7fff0000u, x & 0x7fff0000u));
  }
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
  if (c == 0) t.most[tw][g] = most;
  named_bar_sync(sync, 32 * kTeamWarps);
  auto power_of = [&](int hd) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < kG; ++i) x = max(x, t.most[i][hd]);
    return min(max(static_cast<int>(x >> 23) - 127 - 12, -126), 126);
  };
  const int power = power_of(g);
  const float down = __uint_as_float(static_cast<uint32_t>(127 - power) << 23);
  if (tw < kG) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float f[8];
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[i][j] << 16) * down;
        f[2 * j + 1] = __uint_as_float(w[i][j] & 0xffff0000u) * down;
        sum += f[2 * j] + f[2 * j + 1];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float up = j & 1 ? 0x1p-4f : 1.0f;
        const __half2 z = __floats2half2_rn(f[j] * up, f[j + 4] * up);
        y[j] = *reinterpret_cast<const uint32_t *>(&z);
      }
      t.q[tw][i][lane] = make_uint4(y[0], y[1], y[2], y[3]);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (c == 0) t.qsum[tw][g] = sum * 0x1p-24f;
  }
  // scores come out in units of 2^(power + 24)
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const int all = power_of(2 * c + z) + 24, first = all / 2;
    unit[z] = make_float2(__uint_as_float(static_cast<uint32_t>(127 + first) << 23),
                          a.scale * __uint_as_float(static_cast<uint32_t>(127 + all - first) << 23));
  }
  named_bar_sync(sync, 32 * kTeamWarps);
  // index k of the biases' product: group k % kG of part k / kG of the sums
  float part[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = 2 * c + j + 8 * i, which = k / kG;
      const float all = t.qsum[k % kG][g];
      const float hi = __bfloat162float(__float2bfloat16_rn(all));
      const float mid = __bfloat162float(__float2bfloat16_rn(all - hi));
      part[i][j] = which == 0 ? hi : which == 1 ? mid : which == 2 ? all - hi - mid : 0.0f;
    }
  qbias = make_uint2(bf16x2_bits(part[0][0], part[0][1]), bf16x2_bits(part[1][0], part[1][1]));
}

template <int D>
__global__ void __launch_bounds__(kThreadsD, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tm, const DecodeAttnArgs a) {
  using P = Page<D>;
  constexpr int kG = D / kGroup;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  uint8_t *slots = smem + kTeams * kPagesDeep * P::kBytes;
  DCtl &ctl = *reinterpret_cast<DCtl *>(slots + P::kSlots * P::kOut);
  volatile int *abort_flag = &ctl.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  if (tid < kTeams) {
    Team &t = ctl.team[tid];
    for (int s = 0; s < kPagesDeep; ++s) {
      mbar_init(smem_u32(&t.full[s]), 1);
      mbar_init(smem_u32(&t.empty[s]), kTeamWarps);
    }
    for (int r = 0; r < kRowsDeep; ++r) mbar_init(smem_u32(&t.row[r]), 1);
    t.seq = t.at = 0;
    ctl.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm);
  }
  __syncthreads();
  auto timeout = [&](int site) {
    if (lane == 0) {
      *abort_flag = 1;
      report_error(a.c.status, MOE_ERR_DEVICE_TIMEOUT, KID_ATTN_DECODE * 100 + site);
    }
  };
  constexpr int kSetup = 4, kSync = 5, kVote = 8;  // named barriers; the last two one per team

  if (warp >= kConsumers) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsProducer));
    const int x = tid - 32 * kConsumers, role = warp - kConsumers;
    const int R = a.c.H * a.blocks;
    pdl_wait();
    pdl_launch_dependents();
    // pages before each thread's sequences, and the shares' starts
    const int per = (a.n_seq + 127) / 128, i0 = min(x * per, a.n_seq), i1 = min(i0 + per, a.n_seq);
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
    if (lane == 31) ctl.warp_sum[role] = upto;
    named_bar_sync(kSetup, 128);
    int before = upto - sum, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < role) before += ctl.warp_sum[w];
      total += ctl.warp_sum[w];
    }
    total *= R;
    for (int k = 0; k < kTeams; ++k) {
      // (the first shares, which have units when there are few, are on different SMs)
      const int share = k * kCtas + cta, u0 = share_at(total, share), u1 = share_at(total, share + 1);
      Team &t = ctl.team[k];
      if (u0 < u1 && u0 >= before * R && u0 < (before + sum) * R) {
        int at = u0 - before * R;
        for (int i = i0; i < i1; ++i) {
          int len;
          const int units = pages_of(a, i, len) * R;
          if (at < units) {
            t.seq = i;
            t.at = at;
            break;
          }
          at -= units;
        }
      }
      if (x == k) {
        t.u0 = u0;
        t.u1 = u1;
        a.head[share] = make_int4(0, 0, 0, 0);
      }
    }
    named_bar_sync(kSetup, 128);
    bool ok = true;
    if (role < kTeams) {
      // ---------------------------------------------------------- copies of a team's pages
      Team &t = ctl.team[role];
      uint8_t *stages = smem + role * kPagesDeep * P::kBytes;
      const uint64_t pol = policy_evict_first();
      Row r;
      start_row(r, a, t);
      int st = 0, loads = 0;
      uint32_t phase = 0;
      for (int nr = 0; ok; ++nr) {
        const bool more = next_row(r, a, t);
        if (lane == 0) {
          auto &todo = t.todo[nr % (2 * kRowsDeep)];
          const int share = role * kCtas + cta;
          const bool whole = r.n == r.np;
          todo.n = more ? r.n : 0;
          todo.left = r.len - r.p0 * kPage;
          todo.heads = r.heads;
          todo.seq = r.seq;
          todo.head = r.h * a.group + r.head0;
          todo.out = r.seq * a.Hq + todo.head;
          todo.slot = whole ? -1 : 2 * share + (r.u == t.u0 ? 0 : 1);
          mbar_arrive(smem_u32(&t.row[nr % kRowsDeep]));
        }
        if (!more) break;
        int pages = -1;  // numbers of 32 pages at a time
        for (int i = 0; i < r.n; ++i) {
          if ((i & 31) == 0) {
            pages = -1;
            if (i + lane < r.n) {
              pages = page_of(a.c, r.seq, static_cast<long long>(r.p0 + i + lane) * kPage);
              if (pages < 0) report_error(a.c.status, MOE_ERR_DEVICE_BOUNDS, KID_ATTN_DECODE * 100 + SITE_INDEX);
            }
          }
          const int page = __shfl_sync(0xffffffffu, pages, i & 31);
          ok = __all_sync(0xffffffffu, poll_d(smem_u32(&t.empty[st]), phase ^ 1, abort_flag, a.waits.polls));
          if (!ok) {
            timeout(SITE_PRODUCER_EMPTY);
            break;
          }
          if (loads++ >= a.waits.loads) {
            ok = false;
            break;
          }
          if (lane == 0) {
            t.ok[st] = page >= 0;
            const uint32_t fb = smem_u32(&t.full[st]);
            uint8_t *dst = stages + st * P::kBytes;
            if (page < 0) {
              mbar_arrive(fb);
            } else {
              mbar_arrive_expect_tx(fb, P::kBytes);
              for (int w = 0; w < 2; ++w) {
                const long long row = cache_row(a.c, page, w, r.h, 0);
                tma_load_2d(smem_u32(dst) + w * P::kCodes, &tm, fb, 0, static_cast<int>(row), pol);
                bulk_g2s(dst + 2 * P::kCodes + w * P::kAffine, a.c.affine + row * kG, P::kAffine, &t.full[st]);
              }
            }
          }
          __syncwarp();
          if (++st == kPagesDeep) {
            st = 0;
            phase ^= 1;
          }
        }
        if (lane == 0 && r.p0 == 0 && r.n < r.np) {  // the row starts here: this share's entry says how it goes on
          const int share = role * kCtas + cta, last = r.u + r.np - 1;
          // (an estimate, within one or two; a division of 64 bits took 2 us here)
          int end = total < kShares ? last : min(static_cast<int>(__fdividef(static_cast<float>(last), static_cast<float>(total)) * kShares), kShares - 1);
          while (share_at(total, end + 1) <= last) ++end;
          while (share_at(total, end) > last) --end;
          a.head[share] = make_int4(end - share + 1, 2 * share + (r.u == t.u0 ? 0 : 1),
                                    r.seq * a.Hq + r.h * a.group + r.head0, r.heads);
        }
        __syncwarp();
      }
    } else {
      // sequences without tokens: zeros
      for (int i = cta; i < a.n_seq; i += kCtas)
        if (a.lengths[i] <= 0 || a.c.width == 0)
          for (int y = lane; y < a.Hq * D / 8; y += 32)
            reinterpret_cast<uint4 *>(a.out + static_cast<long long>(i) * a.Hq * D)[y] = make_uint4(0, 0, 0, 0);
    }
  } else {
    // ------------------------------------------------------------ tokens
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsConsumer));
    const int team = warp / kTeamWarps, tw = warp % kTeamWarps;
    const int g = lane >> 2, c = lane & 3, tile = 16 * tw;
    Team &t = ctl.team[team];
    // places in a stage: rows of codes for the matrix loads (matrix m: rows 8 (m & 1)
    // .. of 16, piece m >> 1), scales and biases of this lane's tokens as rows of the
    // scores (g, g + 8 of 16) and as columns (2 c, 2 c + 1, + 8)
    const uint32_t stages = smem_u32(smem) + team * kPagesDeep * P::kBytes;
    const uint32_t mat = piece_at<D>(tile + (lane & 15), lane >> 4);
    const uint32_t rowat = (tile + g) * kG * 4, colat = (tile + 2 * c) * kG * 4;
    const uint32_t sq = smem_u32(&t.q[0][0][lane]);
    int st = 0;
    uint32_t phase = 0;
    bool ok = true;
    pdl_wait();
    for (int nr = 0;; ++nr) {
      if (ok) {
        ok = __all_sync(0xffffffffu, poll_d(smem_u32(&t.row[nr % kRowsDeep]), nr / kRowsDeep & 1, abort_flag, a.waits.polls));
        if (!ok) timeout(SITE_STAGE);
      }
      // the team goes on, or leaves, as one (and all are done with the row before)
      if (named_bar_any(kVote + team, 32 * kTeamWarps, !ok)) break;
      const auto &todo = t.todo[nr % (2 * kRowsDeep)];
      const int n = todo.n;
      if (n == 0) break;
      int left = todo.left;  // tokens of the sequence from the page on
      uint2 qb;
      float2 unit[2];
      make_queries<D>(a, t, tw, kSync + team, todo.seq, todo.head, todo.heads, qb, unit);
      // heads 2 c, 2 c + 1
      float o[kG][4][4] = {}, e[4] = {}, m[2] = {-INFINITY, -INFINITY}, ref[2] = {0.0f, 0.0f}, l[2] = {0.0f, 0.0f};
      for (int i = 0; ok && i < n; ++i, left -= kPage) {
        ok = __all_sync(0xffffffffu, poll_d(smem_u32(&t.full[st]), phase, abort_flag, a.waits.polls));
        if (!ok) {
          timeout(SITE_MMA_FULL);
          break;
        }
        if (t.ok[st] && tile < left) {
          const uint32_t sk = stages + st * P::kBytes, sv = sk + P::kCodes;
          const uint32_t fk = sv + P::kCodes, fv = fk + P::kAffine;
          // scores of 16 tokens (rows g, g + 8; heads 2 c, 2 c + 1): first the biases' part
          float s[4];
          uint32_t ka[2][kG], bb[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t at4 = fk + rowat + 8 * y * kG * 4;
            const uint2 w = lds64(at4 + (D == 256 ? 8 * (c & 1) : 0));
            bb[y] = __byte_perm(w.x, w.y, 0x7632);
            lds_words<kG>(at4, ka[y]);
          }
          mma0_bf16(s, bb[0], bb[1], bb[0], bb[1], qb.x, qb.y);
#pragma unroll
          for (int x = 0; x < kG; ++x) {
            const uint4 q0 = lds128(sq + x * 1024), q1 = lds128(sq + x * 1024 + 512);
            uint32_t w[4], u[4];  // 8 columns of the keys 0 .. 7, 8 .. 15, then 32 columns on
            float acc[4];
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
          // (not below the lowest number: m is minus infinity where no token was attended to,
          // and there alone the result is zero)
          float top[2] = {fmaxf(fmaxf(s[0], s[2]), kLowest), fmaxf(fmaxf(s[1], s[3]), kLowest)};
          if (__any_sync(0xffffffffu, top[0] > m[0] + kLateDecode || top[1] > m[1] + kLateDecode)) {
            float f[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
#pragma unroll
              for (int x = 4; x < 32; x *= 2) top[z] = fmaxf(top[z], __shfl_xor_sync(0xffffffffu, top[z], x));
              const float to = top[z] > m[z] + kLateDecode ? top[z] : m[z];
              f[z] = to == m[z] ? 1.0f : fast_exp2(m[z] - to);
              m[z] = to;
              ref[z] = to;
              l[z] *= f[z];
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              e[y] *= f[y & 1];
#pragma unroll
              for (int x = 0; x < kG; ++x)
#pragma unroll
                for (int z = 0; z < 4; ++z) o[x][z][y] *= f[y & 1];
            }
          }
          // P turned (head g, tokens 2 c, 2 c + 1 of both halves), in two bf16 parts
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            s[y] = fast_exp2(s[y] - ref[y & 1]);
            l[y & 1] += s[y];
          }
          float pt[4];
          uint32_t hi[2], lo[2], ve[4], va[4][kG];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float a0 = s[2 * z], a1 = s[2 * z + 1];
            hi[z] = bf16x2_bits(a0, a1);
            lo[z] = bf16x2_bits(a0 - __uint_as_float(hi[z] << 16), a1 - __uint_as_float(hi[z] & 0xffff0000u));
            hi[z] = turned(hi[z]);
            lo[z] = turned(lo[z]);
            pt[2 * z] = __uint_as_float(hi[z] << 16) + __uint_as_float(lo[z] << 16);
            pt[2 * z + 1] = __uint_as_float(hi[z] & 0xffff0000u) + __uint_as_float(lo[z] & 0xffff0000u);
          }
          // scales of the values; of what is behind the end nothing may be seen (0 x NaN
          // is NaN)
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const uint32_t at4 = fv + colat + (8 * (z >> 1) + (z & 1)) * kG * 4;
            ve[z] = lds32(at4 + (g & (kG - 1)) * 4);
            lds_words<kG>(at4, va[z]);
          }
          if (end) {
#pragma unroll
            for (int z = 0; z < 4; ++z)
              if (tile + 2 * c + 8 * (z >> 1) + (z & 1) >= left) {
                ve[z] = 0u;
#pragma unroll
                for (int x = 0; x < kG; ++x) va[z][x] = 0u;
              }
          }
          {  // sums of p b' (rows g, group g % kG) and p s' (rows g + 8)
            const uint32_t a0 = __byte_perm(ve[0], ve[1], 0x7632), a1 = __byte_perm(ve[0], ve[1], 0x5410);
            const uint32_t a2 = __byte_perm(ve[2], ve[3], 0x7632), a3 = __byte_perm(ve[2], ve[3], 0x5410);
            mma_bf16(e, a0, a1, a2, a3, hi[0], hi[1]);
            mma_bf16(e, a0, a1, a2, a3, lo[0], lo[1]);
          }
          // the values: transposed, so that a word has four columns of two tokens
#pragma unroll
          for (int x = 0; x < kG; ++x) {
            float p[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) p[z] = pt[z] * __uint_as_float(va[z][x] << 16);
            const uint32_t b0 = bf16x2_bits(p[0], p[1]), b1 = bf16x2_bits(p[2], p[3]);
            uint32_t w[4];  // tokens 0 .. 7, 8 .. 15 of 32 columns, then 32 columns on
            ldsm4_t((sv + mat) ^ (32 * x), w);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t v0 = w[z & 2] >> (8 * (z & 1)), v1 = w[(z & 2) + 1] >> (8 * (z & 1));
              mma_bf16(o[x][z], plus128(v0), plus128(v0 >> 4), plus128(v1), plus128(v1 >> 4), b0, b1);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z) mma_bf16(o[x][z], kMinus136, kMinus136, kMinus136, kMinus136, b0, b1);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&t.empty[st]));
        if (++st == kPagesDeep) {
          st = 0;
          phase ^= 1;
        }
      }
      // join the warps' parts (also after an abort: all warps meet here): the biases'
      // sums of group x are with the lanes g = x
      e[0] = fmaf(8.0f, e[2], e[0]);
      e[1] = fmaf(8.0f, e[3], e[1]);
#pragma unroll
      for (int x = 0; x < kG; ++x) {
        const float e0 = __shfl_sync(0xffffffffu, e[0], 4 * x + c), e1 = __shfl_sync(0xffffffffu, e[1], 4 * x + c);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          o[x][z][0] += e0;
          o[x][z][1] += e1;
          o[x][z][2] += e0;
          o[x][z][3] += e1;
        }
      }
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[z] += __shfl_xor_sync(0xffffffffu, l[z], x);
      // warps 2, 3 to 0, 1, then 1 to 0: four registers of a lane side by side
      float4 *slot = reinterpret_cast<float4 *>(slots + (team * 2 + (tw & 1)) * P::kOut) + lane;
      auto put = [&] {
#pragma unroll
        for (int x = 0; x < kG; ++x)
#pragma unroll
          for (int z = 0; z < 4; ++z) slot[(x * 4 + z) * 32] = make_float4(o[x][z][0], o[x][z][1], o[x][z][2], o[x][z][3]);
        if (g == 0) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            t.m[tw][2 * c + z] = m[z];
            t.l[tw][2 * c + z] = l[z];
          }
        }
      };
      auto take = [&](int from, const float4 *src) {
        float f[2], to[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float other = t.m[from][2 * c + z], M = fmaxf(m[z], other);
          f[z] = m[z] == M ? 1.0f : fast_exp2(m[z] - M);
          to[z] = other == M ? 1.0f : fast_exp2(other - M);
          m[z] = M;
          l[z] = l[z] * f[z] + to[z] * t.l[from][2 * c + z];
        }
#pragma unroll
        for (int x = 0; x < kG; ++x)
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float4 v = src[(x * 4 + z) * 32];
            o[x][z][0] = fmaf(to[0], v.x, f[0] * o[x][z][0]);
            o[x][z][1] = fmaf(to[1], v.y, f[1] * o[x][z][1]);
            o[x][z][2] = fmaf(to[0], v.z, f[0] * o[x][z][2]);
            o[x][z][3] = fmaf(to[1], v.w, f[1] * o[x][z][3]);
          }
      };
      if (tw >= 2) put();
      named_bar_sync(kSync + team, 32 * kTeamWarps);
      if (tw < 2) take(tw + 2, slot);
      if (tw == 1) put();  // (over what it has read itself)
      named_bar_sync(kSync + team, 32 * kTeamWarps);
      if (tw == 0 && ok) {
        take(1, slot + P::kOut / 16);
        // o[x][z]: columns 64 x + 32 (z / 2) + 4 g + 2 (z % 2) + 0 (registers 0, 1), + 1 (2, 3)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (2 * c + y >= todo.heads) continue;
          if (todo.slot < 0) {
            const float inv = m[y] == -INFINITY ? 0.0f : 1.0f / l[y];
            __nv_bfloat16 *to = a.out + static_cast<long long>(todo.out + 2 * c + y) * D + 4 * g;
#pragma unroll
            for (int x = 0; x < kG; ++x)
#pragma unroll
              for (int z = 0; z < 4; z += 2)
                *reinterpret_cast<uint2 *>(to + 64 * x + 16 * z) =
                    make_uint2(bf16x2_bits(o[x][z][y] * inv, o[x][z][2 + y] * inv),
                               bf16x2_bits(o[x][z + 1][y] * inv, o[x][z + 1][2 + y] * inv));
          } else {
            float *to = a.part + (static_cast<long long>(todo.slot) * kHeads + 2 * c + y) * (D + 4) + 4 * g;
#pragma unroll
            for (int x = 0; x < kG; ++x)
#pragma unroll
              for (int z = 0; z < 4; z += 2)
                *reinterpret_cast<float4 *>(to + 64 * x + 16 * z) =
                    make_float4(o[x][z][y], o[x][z][2 + y], o[x][z + 1][y], o[x][z + 1][2 + y]);
            if (g == 0) *reinterpret_cast<float2 *>(to + D) = make_float2(m[y], l[y]);
          }
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag)  // after an abort the copies in flight get time to land
    for (int i = 0; i < 200; ++i) __nanosleep(1000);
}

// Joins the parts of the rows that are cut.  Each block lists them (the shares whose
// entry says that the row that starts there goes on) and takes every so many'th
// piece of 64 or more columns of their 8 heads, more of them the fewer rows there are;
// its threads take 4 columns of every so many'th part, with a running maximum and
// sum, and add up through shared memory.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const DecodeAttnArgs a) {
  __shared__ int4 s_head[kShares];
  __shared__ int s_row[kShares], s_warp[kJoinThreads / 32];
  __shared__ float4 s_o[kJoinThreads];
  __shared__ float2 s_ml[kJoinThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  static_assert(kShares <= kJoinThreads, "a thread per entry");
  int rows = 0;
  {
    const int4 head = tid < kShares ? a.head[tid] : make_int4(0, 0, 0, 0);
    const bool cut = head.x > 1;
    const uint32_t mask = __ballot_sync(0xffffffffu, cut);
    if (lane == 0) s_warp[warp] = __popc(mask);
    __syncthreads();
    // lane w: the entries of warp w, those up to it, all
    int upto = lane < kJoinThreads / 32 ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < kJoinThreads / 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    rows = __shfl_sync(0xffffffffu, upto, kJoinThreads / 32 - 1);
    const int before = __shfl_sync(0xffffffffu, upto, max(warp - 1, 0));
    if (cut) {
      const int at = (warp ? before : 0) + __popc(mask & ((1u << lane) - 1));
      s_row[at] = tid;
      s_head[at] = head;
    }
    __syncthreads();
  }
  // columns of a piece: a power of two that gives every block a piece if it can
  constexpr int kLeast = 64, kMost = kHeads * D, kU = 8;
  int wide = kLeast;
  while (wide < kMost && rows * (kHeads * D / wide) > static_cast<int>(gridDim.x)) wide *= 2;
  const int pieces = kHeads * D / wide, lanes = wide / 4, groups = kJoinThreads / lanes;
  const int grp = tid / lanes;
  for (int piece = blockIdx.x; piece < rows * pieces; piece += static_cast<int>(gridDim.x)) {
    const int share = s_row[piece / pieces], col = piece % pieces * wide + 4 * (tid % lanes);
    const int hd = col / D, d = col % D;
    const int4 head = s_head[piece / pieces];
    float M = -INFINITY, L = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (hd < head.w)
      for (int i0 = grp; i0 < head.x; i0 += kU * groups) {
        float4 x[kU];
        float2 ml[kU];
#pragma unroll
        for (int j = 0; j < kU; ++j) {
          const int i = i0 + j * groups;
          ml[j] = make_float2(-INFINITY, 0.0f);
          x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (i < head.x) {
            const float *p = a.part + (static_cast<long long>(i == 0 ? head.y : 2 * (share + i)) * kHeads + hd) * (D + 4);
            ml[j] = *reinterpret_cast<const float2 *>(p + D);
            x[j] = *reinterpret_cast<const float4 *>(p + d);
          }
        }
#pragma unroll
        for (int j = 0; j < kU; ++j) {
          if (i0 + j * groups >= head.x) break;
          const float to = fmaxf(M, ml[j].x);
          const float f = M == to ? 1.0f : fast_exp2(M - to), w = ml[j].x == to ? 1.0f : fast_exp2(ml[j].x - to);
          M = to;
          L = L * f + w * ml[j].y;
          v.x = v.x * f + w * x[j].x;
          v.y = v.y * f + w * x[j].y;
          v.z = v.z * f + w * x[j].z;
          v.w = v.w * f + w * x[j].w;
        }
      }
    s_o[tid] = v;
    s_ml[tid] = make_float2(M, L);
    __syncthreads();
    // four groups' sums into one until one is left
    for (int left = groups; left > 1; left = (left + 3) / 4) {
      const int next = (left + 3) / 4;
      if (grp < next) {
        for (int w = grp + next; w < left; w += next) {
          const int at = w * lanes + tid % lanes;
          const float2 ml = s_ml[at];
          const float4 y = s_o[at];
          const float to = fmaxf(M, ml.x);
          const float f = M == to ? 1.0f : fast_exp2(M - to), u = ml.x == to ? 1.0f : fast_exp2(ml.x - to);
          M = to;
          L = L * f + u * ml.y;
          v.x = v.x * f + u * y.x;
          v.y = v.y * f + u * y.y;
          v.z = v.z * f + u * y.z;
          v.w = v.w * f + u * y.w;
        }
        if (next > 1) {
          s_o[tid] = v;
          s_ml[tid] = make_float2(M, L);
        }
      }
      __syncthreads();
    }
    if (grp == 0 && hd < head.w) {
      const float inv = M == -INFINITY ? 0.0f : 1.0f / L;
      *reinterpret_cast<uint2 *>(a.out + (static_cast<long long>(head.z) + hd) * D + d) =
          make_uint2(bf16x2_bits(v.x * inv, v.y * inv), bf16x2_bits(v.z * inv, v.w * inv));
    }
    __syncthreads();
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
  const cudaError_t e = launch_attn(attn_decode_kernel<D>, dim3(kCtas), kThreadsD, Page<D>::kTotal, st, tm, a);
  if (e != cudaSuccess) return e;
  return launch_attn(attn_join_kernel<D>, dim3(3 * kCtas), kJoinThreads, 0, st, a);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_attention_decode_workspace(int n_seq, int table_width, int n_q_heads,
                                              int n_kv_heads, int head_dim, size_t *bytes) {
  if (!bytes || n_seq < 0 || table_width < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0)
    return MOE_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || n_q_heads > 4096 || table_width > (1 << 25)) return MOE_ERR_UNSUPPORTED;
  *bytes = n_seq == 0 ? 0 : kShares * sizeof(int4) + 2 * kShares * sizeof(float) * kHeads * (head_dim + 4);
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
  if (n_pages < 0 || !(scale > 0.0f) || scale > kMostScale || q_stride < static_cast<long long>(n_q_heads) * head_dim)
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
  a.scale = scale * kLog2e;
  a.waits = attn_waits();
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
