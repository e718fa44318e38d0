// attn_prefill.cu -- causal attention of packed prompts, several query heads on
// one key/value head (moe_attention_prefill in include/moe.h), on the tcgen05
// tensor cores:
//     o_i = sum_j softmax_j(scale q_i . k_j) v_j   over keys j <= i + (keys - queries)
//
// Work split.  Query heads that share a key/value head are rows of one tile: row
// r of a CTA is token r / G, head r % G of the group of G heads, so that a short
// prompt fills tiles and the causal edge costs few masked tiles.  A cluster of
// two CTAs multiplies 2 x 128 rows with one stream of keys and values on the
// two-CTA MMA: each CTA stages half of the keys' rows and half of the values'
// columns, which halves the traffic from L2 and into shared memory (one CTA with
// 128 rows of 256 columns would move 156 bytes a cycle through a shared memory
// that has 128).
//
// Per tile of 128 keys, S and P double-buffered in TMEM (P, bf16, over S):
//     S = Q K^T (M 256, N 128),  P = exp2(c S - c m),  O += P V (M 256, N D)
// The tensor cores run S of the next tile while P is made.  The running maximum m
// moves only when a row's maximum has grown by 2^8: P then stays below 2^8, fp32
// sums lose nothing, and O is rarely scaled again.  P is rounded to bf16 (2^-8 of
// each weight, as large as the result's own rounding; an output's rms error grows
// by sqrt 2); the sum of the softmax is taken before that, in fp32.
//
// A key or value row that some of the tile's queries must not see is masked in
// the scores; but 0 x NaN is NaN, so in the tiles at the causal edge (and at a
// sequence's end) values that are not finite are taken out of V in shared memory,
// and the queries that do see them are set to NaN in the end.
//
// Roles (320 threads): warp 0 TMA copies; warp 1 the MMAs (CTA 0), or telling CTA 0
// that P is there (CTA 1); warps 2-9 the softmax, a warp per 16 rows, so that a row
// lies in one quad and its maximum takes two shuffles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/moe.h"
#include "attn_common.cuh"

namespace moe {

namespace {

constexpr int kThreadsA = 320;
constexpr int kKeys = 128;  // keys per tile
constexpr int kCtlBytes = 3072;
constexpr uint32_t kTmemCols = 512;
constexpr float kLate = 8.0f;  // log2 of how far a row's maximum may grow before m follows

template <int D>
struct Plan {
  static constexpr int kSlot = 64 * D * 2;  // a CTA's half of a tile of keys or of values
  static constexpr int kSlots = D == 256 ? 5 : 10;
  static constexpr int kQ = 128 * D * 2;
  static constexpr int kTotal = kCtlBytes + kQ + kSlots * kSlot;
  static constexpr uint32_t O = 0, S = D;  // TMEM columns: O, then two of S
  static_assert(kTotal <= 227 * 1024, "shared memory");
};

struct PrefillArgs {
  __nv_bfloat16 *out;
  const int *offsets, *k_offsets;
  long long n_q, n_k;
  int n_seq, Hq, Hk, group, tokens;  // tokens: of a CTA's tile
  float scale;                       // times log2(e)
  int *status;
};

struct Item {
  int q0, lq;    // first query and queries of the sequence
  int k0, lk;    // first key and keys
  int t0, head;  // first query of the cluster's tile (in the sequence), key/value head
  int valid;
};

struct Ctl {
  uint64_t full[10], empty[10], vloc[10];
  uint64_t q_full, s_full[2], p_full[2], p_loc[2], pv_done, drain;
  uint32_t tmem, sink;
  int abort_flag;
  Item item;
  float sum[128];
  uint32_t bad[128];  // two columns per word: first key (from the first masked tile on) that is not finite
};
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

// operand whose N index is contiguous (see the same layout in decay_chunk.cu)
__device__ __forceinline__ uint64_t sdesc_cols(uint32_t saddr, uint32_t lbo) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lbo >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kTransposeB = 1u << 16;

// two-CTA MMA with the A operand in TMEM
__device__ __forceinline__ void mma2_ts_bf16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                                 int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 16 lanes x 64 fp32 columns: lane l of the warp has, for each 8 columns n,
// v[4 n], v[4 n + 1] = row l / 4, columns 8 n + 2 (l % 4), + 1, and v[4 n + 2],
// v[4 n + 3] = row l / 4 + 8
__device__ __forceinline__ void ld_16x64(uint32_t ta, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(ta)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void st_16x64(uint32_t ta, const float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x8.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(ta)
      : "memory");
}
// 16 lanes x 32 columns of pairs: lane l has rows l / 4 (even registers) and
// l / 4 + 8 (odd) of column l % 4 of each group of four
__device__ __forceinline__ void st_pairs_16x32(uint32_t ta, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(ta)
      : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void fail(const PrefillArgs &a, volatile int *abort_flag, int site) {
  *abort_flag = 1;
  report_error(a.status, MOE_ERR_DEVICE_TIMEOUT, KID_ATTN_PREFILL * 100 + site);
}
// A warp's wait for phase `parity`: false in every lane when the CTA aborted or
// the polls, each of which sleeps in the barrier for a while, ran out.
constexpr int kPolls = 1 << 21;
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < kPolls; ++i) {
    if (mbar_try_wait_sleep(bar, parity, 2000u)) return true;
    if (abort_flag && *abort_flag) return false;
  }
  return false;
}
__device__ __forceinline__ bool warp_wait(const PrefillArgs &a, uint32_t bar, uint32_t parity,
                                          volatile int *abort_flag, int site) {
  if (__all_sync(0xffffffffu, poll(bar, parity, abort_flag))) return true;
  if ((threadIdx.x & 31) == 0) fail(a, abort_flag, site);
  return false;
}

// The n-th tile of the call (one warp): sequences in order, in a sequence the
// last tile, which sees the most keys, first.
__device__ __forceinline__ Item find_item(const PrefillArgs &a, long long n) {
  const int lane = threadIdx.x & 31, per = 2 * a.tokens;
  Item it = {};
  it.head = static_cast<int>(n % a.Hk);
  long long left = n / a.Hk;
  for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
    const int i = i0 + lane;
    int lo = 0, hi = 0;
    if (i < a.n_seq) seq_rows(a.offsets, a.n_seq, a.n_q, i, lo, hi);
    const int tiles = (hi - lo + per - 1) / per;
    long long upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, upto > left);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const long long back = upto - 1 - left;  // tiles behind it in the sequence
      it.valid = 1;
      it.q0 = __shfl_sync(0xffffffffu, lo, src);
      it.lq = __shfl_sync(0xffffffffu, hi, src) - it.q0;
      it.t0 = __shfl_sync(0xffffffffu, static_cast<int>(back), src) * per;
      seq_rows(a.k_offsets, a.n_seq, a.n_k, i0 + src, it.k0, it.lk);
      it.lk -= it.k0;
      return it;
    }
    left -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return it;
}

// Values of a masked tile that are not finite become zeros in this CTA's half of
// V (blocks of [128 keys][64 columns], 128-byte swizzle), thread e of 256; the
// first such key of each column is noted in both CTAs.
template <int D>
__device__ __noinline__ void take_out(Ctl &ctl, uint32_t v, int e, int rank, int key0, int lk, int base) {
  constexpr int kPer = D / 128 * 128 * 8 / 256;  // 16-byte pieces per thread
  const int r = e & 127, part = e >> 7;
  const uint32_t row = v + (D == 256 ? part * 16384 : 0) + r * 128;
  for (int i = 0; i < kPer; ++i) {
    const int piece = ((D == 256 ? i : part * 4 + i) ^ (r & 7));
    uint32_t w[4];
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(row + piece * 16)
                 : "memory");
    bool hit = false;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      hit = hit || (w[x] & 0x7f80u) == 0x7f80u || (w[x] & 0x7f800000u) == 0x7f800000u;
    if (!hit) continue;
    const int c0 = rank * (D / 2) + (D == 256 ? part * 64 : 0) + (piece ^ (r & 7)) * 8;
    for (int x = 0; x < 8; ++x) {
      const uint32_t half = 0xffffu << (16 * (x & 1));
      if ((w[x >> 1] & half & 0x7f807f80u) != (half & 0x7f807f80u)) continue;
      w[x >> 1] &= ~half;
      if (key0 + r >= lk) continue;  // (another sequence's: nobody sees it)
      const uint32_t mark = static_cast<uint32_t>(key0 + r - base);
      const uint32_t at = smem_u32(&ctl.bad[(c0 + x) >> 1]);
      for (uint32_t to = 0; to < 2; ++to) {
        const uint32_t p = cluster_map(at, to);
        uint32_t old;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(old) : "r"(p) : "memory");
        for (int tries = 0; tries < 1 << 16; ++tries) {
          const uint32_t now = (old >> (16 * (x & 1))) & 0xffffu;
          if (now <= mark) break;
          const uint32_t want = (old & ~half) | mark << (16 * (x & 1));
          uint32_t got;
          asm volatile("atom.shared::cluster.cas.b32 %0, [%1], %2, %3;"
                       : "=r"(got)
                       : "r"(p), "r"(old), "r"(want)
                       : "memory");
          if (got == old) break;
          old = got;
        }
      }
    }
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + piece * 16), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
  }
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  fence_proxy_async_smem();
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreadsA, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const PrefillArgs a) {
  using P = Plan<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl &ctl = *reinterpret_cast<Ctl *>(smem);
  volatile int *abort_flag = &ctl.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const uint32_t sQ = smem_u32(smem) + kCtlBytes, ring = sQ + P::kQ;
  constexpr uint16_t kBoth = 3;

  pdl_wait();
  if (warp == 0) {
    const Item it = find_item(a, blockIdx.x >> 1);
    if (lane == 0) ctl.item = it;
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < P::kSlots; ++s) {
      mbar_init(smem_u32(&ctl.full[s]), 1);
      mbar_init(smem_u32(&ctl.empty[s]), 1);
      mbar_init(smem_u32(&ctl.vloc[s]), 1);
    }
    mbar_init(smem_u32(&ctl.q_full), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctl.s_full[b]), 1);
      mbar_init(smem_u32(&ctl.p_full[b]), 8);
      mbar_init(smem_u32(&ctl.p_loc[b]), 8);
    }
    mbar_init(smem_u32(&ctl.pv_done), 1);
    mbar_init(smem_u32(&ctl.drain), 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  for (int i = static_cast<int>(threadIdx.x); i < 128; i += kThreadsA) ctl.bad[i] = 0xffffffffu;
  __syncthreads();
  const Item it = ctl.item;
  // (the whole cluster leaves; a misplaced shared memory, which the attribute
  // above excludes, would break the swizzle)
  if (!it.valid || (smem_u32(smem) & 1023u) != 0) {
    if (it.valid && threadIdx.x == 0) report_error(a.status, MOE_ERR_DEVICE_BOUNDS, KID_ATTN_PREFILL * 100 + SITE_INDEX);
    pdl_launch_dependents();
    return;
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(&ctl.tmem), kTmemCols);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist
  tc_fence_after();
  pdl_launch_dependents();
  // (all 512 columns are this CTA's: their addresses start at 0)

  const int shift = it.lk - it.lq, per = 2 * a.tokens;
  const int t_end = min(it.t0 + per, it.lq);           // the cluster's queries end here
  const int seen = max(0, t_end + shift);              // keys that its last query sees
  const int nk = (seen + kKeys - 1) / kKeys;
  const int jm = max(0, it.t0 + shift + 1) / kKeys;    // first tile that hides keys from a query
  const int mine = it.t0 + rank * a.tokens;            // this CTA's first query

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (lane == 0 && nk > 0) {
      const uint64_t pol = policy_evict_last();
      const uint32_t q0 = cluster_map(smem_u32(&ctl.q_full), 0);
      if (rank == 0) mbar_arrive_expect_tx(smem_u32(&ctl.q_full), 2 * a.tokens * a.group * D * 2);
      for (int b = 0; b < D / 64; ++b)
        tma_load_3d_pair(sQ + b * 16384, &tmQ, q0, 64 * b, it.head * a.group, it.q0 + mine);
      int r = 0;
      auto load = [&](bool values, int j) {
        const int s = r % P::kSlots;
        const uint32_t fb = smem_u32(&ctl.full[s]), dst = ring + s * P::kSlot;
        if (!poll(smem_u32(&ctl.empty[s]), ((r / P::kSlots) & 1) ^ 1, abort_flag)) {
          fail(a, abort_flag, SITE_PRODUCER_EMPTY);
          return false;
        }
        if (!values) {
          if (rank == 0) mbar_arrive_expect_tx(fb, 2 * P::kSlot);
          const uint32_t to = cluster_map(fb, 0);
          for (int b = 0; b < D / 64; ++b)
            tma_load_2d_pair(dst + b * 8192, &tmK, to, it.head * D + 64 * b, it.k0 + j * kKeys + rank * 64, pol);
        } else {
          uint32_t to = cluster_map(fb, 0);
          if (j >= jm) {  // the softmax's warps see to these first: their copy is this CTA's matter
            if (rank == 0) mbar_arrive(fb);
            mbar_arrive_expect_tx(smem_u32(&ctl.vloc[s]), P::kSlot);
            to = cluster_map(smem_u32(&ctl.vloc[s]), rank);
          } else if (rank == 0) {
            mbar_arrive_expect_tx(fb, 2 * P::kSlot);
          }
          for (int b = 0; b < D / 128; ++b)
            tma_load_2d_pair(dst + b * 16384, &tmV, to, it.head * D + rank * (D / 2) + 64 * b, it.k0 + j * kKeys, pol);
        }
        ++r;
        return true;
      };
      bool ok = load(false, 0);
      for (int j = 0; ok && j < nk; ++j) {
        if (j + 1 < nk) ok = load(false, j + 1);
        if (ok) ok = load(true, j);
      }
      // the commits of the last slots arrive here too: none may land after the
      // CTA has ended
      for (int i = 0; ok && i < P::kSlots; ++i, ++r)
        if (r >= P::kSlots && !poll(smem_u32(&ctl.empty[r % P::kSlots]), ((r / P::kSlots) & 1) ^ 1, abort_flag)) {
          fail(a, abort_flag, SITE_DRAIN);
          ok = false;
        }
    }
  } else if (warp == 1) {
    if (rank == 0 && nk > 0) {
      // ------------------------------------------------------------ MMAs
      // (the whole warp runs the loop, so that descriptors stay in uniform
      // registers; one lane issues)
      constexpr uint32_t id_s = idesc_make(256, kKeys, 1), id_o = idesc_make(256, D, 1) | kTransposeB;
      const bool one = elect_one();
      const uint64_t dq = sdesc_sw128(sQ), dk = sdesc_sw128(ring), dv = sdesc_cols(ring, 16384);
      int r = 0;
      bool ok = warp_wait(a, smem_u32(&ctl.q_full), 0, abort_flag, SITE_MMA_FULL);
      auto scores = [&](int j) {
        const int s = r % P::kSlots;
        if (!warp_wait(a, smem_u32(&ctl.full[s]), (r / P::kSlots) & 1, abort_flag, SITE_MMA_FULL)) return false;
        tc_fence_after();
        if (one) {
          const uint64_t k = dk + s * (P::kSlot >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma2_bf16(P::S + (j & 1) * kKeys, dq + (((kk >> 2) * 16384 + 32 * (kk & 3)) >> 4),
                      k + (((kk >> 2) * 8192 + 32 * (kk & 3)) >> 4), id_s, kk > 0 ? 1u : 0u);
          tc_commit2_mc(smem_u32(&ctl.s_full[j & 1]), kBoth);
          tc_commit2_mc(smem_u32(&ctl.empty[s]), kBoth);
        }
        ++r;
        return true;
      };
      auto output = [&](int j) {
        const int s = r % P::kSlots;
        if (!warp_wait(a, smem_u32(&ctl.full[s]), (r / P::kSlots) & 1, abort_flag, SITE_MMA_FULL) ||
            !warp_wait(a, smem_u32(&ctl.p_full[j & 1]), (j >> 1) & 1, abort_flag, SITE_STAGE))
          return false;
        tc_fence_after();
        if (one) {
          const uint64_t v = dv + s * (P::kSlot >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma2_ts_bf16(P::O, P::S + (j & 1) * kKeys + 8 * kk, v + kk * (2048 >> 4), id_o, (j | kk) != 0 ? 1u : 0u);
          tc_commit2_mc(smem_u32(&ctl.pv_done), kBoth);
          tc_commit2_mc(smem_u32(&ctl.empty[s]), kBoth);
        }
        ++r;
        return true;
      };
      if (ok) ok = scores(0);
      for (int j = 0; ok && j < nk; ++j) {
        if (j + 1 < nk) ok = scores(j + 1);
        if (ok) ok = output(j);
      }
      if (!ok) {  // the MMAs issued so far end before TMEM or shared memory go away
        if (one) tc_commit2(smem_u32(&ctl.drain));
        if (!poll(smem_u32(&ctl.drain), 0, nullptr) && lane == 0) fail(a, abort_flag, SITE_DRAIN);
      }
    } else if (rank == 1) {
      // ------------------------------------------------------------ P is there
      for (int j = 0; j < nk; ++j) {
        if (!warp_wait(a, smem_u32(&ctl.p_loc[j & 1]), (j >> 1) & 1, abort_flag, SITE_STAGE)) break;
        const uint32_t to = cluster_map(smem_u32(&ctl.p_full[j & 1]), 0);
        if (lane == 0) st_async_tx4(cluster_map(smem_u32(&ctl.sink), 0), 0u, to);  // (nothing reads the word)
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int wq = warp & 3, half = (warp - 2) >> 2, e = static_cast<int>(threadIdx.x) - 64;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32 + half * 16) << 16;
    // this thread's two rows: the last key each sees, -1 where it is no query
    int limit[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = wq * 32 + half * 16 + 8 * x + (lane >> 2), t = mine + row / a.group;
      limit[x] = row < a.tokens * a.group && t < it.lq ? min(t + shift, it.lk - 1) : -1;
    }
    const int own = max(0, mine + shift + 1) / kKeys;  // first tile masked for this CTA
    float m[2] = {-INFINITY, -INFINITY}, ref[2] = {0.0f, 0.0f}, l[2] = {0.0f, 0.0f};
    const float c = a.scale, late = kLate / c;
    uint32_t vphase = 0;
    bool ok = true;
    for (int j = 0; j < nk; ++j) {
      const uint32_t ts = P::S + (j & 1) * kKeys + lanes;
      ok = warp_wait(a, smem_u32(&ctl.s_full[j & 1]), (j >> 1) & 1, abort_flag, SITE_EPI_TMEM_FULL);
      if (!ok) break;
      tc_fence_after();
      float x[2][32];
      ld_16x64(ts, x[0]);
      ld_16x64(ts + 64, x[1]);
      if (j >= own) {
        const int key = j * kKeys + 2 * (lane & 3);
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (key + 64 * y + 8 * (i >> 2) + (i & 1) > limit[(i >> 1) & 1]) x[y][i] = -INFINITY;
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int i = 0; i < 32; ++i) top[(i >> 1) & 1] = fmaxf(top[(i >> 1) & 1], x[y][i]);
      bool grown = false;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        top[z] = fmaxf(top[z], __shfl_xor_sync(0xffffffffu, top[z], 1));
        top[z] = fmaxf(top[z], __shfl_xor_sync(0xffffffffu, top[z], 2));
        grown = grown || top[z] > m[z] + late;
      }
      if (__any_sync(0xffffffffu, grown)) {
        float f[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float to = top[z] > m[z] + late ? top[z] : m[z];
          f[z] = to == m[z] ? 1.0f : fast_exp2((m[z] - to) * c);
          m[z] = to;
          ref[z] = to == -INFINITY ? 0.0f : to * c;
          l[z] *= f[z];
        }
        if (j > 0) {  // O of the tiles before
          ok = warp_wait(a, smem_u32(&ctl.pv_done), (j - 1) & 1, abort_flag, SITE_STAGE);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 64) {
            float o[32];
            ld_16x64(P::O + lanes + d, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f[(i >> 1) & 1];
            st_16x64(P::O + lanes + d, o);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int z = i & 1;
          const float u = fast_exp2(fmaf(x[y][2 * i], c, -ref[z])), w = fast_exp2(fmaf(x[y][2 * i + 1], c, -ref[z]));
          l[z] += u + w;
          p[i] = bf16x2_bits(u, w);
        }
        st_pairs_16x32(ts + 32 * y, p);
      }
      wait_st();
      if (j >= jm) {
        const int rv = j + 1 < nk ? 2 * j + 2 : 2 * j + 1, s = rv % P::kSlots;  // V's place in the ring
        ok = warp_wait(a, smem_u32(&ctl.vloc[s]), (vphase >> s) & 1, abort_flag, SITE_MMA_FULL);
        if (!ok) break;
        vphase ^= 1u << s;
        take_out<D>(ctl, ring + s * P::kSlot, e, rank, j * kKeys, it.lk, jm * kKeys);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 1) {
          mbar_arrive(smem_u32(&ctl.p_loc[j & 1]));
        } else if (warp == 2) {
          mbar_arrive_expect_tx(smem_u32(&ctl.p_full[j & 1]), 4);  // the other CTA's word
        } else {
          mbar_arrive(smem_u32(&ctl.p_full[j & 1]));
        }
      }
    }
    // ------------------------------------------------------------ outputs
    if (ok && nk > 0) {
      ok = (nk < 2 || warp_wait(a, smem_u32(&ctl.pv_done), (nk - 2) & 1, abort_flag, SITE_EPI_TMEM_FULL)) &&
           warp_wait(a, smem_u32(&ctl.pv_done), (nk - 1) & 1, abort_flag, SITE_EPI_TMEM_FULL);
      tc_fence_after();
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        l[z] += __shfl_xor_sync(0xffffffffu, l[z], 1);
        l[z] += __shfl_xor_sync(0xffffffffu, l[z], 2);
        if ((lane & 3) == 0) ctl.sum[wq * 32 + half * 16 + 8 * z + (lane >> 2)] = l[z];
      }
    }
    // the two warps of a TMEM quarter take half of the columns each, a row per thread
    named_bar_sync(1 + wq, 64);
    const int row = wq * 32 + lane, t = mine + row / a.group;
    const bool valid = ok && row < a.tokens * a.group && t < it.lq;
    const int lim = t + shift;
    const float inv = nk > 0 && lim >= 0 ? 1.0f / ctl.sum[row] : 0.0f;
    __nv_bfloat16 *o = a.out + (static_cast<long long>(it.q0 + t) * a.Hq + it.head * a.group + row % a.group) * D;
    const int mark = lim - jm * kKeys;
#pragma unroll 1
    for (int d = half * (D / 2); ok && d < (half + 1) * (D / 2); d += 32) {
      float v[32];
      if (nk > 0) {
        tmem_ld32_sync(P::O + (static_cast<uint32_t>(wq * 32) << 16) + d, v);
      }
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t bad = ctl.bad[d / 2 + i];
        float x0 = nk > 0 && lim >= 0 ? v[2 * i] * inv : 0.0f, x1 = nk > 0 && lim >= 0 ? v[2 * i + 1] * inv : 0.0f;
        if (mark >= static_cast<int>(bad & 0xffffu)) x0 = __uint_as_float(0x7fffffffu);
        if (mark >= static_cast<int>(bad >> 16)) x1 = __uint_as_float(0x7fffffffu);
        w[i] = bf16x2_bits(x0, x1);
      }
      if (valid)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<uint4 *>(o + d + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no MMA of the pair is in flight, no arrival is pending
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(0, kTmemCols);
  if (*abort_flag)  // after an abort the copies in flight get time to land
    for (int i = 0; i < 200; ++i) __nanosleep(1000);
}

namespace {

struct PrefillDevice {
  int *status = nullptr;
  int rc = MOE_ERR_CUDA;
};

const PrefillDevice &prefill_device() {
  static PrefillDevice devs[64];
  static std::once_flag once[64];
  static const PrefillDevice none;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return none;
  std::call_once(once[dev], [dev] {
    PrefillDevice &d = devs[dev];
    d.status = noalloc_status_word();
    auto set = [](auto kern, int bytes) {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
    };
    if (d.status && set(attn_prefill_kernel<128>, Plan<128>::kTotal) && set(attn_prefill_kernel<256>, Plan<256>::kTotal))
      d.rc = MOE_OK;
  });
  return devs[dev];
}

template <int D>
cudaError_t launch_prefill(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                           const PrefillArgs &a, long long clusters, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters));
  cfg.blockDim = dim3(kThreadsA);
  cfg.dynamicSmemBytes = Plan<D>::kTotal;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, attn_prefill_kernel<D>, mq, mk, mv, a);
}

}  // namespace

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
  const PrefillDevice &dev = prefill_device();
  if (dev.rc != MOE_OK) return dev.rc;
  PrefillArgs a = {};
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.offsets = offsets;
  a.k_offsets = k_offsets ? k_offsets : offsets;
  a.n_q = n_q;
  a.n_k = n_k;
  a.n_seq = n_seq;
  a.Hq = n_q_heads;
  a.Hk = n_kv_heads;
  a.group = n_q_heads / n_kv_heads;
  a.tokens = 128 / a.group;
  a.scale = scale * 1.4426950408889634f;
  a.status = dev.status;
  // tiles of the call, or as many as there can be
  const long long per = 2 * a.tokens;
  const long long tiles = offsets ? n_q / per + n_seq : n_seq * ((n_q / n_seq + per - 1) / per);
  const long long clusters = tiles * n_kv_heads;
  if (clusters > 0x3fffffffLL) return MOE_ERR_UNSUPPORTED;
  const uint64_t d = head_dim, hk = n_kv_heads;
  const uint64_t keys = n_k > 0 ? n_k : 1;  // (no key is read where there is none)
  const void *kb = n_k > 0 ? k : q, *vb = n_k > 0 ? v : q;
  CUtensorMap mq, mk, mv;
  if (!encode_map_3d(&mq, q, d, n_q_heads, n_q, 2 * d, 2 * q_stride, 64, a.group, a.tokens) ||
      !encode_map_2d(&mk, kb, 2, keys, hk * d, 64, 64, true, 2 * k_stride) ||
      !encode_map_2d(&mv, vb, 2, keys, hk * d, 64, 128, true, 2 * v_stride))
    return MOE_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = head_dim == 128 ? launch_prefill<128>(mq, mk, mv, a, clusters, st)
                                        : launch_prefill<256>(mq, mk, mv, a, clusters, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
