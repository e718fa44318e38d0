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
//   * D = 256: O takes half of TMEM.  All eight softmax warps make each tile's P,
//     16 rows each (a row lies in a quad, its maximum takes two shuffles); the
//     products of a tile, 2,048 cycles, hide that.
//   * D = 128: a tile's products take 1,024 cycles, less than the softmax of one
//     tile from end to end.  Even and odd tiles are therefore two streams, each with
//     an O, a maximum and a sum of its own, four warps with a row per thread for
//     either; they are joined at a row's end.
//
// Schedule.  As many clusters as fit stay; one warp per CTA looks up the next tile of
// rows while the others work.  Tiles are numbered by falling number of key tiles over
// all sequences, and cluster c of P takes the numbers c, 2P - 1 - c, 2P + c, ..: the
// largest go first and the sums stay even.  The next tile's copies and scores run
// during the outputs of the one before.  Where tiles are few, or some see many more
// keys than others, their keys are cut into parts: outputs without the division,
// maxima and sums go to the workspace, and a second kernel joins them in order.
//
// A key or value row that some of the tile's queries must not see is masked in
// the scores; but 0 x NaN is NaN, so in the tiles at the causal edge (and at a
// sequence's end) values that are not finite are taken out of V in shared memory,
// and infinity, its negative, or both for a NaN, are added to the outputs of the
// queries that do see them.
//
// Measured, back to back in a graph (in brackets: calls one after another, under the
// power limit): 4,096 tokens of 16 heads of 256 on 2 in 83 us, 1.66 PFLOP/s (90, 1.53),
// tensor pipes busy 73 % of the cycles; the rest goes at the changes of tile, about 4,500
// cycles each.  8,192 tokens behind 24,576 in 1.83 to 1.87 ms, 2.1 PFLOP/s (2.12, 1.82).
// 2 x 2,048 tokens of 32 heads of 128 on 8 in 85 us, 0.81 PFLOP/s, tensor pipes 35 %: the
// handover between softmax and products, about 1,700 cycles a tile.
//
// Roles (352 threads): warp 0 TMA copies; warp 1 the MMAs (CTA 0); warps 2-9 the
// softmax and the outputs, each telling CTA 0 that its P is there (through a warp of
// CTA 1 that gathered these, 2 x 2,048 tokens of 128 took 87.4 us in place of 84.2);
// warp 10 the schedule.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/moe.h"
#include "attn_common.cuh"

namespace moe {

namespace {

constexpr int kThreadsA = 352;
constexpr int kKeys = 128;  // keys per tile
constexpr int kItems = 2;   // tiles of rows looked up ahead
constexpr int kReaders = 10;  // warps that read an item
constexpr uint32_t kTmemCols = 512;
constexpr float kLate = 8.0f;  // log2 of how far a row's maximum may grow before m follows
// A weight is exp2(c x - c m) by one fused sum, in which c m is rounded: off by up to
// 2^-24 of itself, the same for all of a row's weights, but past 2^30 a weight of 1 then
// leaves fp32, and two streams or parts are weighed against each other by it.  Past this
// size m is therefore taken off x first, which costs a sum per weight in rows that large.
constexpr float kFar = 1024.0f;

struct PrefillArgs {
  __nv_bfloat16 *out;
  const int *offsets, *k_offsets;
  long long n_q, n_k;
  int n_seq, Hq, Hk, group, tokens;  // tokens: of a CTA's tile
  uint32_t per_mul, per_shift;       // x / (2 tokens) = (x per_mul >> 32) >> per_shift, x < 2^31
  float scale;                       // times log2(e)
  int *status;
  AttnWaits waits;
  int parts, length;  // most parts of a tile's keys (1: none are cut), key tiles of a part
  float *part;        // (parts > 1) [parts][n_q][Hq][D]: outputs before the division
  float2 *stat;       // [parts][n_q][Hq]: maximum, sum
};

struct Item {
  int q0, lq;    // first query and queries of the sequence
  int k0, lk;    // first key and keys
  int t0, head;  // first query of the cluster's tile (in the sequence), key/value head
  int valid, part;
};

template <int D>
struct Ctl {
  uint64_t full[10], empty[10], vloc[10];
  uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done, o_full, drain;
  uint64_t it_full[kItems], it_empty[kItems];
  uint32_t tmem, sink;
  int abort_flag;
  Item item[kItems];
  // of three tiles of rows in turn, three columns per word: first key (from the first
  // masked tile on) whose value is infinity, and minus infinity, or in both a NaN
  uint32_t bad[3][2][(D + 2) / 3], hit[3];  // hit: whether there is one
  float2 stream[2][D == 128 ? 128 : 1];      // D = 128: maximum and sum of each stream's rows
};

template <int D>
struct Plan {
  static constexpr int kCtlBytes = D == 256 ? 3072 : 5120;
  static constexpr int kSlot = 64 * D * 2;  // a CTA's half of a tile of keys or of values
  static constexpr int kSlots = D == 256 ? 5 : 10;
  static constexpr int kQ = 128 * D * 2;
  static constexpr int kTotal = kCtlBytes + kQ + kSlots * kSlot;
  static constexpr int kStreams = D == 128 ? 2 : 1;
  static constexpr uint32_t O = 0, S = kStreams * D;  // TMEM columns: O of each stream, then two of S
  static constexpr int kMakers = kStreams == 2 ? 4 : 8;  // warps of a tile's P
  static_assert(kTotal <= 227 * 1024 && sizeof(Ctl<D>) <= kCtlBytes && S + 2 * kKeys <= kTmemCols, "room");
  static_assert(sizeof(Ctl<D>::bad) / 12 <= 256, "a thread of the softmax per word");
};

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
// 32 lanes x 16 or 32 columns, a lane per thread
__device__ __forceinline__ void st_32x16(uint32_t ta, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(ta)
      : "memory");
}
__device__ __forceinline__ void st_32x32(uint32_t ta, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(ta)
      : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 4 x 4 words of a quad's lanes turned: r[i] of lane q becomes r[q] of lane i
__device__ __forceinline__ void turn_quad(uint32_t (&r)[4]) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t t = __shfl_xor_sync(0xffffffffu, odd ? r[i] : r[i + 1], 1);
    if (odd) r[i] = t; else r[i + 1] = t;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t t = __shfl_xor_sync(0xffffffffu, high ? r[i] : r[i + 2], 2);
    if (high) r[i] = t; else r[i + 2] = t;
  }
}

__device__ __forceinline__ void fail(const PrefillArgs &a, volatile int *abort_flag, int site) {
  *abort_flag = 1;
  report_error(a.status, MOE_ERR_DEVICE_TIMEOUT, KID_ATTN_PREFILL * 100 + site);
}
// A warp's wait for phase `parity`: false in every lane when the CTA aborted or
// the polls, each of which sleeps in the barrier for a while, ran out.
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, const volatile int *abort_flag, int polls) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < polls; ++i) {
    if (mbar_try_wait_sleep(bar, parity, 2000u)) return true;
    if (abort_flag && *abort_flag) return false;
  }
  return false;
}
__device__ __forceinline__ bool warp_wait(const PrefillArgs &a, uint32_t bar, uint32_t parity,
                                          volatile int *abort_flag, int site, int times = 1) {
  if (__all_sync(0xffffffffu, poll(bar, parity, abort_flag, times * a.waits.polls))) return true;
  if ((threadIdx.x & 31) == 0) fail(a, abort_flag, site);
  return false;
}

// The schedule (one warp): tiles of rows by falling number of key tiles; kCut: keys of
// some are cut into parts.  Past 32 sequences a tile is found by a search whose every
// step reads all offsets, so that many short ones cost the square of their number: 64
// prompts of 64 tokens 31 us, 256 244 us, 1,024 3.8 ms (16 heads of 256 on 2).
template <bool kCut>
struct Schedule {
  const PrefillArgs &a;
  int per;           // queries of a tile
  int lq, shift;     // (n_seq <= 32) this lane's sequence: queries, keys less queries
  bool alike;        // all sequences are of one length

  __device__ __forceinline__ Schedule(const PrefillArgs &args) : a(args), per(2 * args.tokens) {
    lq = shift = 0;
    alike = !a.offsets || a.n_seq == 1;
    if (a.n_seq <= 32 && (threadIdx.x & 31) < a.n_seq) lengths(threadIdx.x & 31, lq, shift);
  }
  __device__ __forceinline__ int tiles_of(int x) const {  // x / per
    return static_cast<int>(__umulhi(static_cast<uint32_t>(x), a.per_mul) >> a.per_shift);
  }
  __device__ __forceinline__ void lengths(int i, int &queries, int &ahead) const {
    int q0, q1, k0, k1;
    seq_rows(a.offsets, a.n_seq, a.n_q, i, q0, q1);
    seq_rows(a.k_offsets, a.n_seq, a.n_k, i, k0, k1);
    queries = q1 - q0;
    ahead = (k1 - k0) - queries;
  }
  // tiles of a sequence with at least c key tiles: the last query of tile b, at
  // min((b + 1) per, queries) - 1, sees more than 128 (c - 1) keys
  __device__ __forceinline__ int least(int queries, int ahead, int c) const {
    const int tiles = tiles_of(queries + per - 1);
    const long long from = 128LL * (c - 1) - ahead;
    if (c <= 0 || from < 0) return tiles;
    return from >= queries ? 0 : tiles - tiles_of(static_cast<int>(from));
  }
  // that of the sequence i0 + lane
  __device__ __forceinline__ int mine(int i0, int c) const {
    const int i = i0 + static_cast<int>(threadIdx.x & 31);
    if (a.n_seq <= 32) return least(lq, shift, c);
    if (i >= a.n_seq) return 0;
    int queries, ahead;
    lengths(i, queries, ahead);
    return least(queries, ahead, c);
  }
  __device__ __forceinline__ long long all(int c) const {
    if (alike && c == 0) {
      int queries, ahead;
      lengths(0, queries, ahead);
      return static_cast<long long>(tiles_of(queries + per - 1)) * a.n_seq;
    }
    long long sum = 0;
    for (int i0 = 0; i0 < a.n_seq; i0 += 32) sum += __reduce_add_sync(0xffffffffu, mine(i0, c));
    return sum;
  }
  // tiles that have a p-th part: the first so many, as they are in falling order
  __device__ __forceinline__ int from(int p) const { return p == 0 ? 0 : p * a.length + 1; }
  // Parts in their order: all second ones, all third ones, .., then the first, which
  // alone may be short in great number; lane i has those up to the i-th kind.
  __device__ __forceinline__ int kind(int i) const { return i + 1 < a.parts ? i + 1 : 0; }
  __device__ __forceinline__ long long parts_upto(long long &mine_of) const {
    const int lane = threadIdx.x & 31;
    mine_of = 0;
    if (a.n_seq <= 32) {
      for (int i = 0; i < a.n_seq; ++i) {
        const int queries = __shfl_sync(0xffffffffu, lq, i), ahead = __shfl_sync(0xffffffffu, shift, i);
        if (lane < a.parts) mine_of += least(queries, ahead, from(kind(lane)));
      }
    } else {
      for (int i = 0; i < a.parts; ++i) {
        const long long tiles = all(from(kind(i)));
        if (lane == i) mine_of = tiles;
      }
    }
    long long upto = mine_of;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    return upto;
  }
  __device__ __forceinline__ long long total() const {
    if (!kCut) return all(0) * a.Hk;
    long long own;
    return __shfl_sync(0xffffffffu, parts_upto(own), 31) * a.Hk;
  }
  // the n-th part of a tile; n < total()
  __device__ __forceinline__ Item find(long long n) const {
    const int head = static_cast<int>(n % a.Hk);
    long long left = n / a.Hk;
    int part = 0;
    if (kCut) {
      long long own;
      const long long upto = parts_upto(own);
      const int i = __ffs(__ballot_sync(0xffffffffu, upto > left)) - 1;
      left -= __shfl_sync(0xffffffffu, upto - own, i);
      part = kind(i);
    }
    return tile(left, head, part);
  }
  // the left-th tile
  __device__ __forceinline__ Item tile(long long left, int head, int part) const {
    const int lane = threadIdx.x & 31;
    Item it = {};
    it.valid = 1;
    it.head = head;
    it.part = part;
    if (alike) {  // the last tiles of all sequences, then those before
      const int back = static_cast<int>(left / a.n_seq), i = static_cast<int>(left % a.n_seq);
      int k1;
      seq_rows(a.offsets, a.n_seq, a.n_q, i, it.q0, it.lq);
      seq_rows(a.k_offsets, a.n_seq, a.n_k, i, it.k0, k1);
      it.lq -= it.q0;
      it.lk = k1 - it.k0;
      it.t0 = (tiles_of(it.lq + per - 1) - 1 - back) * per;
      return it;
    }
    int lo = 0, hi = static_cast<int>((a.n_k + kKeys - 1) / kKeys) + 1;  // all(lo) > left >= all(hi)
    long long behind = 0;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      const long long m = all(mid);
      if (m > left) {
        lo = mid;
      } else {
        hi = mid;
        behind = m;
      }
    }
    left -= behind;
    for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
      const int from = mine(i0, lo), count = from - mine(i0, hi);
      int upto = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, upto > left);
      if (hit) {
        const int src = __ffs(hit) - 1, i = i0 + src;
        const int nth = static_cast<int>(left) - __shfl_sync(0xffffffffu, upto - count, src);
        const int first = __shfl_sync(0xffffffffu, from, src);  // tiles from its level on
        int k1;
        seq_rows(a.offsets, a.n_seq, a.n_q, i, it.q0, it.lq);
        seq_rows(a.k_offsets, a.n_seq, a.n_k, i, it.k0, k1);
        it.lq -= it.q0;
        it.lk = k1 - it.k0;
        it.t0 = (tiles_of(it.lq + per - 1) - first + nth) * per;
        return it;
      }
      left -= __shfl_sync(0xffffffffu, upto, 31);
    }
    it.valid = 0;  // (not reached)
    return it;
  }
};

// Values of a masked tile that are not finite become zeros in this CTA's half of
// V (blocks of [128 keys][64 columns], 128-byte swizzle), thread e of kN; the first
// such key of each column is noted in both CTAs.
template <int D, int kN>
struct Cleaner {
  static constexpr int kWords = (D + 2) / 3;
  static constexpr uint32_t kMark = 0x3ffu;
  static constexpr int kPer = D * 8 / kN;  // 16-byte pieces per thread, of one row
  static __device__ __forceinline__ uint32_t where(uint32_t v, int e, int i) {
    const int r = e & 127, at = (e >> 7) * kPer + i;  // piece of the row: block at / 8
    return v + (at >> 3) * 16384 + r * 128 + (((at & 7) ^ (r & 7)) << 4);
  }
  static __device__ __forceinline__ void clean(uint32_t bad, uint32_t flag, uint32_t v, int e, int rank, int key0,
                                               int lk, int base) {
    uint32_t top = 0;  // bit 15 or 31 of a sum: an exponent of ones
    uint32_t w[kPer][4];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                   : "r"(where(v, e, i))
                   : "memory");
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) top |= (w[i][x] & 0x7f807f80u) + 0x00800080u;
    if (top & 0x80008000u) take_out(bad, flag, v, e, rank, key0, lk, base);
  }
  static __device__ __noinline__ void take_out(uint32_t bad, uint32_t flag, uint32_t v, int e, int rank, int key0,
                                               int lk, int base) {
    const int key = key0 + (e & 127);
    for (int i = 0; i < kPer; ++i)
      for (int x = 0; x < 8; ++x) {
        const uint32_t at = where(v, e, i) + 2 * x;
        uint16_t bits;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(at) : "memory");
        if ((bits & 0x7f80u) != 0x7f80u) continue;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(0)) : "memory");
        if (key >= lk) continue;  // (another sequence's: nobody sees it)
        const int c = rank * (D / 2) + ((e >> 7) * kPer + i) * 8 + x;
        // (masked tiles are three at most)
        const uint32_t mark = static_cast<uint32_t>(key - base), shift = 10 * (c % 3);
        for (int y = 0; y < 4; ++y) {
          const uint32_t to = y & 1, minus = y >> 1;
          if ((bits & 0x7fu) == 0 && (bits >> 15) != minus) continue;
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_map(flag, to)), "r"(1u) : "memory");
          const uint32_t p = cluster_map(bad + (minus * kWords + c / 3) * 4, to);
          uint32_t old;
          asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(old) : "r"(p) : "memory");
          for (int tries = 0; tries < 1 << 16 && (old >> shift & kMark) > mark; ++tries) {
            const uint32_t want = (old & ~(kMark << shift)) | mark << shift;
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
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  // The marks' infinities into what a thread has stored of a row: its columns
  // 4 wide n + wide sub + 0 .. wide - 1; seen: of the keys from base on, the last that the row sees.
  template <typename T>
  static __device__ __forceinline__ void put_back(const uint32_t (&bad)[2][kWords], T *row, int seen, int sub) {
    constexpr int kWide = sizeof(T) == 2 ? 8 : 2;
#pragma unroll 1
    for (int i = 0; i < D / 4; ++i) {
      const int c = i / kWide * (4 * kWide) + kWide * sub + i % kWide;
      for (int y = 0; y < 2; ++y)
        if (seen >= static_cast<int>(bad[y][c / 3] >> 10 * (c % 3) & kMark))
          row[c] = static_cast<T>(static_cast<float>(row[c]) + (y ? -INFINITY : INFINITY));
    }
  }
};

// What the roles derive from an item
template <bool kCut>
struct Tile {
  int shift, mine;  // keys less queries, this CTA's first query
  int j0, nk, jm;   // first key tile of this part, how many, from which of them on some query must not see a key
  int parts;        // of the tile
  __device__ __forceinline__ Tile(const PrefillArgs &a, const Item &it, int rank) {
    shift = it.lk - it.lq;
    const int end = min(it.t0 + 2 * a.tokens, it.lq);
    nk = (max(0, end + shift) + kKeys - 1) / kKeys;
    j0 = 0;
    parts = 1;
    if (kCut && nk > a.length) {
      parts = (nk + a.length - 1) / a.length;
      j0 = it.part * a.length;
      nk = min(nk - j0, a.length);
    }
    jm = max(0, max(0, it.t0 + shift + 1) / kKeys - j0);
    mine = it.t0 + rank * a.tokens;
  }
};

}  // namespace

template <int D, bool kCut>
__global__ void __launch_bounds__(kThreadsA, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const PrefillArgs a) {
  using P = Plan<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl<D> &ctl = *reinterpret_cast<Ctl<D> *>(smem);
  volatile int *abort_flag = &ctl.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const uint32_t sQ = smem_u32(smem) + P::kCtlBytes, ring = sQ + P::kQ;
  constexpr uint16_t kBoth = 3;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P::kSlots; ++s) {
      mbar_init(smem_u32(&ctl.full[s]), 1);
      mbar_init(smem_u32(&ctl.empty[s]), 1);
      mbar_init(smem_u32(&ctl.vloc[s]), 1);
    }
    mbar_init(smem_u32(&ctl.q_full), 1);
    mbar_init(smem_u32(&ctl.q_empty), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctl.s_full[b]), 1);
      mbar_init(smem_u32(&ctl.p_full[b]), P::kMakers);
    }
    mbar_init(smem_u32(&ctl.pv_done), 1);
    mbar_init(smem_u32(&ctl.o_full), 1);
    mbar_init(smem_u32(&ctl.drain), 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(smem_u32(&ctl.it_full[i]), 1);
      mbar_init(smem_u32(&ctl.it_empty[i]), rank == 0 ? kReaders : kReaders - 1);  // (no MMAs in CTA 1)
    }
    ctl.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (threadIdx.x < 3) ctl.hit[threadIdx.x] = 0;
  for (int i = static_cast<int>(threadIdx.x); i < static_cast<int>(sizeof ctl.bad / 4); i += kThreadsA)
    (&ctl.bad[0][0][0])[i] = 0xffffffffu;
  // (a misplaced shared memory, which the attribute above excludes, would break the
  // swizzle)
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) report_error(a.status, MOE_ERR_DEVICE_BOUNDS, KID_ATTN_PREFILL * 100 + SITE_INDEX);
    pdl_wait();
    return;
  }
  // Rows of Q past the tile's last token, which no copy writes: zeros, so that their
  // scores, which the MMAs form all the same, never count as far or as grown.
  const int rows = a.tokens * a.group;
  for (int i = static_cast<int>(threadIdx.x); i < (128 - rows) * (D / 8); i += kThreadsA) {
    const uint32_t at = sQ + i / ((128 - rows) * 8) * 16384 + rows * 128 + i % ((128 - rows) * 8) * 16;
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
  }
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc2(smem_u32(&ctl.tmem), kTmemCols);
    tmem_relinquish2();
  }
  long long total = 0;
  if (warp == 10) {  // the first item, meanwhile
    pdl_wait();
    const Schedule<kCut> plan(a);
    total = plan.total();
    Item it = {};
    if ((blockIdx.x >> 1) < total) it = plan.find(blockIdx.x >> 1);
    if (lane == 0) ctl.item[0] = it;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist
  tc_fence_after();
  // Only now: a CTA of the next kernel may take TMEM columns before it waits for this
  // grid.  (All 512 columns are this CTA's: their addresses start at 0.)
  pdl_launch_dependents();
  pdl_wait();

  // the k-th item of this cluster, read by a warp; false: an abort or the end
  auto next_item = [&](int k, Item &it) {
    const int i = k % kItems;
    if (!warp_wait(a, smem_u32(&ctl.it_full[i]), (k / kItems) & 1, abort_flag, SITE_STAGE)) return false;
    it = ctl.item[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ctl.it_empty[i]));
    return it.valid != 0;
  };

  if (warp == 10) {
    // ------------------------------------------------------------ schedule
    const Schedule<kCut> plan(a);
    const long long clusters = gridDim.x >> 1, c = blockIdx.x >> 1;
    if (lane == 0) mbar_arrive(smem_u32(&ctl.it_full[0]));
    __syncwarp();
    if (c < total)
      for (int k = 1;; ++k) {
        const long long n = k & 1 ? (k + 1) * clusters - 1 - c : k * clusters + c;
        Item it = {};
        if (n < total) it = plan.find(n);
        // (the one wait that may be as long as a tile of rows, which over 2^28 keys is seconds)
        if (!warp_wait(a, smem_u32(&ctl.it_empty[k % kItems]), ((k / kItems) & 1) ^ 1, abort_flag, SITE_STAGE, 64)) break;
        if (lane == 0) {
          ctl.item[k % kItems] = it;
          mbar_arrive(smem_u32(&ctl.it_full[k % kItems]));
        }
        __syncwarp();
        if (!it.valid) break;
      }
  } else if (warp == 0) {
    // ------------------------------------------------------------ copies
    const uint64_t pol = policy_evict_last();
    int r = 0;  // uses of the ring
    bool ok = true;
    Item it;
    for (int k = 0, used = 0; ok && next_item(k, it); ++k) {
      const Tile<kCut> t(a, it, rank);
      if (t.nk == 0) continue;
      if (lane == 0) {
        // Q, once the scores of the tile before are made
        if (!poll(smem_u32(&ctl.q_empty), (used & 1) ^ 1, abort_flag, a.waits.polls)) {
          fail(a, abort_flag, SITE_PRODUCER_EMPTY);
          ok = false;
        }
        const uint32_t q0 = cluster_map(smem_u32(&ctl.q_full), 0);
        if (ok) {
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&ctl.q_full), 2 * a.tokens * a.group * D * 2);
          for (int b = 0; b < D / 64; ++b)
            tma_load_3d_pair(sQ + b * 16384, &tmQ, q0, 64 * b, it.head * a.group, it.q0 + t.mine);
        }
        auto load = [&](bool values, int j) {
          if (r >= a.waits.loads) return false;
          const int s = r % P::kSlots;
          const uint32_t fb = smem_u32(&ctl.full[s]), dst = ring + s * P::kSlot;
          if (!poll(smem_u32(&ctl.empty[s]), ((r / P::kSlots) & 1) ^ 1, abort_flag, a.waits.polls)) {
            fail(a, abort_flag, SITE_PRODUCER_EMPTY);
            return false;
          }
          if (!values) {
            if (rank == 0) mbar_arrive_expect_tx(fb, 2 * P::kSlot);
            const uint32_t to = cluster_map(fb, 0);
            for (int b = 0; b < D / 64; ++b)
              tma_load_2d_pair(dst + b * 8192, &tmK, to, it.head * D + 64 * b, it.k0 + (t.j0 + j) * kKeys + rank * 64, pol);
          } else {
            uint32_t to = cluster_map(fb, 0);
            if (j >= t.jm) {  // the softmax's warps see to these first: their copy is this CTA's matter
              if (rank == 0) mbar_arrive(fb);
              mbar_arrive_expect_tx(smem_u32(&ctl.vloc[s]), P::kSlot);
              to = cluster_map(smem_u32(&ctl.vloc[s]), rank);
            } else if (rank == 0) {
              mbar_arrive_expect_tx(fb, 2 * P::kSlot);
            }
            for (int b = 0; b < D / 128; ++b)
              tma_load_2d_pair(dst + b * 16384, &tmV, to, it.head * D + rank * (D / 2) + 64 * b, it.k0 + (t.j0 + j) * kKeys, pol);
          }
          ++r;
          return true;
        };
        if (ok) ok = load(false, 0);
        for (int j = 0; ok && j < t.nk; ++j) {
          if (j + 1 < t.nk) ok = load(false, j + 1);
          if (ok) ok = load(true, j);
        }
      }
      ++used;
      ok = __all_sync(0xffffffffu, ok);
    }
    // the commits of the last slots and of Q arrive here too: none may land after the
    // CTA has ended
    if (lane == 0 && ok && !*abort_flag) {
      for (int i = 0; ok && i < P::kSlots; ++i, ++r)
        if (r >= P::kSlots && !poll(smem_u32(&ctl.empty[r % P::kSlots]), ((r / P::kSlots) & 1) ^ 1, abort_flag, a.waits.polls)) {
          fail(a, abort_flag, SITE_DRAIN);
          ok = false;
        }
    }
  } else if (warp == 1) {
    Item it;
    if (rank == 0) {
      // ------------------------------------------------------------ MMAs
      // (the whole warp runs the loop, so that descriptors stay in uniform
      // registers; one lane issues)
      constexpr uint32_t id_s = idesc_make(256, kKeys, 1), id_o = idesc_make(256, D, 1) | kTransposeB;
      const bool one = elect_one();
      const uint64_t dq = sdesc_sw128(sQ), dk = sdesc_sw128(ring), dv = sdesc_cols(ring, 16384);
      int r = 0, done = 0;  // uses of the ring; key tiles of the items before
      bool ok = true;
      for (int k = 0, used = 0; ok && next_item(k, it); ++k) {
        const Tile<kCut> t(a, it, rank);
        if (t.nk == 0) continue;
        ok = warp_wait(a, smem_u32(&ctl.q_full), used & 1, abort_flag, SITE_MMA_FULL);
        ++used;
        auto scores = [&](int j) {
          const int s = r % P::kSlots, b = (done + j) & 1;
          if (!warp_wait(a, smem_u32(&ctl.full[s]), (r / P::kSlots) & 1, abort_flag, SITE_MMA_FULL)) return false;
          tc_fence_after();
          if (one) {
            const uint64_t keys = dk + s * (P::kSlot >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma2_bf16(P::S + b * kKeys, dq + (((kk >> 2) * 16384 + 32 * (kk & 3)) >> 4),
                        keys + (((kk >> 2) * 8192 + 32 * (kk & 3)) >> 4), id_s, kk > 0 ? 1u : 0u);
            tc_commit2_mc(smem_u32(&ctl.s_full[b]), kBoth);
            tc_commit2_mc(smem_u32(&ctl.empty[s]), kBoth);
            if (j == t.nk - 1) tc_commit2_mc(smem_u32(&ctl.q_empty), kBoth);
          }
          ++r;
          return true;
        };
        auto output = [&](int j) {
          const int s = r % P::kSlots, n = done + j, b = n & 1;
          if (!warp_wait(a, smem_u32(&ctl.full[s]), (r / P::kSlots) & 1, abort_flag, SITE_MMA_FULL) ||
              !warp_wait(a, smem_u32(&ctl.p_full[b]), (n >> 1) & 1, abort_flag, SITE_STAGE))
            return false;
          tc_fence_after();
          if (one) {
            const uint64_t v = dv + s * (P::kSlot >> 4);
            const uint32_t o = P::O + (P::kStreams == 2 ? b * D : 0);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma2_ts_bf16(o, P::S + b * kKeys + 8 * kk, v + kk * (2048 >> 4), id_o,
                           j >= P::kStreams || kk != 0 ? 1u : 0u);
            if (P::kStreams == 1) tc_commit2_mc(smem_u32(&ctl.pv_done), kBoth);
            tc_commit2_mc(smem_u32(&ctl.empty[s]), kBoth);
            if (j == t.nk - 1) tc_commit2_mc(smem_u32(&ctl.o_full), kBoth);
          }
          ++r;
          return true;
        };
        if (ok) ok = scores(0);
        for (int j = 0; ok && j < t.nk; ++j) {
          if (j + 1 < t.nk) ok = scores(j + 1);
          if (ok) ok = output(j);
        }
        done += t.nk;
      }
      // The MMAs issued so far end before TMEM or shared memory go away: always, as the
      // warps that wait for them otherwise may abort after this one has ended.
      if (one) tc_commit2(smem_u32(&ctl.drain));
      __syncwarp();
      if (!__all_sync(0xffffffffu, poll(smem_u32(&ctl.drain), 0, nullptr, 1 << 21)) && lane == 0)
        fail(a, abort_flag, SITE_DRAIN);
    }
  } else {
    // ------------------------------------------------------------ softmax, outputs
    const int wq = warp & 3, half = (warp - 2) >> 2;
    const float c = a.scale, late = kLate / c;
    int done = 0, base = 0, used = 0;  // key tiles, uses of the ring of the items before; items with keys, of three
    uint32_t vphase = 0, o_phase = 0;
    bool ok = true;
    Item it;
    // this thread's rows of the outputs (and, with 256 columns, of the scores) as token
    // and head of the tile
    int token[2], head[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int row = wq * 32 + half * 16 + 8 * z + (lane >> 2);
      token[z] = row < a.tokens * a.group ? row / a.group : 1 << 30;
      head[z] = row % a.group;
    }
    const int mine = wq * 32 + lane < a.tokens * a.group ? (wq * 32 + lane) / a.group : 1 << 30;
    // P of tile n is in TMEM: CTA 0 hears of it
    auto made = [&](int n) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 1) {
          // (A remote arrival would hold the warp for a round trip; nothing reads the word.)
          // Its release is an asynchronous store's, which need not cover the warp's earlier
          // stores; there are none left to cover.  What it tells of is done when it is
          // issued, not only ordered before it: P is in TMEM when wait::st has returned,
          // the values that a lane has cleaned are visible to the pair and to the MMAs when
          // its own fences have (take_out), and __syncwarp comes after both in every lane.
          // (A fence of the cluster here as well waits for a round trip, too: 4,096 tokens
          // took 107 us in place of 82.)
          st_async_tx4(cluster_map(smem_u32(&ctl.sink), 0), 0u, cluster_map(smem_u32(&ctl.p_full[n & 1]), 0));
        } else if (wq == 2 && (P::kStreams == 2 || half == 0)) {
          mbar_arrive_expect_tx(smem_u32(&ctl.p_full[n & 1]), 4 * P::kMakers);  // the other CTA's words
        } else {
          mbar_arrive(smem_u32(&ctl.p_full[n & 1]));
        }
      }
    };
    for (int k = 0;; ++k) {
      const bool more = ok && next_item(k, it);
      // D = 128: the two warps of a quarter meet in every item, so they go on, or leave, as
      // one; and both have read the streams' sums of the item before.
      if (D == 128 ? named_bar_any(1 + wq, 64, !more) : !more) break;
      const Tile<kCut> t(a, it, rank);
      const uint32_t bad = smem_u32(&ctl.bad[used][0][0]), flag = smem_u32(&ctl.hit[used]);
      const int own = max(0, t.mine + t.shift + 1) / kKeys - t.j0;  // first tile masked for this CTA
      float f0[2], f1[2];  // factors of the outputs of this thread's two rows there
      float2 stat[2];      // their maximum and sum
      // the values of a masked tile
      auto clean = [&](int j) {
        const int s = (base + (j + 1 < t.nk ? 2 * j + 2 : 2 * j + 1)) % P::kSlots;  // V's place in the ring
        if (!warp_wait(a, smem_u32(&ctl.vloc[s]), (vphase >> s) & 1, abort_flag, SITE_MMA_FULL)) return false;
        const int e = static_cast<int>(threadIdx.x) - 64 - (P::kStreams == 2 ? half * 128 : 0);
        Cleaner<D, P::kMakers * 32>::clean(bad, flag, ring + s * P::kSlot, e, rank, (t.j0 + j) * kKeys, it.lk,
                                            (t.j0 + t.jm) * kKeys);
        return true;
      };
      auto passed = [&](int j) {  // (every softmax warp follows the phases of the masked tiles' copies)
        if (j >= t.jm) vphase ^= 1u << (base + (j + 1 < t.nk ? 2 * j + 2 : 2 * j + 1)) % P::kSlots;
      };
      if constexpr (D == 256) {
        const uint32_t lanes = static_cast<uint32_t>(wq * 32 + half * 16) << 16;
        // this thread's two rows: the last key each sees, -1 where it is no query
        int limit[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int at = t.mine + token[x];
          limit[x] = at < it.lq ? min(at + t.shift, it.lk - 1) : -1;
        }
        float m[2] = {-INFINITY, -INFINITY}, ref[2] = {0.0f, 0.0f}, l[2] = {0.0f, 0.0f};
        for (int j = 0; ok && j < t.nk; ++j) {
          const int n = done + j;
          const uint32_t ts = P::S + (n & 1) * kKeys + lanes;
          ok = warp_wait(a, smem_u32(&ctl.s_full[n & 1]), (n >> 1) & 1, abort_flag, SITE_EPI_TMEM_FULL);
          if (!ok) break;
          tc_fence_after();
          float x[2][32];
          ld_16x64(ts, x[0]);
          ld_16x64(ts + 64, x[1]);
          if (j >= own) {
            const int key = (t.j0 + j) * kKeys + 2 * (lane & 3);
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
              ok = warp_wait(a, smem_u32(&ctl.pv_done), (n - 1) & 1, abort_flag, SITE_STAGE);
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
          float b0 = -ref[0], b1 = -ref[1];
          if (__any_sync(0xffffffffu, fmaxf(fabsf(b0), fabsf(b1)) > kFar)) {
            const float off[2] = {fabsf(b0) > kFar ? m[0] : 0.0f, fabsf(b1) > kFar ? m[1] : 0.0f};
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int i = 0; i < 32; ++i) x[y][i] -= off[(i >> 1) & 1];
            if (fabsf(b0) > kFar) b0 = 0.0f;
            if (fabsf(b1) > kFar) b1 = 0.0f;
          }
          const uint64_t c2 = pair_of(c, c), back[2] = {pair_of(b0, b0), pair_of(b1, b1)};
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float u, w;
              split(fma2(pair_of(x[y][2 * i], x[y][2 * i + 1]), c2, back[i & 1]), u, w);
              u = fast_exp2(u);
              w = fast_exp2(w);
              sums[i & 1] = add2(sums[i & 1], pair_of(u, w));
              p[i] = bf16x2_bits(u, w);
            }
            st_pairs_16x32(ts + 32 * y, p);
          }
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            float u, w;
            split(sums[z], u, w);
            l[z] += u + w;
          }
          wait_st();
          if (j >= t.jm) ok = clean(j);
          passed(j);
          if (!ok) break;
          made(n);
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          l[z] += __shfl_xor_sync(0xffffffffu, l[z], 1);
          l[z] += __shfl_xor_sync(0xffffffffu, l[z], 2);
          f0[z] = kCut && t.parts > 1 ? 1.0f : 1.0f / l[z];
          stat[z] = make_float2(m[z], l[z]);
        }
      } else {
        const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
        const int at = t.mine + mine, limit = at < it.lq ? min(at + t.shift, it.lk - 1) : -1;
        float m = -INFINITY, ref = 0.0f, l = 0.0f;
        bool far = false;  // (kept with m: with a vote per tile 2 x 2,048 tokens took 86.4 us in place of 84.9)
        for (int j = 0; ok && j < t.nk; ++j) {
          const int n = done + j;
          if ((n & 1) != half) {  // the other stream's
            passed(j);
            continue;
          }
          const uint32_t ts = P::S + half * kKeys + lanes, to = P::O + half * D + lanes;
          ok = warp_wait(a, smem_u32(&ctl.s_full[half]), (n >> 1) & 1, abort_flag, SITE_EPI_TMEM_FULL);
          if (!ok) break;
          tc_fence_after();
          // once for the maximum, once more for P (128 values a thread would not stay in
          // registers)
          const bool masked = j >= own;
          const int hidden = limit - (t.j0 + j) * kKeys;  // columns past this are masked
          float top = -INFINITY;
#pragma unroll
          for (int y = 0; y < kKeys; y += 64) {
            float x0[32], x1[32];
            tmem_ld32x2_sync(ts + y, ts + y + 32, x0, x1);
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if (y + i > hidden) x0[i] = -INFINITY;
                if (y + 32 + i > hidden) x1[i] = -INFINITY;
              }
            }
            float t4[4] = {x0[0], x0[1], x1[0], x1[1]};
#pragma unroll
            for (int i = 2; i < 32; ++i) {
              t4[i & 1] = fmaxf(t4[i & 1], x0[i]);
              t4[2 + (i & 1)] = fmaxf(t4[2 + (i & 1)], x1[i]);
            }
            top = fmaxf(top, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])));
          }
          if (__any_sync(0xffffffffu, top > m + late)) {
            const float next = top > m + late ? top : m;
            const float f = next == m ? 1.0f : fast_exp2((m - next) * c);
            m = next;
            ref = next == -INFINITY ? 0.0f : next * c;
            far = __any_sync(0xffffffffu, fabsf(ref) > kFar);
            l *= f;
            // O of the stream's tiles before: their products are done, the scores of this
            // tile were issued behind them
            if (j >= 2) {
#pragma unroll 1
              for (int d = 0; d < D; d += 32) {
                float o[32];
                uint32_t w[32];
                tmem_ld32_sync(to + d, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * f);
                st_32x32(to + d, w);
              }
            }
          }
          const uint64_t c2 = pair_of(c, c);
          uint64_t sums[4] = {0, 0, 0, 0};
          auto weights = [&](int y, uint64_t back, bool less, float off) {
            float x[32];
            uint32_t p[16];
            tmem_ld32_sync(ts + y, x);
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (y + i > hidden) x[i] = -INFINITY;
            }
            if (less) {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] -= off;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float u, w;
              split(fma2(pair_of(x[2 * i], x[2 * i + 1]), c2, back), u, w);
              u = fast_exp2(u);
              w = fast_exp2(w);
              sums[i & 3] = add2(sums[i & 3], pair_of(u, w));
              p[i] = bf16x2_bits(u, w);
            }
            st_32x16(ts + y / 2, p);
          };
          // (P of 32 columns goes over scores that are read)
          if (far) {
            const bool mine = fabsf(ref) > kFar;
            const float b = mine ? 0.0f : -ref;
#pragma unroll 1
            for (int y = 0; y < kKeys; y += 32) weights(y, pair_of(b, b), true, mine ? m : 0.0f);
          } else {
#pragma unroll
            for (int y = 0; y < kKeys; y += 32) weights(y, pair_of(-ref, -ref), false, 0.0f);
          }
          {
            float u, w;
            split(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])), u, w);
            l += u + w;
          }
          wait_st();
          if (j >= t.jm) ok = clean(j);
          passed(j);
          if (!ok) break;
          made(n);
        }
        ctl.stream[half][wq * 32 + lane] = make_float2(m, l);
      }
      // ------------------------------------------------------------ outputs
      if (ok && t.nk > 0) {
        ok = warp_wait(a, smem_u32(&ctl.o_full), o_phase, abort_flag, SITE_EPI_TMEM_FULL);
        o_phase ^= 1;
        tc_fence_after();
        // All warps of both CTAs have made P of this item, so they are past the outputs of
        // the one before: its marks make room for the item after the next, whose scores
        // wait for this warp's P of the next.
        const int e = static_cast<int>(threadIdx.x) - 64;
        const int before = used == 0 ? 2 : used - 1;
        if (e < static_cast<int>(sizeof ctl.bad / 12)) (&ctl.bad[before][0][0])[e] = 0xffffffffu;
        if (e == 0) ctl.hit[before] = 0;
      }
      // 16 rows per warp, 64 columns at a time (lane l: rows l / 4, + 8); the words of a
      // quad are turned, so that a lane stores 16 bytes and a row gets 64 at once
      int lim[2];
      bool valid[2], any[2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int at = t.mine + token[z];
        lim[z] = at + t.shift;
        valid[z] = ok && at < it.lq;
        any[z] = t.nk > 0 && lim[z] >= 0;
      }
      if constexpr (D == 128) {
        named_bar_sync(1 + wq, 64);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int row = wq * 32 + half * 16 + 8 * z + (lane >> 2);
          const float2 s0 = ctl.stream[0][row], s1 = ctl.stream[1][row];
          const float M = fmaxf(s0.x, s1.x);
          f0[z] = s0.x == M ? 1.0f : fast_exp2((s0.x - M) * c);
          f1[z] = s1.x == M ? 1.0f : fast_exp2((s1.x - M) * c);
          stat[z] = make_float2(M, f0[z] * s0.y + f1[z] * s1.y);
          const float inv = kCut && t.parts > 1 ? 1.0f : 1.0f / stat[z].y;
          f0[z] *= inv;
          f1[z] *= inv;
        }
      }
      long long row[2];  // of out
#pragma unroll
      for (int z = 0; z < 2; ++z)
        row[z] = static_cast<long long>(it.q0 + t.mine + (valid[z] ? token[z] : 0)) * a.Hq + it.head * a.group + head[z];
      if (kCut && t.parts > 1) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          row[z] += it.part * a.n_q * a.Hq;
          if (valid[z] && (lane & 3) == 0) a.stat[row[z]] = stat[z];
        }
      }
      const bool marked = t.nk > 0 && *static_cast<volatile uint32_t *>(&ctl.hit[used]) != 0;
      const uint32_t from = P::O + (static_cast<uint32_t>(wq * 32 + half * 16) << 16);
#pragma unroll 1
      for (int d = 0; ok && d < D; d += 64) {
        float v[32];
        if (t.nk > 0) {
          if constexpr (D == 256) {
            ld_16x64(from + d, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= f0[(i >> 1) & 1];
          } else {
            // (with one tile, the other stream's O is another row's)
            const int first = done & 1;
            ld_16x64(from + first * D + d, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= first ? f1[(i >> 1) & 1] : f0[(i >> 1) & 1];
            if (t.nk > 1) {
              float w[32];
              ld_16x64(from + (first ^ 1) * D + d, w);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = fmaf(w[i], first ? f0[(i >> 1) & 1] : f1[(i >> 1) & 1], v[i]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = any[(i >> 1) & 1] ? v[i] : 0.0f;
        if (kCut && t.parts > 1) {
#pragma unroll
          for (int z = 0; z < 2; ++z)
            if (valid[z]) {
              float *to = a.part + row[z] * D + d + 2 * (lane & 3);
#pragma unroll
              for (int n = 0; n < 8; ++n)
                *reinterpret_cast<float2 *>(to + 8 * n) = make_float2(v[4 * n + 2 * z], v[4 * n + 2 * z + 1]);
            }
          continue;
        }
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = bf16x2_bits(v[16 * h + 4 * i + 2 * z], v[16 * h + 4 * i + 2 * z + 1]);
            turn_quad(w);
            if (valid[z])
              *reinterpret_cast<uint4 *>(a.out + row[z] * D + d + 32 * h + 8 * (lane & 3)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
      }
      if (marked && ok) {
        asm volatile("" ::: "memory");  // (what was stored as words is read as numbers)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          if (!valid[z]) continue;
          const int seen = lim[z] - (t.j0 + t.jm) * kKeys;
          if (kCut && t.parts > 1) {
            Cleaner<D, 256>::put_back(ctl.bad[used], a.part + row[z] * D, seen, lane & 3);
          } else {
            Cleaner<D, 256>::put_back(ctl.bad[used], a.out + row[z] * D, seen, lane & 3);
          }
        }
      }
      tc_fence_before();
      if (t.nk > 0) used = used == 2 ? 0 : used + 1;
      done += t.nk;
      base += 2 * t.nk;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag)  // the other CTA hears of an abort
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_map(smem_u32(&ctl.abort_flag), rank ^ 1)), "r"(1) : "memory");
  __syncwarp();
  cluster_sync_all();  // no MMA of the pair is in flight, no arrival is pending
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(0, kTmemCols);
  if (*abort_flag)  // after an abort the copies and arrivals in flight, in either, get time to land
    for (int i = 0; i < 200; ++i) __nanosleep(1000);
}

// Joins the parts of tiles whose keys were cut: a block has some of a tile's 256 rows,
// found as the main kernel finds them; D / 4 threads per row.
constexpr int kJoinThreads = 1024;
template <int D>
constexpr int kJoinRows = kJoinThreads / (D / 4);

template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_prefill_join_kernel(const PrefillArgs a) {
  constexpr int kBlocks = 256 / kJoinRows<D>;  // of a tile
  __shared__ Item s_item;
  pdl_wait();
  pdl_launch_dependents();
  const int d = static_cast<int>(threadIdx.x) % (D / 4) * 4, lane = static_cast<int>(threadIdx.x) & 31;
  const int at = static_cast<int>(blockIdx.x % kBlocks) * kJoinRows<D> + static_cast<int>(threadIdx.x) / (D / 4);
  const int rank = at >> 7, r = at & 127;
  const long long step = a.n_q * a.Hq;
  // (more tiles than the grid has room for only where offsets run backwards)
  for (long long n = blockIdx.x / kBlocks;; n += gridDim.x / kBlocks) {
    if (threadIdx.x < 32) {
      const Schedule<true> plan(a);
      Item it = {};
      if (n / a.Hk < plan.all(plan.from(1))) it = plan.tile(n / a.Hk, static_cast<int>(n % a.Hk), 0);
      if (threadIdx.x == 0) s_item = it;
    }
    __syncthreads();
    const Item it = s_item;
    __syncthreads();
    if (!it.valid) return;
    const int t = it.t0 + rank * a.tokens + r / a.group;
    if (r >= a.tokens * a.group || t >= it.lq) continue;  // (whole warps)
    const long long row = static_cast<long long>(it.q0 + t) * a.Hq + it.head * a.group + r % a.group;
    // Lane s of a warp, all of one row, has part s's maximum and sum, of the parts that
    // have keys for this row.  (By their place, not by the sums: one may be 0 as all its
    // scores are minus infinity, and where all are, the row is 0 / 0 as it is uncut.)
    const int last = t + it.lk - it.lq;
    const int parts = last < 0 ? 0 : min(Tile<true>(a, it, 0).parts, last / (a.length * kKeys) + 1);
    const float2 ml = lane < parts ? a.stat[row + lane * step] : make_float2(-INFINITY, 0.0f);
    float M = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mine = lane >= parts ? 0.0f : ml.x == M ? 1.0f : fast_exp2((ml.x - M) * a.scale);
    float L = mine * ml.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int s0 = 0; s0 < parts; s0 += 8) {
      float4 y[8];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < parts) y[s] = *reinterpret_cast<const float4 *>(a.part + (row + (s0 + s) * step) * D + d);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float f = __shfl_sync(0xffffffffu, mine, s0 + s);
        if (s0 + s >= parts) break;
        o.x = fmaf(f, y[s].x, o.x);
        o.y = fmaf(f, y[s].y, o.y);
        o.z = fmaf(f, y[s].z, o.z);
        o.w = fmaf(f, y[s].w, o.w);
      }
    }
    const float inv = parts == 0 ? 0.0f : 1.0f / L;
    *reinterpret_cast<uint2 *>(a.out + row * D + d) =
        make_uint2(bf16x2_bits(o.x * inv, o.y * inv), bf16x2_bits(o.z * inv, o.w * inv));
  }
}

namespace {

struct PrefillDevice {
  int clusters[2] = {0, 0};  // that can be resident at once (D = 128, 256)
  int *status = nullptr;
  int rc = MOE_ERR_CUDA;
};

// clusters of two CTAs, as a programmatic dependent of the kernel before (attr[1])
void prefill_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, int ctas, int smem, cudaStream_t st) {
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreadsA);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
}

const PrefillDevice &prefill_device() {
  static PrefillDevice devs[64];
  static std::once_flag once[64];
  static const PrefillDevice none;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return none;
  std::call_once(once[dev], [dev] {
    PrefillDevice &d = devs[dev];
    d.status = noalloc_status_word();
    auto set = [](auto kern, int bytes, int &clusters) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr;
      prefill_config(cfg, &attr, 2, bytes, nullptr);
      cfg.numAttrs = 1;
      return cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0;
    };
    int cut[2];  // (as many)
    if (d.status && set(attn_prefill_kernel<128, false>, Plan<128>::kTotal, d.clusters[0]) &&
        set(attn_prefill_kernel<256, false>, Plan<256>::kTotal, d.clusters[1]) &&
        set(attn_prefill_kernel<128, true>, Plan<128>::kTotal, cut[0]) &&
        set(attn_prefill_kernel<256, true>, Plan<256>::kTotal, cut[1]))
      d.rc = MOE_OK;
  });
  return devs[dev];
}

// Where there are few tiles of rows, or some see many more keys than others, keys
// are cut into parts.  Times are in tiles of 128 keys (about 1 us): rounds of clusters
// of a part's tiles and 3 for its start and end, 5 for the second kernel, and the
// parts' outputs, which move to and fro at 3 MB a tile's time.  Measured, 16 query heads
// on 2 of 256: 1 query over 4,096 keys in 18 us (16 parts) against 41, over 16,384 in
// 25 against 142, 64 over 4,096 in 23 against 42, 300 over 8,192 in 47 (3 parts) against
// 76 (4 parts, more than there are clusters: 60); not cut: 700 over 2,000 26 (48 with 2),
// 1,300 over 4,000 61 (97).  1,016 queries over 16,484 keys packed with a prompt of 3,765,
// 4 heads on 1: 100 in place of 149.  Not cut, though it should be: one query over 131,072
// keys next to 63 over 600, 16 heads of 128 on 4, 0.91 ms.
struct Cut {
  int parts, length;
};
Cut cut_of(long long n_q, long long n_k, int n_seq, int n_q_heads, int n_kv_heads, int head_dim) {
  constexpr int kPairs = 76, kMost = 16, kUneven = 8;
  const long long per = 2 * (128 / (n_q_heads / n_kv_heads));
  const long long tiles = ((n_q + per - 1) / per + n_seq - 1) * n_kv_heads;
  // The lengths are on the device: for the first rule the longest sequence counts as of
  // twice the mean length.
  const long long all = (n_k + kKeys - 1) / kKeys, mean = (n_k / n_seq + kKeys - 1) / kKeys;
  const long long keys = n_seq > 2 ? 2 * mean : all;
  const double moved = static_cast<double>(n_q) * n_q_heads * head_dim * 4 / 3e6;
  auto time = [&](int s) {
    const long long rounds = (tiles * s + kPairs - 1) / kPairs;
    return rounds * ((keys + s - 1) / s + 3) + (s > 1 ? 5 + s * moved : 0.0);
  };
  int best = 1;
  double least = 0.9 * time(1);  // (what is cut should gain)
  for (int s = 2; s <= kMost && s <= keys && tiles * s <= 4 * kPairs; ++s)
    if (time(s) < least) {
      least = time(s);
      best = s;
    }
  long long length = (keys + best - 1) / best, most = kMost;
  if (best == 1) {
    // Several sequences with keys before their queries may differ by any factor (where
    // all keys have their queries a long sequence has many tiles, and all clusters
    // work).  The longest are cut to about a cluster's share of the work, if one
    // sequence of all the keys would be far longer than that.
    if (n_seq == 1 || n_k == n_q || tiles > 2 * kPairs) return {1, 0};
    length = tiles * mean / (2 * kPairs);
    if (length < 16) length = 16;
    if (all < 2 * length) return {1, 0};
    most = kUneven;
  }
  if (length < (all + most - 1) / most) length = (all + most - 1) / most;
  return {static_cast<int>((all + length - 1) / length), static_cast<int>(length)};
}

template <int D>
cudaError_t launch_prefill(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                           const PrefillArgs &a, int clusters, long long tiles, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  prefill_config(cfg, attr, 2 * clusters, Plan<D>::kTotal, st);
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  if (a.parts == 1) return cudaLaunchKernelEx(&cfg, attn_prefill_kernel<D, false>, mq, mk, mv, a);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_prefill_kernel<D, true>, mq, mk, mv, a);
  if (e != cudaSuccess) return e;
  return launch_attn(attn_prefill_join_kernel<D>, dim3(static_cast<unsigned>(tiles * (256 / kJoinRows<D>))), kJoinThreads, 0, st,
                     a);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_attention_prefill_workspace(long long n_q, long long n_k, int n_seq, int n_q_heads,
                                               int n_kv_heads, int head_dim, size_t *bytes) {
  if (!bytes || n_q < 0 || n_k < 0 || n_seq < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0)
    return MOE_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || n_q_heads / n_kv_heads > 64 || n_kv_heads > 4096 ||
      n_q > (1LL << 29) || n_k > (1LL << 29))
    return MOE_ERR_UNSUPPORTED;
  *bytes = 0;
  if (n_q == 0 || n_seq == 0) return MOE_OK;
  const int parts = cut_of(n_q, n_k, n_seq, n_q_heads, n_kv_heads, head_dim).parts;
  if (parts > 1) *bytes = parts * static_cast<size_t>(n_q) * n_q_heads * (head_dim * sizeof(float) + sizeof(float2));
  return MOE_OK;
}

extern "C" int moe_attention_prefill(const void *q, const void *k, const void *v,
                                     const int32_t *offsets, const int32_t *k_offsets,
                                     long long n_q, long long n_k, int n_seq, int n_q_heads,
                                     int n_kv_heads, int head_dim, long long q_stride,
                                     long long k_stride, long long v_stride, float scale, void *out,
                                     void *workspace, size_t workspace_bytes, void *cuda_stream) {
  size_t need = 0;
  const int rc = moe_attention_prefill_workspace(n_q, n_k, n_seq, n_q_heads, n_kv_heads, head_dim, &need);
  if (rc != MOE_OK) return rc;
  if (!(scale > 0.0f) || scale > kMostScale) return MOE_ERR_INVALID_ARG;
  if (k_offsets && !offsets) return MOE_ERR_INVALID_ARG;
  if (offsets ? (!k_offsets && n_q != n_k) : (n_seq > 0 && (n_q % n_seq != 0 || n_k % n_seq != 0)))
    return MOE_ERR_INVALID_ARG;
  const long long qw = static_cast<long long>(n_q_heads) * head_dim, kw = static_cast<long long>(n_kv_heads) * head_dim;
  if (q_stride < qw || k_stride < kw || v_stride < kw) return MOE_ERR_INVALID_ARG;
  const long long strides[] = {q_stride, k_stride, v_stride};
  for (long long s : strides) {
    if (s >= (1LL << 38)) return MOE_ERR_UNSUPPORTED;
    if (s % 8 != 0) return MOE_ERR_ALIGNMENT;
  }
  if (n_q == 0 || n_seq == 0) return MOE_OK;
  if (!q || !out || (n_k > 0 && (!k || !v)) || (need > 0 && !workspace) || workspace_bytes < need)
    return MOE_ERR_INVALID_ARG;
  if (off_boundary(q, 16) || off_boundary(k, 16) || off_boundary(v, 16) || off_boundary(out, 16) ||
      off_boundary(workspace, 16) ||
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
  a.scale = scale * kLog2e;
  a.status = dev.status;
  a.waits = attn_waits();
  const Cut cut = cut_of(n_q, n_k, n_seq, n_q_heads, n_kv_heads, head_dim);
  a.parts = cut.parts;
  a.length = cut.length;
  a.part = static_cast<float *>(workspace);
  if (a.parts > 1) a.stat = reinterpret_cast<float2 *>(a.part + a.parts * n_q * n_q_heads * head_dim);
  // x / d = (x m) >> (31 + s), x < 2^31, with 2^(s - 1) < d <= 2^s and m = 2^(31 + s) / d + 1
  const uint32_t divisor = 2 * a.tokens;
  uint32_t s = 1;
  while ((1u << s) < divisor) ++s;
  a.per_mul = static_cast<uint32_t>((1ULL << (31 + s)) / divisor + 1);
  a.per_shift = s - 1;
  // tiles of the call, or as many as there can be
  const long long per = 2 * a.tokens;
  const long long tiles = (offsets ? n_q / per + n_seq : n_seq * ((n_q / n_seq + per - 1) / per)) * n_kv_heads;
  const int most = dev.clusters[head_dim == 256];
  const int clusters = tiles * a.parts < most ? static_cast<int>(tiles * a.parts) : most;
  const uint64_t d = head_dim, hk = n_kv_heads;
  const uint64_t keys = n_k > 0 ? n_k : 1;  // (no key is read where there is none)
  const void *kb = n_k > 0 ? k : q, *vb = n_k > 0 ? v : q;
  CUtensorMap mq, mk, mv;
  if (!encode_map_3d(&mq, q, d, n_q_heads, n_q, 2 * d, 2 * q_stride, 64, a.group, a.tokens) ||
      !encode_map_2d(&mk, kb, 2, keys, hk * d, 64, 64, true, 2 * k_stride) ||
      !encode_map_2d(&mv, vb, 2, keys, hk * d, 64, 128, true, 2 * v_stride))
    return MOE_ERR_CUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = head_dim == 128 ? launch_prefill<128>(mq, mk, mv, a, clusters, tiles, st)
                                        : launch_prefill<256>(mq, mk, mv, a, clusters, tiles, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
