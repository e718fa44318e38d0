// decay_chunk.cu -- the chunked form of linear attention with a decay per head
// (gdn_decay_scan in include/gdn.h), on the tcgen05 tensor cores.
//
// With the tokens of a sequence in chunks of C = 64 and S the state before a
// chunk, lambda the head's decay, i and j tokens of the chunk:
//     o_i = lambda^(i+1) S q_i + sum_{j <= i} lambda^(i-j) (q_i . k_j) v_j
//     S  <- lambda^C S + U,   U = sum_j lambda^(C-1-j) v_j k_j^T
// as matrix products, d_v along the MMA's 128 rows (TMEM lanes):
//     scores  [i][j]     = Q K^T                          (bf16, exact operands)
//     O1^T    [d_v][i]   = S Q^T                          (S rounded to bf16)
//     O2^T    [d_v][i]   = V^T P^T,  P_ij = lambda^(i-j) scores   (P in bf16)
//     o_i                = lambda^(i+1) O1_i + O2_i
//     U       [d_v][d_k] = V~^T K,  V~_j = lambda^(C-1-j) v_j  (bf16, four parts)
// Every decay is a power <= 1 of lambda: nothing is divided by a decay.
//
// Precision.  V~ is four bf16 parts.  With the weight w = lambda^(C-1-j) as three
// bf16 parts w1 + w2 + w3 (24 bits) and v of 8 bits, v w1 and v w2 have 16
// bits each: a rounded bf16 product and its remainder, which a bf16 fused
// multiply-add returns exactly; v w3 goes with the second remainder.  That is
// five packed instructions for two values, where cutting fp32 products into
// three parts took twelve (and those of the slower kind).  The parts are
// multiplied smallest first, each chunk's U starts from zero in TMEM, and the
// state lives in registers, where lambda^C S + U is one fp32 fused
// multiply-add per element: tensor-core accumulation truncates, and adding
// chunk after chunk into one accumulator drifted to several 1e-6 of the state
// (now 1.3e-7 to 1.4e-7).  One float for lambda^64 would be off
// by the same part of an ulp at each chunk; the chunks use the floats below and
// above it in turn, so that their products stay within an ulp of the power (the
// state's error was up to 1e-6 at 32,768 tokens, where torch has 3e-7 to 5e-7).  The outputs are rounded to
// bf16 (rms 1.7e-3) in the end; S (the state's part of an output) and P (the
// chunk's own part) enter their products as bf16, as large a rounding each on
// its part, so that an output's rms error is sqrt(2) times that of the last
// rounding alone (2.35e-3).  Two bf16 parts of S and of P take that away
// (1.66e-3) and cost a quarter of the time: 4,096 tokens 63 us, 32,768 334 us,
// because S's second part finds no free TMEM columns and waits for the first
// one's product (60 / 308 us; P's alone 53 / 272); with one accumulator for both
// products of an output, which frees columns, 65 / 345.
//
// Work split.  One CTA scans one segment of one (sequence, value head, 128
// columns of d_v).  A sequence is one segment when the batch has enough heads
// to fill the GPU; otherwise it is cut (equal segments, or all heads' chunks in
// equal shares, one per SM; make_plan chooses): a first launch of the same kernel
// without the outputs computes what each segment leaves, a small kernel
// chains these into the state before each segment, and the main launch runs
// all segments at once.  Each lets the next one start its CTAs early (they wait
// for its results).
//
// Roles (512 threads): warp 0 TMA copies and the products S Q^T, V^T P^T and
// scores, warp 1 U's products (one issuer for all left the tensor cores idle
// while it waited for one operand or another); warps 2-5 P (the warps of each
// TMEM quarter that are free); warps 4-7 V~; warps 8-15 the state (a thread
// per row and half of d_k) and the outputs.  Shared memory is the scarce
// resource (an M = 128, N = 64 product reads 6 KB in its 48 cycles, all of the
// 128 bytes a cycle): operands that threads make go to TMEM where the MMA can
// take them from there (V~, S), and the scores use 64 rows.
//
// Measured, 32 value heads on 16 key heads of 128 x 128: 51 us for 4,096
// tokens (segments 20, chain 5, main 33, their starts overlapped; one CTA per
// head without segments 95), 257 us for 32,768 (3.1 TB/s of q, k, v, o)
// in a graph.
// A chunk of the main launch takes 1.4 us, 2,650 cycles, for products of 1,984
// cycles: its time is the chain V~ -> U -> the TMEM columns of V~ free again,
// V~'s warps sharing their schedulers with the state's and P's.  A CTA's start
// and end cost 3 chunks more, and an SM has room for one CTA only.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "decay_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kC = kChunkTok;
constexpr int kBlk = kC * 128;  // a 64-token tile of 128 bytes (64 bf16) per token: 8 KB
// threads: four warps for copies and MMAs, one warpgroup for V~ and P (two for
// V~ where there are no outputs), two for the state
constexpr int kThreadsC(bool out) { return out ? 512 : 640; }
constexpr int kStg = 4;    // TMA stages
constexpr int kTerms = 4;  // bf16 parts of V~
constexpr uint32_t kTmemAll = 512;

// TMEM columns
template <int kDk, bool kOut>
struct Cols {
  static constexpr int kBufs = kOut ? 1 : 2;            // of U and V~
  static constexpr uint32_t U = 0;                      // kDk each
  static constexpr uint32_t V = kBufs * kDk;            // kTerms x 32 each, two tokens per column
  static constexpr uint32_t S = V + kBufs * kTerms * 32;  // S, two columns of d_k per TMEM column
  static constexpr uint32_t O1 = S + kDk / 2;        // 64
  static constexpr uint32_t O2 = O1 + 64;            // 64
  static constexpr uint32_t P = O2 + 64;             // scores: 64
  static_assert((kOut ? P + 64 : S) <= kTmemAll, "TMEM columns");
};

// Shared-memory descriptor of an operand whose M or N index is contiguous
// (128-byte swizzle): 128-byte rows of 64 bf16, one per K index; 8 rows make a
// 1024-byte swizzle atom (stride byte offset, along K), `lbo` bytes lie
// between blocks of 64 along M / N.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t lbo) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lbo >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;  // A / B contiguous along M / N

// A operand in TMEM
__device__ __forceinline__ void mma_ts_bf16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t ta, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(ta),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 16 lanes x 64 fp32 columns: lane l of the warp gets, for each 8 columns n,
// v[4 n], v[4 n + 1] = row l / 4, columns 8 n + 2 (l % 4), + 1, and v[4 n + 2],
// v[4 n + 3] = row l / 4 + 8
__device__ __forceinline__ void tmem_ld_16x64_sync(uint32_t ta, float (&v)[32]) {
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
// the same for 32 columns of two accumulators
__device__ __forceinline__ void tmem_ld_16x32x2_sync(uint32_t ta, uint32_t tb, float (&a)[16],
                                                     float (&b)[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(r[16 + i]);
  }
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// shared-memory accesses by 32-bit address
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
// four 8 x 8 matrices of 16-bit values, transposed: lane l gets entries
// (column l / 4; rows 2 (l % 4), + 1) of each; lanes 8 m .. 8 m + 7 give the
// addresses of matrix m's rows
__device__ __forceinline__ void ldsm4_trans(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// four 8 x 8 matrices of 16-bit values: lane l gives row l / 4, columns
// 2 (l % 4), + 1 of each; lanes 8 m .. 8 m + 7 the addresses of matrix m's rows
__device__ __forceinline__ void stsm4(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(r0),
               "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}
// the same, each matrix stored transposed
__device__ __forceinline__ void stsm4_trans(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(r0),
               "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
// a 32 x 32 bf16 tile (64-byte swizzle) to columns x .. of rows y .. of a matrix
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t tile, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(tile), "r"(x), "r"(y)
      : "memory");
}
// this thread's stores have read their tiles; are done
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// 16 lanes x 16 columns: lane l of the warp holds rows l / 4 (even registers)
// and l / 4 + 8 (odd) of column l % 4 of each group of four
__device__ __forceinline__ void tmem_st_16x16(uint32_t ta, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(ta),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// The weights of two tokens as bf16 parts.
struct VtWeight {
  __nv_bfloat162 w1, w2, w3;
};

// V~ of 32 tokens of a chunk for a warp's 32 columns of V: the staged V
// (address `v` of the first token's row, 128-byte swizzle) times a weight per
// token, as kTerms bf16 parts of two tokens per TMEM column, [d_v lane][token
// pair].  Transposed matrix loads give lane l tokens 8 i + 2 (l % 4), + 1 of
// columns l / 4, + 8 of each 16, the layout of a 16-lane TMEM store; w[4 kHalf
// + i] are those tokens' weights.  The leading parts are left to the caller,
// because their TMEM columns are the last to become free.
template <int kHalf>
__device__ __forceinline__ void make_vt(uint32_t v, int wq, const VtWeight (&w)[8], uint32_t ta,
                                        uint32_t (&lead)[2][8]) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  const uint32_t row = v + (wq >> 1) * kBlk + (8 * (m >> 1) + (lane & 7)) * 128;
  uint32_t r[4][4];  // [16 columns, 16 tokens]
#pragma unroll
  for (int x = 0; x < 4; ++x)
    ldsm4_trans(row + ((((wq & 1) * 4 + 2 * (x >> 1) + (m & 1)) ^ (lane & 7)) << 4) + (x & 1) * 2048, r[x]);
#pragma unroll
  for (int hl = 0; hl < 2; ++hl) {
    uint32_t p[kTerms - 1][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&r[2 * hl + (e >> 2)][e & 3]);
      const VtWeight &u = w[4 * kHalf + (e >> 1)];
      const __nv_bfloat162 t1 = __hmul2_rn(x, u.w1), t2 = __hmul2_rn(x, u.w2);
      const __nv_bfloat162 t[kTerms - 1] = {__hfma2(x, u.w1, __hneg2(t1)), t2,
                                            __hfma2(x, u.w3, __hfma2(x, u.w2, __hneg2(t2)))};
      lead[hl][e] = *reinterpret_cast<const uint32_t *>(&t1);
#pragma unroll
      for (int y = 0; y < kTerms - 1; ++y) p[y][e] = *reinterpret_cast<const uint32_t *>(&t[y]);
    }
#pragma unroll
    for (int t = 1; t < kTerms; ++t)
      tmem_st_16x16(ta + 32 * t + (static_cast<uint32_t>(16 * hl) << 16), p[t - 1]);
  }
}

// the weights of make_vt for a chunk of n tokens: tab[n - 1 - t] of token t
__device__ __forceinline__ void vt_weights(const float *tab, int n, VtWeight (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = 8 * i + 2 * (threadIdx.x & 3);
    float a = t < n ? tab[n - 1 - t] : 0.0f, b = t + 1 < n ? tab[n - 2 - t] : 0.0f;
    w[i].w1 = __floats2bfloat162_rn(a, b);
    a -= __low2float(w[i].w1);
    b -= __high2float(w[i].w1);
    w[i].w2 = __floats2bfloat162_rn(a, b);
    w[i].w3 = __floats2bfloat162_rn(a - __low2float(w[i].w2), b - __high2float(w[i].w2));
  }
}

// A warp's 32 rows of kN floats, `pitch` floats apart in global memory, one row
// per lane: whole lines in global memory, turned in the warp's `tile` of shared
// memory (16-byte pieces swizzled by row).  Rows from `rows` on are zeros, not
// touched in global memory.
template <int kN>
__device__ __forceinline__ void load_rows(float (&v)[kN], uint32_t tile, const float *src, int pitch,
                                          int rows) {
  constexpr int kP = kN / 4;
  const int lane = threadIdx.x & 31;
  uint4 u[kP];  // (all of them in flight at once)
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int r = (i * 32 + lane) / kP, p = (i * 32 + lane) % kP;
    u[i] = make_uint4(0, 0, 0, 0);
    if (src && r < rows)
      u[i] = *reinterpret_cast<const uint4 *>(src + static_cast<long long>(r) * pitch + 4 * p);
  }
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int r = (i * 32 + lane) / kP, p = (i * 32 + lane) % kP;
    sts128(tile + (r * kP + (p ^ (r & (kP - 1)))) * 16, u[i].x, u[i].y, u[i].z, u[i].w);
  }
  __syncwarp();
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    const uint4 w = lds128(tile + (lane * kP + (p ^ (lane & (kP - 1)))) * 16);
    v[4 * p] = __uint_as_float(w.x);
    v[4 * p + 1] = __uint_as_float(w.y);
    v[4 * p + 2] = __uint_as_float(w.z);
    v[4 * p + 3] = __uint_as_float(w.w);
  }
  __syncwarp();
}
// and back: into the tile, then from the tile to global memory
template <int kN>
__device__ __forceinline__ void tile_rows(const float (&v)[kN], uint32_t tile) {
  constexpr int kP = kN / 4;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int p = 0; p < kP; ++p)
    sts128(tile + (lane * kP + (p ^ (lane & (kP - 1)))) * 16, __float_as_uint(v[4 * p]),
           __float_as_uint(v[4 * p + 1]), __float_as_uint(v[4 * p + 2]), __float_as_uint(v[4 * p + 3]));
  __syncwarp();
}
template <int kN>
__device__ __forceinline__ void store_rows(uint32_t tile, float *dst, int pitch, int rows) {
  constexpr int kP = kN / 4;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int r = (i * 32 + lane) / kP, p = (i * 32 + lane) % kP;
    if (r < rows)
      *reinterpret_cast<uint4 *>(dst + static_cast<long long>(r) * pitch + 4 * p) =
          lds128(tile + (r * kP + (p ^ (r & (kP - 1)))) * 16);
  }
}

// Rows [n, 64) of the staged K and of warp wq's columns of V become zero: the
// tokens after a sequence's end belong to others, and 0 x NaN is NaN.  Each
// warp reads only its own columns of V.
template <int kDk>
__device__ __forceinline__ void zero_rows(uint32_t k, uint32_t v, int wq, int n) {
  const int lane = threadIdx.x & 31, rows = kC - n;
  for (int i = lane; i < rows * 4; i += 32) {
    const int r = n + (i >> 2), p = ((wq & 1) * 4 + (i & 3)) ^ (r & 7);
    sts128(v + (wq >> 1) * kBlk + r * 128 + (p << 4), 0u, 0u, 0u, 0u);
  }
  for (int i = wq * 32 + lane; i < kDk / 64 * rows * 8; i += 128) {
    const int b = i / (rows * 8), p = i - b * rows * 8;
    sts128(k + b * kBlk + n * 128 + p * 16, 0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// A NaN or infinity in v reaches the earlier tokens of its chunk, too: V^T P^T
// multiplies it by their zeros in P.  It also leaves its row of the state NaN
// for good, so a row of S that ends as NaN is the sign, and costs the others
// nothing.  A warp then goes over column j of v: if token t is the first that
// is not finite, the outputs of the tokens before it in its chunk are made
// again by the recurrence along the row, from the state before the segment.
template <int kDk>
__device__ __noinline__ void redo_row(const DecayArgs &a, int first, int len, int h, int j,
                                      const float *row) {
  constexpr int kE = kDk / 32;
  const int lane = threadIdx.x & 31;
  const long long hk = static_cast<long long>(h / (a.Hv / a.Hk)) * kDk + kE * lane;
  const long long hv = static_cast<long long>(h) * a.dv + j;
  int bad = len;
  for (int t0 = 0; t0 < len && bad == len; t0 += 32) {
    const int t = t0 + lane;
    const bool b = t < len && !isfinite(__bfloat162float(a.v[static_cast<long long>(first + t) * a.v_stride + hv]));
    const uint32_t m = __ballot_sync(0xffffffffu, b);
    if (m) bad = t0 + __ffs(m) - 1;
  }
  if (bad == len || bad % kC == 0) return;
  const float lam = a.decay[h];
  float S[kE];
#pragma unroll
  for (int i = 0; i < kE; ++i) S[i] = row ? row[kE * lane + i] : 0.0f;
  for (int t = 0; t < bad; ++t) {
    const long long at = first + t;
    const float v = __bfloat162float(a.v[at * a.v_stride + hv]);
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      S[i] = fmaf(lam, S[i], v * __bfloat162float(a.k[at * a.k_stride + hk + i]));
      d = fmaf(S[i], __bfloat162float(a.q[at * a.q_stride + hk + i]), d);
    }
    if (t < bad - bad % kC) continue;
#pragma unroll
    for (int m = 16; m; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
    if (lane == 0) a.o[at * a.Hv * a.dv + hv] = __float2bfloat16_rn(d);
  }
}

// One part of the update product U[d_v][d_k] = V~^T K over k steps kk0, kk0 + 1
// (16 tokens each)
template <int kDk>
__device__ __forceinline__ void mma_update(uint32_t u, uint32_t vt, uint64_t k, int t, int kk0,
                                           bool accumulate) {
  constexpr uint32_t idesc = idesc_make(128, kDk, 1) | kTransB;
#pragma unroll
  for (int kk = kk0; kk < kk0 + 2; ++kk)
    mma_ts_bf16(u, vt + 32 * t + 8 * kk, k + kk * (2048 >> 4), idesc, (accumulate || kk > kk0) ? 1u : 0u);
}

__device__ __forceinline__ void fail(const DecayArgs &a, volatile int *abort_flag, int site) {
  *abort_flag = 1;
  report_error(a.status, MOE_ERR_DEVICE_TIMEOUT, KID_DECAY * 100 + site);
}

// A warp's wait for phase `parity`: false in every lane when the CTA aborted
// or the polls (each sleeps in the barrier for a while) ran out.  Short on
// purpose: it is inlined at each wait, and the roles share one instruction
// cache.
constexpr int kPolls = 1 << 22;
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < kPolls; ++i) {
    if (mbar_try_wait_sleep(bar, parity, 2000u)) return true;
    if (abort_flag && *abort_flag) return false;
  }
  return false;
}
__device__ __forceinline__ bool warp_wait(const DecayArgs &a, uint32_t bar, uint32_t parity,
                                          volatile int *abort_flag, int site) {
  if (__all_sync(0xffffffffu, poll(bar, parity, abort_flag))) return true;
  if ((threadIdx.x & 31) == 0) fail(a, abort_flag, site);
  return false;
}
// this warp's writes (TMEM and shared memory) before its arrival
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Shared memory: the stages of (Q, K, V), P, a 32 x 32 output tile for each of
// the state's warps, control
template <int kDk, bool kOut>
struct Smem {
  static constexpr int kQ = kOut ? kDk / 64 * kBlk : 0, kK = kDk / 64 * kBlk, kV = 2 * kBlk;
  static constexpr int kStage = kQ + kK + kV;
  static constexpr int kP = kStg * kStage;
  static constexpr int kO = kP + (kOut ? kBlk : 0);
  static constexpr int kCtl = kO + (kOut ? 8 * 2048 : 0);
  static constexpr int kTotal = kCtl + 2048 + 1024;
};

struct Ctl {
  uint64_t bars[32];
  uint32_t tmem;
  int abort_flag;
  // lambda^63 .. lambda^0, then zeros, in copies that start 0 and 1 words late
  alignas(16) float rtab[2][2 * kC + 8];
  float tab[kC + 1];  // lambda^0 .. lambda^64
  float step[2], frac;  // the floats around lambda^64, its place between them
};
static_assert(sizeof(Ctl) <= 2048, "control block");

}  // namespace

// ws: what each segment leaves -> the state before the next segment, in place,
// along each sequence.  A thread has 4 elements of the state of a (sequence,
// head, tile of d_v); with offsets its block works if its item is the first
// segment of several.  Where the final state goes over the initial one, that is
// copied for the first segment.
__global__ void __launch_bounds__(512, 2) decay_chain_kernel(const DecayArgs a, int dk) {
  const int per = 32 * dk;  // vectors of a tile
  const int in = blockIdx.y, e = static_cast<int>(blockIdx.z * 512 + threadIdx.x);
  if (a.table) pdl_wait();
  int seq, h, d0, n;                // n: states to make
  long long at, copy, step;         // places in ws: of the first one, of the initial one, between two
  float first, len;                 // tokens of the first segment, of the others
  if (a.table) {
    const int item = blockIdx.x;
    step = a.Hv * a.tiles;
    const Segment g = a.table[item];
    if (g.seq < 0 || g.index != 0 || g.last) return;
    long long lo, tokens;
    seq_range(a, g.seq, lo, tokens);
    n = (static_cast<int>(tokens) + a.seg_len - 1) / a.seg_len - 1;
    if (item + n >= a.cuts) return;
    seq = g.seq;
    h = in / a.tiles;
    d0 = in % a.tiles * 128;
    copy = item * step + in;
    at = copy + step;
    first = len = static_cast<float>(a.seg_len);
  } else {
    const int r = blockIdx.x, bundle = a.bundle, sub = in / a.tiles;
    const int row = r * a.pitch, cut = row / a.width + 1;
    n = (row + a.chunks - 1) / a.width - cut + 1;
    seq = r / a.Hk;
    h = (r - seq * a.Hk) * a.group + sub;
    d0 = (in - sub * a.tiles) * 128;
    step = bundle;
    at = static_cast<long long>(cut) * bundle + in;
    copy = static_cast<long long>(a.shares + r) * bundle + in;
    first = static_cast<float>((cut * a.width - row) * kC);
    len = static_cast<float>(a.width * kC);
  }
  if (!a.table) pdl_wait();
  pdl_launch_dependents();
  if (n <= 0 || e >= min(128, a.dv - d0) * dk / 4) return;
  const float f0 = decay_pow(a.decay[h], first), f = decay_pow(a.decay[h], len);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.s_in)
    s = reinterpret_cast<const float4 *>(a.s_in + ((static_cast<long long>(seq) * a.Hv + h) * a.dv + d0) * dk)[e];
  const float4 s0 = s;
  float4 *w = reinterpret_cast<float4 *>(a.ws) + at * per + e;
  step *= per;
  for (int i0 = 0; i0 < n; i0 += 8) {
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i0 + i < n) v[i] = w[(i0 + i) * step];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i0 + i < n) {
        const float g = i0 + i == 0 ? f0 : f;
        s.x = fmaf(g, s.x, v[i].x);
        s.y = fmaf(g, s.y, v[i].y);
        s.z = fmaf(g, s.z, v[i].z);
        s.w = fmaf(g, s.w, v[i].w);
        w[(i0 + i) * step] = s;
      }
  }
  if (a.s_in && a.s_in == a.s_out) reinterpret_cast<float4 *>(a.ws)[copy * per + e] = s0;
}

// kOut: the segment's outputs, from the state before it, and the final state if
// it is the sequence's last.  Otherwise: what the segment leaves from a zero
// state, unless it is the last.
template <int kDk, bool kOut>
__global__ void __launch_bounds__(kThreadsC(kOut), 1)
    decay_chunk_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmO, const DecayArgs a) {
  using L = Smem<kDk, kOut>;
  using M = Cols<kDk, kOut>;
  constexpr int kHalfDk = kDk / 2;
  constexpr int kState = kOut ? 8 : 12;  // the state's first warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  Ctl &ctl = *reinterpret_cast<Ctl *>(smem + L::kCtl);
  volatile int *abort_flag = &ctl.abort_flag;
  const uint32_t full0 = smem_u32(ctl.bars), empty0 = full0 + 8 * kStg;
  const uint32_t bar = empty0 + 8 * kStg;
  const uint32_t sc_full = bar, p_full = bar + 8, s_ready = bar + 24;
  const uint32_t o_full = bar + 32, drain = bar + 40;
  const uint32_t vt_full0 = bar + 64, u_full0 = bar + 80, u_empty0 = bar + 96, vt_part0 = bar + 112;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wq = warp & 3;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStg; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, kOut ? 2 : 1);  // both issuers are done with the stage
    }
    mbar_init(sc_full, 1);
    mbar_init(p_full, 4);
    mbar_init(s_ready, 8);  // the chunk's S is in TMEM, the last chunk's O1, O2 are read
    mbar_init(o_full, 1);
    mbar_init(drain, kOut ? 2 : 1);
    for (int b = 0; b < 4; ++b) mbar_init(vt_part0 + 8 * b, 1);
    for (int b = 0; b < 2; ++b) {
      // (with outputs, also the last U read: U has one buffer then)
      mbar_init(vt_full0 + 8 * b, kOut ? 4 + 8 : 4);
      mbar_init(u_full0 + 8 * b, 1);
      mbar_init(u_empty0 + 8 * b, 8);
    }
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  Piece g;
  if (!a.table) g = find_piece<kOut>(a, static_cast<int>(blockIdx.x));
  pdl_wait();  // (all above, while the kernel before this one ends)
  if (a.table) g = find_piece<kOut>(a, static_cast<int>(blockIdx.x));
  if (g.seq < 0) return;
  const int h = g.h, d0 = g.d0;
  const int nc = static_cast<int>((g.len + kC - 1) / kC);
  const uint32_t stages = smem_u32(smem);
  // (one thread) the copies of chunk c
  auto load = [&](int c) {
    const uint64_t pol = policy_evict_last();
    const int s = c % kStg, hk = h / (a.Hv / a.Hk);
    const uint32_t dst = stages + s * L::kStage, fb = full0 + 8 * s;
    const int y = static_cast<int>(g.first) + c * kC;
    mbar_arrive_expect_tx(fb, L::kStage);
    for (int b = 0; b < kDk / 64; ++b) {
      tma_load_2d(dst + L::kQ + b * kBlk, &tmK, fb, hk * kDk + 64 * b, y, pol);
      if (kOut) tma_load_2d(dst + b * kBlk, &tmQ, fb, hk * kDk + 64 * b, y, pol);
    }
    for (int b = 0; b < 2; ++b)
      tma_load_2d(dst + L::kQ + L::kK + b * kBlk, &tmV, fb, h * a.dv + d0 + 64 * b, y, pol);
  };
  constexpr int kFirst = kStg - 2;  // chunks whose copies start before the CTA is set up
  if (threadIdx.x == 0)
    for (int c = 0; c < nc && c < kFirst; ++c) load(c);
  if (const int t = static_cast<int>(threadIdx.x) - 64; t >= 0 && t <= kC) {
    const float p = decay_pow(a.decay[h], static_cast<float>(t));
    ctl.tab[t] = p;
    if (kOut && t < kC)
      for (int m = 0; m < 2; ++m) {
        ctl.rtab[m][m + kC - 1 - t] = p;
        ctl.rtab[m][m + kC + t] = 0.0f;
      }
    if (t == 0) {  // lambda^64 by squaring, as a sum of two floats
      float near = a.decay[h], off = 0.0f;
#pragma unroll
      for (int i = 1; i < kC; i *= 2) {
        const float sq = near * near, e = fmaf(2.0f * near, off, fmaf(near, near, -sq));
        near = sq + e;
        off = e - (near - sq);
      }
      const float other = off == 0.0f ? near : __int_as_float(__float_as_int(near) + (off > 0.0f ? 1 : -1));
      ctl.step[0] = near;
      ctl.step[1] = other;
      ctl.frac = off == 0.0f ? 0.0f : __fdividef(off, other - near);
    }
  }
  // the state's warps fetch its rows meanwhile
  const int half = (warp - kState) >> 2;
  const long long srow =
      ((static_cast<long long>(g.seq) * a.Hv + h) * a.dv + d0 + wq * 32) * kDk + half * kHalfDk;
  const uint32_t srows = stages + kFirst * L::kStage + (warp - kState) * 32 * kHalfDk * 4;
  // this warp's rows of the state before the segment (null: zeros)
  auto before_rows = [&]() -> const float * {
    if (g.from < 0) return a.s_in ? a.s_in + srow : nullptr;
    return a.ws + (static_cast<long long>(g.from) * 128 + wq * 32) * kDk + half * kHalfDk;
  };
  float S[kHalfDk];
  if (warp >= kState) {
    if (kOut) {
      load_rows<kHalfDk>(S, srows, before_rows(), kDk, a.dv - d0 - wq * 32);
      fence_proxy_async_smem();  // (TMA writes over these rows, once s_ready says they are read)
    } else {
#pragma unroll
      for (int i = 0; i < kHalfDk; ++i) S[i] = 0.0f;
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl.tmem), kTmemAll);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Only now: a CTA of the next kernel may take TMEM columns before it waits
  // for this grid, and this CTA's allocation has no limit to its wait.
  pdl_launch_dependents();
  const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
  const int tail = static_cast<int>(g.len - static_cast<long long>(nc - 1) * kC);  // tokens of the last chunk

  // P of a quarter (16 tokens) by a warp of that TMEM quarter: rows 16 wq +
  // lane / 4, + 8; columns 8 n + 2 (lane % 4), + 1.  Past column 16 wq + 15
  // these rows have nothing: zeros, written once.
  const int pi = 16 * wq + (lane >> 2), pj = 2 * (lane & 3), pm = lane >> 3;
  // this lane's row address for the matrix stores: rows 0..7, 8..15 of two
  // neighbouring column groups
  const uint32_t prow = smem_u32(smem) + L::kP + (16 * wq + 8 * (pm & 1) + (lane & 7)) * 128;
  int loaded = min(nc, kFirst);  // (warp 0) chunks whose copies were issued
  auto p_zeros = [&] {
    for (int n = 2 * wq + 2; n < 8; n += 2) stsm4(prow + (((n + (pm >> 1)) ^ (lane & 7)) << 4), 0u, 0u, 0u, 0u);
  };
  auto make_p = [&](int c) {
    // weights lambda^(row - column): pairs in the copy of the table in which
    // this lane's pairs start on 8-byte boundaries
    const float *pw = ctl.rtab[(pi + 1) & 1] + (kC - 1 - pi + ((pi + 1) & 1)) + pj;
    if (!warp_wait(a, sc_full, c & 1, abort_flag, SITE_EPI_TMEM_FULL)) return false;
    tc_fence_after();
    float v[32];
    tmem_ld_16x64_sync(M::P + lanes, v);
#pragma unroll
    for (int n = 0; n < 8; n += 2) {
      if (n > 2 * wq) break;
      uint32_t p[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int nn = n + (y >> 1), e = y & 1;
        float lo = v[4 * nn + 2 * e], hi = v[4 * nn + 2 * e + 1];
        if (n == 2 * wq) {  // (a score past the diagonal may be anything)
          const int d = pi + 8 * e - 8 * nn - pj;
          lo = d >= 0 ? lo : 0.0f;
          hi = d >= 1 ? hi : 0.0f;
        }
        const float2 w = *reinterpret_cast<const float2 *>(pw + 8 * nn - 8 * e);
        p[y] = bf16x2_bits(lo * w.x, hi * w.y);
      }
      stsm4(prow + (((n + (pm >> 1)) ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
    }
    fence_proxy_async_smem();
    warp_arrive(p_full);
    return true;
  };

  if (kOut && warp == 0) {
    // ------------------------------------------------------------ copies; issuer of the scores, O1, O2
    constexpr uint32_t id_sc = idesc_make(64, kC, 1);
    constexpr uint32_t id_o1 = idesc_make(128, kC, 1);
    constexpr uint32_t id_o2 = idesc_make(128, kC, 1) | kTransA;
    const bool one = elect_one();
    const uint64_t dp = sdesc_sw128(smem_u32(smem) + L::kP), dv = sdesc_mn(stages + L::kQ + L::kK, kBlk);
    const uint64_t dk = sdesc_sw128(stages + L::kQ), dq = sdesc_sw128(stages);
    uint32_t s = 0;
    for (int c = 0; c <= nc; ++c) {  // scores of chunk c, after the outputs of chunk c - 1
      const uint32_t ph = c & 1, at = s * (L::kStage >> 4);
      if (c > 0) {
        const uint32_t sb = s == 0 ? kStg - 1 : s - 1, before = sb * (L::kStage >> 4);
        if (!warp_wait(a, s_ready, ph ^ 1, abort_flag, SITE_STAGE)) break;
        tc_fence_after();
        if (one) {
#pragma unroll
          for (int kk = 0; kk < kDk / 16; ++kk)
            mma_ts_bf16(M::O1, M::S + 8 * kk, dq + before + (((kk >> 2) * kBlk + 32 * (kk & 3)) >> 4), id_o1,
                        kk > 0 ? 1u : 0u);
        }
        // (the rows past a sequence's end leave V with the last V~)
        if (!warp_wait(a, p_full, ph ^ 1, abort_flag, SITE_STAGE) ||
            (c == nc && tail < kC && !warp_wait(a, vt_full0, ph ^ 1, abort_flag, SITE_STAGE)))
          break;
        tc_fence_after();
        if (one) {
#pragma unroll
          for (int kk = 0; kk < kC / 16; ++kk)
            MmaKind<__nv_bfloat16>::mma(M::O2, dv + before + kk * (2048 >> 4), dp + ((32 * kk) >> 4), id_o2,
                                        kk > 0 ? 1u : 0u);
          tc_commit(o_full);
          tc_commit(empty0 + 8 * sb);
        }
      }
      // the copies of chunk c + 2, into the stage of chunk c - 2 (the last two
      // stages hold the initial state's rows until that is in TMEM)
      if (c + kFirst < nc) {
        const int sn = (c + kFirst) % kStg;
        if (!warp_wait(a, empty0 + 8 * sn, (((c + kFirst) / kStg) & 1) ^ 1, abort_flag, SITE_PRODUCER_EMPTY) ||
            (c == 0 && !warp_wait(a, s_ready, 0, abort_flag, SITE_STAGE)))
          break;
        if (one) load(c + kFirst);
        loaded = c + kFirst + 1;
      }
      if (c < nc) {
        if (!warp_wait(a, full0 + 8 * s, (c / kStg) & 1, abort_flag, SITE_MMA_FULL)) break;
        tc_fence_after();
        if (one) {
          // rows 16 g .. 16 g + 15 of a 64-row accumulator are lanes 32 g ..
#pragma unroll
          for (int kk = 0; kk < kDk / 16; ++kk) {
            const uint32_t off = at + (((kk >> 2) * kBlk + 32 * (kk & 3)) >> 4);
            MmaKind<__nv_bfloat16>::mma(M::P, dq + off, dk + off, id_sc, kk > 0 ? 1u : 0u);
          }
          tc_commit(sc_full);
        }
      }
      s = s + 1 == kStg ? 0 : s + 1;
    }
    if (one) tc_commit(drain);
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int c = min(nc, kFirst);
      for (; c < nc; ++c) {
        const int s = c % kStg;
        if (!poll(empty0 + 8 * s, ((c / kStg) & 1) ^ 1, abort_flag)) {
          fail(a, abort_flag, SITE_PRODUCER_EMPTY);
          break;
        }
        load(c);
      }
      loaded = c;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ issuer of U
    // A whole warp runs an issuer's loop, so that descriptors stay in uniform
    // registers; one lane issues.  All 512 TMEM columns are this CTA's, so
    // their addresses start at 0.
    const bool one = elect_one();
    const uint64_t dk = sdesc_mn(stages + L::kQ, kBlk);
    uint32_t s = 0;
    for (int c = 0; c < nc; ++c) {
      const int ub = c % M::kBufs;
      const uint32_t u = M::U + ub * kDk, v = M::V + ub * kTerms * 32;
      const uint64_t k = dk + s * (L::kStage >> 4);
      // (V~ is made after the chunk's copies have landed; with outputs its
      // barrier also says that U's one buffer has been read)
      if ((!kOut && !warp_wait(a, u_empty0 + 8 * ub, ((c >> 1) & 1) ^ 1, abort_flag, SITE_MMA_TMEM_EMPTY)) ||
          !warp_wait(a, vt_full0 + 8 * ub, (c / M::kBufs) & 1, abort_flag, SITE_STAGE))
        break;
      tc_fence_after();
      if (one) {
        // the small parts of each half of the tokens, then the leading ones:
        // few sums are truncated at the size of the result, and V~ of the
        // next chunk can follow part by part
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
          for (int t = kTerms - 1; t > 0; --t) mma_update<kDk>(u, v, k, t, 2 * b, b > 0 || t < kTerms - 1);
          tc_commit(vt_part0 + 8 * (2 * ub + b));
        }
        mma_update<kDk>(u, v, k, 0, 0, true);
        mma_update<kDk>(u, v, k, 0, 2, true);
        tc_commit(u_full0 + 8 * ub);
        tc_commit(empty0 + 8 * s);
      }
      s = s + 1 == kStg ? 0 : s + 1;
    }
    if (one) tc_commit(drain);
  } else if (kOut && warp < 4) {
    // ------------------------------------------------------------ P of quarters 2, 3
    p_zeros();
    for (int c = 0; c < nc; ++c)
      if (!make_p(c)) break;
  } else if (warp >= 4 && warp < kState) {
    // ------------------------------------------------------------ V~ (and P of quarters 0, 1)
    if (kOut && wq < 2) p_zeros();
    VtWeight w[8];
    vt_weights(ctl.tab, kC, w);
    for (int c = (warp - 4) >> 2; c < nc; c += M::kBufs) {  // (one warpgroup per buffer)
      const int s = c % kStg, vb = c % M::kBufs;
      const uint32_t st = stages + s * L::kStage;
      // the products that last used this buffer of V~ end part by part
      const uint32_t before = ((c / M::kBufs) & 1) ^ 1;
      if (!warp_wait(a, full0 + 8 * s, (c / kStg) & 1, abort_flag, SITE_MMA_FULL) ||
          !warp_wait(a, vt_part0 + 16 * vb, before, abort_flag, SITE_MMA_TMEM_EMPTY))
        break;
      tc_fence_after();
      if (c == nc - 1 && tail < kC) {
        zero_rows<kDk>(st + L::kQ, st + L::kQ + L::kK, wq, tail);
        vt_weights(ctl.tab, tail, w);
      }
      const uint32_t v = st + L::kQ + L::kK, ta = M::V + vb * kTerms * 32 + lanes;
      uint32_t lead[2][2][8];
      make_vt<0>(v, wq, w, ta, lead[0]);
      if (!warp_wait(a, vt_part0 + 16 * vb + 8, before, abort_flag, SITE_MMA_TMEM_EMPTY)) break;
      tc_fence_after();
      make_vt<1>(v + 32 * 128, wq, w, ta + 16, lead[1]);
      if (!warp_wait(a, u_full0 + 8 * vb, before, abort_flag, SITE_MMA_TMEM_EMPTY)) break;
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int hl = 0; hl < 2; ++hl)
          tmem_st_16x16(ta + 16 * b + (static_cast<uint32_t>(16 * hl) << 16), lead[b][hl]);
      tmem_wait_st();
      warp_arrive(vt_full0 + 8 * vb);
      if (kOut && wq < 2 && !make_p(c)) break;
    }
  } else if (warp >= kState) {
    // ------------------------------------------------------------ state, outputs
    // outputs: weights lambda^(i + 1) of this lane's tokens, its places in the
    // warp's tile (rows of 64 bytes, pieces of 16 swizzled over pairs of rows)
    float ow[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 32 * half + 8 * i + 2 * (lane & 3);
      ow[i][0] = ctl.tab[t + 1];
      ow[i][1] = ctl.tab[t + 2];
    }
    const int mm = lane >> 3;
    const uint32_t tile = smem_u32(smem) + L::kO + (warp - kState) * 2048;
    const uint32_t otile = tile + (8 * (mm >> 1) + (lane & 7)) * 64;
    const uint32_t oread = tile + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
    const bool one = elect_one(), whole = d0 + wq * 32 + 32 <= a.dv;
    const bool ovalid = d0 + wq * 32 + 8 * (lane & 3) < a.dv;
    const long long ostride = static_cast<long long>(a.Hv) * a.dv;
    __nv_bfloat16 *obase = a.o + (g.first + 32 * half + (lane >> 2)) * ostride +
                           static_cast<long long>(h) * a.dv + d0 + wq * 32 + 8 * (lane & 3);
    const uint32_t ts = M::S + half * (kHalfDk / 2) + lanes;
    auto put_state = [&] {
#pragma unroll
      for (int x = 0; x < kHalfDk / 2; x += 8) {
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = bf16x2_bits(S[2 * (x + i)], S[2 * (x + i) + 1]);
        tmem_st8(ts + x, r);
      }
      tmem_wait_st();
    };
    if (kOut) {
      warp_arrive(vt_full0);
      put_state();
      warp_arrive(s_ready);
    }
    bool ok = true;
    for (int c = 0; c < nc; ++c) {
      const int n = c == nc - 1 ? tail : kC;
      const int ub = c % M::kBufs, use = c / M::kBufs;
      const float turn = fmaf(ctl.frac, static_cast<float>(c), 0.5f);
      const float f = n < kC ? ctl.tab[n] : ctl.step[floorf(turn + ctl.frac) > floorf(turn)];
      ok = warp_wait(a, u_full0 + 8 * ub, use & 1, abort_flag, SITE_EPI_TMEM_FULL);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < kHalfDk; x += 16) {
        float u[16];
        tmem_ld16_sync(M::U + ub * kDk + half * kHalfDk + x + lanes, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) S[x + i] = fmaf(f, S[x + i], u[i]);
      }
      if (!kOut) warp_arrive(u_empty0 + 8 * ub);
      if (kOut) {
        if (c + 1 < nc) warp_arrive(vt_full0);
        ok = warp_wait(a, o_full, c & 1, abort_flag, SITE_EPI_TMEM_FULL);
        if (!ok) break;
        tc_fence_after();
        // tokens 32 half .. of the warp's 32 rows of d_v: combined 16 rows at a
        // time, two tokens per word, and stored transposed into the warp's tile
        // of 32 tokens x 64 bytes
        bulk_wait_read();  // (the last chunk's tile has left)
        __syncwarp();
#pragma unroll
        for (int hl = 0; hl < 2; ++hl) {
          float u[16], v[16];
          const uint32_t at = 32 * half + lanes + (static_cast<uint32_t>(16 * hl) << 16);
          tmem_ld_16x32x2_sync(M::O1 + at, M::O2 + at, u, v);
          uint32_t p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            p[i] = bf16x2_bits(fmaf(ow[i >> 1][0], u[2 * i], v[2 * i]),
                               fmaf(ow[i >> 1][1], u[2 * i + 1], v[2 * i + 1]));
          }
          const uint32_t to = otile + (((2 * hl + (mm & 1)) ^ ((lane >> 1) & 3)) << 4);
          stsm4_trans(to, p[0], p[1], p[2], p[3]);
          stsm4_trans(to + 16 * 64, p[4], p[5], p[6], p[7]);
        }
        if (c + 1 < nc) {
          put_state();  // (S Q^T of this chunk is done: O1 was)
          warp_arrive(s_ready);
        }
        if (32 * half + 32 <= n && whole) {
          fence_proxy_async_smem();
          __syncwarp();
          if (one)
            tma_store_2d(&tmO, tile, h * a.dv + d0 + wq * 32, g.first + c * kC + 32 * half);
        } else {
          // a sequence's end, or columns past d_v: 16 bytes of a token per lane
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 8 * i + (lane >> 2);
            const uint4 r = lds128(oread + 512 * i);
            if (ovalid && 32 * half + t < n)
              *reinterpret_cast<uint4 *>(obase + (static_cast<long long>(c) * kC + 8 * i) * ostride) = r;
          }
        }
      }
    }
    if (kOut) bulk_wait_all();
    float *dst = nullptr;
    if (ok) {
      if (!kOut)
        dst = a.ws + (static_cast<long long>(g.to) * 128 + wq * 32) * kDk + half * kHalfDk;
      else if (g.to < 0 && a.s_out)
        dst = a.s_out + srow;
    }
    // (every product of the CTA that reads the stages is done)
    if (ok) tile_rows<kHalfDk>(S, srows);
    if (kOut) {
      // (outputs are written, and later the state before is read, by all of
      // these warps before the next one goes on)
      asm volatile("bar.sync 1, 256;" ::: "memory");
      uint32_t nan = __ballot_sync(0xffffffffu, ok && isnan(S[0]) && d0 + wq * 32 + lane < a.dv);
      nan &= 0xffffu << (16 * half);  // (the rows' other half has the others)
      const float *src = before_rows();
      for (; nan; nan &= nan - 1) {
        const int r = __ffs(nan) - 1;
        redo_row<kDk>(a, g.first, g.len, h, d0 + wq * 32 + r, src ? src + r * kDk - half * kHalfDk : nullptr);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if (dst) store_rows<kHalfDk>(srows, dst, kDk, a.dv - d0 - wq * 32);
  }
  __syncwarp();
  if (warp == 0 && *abort_flag) {  // copies in flight land before the shared memory goes away
    loaded = __shfl_sync(0xffffffffu, loaded, 0);
    for (int i = max(0, loaded - kStg); i < loaded; ++i)
      poll(full0 + 8 * (i % kStg), (i / kStg) & 1, nullptr);
  }
  const bool fin = poll(drain, 0, nullptr);
  if (!__all_sync(0xffffffffu, fin) && lane == 0) fail(a, abort_flag, SITE_DRAIN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(ctl.tmem, kTmemAll);
}

namespace {

template <int kDk>
cudaError_t launch_chunked(const DecayArgs &a, const CUtensorMap &mq, const CUtensorMap &mk,
                           const CUtensorMap &mv, const CUtensorMap &mo, bool segmented,
                           cudaStream_t st) {
  const long long per = static_cast<long long>(a.Hv) * a.tiles, bundle = a.bundle;
  if (segmented) {
    cudaError_t e = launch_pdl(decay_chunk_kernel<kDk, false>, grid_of(a.table ? a.cuts * per : (a.shares - 1) * bundle),
                               kThreadsC(false), Smem<kDk, false>::kTotal, st, mq, mk, mv, mo, a);
    if (e != cudaSuccess) return e;
    const long long rows = static_cast<long long>(a.n_seq) * a.Hk;
    const dim3 grid(static_cast<unsigned>(a.table ? a.cuts : rows), static_cast<unsigned>(a.table ? per : bundle), 32 * kDk / 512);
    e = launch_pdl(decay_chain_kernel, grid, 512, 0, st, a, kDk);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(decay_chunk_kernel<kDk, true>, grid_of(a.table ? a.items * per : (a.shares + a.smalls) * bundle),
                    kThreadsC(true), Smem<kDk, true>::kTotal, st, mq, mk, mv, mo, a);
}

}  // namespace

bool decay_chunk_setup() {
  auto set = [](auto kern, int bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  return set(decay_chunk_kernel<128, true>, Smem<128, true>::kTotal) &&
         set(decay_chunk_kernel<64, true>, Smem<64, true>::kTotal) &&
         set(decay_chunk_kernel<128, false>, Smem<128, false>::kTotal) &&
         set(decay_chunk_kernel<64, false>, Smem<64, false>::kTotal);
}

cudaError_t launch_decay_chunked(const DecayArgs &a, int dk, const CUtensorMap &mq,
                                 const CUtensorMap &mk, const CUtensorMap &mv,
                                 const CUtensorMap &mo, bool segmented, cudaStream_t st) {
  return dk == 128 ? launch_chunked<128>(a, mq, mk, mv, mo, segmented, st)
                   : launch_chunked<64>(a, mq, mk, mv, mo, segmented, st);
}

}  // namespace moe
