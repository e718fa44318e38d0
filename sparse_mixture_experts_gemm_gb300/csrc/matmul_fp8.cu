// matmul_fp8.cu -- matrix product of e4m3 codes with a scale per token and a
// scale per output channel (moe_matmul_fp8 in include/moe.h):
//     out[t][n] = x_scale[t] * w_scale[n] * sum_k x[t][k] * w[n][k]
// The scales do not depend on k, so the sum runs over the codes alone on the
// tensor cores (e4m3 products, fp32 accumulators in TMEM), and each output is
// scaled in fp32 and rounded to bf16 once.  Codes arrive by TMA in blocks of
// 128 bytes of K in the 128-byte swizzle; what lies past T, N or K reads as
// zero, so any number of tokens and channels takes the same code.
//
// Two kernels:
//   * few tokens: the channels take the MMA's 128 rows and the tokens its
//     columns (16 to 256 of them), so that a handful of tokens wastes no
//     weight bandwidth; a cluster of up to 8 CTAs splits K and adds its
//     partial sums through distributed shared memory in a fixed order;
//   * many tokens: persistent CTA pairs compute 256 tokens x 256 channels on
//     the two-CTA MMA, each CTA holding its 128 tokens' accumulator twice
//     (512 TMEM columns), so that one tile is drained while the next is
//     multiplied.
// Measured (calls back to back in a graph, weights from DRAM): one token x 8192
// x 2048 6.8 us (2.5 for its weights at a copy's rate; the rest is the start,
// the sums' exchange and the end), 16 x 2048 x 4096 6.0 us, 301 x 2500 x 2048
// 9.7 us, 4096 x 8192 x 2048 40.6 us (3.4 PFLOP/s; tensor pipes busy 82 % of an
// SM's cycles), 16384 x 8192 x 2048 152 us (3.6 PFLOP/s); over seconds 178 us
// (3.1 PFLOP/s), where the power limit holds the SMs at 1,335 MHz.
// Every wait is bounded; one that runs out raises the CTA's abort flag and
// records a timeout in the status word of the calls without a handle.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kBK = 128;         // bytes of K per column block (one swizzle row)
constexpr int kRowsM = 128;      // MMA rows of one CTA
constexpr int kBlkBytes = kRowsM * kBK;
constexpr int kMmThreads = 192;  // TMA producer, MMA issuer, four epilogue warps
constexpr int kCtrl = 2048;      // barriers, TMEM address, abort flag, token scales
constexpr int kMaxSmem = 227 * 1024;

struct MatmulArgs {
  const float *xs, *ws;
  __nv_bfloat16 *out;
  long long out_stride;
  int T, N, nkb;   // nkb: K blocks of 128
  int *status;
  // few tokens
  int bt, split, stages, tt;  // tokens per tile, CTAs along K, ring stages, token tiles
  // many tokens
  int mt, nt;  // 256-token and 256-channel tiles
  int align;   // every row of out starts on a boundary of so many bytes: 32, 16, 8, 4 or 2
};

__device__ __forceinline__ void fail(const MatmulArgs &p, volatile int *abort_flag, int site) {
  *abort_flag = 1;
  report_error(p.status, MOE_ERR_DEVICE_TIMEOUT, KID_MATMUL_FP8 * 100 + site);
}

}  // namespace

// Few tokens.  Cluster of p.split CTAs per (128 channels, p.bt tokens); CTA r
// multiplies the K blocks [r nkb / split, (r + 1) nkb / split).  TMEM lane =
// channel, column = token.  The partial sums are laid out in shared memory
// [token][128 channels] over the stages, each CTA's share of the tokens goes to
// it in one bulk copy from every CTA of the cluster (stores into another CTA's
// shared memory, lane by lane, took 3 us more for 64 tokens), and each adds
// and stores its share.
__global__ void __launch_bounds__(kMmThreads, 1)
    matmul_fp8_few_kernel(const __grid_constant__ CUtensorMap tmX,
                          const __grid_constant__ CUtensorMap tmW, const MatmulArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  const int stage_bytes = kBlkBytes + p.bt * kBK;
  float *part = reinterpret_cast<float *>(smem);  // this CTA's sums, [bt][128], over the stages
  // the sums handed over: [split][bt / split][128]
  float *exch = reinterpret_cast<float *>(smem + max(p.stages * stage_bytes, p.bt * kRowsM * 4));
  uint8_t *ctrl = reinterpret_cast<uint8_t *>(exch) + (p.split > 1 ? p.bt * kRowsM * 4 : 0);
  uint64_t *bars = reinterpret_cast<uint64_t *>(ctrl);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctrl + 512);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(ctrl + 516);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * p.stages, tfull = empty0 + 8 * p.stages;
  const uint32_t xbar = tfull + 8;  // counts the bytes of the sums handed over
  float *s_xs = reinterpret_cast<float *>(ctrl + 1024);  // [bt] the tile's token scales
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long limit = MOE_WAIT_LIMIT_CYCLES;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int n0 = tile / p.tt * kRowsM, t0 = tile % p.tt * p.bt;
  const int kb0 = static_cast<int>(static_cast<long long>(p.nkb) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<long long>(p.nkb) * (rank + 1) / p.split);
  uint32_t cols = 32;
  while (static_cast<int>(cols) < p.bt) cols *= 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(tfull, 1);
    mbar_init(xbar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (p.split > 1) mbar_arrive_expect_tx(xbar, p.bt * kRowsM * 4);
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (p.split > 1) cluster_sync_all();  // every CTA of the cluster runs, its barriers exist
  pdl_wait();
  pdl_launch_dependents();

  bool ok = true;
  // the epilogue's scales, under the products: two channels per thread
  const int e = static_cast<int>(threadIdx.x) - 64, c = 2 * (e & 63), n = n0 + c;
  float w0 = 0.0f, w1 = 0.0f;
  if (warp >= 2) {
    for (int i = e; i < p.bt; i += 128) s_xs[i] = t0 + i < p.T ? p.xs[t0 + i] : 0.0f;
    if (n < p.N) w0 = p.ws[n];
    if (n + 1 < p.N) w1 = p.ws[n + 1];
  }
  if (warp == 0 && lane == 0) {
    const uint64_t pol = policy_evict_last();
    int stage = 0;
    uint32_t phase = 0;
    int kb = kb0;
    for (; kb < kb1; ++kb) {
      if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, limit, abort_flag)) {
        fail(p, abort_flag, SITE_PRODUCER_EMPTY);
        break;
      }
      const uint32_t fb = full0 + 8 * stage, dst = smem_u32(smem) + stage * stage_bytes;
      mbar_arrive_expect_tx(fb, stage_bytes);
      tma_load_2d(dst, &tmW, fb, kb * kBK, n0, pol);
      tma_load_2d(dst + kBlkBytes, &tmX, fb, kb * kBK, t0, pol);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (*abort_flag) {  // copies in flight land before the shared memory goes away
      const int issued = kb - kb0;
      for (int i = max(0, issued - p.stages); i < issued; ++i)
        if (!mbar_wait(full0 + 8 * (i % p.stages), (i / p.stages) & 1, limit, nullptr))
          fail(p, abort_flag, SITE_DRAIN);
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_make(kRowsM, p.bt, 0);
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(full0 + 8 * stage, phase, limit, abort_flag)) {
        fail(p, abort_flag, SITE_MMA_FULL);
        break;
      }
      tc_fence_after();
      const uint32_t a0 = smem_u32(smem) + stage * stage_bytes, b0 = a0 + kBlkBytes;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_e4m3(tmem, sdesc_sw128(a0 + 32 * kk), sdesc_sw128(b0 + 32 * kk), idesc,
                 (kb != kb0 || kk != 0) ? 1u : 0u);
      tc_commit(empty0 + 8 * stage);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    tc_commit(tfull);  // (also after an abort: the MMAs issued so far)
  }
  __syncwarp();
  // every warp waits for the accumulator: after this the CTA's copies and
  // MMAs are done
  ok = mbar_wait(tfull, 0, limit, nullptr);
  if (!__all_sync(0xffffffffu, ok)) {
    if (lane == 0) fail(p, abort_flag, SITE_EPI_TMEM_FULL);
    ok = false;
  }
  tc_fence_after();

  const int per = p.bt / p.split;
  if (warp >= 2) {
    const int wq = warp & 3;       // TMEM lane quarter of an epilogue warp
    float *to = part + wq * 32 + lane;
    for (int j = 0; j < p.bt; j += 16) {
      float v[16];
      tmem_ld16_sync(tmem + j + (static_cast<uint32_t>(wq * 32) << 16), v);
#pragma unroll
      for (int i = 0; i < 16; ++i) to[(j + i) * kRowsM] = v[i];
    }
    if (p.split > 1) fence_proxy_async_smem();
    named_bar_sync(1, 128);
    if (e < p.split && p.split > 1) {
      const uint32_t bytes = per * kRowsM * 4;
      asm volatile(
          "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              cluster_map(smem_u32(exch) + rank * bytes, e)),
          "r"(smem_u32(part) + e * bytes), "r"(bytes), "r"(cluster_map(xbar, e))
          : "memory");
    }
    __syncwarp();
    if (p.split > 1) {
      ok = mbar_wait(xbar, 0, limit, nullptr);
      if (!__all_sync(0xffffffffu, ok) && lane == 0) fail(p, abort_flag, SITE_STAGE);
    }
    // two channels of every other token per thread
    const float *sums = p.split > 1 ? exch : part;
    const int first = rank * per, count = min(per, p.T - t0 - first);
    __nv_bfloat16 *o = p.out + (t0 + first) * p.out_stride + n;
    if (n < p.N) {
      constexpr int kU = 8;  // tokens in flight
      const bool pair = n + 1 < p.N;
      for (int i0 = e >> 6; i0 < count; i0 += 2 * kU) {
        float2 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = make_float2(0.0f, 0.0f);
        for (int s = 0; s < p.split; ++s)
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int i = min(i0 + 2 * u, per - 1);
            const float2 x = *reinterpret_cast<const float2 *>(sums + (s * per + i) * kRowsM + c);
            v[u].x += x.x;
            v[u].y += x.y;
          }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = i0 + 2 * u;
          if (i >= count) break;
          const float xs = s_xs[first + i];
          const float y0 = v[u].x * (w0 * xs), y1 = v[u].y * (w1 * xs);
          if (p.align >= 4 && pair) {
            *reinterpret_cast<uint32_t *>(o + i * p.out_stride) = bf16x2_bits(y0, y1);
          } else {
            o[i * p.out_stride] = __float2bfloat16_rn(y0);
            if (pair) o[i * p.out_stride + 1] = __float2bfloat16_rn(y1);
          }
        }
      }
    }
  }
  if (p.split > 1) {
    __syncwarp();
    cluster_sync_all();  // every CTA has its sums: none leaves while one reads from it
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, cols);
}

namespace {

// many tokens: a stage holds one column block of the CTA's 128 tokens and of
// its 128 of the tile's 256 channels
constexpr int kHalf = kBlkBytes;
constexpr int kStages = 6;
constexpr int kPairCols = 512;
constexpr int kOutPitch = 20;                       // words per row of an output tile
constexpr int kStageOut = 4 * 32 * kOutPitch * 4;  // per epilogue warp: 32 rows of 32 bf16
constexpr int kScales = 4 * 256 * 4;       // per epilogue warp: the tile's channel scales
constexpr int kPairSmem = kStages * 2 * kHalf + 1024 + kCtrl + kStageOut + kScales;
constexpr int kBand = 16;  // 256-token tiles per band
static_assert(kPairSmem <= kMaxSmem, "shared memory");

// Tile i of the fixed order: bands of kBand token tiles, in a band one channel
// tile after another with the token tiles innermost, so that the CTA pairs
// at work share few weight tiles and a band of tokens that stays in L2.
__device__ __forceinline__ void pair_tile(const MatmulArgs &p, int i, int &m, int &n) {
  const int per = kBand * p.nt, b = i / per, m0 = b * kBand, h = min(kBand, p.mt - m0);
  const int r = i - b * per;
  n = r / h;
  m = m0 + r - n * h;
}

}  // namespace

namespace {

// rows x min(left, 32) bf16 of a warp's output tile (rows kOutPitch words
// apart) to global memory, U's width per lane
template <typename U>
__device__ __forceinline__ void store_tile(__nv_bfloat16 *o, long long stride, const uint32_t *tile,
                                           int lane, int rows, int left) {
  constexpr int kE = sizeof(U) / 2, kLanes = 32 / kE;  // bf16 per lane, lanes per row
  const int c = lane % kLanes * kE;
#pragma unroll 4
  for (int r = lane / kLanes; r < rows; r += kE) {
    const uint16_t *src = reinterpret_cast<const uint16_t *>(tile + r * kOutPitch) + c;
    if (c + kE <= left) {
      *reinterpret_cast<U *>(o + r * stride + c) = *reinterpret_cast<const U *>(src);
    } else {
      for (int x = 0; x < kE && c + x < left; ++x)
        reinterpret_cast<uint16_t *>(o + r * stride + c)[x] = src[x];
    }
  }
}

}  // namespace

// Many tokens: CTA pairs (clusters of two) on the two-CTA MMA.  CTA r of a pair
// stages its own 128 tokens and 128 of the tile's 256 channels; CTA 0 issues
// the MMAs, which read both CTAs' halves and leave 128 tokens x 256 channels
// in each CTA's TMEM.  Barriers: full[s] in CTA 0 counts the bytes of both
// CTAs; empty[s] and tfull[a] in both, by the MMA's multicast commit;
// tempty[a] in CTA 0, by the eight epilogue warps of the pair.
__global__ void __launch_bounds__(kMmThreads, 1)
    matmul_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmX,
                           const __grid_constant__ CUtensorMap tmW, const MatmulArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  uint8_t *sA = smem, *sB = smem + kStages * kHalf;
  uint8_t *ctrl = smem + kStages * 2 * kHalf;
  uint64_t *bars = reinterpret_cast<uint64_t *>(ctrl);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctrl + 512);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(ctrl + 516);
  uint32_t *s_out = reinterpret_cast<uint32_t *>(ctrl + kCtrl);              // [4 warps][32][kOutPitch]
  float *s_ws = reinterpret_cast<float *>(ctrl + kCtrl + kStageOut);         // [4 warps][256]
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages;
  const uint32_t tfull0 = empty0 + 8 * kStages, tempty0 = tfull0 + 16, drain_bar = tempty0 + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long limit = MOE_WAIT_LIMIT_CYCLES;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cl = static_cast<int>(blockIdx.x >> 1), ncl = static_cast<int>(gridDim.x >> 1);
  constexpr uint16_t kBoth = 3;
  const int tiles = p.mt * p.nt;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 8);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmW);
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(tmem_slot), kPairCols);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      uint32_t pend_mask = 0, pend_phase = 0;
      bool ok = true;
      for (int ti = cl; ok && ti < tiles; ti += ncl) {
        int m, n;
        pair_tile(p, ti, m, n);
        const int xrow = (2 * m + rank) * kRowsM, wrow = (2 * n + rank) * kRowsM;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, limit, abort_flag)) {
            fail(p, abort_flag, SITE_PRODUCER_EMPTY);
            ok = false;
            break;
          }
          const uint32_t fb = full0 + 8 * stage, fb0 = cluster_map(fb, 0);
          if (rank == 0) mbar_arrive_expect_tx(fb, 4 * kBlkBytes);
          tma_load_2d_pair(smem_u32(sA + stage * kHalf), &tmX, fb0, kb * kBK, xrow, pol);
          tma_load_2d_pair(smem_u32(sB + stage * kHalf), &tmW, fb0, kb * kBK, wrow, pol);
          pend_mask |= 1u << stage;
          pend_phase = (pend_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // the commits of the last stages arrive here too: none may land after
      // the CTA has ended
      for (int j = 0; ok && j < kStages; ++j) {
        if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, limit, abort_flag)) {
          fail(p, abort_flag, SITE_DRAIN);
          ok = false;
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok && rank == 0)  // copies of both CTAs that complete here
        for (int s = 0; s < kStages; ++s)
          if ((pend_mask >> s) & 1)
            if (!mbar_wait(full0 + 8 * s, (pend_phase >> s) & 1, limit, nullptr))
              fail(p, abort_flag, SITE_DRAIN);
    }
  } else if (warp == 1) {
    // The whole warp runs the loop, so that descriptors stay in uniform
    // registers; one lane issues.  All 512 TMEM columns are this CTA's, so
    // their addresses start at 0.
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_make(2 * kRowsM, 256, 0);
      const bool one = elect_one();
      const uint64_t da = sdesc_sw128(smem_u32(sA)), db = sdesc_sw128(smem_u32(sB));
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity, int site) {
        const bool w = mbar_wait(bar, parity, limit, abort_flag);
        if (__all_sync(0xffffffffu, w)) return true;
        if (lane == 0) fail(p, abort_flag, site);
        return false;
      };
      for (int ti = cl; ok && ti < tiles; ti += ncl) {
        ok = wait(tempty0 + 8 * acc, acc_phase ^ 1, SITE_MMA_TMEM_EMPTY);
        if (!ok) break;
        tc_fence_after();
        for (int kb = 0; kb < p.nkb; ++kb) {
          ok = wait(full0 + 8 * stage, phase, SITE_MMA_FULL);
          if (!ok) break;
          tc_fence_after();
          if (one) {
            const uint32_t at = stage * (kHalf >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma2_e4m3(acc * 256, da + at + 2 * kk, db + at + 2 * kk, idesc, (kb | kk) != 0 ? 1u : 0u);
            tc_commit2_mc(empty0 + 8 * stage, kBoth);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (one) tc_commit2_mc(tfull0 + 8 * acc, kBoth);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (!ok) {  // the MMAs issued so far end before TMEM or shared memory go away
        if (one) tc_commit2(drain_bar);
        if (!mbar_wait(drain_bar, 0, limit, nullptr) && lane == 0) fail(p, abort_flag, SITE_DRAIN);
      }
    }
  } else {
    const int wq = warp & 3;
    float *ws = s_ws + wq * 256;
    uint32_t *so = s_out + wq * 32 * kOutPitch;
    const uint32_t tempty_r = cluster_map(tempty0, 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int ti = cl; ti < tiles; ti += ncl) {
      int m, n;
      pair_tile(p, ti, m, n);
      // the tile's scales, under its products
      const int t0 = (2 * m + rank) * kRowsM + wq * 32, t = t0 + lane;
      const float xs = t < p.T ? p.xs[t] : 0.0f;
      float w8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int nn = n * 256 + 32 * i + lane;
        w8[i] = nn < p.N ? p.ws[nn] : 0.0f;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) ws[32 * i + lane] = w8[i];
      __syncwarp();
      const bool ok = mbar_wait(tfull0 + 8 * acc, acc_phase, limit, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) fail(p, abort_flag, SITE_EPI_TMEM_FULL);
        break;
      }
      tc_fence_after();
      const uint32_t tb =
          tmem + static_cast<uint32_t>(acc * 256) + (static_cast<uint32_t>(wq * 32) << 16);
      const int rows = min(32, p.T - t0);
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {
        const int nc = n * 256 + c;
        if (nc >= p.N) break;
        float v[32];
        tmem_ld32_sync(tb + c, v);
        __syncwarp();  // (the last columns' readers of the output tile are done)
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 w4 = *reinterpret_cast<const float4 *>(ws + c + i);
          v[i] *= w4.x * xs;
          v[i + 1] *= w4.y * xs;
          v[i + 2] *= w4.z * xs;
          v[i + 3] *= w4.w * xs;
        }
        if (p.align == 32 && nc + 32 <= p.N) {
          // 32 bytes per thread and store: whole sectors
          if (t < p.T) {
            __nv_bfloat16 *o = p.out + t * p.out_stride + nc;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t b[8];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                b[j] = bf16x2_bits(v[16 * q + 2 * j], v[16 * q + 2 * j + 1]);
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + 16 * q),
                           "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3]), "r"(b[4]), "r"(b[5]),
                           "r"(b[6]), "r"(b[7])
                           : "memory");
            }
          }
        } else {
          // rows off the 32-byte grid, or the last columns: through shared
          // memory, so that the lanes of a store lie side by side in a row,
          // with as many bytes each as the rows' alignment allows
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<uint4 *>(so + lane * kOutPitch + j) =
                make_uint4(bf16x2_bits(v[2 * j], v[2 * j + 1]), bf16x2_bits(v[2 * j + 2], v[2 * j + 3]),
                           bf16x2_bits(v[2 * j + 4], v[2 * j + 5]), bf16x2_bits(v[2 * j + 6], v[2 * j + 7]));
          __syncwarp();
          __nv_bfloat16 *o = p.out + t0 * p.out_stride + nc;
          const int left = p.N - nc;
          if (p.align >= 8) {
            store_tile<uint2>(o, p.out_stride, so, lane, rows, left);
          } else if (p.align == 4) {
            store_tile<uint32_t>(o, p.out_stride, so, lane, rows, left);
          } else {
            store_tile<uint16_t>(o, p.out_stride, so, lane, rows, left);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_r + 8 * acc);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no MMA of the pair is in flight, no arrival is pending
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem, kPairCols);
  if (*abort_flag)  // after an abort the partner's copies get time to land
    for (int i = 0; i < 200; ++i) __nanosleep(1000);
}

namespace {

template <typename K>
cudaError_t launch_clusters(K kern, int grid, int cluster, int smem, cudaStream_t st,
                            const CUtensorMap &x, const CUtensorMap &w, const MatmulArgs &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, x, w, p);
}

// Which kernel, and for few tokens how many per tile (bt; 0: the CTA pairs) and
// how many CTAs along K.
struct Shape {
  int bt, split;
};

// The least of the times that these fits of measured calls give, in us (weights
// from DRAM, N 512 .. 8192, K 512 .. 4096, T 1 .. 2048; within 20 %).  Few
// tokens: 0.285 per K block of a CTA, 0.044 per token of its share to store, a
// cluster's start and exchange.  Pairs: 0.266 per K block, more where out's
// rows are not on 32-byte boundaries.  E.g. 16 x 2048 x 4096: 6.0 with 8 CTAs
// along K, 11.9 with one, 13.1 by pairs; 301 x 2500 x 2048: 9.8 in tiles of 64
// tokens, 16.4 of 32, 12.3 by pairs; 128 x 8192 x 2048: 12.3 in one tile of
// 128, 10.2 by pairs.
Shape pick_shape(int T, int N, int nkb, int align, int sms) {
  auto waves = [](long long ctas, int slots) { return static_cast<double>((ctas + slots - 1) / slots); };
  const long long tiles = static_cast<long long>((T + 255) / 256) * ((N + 255) / 256);
  Shape best = {0, 1};
  double least = 4.2 + waves(tiles, sms / 2) * (0.266 * nkb + 0.7) + (align < 32 ? 2.5 : 0.0);
  const int most[] = {32, 64, 128};
  const double start[] = {0.0, 1.1, 1.9, 3.2};
  for (int m : most) {
    const int tt = (T + m - 1) / m, bt = ((T + tt - 1) / tt + 15) / 16 * 16;
    for (int k = 0, split = 1; k < 4 && split <= nkb; ++k, split *= 2) {
      const long long ctas = static_cast<long long>((N + kRowsM - 1) / kRowsM) * tt * split;
      const double t = 1.84 + waves(ctas, sms) * (0.285 * ((nkb + split - 1) / split) + 0.0435 * bt / split +
                                                  start[k] + (split > 1 ? 0.02 * bt : 0.0));
      if (t < least) {
        least = t;
        best = {bt, split};
      }
    }
  }
  return best;
}

// Per device: what the launches need to know, looked up once.
struct MatmulDevice {
  int sms = 0;
  int *status = nullptr;
  int rc = MOE_ERR_CUDA;
};

const MatmulDevice &matmul_device() {
  static MatmulDevice devs[64];
  static std::once_flag once[64];
  static const MatmulDevice none;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return none;
  std::call_once(once[dev], [dev] {
    MatmulDevice &d = devs[dev];
    d.status = noalloc_status_word();
    if (d.status &&
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
        cudaFuncSetAttribute(matmul_fp8_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxSmem) == cudaSuccess &&
        cudaFuncSetAttribute(matmul_fp8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kPairSmem) == cudaSuccess)
      d.rc = MOE_OK;
  });
  return devs[dev];
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_matmul_fp8(const uint8_t *x, const float *x_scales, int T, long long x_stride,
                              const uint8_t *w, const float *w_scales, int N, int K,
                              long long w_stride, void *out, long long out_stride,
                              void *cuda_stream) {
  if (T < 0 || N <= 0 || K <= 0 || x_stride < K || w_stride < K || out_stride < N)
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !x_scales || !w || !w_scales || !out)) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || T > (1 << 22) || N > (1 << 20) || K > (1 << 17) ||
      x_stride >= (1LL << 40) || w_stride >= (1LL << 40))
    return MOE_ERR_UNSUPPORTED;
  auto misaligned = [](const void *p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) % n) != 0;
  };
  if (misaligned(x, 16) || misaligned(w, 16) || x_stride % 16 != 0 || w_stride % 16 != 0 ||
      misaligned(x_scales, 4) || misaligned(w_scales, 4) || misaligned(out, 2))
    return MOE_ERR_ALIGNMENT;
  if (T == 0) return MOE_OK;
  const MatmulDevice &dev = matmul_device();
  if (dev.rc != MOE_OK) return dev.rc;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  MatmulArgs p = {};
  p.xs = x_scales;
  p.ws = w_scales;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.out_stride = out_stride;
  p.T = T;
  p.N = N;
  p.nkb = (K + kBK - 1) / kBK;
  p.status = dev.status;
  p.align = 32;
  while (misaligned(out, p.align) || 2 * out_stride % p.align != 0) p.align /= 2;
  p.mt = (T + 255) / 256;
  p.nt = (N + 255) / 256;
  const Shape shape = pick_shape(T, N, p.nkb, p.align, dev.sms);
  CUtensorMap mx, mw;
  if (!encode_map_2d(&mw, w, 1, N, K, kBK, kRowsM, true, w_stride) ||
      !encode_map_2d(&mx, x, 1, T, K, kBK, shape.bt ? shape.bt : kRowsM, true, x_stride))
    return MOE_ERR_CUDA;
  cudaError_t e;
  if (shape.bt == 0) {
    const int pairs = dev.sms / 2, tiles = p.mt * p.nt;
    e = launch_clusters(matmul_fp8_pair_kernel, 2 * (tiles < pairs ? tiles : pairs), 2, kPairSmem, st, mx,
                        mw, p);
  } else {
    p.bt = shape.bt;
    p.split = shape.split;
    p.tt = (T + p.bt - 1) / p.bt;
    const int stage = kBlkBytes + p.bt * kBK, part = p.bt * kRowsM * 4, exch = p.split > 1 ? part : 0;
    const int mine = (p.nkb + p.split - 1) / p.split;
    p.stages = (kMaxSmem - 1024 - kCtrl - exch) / stage;
    if (p.stages > mine) p.stages = mine;
    if (p.stages > 16) p.stages = 16;
    const int ring = p.stages * stage;
    e = launch_clusters(matmul_fp8_few_kernel, (N + kRowsM - 1) / kRowsM * p.tt * p.split, p.split,
                        (ring > part ? ring : part) + exch + kCtrl + 1024, st, mx, mw, p);
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
