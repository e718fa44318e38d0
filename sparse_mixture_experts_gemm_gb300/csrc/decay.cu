// decay.cu -- linear attention with one decay per value head (gdn_decay_scan
// in include/gdn.h).  With S the state [d_v][d_k] of a value head and lambda
// its decay:
//     S <- lambda S + v_t k_t^T,   o_t = S q_t
//
// The recurrent form (up to kRecur tokens): rows of S are independent, so a
// warp holds eight of them (d_k = 128; sixteen of 64) in registers for the
// whole call, a row spread over d_k / 4 lanes; each token costs one decay and
// write (2 operations an element) and one dot product per row.  One token per
// sequence reads and writes the state once and little else, so it is bound by
// memory: 64 sequences of 32 heads of 128 x 128 take 40.8 us (6.6 TB/s, a
// plain copy's rate), one sequence 2.2 us.  With more tokens the dot
// products' sums count: the lanes trade rows while they add (9 shuffles for 8
// rows, where a tree per row takes 40), and the next token is fetched ahead:
// 8 tokens of 64 sequences 113 -> 73 us.  Four rows a lane are as fast for
// single tokens and slower after (84 us), as fewer products share q and k.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "../../include/gdn.h"
#include "decay_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kRecWarps = 4, kR = 8;  // warps of a CTA, rows of a lane

// kN bf16 values (4 or 8) by one load
template <int kN>
struct Bf16Vec {
  uint32_t w[kN / 2];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    if constexpr (kN == 8) {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2 *>(p);
      w[0] = u.x, w[1] = u.y;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};

// Sums of kR values over kLpr neighbouring lanes: halves of the lanes trade
// halves of the values until each has one, then add up what is left.  Lane c
// of the kLpr ends with the sum of value c / (kLpr / kR).
template <int kLpr>
__device__ __forceinline__ float sum_rows(float (&d)[kR], int c) {
  int n = kR;
#pragma unroll
  for (int m = kLpr / 2; m; m >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = c & m;
#pragma unroll
      for (int r = 0; r < kR / 2; ++r) {
        if (r >= n) break;
        const float give = up ? d[r] : d[r + n], keep = up ? d[r + n] : d[r];
        d[r] = keep + __shfl_xor_sync(0xffffffffu, give, m);
      }
    } else {
      d[0] += __shfl_xor_sync(0xffffffffu, d[0], m);
    }
  }
  return d[0];
}

}  // namespace

// One CTA: kRecWarps * kR * (128 / kDk) rows of one (sequence, value head).
template <int kDk>
__global__ void __launch_bounds__(kRecWarps * 32) decay_recurrent_kernel(const DecayArgs a) {
  constexpr int kLpr = kDk / 4;               // lanes per row
  constexpr int kRowsWarp = kR * (32 / kLpr);  // rows of a warp
  constexpr int kRows = kRecWarps * kRowsWarp;
  const int tiles = (a.dv + kRows - 1) / kRows;
  pdl_wait();
  pdl_launch_dependents();
  if (a.table && blockIdx.x == gridDim.x - 1) {  // one block more: the chunked kernels' segments
    make_table(a);
    return;
  }
  const int tile = blockIdx.x % tiles;
  const int sh = blockIdx.x / tiles, h = sh % a.Hv, seq = sh / a.Hv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kLpr;
  // this lane's rows: j .. j + kR - 1, all of them below d_v or none (d_v is a
  // multiple of 16, as are a warp's rows or they divide it)
  const int j = tile * kRows + warp * kRowsWarp + lane / kLpr * kR;
  if (j - lane / kLpr * kR >= a.dv) return;
  long long first, len;
  seq_range(a, seq, first, len);
  if (len > a.recur) return;  // the chunked kernels take it
  const long long sbase = ((static_cast<long long>(seq) * a.Hv + h) * a.dv + j) * kDk + 4 * c;
  float4 S[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r)
    S[r] = a.s_in ? *reinterpret_cast<const float4 *>(a.s_in + sbase + r * kDk) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float lam = a.decay[h];
  const int hk = h / (a.Hv / a.Hk);
  const __nv_bfloat16 *qp = a.q + first * a.q_stride + hk * kDk + 4 * c;
  const __nv_bfloat16 *kp = a.k + first * a.k_stride + hk * kDk + 4 * c;
  const __nv_bfloat16 *vp = a.v + first * a.v_stride + h * a.dv + j;
  __nv_bfloat16 *op = a.o + (first * a.Hv + h) * a.dv + j + c / (kLpr / kR);
  Bf16Vec<4> q, k;
  Bf16Vec<kR> v;
  auto fetch = [&] {
    q.load(qp);
    k.load(kp);
    v.load(vp);
    qp += a.q_stride;
    kp += a.k_stride;
    vp += a.v_stride;
  };
  if (len > 0) fetch();
  for (int t = 0; t < static_cast<int>(len); ++t) {
    const Bf16Vec<4> qt = q, kt = k;
    const Bf16Vec<kR> vt = v;
    if (t + 1 < len) fetch();
    float d[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      S[r].x = fmaf(lam, S[r].x, vt.at(r) * kt.at(0));
      S[r].y = fmaf(lam, S[r].y, vt.at(r) * kt.at(1));
      S[r].z = fmaf(lam, S[r].z, vt.at(r) * kt.at(2));
      S[r].w = fmaf(lam, S[r].w, vt.at(r) * kt.at(3));
      d[r] = S[r].x * qt.at(0) + S[r].y * qt.at(1) + S[r].z * qt.at(2) + S[r].w * qt.at(3);
    }
    const float o = sum_rows<kLpr>(d, c);
    if (c % (kLpr / kR) == 0) *op = __float2bfloat16_rn(o);
    op += static_cast<long long>(a.Hv) * a.dv;
  }
  if (a.s_out) {
#pragma unroll
    for (int r = 0; r < kR; ++r) *reinterpret_cast<float4 *>(a.s_out + sbase + r * kDk) = S[r];
  }
}

namespace {

template <int kDk>
cudaError_t launch_recurrent(const DecayArgs &a, cudaStream_t st) {
  constexpr int kRows = kRecWarps * kR * (128 / kDk);
  const int tiles = (a.dv + kRows - 1) / kRows;
  const unsigned blocks = static_cast<unsigned>(a.n_seq) * a.Hv * tiles + (a.table ? 1 : 0);
  return launch_pdl(decay_recurrent_kernel<kDk>, grid_of(blocks), kRecWarps * 32, 0, st, a);
}

}  // namespace

}  // namespace moe

using namespace moe;

namespace {

// Longest sequence that takes the recurrent form.  Its time grows with the
// tokens, a chunk's does not (32 heads of 128 x 128; recurrent / chunked, us):
//   tokens   1 sequence   4          16          64
//   12       4.7 / 7.5    8.6 / 9.6  23.8 / 36    92 / 125
//   16       5.8 / 7.5   10.4 / 9.6  29.7 / 36   111 / 125
//   24       8.2 / 7.6   14.5 / 9.7  42.6 / 36   156 / 126
constexpr long long kRecur = 16;

// How a call is cut: the sequences that are not recurrent, their segments.
struct Plan {
  bool recurrent, chunked, segmented;
  // without offsets: rows of chunks on a line cut into shares
  long long rows, chunks, pitch, width, shares;
  // with offsets: items of the table, at most `cuts` of them of cut sequences
  long long seg_len, cut_from, cuts, items;
  long long table;  // bytes of the table of segments, at the workspace's start
  long long slots;  // states in the workspace
};

// bytes of a call's workspace
size_t workspace_bytes_of(const Plan &p, int d_k) {
  return static_cast<size_t>(p.table) + static_cast<size_t>(p.slots) * 128 * d_k * sizeof(float);
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// How the rows are cut, by the time of the kernels in units of one chunk of the
// main kernel (1.4 us): a CTA takes its chunks and 3 more to start and end; where
// a sequence has several segments the first launch (0.52 per chunk and 4) and
// the chain (3.5, its steps and its traffic) come before.  The constants were
// fitted to the times of 1 to 32 segments at 43 sizes (1 to 8 sequences of 256
// to 32,768 tokens, 2 to 64 heads).  Two ways to cut are compared: each row
// into equal segments; and the whole line into one share per SM, whatever row
// ends inside it.  A share that holds the end of one row and the start of the
// next is two CTAs: the larger piece starts at once, and the smaller ones,
// largest first, follow on the SMs whose piece was the smallest, so that each
// SM gets a share and two CTAs' start at most (counted as 10 here, for 3: with 6
// shares won by the model where they lose by 1 to 2 %).  In equal segments /
// in shares: 16,384 tokens x 32 heads 150 / 142 us, 32,768 x 32 272 / 259,
// 8,192 x 64 157 / 147; 8,192 x 32 83.8 / 84.5, 16,384 x 16 81.5 / 83.5.
// With offsets the lengths are not known here: a segment is as long as for one
// sequence of all tokens, but no shorter than the SMs that the uncut batch
// leaves idle can take: the sequences have a CTA per head, or one segment each
// that is not whole, and the rest of the CTAs that run at once goes to whole
// segments.  Where no SM is left the cut helps the longest sequence only and
// costs the others: from 64 chunks, or an SM's share of all the work, on.
// With that bound / with 64 chunks for every batch: one of 2,900 tokens 25.8 /
// 71.9 us with 1 head, 29.5 / 73.1 with 4, 53.6 / 73.4 with 32; nine of 0 to
// 2,049 tokens 30.9 / 55.1 with 4 heads, 39.7 / 56.2 with 8, not cut with 32
// (62; the longest two cut in two 93); sixteen of 512 with 4 heads, where the
// launches for cuts find none, 26.3 / 22.6.
Plan make_plan(bool ragged, long long n_tokens, long long n_seq, long long n_k_heads, long long heads) {
  Plan p = {};
  const long long len = ragged ? n_tokens : n_seq ? n_tokens / n_seq : 0;
  const long long seqs = ragged ? 1 : n_seq;  // of length len at most
  p.chunked = len > kRecur;
  p.recurrent = ragged || !p.chunked;
  if (!p.chunked) return p;
  const long long chunks = ceil_div(len, kChunkTok), bundle = heads / n_k_heads;
  const long long share = ceil_div(chunks * heads, kGpuSms);
  const long long idle = kGpuSms - n_seq * heads;
  const long long least = !ragged ? 1 : std::max(share, idle > 0 ? std::min(ceil_div(chunks * heads, idle), 64LL) : 64LL);
  p.rows = seqs * n_k_heads;
  p.chunks = chunks;
  double best = 0;
  for (long long n = 1; n <= 256 && n <= chunks; ++n) {
    const long long lc = ceil_div(chunks, n);
    if (n > 1 && lc < least) break;
    const long long ns = ceil_div(chunks, lc);
    double t = static_cast<double>(ceil_div(ns * seqs * heads, kGpuSms)) * (lc + 3);
    if (ns > 1)
      t += static_cast<double>(ceil_div((ns - 1) * seqs * heads, kGpuSms)) * (0.52 * lc + 4) + 3.5 +
           0.1 * ns + 0.015 * (ns - 1) * seqs * heads;
    if (n == 1 || t < best) {
      best = t;
      p.width = lc;
      p.pitch = ns * lc;
      p.shares = p.rows * ns;
    }
  }
  p.segmented = p.width < chunks;
  if (ragged) {
    // if the longest has more than cut_from tokens, where the launches that come
    // before cost less (by the costs above) than the chunks that run elsewhere,
    // all sequences of more than seg_len are cut (those launches delay the short
    // ones too); each has one segment more than whole seg_len in it at most.  Only their segments have states in the
    // workspace: 192 prompts in 32,768 tokens, 32 heads of 128 x 128, 15 MB
    // and 538 us (411 MB and 627 us with states for all that may be chunked).
    p.seg_len = p.width * kChunkTok;
    const auto sequences = [&](long long longer) { return std::min(n_seq, n_tokens / (longer + 1)); };
    p.cut_from = (p.width + (52 * p.width + 750) / 100) * kChunkTok;
    p.cuts = p.segmented ? n_tokens / p.seg_len + sequences(p.seg_len) : 0;
    p.items = p.cuts + sequences(kRecur);
    p.table = p.items * static_cast<long long>(sizeof(Segment));
    p.slots = p.cuts * heads;
    return p;
  }
  if (bundle <= kGpuSms && p.rows <= kGpuSms / bundle) {
    const long long w = ceil_div(p.rows * chunks, kGpuSms / bundle);
    const long long shares = ceil_div(p.rows * chunks, w);
    const double t = (w + 10) + (0.52 * w + 4) + 3.5 + 0.1 * (ceil_div(chunks, w) + 1) + 0.015 * shares * bundle;
    if (w < chunks && t < best) {
      p.segmented = true;
      p.width = w;
      p.pitch = chunks;
      p.shares = shares;
    }
  }
  p.slots = p.segmented ? (p.shares + p.rows) * bundle : 0;
  return p;
}

// The rows whose end lies inside a share that the next row starts in, by the
// size of the share's smaller piece; returns their number.
int small_pieces(const Plan &p, uint8_t *order) {
  long long size[kGpuSms];
  int n = 0;
  if (p.rows > kGpuSms || p.pitch % p.width == 0) return 0;
  for (long long r = 0; r + 1 < p.rows; ++r) {
    const long long end = (r + 1) * p.pitch, before = end % p.width;
    if (before == 0) continue;
    const long long after = p.width - before < p.chunks ? p.width - before : p.chunks;
    const long long s = before < after ? before : after;
    int i = n++;
    for (; i > 0 && size[i - 1] < s; --i) {
      size[i] = size[i - 1];
      order[i] = order[i - 1];
    }
    size[i] = s;
    order[i] = static_cast<uint8_t>(r);
  }
  return n;
}

struct DecayDevice {
  int *status = nullptr;
  int rc = MOE_ERR_CUDA;
};

// Per device, looked up once.
const DecayDevice &decay_device() {
  static DecayDevice devs[64];
  static std::once_flag once[64];
  static const DecayDevice none;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return none;
  std::call_once(once[dev], [dev] {
    devs[dev].status = noalloc_status_word();
    if (devs[dev].status && decay_chunk_setup()) devs[dev].rc = MOE_OK;
  });
  return devs[dev];
}

}  // namespace

extern "C" int gdn_decay_workspace(long long n_tokens, int n_seq, int ragged, int n_v_heads, int d_k,
                                   int d_v, size_t *bytes) {
  if (!bytes || n_tokens < 0 || n_seq < 0 || n_v_heads <= 0 || d_k <= 0 || d_v <= 0)
    return MOE_ERR_INVALID_ARG;
  // (how heads share keys, which the plan looks at, is not asked for here)
  *bytes = 0;
  for (int hk = 1; hk <= n_v_heads; ++hk) {
    if (n_v_heads % hk != 0) continue;
    const Plan p = make_plan(ragged != 0, n_tokens, n_seq, hk, n_v_heads * ceil_div(d_v, 128));
    const size_t need = workspace_bytes_of(p, d_k);
    if (need > *bytes) *bytes = need;
  }
  return MOE_OK;
}

extern "C" int gdn_decay_scan(const void *q, const void *k, const void *v, const float *decay,
                              const float *state_in, float *state_out, void *o, const int *offsets,
                              long long n_tokens, int n_seq, int n_k_heads, int n_v_heads, int d_k,
                              int d_v, long long q_stride, long long k_stride, long long v_stride,
                              void *workspace, size_t workspace_bytes, void *cuda_stream) {
  if (n_tokens < 0 || n_seq < 0 || n_k_heads <= 0 || n_v_heads <= 0 || d_k <= 0 || d_v <= 0)
    return MOE_ERR_INVALID_ARG;
  if (n_v_heads % n_k_heads != 0 || (n_seq == 0 && n_tokens > 0)) return MOE_ERR_INVALID_ARG;
  if (!offsets && n_seq > 0 && n_tokens % n_seq != 0) return MOE_ERR_INVALID_ARG;
  if (n_seq == 0) return MOE_OK;
  if (!decay || (n_tokens > 0 && (!q || !k || !v || !o))) return MOE_ERR_INVALID_ARG;
  if (q_stride < static_cast<long long>(n_k_heads) * d_k ||
      k_stride < static_cast<long long>(n_k_heads) * d_k ||
      v_stride < static_cast<long long>(n_v_heads) * d_v)
    return MOE_ERR_INVALID_ARG;
  if ((d_k != 64 && d_k != 128) || d_v % 16 != 0 || d_v > 1024 || n_v_heads > 4096 ||
      n_tokens > 0x7fffffffLL || std::max({q_stride, k_stride, v_stride}) >= 1LL << 39 ||
      static_cast<long long>(n_seq) * n_v_heads * (d_v / 16) > 0x7fffffffLL)
    return MOE_ERR_UNSUPPORTED;
  auto misaligned = [](const void *p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) % n) != 0;
  };
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || misaligned(state_in, 16) ||
      misaligned(state_out, 16) || misaligned(decay, 4) || misaligned(offsets, 4) ||
      misaligned(workspace, 16))
    return MOE_ERR_ALIGNMENT;
  DecayArgs a = {};
  a.tiles = (d_v + 127) / 128;
  a.group = n_v_heads / n_k_heads;
  a.bundle = a.group * a.tiles;
  const long long heads = static_cast<long long>(n_v_heads) * a.tiles;
  const Plan plan = make_plan(offsets != nullptr, n_tokens, n_seq, n_k_heads, heads);
  const size_t need = workspace_bytes_of(plan, d_k);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_INVALID_ARG;
  // (CTAs of the largest launch; chunks of all rows)
  if (plan.rows * plan.pitch > 1 << 30) return MOE_ERR_UNSUPPORTED;
  if (plan.items * heads * 8 > 0x7fffffffLL || (plan.shares + plan.rows * 8) * (heads / n_k_heads) > 0x7fffffffLL)
    return MOE_ERR_UNSUPPORTED;
  const DecayDevice &dev = decay_device();
  if (dev.rc != MOE_OK) return dev.rc;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.v = static_cast<const __nv_bfloat16 *>(v);
  a.decay = decay;
  a.s_in = state_in;
  a.s_out = state_out;
  a.o = static_cast<__nv_bfloat16 *>(o);
  a.offsets = offsets;
  a.n_tokens = n_tokens;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.n_seq = n_seq;
  a.Hk = n_k_heads;
  a.Hv = n_v_heads;
  a.dv = d_v;
  a.recur = static_cast<int>(kRecur);
  a.seg_len = static_cast<int>(plan.seg_len);
  a.cut_from = static_cast<int>(std::min(plan.cut_from, n_tokens));
  a.seq_len = static_cast<int>(n_tokens / n_seq);
  a.cuts = plan.cuts;
  a.items = plan.items;
  if (!offsets && plan.chunked) {
    a.chunks = static_cast<int>(plan.chunks);
    a.width = static_cast<int>(plan.width);
    a.shares = static_cast<int>(plan.shares);
    a.pitch = static_cast<int>(plan.pitch);
    a.smalls = small_pieces(plan, a.order);
  }
  a.table = plan.table ? static_cast<Segment *>(workspace) : nullptr;
  a.ws = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.table);
  a.status = dev.status;
  // the maps before the first launch: a call that fails has launched nothing
  CUtensorMap mq, mk, mv, mo;
  if (plan.chunked) {
    const uint64_t kw = static_cast<uint64_t>(n_k_heads) * d_k, vw = static_cast<uint64_t>(n_v_heads) * d_v;
    if (!encode_map_2d(&mq, q, 2, n_tokens, kw, 64, kChunkTok, true, 2 * q_stride) ||
        !encode_map_2d(&mk, k, 2, n_tokens, kw, 64, kChunkTok, true, 2 * k_stride) ||
        !encode_map_2d(&mv, v, 2, n_tokens, vw, 64, kChunkTok, true, 2 * v_stride) ||
        !encode_map_2d(&mo, o, 2, n_tokens, vw, 32, 32, false, 0, true))
      return MOE_ERR_CUDA;
  }
  cudaError_t e = cudaSuccess;
  if (plan.recurrent)
    e = d_k == 128 ? launch_recurrent<128>(a, st) : launch_recurrent<64>(a, st);
  if (e == cudaSuccess && plan.chunked)
    e = launch_decay_chunked(a, d_k, mq, mk, mv, mo, plan.segmented, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
