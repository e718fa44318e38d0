// decay_common.cuh -- what the kernels of gdn_decay_scan share: the call's
// arguments, the sequences, powers of a decay.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kChunkTok = 64;  // tokens per chunk of the chunked form
constexpr int kGpuSms = 152;   // (the plan is the host's alone and asks no device)

// One segment of a packed sequence that takes the chunked form.
struct alignas(16) Segment {
  int seq;         // -1: none
  int index;       // its place in the sequence
  int first, len;  // its tokens
  int last, pad[3];
};
static_assert(sizeof(Segment) == 32, "its first half is read as a vector");

struct DecayArgs {
  const __nv_bfloat16 *q, *k, *v;
  const float *decay, *s_in;
  float *s_out;
  __nv_bfloat16 *o;
  const int *offsets;  // null: n_seq sequences of n_tokens / n_seq tokens
  long long n_tokens, q_stride, k_stride, v_stride;
  int n_seq, Hk, Hv, dv;
  // Sequences of at most `recur` tokens take the recurrent kernel, the others
  // the chunked ones.  ws holds the states between segments, 128 x dk each (a
  // segment belongs to one tile of d_v), and that before a sequence's first
  // segment if the state is updated in place, since the last segment may write
  // it while the first is still to read it.
  int recur, seq_len;  // seq_len: of every sequence without offsets
  int tiles;           // 128-wide tiles of d_v
  int group, bundle;   // value heads of a key head, their tiles
  float *ws;
  int *status;
  // Without offsets: rows of `chunks` chunks, one per sequence and key head (the
  // value heads and tiles of a row, its bundle, are cut alike, so that CTAs that
  // run together read the same q and k), `pitch` chunks apart on a line that is
  // cut every `width` chunks into `shares`.
  int chunks, pitch, width, shares, smalls;
  uint8_t order[kGpuSms];  // rows whose end lies inside a share, by the share's smaller piece
  // With offsets: segments of seg_len tokens (a multiple of 64), if the longest
  // sequence has more than cut_from; else none is cut.
  int seg_len, cut_from;
  long long cuts, items;
  // [items], made by the call's recurrent kernel: first the segments of the
  // sequences that are cut, `cuts` at most, the only ones with states in ws;
  // then the sequences of one segment.
  Segment *table;
};

// What a CTA of the chunked kernels does.
struct Piece {
  int seq, h, d0;       // seq < 0: nothing
  int first, len;       // its tokens
  int from, to;         // states in ws before and after it; -1: the call's initial, final one
};

// first token and number of tokens of sequence i; offsets outside
// [0, n_tokens] or running backwards are clamped
__device__ __forceinline__ void seq_range(const DecayArgs &a, int i, long long &first,
                                          long long &len) {
  if (a.offsets) {
    const long long lo = min(max(static_cast<long long>(a.offsets[i]), 0LL), a.n_tokens);
    const long long hi = min(max(static_cast<long long>(a.offsets[i + 1]), lo), a.n_tokens);
    first = lo;
    len = hi - lo;
  } else {
    len = a.seq_len;
    first = len * i;
  }
}

// The table of a call with offsets, by one block: segments in order of their
// sequences.  All threads of the block call it.
__device__ __forceinline__ void make_table(const DecayArgs &a) {
  __shared__ int s_cut[32], s_whole[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = static_cast<int>(blockDim.x) >> 5;
  int longest = 0;
  if (a.cuts > 0) {
    for (int i = static_cast<int>(threadIdx.x); i < a.n_seq; i += static_cast<int>(blockDim.x)) {
      long long first, len;
      seq_range(a, i, first, len);
      longest = max(longest, static_cast<int>(len));
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) s_cut[warp] = longest;
    __syncthreads();
    for (int w = 0; w < nw; ++w) longest = max(longest, s_cut[w]);
    __syncthreads();
  }
  const int uncut = longest > a.cut_from ? a.seg_len : static_cast<int>(a.n_tokens);
  long long cuts = 0, wholes = a.cuts;  // the next free place of each part
  for (int i0 = 0; i0 < a.n_seq; i0 += static_cast<int>(blockDim.x)) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    long long first = 0, len = 0;
    int n = 0;
    if (i < a.n_seq) {
      seq_range(a, i, first, len);
      n = len <= a.recur ? 0 : len <= uncut ? 1 : (static_cast<int>(len) + a.seg_len - 1) / a.seg_len;
    }
    const int whole = n == 1 ? 1 : 0, cut = n > 1 ? n : 0;
    int inc = cut;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, whole);
    if (lane == 31) {
      s_cut[warp] = inc;
      s_whole[warp] = __popc(mask);
    }
    __syncthreads();
    // (a sequence has places in one part only)
    long long at = cuts + inc - cut, end = a.cuts;
    if (whole) {
      at = wholes + __popc(mask & ((1u << lane) - 1));
      end = a.items;
    }
    for (int w = 0; w < nw; ++w) {
      if (w < warp) at += whole ? s_whole[w] : s_cut[w];
      cuts += s_cut[w];
      wholes += s_whole[w];
    }
    // (offsets that overlap may ask for more places than there are)
    for (int k = 0; k < n && at + k < end; ++k) {
      Segment g = {};
      g.seq = i;
      g.index = k;
      g.first = static_cast<int>(first) + k * a.seg_len;
      g.last = k == n - 1;
      g.len = g.last ? static_cast<int>(len) - k * a.seg_len : a.seg_len;
      a.table[at + k] = g;
    }
    __syncthreads();
  }
  Segment none = {};
  none.seq = -1;
  for (long long k = cuts + threadIdx.x; k < a.cuts; k += blockDim.x) a.table[k] = none;
  for (long long k = wholes + threadIdx.x; k < a.items; k += blockDim.x) a.table[k] = none;
}

// The piece of CTA `block`: kOut: all of them, the larger one of each share
// before the smaller ones; otherwise those whose end state another one needs.
template <bool kOut>
__device__ __forceinline__ Piece find_piece(const DecayArgs &a, int block) {
  const bool in_place = a.s_in && a.s_in == a.s_out;
  Piece p;
  p.seq = -1;
  if (a.table) {
    const int per = a.Hv * a.tiles, item = block / per, ht = block % per;
    const int4 u = *reinterpret_cast<const int4 *>(a.table + item);
    const bool last = a.table[item].last;
    if (!kOut && (last || item + 1 >= a.cuts)) return p;
    p.seq = u.x;
    p.h = ht / a.tiles;
    p.d0 = ht % a.tiles * 128;
    p.first = u.z;
    p.len = u.w;
    p.from = u.y == 0 && (last || !in_place) ? -1 : item * per + ht;
    p.to = last ? -1 : (item + 1) * per + ht;
    return p;
  }
  // (fewer than 2^30 chunks in all rows: their q alone fills the device before;
  // few and 32-bit unsigned divisions, because a CTA starts with them)
  const unsigned bundle = a.bundle, b = static_cast<unsigned>(block) / bundle;
  const unsigned in = block - b * bundle, chunks = a.chunks, width = a.width, pitch = a.pitch;
  unsigned s = b, r, x, n;  // share, row, first chunk of it, chunks
  if (!kOut) {       // ends at cut b + 1
    const unsigned end = (b + 1) * width;
    r = (end - 1) / pitch;
    const unsigned y = end - r * pitch;
    if (y >= chunks) return p;
    x = y > width ? y - width : 0;
    n = y - x;
  } else {
    const bool small = b >= static_cast<unsigned>(a.shares);
    if (small) s = (a.order[b - a.shares] + 1) * pitch / width;
    r = s * width / pitch;
    x = s * width - r * pitch;
    n = min(width, chunks - x);
    // the share's chunks of the next row
    const unsigned end = (s + 1) * width, row = (r + 1) * pitch;
    const unsigned next = end > row && r + 1 < a.n_seq * static_cast<unsigned>(a.Hk) ? min(end - row, chunks) : 0;
    if ((next > n) != small) {
      ++r;
      x = 0;
      n = next;
    }
  }
  const unsigned seq = r / a.Hk, sub = a.tiles == 1 ? in : in / a.tiles;
  p.seq = seq;
  p.h = (r - seq * a.Hk) * a.group + sub;
  p.d0 = (in - sub * a.tiles) * 128;
  const int at = x * kChunkTok;
  p.first = p.seq * a.seq_len + at;
  p.len = min(static_cast<int>(n * kChunkTok), a.seq_len - at);
  const bool ends = x + n == chunks;
  // what does not start or end with its row does with the share
  p.to = ends ? -1 : static_cast<int>((s + 1) * bundle + in);
  p.from = x > 0                ? static_cast<int>(s * bundle + in)
           : ends || !in_place ? -1
                               : static_cast<int>((a.shares + r) * bundle + in);
  return p;
}

// lam^n for n >= 0 (0^0 = 1).  The exponent n log2(lam) is rounded once: a
// relative error of 2^-24 |n log2(lam)|, large only where the power is small.
__device__ __forceinline__ float decay_pow(float lam, float n) {
  return n == 0.0f ? 1.0f : lam == 0.0f ? 0.0f : exp2f(n * log2f(lam));
}

// Launch of a kernel that may start while the one before it ends (it waits for
// that one's results itself)
inline dim3 grid_of(long long n) { return dim3(static_cast<unsigned>(n)); }
template <typename K, typename... Args>
cudaError_t launch_pdl(K kern, dim3 grid, int threads, int smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// decay_chunk.cu
bool decay_chunk_setup();  // shared-memory attributes; once per device
cudaError_t launch_decay_chunked(const DecayArgs &a, int dk, const CUtensorMap &mq,
                                 const CUtensorMap &mk, const CUtensorMap &mv,
                                 const CUtensorMap &mo, bool segmented,
                                 cudaStream_t st);

}  // namespace moe
