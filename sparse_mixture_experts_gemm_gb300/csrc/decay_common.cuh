// decay_common.cuh -- what the kernels of gdn_decay_scan share: the call's
// arguments, the sequences, powers of a decay.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kChunkTok = 64;  // tokens per chunk of the chunked form

// One segment of a sequence that takes the chunked form.
struct alignas(16) Segment {
  int seq;         // -1: none
  int index;       // its place in the sequence
  int first, len;  // its tokens
  long long slot;  // of the state before it (index > 0); slot + 1: before the next one
  int last, pad;
};
static_assert(sizeof(Segment) == 32, "read as two vectors");

struct DecayArgs {
  const __nv_bfloat16 *q, *k, *v;
  const float *decay, *s_in;
  float *s_out;
  __nv_bfloat16 *o;
  const int *offsets;  // null: n_seq sequences of n_tokens / n_seq tokens
  long long n_tokens, q_stride, k_stride, v_stride;
  int n_seq, Hk, Hv, dv;
  // Sequences of at most `recur` tokens take the recurrent kernel, the others
  // the chunked ones, in segments of seg_len tokens (a multiple of 64); ws
  // holds the state before each segment but a sequence's first, `slots` of
  // them at most, [slot][Hv][dv][dk].
  int recur, seg_len, seq_len;  // seq_len: of every sequence without offsets
  long long slots, items;
  float *ws;
  Segment *table;  // [items], of a call with offsets (made by its recurrent kernel)
  int tiles;  // 128-wide tiles of d_v
  int *status;
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
  __shared__ int s_seg[32], s_seq[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = static_cast<int>(blockDim.x) >> 5;
  long long base = 0;  // segments and sequences before this block's worth
  int rank0 = 0;
  for (int i0 = 0; i0 < a.n_seq; i0 += static_cast<int>(blockDim.x)) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    long long first = 0, len = 0;
    int n = 0;
    if (i < a.n_seq) {
      seq_range(a, i, first, len);
      n = len <= a.recur ? 0 : (static_cast<int>(len) + a.seg_len - 1) / a.seg_len;
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const uint32_t mine = __ballot_sync(0xffffffffu, n > 0);
    if (lane == 31) s_seg[warp] = inc;
    if (lane == 0) s_seq[warp] = __popc(mine);
    __syncthreads();
    long long at = base + inc - n;
    int rank = rank0 + __popc(mine & ((1u << lane) - 1u));
    for (int w = 0; w < nw; ++w) {
      if (w < warp) {
        at += s_seg[w];
        rank += s_seq[w];
      }
      base += s_seg[w];
      rank0 += s_seq[w];
    }
    for (int k = 0; k < n && at + k < a.items; ++k) {
      Segment g;
      g.seq = i;
      g.index = k;
      g.first = static_cast<int>(first) + k * a.seg_len;
      g.last = k == n - 1;
      g.len = g.last ? static_cast<int>(len) - k * a.seg_len : a.seg_len;
      g.slot = at - rank + k - 1;  // each earlier sequence has one slot fewer than segments
      g.pad = 0;
      a.table[at + k] = g;
    }
    __syncthreads();
  }
  Segment none = {};
  none.seq = -1;
  for (long long k = base + threadIdx.x; k < a.items; k += blockDim.x) a.table[k] = none;
}

// The segment that work item `item` stands for.
__device__ __forceinline__ Segment find_segment(const DecayArgs &a, int item) {
  Segment g;
  if (a.table) {
    const int4 *t = reinterpret_cast<const int4 *>(a.table + item);
    const int4 u = t[0], v = t[1];
    g.seq = u.x;
    g.index = u.y;
    g.first = u.z;
    g.len = u.w;
    g.slot = static_cast<long long>(static_cast<unsigned long long>(static_cast<unsigned>(v.y)) << 32 |
                                    static_cast<unsigned>(v.x));
    g.last = v.z;
  } else {  // (fewer than 2^31 tokens, segments and items)
    const int n = (a.seq_len + a.seg_len - 1) / a.seg_len, seq = item / n;
    g.seq = seq < a.n_seq ? seq : -1;
    g.index = item - seq * n;
    const int at = g.index * a.seg_len;
    g.first = seq * a.seq_len + at;
    g.last = at + a.seg_len >= a.seq_len;
    g.len = g.last ? a.seq_len - at : a.seg_len;
    g.slot = static_cast<long long>(seq) * (n - 1) + g.index - 1;
  }
  g.pad = 0;
  return g;
}

// lam^n for n >= 0 (0^0 = 1).  The exponent n log2(lam) is rounded once: a
// relative error of 2^-24 |n log2(lam)|, large only where the power is small.
__device__ __forceinline__ float decay_pow(float lam, float n) {
  return n == 0.0f ? 1.0f : lam == 0.0f ? 0.0f : exp2f(n * log2f(lam));
}

// decay_chunk.cu
bool decay_chunk_setup();  // shared-memory attributes; once per device
cudaError_t launch_decay_chunked(const DecayArgs &a, int dk, const CUtensorMap &mq,
                                 const CUtensorMap &mk, const CUtensorMap &mv,
                                 const CUtensorMap &mo, bool segmented,
                                 cudaStream_t st);

}  // namespace moe
