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
  // the chunked ones, in segments of seg_len tokens (a multiple of 64), one per
  // work item.  ws holds the state before each item's segment, [item][Hv][dv][dk]
  // (before a sequence's first one only if the state is updated in place, since
  // the last segment may write it while the first is still to read it).
  int recur, seg_len, seq_len;  // seq_len: of every sequence without offsets
  long long items;
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
  __shared__ int s_seg[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = static_cast<int>(blockDim.x) >> 5;
  long long base = 0;  // segments before this block's worth of sequences
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
    if (lane == 31) s_seg[warp] = inc;
    __syncthreads();
    long long at = base + inc - n;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) at += s_seg[w];
      base += s_seg[w];
    }
    for (int k = 0; k < n && at + k < a.items; ++k) {
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
  for (long long k = base + threadIdx.x; k < a.items; k += blockDim.x) a.table[k] = none;
}

// The segment that work item `item` stands for.
__device__ __forceinline__ Segment find_segment(const DecayArgs &a, int item) {
  Segment g = {};
  if (a.table) {
    const int4 u = *reinterpret_cast<const int4 *>(a.table + item);
    g.seq = u.x;
    g.index = u.y;
    g.first = u.z;
    g.len = u.w;
    g.last = a.table[item].last;
  } else {  // (fewer than 2^31 tokens, segments and items)
    const int n = (a.seq_len + a.seg_len - 1) / a.seg_len, seq = item / n;
    g.seq = seq < a.n_seq ? seq : -1;
    g.index = item - seq * n;
    const int at = g.index * a.seg_len;
    g.first = seq * a.seq_len + at;
    g.last = at + a.seg_len >= a.seq_len;
    g.len = g.last ? a.seq_len - at : a.seg_len;
  }
  return g;
}

// lam^n for n >= 0 (0^0 = 1).  The exponent n log2(lam) is rounded once: a
// relative error of 2^-24 |n log2(lam)|, large only where the power is small.
__device__ __forceinline__ float decay_pow(float lam, float n) {
  return n == 0.0f ? 1.0f : lam == 0.0f ? 0.0f : exp2f(n * log2f(lam));
}

// Launch of a kernel that may start while the one before it ends (it waits for
// that one's results itself)
template <typename K, typename... Args>
cudaError_t launch_pdl(K kern, long long grid, int threads, int smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
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
