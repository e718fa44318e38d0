// decay_common.cuh -- what the kernels of gdn_decay_scan share: the call's
// arguments, the sequences, powers of a decay.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kChunkTok = 64;  // tokens per chunk of the chunked form

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

// lam^n for n >= 0 (0^0 = 1).  The exponent n log2(lam) is rounded once: a
// relative error of 2^-24 |n log2(lam)|, large only where the power is small.
__device__ __forceinline__ float decay_pow(float lam, float n) {
  return n == 0.0f ? 1.0f : lam == 0.0f ? 0.0f : exp2f(n * log2f(lam));
}

// decay_chunk.cu
bool decay_chunk_setup();  // shared-memory attributes; once per device
cudaError_t launch_decay_chunked(const DecayArgs &a, int dk, const CUtensorMap &mq,
                                 const CUtensorMap &mk, const CUtensorMap &mv, bool segmented,
                                 cudaStream_t st);

}  // namespace moe
