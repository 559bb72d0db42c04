// Internal declarations of the operators around the tree verification: prompt prefill,
// single-token steps, sampling and tree acceptance (not installed).
#pragma once

#include "tv_internal.cuh"

namespace tv {

// A batch of token sequences through the recurrence.  T is the row count of q, k, v, out;
// offsets may end before it.  S_in may be NULL (zero states).
struct SequenceArgs {
  const void *q, *k, *v;
  const float *log_a, *b;
  const int32_t *offsets;
  const float *S_in;
  void *out;
  float *S_out;
  int *ws;
  int B, H, Hk, dk, dv, T, max_len;
};

struct SampleArgs {
  const void *logits;
  long long stride;              // elements from row to row
  const float *uniform, *temperature, *top_p, *min_p;   // the last three may be NULL
  const int32_t *top_k;          // may be NULL
  int32_t *token;
  float *logprob;                // may be NULL
  int *ws;
  int R, V;
};

struct AcceptArgs {
  const int32_t *draft, *target, *root, *parent, *node_offsets;
  int32_t *path, *count, *next;
  int *ws;
  int B, T, max_nodes, max_path;
};

// Node or token range of sequence s; false if it is not inside [0, T] or too long.
__device__ __forceinline__ bool sequence_range(const int32_t *offsets, int s, int T, int max_len,
                                               int &lo, int &n) {
  lo = offsets[s];
  const int hi = offsets[s + 1];
  n = hi - lo;
  return lo >= 0 && hi >= lo && hi <= T && n <= max_len;
}

// Whether no offset up to sequence s is larger than its start, as far as threads tid, tid + step, ...
// see: sequences then never share rows or a place in the workspace.
__device__ __forceinline__ bool sequence_rises(const int32_t *offsets, int s, int lo, int tid, int step) {
  bool ok = true;
  for (int i = tid; i < s; i += step) ok &= offsets[i] <= lo;
  return ok;
}

cudaError_t launch_prefill_simt(const SequenceArgs &a, int mode, int in_dtype, int out_dtype,
                                cudaStream_t st);
size_t prefill_tc_workspace(long long T, long long B, long long H, int mode);
cudaError_t launch_prefill_prepare(const SequenceArgs &a, int mode, cudaStream_t st);
cudaError_t launch_prefill_tc(const SequenceArgs &a, int mode, int out_dtype, cudaStream_t st);
cudaError_t launch_decode_step(const SequenceArgs &a, int mode, int in_dtype, int out_dtype,
                               cudaStream_t st);
cudaError_t launch_sample(const SampleArgs &a, int in_dtype, cudaStream_t st);
cudaError_t launch_accept(const AcceptArgs &a, cudaStream_t st);

}  // namespace tv
