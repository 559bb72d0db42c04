// C ABI entry points of the operators around the tree verification (prefill, single-token
// steps, sampling, tree acceptance): argument validation, kernel choice, launches.
#include "serving.cuh"

namespace {

using namespace tv;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// An array that is read or written: present and 16-byte aligned, unless it has no elements.
bool arr(const void *p, bool empty) { return empty || (p && aligned(p, 16)); }
bool opt(const void *p) { return aligned(p, 16); }

int heads_of(const tv_problem *p) { return p->qk_heads ? p->qk_heads : p->H; }

// The checks of a batch of token sequences: as for trees, without a bound on a sequence's
// length (kernels index with 64 bits).
tv_status check_sequence(const tv_problem *p) {
  if (!p) return TV_ERR_INVALID_ARG;
  if (p->B < 0 || p->H < 1 || p->total_nodes < 0 || p->max_nodes < 0) return TV_ERR_INVALID_ARG;
  if (p->mode != TV_MODE_GDN && p->mode != TV_MODE_SCALAR_DECAY) return TV_ERR_INVALID_ARG;
  if (p->in_dtype != TV_F32 && p->in_dtype != TV_BF16) return TV_ERR_INVALID_ARG;
  if (p->out_dtype != TV_F32 && p->out_dtype != TV_BF16) return TV_ERR_INVALID_ARG;
  if (p->kernel < TV_KERNEL_AUTO || p->kernel > TV_KERNEL_SIMT) return TV_ERR_INVALID_ARG;
  if (p->dk < 1 || p->dv < 1) return TV_ERR_INVALID_ARG;
  if (p->qk_heads < 0 || p->qk_heads > p->H || (p->qk_heads && p->H % p->qk_heads))
    return TV_ERR_INVALID_ARG;
  if (p->dk % 16 || p->dv % 16 || p->dk > 128 || p->dv > 128) return TV_ERR_UNSUPPORTED;
  if (p->in_dtype == TV_F32 && p->out_dtype == TV_BF16) return TV_ERR_UNSUPPORTED;
  // grids of up to 8 blocks for each (sequence, head)
  if ((long long)p->B * p->H > 0x7fffffffLL / 8) return TV_ERR_UNSUPPORTED;
  return TV_OK;
}

// Shapes of the tensor-core prefill, and whether it is the one that runs.
bool prefill_tc_takes(const tv_problem *p) {
  return p->in_dtype == TV_BF16 && p->dk == 128 && p->dv == 128 &&
         (p->total_nodes / 64 + (long long)p->B) * p->H <= 0x7fffffffLL;
}
// Token by token costs 0.21 us a token, or 7 ns for each (sequence, head) where those are more; by
// chunks 30 us and 3 to 5 us a chunk for each 148 of them.  Measured, us with inputs from HBM (token by
// token / by chunks, gated delta rule): 16 heads 29 / 36 at 96 tokens, 49 / 40 at 192, 64 / 46 at 256;
// 32 heads 27 / 32 at 64, 37 / 36 at 96; 128 (sequence, head) pairs 25 / 34 at 16 tokens, 39 / 36 at 32;
// 1024 pairs 135 / 124 at 16, 246 / 126 at 32, 470 / 132 at 64.
bool prefill_on_tc(const tv_problem *p) {
  if (p->total_nodes == 0 || p->B == 0 || p->kernel == TV_KERNEL_SIMT || !prefill_tc_takes(p)) return false;
  const long long len = p->max_nodes, pairs = (long long)p->B * p->H;
  return p->kernel == TV_KERNEL_TC || len >= 112 || (len >= 24 && len * pairs >= 80 * 32);
}

// S_out either is S_in or does not overlap it.
bool states_apart(const tv_problem *p, const float *S_in, const float *S_out) {
  const size_t bytes = (size_t)p->B * p->H * p->dv * p->dk * sizeof(float);
  const uintptr_t x = reinterpret_cast<uintptr_t>(S_in), y = reinterpret_cast<uintptr_t>(S_out);
  return !S_in || x == y || x + bytes <= y || y + bytes <= x;
}

SequenceArgs sequence_args(const tv_problem *p, const void *q, const void *k, const void *v,
                           const float *log_a, const float *b, const int32_t *offsets,
                           const float *S_in, void *out, float *S_out, void *workspace) {
  SequenceArgs a;
  a.q = q; a.k = k; a.v = v; a.log_a = log_a; a.b = b; a.offsets = offsets; a.S_in = S_in;
  a.out = out; a.S_out = S_out; a.ws = static_cast<int *>(workspace);
  a.B = p->B; a.H = p->H; a.Hk = heads_of(p); a.dk = p->dk; a.dv = p->dv;
  a.T = p->total_nodes; a.max_len = p->max_nodes;
  return a;
}

tv_status check_sample(const tv_sample_problem *p) {
  if (!p || p->rows < 0 || p->vocab < 1 || p->row_stride < p->vocab) return TV_ERR_INVALID_ARG;
  if (p->in_dtype != TV_F32 && p->in_dtype != TV_BF16) return TV_ERR_INVALID_ARG;
  if (p->vocab > 1 << 20) return TV_ERR_UNSUPPORTED;
  return TV_OK;
}

}  // namespace

extern "C" {

size_t tv_prefill_workspace_size(const tv_problem *p) {
  if (check_sequence(p) != TV_OK) return 0;
  return prefill_on_tc(p) ? prefill_tc_workspace(p->total_nodes, p->B, p->H, p->mode) : kWorkspaceBytes;
}

tv_status tv_prefill(const tv_problem *p, const void *q, const void *k, const void *v,
                     const float *log_a, const float *b, const int32_t *seq_offsets,
                     const float *S_in, void *out, float *S_out, void *workspace,
                     size_t workspace_bytes, tv_stream_t stream) {
  tv_status st = check_sequence(p);
  if (st != TV_OK) return st;
  const bool none = p->total_nodes == 0;
  if (!arr(q, none) || !arr(k, none) || !arr(v, none) || !arr(log_a, none) || !arr(out, none) ||
      !arr(seq_offsets, false) || !opt(S_in) || !arr(S_out, p->B == 0) || !arr(workspace, false))
    return TV_ERR_INVALID_ARG;
  if (p->mode == TV_MODE_GDN ? !arr(b, none) : !opt(b)) return TV_ERR_INVALID_ARG;
  if (!states_apart(p, S_in, S_out)) return TV_ERR_INVALID_ARG;
  if (p->kernel == TV_KERNEL_TC && !prefill_tc_takes(p)) return TV_ERR_UNSUPPORTED;
  if (workspace_bytes < tv_prefill_workspace_size(p)) return TV_ERR_INVALID_ARG;
  if (p->B == 0) return TV_OK;
  const SequenceArgs a = sequence_args(p, q, k, v, log_a, b, seq_offsets, S_in, out, S_out, workspace);
  if (prefill_on_tc(p))
    return record_cuda_error(
        launch_prefill_tc(a, p->mode, p->out_dtype, reinterpret_cast<cudaStream_t>(stream)));
  return record_cuda_error(launch_prefill_simt(a, p->mode, p->in_dtype, p->out_dtype,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

tv_status tv_decode_step(const tv_problem *p, const void *q, const void *k, const void *v,
                         const float *log_a, const float *b, const float *S, void *out,
                         float *S_new, tv_stream_t stream) {
  tv_status st = check_sequence(p);
  if (st != TV_OK) return st;
  if (p->total_nodes != p->B) return TV_ERR_INVALID_ARG;
  if (p->kernel == TV_KERNEL_TC) return TV_ERR_UNSUPPORTED;
  if (p->B == 0) return TV_OK;
  if (!arr(q, false) || !arr(k, false) || !arr(v, false) || !arr(log_a, false) || !arr(S, false) ||
      !arr(out, false) || !arr(S_new, false))
    return TV_ERR_INVALID_ARG;
  if (p->mode == TV_MODE_GDN ? !arr(b, false) : !opt(b)) return TV_ERR_INVALID_ARG;
  if (!states_apart(p, S, S_new)) return TV_ERR_INVALID_ARG;
  const SequenceArgs a = sequence_args(p, q, k, v, log_a, b, nullptr, S, out, S_new, nullptr);
  return record_cuda_error(launch_decode_step(a, p->mode, p->in_dtype, p->out_dtype,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

size_t tv_sample_workspace_size(const tv_sample_problem *p) {
  return check_sample(p) == TV_OK ? kWorkspaceBytes : 0;
}

tv_status tv_sample(const tv_sample_problem *p, const void *logits, const float *uniform,
                    const float *temperature, const int32_t *top_k, const float *top_p,
                    const float *min_p, int32_t *token, float *logprob, void *workspace,
                    size_t workspace_bytes, tv_stream_t stream) {
  tv_status st = check_sample(p);
  if (st != TV_OK) return st;
  if (p->rows == 0) return TV_OK;
  if (!logits || !aligned(logits, p->in_dtype == TV_BF16 ? 2 : 4) || !uniform || !token ||
      !aligned(uniform, 4) || !aligned(token, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(logprob, 4) ||
      !arr(workspace, false))
    return TV_ERR_INVALID_ARG;
  if (workspace_bytes < tv_sample_workspace_size(p)) return TV_ERR_INVALID_ARG;
  SampleArgs a;
  a.logits = logits; a.stride = p->row_stride; a.uniform = uniform; a.temperature = temperature;
  a.top_p = top_p; a.min_p = min_p; a.top_k = top_k; a.token = token; a.logprob = logprob;
  a.ws = static_cast<int *>(workspace); a.R = p->rows; a.V = p->vocab;
  return record_cuda_error(launch_sample(a, p->in_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

tv_status tv_tree_accept(const tv_problem *p, const int32_t *draft_token,
                         const int32_t *target_token, const int32_t *root_token,
                         const int32_t *parent, const int32_t *node_offsets,
                         int32_t *accepted_path, int32_t *accepted_len, int32_t *next_token,
                         void *workspace, size_t workspace_bytes, tv_stream_t stream) {
  const size_t need = tv_workspace_size(p);
  if (!need) {                            // tell what is invalid from what is unsupported
    return p && p->max_nodes > kMaxNodes ? TV_ERR_UNSUPPORTED : TV_ERR_INVALID_ARG;
  }
  if (p->max_path < 1) return TV_ERR_INVALID_ARG;
  const bool none = p->total_nodes == 0;
  if (!arr(draft_token, none) || !arr(target_token, none) || !arr(parent, none) ||
      !arr(node_offsets, false) || !arr(root_token, p->B == 0) ||
      !arr(accepted_path, p->B == 0) || !arr(accepted_len, p->B == 0) ||
      !arr(next_token, p->B == 0) || !arr(workspace, false) || workspace_bytes < need)
    return TV_ERR_INVALID_ARG;
  if (p->B == 0) return TV_OK;
  AcceptArgs a;
  a.draft = draft_token; a.target = target_token; a.root = root_token; a.parent = parent;
  a.node_offsets = node_offsets; a.path = accepted_path; a.count = accepted_len;
  a.next = next_token; a.ws = static_cast<int *>(workspace);
  a.B = p->B; a.T = p->total_nodes; a.max_nodes = p->max_nodes; a.max_path = p->max_path;
  return record_cuda_error(launch_accept(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
