"""B200 (sm_100a) draft-tree verification through a recurrent linear-attention layer.

`tree_verify` gives every node of a speculative draft tree the output the sequential
scalar-decay or gated-delta recurrence would produce along its root-to-node path, without
per-node state snapshots, and writes one pseudo-value row per node; `tree_commit` rebuilds
the accepted path's state from those pseudo-values.  `prefill` and `decode_step` run the same
recurrence over prompts and single tokens; `sample` and `tree_accept` turn a verified tree's
logits into the accepted path.  All are CUDA kernels behind the C
ABI of ``include/tree_verify.h``; this package is the Python binding over it.
"""
from .binding import (TreeVerifyError, get_status, lib, make_problem, snapshot_commit,
                      snapshot_verify, tree_commit, tree_commit_verify, tree_meta, tree_verify)
from .serving import (decode_step, make_sample_problem, make_sequence_problem, new_workspace,
                      prefill, sample, tree_accept, workspace_size)

__all__ = ["tree_verify", "tree_commit", "tree_commit_verify", "snapshot_verify",
           "snapshot_commit", "tree_meta", "prefill", "decode_step", "sample", "tree_accept",
           "get_status", "workspace_size", "new_workspace", "make_problem",
           "make_sequence_problem", "make_sample_problem", "lib", "TreeVerifyError"]
