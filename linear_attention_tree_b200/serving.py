"""The operators around the tree verification: prompts, single tokens, sampling, acceptance.

Argument marshalling only, as in `binding`.  A decode loop is `prefill` (the prompt's state),
then per step `tree_verify`, the model's logits, `sample` (one target token per node),
`tree_accept` and `tree_commit`; `decode_step` takes the place of a tree for sequences without
a draft.

Tensors may live on another device than the current one.  Outputs and workspaces that are not
given are allocated on the call's stream (``stream``, or the device's current one).

Python name  -> C entry point
  prefill         tv_prefill
  decode_step     tv_decode_step
  sample          tv_sample
  tree_accept     tv_tree_accept
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding
from .binding import DTYPE, KERNEL, MODE, Problem, TreeVerifyError, TV_ERR_INVALID_ARG, make_problem

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_FLOATS = (_F32, _BF16)


class SequenceProblem(Problem):
    """A batch of token sequences (`prefill`, `decode_step`)."""


class SampleProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("row_stride", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


_lib = None


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = binding.lib()
        vp, P, S = ctypes.c_void_p, ctypes.POINTER(Problem), ctypes.POINTER(SampleProblem)
        size = ctypes.c_size_t
        L.tv_prefill_workspace_size.argtypes, L.tv_prefill_workspace_size.restype = [P], size
        L.tv_sample_workspace_size.argtypes, L.tv_sample_workspace_size.restype = [S], size
        L.tv_prefill.argtypes = [P] + [vp] * 10 + [size, vp]
        L.tv_decode_step.argtypes = [P] + [vp] * 9
        L.tv_sample.argtypes = [S] + [vp] * 9 + [size, vp]
        L.tv_tree_accept.argtypes = [P] + [vp] * 9 + [size, vp]
        _lib = L
    return _lib


def make_sequence_problem(B, H, dk, dv, total_tokens, max_len, mode="gdn", in_dtype=_BF16,
                          out_dtype=None, kernel="auto", qk_heads=0) -> SequenceProblem:
    """``max_len``: upper bound on any sequence's length; ``qk_heads``: 0 = H."""
    return SequenceProblem(B, H, dk, dv, total_tokens, max_len, 1, MODE[mode], DTYPE[in_dtype],
                           DTYPE[out_dtype or in_dtype], KERNEL[kernel], 0, qk_heads)


def make_sample_problem(rows, vocab, row_stride=None, in_dtype=_F32) -> SampleProblem:
    return SampleProblem(rows, vocab, vocab if row_stride is None else row_stride,
                         DTYPE[in_dtype], 0)


def workspace_size(problem) -> int:
    """Bytes of device workspace for a problem of any kind (0 if it is invalid)."""
    L = _library()
    if isinstance(problem, SampleProblem):
        return int(L.tv_sample_workspace_size(ctypes.byref(problem)))
    if isinstance(problem, SequenceProblem):
        return int(L.tv_prefill_workspace_size(ctypes.byref(problem)))
    return binding.workspace_size(problem)


def new_workspace(problem, device=None) -> torch.Tensor:
    """Zero-filled device workspace for a problem of any kind (the status word starts clear)."""
    n = workspace_size(problem)
    if n == 0:
        raise TreeVerifyError(TV_ERR_INVALID_ARG, "workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _arr(t, name, dtype, shape, device):
    """Address of a contiguous array of the given shape (None stays None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name} must live on the CUDA device of the call")
    if t.dtype is not dtype and not (type(dtype) is tuple and t.dtype in dtype):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected {n}")
    return t.shape


class _Call:
    """The device and stream of a call: entered, it makes them current, so that what is
    allocated inside belongs to the stream."""

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError("the arguments must live on a CUDA device")
        if stream is not None and stream.device != device:
            raise ValueError("the stream belongs to another device than the arguments")
        here = device.index == torch.cuda.current_device()
        self.context = contextlib.nullcontext() if here and stream is None else \
            torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(device))
        self.raw = (stream or torch.cuda.current_stream(device)).cuda_stream

    def __enter__(self):
        self.context.__enter__()
        return self.raw

    def __exit__(self, *exc):
        return self.context.__exit__(*exc)


def _sequence_call(q, k, v, mode, out, out_dtype):
    T, Hk, dk = _dims(q, "q", 3)
    _, H, dv = _dims(v, "v", 3)
    if mode not in MODE:
        raise ValueError(f"mode is {mode!r}, expected one of {tuple(MODE)}")
    if q.dtype not in DTYPE:
        raise TypeError(f"q has dtype {q.dtype}, expected {_FLOATS}")
    return T, Hk, dk, H, dv, (out.dtype if out is not None else out_dtype or q.dtype)


def prefill(q, k, v, log_a, b, seq_offsets, S_in=None, *, max_len: int, mode: str = "gdn",
            out=None, S_out=None, out_dtype=None, workspace=None, kernel: str = "auto",
            stream=None):
    """The recurrence over whole prompts; returns (out [T][H][dv], S_out [B][H][dv][dk] fp32).

    q, k [T][Hk][dk]; v [T][H][dv] (fp32 or bf16); log_a, b [T][H] fp32 (b may be None in
    scalar mode); seq_offsets [B+1] int32: sequence s owns rows seq_offsets[s] to
    seq_offsets[s+1] - 1, rows behind the last one are left as they were; S_in [B][H][dv][dk]
    fp32 or None (zero states); ``S_out`` may be ``S_in`` itself.  ``max_len`` bounds every
    sequence's length.
    """
    T, Hk, dk, H, dv, odt = _sequence_call(q, k, v, mode, out, out_dtype)
    B = _dims(seq_offsets, "seq_offsets", 1)[0] - 1
    dev = q.device
    with _Call(dev, stream) as raw:
        prob = make_sequence_problem(B, H, dk, dv, T, max_len, mode, q.dtype, odt, kernel, Hk)
        if out is None:
            out = torch.empty((T, H, dv), dtype=odt, device=dev)
        if S_out is None:
            S_out = torch.empty((B, H, dv, dk), dtype=_F32, device=dev)
        if workspace is None:
            workspace = new_workspace(prob, dev)
        st = _library().tv_prefill(
            prob, _arr(q, "q", _FLOATS, (T, Hk, dk), dev), _arr(k, "k", q.dtype, (T, Hk, dk), dev),
            _arr(v, "v", q.dtype, (T, H, dv), dev), _arr(log_a, "log_a", _F32, (T, H), dev),
            _arr(b, "b", _F32, (T, H), dev), _arr(seq_offsets, "seq_offsets", _I32, (B + 1,), dev),
            _arr(S_in, "S_in", _F32, (B, H, dv, dk), dev), _arr(out, "out", _FLOATS, (T, H, dv), dev),
            _arr(S_out, "S_out", _F32, (B, H, dv, dk), dev),
            _arr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), raw)
    if st:
        raise TreeVerifyError(st, "tv_prefill")
    return out, S_out


def decode_step(q, k, v, log_a, b, S, *, mode: str = "gdn", out=None, S_new=None, out_dtype=None,
                stream=None):
    """The recurrence for one token of every sequence; returns (out [B][H][dv], S_new).

    q, k [B][Hk][dk]; v [B][H][dv] (fp32 or bf16); log_a, b [B][H] fp32 (b may be None in
    scalar mode); S [B][H][dv][dk] fp32; ``S_new`` may be ``S`` itself (in place).
    """
    B, Hk, dk, H, dv, odt = _sequence_call(q, k, v, mode, out, out_dtype)
    dev = q.device
    with _Call(dev, stream) as raw:
        prob = make_sequence_problem(B, H, dk, dv, B, 1, mode, q.dtype, odt, "auto", Hk)
        if out is None:
            out = torch.empty((B, H, dv), dtype=odt, device=dev)
        if S_new is None:
            S_new = torch.empty((B, H, dv, dk), dtype=_F32, device=dev)
        st = _library().tv_decode_step(
            prob, _arr(q, "q", _FLOATS, (B, Hk, dk), dev), _arr(k, "k", q.dtype, (B, Hk, dk), dev),
            _arr(v, "v", q.dtype, (B, H, dv), dev), _arr(log_a, "log_a", _F32, (B, H), dev),
            _arr(b, "b", _F32, (B, H), dev), _arr(S, "S", _F32, (B, H, dv, dk), dev),
            _arr(out, "out", _FLOATS, (B, H, dv), dev),
            _arr(S_new, "S_new", _F32, (B, H, dv, dk), dev), raw)
    if st:
        raise TreeVerifyError(st, "tv_decode_step")
    return out, S_new


def sample(logits, uniform, *, temperature=None, top_k=None, top_p=None, min_p=None, token=None,
           logprob=None, workspace=None, stream=None):
    """One token per row of logits; returns (token [R] int32, logprob [R] fp32).

    logits [R][V] (fp32 or bf16; rows may be strided, values of a row adjacent); uniform [R]
    fp32 in [0, 1]; temperature, top_p, min_p [R] fp32 and top_k [R] int32, each may be None
    (1, 1, 0, all).  The token is the first in vocabulary order whose cumulated kept weight
    exceeds uniform times the total; temperature 0 takes the largest logit.  A row that is
    -inf throughout gives -1.
    """
    R, V = _dims(logits, "logits", 2)
    dev = logits.device
    if logits.dtype not in DTYPE:
        raise TypeError(f"logits has dtype {logits.dtype}, expected {_FLOATS}")
    stride = logits.stride(0) if R > 1 else V
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("the values of a row of logits must be adjacent")
    with _Call(dev, stream) as raw:
        prob = SampleProblem(R, V, stride, DTYPE[logits.dtype], 0)
        if token is None:
            token = torch.empty(R, dtype=_I32, device=dev)
        if logprob is None:
            logprob = torch.empty(R, dtype=_F32, device=dev)
        if workspace is None:
            workspace = new_workspace(prob, dev)
        st = _library().tv_sample(
            prob, logits.data_ptr(), _arr(uniform, "uniform", _F32, (R,), dev),
            _arr(temperature, "temperature", _F32, (R,), dev), _arr(top_k, "top_k", _I32, (R,), dev),
            _arr(top_p, "top_p", _F32, (R,), dev), _arr(min_p, "min_p", _F32, (R,), dev),
            _arr(token, "token", _I32, (R,), dev), _arr(logprob, "logprob", _F32, (R,), dev),
            _arr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), raw)
    if st:
        raise TreeVerifyError(st, "tv_sample")
    return token, logprob


def tree_accept(draft_token, target_token, root_token, parent, node_offsets, *, max_nodes: int,
                max_path: int, accepted_path=None, accepted_len=None, next_token=None,
                workspace=None, stream=None):
    """The accepted path of every draft tree; returns (accepted_path [B][max_path],
    accepted_len [B], next_token [B]), all int32, the first as `tree_commit` takes it.

    draft_token, target_token, parent [T], root_token [B], node_offsets [B+1], all int32.
    From the root, the lowest-index child whose draft token equals the target token of the
    current node (root_token at first) is accepted; next_token is the last target token.
    """
    T = _dims(draft_token, "draft_token", 1)[0]
    B = _dims(node_offsets, "node_offsets", 1)[0] - 1
    dev = draft_token.device
    with _Call(dev, stream) as raw:
        prob = make_problem(B, 1, 16, 16, T, max_nodes, max_path)
        new = lambda t, shape: torch.empty(shape, dtype=_I32, device=dev) if t is None else t
        accepted_path = new(accepted_path, (B, max_path))
        accepted_len, next_token = new(accepted_len, B), new(next_token, B)
        if workspace is None:
            workspace = new_workspace(prob, dev)
        ints = lambda t, name, shape: _arr(t, name, _I32, shape, dev)
        st = _library().tv_tree_accept(
            prob, ints(draft_token, "draft_token", (T,)), ints(target_token, "target_token", (T,)),
            ints(root_token, "root_token", (B,)), ints(parent, "parent", (T,)),
            ints(node_offsets, "node_offsets", (B + 1,)),
            ints(accepted_path, "accepted_path", (B, max_path)),
            ints(accepted_len, "accepted_len", (B,)), ints(next_token, "next_token", (B,)),
            _arr(workspace, "workspace", torch.uint8, None, dev), workspace.numel(), raw)
    if st:
        raise TreeVerifyError(st, "tv_tree_accept")
    return accepted_path, accepted_len, next_token
