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

import ctypes
import functools
import inspect

import torch

from . import binding
from .binding import DTYPE, KERNEL, MODE, Problem, TreeVerifyError, TV_ERR_INVALID_ARG, make_problem

# handle of a device's current stream, without making a Stream object of it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32


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


def _int32(*values):
    """The values, whole; ctypes would cut them to 32 bits without a word."""
    whole = [int(x) for x in values]
    if whole and (max(whole) > 0x7fffffff or min(whole) < -0x80000000):
        raise ValueError(f"a size or bound is beyond 32 bits: {whole}")
    return whole


@functools.lru_cache(maxsize=256)
def _sequence_problem(*fields) -> SequenceProblem:
    return SequenceProblem(*_int32(*fields))


def make_sequence_problem(B, H, dk, dv, total_tokens, max_len, mode="gdn", in_dtype=_BF16,
                          out_dtype=None, kernel="auto", qk_heads=0) -> SequenceProblem:
    """``max_len``: upper bound on any sequence's length; ``qk_heads``: 0 = H."""
    return SequenceProblem(*_int32(B, H, dk, dv, total_tokens, max_len, 1, MODE[mode],
                                   DTYPE[in_dtype], DTYPE[out_dtype or in_dtype], KERNEL[kernel],
                                   0, qk_heads))


def make_sample_problem(rows, vocab, row_stride=None, in_dtype=_F32) -> SampleProblem:
    rows, vocab = _int32(rows, vocab)
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


def _arr(t, name, dtype, shape, index):
    """Address of a contiguous array of the given dtype and shape on device `index` (None stays
    None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != index:
        raise ValueError(f"{name} must live on the CUDA device of the call")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected {n}")
    return t.shape


def _workspace(t, problem, device):
    """(address, bytes) of the workspace given, or of a new one (kept alive by the third)."""
    if t is None:
        t = new_workspace(problem, device)
    elif not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    return _arr(t, "workspace", torch.uint8, t.shape, device.index), t.numel(), t


def _on_stream(f):
    """Calls f with the call's stream handle as ``_raw``.  Where ``stream`` or the device of the
    first argument is not the current one, they are made current, so that what f allocates
    belongs to the stream."""
    name = next(iter(inspect.signature(f).parameters))

    @functools.wraps(f)
    def call(*args, stream=None, **kwargs):
        first = args[0] if args else kwargs.get(name)
        if not isinstance(first, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        index = first.get_device()
        if index < 0:
            raise ValueError(f"{name} must live on a CUDA device")
        if stream is None and index == torch.cuda.current_device():
            return f(*args, _raw=_raw_stream(index), **kwargs)
        if stream is None:
            stream = torch.cuda.current_stream(index)
        elif stream.device.index != index:
            raise ValueError("the stream belongs to another device than the arguments")
        with torch.cuda.stream(stream):
            return f(*args, _raw=stream.cuda_stream, **kwargs)
    return call


def _sequence_call(q, v, mode, out, out_dtype):
    T, Hk, dk = _dims(q, "q", 3)
    _, H, dv = _dims(v, "v", 3)
    if mode not in MODE:
        raise ValueError(f"mode is {mode!r}, expected one of {tuple(MODE)}")
    if out is not None:
        out_dtype = _dims(out, "out", 3) and out.dtype
    elif out_dtype is None:
        out_dtype = q.dtype
    for name, dtype in (("q", q.dtype), ("out", out_dtype)):
        if dtype not in DTYPE:
            raise TypeError(f"{name} has dtype {dtype}, expected {tuple(DTYPE)}")
    return T, Hk, dk, H, dv, out_dtype


@_on_stream
def prefill(q, k, v, log_a, b, seq_offsets, S_in=None, *, max_len: int, mode: str = "gdn",
            out=None, S_out=None, out_dtype=None, workspace=None, kernel: str = "auto",
            _raw=None):
    """The recurrence over whole prompts; returns (out [T][H][dv], S_out [B][H][dv][dk] fp32).

    q, k [T][Hk][dk]; v [T][H][dv] (fp32 or bf16); log_a, b [T][H] fp32 (b may be None in
    scalar mode); seq_offsets [B+1] int32: sequence s owns rows seq_offsets[s] to
    seq_offsets[s+1] - 1, rows behind the last one are left as they were; S_in [B][H][dv][dk]
    fp32 or None (zero states); ``S_out`` may be ``S_in`` itself.  ``max_len`` bounds every
    sequence's length.  ``stream``: a torch stream, the device's current one by default.
    """
    T, Hk, dk, H, dv, odt = _sequence_call(q, v, mode, out, out_dtype)
    B = _dims(seq_offsets, "seq_offsets", 1)[0] - 1
    dev, dt = q.device, q.dtype
    at = dev.index
    prob = _sequence_problem(B, H, dk, dv, T, int(max_len), 1, MODE[mode], DTYPE[dt], DTYPE[odt],
                             KERNEL[kernel], 0, Hk)
    if out is None:
        out = torch.empty_like(v) if odt is v.dtype else torch.empty_like(v, dtype=odt)
    if S_out is None:
        S_out = torch.empty((B, H, dv, dk), dtype=_F32, device=dev)
    ws, ws_bytes, _kept = _workspace(workspace, prob, dev)
    st = _library().tv_prefill(
        prob, _arr(q, "q", dt, (T, Hk, dk), at), _arr(k, "k", dt, (T, Hk, dk), at),
        _arr(v, "v", dt, (T, H, dv), at), _arr(log_a, "log_a", _F32, (T, H), at),
        _arr(b, "b", _F32, (T, H), at), _arr(seq_offsets, "seq_offsets", _I32, (B + 1,), at),
        _arr(S_in, "S_in", _F32, (B, H, dv, dk), at), _arr(out, "out", odt, (T, H, dv), at),
        _arr(S_out, "S_out", _F32, (B, H, dv, dk), at), ws, ws_bytes, _raw)
    if st:
        raise TreeVerifyError(st, "tv_prefill")
    return out, S_out


@_on_stream
def decode_step(q, k, v, log_a, b, S, *, mode: str = "gdn", out=None, S_new=None, out_dtype=None,
                _raw=None):
    """The recurrence for one token of every sequence; returns (out [B][H][dv], S_new).

    q, k [B][Hk][dk]; v [B][H][dv] (fp32 or bf16); log_a, b [B][H] fp32 (b may be None in
    scalar mode); S [B][H][dv][dk] fp32; ``S_new`` may be ``S`` itself (in place).
    ``stream``: a torch stream, the device's current one by default.
    """
    B, Hk, dk, H, dv, odt = _sequence_call(q, v, mode, out, out_dtype)
    dev, dt = q.device, q.dtype
    at = dev.index
    prob = _sequence_problem(B, H, dk, dv, B, 1, 1, MODE[mode], DTYPE[dt], DTYPE[odt], 0, 0, Hk)
    if out is None:
        out = torch.empty_like(v) if odt is v.dtype else torch.empty_like(v, dtype=odt)
    if S_new is None:
        S_new = torch.empty((B, H, dv, dk), dtype=_F32, device=dev)
    st = _library().tv_decode_step(
        prob, _arr(q, "q", dt, (B, Hk, dk), at), _arr(k, "k", dt, (B, Hk, dk), at),
        _arr(v, "v", dt, (B, H, dv), at), _arr(log_a, "log_a", _F32, (B, H), at),
        _arr(b, "b", _F32, (B, H), at), _arr(S, "S", _F32, (B, H, dv, dk), at),
        _arr(out, "out", odt, (B, H, dv), at), _arr(S_new, "S_new", _F32, (B, H, dv, dk), at), _raw)
    if st:
        raise TreeVerifyError(st, "tv_decode_step")
    return out, S_new


@_on_stream
def sample(logits, uniform, *, temperature=None, top_k=None, top_p=None, min_p=None, token=None,
           logprob=None, workspace=None, _raw=None):
    """One token per row of logits; returns (token [R] int32, logprob [R] fp32).

    logits [R][V] (fp32 or bf16; rows may be strided, values of a row adjacent); uniform [R]
    fp32 in [0, 1]; temperature, top_p, min_p [R] fp32 and top_k [R] int32, each may be None
    (1, 1, 0, all).  The token is the first in vocabulary order whose cumulated kept weight
    exceeds uniform times the total; temperature 0 takes the largest logit.  A row that is
    -inf throughout gives -1.  ``stream``: a torch stream, the device's current one by default.
    """
    R, V = _dims(logits, "logits", 2)
    if logits.dtype not in DTYPE:
        raise TypeError(f"logits has dtype {logits.dtype}, expected {tuple(DTYPE)}")
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("the values of a row of logits must be adjacent")
    if R > 0x7fffffff or V > 0x7fffffff:
        raise ValueError(f"logits have shape {tuple(logits.shape)}, beyond 32 bits")
    dev = logits.device
    at = dev.index
    prob = SampleProblem(R, V, logits.stride(0) if R > 1 else V, DTYPE[logits.dtype], 0)
    uniform_at = _arr(uniform, "uniform", _F32, (R,), at)
    if token is None:
        token = torch.empty_like(uniform, dtype=_I32)
    if logprob is None:
        logprob = torch.empty_like(uniform)
    ws, ws_bytes, _kept = _workspace(workspace, prob, dev)
    st = _library().tv_sample(
        prob, logits.data_ptr(), uniform_at,
        _arr(temperature, "temperature", _F32, (R,), at), _arr(top_k, "top_k", _I32, (R,), at),
        _arr(top_p, "top_p", _F32, (R,), at), _arr(min_p, "min_p", _F32, (R,), at),
        _arr(token, "token", _I32, (R,), at), _arr(logprob, "logprob", _F32, (R,), at),
        ws, ws_bytes, _raw)
    if st:
        raise TreeVerifyError(st, "tv_sample")
    return token, logprob


@functools.lru_cache(maxsize=256)
def _tree_problem(B, T, max_nodes, max_path) -> Problem:
    return make_problem(*_int32(B, 1, 16, 16, T, max_nodes, max_path))


@_on_stream
def tree_accept(draft_token, target_token, root_token, parent, node_offsets, *, max_nodes: int,
                max_path: int, accepted_path=None, accepted_len=None, next_token=None,
                workspace=None, _raw=None):
    """The accepted path of every draft tree; returns (accepted_path [B][max_path],
    accepted_len [B], next_token [B]), all int32, the first as `tree_commit` takes it.

    draft_token, target_token, parent [T], root_token [B], node_offsets [B+1], all int32.
    From the root, the lowest-index child whose draft token equals the target token of the
    current node (root_token at first) is accepted; next_token is the last target token.
    ``stream``: a torch stream, the device's current one by default.
    """
    T = _dims(draft_token, "draft_token", 1)[0]
    B = _dims(node_offsets, "node_offsets", 1)[0] - 1
    dev = draft_token.device
    at = dev.index
    prob = _tree_problem(B, T, int(max_nodes), int(max_path))
    if not isinstance(root_token, torch.Tensor):
        raise TypeError("root_token must be a torch.Tensor")
    if root_token.dtype is not _I32:
        raise TypeError(f"root_token has dtype {root_token.dtype}, expected {_I32}")
    if accepted_path is None:
        accepted_path = root_token.new_empty((B, max_path))
    if accepted_len is None:
        accepted_len = torch.empty_like(root_token)
    if next_token is None:
        next_token = torch.empty_like(root_token)
    ws, ws_bytes, _kept = _workspace(workspace, prob, dev)
    nodes, seqs = (T,), (B,)
    st = _library().tv_tree_accept(
        prob, _arr(draft_token, "draft_token", _I32, nodes, at),
        _arr(target_token, "target_token", _I32, nodes, at),
        _arr(root_token, "root_token", _I32, seqs, at), _arr(parent, "parent", _I32, nodes, at),
        _arr(node_offsets, "node_offsets", _I32, (B + 1,), at),
        _arr(accepted_path, "accepted_path", _I32, (B, max_path), at),
        _arr(accepted_len, "accepted_len", _I32, seqs, at),
        _arr(next_token, "next_token", _I32, seqs, at), ws, ws_bytes, _raw)
    if st:
        raise TreeVerifyError(st, "tv_tree_accept")
    return accepted_path, accepted_len, next_token
