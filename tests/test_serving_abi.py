"""The entry points around the verification refuse bad arguments before any CUDA call, and the
oracle of their tests agrees with closed forms and with the tree oracle on chains (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_tree_b200 as L
from linear_attention_tree_b200 import binding, serving
from linear_attention_tree_b200 import workloads as W
from oracle import oracle as O
from oracle import serving as OS

INVALID, UNSUPPORTED = binding.TV_ERR_INVALID_ARG, binding.TV_ERR_UNSUPPORTED
size = ctypes.c_size_t


def _ptrs(n, null=None, off=None, by=4):
    # fake device addresses: the call must fail before it dereferences anything
    p = [0x10000000 * (i + 1) for i in range(n)]
    if null is not None:
        p[null] = None
    if off is not None:
        p[off] += by
    return p


def _prefill(prob, ptrs, bytes_=256):
    return serving._library().tv_prefill(prob, *ptrs, size(bytes_), None)


def _sequence(**change):
    p = L.make_sequence_problem(4, 2, 128, 128, 64, 40, qk_heads=2)
    for name, value in change.items():
        setattr(p, name, value)
    return p


@pytest.mark.parametrize("change,expect", [
    ({"H": 0}, INVALID), ({"B": -1}, INVALID), ({"total_nodes": -1}, INVALID),
    ({"max_nodes": -1}, INVALID), ({"mode": 5}, INVALID), ({"in_dtype": 3}, INVALID),
    ({"out_dtype": 3}, INVALID), ({"kernel": 3}, INVALID), ({"dk": 0}, INVALID),
    ({"qk_heads": 3}, INVALID), ({"dk": 100}, UNSUPPORTED), ({"dv": 144}, UNSUPPORTED),
    ({"in_dtype": 0, "out_dtype": 1}, UNSUPPORTED), ({"B": 1 << 30}, UNSUPPORTED)])
def test_bad_sequence_problem(change, expect):
    prob = _sequence(**change)
    assert _prefill(prob, _ptrs(10)) == expect
    assert L.workspace_size(prob) == 0
    assert serving._library().tv_decode_step(prob, *_ptrs(8), None) == expect


@pytest.mark.parametrize("i", range(10))
def test_prefill_null_and_misaligned(i):
    if i != 6:                                      # S_in may be NULL
        assert _prefill(_sequence(), _ptrs(10, null=i)) == INVALID
    assert _prefill(_sequence(), _ptrs(10, off=i)) == INVALID


def test_prefill_refusals():
    assert _prefill(_sequence(), _ptrs(10), 8) == INVALID
    ptrs = _ptrs(10)
    ptrs[8] = ptrs[6] + 1024                        # S_out over a part of S_in
    assert _prefill(_sequence(), ptrs) == INVALID
    prob = L.make_sequence_problem(4, 2, 64, 128, 64, 40, kernel="tc")
    assert _prefill(prob, _ptrs(10)) == UNSUPPORTED
    # scalar decay: b may be NULL, not misaligned
    prob = _sequence(mode=1)
    assert _prefill(prob, _ptrs(10, off=4)) == INVALID


@pytest.mark.parametrize("i", range(8))
def test_decode_step_null_and_misaligned(i):
    prob = L.make_sequence_problem(4, 2, 128, 128, 4, 1)
    fn = serving._library().tv_decode_step
    assert fn(prob, *_ptrs(8, null=i), None) == INVALID
    assert fn(prob, *_ptrs(8, off=i), None) == INVALID


def test_decode_step_refusals():
    fn = serving._library().tv_decode_step
    assert fn(_sequence(), *_ptrs(8), None) == INVALID          # 64 rows, 4 sequences
    prob = L.make_sequence_problem(4, 2, 128, 128, 4, 1)
    ptrs = _ptrs(8)
    ptrs[7] = ptrs[5] + 256
    assert fn(prob, *ptrs, None) == INVALID
    assert fn(L.make_sequence_problem(0, 2, 128, 128, 0, 1), *[None] * 8, None) == binding.TV_OK


def _sample(prob, ptrs, bytes_=None):
    n = serving._library().tv_sample_workspace_size(prob) if bytes_ is None else bytes_
    return serving._library().tv_sample(prob, *ptrs, size(n), None)


@pytest.mark.parametrize("args,expect", [
    ((-1, 10), INVALID), ((3, 0), INVALID), ((3, 10, 9), INVALID), ((3, (1 << 20) + 1), UNSUPPORTED)])
def test_bad_sample_problem(args, expect):
    prob = L.make_sample_problem(*args)
    assert L.workspace_size(prob) == 0
    assert _sample(prob, _ptrs(9), 1 << 20) == expect


@pytest.mark.parametrize("i", range(9))
def test_sample_null_and_misaligned(i):
    prob = L.make_sample_problem(3, 100)
    if i in (0, 1, 6, 8):
        assert _sample(prob, _ptrs(9, null=i)) == INVALID
    assert _sample(prob, _ptrs(9, off=i, by=2)) == INVALID
    assert _sample(prob, _ptrs(9), 8) == INVALID


def _accept(prob, ptrs, bytes_=256):
    return serving._library().tv_tree_accept(prob, *ptrs, size(bytes_), None)


@pytest.mark.parametrize("i", range(9))
def test_accept_null_and_misaligned(i):
    prob = L.make_problem(4, 1, 16, 16, 64, 16, 4)
    assert _accept(prob, _ptrs(9, null=i)) == INVALID
    assert _accept(prob, _ptrs(9, off=i)) == INVALID


def test_accept_refusals():
    assert _accept(L.make_problem(4, 1, 16, 16, 64, 16, 0), _ptrs(9)) == INVALID
    assert _accept(L.make_problem(4, 1, 16, 16, 65, 16, 4), _ptrs(9)) == INVALID
    assert _accept(L.make_problem(4, 1, 16, 16, 64, 257, 4), _ptrs(9)) == UNSUPPORTED
    assert _accept(L.make_problem(4, 1, 16, 16, 64, 16, 4), _ptrs(9), 8) == INVALID


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 16)
    g = torch.zeros(4, 2)
    S = torch.zeros(4, 2, 16, 16)
    with pytest.raises(ValueError):
        L.decode_step(x, x, x, g, g, S)
    with pytest.raises(ValueError):
        L.prefill(x, x, x, g, g, torch.zeros(2, dtype=torch.int32), max_len=4)
    with pytest.raises(ValueError):
        L.sample(torch.zeros(2, 8), torch.zeros(2))
    with pytest.raises(TypeError):
        L.sample(None, torch.zeros(2))
    with pytest.raises(ValueError):
        L.sample(torch.zeros(8), torch.zeros(2))
    with pytest.raises(ValueError):
        i = torch.zeros(4, dtype=torch.int32)
        L.tree_accept(i, i, i, i, i, max_nodes=4, max_path=2)


@pytest.mark.parametrize("i", range(6))
def test_sizes_beyond_32_bits_are_refused(i):
    """Not cut to their low 32 bits, which would be a valid size here."""
    args = [4, 2, 128, 128, 64, 40]
    args[i] += 1 << 32
    with pytest.raises(ValueError):
        L.make_sequence_problem(*args)
    with pytest.raises(ValueError):
        serving._sequence_problem(*args, 1, 0, 1, 1, 0, 0, 2)
    with pytest.raises(ValueError):
        serving._tree_problem(*[n + (1 << 32) * (i % 4 == j) for j, n in enumerate((4, 64, 16, 4))])
    with pytest.raises(ValueError):
        L.make_sample_problem(*[n + (1 << 32) * (i % 2 == j) for j, n in enumerate((3, 100))])


# ---- the oracle itself ---------------------------------------------------------------------


@pytest.mark.parametrize("mode", ["gdn", "scalar"])
def test_prefill_oracle_is_the_tree_oracle_on_a_chain(mode):
    w = W.synthetic([np.arange(-1, 11)], H=2, dk=32, dv=16, seed=3, mode=mode)
    o, U = O.tree_verify(w)
    out, S = OS.prefill(w.q, w.k, w.v, w.log_a, w.b, [0, w.T], w.S_root, mode)
    assert np.allclose(out, o, rtol=0, atol=1e-12)
    want = np.stack([O.commit_sequence(w, 0, h, np.arange(12)) for h in range(2)])
    assert np.allclose(S[0], want, rtol=0, atol=1e-12)


def test_sample_oracle_closed_forms():
    x = np.zeros(1000)
    assert OS.sample_row(x, 0.5) == (500, np.log(1 / 1000))       # equal weights: exact borders
    assert OS.sample_row(x, 0.0)[0] == 0 and OS.sample_row(x, 1.0)[0] == 999
    assert OS.sample_row(x, 1.0, top_k=7)[0] == 6                 # ties go to the lowest index
    assert OS.sample_row(x, 1.0, top_p=0.5)[0] == 499
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    assert OS.sample_row(x, 0.99, top_p=0.5)[0] == 1              # 4/8 of the mass: one token
    assert OS.sample_row(x, 0.99, top_p=0.51)[0] == 2
    assert OS.sample_row(x, 0.99, top_k=3, top_p=0.9)[0] == 2     # 7 of mass: 4, 2, then 1
    assert OS.sample_row(x, 0.0, top_k=3, top_p=0.9)[0] == 0
    assert OS.sample_row(x, 0.99, min_p=0.3)[0] == 2
    assert OS.sample_row(x, 0.3, t=0.0) == (1, 0.0)
    assert OS.sample_row(np.full(4, -np.inf), 0.3) == (-1, -np.inf)


def test_accept_oracle_by_hand():
    parent = [-1, 0, 0, 1, 2]
    draft = [5, 7, 7, 9, 9]
    target = [7, 9, 1, 4, 1]
    path, n, nxt = OS.accept(draft, target, [5], parent, [0, 5], 4)
    assert path.tolist() == [[0, 1, 3, -1]] and n.tolist() == [3] and nxt.tolist() == [4]
    path, n, nxt = OS.accept(draft, target, [6], parent, [0, 5], 4)
    assert n.tolist() == [0] and nxt.tolist() == [6]
