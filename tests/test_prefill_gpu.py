"""Prompts and single tokens through the recurrence against 64 bits, token by token.

Tolerances.  A token's step rounds each value of S about four times (the decay, its product,
the update) and u by a dot product of 128 terms (depth 22 in the kernels' order); roundings are
of either sign, so a step adds about (sqrt(22) + 4) 2^-24 < 9 * 2^-24 of the state's norm, and
n of them sqrt(n) times that.  A step back of 100 tokens has decayed to e^-2, so n <= 100:
    tol(T) = 9 sqrt(min(T, 100)) 2^-24        (2-norm of the error over 2-norm of the result)
for states, and for out in fp32 5 * 2^-24 more (its own dot product).  out in bf16 adds one
rounding of up to 2^-8 of each value; its 2-norm stays under 2^-8 with as much again, of random
sign, for a bf16 operand in a matrix product before it.  The tensor-core kernel rounds per chunk of
64 tokens what the other rounds per token, its products being exact to 2^-21, and is held to the same.
"""
import math

import numpy as np
import pytest
import torch

import linear_attention_tree_b200 as L
from oracle import serving as OS

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def tol(T, dtype=None):
    t = 9 * math.sqrt(min(max(T, 1), 100)) * 2.0 ** -24
    if dtype is None:
        return t
    return t + 5 * 2.0 ** -24 if dtype is F32 else 2.0 ** -8


def inputs(lens, H, dk, dv, *, seed, Hk=None, dtype=BF16, mode="gdn", zero=False, log_a=-4.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, Hk = sum(lens), Hk or H
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda *s: torch.nn.functional.normalize(rnd(*s), dim=-1).to(dtype)
    d = {"q": unit(T, Hk, dk), "k": unit(T, Hk, dk), "v": rnd(T, H, dv).to(dtype),
         "log_a": -torch.nn.functional.softplus(log_a + 0.5 * rnd(T, H)),
         "b": torch.sigmoid(rnd(T, H)) if mode == "gdn" else None,
         "S": None if zero else 0.02 * rnd(len(lens), H, dv, dk)}
    d["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32,
                                device="cuda")
    return d


def recurrence(d, lens, mode):
    """64 bits on the GPU, one token of every sequence at a time."""
    H = d["v"].shape[1]
    rep = lambda x: x.double().repeat_interleave(H // x.shape[1], dim=1)
    q, k, v, a = rep(d["q"]), rep(d["k"]), d["v"].double(), d["log_a"].double().exp()
    dv, dk = v.shape[2], q.shape[2]
    out = torch.zeros_like(v)
    S = torch.zeros(len(lens), H, dv, dk, dtype=torch.float64, device="cuda")
    if d["S"] is not None:
        S += d["S"].double()
    off = d["offsets"].tolist()
    for s in range(len(lens)):
        X = S[s]
        for t in range(off[s], off[s + 1]):
            X = torch.where(a[t, :, None, None] > 0, X * a[t, :, None, None], 0.0)
            u = v[t]
            if mode == "gdn":
                u = d["b"][t].double()[:, None] * (u - (X @ k[t, :, :, None])[..., 0])
            X = X + u[:, :, None] * k[t, :, None, :]
            out[t] = (X @ q[t, :, :, None])[..., 0]
        S[s] = X
    return out, S


def check(got, want, bound, what, spread=8.0):
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all(), what
    norm = want.norm().item()
    err = (got - want).norm().item()
    assert err <= bound * norm, f"{what}: {err / max(norm, 1e-300):.3e} > {bound:.3e}"
    if want.numel():
        rms = norm / math.sqrt(want.numel())
        worst = ((got - want).abs() / want.abs().clamp(min=rms)).max().item()
        assert worst <= spread * bound, f"{what}: worst value {worst:.3e} > {spread * bound:.3e}"


def run_prefill(d, lens, mode, kernel="auto", out_dtype=None, **kw):
    ws = L.new_workspace(L.make_sequence_problem(
        len(lens), d["v"].shape[1], d["q"].shape[2], d["v"].shape[2], d["q"].shape[0], max(lens),
        mode, d["q"].dtype, kernel=kernel, qk_heads=d["q"].shape[1]))
    got = L.prefill(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], d["S"],
                    max_len=max(lens), mode=mode, kernel=kernel, out_dtype=out_dtype,
                    workspace=ws, **kw)
    assert L.get_status(ws) == 0
    return got


def compare(d, lens, mode, got, want=None):
    o, S = recurrence(d, lens, mode) if want is None else want
    n = max(lens)
    check(got[1], S, tol(n), "state")
    check(got[0], o, tol(n, got[0].dtype), "out")


def test_recurrence_is_the_oracle():
    lens = [5, 0, 9]
    d = inputs(lens, 4, 32, 16, seed=1, Hk=2)
    o, S = recurrence(d, lens, "gdn")
    h = {n: None if x is None else x.float().cpu().numpy() for n, x in d.items()}
    oo, So = OS.prefill(h["q"], h["k"], h["v"], h["log_a"], h["b"], d["offsets"].tolist(), h["S"])
    assert np.abs(o.cpu().numpy() - oo).max() < 1e-12
    assert np.abs(S.cpu().numpy() - So).max() < 1e-12


@pytest.mark.parametrize("mode", ["gdn", "scalar"])
@pytest.mark.parametrize("lens", [[1], [2], [16], [17], [63], [64], [65], [127], [128], [129],
                                  [0, 1, 0], [200, 3, 0, 64, 65]])
def test_lengths(mode, lens):
    d = inputs(lens, 2, 128, 128, seed=sum(lens), mode=mode)
    want = recurrence(d, lens, mode)
    for odt in (BF16, F32):
        for kernel in ("tc", "simt", "auto"):
            compare(d, lens, mode, run_prefill(d, lens, mode, kernel, odt), want)


@pytest.mark.parametrize("kernel", ["tc", "simt"])
@pytest.mark.parametrize("mode", ["gdn", "scalar"])
def test_rows_of_others_may_hold_anything(kernel, mode):
    """NaN and infinity in the rows before, between and behind: no sequence sees them."""
    lens = [70, 1, 64, 100]
    d = inputs(lens, 3, 128, 128, seed=41, mode=mode)
    want = recurrence(d, lens, mode)
    off = d["offsets"].tolist()
    for s in range(4):
        e = dict(d)
        for name in ("q", "k", "v", "log_a", "b"):
            if d[name] is not None:
                x = d[name].clone()
                x[:off[s]] = math.nan
                x[off[s + 1]:] = math.inf
                e[name] = torch.cat([x, torch.full_like(x, math.nan)])
        e["offsets"] = torch.tensor([off[s], off[s + 1]], dtype=torch.int32, device="cuda")
        e["S"] = d["S"][s:s + 1].contiguous()
        for odt in (BF16, F32):
            o, S = run_prefill(e, lens[s:s + 1], mode, kernel, odt)
            check(S, want[1][s:s + 1], tol(100), "state")
            check(o[off[s]:off[s + 1]], want[0][off[s]:off[s + 1]], tol(100, odt), "out")


@pytest.mark.parametrize("mode", ["gdn", "scalar"])
@pytest.mark.parametrize("n", [64, 130])
def test_equal_prompts_give_equal_bits(mode, n):
    """Thousands of chunks of the same tokens: every one has the first one's bits, whichever warp
    of its CTA comes first at each step."""
    B, H = 1200, 4
    d = inputs([n], H, 128, 128, seed=59, mode=mode, zero=True)
    want = recurrence(d, [n], mode)
    d["offsets"] = torch.arange(0, (B + 1) * n, n, dtype=torch.int32, device="cuda")
    for name in ("q", "k", "v", "log_a", "b"):
        if d[name] is not None:
            d[name] = d[name].repeat((B,) + (1,) * (d[name].dim() - 1))
    for _ in range(3):
        o, S = run_prefill(d, [n] * B, mode, "tc", F32)
        o = o.view(B, n, H, 128)
        assert (o == o[0]).all() and (S == S[0]).all()
        check(o[0], want[0], tol(n, F32), "out")
        check(S[:1], want[1], tol(n), "state")


@pytest.mark.parametrize("kernel", ["tc", "simt"])
def test_many_ragged_sequences(kernel):
    g = np.random.default_rng(5)
    lens = [int(n) for n in g.integers(0, 150, 61)]
    d = inputs(lens, 2, 128, 128, seed=43)
    compare(d, lens, "gdn", run_prefill(d, lens, "gdn", kernel, F32))


@pytest.mark.parametrize("kernel", ["tc", "simt"])
def test_offsets_that_do_not_rise(kernel):
    """Sequences that start before an earlier one ends are refused; the others are computed."""
    H, T = 2, 200
    d = inputs([T], H, 128, 128, seed=47)
    d["S"] = 0.02 * torch.randn(5, H, 128, 128, device="cuda")
    d["offsets"] = torch.tensor([0, 150, 40, 140, 150, 200], dtype=torch.int32, device="cuda")
    S = torch.full((5, H, 128, 128), math.nan, device="cuda")
    out = torch.full((T, H, 128), math.nan, dtype=BF16, device="cuda")
    ws = L.new_workspace(L.make_sequence_problem(5, H, 128, 128, T, T, kernel=kernel))
    L.prefill(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], d["S"], max_len=T, out=out,
              S_out=S, kernel=kernel, workspace=ws)
    assert L.get_status(ws) == L.binding.TV_ERR_BAD_TREE
    assert torch.isnan(S[1:4]).all()
    for s, lo, hi in ((0, 0, 150), (4, 150, 200)):
        e = {n: x[lo:hi] for n, x in d.items() if n in ("q", "k", "v", "log_a", "b")}
        e.update(offsets=torch.tensor([0, hi - lo], dtype=torch.int32), S=d["S"][s:s + 1])
        o, Sw = recurrence(e, [hi - lo], "gdn")
        check(S[s:s + 1], Sw, tol(150), "state")
        check(out[lo:hi], o, tol(150, BF16), "out")


@pytest.mark.parametrize("mode", ["gdn", "scalar"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (48, 80), (64, 48), (112, 32), (128, 128)])
def test_shapes(mode, dtype, dk, dv):
    lens = [37, 1, 50]
    d = inputs(lens, 4, dk, dv, seed=dk + dv, Hk=2, dtype=dtype, mode=mode)
    want = recurrence(d, lens, mode)
    compare(d, lens, mode, run_prefill(d, lens, mode), want)
    compare(d, lens, mode, run_prefill(d, lens, mode, kernel="simt"), want)


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 5), (3, 6), (7, 7)])
def test_shared_heads(Hk, H):
    lens = [90, 33]
    d = inputs(lens, H, 128, 128, seed=H, Hk=Hk)
    for kernel in ("tc", "simt"):
        compare(d, lens, "gdn", run_prefill(d, lens, "gdn", kernel, F32))


@pytest.mark.parametrize("mode", ["gdn", "scalar"])
def test_long_prompt(mode):
    lens = [2500]
    d = inputs(lens, 3, 128, 128, seed=7, mode=mode, zero=True)
    compare(d, lens, mode, run_prefill(d, lens, mode, out_dtype=F32))


@pytest.mark.parametrize("what", ["slow decay", "no decay", "fast decay", "repeated key", "b one"])
def test_values(what):
    """Gates at their ends and keys that repeat (the chunk's system at its least benign)."""
    lens = [150, 70]
    d = inputs(lens, 2, 128, 128, seed=11,
               log_a={"slow decay": -9.0, "fast decay": 4.0}.get(what, -4.0))
    if what == "no decay":
        d["log_a"].zero_()
    if what in ("repeated key", "b one"):
        d["b"].fill_(1.0)
    if what == "repeated key":
        d["k"][:] = d["k"][:1]
    for kernel in ("tc", "simt"):
        compare(d, lens, "gdn", run_prefill(d, lens, "gdn", kernel, F32))


@pytest.mark.parametrize("mode", ["gdn", "scalar"])
@pytest.mark.parametrize("repeated", [False, True])
def test_long_memory(mode, repeated):
    """4000 tokens without decay (of one key, b = 1): roundings of all of them add up, so the bound is
    tol's with n = 4000 tokens in place of 100."""
    T = 4000
    d = inputs([T], 2, 128, 128, seed=73, mode=mode)
    d["log_a"].zero_()
    if repeated:
        d["k"][:] = d["k"][:1]
        if mode == "gdn":
            d["b"].fill_(1.0)
    want = recurrence(d, [T], mode)
    bound = 9 * math.sqrt(T) * 2.0 ** -24
    for kernel in ("tc", "simt"):
        o, S = run_prefill(d, [T], mode, kernel, F32)
        check(S, want[1], bound, "state")
        check(o, want[0], bound + 5 * 2.0 ** -24, "out")


@pytest.mark.parametrize("kernel", ["tc", "simt"])
@pytest.mark.parametrize("mode", ["gdn", "scalar"])
@pytest.mark.parametrize("value", [-math.inf, -1e30, -3000.0, -80.0])
def test_reset(kernel, mode, value):
    """A decay of (nearly) zero starts the state afresh and spoils no later decay ratio."""
    lens = [140]
    d = inputs(lens, 2, 128, 128, seed=13, mode=mode)
    d["log_a"][[10, 64, 100, 139]] = value
    compare(d, lens, mode, run_prefill(d, lens, mode, kernel=kernel, out_dtype=F32))


@pytest.mark.parametrize("kernel", ["tc", "simt", "decode"])
@pytest.mark.parametrize("mode", ["gdn", "scalar"])
@pytest.mark.parametrize("value", [-math.inf, -200.0])
@pytest.mark.parametrize("held", [math.nan, math.inf])
def test_reset_of_a_recycled_state(kernel, mode, value, held):
    """A first decay of zero starts afresh from a state that holds anything, in place too."""
    lens = [1, 1, 1] if kernel == "decode" else [140, 3, 64]
    d = inputs(lens, 2, 128, 128, seed=71, mode=mode)
    d["log_a"][d["offsets"][:-1].long()] = value
    d["S"][:2] = held
    # (a decay that is zero in fp32 is zero; in 64 bits e^-200 would keep the NaN)
    zero = torch.where(d["log_a"].exp() == 0, -math.inf, d["log_a"])
    want = recurrence(dict(d, log_a=zero), lens, mode)
    if kernel == "decode":
        got = L.decode_step(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["S"], mode=mode,
                            S_new=d["S"], out_dtype=F32)
    else:
        got = run_prefill(d, lens, mode, kernel, F32, S_out=d["S"])
    check(got[1], want[1], tol(max(lens)), "state")
    check(got[0], want[0], tol(max(lens), F32), "out")


@pytest.mark.parametrize("mode", ["gdn", "scalar"])
def test_splitting_a_prompt(mode):
    """A prompt in two calls, the state carried (in place), is the prompt in one."""
    d = inputs([211], 3, 128, 128, seed=17, mode=mode)
    whole = run_prefill(d, [211], mode, out_dtype=F32)
    S = d["S"].clone()
    parts = []
    for lo, hi in ((0, 100), (100, 211)):
        off = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        cut = lambda x: None if x is None else x[lo:hi].clone()
        o, S2 = L.prefill(cut(d["q"]), cut(d["k"]), cut(d["v"]), cut(d["log_a"]), cut(d["b"]),
                          off, S, max_len=hi - lo, mode=mode, S_out=S, out_dtype=F32)
        assert S2 is S
        parts.append(o)
    check(torch.cat(parts), whole[0], 2 * tol(211, F32), "out")
    check(S, whole[1], 2 * tol(211), "state")


@pytest.mark.parametrize("kernel", ["tc", "simt"])
def test_nothing_else_is_written(kernel):
    """Guards around out and S_out, rows behind the last sequence, a sequence out of range."""
    H, G = 2, 2048
    lens = [65, 0, 30]
    T = 128
    d = inputs([T], H, 128, 128, seed=19)
    d["S"] = 0.02 * torch.randn(3, H, 128, 128, device="cuda")
    d["offsets"] = torch.tensor([0, 65, 65, 95], dtype=torch.int32, device="cuda")
    obuf = torch.full((2 * G + T * H * 128,), math.nan, dtype=BF16, device="cuda")
    sbuf = torch.full((2 * G + 3 * H * 128 * 128,), math.nan, device="cuda")
    out = obuf[G:-G].view(T, H, 128)
    S_out = sbuf[G:-G].view(3, H, 128, 128)
    L.prefill(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], d["S"], max_len=65,
              out=out, S_out=S_out, kernel=kernel)
    for g in (obuf[:G], obuf[-G:], sbuf[:G], sbuf[-G:], out[95:]):
        assert torch.isnan(g.float()).all()
    assert torch.equal(S_out[1], d["S"][1])
    compare(d, lens, "gdn", (out[:95], S_out),
            [x[:95] if i == 0 else x for i, x in enumerate(recurrence(d, lens, "gdn"))])
    # the middle sequence's range is bad: it alone is left as it was, and the status says so
    ws = L.new_workspace(L.make_sequence_problem(3, H, 128, 128, T, 65, kernel=kernel))
    for bad in ([0, 65, 300, 95], [0, 40, 20, 20], [-1, 40, 40, 40]):
        out.fill_(math.nan)
        S_out.fill_(math.nan)
        d["offsets"].copy_(torch.tensor(bad, dtype=torch.int32))
        L.prefill(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], d["S"], max_len=65,
                  out=out, S_out=S_out, kernel=kernel, workspace=ws)
        assert L.get_status(ws) == L.binding.TV_ERR_BAD_TREE
        bad_seq = 0 if bad[0] < 0 else 1
        assert torch.isnan(S_out[bad_seq]).all()
        assert not torch.isnan(S_out[(bad_seq + 1) % 2]).any() or bad[2] == 300
        for g in (obuf[:G], obuf[-G:], sbuf[:G], sbuf[-G:]):
            assert torch.isnan(g.float()).all()
    # longer than max_len
    d["offsets"].copy_(torch.tensor([0, 66, 66, 66], dtype=torch.int32))
    L.prefill(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], d["S"], max_len=65,
              out=out, S_out=S_out, kernel=kernel, workspace=ws)
    assert L.get_status(ws) == L.binding.TV_ERR_BAD_TREE


@pytest.mark.parametrize("kernel", ["tc", "simt"])
@pytest.mark.parametrize("mode", ["gdn", "scalar"])
@pytest.mark.parametrize("offsets,max_len,good", [
    ([0, 65, 300, 95], 65, [0]),            # past the rows; the third starts behind its end
    ([0, 65, 300, 95], 128, [0]),
    ([0, 40, 20, 20], 65, [0]),             # ends before it starts; an end before the first's
    ([-1, 40, 40, 40], 65, [1, 2]),
    ([0, 66, 66, 66], 65, [1, 2]),          # longer than max_len
    ([0, 66, 100, 128], 65, [1, 2]),
    ([30, 30, 95, 129], 128, [0, 1]),       # rows before the first, one row too many
    ([128, 128, 128, 128], 1, [0, 1, 2]),
    ([0, 2 ** 31 - 1, -2 ** 31, 5], 128, [])])
def test_good_sequences_beside_bad_ones(kernel, mode, offsets, max_len, good):
    """Every sequence that the offsets define is computed; nothing else is written."""
    H, T = 2, 128
    d = inputs([T], H, 128, 128, seed=79, mode=mode)
    d["S"] = 0.02 * torch.randn(3, H, 128, 128, device="cuda",
                                generator=torch.Generator("cuda").manual_seed(79))
    d["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out = torch.full((T, H, 128), math.nan, device="cuda")
    S = torch.full((3, H, 128, 128), math.nan, device="cuda")
    ws = L.new_workspace(L.make_sequence_problem(3, H, 128, 128, T, max_len, mode, kernel=kernel))
    L.prefill(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], d["S"], max_len=max_len,
              mode=mode, out=out, S_out=S, kernel=kernel, workspace=ws)
    assert L.get_status(ws) == (0 if len(good) == 3 else L.binding.TV_ERR_BAD_TREE)
    rows = torch.zeros(T, dtype=torch.bool, device="cuda")
    for s in range(3):
        if s not in good:
            assert torch.isnan(S[s]).all()
            continue
        lo, hi = offsets[s], offsets[s + 1]
        rows[lo:hi] = True
        e = {n: None if d[n] is None else d[n][lo:hi] for n in ("q", "k", "v", "log_a", "b")}
        e.update(offsets=torch.tensor([0, hi - lo]), S=d["S"][s:s + 1])
        o, Sw = recurrence(e, [hi - lo], mode)
        check(S[s:s + 1], Sw, tol(hi - lo), "state")
        check(out[lo:hi], o, tol(hi - lo, F32), "out")
    assert torch.isnan(out[~rows]).all()


@pytest.mark.parametrize("kernel", ["tc", "simt"])
@pytest.mark.parametrize("mode", ["gdn", "scalar"])
@pytest.mark.parametrize("name", ["q", "k", "v", "log_a", "b"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_token_that_is_not_finite(kernel, mode, name, bad):
    """It spoils its own sequence and heads, from its token (by chunks: its chunk) on."""
    if name == "b" and mode == "scalar":
        pytest.skip("scalar decay has no b")
    lens, at = [200, 70], 100
    d = inputs(lens, 4, 128, 128, Hk=2, seed=61, mode=mode)
    want = run_prefill(d, lens, mode, kernel, F32)
    d[name] = d[name].clone()
    d[name][at, 1] = bad
    o, S = run_prefill(d, lens, mode, kernel, F32)
    heads = [2, 3] if name in ("q", "k") else [1]
    others = [h for h in range(4) if h not in heads]
    first = at // 64 * 64 if kernel == "tc" else at
    assert torch.equal(o[200:], want[0][200:]) and torch.equal(S[1], want[1][1])
    assert torch.equal(o[:, others], want[0][:, others])
    assert torch.equal(S[0, others], want[1][0, others])
    assert torch.equal(o[:first], want[0][:first])
    assert not torch.isfinite(o[at, heads]).any()
    if name == "q":
        assert torch.equal(o[:at], want[0][:at]) and torch.equal(o[at + 1:], want[0][at + 1:])
        assert torch.equal(S, want[1])
    else:
        assert not torch.isfinite(S[0, heads]).all(-1).all(-1).any()


def test_empty_calls():
    d = inputs([0, 0], 2, 128, 128, seed=3)
    o, S = L.prefill(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], d["S"], max_len=0)
    assert o.shape[0] == 0 and torch.equal(S, d["S"])
    o, S = L.prefill(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], None, max_len=0)
    assert not S.any()
    o, S = L.prefill(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"][:1], None, max_len=0)
    assert S.shape[0] == 0


@pytest.mark.parametrize("lens", [[300, 41], [20, 7]])
def test_streams_and_graphs(lens):
    """The same inputs on two streams at once, each with its own outputs, and captured."""
    d = inputs(lens, 4, 128, 128, seed=23)
    want = run_prefill(d, lens, "gdn")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    args = (d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], d["S"])
    got = [L.prefill(*args, max_len=max(lens), stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for o, S in got:                                   # deterministic bit for bit
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])
    ws = L.new_workspace(L.make_sequence_problem(len(lens), 4, 128, 128, sum(lens), max(lens)))
    graph = torch.cuda.CUDAGraph()
    S = d["S"].clone()
    out = torch.empty_like(want[0])
    with torch.cuda.graph(graph):
        L.prefill(*args[:6], S, max_len=max(lens), out=out, S_out=S, workspace=ws)
    S.copy_(d["S"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(S, want[1])


def test_rows_past_32_bits():
    """q, k, v and out of over 2^31 elements: the last sequence is computed where it lies."""
    H, T = 32, 530_000
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    n = 100
    d = inputs([n], H, 128, 128, seed=29)
    want = run_prefill(d, [n], "gdn")
    big = {}
    for name in ("q", "k", "v", "log_a", "b"):
        big[name] = torch.zeros((T,) + tuple(d[name].shape[1:]), dtype=d[name].dtype, device="cuda")
        big[name][T - n:] = d[name]
    out = torch.zeros_like(big["v"])
    off = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    _, S = L.prefill(big["q"], big["k"], big["v"], big["log_a"], big["b"], off, d["S"],
                     max_len=n, out=out)
    assert torch.equal(S, want[1]) and torch.equal(out[T - n:], want[0])
    assert not out[:T - n].any()


@pytest.mark.parametrize("kernel", ["tc", "simt", "decode"])
@pytest.mark.parametrize("mode", ["gdn", "scalar"])
def test_out_is_rounded_once(kernel, mode):
    """out in bf16 is out in fp32 rounded, bit for bit: its products are no coarser."""
    lens = [1] * 300 if kernel == "decode" else [300, 70, 1]
    d = inputs(lens, 4, 128, 128, seed=67, Hk=2, mode=mode)

    def run(odt):
        if kernel == "decode":
            return L.decode_step(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["S"], mode=mode,
                                 out_dtype=odt)
        return run_prefill(d, lens, mode, kernel, odt)
    (o16, S16), (o32, S32) = run(BF16), run(F32)
    assert torch.equal(o16, o32.to(BF16)) and torch.equal(S16, S32)


# ---- single tokens ---------------------------------------------------------------------------


@pytest.mark.parametrize("mode", ["gdn", "scalar"])
@pytest.mark.parametrize("dtype,odt", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (48, 80), (96, 112), (128, 128)])
def test_decode_step(mode, dtype, odt, dk, dv):
    B = 5
    d = inputs([1] * B, 6, dk, dv, seed=dk * dv, Hk=3, dtype=dtype, mode=mode)
    o, S = L.decode_step(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["S"], mode=mode,
                         out_dtype=odt)
    compare(d, [1] * B, mode, (o, S))


def test_decode_steps_follow_prefill_in_place():
    """Eight single-token steps in place are a prompt of eight tokens."""
    B, n = 3, 8
    d = inputs([n] * B, 4, 128, 128, seed=31)
    want = run_prefill(d, [n] * B, "gdn", kernel="simt", out_dtype=F32)
    S = d["S"].clone()
    at = lambda x, t: x[t::n].contiguous()
    for t in range(n):
        o, S2 = L.decode_step(at(d["q"], t), at(d["k"], t), at(d["v"], t), at(d["log_a"], t),
                              at(d["b"], t), S, S_new=S, out_dtype=F32)
        assert S2 is S
        check(o, at(want[0], t), 2 * tol(n, F32), f"out {t}")
    check(S, want[1], 2 * tol(n), "state")


def test_decode_step_resets_and_streams():
    d = inputs([1] * 4, 2, 128, 128, seed=37)
    d["log_a"][1] = -math.inf
    o, S = L.decode_step(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["S"], out_dtype=F32)
    compare(d, [1] * 4, "gdn", (o, S))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, S2 = L.decode_step(d["q"], d["k"], d["v"], d["log_a"], d["b"], d["S"], out_dtype=F32,
                           stream=s)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2)


def test_keyword_calls():
    d = inputs([5, 4], 2, 128, 128, seed=53)
    kw = {n: d[n] for n in ("q", "k", "v", "log_a", "b")}
    a = L.prefill(*kw.values(), d["offsets"], d["S"], max_len=5)
    b = L.prefill(seq_offsets=d["offsets"], S_in=d["S"], max_len=np.int64(5), **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = {n: x[:2].contiguous() for n, x in kw.items()}
    a, b = L.decode_step(*one.values(), d["S"]), L.decode_step(S=d["S"], **one)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals_by_the_binding():
    d = inputs([4], 2, 128, 128, seed=1)
    args = [d["q"], d["k"], d["v"], d["log_a"], d["b"], d["offsets"], d["S"]]
    for i, bad, error in ((1, d["k"].float(), TypeError), (3, d["log_a"].double(), TypeError),
                          (2, d["v"][:3], ValueError), (5, d["offsets"].long(), TypeError),
                          (6, d["S"].transpose(2, 3), ValueError), (0, d["q"].half(), TypeError)):
        with pytest.raises(error):
            L.prefill(*args[:i], bad, *args[i + 1:], max_len=4)
    with pytest.raises(L.TreeVerifyError):
        L.prefill(*args[:4], None, *args[5:], max_len=4)           # gdn needs b
    with pytest.raises(ValueError):
        L.prefill(*args, max_len=4, mode="other")
    with pytest.raises(L.TreeVerifyError):
        L.decode_step(*args[:5], d["S"].expand(4, 2, 128, 128).contiguous(), out_dtype=F32,
                      S_new=d["S"].new_empty(5 * 2 * 128 * 128)[1:1 + 4 * 2 * 128 * 128]
                      .view(4, 2, 128, 128))                        # misaligned
