"""Sampling against a full sort of every row in 64 bits, and acceptance against a walk.

Tokens have to be equal.  Both sides sum weights in 64 bits (top-p's border in 2^-43 steps of
the largest weight on the GPU): over V tokens their sums differ by less than V * 2^-43 of the
total, so one of the some 1e4 random borders here is within that of its goal with a
probability below 1e-3 in all.  logprob is a logarithm in 64 bits rounded to fp32, of a
quotient that top-p's border leaves as it is: 2^-24 relative, and 2^-40 absolute for the sums.
"""
import math

import numpy as np
import pytest
import torch

import linear_attention_tree_b200 as L
from linear_attention_tree_b200 import workloads as W
from oracle import serving as OS

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


def logits(R, V, seed, dtype=F32, scale=2.0):
    g = np.random.default_rng(seed)
    return torch.from_numpy((scale * g.standard_normal((R, V))).astype(np.float32)).to(dtype).cuda()


def compare(x, u, **p):
    ws = L.new_workspace(L.make_sample_problem(*x.shape, in_dtype=x.dtype))
    dev = {k: None if a is None else torch.as_tensor(a).cuda() for k, a in p.items()}
    token, lp = L.sample(x, torch.as_tensor(u, dtype=F32).cuda(), workspace=ws, **dev)
    assert L.get_status(ws) == 0
    want, wlp = OS.sample(x.float().cpu().numpy(), np.float32(u), **p)
    got = token.cpu().numpy()
    assert np.array_equal(got, want), np.nonzero(got != want)[0][:10]
    lp = lp.cpu().numpy().astype(np.float64)
    fin = np.isfinite(wlp)
    assert np.array_equal(fin, np.isfinite(lp)) and np.all(lp[~fin] == -np.inf)
    assert np.all(np.abs(lp[fin] - wlp[fin]) <= 2.0 ** -24 * np.abs(wlp[fin]) + 2.0 ** -40)
    return got


def mixed(R, seed):
    g = np.random.default_rng(seed)
    f = lambda x: x.astype(np.float32)
    return {"temperature": f(np.where(g.random(R) < 0.1, 0.0, 0.3 + 1.5 * g.random(R))),
            "top_k": np.where(g.random(R) < 0.4, 0, g.integers(1, 60, R)).astype(np.int32),
            "top_p": f(np.where(g.random(R) < 0.3, 1.0, g.random(R))),
            "min_p": f(np.where(g.random(R) < 0.5, 0.0, 0.2 * g.random(R)))}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 511, 513, 1000, 4097, 50257])
def test_sizes(dtype, V):
    R = 40
    x, u = logits(R, V, V, dtype), np.random.default_rng(V).random(R)
    compare(x, u)
    compare(x, u, **mixed(R, V + 1))


@pytest.mark.parametrize("only", ["temperature", "top_k", "top_p", "min_p"])
def test_each_filter_alone(only):
    R, V = 64, 3001
    p = mixed(R, 5)
    compare(logits(R, V, 6), np.random.default_rng(7).random(R), **{only: p[only]})


@pytest.mark.parametrize("V", [100_003, 1 << 18, 1 << 20])
def test_large_vocabulary(V):
    R = 3
    compare(logits(R, V, 8), [0.1, 0.5, 0.99], **{k: a[:R] for k, a in mixed(64, 9).items()})
    compare(logits(R, V, 8), [0.1, 0.5, 0.999999])
    compare(logits(R, V, 8, scale=0.0), [0.25, 0.5, 0.75], top_p=np.float32([0.5, 0.25, 1.0]))


def test_ties():
    """Logits on a grid of halves: most borders fall among equals, which go by index."""
    R, V = 200, 700
    x = (logits(R, V, 10) * 2).round() / 2
    u = np.random.default_rng(11).random(R)
    compare(x, u, **mixed(R, 12))
    compare(x, u, top_k=np.arange(1, R + 1, dtype=np.int32))
    compare(x.to(BF16), u, **mixed(R, 13))
    z = torch.zeros(6, 1000, device="cuda")
    z[:, 500:] = -0.0                              # equal to +0
    assert compare(z, [0.0, 0.5, 1.0, 0.5, 0.0, 0.999])[1] == 500
    compare(z, [0.0, 0.5, 1.0, 0.5, 0.0, 0.999], top_p=np.float32([0.5] * 6))
    compare(z, [0.0, 0.5, 1.0, 0.5, 0.0, 0.999], top_k=np.int32([501, 7, 1, 999, 1000, 2000]))


@pytest.mark.parametrize("scale,shift", [(0.01, 0.0), (1.0, 0.0), (6.0, 3.0), (1e-3, 0.0), (80.0, 0.0),
                                         (3.0, 300.0), (3.0, -300.0), (1.0, 0.004)])
def test_bf16_magnitudes(scale, shift):
    """bf16 logits of magnitudes with and without a place of their own, zeros among them."""
    R, V = 48, 6000
    x = (logits(R, V, 30, scale=scale) + shift).to(BF16)
    x[::2, ::7] = 0.0
    x[1::4, ::5] = -math.inf
    u = np.random.default_rng(31).random(R)
    compare(x, u, **mixed(R, 32))
    compare(x, u, top_p=np.linspace(0.02, 0.9999, R).astype(np.float32))
    compare(x, u, min_p=np.linspace(0.0, 0.5, R).astype(np.float32))
    compare(x.float(), u, top_p=np.linspace(0.02, 0.9999, R).astype(np.float32))
    compare(x, u, top_k=np.full(R, 2000, np.int32), top_p=np.full(R, 0.7, np.float32))


def kept_of_top_p(x, k, p):
    """Mask of the tokens that top-k and top-p keep, sums in 64-bit mantissas."""
    w = np.exp(x.astype(np.longdouble) - x.max())
    order = np.argsort(-x, kind="stable")[:k]
    mass = np.cumsum(w[order])
    kept = np.zeros(len(x), bool)
    kept[order[mass - w[order] < np.longdouble(p) * mass[-1]]] = True
    return kept, w


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("spread", [0.0, 2.0])
@pytest.mark.parametrize("by_k", [True, False])
@pytest.mark.parametrize("rows", [1, 160])
def test_top_p_next_to_one(dtype, spread, by_k, rows):
    """A million weights around e^-30 behind one of 1: half of them lie below top_p's border, and
    tokens on either side of what they add up to are told apart."""
    V, p = 1 << 20, np.float32(1 - 2.0 ** -24)
    g = np.random.default_rng(33)
    x = torch.from_numpy((-30 - spread * (g.random(V) - 0.5)).astype(np.float32))
    x[-1] = 0.0
    x = x.to(dtype)
    k = V - 1 if by_k else V
    kept, w = kept_of_top_p(x.float().numpy().astype(np.float64), k, p)
    assert 0.2 * V < kept.sum() < 0.8 * V
    c = np.cumsum(np.where(kept, w, 0))
    share = float((c[-1] - 1) / c[-1])
    u = np.resize(np.float32([0.0, 0.01 * share, 0.3 * share, 0.99 * share, 1.01 * share]), rows)
    if rows == 1:
        u[0] = np.float32(0.99 * share)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    ws = L.new_workspace(L.make_sample_problem(rows, V, in_dtype=dtype))
    xs = x.cuda()[None].expand(rows, V).contiguous()
    token, lp = L.sample(xs, dev(u), top_p=dev(np.full(rows, p)), workspace=ws,
                         top_k=dev(np.full(rows, k, np.int32)) if by_k else None)
    assert L.get_status(ws) == 0
    want = [int(np.nonzero((c > np.longdouble(v) * c[-1]) & kept)[0][0]) for v in u]
    got = token.cpu().numpy()
    # the sums' order leaves the border and the token open by a few thousandths of a token
    assert np.array_equal(got, want), (got[:5], want[:5])
    assert np.all(np.abs(lp.cpu().numpy() - np.log((w[want] / c[-1]).astype(float))) <= 2.0 ** -24 * 32)


def test_ends_of_the_parameters():
    R, V = 12, 333
    x = logits(R, V, 14)
    u = np.linspace(0, 1, R)
    one = lambda v, t=np.float32: np.full(R, v, t)
    for p in ({"top_p": one(0.0)}, {"top_p": one(1.0)}, {"top_p": one(1 - 2.0 ** -24)},
              {"top_p": one(1e-30)}, {"min_p": one(1.0)}, {"min_p": one(1e-30)},
              {"top_k": one(1, np.int32)}, {"top_k": one(-5, np.int32)},
              {"top_k": one(V, np.int32)}, {"top_k": one(2 ** 31 - 1, np.int32)},
              {"temperature": one(0.0)}, {"temperature": one(1e-30)}, {"temperature": one(1e-45)},
              {"temperature": one(1e30)}, {"temperature": one(3e38), "top_p": one(0.5)}):
        compare(x, u, **p)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_rows(dtype):
    """-inf, NaN and +inf among the logits; rows that leave one token or none."""
    R, V = 10, 257
    x = logits(R, V, 15, dtype)
    x[0] = -math.inf
    x[1] = -math.inf
    x[1, 77] = -3.0
    x[2, ::2] = -math.inf
    x[3, 1::2] = math.nan
    x[4] = math.nan
    x[5, [3, 200]] = math.inf
    x[6, 1:] = -math.inf
    x[7, :-1] = -math.inf
    x[8] = torch.finfo(dtype).min
    x[9, :250] = torch.finfo(dtype).min
    for s in range(3):
        u = np.random.default_rng(s).random(R)
        got = compare(x, u)
        assert got[0] == -1 and got[1] == 77 and got[4] == -1 and got[6] == 0 and got[7] == V - 1
        compare(x, u, **mixed(R, s))
        compare(x, u, top_k=np.full(R, 200, np.int32), top_p=np.full(R, 0.9, np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("start,pad", [(0, 3), (1, 2), (5, 64)])
def test_strided_rows(dtype, start, pad):
    """Rows of a padded matrix, at any alignment; what lies between them is not looked at."""
    R, V = 9, 1001
    wide = torch.full((R, start + V + pad), math.nan, dtype=dtype, device="cuda")
    wide[:, :start] = math.inf
    wide[:, start + V:] = math.inf
    x = wide[:, start:start + V]
    x.copy_(logits(R, V, 16, dtype))
    compare(x, np.random.default_rng(17).random(R), **mixed(R, 18))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [12, 160])
@pytest.mark.parametrize("V", [400, 5000, 60_000])
def test_large_top_k(dtype, rows, V):
    """top_k of 257 and more: the border by counts through the bits, then top-p's among what is left."""
    x, u = logits(rows, V, V + 40, dtype), np.random.default_rng(41).random(rows)
    g = np.random.default_rng(42)
    k = g.integers(257, V, rows).astype(np.int32)
    k[:2] = 257, V - 1
    p = g.random(rows).astype(np.float32)
    compare(x, u, top_k=k)
    compare(x, u, top_k=k, top_p=p)
    compare(x, u, top_k=k, min_p=(0.2 * p).astype(np.float32),
            temperature=(0.3 + 1.5 * p).astype(np.float32))
    compare((x * 2).round() / 2, u, top_k=k, top_p=p)
    compare(-x.abs(), u, top_k=k, top_p=p)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [8, 160])
def test_small_top_k_among_many_equals(dtype, rows):
    """More than a thousand logits reach the bound that the stripes give a top_k of up to 256."""
    V = 6000
    x = (logits(rows, V, 43) / 2).round().to(dtype)        # some 2300 zeros, 1500 ones
    u = np.random.default_rng(44).random(rows)
    for k in (2, 100, 256):
        k = np.full(rows, k, np.int32)
        compare(x, u, top_k=k)
        compare(x, u, top_k=k, top_p=np.full(rows, 0.6, np.float32))
    z = torch.zeros_like(x)
    z[:, 5000:] = -1.0
    compare(z, u, top_k=np.full(rows, 200, np.int32), top_p=np.full(rows, 0.37, np.float32))


# more rows than SMs: 512 threads to a row


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1, 33, 1000, 4097, 50257, 200_003])
def test_many_rows(dtype, V):
    R = 160
    x, u = logits(R, V, V + 50, dtype), np.random.default_rng(V).random(R)
    compare(x, u)
    compare(x, u, **mixed(R, V + 51))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_masked_rows(dtype):
    R, V = 160, 5003
    x = logits(R, V, 52, dtype)
    low = torch.finfo(dtype).min
    x[0::10] = -math.inf
    x[1::10] = -math.inf
    x[1::10, 4077] = -3.0
    x[2::10, ::2] = -math.inf
    x[3::10, 1::2] = math.nan
    x[4::10] = math.nan
    x[5::10, [3, 4200]] = math.inf
    x[6::10, 1:] = -math.inf
    x[7::10, :-1] = -math.inf
    x[8::10] = low
    x[9::10, :4990] = low
    for s in range(2):
        u = np.random.default_rng(s).random(R)
        got = compare(x, u)
        assert (got[0::10] == -1).all() and (got[1::10] == 4077).all() and (got[4::10] == -1).all()
        compare(x, u, **mixed(R, s + 53))
        compare(x, u, top_k=np.full(R, 2000, np.int32), top_p=np.full(R, 0.9, np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows_at_the_ends_of_the_parameters(dtype):
    R, V = 160, 2333
    x = logits(R, V, 54, dtype)
    u = np.linspace(0, 1, R)
    one = lambda v, t=np.float32: np.full(R, v, t)
    for p in ({"top_p": one(0.0)}, {"top_p": one(1 - 2.0 ** -24)}, {"top_p": one(1e-30)},
              {"min_p": one(1.0)}, {"min_p": one(1e-30)}, {"top_k": one(1, np.int32)},
              {"top_k": one(V - 1, np.int32)}, {"temperature": one(1e-30)},
              {"temperature": one(1e30)}, {"temperature": one(3e38), "top_p": one(0.5)}):
        compare(x, u, **p)


@pytest.mark.parametrize("scale,shift", [(0.01, 0.0), (6.0, 3.0), (80.0, 0.0), (3.0, 300.0),
                                         (3.0, -300.0)])
def test_many_rows_of_bf16_magnitudes(scale, shift):
    R, V = 160, 9001
    x = (logits(R, V, 55, scale=scale) + shift).to(BF16)
    x[::2, ::7] = 0.0
    x[1::4, ::5] = -math.inf
    u = np.random.default_rng(56).random(R)
    compare(x, u, **mixed(R, 57))
    compare(x, u, top_p=np.linspace(0.02, 0.9999, R).astype(np.float32))
    compare(x.float(), u, top_p=np.linspace(0.02, 0.9999, R).astype(np.float32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("start,pad", [(1, 2), (5, 64)])
def test_many_strided_rows(dtype, start, pad):
    R, V = 160, 9001
    wide = torch.full((R, start + V + pad), math.nan, dtype=dtype, device="cuda")
    wide[:, :start] = math.inf
    wide[:, start + V:] = math.inf
    x = wide[:, start:start + V]
    x.copy_(logits(R, V, 58, dtype))
    compare(x, np.random.default_rng(59).random(R), **mixed(R, 60))


def test_bad_parameters_leave_the_row():
    R, V = 8, 100
    x = logits(R, V, 19)
    u = torch.full((R,), 0.5, device="cuda")
    t = torch.ones(R, device="cuda")
    p, m = torch.ones(R, device="cuda"), torch.zeros(R, device="cuda")
    t[0], t[1], t[2] = -1.0, math.nan, math.inf
    p[3], p[4] = 1.5, -0.1
    m[5] = math.nan
    u[6] = 1.5
    token = torch.full((R,), -7, dtype=I32, device="cuda")
    ws = L.new_workspace(L.make_sample_problem(R, V))
    L.sample(x, u, temperature=t, top_p=p, min_p=m, token=token, workspace=ws)
    assert L.get_status(ws) == L.binding.TV_ERR_BAD_PARAM
    assert (token[:7] == -7).all() and token[7] >= 0
    assert L.get_status(ws) == 0


def test_sampled_shares():
    """Tokens at evenly spread random numbers come with their shares, to one number each."""
    V, R = 50, 4000
    x = logits(1, V, 20).expand(R, V).contiguous()
    u = (torch.arange(R, device="cuda") + 0.5) / R
    token, lp = L.sample(x, u)
    share = torch.bincount(token.long(), minlength=V).double() / R
    want = torch.softmax(x[0].double(), 0)
    assert ((share - want).abs() <= 1.0 / R + 1e-9).all()
    assert torch.allclose(lp.double(), want.log()[token.long()], rtol=1e-6, atol=1e-12)


@pytest.mark.parametrize("R,V", [(1, 40000), (300, 5000)])
def test_streams_and_graphs(R, V):
    x, u = logits(R, V, 21), torch.from_numpy(np.random.default_rng(22).random(R)).float().cuda()
    p = {k: torch.from_numpy(a).cuda() for k, a in mixed(R, 23).items()}
    want = L.sample(x, u, **p)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [L.sample(x, u, stream=s, **p) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for token, lp in got:
        assert torch.equal(token, want[0]) and torch.equal(lp, want[1])
    ws = L.new_workspace(L.make_sample_problem(R, V))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token, lp = L.sample(x, u, workspace=ws, **p)
    for _ in range(2):
        token.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(token, want[0]) and torch.equal(lp, want[1])


def test_no_rows():
    token, lp = L.sample(torch.empty(0, 10, device="cuda"), torch.empty(0, device="cuda"))
    assert token.shape == (0,) and lp.shape == (0,)


# ---- acceptance ------------------------------------------------------------------------------


def trees(lens, seed, tokens=3):
    g = np.random.default_rng(seed)
    parent = [int(g.integers(max(-1, i // 2 - 2), i)) for n in lens for i in range(n)]
    T = len(parent)
    i32 = lambda a: np.asarray(a, np.int32)
    return {"draft": i32(g.integers(0, tokens, T)), "target": i32(g.integers(0, tokens, T)),
            "root": i32(g.integers(0, tokens, len(lens))), "parent": i32(parent),
            "offsets": i32(np.concatenate([[0], np.cumsum(lens)]))}


def accept(t, lens, max_path, **kw):
    d = {k: torch.from_numpy(a).cuda() for k, a in t.items()}
    return L.tree_accept(d["draft"], d["target"], d["root"], d["parent"], d["offsets"],
                         max_nodes=max(max(lens), 1), max_path=max_path, **kw)


@pytest.mark.parametrize("lens", [[1], [6], [32, 33, 0, 64], [256, 1, 255], [0, 0], list(range(40))])
@pytest.mark.parametrize("max_path", [1, 5, 64])
def test_accept(lens, max_path):
    for seed in range(6):
        t = trees(lens, seed, tokens=1 + seed % 3)
        got = [x.cpu().numpy() for x in accept(t, lens, max_path)]
        want = OS.accept(t["draft"], t["target"], t["root"], t["parent"], t["offsets"], max_path)
        for a, b, name in zip(got, want, ("path", "length", "next")):
            assert np.array_equal(a, b), name


def test_accept_negative_tokens_and_chains():
    n = 200
    t = {"draft": np.arange(n, dtype=np.int32), "target": np.arange(1, n + 1, dtype=np.int32),
         "root": np.zeros(1, np.int32), "parent": np.arange(-1, n - 1, dtype=np.int32),
         "offsets": np.array([0, n], np.int32)}
    path, count, nxt = accept(t, [n], 300)
    assert count.item() == n and nxt.item() == n and path[0, :n].tolist() == list(range(n))
    assert (path[0, n:] == -1).all()
    t["draft"][50] = -1
    t["target"][49] = -1
    path, count, nxt = accept(t, [n], 300)
    assert count.item() == 50 and nxt.item() == -1


@pytest.mark.parametrize("bad", ["self", "forward", "below", "long", "end"])
def test_accept_bad_trees(bad):
    lens = [10, 12, 9]
    t = trees(lens, 3)
    if bad in ("self", "forward", "below"):
        t["parent"][15] = {"self": 5, "forward": 9, "below": -2}[bad]
    elif bad == "long":
        t["offsets"][1], t["offsets"][2] = 4, 22
    else:
        t["offsets"][3] = 30
    out = torch.full((3, 4), -9, dtype=I32, device="cuda")
    ws = L.new_workspace(L.make_problem(3, 1, 16, 16, 31, 12, 4))
    accept(t, lens, 4, accepted_path=out, workspace=ws)
    assert L.get_status(ws) == L.binding.TV_ERR_BAD_TREE
    row = 2 if bad == "end" else 1
    assert (out[row] == -9).all() and (out[0] >= -1).all()


def test_decode_loop_of_the_operators():
    """Prompt, then two steps of verify, logits, sample, accept and commit: the committed state
    and the tokens are those of a token-by-token decode with the same random numbers."""
    B, H, d, V = 2, 2, 128, 19
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1).to(BF16)
    # one embedding per token for q, k, v and the gates, and a read-out of the layer's output
    eq, ek, ev = unit(rnd(V, H, d)), unit(rnd(V, H, d)), rnd(V, H, d).to(BF16)
    la, b = -torch.nn.functional.softplus(-3 + rnd(V, H)), torch.sigmoid(rnd(V, H))
    head = 0.3 * rnd(H * d, V)
    read = lambda o: (o.float().reshape(o.shape[0], -1) @ head).contiguous()
    prompt = torch.randint(0, V, (B * 70,), generator=g, device="cuda")
    offsets = torch.tensor([0, 70, 140], dtype=I32, device="cuda")
    out, S = L.prefill(eq[prompt], ek[prompt], ev[prompt], la[prompt], b[prompt], offsets,
                       max_len=70, out_dtype=F32)
    last, _ = L.sample(read(out[[69, 139]]), torch.rand(B, generator=g, device="cuda"))
    plain = S.clone()
    for step in range(2):
        # each tree: every token under the root is not possible, so a chain of greedy guesses
        # and random siblings; the first node is the token already sampled
        parent, draft = [], []
        for s in range(B):
            base = [int(last[s])] + torch.randint(0, V, (11,), generator=g, device="cuda").tolist()
            parent += [-1, 0, 0, 0, 1, 1, 2, 2, 3, 3, 4, 6]
            draft += base
        draft_t = torch.tensor(draft, dtype=I32, device="cuda")
        parent_t = torch.tensor(parent, dtype=I32, device="cuda")
        off = torch.tensor([0, 12, 24], dtype=I32, device="cuda")
        n = draft_t.long()
        o, U = L.tree_verify(eq[n], ek[n], ev[n], la[n].contiguous(), b[n].contiguous(), parent_t,
                             off, S, max_nodes=12, out_dtype=F32)
        u = torch.rand(24, generator=g, device="cuda")
        target, _ = L.sample(read(o), u, top_k=torch.full((24,), 3, dtype=I32, device="cuda"))
        path, count, nxt = L.tree_accept(draft_t, target, last, parent_t, off, max_nodes=12,
                                         max_path=4)
        S = L.tree_commit(U, ek[n], la[n].contiguous(), S, off, path, max_nodes=12,
                          parent=parent_t)
        assert (count >= 1).all()                    # the token already sampled is in its tree
        for s in range(B):                           # the accepted tokens, one at a time
            for j in range(int(count[s])):
                tok = torch.tensor([draft[12 * s + int(path[s, j])]], device="cuda")
                one, X = L.decode_step(eq[tok], ek[tok], ev[tok], la[tok], b[tok],
                                       plain[s:s + 1].contiguous(), out_dtype=F32)
                plain[s] = X[0]
            # the verified output of the last accepted node is the step's (bf16 products there)
            node = 12 * s + int(path[s, int(count[s]) - 1])
            rms = one.double().pow(2).mean().sqrt()
            assert (one[0] - o[node]).abs().max() <= 2e-2 * rms
            assert int(nxt[s]) == int(target[node])
        rms = plain.double().pow(2).mean().sqrt()
        assert (S - plain).abs().max() <= 2e-2 * rms
        S.copy_(plain)
        last = nxt
