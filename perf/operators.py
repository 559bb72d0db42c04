"""Cases, plain forms and exact values of the operators around a tree-verifying decode loop.

  prefill      the layer's recurrence (gated delta rule or scalar decay) over whole prompts:
               outputs of every token and the state after the last one
  decode_step  the same recurrence for one token of every sequence, the state updated in place
  sample       one token per row of logits: temperature, top-k, top-p and min-p from a given
               random number
  tree_accept  sampled target tokens walked against the draft trees: the accepted path that
               the commit takes, its length and the next token

The plain forms are elementary torch operations.  Prompts are computed in chunks of 64
tokens (the recurrence's closed form inside a chunk, every chunk at once; the state carried
from chunk to chunk in a loop, since it is sequential).  Sampling sorts in full and sums in
64 bits, because a token is decided by comparing sums next to a border.
"""
import math
import random

import torch

own = False

CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one long prompt of one user: the chain of states is the whole of the latency
        {"name": "prefill gdn 1x8192", "op": "prefill", "mode": "gdn", "type": "bf16", "B": 1,
         "T": 8192, "H": 32, "Hk": 32, "dk": 128, "dv": 128, "ragged": False, "zero": True},
        # a batch of prompts of mixed lengths, two value heads to a key head, from kept states
        {"name": "prefill gdn ragged 16", "op": "prefill", "mode": "gdn", "type": "bf16", "B": 16,
         "T": 16384, "H": 32, "Hk": 16, "dk": 128, "dv": 128, "ragged": True, "zero": False},
        # a scalar-decay layer's batch of equal prompts
        {"name": "prefill scalar 8x1000", "op": "prefill", "mode": "scalar", "type": "bf16",
         "B": 8, "T": 8000, "H": 16, "Hk": 16, "dk": 128, "dv": 128, "ragged": False,
         "zero": False},
        # a small layer in 32 bits, odd lengths
        {"name": "prefill gdn f32 small", "op": "prefill", "mode": "gdn", "type": "f32", "B": 3,
         "T": 219, "H": 4, "Hk": 2, "dk": 64, "dv": 48, "ragged": True, "zero": False},
        # single-token steps: one user (latency), a usual batch, a large one with shared keys
        {"name": "decode gdn 1", "op": "decode", "mode": "gdn", "type": "bf16", "B": 1, "H": 16,
         "Hk": 16, "dk": 128, "dv": 128},
        {"name": "decode gdn 32", "op": "decode", "mode": "gdn", "type": "bf16", "B": 32, "H": 32,
         "Hk": 32, "dk": 128, "dv": 128},
        {"name": "decode scalar f32 128", "op": "decode", "mode": "scalar", "type": "f32",
         "B": 128, "H": 32, "Hk": 16, "dk": 128, "dv": 128},
        # one user's next token; a decode batch with every filter; every node of 32 draft trees
        {"name": "sample 1x32768", "op": "sample", "type": "f32", "R": 1, "V": 32768,
         "pad": 0, "filters": "top-p"},
        {"name": "sample mixed 128x100003", "op": "sample", "type": "f32", "R": 128, "V": 100003,
         "pad": 61, "filters": "mixed"},
        {"name": "sample nodes 2048x65536", "op": "sample", "type": "bf16", "R": 2048,
         "V": 65536, "pad": 0, "filters": "mixed"},
        # the draft trees of one user, and of a batch with ragged trees
        {"name": "accept 1x16", "op": "accept", "B": 1, "N": 16, "ragged": False},
        {"name": "accept ragged 128x64", "op": "accept", "B": 128, "N": 64, "ragged": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "sample", "sample",
                     "sample", "accept"])
    if op in ("prefill", "decode"):
        share = rng.choice([1, 1, 2, 4])
        c = {"op": op, "mode": rng.choice(["gdn", "gdn", "scalar"]), "type": "bf16", "dk": 128,
             "dv": 128}
        if rng.random() < 0.3:
            c.update(type=rng.choice(["bf16", "f32"]), dk=16 * rng.randint(1, 8),
                     dv=16 * rng.randint(1, 8))
        c["H"] = share * rng.randint(1, 32 // share)
        c["Hk"] = c["H"] // share
        if op == "decode":
            c["B"] = _log_int(rng, 1, 128)
            return c
        # shapes off the usual widths, and 32-bit inputs, up to 2048 tokens
        wide = c["type"] == "bf16" and c["dk"] == c["dv"] == 128
        c["T"] = _log_int(rng, 1, 12000 if wide else 2048)
        c["B"] = min(c["T"], _log_int(rng, 1, 32))
        c["ragged"] = rng.random() < 0.7
        c["zero"] = rng.random() < 0.5
        if not c["ragged"]:
            c["T"] -= c["T"] % c["B"]
        return c
    if op == "sample":
        V = _log_int(rng, 17, 150000)
        return {"op": op, "type": rng.choice(["bf16", "f32"]),
                "R": _log_int(rng, 1, max(1, min(2048, 100_000_000 // V))), "V": V,
                "pad": rng.choice([0, 0, 3, 64]),
                "filters": rng.choice(["mixed", "mixed", "top-p", "none", "greedy"])}
    return {"op": op, "B": _log_int(rng, 1, 128), "N": rng.randint(1, 256),
            "ragged": rng.random() < 0.6}


def _lengths(total, parts, ragged, most=None):
    """`parts` lengths with the sum `total` (or, with `most`, up to `most` each)."""
    r = random.Random(total * 1009 + parts)
    if most is not None:
        return [r.randint(0, most) if ragged else most for _ in range(parts)]
    if not ragged:
        return [total // parts] * parts
    cuts = sorted(r.randint(0, total) for _ in range(parts - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# ---- inputs -------------------------------------------------------------------------------


def _gates(rng, shape, mode):
    """log_a and b as a gated layer makes them: a decay near one, a write strength in (0, 1)."""
    n = torch.randn(shape, generator=rng, device="cuda")
    log_a = -torch.nn.functional.softplus(-4.0 + 0.5 * n)
    b = torch.sigmoid(torch.randn(shape, generator=rng, device="cuda")) if mode == "gdn" else None
    return log_a, b


def _unit(rng, shape, dtype):
    x = torch.randn(shape, generator=rng, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def _prepare_sequences(c, rng):
    dt = TYPES[c["type"]]
    lens = _lengths(c["T"], c["B"], c["ragged"]) if c["op"] == "prefill" else [1] * c["B"]
    T, B, H, Hk, dk, dv = sum(lens), c["B"], c["H"], c["Hk"], c["dk"], c["dv"]
    st = {"op": c["op"], "mode": c["mode"], "lens": lens,
          "q": _unit(rng, (T, Hk, dk), dt), "k": _unit(rng, (T, Hk, dk), dt),
          "v": torch.randn((T, H, dv), generator=rng, device="cuda").to(dt),
          "S": 0.02 * torch.randn((B, H, dv, dk), generator=rng, device="cuda")}
    st["log_a"], st["b"] = _gates(rng, (T, H), c["mode"])
    if c["op"] == "prefill":
        if c["zero"]:
            st["S"] = None
        st["offsets"] = torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda")
        st["plan"] = _chunk_plan(lens)
    return st


def _chunk_plan(lens):
    """Index lists of the chunked form: token row and validity of every place of every chunk,
    sequences by falling length, and the chunks of each step of the chain."""
    order = sorted(range(len(lens)), key=lambda s: -lens[s])
    off = _offsets(lens)
    first, starts, counts = [], [], []
    for s in order:
        first.append(len(starts))
        for t in range(0, lens[s], CHUNK):
            starts.append(off[s] + t)
            counts.append(min(CHUNK, lens[s] - t))
    dev = {"device": "cuda"}
    place = torch.arange(CHUNK, **dev)
    counts_t = torch.tensor(counts, dtype=torch.int64, **dev)
    rows = torch.tensor(starts, dtype=torch.int64, **dev)[:, None] + place
    valid = place < counts_t[:, None]
    steps = []
    for j in range(-(-max(lens) // CHUNK)):
        steps.append(torch.tensor([first[i] + j for i, s in enumerate(order)
                                   if lens[s] > j * CHUNK], dtype=torch.int64, **dev))
    return {"order": torch.tensor(order, dtype=torch.int64, **dev), "steps": steps,
            "rows": torch.where(valid, rows, 0), "valid": valid, "tokens": rows[valid]}


def _prepare_sample(c, rng):
    R, V, W = c["R"], c["V"], c["V"] + c["pad"]
    dev = {"device": "cuda", "generator": rng}
    # logits that fall off with the logarithm of a token's rank, as a language model's do
    x = -1.1 * torch.log1p(V * torch.rand((R, W), **dev))
    x += 0.5 * torch.randn((R, W), **dev)
    if c["filters"] == "mixed":
        # a tenth of the rows allow a tenth of the tokens only, as under a grammar
        shut = (torch.rand((R, 1), **dev) < 0.1) & (torch.rand((R, W), **dev) < 0.9)
        x.masked_fill_(shut, -math.inf)
    ones = torch.ones(R, device="cuda")
    st = {"op": "sample", "logits": x.to(TYPES[c["type"]])[:, :V],
          "uniform": torch.rand(R, **dev), "temperature": ones, "top_k": None, "top_p": None,
          "min_p": None}
    pick = torch.rand((4, R), **dev)
    if c["filters"] == "greedy":
        st["temperature"] = 0 * ones
    elif c["filters"] == "top-p":
        st["temperature"] = 0.6 + 0.6 * pick[0]
        st["top_p"] = 0.8 + 0.19 * pick[1]
    elif c["filters"] == "mixed":
        st["temperature"] = torch.where(pick[0] < 0.1, 0.0, 0.5 + pick[0])
        st["top_k"] = torch.where(pick[1] < 0.5, 0, 1 + 99 * pick[1]).to(torch.int32)
        st["top_p"] = torch.where(pick[2] < 0.3, 1.0, 0.6 + 0.39 * pick[2])
        st["min_p"] = torch.where(pick[3] < 0.5, 0.0, 0.1 * pick[3])
    return st


def _prepare_accept(c, rng):
    lens = _lengths(0, c["B"], c["ragged"], most=c["N"])
    T, B = sum(lens), c["B"]
    host = random.Random(c["N"] * 31 + B)
    parent, depth = [], []
    for n in lens:
        base = len(depth)
        for i in range(n):
            # one to a few children to a node, near the front of the tree, no path over 32
            p = -1 if i == 0 else host.randint(max(-1, i // 3 - 2), i - 1)
            while p >= 0 and depth[base + p] >= 32:
                p -= 1
            parent.append(p)
            depth.append(1 if p < 0 else depth[base + p] + 1)
    dev = {"device": "cuda"}
    # a draft that is right most of the time: four token values, the target's one of them
    draft = torch.randint(0, 4, (T,), generator=rng, **dev, dtype=torch.int32)
    return {"op": "accept", "lens": lens, "draft": draft,
            "target": torch.randint(0, 4, (T,), generator=rng, **dev, dtype=torch.int32),
            "root": torch.randint(0, 4, (B,), generator=rng, **dev, dtype=torch.int32),
            "parent": torch.tensor(parent, dtype=torch.int32, **dev),
            "offsets": torch.tensor(_offsets(lens), dtype=torch.int32, **dev),
            "max_nodes": c["N"], "max_path": 32}


def prepare(case, seed):
    rng = torch.Generator(device="cuda")
    rng.manual_seed(seed)
    if case["op"] in ("prefill", "decode"):
        return _prepare_sequences(case, rng)
    if case["op"] == "sample":
        return _prepare_sample(case, rng)
    return _prepare_accept(case, rng)


# ---- plain forms --------------------------------------------------------------------------


def _plain_prefill(st):
    plan, gdn = st["plan"], st["mode"] == "gdn"
    T, Hk, dk = st["q"].shape
    H, dv = st["v"].shape[1:]
    rows, valid = plan["rows"], plan["valid"]
    v = torch.where(valid[..., None, None], st["v"].float()[rows], 0).transpose(1, 2)
    k = torch.where(valid[..., None, None], st["k"].float()[rows], 0).transpose(1, 2)
    q = st["q"].float()[rows].transpose(1, 2)
    k, q = (x.repeat_interleave(H // Hk, dim=1) for x in (k, q))
    la = torch.where(valid[..., None], st["log_a"].double()[rows], 0).transpose(1, 2)
    cl = la.cumsum(-1)                                                 # [chunk, head, place]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(low, torch.exp(cl[..., :, None] - cl[..., None, :]), 0).float()
    gamma = torch.exp(cl).float()[..., None]
    tail = torch.exp(cl[..., -1:] - cl).float()[..., None]
    if gdn:
        b = torch.where(valid[..., None], st["b"][rows], 0).transpose(1, 2)[..., None]
        a = -(b * decay * (k @ k.transpose(-1, -2))).tril(-1)
        inv = a + torch.eye(CHUNK, device=q.device)
        for _ in range(5):                    # (I - A)^-1 = (I + A)(I + A^2)(I + A^4)...
            a = a @ a
            inv = inv + a @ inv
        w, u0 = inv @ (b * gamma * k), inv @ (b * v)
    else:
        u0 = v
    qk, qg, kt, g = decay * (q @ k.transpose(-1, -2)), gamma * q, tail * k, gamma[..., -1:, :]
    S0 = st["S"]
    B = len(st["lens"])
    S = torch.zeros(B, H, dv, dk, device=q.device) if S0 is None else S0[plan["order"]]
    o = torch.empty_like(u0)
    for ids in plan["steps"]:
        live = S[:len(ids)]
        u = u0[ids] - w[ids] @ live.transpose(-1, -2) if gdn else u0[ids]
        o[ids] = qg[ids] @ live.transpose(-1, -2) + qk[ids] @ u
        S[:len(ids)] = g[ids] * live + u.transpose(-1, -2) @ kt[ids]
    out = torch.empty(T, H, dv, dtype=st["q"].dtype, device=q.device)
    out[plan["tokens"]] = o.transpose(1, 2)[valid].to(out.dtype)
    S_new = torch.empty_like(S)
    S_new[plan["order"]] = S
    return out, S_new


def _plain_decode(st):
    S, v = st["S"], st["v"].float()
    share = v.shape[1] // st["q"].shape[1]
    q, k = (st[n].float().repeat_interleave(share, dim=1)[..., None] for n in ("q", "k"))
    S *= torch.exp(st["log_a"])[..., None, None]
    u = st["b"][..., None] * (v - (S @ k)[..., 0]) if st["mode"] == "gdn" else v
    S += u[..., None] * k.transpose(-1, -2)
    return (S @ q)[..., 0].to(st["q"].dtype), S


def _plain_sample(st):
    x = st["logits"].float()
    R, V = x.shape
    x = torch.where(x.isnan(), -math.inf, x)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    y = x.double()
    top = y.max(-1, keepdim=True).values
    t = st["temperature"].double()[:, None]
    w = torch.where(y == top, 0.0, (y - top) / torch.where(t > 0, t, 1.0)).exp()
    ws = w.gather(-1, order)
    place = torch.arange(V, device=x.device)
    keep = (place == 0) | (t > 0)
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep &= (place < k) | (k <= 0)
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        wk = torch.where(keep, ws, 0.0)
        mass = wk.cumsum(-1)
        keep &= (mass - wk < p * mass[:, -1:]) | (p >= 1) | (place == 0)
    if st["min_p"] is not None:
        keep &= ws >= st["min_p"].double()[:, None]
    wv = torch.zeros_like(w).scatter_(-1, order, torch.where(keep, ws, 0.0))
    mass = wv.cumsum(-1)
    total = mass[:, -1:]
    past = (mass > st["uniform"].double()[:, None] * total) & (wv > 0)
    last = V - 1 - (wv > 0).flip(-1).to(torch.int32).argmax(-1)
    token = torch.where(past.any(-1), past.to(torch.int32).argmax(-1), last)
    logprob = (wv.gather(-1, token[:, None]) / total).log()[:, 0].float()
    empty = top[:, 0] == -math.inf
    return (torch.where(empty, -1, token).to(torch.int32),
            torch.where(empty, -math.inf, logprob))


def _plain_accept(st):
    dev, B, N, P = st["draft"].device, len(st["lens"]), st["max_nodes"], st["max_path"]
    off = st["offsets"].long()
    node = torch.arange(N, device=dev)
    valid = node < (off[1:] - off[:-1])[:, None]
    rows = torch.where(valid, off[:-1, None] + node, 0)
    at = lambda x, none: (torch.where(valid, x[rows], none) if x.numel()
                          else torch.full((B, N), none, device=dev))
    draft, target, parent = at(st["draft"], -1), at(st["target"], -1), at(st["parent"], -1).long()
    root = st["root"][:, None].to(target.dtype)
    up = parent.clamp(min=0)
    want = torch.where(parent < 0, root, target.gather(1, up))
    good = valid & (draft == want) & (draft >= 0)
    # of siblings with the same token the first counts
    twin = (parent[:, :, None] == parent[:, None, :]) & (good[:, :, None] & good[:, None, :])
    good &= ~(twin & (node[:, None] > node)).any(-1)
    # a node is accepted if every node of its path is good: parents by doubling, N to a root
    depth = torch.ones_like(parent)
    jump = torch.where(parent < 0, N, parent)
    pad = lambda x, v: torch.cat([x, torch.full((B, 1), v, dtype=x.dtype, device=dev)], 1)
    good, depth, jump = pad(good, True), pad(depth, 0), pad(jump, N)
    for _ in range(max(1, (N - 1).bit_length())):
        good = good & good.gather(1, jump)
        depth = depth + depth.gather(1, jump)
        jump = jump.gather(1, jump)
    got = good[:, :N] & (depth[:, :N] <= P)
    place = torch.where(got, depth[:, :N] - 1, P)
    path = torch.full((B, P + 1), -1, dtype=torch.int64, device=dev)
    path = path.scatter(1, place, node.expand(B, N))[:, :P]
    count = got.sum(1)
    leaf = path.gather(1, (count - 1).clamp(min=0)[:, None])
    nxt = torch.where(count > 0, target.gather(1, leaf.clamp(min=0))[:, 0], root[:, 0])
    return path.to(torch.int32), count.to(torch.int32), nxt.to(torch.int32)


# ---- the framework's calls ----------------------------------------------------------------


def _kept(st, name, make):
    """A buffer or workspace that a user's program keeps from call to call."""
    if name not in st:
        st[name] = make()
    return st[name]


def _own(st):
    import linear_attention_tree_b200 as L
    if st["op"] == "prefill":
        ws = _kept(st, "workspace", lambda: L.new_workspace(L.make_sequence_problem(
            len(st["lens"]), st["v"].shape[1], st["q"].shape[2], st["v"].shape[2],
            st["q"].shape[0], max(st["lens"]), mode=st["mode"], in_dtype=st["q"].dtype,
            qk_heads=st["q"].shape[1])))
        return L.prefill(st["q"], st["k"], st["v"], st["log_a"], st["b"], st["offsets"], st["S"],
                         max_len=max(st["lens"]), mode=st["mode"], workspace=ws)
    if st["op"] == "decode":
        return L.decode_step(st["q"], st["k"], st["v"], st["log_a"], st["b"], st["S"],
                             mode=st["mode"], S_new=st["S"])
    if st["op"] == "sample":
        ws = _kept(st, "workspace", lambda: L.new_workspace(
            L.make_sample_problem(*st["logits"].shape, in_dtype=st["logits"].dtype)))
        return L.sample(st["logits"], st["uniform"], temperature=st["temperature"],
                        top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"], workspace=ws)
    ws = _kept(st, "workspace", lambda: L.new_workspace(L.make_problem(
        len(st["lens"]), 1, 16, 16, st["draft"].shape[0], st["max_nodes"], st["max_path"])))
    return L.tree_accept(st["draft"], st["target"], st["root"], st["parent"], st["offsets"],
                         max_nodes=st["max_nodes"], max_path=st["max_path"], workspace=ws)


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "sample": _plain_sample,
            "accept": _plain_accept}[state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------


def work(case):
    if case["op"] in ("prefill", "decode"):
        size = 2 if case["type"] == "bf16" else 4
        B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
        T = case["T"] if case["op"] == "prefill" else B
        gdn = case["mode"] == "gdn"
        states = 1 if case.get("zero") else 2
        return {"bytes": T * (2 * Hk * dk + 2 * H * dv) * size + T * H * (8 if gdn else 4)
                + states * B * H * dk * dv * 4,
                "flops": (6 if gdn else 4) * T * H * dk * dv}
    if case["op"] == "sample":
        R, V = case["R"], case["V"]
        # an exponential, a sum and the comparisons of the filters for each logit
        return {"bytes": R * V * (2 if case["type"] == "bf16" else 4) + 28 * R,
                "flops": 6 * R * V}
    nodes = sum(_lengths(0, case["B"], case["ragged"], most=case["N"]))
    return {"bytes": 12 * nodes + case["B"] * (4 * 32 + 16), "flops": 2 * nodes}


# ---- exact values ---------------------------------------------------------------------------


def _exact_recurrence(st):
    """Token by token in 64 bits: S = a S; S += b (v - S k) k^T (or v k^T); o = S q."""
    lens, gdn = st["lens"], st["mode"] == "gdn"
    T, Hk, dk = st["q"].shape
    H, dv = st["v"].shape[1:]
    head = torch.arange(H, device="cuda") // (H // Hk)
    q, k = (st[n].double() for n in ("q", "k"))
    v, decay = st["v"].double(), st["log_a"].double().exp()
    b = st["b"].double() if gdn else None
    order = sorted(range(len(lens)), key=lambda s: -lens[s])
    off = _offsets(lens)
    start = torch.tensor([off[s] for s in order], device="cuda")
    S = torch.zeros(len(lens), H, dv, dk, dtype=torch.float64, device="cuda")
    if st["S"] is not None:
        S += st["S"].double()[order]
    out = torch.empty(T, H, dv, dtype=torch.float64, device="cuda")
    live = len(order)
    for t in range(max(lens)):
        while lens[order[live - 1]] <= t:
            live -= 1
        r = start[:live] + t
        kt, qt = k[r][:, head], q[r][:, head]
        X = S[:live]
        X *= decay[r][:, :, None, None]
        u = v[r]
        if gdn:
            u = b[r][..., None] * (u - torch.einsum("shvk,shk->shv", X, kt))
        X += torch.einsum("shv,shk->shvk", u, kt)
        out[r] = torch.einsum("shvk,shk->shv", X, qt)
    back = torch.empty_like(S)
    back[order] = S
    return out, back


def _exact_sample(st):
    """The log-probability of the sampled token in 64 bits: the kept tokens are those above
    the last kept value, and the first few in order that equal it."""
    R = st["logits"].shape[0]
    tokens, logprob = [], []
    for lo in range(0, R, 64):
        row = slice(lo, min(R, lo + 64))
        y = st["logits"][row].double()
        y = torch.where(y.isnan(), torch.full_like(y, -math.inf), y)
        n, V = y.shape
        t = st["temperature"][row].double()
        desc = torch.sort(y, dim=-1, descending=True).values
        z = torch.where(t[:, None] > 0, desc - desc[:, :1], 0.0) / t.clamp(min=1e-300)[:, None]
        e = torch.where(desc == desc[:, :1], 1.0, torch.exp(z))
        count = torch.where(t > 0, V, 1)
        if st["top_k"] is not None:
            k = st["top_k"][row].long()
            count = torch.where((k > 0) & (k < count), k, count)
        before = torch.cat([torch.zeros(n, 1, dtype=e.dtype, device=e.device),
                            e.cumsum(-1)[:, :-1]], 1)
        within = torch.arange(V, device=e.device) < count[:, None]
        if st["top_p"] is not None:
            p = st["top_p"][row].double()
            mass = torch.where(within, e, 0.0).sum(-1)
            need = (within & (before < (p * mass)[:, None])).sum(-1).clamp(min=1)
            count = torch.where(p < 1, torch.minimum(count, need), count)
        if st["min_p"] is not None:
            count = torch.minimum(count, (e >= st["min_p"][row].double()[:, None]).sum(-1))
        edge = desc.gather(-1, count[:, None] - 1)
        above = y > edge
        same = y == edge
        kept = above | (same & (same.cumsum(-1) <= (count - above.sum(-1))[:, None]))
        d = torch.where(y == desc[:, :1], torch.zeros_like(y),
                        (y - desc[:, :1]) / torch.where(t > 0, t, 1.0)[:, None])
        w = torch.where(kept, torch.exp(d), 0.0)
        total = w.sum(-1)
        token = (w.cumsum(-1) <= (st["uniform"][row].double() * total)[:, None]).sum(-1)
        token = token.clamp(max=V - 1)
        tokens.append(token.to(torch.int32))
        logprob.append(torch.log(w.gather(-1, token[:, None])[:, 0] / total))
    return torch.cat(tokens), torch.cat(logprob)


def exact(case, seed):
    if case["op"] == "accept":
        return None
    st = prepare(case, seed)
    return _exact_sample(st) if case["op"] == "sample" else _exact_recurrence(st)
