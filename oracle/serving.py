"""Float64 CPU oracle of the operators around the tree verification: prompts token by token,
sampling by a full sort of every row, tree acceptance by walking.  Plain numpy; shares nothing
with the CUDA path."""
from __future__ import annotations

import numpy as np


def prefill(q, k, v, log_a, b, offsets, S_in=None, mode="gdn"):
    """(out [T][H][dv], S_out [B][H][dv][dk]): S = a S; S += b (v - S k) k^T (scalar: v k^T);
    out = S q, one token at a time.  Rows that no sequence owns are NaN."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    H, dv, dk = v.shape[1], v.shape[2], q.shape[2]
    share = H // q.shape[1]
    a = np.exp(np.asarray(log_a, np.float64))
    B = len(offsets) - 1
    S = np.zeros((B, H, dv, dk)) if S_in is None else np.array(S_in, np.float64)
    out = np.full(v.shape, np.nan)
    for s in range(B):
        for h in range(H):
            X = S[s, h]
            for t in range(offsets[s], offsets[s + 1]):
                kt, qt = k[t, h // share], q[t, h // share]
                X = a[t, h] * X if a[t, h] else np.zeros_like(X)
                u = b[t, h] * (v[t, h] - X @ kt) if mode == "gdn" else v[t, h]
                X = X + np.outer(u, kt)
                out[t, h] = X @ qt
            S[s, h] = X
    return out, S


def sample_row(x, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob) of one row of logits."""
    x = np.asarray(x, np.float64).copy()
    x[np.isnan(x)] = -np.inf
    V, m = len(x), x.max()
    if m == -np.inf:
        return -1, -np.inf
    order = np.argsort(-x, kind="stable")
    if t == 0:
        return int(order[0]), 0.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == m, 1.0, np.exp((x - m) / t))
    n_k = top_k if 0 < top_k < V else V
    ws = w[order]
    n = n_k
    if top_p < 1:
        mass = np.cumsum(ws[:n_k])
        before = mass - ws[:n_k]
        n = max(1, int(np.sum(before < top_p * mass[-1])))
    n = min(n, int(np.sum(ws >= min_p)))
    kept = np.zeros(V, bool)
    kept[order[:n]] = True
    c = np.cumsum(np.where(kept, w, 0.0))
    hit = np.nonzero((c > u * c[-1]) & kept & (w > 0))[0]
    token = int(hit[0]) if len(hit) else int(np.nonzero(kept & (w > 0))[0][-1])
    return token, float(np.log(w[token] / c[-1]))


def sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None):
    at = lambda x, r, none: none if x is None else x[r]
    got = [sample_row(logits[r], float(uniform[r]), float(at(temperature, r, 1.0)),
                      int(at(top_k, r, 0)), float(at(top_p, r, 1.0)), float(at(min_p, r, 0.0)))
           for r in range(len(uniform))]
    return (np.array([g[0] for g in got], np.int32).reshape(-1),
            np.array([g[1] for g in got], np.float64).reshape(-1))


def accept(draft, target, root, parent, offsets, max_path):
    """(path [B][max_path], length [B], next token [B])."""
    B = len(offsets) - 1
    path = np.full((B, max_path), -1, np.int32)
    count, nxt = np.zeros(B, np.int32), np.zeros(B, np.int32)
    for s in range(B):
        lo, hi = offsets[s], offsets[s + 1]
        cur, want = -1, int(root[s])
        while count[s] < max_path and want >= 0:
            child = [i for i in range(hi - lo)
                     if parent[lo + i] == cur and draft[lo + i] == want]
            if not child:
                break
            cur = child[0]
            path[s, count[s]] = cur
            count[s] += 1
            want = int(target[lo + cur])
        nxt[s] = want
    return path, count, nxt
