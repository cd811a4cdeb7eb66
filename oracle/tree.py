"""Float64 reference of a decoding step over a tree of drafted tokens.

Plain definitions in NumPy and Python, one sequence and one head at a time.
Test infrastructure only; it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from oracle.scored import _probabilities, append


def lineages(parents):
    """Each place's ancestors and itself, root first; empty where there is no node."""
    lines = []
    for i, p in enumerate(parents):
        p = int(p)
        if p == -1:
            lines.append([i])
        elif 0 <= p < i and lines[p]:
            lines.append(lines[p] + [i])
        else:
            lines.append([])
    return lines


def attention(q, k_tree, v_tree, k, v, parents, lens, scale, softcap=0.0, slopes=None,
              window=None):
    """q [B, h, n, d], k_tree and v_tree [B, h_kv, n, d], k and v [B, h_kv, L_max, d] float64.
    Returns O and LSE."""
    B, h, n, d = q.shape
    group = h // k.shape[1]
    o, lse = np.zeros(q.shape), np.full((B, h, n), -np.inf)
    for b in range(B):
        L = int(lens[b])
        lines = lineages(parents[b])
        for hh in range(h):
            g = hh // group
            for i, line in enumerate(lines):
                if not line:
                    continue
                here = L + len(line) - 1
                place = np.concatenate([np.arange(L), L + np.arange(len(line))])
                keys = np.concatenate([k[b, g, :L], k_tree[b, g, line]])
                values = np.concatenate([v[b, g, :L], v_tree[b, g, line]])
                if window is not None:
                    near = place >= here - window
                    place, keys, values = place[near], keys[near], values[near]
                x = keys @ q[b, hh, i] * scale
                if softcap > 0:
                    x = softcap * np.tanh(x / softcap)
                if slopes is not None:
                    x = x - slopes[hh] * (here - place)
                p, lse[b, hh, i:i + 1] = _probabilities(x[None], np.ones((1, x.size), bool))
                o[b, hh, i] = p[0] @ values
    return o, lse


def verify(target, tokens, parents, uniforms, draft=None):
    """One sequence: target and draft [n, V], tokens, parents, uniforms [n].  Returns the path, the
    row that the next token is drawn from, its total, and the least relative distance of a test
    from its border."""
    target = np.where(target > 0, target.astype(np.float64), 0.0)
    draft = None if draft is None else np.where(draft > 0, draft.astype(np.float64), 0.0)
    n, V = target.shape
    path, margin = [0], np.inf
    while True:
        node = path[-1]
        r, Z = target[node], 1.0
        went = False
        for c in range(node + 1, n):
            if int(parents[c]) != node:
                continue
            x = int(tokens[c])
            known = 0 <= x < V
            left = r[x] if known else 0.0
            asked = float(uniforms[c]) * Z * (1.0 if draft is None else
                                              (draft[node, x] if known else 0.0))
            if max(left, asked) > 0:
                margin = min(margin, abs(asked - left) / max(left, asked))
            if asked < left:
                path.append(c)
                went = True
                break
            if draft is None:
                Z -= left
                r = r.copy()
                if known:
                    r[x] = 0.0
            else:
                r = np.maximum(r - Z * draft[node], 0.0)
                Z = r.sum()
        if not went:
            break
    if r.sum() == 0:
        r = target[path[-1]]
    return path, r, margin


def next_tokens(r, u, slack):
    """The tokens that may follow for the random number u when the borders between
    them are known to `slack` of the total: those whose part of [0, 1) is that near."""
    total = r.sum()
    if total == 0:
        return {-1}
    upto = np.cumsum(r) / total
    low = upto - r / total
    return set(np.nonzero((r > 0) & (low <= u + slack) & (upto > u - slack))[0].tolist())


def append_path(cache, scale, tree, path, path_lens, lens, block, int8):
    """Every layer: cache [layers, B, h, L, d] (values of codes, or rows when scale is None),
    scale [layers, B, h, nblk] float32, tree [layers, B, h, n, d].  In place."""
    layers, B, h, L, d = cache.shape
    n = tree.shape[3]
    for b in range(B):
        rows = []
        for node in path[b][:max(0, min(int(path_lens[b]), n))]:
            if not 0 <= node < n:
                break
            rows.append(int(node))
        start = max(0, min(int(lens[b]), L))
        rows = rows[:L - start]
        if not rows:
            continue
        for layer in range(layers):
            new = tree[layer, b:b + 1][:, :, rows]
            if scale is None:
                cache[layer, b, :, start:start + len(rows)] = new[0]
            else:
                append(cache[layer, b:b + 1], scale[layer, b:b + 1], new, [start], [len(rows)],
                       block, int8)
