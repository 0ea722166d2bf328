"""Float64 reference of the draft-tree operators, written from their formulas.

``rope_axes``: "hf2q 0.1.13 src/inference/models/qwen35/mtp.rs" apply_imrope (position ids per
axis, interleaved sections).  ``tree_attention``: the attention of ``mtp_oracle.attention`` with a
visible-key list per row instead of a causal order.  ``tree_accept``, ``tree_commit``: the accepted
prefix and rewind of "cortiq-engine 0.8.49 src/mimo_mtp.rs" on a tree.
"""

from __future__ import annotations

import numpy as np


def axis_of_pair(sections, interleaved):
    n, half = len(sections), sum(sections)
    if not interleaved:
        return [a for a in range(n) for _ in range(sections[a])]
    out = []
    for i in range(half):
        a = i % n
        out.append(a if a and i < n * sections[a] else 0)
    return out


def head_norm(x, w, eps):
    x = np.asarray(x, np.float64)
    if w is None:
        return x
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(w, np.float64)


def rope_axes(x, pos, sections, interleaved, theta):
    """x [rows, heads, d], pos [n_axes, rows]."""
    x = np.array(x, np.float64)
    half = sum(sections)
    axis = axis_of_pair(sections, interleaved)
    for r in range(x.shape[0]):
        ang = np.array([pos[axis[i]][r] * theta ** (-2.0 * i / (2 * half)) for i in range(half)])
        a, b = x[r, :, :half].copy(), x[r, :, half:2 * half].copy()
        x[r, :, :half] = a * np.cos(ang) - b * np.sin(ang)
        x[r, :, half:2 * half] = a * np.sin(ang) + b * np.cos(ang)
    return x


def tree_plan(parents):
    mask, depth = [], []
    for i, p in enumerate(parents):
        mask.append((1 << i) | (mask[p] if p >= 0 else 0))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return mask, depth


def tree_attention(q, k_cache, v_cache, k_new, v_new, mask, depth, window=0, sinks=None, gate=None, scale=None):
    """q [n, nh, dqk], caches [nkv, L, d], new rows [n, nkv, d] (normalised and rotated).  Hidden
    keys take no part at all."""
    n, nh, dqk = q.shape
    nkv, L, _ = k_cache.shape
    dv = v_new.shape[-1]
    scale = 1 / np.sqrt(dqk) if scale is None else scale
    out = np.zeros((n, nh, dv))
    for i in range(n):
        lo = max(0, L + depth[i] - window + 1) if window > 0 else 0
        new = [j for j in range(n) if (mask[i] >> j) & 1 and (window <= 0 or depth[j] > depth[i] - window)]
        for h in range(nh):
            g = h // (nh // nkv)
            K = np.concatenate([k_cache[g, lo:].astype(np.float64), k_new[new, g].reshape(-1, dqk)])
            V = np.concatenate([v_cache[g, lo:].astype(np.float64), v_new[new, g].reshape(-1, dv)])
            lg = K @ q[i, h] * scale
            top = max([-np.inf] + list(lg) + ([float(sinks[h])] if sinks is not None else []))
            if not len(lg):
                continue
            p = np.exp(lg - top)
            den = p.sum() + (np.exp(float(sinks[h]) - top) if sinks is not None else 0.0)
            out[i, h] = p @ V / den
    if gate is not None:
        out = out / (1 + np.exp(-np.asarray(gate, np.float64)))
    return out


def logit_rules(logits, counts=None, repetition=1.0, frequency=0.0, presence=0.0, bias=(), allow=None,
                path_tokens=(), path_mask=None, dtype=np.float64):
    """Rows of final logits; with dtype float32 every step rounds as the device's does."""
    f = dtype
    out = np.array(logits, f)
    V = out.shape[1]
    rep, fr, pr = f(np.float32(repetition)), f(np.float32(frequency)), f(np.float32(presence))
    word = np.zeros(V, np.int64) if counts is None else np.asarray(counts).astype(np.int64) & 0xFFFFFFFF
    for r in range(out.shape[0]):
        c = word & 0x7FFFFFFF
        seen = word != 0
        for j, t in enumerate(path_tokens):
            if path_mask is not None and (path_mask[r] >> j) & 1 and 0 <= t < V:
                c[t] += 1
                seen[t] = True
        l = out[r]
        with np.errstate(invalid="ignore", over="ignore"):
            l = np.where(seen, np.where(l > 0, l / rep, l * rep), l).astype(f)
            l = np.where(seen, l - (c.astype(f) * fr + np.where(c > 0, pr, f(0))), l).astype(f)
            add = {}
            for t, b in bias:
                if 0 <= t < V:
                    add[t] = f(add.get(t, f(0)) + f(np.float32(b)))
            for t, b in add.items():
                l[t] = l[t] + b
        if allow is not None:
            m = np.asarray(allow[r] if np.ndim(allow) == 2 else allow).astype(np.int64) & 0xFFFFFFFF
            v = np.arange(V)
            l = np.where((m[v >> 5] >> (v & 31)) & 1, l, f(-np.inf))
        out[r] = l
    return out


def greedy(rows):
    """(token, value) of each row: lowest index of the largest value, -1 where nothing is above -inf."""
    res = []
    for l in rows:
        x = np.where(np.isnan(l), -np.inf, l)
        t = int(np.argmax(x))
        res.append((t, float(x[t])) if x[t] > -np.inf else (-1, -np.inf))
    return res


def tree_accept(parents, tokens, verify):
    path = [0]
    while True:
        kids = [j for j in range(path[-1] + 1, len(parents))
                if parents[j] == path[-1] and tokens[j] == verify[path[-1]]]
        if not kids:
            return path, [int(verify[i]) for i in path]
        path.append(kids[0])
