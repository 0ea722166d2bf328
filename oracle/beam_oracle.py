"""Float64 reference of the operators of a beam search's step, written from their formulas.

``prefix_attention``: every sequence alone, over its prompt's rows followed by its own (the attention of
``mtp_oracle.attention``, causal, with a window and sinks).  ``beam_select``: all candidates of a prompt
listed and sorted.  ``beam_reorder``: tails copied from a copy.
"""

from __future__ import annotations

import math

import numpy as np


def prefix_attention(q, k_new, v_new, k_prefix, v_prefix, k_tail, v_tail, prefix_len, tail_len, m, window=0,
                     sinks=None, gate=None, scale=None):
    """q [seqs*m, nh, dqk], new rows [seqs*m, nkv, d] (normalised and rotated), prompts
    [groups][nkv, cap, d], tails [seqs, nkv, cap, d].  Rows of sequences of negative length are None."""
    nh, dqk = q.shape[1:]
    nkv, dv = v_new.shape[1:]
    seqs, groups = len(tail_len), len(prefix_len)
    scale = 1 / math.sqrt(dqk) if scale is None else scale
    out = [None] * (seqs * m)
    for b in range(seqs):
        t, p = int(tail_len[b]), b // (seqs // groups)
        if t < 0:
            continue
        P = int(prefix_len[p])
        for i in range(m):
            row, pos = np.zeros((nh, dv)), P + t + i
            lo = max(0, pos - window + 1) if window > 0 else 0
            for h in range(nh):
                g = h // (nh // nkv)
                own, new = max(0, lo - P), range(b * m + max(0, lo - P - t), b * m + i + 1)
                K = np.concatenate([k_prefix[p][g][lo:P], k_tail[b][g][own:t], [k_new[j][g] for j in new]]).astype(np.float64)
                V = np.concatenate([v_prefix[p][g][lo:P], v_tail[b][g][own:t], [v_new[j][g] for j in new]]).astype(np.float64)
                lg = K @ np.asarray(q[b * m + i, h], np.float64) * scale
                top = max(list(lg) + ([float(sinks[h])] if sinks is not None else []))
                e = np.exp(lg - top)
                den = e.sum() + (math.exp(float(sinks[h]) - top) if sinks is not None else 0.0)
                row[h] = e @ V / den
            if gate is not None:
                row = row / (1 + np.exp(-np.asarray(gate[b * m + i], np.float64)))
            out[b * m + i] = row
    return out


def beam_candidates(logits, score, length=None, done=None, eos=-1, alpha=0.0):
    """Every candidate of one prompt as (rank, beam, token, score, length, finished), best first."""
    res = []
    for b in range(len(score)):
        s = float(score[b])
        n = 0 if length is None else int(length[b])
        if not math.isfinite(s):
            continue
        if done is not None and done[b]:
            res.append((s / max(n, 1) ** alpha, b, eos, s, n, 1))
            continue
        x = np.asarray(logits[b], np.float64)
        x = np.where(np.isnan(x), -np.inf, x)
        top = x.max()
        if not math.isfinite(top):
            continue
        lse = top + math.log(np.exp(x - top).sum())
        for v in np.flatnonzero(x > -np.inf):
            c = s + (x[v] - lse)
            res.append((c / max(n + 1, 1) ** alpha, b, int(v), c, n + 1, int(v == eos)))
    return sorted(res, key=lambda c: (-c[0], c[1], c[2]))


def beam_select(logits, n_seqs, beams, k, score, length=None, done=None, eos=-1, alpha=0.0):
    """(parent, token, score, length, done), each [n_seqs, k]."""
    at = lambda a, s: None if a is None else a[s * beams:(s + 1) * beams]  # noqa: E731
    none = (-math.inf, -1, -1, -math.inf, 0, 0)
    rows = []
    for s in range(n_seqs):
        c = beam_candidates(at(logits, s), at(score, s), at(length, s), at(done, s), eos, alpha)[:k]
        rows.append(c + [none] * (k - len(c)))
    return tuple(np.array([[c[i] for c in row] for row in rows]) for i in (1, 2, 3, 4, 5))


def beam_reorder(tails, parent, length, beams):
    """tails [rows, nkv, cap, d]."""
    out = np.array(tails)
    for r, (p, n) in enumerate(zip(np.ravel(parent), np.ravel(length))):
        if p >= 0 and n > 0:
            out[r, :, :n] = tails[r // beams * beams + p, :, :n]
    return out
