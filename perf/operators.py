"""The operators of a draft tree's verification round, as they are measured.

A round over a tree of drafted tokens rotates the queries and keys of its rows (positions on one
or several axes), attends from every node to the cache and to the node's own ancestors, corrects
the head's logits by the request's rules, takes each row's greedy token, walks the accepted path
and moves that path's K/V rows to the end of the cache.  Four kinds of cases:

  rope     per-head norm and rotary positions with several axes, for q and k rows
  attn     attention of a tree of drafted tokens over a cache
  rules    penalties, biases and a grammar mask on logits, and each row's argmax
  commit   the accepted path of a tree and the move of its K/V rows

With ``own`` false, ``run`` computes them with elementary torch operations in float32.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
SEEN = -(1 << 31)  # bit 31 of a count word: the token occurs in the prompt


# ------------------------------------------------------------------------------------- cases
def _attn(name, nh, nkv, dqk, dv, L, n, **kw):
    c = dict(kind="attn", name=name, nh=nh, nkv=nkv, dqk=dqk, dv=dv, rot=dqk, L=L, n=n, window=0,
             gated=False, norm=True, sinks=False, axes=1, theta=1e6, chain=False)
    c.update(kw)
    return c


def listed():
    return [
        # one pending token on the small test layer: the smallest call, where latency counts
        _attn("attn tiny, 1 token", 4, 2, 64, 64, 64, 1),
        # a usual tree of 16 nodes on the 40/8-head layer with gated queries
        _attn("attn 40/8, 16 nodes, 4096", 40, 8, 128, 128, 4096, 16, gated=True),
        # the MoE layer's two wide KV heads, odd counts, image positions on three axes
        _attn("attn 16/2, 13 nodes, 2047", 16, 2, 256, 256, 2047, 13, axes=3),
        # sliding window with sinks, wide keys, no q/k norm, a full tree
        _attn("attn 32/8 window, 64 nodes", 32, 8, 192, 128, 320, 64, window=128, norm=False,
              sinks=True, theta=1e4),
        # the largest: a full tree over a long cache
        _attn("attn 40/8, 64 nodes, 32768", 40, 8, 128, 128, 32768, 64, gated=True),
        # greedy decoding of one token on the small test vocabulary
        dict(kind="rules", name="rules 1 x 4096", rows=1, vocab=4096, nodes=1, bias=4, allow=True,
             logits=False, pen=True),
        # a tree's rows on the 40/8-head layer's vocabulary, logits kept for sampling
        dict(kind="rules", name="rules 16 x 151936", rows=16, vocab=151936, nodes=16, bias=64,
             allow=True, logits=True, pen=True),
        # a full tree and an odd vocabulary, whose rows start at every alignment
        dict(kind="rules", name="rules 64 x 152577", rows=64, vocab=152577, nodes=64, bias=300,
             allow=True, logits=True, pen=True),
        # one token's q and k heads
        dict(kind="rope", name="rope 1 row", rows=1, nh=40, nkv=8, d=128, rot=128, axes=3,
             inter=True, norm=True, gated=True, theta=1e6),
        # a prompt with images: rotation of every q and k head
        dict(kind="rope", name="rope 8192 rows", rows=8192, nh=40, nkv=8, d=128, rot=128, axes=3,
             inter=True, norm=True, gated=True, theta=1e6),
        # a short tree on one draft layer's cache
        dict(kind="commit", name="commit 4 nodes, 1 layer", n=4, layers=1, nkv=2, dqk=64, dv=64,
             L=64),
        # a full tree on the caches of a deep target model
        dict(kind="commit", name="commit 64 nodes, 48 layers", n=64, layers=48, nkv=8, dqk=128,
             dv=128, L=501),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn", "rules", "rules", "rope", "rope", "commit"])
    if kind == "attn":
        while True:
            nkv = rng.choice([1, 2, 3, 4, 8])
            group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
            dqk = 32 * rng.randint(1, 8)
            dv = dqk if rng.random() < 0.7 else 32 * rng.randint(1, 8)
            rot = dqk if rng.random() < 0.7 else 2 * rng.randint(4, dqk // 2)
            L = 0 if rng.random() < 0.08 else _logint(rng, 1, 32768)
            n = _logint(rng, 1, 64)
            c = dict(kind="attn", nh=nkv * group, nkv=nkv, dqk=dqk, dv=dv, rot=rot, L=L, n=n,
                     window=rng.choice([0, 0, 0, _logint(rng, 16, 4096)]),
                     gated=dqk == dv and rng.random() < 0.5, norm=rng.random() < 0.6,
                     sinks=rng.random() < 0.4, axes=rng.choice([1, 1, 3]),
                     theta=rng.choice([1e4, 1e6]), chain=rng.random() < 0.2)
            if c["nh"] * n * (L + 1) * (dqk + dv) <= 40 * 64 * 32768 * 256 and nkv * L * (dqk + dv) <= 8 * 32768 * 256:
                return c
    if kind == "rules":
        rows = _logint(rng, 1, 64)
        return dict(kind="rules", rows=rows, vocab=_logint(rng, 1000, 152000), nodes=rng.randint(1, 64),
                    bias=rng.choice([0, _logint(rng, 1, 300)]), allow=rng.random() < 0.7,
                    logits=rng.random() < 0.6, pen=rng.random() < 0.8)
    if kind == "rope":
        d = 32 * rng.randint(1, 8)
        nkv = rng.choice([1, 2, 3, 4, 8])
        nh = nkv * rng.choice([1, 2, 3, 4, 5])
        return dict(kind="rope", rows=_logint(rng, 1, 8 * 8192 * 48 * 128 // (8 * (nh + nkv) * d) if (nh + nkv) * d > 6144 else 8192),
                    nh=nh, nkv=nkv, d=d, rot=d if rng.random() < 0.5 else 2 * rng.randint(4, d // 2),
                    axes=rng.choice([1, 2, 3, 4]), inter=rng.random() < 0.5, norm=rng.random() < 0.6,
                    gated=rng.random() < 0.4, theta=rng.choice([1e4, 1e6]))
    return dict(kind="commit", n=_logint(rng, 1, 64), layers=rng.randint(1, 48), nkv=rng.randint(1, 8),
                dqk=32 * rng.randint(1, 4), dv=32 * rng.randint(1, 4), L=rng.randint(0, 500))


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _tree(rng, n, chain=False):
    """Parents, ancestor masks (self among them) and depths of a random tree rooted at node 0."""
    parents = [-1] + [i - 1 if chain else rng.randrange(max(0, (i - 1) // 3), i) for i in range(1, n)]
    mask, depth = [], []
    for i, p in enumerate(parents):
        mask.append((1 << i) | (mask[p] if p >= 0 else 0))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return parents, mask, depth


def _i64(words):
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device=DEV)


def _sections(axes, half):
    """Rotary pairs of each axis: the later axes a share each, the first the rest."""
    share = half // (axes + 1)
    return [half - share * (axes - 1)] + [share] * (axes - 1)


def _axis_of_pair(sections, interleaved):
    """Axis of each rotary pair: sections one after another, or dealt in turn (pair i goes to axis
    i mod n while that axis has pairs left, else to axis 0)."""
    n, half = len(sections), sum(sections)
    if not interleaved:
        return [a for a in range(n) for _ in range(sections[a])]
    return [i % n if i % n and i < n * sections[i % n] else 0 for i in range(half)]


def _rope_table(max_pos, rot, theta):
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    ang = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * theta ** (-2.0 * i / rot)
    return torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()


def prepare(case, seed):
    g, rng = _gen(seed), random.Random(seed)
    return {"attn": _prepare_attn, "rules": _prepare_rules, "rope": _prepare_rope,
            "commit": _prepare_commit}[case["kind"]](case, g, rng)


def _prepare_attn(c, g, rng):
    nh, nkv, dqk, dv, L, n = (c[k] for k in ("nh", "nkv", "dqk", "dv", "L", "n"))
    cap = L + n
    parents, mask, depth = _tree(rng, n, c["chain"])
    s = dict(case=c, cap=cap, mask=_i64(mask), depth=torch.tensor(depth, dtype=torch.int32, device=DEV))
    s["qp"] = _randn(g, n, nh * dqk * (2 if c["gated"] else 1))
    s["kp"] = _randn(g, n, nkv * dqk)
    s["vp"] = _randn(g, n, nkv * dv)
    s["k_cache"], s["v_cache"] = _randn(g, nkv, cap, dqk), _randn(g, nkv, cap, dv)
    s["q_norm"] = 1 + 0.1 * _randn(g, dqk) if c["norm"] else None
    s["k_norm"] = 1 + 0.1 * _randn(g, dqk) if c["norm"] else None
    s["sinks"] = _randn(g, nh) if c["sinks"] else None
    s["rope"] = _rope_table(cap, c["rot"], c["theta"])
    s["sections"] = _sections(c["axes"], c["rot"] // 2)
    s["axis"] = torch.tensor(_axis_of_pair(s["sections"], True), device=DEV)
    # text tokens after an image: every axis at its own offset, advancing with the depth
    s["pos"] = torch.stack([s["depth"] + max(0, L - 7 * a) for a in range(c["axes"])]).to(torch.int32).contiguous()
    s["out"] = torch.zeros(n, nh * dv, device=DEV)
    return s


def _prepare_rules(c, g, rng):
    rows, V, nodes = c["rows"], c["vocab"], c["nodes"]
    s = dict(case=c, logits=3 * _randn(g, rows, V))
    _, mask, _ = _tree(rng, nodes)
    # a text's token statistics: few tokens many times
    hist = (V * torch.rand(2048, generator=g, device=DEV) ** 4).long().clamp_(max=V - 1)
    counts = torch.bincount(hist[:1024], minlength=V).to(torch.int32)
    counts[hist[1024:]] |= SEEN
    s["counts"] = counts if c["pen"] else None
    s["rep"], s["freq"], s["pres"] = (1.1, 0.25, 0.5) if c["pen"] else (1.0, 0.0, 0.0)
    s["rep_t"] = torch.tensor(s["rep"], dtype=torch.float32, device=DEV)
    s["path_tokens"] = torch.randint(0, V, (nodes,), generator=g, device=DEV, dtype=torch.int32)
    s["path_mask"] = _i64([mask[i % nodes] for i in range(rows)])
    s["bias_tokens"] = torch.randperm(V, generator=g, device=DEV)[:c["bias"]].to(torch.int32) if c["bias"] else None
    s["bias"] = 2 * _randn(g, c["bias"]) if c["bias"] else None
    if c["allow"]:
        words = (V + 31) // 32
        w = torch.randint(0, 1 << 32, (2, rows, words), generator=g, device=DEV)
        # a grammar allows anything from a few tokens to most of them
        half = torch.rand(rows, 1, generator=g, device=DEV) < 0.5
        w = torch.where(half, w[0] & w[1], w[0] | w[1])
        s["allow"] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous()
    else:
        s["allow"] = None
    s["tokens"] = torch.zeros(rows, dtype=torch.int32, device=DEV)
    s["values"] = torch.zeros(rows, device=DEV)
    s["out"] = torch.zeros(rows, V, device=DEV) if c["logits"] else None
    return s


def _prepare_rope(c, g, rng):
    T, nh, nkv, d = c["rows"], c["nh"], c["nkv"], c["d"]
    s = dict(case=c, max_pos=T + 64)
    s["q"] = _randn(g, T, nh, (2 if c["gated"] else 1) * d)
    s["k"] = _randn(g, T, nkv, d)
    s["q_norm"] = 1 + 0.1 * _randn(g, d) if c["norm"] else None
    s["k_norm"] = 1 + 0.1 * _randn(g, d) if c["norm"] else None
    s["rope"] = _rope_table(s["max_pos"], c["rot"], c["theta"])
    s["sections"] = _sections(c["axes"], c["rot"] // 2)
    s["axis"] = torch.tensor(_axis_of_pair(s["sections"], c["inter"]), device=DEV)
    # time, height and width of image patches: a grid of rows of about 1/64 of the prompt
    t, w = torch.arange(T, device=DEV), max(1, T // 64)
    axes = [t // (w * w), (t // w) % w, t % w, t]
    s["pos"] = torch.stack([axes[a if c["axes"] > 1 else 3] + rng.randrange(64) % (s["max_pos"] - T)
                            for a in range(c["axes"])]).to(torch.int32).contiguous()
    s["yq"], s["yk"] = torch.zeros(T, nh, d, device=DEV), torch.zeros(T, nkv, d, device=DEV)
    return s


def _prepare_commit(c, g, rng):
    n, L = c["n"], c["L"]
    parents, mask, depth = _tree(rng, n)
    kids = [[j for j in range(n) if parents[j] == i] for i in range(n)]
    tokens = [rng.randrange(1000) for _ in range(n)]
    # the verifier agrees with one of a node's children four times out of five
    verify = [tokens[rng.choice(k)] if k and rng.random() < 0.8 else 1000 + rng.randrange(1000) for k in kids]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = dict(case=c, cap=L + n + 11, parents=i32(parents), tokens=i32(tokens), verify=i32(verify))
    s["k"] = _randn(g, c["layers"], c["nkv"], s["cap"], c["dqk"])
    s["v"] = _randn(g, c["layers"], c["nkv"], s["cap"], c["dv"])
    s["path"], s["emitted"] = i32([0] * n), i32([0] * n)
    s["count"] = i32([0])
    return s


# ------------------------------------------------------------------------------------- passes
def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"attn": _own_attn, "rules": _own_rules, "rope": _own_rope, "commit": _own_commit}[kind](s)
    return {"attn": _plain_attn, "rules": _plain_rules, "rope": _plain_rope, "commit": _plain_commit}[kind](s)


def _norm(x, w, eps=1e-6):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _rotate(x, table, pos, axis, rot):
    """x [T, heads, d]: pairs (i, i + rot/2) turned by the angle of pair i at its axis' position."""
    half = rot // 2
    cs = table[pos[axis].T.long(), torch.arange(half, device=x.device)][:, None]  # [T, 1, half, 2]
    a, b = x[..., :half], x[..., half:rot]
    return torch.cat([a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0], x[..., rot:]], -1)


def _bits(words, n):
    return (words[:, None] >> torch.arange(n, device=words.device)) & 1 == 1


def _plain_attn(s):
    c = s["case"]
    nh, nkv, dqk, dv, L, n = (c[k] for k in ("nh", "nkv", "dqk", "dv", "L", "n"))
    G = nh // nkv
    qp = s["qp"].view(n, nh, -1)
    q = _rotate(_norm(qp[..., :dqk], s["q_norm"]), s["rope"], s["pos"], s["axis"], c["rot"])
    k = _rotate(_norm(s["kp"].view(n, nkv, dqk), s["k_norm"]), s["rope"], s["pos"], s["axis"], c["rot"])
    s["k_cache"][:, L:L + n] = k.transpose(0, 1)
    s["v_cache"][:, L:L + n] = s["vp"].view(n, nkv, dv).transpose(0, 1)
    K, V = s["k_cache"][:, :L + n], s["v_cache"][:, :L + n]
    qg = q.view(n, nkv, G, dqk).permute(1, 2, 0, 3).reshape(nkv, G * n, dqk)
    logit = (qg @ K.transpose(1, 2)).view(nkv, G, n, L + n) / math.sqrt(dqk)
    seen = torch.cat([torch.ones(n, L, dtype=torch.bool, device=DEV), _bits(s["mask"], n)], 1)
    if c["window"]:
        at = torch.cat([torch.arange(L, device=DEV), L + s["depth"].long()])
        seen = seen & (at[None] > (L + s["depth"].long())[:, None] - c["window"])
    logit = torch.where(seen, logit, -math.inf)
    top = logit.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(nkv, G, 1, 1)
        top = torch.maximum(top, sink)
    p = torch.exp(logit - top)
    den = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        den = den + torch.exp(sink - top)
    o = (p.view(nkv, G * n, L + n) @ V).view(nkv, G, n, dv) / den
    o = o.permute(2, 0, 1, 3).reshape(n, nh, dv)
    if c["gated"]:
        o = o * torch.sigmoid(qp[..., dqk:])
    return o.reshape(n, nh * dv), s["k_cache"][:, L:], s["v_cache"][:, L:]


def _plain_rules(s):
    c = s["case"]
    rows, V, nodes = c["rows"], c["vocab"], c["nodes"]
    l = s["logits"]
    if c["pen"]:
        path = torch.zeros(rows, V, dtype=torch.int32, device=DEV)
        path.scatter_add_(1, s["path_tokens"].long().expand(rows, nodes), _bits(s["path_mask"], nodes).int())
        cnt = (s["counts"] & 0x7FFFFFFF) + path
        seen = (s["counts"] != 0) | (path > 0)
        l = torch.where(seen, torch.where(l > 0, l / s["rep_t"], l * s["rep_t"]), l)
        l = l - (cnt.float() * s["freq"] + (cnt > 0).float() * s["pres"])
    if s["bias"] is not None:
        l = l.clone()
        l[:, s["bias_tokens"].long()] += s["bias"]
    if s["allow"] is not None:
        word = s["allow"][:, torch.arange(V, device=DEV) >> 5]
        l = torch.where((word >> (torch.arange(V, device=DEV) & 31)) & 1 == 1, l, -math.inf)
    top = l.amax(-1)
    # the lowest index among equal values; -1 where nothing is above -inf
    at = torch.where(l == top[:, None], torch.arange(V, device=DEV), V).amin(-1)
    tok = torch.where(top > -math.inf, at, -1).to(torch.int32)
    return (tok, top, l) if c["logits"] else (tok, top)


def _plain_rope(s):
    c = s["case"]
    q = _rotate(_norm(s["q"][..., :c["d"]], s["q_norm"]), s["rope"], s["pos"], s["axis"], c["rot"])
    k = _rotate(_norm(s["k"], s["k_norm"]), s["rope"], s["pos"], s["axis"], c["rot"])
    return q, k


def _plain_commit(s):
    c = s["case"]
    n, L = c["n"], c["L"]
    parents, tokens, verify = s["parents"].long(), s["tokens"], s["verify"]
    i = torch.arange(n, device=DEV)
    up = parents.clamp(min=0)
    match = (parents >= 0) & (tokens == verify[up])
    # of several matching children the lowest index is taken
    same = match[:, None] & match[None] & (parents[:, None] == parents[None])
    first = match & ~(same & (i[None] < i[:, None])).any(1)
    # a node is on the path when its whole line of ancestors is: 2^k steps up in k doublings
    step = torch.zeros(n, n, device=DEV)
    step[i, up] = 1.0
    reach = step + torch.eye(n, device=DEV)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    ok = first | (i == 0)
    on = ~((reach > 0) & ~ok[None]).any(1)
    count = on.sum().to(torch.int32).view(1)
    order = torch.sort(torch.where(on, i, n + i)).values  # the path's nodes first, in order
    keep = i < count
    path = torch.where(keep, order, -1)
    src = torch.where(keep, order, i)
    emitted = torch.where(keep, verify[src], -1)
    for_k = s["k"][:, :, L + src]
    for_v = s["v"][:, :, L + src]
    s["k"][:, :, L:L + n] = torch.where(keep[:, None], for_k, s["k"][:, :, L:L + n])
    s["v"][:, :, L:L + n] = torch.where(keep[:, None], for_v, s["v"][:, :, L:L + n])
    return path.to(torch.int32), emitted, count, s["k"][:, :, L:L + n], s["v"][:, :, L:L + n]


def _own_attn(s):
    import mtp_speculative_draft_gb300 as M
    c = s["case"]
    h = s.get("handle")
    if h is None:  # what a program makes once for a layer: geometry, positions, workspace
        geom = M.attn_geom(c["nh"], c["nkv"], c["dqk"], c["dv"], c["rot"], c["window"], c["gated"])
        axes = M.rope_axes(s["sections"], s["pos"], s["rope"], interleaved=True) if c["axes"] > 1 else None
        tree = M.draft_tree(s["mask"], s["depth"], axes=axes)
        h = s["handle"] = (geom, tree, M.workspace(M.attn_tree_sink_workspace_bytes(geom, c["n"], c["L"])))
    M.attn_tree_sink(h[0], h[1], s["qp"], s["kp"], s["vp"], s["q_norm"], s["k_norm"], s["rope"], s["sinks"],
                     s["k_cache"], s["v_cache"], c["L"], s["out"], h[2])
    return s["out"], s["k_cache"][:, c["L"]:], s["v_cache"][:, c["L"]:]


def _own_rules(s):
    import mtp_speculative_draft_gb300 as M
    c = s["case"]
    h = s.get("handle")
    if h is None:
        rules = M.logit_rules(c["vocab"], repetition=s["rep"], frequency=s["freq"], presence=s["pres"],
                              counts=s["counts"], bias_tokens=s["bias_tokens"], bias=s["bias"], allow=s["allow"],
                              path_tokens=s["path_tokens"] if c["pen"] else None,
                              path_mask=s["path_mask"] if c["pen"] else None)
        h = s["handle"] = (rules, M.workspace(M.logit_rules_argmax_workspace_bytes(c["rows"])))
    M.logit_rules_argmax(h[0], s["logits"], s["tokens"], s["values"], s["out"], h[1])
    return (s["tokens"], s["values"], s["out"]) if c["logits"] else (s["tokens"], s["values"])


def _own_rope(s):
    import mtp_speculative_draft_gb300 as M
    c = s["case"]
    h = s.get("handle")
    if h is None:
        axes = M.rope_axes(s["sections"], s["pos"], s["rope"], interleaved=c["inter"])
        h = s["handle"] = (axes, M.workspace(M.rope_axes_rows_workspace_bytes()))
    M.rope_axes_rows(h[0], [(s["q"][..., :c["d"]], s["yq"], s["q_norm"]), (s["k"], s["yk"], s["k_norm"])], h[1])
    return s["yq"], s["yk"]


def _own_commit(s):
    import mtp_speculative_draft_gb300 as M
    c = s["case"]
    h = s.get("handle")
    if h is None:
        h = s["handle"] = (M.kv_caches(s["k"].unbind(0), s["v"].unbind(0)), M.workspace(M.mtp_tree_workspace_bytes()))
    M.mtp_tree_accept(s["parents"], s["tokens"], s["verify"], s["path"], s["emitted"], s["count"])
    M.kv_tree_commit(h[0], s["path"], c["L"], h[1])
    L = c["L"]
    return s["path"], s["emitted"], s["count"], s["k"][:, :, L:L + c["n"]], s["v"][:, :, L:L + c["n"]]


# ------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["kind"] == "attn":
        nh, nkv, dqk, dv, L, n = (c[k] for k in ("nh", "nkv", "dqk", "dv", "L", "n"))
        keys = min(L, c["window"] - 1 + n) if c["window"] else L
        rows = n * (nh * dqk * (2 if c["gated"] else 1) + nh * dv + 2 * nkv * (dqk + dv) + c["rot"])
        seen = (min(L, c["window"]) if c["window"] else L) + 1
        return {"bytes": 4 * (nkv * keys * (dqk + dv) + rows), "flops": 2 * nh * n * seen * (dqk + dv)}
    if c["kind"] == "rules":
        rows, V = c["rows"], c["vocab"]
        b = 4 * rows * V * (2 if c["logits"] else 1) + (rows * V // 8 if c["allow"] else 0)
        b += 4 * V if c["pen"] else 0
        return {"bytes": b + 8 * c["bias"] + 8 * rows, "flops": 4 * rows * V}
    if c["kind"] == "rope":
        values = c["rows"] * (c["nh"] + c["nkv"]) * c["d"]
        return {"bytes": 8 * values + 4 * c["rows"] * (c["axes"] + c["rot"]), "flops": (7 if c["norm"] else 3) * values}
    # the expected path has about five nodes whatever the tree: the rows of one node are the floor
    row = 4 * c["layers"] * c["nkv"] * (c["dqk"] + c["dv"])
    return {"bytes": 2 * row * min(c["n"], 4) + 20 * c["n"], "flops": c["n"]}


# ------------------------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "rules": _exact_rules, "rope": _exact_rope, "commit": _exact_commit}[case["kind"]](s)


def _exact_heads(x, w, pos, axis, rot, theta):
    """[T, heads, d] in 64 bits: x / rms(x) * w, then the rotation as a complex product."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
    half = rot // 2
    freq = theta ** (-torch.arange(half, device=DEV, dtype=torch.float64) * 2 / rot)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[axis].T * freq)
    z = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous()) * turn[:, None]
    return torch.cat([z.real, z.imag, x[..., rot:]], -1)


def _exact_attn(s):
    c = s["case"]
    nh, nkv, dqk, dv, L, n = (c[k] for k in ("nh", "nkv", "dqk", "dv", "L", "n"))
    raw = s["qp"].view(n, nh, -1)
    q = _exact_heads(raw[..., :dqk], s["q_norm"], s["pos"], s["axis"], c["rot"], c["theta"])
    k = _exact_heads(s["kp"].view(n, nkv, dqk), s["k_norm"], s["pos"], s["axis"], c["rot"], c["theta"])
    v = s["vp"].view(n, nkv, dv).double()
    words = [int(w) & ((1 << 64) - 1) for w in s["mask"].tolist()]
    line = torch.tensor([[(w >> j) & 1 for j in range(n)] for w in words], device=DEV, dtype=torch.bool)
    depth = s["depth"].long()
    cached = torch.ones(n, L, device=DEV, dtype=torch.bool)
    if c["window"]:
        cached = torch.arange(L, device=DEV)[None] > (L + depth - c["window"])[:, None]
        line = line & (depth[None] > (depth - c["window"])[:, None])
    sees = torch.cat([cached, line], 1)
    out = torch.zeros(n, nh, dv, device=DEV, dtype=torch.float64)
    for h in range(nh):  # one head at a time, to bound the memory
        kv = h // (nh // nkv)
        keys = torch.cat([s["k_cache"][kv, :L].double(), k[:, kv]])
        vals = torch.cat([s["v_cache"][kv, :L].double(), v[:, kv]])
        e = torch.einsum("td,kd->tk", q[:, h], keys) * dqk ** -0.5
        e = e.masked_fill(~sees, -math.inf)
        if s["sinks"] is not None:
            e = torch.cat([e, s["sinks"][h].double().expand(n, 1)], 1)
        out[:, h] = torch.softmax(e, -1)[:, :L + n] @ vals
    if c["gated"]:
        out = out / (1 + torch.exp(-raw[..., dqk:].double()))
    return out.reshape(n, nh * dv), k.transpose(0, 1), v.transpose(0, 1)


def _exact_rules(s):
    c = s["case"]
    V = c["vocab"]
    words = [int(w) & ((1 << 64) - 1) for w in s["path_mask"].tolist()]
    path = s["path_tokens"].tolist()
    rows = s["logits"].double().cpu().numpy()
    if c["pen"]:
        word = s["counts"].cpu().numpy().astype(np.int64)
        rep = float(np.float32(s["rep"]))
        for r, w in enumerate(words):
            own_path = np.bincount([path[j] for j in range(c["nodes"]) if (w >> j) & 1], minlength=V)
            made = (word & 0x7FFFFFFF) + own_path
            hit = (word != 0) | (own_path > 0)
            rows[r] = np.where(hit, rows[r] * np.where(rows[r] > 0, 1 / rep, rep), rows[r])
            rows[r] -= s["freq"] * made + s["pres"] * (made > 0)
    if s["bias"] is not None:
        np.add.at(rows, (slice(None), s["bias_tokens"].cpu().numpy()), s["bias"].double().cpu().numpy())
    if s["allow"] is not None:
        bits = np.unpackbits(s["allow"].cpu().numpy().view(np.uint8).reshape(c["rows"], -1), axis=1, bitorder="little")
        rows[bits[:, :V] == 0] = -math.inf
    top = torch.from_numpy(rows.max(1))
    return (None, top, torch.from_numpy(rows)) if c["logits"] else (None, top)


def _exact_rope(s):
    c = s["case"]
    return tuple(_exact_heads(x, w, s["pos"], s["axis"], c["rot"], c["theta"])
                 for x, w in ((s["q"][..., :c["d"]], s["q_norm"]), (s["k"], s["k_norm"])))


def _exact_commit(s):
    c = s["case"]
    parents, tokens, verify = (s[k].tolist() for k in ("parents", "tokens", "verify"))
    path = [0]
    while True:
        nxt = [j for j in range(c["n"]) if parents[j] == path[-1] and tokens[j] == verify[path[-1]]]
        if not nxt:
            break
        path.append(nxt[0])
    L = c["L"]
    k, v = (s[x][:, :, L:L + c["n"]].double() for x in ("k", "v"))
    k2, v2 = k.clone(), v.clone()
    for j, node in enumerate(path):
        k2[:, :, j], v2[:, :, j] = k[:, :, node], v[:, :, node]
    return None, None, None, k2, v2
