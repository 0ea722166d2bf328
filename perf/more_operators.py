"""The operators of a beam search over prompts, as they are measured.

Many sequences continue one prompt: each step attends from every sequence's new rows to the prompt's
K/V rows, which are kept once, and to the sequence's own tail of rows; the head's logits then extend
the beams of a prompt, the best of all extensions survive, and the survivors' tails move to their
places.  Three kinds of cases:

  attn     attention of a batch that shares prefixes (beams, samples, or chains of drafts to verify)
  select   log-probabilities, scores and the selection over beams and vocabulary
  reorder  the tails of K/V rows of the beams that survived

With ``own`` false, ``run`` computes them with elementary torch operations: attention in float32, the
selection's scores in 64 bits, as values next to the border decide which tokens are taken.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------- cases
def _attn(name, nh, nkv, dqk, dv, groups, per, prefix, tail, **kw):
    """``per`` sequences for each of ``groups`` prompts of up to ``prefix`` rows, tails of up to ``tail`` rows,
    ``m`` new rows a sequence."""
    c = dict(kind="attn", name=name, nh=nh, nkv=nkv, dqk=dqk, dv=dv, rot=dqk, groups=groups, per=per,
             prefix=prefix, tail=tail, m=1, window=0, gated=False, norm=True, sinks=False, theta=1e6,
             even=False, idle=False)
    c.update(kw)
    return c


def listed():
    return [
        # four beams on the small test layer, a short prompt: the smallest call, where latency counts
        _attn("attn tiny, 4 beams", 4, 2, 64, 64, 1, 4, 64, 3, even=True),
        # eight beams of one prompt on the 40/8-head layer with gated queries
        _attn("attn 40/8, 8 beams, 4096", 40, 8, 128, 128, 1, 8, 4096, 63, gated=True, even=True),
        # the MoE layer's two wide KV heads: three prompts of odd lengths, five samples each, one of them ended
        _attn("attn 16/2, 3 x 5, 2047", 16, 2, 256, 256, 3, 5, 2047, 301, idle=True),
        # chains of four drafts to verify: sliding window with sinks, wide keys, no q/k norm
        _attn("attn 32/8 window, 16 x 4 rows", 32, 8, 192, 128, 1, 16, 320, 77, m=4, window=128, norm=False,
              sinks=True, theta=1e4),
        # samples that have grown longer than their prompt: the tails are most of the work
        _attn("attn 40/8, 24 samples, tails 2048", 40, 8, 128, 128, 1, 24, 1024, 2048),
        # the largest: 64 samples of a long prompt
        _attn("attn 40/8, 64 samples, 32768", 40, 8, 128, 128, 1, 64, 32768, 256, gated=True),
        # four beams on the small test vocabulary
        dict(kind="select", name="select 4 x 4096", seqs=1, beams=4, vocab=4096, k=4, alpha=0.0, mask=0.0, done=False),
        # eight beams on the 40/8-head layer's vocabulary, twice as many candidates, length penalty
        dict(kind="select", name="select 8 x 151936", seqs=1, beams=8, vocab=151936, k=16, alpha=0.6, mask=0.0,
             done=True),
        # sixteen prompts of four beams, an odd vocabulary whose rows start at every alignment, a grammar's mask
        dict(kind="select", name="select 16 x 4 x 152577", seqs=16, beams=4, vocab=152577, k=8, alpha=1.0, mask=0.5,
             done=True),
        # five beams' short tails on one layer
        dict(kind="reorder", name="reorder 5 beams, 1 layer", seqs=1, beams=5, layers=1, nkv=2, dqk=64, dv=64, tail=17),
        # eight prompts of four beams on the caches of a deep target model
        dict(kind="reorder", name="reorder 8 x 4 beams, 48 layers", seqs=8, beams=4, layers=48, nkv=8, dqk=128, dv=128,
             tail=101),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn", "attn", "select", "select", "reorder"])
    if kind == "attn":
        while True:
            nkv = rng.choice([1, 2, 3, 4, 8])
            nh = nkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
            dqk = 32 * rng.randint(1, 8)
            dv = dqk if rng.random() < 0.7 else 32 * rng.randint(1, 8)
            c = _attn("", nh, nkv, dqk, dv, rng.choice([1, 1, 1, 2, 3, 4]), _logint(rng, 1, 64),
                      0 if rng.random() < 0.08 else _logint(rng, 1, 32768),
                      0 if rng.random() < 0.15 else _logint(rng, 1, 2048),
                      rot=dqk if rng.random() < 0.7 else 2 * rng.randint(4, dqk // 2),
                      m=rng.choice([1, 1, 1, 1, 2, 3, 5, 8]), window=rng.choice([0, 0, 0, _logint(rng, 16, 4096)]),
                      gated=dqk == dv and rng.random() < 0.5, norm=rng.random() < 0.6, sinks=rng.random() < 0.4,
                      theta=rng.choice([1e4, 1e6]), even=rng.random() < 0.4, idle=rng.random() < 0.3)
            del c["name"]
            seqs = c["groups"] * c["per"]
            if (c["nh"] * seqs * c["m"] * (c["prefix"] + c["tail"]) <= 40 * 64 * 33024 // 2
                    and nkv * c["groups"] * c["prefix"] * (dqk + dv) <= 8 * 32768 * 256
                    and nkv * seqs * c["tail"] * (dqk + dv) <= 8 * 24 * 2048 * 256):
                return c
    if kind == "select":
        beams = _logint(rng, 1, 16)
        return dict(kind="select", seqs=_logint(rng, 1, 64 // beams), beams=beams, vocab=_logint(rng, 1000, 152000),
                    k=rng.choice([1, beams, 2 * beams, rng.randint(1, 32)]), alpha=rng.choice([0.0, 0.6, 1.0]),
                    mask=rng.choice([0.0, 0.0, 0.5, 0.999]), done=rng.random() < 0.5)
    return dict(kind="reorder", seqs=_logint(rng, 1, 8), beams=_logint(rng, 1, 8), layers=rng.randint(1, 24),
                nkv=rng.randint(1, 8), dqk=32 * rng.randint(1, 4), dv=32 * rng.randint(1, 4), tail=_logint(rng, 1, 200))


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _lengths(c):
    """Rows of each prompt, and of each sequence's tail (-1: a sequence that has ended)."""
    prefix = [max(0, c["prefix"] - 17 * i) for i in range(c["groups"])]
    n = c["groups"] * c["per"]
    # beams are of one length; samples began at different times
    tail = [c["tail"] if c["even"] else c["tail"] - c["tail"] * ((7 * i) % n) // n for i in range(n)]
    if c["idle"] and n > 1:
        tail[n // 2] = -1
    return prefix, tail


def _rope_table(max_pos, rot, theta):
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    ang = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * theta ** (-2.0 * i / rot)
    return torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()


def prepare(case, seed):
    return {"attn": _prepare_attn, "select": _prepare_select, "reorder": _prepare_reorder}[case["kind"]](case, seed)


def _prepare_attn(c, seed):
    g = _gen(seed)
    nh, nkv, dqk, dv, m = (c[k] for k in ("nh", "nkv", "dqk", "dv", "m"))
    n, cap = c["groups"] * c["per"], c["tail"] + m + 5
    prefix, tail = _lengths(c)
    s = dict(case=c, prefix_len=_i32(prefix), tail_len=_i32(tail))
    s["qp"] = _randn(g, n * m, nh * dqk * (2 if c["gated"] else 1))
    s["kp"], s["vp"] = _randn(g, n * m, nkv * dqk), _randn(g, n * m, nkv * dv)
    s["k_prefix"] = _randn(g, c["groups"], nkv, max(1, c["prefix"]), dqk)
    s["v_prefix"] = _randn(g, c["groups"], nkv, max(1, c["prefix"]), dv)
    s["k_tail"], s["v_tail"] = _randn(g, n, nkv, cap, dqk), _randn(g, n, nkv, cap, dv)
    s["q_norm"] = 1 + 0.1 * _randn(g, dqk) if c["norm"] else None
    s["k_norm"] = 1 + 0.1 * _randn(g, dqk) if c["norm"] else None
    s["sinks"] = _randn(g, nh) if c["sinks"] else None
    s["rope"] = _rope_table(c["prefix"] + c["tail"] + m, c["rot"], c["theta"])
    s["out"] = torch.zeros(n * m, nh * dv, device=DEV)
    return s


def _prepare_select(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    rows, V = c["seqs"] * c["beams"], c["vocab"]
    s = dict(case=c, logits=3 * _randn(g, rows, V), eos=2)
    if c["mask"]:  # what a grammar forbids is at -inf; every row keeps some tokens
        gone = torch.rand(rows, V, generator=g, device=DEV) < c["mask"]
        gone[:, 5:9] = False
        s["logits"].masked_fill_(gone, -math.inf)
    length = [rng.randint(10, 30) for _ in range(c["seqs"])]
    # the beams of a prompt lie a few nats apart, best first
    score = [-2.0 * n - 0.7 * b - rng.random() for n in length for b in range(c["beams"])]
    done = [int(c["done"] and c["beams"] > 1 and b == 1 and rng.random() < 0.7) for _ in length for b in range(c["beams"])]
    length = [n - 3 * d for n, d in zip([n for n in length for _ in range(c["beams"])], done)]
    s["score"] = torch.tensor(score, dtype=torch.float32, device=DEV)
    s["length"], s["done"] = _i32(length), _i32(done) if c["done"] else None
    out = (c["seqs"], c["k"])
    s["parent"], s["token"], s["new_length"], s["new_done"] = (
        torch.zeros(out, dtype=torch.int32, device=DEV) for _ in range(4))
    s["new_score"] = torch.zeros(out, device=DEV)
    return s


def _parents(c, rng):
    """Parents as a selection leaves them: the better beams have more children, some beams none."""
    return [[min(rng.randrange(c["beams"]), rng.randrange(c["beams"])) for _ in range(c["beams"])]
            for _ in range(c["seqs"])]


def _prepare_reorder(c, seed):
    g, rng = _gen(seed), random.Random(seed)
    n, cap = c["seqs"] * c["beams"], c["tail"] + 6
    s = dict(case=c, parent=_i32(_parents(c, rng)))
    s["length"] = _i32([c["tail"] - (i // c["beams"]) % max(1, c["tail"]) for i in range(n)])
    s["k"], s["v"] = _randn(g, c["layers"], n, c["nkv"], cap, c["dqk"]), _randn(g, c["layers"], n, c["nkv"], cap, c["dv"])
    return s


# ------------------------------------------------------------------------------------- passes
def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"attn": _own_attn, "select": _own_select, "reorder": _own_reorder}[kind](s)
    return {"attn": _plain_attn, "select": _plain_select, "reorder": _plain_reorder}[kind](s)


def _norm(x, w, eps=1e-6):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _rotate(x, table, pos, rot):
    """x [rows, heads, d]: pairs (i, i + rot/2) turned by the angle of pair i at the row's position."""
    half = rot // 2
    cs = table[pos][:, None]  # [rows, 1, half, 2]
    a, b = x[..., :half], x[..., half:rot]
    return torch.cat([a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0], x[..., rot:]], -1)


def _append(cache, rows, at, active):
    """Row r of sequence b to cache row at[b, r], of the sequences that are active."""
    i = torch.arange(cache.shape[0], device=DEV)[:, None]
    cache[i, :, at] = torch.where(active[:, None, None, None], rows, cache[i, :, at])


def _plain_attn(s):
    c = s["case"]
    nh, nkv, dqk, dv, m = (c[k] for k in ("nh", "nkv", "dqk", "dv", "m"))
    G, groups, per = nh // nkv, c["groups"], c["per"]
    n = groups * per
    plen, tlen = s["prefix_len"].long().repeat_interleave(per), s["tail_len"].long()
    active, first = tlen >= 0, tlen.clamp(min=0)
    step = torch.arange(m, device=DEV)
    at = first[:, None] + step                      # tail row of each new row [n, m]
    pos = plen[:, None] + at                        # and its position
    qp = s["qp"].view(n * m, nh, -1)
    q = _rotate(_norm(qp[..., :dqk], s["q_norm"]), s["rope"], pos.view(-1), c["rot"])
    k = _rotate(_norm(s["kp"].view(n * m, nkv, dqk), s["k_norm"]), s["rope"], pos.view(-1), c["rot"])
    _append(s["k_tail"], k.view(n, m, nkv, dqk), at, active)
    _append(s["v_tail"], s["vp"].view(n, m, nkv, dv), at, active)
    kp, vp, kt, vt = s["k_prefix"], s["v_prefix"], s["k_tail"], s["v_tail"]
    P, cap = kp.shape[2], kt.shape[2]
    q = q.view(n, m, nkv, G, dqk).permute(0, 2, 1, 3, 4)  # [n, nkv, m, G, dqk]
    # all rows of a prompt against its keys at once, each sequence's against its own
    shared = q.reshape(groups, per, nkv, m * G, dqk).transpose(1, 2).reshape(groups, nkv, per * m * G, dqk) @ kp.transpose(2, 3)
    shared = shared.view(groups, nkv, per, m, G, P).transpose(1, 2).reshape(n, nkv, m, G, P)
    mine = (q.reshape(n, nkv, m * G, dqk) @ kt.transpose(2, 3)).view(n, nkv, m, G, cap)
    key, tkey = torch.arange(P, device=DEV), torch.arange(cap, device=DEV)
    seen = (key < plen[:, None, None]).expand(n, m, P)
    tseen = tkey <= at[..., None]
    if c["window"]:
        low = pos[..., None] - c["window"]
        seen, tseen = seen & (key > low), tseen & (plen[:, None, None] + tkey > low)
    logit = torch.cat([torch.where(seen[:, None, :, None], shared, -math.inf),
                       torch.where(tseen[:, None, :, None], mine, -math.inf)], -1) / math.sqrt(dqk)
    top = logit.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(nkv, 1, G, 1)
        top = torch.maximum(top, sink)
    p = torch.exp(logit - top)
    den = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        den = den + torch.exp(sink - top)
    ps = p[..., :P].reshape(groups, per, nkv, m * G, P).transpose(1, 2).reshape(groups, nkv, per * m * G, P)
    o = (ps @ vp).view(groups, nkv, per, m, G, dv).transpose(1, 2).reshape(n, nkv, m, G, dv)
    o = (o + (p[..., P:].reshape(n, nkv, m * G, cap) @ vt).view(n, nkv, m, G, dv)) / den
    o = o.permute(0, 2, 1, 3, 4).reshape(n, m, nh, dv)
    if c["gated"]:
        o = o * torch.sigmoid(qp[..., dqk:].view(n, m, nh, dv))
    s["out"].copy_(torch.where(active[:, None, None, None], o, s["out"].view(n, m, nh, dv)).reshape(n * m, nh * dv))
    return s["out"], kt, vt


def _plain_select(s):
    c = s["case"]
    S, B, V, k = c["seqs"], c["beams"], c["vocab"], c["k"]
    l = s["logits"].double()
    top = l.amax(-1, keepdim=True)
    logp = l - (top + torch.exp(l - top).sum(-1, keepdim=True).log())
    done = s["done"].bool() if s["done"] is not None else torch.zeros(S * B, dtype=torch.bool, device=DEV)
    # an ended beam has one way to go on: as it is
    keep = torch.where(torch.arange(V, device=DEV) == s["eos"], 0.0, -math.inf).double()
    score = s["score"].double()[:, None] + torch.where(done[:, None], keep, logp)
    length = s["length"] + (~done).int()
    rank = (score / (length.clamp(min=1).double() ** c["alpha"])[:, None]).view(S, B * V)
    if B * V < k:
        rank = torch.cat([rank, rank.new_full((S, k - B * V), -math.inf)], 1)
    # equal ranks: the lower beam, then the lower token
    rank, at = torch.sort(rank, dim=-1, descending=True, stable=True)
    rank, at = rank[:, :k], at[:, :k].clamp(max=B * V - 1)
    there = rank > -math.inf
    token = torch.where(there, at % V, -1)
    parent = torch.where(there, at // V, -1)
    row = parent.clamp(min=0) + B * torch.arange(S, device=DEV)[:, None]
    new = torch.where(there, score.view(S, B * V).gather(1, at), -math.inf).float()
    new_len = torch.where(there, length[row], 0).to(torch.int32)
    new_done = (there & (done[row] | (token == s["eos"]))).to(torch.int32)
    return parent.to(torch.int32), token.to(torch.int32), new, new_len, new_done


def _plain_reorder(s):
    c = s["case"]
    S, B = c["seqs"], c["beams"]
    src = (s["parent"].long() + B * torch.arange(S, device=DEV)[:, None]).view(-1)
    take = torch.arange(s["k"].shape[3], device=DEV) < s["length"][:, None]  # [rows, cap]
    for x in (s["k"], s["v"]):
        for layer in x:
            layer.copy_(torch.where(take[:, None, :, None], layer[src], layer))
    return s["k"], s["v"]


def _own_attn(s):
    import mtp_speculative_draft_gb300 as M
    c = s["case"]
    h = s.get("handle")
    if h is None:  # what a program makes once: geometry, lengths, workspace
        geom = M.attn_geom(c["nh"], c["nkv"], c["dqk"], c["dv"], c["rot"], c["window"], c["gated"])
        batch = M.prefix_batch(s["prefix_len"], s["tail_len"], c["prefix"], c["tail"], m=c["m"])
        h = s["handle"] = (geom, batch, M.workspace(M.attn_prefix_sink_workspace_bytes(geom, batch)))
    M.attn_prefix_sink(h[0], h[1], s["qp"], s["kp"], s["vp"], s["q_norm"], s["k_norm"], s["rope"], s["sinks"],
                       s["k_prefix"], s["v_prefix"], s["k_tail"], s["v_tail"], s["out"], h[2])
    return s["out"], s["k_tail"], s["v_tail"]


def _own_select(s):
    import mtp_speculative_draft_gb300 as M
    c = s["case"]
    h = s.get("handle")
    if h is None:
        beams = M.beam_set(c["seqs"], c["beams"], c["vocab"], s["score"], length=s["length"], done=s["done"],
                           eos=s["eos"], length_penalty=c["alpha"])
        h = s["handle"] = (beams, M.workspace(M.beam_select_workspace_bytes(beams, c["k"])))
    M.beam_select(h[0], s["logits"], c["k"], s["parent"], s["token"], s["new_score"], s["new_length"], s["new_done"], h[1])
    return s["parent"], s["token"], s["new_score"], s["new_length"], s["new_done"]


def _own_reorder(s):
    import mtp_speculative_draft_gb300 as M
    c = s["case"]
    h = s.get("handle")
    if h is None:
        h = s["handle"] = (M.kv_tails(s["k"].unbind(0), s["v"].unbind(0), c["beams"]), M.workspace(M.kv_beam_workspace_bytes()))
    M.kv_beam_reorder(h[0], s["parent"], s["length"], c["tail"], h[1])
    return s["k"], s["v"]


# ------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["kind"] == "attn":
        nh, nkv, dqk, dv, m, W = (c[k] for k in ("nh", "nkv", "dqk", "dv", "m", "window"))
        prefix, tail = _lengths(c)
        keys = seen = 0
        for g, P in enumerate(prefix):
            own_tails = [t for t in tail[g * c["per"]:(g + 1) * c["per"]] if t >= 0]
            low = min([max(0, P + t + 1 - W) if W else 0 for t in own_tails], default=P)
            keys += max(0, P - low)                                   # the prompt's rows that any row sees
            for t in own_tails:
                see = min(P + t + 1, W) if W else P + t + 1
                keys += min(t, see)
                seen += m * see
        rows = sum(t >= 0 for t in tail) * m
        row = nh * dqk * (2 if c["gated"] else 1) + nh * dv + 2 * nkv * (dqk + dv) + c["rot"]
        return {"bytes": 4 * (nkv * keys * (dqk + dv) + rows * row), "flops": 2 * nh * seen * (dqk + dv)}
    if c["kind"] == "select":
        rows = c["seqs"] * c["beams"]
        return {"bytes": 4 * rows * c["vocab"] + 12 * rows + 20 * c["seqs"] * c["k"], "flops": 4 * rows * c["vocab"]}
    # of the expected selection: beams that are somebody's parent elsewhere are read, beams that change are written
    B = c["beams"]
    p = [((B - i) ** 2 - (B - i - 1) ** 2) / B ** 2 for i in range(B)]  # beam i is a given child's parent
    moved = B - sum(p)                                                 # children whose parent is another beam
    read = sum(1 - (1 - x) ** (B - 1) for x in p)
    row = 4 * c["layers"] * c["seqs"] * c["nkv"] * (c["dqk"] + c["dv"]) * c["tail"]
    return {"bytes": int(row * (moved + read)) + 8 * c["seqs"] * B, "flops": 0}


# ------------------------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "select": _exact_select, "reorder": _exact_reorder}[case["kind"]](s)


def _exact_heads(x, w, pos, rot, theta):
    """[rows, heads, d] in 64 bits: x / rms(x) * w, then the rotation as a complex product."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
    half = rot // 2
    freq = theta ** (-torch.arange(half, device=DEV, dtype=torch.float64) * 2 / rot)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None] * freq)
    z = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous()) * turn[:, None]
    return torch.cat([z.real, z.imag, x[..., rot:]], -1)


def _exact_attn(s):
    c = s["case"]
    nh, nkv, dqk, dv, m, W = (c[k] for k in ("nh", "nkv", "dqk", "dv", "m", "window"))
    G = nh // nkv
    prefix, tail = _lengths(c)
    out = torch.zeros(len(tail), m, nh, dv, device=DEV, dtype=torch.float64)
    kt, vt = s["k_tail"].double(), s["v_tail"].double()
    for b, t in enumerate(tail):  # one sequence at a time, as if it were alone
        if t < 0:
            continue
        P = prefix[b // c["per"]]
        rows = slice(b * m, b * m + m)
        pos = torch.arange(P + t, P + t + m, device=DEV)
        raw = s["qp"][rows].view(m, nh, -1)
        q = _exact_heads(raw[..., :dqk], s["q_norm"], pos, c["rot"], c["theta"])
        kt[b, :, t:t + m] = _exact_heads(s["kp"][rows].view(m, nkv, dqk), s["k_norm"], pos, c["rot"], c["theta"]).transpose(0, 1)
        vt[b, :, t:t + m] = s["vp"][rows].view(m, nkv, dv).double().transpose(0, 1)
        where = torch.arange(P + t + m, device=DEV)
        sees = where[None] <= pos[:, None]
        if W:
            sees &= where[None] > pos[:, None] - W
        for h in range(nkv):
            keys = torch.cat([s["k_prefix"][b // c["per"], h, :P].double(), kt[b, h, :t + m]])
            vals = torch.cat([s["v_prefix"][b // c["per"], h, :P].double(), vt[b, h, :t + m]])
            e = torch.einsum("rgd,kd->rgk", q[:, h * G:(h + 1) * G], keys) * dqk ** -0.5
            e = e.masked_fill(~sees[:, None], -math.inf)
            if s["sinks"] is not None:
                e = torch.cat([e, s["sinks"][h * G:(h + 1) * G].double().expand(m, G)[..., None]], -1)
            out[b, :, h * G:(h + 1) * G] = torch.softmax(e, -1)[..., :P + t + m] @ vals
        if c["gated"]:
            out[b] /= 1 + torch.exp(-raw[..., dqk:].double())
    return out.view(-1, nh * dv), kt, vt


def _exact_select(s):
    c = s["case"]
    S, B, V, k = c["seqs"], c["beams"], c["vocab"], c["k"]
    alpha, eos = c["alpha"], s["eos"]
    length = s["length"].tolist()
    done = s["done"].tolist() if s["done"] is not None else [0] * (S * B)
    out = torch.full((S, k), -math.inf, dtype=torch.float64)
    for i in range(S):
        best = []
        for r in range(i * B, i * B + B):
            start = float(s["score"][r])
            if done[r]:
                best.append((start / max(1, length[r]) ** alpha, start))
                continue
            row = s["logits"][r].double()
            row = start + row - torch.logsumexp(row, 0)
            for v in torch.topk(row, min(k, V)).values.tolist():
                if v > -math.inf:
                    best.append((v / (length[r] + 1) ** alpha, v))
        best.sort(key=lambda t: -t[0])
        for j, (_, v) in enumerate(best[:k]):
            out[i, j] = v
    return None, None, out.to(DEV), None, None


def _exact_reorder(s):
    c = s["case"]
    parent, length = s["parent"].tolist(), s["length"].tolist()
    out = []
    for x in (s["k"], s["v"]):
        y = x.double()
        for i in range(c["seqs"]):
            for j, p in enumerate(parent[i]):
                at, n = i * c["beams"] + j, length[i * c["beams"] + j]
                y[:, at, :, :n] = x[:, i * c["beams"] + p, :, :n].double()
        out.append(y)
    return tuple(out)
