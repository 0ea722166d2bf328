"""Torch-facing wrappers of the calls of a beam search's step (argument marshalling only).

Descriptors (``prefix_batch``, ``beam_set``, ``kv_tails``) hold the device pointers of the tensors they
were made from and keep those tensors alive; a program makes them once and fills the tensors in place
each step.  Tensors have to be on the current CUDA device.
"""

from __future__ import annotations

import ctypes as C

import torch

from . import _lib as L
from ._lib import AttnGeom, BeamSet, KvCaches, PrefixBatch, RopeAxes, check
from .api import workspace
from .tree import _F32, _I32, _MOST, _device, _here, _int, _on, _ptr, _rows, _ws


# ------------------------------------------------------------------------------- shared prompts
def prefix_batch(prefix_len: torch.Tensor, tail_len: torch.Tensor, prefix_max, tail_max, m=1,
                 axes: RopeAxes | None = None, pos_base=0) -> PrefixBatch:
    """The new rows of sequences that share prompts: ``prefix_len [n_groups]`` and ``tail_len [n_seqs]``
    (int32, negative: no sequence), at most ``prefix_max`` and ``tail_max``, ``m`` new rows a sequence."""
    dev = _device()
    groups, seqs = _int(prefix_len.numel(), "prefix_len"), _int(tail_len.numel(), "tail_len")
    if axes is not None:
        _here(axes, dev)
    b = PrefixBatch(_ptr(prefix_len, _I32, 1, "prefix_len", dev), _ptr(tail_len, _I32, 1, "tail_len", dev),
                    C.pointer(axes) if axes is not None else None, groups, seqs, _int(m, "m"),
                    _int(prefix_max, "prefix_max"), _int(tail_max, "tail_max"), _int(pos_base, "pos_base"), 0, 0, 0)
    b.tensors, b.device = (prefix_len, tail_len, axes), dev
    return b


def attn_prefix_sink_workspace_bytes(g: AttnGeom, batch: PrefixBatch) -> int:
    return L.load().attn_prefix_sink_workspace_bytes(C.byref(g), batch.n_groups, batch.n_seqs, batch.m, batch.prefix_max)


def attn_prefix_sink(g: AttnGeom, batch: PrefixBatch, qp, kp, vp, q_norm, k_norm, rope, sinks, k_prefix,
                     v_prefix, k_tail, v_tail, out, ws=None, stream=None):
    """Attention of the rows ``qp [n_seqs * m, q_rows]``, ``kp``, ``vp`` (any row stride) over their
    prompts ``[n_groups, n_kv, cap, dim]`` and tails ``[n_seqs, n_kv, cap, dim]``; appends the rows to
    the tails.  ``k_prefix`` and ``v_prefix`` may be None where ``prefix_max`` is 0."""
    dev = _device()
    if batch.device != dev:
        _here(batch, dev)
    lib = L.load()
    groups, seqs, rows = batch.n_groups, batch.n_seqs, batch.n_seqs * batch.m
    nh, nkv, dqk, dv = g.n_heads, g.n_kv_heads, g.head_dim_qk, g.head_dim_v
    pq, ldq = _rows(qp, rows, nh * dqk * (2 if g.gated_q else 1), "qp", dev)
    pk, ldk = _rows(kp, rows, nkv * dqk, "kp", dev)
    pv, ldv = _rows(vp, rows, nkv * dv, "vp", dev)
    if ldq or ldk or ldv:  # a call's own strides: the descriptor stays as it is
        b = PrefixBatch()
        C.pointer(b)[0] = batch
        b.ld_q, b.ld_k, b.ld_v, b.tensors = ldq, ldk, ldv, batch.tensors
        batch = b
    pcap = k_prefix.shape[2] if k_prefix is not None and k_prefix.dim() == 4 else 0
    if (k_prefix is not None or batch.prefix_max > 0) and (
            k_prefix is None or v_prefix is None or k_prefix.shape != (groups, nkv, pcap, dqk)
            or v_prefix.shape != (groups, nkv, pcap, dv)):
        raise ValueError("attn_prefix_sink: prompts [n_groups, n_kv, cap, dim] of the geometry are required")
    tcap = k_tail.shape[2] if k_tail.dim() == 4 else 0
    if k_tail.shape != (seqs, nkv, tcap, dqk) or v_tail.shape != (seqs, nkv, tcap, dv):
        raise ValueError("attn_prefix_sink: tails [n_seqs, n_kv, cap, dim] of the geometry are required")
    if ws is None:
        ws = workspace(attn_prefix_sink_workspace_bytes(g, batch), stream=stream)
    check(lib.attn_prefix_sink(
        C.byref(g), C.byref(batch), pq, pk, pv, _ptr(q_norm, _F32, dqk, "q_norm", dev),
        _ptr(k_norm, _F32, dqk, "k_norm", dev), _ptr(rope, _F32, 0, "rope", dev),
        min(rope.numel() // g.rot_dim, _MOST) if rope is not None and g.rot_dim > 0 else 0,
        _ptr(sinks, _F32, nh, "sinks", dev), _ptr(k_prefix, _F32, 0, "k_prefix", dev),
        _ptr(v_prefix, _F32, 0, "v_prefix", dev), pcap, _ptr(k_tail, _F32, 0, "k_tail", dev),
        _ptr(v_tail, _F32, 0, "v_tail", dev), tcap, _ptr(out, _F32, rows * nh * dv, "out", dev), *_ws(ws, dev),
        _on(stream, dev)), "attn_prefix_sink")
    return ws


# ------------------------------------------------------------------------------- selection
def beam_set(n_seqs, beams, vocab, score: torch.Tensor, length=None, done=None, eos=-1, length_penalty=0.0) -> BeamSet:
    """The beams of ``n_seqs`` prompts: ``score [n_seqs * beams]`` (float32), ``length`` and ``done`` (int32)."""
    dev = _device()
    n_seqs, beams, vocab = _int(n_seqs, "n_seqs"), _int(beams, "beams"), _int(vocab, "vocab")
    rows = max(1, n_seqs * beams)
    b = BeamSet(_ptr(score, _F32, rows, "score", dev), _ptr(length, _I32, rows, "length", dev),
                _ptr(done, _I32, rows, "done", dev), n_seqs, beams, vocab, _int(eos, "eos"), length_penalty)
    b.tensors, b.device = (score, length, done), dev
    return b


def beam_select_workspace_bytes(beams: BeamSet, k: int) -> int:
    return L.load().beam_select_workspace_bytes(beams.n_seqs, beams.beams, beams.vocab, _int(k, "k"))


def beam_select(beams: BeamSet, logits, k, parent, token, score, length=None, done=None, ws=None, stream=None):
    """The ``k`` best extensions of each prompt's beams by ``logits [n_seqs * beams, vocab]`` (any row
    stride) into ``parent``, ``token``, ``score`` and, if given, ``length`` and ``done [n_seqs, k]``."""
    dev = _device()
    if beams.device != dev:
        _here(beams, dev)
    lib = L.load()
    if type(k) is not int or not -_MOST <= k <= _MOST:
        k = _int(k, "k")
    n, vocab = beams.n_seqs * k, beams.vocab
    px, ld = _rows(logits, beams.n_seqs * beams.beams, vocab, "logits", dev)
    if ws is None:
        ws = workspace(lib.beam_select_workspace_bytes(beams.n_seqs, beams.beams, vocab, k), stream=stream)
    check(lib.beam_select(C.byref(beams), px, ld or vocab, k, _ptr(parent, _I32, n, "parent", dev),
                          _ptr(token, _I32, n, "token", dev), _ptr(score, _F32, n, "score", dev),
                          _ptr(length, _I32, n, "length", dev), _ptr(done, _I32, n, "done", dev), *_ws(ws, dev),
                          _on(stream, dev)), "beam_select")
    return ws


# ------------------------------------------------------------------------------- survivors' tails
def kv_tails(k_tails, v_tails, beams) -> KvCaches:
    """The K and V tails ``[n_seqs * beams, n_kv, cap, dim]`` of layers with one geometry."""
    dev = _device()
    k_tails, v_tails = list(k_tails), list(v_tails)
    n, beams = len(k_tails), _int(beams, "beams")
    if n < 1 or len(v_tails) != n:
        raise ValueError("kv_tails: one K and one V tail a layer")
    if k_tails[0].dim() != 4:
        raise ValueError("kv_tails: tails [n_seqs * beams, n_kv, cap, dim] are required")
    rows, nkv, cap, dqk = k_tails[0].shape
    dv = v_tails[0].shape[-1]
    if beams < 1 or rows % beams:
        raise ValueError(f"kv_tails: {rows} tails are no whole number of prompts of {beams} beams")
    for k, v in zip(k_tails, v_tails):
        if tuple(k.shape) != (rows, nkv, cap, dqk) or tuple(v.shape) != (rows, nkv, cap, dv):
            raise ValueError("kv_tails: tails [n_seqs * beams, n_kv, cap, dim] of one geometry are required")
    ks = (L.vp * n)(*[_ptr(k, _F32, 1, "k_tail", dev) for k in k_tails])
    vs = (L.vp * n)(*[_ptr(v, _F32, 1, "v_tail", dev) for v in v_tails])
    if len({*ks, *vs}) != 2 * n:
        raise ValueError("kv_tails: a tail is given twice")
    c = KvCaches(ks, vs, n, nkv, dqk, dv, _int(cap, "cap"))
    c.tensors, c.device, c.seqs, c.beams = (k_tails, v_tails, ks, vs), dev, rows // beams, beams
    return c


def kv_beam_workspace_bytes() -> int:
    return L.load().kv_beam_workspace_bytes()


def kv_beam_reorder(tails: KvCaches, parent, length, max_len, ws=None, stream=None):
    """Rows ``0 .. length[r] - 1`` of beam r become those of its ``parent``, in all layers (``parent`` and
    ``length [n_seqs * beams]``, int32; a negative parent: the beam stays)."""
    dev = _device()
    if tails.device != dev:
        _here(tails, dev)
    if not tails.beams:
        raise ValueError("kv_beam_reorder: tails [n_seqs * beams, n_kv, cap, dim] are required (kv_tails)")
    lib = L.load()
    if ws is None:
        ws = workspace(lib.kv_beam_workspace_bytes(), stream=stream)
    rows = tails.seqs * tails.beams
    check(lib.kv_beam_reorder(C.byref(tails), _ptr(parent, _I32, rows, "parent", dev), tails.seqs, tails.beams,
                              _ptr(length, _I32, rows, "length", dev), _int(max_len, "max_len"), *_ws(ws, dev),
                              _on(stream, dev)), "kv_beam_reorder")
    return ws
