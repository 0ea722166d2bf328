"""Torch-facing wrappers of the draft-tree calls (argument marshalling only).

Descriptors (``rope_axes``, ``draft_tree``, ``logit_rules``, ``kv_caches``) hold the device
pointers of the tensors they were made from and keep those tensors alive; a program makes them once
and fills the tensors in place each round.  Tensors have to be on the current CUDA device.
"""

from __future__ import annotations

import ctypes as C

import torch

from . import _lib as L
from ._lib import AttnGeom, DraftTree, HeadRows, KvCaches, LogitRules, RopeAxes, check
from .api import workspace

_I32, _F32 = torch.int32, torch.float32
_MOST = (1 << 31) - 1


def _refuse(t, dtype, numel, name):
    if not t.is_cuda or t.get_device() != _device():
        raise ValueError(f"{name}: a tensor on the current CUDA device is required")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} is required, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is required")
    raise ValueError(f"{name}: {numel} values are needed, got {t.numel()}")


def _ptr(t, dtype, numel, name, device):
    """Device pointer of a contiguous tensor of ``dtype`` with at least ``numel`` values."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous() or t.numel() < numel:
        _refuse(t, dtype, numel, name)
    return t.data_ptr()


def _int(v, name):
    """A number that the library takes in 32 bits (ctypes would cut a longer one off)."""
    v = int(v)
    if not -_MOST <= v <= _MOST:
        raise ValueError(f"{name}: {v} does not fit in 32 bits")
    return v


def _device():
    """The current CUDA device."""
    try:
        return torch._C._cuda_getDevice()
    except (AttributeError, RuntimeError):
        raise ValueError("a CUDA device is required") from None


def _on(stream, device):
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _rows(t, rows, width, name, device):
    """Pointer and row stride (0: contiguous rows) of a float32 ``[rows, width]`` matrix whose rows are
    contiguous."""
    if t is None or t.get_device() != device:
        raise ValueError(f"{name}: a tensor on the current CUDA device is required")
    if t.dtype is not _F32:
        raise TypeError(f"{name}: torch.float32 is required, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] < rows or shape[1] != width:
        raise ValueError(f"{name}: [{rows}, {width}] with contiguous rows is required, got {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    if (width > 1 and t.stride(1) != 1) or (shape[0] > 1 and t.stride(0) < width):
        raise ValueError(f"{name}: [{rows}, {width}] with contiguous rows is required, got strides {t.stride()}")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else 0


def _ws(ws, device):
    if ws.get_device() != device or not ws.is_contiguous() or ws.dtype is not torch.uint8:
        raise ValueError("workspace: a contiguous uint8 tensor on the current CUDA device is required")
    return ws.data_ptr(), ws.numel()


def _here(desc, device):
    """Refuses a descriptor whose tensors are on another device than the current one (one that a program filled
    in by itself has no device)."""
    if desc.device not in (None, device):
        raise ValueError(f"{type(desc).__name__}: its tensors are on device {desc.device}, the current one is {device}")


# ------------------------------------------------------------------------------- rotary axes
def rope_axes(sections, pos: torch.Tensor, rope: torch.Tensor, interleaved=False) -> RopeAxes:
    """Rotary positions ``pos [n_axes, rows]`` (int32) on the axes whose rotary pairs ``sections``
    counts, with the table of ``mtp_rope_table`` for ``2 * sum(sections)`` rotated dims."""
    dev = _device()
    n, half = len(sections), int(sum(sections))
    if not 1 <= n <= 4 or half < 1:
        raise ValueError("rope_axes: 1..4 sections with at least one rotary pair")
    if pos.dim() != 2 or pos.shape[0] != n:
        raise ValueError(f"rope_axes: pos [{n}, rows] is required")
    ax = RopeAxes(_ptr(pos, _I32, n, "pos", dev), _ptr(rope, _F32, 2 * half, "rope", dev), n,
                  (L.i32 * 4)(*[_int(s, "sections") for s in sections]), int(bool(interleaved)),
                  _int(pos.shape[1], "pos"), min(rope.numel() // (2 * half), _MOST))
    ax.tensors, ax.device = (pos, rope), dev
    return ax


def rope_axes_rows_workspace_bytes() -> int:
    return L.load().rope_axes_rows_workspace_bytes()


def rope_axes_rows(axes: RopeAxes, tensors, ws=None, eps=1e-6, stream=None):
    """Norm and rotation of rows of heads.  ``tensors``: up to four ``(x, y, norm_w)`` with x and y
    ``[rows, heads, head_dim]`` (any row and head stride, contiguous head rows; y may be x) and
    norm_w ``[head_dim]`` or None."""
    dev = _device()
    if axes.device != dev:
        _here(axes, dev)
    lib = L.load()
    rows, _, d = tensors[0][0].shape
    descs = []
    for x, y, w in tensors:
        shape = x.shape
        if x.get_device() != dev or y.get_device() != dev:
            raise ValueError("rope_axes_rows: tensors on the current CUDA device are required")
        if len(shape) != 3 or shape[0] != rows or shape[2] != d or y.shape != shape:
            raise ValueError("rope_axes_rows: x and y [rows, heads, head_dim] of one row count and head_dim are required")
        n = shape[1]
        (xr, xh, x1), (yr, yh, y1) = x.stride(), y.stride()
        if x.dtype is not _F32 or y.dtype is not _F32 or x1 != 1 or y1 != 1:
            raise TypeError("rope_axes_rows: float32 with contiguous head rows is required")
        if n == 1:  # a stride that is never stepped may be anything
            xh = yh = d
        if rows == 1:
            xr, yr = n * xh, n * yh
        if xh > _MOST or yh > _MOST:
            raise ValueError("rope_axes_rows: a head stride does not fit in 32 bits")
        descs.append(HeadRows(x.data_ptr(), y.data_ptr(), _ptr(w, _F32, d, "norm_w", dev), xr, yr, xh, yh, n))
    arr = (HeadRows * len(descs))(*descs)
    if ws is None:
        ws = workspace(lib.rope_axes_rows_workspace_bytes(), stream=stream)
    check(lib.rope_axes_rows(C.byref(axes), arr, len(arr), rows, d, eps, *_ws(ws, dev), _on(stream, dev)),
          "rope_axes_rows")
    return ws


# ------------------------------------------------------------------------------- tree attention
def draft_tree(mask: torch.Tensor, depth: torch.Tensor, axes: RopeAxes | None = None, pos_base=0) -> DraftTree:
    """The new rows of a tree: ancestor words ``mask [n]`` (int64 or uint64) and ``depth [n]``."""
    dev = _device()
    n = _int(mask.numel(), "mask")
    if mask.dtype not in (torch.int64, torch.uint64):
        raise TypeError("draft_tree: mask holds 64-bit words")
    if axes is not None:
        _here(axes, dev)
    t = DraftTree(_ptr(mask, mask.dtype, 1, "mask", dev), _ptr(depth, _I32, n, "depth", dev),
                  C.pointer(axes) if axes is not None else None, n, _int(pos_base, "pos_base"), 0, 0, 0)
    t.tensors, t.device = (mask, depth, axes), dev
    return t


def mtp_tree_workspace_bytes() -> int:
    return L.load().mtp_tree_workspace_bytes()


def mtp_tree_plan(parents, mask, depth, ws=None, stream=None):
    """Ancestor words and depths of a tree from its ``parents [n]`` (int32, -1 for a root)."""
    dev = _device()
    n = parents.numel()
    if n > _MOST:
        _int(n, "parents")
    if ws is None:
        ws = workspace(mtp_tree_workspace_bytes(), stream=stream)
    if mask.dtype not in (torch.int64, torch.uint64):
        raise TypeError("mtp_tree_plan: mask holds 64-bit words")
    check(L.load().mtp_tree_plan(_ptr(parents, _I32, n, "parents", dev), n,
                                 _ptr(mask, mask.dtype, n, "mask", dev),
                                 _ptr(depth, _I32, n, "depth", dev), *_ws(ws, dev), _on(stream, dev)),
          "mtp_tree_plan")
    return ws


def attn_tree_sink_workspace_bytes(g: AttnGeom, n: int, cache_len: int) -> int:
    return L.load().attn_tree_sink_workspace_bytes(C.byref(g), _int(n, "n"), _int(cache_len, "cache_len"))


def attn_tree_sink(g: AttnGeom, tree: DraftTree, qp, kp, vp, q_norm, k_norm, rope, sinks, k_cache,
                   v_cache, cache_len, out, ws=None, stream=None):
    """Attention of a tree's rows ``qp [n, q_rows]``, ``kp``, ``vp`` (any row stride) over the cache
    ``[n_kv, cap, dim]`` and their ancestors; appends the rows at ``cache_len`` onwards."""
    dev = _device()
    if tree.device != dev:
        _here(tree, dev)
    if type(cache_len) is not int or not -_MOST <= cache_len <= _MOST:
        cache_len = _int(cache_len, "cache_len")
    lib = L.load()
    n, nh, nkv, dqk, dv = tree.n, g.n_heads, g.n_kv_heads, g.head_dim_qk, g.head_dim_v
    pq, ldq = _rows(qp, n, nh * dqk * (2 if g.gated_q else 1), "qp", dev)
    pk, ldk = _rows(kp, n, nkv * dqk, "kp", dev)
    pv, ldv = _rows(vp, n, nkv * dv, "vp", dev)
    if ldq or ldk or ldv:  # a call's own strides: the descriptor stays as it is
        tree = DraftTree(tree.d_mask, tree.d_depth, tree.axes, n, tree.pos_base, ldq, ldk, ldv)
    cap = k_cache.shape[1] if k_cache.dim() == 3 else 0
    if k_cache.shape != (nkv, cap, dqk) or v_cache.shape != (nkv, cap, dv):
        raise ValueError("attn_tree_sink: caches [n_kv, cap, dim] of the geometry are required")
    if ws is None:
        ws = workspace(lib.attn_tree_sink_workspace_bytes(C.byref(g), n, cache_len), stream=stream)
    check(lib.attn_tree_sink(
        C.byref(g), C.byref(tree), pq, pk, pv, _ptr(q_norm, _F32, dqk, "q_norm", dev),
        _ptr(k_norm, _F32, dqk, "k_norm", dev), _ptr(rope, _F32, 0, "rope", dev),
        min(rope.numel() // g.rot_dim, _MOST) if rope is not None and g.rot_dim > 0 else 0,
        _ptr(sinks, _F32, nh, "sinks", dev), _ptr(k_cache, _F32, 0, "k_cache", dev),
        _ptr(v_cache, _F32, 0, "v_cache", dev), cache_len, cap,
        _ptr(out, _F32, n * nh * dv, "out", dev), *_ws(ws, dev), _on(stream, dev)), "attn_tree_sink")
    return ws


# ------------------------------------------------------------------------------- logit rules
def logit_rules(vocab, repetition=1.0, frequency=0.0, presence=0.0, counts=None, bias_tokens=None,
                bias=None, allow=None, path_tokens=None, path_mask=None) -> LogitRules:
    """Rules of a request: penalties with the count table ``counts [vocab]`` (int32 or uint32 words),
    biases, a grammar's mask ``allow [rows, words]`` (``[words]``: one for all rows), and the draft
    tree's ``path_tokens [n]`` with each row's ancestor word ``path_mask [rows]``."""
    dev = _device()
    word = lambda t: t.dtype if t is not None and t.dtype in (_I32, torch.uint32) else _I32  # noqa: E731
    nb = 0 if bias is None else _int(bias.numel(), "bias")
    npath = 0 if path_tokens is None else _int(path_tokens.numel(), "path_tokens")
    vocab = _int(vocab, "vocab")
    words = (vocab + 31) // 32
    if (bias is None) != (bias_tokens is None) or (path_tokens is None) != (path_mask is None):
        raise ValueError("logit_rules: bias with bias_tokens, path_tokens with path_mask")
    if allow is not None and (allow.dim() not in (1, 2) or allow.shape[-1] < words):
        raise ValueError(f"logit_rules: allow needs {words} words a row")
    if path_mask is not None and path_mask.dtype not in (torch.int64, torch.uint64):
        raise TypeError("logit_rules: path_mask holds 64-bit words")
    r = LogitRules(vocab, repetition, frequency, presence,
                   _ptr(counts, word(counts), vocab, "counts", dev),
                   _ptr(bias_tokens, _I32, nb, "bias_tokens", dev), _ptr(bias, _F32, nb, "bias", dev), nb,
                   _ptr(allow, word(allow), words, "allow", dev),
                   _int(allow.shape[1], "allow") if allow is not None and allow.dim() == 2 else 0,
                   _ptr(path_tokens, _I32, npath, "path_tokens", dev),
                   _ptr(path_mask, None if path_mask is None else path_mask.dtype, 1, "path_mask", dev), npath)
    r.rows = min([1 << 30] + [t.shape[0] for t in (allow if allow is not None and allow.dim() == 2 else None,
                                                   path_mask) if t is not None])
    r.tensors = (counts, bias_tokens, bias, allow, path_tokens, path_mask)
    if any(t is not None for t in r.tensors):
        r.device = dev
    return r


def logit_rules_argmax_workspace_bytes(rows: int) -> int:
    return L.load().logit_rules_argmax_workspace_bytes(_int(rows, "rows"))


def logit_rules_argmax(rules: LogitRules, logits, tokens, values, out=None, ws=None, stream=None):
    """Applies ``rules`` to ``logits [rows, vocab]`` (any row stride) and takes each row's argmax;
    ``out`` (or ``logits`` itself) receives the final logits."""
    dev = _device()
    if rules.device != dev:
        _here(rules, dev)
    lib = L.load()
    rows = logits.shape[0]
    if rows > rules.rows:
        raise ValueError(f"logit_rules_argmax: the rules' mask has {rules.rows} rows, the logits {rows}")
    vocab = rules.vocab
    px, ld = _rows(logits, rows, vocab, "logits", dev)
    py, ldy = (None, 0) if out is None else _rows(out, rows, vocab, "out", dev)
    if ws is None:
        ws = workspace(lib.logit_rules_argmax_workspace_bytes(rows), stream=stream)
    check(lib.logit_rules_argmax(C.byref(rules), px, ld or vocab, rows, _ptr(tokens, _I32, rows, "tokens", dev),
                                 _ptr(values, _F32, rows, "values", dev), py, ldy or vocab, *_ws(ws, dev),
                                 _on(stream, dev)), "logit_rules_argmax")
    return ws


def mtp_token_counts(counts, tokens, prompt=False, ws=None, stream=None):
    """Adds ``tokens`` (negative ids skipped) to the count table ``counts [vocab]``."""
    dev = _device()
    if counts.dtype not in (_I32, torch.uint32):
        raise TypeError("mtp_token_counts: counts holds 32-bit words")
    vocab, n = _int(counts.numel(), "counts"), _int(tokens.numel(), "tokens")
    if ws is None:
        ws = workspace(mtp_tree_workspace_bytes(), stream=stream)
    check(L.load().mtp_token_counts(_ptr(counts, counts.dtype, 1, "counts", dev), vocab,
                                    _ptr(tokens, _I32, n, "tokens", dev), n, int(bool(prompt)), *_ws(ws, dev),
                                    _on(stream, dev)), "mtp_token_counts")
    return ws


# ------------------------------------------------------------------------------- accepted path
def mtp_tree_accept(parents, tokens, verify, path, emitted, count, stream=None):
    """The accepted path of a tree: nodes into ``path [n]``, the verifier's tokens on it into
    ``emitted [n]`` (both -1 past the end), their number into ``count [1]``."""
    dev = _device()
    n = parents.numel()
    if n > _MOST:
        _int(n, "parents")
    check(L.load().mtp_tree_accept(
        _ptr(parents, _I32, n, "parents", dev), _ptr(tokens, _I32, n, "tokens", dev),
        _ptr(verify, _I32, n, "verify", dev), n, _ptr(path, _I32, n, "path", dev),
        _ptr(emitted, _I32, n, "emitted", dev), _ptr(count, _I32, 1, "count", dev), _on(stream, dev)),
        "mtp_tree_accept")


def kv_caches(k_caches, v_caches) -> KvCaches:
    """The K and V caches ``[n_kv, cap, dim]`` of layers with one geometry."""
    dev = _device()
    k_caches, v_caches = list(k_caches), list(v_caches)
    n = len(k_caches)
    if n < 1 or len(v_caches) != n:
        raise ValueError("kv_caches: one K and one V cache a layer")
    nkv, cap, dqk = k_caches[0].shape
    dv = v_caches[0].shape[-1]
    for k, v in zip(k_caches, v_caches):
        if tuple(k.shape) != (nkv, cap, dqk) or tuple(v.shape) != (nkv, cap, dv):
            raise ValueError("kv_caches: caches [n_kv, cap, dim] of one geometry are required")
    ks = (L.vp * n)(*[_ptr(k, _F32, 1, "k_cache", dev) for k in k_caches])
    vs = (L.vp * n)(*[_ptr(v, _F32, 1, "v_cache", dev) for v in v_caches])
    if len({*ks, *vs}) != 2 * n:
        raise ValueError("kv_caches: a cache is given twice")
    c = KvCaches(ks, vs, n, nkv, dqk, dv, _int(cap, "cap"))
    c.tensors, c.device = (k_caches, v_caches, ks, vs), dev
    return c


def kv_tree_commit(caches: KvCaches, path, cache_len, ws=None, stream=None):
    """Moves the rows of ``path [n]`` (nodes of the tree, -1 past the end) to ``cache_len`` onwards."""
    dev = _device()
    if caches.device != dev:
        _here(caches, dev)
    if caches.beams:
        raise ValueError("kv_tree_commit: caches [n_kv, cap, dim] are required (kv_caches), not beams' tails")
    if ws is None:
        ws = workspace(mtp_tree_workspace_bytes(), stream=stream)
    n = path.numel()
    if n > _MOST or type(cache_len) is not int or not -_MOST <= cache_len <= _MOST:
        n, cache_len = _int(n, "path"), _int(cache_len, "cache_len")
    check(L.load().kv_tree_commit(C.byref(caches), _ptr(path, _I32, n, "path", dev), n, cache_len,
                                  *_ws(ws, dev), _on(stream, dev)), "kv_tree_commit")
    return ws
