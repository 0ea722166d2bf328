"""Attention over shared prompts where the launches are three (prep, split, tail), and where a size decides that they
are one.  Tolerances as in test_gpu_beams.py."""

import numpy as np
import pytest

from helpers import assert_close
from test_gpu_beams import ATTN_TOL, Call, _attn_case, _reference, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_most_prompts_of_most_kv_heads(dev):  # noqa: F811
    """1024 prompts of 64 KV heads, one more than a grid's third axis holds: a few of them against the reference,
    every tail's rows outside the new ones as they were."""
    rng = np.random.default_rng(5)
    c = _attn_case(60, nh=192, nkv=64, dqk=32, dv=32, plen=[int(n) for n in rng.integers(0, 9, 1023)] + [8],
                   tlen=[int(t) for t in rng.integers(-1, 4, 1023)] + [3], m=2)
    call = Call(c, dev)
    call()
    got, m = call.out.cpu().numpy().reshape(1024, 2, 192, 32), 2
    kt, vt = call.kt.cpu().numpy(), call.vt.cpu().numpy()
    pick = [0, 1, 511, 512, 1022, 1023]
    rows = np.concatenate([np.arange(b * m, b * m + m) for b in pick])
    sub = {**c, **{n: [c[n][b] for b in pick] for n in ("plen", "tlen")}, **{n: c[n][pick] for n in ("kpre", "vpre", "kt", "vt")},
           **{n: c[n][rows] for n in ("qp", "kp", "vp")}}
    ref, k, _ = _reference(sub)
    for x, b in enumerate(pick):
        t = c["tlen"][b]
        if t >= 0:
            assert_close(got[b], np.array(ref[x * m:x * m + m]), f"sequence {b}", ATTN_TOL)
            assert_close(kt[b, :, t:t + m], k[x * m:x * m + m].transpose(1, 0, 2), f"keys of {b}", 2e-6)
    for b, t in enumerate(c["tlen"]):
        keep = np.ones(kt.shape[2], bool)
        if t >= 0:
            keep[t:t + m] = False
            np.testing.assert_array_equal(vt[b, :, t:t + m], c["vp"][b * m:b * m + m].reshape(m, 64, 32).transpose(1, 0, 2))
        else:
            assert (got[b] == 7).all()
        np.testing.assert_array_equal(kt[b][:, keep], c["kt"][b][:, keep])
        np.testing.assert_array_equal(vt[b][:, keep], c["vt"][b][:, keep])
