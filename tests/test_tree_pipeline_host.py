"""The barriers of the tree attention's split kernel, walked through on the host.

The kernel's threads that hand tiles to one another (K and V converters, two softmax warpgroups on
alternate tiles, the tensor pipe) are reduced to their waits and arrivals, and every order in which
they can run is visited.  A tile's scale of K lies in a ring; no order may overwrite an entry that
the tile's warpgroup has not read.  The ring's size and the place of its write are taken from the
source.
"""

import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mtp_speculative_draft_gb300",
                   "csrc", "treeattn.cu")


def overwritten_early(ring, write_after_wait, tiles=9):
    """Whether some order of the steps lets a warpgroup read another tile's scale.

    State: steps done by the K converters (two a tile: the write into the ring, the wait for the tile's
    buffer with the arrival on its barrier), tiles of V converted, each warpgroup's place, tiles whose
    scores and whose outputs the tensor pipe has finished, what the ring holds.
    """
    first, second = (("wait", "write") if write_after_wait else ("write", "wait"))
    start = (0, 0, (0, 1), (0, 0), frozenset(), frozenset(), frozenset(), (-1,) * ring)
    seen, todo = {start}, [start]
    while todo:
        k, v, tile, at, issued, qk, pv, held = todo.pop()
        nxt = []
        t = k // 2  # the K converters' tile
        if t < tiles:
            what = first if k % 2 == 0 else second
            if what == "write":
                h = list(held)
                h[t % ring] = t
                nxt.append((k + 1, v, tile, at, issued, qk, pv, tuple(h)))
            elif t < 2 or t - 2 in qk:  # the buffer is free once the scores of tile t - 2 are done
                nxt.append((k + 1, v, tile, at, issued, qk, pv, held))
        if v < tiles and (v < 2 or v - 2 in pv):
            nxt.append((k, v + 1, tile, at, issued, qk, pv, held))
        for i in issued:  # the tensor pipe finishes a tile's scores
            nxt.append((k, v, tile, at, issued - {i}, qk | {i}, pv, held))
        for g in (0, 1):
            t = tile[g]
            if t >= tiles:
                continue
            step = lambda x: at[:g] + (x,) + at[g + 1:]  # noqa: E731
            if at[g] == 0 and k >= 2 * (t + 1):  # K of the tile is converted: its scores are issued
                nxt.append((k, v, tile, step(1), issued | {t}, qk, pv, held))
            elif at[g] == 1 and t in qk and v > t:  # scores and V are there: the scale is read
                if held[t % ring] != t:
                    return True
                nxt.append((k, v, tile, step(2), issued, qk, pv, held))
            elif at[g] == 2:  # weights, P V, then the warpgroup's next tile
                nxt.append((k, v, tile[:g] + (t + 2,) + tile[g + 1:], step(0), issued, qk, pv | {t}, held))
        for s in nxt:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return False


@pytest.mark.parametrize("ring,after,early", [(4, False, True), (5, False, False), (3, True, True), (4, True, False)])
def test_the_model_tells_the_orders_apart(ring, after, early):
    assert overwritten_early(ring, after) is early


def test_scale_ring_is_not_overwritten_before_it_is_read():
    src = open(SRC).read()
    ring = int(re.search(r"constexpr int kScaleRing = (\d+);", src).group(1))
    stages = int(re.search(r"constexpr int kStages = (\d+);", src).group(1))
    assert stages == 2  # the model's buffers
    write, wait = src.index("inv[t % kScaleRing] = iv"), src.index("wait(&empty[s]")
    assert write < src.index("tc5::mbar_arrive(&full[s])")
    assert not overwritten_early(ring, write > wait)
