"""Draft-tree calls as a program may make them: streams, devices, layouts, numbers at the ends of their ranges."""

import numpy as np
import pytest

from test_gpu_tree import dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_workspaces_come_from_the_pool_of_their_stream(dev):  # noqa: F811
    import torch
    import mtp_speculative_draft_gb300 as M
    side = torch.cuda.Stream()
    par = torch.tensor([-1, 0, 0], dtype=torch.int32, device=dev)
    mask, depth = torch.zeros(3, dtype=torch.int64, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    kept = [M.mtp_tree_plan(par, mask, depth, stream=side), M.workspace(100000, stream=side)]
    side.synchronize()
    assert mask.tolist() == [1, 3, 5]
    for ws in kept:
        at = [s["stream"] for s in torch.cuda.memory_snapshot()
              if s["address"] <= ws.data_ptr() < s["address"] + s["total_size"]]
        assert at == [side.cuda_stream]
