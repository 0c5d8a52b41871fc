"""What the cache's calls keep between one another: lengths in place, the workspace's counters."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
from test_gpu_cache import BF16, DEV, check_attention, filled, gen, make_cache, normal
from test_gpu_window import make

pytestmark = pytest.mark.gpu


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("windowed", [False, True])
def test_append_on_a_workspace_that_served_other_calls(windowed):
    """The lengths advance whatever the workspace's other words hold."""
    lens = [300, 40]
    x, _ = make(lens, lens, 2, 2, 64, 60)
    ws = (jfa.new_window_workspace(2, 2, 2, 64, 340, 340, 0, False, DEV) if windowed
          else jfa.jfa.new_workspace(2, 2, 64, 340, 340, False, DEV))
    g = gen(61)
    k, v, table = make_cache(g, [50, 50], 2, 64, 16)
    n = int32([3, 20])
    rows, off = normal(g, 5, 2, 64), torch.tensor([0, 2, 5], device=DEV)
    for step in range(3):
        if windowed:
            jfa.jfa_window_forward(**x, window=9, workspace=ws)
        else:
            jfa.jfa_forward(**x, workspace=ws)
        jfa.jfa_cache_append(rows, rows, off, k, v, table, n, lengths_out=n, workspace=ws)
        assert jfa.jfa_check_status(ws) == 0
        assert n.tolist() == [3 + 2 * (step + 1), 20 + 3 * (step + 1)]
