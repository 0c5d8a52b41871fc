"""Tensors that end with their allocation: loads of the last sequences' partial tiles must not touch
the memory behind them.  Sizes are whole 2 MB pages, token rows narrow (128 to 1024 bytes)."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
import oracle.window_oracle as orc
from test_gpu_window import close, make, offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,d,T", [(1, 64, 163840), (2, 64, 81920), (4, 64, 40960), (4, 128, 20480)])
@pytest.mark.parametrize("longest", [20, 300])
def test_plain_causal(H, d, T, longest):
    lens = np.random.RandomState(H).randint(0, longest + 1, T)
    lens = lens[:np.searchsorted(np.cumsum(lens), T)]
    lens = [int(n) for n in lens] + [T - int(lens.sum())]
    torch.cuda.empty_cache()
    x, dout = make(lens, lens, H, H, d, 20)
    out, lse, ws = jfa.jfa_forward(**x, causal=True)
    dq, dk, dv, wb = jfa.jfa_backward(dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"], x["kv_offsets"], causal=True)
    assert jfa.jfa_check_status(ws) == 0 and jfa.jfa_check_status(wb) == 0
    part = slice(len(lens) - 400 // longest - 3, None)
    n = sum(lens[part])
    r, off = slice(T - n, T), offsets(lens[part])
    ref = orc.window_attention(x["q"][r], x["k"][r], x["v"][r], off, off, 1 << 40, 0, d ** -0.5, dout[r])
    for name, t in (("out", out[r]), ("lse", lse[:, r]), ("dq", dq[r]), ("dk", dk[r]), ("dv", dv[r])):
        close(t, ref[name], name)
