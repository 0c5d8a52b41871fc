"""The plain call's rows that meet a NaN: out = NaN and lse = NaN, not the -inf of a row without keys."""
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
from test_gpu_window import make

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("biased", [False, True])
def test_query_and_key(causal, d, biased):
    lens = [300, 0, 130]
    x, _ = make(lens, lens, 2, 2, d, 53)
    bias = torch.randn(2, 700, device="cuda:0") * 0.1 if biased else None
    run = lambda: jfa.jfa_forward(**x, causal=causal, bias=bias, bias_center=350)
    want = run()
    x["q"][77, 1] = NAN
    out, lse, ws = run()
    assert jfa.jfa_check_status(ws) == 0
    assert torch.isnan(lse[1, 77]) and torch.isnan(out[77, 1]).all() and int(torch.isnan(lse).sum()) == 1
    assert torch.equal(lse[0], want[1][0]) and torch.equal(out[:, 0], want[0][:, 0])
    x["q"][77, 1] = 1.0
    x["k"][200, 0] = NAN
    out, lse, _ = run()
    rows = slice(200 if causal else 0, 300)
    assert torch.isnan(lse[0, rows]).all() and torch.isnan(out[rows, 0]).all()
    assert torch.equal(lse[:, 300:], want[1][:, 300:]) and torch.equal(out[300:], want[0][300:])
