"""Items of the windowed backward that run for seconds: 4096 query heads share one key head."""
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("d,tiles", [(64, 256), (128, 288)])
def test_key_tiles_of_a_large_group(d, tiles):
    """The first key tile sums over 4096 x `tiles` query tiles, 2.5 and 3.6 s.  Keys are zeros, so P_ij =
    1 / (i + 1) for j <= i; values ones, so out = 1, dS = 0, and with dout = 1 in a few heads dv_j =
    sum over i >= j of (number of those heads) / (i + 1).  Everything that is zero or one is exact; P
    is off by half a bf16 step (and by the roundings of lse, below 16, and its product with log2 e: 2^-19),
    dv by half a step more, and its fp32 sum over `n` nonzero products of 16 queries by at most n 2^-23
    of its size."""
    H, T = 4096, 128 * tiles
    torch.cuda.empty_cache()
    ones = torch.ones(T, H, d, dtype=torch.bfloat16, device=DEV)  # q and out
    dout = torch.zeros_like(ones)
    heads = [0, 1000, 4095]
    dout[:, heads] = 1
    k, v = torch.zeros(T, 1, d, dtype=torch.bfloat16, device=DEV), torch.ones(T, 1, d, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, T], device=DEV)
    i = torch.arange(T, device=DEV)
    lse = (i + 1).double().log().float().expand(H, T).contiguous()
    dq, dk, dv, ws = jfa.jfa_window_backward(dout, ones, k, v, ones, lse, off, off)
    assert jfa.jfa_check_status(ws) == 0
    # dP_ij = D_i = d in the heads of dout, both exact
    assert not dq.any() and not dk.any()
    want = len(heads) * torch.flip(torch.cumsum(torch.flip(1.0 / (i + 1).double(), [0]), 0), [0])
    n = len(heads) * T / 16
    bound = want * (2 * 2.0 ** -8 + 2.0 ** -19 + n * 2.0 ** -23 + 2.0 ** -15)  # 2^-15: the terms' products
    assert ((dv[:, 0].double() - want[:, None]).abs() <= bound[:, None]).all()
