"""What a NaN leaves behind: the rows that see it get out = NaN and lse = NaN (not the -inf of a row
without keys), the backward pass carries it into their gradients, and nothing else changes."""
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
import oracle.window_oracle as orc
from test_gpu_window import make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
NAN = float("nan")
LENS, W, S = [300, 0, 130], 50, 3


def seeing(key):
    """Rows of the first sequence that see its key."""
    return torch.as_tensor(orc.visible(LENS[0], LENS[0], W, S)[:, key], device=DEV)


def run(x, dout):
    out, lse, ws = jfa.jfa_window_forward(**x, window=W, sinks=S)
    g = jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"], x["kv_offsets"], W, S)
    assert jfa.jfa_check_status(ws) == 0 and jfa.jfa_check_status(g[3]) == 0
    return out, lse, *g[:3]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("key", [1, 40, 200, 299])  # a sink, keys of the window part, the last
def test_windowed_key(d, key):
    x, dout = make(LENS, LENS, 4, 2, d, 50)
    want = run(x, dout)
    x["k"][key, 1] = NAN  # of query heads 2 and 3
    out, lse, dq, dk, dv = run(x, dout)
    rows = torch.zeros(sum(LENS), dtype=torch.bool, device=DEV)
    rows[:LENS[0]] = seeing(key)
    assert torch.isnan(lse[2:, rows]).all() and torch.isnan(out[rows, 2:]).all() and torch.isnan(dq[rows, 2:]).all()
    assert torch.equal(lse[2:, ~rows], want[1][2:, ~rows]) and torch.equal(out[~rows, 2:], want[0][~rows, 2:])
    seen = torch.as_tensor(orc.visible(LENS[0], LENS[0], W, S), device=DEV)[rows[:LENS[0]]].any(0).nonzero()[:, 0]
    assert torch.isnan(dk[seen, 1]).all() and torch.isnan(dv[seen, 1]).all()
    for got, ref in zip((out[:, :2], lse[:2], dq[:, :2], dk[:, 0], dv[:, 0]),
                        (want[0][:, :2], want[1][:2], want[2][:, :2], want[3][:, 0], want[4][:, 0])):
        assert torch.equal(got, ref)
    for got, ref in zip((out, dq, dk, dv), (want[0], want[2], want[3], want[4])):
        assert torch.equal(got[LENS[0]:], ref[LENS[0]:])


@pytest.mark.parametrize("d", [64, 128])
def test_windowed_query(d):
    x, dout = make(LENS, LENS, 4, 2, d, 51)
    want = run(x, dout)
    x["q"][77, 3] = NAN
    out, lse, dq, _, _ = run(x, dout)
    assert torch.isnan(lse[3, 77]) and torch.isnan(out[77, 3]).all() and torch.isnan(dq[77, 3]).all()
    assert int(torch.isnan(lse).sum()) == 1 and int(torch.isnan(out).sum()) == d
    assert torch.equal(lse[:3], want[1][:3]) and torch.equal(out[:, :3], want[0][:, :3])


@pytest.mark.parametrize("where", ["k", "q"])
@pytest.mark.parametrize("lens,d,H,G", [([0, 100, 70], 64, 4, 2), ([30000, 5], 128, 2, 1)])  # whole units, a split one
def test_cache_attention(where, lens, d, H, G):
    g = torch.Generator(device=DEV)
    g.manual_seed(52)
    n = lambda *s: torch.empty(s, dtype=BF16, device=DEV).normal_(generator=g)
    page, B = 64, len(lens)
    width = (max(lens) + page - 1) // page
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    k, v, q = n(B * width, G, page, d), n(B * width, G, page, d), n(B, H, d)
    length = torch.tensor(lens, dtype=torch.int32, device=DEV)
    b = max(range(B), key=lambda i: lens[i])
    want = jfa.jfa_cache_attention(q, k, v, table, length)
    heads = torch.zeros(H, dtype=torch.bool, device=DEV)
    if where == "k":
        k[table[b, lens[b] // 2 // page].long(), G - 1, lens[b] // 2 % page] = NAN
        heads[H - H // G:] = True
    else:
        q[b, 1] = NAN
        heads[1] = True
    out, lse, ws = jfa.jfa_cache_attention(q, k, v, table, length)
    assert jfa.jfa_check_status(ws) == 0
    hit = torch.zeros(B, H, dtype=torch.bool, device=DEV)
    hit[b, heads] = True
    assert torch.isnan(lse.t()[hit]).all() and torch.isnan(out[hit]).all()
    assert torch.equal(lse.t()[~hit], want[1].t()[~hit]) and torch.equal(out[~hit], want[0][~hit])
