"""Calls of the windowed attention that need no gradient, and malformed ones."""
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
from test_gpu_window import make

pytestmark = pytest.mark.gpu


def leaves(seed):
    x, dout = make([140, 33], [140, 33], 2, 2, 64, seed)
    want = jfa.jfa_window_forward(**x, window=20, sinks=2)[0]
    for n in ("q", "k", "v"):
        x[n].requires_grad_()
    return x, dout, want


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_without_gradients(mode):
    """Leaves that require a gradient may be given where none is recorded."""
    x, _, want = leaves(70)
    with mode():
        out = jfa.window_attention(*x.values(), 20, 2)
    assert torch.equal(out, want) and not out.requires_grad


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_captured_without_gradients(mode):
    """Such a call accumulates nothing, so it is captured whatever eager graphs live; and it does not
    keep a training step of the same leaves from being captured."""
    x, dout, want = leaves(71)
    eager = jfa.window_attention(*x.values(), 20, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph), mode():  # (a capture begun in inference mode leaves torch unable to begin another outside)
        out = jfa.window_attention(*x.values(), 20, 2)
    graph.replay()
    assert torch.equal(out, want)
    del eager
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kept = jfa.window_attention(*x.values(), 20, 2)
        kept.backward(dout, retain_graph=True)
    torch.cuda.current_stream().wait_stream(side)
    with mode():
        jfa.window_attention(*x.values(), 20, 2)  # on the default stream, `kept` alive
    first = [x[n].grad.clone() for n in ("q", "k", "v")]
    for n in ("q", "k", "v"):
        x[n].grad = None
    step = torch.cuda.CUDAGraph()
    with torch.cuda.graph(step):
        jfa.window_attention(*x.values(), 20, 2).backward(dout)
    step.replay()
    assert all(torch.equal(x[n].grad, g) for n, g in zip(("q", "k", "v"), first))
    del kept


def test_missing_offsets_are_refused():
    x, dout, _ = leaves(72)
    out, lse, _ = jfa.jfa_window_forward(**x, window=20)
    for name in ("q_offsets", "kv_offsets"):
        for bad in (None, [0, 140, 173]):
            y = {**x, name: bad}
            with pytest.raises(ValueError, match="offsets"):
                jfa.jfa_window_forward(**y, window=20)
            with pytest.raises(ValueError, match="offsets"):
                jfa.jfa_window_backward(dout, y["q"], y["k"], y["v"], out, lse, y["q_offsets"], y["kv_offsets"], 20)
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda:0")
    t, n = torch.zeros(1, 4, dtype=torch.int32, device="cuda:0"), torch.zeros(1, dtype=torch.int32, device="cuda:0")
    for bad in (None, [0, 173]):
        with pytest.raises(ValueError, match="offsets"):
            jfa.jfa_cache_append(x["k"].detach(), x["v"].detach(), bad, c, c.clone(), t, n)


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_in_the_place_of_queries(d):
    """out may be q, and dq may be q, dout or out."""
    x, dout = make([300, 0, 5, 129], [300, 7, 5, 200], 4, 2, d, 73)
    want, wl, _ = jfa.jfa_window_forward(**x, window=40, sinks=3)
    q = x["q"].clone()
    out, lse, ws = jfa.jfa_window_forward(**{**x, "q": q}, window=40, sinks=3, out=q)
    assert jfa.jfa_check_status(ws) == 0 and torch.equal(out, want) and torch.equal(lse, wl)
    rest = (wl, x["q_offsets"], x["kv_offsets"], 40, 3)
    ref = jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], want, *rest)[:3]
    for i in range(3):
        a = [dout.clone(), x["q"].clone(), want.clone()]
        got = jfa.jfa_window_backward(a[0], a[1], x["k"], x["v"], a[2], *rest, dq=a[i])[:3]
        assert all(torch.equal(s, t) for s, t in zip(got, ref))
