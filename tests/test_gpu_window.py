"""Windowed jagged attention with sinks on the GPU, both directions, against float64 with
elementwise bounds (oracle/window_oracle.py)."""
import types

import numpy as np
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
import oracle.window_oracle as orc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64, device=DEV)


def make(lq, lk, H, G, d, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = lambda t, h: torch.empty(t, h, d, dtype=BF16, device=DEV).normal_(generator=g)
    return dict(q=n(sum(lq), H), k=n(sum(lk), G), v=n(sum(lk), G), q_offsets=offsets(lq), kv_offsets=offsets(lk)), n(sum(lq), H)


def close(got, ref, what):
    val, err = ref
    g = orc.f64(got)
    assert np.array_equal(np.isneginf(g), np.isneginf(val)), f"{what}: -inf pattern"
    fin = np.isfinite(val)
    bad = np.abs(g[fin] - val[fin]) - err[fin]
    assert np.all(np.isfinite(g[fin])) and (not bad.size or bad.max() <= 0), \
        f"{what}: {int((~(bad <= 0)).sum())} of {bad.size} values beyond their bound, worst by {np.nanmax(bad):.3g}"


def check(x, dout, W, S, scale=None):
    d = x["q"].shape[2]
    out, lse, ws = jfa.jfa_window_forward(**x, window=W, sinks=S, scale=scale)
    assert jfa.jfa_check_status(ws) == 0
    ref = orc.window_attention(*x.values(), W or 1 << 40, S, scale or d ** -0.5, dout)
    close(out, ref["out"], "out")
    close(lse, ref["lse"], "lse")
    if dout is None:
        return out, lse
    dq, dk, dv, ws = jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"], x["kv_offsets"], W, S,
                                             scale)
    assert jfa.jfa_check_status(ws) == 0
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        close(t, ref[n], n)
    return out, lse, dq, dk, dv


SELF = [1, 2, 127, 128, 129, 0, 255, 256, 257, 385, 513, 700]
MIXED = ([1, 130, 300, 0, 50, 128, 257, 5, 1, 300, 200], [500, 700, 100, 50, 0, 1281, 256, 3, 1, 900, 600])


@pytest.mark.parametrize("W,S", [(1, 0), (1, 1), (2, 3), (16, 4), (127, 0), (128, 1), (129, 16), (200, 17), (256, 128),
                                 (300, 64), (1000, 5), (None, 0), (None, 100)])
@pytest.mark.parametrize("d,H,G", [(64, 2, 1), (128, 2, 2)])
def test_self_attention(W, S, d, H, G):
    check(*make(SELF, SELF, H, G, d, 1), W, S)


@pytest.mark.parametrize("W,S", [(1, 0), (7, 2), (128, 4), (130, 128), (255, 33), (None, 0), (400, 0), (40, 100)])
@pytest.mark.parametrize("d,H,G", [(64, 3, 1), (128, 4, 2)])
def test_queries_and_keys_of_different_lengths(W, S, d, H, G):
    check(*make(*MIXED, H, G, d, 2), W, S)


@pytest.mark.parametrize("H,G", [(1, 1), (8, 1), (5, 5), (12, 3), (16, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_head_layouts(H, G, d):
    check(*make([200, 3, 129], [200, 3, 300], H, G, d, 3), 70, 4)


@pytest.mark.parametrize("d", [64, 128])
def test_long_sequences(d):
    """Several chunks of the sinks' gradient, long ranges of tiles per item."""
    check(*make([4500, 90, 2049], [4500, 90, 2600], 2, 1, d, 4), 300, 5)


@pytest.mark.parametrize("lq,lk", [([1], [1]), ([0, 0], [0, 3]), ([3, 0], [0, 0]), ([0], [200]), ([0, 5], [130, 0])])
@pytest.mark.parametrize("S", [0, 4])
def test_almost_nothing(lq, lk, S):
    x, dout = make(lq, lk, 2, 1, 64, 5)
    if sum(lk) == 0:
        x["k"], x["v"] = x["k"][:0], x["v"][:0]
    check(x, dout, 3, S)


@pytest.mark.parametrize("B", [300, 1500])
def test_many_sequences(B):
    r = np.random.RandomState(B)
    lq = [int(n) for n in r.randint(0, 40, B)]
    check(*make(lq, [n + int(m) for n, m in zip(lq, r.randint(0, 30, B))], 2, 1, 64, 6), 9, 3)


@pytest.mark.parametrize("d,G", [(64, 1), (128, 2)])
def test_unseen_keys_are_not_read(d, G):
    """Keys that no query sees may hold NaN, in every position relative to the tiles."""
    lq, lk, W, S = [1, 128, 100, 5, 1], [900, 600, 500, 140, 129], 60, 5
    x, dout = make(lq, lk, 2, G, d, 7)
    at = 0
    for n, m in zip(lq, lk):
        lo = max(0, m - n - W + 1)
        if lo > S:
            x["k"][at + S:at + lo] = float("nan")
            x["v"][at + S:at + lo] = float("inf")
        at += m
    _, _, _, dk, dv = check(x, dout, W, S)
    unseen = torch.isnan(x["k"].float())
    assert (dk[unseen] == 0).all() and (dv[unseen] == 0).all()


def test_neighbouring_sequences_do_not_mix():
    """A sequence of NaN leaves the others' results as they were, bit for bit."""
    lens = [130, 60, 257, 1]
    x, dout = make(lens, lens, 2, 1, 64, 8)
    run = lambda: jfa.jfa_window_forward(**x, window=50, sinks=3)[:2]
    out, lse = run()
    rows = torch.ones(sum(lens), dtype=torch.bool, device=DEV)
    rows[130:190] = False
    x["k"][130:190] = float("nan")
    x["v"][130:190] = float("inf")
    x["q"][130:190] = float("nan")
    out2, lse2 = run()
    assert torch.equal(out[rows], out2[rows]) and torch.equal(lse[:, rows], lse2[:, rows])
    do = torch.where(rows[:, None, None], dout, float("nan")).to(BF16)
    grads = jfa.jfa_window_backward(do, x["q"], x["k"], x["v"], out2, lse2, x["q_offsets"], x["kv_offsets"], 50, 3)[:3]
    assert all(torch.isfinite(g[rows]).all() for g in grads)


def test_a_wide_window_is_causal_attention():
    lens = [300, 70, 1, 513]
    x, dout = make(lens, lens, 2, 2, 64, 9)
    a, la = check(x, dout, 513, 0)[:2]
    b, lb, _ = jfa.jfa_forward(*x.values(), causal=True)
    assert torch.allclose(la, lb, rtol=0, atol=1e-5) and float((a.float() - b.float()).abs().max()) < 0.05
    ga = jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], a, la, x["q_offsets"], x["kv_offsets"], 513, 0)[:3]
    gb = jfa.jfa_backward(dout, x["q"], x["k"], x["v"], b, lb, x["q_offsets"], x["kv_offsets"], causal=True)[:3]
    for s, t in zip(ga, gb):
        assert float((s.float() - t.float()).norm() / t.float().norm()) < 4e-3  # other passes, both bf16


def test_results_are_reproducible():
    x, dout = make([2000, 700], [2000, 900], 4, 2, 64, 10)
    runs = []
    for _ in range(3):
        out, lse, _ = jfa.jfa_window_forward(**x, window=100, sinks=6)
        g = jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"], x["kv_offsets"], 100, 6)[:3]
        runs.append((out, lse, *g))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


def test_large_scores():
    x, dout = make([300, 20], [300, 20], 2, 1, 64, 11)
    x["q"] *= 20
    check(x, None, 40, 3, scale=1.0)


def test_autograd_with_shared_heads():
    x, dout = make([150, 40], [150, 90], 4, 2, 64, 12)
    for n in ("q", "k", "v"):
        x[n].requires_grad_()
    out = jfa.window_attention(*x.values(), 60, 4)
    out.backward(dout)
    ref = orc.window_attention(*(t.detach() for t in x.values()), 60, 4, 0.125, dout)
    close(out, ref["out"], "out")
    for n in ("q", "k", "v"):
        close(x[n].grad, ref["d" + n], "d" + n)
    # through a transposed upstream gradient, and only one input wanting it
    q = x["q"].detach().requires_grad_()
    out = jfa.window_attention(q, x["k"].detach(), x["v"].detach(), x["q_offsets"], x["kv_offsets"], 60, 4)
    (g,) = torch.autograd.grad(out.transpose(0, 1), q, dout.transpose(0, 1).contiguous())
    assert torch.equal(g, x["q"].grad)


def test_gradients_are_not_differentiable():
    x, dout = make([40], [40], 1, 1, 64, 14)
    q = x["q"].requires_grad_()
    out = jfa.window_attention(*x.values(), 8, 1)
    (g,) = torch.autograd.grad(out, q, dout.requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.float().sum().backward()


def test_autograd_in_a_graph():
    """A captured forward and backward pass of leaf tensors; refused while an eager graph of them,
    made on the default stream, is alive (its accumulators would run outside the capture)."""
    lens = [140, 33]
    x, dout = make(lens, lens, 2, 2, 64, 15)
    for n in ("q", "k", "v"):
        x[n].requires_grad_()
    out = jfa.window_attention(*x.values(), 20, 2)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="eager graph"):
        with torch.cuda.graph(graph):
            jfa.window_attention(*x.values(), 20, 2)
    del out, graph
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        jfa.window_attention(*x.values(), 20, 2).backward(dout)
    torch.cuda.current_stream().wait_stream(side)
    for n in ("q", "k", "v"):
        x[n].grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = jfa.window_attention(*x.values(), 20, 2)
        out.backward(dout)
    y, do = make(lens, lens, 2, 2, 64, 16)
    with torch.no_grad():
        for n in ("q", "k", "v"):
            x[n].copy_(y[n])
        dout.copy_(do)
    graph.replay()
    ref = orc.window_attention(*(t.detach() for t in x.values()), 20, 2, 0.125, dout)
    close(out, ref["out"], "out")
    for n in ("q", "k", "v"):
        close(x[n].grad, ref["d" + n], "d" + n)


def test_outputs_aligned_to_16_bytes():
    """Outputs that start on an odd multiple of 16 bytes."""
    lens, H, G, d = [130, 5], 2, 1, 128
    x, dout = make(lens, lens, H, G, d, 17)
    like = lambda t: torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[8:].view(t.shape)
    lse = torch.empty(H * sum(lens) + 4, device=DEV)[4:].view(H, sum(lens))
    out, _, _ = jfa.jfa_window_forward(**x, window=50, sinks=3, out=like(x["q"]), lse=lse)
    assert out.data_ptr() % 32 == 16
    want, wl, _ = jfa.jfa_window_forward(**x, window=50, sinks=3)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    args = (dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"], x["kv_offsets"], 50, 3)
    got = jfa.jfa_window_backward(*args, dq=like(x["q"]), dk=like(x["k"]), dv=like(x["v"]))
    for a, b in zip(got[:3], jfa.jfa_window_backward(*args)[:3]):
        assert torch.equal(a, b)


def test_training_step_in_a_graph():
    lens = [200, 129, 7]
    x, dout = make(lens, lens, 2, 1, 128, 13)
    H, G, d, T = 2, 1, 128, sum(lens)
    wf = jfa.new_window_workspace(3, H, G, d, T, T, 4, False, DEV)
    wb = jfa.new_window_workspace(3, H, G, d, T, T, 4, True, DEV)

    def step():
        out, lse, _ = jfa.jfa_window_forward(**x, window=33, sinks=4, workspace=wf)
        return out, lse, *jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"], x["kv_offsets"],
                                                  33, 4, workspace=wb)[:3]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (20, 21):
        y, do = make(lens, lens, H, G, d, seed)
        for n in ("q", "k", "v"):
            x[n].copy_(y[n])
        dout.copy_(do)
        graph.replay()
        assert jfa.jfa_check_status(wf) == 0 and jfa.jfa_check_status(wb) == 0
        ref = orc.window_attention(*x.values(), 33, 4, d ** -0.5, dout)
        for n, t in zip(("out", "lse", "dq", "dk", "dv"), got):
            close(t, ref[n], n)


def test_malformed_offsets_are_reported():
    x, dout = make([50, 30], [50, 30], 2, 1, 64, 14)
    ws = jfa.new_window_workspace(2, 2, 1, 64, 80, 80, 4, False, DEV)
    wb = jfa.new_window_workspace(2, 2, 1, 64, 80, 80, 4, True, DEV)
    out, lse, _ = jfa.jfa_window_forward(**x, window=8, sinks=4, workspace=ws)
    for bad in ([0, 90, 80], [1, 50, 80], [0, 50, 79], [0, -3, 80]):
        y = dict(x, kv_offsets=torch.tensor(bad, device=DEV))
        jfa.jfa_window_forward(**y, window=8, sinks=4, workspace=ws)
        assert jfa.jfa_check_status(ws) == 5
        jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"], y["kv_offsets"], 8, 4, workspace=wb)
        assert jfa.jfa_check_status(wb) == 5
    again, _, _ = jfa.jfa_window_forward(**x, window=8, sinks=4, workspace=ws)
    assert jfa.jfa_check_status(ws) == 0 and torch.equal(again, out)


@pytest.mark.parametrize("S", [0, 3, 16, 40])
def test_tensors_that_fill_their_memory(S):
    """Short sequences at the end of tensors that end with their allocation: loads of partial tiles
    must not touch what lies behind.  (A key row of 128 bytes; the sizes are whole 2 MB pages.)"""
    H, G, d, W = 8, 1, 64, 64
    lens = np.random.RandomState(3).randint(0, 21, 20000)
    lens = lens[:np.searchsorted(np.cumsum(lens), 163840)]
    lens = [int(x) for x in lens] + [163840 - int(lens.sum())]
    torch.cuda.empty_cache()
    x, dout = make(lens, lens, H, G, d, 19)
    out, lse, ws = jfa.jfa_window_forward(**x, window=W, sinks=S)
    dq, dk, dv, wb = jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"], x["kv_offsets"], W, S)
    assert jfa.jfa_check_status(ws) == 0 and jfa.jfa_check_status(wb) == 0
    for part in (slice(0, 120), slice(len(lens) - 120, None)):
        first = sum(lens[:part.start])
        n = sum(lens[part])
        r, off = slice(first, first + n), offsets(lens[part])
        ref = orc.window_attention(x["q"][r], x["k"][r], x["v"][r], off, off, W, S, d ** -0.5, dout[r])
        for name, t in (("out", out[r]), ("lse", lse[:, r]), ("dq", dq[r]), ("dk", dk[r]), ("dv", dv[r])):
            close(t, ref[name], name)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_beyond_2_billion_elements(d):
    """A short sequence behind one whose rows fill 2^31 elements: as if it were alone."""
    H, G, W, S = 16, 1, 16, 2
    lens = [(1 << 31) // (H * d) + 77, 40, 0, 130]
    x, dout = make(lens, lens, H, G, d, 18)
    out, lse, _ = jfa.jfa_window_forward(**x, window=W, sinks=S)
    dq, dk, dv, ws = jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"], x["kv_offsets"], W, S)
    assert jfa.jfa_check_status(ws) == 0
    r = slice(lens[0], None)
    off = offsets(lens[1:])
    ref = orc.window_attention(x["q"][r], x["k"][r], x["v"][r], off, off, W, S, d ** -0.5, dout[r])
    for n, t in (("out", out[r]), ("lse", lse[:, r]), ("dq", dq[r]), ("dk", dk[r]), ("dv", dv[r])):
        close(t, ref[n], n)


def test_one_workspace_for_calls_of_different_sizes():
    """A workspace made for the largest call serves every smaller one, forward and backward in turn."""
    ws = jfa.new_window_workspace(300, 8, 4, 128, 60000, 60000, 128, True, DEV)
    calls = []
    for i, (lens, H, G, d, W, S) in enumerate([([700, 1, 300, 0, 1290], 4, 2, 64, 100, 7), ([20] * 300, 8, 4, 128, 9, 128),
                                               ([5000, 3, 8000], 2, 1, 128, 999, 0), ([1], 1, 1, 64, 1, 1)]):
        x, dout = make(lens, lens, H, G, d, 40 + i)
        o = jfa.jfa_window_forward(**x, window=W, sinks=S)[:2]
        b = lambda ws, x=x, dout=dout, o=o, W=W, S=S: jfa.jfa_window_backward(
            dout, x["q"], x["k"], x["v"], *o, x["q_offsets"], x["kv_offsets"], W, S, workspace=ws)[:3]
        calls.append((lambda ws, x=x, W=W, S=S: jfa.jfa_window_forward(**x, window=W, sinks=S, workspace=ws)[:2], b, o, b(None)))
    for i in (0, 1, 2, 3, 1, 0, 3, 2, 0):
        f, b, o, g = calls[i]
        assert all(torch.equal(p, r) for p, r in zip(f(ws), o)) and all(torch.equal(p, r) for p, r in zip(b(ws), g))
    assert jfa.jfa_check_status(ws) == 0


def test_two_calls_at_once():
    calls = []
    for i, (lens, H, G, d) in enumerate([([700, 1, 300, 0, 1290], 4, 2, 64), ([513] * 9, 2, 2, 128)]):
        x, dout = make(lens, lens, H, G, d, 30 + i)
        want = check(x, None, 100, 7)
        grads = jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], *want, x["q_offsets"], x["kv_offsets"], 100, 7)[:3]
        calls.append((x, dout, (*want, *grads), torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for _ in range(6):
        for x, dout, _, side, got in calls:
            out, lse, _ = jfa.jfa_window_forward(**x, window=100, sinks=7, stream=side)
            got.append((out, lse, *jfa.jfa_window_backward(dout, x["q"], x["k"], x["v"], out, lse, x["q_offsets"],
                                                           x["kv_offsets"], 100, 7, stream=side)[:3]))
    torch.cuda.synchronize()
    for _, _, want, _, got in calls:
        assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))


def test_side_stream():
    x, dout = make([300], [300], 2, 1, 64, 15)
    want = jfa.jfa_window_forward(**x, window=64, sinks=2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = jfa.jfa_window_forward(**x, window=64, sinks=2, stream=side)
    assert jfa.jfa_check_status(got[2], side) == 0 and torch.equal(got[0], want[0])


def test_refusals_of_the_binding():
    x, dout = make([20], [20], 4, 2, 64, 16)
    for bad in (dict(q=x["q"].float()), dict(k=x["k"][:, :1].expand(20, 3, 64).contiguous()), dict(v=x["v"][:10]),
                dict(q=x["q"][:, ::2]), dict(window=0), dict(sinks=-1), dict(kv_offsets=offsets([10, 10])),
                dict(q_offsets=x["q_offsets"].int()), dict(out=x["k"]), dict(lse=torch.empty(4, 4, device=DEV)),
                dict(workspace=torch.zeros(256, dtype=torch.uint8, device=DEV)),
                dict(stream=types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0))):
        with pytest.raises(ValueError):
            jfa.jfa_window_forward(**{**dict(x, window=4, sinks=0), **bad})
    with pytest.raises(jfa.JfaError):
        jfa.jfa_window_forward(**x, window=4, sinks=129, workspace=torch.zeros(1 << 22, dtype=torch.uint8, device=DEV))


# ------------------------------------------------------------------ with the cache

def test_prompt_then_decoding():
    """A prompt (rotated and cached on the way, attended over jagged) and decoding steps over the
    cache give what one windowed pass over the whole sequences gives."""
    B, H, G, d, page, W, S, new = 3, 4, 2, 64, 16, 50, 4, 6
    prompt = [70, 3, 130]
    total = [n + new for n in prompt]
    g = torch.Generator(device=DEV)
    g.manual_seed(17)
    toks = [torch.empty(n, H + 2 * G, d, dtype=BF16, device=DEV).normal_(generator=g) for n in total]
    pages = sum((n + page - 1) // page for n in total)
    kc = torch.full((pages, G, page, d), float("nan"), dtype=BF16, device=DEV)
    vc = kc.clone()
    width = max((n + page - 1) // page for n in total)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    order, at = torch.randperm(pages, generator=g, device=DEV).to(torch.int32), 0
    for b, n in enumerate(total):
        m = (n + page - 1) // page
        table[b, :m] = order[at:at + m]
        at += m
    f = jfa.rotary_frequencies(d)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    x = torch.cat([t[:n] for t, n in zip(toks, prompt)])
    off = offsets(prompt)
    k_rot = torch.empty(sum(prompt), G, d, dtype=BF16, device=DEV)
    q_rot, k_rot, _, _ = jfa.jfa_cache_append(x[:, H:H + G], x[:, H + G:], off, kc, vc, table, lens, q=x[:, :H],
                                              frequencies=f, k_out=k_rot, lengths_out=lens)
    out, lse, _ = jfa.jfa_window_forward(q_rot, k_rot, x[:, H + G:].contiguous(), off, off, W, S)
    got, qs = [[o] for o in out.split(prompt)], [[q] for q in q_rot.split(prompt)]
    one = torch.arange(B + 1, device=DEV)
    for t in range(new):
        y = torch.stack([tk[n + t] for tk, n in zip(toks, prompt)])
        q1, _, _, _ = jfa.jfa_cache_append(y[:, H:H + G], y[:, H + G:], one, kc, vc, table, lens, q=y[:, :H], frequencies=f,
                                           lengths_out=lens)
        o, _, ws = jfa.jfa_cache_attention(q1, kc, vc, table, lens, W, S)
        assert jfa.jfa_check_status(ws) == 0
        for b in range(B):
            got[b].append(o[b:b + 1])
            qs[b].append(q1[b:b + 1])
    assert lens.tolist() == total
    for b in range(B):
        xs, pos = orc.f64(toks[b]), np.arange(total[b])
        q, k = torch.cat(qs[b]), torch.from_numpy(orc.cache_rows(kc, table, b, pos)).to(BF16)
        close(q, orc.rotate(xs[:, :H], pos, f), "queries")
        close(k, orc.rotate(xs[:, H:H + G], pos, f), "keys")
        ref = orc.window_attention(q, k, xs[:, H + G:], [0, total[b]], [0, total[b]], W, S, d ** -0.5)
        close(torch.cat(got[b]), ref["out"], f"sequence {b}")
