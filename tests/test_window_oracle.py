"""The float64 reference of the windowed attention pinned against an independent dense
formulation (torch autograd in float64), finite differences and closed forms; and the windowed
calls' host-side refusals (CPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
import oracle.window_oracle as orc


def problem(lq, lk, H, G, d, seed):
    r = np.random.RandomState(seed)
    q_off, k_off = np.concatenate([[0], np.cumsum(lq)]), np.concatenate([[0], np.cumsum(lk)])
    n = lambda t, h: r.standard_normal((t, h, d))
    return n(q_off[-1], H), n(k_off[-1], G), n(k_off[-1], G), q_off, k_off, n(q_off[-1], H)


CASES = [([5, 0, 9, 1, 7], [5, 3, 20, 1, 4], 4, 2, 3, 2), ([12], [12], 2, 1, 5, 0), ([6, 6], [6, 30], 3, 3, 100, 4),
         ([8, 3], [3, 8], 2, 2, 1, 1), ([10], [10], 2, 2, 2, 10)]


@pytest.mark.parametrize("lq,lk,H,G,W,S", CASES)
def test_against_autograd(lq, lk, H, G, W, S):
    q, k, v, qo, ko, do = problem(lq, lk, H, G, 8, 1)
    ref = orc.window_attention(q, k, v, qo, ko, W, S, 0.3, do)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    outs = []
    for b in range(len(lq)):
        Q, K, V = tq[qo[b]:qo[b + 1]], tk[ko[b]:ko[b + 1]], tv[ko[b]:ko[b + 1]]
        for i in range(lq[b]):
            p = i + lk[b] - lq[b]
            keys = [j for j in range(lk[b]) if j <= p and (p - j < W or j < S)]
            for h in range(H):
                if not keys:
                    outs.append(torch.zeros(8, dtype=torch.float64))
                    continue
                s = 0.3 * K[keys, h // (H // G)] @ Q[i, h]
                assert abs(float(torch.logsumexp(s, 0)) - ref["lse"][0][h, qo[b] + i]) < 1e-12
                outs.append(torch.softmax(s, 0) @ V[keys, h // (H // G)])
    out = torch.stack(outs).view(-1, H, 8)
    assert np.abs(out.detach().numpy() - ref["out"][0]).max() < 1e-13
    out.backward(torch.tensor(do))
    for n, t in (("dq", tq), ("dk", tk), ("dv", tv)):
        assert np.abs(t.grad.numpy() - ref[n][0]).max() < 1e-12, n


def test_finite_differences():
    lq, lk, H, G, W, S = CASES[0]
    q, k, v, qo, ko, do = problem(lq, lk, H, G, 4, 2)
    ref = orc.window_attention(q, k, v, qo, ko, W, S, 0.5, do)
    f = lambda: float((orc.window_attention(q, k, v, qo, ko, W, S, 0.5)["out"][0] * do).sum())
    r = np.random.RandomState(3)
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        for _ in range(12):
            i = tuple(r.randint(0, m) for m in x.shape)
            old, h = x[i], 1e-5
            x[i] = old + h
            up = f()
            x[i] = old - h
            down = f()
            x[i] = old
            assert abs((up - down) / (2 * h) - ref[n][0][i]) < 1e-7


def test_closed_forms():
    q, k, v, qo, ko, do = problem([6], [6], 1, 1, 4, 3)
    r = orc.window_attention(q, k, v, qo, ko, 1, 0, 1.0, do)  # itself alone
    assert np.allclose(r["out"][0], v) and np.allclose(r["dv"][0], do) and np.allclose(r["dq"][0], 0)
    r = orc.window_attention(q * 0, k, v, qo, ko, 2, 1, 1.0)  # the mean of the visible values
    assert np.allclose(r["out"][0][4, 0], (v[0, 0] + v[3, 0] + v[4, 0]) / 3)
    k[1:4] = np.nan  # keys that one late query does not see
    r = orc.window_attention(q[:1], k, v, [0, 1], ko, 2, 1, 1.0, do[:1])
    assert np.isfinite(r["out"][0]).all() and np.all(r["dk"][0][1:4] == 0)


def test_a_wrong_mask_is_caught():
    q, k, v, qo, ko, do = problem([9], [20], 2, 1, 8, 4)
    ref = orc.window_attention(q, k, v, qo, ko, 4, 2, 0.4)["out"]
    for W, S in ((5, 2), (3, 2), (4, 1), (4, 3)):
        other = orc.window_attention(q, k, v, qo, ko, W, S, 0.4)["out"][0]
        assert (np.abs(other - ref[0]) > ref[1]).any()


def test_rotation_against_complex_numbers():
    r = np.random.RandomState(5)
    x, pos, f = r.standard_normal((7, 2, 16)), np.array([0, 1, 2, 50, 1000, 10 ** 6, 3]), jfa.rotary_frequencies(12).numpy()
    z = np.exp(1j * pos[:, None] * f)[:, None]
    a = orc.rotate(x, pos, f)[0]
    w = (x[..., :6] + 1j * x[..., 6:12]) * z
    assert np.allclose(a[..., :6], w.real) and np.allclose(a[..., 6:12], w.imag) and np.array_equal(a[..., 12:], x[..., 12:])
    a = orc.rotate(x, pos, f, True)[0]
    w = (x[..., 0:12:2] + 1j * x[..., 1:12:2]) * z
    assert np.allclose(a[..., 0:12:2], w.real) and np.allclose(a[..., 1:12:2], w.imag)


# ------------------------------------------------------------------ refusals

def fwd(**over):
    a = dict(q=16, k=16, v=16, qo=16, ko=16, B=2, H=4, G=2, d=64, tq=10, tk=10, window=8, sinks=4, scale=0.125, out=16,
             lse=16, ws=256, wsb=1 << 30)
    a.update(over)
    return jfa.load_library().jfa_window_forward(a["q"], a["k"], a["v"], a["qo"], a["ko"], a["B"], a["H"], a["G"], a["d"],
                                                 a["tq"], a["tk"], a["window"], a["sinks"], a["scale"], a["out"],
                                                 a["lse"], a["ws"], a["wsb"], None)


def bwd(**over):
    a = dict(dout=16, q=16, k=16, v=16, out=16, lse=16, qo=16, ko=16, B=2, H=4, G=2, d=64, tq=10, tk=10, window=8,
             sinks=4, scale=0.125, dq=16, dk=16, dv=16, ws=256, wsb=1 << 30)
    a.update(over)
    return jfa.load_library().jfa_window_backward(a["dout"], a["q"], a["k"], a["v"], a["out"], a["lse"], a["qo"], a["ko"],
                                                  a["B"], a["H"], a["G"], a["d"], a["tq"], a["tk"], a["window"], a["sinks"],
                                                  a["scale"], a["dq"], a["dk"], a["dv"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("over,status", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(G=8), 1), (dict(d=96), 2), (dict(window=0), 1),
    (dict(window=-5), 1), (dict(sinks=-1), 1), (dict(sinks=129), 2), (dict(scale=0.0), 1), (dict(scale=math.inf), 1),
    (dict(q=18), 1), (dict(k=None), 1), (dict(v=24), 1), (dict(out=None), 1), (dict(lse=20), 1), (dict(qo=None), 1),
    (dict(tq=-1), 1), (dict(tk=1 << 40), 1), (dict(ws=None), 3), (dict(ws=128), 3), (dict(wsb=512), 3)])
def test_windowed_calls_check_their_arguments(call, over, status):
    assert call(**over) == status


def test_backward_checks_gradients():
    for n in ("dout", "dq", "dk", "dv"):
        assert bwd(**{n: None}) == 1 and bwd(**{n: 24}) == 1


def test_no_rows_is_no_work():
    assert fwd(tq=0, q=None, out=None, lse=None) == 0
    assert bwd(tq=0, tk=0, dout=None, q=None, k=None, v=None, out=None, lse=None, dq=None, dk=None, dv=None) == 0


def test_workspace_size():
    f = jfa.window_workspace_size
    assert f(2, 4, 3, 64, 10, 10, 0, False) == 0 and f(2, 4, 2, 64, 10, 10, 129, False) == 0
    assert 0 < f(2, 4, 2, 64, 1000, 1000, 0, False) < f(2, 4, 2, 64, 1000, 1000, 4, False)
    assert f(2, 4, 2, 64, 1000, 1000, 4, True) < f(2, 4, 2, 64, 1000, 1000, 64, True)
    with pytest.raises(ValueError):
        jfa.new_window_workspace(2, 4, 3, 64, 10, 10, 0, False, "cpu")


def test_cpu_tensors_are_refused():
    x, off = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 3])
    with pytest.raises(ValueError, match="CUDA"):
        jfa.jfa_window_forward(x, x, x, off, off, 4)
    with pytest.raises(ValueError, match="CUDA"):
        jfa.window_attention(x, x, x, off, off, 4)
