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


@pytest.mark.parametrize("in_place", [False, True])
def test_lengths_after_an_error(in_place):
    """A sequence keeps its length when a token of it was not stored; malformed offsets change none."""
    g = gen(62)
    kc, vc, table = make_cache(g, [40, 40, 40], 1, 64, 16, spare_cols=0)  # three pages each
    k = normal(g, 90, 1, 64)
    ws = jfa.new_cache_workspace(3, 1, 1, 64, DEV)

    def run(lens, offs, table=table):
        n = int32(lens)
        out = n if in_place else torch.full((3,), 77, dtype=torch.int32, device=DEV)
        jfa.jfa_cache_append(k, k, torch.tensor(offs, device=DEV), kc, vc, table, n, lengths_out=out, workspace=ws)
        return jfa.jfa_check_status(ws), out.tolist()

    def with_page(b, i, page):
        t = table.clone()
        t[b, i] = page
        return t

    assert run((30, 0, 7), (0, 2, 4, 4)) == (0, [32, 2, 7])
    assert run((47, 0, 7), (0, 2, 4, 9)) == (7, [47, 2, 12])              # position 48 lies past the table
    assert run((46, 48, 7), (0, 2, 3, 9)) == (7, [48, 48, 13])
    assert run((2 ** 31 - 1, 0, 0), (0, 2, 4, 9)) == (7, [2 ** 31 - 1, 2, 5])
    for bad in (-1, kc.shape[0], 1 << 30):
        assert run((14, 0, 7), (0, 2, 4, 4), with_page(0, 1, bad)) == (0, [16, 2, 7])       # not needed
        assert run((15, 0, 7), (0, 2, 4, 4), with_page(0, 1, bad)) == (7, [15, 2, 7])
        assert run((0, 40, 0), (0, 40, 42, 90), with_page(0, 2, bad)) == (7, [0, 42, 48])   # its last page
        assert run((0, 40, 0), (0, 40, 42, 82), with_page(2, 0, bad)) == (7, [40, 42, 0])   # its first
    assert run((-3, 30, 5), (0, 2, 4, 4)) == (5, [-3, 32, 5])
    assert run((5, 6, 7), (0, 2, 4, 4), with_page(2, 0, -1)) == (0, [7, 8, 7])              # nothing for it to store
    for offs in ([0, 3, 2, 4], [0, 3, 5, 91], [1, 3, 4, 5], [0, -1, 3, 5], [0, 2, 4, 1 << 40]):
        status, after = run((5, 6, 7), offs)  # such offsets also put tokens past the table: either error may be the first
        assert status in (5, 7) and after == [5, 6, 7]
    assert run((5, 6, 7), (0, 2, 4, 4)) == (0, [7, 8, 7])
    # a status that nobody has read yet does not hold later calls back
    n = int32([47, 0, 7])
    jfa.jfa_cache_append(k, k, torch.tensor([0, 2, 4, 9], device=DEV), kc, vc, table, n, lengths_out=n, workspace=ws)
    jfa.jfa_cache_append(k, k, torch.tensor([0, 0, 4, 9], device=DEV), kc, vc, table, n, lengths_out=n, workspace=ws)
    assert n.tolist() == [47, 6, 17] and jfa.jfa_check_status(ws) == 7


def test_decoding_without_a_pause():
    """Steps enqueued one behind the other give what synchronised steps give, bit for bit."""
    B, H, G, d, page, steps = 48, 8, 2, 64, 16, 300
    g = gen(63)
    start = [int(x) for x in np.random.RandomState(2).randint(0, 200, B)]
    k0, v0, table = make_cache(g, [n + steps for n in start], G, d, page)
    k0.zero_(), v0.zero_()
    x = normal(g, steps, B, H + 2 * G, d)
    off, f = torch.arange(B + 1, device=DEV), jfa.rotary_frequencies(d)

    def run(wait):
        kc, vc, n = k0.clone(), v0.clone(), int32(start)
        ws = jfa.new_cache_workspace(B, H, G, d, DEV)
        q_rot = torch.empty(B, H, d, dtype=BF16, device=DEV)
        outs = torch.empty(steps, B, H, d, dtype=BF16, device=DEV)
        lses = torch.empty(steps, H, B, device=DEV)
        torch.cuda.synchronize()
        for t in range(steps):
            jfa.jfa_cache_append(x[t][:, H:H + G], x[t][:, H + G:], off, kc, vc, table, n, q=x[t][:, :H], frequencies=f,
                                 q_out=q_rot, lengths_out=n, workspace=ws)
            if wait:
                torch.cuda.synchronize()
            jfa.jfa_cache_attention(q_rot, kc, vc, table, n, 150, 3, out=outs[t], lse=lses[t], workspace=ws)
            if wait:
                torch.cuda.synchronize()
        assert jfa.jfa_check_status(ws) == 0 and n.tolist() == [a + steps for a in start]
        return outs, lses, kc, vc

    want = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))


def test_attention_refuses_a_workspace_that_served_other_calls():
    """Where another call's data may have reached its counters: an error instead of wrong sums, until
    the workspace is zeroed.  A call that did not reach them changes nothing."""
    g = gen(65)
    k, v, table, n = filled(g, [9000, 700, 3], 2, 64, 64)
    q = normal(g, 3, 2, 64)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    check_attention(q, k, v, table, n, None, 0, workspace=ws)
    for lens, refused in (([1] * 20000, True), ([2000], False)):
        x, _ = make(lens, lens, 2, 2, 64, 64)
        for call in (lambda: jfa.jfa_window_forward(**x, window=90, sinks=2, workspace=ws),
                     lambda: jfa.jfa_forward(**x, workspace=ws)):
            call()
            if refused:
                for _ in range(2):
                    jfa.jfa_cache_attention(q, k, v, table, n, workspace=ws)
                    assert jfa.jfa_check_status(ws) == 3
                ws.zero_()
            check_attention(q, k, v, table, n, None, 0, workspace=ws)
