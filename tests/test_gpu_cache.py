"""The paged cache on the GPU: appending with the position rotation, and the attention of one
new token per sequence, against float64 with elementwise bounds (oracle/window_oracle.py)."""
import math

import numpy as np
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
import oracle.window_oracle as orc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.empty(shape, dtype=BF16, device=DEV).normal_(generator=g)


def make_cache(g, lens, G, d, page, spare_cols=1):
    """A cache whose every row holds NaN, and a shuffled page table (-1 where not needed)."""
    need = [(n + page - 1) // page for n in lens]
    P = sum(need) + 2
    order = torch.randperm(P, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((len(lens), max(need + [1]) + spare_cols), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    nan = torch.full((P, G, page, d), float("nan"), dtype=BF16, device=DEV)
    return nan.clone(), nan.clone(), table.to(DEV)


def fill(cache, table, b, positions, rows):
    page = cache.shape[2]
    pos = torch.as_tensor(positions, device=DEV)
    cache[table[b].long()[pos // page], :, pos % page] = rows


def filled(g, lens, G, d, page, window=None, sinks=0):
    """A cache that holds numbers at the visible keys and NaN everywhere else."""
    k, v, table = make_cache(g, lens, G, d, page)
    for b, n in enumerate(lens):
        pos = [j for j in range(n) if window is None or j >= n - window or j < sinks]
        if pos:
            fill(k, table, b, pos, normal(g, len(pos), G, d))
            fill(v, table, b, pos, normal(g, len(pos), G, d))
    return k, v, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def close(got, ref, what):
    val, err = ref
    g = orc.f64(got)
    assert np.array_equal(np.isneginf(g), np.isneginf(val)), f"{what}: -inf pattern"
    fin = np.isfinite(val)
    bad = np.abs(g[fin] - val[fin]) - err[fin]
    assert np.all(np.isfinite(g[fin])) and (not bad.size or bad.max() <= 0), \
        f"{what}: {int((~(bad <= 0)).sum())} of {bad.size} values beyond their bound, worst by {np.nanmax(bad):.3g}"


def check_attention(q, k, v, table, lens, window, sinks, scale=None, **kw):
    out, lse, ws = jfa.jfa_cache_attention(q, k, v, table, lens, window, sinks, scale, **kw)
    assert jfa.jfa_check_status(ws) == 0
    ref = orc.cache_attention(q, k, v, table, lens, window or 1 << 40, sinks, scale or 1 / math.sqrt(q.shape[-1]))
    close(out, ref["out"], "out")
    close(lse, ref["lse"], "lse")
    return out, lse


# lengths: none, one, around a page and a 64-key tile, several tiles
LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,H,G", [(64, 2, 2), (128, 4, 1), (128, 6, 2), (64, 16, 1)])
def test_attention_over_everything(page, d, H, G):
    g = gen(1)
    k, v, table, lens = filled(g, LENS, G, d, page)
    check_attention(normal(g, len(LENS), H, d), k, v, table, lens, None, 0)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 64), (65, 1), (100, 70), (128, 130), (1000, 4)])
@pytest.mark.parametrize("d,H,G,page", [(64, 8, 2, 16), (128, 3, 3, 64)])
def test_attention_with_window_and_sinks(window, sinks, d, H, G, page):
    g = gen(2)
    k, v, table, lens = filled(g, LENS + [777], G, d, page, window, sinks)
    # pages without a visible key are never looked up
    for b, n in enumerate(LENS + [777]):
        for pg in range(table.shape[1]):
            keys = range(pg * page, min(n, (pg + 1) * page))
            if not any(j >= n - window or j < sinks for j in keys):
                table[b, pg] = 1 << 30
    check_attention(normal(g, len(LENS) + 1, H, d), k, v, table, lens, window, sinks)


@pytest.mark.parametrize("H,G", [(16, 1), (17, 1), (40, 2), (33, 1)])
def test_attention_with_more_query_heads_than_one_block(H, G):
    g = gen(3)
    k, v, table, lens = filled(g, [5, 200, 0, 64], G, 64, 16)
    check_attention(normal(g, 4, H, 64), k, v, table, lens, None, 0)


@pytest.mark.parametrize("lens", [[20000], [1, 30000, 3], [4097, 5000, 1, 0, 9000]])
def test_attention_splits_long_sequences(lens):
    g = gen(4)
    k, v, table, n = filled(g, lens, 2, 128, 32)
    q = normal(g, len(lens), 4, 128)
    ws = jfa.new_cache_workspace(len(lens), 4, 2, 128, DEV)
    a = check_attention(q, k, v, table, n, None, 0, workspace=ws)
    at = ws.numel() - -(-len(lens) * 2 * 4 // 256) * 256  # the counters are the workspace's last part
    assert int(ws[at:].view(torch.int32).abs().sum()) == 0  # left at zero
    for _ in range(3):  # the order of the joins is fixed: the same bits every time
        b = jfa.jfa_cache_attention(q, k, v, table, n, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_one_workspace_for_calls_of_different_sizes():
    """A workspace made for the largest call serves the others in between: what one call leaves
    behind is never where another expects its counters at zero."""
    g = gen(13)
    ws = jfa.new_cache_workspace(900, 16, 2, 128, DEV)
    r = np.random.RandomState(1)
    sizes = [([20000], 16, 1, 128), ([int(x) for x in r.randint(100, 900, 900)], 2, 2, 64),
             ([9000, 5], 3, 1, 64), ([30000], 34, 2, 64)]
    calls = []
    for lens, H, G, d in sizes:
        k, v, table, n = filled(g, lens, G, d, 64)
        q = normal(g, len(lens), H, d)
        calls.append((q, k, v, table, n))
    alone = [jfa.jfa_cache_attention(*c)[:2] for c in calls]
    for i in (0, 1, 0, 2, 3, 1, 2, 0):
        out, lse, _ = jfa.jfa_cache_attention(*calls[i], workspace=ws)
        assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])
    check_attention(*calls[1], None, 0, workspace=ws)
    # an append in between, its lengths among the results
    rows = normal(g, 900, 2, 64)
    k, v, table, n = make_cache(g, [1] * 900, 2, 64, 16) + (torch.zeros(900, dtype=torch.int32, device=DEV),)
    jfa.jfa_cache_append(rows, rows, torch.arange(901, device=DEV), k, v, table, n, lengths_out=n, workspace=ws)
    assert bool((n == 1).all())
    out, lse, _ = jfa.jfa_cache_attention(*calls[3], workspace=ws)
    assert torch.equal(out, alone[3][0]) and torch.equal(lse, alone[3][1])
    assert jfa.jfa_check_status(ws) == 0


def test_attention_of_many_sequences():
    g = gen(5)
    r = np.random.RandomState(0)
    lens = [int(x) for x in r.randint(0, 90, 700)]
    k, v, table, n = filled(g, lens, 1, 64, 16)
    check_attention(normal(g, len(lens), 1, 64), k, v, table, n, 33, 2)


def test_attention_extreme_scores():
    """Scores of several hundred: the running maximum has to carry them."""
    g = gen(6)
    k, v, table, n = filled(g, [500, 64, 3], 1, 64, 16)
    check_attention(normal(g, 3, 2, 64) * 30, k, v, table, n, None, 0, scale=1.0)


def test_attention_reports_bad_pages_and_lengths():
    g = gen(7)
    k, v, table, n = filled(g, [40, 40], 1, 64, 16)
    q = normal(g, 2, 1, 64)
    ws = jfa.new_cache_workspace(2, 1, 1, 64, DEV)
    for bad in (-1, k.shape[0], 1 << 30):
        t = table.clone()
        t[1, 2] = bad
        out, _, _ = jfa.jfa_cache_attention(q, k, v, t, n, workspace=ws)
        assert jfa.jfa_check_status(ws) == 7
        assert torch.equal(out[0], jfa.jfa_cache_attention(q, k, v, table, n)[0][0])  # the others are right
    for bad in (-1, table.shape[1] * 16 + 1):
        n2 = n.clone()
        n2[0] = bad
        jfa.jfa_cache_attention(q, k, v, table, n2, workspace=ws)
        assert jfa.jfa_check_status(ws) == 5
    assert jfa.jfa_check_status(ws) == 0
    check_attention(q, k, v, table, n, None, 0, workspace=ws)  # the workspace is usable again


# ------------------------------------------------------------------ append

def check_append(lens, new, G, H, d, page, rot, interleaved=False, strided=False, pad_rows=0, in_place=False, base=1e4):
    g = gen(8)
    total = [a + n for a, n in zip(lens, new)]
    kc, vc, table = make_cache(g, total, G, d, page)
    T = sum(new) + pad_rows
    if strided:  # slices of one projection
        x = normal(g, T, (H + 2 * G) * d)
        q, k, v = (y.view(T, -1, d) for y in x.split([H * d, G * d, G * d], 1))
    else:
        q, k, v = normal(g, T, H, d), normal(g, T, G, d), normal(g, T, G, d)
    off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int64, device=DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    f = jfa.rotary_frequencies(rot, base) if rot else None
    pos = np.concatenate([np.arange(a, a + m) for a, m in zip(lens, new)] or [[]])
    kr, vr, qr = (orc.f64(y[:len(pos)]) for y in (k, v, q))
    k_out = k if in_place else torch.full((T, G, d), 7.0, dtype=BF16, device=DEV)
    q_out = q if in_place else torch.full((T, H, d), 7.0, dtype=BF16, device=DEV)
    tail = (q[len(pos):].clone(), k[len(pos):].clone()) if in_place else (q_out[len(pos):].clone(), k_out[len(pos):].clone())
    got_q, got_k, n_out, ws = jfa.jfa_cache_append(k, v, off, kc, vc, table, n, q=q, frequencies=f,
                                                   interleaved=interleaved, q_out=q_out, k_out=k_out)
    assert jfa.jfa_check_status(ws) == 0
    assert n_out.tolist() == total and n.tolist() == lens
    ff = f if f is not None else np.zeros(0)
    kref, qref = orc.rotate(kr, pos, ff, interleaved), orc.rotate(qr, pos, ff, interleaved)
    close(got_k[:len(pos)], kref, "k_out")
    close(got_q[:len(pos)], qref, "q_out")
    assert torch.equal(got_q[len(pos):], tail[0]) and torch.equal(got_k[len(pos):], tail[1])  # rows behind the last
    at = 0
    written = torch.zeros(kc.shape[0], page, dtype=torch.bool, device=DEV)
    for b, m in enumerate(new):
        if m:
            p = np.arange(lens[b], total[b])
            assert np.array_equal(orc.cache_rows(kc, table, b, p), orc.f64(got_k[at:at + m]))
            assert np.array_equal(orc.cache_rows(vc, table, b, p), vr[at:at + m])
            pt = torch.as_tensor(p, device=DEV)
            written[table[b].long()[pt // page], pt % page] = True
        at += m
    untouched = ~written[:, None, :, None].expand(kc.shape)
    assert torch.isnan(kc[untouched]).all() and torch.isnan(vc[untouched]).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (128, 128, False), (128, 32, False), (64, 16, False),
                                               (64, 64, True), (128, 48, True), (128, 0, False)])
def test_append(page, d, rot, interleaved):
    check_append([0, 5, 100, 17, 31, 0], [3, 1, 0, 40, 130, 1], 2, 6, d, page, rot, interleaved)


@pytest.mark.parametrize("kw", [dict(strided=True), dict(pad_rows=9), dict(in_place=True), dict(strided=True, pad_rows=3)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_strided_padded_in_place(kw, interleaved):
    check_append([4, 0, 60], [1, 2, 9], 3, 3, 64, 16, 64, interleaved, **kw)


@pytest.mark.parametrize("B,m", [(1, 1), (33, 1), (200, 1), (1025, 1), (3, 900), (40, 61)])
def test_append_many_sequences_and_long_prompts(B, m):
    r = np.random.RandomState(B)
    new = [int(x) for x in r.randint(0, m + 1, B)]
    check_append([int(x) for x in r.randint(0, 50, B)], new, 1, 2, 64, 16, 64)


def test_append_nothing():
    check_append([3, 0], [0, 0], 1, 1, 64, 16, 64)


def test_append_far_positions_and_odd_frequencies():
    """Angles stay exact at positions where an fp32 product would be off by radians."""
    d, page = 64, 128
    start = (1 << 30) + 12345
    pages = start // page + 2
    table = torch.zeros(1, pages, dtype=torch.int32, device=DEV)
    kc, vc = torch.zeros(1, 1, page, d, dtype=BF16, device=DEV), torch.zeros(1, 1, page, d, dtype=BF16, device=DEV)
    g = gen(9)
    k = normal(g, 4, 1, d)
    f = torch.cat([jfa.rotary_frequencies(d)[:29], torch.tensor([-0.7, 100.0, 0.0], dtype=torch.float64)])
    out = torch.empty_like(k)
    _, _, n, ws = jfa.jfa_cache_append(k, k, torch.tensor([0, 4], device=DEV), kc, vc, table,
                                       torch.tensor([start], dtype=torch.int32, device=DEV), frequencies=f, k_out=out)
    assert jfa.jfa_check_status(ws) == 0 and n.tolist() == [start + 4]
    # the frequency itself is a double: at 2^30 its last bit is 2^-23 radians of a radian
    val, err = orc.rotate(k, np.arange(start, start + 4), f)
    x = np.abs(orc.f64(k))
    size = np.concatenate([x[..., :32] + x[..., 32:]] * 2, -1)
    slack = np.abs(np.concatenate([f.numpy()] * 2)) * (start + 4) * 2.0 ** -52
    close(out, (val, err + size * slack), "k_out")


def test_append_reports_errors():
    g = gen(10)
    kc, vc, table = make_cache(g, [40, 40], 1, 64, 16, spare_cols=0)
    k = normal(g, 4, 1, 64)
    off = torch.tensor([0, 2, 4], device=DEV)
    ws = jfa.new_cache_workspace(2, 1, 1, 64, DEV)

    def run(lens=(30, 30), off=off, table=table):
        jfa.jfa_cache_append(k, k, off, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device=DEV), workspace=ws)
        return jfa.jfa_check_status(ws)

    assert run() == 0
    before = kc.clone()
    assert run(lens=(47, 0)) == 7                      # position 48 lies past the table
    assert run(lens=(2 ** 31 - 2, 0)) == 7
    t = table.clone()
    t[0, 1] = kc.shape[0]
    assert run(lens=(16, 30), table=t) == 7
    t[0, 1] = -1
    assert run(lens=(16, 30), table=t) == 7
    assert run(lens=(-3, 30)) == 5
    assert run(off=torch.tensor([0, 3, 2], device=DEV)) == 5
    assert run(off=torch.tensor([0, 3, 5], device=DEV)) == 5
    assert run(off=torch.tensor([1, 3, 4], device=DEV)) == 5
    assert run() == 0
    assert torch.isnan(before).sum() >= torch.isnan(kc).sum()


# ------------------------------------------------------------------ together

def test_decoding_steps_in_a_graph():
    """append (lengths advanced in place) and attention, captured once and replayed: each replay
    is the next step, and matches attention over the rotated history in float64."""
    B, G, H, d, page, W, S, steps = 3, 2, 4, 64, 16, 40, 3, 50
    g = gen(11)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    kc, vc, table = make_cache(g, [steps + 2] * B, G, d, page)
    x = normal(g, steps, B, H + 2 * G, d)
    cur = torch.empty_like(x[0])
    off = torch.arange(B + 1, device=DEV)
    f = jfa.rotary_frequencies(d)
    ws = jfa.new_cache_workspace(B, H, G, d, DEV)
    out, lse, q_rot = torch.empty(B, H, d, dtype=BF16, device=DEV), torch.empty(H, B, device=DEV), torch.empty(
        B, H, d, dtype=BF16, device=DEV)

    def step():
        jfa.jfa_cache_append(cur[:, H:H + G], cur[:, H + G:], off, kc, vc, table, lens, q=cur[:, :H], frequencies=f,
                             q_out=q_rot, lengths_out=lens, workspace=ws)
        jfa.jfa_cache_attention(q_rot, kc, vc, table, lens, W, S, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cur.copy_(x[0])
        step()  # the first step runs eagerly
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(1, steps):
        cur.copy_(x[t])
        graph.replay()
        if t in (1, 15, 16, 39, 40, 41, 49):
            assert lens.tolist() == [t + 1] * B
            ref = orc.cache_attention(q_rot, kc, vc, table, lens, W, S, d ** -0.5)
            close(out, ref["out"], f"step {t}")
            close(lse, ref["lse"], f"step {t}")
            hist = orc.rotate(orc.f64(x[:t + 1, :, H:H + G]).reshape(-1, G, d), np.repeat(np.arange(t + 1), B), f)
            for b in range(B):
                rows = slice(b, None, B)
                close(torch.as_tensor(orc.cache_rows(kc, table, b, np.arange(t + 1))), (hist[0][rows], hist[1][rows]), "keys")
    assert jfa.jfa_check_status(ws) == 0


def test_pages_beyond_4_billion_elements():
    """The last pages of caches of 2^32 elements and more."""
    g, G, d, page, B = gen(14), 2, 128, 128, 3
    P = (1 << 32) // (G * page * d) + 8
    kc = torch.empty(P, G, page, d, dtype=BF16, device=DEV)
    vc = torch.empty_like(kc)
    table = (P - 1 - torch.arange(2 * B, device=DEV, dtype=torch.int32)).view(B, 2)
    n = torch.tensor([0, 100, 255], dtype=torch.int32, device=DEV)
    for b in range(B):
        for t in (kc, vc):
            if n[b]:
                fill(t, table, b, range(int(n[b])), normal(g, int(n[b]), G, d))
    k, v, q, off = normal(g, B, G, d), normal(g, B, G, d), normal(g, B, 4, d), torch.arange(B + 1, device=DEV)
    f = jfa.rotary_frequencies(d)
    k_out = torch.empty_like(k)
    q2, _, n2, ws = jfa.jfa_cache_append(k, v, off, kc, vc, table, n, q=q, frequencies=f, k_out=k_out)
    assert jfa.jfa_check_status(ws) == 0 and n2.tolist() == [1, 101, 256]
    close(k_out, orc.rotate(k, n.cpu().numpy(), f), "k_out")
    for b in range(B):
        at = table[b, int(n[b]) // page].long(), slice(None), int(n[b]) % page
        assert torch.equal(kc[at], k_out[b]) and torch.equal(vc[at], v[b])
    check_attention(q2, kc, vc, table, n2, None, 0)


def test_two_calls_at_once():
    g = gen(15)
    calls = []
    for lens, H, G in (([9000, 300, 0, 5000], 4, 2), ([200] * 150 + [7000], 8, 1)):
        k, v, table, n = filled(g, lens, G, 128, 64)
        q = normal(g, len(lens), H, 128)
        ws = jfa.new_cache_workspace(len(lens), H, G, 128, DEV)
        calls.append(((q, k, v, table, n, 4000, 9), ws, torch.cuda.Stream(), jfa.jfa_cache_attention(q, k, v, table, n, 4000, 9)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (args, ws, side, _) in enumerate(calls):
            got[i].append(jfa.jfa_cache_attention(*args, workspace=ws, stream=side))
    torch.cuda.synchronize()
    for (_, ws, side, want), results in zip(calls, got):
        assert jfa.jfa_check_status(ws, side) == 0
        assert all(torch.equal(r[0], want[0]) and torch.equal(r[1], want[1]) for r in results)


def test_calls_on_a_side_stream():
    g = gen(12)
    k, v, table, n = filled(g, [300, 70], 2, 64, 16)
    q = normal(g, 2, 4, 64)
    want = jfa.jfa_cache_attention(q, k, v, table, n, 100, 4)[:2]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = jfa.jfa_cache_attention(q, k, v, table, n, 100, 4, stream=side)
    assert jfa.jfa_check_status(got[2], side) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals_of_the_binding():
    g = gen(13)
    k, v, table, n = filled(g, [30], 2, 64, 16)
    q = normal(g, 1, 4, 64)
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q.expand(2, 4, 64)), dict(k_cache=k.float()),
                dict(v_cache=v[:-1]), dict(page_table=table.long()), dict(lengths=n.long()), dict(lengths=n.repeat(2)),
                dict(window=0), dict(sinks=-1), dict(page_table=table[:, ::2]), dict(k_cache=k.cpu()),
                dict(lse=torch.empty(1, 4, device=DEV)), dict(out=q[:, :2]), dict(workspace=torch.zeros(64, device=DEV))):
        a = dict(q=q, k_cache=k, v_cache=v, page_table=table, lengths=n)
        a.update(bad)
        with pytest.raises(ValueError):
            jfa.jfa_cache_attention(**a)
    kn, off = normal(g, 3, 2, 64), torch.tensor([0, 3], device=DEV)
    for bad in (dict(k=kn[:, :1]), dict(v=kn[:2]), dict(k=kn.float()), dict(offsets=off.int()), dict(offsets=off[:1]),
                dict(q_out=kn), dict(k_out=kn[:2]), dict(frequencies=torch.ones(8)), dict(lengths_out=n.long()),
                dict(frequencies=torch.ones(8, dtype=torch.float64, device=DEV)), dict(k=kn.transpose(0, 1)),
                dict(k=torch.empty(3, 2, 65, dtype=BF16, device=DEV)[..., 1:])):
        a = dict(k=kn, v=kn, offsets=off, k_cache=k, v_cache=v, page_table=table, lengths=n)
        a.update(bad)
        with pytest.raises(ValueError):
            jfa.jfa_cache_append(**a)
    with pytest.raises(jfa.JfaError):
        jfa.jfa_cache_append(kn, kn, off, k, v, table, n, frequencies=torch.ones(12, dtype=torch.float64))
