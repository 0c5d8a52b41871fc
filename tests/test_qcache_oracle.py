"""Pins of the 8-bit cache's reference (CPU): codes against PyTorch's casts, scales against their definition,
the attention against a dense softmax, and mistakes that the pins have to catch."""
import numpy as np
import pytest
import torch

import oracle.qcache_oracle as qo
import oracle.window_oracle as wo


def test_e4m3_codes_are_pytorchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(qo.decode(codes, "e4m3"), codes.double().numpy(), equal_nan=True)
    assert np.array_equal(qo.decode(torch.arange(-128, 128).to(torch.int8), "int8"), np.arange(-128.0, 128.0))


def test_nearest_is_the_cast():
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(20000, generator=g) * 2.0 ** torch.randint(-12, 9, (20000,), generator=g)]).clamp(-448, 448)
    # every code, and every point half-way between two
    v = np.unique(qo.e4m3_values()[np.isfinite(qo.e4m3_values())])
    x = torch.cat([x, torch.from_numpy(np.concatenate([v, (v[1:] + v[:-1]) / 2])).float()])
    assert np.array_equal(qo.nearest(x.numpy(), "e4m3"), x.to(torch.float8_e4m3fn).double().numpy())
    y = torch.cat([x[x.abs() <= 127], torch.arange(-127, 127) + 0.5])
    assert np.array_equal(qo.nearest(y.numpy(), "int8"), y.round().double().numpy())
    assert qo.nearest(1e9, "e4m3") == 448 and qo.nearest(-1e9, "int8") == -127


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("rotated", [False, True])
def test_scales_hold_their_values(kind, rotated):
    amax = torch.arange(0, 0x7f80, dtype=torch.int16).view(torch.bfloat16).double().numpy()[::7]
    c = np.sqrt(2.0) if rotated else 1.0
    for a in amax:
        s = qo.needed_scale(a, kind, rotated)
        assert qo.MOST[kind] * s >= c * a and (s == 2.0 ** -126 or qo.MOST[kind] * s / 2 < c * a)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_rule_of_the_exponent(kind):
    """The kernels take a scale's exponent from the bits of the largest element, with a limit for its fraction."""
    for rotated, base, limit in ((False, {"e4m3": 8, "int8": 6}[kind], {"e4m3": 96, "int8": 126}[kind]),
                                 (True, {"e4m3": 8, "int8": 6}[kind], {"e4m3": 30, "int8": 51}[kind])):
        for m in range(0, 0x7f80, 3):
            a = float(torch.tensor(m, dtype=torch.int16).view(torch.bfloat16))
            e = max((m >> 7) - base + ((m & 127) > limit), 1)
            assert 2.0 ** (e - 127) == qo.needed_scale(a, kind, rotated), (m, rotated)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_a_scale_that_grows_keeps_old_values(kind):
    """e4m3 codes move exactly between powers of two (but for subnormal ones); int8 errors stay below a step."""
    r = np.random.RandomState(1)
    y = r.randn(1000) * 0.5
    s = qo.needed_scale(np.abs(y).max(), kind, False)
    c = qo.nearest(y / s, kind)
    for grow in range(1, 6):
        c = qo.nearest(c / 2, kind)
        s *= 2
        if kind == "int8":
            assert np.abs(c * s - y).max() < s
        else:
            assert np.all(np.abs(c * s - y) <= 2.0 ** -4 * np.abs(y) + 2.0 ** -9 * s)


def small(kind="e4m3", seed=0):
    r = np.random.RandomState(seed)
    P, G, page, d, block = 6, 2, 32, 64, 16
    codes = [qo.nearest(r.randn(P, G, page, d) * 40, kind) for _ in range(2)]
    scales = [np.exp(0.3 * r.randn(P, G, page // block)) * 0.02 for _ in range(2)]
    table = np.array([[0, 3, 5], [4, 1, 2]])
    return r.randn(2, 4, d), *codes, *scales, table, np.array([70, 33])


@pytest.mark.parametrize("window,sinks", [(1 << 30, 0), (20, 3)])
def test_attention_is_a_softmax(window, sinks):
    q, kc, vc, ks, vs, table, lengths = small()
    got = qo.attention(q, kc, vc, ks, vs, table, lengths, window, sinks, 0.125)
    wide = [np.repeat(s, 16, axis=2)[..., None] for s in (ks, vs)]
    # the bf16 cache's reference on the values the codes stand for
    ref = wo.cache_attention(q, kc * wide[0], vc * wide[1], table, lengths, window, sinks, 0.125)
    for n in ("out", "lse"):
        assert np.allclose(got[n][0], ref[n][0], rtol=1e-12, atol=1e-12)
        assert np.all(got[n][1] > 0)


@pytest.mark.parametrize("mistake", ["scale of the next block", "scales exchanged", "window off by one", "no scale"])
def test_mistakes_are_caught(mistake):
    q, kc, vc, ks, vs, table, lengths = small()
    args = [q, kc, vc, ks, vs, table, lengths, 20, 3, 0.125]
    ref = qo.attention(*args)
    if mistake == "scale of the next block":
        args[3] = np.roll(ks, 1, axis=2)
    elif mistake == "scales exchanged":
        args[3], args[4] = vs, ks
    elif mistake == "window off by one":
        args[7] = 21
    else:
        args[4] = np.full_like(vs, 0.02)
    got = qo.attention(*args)
    assert np.any(np.abs(got["out"][0] - ref["out"][0]) > ref["out"][1])


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_by_hand(kind):
    """Two tokens behind one cached: the block's scale doubles and the cached code halves."""
    codes, scales = np.zeros((2, 1, 16, 64)), np.full((2, 1, 1), 2.0 ** -3)
    codes[1, 0, 0] = 5.0
    x = np.zeros((2, 1, 64))
    x[0, 0, 0], x[1, 0, 5] = qo.MOST[kind] * 2.0 ** -2, -3.0
    lo, hi, s = qo.append(codes, scales, np.array([[1]]), [1], [2], x, kind)
    assert s[1, 0, 0] == 2.0 ** -2 and s[0, 0, 0] == 2.0 ** -3 and np.array_equal(lo, hi)
    assert np.all(lo[1, 0, 0] == (2.5 if kind == "e4m3" else 2.0))  # 2.5: a tie for int8, to the even 2
    assert lo[1, 0, 1, 0] == qo.MOST[kind] and lo[1, 0, 2, 5] == -12.0
    assert np.all(lo[0] == 0) and np.all(lo[1, 0, 3:] == 0)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_append_not_finite_by_hand(kind, value):
    """A value that is not finite makes its block's scale NaN, behind earlier tokens too; so does an earlier scale."""
    codes, scales = np.full((2, 2, 16, 64), 5.0), np.full((2, 2, 1), 2.0 ** -3)
    x = np.ones((2, 2, 64))
    x[1, 0, 7] = value
    lo, hi, s = qo.append(codes, scales, np.array([[1]]), [3], [2], x, kind)
    assert np.isnan(s[1, 0, 0]) and s[1, 1, 0] == 2.0 ** -3 and np.all(s[0] == 2.0 ** -3)
    assert np.all(np.isneginf(lo[1, 0, 3:5])) and np.all(np.isposinf(hi[1, 0, 3:5])) and np.all(lo[1, 0, :3] == 5.0)
    assert np.all(lo[1, 1, 3:5] == 8.0) and np.array_equal(lo[1, 1], hi[1, 1])
    lo, hi, s = qo.append(codes, s, np.array([[1]]), [5], [1], np.ones((1, 2, 64)), kind)
    assert np.isnan(s[1, 0, 0]) and s[1, 1, 0] == 2.0 ** -3
    lo, hi, s = qo.append(codes, s, np.array([[1]]), [0], [1], np.ones((1, 2, 64)), kind)
    assert s[1, 0, 0] == s[1, 1, 0] == qo.needed_scale(1.0, kind, False) and np.array_equal(lo, hi)


def test_append_behind_the_lowest_int8_code():
    """-128 stays where its scale does, and becomes the nearest code where that changes: 127 by a factor of -1."""
    for old, want in ((2.0 ** -5, -128), (-2.0 ** -5, 127), (-2.0 ** -6, 64), (2.0 ** -6, -64), (0.996 * 2.0 ** -5, -127),
                      (0.999 * 2.0 ** -5, -128), (-0.999 * 2.0 ** -5, 127)):
        codes, scales = np.full((1, 1, 16, 64), -128.0), np.full((1, 1, 1), old)
        lo, hi, s = qo.append(codes, scales, np.array([[0]]), [3], [1], np.full((1, 1, 64), 3.0), "int8")
        assert s[0, 0, 0] == 2.0 ** -5 and np.all(lo[0, 0, :3] == want) and np.array_equal(lo, hi)


def test_pages_by_hand():
    table = np.full((3, 4), -1)
    table[0, :2], table[2, 0] = [7, 8], 9
    free = np.array([0, 1, 2, 3, 4, 5, 6, -1, -1, -1])
    t, slots, n = qo.reserve(table, [20, 0, 16], [0, 13, 14, 15], 17, free, 7, 16)
    # sequence 0 goes to 33 tokens (a third page), 1 takes its first, 2's one page is full
    assert n == 4 and t[0].tolist() == [7, 8, 6, -1] and t[1, 0] == 5 and t[2].tolist() == [9, 4, -1, -1]
    assert slots.tolist() == [8 * 16 + i for i in range(4, 16)] + [6 * 16] + [5 * 16] + [4 * 16] + [-1, -1]
    f, n = qo.release(t, [33, 1, 17], [16, 0, 17], free, 4, 16)
    assert n == 7 and f[:7].tolist() == [0, 1, 2, 3, 8, 6, 5]
