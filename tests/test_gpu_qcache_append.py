"""Appends to the 8-bit cache that need more than a few blocks or more than one call, against float64."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
import oracle.qcache_oracle as qo
import oracle.window_oracle as wo
from test_gpu_qcache import DEV, KINDS, check_append, filled, gen, int32, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,longest,past,G,H,d,block,rot", [
    (1500, 150, 60, 1, 1, 64, 64, 64), (1500, 150, 60, 2, 1, 64, 64, 0), (1250, 70, 30, 2, 1, 128, 32, 128),
    (1400, 70, 30, 2, 1, 128, 32, 0), (1400, 200, 100, 1, 2, 64, 128, 64)])
def test_append_several_blocks_to_a_cta(kind, B, longest, past, G, H, d, block, rot):
    """A CTA's blocks have different numbers of new rows, and its warps share them in other teams each time: every team
    agrees on a scale.  (Rows differ in size by much, so that a neighbour's largest element would give another scale.)"""
    r = np.random.RandomState(B)
    new = [int(x) for x in r.randint(1, longest + 1, B)]
    lens = [int(x) for x in r.randint(0, past + 1, B)]
    ctas = (3 if d == 64 else 2) * torch.cuda.get_device_properties(DEV).multi_processor_count
    assert sum(new) // block + 2 * B >= 2 * 4 * ctas  # then a CTA takes two blocks' numbers or more
    amplitude = torch.empty(sum(new), 1, 1, device=DEV).normal_(0.0, 3.0, generator=gen(31)).exp_().to(torch.bfloat16)
    check_append(lens, new, G, H, d, 128, block, kind, rot, amplitude=amplitude)


def check_scales_and_codes(kind, codes, scales, before, table, lens, new, x, freq):
    """Scales equal to the reference's, NaN where that is; codes within its bounds where the scale is a number."""
    lo, hi, s = qo.append(before[0], before[1], table, lens, new, wo.f64(x), kind, freq)
    assert np.array_equal(wo.f64(scales), s, equal_nan=True)
    known = ~np.isnan(np.repeat(s, codes.shape[2] // s.shape[2], axis=2))
    c, lo, hi = qo.decode(codes, kind)[known], lo[known], hi[known]
    assert np.all(np.isnan(c) & np.isnan(lo) | (c >= lo) & (c <= hi))  # (rows that hold no token are NaN)
    return s


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("page,block,lens,new,bad", [
    (16, 16, [5, 20], [1, 1], 0),          # one token each, the first sequence's is bad
    (32, 32, [1, 40], [3, 1], 2),          # the last of three
    (128, 128, [5, 130], [100, 2], 0),     # a block whose rows several warps share: a row of the first warp's,
    (128, 128, [5, 130], [100, 2], 99)])   # one of the last's
def test_append_not_finite_behind_earlier_tokens(kind, value, rot, page, block, lens, new, bad):
    """The scale of the block and head becomes NaN although earlier tokens had one, and stays so; others do not."""
    G, d = 2, 64
    g = gen(32)
    total = [a + n for a, n in zip(lens, new)]
    kc, vc, ks, vs, table, _ = filled(g, [n + 1 for n in total], G, d, page, block, kind)
    for s in (ks, vs):
        s.copy_(torch.pow(2.0, torch.randint(-8, -3, s.shape, generator=g, device=DEV).float()))
    before = [(qo.decode(c, kind), wo.f64(s)) for c, s in ((kc, ks), (vc, vs))]
    k, v = normal(g, sum(new), G, d), normal(g, sum(new), G, d)
    k[bad, 1, 5] = value
    v[bad, 0, 60] = value
    f = jfa.rotary_frequencies(rot) if rot else None
    ff = f.numpy() if rot else ()
    ws = jfa.new_cache_workspace(2, 2, G, d, DEV)

    def append(lens, k, v):
        off = torch.tensor(np.concatenate([[0], np.cumsum([n for _, n in lens])]), device=DEV)
        jfa.jfa_qcache_append(k, v, off, kc, vc, ks, vs, table, int32([a for a, _ in lens]), frequencies=f, workspace=ws)
        assert jfa.jfa_check_status(ws) == 0

    append(list(zip(lens, new)), k, v)
    sk = check_scales_and_codes(kind, kc, ks, before[0], table, lens, new, k, ff)
    sv = check_scales_and_codes(kind, vc, vs, before[1], table, lens, new, v, ())
    at = int(table[0, (lens[0] + bad) // page]), (lens[0] + bad) % page // block
    assert np.argwhere(np.isnan(sk)).tolist() == [[at[0], 1, at[1]]]
    assert np.argwhere(np.isnan(sv)).tolist() == [[at[0], 0, at[1]]]
    q = normal(g, 2, G, d)
    out, lse, _ = jfa.jfa_qcache_attention(q, kc, vc, ks, vs, table, int32(total), workspace=ws)
    assert torch.isnan(lse).tolist() == [[False, False], [True, False]]
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isfinite(out[1]).all())
    append([(n, 1) for n in total], normal(g, 2, G, d), normal(g, 2, G, d))  # finite values behind it, in the same block
    assert bool(torch.isnan(ks[at[0], 1, at[1]])) and bool(torch.isnan(vs[at[0], 0, at[1]]))
    assert int(torch.isnan(ks).sum()) == int(torch.isnan(vs).sum()) == 1
    assert jfa.jfa_check_status(ws) == 0


@pytest.mark.parametrize("old", [-2.0 ** -5, 2.0 ** -5, -2.0 ** -6, -0.999 * 2.0 ** -5, 0.999 * 2.0 ** -5])
def test_append_behind_the_lowest_int8_code(old):
    """Earlier codes of -128, of another origin, become the nearest ones at a scale that is exactly minus theirs, or next
    to it.  (The new rows need 2^-5: their largest element lies between 127 / 64 and 127 / 32.)"""
    start = filled(gen(33), [40, 40], 2, 64, 32, 32, "int8")
    for codes, scales in (start[:1] + start[2:3], start[1:2] + start[3:4]):
        codes[:, :, ::2] = -128
        scales.fill_(old)
    check_append([5, 37], [3, 2], 2, 1, 64, 32, 32, "int8", 0, start=start)
    first, second = start[4][0, 0].long(), start[4][1, 1].long()
    for codes, scales in (start[:1] + start[2:3], start[1:2] + start[3:4]):
        assert bool((scales[first] == 2.0 ** -5).all()) and bool((scales[second] == 2.0 ** -5).all())
        assert bool((codes[first, :, 0:5:2] == {-2.0 ** -5: 127, -2.0 ** -6: 64, -0.999 * 2.0 ** -5: 127}.get(old, -128)).all())
