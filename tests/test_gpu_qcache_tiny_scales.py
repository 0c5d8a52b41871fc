"""The attention over an 8-bit cache whose values are next to the smallest that a scale can hold."""
import numpy as np
import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
from test_gpu_qcache import DEV, KINDS, filled, gen, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", [1, 12, 24])  # to a key: a kernel each
@pytest.mark.parametrize("scale", [2.0 ** -126, 1.7 * 2.0 ** -125])
def test_smallest_value_scales_over_long_sequences(kind, heads, scale):
    """Every value is the largest code by one scale, so that the output is that value, whatever the weights are; a CTA
    adds up dozens of tiles.  Off by half an f16 step of each weight, fp32 sums, and half a bf16 step of the output."""
    G, d = 8, 64
    lens = [int(x) for x in np.random.RandomState(4).randint(3000, 4500, 48)]
    g = gen(34)
    kc, vc, ks, vs, table, n = filled(g, lens, G, d, 128, 64, kind)
    most = 448.0 if kind == "e4m3" else 127.0
    vc.copy_(torch.full_like(vs[0, 0, :1], most).to(vc.dtype).expand_as(vc))
    vs.fill_(scale)
    ks.copy_(ks.nan_to_num(0.0) * 0.1)  # scores of a few units: no key outweighs the others
    out, lse, ws = jfa.jfa_qcache_attention(normal(g, len(lens), heads * G, d), kc, vc, ks, vs, table, n)
    assert jfa.jfa_check_status(ws) == 0 and bool(torch.isfinite(lse).all())
    want = most * float(torch.tensor(scale, dtype=torch.float32))
    assert float((out.double() / want - 1).abs().max()) <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18
