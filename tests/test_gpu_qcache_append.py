"""Appends to the 8-bit cache that need more than a few blocks or more than one call, against float64."""
import numpy as np
import pytest
import torch

from test_gpu_qcache import DEV, KINDS, check_append, gen

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
