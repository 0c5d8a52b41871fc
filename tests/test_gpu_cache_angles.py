"""The rotation's angles where they show: next to a multiple of a quarter turn a sine or cosine is
small, so that its bf16 value still carries the angle's last bits."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
getcontext().prec = 80
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def turned(position, frequency):
    """cos and sin of position * frequency, the product and its remainder in 80 digits."""
    turns = Decimal(position) * Decimal(frequency) / TWO_PI
    quarters = int((turns * 4).to_integral_value())
    r = float((turns - Decimal(quarters) / 4) * TWO_PI)
    c, s = math.cos(r), math.sin(r)
    return [(c, s), (-s, c), (-c, -s), (s, -c)][quarters % 4]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("position", [1, 7, 1000, 123457, 10 ** 6 + 3, (1 << 30) + 12345])
def test_angles_next_to_quarter_turns(position, interleaved):
    """Bound: half a bf16 step and 2^-21 for fp32, relative to the value, and 2^-32 of a turn.  The
    frequencies are near quarter turns of the position, from both sides, and the usual ones."""
    d, page = 64, 128
    f = []
    for i in range(32):
        quarters = [1, 2, 3, 4, 6, 9, 17, 1003][i % 8]
        off = (1e-7, -1e-6, 3e-5, -1e-3)[i // 8]
        f.append((quarters * math.pi / 2 + off) / position)
    kc = torch.zeros(1, 1, page, d, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(1, position // page + 2, dtype=torch.int32, device=DEV)
    for freq in (f, jfa.rotary_frequencies(d).tolist(), [-x for x in f], [x + 2 * math.pi * 5 for x in f]):
        k = torch.zeros(1, 1, d, dtype=torch.bfloat16, device=DEV)
        first = slice(0, d, 2) if interleaved else slice(0, d // 2)
        second = slice(1, d, 2) if interleaved else slice(d // 2, d)
        k[..., first] = 1.0
        out = torch.empty_like(k)
        _, _, _, ws = jfa.jfa_cache_append(k, k, torch.tensor([0, 1], device=DEV), kc, kc.clone(), table,
                                           torch.tensor([position], dtype=torch.int32, device=DEV), interleaved=interleaved,
                                           frequencies=torch.tensor(freq, dtype=torch.float64), k_out=out)
        assert jfa.jfa_check_status(ws) == 0
        got = list(zip(out[0, 0, first].tolist(), out[0, 0, second].tolist()))
        for i, x in enumerate(freq):
            for a, ref in zip(got[i], turned(position, x)):
                assert abs(a - ref) <= (2.0 ** -8 + 2.0 ** -21) * abs(ref) + 2 * math.pi * 2.0 ** -32, (i, x, a, ref)
