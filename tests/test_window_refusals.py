"""The windowed calls refuse bad arguments on the host, before any device work (CPU)."""
import pytest

import jagged_attention_recsys_jfa_gb300 as jfa

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def forward(**over):
    a = dict(q=16, k=32, v=48, qo=64, ko=64, B=2, H=4, G=4, d=64, tq=10, tk=10, window=4, sinks=1, scale=0.125, out=80,
             lse=96, ws=None, wsb=0)
    a.update(over)
    return jfa.load_library().jfa_window_forward(*a.values(), None)


def backward(**over):
    a = dict(dout=112, q=16, k=32, v=48, out=80, lse=96, qo=64, ko=64, B=2, H=4, G=4, d=64, tq=10, tk=10, window=4, sinks=1,
             scale=0.125, dq=128, dk=144, dv=160, ws=None, wsb=0)
    a.update(over)
    return jfa.load_library().jfa_window_backward(*a.values(), None)


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("over,status", [
    (dict(), WORKSPACE),  # everything else is right
    (dict(G=3), INVALID), (dict(G=0), INVALID), (dict(window=0), INVALID), (dict(sinks=-1), INVALID),
    (dict(sinks=129), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(k=40), INVALID), (dict(q=None), INVALID),
    (dict(scale=0.0), INVALID), (dict(qo=None), INVALID),
])
def test_arguments(call, over, status):
    assert call(**over) == status


ROOM = dict(ws=256, wsb=1 << 30)  # these are looked at last


@pytest.mark.parametrize("over", [dict(out=32), dict(out=48)])
def test_forward_outputs_in_the_place_of_keys(over):
    assert forward(**over, **ROOM) == INVALID


@pytest.mark.parametrize("over", [dict(dk=32), dict(dk=48), dict(dv=32), dict(dv=48), dict(dk=160), dict(dk=16), dict(dv=16),
                                  dict(dk=112), dict(dv=112), dict(dq=32), dict(dq=48), dict(dq=144), dict(dq=160)])
def test_backward_outputs_in_the_place_of_inputs(over):
    assert backward(**over, **ROOM) == INVALID
