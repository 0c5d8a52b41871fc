"""The paged cache's calls refuse bad arguments on the host, before any device work (CPU)."""
import ctypes
import math

import pytest
import torch

import jagged_attention_recsys_jfa_gb300 as jfa
from jagged_attention_recsys_jfa_gb300.jfa import _Cache

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def cache(**over):
    a = dict(k=4096, v=8192, num_pages=8, H_kv=2, page_size=16, d=64, page_table=64, max_pages=4, lengths=128, B=3)
    a.update(over)
    return _Cache(*(a[n] for n, _ in _Cache._fields_))


def append(c=None, freq=(1.0,) * 32, **over):
    a = dict(k=16, ks=128, v=32, vs=128, q=None, qs=0, H=0, off=64, total=5, rot=2 * len(freq), il=0, q_out=None,
             k_out=None, lengths_out=None, ws=256, wsb=1 << 20)
    a.update(over)
    f = (ctypes.c_double * max(len(freq), 1))(*freq) if freq is not None else None
    return jfa.load_library().jfa_cache_append(
        ctypes.byref(c or cache()), a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["H"], a["off"], a["total"],
        ctypes.cast(f, ctypes.c_void_p) if a.get("freq", 1) else None, a["rot"], a["il"], a["q_out"], a["k_out"],
        a["lengths_out"], a["ws"], a["wsb"], None)


def attend(c=None, **over):
    a = dict(q=16, H=4, window=8, sinks=0, scale=0.125, out=16, lse=16, ws=256, wsb=1 << 30)
    a.update(over)
    return jfa.load_library().jfa_cache_attention(ctypes.byref(c or cache()), a["q"], a["H"], a["window"], a["sinks"],
                                                  a["scale"], a["out"], a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("over,status", [
    (dict(B=0), INVALID), (dict(H_kv=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(v=8200), INVALID), (dict(page_table=None), INVALID), (dict(page_table=66), INVALID),
    (dict(lengths=None), INVALID), (dict(lengths=130), INVALID),
    (dict(num_pages=1 << 27), INVALID),   # 2^27 pages x 2 heads x 16 rows: row numbers past 31 bits
    (dict(num_pages=1 << 62), INVALID), (dict(max_pages=1 << 27), INVALID), (dict(max_pages=(1 << 27) - 7), INVALID),
])
def test_cache_is_checked(call, over, status):
    assert call(cache(**over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(k=None), INVALID), (dict(k=24), INVALID), (dict(v=None), INVALID), (dict(off=None), INVALID),
    (dict(off=68), INVALID), (dict(total=-1), INVALID), (dict(total=1 << 31), INVALID), (dict(ks=120), INVALID),
    (dict(ks=132), INVALID), (dict(vs=64), INVALID), (dict(lengths_out=6), INVALID), (dict(k_out=8), INVALID),
    (dict(q=16, qs=256, H=4), INVALID),               # no q_out
    (dict(q=16, qs=128, H=4, q_out=16), INVALID),     # q rows overlap
    (dict(q=16, qs=264, H=4, q_out=16), INVALID),     # in place, but strided
    (dict(k_out=16, ks=136), INVALID),
    (dict(k_out=32), INVALID),                        # k_out is v
    (dict(q=48, qs=256, H=4, q_out=16), INVALID), (dict(q=48, qs=256, H=4, q_out=32), INVALID),
    (dict(q=48, qs=256, H=4, q_out=64, k_out=64), INVALID), (dict(q=48, qs=256, H=4, q_out=64, k_out=48), INVALID),
    (dict(rot=66), INVALID), (dict(rot=-16), INVALID), (dict(rot=24), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=128), WORKSPACE), (dict(wsb=255), WORKSPACE),
])
def test_append_is_checked(over, status):
    assert append(**over) == status


def test_append_frequencies_are_finite():
    assert append(freq=(1.0,) * 31 + (math.inf,)) == INVALID
    assert append(freq=(math.nan,) * 8) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(H=3), INVALID), (dict(H=1), INVALID), (dict(window=0), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(q=None), INVALID),
    (dict(q=24), INVALID), (dict(out=None), INVALID), (dict(lse=20), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=64), WORKSPACE), (dict(wsb=1000), WORKSPACE),
])
def test_attention_is_checked(over, status):
    assert attend(**over) == status


def test_workspace_size():
    f = jfa.cache_workspace_size
    assert f(0, 4, 2, 64) == 0 and f(2, 3, 2, 64) == 0 and f(2, 4, 2, 80) == 0 and f(2, 1, 2, 64) == 0
    assert f(2, 4, 2, 64) > 256 and f(2, 4, 2, 64) % 256 == 0
    assert f(100000, 64, 2, 128) > f(2, 64, 2, 128)
    # calls of different sizes share a workspace, so only the number of units makes it larger
    assert f(7, 16, 4, 64) == f(7, 4, 4, 128)
    with pytest.raises(ValueError):
        jfa.new_cache_workspace(2, 3, 2, 64, "cpu")


def test_cpu_tensors_are_refused():
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, n = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        jfa.jfa_cache_attention(x, kc, kc, table, n)
    with pytest.raises(ValueError, match="CUDA"):
        jfa.jfa_cache_append(x, x, torch.zeros(4, dtype=torch.int64), kc, kc, table, n)


def test_rotary_frequencies():
    f = jfa.rotary_frequencies(64, 1000.0)
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1.0
    assert abs(float(f[16]) - 1000.0 ** -0.5) < 1e-15
