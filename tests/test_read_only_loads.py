"""Which data the kernels read through the read-only path (CPU, from the source).

A kernel of the library may become resident while the one in front of it still runs (programmatic
launch).  The read-only path is for data that nothing writes while a grid lives, so it must not be used
for what the kernel directly in front may write.  The kernel before that one has finished by then: a
kernel lets its successor start only behind its own wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "jagged_attention_recsys_jfa_gb300", "csrc")

# what may be read so, by file: arrays that only callers write, and what comes from a kernel at least two in front
ALLOWED = {
    "jfa_cache.cu": {"p.offsets", "offsets", "p.page_table", "table"},
    "jfa_fwd.cu": set(),
    # dout, out and lse: from callers, or the forward, behind which the planner runs; brow: the bias table, from
    # the planner, behind which the preprocess runs; lse2, delta: from the preprocess, read by the dQ pass behind dK/dV
    "jfa_bwd.cu": {"p.dout", "p.out", "drow", "orow", "p.lse", "p.q_off", "brow", "p.lse2", "p.delta"},
    "jfa_win.cu": set(),
    "jfa_win_bwd.cu": {"p.lse2", "p.delta", "part", "pv"},  # part, pv: from dK/dV, read by the join behind dQ
    "jfa_win_dkdv.cu": set(),
    "jfa_win_dq.cu": {"p.lse2", "p.delta"},
    "jfa_plan.cu": set(),
    "jfa_win_plan.cu": set(),
}


def read_only_loads(text):
    """The array of each __ldg: its argument without casts and index arithmetic."""
    for m in re.finditer(r"__ldg\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        arg = re.sub(r"reinterpret_cast<[^>]*>\(", "", text[m.end():at - 1])
        yield re.match(r"[\w.]+", arg).group(0)


@pytest.mark.parametrize("name", sorted(ALLOWED))
def test_read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        found = set(read_only_loads(f.read()))
    assert found <= ALLOWED[name], found - ALLOWED[name]
