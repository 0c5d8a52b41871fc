"""The limits of the waits that last a whole item (CPU): large enough for the longest item that the
accepted sizes allow, and used where a role waits that long."""
import os
import re

import pytest

import jagged_attention_recsys_jfa_gb300 as jfa

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "jagged_attention_recsys_jfa_gb300", "csrc")

# barriers that a role meets only at an item's ends
ITEM_LONG = {
    "jfa_fwd.cu": {"q_empty": 1},
    "jfa_bwd.cu": {"kv_empty": 2, "dv_full": 3, "dk_full": 3, "qdo_empty": 1, "acc_full": 1, "q_empty": 1, "dq_full": 2},
    "jfa_win_bwd.cu": {"kv_empty": 1, "dv_full": 2, "dk_full": 2, "qdo_empty": 1, "acc_full": 1},
    "jfa_win_dkdv.cu": {"kv_empty": 1},
}


@pytest.mark.parametrize("name", sorted(ITEM_LONG))
def test_item_long_waits_take_the_planned_limit(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    for barrier, count in ITEM_LONG[name].items():
        limits = re.findall(r"mbar_wait\(&" + barrier + r", [^;{]*?abort_flag, ([^)]*)\)", text)
        assert limits == ["meta.wait_ns, kWaitTimeoutNs"] * count, (barrier, limits)


@pytest.mark.parametrize("group,queries,window", [(64, 2 << 20, None), (4096, 40000, None), (1, 1 << 28, None),
                                                  (4096, 1 << 18, 1 << 16), (8, 4096, 512)])
def test_limit_covers_the_longest_item(group, queries, window):
    """Ten times the 3.2 us that the slowest pass takes for a pair of 128-row tiles."""
    tiles = -(-queries // 128)
    if window is not None:
        tiles = min(tiles, window // 128 + 2)
    pairs = group * tiles  # of a key tile that every one of these query tiles sees
    limit = int(jfa.load_library().jfa_wait_limit_ns(pairs, 152, pairs))
    assert limit >= 2_000_000_000 + min(pairs * 32_000, 3_600_000_000_000) >= 10 * min(pairs * 3_200, 360_000_000_000)
