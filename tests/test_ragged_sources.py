"""What the packed kernels' sources promise: arrays that the grid before may still write are read by plain
loads (after its end), and what all lanes of a warp wait for has one answer for all of them."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "streaming_kv_cache_duo_gb300",
                    "csrc")


def _text(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", ["attn_ragged.cu", "append_ragged.cu"])
def test_nothing_is_read_as_constant(name):
    text = _text(name)
    assert "griddepcontrol.wait" in text and "__ldg(" not in text


def test_softmax_and_mma_warps_wait_together():
    """Barriers that only whole warps wait for: one answer for all lanes (single looks are voted on)."""
    text = _text("attn_ragged.cu")
    waits = [line.strip() for line in text.splitlines()
             if re.search(r"wait\w*\(&?bars->(s_full|o_final|p_full|pair_ml|pair_done)", line)]
    looks = [line for line in waits if "mbar_try_wait(" in line]
    assert waits and all("wait_warp(" in line or line in looks for line in waits), waits
    assert re.search(r"__all_sync\(0xffffffffu, v && k && p0\)", text) and len(looks) == 1
