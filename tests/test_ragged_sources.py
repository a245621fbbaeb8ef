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
    for line in _text("attn_ragged.cu").splitlines():
        if re.search(r"wait\w*\(&?bars->(s_full|o_final|p_full|pair_ml|pair_done|v_full)", line):
            assert "wait_warp(" in line or "ready(" in line or "mbar_wait(&bars->k_full" in line or "wait_for(&bars->v_full" in line, line
