"""Waits of whole warps in the kernels' sources: what all lanes of a warp wait for goes through the
form with one answer (a lane that gave up while the others go on would leave them alone in front of
shuffles, matrix loads and products, and TMEM accesses, which need all 32 lanes)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "streaming_kv_cache_duo_gb300",
                    "csrc")


def _lines(name, pattern):
    with open(os.path.join(CSRC, name)) as f:
        return [line.strip() for line in f if re.search(pattern, line)]


@pytest.mark.parametrize("name,barriers", [
    ("decode_kv8.cu", r"bars\[b\]"),              # a slice's copies
    ("prefill.cu", r"s_full\[x\]|o_final\[x\]"),  # scores and outputs, by the softmax warps
])
def test_waits_of_whole_warps_have_one_answer(name, barriers):
    waits = _lines(name, r"mbar_wait\w*\(&?[\w>-]*(" + barriers + ")")
    assert waits
    for line in waits:
        assert "mbar_wait_warp(" in line, line


def test_bf16_decode_warps_wait_together():
    """Its slices (wfull[s]) and the warps' meeting point (bar); lane 0 alone collects what is left."""
    waits = _lines("decode.cu", r"mbar_wait\w*\((&wfull\[s\]|bar,)")
    assert len(waits) == 2 and all("mbar_wait_warp(" in line for line in waits), waits
