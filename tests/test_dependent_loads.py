"""Kernels launched as programmatic dependents live while the grid before them still writes. What that
grid writes (lengths and block tables, ring positions, the factors of an expanded cache) is read by plain
loads after the wait, not through the read-only path (__ldg), which may be served from before it."""

import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "streaming_kv_cache_duo_gb300",
                    "csrc")


@pytest.mark.parametrize("name,arrays", [
    ("decode_kv8.cu", ("seq_lens", "pages", "p.pos")),
    ("decode.cu", ("seq_lens", "p.pos")),
    ("prefill.cu", ("k_fac", "v_fac")),
    ("append_kv8.cu", ("cu_new", "token_seq", "token_pos", "slots", "pg.table", "tail")),
    ("block_tables.cu", ("",)),
])
def test_what_the_grid_before_writes_is_not_read_as_constant(name, arrays):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert "griddepcontrol.wait" in text
    for line in text.splitlines():
        if "__ldg(" in line:
            argument = line.split("__ldg(", 1)[1]
            assert not any(a in argument for a in arrays), line.strip()
