"""What DuoRope.rotate refuses before it calls the library (CPU: no device is asked for)."""

import pytest
import torch


@pytest.fixture
def rope(monkeypatch):
    import streaming_kv_cache_duo_gb300 as duo
    monkeypatch.setattr(duo._lib, "_current_device", lambda: -1)
    monkeypatch.setattr(duo._lib, "duo_rope_rotate", lambda *a: None)
    x = duo.DuoRope.__new__(duo.DuoRope)
    x.head_dim, x.index, x.bf16, x.int32, x.empty_like, x.c = 64, -1, torch.bfloat16, torch.int32, torch.empty_like, None
    return x


def test_an_output_for_keys_without_keys(rope):
    """It came back unwritten, as if it held rotated keys."""
    q, pos = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_out"):
        rope.rotate(q, None, pos, k_out=torch.zeros_like(q))
    assert rope.rotate(q, None, pos)[1] is None
    out = torch.zeros_like(q)
    assert rope.rotate(q, q, pos, k_out=out)[1] is out
