"""The block table that a paged 8-bit layer takes: on the layer's own device, its kernels read it."""

import pytest
import torch

import streaming_kv_cache_duo_gb300 as duo


class Table:
    """Looks like a CUDA tensor on device `index`."""

    def __init__(self, shape=(2, 3, 4), dtype=torch.int32, index=0, contiguous=True, is_cuda=True):
        self.shape, self.dtype, self.index, self.contiguous, self.is_cuda = shape, dtype, index, contiguous, is_cuda
        self.device = f"cuda:{index}"

    def is_contiguous(self):
        return self.contiguous

    def get_device(self):
        return self.index


def test_a_table_on_the_layers_device_is_taken():
    duo._check_table(Table(index=0), (2, 3, 4), 0)
    duo._check_table(Table(index=1), (2, 3, 4), 1)


@pytest.mark.parametrize("bad", [dict(index=1), dict(shape=(2, 3, 5)), dict(dtype=torch.int64), dict(contiguous=False),
                                 dict(is_cuda=False)])
def test_other_tables_are_refused(bad):
    with pytest.raises(ValueError, match="block_table"):
        duo._check_table(Table(**bad), (2, 3, 4), 0)


@pytest.mark.gpu
def test_a_paged_layer_checks_its_table(monkeypatch):
    table = torch.zeros((1, 1, 2), dtype=torch.int32, device="cuda")
    make = lambda t: duo.DuoKv8PagedLayer(1, 2, 2, 64, 4, 32, 128, 2, 4, t, [1, 0])
    make(table)
    for bad in (table.long(), table.cpu(), table[:, :, :1].contiguous(), torch.zeros((1, 1, 4), device="cuda").int()[:, :, ::2]):
        with pytest.raises(ValueError, match="block_table"):
            make(bad)
    seen = []
    monkeypatch.setattr(duo, "_check_table", lambda t, shape, index: seen.append((t, tuple(shape), index)))
    layer = make(table)
    assert len(seen) == 1 and seen[0][0] is table and seen[0][1:] == ((1, 1, 2), layer.index)
