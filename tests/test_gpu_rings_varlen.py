"""Single tokens over rings alone in a paged layer, with lengths on the device: short rings give what the kernel of
contiguous caches gives, bit for bit, and rings on either side of the limits are right."""

import numpy as np
import pytest
import torch

from test_gpu_attn_ragged import Batch, _decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D,S,R,lens", [
    (8, 2, 128, 4, 32, [300, 1, 0, 35, 36, 37]), (4, 4, 64, 64, 256, [320, 700, 5, 0]), (16, 2, 64, 0, 640, [2000, 640, 641]),
    (8, 1, 128, 24, 1000, [1500, 1023]),
])
def test_short_rings_keep_their_kernel(Hq, Hkv, D, S, R, lens):
    from streaming_kv_cache_duo_gb300 import duo_attn_decode_varlen, duo_device_error
    x = Batch(51, [(max(n - 1, 0), min(n, 1)) for n in lens], Hq, Hkv, 0, D, S, R, 128, appended=True)
    q = torch.randn(len(lens), Hq, D, device="cuda").to(torch.bfloat16)
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref = torch.empty_like(q)
    for most in (max(lens), max(max(lens) - 1, 1), 2 ** 31 - 1):
        duo_attn_decode_varlen(x.layer.handle, x.layer.cache, L, most, q, ref, x.layer.workspace)
        assert torch.equal(x.layer.decode_varlen(q, L, most), ref)
    assert duo_device_error() == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 8, 2)])
@pytest.mark.parametrize("rows", [640, 641, 1024, 1025])
def test_rings_on_either_side_of_the_limits(D, Hq, Hkv, rows):
    rng = np.random.default_rng(rows)
    lens = [rows + 300, rows, rows - 1, 1, 0] + [int(n) for n in rng.integers(1, 2 * rows, 3)]
    _decode(Batch(52, [(max(n - 1, 0), min(n, 1)) for n in lens], Hq, Hkv, 0, D, 4, rows - 4, 128, appended=True))


def test_rings_of_many_sequences():
    rng = np.random.default_rng(9)
    lens = [0] + [int(n) for n in rng.integers(0, 1500, 318)] + [1400]
    for rows in (100, 700):
        _decode(Batch(53, [(max(n - 1, 0), min(n, 1)) for n in lens], 2, 1, 0, 64, 4, rows - 4, 128, appended=True), most=30)
