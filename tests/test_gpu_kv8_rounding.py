"""How much of a decode's error over bf16 rows (rings, tails) is its own. The outputs are rounded to bf16,
which alone puts them e0 = |bf16(o) - o| from the outputs o in 64 bits (by norm). What the kernel adds is
in fp32 and p in two bf16 terms, 2^-17: over a sum of p |v| of some ten times |o| here less than 2^-13 of
it, against e0 of about 2^-9, so in squares less than a hundredth. p rounded to one bf16 term would add
as much as e0 again, since both roundings are alike: a factor of sqrt 2."""

import numpy as np
import pytest
import torch

from kv8_util import Batch, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,S,R,kinds,n,code", [
    (128, 64, 256, [0, 0], 1000, "int8"), (64, 4, 100, [0, 0], 600, "e4m3"), (128, 4, 32, [1, 1], 63, "int8"),
    (64, 4, 700, [0, 0], 2000, "int8"), (64, 4, 32, [1, 1], 47, "e4m3"),
])
def test_the_error_is_the_outputs_rounding(D, S, R, kinds, n, code):
    from streaming_kv_cache_duo_gb300 import DuoKv8Layer
    B = 8
    c = Batch(95, [n] * B, 16, 2, D, S, R, kinds, code, scale=0.7)
    layer = DuoKv8Layer(B, 16, 2, D, S, R, n, kinds, code=code)
    c.fill(layer)
    got = f64(layer.decode(c.query([n] * B)))
    want = np.stack([c.decode(b, n)[0] for b in range(B)])
    rounded = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    e0 = np.linalg.norm(rounded - want)
    assert np.linalg.norm(got - want) <= 1.05 * e0
