"""Calls on another stream that make their own outputs: right, and of that stream's memory."""

import numpy as np
import pytest
import torch

from ragged_util import normal
from test_gpu_attn_ragged import Batch

pytestmark = pytest.mark.gpu


def _calls():
    """name -> call(stream) -> outputs, of a batch of three sequences with a cache."""
    from streaming_kv_cache_duo_gb300 import DuoRope
    x = Batch(41, [(700, 60), (0, 200), (40, 1)], 8, 2, 1, 128, 4, 32, 128)
    start, new = [700, 0, 40], [60, 200, 1]
    q, k, v = (x.packed(y, start, new) for y in (x.q, x.k, x.v))
    fused = torch.cat([q, k, v], 1)
    qs, ks, vs = fused.split([8, 2, 2], 1)
    m, rope = x.map(start, new), DuoRope(128)
    three = x.map([None, 100, None], [0, 3, 0])  # (of a sequence that holds nothing for the other calls)
    lens = torch.tensor([700, 0, 40], dtype=torch.int32, device="cuda")
    return {"rotate": lambda s: rope.rotate(qs, ks, m.token_pos, stream=s),
            "rotate dense": lambda s: rope.rotate(q, k, m.token_pos, stream=s),
            "prefill": lambda s: [x.layer.prefill_ragged(qs, ks, vs, m, stream=s)],
            "decode": lambda s: [x.layer.decode_varlen(q[:3], lens, 700, stream=s)],
            "append": lambda s: [x.layer.append_ragged(ks[:3], vs[:3], three, rope=rope, q=qs[:3], stream=s)]}


def test_outputs_made_on_another_stream():
    from streaming_kv_cache_duo_gb300 import duo_device_error
    for name, call in _calls().items():
        ref = [o.clone() for o in call(None)]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for stream in (side, side.cuda_stream):
            freed = [torch.empty_like(o) for o in ref]  # memory that the current stream is through with on the host
            taken = {t.data_ptr() for t in freed}
            del freed
            side.wait_stream(torch.cuda.current_stream())
            out = call(stream)
            assert all(o.data_ptr() not in taken for o in out), name
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), name
            own = {o.data_ptr() for o in out}
            del out
            assert all(torch.empty_like(o).data_ptr() not in own for o in ref), name
        with torch.cuda.stream(side):  # the default stream by its handle, while another one is current
            out = call(0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref)), name
    assert duo_device_error() == 0


def test_outputs_of_calls_captured_on_their_own_stream():
    from streaming_kv_cache_duo_gb300 import duo_device_error
    calls = _calls()
    ref = [o.clone() for name in calls for o in calls[name](None)]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = [o for name in calls for o in calls[name](side)]
    for o in out:
        o.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert duo_device_error() == 0 and all(torch.equal(a, b) for a, b in zip(out, ref))


def test_uniform_calls_on_another_stream():
    """The calls of one length: bf16 caches, contiguous and paged."""
    from streaming_kv_cache_duo_gb300 import DuoLayer, duo_device_error
    rng = np.random.default_rng(43)
    layer = DuoLayer(1, 4, 2, 64, 4, 32, 600, [1, 0])
    (k, _), (v, _), (q, _) = (normal(rng, 1, 300, h, 64) for h in (2, 2, 4))
    layer.append(k.cuda(), v.cuda())
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    for call in (lambda s: layer.prefill(q, k, v, stream=s), lambda s: layer.decode(q[:, 0].contiguous(), stream=s),
                 lambda s: layer.decode_varlen(q[:, 0].contiguous(), lens, 300, stream=s)):
        ref = call(None)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        out = call(side)
        side.synchronize()
        assert torch.equal(out, ref)
    assert duo_device_error() == 0
