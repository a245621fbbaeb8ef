"""Outputs that a call makes itself come from the allocator in the order of the stream the call runs on (CPU:
torch's current stream, the allocations and the library are recorded)."""

import inspect

import pytest
import torch

import streaming_kv_cache_duo_gb300 as duo
from streaming_kv_cache_duo_gb300 import _lib

B, T, Hq, Hkv, D = 2, 3, 4, 2, 64
STREAM, CURRENT = 0x5eed0, 0xc0de0


@pytest.fixture
def record(monkeypatch):
    """[(stream in effect, tensor)] of every allocation; library calls do nothing."""
    made, within = [], []
    real_like, real_empty = torch.empty_like, torch.empty

    def on(stream):
        within[:] = [] if stream == CURRENT else [stream]

    def like(*a, **kw):
        t = real_like(*a, **kw)
        made.append((within[-1] if within else None, t))
        return t

    def empty(*a, **kw):
        t = real_empty(*a, **kw)
        made.append((within[-1] if within else None, t))
        return t

    monkeypatch.setattr(torch, "empty_like", like)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "set_stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: CURRENT)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: ptr)
    monkeypatch.setattr(_lib, "_bf16", lambda *a: None)
    monkeypatch.setattr(_lib, "_current_device", lambda: -1)
    monkeypatch.setattr(_lib, "_stream_ptr", lambda s: CURRENT if s is None else s)
    monkeypatch.setattr(duo, "_check_lens", lambda *a: None)
    for module in (_lib, duo):
        for name in list(vars(module)):
            if name.startswith("duo_") and callable(getattr(module, name)) and not isinstance(getattr(module, name), type):
                monkeypatch.setattr(module, name, lambda *a, **kw: 1024)
    yield made
    assert not within  # (the current stream is what it was)


def _layer(cls):
    x = cls.__new__(cls)
    x.B, x.Hq, x.Hkv, x.D, x.n_ret, x.n_str = B, Hq, Hkv, D, 1, 1
    x.handle = x.paged = x.kv4 = x.kv8 = x.stream_table = None
    x.cache = _lib.duo_kv_cache(None, None, None, None, None, 0)
    x.workspace, x.index, x.bf16 = None, -1, torch.bfloat16
    x.empty_like, x.row = torch.empty_like, (B, Hq, D)
    return x


def _map(N):
    m = duo.DuoSlotMap.__new__(duo.DuoSlotMap)
    m.batch, m.num_tokens, m.planes, m.index, m.c = B, N, 1, -1, None
    return m


def _rope():
    x = duo.DuoRope.__new__(duo.DuoRope)
    x.head_dim, x.index, x.bf16, x.int32 = D, -1, torch.bfloat16, torch.int32
    x.empty_like, x.c = torch.empty_like, None
    return x


def _rows(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _fused(N):
    return _rows(N, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 1)


def _packed(method):
    def call(stream, dense):
        N = 5
        q, k, v = _fused(N)
        if dense:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        layer = _layer(duo.DuoPagedLayer)
        if method == "append_ragged":
            return [layer.append_ragged(k, v, _map(N), rope=_rope(), q=q, stream=stream)]
        if method == "prefill_ragged":
            return [layer.prefill_ragged(q, k, v, _map(N), stream=stream)]
        return list(_rope().rotate(q, k, torch.zeros(N, dtype=torch.int32), stream=stream))
    return call


def _uniform(cls, method):
    def call(stream, dense):
        layer = _layer(cls)
        q, chunk = _rows(B, Hq, D), [_rows(B, T, h, D) for h in (Hq, Hkv, Hkv)]
        lens = torch.zeros(B, dtype=torch.int32)
        args = {"decode": (q,), "decode_varlen": (q, lens, 10), "prefill": chunk, "dca_decode": (q, q, q, 256),
                "dca_prefill": (chunk[0], chunk[0], chunk[0], chunk[1], chunk[2], 256)}[method]
        return [getattr(layer, method)(*args, stream=stream)]
    return call


CALLS = {name: _packed(name) for name in ("append_ragged", "prefill_ragged", "rotate")}
for _cls, _methods in ((duo.DuoLayer, ("prefill", "decode", "dca_prefill", "dca_decode", "decode_varlen")),
                       (duo.DuoPagedLayer, ("prefill", "decode", "decode_varlen")), (duo.DuoKv4Layer, ("prefill", "decode")),
                       (duo.DuoKv4PagedLayer, ("decode",)), (duo.DuoKv8Layer, ("prefill", "decode", "decode_varlen"))):
    CALLS.update({f"{_cls.__name__}.{m}": _uniform(_cls, m) for m in _methods})


@pytest.mark.parametrize("dense", [True, False], ids=["dense", "slices"])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_outputs_are_the_streams_own(record, name, dense):
    outs = CALLS[name](STREAM, dense)
    assert outs and all(o.is_contiguous() for o in outs)
    for o in outs:
        assert [s for s, t in record if t is o] == [STREAM], name
    assert all(s == STREAM for s, _ in record)  # and so is what the call needs besides
    for stream in (None, CURRENT):  # the current one: nothing to switch
        record.clear()
        outs = CALLS[name](stream, dense)
        assert record and all(s is None for s, _ in record) and all(o.is_contiguous() for o in outs)


def test_every_call_with_a_stream_and_an_output_is_among_them():
    classes = (duo.DuoLayer, duo.DuoPagedLayer, duo.DuoRope, duo.DuoKv4Layer, duo.DuoKv4PagedLayer, duo.DuoKv8Layer,
               duo.DuoKv8PagedLayer)
    for cls in classes:
        for name, f in vars(cls).items():
            if not callable(f) or name.startswith("_"):
                continue
            args = inspect.signature(f).parameters
            if "stream" in args and {"out", "q_out", "k_out"} & set(args):
                assert name in CALLS or f"{cls.__name__}.{name}" in CALLS, (cls, name)
