"""GB300-native mixed-head causal attention (retrieval + streaming heads) for long-context serving.

The product is the C ABI in ``include/duo_attn.h``, implemented by
``libduo_attn.so`` (hand-written sm_103a kernels). This package holds its thin
ctypes binding (``_lib``, the same entry-point names), ``DuoLayer`` -- a small
owner of the torch tensors one layer's caches live in -- and the algorithmic
work counters used to report throughput (``workload``).
"""

from __future__ import annotations

from . import _lib
from ._lib import (DUO_RETRIEVAL, DUO_STREAMING, DuoError, duo_attn_decode, duo_attn_decode_varlen,  # noqa: F401
                   duo_attn_prefill, duo_attn_prefill_select, duo_cache_reset, duo_classify_heads, duo_create,
                   duo_decode_workspace_size, duo_destroy, duo_device_error, duo_kv_append, duo_kv_append_varlen,
                   duo_last_error, duo_paged_stream_dead_blocks)


class DuoLayer:
    """Caches of one attention layer in torch device memory plus a library handle.

    k_full/v_full: bf16 [B, n_ret, max_seq_len, D]; k_sr/v_sr: bf16 [B, n_str, S+R, D];
    pos: int32 [B, S+R]; ``n`` tokens appended so far. ``workspace`` is the decode
    workspace (zero-filled once)."""

    def __init__(self, batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, max_seq_len,
                 is_retrieval, device="cuda"):
        import torch
        self.B, self.Hq, self.Hkv, self.D = batch, num_q_heads, num_kv_heads, head_dim
        self.S, self.R, self.cap = sink_size, recent_size, max_seq_len
        self.is_retrieval = [1 if x else 0 for x in is_retrieval]
        self.kind_index, self.n_ret = duo_classify_heads(self.is_retrieval)
        self.n_str = num_kv_heads - self.n_ret
        self.device = torch.device(device)
        with torch.cuda.device(self.device):
            self.handle = duo_create(batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size,
                                     max_seq_len, self.is_retrieval)
        bf = dict(dtype=torch.bfloat16, device=self.device)
        SR = sink_size + recent_size
        self.k_full = torch.empty((batch, self.n_ret, max_seq_len if self.n_ret else 0, head_dim), **bf)
        self.v_full = torch.empty_like(self.k_full)
        self.k_sr = torch.empty((batch, self.n_str, SR, head_dim), **bf)
        self.v_sr = torch.empty_like(self.k_sr)
        self.pos = torch.empty((batch, SR), dtype=torch.int32, device=self.device)
        ws = duo_decode_workspace_size(self.handle, 1)
        self.workspace = torch.zeros(((ws + 255) // 256) * 256, dtype=torch.uint8, device=self.device)
        self.cache = _lib.duo_kv_cache(self.k_full.data_ptr() if self.n_ret else None,
                                       self.v_full.data_ptr() if self.n_ret else None,
                                       self.k_sr.data_ptr() if self.n_str else None,
                                       self.v_sr.data_ptr() if self.n_str else None,
                                       self.pos.data_ptr(), 0)
        self.reset()

    @property
    def n(self) -> int:
        return int(self.cache.n)

    def reset(self, stream=None) -> None:
        duo_cache_reset(self.handle, self.cache, stream)

    def append(self, k_new, v_new, stream=None) -> None:
        T = k_new.shape[1]
        _lib._bf16(k_new, (self.B, T, self.Hkv, self.D), "k_new")
        _lib._bf16(v_new, (self.B, T, self.Hkv, self.D), "v_new")
        duo_kv_append(self.handle, self.cache, k_new, v_new, T, stream)

    def prefill(self, q, k, v, out=None, kind_mask=3, stream=None):
        import torch
        T = q.shape[1]
        _lib._bf16(q, (self.B, T, self.Hq, self.D), "q")
        _lib._bf16(k, (self.B, T, self.Hkv, self.D), "k")
        _lib._bf16(v, (self.B, T, self.Hkv, self.D), "v")
        if out is None:
            out = torch.empty_like(q)
        _lib._bf16(out, (self.B, T, self.Hq, self.D), "o")
        duo_attn_prefill_select(self.handle, self.cache, q, k, v, T, out, kind_mask, stream)
        return out

    def decode(self, q, out=None, stream=None):
        import torch
        _lib._bf16(q, (self.B, self.Hq, self.D), "q")
        if out is None:
            out = torch.empty_like(q)
        _lib._bf16(out, (self.B, self.Hq, self.D), "o")
        duo_attn_decode(self.handle, self.cache, q, out, self.workspace, stream)
        return out

    def dca_prefill(self, q, q_succ, q_inter, k, v, chunk_len, mscale=None, out=None, stream=None):
        """Dual Chunk Attention prefill of T tokens at positions n ... n+T-1 against the cache
        (n = tokens appended so far, a multiple of 256; every head full attention); mscale:
        fp32 [B, T] on the device or None."""
        import torch
        T = q.shape[1]
        for name, t in (("q", q), ("q_succ", q_succ), ("q_inter", q_inter)):
            _lib._bf16(t, (self.B, T, self.Hq, self.D), name)
        _lib._bf16(k, (self.B, T, self.Hkv, self.D), "k")
        _lib._bf16(v, (self.B, T, self.Hkv, self.D), "v")
        _check_mscale(mscale, (self.B, T))
        if out is None:
            out = torch.empty_like(q)
        _lib._bf16(out, (self.B, T, self.Hq, self.D), "o")
        _lib.duo_dca_prefill(self.handle, self.cache, q, q_succ, q_inter, k, v, mscale, T, chunk_len, out, stream)
        return out

    def dca_decode(self, q, q_succ, q_inter, chunk_len, mscale=None, out=None, stream=None):
        """Dual Chunk Attention decode of the token at position n - 1; mscale fp32 [B] or None."""
        import torch
        for name, t in (("q", q), ("q_succ", q_succ), ("q_inter", q_inter)):
            _lib._bf16(t, (self.B, self.Hq, self.D), name)
        _check_mscale(mscale, (self.B,))
        if out is None:
            out = torch.empty_like(q)
        _lib._bf16(out, (self.B, self.Hq, self.D), "o")
        _lib.duo_dca_decode(self.handle, self.cache, q, q_succ, q_inter, mscale, chunk_len, out, self.workspace, stream)
        return out

    def append_varlen(self, k_new, v_new, seq_lens, stream=None) -> None:
        """One token per sequence at positions seq_lens (device int32 [B]), which advance by one."""
        _lib._bf16(k_new, (self.B, 1, self.Hkv, self.D), "k_new")
        _lib._bf16(v_new, (self.B, 1, self.Hkv, self.D), "v_new")
        _check_lens(seq_lens, self.B)
        duo_kv_append_varlen(self.handle, self.cache, seq_lens, k_new, v_new, stream)

    def decode_varlen(self, q, seq_lens, max_len, out=None, stream=None):
        """Decode where sequence b holds seq_lens[b] tokens (device int32 [B], <= max_len)."""
        import torch
        _lib._bf16(q, (self.B, self.Hq, self.D), "q")
        _check_lens(seq_lens, self.B)
        if out is None:
            out = torch.empty_like(q)
        _lib._bf16(out, (self.B, self.Hq, self.D), "o")
        duo_attn_decode_varlen(self.handle, self.cache, seq_lens, max_len, q, out, self.workspace, stream)
        return out

    def close(self) -> None:
        if getattr(self, "handle", None) is not None:
            duo_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DuoPagedLayer(DuoLayer):
    """A layer whose caches live in a shared pool of blocks addressed through block
    tables (device int32): retrieval heads through ``block_table`` [B, n_ret,
    max_blocks]; streaming heads through ``stream_table`` [B, n_str, max_blocks] when
    given (block-granular eviction: ``dead_blocks()`` names the blocks the caller may
    free), else they keep the sink + ring cache."""

    def __init__(self, batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, block_size,
                 max_blocks, num_blocks, block_table, is_retrieval, device="cuda", stream_table=None):
        import torch
        super().__init__(batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, 1, is_retrieval,
                         device=device)
        bf = dict(dtype=torch.bfloat16, device=self.device)
        self.block_size = block_size
        self.k_full = torch.empty((num_blocks, block_size, head_dim), **bf)
        self.v_full = torch.empty_like(self.k_full)
        self.cache.k_full = self.k_full.data_ptr()
        self.cache.v_full = self.v_full.data_ptr()
        for name, t, rows in (("block_table", block_table, self.n_ret), ("stream_table", stream_table, self.n_str)):
            if t is not None:
                assert t.dtype == torch.int32 and t.is_cuda and t.is_contiguous(), name
                assert tuple(t.shape) == (batch, rows, max_blocks), name
        self.block_table = block_table
        self.stream_table = stream_table
        self.paged = _lib.duo_paged(block_table.data_ptr() if block_table is not None else None, block_size,
                                    max_blocks, num_blocks,
                                    stream_table.data_ptr() if stream_table is not None else None)

    def dead_blocks(self, n=None) -> tuple:
        """Logical blocks [lo, hi) of every streaming head that no query can see any more."""
        return _lib.duo_paged_stream_dead_blocks(self.S, self.R, self.block_size, self.n if n is None else n)

    def append(self, k_new, v_new, stream=None) -> None:
        T = k_new.shape[1]
        _lib._bf16(k_new, (self.B, T, self.Hkv, self.D), "k_new")
        _lib._bf16(v_new, (self.B, T, self.Hkv, self.D), "v_new")
        _lib.duo_kv_append_paged(self.handle, self.cache, self.paged, k_new, v_new, T, stream)

    def prefill(self, q, k, v, out=None, kind_mask=3, stream=None):
        import torch
        assert kind_mask == 3
        T = q.shape[1]
        _lib._bf16(q, (self.B, T, self.Hq, self.D), "q")
        if out is None:
            out = torch.empty_like(q)
        _lib.duo_attn_prefill_paged(self.handle, self.cache, self.paged, q, k, v, T, out, stream)
        return out

    def decode(self, q, out=None, stream=None):
        import torch
        _lib._bf16(q, (self.B, self.Hq, self.D), "q")
        if out is None:
            out = torch.empty_like(q)
        _lib.duo_attn_decode_paged(self.handle, self.cache, self.paged, q, out, self.workspace, stream)
        return out


class DuoKv4Layer(DuoLayer):
    """A layer whose caches hold 4-bit codes with an fp16 (scale, zero) pair per row
    (layout in include/duo_attn.h): codes u8 [B, planes, pitch, D/2] and pairs int32
    [B, planes, pitch], pitch = capacity rounded up to 16 rows. Prefill attention is
    computed from bf16 inputs as usual; appends quantize; decode reads the codes."""

    def __init__(self, batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, max_seq_len,
                 is_retrieval, device="cuda"):
        import torch
        super().__init__(batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, 1, is_retrieval,
                         device=device)
        self.cap = max_seq_len
        cap16 = -(-max_seq_len // 16) * 16
        sr16 = -(-(sink_size + recent_size) // 16) * 16
        u8 = dict(dtype=torch.uint8, device=self.device)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.k_codes = torch.zeros((batch, self.n_ret, cap16 if self.n_ret else 0, head_dim // 2), **u8)
        self.v_codes = torch.zeros_like(self.k_codes)
        self.k_sz = torch.zeros((batch, self.n_ret, cap16 if self.n_ret else 0), **i32)
        self.v_sz = torch.zeros_like(self.k_sz)
        self.ks_codes = torch.zeros((batch, self.n_str, sr16, head_dim // 2), **u8)
        self.vs_codes = torch.zeros_like(self.ks_codes)
        self.ks_sz = torch.zeros((batch, self.n_str, sr16), **i32)
        self.vs_sz = torch.zeros_like(self.ks_sz)
        # the handle's capacity is max_seq_len: recreate it with the real value
        duo_destroy(self.handle)
        with torch.cuda.device(self.device):
            self.handle = duo_create(batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, max_seq_len,
                                     self.is_retrieval)
        ptr = lambda t: t.data_ptr() if t.numel() else None
        self.kv4 = _lib.duo_kv4_cache(ptr(self.k_codes), ptr(self.v_codes), ptr(self.k_sz), ptr(self.v_sz),
                                      ptr(self.ks_codes), ptr(self.vs_codes), ptr(self.ks_sz), ptr(self.vs_sz))
        self.reset()

    def append(self, k_new, v_new, stream=None) -> None:
        T = k_new.shape[1]
        _lib._bf16(k_new, (self.B, T, self.Hkv, self.D), "k_new")
        _lib._bf16(v_new, (self.B, T, self.Hkv, self.D), "v_new")
        _lib.duo_kv_append_kv4(self.handle, self.cache, self.kv4, k_new, v_new, T, stream)

    def decode(self, q, out=None, stream=None):
        import torch
        _lib._bf16(q, (self.B, self.Hq, self.D), "q")
        if out is None:
            out = torch.empty_like(q)
        _lib._bf16(out, (self.B, self.Hq, self.D), "o")
        _lib.duo_attn_decode_kv4(self.handle, self.cache, self.kv4, q, out, self.workspace, stream)
        return out

    def prefill(self, q, k, v, out=None, kind_mask=3, stream=None):
        """A chunk of T new tokens against the 4-bit caches (dequantized in the kernel)."""
        import torch
        assert kind_mask == 3
        T = q.shape[1]
        _lib._bf16(q, (self.B, T, self.Hq, self.D), "q")
        _lib._bf16(k, (self.B, T, self.Hkv, self.D), "k")
        _lib._bf16(v, (self.B, T, self.Hkv, self.D), "v")
        if out is None:
            out = torch.empty_like(q)
        _lib._bf16(out, (self.B, T, self.Hq, self.D), "o")
        _lib.duo_attn_prefill_kv4(self.handle, self.cache, self.kv4, q, k, v, T, out, stream)
        return out


class DuoKv4PagedLayer(DuoKv4Layer):
    """4-bit caches whose retrieval rows live in a pool of blocks shared by every sequence
    and head: codes u8 [num_blocks, block_size, D/2] and (scale, zero) pairs int32
    [num_blocks, block_size], row t of retrieval head r of sequence b at row t %
    block_size of block block_table[b, r, t // block_size] (block_table: device int32
    [B, n_ret, max_blocks]; block_size a multiple of 128). Streaming heads keep their 4-bit
    sink + ring arrays."""

    def __init__(self, batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, block_size,
                 max_blocks, num_blocks, block_table, is_retrieval, device="cuda"):
        import torch
        super().__init__(batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, 16, is_retrieval,
                         device=device)
        u8 = dict(dtype=torch.uint8, device=self.device)
        i32 = dict(dtype=torch.int32, device=self.device)
        rows = num_blocks * block_size if self.n_ret else 0
        self.k_codes = torch.zeros((rows, head_dim // 2), **u8)
        self.v_codes = torch.zeros_like(self.k_codes)
        self.k_sz = torch.zeros((rows,), **i32)
        self.v_sz = torch.zeros_like(self.k_sz)
        if block_table is not None:
            assert block_table.dtype == torch.int32 and block_table.is_cuda and block_table.is_contiguous()
            assert tuple(block_table.shape) == (batch, self.n_ret, max_blocks)
        self.block_size = block_size
        self.block_table = block_table
        self.paged = _lib.duo_paged(block_table.data_ptr() if block_table is not None else None, block_size,
                                    max_blocks, num_blocks, None)
        ptr = lambda t: t.data_ptr() if t.numel() else None
        self.kv4 = _lib.duo_kv4_cache(ptr(self.k_codes), ptr(self.v_codes), ptr(self.k_sz), ptr(self.v_sz),
                                      ptr(self.ks_codes), ptr(self.vs_codes), ptr(self.ks_sz), ptr(self.vs_sz))

    def append(self, k_new, v_new, stream=None) -> None:
        T = k_new.shape[1]
        _lib._bf16(k_new, (self.B, T, self.Hkv, self.D), "k_new")
        _lib._bf16(v_new, (self.B, T, self.Hkv, self.D), "v_new")
        _lib.duo_kv_append_kv4_paged(self.handle, self.cache, self.paged, self.kv4, k_new, v_new, T, stream)

    def prefill(self, *args, **kwargs):
        raise NotImplementedError("prefill against 4-bit rows in a paged pool is not provided")

    def decode(self, q, out=None, stream=None):
        import torch
        _lib._bf16(q, (self.B, self.Hq, self.D), "q")
        if out is None:
            out = torch.empty_like(q)
        _lib._bf16(out, (self.B, self.Hq, self.D), "o")
        _lib.duo_attn_decode_kv4_paged(self.handle, self.cache, self.paged, self.kv4, q, out, self.workspace, stream)
        return out


class DuoKv8Layer(DuoLayer):
    """A layer whose retrieval heads' caches hold 8-bit codes (``code``: "int8" or "e4m3") with
    one fp32 scale per block of 64 tokens of a head (layout and rounding in include/duo_attn.h):
    k_codes/v_codes [B, n_ret, cap64, D], k_scale/v_scale fp32 [B, n_ret, cap64 / 64] and the
    open block's rows in bf16, k_tail/v_tail [B, n_ret, 64, D]. Streaming heads keep their bf16
    sink + ring caches."""

    def __init__(self, batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, max_seq_len,
                 is_retrieval, code="int8", device="cuda"):
        super().__init__(batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, 1, is_retrieval,
                         device=device)
        self.cap = max_seq_len
        self._set_capacity(max_seq_len)
        cap64 = -(-max_seq_len // _lib.DUO_KV8_BLOCK) * _lib.DUO_KV8_BLOCK if self.n_ret else 0
        self._codes(code, (batch, self.n_ret, cap64), (batch, self.n_ret, cap64 // _lib.DUO_KV8_BLOCK))
        self.reset()

    def _set_capacity(self, max_seq_len):
        """The handle's capacity is max_seq_len: create it again with that value."""
        import torch
        duo_destroy(self.handle)
        self.handle = None
        with torch.cuda.device(self.device):
            self.handle = duo_create(self.B, self.Hq, self.Hkv, self.D, self.S, self.R, max_seq_len,
                                     self.is_retrieval)

    def _codes(self, code, rows, blocks):
        import torch
        if code not in ("int8", "e4m3"):
            raise ValueError(f'code: "int8" or "e4m3", got {code!r}')
        self.code = code
        dtype = torch.int8 if code == "int8" else torch.float8_e4m3fn
        dev = dict(device=self.device)
        self.k_codes = torch.zeros(rows + (self.D,), dtype=torch.uint8, **dev).view(dtype)
        self.v_codes = torch.zeros(rows + (self.D,), dtype=torch.uint8, **dev).view(dtype)
        self.k_scale = torch.zeros(blocks, dtype=torch.float32, **dev)
        self.v_scale = torch.zeros(blocks, dtype=torch.float32, **dev)
        self.k_tail = torch.zeros((self.B, self.n_ret, _lib.DUO_KV8_BLOCK, self.D), dtype=torch.bfloat16, **dev)
        self.v_tail = torch.zeros_like(self.k_tail)
        ptr = lambda t: t.data_ptr() if t.numel() else None
        self.kv8 = _lib.duo_kv8_cache(ptr(self.k_codes), ptr(self.v_codes), ptr(self.k_scale), ptr(self.v_scale),
                                      ptr(self.k_tail), ptr(self.v_tail),
                                      _lib.DUO_KV8_INT8 if code == "int8" else _lib.DUO_KV8_E4M3)
        self.paged = None
        # (looked up here: a small call's time is the host's)
        self.index, self.bf16, self.empty_like = self.pos.get_device(), torch.bfloat16, torch.empty_like
        self.row = (self.B, self.Hq, self.D)

    def append(self, k_new, v_new, stream=None) -> None:
        T = k_new.shape[1]
        _on(self, "k_new", k_new, (self.B, T, self.Hkv, self.D))
        _on(self, "v_new", v_new, (self.B, T, self.Hkv, self.D))
        if self.paged is None:
            _lib.duo_kv_append_kv8(self.handle, self.cache, self.kv8, k_new, v_new, T, stream)
        else:
            _lib.duo_kv_append_kv8_paged(self.handle, self.cache, self.paged, self.kv8, k_new, v_new, T, stream)

    def decode(self, q, out=None, stream=None):
        out = self._out(q, self.row, out)
        if self.paged is None:
            _lib.duo_attn_decode_kv8(self.handle, self.cache, self.kv8, q, out, self.workspace, stream)
        else:
            _lib.duo_attn_decode_kv8_paged(self.handle, self.cache, self.paged, self.kv8, q, out, self.workspace,
                                           stream)
        return out

    def decode_varlen(self, q, seq_lens, max_len, out=None, stream=None):
        """Decode where sequence b holds seq_lens[b] tokens, the new one included (device int32
        [B], <= max_len); a sequence of length 0 gets zeros."""
        out = self._out(q, self.row, out)
        _check_lens(seq_lens, self.B)
        if seq_lens.get_device() != self.index:
            raise ValueError(f"seq_lens: on {seq_lens.device}, the layer is on CUDA device {self.index}")
        _lib.duo_attn_decode_kv8_varlen(self.handle, self.cache, self.paged, self.kv8, seq_lens, max_len, q, out,
                                        self.workspace, stream)
        return out

    def _out(self, q, shape, out):
        _on(self, "q", q, shape)
        if out is None:
            return self.empty_like(q)
        _on(self, "o", out, shape)
        return out

    def append_varlen(self, *args, **kwargs):
        raise NotImplementedError("8-bit caches: append_ragged (a paged layer) takes lengths from the device")

    def prefill(self, q, k, v, out=None, kind_mask=3, stream=None):
        """A chunk of T new tokens against the 8-bit caches. Their rows are written as bf16 to a
        workspace first (4 D bytes per cached token and retrieval head), taken from torch's
        allocator on the stream the call runs on."""
        import torch
        if kind_mask != 3:
            raise NotImplementedError("8-bit caches: prefill takes the heads of both kinds")
        T = q.shape[1]
        out = self._out(q, (self.B, T, self.Hq, self.D), out)
        _on(self, "k", k, (self.B, T, self.Hkv, self.D))
        _on(self, "v", v, (self.B, T, self.Hkv, self.D))
        need = _lib.duo_prefill_kv8_workspace_size(self.handle, self.n, T)
        if stream is None:
            ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:  # its memory may be given out again as soon as this returns: in that stream's order
            handle = _lib._stream_ptr(stream)
            with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=q.device)):
                ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        if self.paged is None:
            _lib.duo_attn_prefill_kv8(self.handle, self.cache, self.kv8, q, k, v, T, out, ws, stream)
        else:
            _lib.duo_attn_prefill_kv8_paged(self.handle, self.cache, self.paged, self.kv8, q, k, v, T, out, ws, stream)
        return out

    def dca_prefill(self, *args, **kwargs):
        raise NotImplementedError("Dual Chunk Attention over 8-bit caches is not provided")

    dca_decode = dca_prefill


class DuoKv8PagedLayer(DuoKv8Layer):
    """8-bit caches whose codes and scales live in a pool of blocks shared by every sequence
    and head: k_codes/v_codes [num_blocks, block_size, D], k_scale/v_scale [num_blocks,
    block_size / 64], row t of retrieval head r of sequence b at row t % block_size of block
    block_table[b, r, t // block_size] (device int32 [B, n_ret, max_blocks]; block_size a
    multiple of 128). ``append_ragged`` and ``decode_varlen`` take every length from the device
    (see DuoBlockPool)."""

    def __init__(self, batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, block_size,
                 max_blocks, num_blocks, block_table, is_retrieval, code="int8", device="cuda"):
        super().__init__(batch, num_q_heads, num_kv_heads, head_dim, sink_size, recent_size, 1, is_retrieval,
                         code=code, device=device)
        if block_table is not None:
            _check_table(block_table, (batch, self.n_ret, max_blocks), self.index)
        blocks = num_blocks if self.n_ret else 0
        self._codes(code, (blocks, block_size), (blocks, block_size // _lib.DUO_KV8_BLOCK))
        self.block_size = block_size
        self.block_table = block_table
        self.paged = _lib.duo_paged(block_table.data_ptr() if block_table is not None else None, block_size,
                                    max_blocks, num_blocks, None)

    def append_ragged(self, k_new, v_new, slot_map, stream=None) -> None:
        """A packed batch of tokens [num_tokens, Hkv, D], each at its own place (a DuoSlotMap). The lengths
        stay on the device: ``n`` does not change, so ``decode`` and ``prefill``, which go by it, need
        ``cache.n`` set by the caller (and sequences of one length)."""
        N = k_new.shape[0]
        _on(self, "k_new", k_new, (N, self.Hkv, self.D))
        _on(self, "v_new", v_new, (N, self.Hkv, self.D))
        if slot_map.cu_new.get_device() != self.index:
            raise ValueError(f"slot_map: on {slot_map.cu_new.device}, the layer is on CUDA device {self.index}")
        if slot_map.batch != self.B or slot_map.num_tokens != N or (self.n_ret and slot_map.planes != self.n_ret):
            raise ValueError(f"slot_map: of {slot_map.batch} sequences, {slot_map.num_tokens} tokens and "
                             f"{slot_map.planes} planes; need {self.B}, {N} and {self.n_ret}")
        _lib.duo_kv_append_kv8_ragged(self.handle, self.cache, self.paged, self.kv8, slot_map.c, N, k_new, v_new,
                                      stream)


class DuoSlotMap:
    """Where the tokens of a packed batch go: cu_new int32 [B + 1], token_seq and token_pos int32
    [num_tokens], slots int64 [num_tokens, planes], all on the device (include/duo_attn.h)."""

    def __init__(self, cu_new, token_seq, token_pos, slots):
        import torch
        N = token_seq.shape[0]
        for name, t, dtype, dims in (("cu_new", cu_new, torch.int32, 1), ("token_seq", token_seq, torch.int32, 1),
                                     ("token_pos", token_pos, torch.int32, 1), ("slots", slots, torch.int64, 2)):
            if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or t.dim() != dims or t.device != cu_new.device:
                raise ValueError(f"{name}: need a contiguous CUDA {dtype} tensor of {dims} dimension(s), all on one device")
        if token_pos.shape[0] != N or slots.shape[0] != N:
            raise ValueError("token_seq, token_pos and slots: different numbers of tokens")
        self.cu_new, self.token_seq, self.token_pos, self.slots = cu_new, token_seq, token_pos, slots
        self.batch, self.num_tokens, self.planes = cu_new.shape[0] - 1, N, slots.shape[1]
        self.c = _lib.duo_slot_map(cu_new.data_ptr(), token_seq.data_ptr(), token_pos.data_ptr(), slots.data_ptr())


class DuoBlockPool:
    """Block tables, free list and lengths of a batch kept on the device, and the slot map of
    its packed steps of up to max_tokens tokens. block_table int32 [B, planes, max_blocks],
    free_list int32 [num_blocks] (at first every block, taken from the end), free_count int32
    [1], seq_lens int32 [B]. ``planes`` is a layer's number of retrieval heads."""

    def __init__(self, batch, planes, block_size, max_blocks, num_blocks, max_tokens, device="cuda"):
        import torch
        self.device = torch.device(device)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.block_table = torch.full((batch, planes, max_blocks), -1, **i32)
        self.free_list = torch.arange(num_blocks, **i32)
        self.free_count = torch.full((1,), num_blocks, **i32)
        self.seq_lens = torch.zeros(batch, **i32)
        self.batch, self.max_tokens = batch, max_tokens
        self.index, self.int32 = self.seq_lens.get_device(), torch.int32
        self.slot_map = DuoSlotMap(torch.zeros(batch + 1, **i32), torch.full((max_tokens,), -1, **i32),
                                   torch.full((max_tokens,), -1, **i32),
                                   torch.full((max_tokens, planes), -1, dtype=torch.int64, device=self.device))
        self.workspace = torch.empty(_lib.duo_block_tables_workspace_size(batch), dtype=torch.uint8,
                                     device=self.device)
        self.c = _lib.duo_block_pool(self.block_table.data_ptr(), self.free_list.data_ptr(),
                                     self.free_count.data_ptr(), self.seq_lens.data_ptr(), batch, planes, block_size,
                                     max_blocks, num_blocks)

    def update(self, new_lens, seq_lens_out=None, free_count_out=None, stream=None):
        """Sequence b takes new_lens[b] more tokens (-1: it has finished; device int32 [B]).
        Updates tables, free list and lengths (into the *_out tensors if given) and returns
        the slot map of the packed tokens, whose arrays the next update overwrites."""
        lens = self.seq_lens if seq_lens_out is None else seq_lens_out
        count = self.free_count if free_count_out is None else free_count_out
        for name, t, n in (("new_lens", new_lens, self.batch), ("seq_lens_out", lens, self.batch),
                           ("free_count_out", count, 1)):
            if t.dtype is not self.int32 or t.get_device() != self.index or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"{name}: need a contiguous int32 tensor of {n} element(s) on CUDA device {self.index}")
        if _lib._current_device() != self.index:
            raise ValueError(f"the current device is not the pool's (CUDA device {self.index})")
        _lib.duo_block_tables_update(self.c, new_lens, self.max_tokens, lens, count, self.slot_map.c, self.workspace,
                                     stream)
        return self.slot_map


def _on(layer, name, t, shape):
    """_lib._bf16, and on the layer's own device."""
    if (t.dtype is not layer.bf16 or t.get_device() != layer.index or t.shape != shape or not t.is_contiguous()):
        _lib._bf16(t, shape, name)
        raise ValueError(f"{name}: on {t.device}, the layer is on CUDA device {layer.index}")


def _check_table(t, shape, index):
    """A block table of a layer on CUDA device `index`."""
    import torch
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"block_table: need a contiguous CUDA int32 tensor of shape {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"block_table: on {t.device}, the layer is on CUDA device {index}")


def _check_mscale(mscale, shape):
    import torch
    if mscale is None:
        return
    if (mscale.dtype != torch.float32 or not mscale.is_cuda or not mscale.is_contiguous()
            or tuple(mscale.shape) != tuple(shape)):
        raise ValueError(f"mscale: need a contiguous CUDA float32 tensor of shape {tuple(shape)}")


def _check_lens(seq_lens, B):
    import torch
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda or not seq_lens.is_contiguous() or seq_lens.numel() != B:
        raise ValueError(f"seq_lens: need a contiguous CUDA int32 tensor of {B} elements")
