"""GB300 TurboQuant compressed KV cache: Python binding of libtq.so.

The functions below carry the names of the C ABI (include/tq.h) and only
marshal arguments: tensors become device pointers, the current torch stream
becomes the cudaStream_t. Every step of encode and decode runs in the
library's CUDA kernels. PyTorch provides device memory and streams.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import NamedTuple, Optional

import numpy as np

from . import _lib
from ._lib import (TQ_BF16, TQ_DEVERR_BLOCK, TQ_DEVERR_CAPACITY, TQ_DEVERR_NONFINITE, TQ_DEVERR_SEQLEN, TQ_ENCODE_AUTO,
                   TQ_ENCODE_EXACT, TQ_F16, TQ_F32, TQ_KV8_E4M3, TQ_KV8_INT8, TQ_MODE_GROUP, TQ_MODE_MSE, TQ_MODE_PROD,
                   TQ_OK, TQError, check, lib, library_path, status_string, tq_batch, tq_cache_desc, tq_codec_info_t,
                   tq_blocks, tq_kv8_cache, tq_kv8_scores, tq_places, tq_rope, tq_rows, tq_split_state)

__all__ = [
    "tq_codec_create", "tq_codec_create_group", "tq_codec_destroy", "tq_codec_info",
    "tq_bits_split", "tq_codec_pair_for_bits",
    "tq_codec_build_host", "tq_codec_export", "tq_cache_desc_init", "tq_encode_append",
    "tq_quantize", "tq_decode_workspace_bytes", "tq_decode_attention", "tq_decode_attention_noalloc",
    "tq_decode_step", "tq_decode_plan",
    "tq_prefill_workspace_bytes", "tq_prefill_attention", "tq_cache_copy_blocks",
    "tq_decode_partials", "tq_decode_merge",
    "tq_encode_append_split", "tq_decode_workspace_bytes_split", "tq_decode_attention_split", "SplitCache",
    "tq_batch_filter", "tq_batch_extend", "tq_batch_merge", "tq_batch_extract", "Batch",
    "tq_kv8_append", "tq_kv8_attention", "tq_kv8_workspace_bytes", "KV8Cache", "Rope",
    "tq_rope_apply", "tq_blocks_reserve", "tq_blocks_release", "tq_verify_drafts", "BlockTable", "Places", "Verified",
    "tq_device_error", "tq_selftest_wait_timeout",
    "tq_launch_count", "tq_abi_version", "Codec", "CompressedKVCache", "TQError",
    "TQ_MODE_MSE", "TQ_MODE_PROD", "TQ_MODE_GROUP", "TQ_F32", "TQ_BF16", "TQ_F16",
    "TQ_ENCODE_AUTO", "TQ_ENCODE_EXACT", "TQ_KV8_E4M3", "TQ_KV8_INT8",
]


def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return TQ_F32
    if t.dtype == torch.bfloat16:
        return TQ_BF16
    if t.dtype == torch.float16:
        return TQ_F16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _torch().cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


# ----------------------------------------------------------------- raw ABI

def tq_abi_version() -> int:
    return lib().tq_abi_version()


def tq_launch_count() -> int:
    return int(lib().tq_launch_count())


def tq_codec_create(head_dim: int, bits: int, mode: int, seed: int) -> int:
    h = ctypes.c_void_p()
    check(lib().tq_codec_create(head_dim, bits, mode, seed, ctypes.byref(h)), "tq_codec_create")
    return h.value


def tq_codec_create_group(head_dim: int, bits: int, group_size: int) -> int:
    h = ctypes.c_void_p()
    check(lib().tq_codec_create_group(head_dim, bits, group_size, ctypes.byref(h)),
          "tq_codec_create_group")
    return h.value


def tq_bits_split(bits: float) -> tuple:
    """(key bits, value bits) of a possibly fractional width: floor/ceil, or b/b."""
    kb, vb = ctypes.c_int(), ctypes.c_int()
    check(lib().tq_bits_split(float(bits), ctypes.byref(kb), ctypes.byref(vb)), "tq_bits_split")
    return kb.value, vb.value


def tq_codec_pair_for_bits(head_dim: int, bits: float, seed: int) -> tuple:
    kh, vh = ctypes.c_void_p(), ctypes.c_void_p()
    check(lib().tq_codec_pair_for_bits(head_dim, float(bits), seed, ctypes.byref(kh), ctypes.byref(vh)),
          "tq_codec_pair_for_bits")
    return kh.value, vh.value


def tq_codec_destroy(handle: int) -> None:
    lib().tq_codec_destroy(handle)


def tq_codec_info(handle: int) -> dict:
    info = tq_codec_info_t()
    check(lib().tq_codec_info(handle, ctypes.byref(info)), "tq_codec_info")
    return {k: getattr(info, k) for k, _ in info._fields_}


def _tables(D: int, ib: int, with_s: bool):
    R = np.empty((D, D), np.float32)
    S = np.empty((D, D), np.float32) if with_s else None
    c = np.empty(1 << ib, np.float32)
    m = np.empty((1 << ib) - 1, np.float32)
    return R, S, c, m


def _np_ptr(a):
    return None if a is None else a.ctypes.data


def tq_codec_build_host(head_dim: int, bits: int, mode: int, seed: int):
    ib = bits - 1 if mode == TQ_MODE_PROD else bits
    R, S, c, m = _tables(head_dim, ib, mode == TQ_MODE_PROD)
    check(lib().tq_codec_build_host(head_dim, bits, mode, seed, _np_ptr(R), _np_ptr(S), _np_ptr(c),
                                    _np_ptr(m)), "tq_codec_build_host")
    return R, S, c, m


def tq_codec_export(handle: int):
    info = tq_codec_info(handle)
    R, S, c, m = _tables(info["head_dim"], info["index_bits"], info["mode"] == TQ_MODE_PROD)
    check(lib().tq_codec_export(handle, _np_ptr(R), _np_ptr(S), _np_ptr(c), _np_ptr(m)),
          "tq_codec_export")
    return R, S, c, m


def tq_cache_desc_init(key_codec: int, value_codec: int, num_layers: int, num_blocks: int,
                       block_tokens: int, num_kv_heads: int, pool=None):
    """Returns (desc, required_bytes). ``pool`` is a device tensor or None."""
    d = tq_cache_desc()
    req = ctypes.c_size_t()
    ptr = None if pool is None else pool.data_ptr()
    nbytes = 0 if pool is None else pool.numel() * pool.element_size()
    check(lib().tq_cache_desc_init(ctypes.byref(d), key_codec, value_codec, num_layers, num_blocks,
                                   block_tokens, num_kv_heads, ptr, nbytes, ctypes.byref(req)),
          "tq_cache_desc_init")
    return d, req.value


def tq_encode_append(key_codec: int, value_codec: int, desc: tq_cache_desc, layer: int, k, v,
                     seq_lens, block_table=None, max_blocks: int = 0, stream=None) -> None:
    batch, _, n_new, _ = k.shape
    check(lib().tq_encode_append(key_codec, value_codec, ctypes.byref(desc), layer, _ptr(k), _ptr(v),
                                 _dtype_code(k), batch, n_new, _ptr(seq_lens), _ptr(block_table),
                                 max_blocks, _stream(stream)), "tq_encode_append")


def tq_quantize(codec: int, x, idx, aux0=None, aux1=None, aux2=None, stream=None) -> None:
    n = x.shape[0]
    check(lib().tq_quantize(codec, _ptr(x), _dtype_code(x), n, _ptr(idx), _ptr(aux0), _ptr(aux1),
                            _ptr(aux2), _stream(stream)), "tq_quantize")


def tq_decode_workspace_bytes(desc: tq_cache_desc, batch: int, num_q_heads: int, q_len: int,
                              max_seq_len: int) -> int:
    out = ctypes.c_size_t()
    check(lib().tq_decode_workspace_bytes(ctypes.byref(desc), batch, num_q_heads, q_len, max_seq_len,
                                          ctypes.byref(out)), "tq_decode_workspace_bytes")
    return out.value


def tq_decode_attention(key_codec: int, value_codec: int, desc: tq_cache_desc, layer: int, q,
                        seq_lens, block_table, max_blocks: int, max_seq_len: int, out, workspace,
                        scale: float = 0.0, stream=None) -> None:
    batch, hq, lq, _ = q.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    check(lib().tq_decode_attention(key_codec, value_codec, ctypes.byref(desc), layer, _ptr(q),
                                    _dtype_code(q), batch, hq, lq, _ptr(seq_lens), _ptr(block_table),
                                    max_blocks, max_seq_len, scale, _ptr(out), _ptr(workspace),
                                    ws_bytes, _stream(stream)), "tq_decode_attention")


def tq_decode_plan(desc: tq_cache_desc, batch: int, num_q_heads: int, q_len: int, max_seq_len: int,
                   num_sms: int) -> dict:
    """The launch shape tq_decode_attention would use (host arithmetic; see include/tq.h)."""
    info = _lib.tq_decode_plan_info()
    check(lib().tq_decode_plan(ctypes.byref(desc), batch, num_q_heads, q_len, max_seq_len, num_sms,
                               ctypes.byref(info)), "tq_decode_plan")
    return {f: getattr(info, f) for f, _ in info._fields_}


def tq_decode_step(key_codec: int, value_codec: int, desc: tq_cache_desc, layer: int, k_new, v_new, q,
                   seq_lens, block_table, max_blocks: int, max_seq_len: int, out, workspace,
                   scale: float = 0.0, stream=None) -> None:
    """Append k_new / v_new [batch][kv heads][n_new][D] at seq_lens (the lengths before the step) and
    decode q over the grown sequences, in one call (see include/tq.h)."""
    batch, hq, lq, _ = q.shape
    n_new = k_new.shape[2]
    ws_bytes = workspace.numel() * workspace.element_size()
    check(lib().tq_decode_step(key_codec, value_codec, ctypes.byref(desc), layer, _ptr(k_new), _ptr(v_new),
                               _dtype_code(k_new), n_new, _ptr(q), _dtype_code(q), batch, hq, lq,
                               _ptr(seq_lens), _ptr(block_table), max_blocks, max_seq_len, scale, _ptr(out),
                               _ptr(workspace), ws_bytes, _stream(stream)), "tq_decode_step")


def tq_cache_copy_blocks(src: tq_cache_desc, dst: tq_cache_desc, src_blocks, dst_blocks, stream=None) -> None:
    n = src_blocks.numel()
    assert dst_blocks.numel() == n
    check(lib().tq_cache_copy_blocks(ctypes.byref(src), ctypes.byref(dst), _ptr(src_blocks), _ptr(dst_blocks), n,
                                     _stream(stream)), "tq_cache_copy_blocks")


def tq_prefill_workspace_bytes(desc: tq_cache_desc, batch: int, num_q_heads: int, q_len: int) -> int:
    out = ctypes.c_size_t()
    check(lib().tq_prefill_workspace_bytes(ctypes.byref(desc), batch, num_q_heads, q_len, ctypes.byref(out)),
          "tq_prefill_workspace_bytes")
    return out.value


def tq_prefill_attention(key_codec: int, value_codec: int, desc: tq_cache_desc, layer: int, q,
                         seq_lens, block_table, max_blocks: int, out, workspace, scale: float = 0.0,
                         stream=None) -> None:
    batch, hq, lq, _ = q.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    check(lib().tq_prefill_attention(key_codec, value_codec, ctypes.byref(desc), layer, _ptr(q),
                                     _dtype_code(q), batch, hq, lq, _ptr(seq_lens), _ptr(block_table),
                                     max_blocks, scale, _ptr(out), _ptr(workspace), ws_bytes,
                                     _stream(stream)), "tq_prefill_attention")


def tq_decode_attention_noalloc(key_codec: int, value_codec: int, desc: tq_cache_desc, layer: int, q,
                                seq_lens, block_table, max_blocks: int, max_seq_len: int, out,
                                scale: float = 0.0, stream=None) -> None:
    """tq_decode_attention with its scratch in the library's fixed device array
    (for callers that cannot allocate device memory); see include/tq.h."""
    batch, hq, lq, _ = q.shape
    check(lib().tq_decode_attention_noalloc(key_codec, value_codec, ctypes.byref(desc), layer, _ptr(q),
                                            _dtype_code(q), batch, hq, lq, _ptr(seq_lens),
                                            _ptr(block_table), max_blocks, max_seq_len, scale, _ptr(out),
                                            _stream(stream)), "tq_decode_attention_noalloc")


def tq_decode_partials(key_codec: int, value_codec: int, desc: tq_cache_desc, layer: int, q, seq_lens,
                       causal_end, block_table, max_blocks: int, max_seq_len: int, part_ml, part_acc, workspace,
                       scale: float = 0.0, stream=None) -> None:
    """Unnormalised softmax state of this shard of every sequence (see include/tq.h)."""
    batch, hq, lq, _ = q.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    check(lib().tq_decode_partials(key_codec, value_codec, ctypes.byref(desc), layer, _ptr(q), _dtype_code(q),
                                   batch, hq, lq, _ptr(seq_lens), _ptr(causal_end), _ptr(block_table), max_blocks,
                                   max_seq_len, scale, _ptr(part_ml), _ptr(part_acc), _ptr(workspace), ws_bytes,
                                   _stream(stream)), "tq_decode_partials")


def tq_decode_merge(value_codec: int, parts_ml, parts_acc, out, stream=None) -> None:
    """Log-sum-exp merge of shards' states: parts_ml [P, ..., 2], parts_acc [P, ..., D] -> out [..., D]."""
    P = parts_ml.shape[0]
    rows = parts_ml[0].numel() // 2
    check(lib().tq_decode_merge(value_codec, P, _ptr(parts_ml), _ptr(parts_acc), rows, _ptr(out),
                                _stream(stream)), "tq_decode_merge")


class SplitCache:
    """Split (low/high) states: the low coordinates [0, DL) of every key and value
    in one cache, the high coordinates [DL, D) in another, each under its own
    codec pair; both caches share one block layout."""

    def __init__(self, key_low: "Codec", value_low: "Codec", key_high: "Codec", value_high: "Codec",
                 num_layers: int, num_blocks: int, block_tokens: int, num_kv_heads: int, device="cuda",
                 exact_encode: bool = False):
        self.low = CompressedKVCache(key_low, value_low, num_layers, num_blocks, block_tokens, num_kv_heads,
                                     device, exact_encode)
        self.high = CompressedKVCache(key_high, value_high, num_layers, num_blocks, block_tokens, num_kv_heads,
                                      device, exact_encode)
        self.low_dim = key_low.info["head_dim"]
        self.head_dim = self.low_dim + key_high.info["head_dim"]

    def state(self) -> tq_split_state:
        return tq_split_state(self.low.key.handle, self.low.value.handle, self.high.key.handle,
                              self.high.value.handle, ctypes.pointer(self.low.desc), ctypes.pointer(self.high.desc))

    def append(self, layer, k_low, v_low, k_high, v_high, seq_lens, block_table=None, max_blocks=0, stream=None):
        tq_encode_append_split(self, layer, k_low, v_low, k_high, v_high, seq_lens, block_table, max_blocks, stream)

    def workspace_bytes(self, batch, num_q_heads, q_len, max_seq_len):
        return tq_decode_workspace_bytes_split(self, batch, num_q_heads, q_len, max_seq_len)

    def decode(self, layer, q, seq_lens, block_table, max_blocks, max_seq_len, out, workspace, scale=0.0,
               stream=None):
        tq_decode_attention_split(self, layer, q, seq_lens, block_table, max_blocks, max_seq_len, out, workspace,
                                  scale, stream)


def tq_encode_append_split(sc: SplitCache, layer: int, k_low, v_low, k_high, v_high, seq_lens, block_table=None,
                           max_blocks: int = 0, stream=None) -> None:
    batch, _, n_new, _ = k_low.shape
    st = sc.state()
    check(lib().tq_encode_append_split(ctypes.byref(st), layer, _ptr(k_low), _ptr(v_low), _ptr(k_high),
                                       _ptr(v_high), _dtype_code(k_low), batch, n_new, _ptr(seq_lens),
                                       _ptr(block_table), max_blocks, _stream(stream)), "tq_encode_append_split")


def tq_decode_workspace_bytes_split(sc: SplitCache, batch: int, num_q_heads: int, q_len: int, max_seq_len: int) -> int:
    out = ctypes.c_size_t()
    st = sc.state()
    check(lib().tq_decode_workspace_bytes_split(ctypes.byref(st), batch, num_q_heads, q_len, max_seq_len,
                                                ctypes.byref(out)), "tq_decode_workspace_bytes_split")
    return out.value


def tq_decode_attention_split(sc: SplitCache, layer: int, q, seq_lens, block_table, max_blocks: int,
                              max_seq_len: int, out, workspace, scale: float = 0.0, stream=None) -> None:
    batch, hq, lq, _ = q.shape
    st = sc.state()
    ws_bytes = workspace.numel() * workspace.element_size()
    check(lib().tq_decode_attention_split(ctypes.byref(st), layer, _ptr(q), _dtype_code(q), batch, hq, lq,
                                          _ptr(seq_lens), _ptr(block_table), max_blocks, max_seq_len, scale,
                                          _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)),
          "tq_decode_attention_split")


class Batch:
    """A batch of sequences in a paged cache: device block table [capacity][max_blocks]
    (-1 = no block) and sequence lengths [capacity], rows 0..batch-1 in use."""

    def __init__(self, cache: "CompressedKVCache", capacity: int, max_blocks: int, table=None, lens=None,
                 batch: int = 0):
        torch = _torch()
        dev = cache.pool.device
        self.cache = cache
        self.table = table if table is not None else torch.full((capacity, max_blocks), -1, dtype=torch.int32,
                                                                 device=dev)
        self.lens = lens if lens is not None else torch.zeros(capacity, dtype=torch.int32, device=dev)
        self.batch = batch
        assert self.table.shape == (capacity, max_blocks) and self.lens.shape == (capacity,)

    @property
    def capacity(self) -> int:
        return self.table.shape[0]

    @property
    def max_blocks(self) -> int:
        return self.table.shape[1]

    def view(self) -> tq_batch:
        return tq_batch(ctypes.pointer(self.cache.desc), _ptr(self.table), _ptr(self.lens), self.batch,
                        self.capacity, self.max_blocks)


def tq_batch_filter(batch: Batch, keep, out: Batch, freed, n_freed, stream=None) -> None:
    """Rows `keep` (host list) of `batch` become rows 0.. of `out` (same pool); the block ids of the
    other rows go to `freed` (device int32) and their count to n_freed (device int32 [1])."""
    keep_arr = (ctypes.c_int32 * max(1, len(keep)))(*[int(i) for i in keep])
    src, dst = batch.view(), out.view()
    check(lib().tq_batch_filter(ctypes.byref(src), keep_arr, len(keep), ctypes.byref(dst), _ptr(freed),
                                _ptr(n_freed), _stream(stream)), "tq_batch_filter")
    out.batch = dst.batch


def tq_batch_extend(dst: Batch, src: Batch, free_blocks=None, n_used=None, stream=None) -> None:
    """Append the sequences of `src` to `dst`, copying their blocks into dst's free blocks
    (free_blocks device int32, consumed from n_used[0]) unless both share a pool."""
    d, s_ = dst.view(), src.view()
    n_free = 0 if free_blocks is None else free_blocks.numel()
    check(lib().tq_batch_extend(ctypes.byref(d), ctypes.byref(s_), _ptr(free_blocks), n_free, _ptr(n_used),
                                _stream(stream)), "tq_batch_extend")
    dst.batch = d.batch


def tq_batch_merge(dst: Batch, srcs, free_blocks=None, n_used=None, stream=None) -> None:
    """tq_batch_extend of `dst` by each of `srcs` in order (one guard over all of them first)."""
    d = dst.view()
    arr = (tq_batch * max(1, len(srcs)))(*[b.view() for b in srcs])
    n_free = 0 if free_blocks is None else free_blocks.numel()
    check(lib().tq_batch_merge(ctypes.byref(d), arr, len(srcs), _ptr(free_blocks), n_free, _ptr(n_used),
                               _stream(stream)), "tq_batch_merge")
    dst.batch = d.batch


def tq_batch_extract(src: Batch, idx: int, dst: Batch, free_blocks=None, n_used=None, stream=None) -> None:
    """Sequence idx of `src` becomes the only sequence of `dst`."""
    s_, d = src.view(), dst.view()
    n_free = 0 if free_blocks is None else free_blocks.numel()
    check(lib().tq_batch_extract(ctypes.byref(s_), idx, ctypes.byref(d), _ptr(free_blocks), n_free,
                                 _ptr(n_used), _stream(stream)), "tq_batch_extract")
    dst.batch = d.batch


def tq_device_error() -> int:
    flags = ctypes.c_uint32()
    st = lib().tq_device_error(ctypes.byref(flags))
    if st not in (TQ_OK, 7):
        check(st, "tq_device_error")
    return flags.value


def tq_selftest_wait_timeout(seconds: float, stream=None) -> None:
    check(lib().tq_selftest_wait_timeout(float(seconds), _stream(stream)), "tq_selftest_wait_timeout")


# ----------------------------------------------------------------- helpers

class Codec:
    """Owns one codec handle."""

    def __init__(self, head_dim: int, bits: int, mode: int, seed: int = 0, group: int = 0,
                 _handle: int = 0):
        if _handle:
            self.handle = _handle
        elif mode == TQ_MODE_GROUP:
            self.handle = tq_codec_create_group(head_dim, bits, group)
        else:
            self.handle = tq_codec_create(head_dim, bits, mode, seed)
        self.info = tq_codec_info(self.handle)

    @classmethod
    def pair_for_bits(cls, head_dim: int, bits: float, seed: int = 0) -> tuple:
        """(key codec, value codec) for a possibly fractional bit width: MSE
        codecs of floor(bits) and ceil(bits) bits, seeds seed and seed + 1."""
        kh, vh = tq_codec_pair_for_bits(head_dim, bits, seed)
        return cls(0, 0, 0, _handle=kh), cls(0, 0, 0, _handle=vh)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            try:
                tq_codec_destroy(h)
            except Exception:
                pass
            self.handle = None

    @property
    def record_bytes(self) -> int:
        return self.info["record_bytes"]

    def export(self):
        return tq_codec_export(self.handle)


class CompressedKVCache:
    """A device pool plus its descriptor (all layers), allocated through torch."""

    def __init__(self, key: Codec, value: Codec, num_layers: int, num_blocks: int,
                 block_tokens: int, num_kv_heads: int, device="cuda", exact_encode: bool = False):
        torch = _torch()
        self.key, self.value = key, value
        _, req = tq_cache_desc_init(key.handle, value.handle, num_layers, num_blocks, block_tokens,
                                    num_kv_heads, None)
        self.pool = torch.zeros(req, dtype=torch.uint8, device=device)
        self.desc, _ = tq_cache_desc_init(key.handle, value.handle, num_layers, num_blocks,
                                          block_tokens, num_kv_heads, self.pool)
        # TQ_ENCODE_EXACT: every append in the sequential fp32 order; AUTO lets
        # long appends rotate on the tensor cores
        self.desc.encode_policy = TQ_ENCODE_EXACT if exact_encode else TQ_ENCODE_AUTO
        self.num_layers, self.num_blocks = num_layers, num_blocks
        self.block_tokens, self.num_kv_heads = block_tokens, num_kv_heads

    @property
    def nbytes(self) -> int:
        return self.pool.numel()

    def append(self, layer, k, v, seq_lens, block_table=None, max_blocks=0, stream=None):
        tq_encode_append(self.key.handle, self.value.handle, self.desc, layer, k, v, seq_lens,
                         block_table, max_blocks, stream)

    def workspace_bytes(self, batch, num_q_heads, q_len, max_seq_len):
        return tq_decode_workspace_bytes(self.desc, batch, num_q_heads, q_len, max_seq_len)

    def copy_blocks_from(self, src: "CompressedKVCache", src_blocks, dst_blocks, stream=None):
        """Blocks src_blocks of `src` (every layer) become blocks dst_blocks of this cache."""
        tq_cache_copy_blocks(src.desc, self.desc, src_blocks, dst_blocks, stream)

    def prefill_workspace_bytes(self, batch, num_q_heads, q_len):
        return tq_prefill_workspace_bytes(self.desc, batch, num_q_heads, q_len)

    def prefill_attention(self, layer, q, seq_lens, block_table, max_blocks, out, workspace, scale=0.0,
                          stream=None):
        tq_prefill_attention(self.key.handle, self.value.handle, self.desc, layer, q, seq_lens, block_table,
                             max_blocks, out, workspace, scale, stream)

    def decode(self, layer, q, seq_lens, block_table, max_blocks, max_seq_len, out, workspace,
               scale=0.0, stream=None):
        tq_decode_attention(self.key.handle, self.value.handle, self.desc, layer, q, seq_lens,
                            block_table, max_blocks, max_seq_len, out, workspace, scale, stream)

    def decode_partials(self, layer, q, seq_lens, causal_end, block_table, max_blocks, max_seq_len, part_ml,
                        part_acc, workspace, scale=0.0, stream=None):
        """This cache holds one shard of each sequence: its unnormalised softmax state."""
        tq_decode_partials(self.key.handle, self.value.handle, self.desc, layer, q, seq_lens, causal_end,
                           block_table, max_blocks, max_seq_len, part_ml, part_acc, workspace, scale, stream)

    def decode_step(self, layer, k_new, v_new, q, seq_lens, block_table, max_blocks, max_seq_len, out,
                    workspace, scale=0.0, stream=None):
        """Append the step's tokens at seq_lens (lengths before the step) and decode, in one call."""
        tq_decode_step(self.key.handle, self.value.handle, self.desc, layer, k_new, v_new, q, seq_lens,
                       block_table, max_blocks, max_seq_len, out, workspace, scale, stream)


# ----------------------------------------------------------------- 8-bit cache

class _KV8:
    """What the calls below need of torch and the library, looked up once (they are short: every lookup counts)."""

    def __init__(self):
        torch = _torch()
        self.empty, self.zeros = torch.empty, torch.zeros
        self.codes = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}
        self.i32, self.f32 = torch.int32, torch.float32
        self.device = torch._C._cuda_getDevice                # of torch.cuda.current_device
        self.stream = torch._C._cuda_getCurrentRawStream      # of torch.cuda.current_stream(device).cuda_stream
        self.append, self.attention = lib().tq_kv8_append, lib().tq_kv8_attention
        self.rope, self.verify = lib().tq_rope_apply, lib().tq_verify_drafts
        self.reserve, self.release = lib().tq_blocks_reserve, lib().tq_blocks_release


_kv8_found = None


def _kv8() -> _KV8:
    global _kv8_found
    if _kv8_found is None:
        _kv8_found = _KV8()
    return _kv8_found


def _raw_stream(t, stream, device) -> int:
    if stream is None:
        return t.stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


_pack_rows = struct.Struct("@Pqqq").pack                 # tq_rows
_pack_scores = struct.Struct("@ffPiPPPP").pack           # tq_kv8_scores


def _on(stream):
    """Allocations and fills on the stream that a call names (None: the current one)."""
    cuda = _torch().cuda
    if stream is not None and not isinstance(stream, cuda.Stream):
        stream = cuda.ExternalStream(stream if isinstance(stream, int) else stream.cuda_stream)
    return cuda.stream(stream)


def _rows(t, name, dtype, device, batch, heads, tokens, dim) -> bytes:
    """tq_rows of a [batch, heads, tokens, head_dim] view, in whatever order its first three axes lie."""
    if t.shape != (batch, heads, tokens, dim):
        raise ValueError(f"{name} must be [batch, heads, tokens, head_dim] = {(batch, heads, tokens, dim)}, not {tuple(t.shape)}")
    if t.dtype != dtype or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} on cuda:{device}, not {t.dtype} on {t.device}")
    sb, sh, st, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the coordinates of a head must be contiguous")
    # the stride of an axis of one element says nothing, whatever it is
    return _pack_rows(t.data_ptr(), sb if batch > 1 else 0, sh if heads > 1 else 0, st if tokens > 1 else 0)


def _array(t, name, dtype, device, shape) -> Optional[int]:
    """Pointer of a small contiguous argument (lengths, tables, slopes), or None."""
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on cuda:{device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


class Rope:
    """Position rotation: pair i of a head's first ``2 * len(inv_freq)`` coordinates turns by position * inv_freq[i].

    ``inv_freq`` is a float64 device tensor, kept by this object; pairs are coordinates (i, i + rot_dim / 2), or
    (2i, 2i + 1) with ``interleaved``; ``scale`` multiplies the rotated coordinates.
    """

    def __init__(self, inv_freq, interleaved: bool = False, scale: float = 1.0):
        torch = _torch()
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous() or not inv_freq.is_cuda:
            raise ValueError("inv_freq must be a contiguous one-dimensional float64 tensor on a CUDA device")
        if not scale:
            raise ValueError("scale must not be 0")
        self.inv_freq = inv_freq
        self.device = inv_freq.get_device()
        self.desc = tq_rope(inv_freq.data_ptr(), 2 * inv_freq.numel(), int(interleaved), scale)
        self.address = ctypes.addressof(self.desc)

    @classmethod
    def of_base(cls, rot_dim: int, base: float = 10000.0, device="cuda", interleaved: bool = False, scale: float = 1.0):
        """inv_freq[i] = base ** (-2 i / rot_dim)."""
        return cls(cls._frequencies(rot_dim, base, device), interleaved, scale)

    # Forms for contexts longer than the trained one, as frequencies of their own.

    @classmethod
    def linear(cls, rot_dim: int, factor: float, base: float = 10000.0, device="cuda", interleaved: bool = False,
               scale: float = 1.0):
        """Positions divided by `factor`."""
        return cls(cls._frequencies(rot_dim, base, device) / factor, interleaved, scale)

    @classmethod
    def ntk(cls, rot_dim: int, factor: float, base: float = 10000.0, device="cuda", interleaved: bool = False,
            scale: float = 1.0):
        """The base times factor ** (rot_dim / (rot_dim - 2)): the slowest pair turns `factor` times slower, the fastest as before."""
        if rot_dim <= 2:
            raise ValueError("rot_dim must be above 2")
        return cls(cls._frequencies(rot_dim, base * factor ** (rot_dim / (rot_dim - 2)), device), interleaved, scale)

    @classmethod
    def by_parts(cls, rot_dim: int, factor: float, original: int, low: float = 1.0, high: float = 32.0,
                 base: float = 10000.0, device="cuda", interleaved: bool = False, scale: float = 1.0):
        """Pairs that turn fewer than `low` times over the `original` trained positions turn `factor` times slower, those
        above `high` turns as before, those between by a ramp in their turns. `scale`: with these defaults usually
        1 + 0.1 ln(factor)."""
        if not low < high:
            raise ValueError("low must be below high")
        f = cls._frequencies(rot_dim, base, device)
        ramp = ((original / (2 * np.pi) * f - low) / (high - low)).clamp(0, 1)
        return cls(f * ((1 - ramp) / factor + ramp), interleaved, scale)

    @staticmethod
    def _frequencies(rot_dim, base, device):
        torch = _torch()
        i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
        return base ** (-i / rot_dim)

    def apply(self, q, k=None, out=None, k_out=None, starts=None, positions=None, new_lens=None, transposed=False,
              stream=None):
        return tq_rope_apply(self, q, k, out, k_out, starts, positions, new_lens, transposed, stream)


def tq_kv8_append(cache: "KV8Cache", layer, k, v, seq_lens, block_table=None, max_blocks=0, new_lens=None, rope=None,
                  positions=None, stream=None):
    """Append k, v [batch, kv heads, n_new, head_dim] (views in any order of the first three axes) at seq_lens."""
    t, device = _kv8(), cache.index
    if t.device() != device:
        with _torch().cuda.device(device):
            return tq_kv8_append(cache, layer, k, v, seq_lens, block_table, max_blocks, new_lens, rope, positions, stream)
    if k.dim() != 4:
        raise ValueError("k must be [batch, heads, tokens, head_dim]")
    batch, _, n_new, _ = k.shape
    dtype, i32, heads, dim = k.dtype, t.i32, cache.num_kv_heads, cache.head_dim
    code = t.codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    if rope is not None and rope.device != device:
        raise ValueError(f"rope must be on cuda:{device}")
    per = (batch,)
    status = t.append(
        cache.ref, layer, _rows(k, "k", dtype, device, batch, heads, n_new, dim),
        _rows(v, "v", dtype, device, batch, heads, n_new, dim), code, batch, n_new,
        _array(seq_lens, "seq_lens", i32, device, per), _array(new_lens, "new_lens", i32, device, per),
        _array(block_table, "block_table", i32, device, (batch, max_blocks)), max_blocks,
        rope.address if rope is not None else None, _array(positions, "positions", i32, device, (batch, n_new)),
        _raw_stream(t, stream, device))
    if status:
        check(status, "tq_kv8_append")


def tq_kv8_workspace_bytes(cache: "KV8Cache", batch, num_q_heads, q_len, max_seq_len) -> int:
    n = ctypes.c_size_t()
    with _torch().cuda.device(cache.index):
        check(lib().tq_kv8_workspace_bytes(cache.ref, batch, num_q_heads, q_len, max_seq_len, ctypes.byref(n)),
              "tq_kv8_workspace_bytes")
    return n.value


def tq_kv8_attention(cache: "KV8Cache", layer, q, seq_lens, block_table=None, max_blocks=0, max_seq_len=0, out=None,
                     workspace=None, q_lens=None, scale=0.0, softcap=0.0, slopes=None, window=0, prefix_lens=None,
                     doc_starts=None, rope=None, positions=None, stream=None):
    """Attention of q [batch, query heads, q_len, head_dim] over the cache; returns out (like q if None).

    Without `out`, rows behind q_lens are zero. An output and a workspace that are not given are made on `stream`, and
    belong to it in torch's allocator.
    """
    t, device = _kv8(), cache.index
    if t.device() != device:
        with _torch().cuda.device(device):
            return tq_kv8_attention(cache, layer, q, seq_lens, block_table, max_blocks, max_seq_len, out, workspace,
                                    q_lens, scale, softcap, slopes, window, prefix_lens, doc_starts, rope, positions,
                                    stream)
    if q.dim() != 4:
        raise ValueError("q must be [batch, heads, tokens, head_dim]")
    batch, heads, q_len, _ = q.shape
    dtype, i32, dim = q.dtype, t.i32, cache.head_dim
    code = t.codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    qr = _rows(q, "q", dtype, device, batch, heads, q_len, dim)
    if out is None:
        with _on(stream):
            out = _torch().empty_like(q) if q_lens is None else _torch().zeros_like(q)
    if rope is not None and rope.device != device:
        raise ValueError(f"rope must be on cuda:{device}")
    per, each, sc = (batch,), (batch, q_len), None
    if rope is not None or scale or softcap or window or slopes is not None or prefix_lens is not None or doc_starts is not None:
        sc = _pack_scores(scale, softcap, _array(slopes, "slopes", t.f32, device, (heads,)) or 0, window,
                          _array(prefix_lens, "prefix_lens", i32, device, per) or 0,
                          _array(doc_starts, "doc_starts", i32, device, each) or 0,
                          rope.address if rope is not None else 0,
                          _array(positions, "positions", i32, device, each) or 0)
    if workspace is None:
        n = tq_kv8_workspace_bytes(cache, batch, heads, q_len, max_seq_len)
        if n:
            with _on(stream):
                workspace = _torch().empty(n, dtype=_torch().uint8, device=cache.device)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{device}")
    status = t.attention(
        cache.ref, layer, qr, code, batch, heads, q_len, _array(seq_lens, "seq_lens", i32, device, per),
        _array(q_lens, "q_lens", i32, device, per),
        _array(block_table, "block_table", i32, device, (batch, max_blocks)), max_blocks, max_seq_len, sc,
        _rows(out, "out", dtype, device, batch, heads, q_len, dim),
        workspace.data_ptr() if workspace is not None else None, workspace.nbytes if workspace is not None else 0,
        _raw_stream(t, stream, device))
    if status:
        check(status, "tq_kv8_attention")
    return out


class KV8Cache:
    """A paged 8-bit cache: codes [layer, block, kv head, token, head_dim], scale bytes [layer, block, kv head]."""

    def __init__(self, num_layers: int, num_blocks: int, block_tokens: int, num_kv_heads: int, head_dim: int,
                 format: int = TQ_KV8_E4M3, device="cuda"):
        torch = _torch()
        codes = (num_layers, num_blocks, num_kv_heads, block_tokens, head_dim)
        self._set(*(torch.zeros(codes, dtype=torch.uint8, device=device) for _ in "kv"),
                  *(torch.full(codes[:3], 127, dtype=torch.uint8, device=device) for _ in "kv"), format)

    @classmethod
    def wrap(cls, k_codes, v_codes, k_scales, v_scales, format: int = TQ_KV8_E4M3) -> "KV8Cache":
        """A cache over tensors of the caller's (uint8; without the layer axis: one layer). Scale bytes in [64, 190], and
        no NaN codes among the tokens that attention is to see."""
        self = cls.__new__(cls)
        if k_codes.dim() == 4:
            k_codes, v_codes, k_scales, v_scales = (t.unsqueeze(0) for t in (k_codes, v_codes, k_scales, v_scales))
        self._set(k_codes, v_codes, k_scales, v_scales, format)
        return self

    def _set(self, k_codes, v_codes, k_scales, v_scales, format):
        torch = _torch()
        if k_codes.dim() != 5 or v_codes.shape != k_codes.shape or k_scales.shape != k_codes.shape[:3] \
                or v_scales.shape != k_scales.shape:
            raise ValueError("codes must be [layers, blocks, kv heads, tokens, head_dim], scales [layers, blocks, kv heads]")
        for t in (k_codes, v_codes, k_scales, v_scales):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.device != k_codes.device or not t.is_cuda:
                raise ValueError("codes and scales must be contiguous uint8 tensors on one CUDA device")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.num_layers, self.num_blocks, self.num_kv_heads, self.block_tokens, self.head_dim = k_codes.shape
        self.format = format
        self.device, self.index = k_codes.device, k_codes.get_device()
        self.desc = tq_kv8_cache(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                 k_codes.stride(0), k_scales.stride(0), self.num_layers, self.num_blocks,
                                 self.block_tokens, self.num_kv_heads, self.head_dim, format)
        self.ref = ctypes.byref(self.desc)

    @property
    def nbytes(self) -> int:
        return 2 * (self.k_codes.numel() + self.k_scales.numel())

    def append(self, layer, k, v, seq_lens, block_table=None, max_blocks=0, new_lens=None, rope=None, positions=None,
               stream=None):
        tq_kv8_append(self, layer, k, v, seq_lens, block_table, max_blocks, new_lens, rope, positions, stream)

    def workspace_bytes(self, batch, num_q_heads, q_len, max_seq_len):
        return tq_kv8_workspace_bytes(self, batch, num_q_heads, q_len, max_seq_len)

    def attention(self, layer, q, seq_lens, block_table=None, max_blocks=0, max_seq_len=0, out=None, workspace=None,
                  q_lens=None, scale=0.0, softcap=0.0, slopes=None, window=0, prefix_lens=None, doc_starts=None,
                  rope=None, positions=None, stream=None):
        return tq_kv8_attention(self, layer, q, seq_lens, block_table, max_blocks, max_seq_len, out, workspace, q_lens,
                                scale, softcap, slopes, window, prefix_lens, doc_starts, rope, positions, stream)


# ----------------------------------------------------------------- around the caches' calls

_here = contextlib.nullcontext()   # the current stream, at once
_pack_drafts = struct.Struct("@PqqPqqPPPPPqPiii4x").pack   # tq_drafts


def tq_rope_apply(rope: Rope, q, k=None, out=None, k_out=None, starts=None, positions=None, new_lens=None,
                  transposed=False, stream=None):
    """q, k [batch, heads, n, head_dim] (views in any order of the first three axes) turned by `rope`: (out, k_out).

    Token i of sequence b is at positions[b, i], or starts[b] + i, or i. An output may be its input; one that is not given
    is made on `stream`, contiguous, rows behind new_lens zero. `transposed`: by the opposite angle (the gradient).
    """
    t, device = _kv8(), rope.device
    if t.device() != device:
        with _torch().cuda.device(device):
            return tq_rope_apply(rope, q, k, out, k_out, starts, positions, new_lens, transposed, stream)
    if q.dim() != 4:
        raise ValueError("q must be [batch, heads, tokens, head_dim]")
    batch, heads, n, dim = q.shape
    dtype, i32 = q.dtype, t.i32
    code = t.codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    qr = _rows(q, "q", dtype, device, batch, heads, n, dim)
    kr = ko = None
    k_heads = 0
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must be [batch, heads, tokens, head_dim]")
        k_heads = k.shape[1]
        kr = _rows(k, "k", dtype, device, batch, k_heads, n, dim)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if out is None or (k is not None and k_out is None):
        make = t.empty if new_lens is None else t.zeros
        with _on(stream) if stream is not None else _here:
            if out is None:
                out = make(q.shape, dtype=dtype, device=q.device)
            if k is not None and k_out is None:
                k_out = make(k.shape, dtype=dtype, device=q.device)
    if k is not None:
        ko = _rows(k_out, "k_out", dtype, device, batch, k_heads, n, dim)
    per = (batch,)
    status = t.rope(
        rope.address, int(transposed), code, dim, batch, n, qr, heads, _rows(out, "out", dtype, device, batch, heads, n, dim),
        kr, k_heads, ko, _array(starts, "starts", i32, device, per), _array(new_lens, "new_lens", i32, device, per),
        _array(positions, "positions", i32, device, (batch, n)), _raw_stream(t, stream, device))
    if status:
        check(status, "tq_rope_apply")
    return out, k_out


class Places:
    """Where the tokens of a reservation lie: per sequence granted [batch] and starts [batch + 1], per packed token
    seq_ids, positions and slots [max_tokens] (max_tokens = 0: no maps)."""

    def __init__(self, batch: int, max_tokens: int = 0, device="cuda"):
        torch = _torch()
        self.granted = torch.zeros(batch, dtype=torch.int32, device=device)
        self.starts = torch.zeros(batch + 1, dtype=torch.int32, device=device)
        self.seq_ids = torch.full((max_tokens,), -1, dtype=torch.int32, device=device)
        self.positions = torch.zeros(max_tokens, dtype=torch.int32, device=device)
        self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=device)
        self.batch, self.max_tokens, self.index = batch, max_tokens, self.granted.get_device()
        maps = (self.seq_ids.data_ptr(), self.positions.data_ptr(), self.slots.data_ptr()) if max_tokens else (None,) * 3
        self.desc = tq_places(self.granted.data_ptr(), self.starts.data_ptr(), *maps, max_tokens)
        self.address = ctypes.addressof(self.desc)


class BlockTable:
    """Rows of block ids (-1 = no block) and the free list of the blocks that no row holds, on the device.

    `table` [rows, max_blocks] goes into the caches' calls; `free_blocks` and `n_used` into tq_batch_extend, tq_batch_merge
    and tq_batch_extract, which take from the same list.
    """

    def __init__(self, rows: int, max_blocks: int, num_blocks: int, block_tokens: int, device="cuda"):
        torch = _torch()
        self._set(torch.full((rows, max_blocks), -1, dtype=torch.int32, device=device),
                  torch.arange(num_blocks, dtype=torch.int32, device=device), torch.zeros(1, dtype=torch.int32, device=device),
                  block_tokens, num_blocks)

    @classmethod
    def wrap(cls, table, free_blocks, n_used, block_tokens: int, num_blocks: int) -> "BlockTable":
        """A table and a free list of the caller's (int32): free_blocks[n_used[0]:] are free."""
        self = cls.__new__(cls)
        self._set(table, free_blocks, n_used, block_tokens, num_blocks)
        return self

    def _set(self, table, free_blocks, n_used, block_tokens, num_blocks):
        i32 = _torch().int32
        if table.dim() != 2 or free_blocks.dim() != 1 or n_used.shape != (1,):
            raise ValueError("table must be [rows, max_blocks], free_blocks one-dimensional, n_used of one element")
        for t in (table, free_blocks, n_used):
            if t.dtype != i32 or not t.is_contiguous() or t.device != table.device or not t.is_cuda:
                raise ValueError("table, free_blocks and n_used must be contiguous int32 tensors on one CUDA device")
        self.table, self.free_blocks, self.n_used = table, free_blocks, n_used
        self.rows, self.max_blocks = table.shape
        self.block_tokens, self.num_blocks = block_tokens, num_blocks
        self.device, self.index = table.device, table.get_device()
        self.desc = tq_blocks(table.data_ptr(), free_blocks.data_ptr(), n_used.data_ptr(), free_blocks.numel(),
                              self.max_blocks, block_tokens, num_blocks)
        self.address = ctypes.addressof(self.desc)

    def batch(self, cache: "CompressedKVCache", lens, batch: int) -> Batch:
        """The first `batch` rows, with lengths `lens` [rows], as the batch calls take them."""
        return Batch(cache, self.rows, self.max_blocks, table=self.table, lens=lens, batch=batch)

    def reserve(self, seq_lens, new_lens=None, n_new: int = 1, places: Optional[Places] = None, stream=None):
        tq_blocks_reserve(self, seq_lens, new_lens, n_new, places, stream)

    def release(self, keep_lens, stream=None):
        tq_blocks_release(self, keep_lens, stream)


def _rows_in_use(blocks: BlockTable, lens, name):
    if lens.dim() != 1 or lens.shape[0] > blocks.rows:
        raise ValueError(f"{name} must be one-dimensional, of at most {blocks.rows} rows")
    return lens.shape[0]


def tq_blocks_reserve(blocks: BlockTable, seq_lens, new_lens=None, n_new: int = 1, places: Optional[Places] = None,
                      stream=None) -> None:
    """Blocks for new_lens[b] <= n_new tokens (None: n_new each) behind seq_lens[b], and where the tokens lie (see include/tq.h)."""
    t, device = _kv8(), blocks.index
    if t.device() != device:
        with _torch().cuda.device(device):
            return tq_blocks_reserve(blocks, seq_lens, new_lens, n_new, places, stream)
    batch = _rows_in_use(blocks, seq_lens, "seq_lens")
    if places is not None and (places.batch != batch or places.index != device):
        raise ValueError(f"places must be of {batch} sequences on cuda:{device}")
    per = (batch,)
    status = t.reserve(blocks.address, batch, _array(seq_lens, "seq_lens", t.i32, device, per),
                       _array(new_lens, "new_lens", t.i32, device, per), n_new,
                       places.address if places is not None else None, _raw_stream(t, stream, device))
    if status:
        check(status, "tq_blocks_reserve")


def tq_blocks_release(blocks: BlockTable, keep_lens, stream=None) -> None:
    """Blocks behind the first keep_lens[b] tokens of each row back to the free list."""
    t, device = _kv8(), blocks.index
    if t.device() != device:
        with _torch().cuda.device(device):
            return tq_blocks_release(blocks, keep_lens, stream)
    batch = _rows_in_use(blocks, keep_lens, "keep_lens")
    status = t.release(blocks.address, batch, _array(keep_lens, "keep_lens", t.i32, device, (batch,)), _raw_stream(t, stream, device))
    if status:
        check(status, "tq_blocks_release")


class Verified(NamedTuple):
    """accepted [batch], tokens and logprobs [batch, drafts + 1], keep_lens [batch] (None without seq_lens)."""
    accepted: object
    tokens: object
    keep_lens: object
    logprobs: object


def _row_strides(x, name, device, shape):
    if x.shape != shape or x.get_device() != device or (shape[-1] > 1 and x.stride(-1) != 1):
        raise ValueError(f"{name} must be {shape} on cuda:{device} with contiguous rows, not {tuple(x.shape)} on {x.device}")
    return x.stride()[:-1]


def tq_verify_drafts(target, draft_tokens=None, draft_probs=None, uniforms=None, noise=None, temperatures=None,
                     draft_lens=None, seq_lens=None, target_probs=False, out: Optional[Verified] = None, stream=None) -> Verified:
    """Which of draft_tokens [batch, drafts] stand against target [batch, drafts + 1, vocab] (logits, or probabilities with
    target_probs), and the token behind them (see include/tq.h). Without draft_tokens: one token of each row target[:, 0].

    draft_probs [batch, drafts, vocab]: what the drafts were drawn from (None: they were not); uniforms [batch, drafts] in
    [0, 1), noise [batch, vocab] exponential; without noise the tokens are the likeliest. What is returned is made on `stream`.
    """
    t = _kv8()
    if target.dim() != 3 or not target.is_cuda:
        raise ValueError("target must be [batch, drafts + 1, vocab] on a CUDA device")
    device = target.get_device()
    if t.device() != device:
        with _torch().cuda.device(device):
            return tq_verify_drafts(target, draft_tokens, draft_probs, uniforms, noise, temperatures, draft_lens, seq_lens,
                                    target_probs, out, stream)
    batch, rows, vocab = target.shape
    drafts = rows - 1
    if drafts < 0 or (drafts > 0 and draft_tokens is None):
        raise ValueError("target must have a row behind the last draft, and drafts their tokens")
    i32, f32 = t.i32, t.f32
    code = t.codes.get(target.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {target.dtype}")
    tb, tr = _row_strides(target, "target", device, (batch, rows, vocab))
    db = dr = nb = draft = dcode = 0
    if draft_probs is not None and drafts:
        db, dr = _row_strides(draft_probs, "draft_probs", device, (batch, drafts, vocab))
        dcode = t.codes.get(draft_probs.dtype)
        if dcode is None:
            raise TypeError(f"unsupported dtype {draft_probs.dtype}")
        draft = draft_probs.data_ptr()
    if noise is not None:
        nb, = _row_strides(noise, "noise", device, (batch, vocab))
        if noise.dtype != f32:
            raise TypeError(f"noise must be float32, not {noise.dtype}")
    per, each, full = (batch,), (batch, drafts), (batch, rows)
    if out is None:
        make, on = t.empty, target.device
        with _on(stream) if stream is not None else _here:
            out = Verified(make(per, dtype=i32, device=on), make(full, dtype=i32, device=on),
                           make(per, dtype=i32, device=on) if seq_lens is not None else None, make(full, dtype=f32, device=on))
        to = (out.accepted.data_ptr(), out.tokens.data_ptr(), out.logprobs.data_ptr(), out.keep_lens.data_ptr() if seq_lens is not None else None)
    else:
        if (seq_lens is None) != (out.keep_lens is None):
            raise ValueError("keep_lens go with seq_lens")
        to = (_array(out.accepted, "accepted", i32, device, per), _array(out.tokens, "tokens", i32, device, full),
              _array(out.logprobs, "logprobs", f32, device, full), _array(out.keep_lens, "keep_lens", i32, device, per))
    packed = _pack_drafts(
        target.data_ptr(), tb, tr, draft, db, dr, (_array(draft_tokens, "draft_tokens", i32, device, each) or 0) if drafts else 0,
        _array(draft_lens, "draft_lens", i32, device, per) or 0, _array(temperatures, "temperatures", f32, device, per) or 0,
        (_array(uniforms, "uniforms", f32, device, each) or 0) if drafts else 0, noise.data_ptr() if noise is not None else 0, nb,
        _array(seq_lens, "seq_lens", i32, device, per) or 0, code, dcode, int(target_probs))
    status = t.verify(packed, batch, drafts, vocab, *to, _raw_stream(t, stream, device))
    if status:
        check(status, "tq_verify_drafts")
    return out
