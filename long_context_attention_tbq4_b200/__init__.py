"""TBQ4 long-context attention on NVIDIA B200 (sm_100a).

A thin binding over libtbq4.so (include/tbq4.h): every function here only
checks and marshals torch tensors (device memory, current stream) and calls
the C ABI of the same name; all arithmetic runs in the library's CUDA
kernels.  There is no CPU path.

TBQ4 stores 128 values in 66 bytes (2-byte scale + 64 bytes of 4-bit
indices) in a Hadamard-rotated domain, and attention dequantises the raw
blocks inside its inner loop (trefon.com, "Kontekst 262K na jednej RTX 4090:
co dodalem do llama.cpp-turboq", section "Od czego zaczalem").
"""
import contextlib
import ctypes as C

import numpy as np
import torch

from ._lib import LIB_PATH, STATUS_NAMES, Tbq4Error, check, lib

D = 128
BLOCK_BYTES = 66

__all__ = [
    "D", "BLOCK_BYTES", "LIB_PATH", "Tbq4Error", "tbq4_block_bytes",
    "tbq4_cache_bytes", "tbq4_signs", "tbq4_quantize_append",
    "tbq4_decode_workspace_bytes", "tbq4_attn_decode", "tbq4_attn_decode_append",
    "tbq4_decode_mq_workspace_bytes", "tbq4_attn_decode_mq",
    "tbq4_prefill_workspace_bytes", "tbq4_attn_prefill_chunk",
    "tbq4_set_timing_events", "tbq4_get_device_status", "tbq4_selftest_bounded_wait",
    "empty_cache",
    "empty_pool", "tbq4_quantize_append_paged", "tbq4_attn_decode_paged",
    "BLOCK_BYTES3", "empty_cache3", "tbq3_quantize_append", "tbq3_attn_decode",
    "tbq4_rope_append", "tbq4_rope_append_paged", "tree_mask", "tbq4_tree_workspace_bytes",
    "tbq4_attn_tree", "tbq4_attn_tree_paged", "tbq4_tree_accept", "tbq4_tree_accept_paged",
]


def _ptr(t):
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _need(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


def tbq4_block_bytes() -> int:
    return int(lib.tbq4_block_bytes())


def tbq4_cache_bytes(batch: int, n_kv_heads: int, capacity: int) -> int:
    return int(lib.tbq4_cache_bytes(batch, n_kv_heads, capacity))


def tbq4_signs(seed: int) -> np.ndarray:
    out = np.zeros(D, np.int8)
    lib.tbq4_signs(C.c_uint64(seed), out.ctypes.data_as(C.c_void_p))
    return out


def empty_cache(batch, n_kv_heads, capacity, device="cuda"):
    """An uninitialised [B][Hkv][capacity][66] uint8 cache (capacity % 8 == 0)."""
    return torch.empty((batch, n_kv_heads, capacity, BLOCK_BYTES), dtype=torch.uint8,
                       device=device)


def tbq4_quantize_append(src, start_pos, cache, sign_seed=0, stream=None):
    """src fp32 [B][n_new][Hkv][128]; start_pos int32 [B]; cache uint8
    [B][Hkv][capacity][66] (written in place)."""
    _need(src, torch.float32, "src", 4)
    _need(start_pos, torch.int32, "start_pos", 1)
    _need(cache, torch.uint8, "cache", 4)
    B, n_new, Hkv, d = src.shape
    if d != D or tuple(cache.shape[:2]) != (B, Hkv) or cache.shape[3] != BLOCK_BYTES:
        raise ValueError("shape mismatch between src and cache")
    check(lib.tbq4_quantize_append(_ptr(src), B, n_new, Hkv, _ptr(start_pos),
                                   cache.shape[2], C.c_uint64(sign_seed), _ptr(cache),
                                   _stream(stream)), "tbq4_quantize_append")
    return cache


def tbq4_decode_workspace_bytes(B, Hq, Hkv, max_len, split_tokens=0) -> int:
    return int(lib.tbq4_decode_workspace_bytes_split(B, Hq, Hkv, max_len, split_tokens))


def tbq4_attn_decode(q, k_cache, v_cache, seq_lens, max_len, softmax_scale,
                     sign_seed=0, workspace=None, out=None, split_tokens=0,
                     stream=None):
    """q fp32 [B][Hq][128]; caches uint8 [B][Hkv][capacity][66]; seq_lens
    int32 [B] (device); returns fp16 [B][Hq][128]."""
    _need(q, torch.float32, "q", 3)
    _need(k_cache, torch.uint8, "k_cache", 4)
    _need(v_cache, torch.uint8, "v_cache", 4)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, d = q.shape
    _, Hkv, cap, nb = k_cache.shape
    if d != D or nb != BLOCK_BYTES or v_cache.shape != k_cache.shape or k_cache.shape[0] != B:
        raise ValueError("shape mismatch between q and caches")
    need = tbq4_decode_workspace_bytes(B, Hq, Hkv, max_len, split_tokens)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float16, device=q.device)
    _need(out, torch.float16, "out", 3)
    check(lib.tbq4_attn_decode_split(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), int(max_len), B, Hq, Hkv,
        cap, float(softmax_scale), C.c_uint64(sign_seed), int(split_tokens),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out),
        _stream(stream)), "tbq4_attn_decode")
    return out


def tbq4_attn_decode_append(q, k_new, v_new, k_cache, v_cache, seq_lens, max_len,
                            softmax_scale, sign_seed=0, workspace=None, out=None, stream=None):
    """One decode step: k_new / v_new fp32 [B][Hkv][128] are encoded into the
    caches at position seq_lens[b]-1, then decode attention over seq_lens[b]
    keys; returns fp16 [B][Hq][128]."""
    _need(q, torch.float32, "q", 3)
    _need(k_new, torch.float32, "k_new", 3)
    _need(v_new, torch.float32, "v_new", 3)
    _need(k_cache, torch.uint8, "k_cache", 4)
    _need(v_cache, torch.uint8, "v_cache", 4)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, d = q.shape
    _, Hkv, cap, nb = k_cache.shape
    if (d != D or nb != BLOCK_BYTES or v_cache.shape != k_cache.shape or k_cache.shape[0] != B
            or tuple(k_new.shape) != (B, Hkv, D) or tuple(v_new.shape) != (B, Hkv, D)):
        raise ValueError("shape mismatch between q, new rows and caches")
    need = tbq4_decode_workspace_bytes(B, Hq, Hkv, max_len)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float16, device=q.device)
    _need(out, torch.float16, "out", 3)
    check(lib.tbq4_attn_decode_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
        int(max_len), B, Hq, Hkv, cap, float(softmax_scale), C.c_uint64(sign_seed),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out),
        _stream(stream)), "tbq4_attn_decode_append")
    return out


def empty_pool(n_pages, n_kv_heads, page_size, device="cuda"):
    """An uninitialised page pool [n_pages][Hkv][page_size][66] uint8
    (page_size a multiple of 32)."""
    return torch.empty((n_pages, n_kv_heads, page_size, BLOCK_BYTES), dtype=torch.uint8,
                       device=device)


def _pool_shape(pool, name):
    _need(pool, torch.uint8, name, 4)
    n_pages, Hkv, page_size, nb = pool.shape
    if nb != BLOCK_BYTES:
        raise ValueError(f"{name}: last dimension must be {BLOCK_BYTES}")
    return n_pages, Hkv, page_size


def tbq4_quantize_append_paged(src, start_pos, block_table, pool, sign_seed=0, stream=None):
    """src fp32 [B][n_new][Hkv][128]; start_pos int32 [B]; block_table int32
    [B][max_pages]; pool uint8 [n_pages][Hkv][page_size][66] (written)."""
    _need(src, torch.float32, "src", 4)
    _need(start_pos, torch.int32, "start_pos", 1)
    _need(block_table, torch.int32, "block_table", 2)
    n_pages, Hkv, page_size = _pool_shape(pool, "pool")
    B, n_new, h, d = src.shape
    if d != D or h != Hkv or block_table.shape[0] != B:
        raise ValueError("shape mismatch between src, block_table and pool")
    check(lib.tbq4_quantize_append_paged(
        _ptr(src), B, n_new, Hkv, _ptr(start_pos), _ptr(block_table), block_table.shape[1],
        page_size, n_pages, C.c_uint64(sign_seed), _ptr(pool), _stream(stream)),
        "tbq4_quantize_append_paged")
    return pool


def tbq4_attn_decode_paged(q, k_pool, v_pool, block_table, seq_lens, max_len, softmax_scale,
                           sign_seed=0, k_new=None, v_new=None, workspace=None, out=None,
                           stream=None):
    """Decode attention over paged caches: q fp32 [B][Hq][128]; pools uint8
    [n_pages][Hkv][page_size][66]; block_table int32 [B][max_pages]; with
    k_new / v_new (fp32 [B][Hkv][128]) the step's rows are written at
    seq_lens[b]-1 first.  Returns fp16 [B][Hq][128]."""
    _need(q, torch.float32, "q", 3)
    _need(block_table, torch.int32, "block_table", 2)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    n_pages, Hkv, page_size = _pool_shape(k_pool, "k_pool")
    if v_pool.shape != k_pool.shape:
        raise ValueError("k_pool and v_pool differ in shape")
    _pool_shape(v_pool, "v_pool")
    B, Hq, d = q.shape
    if d != D or block_table.shape[0] != B:
        raise ValueError("shape mismatch between q, block_table and pools")
    if (k_new is None) != (v_new is None):
        raise ValueError("give both k_new and v_new, or neither")
    if k_new is not None:
        _need(k_new, torch.float32, "k_new", 3)
        _need(v_new, torch.float32, "v_new", 3)
        if tuple(k_new.shape) != (B, Hkv, D) or tuple(v_new.shape) != (B, Hkv, D):
            raise ValueError("k_new / v_new must be [B][Hkv][128]")
    need = tbq4_decode_workspace_bytes(B, Hq, Hkv, max_len)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float16, device=q.device)
    _need(out, torch.float16, "out", 3)
    check(lib.tbq4_attn_decode_paged(
        _ptr(q), _ptr(k_new) if k_new is not None else None,
        _ptr(v_new) if v_new is not None else None, _ptr(k_pool), _ptr(v_pool),
        _ptr(block_table), block_table.shape[1], page_size, n_pages, _ptr(seq_lens),
        int(max_len), B, Hq, Hkv, float(softmax_scale), C.c_uint64(sign_seed), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _stream(stream)),
        "tbq4_attn_decode_paged")
    return out


BLOCK_BYTES3 = 50      # TBQ3: the 3-bit variant (see include/tbq4.h)


def empty_cache3(batch, n_kv_heads, capacity, device="cuda"):
    """An uninitialised 3-bit cache [B][Hkv][capacity][50] (capacity % 8 == 0)."""
    return torch.empty((batch, n_kv_heads, capacity, BLOCK_BYTES3), dtype=torch.uint8,
                       device=device)


def tbq3_quantize_append(src, start_pos, cache, sign_seed=0, stream=None):
    """As tbq4_quantize_append, into a 3-bit cache [B][Hkv][capacity][50]."""
    _need(src, torch.float32, "src", 4)
    _need(start_pos, torch.int32, "start_pos", 1)
    _need(cache, torch.uint8, "cache", 4)
    B, n_new, Hkv, d = src.shape
    if d != D or tuple(cache.shape[:2]) != (B, Hkv) or cache.shape[3] != BLOCK_BYTES3:
        raise ValueError("shape mismatch between src and cache")
    check(lib.tbq3_quantize_append(_ptr(src), B, n_new, Hkv, _ptr(start_pos),
                                   cache.shape[2], C.c_uint64(sign_seed), _ptr(cache),
                                   _stream(stream)), "tbq3_quantize_append")
    return cache


def tbq3_attn_decode(q, k_cache, v_cache, seq_lens, max_len, softmax_scale, sign_seed=0,
                     workspace=None, out=None, stream=None):
    """As tbq4_attn_decode, over 3-bit caches [B][Hkv][capacity][50]."""
    _need(q, torch.float32, "q", 3)
    _need(k_cache, torch.uint8, "k_cache", 4)
    _need(v_cache, torch.uint8, "v_cache", 4)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, d = q.shape
    _, Hkv, cap, nb = k_cache.shape
    if d != D or nb != BLOCK_BYTES3 or v_cache.shape != k_cache.shape or k_cache.shape[0] != B:
        raise ValueError("shape mismatch between q and caches")
    need = tbq4_decode_workspace_bytes(B, Hq, Hkv, max_len)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float16, device=q.device)
    _need(out, torch.float16, "out", 3)
    check(lib.tbq3_attn_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), int(max_len), B, Hq, Hkv, cap,
        float(softmax_scale), C.c_uint64(sign_seed), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _stream(stream)),
        "tbq3_attn_decode")
    return out


def tbq4_decode_mq_workspace_bytes(B, q_len, Hq, Hkv, max_len) -> int:
    return int(lib.tbq4_decode_mq_workspace_bytes(B, q_len, Hq, Hkv, max_len))


def tbq4_attn_decode_mq(q, k_cache, v_cache, seq_lens, max_len, softmax_scale, sign_seed=0,
                        workspace=None, out=None, stream=None):
    """q fp32 [B][q_len][Hq][128]: the last q_len tokens of each sequence
    (already in the caches); returns fp16 [B][q_len][Hq][128]."""
    _need(q, torch.float32, "q", 4)
    _need(k_cache, torch.uint8, "k_cache", 4)
    _need(v_cache, torch.uint8, "v_cache", 4)
    _need(seq_lens, torch.int32, "seq_lens", 1)
    B, q_len, Hq, d = q.shape
    _, Hkv, cap, nb = k_cache.shape
    if d != D or nb != BLOCK_BYTES or v_cache.shape != k_cache.shape or k_cache.shape[0] != B:
        raise ValueError("shape mismatch between q and caches")
    need = tbq4_decode_mq_workspace_bytes(B, q_len, Hq, Hkv, max_len)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, q_len, Hq, D), dtype=torch.float16, device=q.device)
    _need(out, torch.float16, "out", 4)
    check(lib.tbq4_attn_decode_mq(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), int(max_len), B, q_len, Hq, Hkv,
        cap, float(softmax_scale), C.c_uint64(sign_seed), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _stream(stream)),
        "tbq4_attn_decode_mq")
    return out


def tbq4_prefill_workspace_bytes(n_new, Hq, Hkv, n_cached) -> int:
    return int(lib.tbq4_prefill_workspace_bytes(n_new, Hq, Hkv, n_cached))


def tbq4_attn_prefill_chunk(q, n_cached, k_cache, v_cache, softmax_scale, sign_seed=0,
                            workspace=None, out=None, stream=None):
    """q bf16 [n_new][Hq][128]; caches uint8 [Hkv][capacity][66] of one
    sequence holding the chunk at n_cached ..; returns bf16 [n_new][Hq][128]."""
    _need(q, torch.bfloat16, "q", 3)
    _need(k_cache, torch.uint8, "k_cache", 3)
    _need(v_cache, torch.uint8, "v_cache", 3)
    n_new, Hq, d = q.shape
    Hkv, cap, nb = k_cache.shape
    if d != D or nb != BLOCK_BYTES or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch between q and caches")
    need = tbq4_prefill_workspace_bytes(n_new, Hq, Hkv, n_cached)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((n_new, Hq, D), dtype=torch.bfloat16, device=q.device)
    _need(out, torch.bfloat16, "out", 3)
    check(lib.tbq4_attn_prefill_chunk(
        _ptr(q), n_new, int(n_cached), _ptr(k_cache), _ptr(v_cache), Hq, Hkv, cap,
        float(softmax_scale), C.c_uint64(sign_seed), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _stream(stream)),
        "tbq4_attn_prefill_chunk")
    return out


# ---- speculative decoding with draft trees ---------------------------------

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}    # tbq4_dtype


def _one_device(first, *rest):
    """The device that every given tensor (None: not given) lies on."""
    for t in rest:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on {first.device} and {t.device}: one device is needed")
    return first.device


def _on(device):
    """Makes `device` current for a call whose tensors lie on another one."""
    if device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _stream_on(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    return stream.cuda_stream


def _ptr_or_null(t):
    return t.data_ptr() if t is not None else None


def _need_rows(t, name, dtype=None, heads=None, tokens=None):
    """Rows of 128 at any token and head stride; returns those strides."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'float32, float16 or bfloat16'}, got {t.dtype}")
    if t.dim() != 3 or t.shape[2] != D or t.stride(2) != 1:
        raise ValueError(f"{name} must be [tokens][heads][128] with adjacent channels, "
                         f"got {tuple(t.shape)} with strides {t.stride()}")
    if (heads is not None and t.shape[1] != heads) or (tokens is not None and t.shape[0] != tokens):
        raise ValueError(f"{name} must be [{tokens}][{heads}][128], got {tuple(t.shape)}")
    # the stride of a dimension of one is never used
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


def _rope_append(name, k, v, slots, inv_freq, kc, vc, Hkv, B, layout, table, q, positions, seq_ids,
                 interleaved, sign_seed, q_out, stream):
    k_tok, k_head = _need_rows(k, "k", heads=Hkv)
    n = k.shape[0]
    v_tok, v_head = _need_rows(v, "v", k.dtype, Hkv, n)
    _need(slots, torch.int32, "slots", 1)
    rot = 0
    if inv_freq is not None:
        _need(inv_freq, torch.float64, "inv_freq", 1)
        rot = 2 * inv_freq.shape[0]
    for t, what in ((positions, "positions"), (seq_ids, "seq_ids")):
        if t is not None:
            _need(t, torch.int32, what, 1)
            if t.shape[0] != n:
                raise ValueError(f"{what} must be [{n}], got {tuple(t.shape)}")
    if slots.shape[0] != n:
        raise ValueError(f"slots must be [{n}], got {tuple(slots.shape)}")
    Hq = q_tok = q_head = 0
    if q is not None:
        q_tok, q_head = _need_rows(q, "q", k.dtype, tokens=n)
        Hq = q.shape[1]
        if q_out is None:
            q_out = torch.empty((n, Hq, D), dtype=q.dtype, device=q.device)
        _need(q_out, q.dtype, "q_out", 3)
        if q_out.shape != q.shape:
            raise ValueError(f"q_out must be {tuple(q.shape)}, got {tuple(q_out.shape)}")
    elif q_out is not None:
        raise ValueError("q_out without q")
    device = _one_device(k, v, slots, inv_freq, kc, vc, table, q, positions, seq_ids, q_out)
    with _on(device):
        check(getattr(lib, name)(
            _ptr_or_null(q), q_tok, q_head, k.data_ptr(), k_tok, k_head, v.data_ptr(), v_tok, v_head,
            _DTYPES[k.dtype], n, B, Hq, Hkv, _ptr_or_null(seq_ids), slots.data_ptr(),
            _ptr_or_null(positions), _ptr_or_null(inv_freq), rot, int(bool(interleaved)), *layout,
            sign_seed, kc.data_ptr(), vc.data_ptr(), _ptr_or_null(q_out),
            _stream_on(stream, device)), name)
    return q_out


def tbq4_rope_append(k, v, slots, inv_freq, k_cache, v_cache, q=None, positions=None, seq_ids=None,
                     interleaved=False, sign_seed=0, q_out=None, stream=None):
    """Rotary embedding of q and k and quantise-append of k and v, in one
    launch.  k, v [n][Hkv][128] and q [n][Hq][128] in float32, float16 or
    bfloat16, at any token and head stride that is a multiple of 16 bytes;
    slots, positions (default: the slots), seq_ids (default: n / B tokens of
    each sequence in turn; negative: padding) int32 [n]; inv_freq float64
    [rot_dim / 2] (None: no rotation); caches uint8 [B][Hkv][capacity][66]
    (written).  Returns the rotated queries, [n][Hq][128] in q's dtype (None
    without q)."""
    _need(k_cache, torch.uint8, "k_cache", 4)
    _need(v_cache, torch.uint8, "v_cache", 4)
    B, Hkv, cap, nb = k_cache.shape
    if nb != BLOCK_BYTES or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [B][Hkv][capacity][66]")
    return _rope_append("tbq4_rope_append", k, v, slots, inv_freq, k_cache, v_cache, Hkv, B, (cap,),
                        None, q, positions, seq_ids, interleaved, sign_seed, q_out, stream)


def tbq4_rope_append_paged(k, v, slots, inv_freq, block_table, k_pool, v_pool, q=None,
                           positions=None, seq_ids=None, interleaved=False, sign_seed=0, q_out=None,
                           stream=None):
    """As tbq4_rope_append, into page pools uint8 [n_pages][Hkv][page_size][66]
    through block_table int32 [B][max_pages]."""
    _need(block_table, torch.int32, "block_table", 2)
    n_pages, Hkv, page_size = _pool_shape(k_pool, "k_pool")
    _pool_shape(v_pool, "v_pool")
    if v_pool.shape != k_pool.shape:
        raise ValueError("k_pool and v_pool differ in shape")
    return _rope_append("tbq4_rope_append_paged", k, v, slots, inv_freq, k_pool, v_pool, Hkv,
                        block_table.shape[0],
                        (block_table.data_ptr(), block_table.shape[1], page_size, n_pages),
                        block_table, q, positions, seq_ids, interleaved, sign_seed, q_out, stream)


def tree_mask(parents):
    """The masks of draft trees for tbq4_attn_tree: parents [T] or [B][T]
    (integers, -1 for a node that hangs off the context) -> int64 of the same
    shape and device, bit j of node i set where j is i or an ancestor of i."""
    parents = torch.as_tensor(parents).long()
    T = parents.shape[-1]
    if not 1 <= T <= 64:
        raise ValueError(f"1 to 64 nodes, got {T}")
    if bool(((parents < -1) | (parents >= T)).any()):
        raise ValueError("a parent is a node of the tree or -1")
    node = torch.arange(T, device=parents.device)
    sees = torch.zeros((*parents.shape, T), dtype=torch.bool, device=parents.device)
    at = node.expand_as(parents)
    for _ in range(T):                         # one generation at a time
        sees |= at[..., None] == node
        at = torch.where(at >= 0, parents.gather(-1, at.clamp(min=0)), -1)
    if bool((at >= 0).any()):
        raise ValueError("the parents run in a circle")
    return torch.where(sees, torch.ones_like(node) << node, 0).sum(-1)


def tbq4_tree_workspace_bytes(B, T, Hq, Hkv) -> int:
    return int(lib.tbq4_tree_workspace_bytes(B, T, Hq, Hkv))


def _attn_tree(name, q, kc, vc, Hkv, layout, table, ctx_lens, mask, softmax_scale, sign_seed, n_nodes,
               workspace, out, out_dtype, stream):
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise TypeError("q must be a float32, float16 or bfloat16 CUDA tensor")
    _need(q, q.dtype, "q", 4)
    _need(ctx_lens, torch.int32, "ctx_lens", 1)
    _need(mask, torch.int64, "tree_mask")
    B, T, Hq, d = q.shape
    if d != D or ctx_lens.shape[0] != B:
        raise ValueError("shape mismatch between q, caches and ctx_lens")
    if tuple(mask.shape) not in ((T,), (B, T)):
        raise ValueError(f"tree_mask must be [{T}] or [{B}][{T}], got {tuple(mask.shape)}")
    if n_nodes is not None:
        _need(n_nodes, torch.int32, "n_nodes", 1)
        if n_nodes.shape[0] != B:
            raise ValueError(f"n_nodes must be [{B}], got {tuple(n_nodes.shape)}")
    if workspace is None:
        workspace = torch.empty(max(tbq4_tree_workspace_bytes(B, T, Hq, Hkv), 1), dtype=torch.uint8,
                                device=q.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if out is None:
        if out_dtype is None:
            out_dtype = torch.bfloat16 if q.dtype == torch.bfloat16 else torch.float16
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    if out.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"out must be float16 or bfloat16, got {out.dtype}")
    _need(out, out.dtype, "out", 4)
    if out.shape != q.shape:
        raise ValueError(f"out must be {tuple(q.shape)}, got {tuple(out.shape)}")
    device = _one_device(q, kc, vc, table, ctx_lens, mask, n_nodes, workspace, out)
    with _on(device):
        check(getattr(lib, name)(
            q.data_ptr(), _DTYPES[q.dtype], kc.data_ptr(), vc.data_ptr(), *(layout if table is not None else ()),
            ctx_lens.data_ptr(), _ptr_or_null(n_nodes), mask.data_ptr(), T if mask.dim() == 2 else 0,
            B, T, Hq, Hkv, *(layout if table is None else ()), float(softmax_scale), sign_seed,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), out.data_ptr(),
            _DTYPES[out.dtype], _stream_on(stream, device)), name)
    return out


def tbq4_attn_tree(q, k_cache, v_cache, ctx_lens, tree_mask, softmax_scale, sign_seed=0, n_nodes=None,
                   workspace=None, out=None, out_dtype=None, stream=None):
    """Attention of drafted nodes over their context and tree: q [B][T][Hq][128]
    in float32, float16 or bfloat16; caches uint8 [B][Hkv][capacity][66] that
    hold ctx_lens[b] tokens and the nodes right behind them; ctx_lens, n_nodes
    (default: T everywhere) int32 [B]; tree_mask int64 [B][T] or [T] (one tree
    for all): bit j of entry i set where node i sees node j.  Returns
    [B][T][Hq][128] in out's dtype (default: bfloat16 for bfloat16 queries,
    else float16); rows of nodes >= n_nodes[b] are not written."""
    _need(k_cache, torch.uint8, "k_cache", 4)
    _need(v_cache, torch.uint8, "v_cache", 4)
    B, Hkv, cap, nb = k_cache.shape
    if nb != BLOCK_BYTES or v_cache.shape != k_cache.shape or B != q.shape[0]:
        raise ValueError("shape mismatch between q and caches")
    return _attn_tree("tbq4_attn_tree", q, k_cache, v_cache, Hkv, (cap,), None, ctx_lens, tree_mask,
                      softmax_scale, sign_seed, n_nodes, workspace, out, out_dtype, stream)


def tbq4_attn_tree_paged(q, k_pool, v_pool, block_table, ctx_lens, tree_mask, softmax_scale,
                         sign_seed=0, n_nodes=None, workspace=None, out=None, out_dtype=None,
                         stream=None):
    """As tbq4_attn_tree, over page pools uint8 [n_pages][Hkv][page_size][66]
    through block_table int32 [B][max_pages]."""
    _need(block_table, torch.int32, "block_table", 2)
    n_pages, Hkv, page_size = _pool_shape(k_pool, "k_pool")
    _pool_shape(v_pool, "v_pool")
    if v_pool.shape != k_pool.shape or block_table.shape[0] != q.shape[0]:
        raise ValueError("shape mismatch between q, block_table and pools")
    return _attn_tree("tbq4_attn_tree_paged", q, k_pool, v_pool, Hkv,
                      (block_table.data_ptr(), block_table.shape[1], page_size, n_pages), block_table,
                      ctx_lens, tree_mask, softmax_scale, sign_seed, n_nodes, workspace, out,
                      out_dtype, stream)


def _tree_accept(name, ks, vs, shape, B, Hkv, layout, table, ctx_lens, path, n_accept, new_lens, stream):
    if len(ks) != len(vs) or not ks:
        raise ValueError(f"{len(ks)} K and {len(vs)} V caches: as many of each, at least one")
    for c in (*ks, *vs):
        _need(c, torch.uint8, "each cache", 4)
        if c.shape != shape:
            raise ValueError("the caches differ in shape")
    _need(ctx_lens, torch.int32, "ctx_lens", 1)
    _need(path, torch.int32, "path", 2)
    _need(n_accept, torch.int32, "n_accept", 1)
    if new_lens is None:
        new_lens = torch.empty_like(ctx_lens)
    _need(new_lens, torch.int32, "new_lens", 1)
    if not B == ctx_lens.shape[0] == path.shape[0] == n_accept.shape[0] == new_lens.shape[0]:
        raise ValueError("shape mismatch between caches, ctx_lens, path, n_accept and new_lens")
    device = _one_device(ctx_lens, path, n_accept, new_lens, table, *ks, *vs)
    n = len(ks)
    with _on(device):
        check(getattr(lib, name)(
            (C.c_void_p * n)(*[c.data_ptr() for c in ks]), (C.c_void_p * n)(*[c.data_ptr() for c in vs]),
            n, *(layout if table is not None else ()), ctx_lens.data_ptr(), path.data_ptr(),
            n_accept.data_ptr(), path.shape[1], B, Hkv, *(layout if table is None else ()),
            new_lens.data_ptr(), _stream_on(stream, device)), name)
    return new_lens


def tbq4_tree_accept(k_caches, v_caches, ctx_lens, path, n_accept, new_lens=None, stream=None):
    """Keeps the accepted nodes in every layer's caches (lists of uint8
    [B][Hkv][capacity][66], written): block ctx_lens[b] + i becomes block
    ctx_lens[b] + path[b][i] for i < n_accept[b].  path int32 [B][max_path],
    ctx_lens and n_accept int32 [B].  Returns the new lengths, int32 [B]."""
    _need(k_caches[0], torch.uint8, "each cache", 4)
    shape = k_caches[0].shape
    if shape[3] != BLOCK_BYTES:
        raise ValueError("caches must be [B][Hkv][capacity][66]")
    return _tree_accept("tbq4_tree_accept", k_caches, v_caches, shape, shape[0], shape[1], (shape[2],),
                        None, ctx_lens, path, n_accept, new_lens, stream)


def tbq4_tree_accept_paged(k_pools, v_pools, block_table, ctx_lens, path, n_accept, new_lens=None,
                           stream=None):
    """As tbq4_tree_accept, over page pools (lists of uint8
    [n_pages][Hkv][page_size][66]) that share block_table int32 [B][max_pages]."""
    _need(block_table, torch.int32, "block_table", 2)
    n_pages, Hkv, page_size = _pool_shape(k_pools[0], "each pool")
    return _tree_accept("tbq4_tree_accept_paged", k_pools, v_pools, k_pools[0].shape,
                        block_table.shape[0], Hkv,
                        (block_table.data_ptr(), block_table.shape[1], page_size, n_pages), block_table,
                        ctx_lens, path, n_accept, new_lens, stream)


def tbq4_set_timing_events(before=None, after=None):
    """Record torch.cuda.Event `before`/`after` around the main attention
    kernel of every following attention call (None, None to stop)."""
    lib.tbq4_set_timing_events(C.c_void_p(before.cuda_event if before is not None else 0),
                               C.c_void_p(after.cuda_event if after is not None else 0))


def tbq4_get_device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error code."""
    return int(lib.tbq4_get_device_status(_stream(stream)))


def tbq4_selftest_bounded_wait(polls=256, stream=None) -> None:
    """Launches the bounded-wait self-test: one warp waits on a barrier that
    nothing completes, gives up after `polls` polls and records
    TBQ4_ERR_DEVICE_TIMEOUT (read it with tbq4_get_device_status)."""
    check(lib.tbq4_selftest_bounded_wait(C.c_uint32(int(polls)), _stream(stream)),
          "tbq4_selftest_bounded_wait")
