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
import ctypes as C
from array import array
from operator import attrgetter

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


# The calls below serve single decode steps, so the host's share counts: a
# check reads each attribute once, and devices are compared by index.

_dtype_of, _shape_of = attrgetter("dtype"), attrgetter("shape")
# the current stream's handle without a Stream object around it (1.2 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)

def _check(name, t, dtype, ndim, index):
    """A contiguous CUDA tensor of this type and rank on device `index`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()
            and t.get_device() == index):
        _need(t, dtype, name, ndim)
        raise ValueError(f"{name} lies on {t.device}, other tensors on cuda:{index}")


def _device_index(t, name):
    """The index of the device that t, and with it all of a call, lies on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _stream_on(stream, index):
    if stream is None:
        return _raw_stream(index)
    if stream.device.index != index:
        raise ValueError(f"stream on {stream.device}, tensors on cuda:{index}")
    return stream.cuda_stream


def _empty(like, shape, dtype, stream):
    """Memory of the stream that the call runs on: there it is free for use at
    once, and again once this call's work is done."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _call(name, index, *args):
    """The library's function `name`, with device `index` current."""
    if index == torch.cuda.current_device():
        code = getattr(lib, name)(*args)
    else:
        with torch.cuda.device(index):
            code = getattr(lib, name)(*args)
    if code:
        raise Tbq4Error(code, name)


def _rows(name, t, dtype, index, tokens, heads):
    """Rows of 128 at any token and head stride: pointer and strides."""
    shape, (tok, head, one) = t.shape, t.stride()
    if not (t.dtype is dtype and t.get_device() == index and shape[2] == D and one == 1
            and shape[0] == tokens and shape[1] == heads):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != index:
            raise ValueError(f"{name} lies on {t.device}, other tensors on cuda:{index}")
        raise ValueError(f"{name} must be [{tokens}][{heads}][128] with adjacent channels, "
                         f"got {tuple(shape)} with strides {t.stride()}")
    # the stride of a dimension of one is never used
    return t.data_ptr(), tok if tokens > 1 else 0, head if heads > 1 else 0


def _rope_append(name, k, v, slots, inv_freq, kc, vc, Hkv, B, layout, index, q, positions, seq_ids,
                 interleaved, sign_seed, q_out, stream):
    for t, what in ((k, "k"), (v, "v"), (k if q is None else q, "q")):
        if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES or t.dim() != 3:
            raise TypeError(f"{what} must be a [tokens][heads][128] CUDA tensor of float32, float16 or "
                            f"bfloat16")
    dtype, n = k.dtype, k.shape[0]
    krows = _rows("k", k, dtype, index, n, Hkv)
    vrows = _rows("v", v, dtype, index, n, Hkv)
    Hq, qrows, out_ptr = 0, (None, 0, 0), None
    if q is not None:
        Hq = q.shape[1]
        qrows = _rows("q", q, dtype, index, n, Hq)
        if q_out is None:
            q_out = _empty(q, (n, Hq, D), dtype, stream)
        else:
            _check("q_out", q_out, dtype, 3, index)
            if q_out.shape != q.shape:
                raise ValueError(f"q_out must be {tuple(q.shape)}, got {tuple(q_out.shape)}")
        out_ptr = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    ids = pos = freq = None
    rot = 0
    _check("slots", slots, torch.int32, 1, index)
    wrong = slots.shape[0] != n
    if positions is not None:
        _check("positions", positions, torch.int32, 1, index)
        wrong |= positions.shape[0] != n
        pos = positions.data_ptr()
    if seq_ids is not None:
        _check("seq_ids", seq_ids, torch.int32, 1, index)
        wrong |= seq_ids.shape[0] != n
        ids = seq_ids.data_ptr()
    if wrong:
        raise ValueError(f"slots, positions and seq_ids must be [{n}]")
    if inv_freq is not None:
        _check("inv_freq", inv_freq, torch.float64, 1, index)
        rot = 2 * inv_freq.shape[0]
        freq = inv_freq.data_ptr()
    if n == 0:
        return q_out                           # empty tensors have no address to pass on
    _call(name, index, *qrows, *krows, *vrows, _DTYPES[dtype], n, B, Hq, Hkv, ids, slots.data_ptr(),
          pos, freq, rot, 1 if interleaved else 0, *layout, sign_seed, kc.data_ptr(), vc.data_ptr(),
          out_ptr, _stream_on(stream, index))
    return q_out


def _cache_pair(k_cache, v_cache, names, block=BLOCK_BYTES):
    """Device index and [.., .., .., 66] shape of a K and a V cache or pool."""
    index = _device_index(k_cache, names[0])
    _check(names[0], k_cache, torch.uint8, 4, index)
    _check(names[1], v_cache, torch.uint8, 4, index)
    shape = k_cache.shape
    if shape[3] != block or v_cache.shape != shape:
        raise ValueError(f"{names[0]} and {names[1]} must have one shape that ends in {block}, got "
                         f"{tuple(shape)} and {tuple(v_cache.shape)}")
    return index, shape


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
    index, (B, Hkv, cap, _) = _cache_pair(k_cache, v_cache, ("k_cache", "v_cache"))
    return _rope_append("tbq4_rope_append", k, v, slots, inv_freq, k_cache, v_cache, Hkv, B, (cap,),
                        index, q, positions, seq_ids, interleaved, sign_seed, q_out, stream)


def tbq4_rope_append_paged(k, v, slots, inv_freq, block_table, k_pool, v_pool, q=None,
                           positions=None, seq_ids=None, interleaved=False, sign_seed=0, q_out=None,
                           stream=None):
    """As tbq4_rope_append, into page pools uint8 [n_pages][Hkv][page_size][66]
    through block_table int32 [B][max_pages]."""
    index, (n_pages, Hkv, page_size, _) = _cache_pair(k_pool, v_pool, ("k_pool", "v_pool"))
    _check("block_table", block_table, torch.int32, 2, index)
    B, max_pages = block_table.shape
    return _rope_append("tbq4_rope_append_paged", k, v, slots, inv_freq, k_pool, v_pool, Hkv, B,
                        (block_table.data_ptr(), max_pages, page_size, n_pages), index, q, positions,
                        seq_ids, interleaved, sign_seed, q_out, stream)


def tree_mask(parents):
    """The masks of draft trees for tbq4_attn_tree: parents [T] or [B][T]
    (integers, -1 for a node that hangs off the context) -> int64 of the same
    shape and device, bit j of node i set where j is i or an ancestor of i.
    Checks the parents on the host, so it is not for a graph's capture."""
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


def _attn_tree(name, q, kc, vc, Hkv, B, cap, paged, index, ctx_lens, mask, softmax_scale, sign_seed,
               n_nodes, workspace, out, out_dtype, stream):
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise TypeError("q must be a float32, float16 or bfloat16 CUDA tensor")
    _check("q", q, q.dtype, 4, index)
    Bq, T, Hq, d = shape = q.shape
    _check("ctx_lens", ctx_lens, torch.int32, 1, index)
    if d != D or Bq != B or ctx_lens.shape[0] != B:
        raise ValueError("shape mismatch between q, caches and ctx_lens")
    _check("tree_mask", mask, torch.int64, getattr(mask, "ndim", None), index)
    per = mask.numel() // T if T else 0
    if mask.shape[-1:] != (T,) or (mask.dim() == 2 and per != B) or not 1 <= mask.dim() <= 2:
        raise ValueError(f"tree_mask must be [{T}] or [{B}][{T}], got {tuple(mask.shape)}")
    nodes = None
    if n_nodes is not None:
        _check("n_nodes", n_nodes, torch.int32, 1, index)
        if n_nodes.shape[0] != B:
            raise ValueError(f"n_nodes must be [{B}], got {tuple(n_nodes.shape)}")
        nodes = n_nodes.data_ptr()
    if workspace is None:
        workspace = _empty(q, (max(lib.tbq4_tree_workspace_bytes(B, T, Hq, Hkv), 1),), torch.uint8, stream)
    elif not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a CUDA tensor")
    elif not workspace.is_contiguous() or workspace.get_device() != index:
        raise ValueError(f"workspace must be contiguous, on cuda:{index}")
    if out is None:
        if out_dtype is None:
            out_dtype = torch.bfloat16 if q.dtype is torch.bfloat16 else torch.float16
        out = _empty(q, shape, out_dtype, stream)
    elif not isinstance(out, torch.Tensor):
        raise TypeError("out must be a CUDA tensor")
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    if out.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"out must be float16 or bfloat16, got {out.dtype}")
    _check("out", out, out.dtype, 4, index)
    if out.shape != shape:
        raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    _call(name, index, q.data_ptr(), _DTYPES[q.dtype], kc.data_ptr(), vc.data_ptr(), *paged,
          ctx_lens.data_ptr(), nodes, mask.data_ptr(), T if mask.dim() == 2 else 0, B, T, Hq, Hkv, *cap,
          softmax_scale, sign_seed, workspace.data_ptr(), workspace.nbytes, out.data_ptr(),
          _DTYPES[out.dtype], _stream_on(stream, index))
    return out


def tbq4_attn_tree(q, k_cache, v_cache, ctx_lens, tree_mask, softmax_scale, sign_seed=0, n_nodes=None,
                   workspace=None, out=None, out_dtype=None, stream=None):
    """Attention of drafted nodes over their context and tree: q [B][T][Hq][128]
    in float32, float16 or bfloat16; caches uint8 [B][Hkv][capacity][66] that
    hold ctx_lens[b] tokens and the nodes right behind them; ctx_lens, n_nodes
    (default: T everywhere) int32 [B]; tree_mask int64 [B][T] or [T] (one tree
    for all): bit j of entry i set where node i sees node j.  Returns
    [B][T][Hq][128] in out's dtype (default: bfloat16 for bfloat16 queries,
    else float16); rows of nodes >= n_nodes[b] are not written.  bfloat16
    queries with a bfloat16 out are computed in 11 bits (a term per operand),
    every other pair in 22, in up to twice the time."""
    index, (B, Hkv, cap, _) = _cache_pair(k_cache, v_cache, ("k_cache", "v_cache"))
    return _attn_tree("tbq4_attn_tree", q, k_cache, v_cache, Hkv, B, (cap,), (), index, ctx_lens,
                      tree_mask, softmax_scale, sign_seed, n_nodes, workspace, out, out_dtype, stream)


def tbq4_attn_tree_paged(q, k_pool, v_pool, block_table, ctx_lens, tree_mask, softmax_scale,
                         sign_seed=0, n_nodes=None, workspace=None, out=None, out_dtype=None,
                         stream=None):
    """As tbq4_attn_tree, over page pools uint8 [n_pages][Hkv][page_size][66]
    through block_table int32 [B][max_pages]."""
    index, (n_pages, Hkv, page_size, _) = _cache_pair(k_pool, v_pool, ("k_pool", "v_pool"))
    _check("block_table", block_table, torch.int32, 2, index)
    B, max_pages = block_table.shape
    return _attn_tree("tbq4_attn_tree_paged", q, k_pool, v_pool, Hkv, B, (),
                      (block_table.data_ptr(), max_pages, page_size, n_pages), index, ctx_lens,
                      tree_mask, softmax_scale, sign_seed, n_nodes, workspace, out, out_dtype, stream)


def _tree_accept(name, ks, vs, shape, B, cap, paged, index, ctx_lens, path, n_accept, new_lens, stream):
    n, caches = len(ks), [*ks, *vs]
    if len(caches) != 2 * n:
        raise ValueError(f"{n} K and {len(caches) - n} V caches: as many of each")
    # in bulk: a loop over the 56 caches of 28 layers took longer than the kernel
    if not (set(map(torch.Tensor.get_device, caches)) == {index}
            and all(map(torch.Tensor.is_contiguous, caches))
            and set(map(_dtype_of, caches)) == {torch.uint8}
            and list(map(_shape_of, caches)).count(shape) == 2 * n):
        for c in caches:
            _check("each cache", c, torch.uint8, 4, index)
        raise ValueError("the caches differ in shape")
    for t, what, ndim in ((ctx_lens, "ctx_lens", 1), (path, "path", 2), (n_accept, "n_accept", 1)):
        _check(what, t, torch.int32, ndim, index)
    if new_lens is None:
        new_lens = _empty(ctx_lens, ctx_lens.shape, torch.int32, stream)
    else:
        _check("new_lens", new_lens, torch.int32, 1, index)
    if not B == ctx_lens.shape[0] == path.shape[0] == n_accept.shape[0] == new_lens.shape[0]:
        raise ValueError("shape mismatch between caches, ctx_lens, path, n_accept and new_lens")
    ptrs = array("Q", map(torch.Tensor.data_ptr, caches))
    at = ptrs.buffer_info()[0]
    _call(name, index, at, at + 8 * n, n, *paged,
          ctx_lens.data_ptr(), path.data_ptr(), n_accept.data_ptr(), path.shape[1], B, shape[1], *cap,
          new_lens.data_ptr(), _stream_on(stream, index))
    return new_lens


def _first_cache(caches, name):
    """Device index and shape of the first of a list of caches."""
    if not caches:
        raise ValueError("no caches")
    index = _device_index(caches[0], name)
    _check(name, caches[0], torch.uint8, 4, index)
    if caches[0].shape[3] != BLOCK_BYTES:
        raise ValueError(f"{name} must end in {BLOCK_BYTES}, got {tuple(caches[0].shape)}")
    return index, caches[0].shape


def tbq4_tree_accept(k_caches, v_caches, ctx_lens, path, n_accept, new_lens=None, stream=None):
    """Keeps the accepted nodes in every layer's caches (lists of uint8
    [B][Hkv][capacity][66], written): block ctx_lens[b] + i becomes block
    ctx_lens[b] + path[b][i] for i < n_accept[b].  path int32 [B][max_path],
    ctx_lens and n_accept int32 [B].  Returns the new lengths, int32 [B]."""
    index, shape = _first_cache(k_caches, "each cache")
    return _tree_accept("tbq4_tree_accept", k_caches, v_caches, shape, shape[0], (shape[2],), (), index,
                        ctx_lens, path, n_accept, new_lens, stream)


def tbq4_tree_accept_paged(k_pools, v_pools, block_table, ctx_lens, path, n_accept, new_lens=None,
                           stream=None):
    """As tbq4_tree_accept, over page pools (lists of uint8
    [n_pages][Hkv][page_size][66]) that share block_table int32 [B][max_pages]."""
    index, shape = _first_cache(k_pools, "each pool")
    _check("block_table", block_table, torch.int32, 2, index)
    B, max_pages = block_table.shape
    return _tree_accept("tbq4_tree_accept_paged", k_pools, v_pools, shape, B, (),
                        (block_table.data_ptr(), max_pages, shape[2], shape[0]), index, ctx_lens, path,
                        n_accept, new_lens, stream)


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
