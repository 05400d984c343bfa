"""GB300 (sm_103a) fused attention forward -- Python binding of libgbattn.so.

The functions here only marshal arguments (shapes, pointers, the current
CUDA stream) into the C ABI declared in ``include/gbattn.h``; every step of
the computation runs in the library's CUDA kernels.  There is no CPU or
PyTorch fallback: if the library is missing, or the device is not a GB300,
the calls raise.

Entry points (same names as the C ABI):
    attn_fwd_dense(q, k, v, ...)    q [B, Sq, Hq, D], k/v [B, Sk, Hkv, D]
    attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, ...)
    attn_fwd_paged(q, kv_cache, block_table, seq_lens, max_seq_len, ...)
    attn_fwd_paged_workspace_size(num_seqs, Hq, Hkv, D, max_seq_len)
    attn_kv_cache_write, attn_fwd_paged_prefill, attn_mask_to_varlen, attn_pack_rows,
    attn_unpack_rows, attn_unpack_lse, attn_fwd_dense_plan, attn_fwd_varlen_plan, attn_fwd_paged_noalloc,
    attn_set_wait_give_up, attn_fwd_padded
    attn_vsa_layout, attn_vsa_tile_map, attn_gather_rows, attn_vsa_pool, attn_vsa_list_size,
    attn_vsa_block_map, attn_fwd_vsa
    attn_kv_cache_write_fp8, attn_kv_cache_read_fp8, attn_fwd_paged_fp8,
    attn_fwd_paged_fp8_workspace_size: the 8-bit paged KV cache
    attn_bwd_dense, attn_bwd_padded, attn_bwd_varlen, attn_bwd_workspace_size: gradients
    (include/gbattn_bwd.h, and include/gbattn_bwd_strided.h for an out that is not contiguous)
    attn_rotary, attn_rotary_kv_cache_write, attn_rotary_frequencies, attn_rotary_steps: rotary
    positions (include/gbattn_rotary.h), with RotaryPlan holding a head's frequencies on the device
Compositions of those calls: attn_fwd_masked (padding mask), attn_vsa (block-sparse
video attention, with VsaPlan holding one geometry's layout on the device),
attn_fwd_paged_prefill_fp8 (several new tokens a sequence over the 8-bit cache).
"""

from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgbattn.so")

OUT_BF16, OUT_F32 = 0, 1
DEV_BAD_INDEX, DEV_TIMEOUT, DEV_BAD_SEQLEN = 1, 2, 4
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "alignment", 4: "workspace",
                5: "cuda", 6: "device", 7: "scratch limit"}
KV_E4M3, KV_E5M2 = 0, 1
NOALLOC_SCRATCH_BYTES = 32 << 20  # GBATTN_NOALLOC_SCRATCH_BYTES

# (name, restype, argtypes) for every symbol of include/gbattn.h
_P, _I, _F, _Z, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
_D = ctypes.c_double
SIGNATURES = {
    "attn_fwd_dense": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _I, _P, _P, _P]),
    "attn_fwd_varlen": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _I, _P, _P, _P]),
    "attn_fwd_paged_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "attn_fwd_paged": (_I, [_P, _P, _I, _I, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _I, _P, _P, _Z, _P, _P]),
    "attn_status_string": (ctypes.c_char_p, [_I]),
    "attn_fwd_paged_noalloc": (_I, [_P, _P, _I, _I, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _I, _P, _P, _P]),
    "attn_fwd_dense_plan": (_I, [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "attn_fwd_varlen_plan": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_int)]),
    "attn_fwd_padded": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _I, _P, _P, _P]),
    "attn_set_wait_give_up": (_I, [_I, ctypes.POINTER(ctypes.c_int)]),
    "attn_kv_cache_write": (_I, [_P, _P, _P, _I, _P, _I, _I, _I, _I, _P, _P]),
    "attn_fwd_paged_prefill": (_I, [_P, _P, _I, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _I, _P,
                                    _P, _P]),
    "attn_mask_to_varlen": (_I, [_P, _I, _I, _P, _P, _P]),
    "attn_pack_rows": (_I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    "attn_unpack_rows": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "attn_unpack_lse": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "attn_vsa_layout": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, ctypes.POINTER(ctypes.c_int),
                             ctypes.POINTER(ctypes.c_int)]),
    "attn_vsa_tile_map": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, _P, _P, ctypes.POINTER(ctypes.c_int),
                               ctypes.POINTER(ctypes.c_int)]),
    "attn_gather_rows": (_I, [_P, _L, _P, _L, _I, _P, _P, _P]),
    "attn_vsa_pool": (_I, [_P, _I, _I, _I, _P, _P, _P, _P]),
    "attn_vsa_list_size": (_I, [_I, _I, _I, _I, ctypes.POINTER(ctypes.c_longlong)]),
    "attn_vsa_block_map": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P]),
    "attn_kv_cache_write_fp8": (_I, [_P, _P, _L, _L, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "attn_kv_cache_read_fp8": (_I, [_P, _P, _I, _I, _I, _P, _I, _P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "attn_fwd_paged_fp8_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "attn_fwd_paged_fp8": (_I, [_P, _L, _P, _P, _I, _I, _I, _P, _I, _P, _I, _I, _I, _I, _I, _F, _I, _P, _I, _P, _P, _Z,
                                _P, _P]),
    "attn_fwd_vsa": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P, _L, _I, _I, _I, _F, _P, _I, _P, _P, _P]),
    "attn_bwd_workspace_size": (_Z, [_I, _I, _I]),
    "attn_bwd_dense": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P, _Z, _P, _P]),
    "attn_bwd_padded": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P, _Z,
                             _P, _P]),
    "attn_bwd_varlen": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P,
                             _P, _Z, _P, _P]),
    "attn_bwd_padded_strided": (_I, [_P, _P, _P, _P, _I, _L, _L, _L, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P,
                                     _P, _P, _P, _Z, _P, _P]),
    "attn_bwd_varlen_strided": (_I, [_P, _P, _P, _P, _I, _L, _L, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I,
                                     _P, _P, _P, _P, _Z, _P, _P]),
    "attn_rotary_frequencies": (_I, [_I, _D, _I, _D, _D, _D, _D, _P, _P]),
    "attn_rotary_steps": (_I, [_P, _I, _P]),
    "attn_rotary": (_I, [_P, _L, _P, _L, _P, _I, _P, _I, _I, _I, _F, _I, _I, _I, _P, _L, _P, _L, _P]),
    "attn_rotary_kv_cache_write": (_I, [_P, _L, _P, _L, _P, _L, _P, _P, _I, _P, _I, _I, _F, _P, _L, _P, _I, _I, _I, _I, _I,
                                        _P, _P]),
}

_lib = None


class GbattnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({STATUS_NAMES.get(status, '?')})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgbattn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with attention_forward_09_gb300._build.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, st):
    if st != 0:
        raise GbattnError(fn, st)


def _out_code(dtype):
    if dtype == torch.float32:
        return OUT_F32
    if dtype == torch.bfloat16:
        return OUT_BF16
    raise ValueError("out dtype must be float32 or bfloat16")


def _bf16_cuda(name, t):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor")


def attn_fwd_dense(q, k, v, softmax_scale=None, causal=False, out=None, lse=None, out_dtype=torch.float32,
                   dev_status=None, stream=None):
    """Dense batch.  Returns (out [B, Sq, Hq, D], lse [B, Hq, Sq] or None).
    Pass ``lse=True`` to allocate the LSE output, or a float32 tensor."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bf16_cuda(n, t)
    B, Sq, Hq, D = q.shape
    _, Sk, Hkv, _ = k.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != D:
        raise ValueError("k and v must be [B, Sk, Hkv, D] matching q")
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    if out is None:
        out = torch.empty(B, Sq, Hq, D, dtype=out_dtype, device=q.device)
    if lse is True:
        lse = torch.empty(B, Hq, Sq, dtype=torch.float32, device=q.device)
    st = load_library().attn_fwd_dense(_ptr(q), _ptr(k), _ptr(v), B, Sq, Sk, Hq, Hkv, D, scale, int(bool(causal)),
                                       _ptr(out), _out_code(out.dtype), _ptr(lse), _ptr(dev_status),
                                       _stream_handle(stream))
    _check("attn_fwd_dense", st)
    return out, lse


def attn_fwd_padded(q, k, v, lens_q=None, lens_k=None, softmax_scale=None, causal=False, out=None, lse=None,
                    out_dtype=torch.float32, dev_status=None, stream=None):
    """Right-padded batch: entry b uses its first lens_q[b] query rows and
    lens_k[b] keys (int32 CUDA tensors [B], or None for all rows).  q [B, Sq,
    Hq, D], k/v [B, Sk, Hkv, D].  Returns (out [B, Sq, Hq, D], lse [B, Hq, Sq]
    or None); padded query rows get zeros and -inf."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bf16_cuda(n, t)
    B, Sq, Hq, D = q.shape
    _, Sk, Hkv, _ = k.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != D:
        raise ValueError("k and v must be [B, Sk, Hkv, D] matching q")
    for n, t in (("lens_q", lens_q), ("lens_k", lens_k)):
        if t is not None and (t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.numel() != B):
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor of {B} entries")
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    if out is None:
        out = torch.empty(B, Sq, Hq, D, dtype=out_dtype, device=q.device)
    if lse is True:
        lse = torch.empty(B, Hq, Sq, dtype=torch.float32, device=q.device)
    st = load_library().attn_fwd_padded(_ptr(q), _ptr(k), _ptr(v), _ptr(lens_q), _ptr(lens_k), B, Sq, Sk, Hq, Hkv, D,
                                        scale, int(bool(causal)), _ptr(out), _out_code(out.dtype), _ptr(lse),
                                        _ptr(dev_status), _stream_handle(stream))
    _check("attn_fwd_padded", st)
    return out, lse


def attn_fwd_dense_plan(B, Sq, Sk, Hq, Hkv, D, causal=False):
    """(launches, split) attn_fwd_dense makes for these sizes on the current device."""
    n, sp = ctypes.c_int(0), ctypes.c_int(0)
    st = load_library().attn_fwd_dense_plan(B, Sq, Sk, Hq, Hkv, D, int(bool(causal)), ctypes.byref(n),
                                            ctypes.byref(sp))
    _check("attn_fwd_dense_plan", st)
    return n.value, sp.value


def attn_set_wait_give_up(on) -> bool:
    """Make the prefill, gradient and 8-bit decode kernels launched from now on give up their pipeline
    waits at once (a test of the failure path: GBATTN_DEV_TIMEOUT is set,
    the call returns, outputs are undefined); returns the previous setting."""
    prev = ctypes.c_int(0)
    _check("attn_set_wait_give_up", load_library().attn_set_wait_give_up(int(bool(on)), ctypes.byref(prev)))
    return bool(prev.value)


def attn_fwd_varlen_plan(lens_q, D, causal=False, Hq=32, Hkv=8, lens_k=None):
    """Kernel launches attn_fwd_varlen makes for documents of these lengths
    on the current device (host sizes only)."""
    lens_k = lens_q if lens_k is None else lens_k
    n = ctypes.c_int(0)
    st = load_library().attn_fwd_varlen_plan(len(lens_q), int(sum(lens_q)), int(max(list(lens_q) + [0])),
                                             int(max(list(lens_k) + [0])), Hq, Hkv, D, int(bool(causal)),
                                             ctypes.byref(n))
    _check("attn_fwd_varlen_plan", st)
    return n.value


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale=None,
                    causal=False, out=None, lse=None, out_dtype=torch.float32, dev_status=None, stream=None):
    """Packed documents.  q [Tq, Hq, D], k/v [Tk, Hkv, D], cu_seqlens int32
    CUDA tensors [N+1]; max_seqlen_q/k are host ints.  Returns (out [Tq, Hq, D],
    lse [Hq, Tq] or None)."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bf16_cuda(n, t)
    for n, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    if k.shape != v.shape or k.shape[2] != D:
        raise ValueError("k and v must be [Tk, Hkv, D] matching q")
    n_docs = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() - 1 != n_docs:
        raise ValueError("cu_seqlens_q and cu_seqlens_k describe different document counts")
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    if out is None:
        out = torch.empty(Tq, Hq, D, dtype=out_dtype, device=q.device)
    if lse is True:
        lse = torch.empty(Hq, Tq, dtype=torch.float32, device=q.device)
    st = load_library().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), n_docs,
                                        Tq, Tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D, scale,
                                        int(bool(causal)), _ptr(out), _out_code(out.dtype), _ptr(lse),
                                        _ptr(dev_status), _stream_handle(stream))
    _check("attn_fwd_varlen", st)
    return out, lse


def attn_fwd_paged_workspace_size(num_seqs, Hq, Hkv, D, max_seq_len) -> int:
    return int(load_library().attn_fwd_paged_workspace_size(num_seqs, Hq, Hkv, D, max_seq_len))


def attn_fwd_paged(q, kv_cache, block_table, seq_lens, max_seq_len, softmax_scale=None, causal=True, out=None,
                   lse=None, out_dtype=torch.float32, workspace=None, dev_status=None, stream=None):
    """Decode over a paged cache.  q [S, Hq, D]; kv_cache [2, nb, 128, Hkv, D];
    block_table int32 [S, max_blocks]; seq_lens int32 [S]; max_seq_len host int.
    Returns (out [S, Hq, D], lse [S, Hq] or None).  A workspace tensor of at
    least ``attn_fwd_paged_workspace_size`` bytes may be passed (it is
    allocated here otherwise)."""
    _bf16_cuda("q", q)
    _bf16_cuda("kv_cache", kv_cache)
    S, Hq, D = q.shape
    two, nb, bs, Hkv, Dk = kv_cache.shape
    if two != 2 or Dk != D:
        raise ValueError("kv_cache must be [2, num_blocks, block_size, Hkv, D]")
    for n, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    need = attn_fwd_paged_workspace_size(S, Hq, Hkv, D, int(max_seq_len))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(S, Hq, D, dtype=out_dtype, device=q.device)
    if lse is True:
        lse = torch.empty(S, Hq, dtype=torch.float32, device=q.device)
    st = load_library().attn_fwd_paged(_ptr(q), _ptr(kv_cache), nb, bs, _ptr(block_table), block_table.shape[1],
                                       _ptr(seq_lens), S, int(max_seq_len), Hq, Hkv, D, scale, int(bool(causal)),
                                       _ptr(out), _out_code(out.dtype), _ptr(lse), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                       _stream_handle(stream))
    _check("attn_fwd_paged", st)
    return out, lse


def attn_fwd_paged_noalloc(q, kv_cache, block_table, seq_lens, max_seq_len, softmax_scale=None, causal=True,
                           out=None, lse=None, out_dtype=torch.float32, dev_status=None, stream=None):
    """attn_fwd_paged without a workspace argument, for callers that must not
    allocate device memory while it runs (e.g. during CUDA-graph capture): the
    split-K scratch is the library's built-in 32 MiB device array.  Pass
    preallocated ``out`` (and ``lse``) to allocate nothing here either.  The
    first call on a device should happen before any stream capture.  Calls
    that overlap on the GPU share the scratch and race."""
    _bf16_cuda("q", q)
    _bf16_cuda("kv_cache", kv_cache)
    S, Hq, D = q.shape
    two, nb, bs, Hkv, Dk = kv_cache.shape
    if two != 2 or Dk != D:
        raise ValueError("kv_cache must be [2, num_blocks, block_size, Hkv, D]")
    for n, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    if out is None:
        out = torch.empty(S, Hq, D, dtype=out_dtype, device=q.device)
    if lse is True:
        lse = torch.empty(S, Hq, dtype=torch.float32, device=q.device)
    st = load_library().attn_fwd_paged_noalloc(_ptr(q), _ptr(kv_cache), nb, bs, _ptr(block_table),
                                               block_table.shape[1], _ptr(seq_lens), S, int(max_seq_len), Hq, Hkv, D,
                                               scale, int(bool(causal)), _ptr(out), _out_code(out.dtype), _ptr(lse),
                                               _ptr(dev_status), _stream_handle(stream))
    _check("attn_fwd_paged_noalloc", st)
    return out, lse


def attn_kv_cache_write(key, value, slot_mapping, kv_cache, dev_status=None, stream=None):
    """Store key / value [T, Hkv, D] (bf16) into kv_cache [2, nb, bs, Hkv, D]
    in place at slot_mapping [T] (int32 CUDA): token t goes to block
    slot // bs, offset slot % bs; negative slots store nothing."""
    for n, t in (("key", key), ("value", value), ("kv_cache", kv_cache)):
        _bf16_cuda(n, t)
    T, Hkv, D = key.shape
    two, nb, bs, Hc, Dc = kv_cache.shape
    if value.shape != key.shape or two != 2 or (Hc, Dc) != (Hkv, D):
        raise ValueError("key/value must be [T, Hkv, D] and kv_cache [2, num_blocks, block_size, Hkv, D]")
    if slot_mapping.dtype != torch.int32 or not slot_mapping.is_cuda or not slot_mapping.is_contiguous() or \
            slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be a contiguous int32 CUDA tensor of T entries")
    st = load_library().attn_kv_cache_write(_ptr(key), _ptr(value), _ptr(slot_mapping), T, _ptr(kv_cache), nb, bs,
                                            Hkv, D, _ptr(dev_status), _stream_handle(stream))
    _check("attn_kv_cache_write", st)
    return kv_cache


def attn_fwd_paged_prefill(q, kv_cache, block_table, seq_lens, cu_seqlens_q, max_seqlen_q, max_seq_len,
                           softmax_scale=None, causal=True, out=None, lse=None, out_dtype=torch.float32,
                           dev_status=None, stream=None):
    """Several query tokens per sequence (packed by cu_seqlens_q, the last
    tokens of each context) against the paged cache.  Returns
    (out [Tq, Hq, D], lse [Hq, Tq] or None); max_seqlen_q / max_seq_len are
    host ints."""
    _bf16_cuda("q", q)
    _bf16_cuda("kv_cache", kv_cache)
    Tq, Hq, D = q.shape
    two, nb, bs, Hkv, Dk = kv_cache.shape
    if two != 2 or Dk != D:
        raise ValueError("kv_cache must be [2, num_blocks, block_size, Hkv, D]")
    for n, t in (("block_table", block_table), ("seq_lens", seq_lens), ("cu_seqlens_q", cu_seqlens_q)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous int32 CUDA tensor")
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    if out is None:
        out = torch.empty(Tq, Hq, D, dtype=out_dtype, device=q.device)
    if lse is True:
        lse = torch.empty(Hq, Tq, dtype=torch.float32, device=q.device)
    S = cu_seqlens_q.numel() - 1
    st = load_library().attn_fwd_paged_prefill(_ptr(q), _ptr(kv_cache), nb, bs, _ptr(block_table),
                                               block_table.shape[1], _ptr(seq_lens), _ptr(cu_seqlens_q), S, Tq,
                                               int(max_seqlen_q), int(max_seq_len), Hq, Hkv, D, scale,
                                               int(bool(causal)), _ptr(out), _out_code(out.dtype), _ptr(lse),
                                               _ptr(dev_status), _stream_handle(stream))
    _check("attn_fwd_paged_prefill", st)
    return out, lse


# ---- 8-bit paged KV cache.  These calls run on their tensors' device, whichever
# is current, and allocate what they return (and a workspace not given) on the
# stream they run on.
_KV_CODE = {torch.float8_e4m3fn: KV_E4M3, torch.float8_e5m2: KV_E5M2}


def _fp8_cache(kv_cache, kv_scales):
    """(code format, num_blocks, block_size, Hkv, D) of an 8-bit cache."""
    code, shape = _KV_CODE.get(kv_cache.dtype), kv_cache.shape
    if code is None or len(shape) != 5 or shape[0] != 2:
        raise ValueError("kv_cache must be a float8_e4m3fn or float8_e5m2 tensor [2, num_blocks, block_size, Hkv, D]")
    _, nb, bs, hkv, d = shape
    if kv_scales.dtype != torch.uint8 or kv_scales.shape != (2, nb, hkv, bs):
        raise ValueError(f"kv_scales must be a uint8 tensor [2, {nb}, {hkv}, {bs}] (num_blocks, Hkv, block_size)")
    if not (kv_cache.is_contiguous() and kv_scales.is_contiguous()):
        raise ValueError("kv_cache and kv_scales must be contiguous")
    return code, nb, bs, hkv, d


def _on_device(dev, names, *tensors):
    """Raise ValueError unless every tensor given is on CUDA device number dev."""
    if dev < 0:
        raise ValueError("the 8-bit cache calls take CUDA tensors")
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{names.split()[i]} must be on cuda:{dev}, with the cache")


def _index_table(name, t, dim):
    if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {dim} dimension{'s' if dim > 1 else ''}")


def _status_ptr(dev_status):
    if dev_status is None:
        return None
    if dev_status.dtype not in (torch.int32, torch.uint32) or dev_status.numel() < 1:
        raise ValueError("dev_status must be a 32-bit integer tensor")
    return dev_status.data_ptr()


def _host_int(name, x):
    x = int(x)
    if x >= 1 << 31:  # (a negative one is the library's to refuse)
        raise ValueError(f"{name} must be below 2**31")
    return x


def _run_fp8(name, dev, stream, args):
    """One C call on device number dev and stream (None: the device's current one)."""
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream must be of cuda:{dev}, where the cache is")
    fn = getattr(_lib or load_library(), name)
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != 0:
        raise GbattnError(name, st)


def _empty_on(stream, like, shape, dtype):
    """An uninitialised tensor on like's device, of the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _token_rows(name, t, heads, d):
    """Element stride between the tokens of a bf16 [T, heads, D] tensor whose [heads, D] rows are contiguous."""
    shape = t.shape
    if t.dtype != torch.bfloat16 or len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{name} must be a bfloat16 tensor [tokens, {heads}, {d}]")
    tokens, row, col = t.stride()
    if (d > 1 and col != 1) or (heads > 1 and row != d):
        raise ValueError(f"{name}: a token's [heads, D] must be contiguous")
    return tokens if shape[0] > 1 else heads * d


def attn_kv_cache_write_fp8(key, value, slot_mapping, kv_cache, kv_scales, dev_status=None, stream=None):
    """Store key / value [T, Hkv, D] (bf16; tokens may be strided, as parts of
    a fused projection's output) into the 8-bit cache kv_cache [2, nb, bs, Hkv,
    D] (float8_e4m3fn or float8_e5m2) and its exponent bytes kv_scales [2, nb,
    Hkv, bs] (uint8), in place, at slot_mapping [T] (int32): token t goes to
    block slot // bs, offset slot % bs; negative slots store nothing, and a
    slot is to be given once (what one given twice stands for is undefined).
    A row is codes c and a byte b that stand for c * 2^(b - 127).  Returns
    (kv_cache, kv_scales)."""
    code, nb, bs, hkv, d = _fp8_cache(kv_cache, kv_scales)
    ks, vs = _token_rows("key", key, hkv, d), _token_rows("value", value, hkv, d)
    _index_table("slot_mapping", slot_mapping, 1)
    T = slot_mapping.numel()
    if key.shape[0] != T or value.shape[0] != T:
        raise ValueError("key, value and slot_mapping disagree on the token count")
    status, dev = _status_ptr(dev_status), kv_cache.get_device()
    _on_device(dev, "key value slot_mapping kv_scales dev_status", key, value, slot_mapping, kv_scales, dev_status)
    _run_fp8("attn_kv_cache_write_fp8", dev, stream,
             (key.data_ptr(), value.data_ptr(), ks, vs, slot_mapping.data_ptr(), T, kv_cache.data_ptr(),
              kv_scales.data_ptr(), code, nb, bs, hkv, d, status))
    return kv_cache, kv_scales


def attn_kv_cache_read_fp8(kv_cache, kv_scales, block_table, cu_seqlens_k, total_tokens, k=None, v=None,
                           dev_status=None, stream=None):
    """The first cu_seqlens_k[s + 1] - cu_seqlens_k[s] context tokens of every
    sequence s, read from the 8-bit cache through block_table [S, max_blocks]
    (int32), as packed bf16 rows (k, v), each [total_tokens, Hkv, D]: what
    attn_fwd_varlen takes.  total_tokens (host int) is at least
    cu_seqlens_k[S]; rows past that are left as they were, and so are those of a
    sequence whose boundaries make no sense (DEV_BAD_SEQLEN)."""
    code, nb, bs, hkv, d = _fp8_cache(kv_cache, kv_scales)
    _index_table("block_table", block_table, 2)
    _index_table("cu_seqlens_k", cu_seqlens_k, 1)
    S = cu_seqlens_k.numel() - 1
    if S < 0 or block_table.shape[0] != S:
        raise ValueError("block_table must have a row, and cu_seqlens_k a boundary, for each sequence")
    status, dev, T = _status_ptr(dev_status), kv_cache.get_device(), _host_int("total_tokens", total_tokens)
    _on_device(dev, "kv_scales block_table cu_seqlens_k k v dev_status", kv_scales, block_table, cu_seqlens_k, k, v,
               dev_status)
    for name, t in (("k", k), ("v", v)):
        if t is not None and (t.dtype != torch.bfloat16 or tuple(t.shape) != (T, hkv, d) or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous bfloat16 tensor [{T}, {hkv}, {d}]")
    if k is None:
        k = _empty_on(stream, kv_cache, (T, hkv, d), torch.bfloat16)
    if v is None:
        v = _empty_on(stream, kv_cache, (T, hkv, d), torch.bfloat16)
    _run_fp8("attn_kv_cache_read_fp8", dev, stream,
             (kv_cache.data_ptr(), kv_scales.data_ptr(), code, nb, bs, block_table.data_ptr(),
              block_table.shape[1], cu_seqlens_k.data_ptr(), S, T, hkv, d, k.data_ptr(), v.data_ptr(),
              status))
    return k, v


def attn_fwd_paged_fp8_workspace_size(num_seqs, Hq, Hkv, D, max_seq_len) -> int:
    return int(load_library().attn_fwd_paged_fp8_workspace_size(num_seqs, Hq, Hkv, D,
                                                                _host_int("max_seq_len", max_seq_len)))


def attn_fwd_paged_fp8(q, kv_cache, kv_scales, block_table, seq_lens, max_seq_len, softmax_scale=None, causal=True,
                       out=None, lse=None, out_dtype=torch.float32, workspace=None, dev_status=None, stream=None):
    """attn_fwd_paged over an 8-bit cache (attn_kv_cache_write_fp8): q [S, Hq,
    D] bf16 (sequences may be strided); kv_cache [2, nb, 128, Hkv, D] float8;
    kv_scales [2, nb, Hkv, 128] uint8; block_table int32 [S, max_blocks];
    seq_lens int32 [S]; max_seq_len host int.  Returns (out [S, Hq, D], lse
    [S, Hq] or None).  A workspace tensor of at least
    ``attn_fwd_paged_fp8_workspace_size`` bytes may be passed (it is allocated
    here otherwise); calls that can overlap need one each."""
    code, nb, bs, hkv, d = _fp8_cache(kv_cache, kv_scales)
    if q.dim() != 3:
        raise ValueError("q must be [S, Hq, D]")
    S, Hq, _ = q.shape
    qs = _token_rows("q", q, Hq, d)
    _index_table("block_table", block_table, 2)
    _index_table("seq_lens", seq_lens, 1)
    if block_table.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_table and seq_lens must have a row for each of q's sequences")
    status, dev, max_seq_len = _status_ptr(dev_status), kv_cache.get_device(), _host_int("max_seq_len", max_seq_len)
    given = lse if torch.is_tensor(lse) else None
    _on_device(dev, "q kv_scales block_table seq_lens out lse workspace dev_status", q, kv_scales, block_table,
               seq_lens, out, given, workspace, dev_status)
    if out is None:
        out = _empty_on(stream, kv_cache, (S, Hq, d), out_dtype)
    elif out.shape != (S, Hq, d) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous tensor [{S}, {Hq}, {d}]")
    if given is None:
        lse = _empty_on(stream, kv_cache, (S, Hq), torch.float32) if lse else None
    elif lse.dtype != torch.float32 or lse.shape != (S, Hq) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor [{S}, {Hq}]")
    if workspace is None:
        ws_bytes = (_lib or load_library()).attn_fwd_paged_fp8_workspace_size(S, Hq, hkv, d, max_seq_len)
        if ws_bytes:
            workspace = _empty_on(stream, kv_cache, (ws_bytes,), torch.uint8)
    elif workspace.is_contiguous():
        ws_bytes = workspace.numel() * workspace.element_size()
    else:
        raise ValueError("workspace must be contiguous")
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    _run_fp8("attn_fwd_paged_fp8", dev, stream,
             (q.data_ptr(), qs, kv_cache.data_ptr(), kv_scales.data_ptr(), code, nb, bs, block_table.data_ptr(),
              block_table.shape[1], seq_lens.data_ptr(), S, max_seq_len, Hq, hkv, d, scale, 1 if causal else 0,
              out.data_ptr(), _out_code(out.dtype), None if lse is None else lse.data_ptr(),
              None if workspace is None else workspace.data_ptr(), ws_bytes, status))
    return out, lse


def attn_fwd_paged_prefill_fp8(q, kv_cache, kv_scales, block_table, cu_seqlens_q, cu_seqlens_k, total_tokens,
                               max_seqlen_q, max_seq_len, softmax_scale=None, causal=True, out=None, lse=None,
                               out_dtype=torch.float32, dev_status=None, stream=None):
    """Several query tokens a sequence (packed by cu_seqlens_q, the last tokens
    of each context) against the 8-bit cache: the contexts are read back
    (attn_kv_cache_read_fp8) and attended as packed documents
    (attn_fwd_varlen).  cu_seqlens_k [S + 1] (int32) holds the contexts' running
    sum, total_tokens >= cu_seqlens_k[S], max_seqlen_q and max_seq_len are
    host ints.  A sequence whose boundaries decrease or run past total_tokens,
    its length bound or its row of the table sets DEV_BAD_SEQLEN and is
    skipped: its rows of out and lse are left unwritten.  (Boundaries that
    decrease can let two other sequences claim the same rows: the results of
    those two are undefined.)  Returns (out [Tq, Hq, D], lse [Hq, Tq] or None)."""
    _, _, bs, hkv, d = _fp8_cache(kv_cache, kv_scales)
    _index_table("block_table", block_table, 2)
    T, max_seqlen_q, max_seq_len = int(total_tokens), _host_int("max_seqlen_q", max_seqlen_q), _host_int("max_seq_len", max_seq_len)
    # the read-back refuses a context that its row of the table cannot hold and
    # leaves its rows unwritten: attn_fwd_varlen has to skip that sequence too (and
    # takes no bound above the rows there are)
    max_seq_len = min(max_seq_len, bs * block_table.shape[1], T)
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[2] != d or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous bfloat16 tensor [tokens, Hq, {d}]")
    Tq, Hq, _ = q.shape
    _index_table("cu_seqlens_q", cu_seqlens_q, 1)
    if cu_seqlens_q.shape != cu_seqlens_k.shape:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have as many boundaries")
    if out is not None and (out.shape != q.shape or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous tensor [{Tq}, {Hq}, {d}]")
    given = lse if torch.is_tensor(lse) else None
    if given is not None and (lse.dtype != torch.float32 or lse.shape != (Hq, Tq) or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor [{Hq}, {Tq}]")
    _on_device(kv_cache.get_device(), "q cu_seqlens_q out lse", q, cu_seqlens_q, out, given)
    k, v = attn_kv_cache_read_fp8(kv_cache, kv_scales, block_table, cu_seqlens_k, T, dev_status=dev_status,
                                  stream=stream)
    with torch.cuda.device(kv_cache.device):
        s = torch.cuda.current_stream() if stream is None else stream
        with torch.cuda.stream(s):
            if Tq == 0:  # no query, no result
                out = torch.empty(0, Hq, d, dtype=out_dtype, device=q.device) if out is None else out
                return out, given if given is not None else q.new_empty(Hq, 0, dtype=torch.float32) if lse else None
            return attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seq_len, softmax_scale, causal,
                                   out, given if given is not None else True if lse else None, out_dtype,
                                   dev_status, stream)


def attn_mask_to_varlen(mask, stream=None):
    """mask [B, S] (bool or uint8 CUDA, nonzero = token) -> (cu_seqlens [B+1], packed_pos [B*S]) int32."""
    if mask.dim() != 2 or not mask.is_cuda or mask.element_size() != 1:
        raise ValueError("mask must be a [B, S] bool / uint8 CUDA tensor")
    mask = mask.contiguous()
    B, S = mask.shape
    cu = torch.empty(B + 1, dtype=torch.int32, device=mask.device)
    pos = torch.empty(B * S, dtype=torch.int32, device=mask.device)
    st = load_library().attn_mask_to_varlen(_ptr(mask), B, S, _ptr(cu), _ptr(pos), _stream_handle(stream))
    _check("attn_mask_to_varlen", st)
    return cu, pos


def attn_pack_rows(x, packed_pos, cu_seqlens, stream=None):
    """x [B, S, ...] contiguous CUDA -> packed [B*S, ...]: the masked-in rows in order, then zero rows."""
    B, S = x.shape[:2]
    packed = torch.empty((B * S,) + tuple(x.shape[2:]), dtype=x.dtype, device=x.device)
    rb = x[0, 0].numel() * x.element_size()
    st = load_library().attn_pack_rows(_ptr(x), _ptr(packed_pos), _ptr(cu_seqlens), B, S, rb, _ptr(packed),
                                       _stream_handle(stream))
    _check("attn_pack_rows", st)
    return packed


def attn_unpack_rows(packed, packed_pos, B, S, stream=None):
    """packed [B*S, ...] -> [B, S, ...] with zeros at the padding."""
    out = torch.empty((B, S) + tuple(packed.shape[1:]), dtype=packed.dtype, device=packed.device)
    rb = packed[0].numel() * packed.element_size()
    st = load_library().attn_unpack_rows(_ptr(packed), _ptr(packed_pos), B, S, rb, _ptr(out), _stream_handle(stream))
    _check("attn_unpack_rows", st)
    return out


def attn_unpack_lse(lse_packed, packed_pos, B, S, stream=None):
    """lse_packed [H, B*S] -> [B, H, S], -inf at the padding."""
    H = lse_packed.shape[0]
    lse = torch.empty(B, H, S, dtype=torch.float32, device=lse_packed.device)
    st = load_library().attn_unpack_lse(_ptr(lse_packed), _ptr(packed_pos), B, H, S, _ptr(lse), _stream_handle(stream))
    _check("attn_unpack_lse", st)
    return lse


def attn_fwd_masked(q, k, v, mask, softmax_scale=None, causal=False, cross=False, lse=False, out_dtype=torch.float32,
                    dev_status=None, stream=None):
    """Padded batch q [B, Sq, Hq, D], k/v [B, Sk, Hkv, D] with a [B, Sk]
    padding mask: the masked-in tokens are packed, attended as varlen
    documents and put back (zeros, lse -inf at the padding).  cross=True:
    the mask covers the keys only and every query row is kept.  Returns
    (out [B, Sq, Hq, D], lse [B, Hq, Sq] or None)."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _bf16_cuda(n, t)
    B, Sq, Hq, D = q.shape
    _, Sk, Hkv, _ = k.shape
    if not cross and Sq != Sk:
        raise ValueError("self-attention needs Sq == Sk (use cross=True for a key-only mask)")
    cu_k, pos_k = attn_mask_to_varlen(mask, stream)
    kp, vp = attn_pack_rows(k, pos_k, cu_k, stream), attn_pack_rows(v, pos_k, cu_k, stream)
    if cross:
        qp = q.view(B * Sq, Hq, D)
        cu_q = torch.arange(0, (B + 1) * Sq, Sq, dtype=torch.int32, device=q.device)
    else:
        qp, cu_q = attn_pack_rows(q, pos_k, cu_k, stream), cu_k
    out_p, lse_p = attn_fwd_varlen(qp, kp, vp, cu_q, cu_k, Sq, Sk, softmax_scale, causal, lse=True if lse else None,
                                   out_dtype=out_dtype, dev_status=dev_status, stream=stream)
    if cross:
        out = out_p.view(B, Sq, Hq, D)
        lse_out = lse_p.view(Hq, B, Sq).permute(1, 0, 2) if lse else None
    else:
        out = attn_unpack_rows(out_p, pos_k, B, Sq, stream)
        lse_out = attn_unpack_lse(lse_p, pos_k, B, Sq, stream) if lse else None
    return out, lse_out


def attn_vsa_layout(prefix_segments, video_shape, tile=(4, 4, 4), block=64):
    """Token blocks of block-sparse video attention (host computation).
    Returns (order int32 [tokens], block_start int32 [NB + 1], n_prefix_blocks)."""
    lib = load_library()
    seg = (ctypes.c_int32 * max(1, len(prefix_segments)))(*[int(x) for x in prefix_segments])
    nb, npre = ctypes.c_int(0), ctypes.c_int(0)
    t, h, w = (int(x) for x in video_shape)
    args = (seg, len(prefix_segments), t, h, w, int(tile[0]), int(tile[1]), int(tile[2]), int(block))
    _check("attn_vsa_layout", lib.attn_vsa_layout(*args, None, None, ctypes.byref(nb), ctypes.byref(npre)))
    order = torch.empty(sum(int(x) for x in prefix_segments) + t * h * w, dtype=torch.int32)
    start = torch.empty(nb.value + 1, dtype=torch.int32)
    _check("attn_vsa_layout", lib.attn_vsa_layout(*args, _ptr(order), _ptr(start), ctypes.byref(nb),
                                                  ctypes.byref(npre)))
    return order, start, npre.value


def attn_vsa_tile_map(prefix_segments, video_shape, tile=(4, 4, 4)):
    """Tiled layout of block-sparse video attention (host computation, 64-token
    blocks).  Returns (tile_index int32 [nbp * 64], block_sizes int32 [nb],
    n_prefix_blocks), host tensors."""
    lib = load_library()
    seg = (ctypes.c_int32 * max(1, len(prefix_segments)))(*[int(x) for x in prefix_segments])
    nb, npre = ctypes.c_int(0), ctypes.c_int(0)
    t, h, w = (int(x) for x in video_shape)
    args = (seg, len(prefix_segments), t, h, w, int(tile[0]), int(tile[1]), int(tile[2]))
    _check("attn_vsa_tile_map", lib.attn_vsa_tile_map(*args, None, None, ctypes.byref(nb), ctypes.byref(npre)))
    index = torch.empty((nb.value + nb.value % 2) * 64, dtype=torch.int32)
    sizes = torch.empty(nb.value, dtype=torch.int32)
    _check("attn_vsa_tile_map", lib.attn_vsa_tile_map(*args, _ptr(index), _ptr(sizes), ctypes.byref(nb),
                                                      ctypes.byref(npre)))
    return index, sizes, npre.value


def attn_gather_rows(src, index, dev_status=None, stream=None):
    """src [N, ...] contiguous CUDA, index int32 CUDA [M] -> dst [M, ...]:
    dst[w] = src[index[w]], zero rows where index[w] < 0."""
    if not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous CUDA tensor")
    if index.dtype != torch.int32 or not index.is_cuda or not index.is_contiguous():
        raise ValueError("index must be a contiguous int32 CUDA tensor")
    M = index.numel()
    dst = torch.empty((M,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    rb = src[0].numel() * src.element_size() if src.shape[0] > 0 else dst[0].numel() * dst.element_size()
    st = load_library().attn_gather_rows(_ptr(src), src.shape[0], _ptr(index), M, rb, _ptr(dst), _ptr(dev_status),
                                         _stream_handle(stream))
    _check("attn_gather_rows", st)
    return dst


def attn_vsa_pool(x_tiled, block_sizes, dev_status=None, stream=None):
    """x_tiled [rows >= nb * 64, H, D] bf16 CUDA, block_sizes int32 CUDA [nb]
    -> pooled [H, nb, D] fp32 block means."""
    _bf16_cuda("x_tiled", x_tiled)
    if block_sizes.dtype != torch.int32 or not block_sizes.is_cuda or not block_sizes.is_contiguous():
        raise ValueError("block_sizes must be a contiguous int32 CUDA tensor")
    nb = block_sizes.numel()
    _, H, D = x_tiled.shape
    if x_tiled.shape[0] < nb * 64:
        raise ValueError("x_tiled has fewer than 64 rows per block")
    pooled = torch.empty(H, nb, D, dtype=torch.float32, device=x_tiled.device)
    st = load_library().attn_vsa_pool(_ptr(x_tiled), nb, H, D, _ptr(block_sizes), _ptr(pooled), _ptr(dev_status),
                                      _stream_handle(stream))
    _check("attn_vsa_pool", st)
    return pooled


def attn_vsa_list_size(num_blocks, num_prefix_blocks, topk, Hq) -> int:
    n = ctypes.c_longlong(0)
    _check("attn_vsa_list_size", load_library().attn_vsa_list_size(num_blocks, num_prefix_blocks, topk, Hq,
                                                                   ctypes.byref(n)))
    return n.value


def attn_vsa_block_map(pooled_q, pooled_k, block_sizes, num_prefix_blocks, topk, softmax_scale, dev_status=None,
                       stream=None):
    """pooled_q [Hq, nb, D], pooled_k [Hkv, nb, D] fp32 CUDA -> (kv_list, kv_num)
    int32: per head and tile (query blocks 2t, 2t+1), the union of the key
    blocks they keep, entries (block << 9) | (size << 2) | bits."""
    if pooled_q.dim() != 3 or pooled_k.dim() != 3 or pooled_q.shape[1:] != pooled_k.shape[1:]:
        raise ValueError("pooled_q must be [Hq, nb, D] and pooled_k [Hkv, nb, D] with the same nb and D")
    if pooled_q.dtype != torch.float32 or pooled_k.dtype != torch.float32:
        raise ValueError("pooled_q and pooled_k must be float32")
    Hq, nb, D = pooled_q.shape
    Hkv = pooled_k.shape[0]
    if block_sizes.numel() != nb or block_sizes.dtype != torch.int32:
        raise ValueError(f"block_sizes must hold {nb} int32 entries (one per block)")
    for n_, t in (("pooled_q", pooled_q), ("pooled_k", pooled_k), ("block_sizes", block_sizes)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n_} must be a contiguous CUDA tensor")
    n = attn_vsa_list_size(nb, num_prefix_blocks, topk, Hq)
    kv_list = torch.empty(max(n, 1), dtype=torch.int32, device=pooled_q.device)
    kv_num = torch.empty(Hq, (nb + 1) // 2, dtype=torch.int32, device=pooled_q.device)
    st = load_library().attn_vsa_block_map(_ptr(pooled_q), _ptr(pooled_k), nb, num_prefix_blocks, Hq, Hkv, D, topk,
                                           float(softmax_scale), _ptr(block_sizes), _ptr(kv_list), _ptr(kv_num),
                                           _ptr(dev_status), _stream_handle(stream))
    _check("attn_vsa_block_map", st)
    return kv_list, kv_num


def _check_vsa_fwd_shapes(q_tiled, k_tiled, v_tiled, kv_list, kv_num, num_blocks, num_prefix_blocks, topk,
                          out_index, out_rows, out, lse):
    """Raise ValueError unless the tensors have the sizes the C call derives
    from (num_blocks, Hq, Hkv, D): its tensor maps and list reads trust them."""
    if q_tiled.dim() != 3 or k_tiled.dim() != 3 or v_tiled.dim() != 3:
        raise ValueError("q_tiled, k_tiled and v_tiled must be [rows, heads, D]")
    rows, Hq, D = q_tiled.shape
    want = (num_blocks + num_blocks % 2) * 64
    if rows != want:
        raise ValueError(f"q_tiled has {rows} rows; {num_blocks} blocks need {want} (64 per block, even count)")
    if k_tiled.shape != v_tiled.shape or k_tiled.shape[0] != rows or k_tiled.shape[2] != D:
        raise ValueError("k_tiled and v_tiled must both be [rows of q_tiled, Hkv, D of q_tiled]")
    for n_, t in (("kv_list", kv_list), ("kv_num", kv_num)):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{n_} must be a contiguous int32 tensor")
    need = attn_vsa_list_size(num_blocks, num_prefix_blocks, topk, Hq)
    if kv_list.numel() < need:
        raise ValueError(f"kv_list holds {kv_list.numel()} entries; these sizes need {need}")
    if tuple(kv_num.shape) != (Hq, (num_blocks + 1) // 2):
        raise ValueError(f"kv_num must be [Hq, (num_blocks + 1) // 2] = [{Hq}, {(num_blocks + 1) // 2}]")
    if out_index is not None and (out_index.dtype != torch.int32 or out_index.numel() != rows):
        raise ValueError(f"out_index must hold {rows} int32 entries (one per tiled row)")
    if out_index is None and out_rows != rows:
        raise ValueError("without out_index the output stays tiled: out_rows must equal the tiled row count")
    if out is not None and tuple(out.shape) != (out_rows, Hq, D):
        raise ValueError(f"out must be [out_rows, Hq, D] = [{out_rows}, {Hq}, {D}]")
    if torch.is_tensor(lse) and (tuple(lse.shape) != (Hq, out_rows) or lse.dtype != torch.float32):
        raise ValueError(f"lse must be float32 [Hq, out_rows] = [{Hq}, {out_rows}]")


def attn_fwd_vsa(q_tiled, k_tiled, v_tiled, kv_list, kv_num, num_blocks, num_prefix_blocks, topk, out_index=None,
                 out_rows=None, softmax_scale=None, lse=None, out_dtype=torch.float32, out=None, dev_status=None,
                 stream=None):
    """Block-sparse attention over tiled q [nbp*64, Hq, D], k/v [nbp*64, Hkv, D]
    (bf16 CUDA) and the lists of attn_vsa_block_map.  Row r of the tiled layout
    goes to out row out_index[r] (None: out stays tiled).  Returns (out
    [out_rows, Hq, D], lse [Hq, out_rows] or None)."""
    if out_rows is None:
        out_rows = q_tiled.shape[0]
    _check_vsa_fwd_shapes(q_tiled, k_tiled, v_tiled, kv_list, kv_num, num_blocks, num_prefix_blocks, topk,
                          out_index, out_rows, out, lse)
    for n_, t in (("q_tiled", q_tiled), ("k_tiled", k_tiled), ("v_tiled", v_tiled)):
        _bf16_cuda(n_, t)
    for n_, t in (("kv_list", kv_list), ("kv_num", kv_num), ("out_index", out_index), ("out", out), ("lse", lse)):
        if torch.is_tensor(t) and not t.is_cuda:
            raise ValueError(f"{n_} must be a CUDA tensor")
    rows, Hq, D = q_tiled.shape
    Hkv = k_tiled.shape[1]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty(out_rows, Hq, D, dtype=out_dtype, device=q_tiled.device)
    if lse is True:
        lse = torch.empty(Hq, out_rows, dtype=torch.float32, device=q_tiled.device)
    st = load_library().attn_fwd_vsa(_ptr(q_tiled), _ptr(k_tiled), _ptr(v_tiled), num_blocks, num_prefix_blocks, topk,
                                     _ptr(kv_list), _ptr(kv_num), _ptr(out_index), out_rows, Hq, Hkv, D,
                                     float(softmax_scale), _ptr(out), _out_code(out.dtype), _ptr(lse),
                                     _ptr(dev_status), _stream_handle(stream))
    _check("attn_fwd_vsa", st)
    return out, lse


class VsaPlan:
    """One geometry's tiled layout, computed on the host once and kept on the
    device (the page caches the same metadata per geometry)."""

    def __init__(self, prefix_segments, video_shape, device, tile=(4, 4, 4)):
        index, sizes, npre = attn_vsa_tile_map(prefix_segments, video_shape, tile)
        self.tokens = sum(int(x) for x in prefix_segments) + math.prod(int(x) for x in video_shape)
        self.num_blocks = sizes.numel()
        self.num_prefix_blocks = npre
        self.rows = index.numel()
        self.tile_index = index.to(device)
        self.block_sizes = sizes.to(device)


def attn_vsa(q, k, v, plan: VsaPlan, topk=64, softmax_scale=None, lse=False, out_dtype=torch.float32,
             dev_status=None, stream=None):
    """Block-sparse video attention of one sequence: q [S, Hq, D], k/v [S, Hkv, D]
    bf16 CUDA, S = plan.tokens.  Tiles q, k, v, pools q and k, builds the block
    map and attends it; returns (out [S, Hq, D], lse [Hq, S] or None)."""
    for n_, t in (("q", q), ("k", k), ("v", v)):
        _bf16_cuda(n_, t)
    S, Hq, D = q.shape
    if S != plan.tokens or k.shape[0] != S or v.shape[0] != S:
        raise ValueError(f"the plan's geometry has {plan.tokens} tokens, q/k/v have {S}")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    qt = attn_gather_rows(q, plan.tile_index, dev_status, stream)
    kt = attn_gather_rows(k, plan.tile_index, dev_status, stream)
    vt = attn_gather_rows(v, plan.tile_index, dev_status, stream)
    pq = attn_vsa_pool(qt, plan.block_sizes, dev_status, stream)
    pk = attn_vsa_pool(kt, plan.block_sizes, dev_status, stream)
    kv_list, kv_num = attn_vsa_block_map(pq, pk, plan.block_sizes, plan.num_prefix_blocks, topk, softmax_scale,
                                         dev_status, stream)
    return attn_fwd_vsa(qt, kt, vt, kv_list, kv_num, plan.num_blocks, plan.num_prefix_blocks, topk,
                        out_index=plan.tile_index, out_rows=S, softmax_scale=softmax_scale,
                        lse=True if lse else None, out_dtype=out_dtype, dev_status=dev_status, stream=stream)


# ---- gradients (gbattn_bwd.h).  These calls run on their tensors' device,
# whichever one is current, and allocate what they return (and a workspace not
# given) on the stream they run on.
def _run_on(name, dev, stream, args):
    """One C call on device number dev and stream (None: the device's current one)."""
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream must be of cuda:{dev}, where the tensors are")
    fn = getattr(_lib or load_library(), name)
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != 0:
        raise GbattnError(name, st)


def _tensor(name, t, dev, dtype, shape, strided=False):
    """Raise ValueError unless t is a contiguous (or strided) tensor of this type and shape on CUDA device number dev."""
    if t.dtype != dtype or t.shape != shape or not (strided or t.is_contiguous()):
        raise ValueError(f"{name} must be a {'' if strided else 'contiguous '}{str(dtype)[6:]} tensor {list(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, with q")


def _laid_out(stream, t):
    """t, or a contiguous copy of it made on the stream that will read it."""
    if t is None or t.is_contiguous():
        return t
    if stream is None:
        return t.detach().contiguous()
    with torch.cuda.stream(stream):
        return t.detach().contiguous()


def _row_strides(t):
    """Strides, up to the last dimension's, of a tensor whose rows of D values can be read where they lie: side by side, each
    on 16 bytes.  None if they cannot.  (A dimension of one index has no stride.)"""
    *strides, col = (0 if n == 1 else s for n, s in zip(t.shape, t.stride()))
    if col != 1 or t.data_ptr() % 16 or any(s * t.element_size() % 16 for s in strides):
        return None
    return strides


def _like(stream, t):
    """An uninitialised contiguous tensor of t's shape and type, of the stream that will write it."""
    if stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        return torch.empty_like(t, memory_format=torch.contiguous_format)


def attn_bwd_workspace_size(num_docs, Tq, Hq) -> int:
    """Bytes of workspace a backward call needs for num_docs documents (or batch entries) of Tq query rows in all."""
    return int((_lib or load_library()).attn_bwd_workspace_size(_host_int("num_docs", num_docs), _host_int("Tq", Tq), Hq))


def _bwd(name, q, k, v, out, lse, dout, dlse, index, sizes, docs, heads, lse_shape, softmax_scale, causal, dq, dk, dv,
         workspace, dev_status, stream):
    """The part the backward calls share: checks, allocation and the C call.  index: (name, tensor, entries) of the
    int32 tensors the call takes; sizes: its sizes up to D; docs: documents or batch entries."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("the gradients take CUDA tensors")
    Hq, Hkv, D = heads
    bf16, qs, ks = torch.bfloat16, q.shape, k.shape
    f32_out = out.dtype == torch.float32
    if not (q.dtype == k.dtype == v.dtype == dout.dtype == bf16 and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous() and v.shape == ks and dout.shape == qs
            and k.get_device() == v.get_device() == dout.get_device() == dev):
        for n, t, shape in (("q", q, qs), ("k", k, ks), ("v", v, ks), ("dout", dout, qs)):
            _tensor(n, t, dev, bf16, shape, strided=n == "dout")
    _tensor("out", out, dev, torch.float32 if f32_out else bf16, qs, strided=True)
    _tensor("lse", lse, dev, torch.float32, lse_shape, strided=True)
    if dlse is not None:
        _tensor("dlse", dlse, dev, torch.float32, lse_shape, strided=True)
    for n, t, entries in index:
        if t is not None:
            _tensor(n, t, dev, torch.int32, (entries,))
    status = _status_ptr(dev_status)
    if dev_status is not None and dev_status.get_device() != dev:
        raise ValueError(f"dev_status must be on cuda:{dev}, with q")
    for n, t, shape in (("dq", dq, qs), ("dk", dk, ks), ("dv", dv, ks)):
        if t is not None:
            _tensor(n, t, dev, bf16, shape)
    dq = _like(stream, q) if dq is None else dq
    dk = _like(stream, k) if dk is None else dk
    dv = _like(stream, k) if dv is None else dv
    if workspace is None:
        ws_bytes = attn_bwd_workspace_size(docs, q.numel() // (Hq * D) if Hq * D else 0, Hq)
        workspace = _empty_on(stream, q, (ws_bytes,), torch.uint8)
    elif workspace.is_contiguous() and workspace.get_device() == dev:
        ws_bytes = workspace.numel() * workspace.element_size()
    else:
        raise ValueError(f"workspace must be contiguous and on cuda:{dev}, with q")
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    # what other code computed or autograd hands over: out is read where it lies, the others are laid out
    strides = ()
    if not out.is_contiguous():
        strides = _row_strides(out)
        if strides is None:
            out, strides = _laid_out(stream, out), ()
        elif name == "attn_bwd_varlen":
            name = "attn_bwd_varlen_strided"
        else:
            name = "attn_bwd_padded_strided"
            index = index or (("lens_q", None, 0), ("lens_k", None, 0))
    dout, lse, dlse = _laid_out(stream, dout), _laid_out(stream, lse), _laid_out(stream, dlse)
    _run_on(name, dev, stream,
            (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), OUT_F32 if f32_out else OUT_BF16, *strides,
             lse.data_ptr(), dout.data_ptr(), None if dlse is None else dlse.data_ptr(),
             *[None if t is None else t.data_ptr() for _, t, _ in index], *sizes, Hq, Hkv, D, scale, 1 if causal else 0,
             dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), ws_bytes, status))
    return dq, dk, dv


def _bwd_batch(q, k):
    """(B, Sq, Sk, Hq, Hkv, D) of a batch's q and k."""
    if q.dim() != 4 or k.dim() != 4 or k.shape[0] != q.shape[0] or k.shape[3] != q.shape[3]:
        raise ValueError("q must be [B, Sq, Hq, D], k and v [B, Sk, Hkv, D]")
    B, Sq, Hq, D = q.shape
    return B, Sq, k.shape[1], Hq, k.shape[2], D


def attn_bwd_dense(q, k, v, out, lse, dout, softmax_scale=None, causal=False, dlse=None, dq=None, dk=None, dv=None,
                   workspace=None, dev_status=None, stream=None):
    """Gradients of attn_fwd_dense from what it took and returned: q, dout
    [B, Sq, Hq, D] and k, v [B, Sk, Hkv, D] bf16, out (bf16 or fp32) and lse
    [B, Hq, Sq] as it returned them, dout the gradient of out and dlse that of
    lse (None: lse is not used further on).  out, dout, lse and dlse may have
    any strides: an out whose rows of D values lie on 16 bytes is read where it
    is, the others are copied first unless they are contiguous.  Returns (dq,
    dk, dv) in bf16; tensors given for them are written and must not overlap the
    inputs.  A workspace of at least ``attn_bwd_workspace_size(B, B * Sq, Hq)``
    bytes may be passed (it is allocated here otherwise); calls that can overlap
    need one each."""
    B, Sq, Sk, Hq, Hkv, D = _bwd_batch(q, k)
    return _bwd("attn_bwd_dense", q, k, v, out, lse, dout, dlse, (), (B, Sq, Sk), B, (Hq, Hkv, D), (B, Hq, Sq),
                softmax_scale, causal, dq, dk, dv, workspace, dev_status, stream)


def attn_bwd_padded(q, k, v, out, lse, dout, lens_q=None, lens_k=None, softmax_scale=None, causal=False, dlse=None,
                    dq=None, dk=None, dv=None, workspace=None, dev_status=None, stream=None):
    """Gradients of attn_fwd_padded: as attn_bwd_dense, entry b using its first
    lens_q[b] query rows and lens_k[b] keys (int32 [B], or None for all rows).
    Rows past them get zeros and never reach a result, whatever they hold."""
    B, Sq, Sk, Hq, Hkv, D = _bwd_batch(q, k)
    return _bwd("attn_bwd_padded", q, k, v, out, lse, dout, dlse, (("lens_q", lens_q, B), ("lens_k", lens_k, B)),
                (B, Sq, Sk), B, (Hq, Hkv, D), (B, Hq, Sq), softmax_scale, causal, dq, dk, dv, workspace, dev_status, stream)


def attn_bwd_varlen(q, k, v, out, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, softmax_scale=None,
                    causal=False, dlse=None, dq=None, dk=None, dv=None, workspace=None, dev_status=None, stream=None):
    """Gradients of attn_fwd_varlen: q, out, dout [Tq, Hq, D], k, v [Tk, Hkv,
    D], lse [Hq, Tq], cu_seqlens int32 [N + 1], max_seqlen_q/k host ints;
    strides as for attn_bwd_dense.  Returns (dq, dk, dv); rows that belong to no
    document are left as they were.  Workspace: ``attn_bwd_workspace_size(N, Tq,
    Hq)`` bytes."""
    if q.dim() != 3 or k.dim() != 3 or k.shape[2] != q.shape[2]:
        raise ValueError("q must be [Tq, Hq, D], k and v [Tk, Hkv, D]")
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    N = cu_seqlens_q.numel() - 1
    if N < 0:
        raise ValueError("cu_seqlens_q must have a boundary more than there are documents")
    return _bwd("attn_bwd_varlen", q, k, v, out, lse, dout, dlse,
                (("cu_seqlens_q", cu_seqlens_q, N + 1), ("cu_seqlens_k", cu_seqlens_k, N + 1)),
                (N, Tq, Tk, _host_int("max_seqlen_q", max_seqlen_q), _host_int("max_seqlen_k", max_seqlen_k)), N,
                (Hq, Hkv, D), (Hq, Tq), softmax_scale, causal, dq, dk, dv, workspace, dev_status, stream)


# ---- rotary positions (gbattn_rotary.h)
ROTARY_SCALINGS = {"linear": 1, "ntk": 2, "by_parts": 3, "yarn": 4}  # gbattn_rotary_scaling


def attn_rotary_frequencies(rot_dim, base=10000.0, scaling=None):
    """(frequencies, gain) of a head whose first rot_dim values are turned, as
    Python floats.  scaling: None, or a dict with "kind" (linear, ntk, by_parts,
    yarn), "factor", and for the last two "low", "high" and "length" (the
    trained length); gbattn_rotary.h has the formulas."""
    scaling = dict(scaling or {})
    kind = scaling.pop("kind", None)
    if kind is not None and kind not in ROTARY_SCALINGS:
        raise ValueError(f"scaling kind must be one of {sorted(ROTARY_SCALINGS)}")
    takes = () if kind is None else ("factor",) if kind in ("linear", "ntk") else ("factor", "low", "high", "length")
    if sorted(scaling) != sorted(takes):
        raise ValueError(f"scaling {kind} takes {', '.join(takes) or 'nothing'}")
    n = max(int(rot_dim) // 2, 0)
    f, gain = (ctypes.c_double * max(n, 1))(), ctypes.c_double()
    st = load_library().attn_rotary_frequencies(_host_int("rot_dim", rot_dim), float(base), ROTARY_SCALINGS.get(kind, 0),
                                                *(float(scaling.get(x, 0.0)) for x in ("factor", "low", "high", "length")),
                                                f, ctypes.byref(gain))
    _check("attn_rotary_frequencies", st)
    return list(f)[:n], gain.value


def attn_rotary_steps(inv_freq):
    """Frequencies (floats) as fixed-point turns: Python ints, f / 2 pi modulo 1 in units of 2^-64."""
    n = len(inv_freq)
    f, steps = (ctypes.c_double * max(n, 1))(*map(float, inv_freq)), (ctypes.c_uint64 * max(n, 1))()
    _check("attn_rotary_steps", load_library().attn_rotary_steps(f, n, steps))
    return list(steps)[:n]


class RotaryPlan:
    """A head's rotary frequencies on the device, made once and given to
    attn_rotary and attn_rotary_kv_cache_write: the first rot_dim values are
    turned, in pairs (i, i + rot_dim / 2) or, interleaved, (2 i, 2 i + 1).
    scaling as for attn_rotary_frequencies; or inv_freq, rot_dim / 2 frequencies
    of one's own.  gain (None: the scaling's, 1 but for yarn) multiplies what is
    turned."""

    def __init__(self, rot_dim, base=10000.0, interleaved=False, scaling=None, inv_freq=None, gain=None, device="cuda"):
        if inv_freq is None:
            self.inv_freq, own_gain = attn_rotary_frequencies(rot_dim, base, scaling)
        else:
            if scaling is not None:
                raise ValueError("give a scaling or the frequencies themselves")
            self.inv_freq, own_gain = [float(f) for f in inv_freq], 1.0
            if 2 * len(self.inv_freq) != rot_dim:
                raise ValueError(f"inv_freq must hold {rot_dim // 2} frequencies")
        self.rot_dim, self.interleaved = int(rot_dim), bool(interleaved)
        self.gain = own_gain if gain is None else float(gain)
        steps = [s - (1 << 64) if s >> 63 else s for s in attn_rotary_steps(self.inv_freq)]
        self.steps = torch.tensor(steps, dtype=torch.int64).to(device)


def _rotary_rows(name, t, dev, shape):
    """Token stride of a bf16 tensor [T, heads, D] (given as shape) on device number dev, whose [heads, D] rows are
    contiguous."""
    if t.dtype != torch.bfloat16 or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a bfloat16 tensor {list(shape)} on cuda:{dev}, as q")
    T, heads, d = shape
    tokens, row, col = t.stride()
    if col != 1 or (row != d and heads > 1):
        raise ValueError(f"{name}: a token's [heads, D] must be contiguous")
    return tokens if T > 1 else heads * d


def _rotary_shape(name, t):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, D]")
    return t.shape


def attn_rotary(q, k, positions, plan: RotaryPlan, transpose=False, q_out=None, k_out=None, stream=None):
    """Turn queries q [T, Hq, D] and keys k [T, Hkv, D] (bf16; tokens may be
    strided, as parts of a fused projection's output; k may be None) by their
    positions [T] (int32).  transpose=True turns gradients back.  Returns
    (q_out, k_out): new tensors, or those given, which may be q and k
    themselves (in place) and must not overlap the inputs in another way."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("attn_rotary takes CUDA tensors")
    shape = _rotary_shape("q", q)
    T, Hq, D = shape
    qs = _rotary_rows("q", q, dev, shape)
    Hkv = ks = kos = 0
    if k is not None:
        Hkv = _rotary_shape("k", k)[1]
        k_shape = (T, Hkv, D)
        ks = _rotary_rows("k", k, dev, k_shape)
    elif k_out is not None:
        raise ValueError("k_out is given without k")
    _tensor("positions", positions, dev, torch.int32, (T,))
    _tensor("plan.steps", plan.steps, dev, torch.int64, (plan.rot_dim // 2,))
    if q_out is None:
        q_out = _like(stream, q)
        qos = Hq * D
    else:
        qos = _rotary_rows("q_out", q_out, dev, shape)
    if k is not None:
        if k_out is None:
            k_out = _like(stream, k)
            kos = Hkv * D
        else:
            kos = _rotary_rows("k_out", k_out, dev, k_shape)
    _run_on("attn_rotary", dev, stream,
            (q.data_ptr(), qs, None if k is None else k.data_ptr(), ks, positions.data_ptr(), T, plan.steps.data_ptr(),
             plan.rot_dim, 1 if plan.interleaved else 0, 1 if transpose else 0, plan.gain, Hq, Hkv, D, q_out.data_ptr(), qos,
             None if k is None else k_out.data_ptr(), kos))
    return q_out, k_out


def attn_rotary_kv_cache_write(q, key, value, positions, plan: RotaryPlan, slot_mapping, kv_cache, q_out=None,
                               dev_status=None, stream=None):
    """attn_rotary of q, and attn_kv_cache_write of the turned key and of value
    into kv_cache [2, nb, bs, Hkv, D], in place, at slot_mapping [T] (int32;
    negative: not stored; a slot is to be given once), in one pass.  q [T, Hq,
    D], key, value [T, Hkv, D]; tokens may be strided.  Returns q_out: a new
    tensor, or the one given, which may be q itself."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("attn_rotary_kv_cache_write takes CUDA tensors")
    shape = _rotary_shape("q", q)
    T, Hq, D = shape
    Hkv = _rotary_shape("key", key)[1]
    k_shape = (T, Hkv, D)
    qs, ks, vs = (_rotary_rows("q", q, dev, shape), _rotary_rows("key", key, dev, k_shape),
                  _rotary_rows("value", value, dev, k_shape))
    _tensor("positions", positions, dev, torch.int32, (T,))
    _tensor("slot_mapping", slot_mapping, dev, torch.int32, (T,))
    _tensor("plan.steps", plan.steps, dev, torch.int64, (plan.rot_dim // 2,))
    if kv_cache.dim() != 5 or kv_cache.shape[0] != 2 or kv_cache.shape[3:] != (Hkv, D):
        raise ValueError(f"kv_cache must be [2, num_blocks, block_size, {Hkv}, {D}]")
    _tensor("kv_cache", kv_cache, dev, torch.bfloat16, kv_cache.shape)
    status = _status_ptr(dev_status)
    if dev_status is not None and dev_status.get_device() != dev:
        raise ValueError(f"dev_status must be on cuda:{dev}, with q")
    if q_out is None:
        q_out = _like(stream, q)
        qos = Hq * D
    else:
        qos = _rotary_rows("q_out", q_out, dev, shape)
    _run_on("attn_rotary_kv_cache_write", dev, stream,
            (q.data_ptr(), qs, key.data_ptr(), ks, value.data_ptr(), vs, positions.data_ptr(), slot_mapping.data_ptr(), T,
             plan.steps.data_ptr(), plan.rot_dim, 1 if plan.interleaved else 0, plan.gain, q_out.data_ptr(), qos,
             kv_cache.data_ptr(), kv_cache.shape[1], kv_cache.shape[2], Hq, Hkv, D, status))
    return q_out
