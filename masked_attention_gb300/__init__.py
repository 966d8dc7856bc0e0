"""Masked fused attention for one GB300 GPU (sm_103a).

A thin ctypes binding of ``libmattn.so`` (C ABI in ``include/mattn.h``). The
functions here only marshal arguments: every step of the computation runs in
the library's CUDA kernels. There is no CPU fallback: if the library has not
been built (``python -m masked_attention_gb300._build``), loading it raises.

Tensors are passed as torch CUDA tensors (or raw device addresses as ints);
PyTorch provides device memory and streams only.

With the environment variable ``MATTN_DEBUG=1`` set before the first call,
the debug build ``libmattn_debug.so`` is loaded instead (device-side bounds
checks, ``include/mattn_debug.h``; build it with
``python -m masked_attention_gb300._build --debug``); ``debug_record`` and
``debug_selftest`` read and test its checks.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

__all__ = [
    "MASK_CAUSAL", "MASK_WINDOW", "MASK_DOCUMENT", "MASK_PREFIX", "SCORE_ALIBI",
    "SCORE_SOFTCAP", "BF16", "F32", "AttnError", "BlockMask", "attn_fwd", "attn_bwd",
    "attn_decode", "attn_decode_workspace_bytes",
    "build_block_mask", "attn_block_mask_bytes", "attn_bwd_workspace_bytes", "attn_bwd_noalloc",
    "attn_check_status", "attn_status_str", "attn_last_cuda_error", "attn_combine", "lib",
    "LIB_PATH", "LIB_DEBUG_PATH", "debug_record", "debug_selftest",
    "attn_page_plan", "attn_qk_norm_rope", "attn_qk_norm_rope_bwd",
    "attn_qk_norm_rope_bwd_workspace_bytes", "attn_qk_norm_rope_axes",
    "attn_qk_norm_rope_axes_bwd", "attn_cache_q4_bytes", "attn_cache_store_q4",
    "attn_cache_load_q4", "attn_decode_q4", "attn_decode_q4_workspace_bytes",
    "attn_decode_shared", "attn_decode_shared_workspace_bytes", "attn_key_weights",
    "attn_cache_evict",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmattn.so")
LIB_DEBUG_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmattn_debug.so")

# Mirrors of the constants in include/mattn.h (a test checks they agree).
ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_MISALIGNED = 0, 1, 2, 3
ATTN_ERR_WORKSPACE_TOO_SMALL, ATTN_ERR_CUDA, ATTN_ERR_TIMEOUT = 4, 5, 6
MASK_CAUSAL, MASK_WINDOW, MASK_DOCUMENT, MASK_PREFIX = 1 << 0, 1 << 1, 1 << 2, 1 << 3
SCORE_ALIBI, SCORE_SOFTCAP, SCORE_RELBIAS = 1 << 8, 1 << 9, 1 << 10
BF16, F32 = 0, 1
TILE = 128
FAULT_NO_LOADS = 1


class attn_block_mask(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Sq", ctypes.c_int), ("Skv", ctypes.c_int),
                ("nq", ctypes.c_int), ("nkv", ctypes.c_int), ("variant", ctypes.c_uint),
                ("window", ctypes.c_int), ("doc_id", ctypes.c_void_p),
                ("prefix_len", ctypes.c_void_p), ("full_cnt", ctypes.c_void_p),
                ("part_cnt", ctypes.c_void_p), ("full_idx", ctypes.c_void_p),
                ("part_idx", ctypes.c_void_p), ("order", ctypes.c_void_p),
                ("t_full_cnt", ctypes.c_void_p), ("t_part_cnt", ctypes.c_void_p),
                ("t_full_idx", ctypes.c_void_p), ("t_part_idx", ctypes.c_void_p),
                ("t_order", ctypes.c_void_p), ("q_offset", ctypes.c_int),
                ("kv_offset", ctypes.c_int), ("doc_len", ctypes.c_int)]


class attn_params(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("window", ctypes.c_int),
                ("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p),
                ("doc_id", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
                ("block_mask", ctypes.POINTER(attn_block_mask)), ("status", ctypes.c_void_p),
                ("timeout_ns", ctypes.c_ulonglong), ("rel_bias", ctypes.c_void_p),
                ("fault_inject", ctypes.c_uint), ("page_table", ctypes.c_void_p),
                ("page_size", ctypes.c_int), ("pages_per_seq", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("q_offset", ctypes.c_int),
                ("kv_offset", ctypes.c_int), ("doc_len", ctypes.c_int)]


class attn_view(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_longlong),
                ("stride_h", ctypes.c_longlong), ("stride_s", ctypes.c_longlong)]


class attn_rope_params(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p),
                ("max_pos", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("positions", ctypes.c_void_p)]


class attn_debug_info(ctypes.Structure):
    _fields_ = [("count", ctypes.c_ulonglong), ("site", ctypes.c_int), ("pad", ctypes.c_int),
                ("index", ctypes.c_longlong), ("bound", ctypes.c_longlong)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        debug = os.environ.get("MATTN_DEBUG", "0") not in ("", "0")
        path = LIB_DEBUG_PATH if debug else LIB_PATH
        if not os.path.exists(path):
            flag = " --debug" if debug else ""
            raise RuntimeError(f"{path} is missing: build it with "
                               f"`python -m masked_attention_gb300._build{flag}` (no CPU fallback)")
        L = ctypes.CDLL(path)
        vp, i, u, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
        P = ctypes.POINTER(attn_params)
        BM = ctypes.POINTER(attn_block_mask)
        L.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, u, P, vp]
        L.attn_fwd.restype = i
        L.attn_block_mask_bytes.argtypes = [i, i, i, i]
        L.attn_block_mask_bytes.restype = sz
        L.build_block_mask.argtypes = [u, P, i, i, i, vp, sz, i, BM, vp]
        L.build_block_mask.restype = i
        L.attn_bwd_workspace_bytes.argtypes = [i, i, i]
        L.attn_bwd_workspace_bytes.restype = sz
        L.attn_bwd_workspace_bytes_f16.argtypes = [i, i, i, i, i, i]
        L.attn_bwd_workspace_bytes_f16.restype = sz
        L.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, i, i, u, P,
                               vp]
        L.attn_bwd.restype = i
        L.attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, u,
                                       P, vp]
        L.attn_bwd_noalloc.restype = i
        L.attn_doc_ids_from_seqlens.argtypes = [vp, i, i, vp, vp]
        L.attn_doc_ids_from_seqlens.restype = i
        L.attn_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, u, P, vp, sz, vp]
        L.attn_decode.restype = i
        L.attn_decode_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.attn_decode_workspace_bytes.restype = sz
        L.attn_combine.argtypes = [vp, vp, i, ctypes.c_longlong, i, i, vp, vp, vp]
        L.attn_combine.restype = i
        V, R = ctypes.POINTER(attn_view), ctypes.POINTER(attn_rope_params)
        L.attn_page_plan.argtypes = [vp, vp, i, vp, i, i, vp, i, vp, vp, vp, vp, vp, i, vp, vp]
        L.attn_page_plan.restype = i
        L.attn_qk_norm_rope.argtypes = [V, V, V, V, i, i, i, i, i, R, vp]
        L.attn_qk_norm_rope.restype = i
        L.attn_qk_norm_rope_bwd_workspace_bytes.argtypes = [i]
        L.attn_qk_norm_rope_bwd_workspace_bytes.restype = sz
        L.attn_qk_norm_rope_bwd.argtypes = [V, V, V, V, V, V, vp, vp, vp, sz, i, i, i, i, i, R, vp]
        L.attn_qk_norm_rope_bwd.restype = i
        cp = ctypes.c_char_p
        L.attn_qk_norm_rope_axes.argtypes = [V, V, V, V, i, i, i, i, i, R, i, cp, vp]
        L.attn_qk_norm_rope_axes.restype = i
        L.attn_qk_norm_rope_axes_bwd.argtypes = [V, V, V, V, V, V, vp, vp, vp, sz, i, i, i, i, i,
                                                 R, i, cp, vp]
        L.attn_qk_norm_rope_axes_bwd.restype = i
        L.attn_cache_q4_bytes.argtypes = [i, i, i, i]
        L.attn_cache_q4_bytes.restype = sz
        L.attn_cache_store_q4.argtypes = [V, V, vp, vp, i, i, i, i, i, i, vp]
        L.attn_cache_store_q4.restype = i
        L.attn_cache_load_q4.argtypes = [vp, i, i, vp, V, V, i, i, i, i, vp]
        L.attn_cache_load_q4.restype = i
        L.attn_decode_q4.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, u, P, vp, i, vp, sz, vp]
        L.attn_decode_q4.restype = i
        L.attn_decode_q4_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.attn_decode_q4_workspace_bytes.restype = sz
        f = ctypes.c_float
        L.attn_key_weights.argtypes = [vp, vp, vp, vp, f, vp, i, i, i, i, i, i, i, u, P, vp, vp]
        L.attn_key_weights.restype = i
        L.attn_decode_shared.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, u, P, vp, vp, vp, i,
                                         vp, sz, vp]
        L.attn_decode_shared.restype = i
        L.attn_decode_shared_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
        L.attn_decode_shared_workspace_bytes.restype = sz
        L.attn_cache_evict.argtypes = [vp, vp, i, vp, vp, i, i, i, vp, vp, i, i, vp, i, vp, i, i,
                                       i, i, i, vp, vp, vp, i, vp, vp]
        L.attn_cache_evict.restype = i
        L.attn_check_status.argtypes = [vp, vp]
        L.attn_check_status.restype = i
        L.attn_status_str.argtypes = [i]
        L.attn_status_str.restype = ctypes.c_char_p
        L.attn_last_cuda_error.argtypes = []
        L.attn_last_cuda_error.restype = ctypes.c_char_p
        if debug:
            L.attn_debug_record.argtypes = [ctypes.POINTER(attn_debug_info), i]
            L.attn_debug_record.restype = i
            L.attn_debug_site_name.argtypes = [i]
            L.attn_debug_site_name.restype = ctypes.c_char_p
            L.attn_debug_selftest.argtypes = [vp]
            L.attn_debug_selftest.restype = i
        _lib = L
    return _lib


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {attn_status_str(status)} (status {status})"
        if status == ATTN_ERR_CUDA:
            msg += f": {attn_last_cuda_error()}"
        super().__init__(msg)


def _debug_lib():
    L = lib()
    if not hasattr(L, "attn_debug_record"):
        raise RuntimeError("the release library is loaded: set MATTN_DEBUG=1 before the first "
                           "call to load libmattn_debug.so")
    return L


def debug_record(clear: bool = False) -> dict:
    """Debug build: the failed bounds checks of every kernel so far (count,
    and site name, index and bound of the first); ``clear`` resets them."""
    L = _debug_lib()
    info = attn_debug_info()
    _check(L.attn_debug_record(ctypes.byref(info), 1 if clear else 0), "attn_debug_record")
    return {"count": int(info.count), "site": L.attn_debug_site_name(info.site).decode(),
            "index": int(info.index), "bound": int(info.bound)}


def debug_selftest(stream=None) -> None:
    """Debug build: checks that an index planted past a buffer's end is
    refused and recorded (attn_debug_selftest); raises if not."""
    _check(_debug_lib().attn_debug_selftest(_stream(stream)), "attn_debug_selftest")


def attn_last_cuda_error() -> str:
    """Name of the CUDA error behind this thread's most recent ATTN_ERR_CUDA."""
    return lib().attn_last_cuda_error().decode()


def attn_status_str(status: int) -> str:
    return lib().attn_status_str(int(status)).decode()


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != ATTN_OK:
        raise AttnError(status, where)


class BlockMask:
    """A block mask built on the device. Holds the device buffer (a torch
    uint8 tensor) and the host struct that describes it."""

    def __init__(self, buf, struct: attn_block_mask, keep_alive: tuple):
        self.buf = buf
        self.struct = struct
        self._keep = keep_alive

    @property
    def nq(self) -> int:
        return self.struct.nq

    @property
    def nkv(self) -> int:
        return self.struct.nkv

    def to_host(self) -> dict:
        """Copies the lists to the host (for tests and inspection)."""
        import torch
        s = self.struct
        base = self.buf.data_ptr()

        def view(addr, n):
            off = addr - base
            return self.buf[off:off + 4 * n].view(torch.int32).cpu().numpy()

        B, nq, nkv = s.B, s.nq, s.nkv
        out = dict(full_cnt=view(s.full_cnt, B * nq).reshape(B, nq),
                   part_cnt=view(s.part_cnt, B * nq).reshape(B, nq),
                   full_idx=view(s.full_idx, B * nq * nkv).reshape(B, nq, nkv),
                   part_idx=view(s.part_idx, B * nq * nkv).reshape(B, nq, nkv),
                   order=view(s.order, B * nq))
        if s.t_full_cnt:
            out.update(t_full_cnt=view(s.t_full_cnt, B * nkv).reshape(B, nkv),
                       t_part_cnt=view(s.t_part_cnt, B * nkv).reshape(B, nkv),
                       t_full_idx=view(s.t_full_idx, B * nkv * nq).reshape(B, nkv, nq),
                       t_part_idx=view(s.t_part_idx, B * nkv * nq).reshape(B, nkv, nq),
                       t_order=view(s.t_order, B * nkv))
        return out


def _params(dtype: int, scale: float, window: int, softcap: float, alibi_slopes, doc_id,
            prefix_len, block_mask: Optional[BlockMask], status, timeout_ns: int,
            fault_inject: int = 0, rel_bias=None, q_offset: int = 0,
            kv_offset: int = 0) -> attn_params:
    p = attn_params()
    p.dtype = dtype
    p.scale = scale
    p.window = window
    p.softcap = softcap
    p.alibi_slopes = _ptr(alibi_slopes)
    p.doc_id = _ptr(doc_id)
    p.prefix_len = _ptr(prefix_len)
    p.block_mask = ctypes.pointer(block_mask.struct) if block_mask is not None else None
    p.status = _ptr(status)
    p.timeout_ns = timeout_ns
    p.fault_inject = fault_inject
    p.rel_bias = _ptr(rel_bias)
    p.q_offset = q_offset
    p.kv_offset = kv_offset
    # the row length of the document ids, from the tensor ([B, L] or [L])
    p.doc_len = int(doc_id.shape[-1]) if doc_id is not None and hasattr(doc_id, "shape") else 0
    return p


def attn_block_mask_bytes(B: int, Sq: int, Skv: int, transposed: bool = False) -> int:
    return int(lib().attn_block_mask_bytes(B, Sq, Skv, int(transposed)))


def attn_bwd_workspace_bytes(B: int, Hq: int, Sq: int) -> int:
    return int(lib().attn_bwd_workspace_bytes(B, Hq, Sq))


def attn_bwd_workspace_bytes_f16(B: int, Hq: int, Hkv: int, Sq: int, Skv: int, D: int) -> int:
    """Workspace bytes for attn_bwd's fp16 path (fp16 copies of q, k, v, dO)."""
    return int(lib().attn_bwd_workspace_bytes_f16(B, Hq, Hkv, Sq, Skv, D))


def build_block_mask(variant: int, B: int, Sq: int, Skv: int, *, window: int = 0, doc_id=None,
                     prefix_len=None, transposed: bool = False, device="cuda",
                     buf=None, q_offset: int = 0, kv_offset: int = 0,
                     stream=None) -> BlockMask:
    """Builds the block mask on the device (``buf``: optional caller buffer,
    a uint8 CUDA tensor of at least ``attn_block_mask_bytes`` bytes).
    ``q_offset``/``kv_offset``: absolute positions of query row 0 and key 0
    (one shard of a longer sequence)."""
    import torch
    nbytes = attn_block_mask_bytes(B, Sq, Skv, transposed)
    if buf is None:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    p = _params(BF16, 0.0, window, 0.0, None, doc_id, prefix_len, None, None, 0,
                q_offset=q_offset, kv_offset=kv_offset)
    out = attn_block_mask()
    st = lib().build_block_mask(variant, ctypes.byref(p), B, Sq, Skv, _ptr(buf),
                                buf.numel() if hasattr(buf, "numel") else nbytes,
                                int(transposed), ctypes.byref(out), _stream(stream))
    _check(st, "build_block_mask")
    return BlockMask(buf, out, (doc_id, prefix_len))


def attn_fwd(q, k, v, o, lse, variant: int = 0, *, B=None, Hq=None, Hkv=None, Sq=None,
             Skv=None, D=None, dtype: Optional[int] = None, scale: float = 0.0, window: int = 0,
             softcap: float = 0.0, alibi_slopes=None, doc_id=None, prefix_len=None,
             block_mask: Optional[BlockMask] = None, status=None, timeout_ns: int = 0,
             fault_inject: int = 0, rel_bias=None, page_table=None, page_size: int = 0,
             q_offset: int = 0, kv_offset: int = 0, stream=None) -> None:
    """O and LSE of masked attention; writes ``o`` and ``lse`` in place.

    Paged K/V cache: ``k``/``v`` are page pools [num_pages, Hkv, page_size, D]
    and ``page_table`` [B, pages_per_seq] int32 maps logical to physical pages;
    pass ``Skv`` (the shapes cannot tell it).

    One shard of a longer sequence: ``q_offset``/``kv_offset`` are the
    absolute positions of query row 0 and key 0 (mask terms, ALiBi and
    document ids use absolute positions); merge the results over key shards
    with ``attn_combine``.

    ``q`` [B,Hq,Sq,D], ``k``/``v`` [B,Hkv,Skv,D], ``o`` like ``q``, ``lse`` fp32
    [B,Hq,Sq]. Shapes come from the tensors unless given explicitly (needed
    when raw addresses are passed)."""
    if B is None:
        B, Hq, Sq, D = q.shape
        Hkv = k.shape[1]
        if Skv is None:
            Skv = k.shape[2]
    if dtype is None:
        import torch
        dtype = F32 if q.dtype == torch.float32 else BF16
    p = _params(dtype, scale, window, softcap, alibi_slopes, doc_id, prefix_len, block_mask,
                status, timeout_ns, fault_inject, rel_bias, q_offset, kv_offset)
    if page_table is not None:
        p.page_table = _ptr(page_table)
        p.page_size = page_size
        p.pages_per_seq = page_table.shape[1]
        p.num_pages = k.shape[0]
    st = lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Skv, D,
                        variant, ctypes.byref(p), _stream(stream))
    _check(st, "attn_fwd")


def attn_decode_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, Skv: int, D: int) -> int:
    return int(lib().attn_decode_workspace_bytes(B, Hq, Hkv, Sq, Skv, D))


def attn_decode(q, k, v, o, lse, variant: int = 0, *, workspace=None, Skv=None,
                scale: float = 0.0, window: int = 0, softcap: float = 0.0, alibi_slopes=None,
                doc_id=None, prefix_len=None, status=None, timeout_ns: int = 0, rel_bias=None,
                page_table=None, page_size: int = 0, q_offset: int = 0, kv_offset: int = 0,
                stream=None) -> None:
    """Decode: few query rows (q [B,Hq,Sq,D], (Hq/Hkv) * Sq <= 16) against a
    long key/value cache, contiguous [B,Hkv,Skv,D] or paged (``page_table``
    [B, pages_per_seq] into pools [num_pages, Hkv, page_size, D]; pass
    ``Skv``). ``workspace``: optional CUDA tensor for the split partial
    results (``attn_decode_workspace_bytes``). Writes ``o`` and ``lse``."""
    B, Hq, Sq, D = q.shape
    Hkv = k.shape[1]
    if Skv is None:
        Skv = k.shape[2]
    p = _params(BF16, scale, window, softcap, alibi_slopes, doc_id, prefix_len, None, status,
                timeout_ns, 0, rel_bias, q_offset, kv_offset)
    if page_table is not None:
        p.page_table = _ptr(page_table)
        p.page_size = page_size
        p.pages_per_seq = page_table.shape[1]
        p.num_pages = k.shape[0]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Skv,
                           D, variant, ctypes.byref(p), _ptr(workspace), ws_bytes,
                           _stream(stream))
    _check(st, "attn_decode")


def attn_combine(o_parts, lse_parts, o, lse, stream=None) -> None:
    """Merges results over disjoint key sets (e.g. key/value shards):
    ``o_parts`` [n, ...rows..., D] (bf16 or fp32 CUDA tensor), ``lse_parts``
    fp32 [n, ...rows...]; writes ``o`` [...rows..., D] and ``lse``
    [...rows...] in place: LSE = ln sum_k exp(LSE_k), O = sum_k
    exp(LSE_k - LSE) O_k."""
    import torch
    for name, x in (("o_parts", o_parts), ("lse_parts", lse_parts), ("o", o), ("lse", lse)):
        if not x.is_contiguous():
            raise ValueError(f"attn_combine: {name} must be contiguous")
    n, D = o_parts.shape[0], o_parts.shape[-1]
    rows = lse_parts[0].numel()
    if o.numel() != rows * D or lse.numel() != rows or o_parts.numel() != n * rows * D:
        raise ValueError("attn_combine: shapes of the parts and the outputs disagree")
    dtype = F32 if o_parts.dtype == torch.float32 else BF16
    st = lib().attn_combine(_ptr(o_parts), _ptr(lse_parts), n, rows, D, dtype, _ptr(o),
                            _ptr(lse), _stream(stream))
    _check(st, "attn_combine")


def doc_ids_from_seqlens(cu_seqlens, total: Optional[int] = None, doc_id=None,
                         stream=None):
    """Jagged batches: per-position sequence index of ``total`` packed
    positions from the cumulative lengths ``cu_seqlens`` (int32 CUDA tensor,
    n + 1 entries starting at 0). Use the result as ``doc_id`` ([1, total])
    with ``MASK_DOCUMENT`` and B = 1 to attend within each sequence only."""
    import torch
    n = cu_seqlens.numel() - 1
    if total is None:
        total = int(cu_seqlens[-1].item())
    if doc_id is None:
        doc_id = torch.empty(1, total, dtype=torch.int32, device=cu_seqlens.device)
    st = lib().attn_doc_ids_from_seqlens(_ptr(cu_seqlens), n, total, _ptr(doc_id),
                                         _stream(stream))
    _check(st, "attn_doc_ids_from_seqlens")
    return doc_id


def attn_bwd(q, k, v, o, lse, do, dq, dk, dv, workspace, variant: int = 0, *,
             scale: float = 0.0, window: int = 0, softcap: float = 0.0, alibi_slopes=None,
             doc_id=None, prefix_len=None, block_mask: Optional[BlockMask] = None, status=None,
             timeout_ns: int = 0, fault_inject: int = 0, q_offset: int = 0, kv_offset: int = 0,
             rel_bias=None, stream=None) -> None:
    """dQ, dK, dV of ``sum(dO * O)``; writes ``dq``, ``dk``, ``dv`` in place.
    ``workspace``: a CUDA tensor of at least ``attn_bwd_workspace_bytes`` bytes.
    ``q_offset``/``kv_offset``: absolute positions of query row 0 and key 0
    (one shard of a longer sequence; the block mask must be built for them).
    ``rel_bias``: the forward's relative-position bias table (no gradient)."""
    import torch
    B, Hq, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    dtype = F32 if q.dtype == torch.float32 else BF16
    p = _params(dtype, scale, window, softcap, alibi_slopes, doc_id, prefix_len, block_mask,
                status, timeout_ns, fault_inject, rel_bias=rel_bias, q_offset=q_offset,
                kv_offset=kv_offset)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq),
                        _ptr(dk), _ptr(dv), _ptr(workspace), ws_bytes, B, Hq, Hkv, Sq, Skv, D,
                        variant, ctypes.byref(p), _stream(stream))
    _check(st, "attn_bwd")


def attn_bwd_noalloc(q, k, v, o, lse, do, dq, dk, dv, variant: int = 0, *,
                     scale: float = 0.0, window: int = 0, softcap: float = 0.0,
                     alibi_slopes=None, doc_id=None, prefix_len=None,
                     block_mask: Optional[BlockMask] = None, status=None, timeout_ns: int = 0,
                     q_offset: int = 0, kv_offset: int = 0, rel_bias=None,
                     stream=None) -> None:
    """attn_bwd without a workspace argument, for callers that cannot allocate
    device memory: the library's own fixed array holds the row terms (at most
    B*Hq*Sq = 2,097,152; see include/mattn.h). Writes dq, dk, dv in place."""
    import torch
    B, Hq, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    dtype = F32 if q.dtype == torch.float32 else BF16
    p = _params(dtype, scale, window, softcap, alibi_slopes, doc_id, prefix_len, block_mask,
                status, timeout_ns, rel_bias=rel_bias, q_offset=q_offset,
                kv_offset=kv_offset)
    st = lib().attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                                _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Skv, D, variant,
                                ctypes.byref(p), _stream(stream))
    _check(st, "attn_bwd_noalloc")


# The calls below run once per layer of a decode step, where the host's time is
# what counts, so their checks are few attribute reads per tensor; what a refusal
# says is worked out only once one fails.
_torch = _current_device = _current_stream = None


def _lazy_torch():
    """torch and two of its getters; the direct ones where this torch has them
    (torch.cuda.current_stream builds a Stream object around the handle)."""
    global _torch, _current_device, _current_stream
    if _torch is None:
        import torch
        direct = torch._C
        _current_device = getattr(direct, "_cuda_getDevice", torch.cuda.current_device)
        _current_stream = getattr(direct, "_cuda_getCurrentRawStream",
                                  lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        torch.cuda.init()
        _torch = torch
    return _torch


def _refuse(where: str, name: str, x, dtype, dev: int, shape=None) -> None:
    """Raises what is wrong with a tensor argument (shape: contiguous of that shape)."""
    if not isinstance(x, _torch.Tensor):
        raise ValueError(f"{where}: {name} must be a tensor")
    if x.dtype is not dtype:
        raise ValueError(f"{where}: {name} must be {dtype}, not {x.dtype}")
    if not x.is_cuda or x.get_device() != dev:
        raise ValueError(f"{where}: {name} is on {x.device}, not on one CUDA device with the rest")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, not {tuple(x.shape)}")
    if shape is not None and not x.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")
    raise ValueError(f"{where}: the last dimension of {name} must be contiguous")


def _tensor(where: str, name: str, x, dtype, dev: int, shape) -> int:
    """Address of a contiguous tensor argument, checked."""
    try:
        if (x.dtype is dtype and x.get_device() == dev and x.shape == shape
                and x.is_contiguous()):
            return x.data_ptr()
    except AttributeError:
        pass
    _refuse(where, name, x, dtype, dev, shape)


def _view(where: str, name: str, x, dtype, dev: int, shape):
    """A [B, H, S, D] tensor of any strides with contiguous D, checked."""
    try:
        if x.dtype is dtype and x.get_device() == dev and x.shape == shape:
            sb, sh, ss, sd = x.stride()
            if sd == 1 or shape[3] == 1:
                return ctypes.byref(attn_view(x.data_ptr(), sb, sh, ss))
            _refuse(where, name, x, dtype, dev)
    except AttributeError:
        pass
    _refuse(where, name, x, dtype, dev, shape)


def _device(where: str, name: str, x) -> int:
    """Index of the CUDA device that a call's tensors are on."""
    if getattr(x, "is_cuda", False) is not True:
        raise ValueError(f"{where}: {name} must be a CUDA tensor")
    if _torch is None:
        _lazy_torch()
    return x.get_device()


def _run(where: str, fn, dev: int, stream, *args) -> None:
    """Calls fn(*args, stream) on device `dev` (on its current stream unless given)."""
    stream = _current_stream(dev) if stream is None else _stream(stream)
    if dev == _current_device():
        st = fn(*args, stream)
    else:
        with _torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != ATTN_OK:
        raise AttnError(st, where)


def attn_page_plan(cached_lens, new_lens, page_table, free_pages, seq_lens, cu_new, slots,
                   positions, seq_ids, info, *, page_size: int, stream=None) -> None:
    """Page tables and slot maps of a serving step, on the device, from the
    requests' lengths: ``cached_lens`` [B] tokens are held in the pages of
    ``page_table`` [B, pages_per_seq], ``new_lens`` [B] more come; pages they
    need are taken from ``free_pages`` in order and entered. Writes ``seq_lens``
    [B], ``cu_new`` [B + 1], per new token ``slots`` (int64), ``positions`` and
    ``seq_ids`` [max_tokens] (-1 past the last one), and ``info`` [4]: new
    tokens, pages taken, pages lacking, requests longer than their table. All
    int32 but ``slots``. ``free_pages`` is not changed: move its front past the
    pages taken before the next call. See include/mattn.h."""
    w = "attn_page_plan"
    dev = _device(w, "cached_lens", cached_lens)
    i32 = _torch.int32
    B, per = page_table.shape
    n, n_free = slots.numel(), free_pages.numel()
    _run(w, lib().attn_page_plan, dev, stream, _tensor(w, "cached_lens", cached_lens, i32, dev, (B,)),
         _tensor(w, "new_lens", new_lens, i32, dev, (B,)), B,
         _tensor(w, "page_table", page_table, i32, dev, (B, per)), per, page_size,
         _tensor(w, "free_pages", free_pages, i32, dev, (n_free,)), n_free,
         _tensor(w, "seq_lens", seq_lens, i32, dev, (B,)),
         _tensor(w, "cu_new", cu_new, i32, dev, (B + 1,)),
         _tensor(w, "slots", slots, _torch.int64, dev, (n,)),
         _tensor(w, "positions", positions, i32, dev, (n,)),
         _tensor(w, "seq_ids", seq_ids, i32, dev, (n,)), n, _tensor(w, "info", info, i32, dev, (4,)))


def _rope_params(w: str, dt, dev: int, tokens: int, D: int, q_weight, k_weight, eps, cos_sin,
                 positions, interleaved):
    if dt is not _torch.bfloat16 and dt is not _torch.float32:
        raise ValueError(f"{w}: tensors must be bfloat16 or float32, not {dt}")
    f32 = _torch.float32
    max_pos = rot_dim = 0
    qw = kw = table = pos = None
    if q_weight is not None:
        qw = _tensor(w, "q_weight", q_weight, f32, dev, (D,))
    if k_weight is not None:
        kw = _tensor(w, "k_weight", k_weight, f32, dev, (D,))
    if cos_sin is not None:
        max_pos, rot_dim = cos_sin.shape
        table = _tensor(w, "cos_sin", cos_sin, f32, dev, (max_pos, rot_dim))
    if positions is not None:
        pos = _tensor(w, "positions", positions, _torch.int32, dev, positions.shape)
        if positions.numel() != tokens:
            raise ValueError(f"{w}: positions must have {tokens} entries ([B, S])")
    return ctypes.byref(attn_rope_params(F32 if dt is f32 else BF16, eps, qw, kw, table, max_pos,
                                         rot_dim, 1 if interleaved else 0, pos))


def attn_qk_norm_rope(q, k, q_out, k_out, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                      cos_sin=None, positions=None, interleaved: bool = False,
                      stream=None) -> None:
    """Per-head RMS norm of queries and keys and their position rotation, in
    one pass. ``q``, ``q_out`` [B, Hq, S, D] and ``k``, ``k_out`` [B, Hkv, S,
    D], bf16 or fp32, of any strides with contiguous D (slices of a fused
    projection in, the attention's layout out; in place with equal strides);
    ``k`` and ``k_out`` may be None. ``q_weight``, ``k_weight`` fp32 [D] (None:
    no norm), ``cos_sin`` fp32 [max_pos, rot_dim] (rot_dim / 2 cosines, then
    the sines; None: no rotation), ``positions`` int32 [B, S] (None: 0..S-1;
    rows whose position is outside the table are not written)."""
    w = "attn_qk_norm_rope"
    dev = _device(w, "q", q)
    B, Hq, S, D = shape = q.shape
    dt = q.dtype
    p = _rope_params(w, dt, dev, B * S, D, q_weight, k_weight, eps, cos_sin, positions, interleaved)
    kv = ko = None
    Hkv = 0
    if k is not None:
        Hkv = k.shape[1]
        kv = _view(w, "k", k, dt, dev, (B, Hkv, S, D))
        ko = _view(w, "k_out", k_out, dt, dev, (B, Hkv, S, D))
    _run(w, lib().attn_qk_norm_rope, dev, stream, _view(w, "q", q, dt, dev, shape), kv,
         _view(w, "q_out", q_out, dt, dev, shape), ko, B, Hq, Hkv, S, D, p)


def attn_qk_norm_rope_bwd_workspace_bytes(D: int) -> int:
    return int(lib().attn_qk_norm_rope_bwd_workspace_bytes(D))


def attn_qk_norm_rope_bwd(q, k, dq_out, dk_out, dq, dk, *, dq_weight=None, dk_weight=None,
                          workspace, q_weight=None, k_weight=None, eps: float = 1e-6,
                          cos_sin=None, positions=None, interleaved: bool = False,
                          stream=None) -> None:
    """Gradient of ``attn_qk_norm_rope``: from its inputs ``q``, ``k`` (not
    read, and may be None, without a norm) and the gradients ``dq_out``,
    ``dk_out`` of its outputs writes ``dq``, ``dk`` and the weights' gradients
    ``dq_weight``, ``dk_weight`` (fp32 [D]; None: not wanted). Rows whose position
    is outside the table are not written in ``dq``, ``dk``: zero them beforehand
    where something reads those rows. ``workspace``:
    a CUDA tensor of ``attn_qk_norm_rope_bwd_workspace_bytes(D)`` bytes."""
    w = "attn_qk_norm_rope_bwd"
    dev = _device(w, "dq_out", dq_out)
    B, Hq, S, D = qs = dq_out.shape
    Hkv = dk_out.shape[1] if dk_out is not None else 0
    ks = (B, Hkv, S, D)
    dt, f32 = dq_out.dtype, _torch.float32
    p = _rope_params(w, dt, dev, B * S, D, q_weight, k_weight, eps, cos_sin, positions, interleaved)
    _run(w, lib().attn_qk_norm_rope_bwd, dev, stream,
         _view(w, "q", q, dt, dev, qs) if q is not None else None,
         _view(w, "k", k, dt, dev, ks) if Hkv and k is not None else None,
         _view(w, "dq_out", dq_out, dt, dev, qs),
         _view(w, "dk_out", dk_out, dt, dev, ks) if Hkv else None,
         _view(w, "dq", dq, dt, dev, qs), _view(w, "dk", dk, dt, dev, ks) if Hkv else None,
         None if dq_weight is None else _tensor(w, "dq_weight", dq_weight, f32, dev, (D,)),
         None if dk_weight is None else _tensor(w, "dk_weight", dk_weight, f32, dev, (D,)),
         *_workspace(w, workspace, dev), B, Hq, Hkv, S, D, p)


def _rope_axes(w: str, positions, axes, cos_sin) -> tuple:
    """(number of axes, axis of each channel pair as bytes), checked."""
    if cos_sin is None or positions is None:
        raise ValueError(f"{w}: cos_sin and positions are needed")
    if positions.dim() != 3:
        raise ValueError(f"{w}: positions must have shape [axes, B, S]")
    pairs = axes if isinstance(axes, bytes) else bytes([int(a) for a in axes])
    if 2 * len(pairs) != cos_sin.shape[1]:
        raise ValueError(f"{w}: axes must have an entry for each of the {cos_sin.shape[1] // 2} "
                         f"channel pairs, not {len(pairs)}")
    return positions.shape[0], pairs


def attn_qk_norm_rope_axes(q, k, q_out, k_out, *, cos_sin, positions, axes, q_weight=None,
                           k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                           stream=None) -> None:
    """``attn_qk_norm_rope`` with positions on several axes (time, height and
    width of images and video): ``positions`` int32 [A, B, S], A up to 4, and
    ``axes`` the axis of each of the rot_dim / 2 channel pairs (a sequence of
    whole numbers, e.g. ``bytes([0] * 16 + [1] * 24 + [2] * 24)``). A row with a
    position outside the table on any axis is not written."""
    w = "attn_qk_norm_rope_axes"
    dev = _device(w, "q", q)
    B, Hq, S, D = shape = q.shape
    dt = q.dtype
    A, pairs = _rope_axes(w, positions, axes, cos_sin)
    p = _rope_params(w, dt, dev, A * B * S, D, q_weight, k_weight, eps, cos_sin, positions,
                     interleaved)
    kv = ko = None
    Hkv = 0
    if k is not None:
        Hkv = k.shape[1]
        kv = _view(w, "k", k, dt, dev, (B, Hkv, S, D))
        ko = _view(w, "k_out", k_out, dt, dev, (B, Hkv, S, D))
    _run(w, lib().attn_qk_norm_rope_axes, dev, stream, _view(w, "q", q, dt, dev, shape), kv,
         _view(w, "q_out", q_out, dt, dev, shape), ko, B, Hq, Hkv, S, D, p, A, pairs)


def attn_qk_norm_rope_axes_bwd(q, k, dq_out, dk_out, dq, dk, *, cos_sin, positions, axes,
                               workspace, dq_weight=None, dk_weight=None, q_weight=None,
                               k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                               stream=None) -> None:
    """Gradient of ``attn_qk_norm_rope_axes``, with the arguments of
    ``attn_qk_norm_rope_bwd`` beside ``positions`` [A, B, S] and ``axes``."""
    w = "attn_qk_norm_rope_axes_bwd"
    dev = _device(w, "dq_out", dq_out)
    B, Hq, S, D = qs = dq_out.shape
    Hkv = dk_out.shape[1] if dk_out is not None else 0
    ks = (B, Hkv, S, D)
    dt, f32 = dq_out.dtype, _torch.float32
    A, pairs = _rope_axes(w, positions, axes, cos_sin)
    p = _rope_params(w, dt, dev, A * B * S, D, q_weight, k_weight, eps, cos_sin, positions,
                     interleaved)
    _run(w, lib().attn_qk_norm_rope_axes_bwd, dev, stream,
         _view(w, "q", q, dt, dev, qs) if q is not None else None,
         _view(w, "k", k, dt, dev, ks) if Hkv and k is not None else None,
         _view(w, "dq_out", dq_out, dt, dev, qs),
         _view(w, "dk_out", dk_out, dt, dev, ks) if Hkv else None,
         _view(w, "dq", dq, dt, dev, qs), _view(w, "dk", dk, dt, dev, ks) if Hkv else None,
         None if dq_weight is None else _tensor(w, "dq_weight", dq_weight, f32, dev, (D,)),
         None if dk_weight is None else _tensor(w, "dk_weight", dk_weight, f32, dev, (D,)),
         *_workspace(w, workspace, dev), B, Hq, Hkv, S, D, p, A, pairs)


def _workspace(w: str, x, dev: int) -> tuple:
    """(address, bytes) of a workspace tensor of any type, or (None, 0)."""
    if x is None:
        return None, 0
    return (_tensor(w, "workspace", x, getattr(x, "dtype", None), dev, getattr(x, "shape", None)),
            x.numel() * x.element_size())


def attn_cache_q4_bytes(num_pages: int, Hkv: int, page_size: int, D: int) -> int:
    """Bytes of a 4-bit cache pool; as a tensor: uint8 [num_pages, Hkv, bytes
    per record]."""
    return int(lib().attn_cache_q4_bytes(num_pages, Hkv, page_size, D))


def _cache_q4(w: str, load: bool, k, v, slots, pool, page_size: int, stream) -> None:
    dev = _device(w, "k", k)
    B, Hkv, S, D = shape = k.shape
    bf16 = _torch.bfloat16
    pages = pool.shape[0]
    vk, vv = _view(w, "k", k, bf16, dev, shape), _view(w, "v", v, bf16, dev, shape)
    ps = _tensor(w, "slots", slots, _torch.int64, dev, slots.shape)
    if slots.numel() != B * S:
        raise ValueError(f"{w}: slots must have {B * S} entries ([B, S])")
    # codes and scales of a token and head: D + D / 8 bytes (include/mattn.h)
    pp = _tensor(w, "pool", pool, _torch.uint8, dev, (pages, Hkv, page_size * (D + D // 8)))
    if load:
        _run(w, lib().attn_cache_load_q4, dev, stream, pp, pages, page_size, ps, vk, vv, B, Hkv, S,
             D)
    else:
        _run(w, lib().attn_cache_store_q4, dev, stream, vk, vv, ps, pp, pages, page_size, B, Hkv,
             S, D)


def attn_cache_store_q4(k, v, slots, pool, *, page_size: int, stream=None) -> None:
    """Quantises ``k``, ``v`` (bf16 [B, Hkv, S, D], any strides with contiguous
    D) into the 4-bit ``pool`` (uint8 [num_pages, Hkv, record bytes]) at
    ``slots`` (int64 [B, S], page * page_size + row, each at most once; a slot
    outside the pool is skipped). Record layout and rounding: include/mattn.h."""
    _cache_q4("attn_cache_store_q4", False, k, v, slots, pool, page_size, stream)


def attn_cache_load_q4(pool, slots, k, v, *, page_size: int, stream=None) -> None:
    """Reads the rows at ``slots`` of the 4-bit ``pool`` into ``k``, ``v``
    (bf16 [B, Hkv, S, D], any strides with contiguous D); a slot outside the
    pool reads as zeros."""
    _cache_q4("attn_cache_load_q4", True, k, v, slots, pool, page_size, stream)


def attn_decode_q4_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, max_len: int,
                                   D: int) -> int:
    return int(lib().attn_decode_q4_workspace_bytes(B, Hq, Hkv, Sq, max_len, D))


def attn_decode_q4(q, pool, o, lse, variant: int = 0, *, page_table, page_size: int, seq_lens,
                   max_len: Optional[int] = None, workspace=None, scale: float = 0.0,
                   window: int = 0, sink: int = 0, softcap: float = 0.0, alibi_slopes=None,
                   stream=None) -> None:
    """Decode over a 4-bit paged cache: ``q`` [B, Hq, Sq, D] bf16 (the last Sq
    tokens of each sequence, (Hq/Hkv) * Sq <= 16) against the ``seq_lens`` [B]
    int32 tokens that ``page_table`` [B, pages_per_seq] places in ``pool``
    (uint8 [num_pages, Hkv, record bytes]). ``max_len`` (default: all the
    table holds) bounds seq_lens. With ``MASK_WINDOW`` the first ``sink`` keys
    stay visible. Writes ``o`` (bf16, like q) and ``lse`` fp32 [B, Hq, Sq].
    ``workspace``: optional CUDA tensor (``attn_decode_q4_workspace_bytes``)."""
    w = "attn_decode_q4"
    dev = _device(w, "q", q)
    bf16, i32, f32 = _torch.bfloat16, _torch.int32, _torch.float32
    B, Hq, Sq, D = shape = q.shape
    pages, Hkv = pool.shape[:2]
    per = page_table.shape[1]
    p = attn_params(BF16, scale, window, softcap)
    if alibi_slopes is not None:
        p.alibi_slopes = _tensor(w, "alibi_slopes", alibi_slopes, f32, dev, (Hq,))
    p.page_table = _tensor(w, "page_table", page_table, i32, dev, (B, per))
    p.page_size = page_size
    p.pages_per_seq = per
    p.num_pages = pages
    ws, ws_bytes = _workspace(w, workspace, dev)
    _run(w, lib().attn_decode_q4, dev, stream, _tensor(w, "q", q, bf16, dev, shape),
         _tensor(w, "pool", pool, _torch.uint8, dev, (pages, Hkv, page_size * (D + D // 8))),
         _tensor(w, "o", o, bf16, dev, shape), _tensor(w, "lse", lse, f32, dev, (B, Hq, Sq)),
         B, Hq, Hkv, Sq, per * page_size if max_len is None else max_len, D, variant,
         ctypes.byref(p), _tensor(w, "seq_lens", seq_lens, i32, dev, (B,)), sink, ws, ws_bytes)


def _paged_params(w: str, dev: int, B: int, Hq: int, scale, window, softcap, alibi_slopes,
                  page_table, page_size: int, pages: int, status, timeout_ns: int,
                  fault_inject: int) -> attn_params:
    """Parameters of the calls over the bf16 cache with sequences of their own lengths."""
    i32 = _torch.int32
    p = attn_params(BF16, scale, window, softcap)
    if alibi_slopes is not None:
        p.alibi_slopes = _tensor(w, "alibi_slopes", alibi_slopes, _torch.float32, dev, (Hq,))
    if page_table is not None:
        per = page_table.shape[1]
        p.page_table = _tensor(w, "page_table", page_table, i32, dev, (B, per))
        p.page_size = page_size
        p.pages_per_seq = per
        p.num_pages = pages
    if status is not None:
        p.status = _tensor(w, "status", status, i32, dev, status.shape)
    p.timeout_ns = timeout_ns
    p.fault_inject = fault_inject
    return p


def attn_decode_shared_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, G: int, max_len: int,
                                       D: int) -> int:
    return int(lib().attn_decode_shared_workspace_bytes(B, Hq, Hkv, Sq, G, max_len, D))


def attn_decode_shared(q, k, v, o, lse, variant: int = 0, *, page_table, page_size: int, seq_lens,
                       workspace, group_starts=None, shared_lens=None,
                       max_len: Optional[int] = None, scale: float = 0.0, window: int = 0,
                       softcap: float = 0.0, alibi_slopes=None, status=None, timeout_ns: int = 0,
                       fault_inject: int = 0, stream=None) -> None:
    """Decode over a bf16 paged cache for sequences of their own lengths, groups of which share
    their first keys: ``q`` [B, Hq, Sq, D] (the last Sq tokens of each, (Hq/Hkv) * Sq <= 16)
    against the ``seq_lens`` [B] int32 tokens that ``page_table`` [B, pages_per_seq] places in
    the pools ``k``, ``v`` [num_pages, Hkv, page, D]. Sequences ``group_starts[g]`` to
    ``group_starts[g + 1] - 1`` (int32 [G + 1]) hold the same first ``shared_lens[g]`` (int32
    [G]) keys in the same pages: 512 or more of them are read once for all, fewer by each
    sequence. ``max_len`` (default: all the table holds) bounds seq_lens. Writes ``o`` (bf16,
    like q) and ``lse`` fp32 [B, Hq, Sq].
    ``workspace``: a CUDA tensor of ``attn_decode_shared_workspace_bytes`` bytes."""
    w = "attn_decode_shared"
    dev = _device(w, "q", q)
    bf16, i32 = _torch.bfloat16, _torch.int32
    B, Hq, Sq, D = shape = q.shape
    pages, Hkv = k.shape[:2]
    pool = (pages, Hkv, page_size, D)
    p = _paged_params(w, dev, B, Hq, scale, window, softcap, alibi_slopes, page_table, page_size,
                      pages, status, timeout_ns, fault_inject)
    G, gs, sl = 0, None, None
    if group_starts is not None or shared_lens is not None:
        G = shared_lens.numel() if shared_lens is not None else 0
        sl = _tensor(w, "shared_lens", shared_lens, i32, dev, (G,))
        gs = _tensor(w, "group_starts", group_starts, i32, dev, (G + 1,))
    _run(w, lib().attn_decode_shared, dev, stream, _tensor(w, "q", q, bf16, dev, shape),
         _tensor(w, "k", k, bf16, dev, pool), _tensor(w, "v", v, bf16, dev, pool),
         _tensor(w, "o", o, bf16, dev, shape), _tensor(w, "lse", lse, _torch.float32, dev,
                                                       (B, Hq, Sq)),
         B, Hq, Hkv, Sq, p.pages_per_seq * page_size if max_len is None else max_len, D, variant,
         ctypes.byref(p), _tensor(w, "seq_lens", seq_lens, i32, dev, (B,)), gs, sl, G,
         *_workspace(w, workspace, dev))


def attn_key_weights(q, k, lse, weights, variant: int = 0, *, previous=None, decay: float = 1.0,
                     page_table=None, page_size: int = 0, seq_lens=None, scale: float = 0.0,
                     window: int = 0, softcap: float = 0.0, alibi_slopes=None, status=None,
                     timeout_ns: int = 0, fault_inject: int = 0, stream=None) -> None:
    """The attention weight that each cached key received: writes ``weights`` (fp32 [B, Hkv,
    L]) = ``decay`` * ``previous`` + the sum over the query rows of each key/value head of
    exp(score - LSE). ``q`` [B, Hq, Sq, D] bf16 and ``lse`` fp32 [B, Hq, Sq] are those of an
    attention call over the same keys; ``k``: bf16 page pool [num_pages, Hkv, page, D] with
    ``page_table`` [B, pages_per_seq], or contiguous [B, Hkv, Skv, D]. ``seq_lens`` int32 [B]
    counts each sequence's keys (its Sq rows are the last ones; None: all of L or Skv);
    entries of ``weights`` past them are left as they were. ``previous`` (like ``weights``, or
    ``weights`` itself; None: 0). See include/mattn.h."""
    w = "attn_key_weights"
    dev = _device(w, "q", q)
    bf16, f32 = _torch.bfloat16, _torch.float32
    B, Hq, Sq, D = shape = q.shape
    Hkv, L = k.shape[1], weights.shape[-1]
    paged = page_table is not None
    p = _paged_params(w, dev, B, Hq, scale, window, softcap, alibi_slopes, page_table, page_size,
                      k.shape[0], status, timeout_ns, fault_inject)
    max_len = min(L, p.pages_per_seq * page_size) if paged else k.shape[2]
    _run(w, lib().attn_key_weights, dev, stream, _tensor(w, "q", q, bf16, dev, shape),
         _tensor(w, "k", k, bf16, dev, (k.shape[0], Hkv, page_size, D) if paged
                 else (B, Hkv, max_len, D)),
         _tensor(w, "lse", lse, f32, dev, (B, Hq, Sq)),
         None if previous is None else _tensor(w, "previous", previous, f32, dev, (B, Hkv, L)),
         decay, _tensor(w, "weights", weights, f32, dev, (B, Hkv, L)), B, Hq, Hkv, Sq, max_len, D,
         L, variant, ctypes.byref(p),
         None if seq_lens is None else _tensor(w, "seq_lens", seq_lens, _torch.int32, dev, (B,)))


def attn_cache_evict(weights, seq_lens, k, v, page_table, weights_out, kept, new_lens, freed, info,
                     *, page_size: int, recent: int, sink: int = 0, starts=None, new_table=None,
                     stream=None) -> None:
    """Eviction from the bf16 paged cache by attention weight: of every (sequence, key/value
    head)'s keys the first ``sink`` (or ``starts`` [B] int32) stay, and of the others, where
    they are more than ``kept.shape[2]``, the last ``recent`` and the heaviest by ``weights``
    (fp32 [B, Hkv, L]), that many in all. Their rows in the pools ``k``, ``v`` (bf16 [num_pages,
    Hkv, page, D]) move together in order, in place or, with ``new_table`` [B, pages], into its
    pages. Writes ``weights_out`` (may be ``weights``), ``kept`` [B, Hkv, keep] (old positions,
    -1 past the last), ``new_lens`` [B], ``freed`` (page ids no longer used: not those that
    ``new_table`` has in the same place) and ``info`` [2]: pages freed, sequences cut. All int32. See include/mattn.h."""
    w = "attn_cache_evict"
    dev = _device(w, "weights", weights)
    i32, f32, bf16 = _torch.int32, _torch.float32, _torch.bfloat16
    B, Hkv, L = ws = weights.shape
    pages, D = k.shape[0], k.shape[-1]
    pool, per, keep = (pages, Hkv, page_size, D), page_table.shape[1], kept.shape[-1]
    new = None if new_table is None else _tensor(w, "new_table", new_table, i32, dev,
                                                 (B, new_table.shape[1]))
    _run(w, lib().attn_cache_evict, dev, stream, _tensor(w, "weights", weights, f32, dev, ws),
         _tensor(w, "weights_out", weights_out, f32, dev, ws), L,
         _tensor(w, "seq_lens", seq_lens, i32, dev, (B,)),
         None if starts is None else _tensor(w, "starts", starts, i32, dev, (B,)), sink, keep,
         recent, _tensor(w, "k", k, bf16, dev, pool), _tensor(w, "v", v, bf16, dev, pool), pages,
         page_size, _tensor(w, "page_table", page_table, i32, dev, (B, per)), per, new,
         0 if new is None else new_table.shape[1], B, Hkv, min(L, per * page_size), D,
         _tensor(w, "kept", kept, i32, dev, (B, Hkv, keep)),
         _tensor(w, "new_lens", new_lens, i32, dev, (B,)),
         _tensor(w, "freed", freed, i32, dev, (freed.numel(),)), freed.numel(),
         _tensor(w, "info", info, i32, dev, (2,)))


def attn_check_status(status=None, stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status word."""
    return int(lib().attn_check_status(_ptr(status), _stream(stream)))


def default_scale(D: int) -> float:
    return 1.0 / math.sqrt(D)
