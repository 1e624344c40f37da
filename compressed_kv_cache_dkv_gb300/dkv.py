"""Thin ctypes binding of libdkv (include/dkv.h).

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of libdkv.so.  PyTorch supplies device memory and the current CUDA
stream.  The functions keep the C names; tensors are passed where the C ABI
takes device pointers, and outputs the caller does not supply are allocated
with torch on the inputs' device.

There is no CPU fallback: when libdkv.so is missing every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdkv.so")

DKV_OK = 0
DKV_ERR_ARG = -1
DKV_ERR_SHAPE = -2
DKV_ERR_ALIGN = -3
DKV_ERR_UNSUPPORTED = -4
DKV_ERR_CUDA = -5
DKV_ERR_TIMEOUT = -6
DKV_ERR_WORKSPACE = -7
DKV_ERR_DEVICE = -8
DKV_DEVERR_TIMEOUT = 0x1
DKV_DEVERR_INDEX = 0x2
DKV_DEVERR_RANGE = 0x4
BLOCK_SIZE = 256
DKV_LAYOUT_FRAGMENT = 0
DKV_LAYOUT_TC = 1
DKV_FP16 = 0
DKV_BF16 = 1

EXPORTED = (
    "dkv_version", "dkv_status_string", "dkv_layout", "dkv_layout_bytes",
    "dkv_compress_workspace_bytes", "dkv_compress_layout", "dkv_import_factors",
    "dkv_decode_workspace_bytes", "dkv_decode_launches", "dkv_decode_attend", "dkv_decode_route", "dkv_decode_blocks",
    "dkv_decode_combine",
    "dkv_dense_workspace_bytes", "dkv_dense_decode", "dkv_get_error", "dkv_decode_attend_noalloc",
    "dkv_append_workspace_bytes", "dkv_append", "dkv_debug_set_limits", "dkv_debug_set_launch", "dkv_prefill_routed_slots",
    "dkv_prefill_workspace_bytes", "dkv_prefill_attend",
    "dkv_paged_check", "dkv_paged_workspace_bytes", "dkv_paged_append", "dkv_paged_decode", "dkv_paged_prefill",
    "dkv_paged_weights", "dkv_paged_evict",
    "dkv_paged_plan_workspace_bytes", "dkv_paged_plan", "dkv_qk_norm_rope",
    "dkv_qpaged_check", "dkv_qpaged_workspace_bytes", "dkv_qpaged_append", "dkv_qpaged_gather", "dkv_qpaged_decode",
    "dkv_qpaged_prefill",
)


class DkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {dkv_status_string(status)} ({status})")
        self.status = status


class dkv_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "n_q_heads", "n_kv_heads", "head_dim", "block_size", "n_blocks", "window", "rank",
        "n_residual", "layout", "block_capacity", "window_capacity", "residual_bits", "rope_dims")] + [
        ("rope_base", ctypes.c_float)] + [(n, ctypes.c_int32) for n in ("rank_pad", "res_pad", "window_pad",
                                                                         "n_units")] + [
        (n, ctypes.c_uint64) for n in (
            "blk_off_mask", "blk_off_vk", "blk_off_u", "blk_off_res", "blk_off_vv", "block_bytes",
            "off_router", "off_blocks", "off_cold", "off_window", "block_stride", "unit_stride", "total_bytes",
            "off_rope")]

    @property
    def group(self) -> int:
        return self.n_q_heads // self.n_kv_heads


class dkv_factors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "a_k", "a_v", "U", "V_K", "V_V", "res_pos", "K_res", "V_res", "kmin", "kmax", "win_K", "win_V")]


class dkv_paged(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "n_q_heads", "n_kv_heads", "head_dim", "page_size", "n_pages", "max_pages", "dtype", "window", "sinks")] + [
        (n, ctypes.c_int64) for n in ("stride_page", "stride_head", "stride_token")]


class dkv_strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "head", "token")]


class dkv_rotate(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "n_q_heads", "n_kv_heads", "head_dim", "dtype", "norm", "rope_dims")] + [
        ("eps", ctypes.c_float), ("rope_base", ctypes.c_double), ("inv_freq", ctypes.POINTER(ctypes.c_double))]


class dkv_qpaged(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "n_q_heads", "n_kv_heads", "head_dim", "page_size", "n_pages", "max_pages", "dtype", "window", "sinks")] + [
        (n, ctypes.c_int64) for n in ("stride_page", "stride_head")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libdkv.so (built by ``build.py`` / ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdkv.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        pdesc = ctypes.POINTER(dkv_desc)
        L.dkv_version.restype = ctypes.c_int
        L.dkv_status_string.restype = ctypes.c_char_p
        L.dkv_status_string.argtypes = [ctypes.c_int]
        L.dkv_layout.argtypes = [pdesc]
        L.dkv_layout_bytes.restype = sz
        L.dkv_layout_bytes.argtypes = [pdesc]
        L.dkv_compress_workspace_bytes.restype = sz
        L.dkv_compress_workspace_bytes.argtypes = [pdesc]
        L.dkv_compress_layout.argtypes = [pdesc, vp, vp, vp, vp, sz, vp]
        L.dkv_import_factors.argtypes = [pdesc, ctypes.POINTER(dkv_factors), vp, vp, vp]
        L.dkv_decode_workspace_bytes.restype = sz
        L.dkv_decode_workspace_bytes.argtypes = [pdesc, i32]
        L.dkv_decode_launches.restype = i32
        L.dkv_decode_launches.argtypes = [pdesc, i32]
        L.dkv_decode_attend.argtypes = [pdesc, vp, vp, i32, vp, vp, vp, vp, sz, vp]
        L.dkv_decode_route.argtypes = [pdesc, vp, vp, i32, vp, vp, sz, vp]
        L.dkv_decode_blocks.argtypes = [pdesc, vp, vp, i32, vp, vp, vp, sz, vp]
        L.dkv_decode_combine.argtypes = [pdesc, i32, vp, vp, vp, sz, vp]
        L.dkv_dense_workspace_bytes.restype = sz
        L.dkv_dense_workspace_bytes.argtypes = [i32] * 5
        L.dkv_dense_decode.argtypes = [i32] * 5 + [vp] * 6 + [sz, vp]
        L.dkv_get_error.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.dkv_decode_attend_noalloc.argtypes = [pdesc, vp, vp, i32, vp, vp, vp, vp]
        L.dkv_append_workspace_bytes.restype = sz
        L.dkv_append_workspace_bytes.argtypes = [pdesc]
        L.dkv_append.argtypes = [pdesc, vp, vp, i32, vp, vp, sz, vp]
        L.dkv_debug_set_limits.argtypes = [i32, ctypes.c_uint32]
        L.dkv_debug_set_launch.argtypes = [i32]
        L.dkv_prefill_routed_slots.restype = i32
        L.dkv_prefill_routed_slots.argtypes = [i32, i32]
        L.dkv_prefill_workspace_bytes.restype = sz
        L.dkv_prefill_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        L.dkv_prefill_attend.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        ppaged, pstr = ctypes.POINTER(dkv_paged), ctypes.POINTER(dkv_strides)
        L.dkv_paged_check.argtypes = [ppaged]
        L.dkv_paged_workspace_bytes.restype = sz
        L.dkv_paged_workspace_bytes.argtypes = [ppaged, i32]
        L.dkv_paged_append.argtypes = [ppaged, vp, vp, pstr, i32] + [vp] * 6 + [sz, vp]
        L.dkv_paged_decode.argtypes = [ppaged, vp, pstr] + [vp] * 8 + [sz, vp]
        L.dkv_paged_prefill.argtypes = [ppaged, vp, pstr, i32] + [vp] * 6 + [pstr, vp, vp, sz, vp]
        L.dkv_paged_weights.argtypes = [ppaged, vp, pstr, i32] + [vp] * 7 + [sz, vp]
        L.dkv_paged_evict.argtypes = [ppaged] + [vp] * 5 + [i32] * 3 + [vp, i32] + [vp] * 4 + [sz, vp]
        L.dkv_paged_plan_workspace_bytes.restype = sz
        L.dkv_paged_plan_workspace_bytes.argtypes = [i32]
        L.dkv_paged_plan.argtypes = [i32] * 4 + [vp] * 3 + [i32, vp, vp, i32] + [vp] * 7 + [sz, vp]
        pq = ctypes.POINTER(dkv_qpaged)
        L.dkv_qk_norm_rope.argtypes = [ctypes.POINTER(dkv_rotate), vp, pstr, vp, pstr, vp, vp, vp, vp, pstr, vp, pstr,
                                       ppaged, vp, pstr, vp, vp, vp, vp, sz, vp]
        L.dkv_qpaged_check.argtypes = [pq]
        L.dkv_qpaged_workspace_bytes.restype = sz
        L.dkv_qpaged_workspace_bytes.argtypes = [pq]
        L.dkv_qpaged_append.argtypes = [pq, vp, vp, pstr, i32, vp, vp, vp, sz, vp]
        L.dkv_qpaged_gather.argtypes = [pq] + [vp] * 4 + [i32, vp, vp, pstr, vp, sz, vp]
        L.dkv_qpaged_decode.argtypes = [pq, vp, pstr] + [vp] * 6 + [sz, vp]
        L.dkv_qpaged_prefill.argtypes = [pq, vp, pstr, i32, i32] + [vp] * 5 + [pstr, vp, vp, sz, vp]
        _lib = L
    return _lib


def dkv_status_string(status: int) -> str:
    return lib().dkv_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != DKV_OK:
        raise DkvError(status, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def dkv_layout(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int, n_blocks: int, window: int,
               rank: int, n_residual: int, block_size: int = BLOCK_SIZE,
               layout: int | None = None, block_capacity: int = 0, window_capacity: int = 0,
               residual_bits: int = 0, rope_dims: int = 0, rope_base: float = 0.0) -> dkv_desc:
    """Fill a descriptor.  `layout` is DKV_LAYOUT_FRAGMENT (mma.sync decode kernel, the
    default) or DKV_LAYOUT_TC (tcgen05 decode kernel; head_dim 128, rank <= 48, 1 <= R <= 128).
    `block_capacity` / `window_capacity` reserve room for dkv_append (0: the live counts).
    `residual_bits` 0 keeps residual rows fp16; 8 or 4 stores them group-quantised.
    `rope_dims` > 0 makes an un-rotated pool: keys are given and stored before RoPE and the
    decode rotates them to their absolute positions (RoPE base `rope_base`)."""
    d = dkv_desc(batch=batch, n_q_heads=n_q_heads, n_kv_heads=n_kv_heads, head_dim=head_dim,
                 block_size=block_size, n_blocks=n_blocks, window=window, rank=rank, n_residual=n_residual,
                 layout=DKV_LAYOUT_FRAGMENT if layout is None else layout,
                 block_capacity=block_capacity, window_capacity=window_capacity, residual_bits=residual_bits,
                 rope_dims=rope_dims, rope_base=rope_base)
    _check(lib().dkv_layout(ctypes.byref(d)), "dkv_layout")
    return d


def dkv_layout_supported(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int, n_blocks: int, window: int,
                         rank: int, n_residual: int, layout: int) -> bool:
    """True when dkv_layout accepts these sizes under `layout`."""
    try:
        dkv_layout(batch, n_q_heads, n_kv_heads, head_dim, n_blocks, window, rank, n_residual, layout=layout)
    except DkvError:
        return False
    return True


def dkv_layout_bytes(d: dkv_desc) -> int:
    return int(lib().dkv_layout_bytes(ctypes.byref(d)))


def _ws(nbytes: int, device, workspace):
    if workspace is not None:
        return workspace
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)


def dkv_compress_workspace_bytes(d: dkv_desc) -> int:
    return int(lib().dkv_compress_workspace_bytes(ctypes.byref(d)))


def dkv_compress_layout(d: dkv_desc, K: torch.Tensor, V: torch.Tensor, cache: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """K, V: fp16 [B, Hkv, T, d] on the GPU -> packed cache (uint8 [total_bytes])."""
    if cache is None:
        cache = torch.empty(d.total_bytes, dtype=torch.uint8, device=K.device)
    need = int(lib().dkv_compress_workspace_bytes(ctypes.byref(d)))
    workspace = _ws(need, K.device, workspace)
    _check(lib().dkv_compress_layout(ctypes.byref(d), _ptr(K), _ptr(V), _ptr(cache), _ptr(workspace),
                                     workspace.numel(), _stream(stream)), "dkv_compress_layout")
    return cache


def dkv_append_workspace_bytes(d: dkv_desc) -> int:
    return int(lib().dkv_append_workspace_bytes(ctypes.byref(d)))


def dkv_append(d: dkv_desc, K_new: torch.Tensor, V_new: torch.Tensor, cache: torch.Tensor,
               workspace: torch.Tensor | None = None, stream=None) -> dkv_desc:
    """Append K_new, V_new (fp16 [B, Hkv, n_new, d] on the GPU) to the cache; advances d in place."""
    if K_new.shape != V_new.shape or K_new.dim() != 4:
        raise DkvError(DKV_ERR_SHAPE, "dkv_append")
    K_new, V_new = K_new.contiguous(), V_new.contiguous()
    workspace = _ws(dkv_append_workspace_bytes(d), K_new.device, workspace)
    _check(lib().dkv_append(ctypes.byref(d), _ptr(K_new), _ptr(V_new), int(K_new.shape[2]), _ptr(cache),
                            _ptr(workspace), workspace.numel(), _stream(stream)), "dkv_append")
    return d


def dkv_import_factors(d: dkv_desc, f: dict, cache: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """f: dict of device tensors named like the dkv_factors fields (fp16, res_pos int32)."""
    dev = next(v.device for v in f.values() if v is not None)
    if cache is None:
        cache = torch.empty(d.total_bytes, dtype=torch.uint8, device=dev)
    workspace = _ws(256, dev, workspace)
    fac = dkv_factors(**{k: _ptr(f.get(k)) for k, _ in dkv_factors._fields_})
    _check(lib().dkv_import_factors(ctypes.byref(d), ctypes.byref(fac), _ptr(cache), _ptr(workspace),
                                    _stream(stream)), "dkv_import_factors")
    return cache


def dkv_decode_workspace_bytes(d: dkv_desc, top_k: int) -> int:
    return int(lib().dkv_decode_workspace_bytes(ctypes.byref(d), int(top_k)))


def dkv_decode_launches(d: dkv_desc, top_k: int) -> int:
    """Kernel launches one dkv_decode_attend call makes on the current device (1: one grid)."""
    return int(lib().dkv_decode_launches(ctypes.byref(d), int(top_k)))


def dkv_decode_attend(d: dkv_desc, q: torch.Tensor, cache: torch.Tensor, top_k: int,
                      out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = True,
                      routed: torch.Tensor | bool | None = True, workspace: torch.Tensor | None = None,
                      stream=None):
    """q fp16 [B, Hq, d] -> (out fp32 [B, Hq, d], lse fp32 [B, Hq] or None, routed int32 [B, Hkv, K_eff] or None)."""
    dev = q.device
    k_eff = d.n_blocks if (top_k == 0 or top_k >= d.n_blocks) else top_k
    if out is None:
        out = torch.empty(d.batch, d.n_q_heads, d.head_dim, dtype=torch.float32, device=dev)
    if lse is True:
        lse = torch.empty(d.batch, d.n_q_heads, dtype=torch.float32, device=dev)
    elif lse is False:
        lse = None
    if routed is True:
        routed = torch.empty(d.batch, d.n_kv_heads, max(k_eff, 0), dtype=torch.int32, device=dev) if k_eff > 0 else None
    elif routed is False:
        routed = None
    if workspace is None:
        workspace = _ws(dkv_decode_workspace_bytes(d, top_k), dev, None)
    _check(lib().dkv_decode_attend(ctypes.byref(d), _ptr(q), _ptr(cache), int(top_k), _ptr(out), _ptr(lse),
                                   _ptr(routed), _ptr(workspace), workspace.numel(), _stream(stream)),
           "dkv_decode_attend")
    return out, lse, routed


def dkv_decode_route(d: dkv_desc, q, cache, top_k: int, workspace, routed=None, stream=None) -> None:
    _check(lib().dkv_decode_route(ctypes.byref(d), _ptr(q), _ptr(cache), int(top_k), _ptr(routed), _ptr(workspace),
                                  workspace.numel(), _stream(stream)), "dkv_decode_route")


def dkv_decode_blocks(d: dkv_desc, q, cache, top_k: int, workspace, out=None, lse=None, stream=None) -> None:
    _check(lib().dkv_decode_blocks(ctypes.byref(d), _ptr(q), _ptr(cache), int(top_k), _ptr(out), _ptr(lse),
                                   _ptr(workspace), workspace.numel(), _stream(stream)), "dkv_decode_blocks")


def dkv_decode_combine(d: dkv_desc, top_k: int, out, workspace, lse=None, stream=None) -> None:
    _check(lib().dkv_decode_combine(ctypes.byref(d), int(top_k), _ptr(out), _ptr(lse), _ptr(workspace),
                                    workspace.numel(), _stream(stream)), "dkv_decode_combine")


def dkv_dense_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim, T) -> int:
    return int(lib().dkv_dense_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim, T))


def dkv_dense_decode(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, out: torch.Tensor | None = None,
                     lse: torch.Tensor | bool | None = True, workspace: torch.Tensor | None = None, stream=None):
    """Dense decode attention over uncompressed K, V fp16 [B, Hkv, T, d]; q fp16 [B, Hq, d]."""
    B, Hkv, T, dh = K.shape
    Hq = q.shape[1]
    dev = q.device
    if out is None:
        out = torch.empty(B, Hq, dh, dtype=torch.float32, device=dev)
    if lse is True:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=dev)
    elif lse is False:
        lse = None
    if workspace is None:
        workspace = _ws(dkv_dense_workspace_bytes(B, Hq, Hkv, dh, T), dev, None)
    _check(lib().dkv_dense_decode(B, Hq, Hkv, dh, T, _ptr(q), _ptr(K), _ptr(V), _ptr(out), _ptr(lse),
                                  _ptr(workspace), workspace.numel(), _stream(stream)), "dkv_dense_decode")
    return out, lse


def dkv_prefill_routed_slots(T: int, top_k: int) -> int:
    """Slots per query block of dkv_prefill_attend's routed-index output (0 on bad arguments)."""
    return int(lib().dkv_prefill_routed_slots(int(T), int(top_k)))


def dkv_prefill_workspace_bytes(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int, T: int,
                                top_k: int) -> int:
    """Workspace bytes dkv_prefill_attend needs for these sizes (0 on bad arguments)."""
    return int(lib().dkv_prefill_workspace_bytes(int(batch), int(n_q_heads), int(n_kv_heads), int(head_dim), int(T),
                                                 int(top_k)))


def dkv_prefill_attend(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, top_k: int, out: torch.Tensor | None = None,
                       lse: torch.Tensor | bool = True, routed: torch.Tensor | bool = True,
                       workspace: torch.Tensor | None = None, stream=None):
    """Block-sparse prefill: q fp16 [B, Hq, T, d], K, V fp16 [B, Hkv, T, d] on the GPU ->
    (out fp32 [B, Hq, T, d], lse fp32 [B, Hq, T] or None, routed int32 [B, Hkv, nb, slots] or None)."""
    B, Hq, T, d = q.shape
    Hkv = K.shape[1]
    dev = q.device
    if out is None:
        out = torch.empty(B, Hq, T, d, dtype=torch.float32, device=dev)
    if lse is True:
        lse = torch.empty(B, Hq, T, dtype=torch.float32, device=dev)
    nb = -(-T // BLOCK_SIZE)
    if routed is True:
        routed = torch.empty(B, Hkv, nb, dkv_prefill_routed_slots(T, top_k), dtype=torch.int32, device=dev)
    need = dkv_prefill_workspace_bytes(B, Hq, Hkv, d, T, top_k)
    workspace = _ws(need, dev, workspace)
    lse_t = lse if isinstance(lse, torch.Tensor) else None
    routed_t = routed if isinstance(routed, torch.Tensor) else None
    _check(lib().dkv_prefill_attend(B, Hq, Hkv, d, T, int(top_k), _ptr(q), _ptr(K), _ptr(V), _ptr(out),
                                    _ptr(lse_t) if lse_t is not None else None,
                                    _ptr(routed_t) if routed_t is not None else None, _ptr(workspace),
                                    workspace.numel(), _stream(stream)), "dkv_prefill_attend")
    return out, lse_t, routed_t


# ---------------------------------------------------------------- paged cache

_PAGED_DTYPES = {torch.float16: DKV_FP16, torch.bfloat16: DKV_BF16}
_I32, _F32 = torch.int32, torch.float32


class _Geometry:
    """What the calls compare their tensors with, from a descriptor's bytes."""

    __slots__ = ("key", "ref", "dtype", "pool", "strides", "batch", "heads", "kv_heads", "d", "each", "table", "q1", "lse1",
                 "weights", "lib")

    def __init__(self, p: dkv_paged, key: bytes):
        self.key, self.ref = key, ctypes.byref(p)
        self.dtype = torch.bfloat16 if p.dtype == DKV_BF16 else torch.float16
        self.batch, self.heads, self.kv_heads, self.d = p.batch, p.n_q_heads, p.n_kv_heads, p.head_dim
        self.pool = (p.n_pages, p.n_kv_heads, p.page_size, p.head_dim)
        self.strides = (p.stride_page, p.stride_head, p.stride_token, 1)
        self.each, self.table = (p.batch,), (p.batch, p.max_pages)
        self.q1, self.lse1 = (p.batch, p.n_q_heads, p.head_dim), (p.batch, p.n_q_heads)
        self.weights = (p.batch, p.n_kv_heads, p.max_pages * p.page_size)
        self.lib = lib()


def _geometry(p: dkv_paged) -> _Geometry:
    key = bytes(p)
    g = p.__dict__.get("_geometry")
    if g is None or g.key != key:
        g = p._geometry = _Geometry(p, key)
    return g


# The checks below stand in the calls themselves as one expression per tensor (a call into a helper
# costs as much as a check); these say what was wrong.

def _wrong(what: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple, dev: int):
    raise ValueError(f"{what}: expected contiguous {dtype} {tuple(shape)} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} "
                     f"with strides {t.stride()} on {t.device}")


def _wrong_rows(what: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple, dev: int):
    raise ValueError(f"{what}: expected {dtype} {tuple(shape)} with adjacent channels on cuda:{dev}, got {t.dtype} "
                     f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


@functools.lru_cache(maxsize=1024)
def _strides(batch: int, head: int, token: int):
    s = dkv_strides(batch, head, token)
    return ctypes.byref(s)


def _check_pool(g: _Geometry, t: torch.Tensor, dev: int) -> None:
    if t.dtype is not g.dtype or t.shape != g.pool or t.get_device() != dev:
        raise ValueError(f"pool: expected {g.dtype} {g.pool} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.stride() != g.strides and any(n > 1 and a != b for n, a, b in zip(g.pool, t.stride(), g.strides)):
        raise ValueError(f"pool: strides {t.stride()} are not the descriptor's {g.strides}")


def _elsewhere(t: torch.Tensor, dev: int) -> bool:
    """Whether the call has to be made on another device than the current one (its tensors' own)."""
    if dev < 0:
        raise ValueError("device tensor expected")
    return dev != torch._C._cuda_getDevice()


def _place(dev: int, stream):
    """The tensors' device, and the caller's stream as its current one: what a call allocates and fills
    is then in that stream's order, and returns to that stream's memory."""
    if stream is None:
        return torch.cuda.device(dev)
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream), device=dev))


def _paged_ws(p: dkv_paged, workspace, dev: int, with_weights: bool = False) -> torch.Tensor:
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous() or workspace.element_size() != 1:
            raise ValueError("workspace: expected contiguous bytes on the tensors' device")
        return workspace
    ws = torch.empty(dkv_paged_workspace_bytes(p, with_weights), dtype=torch.uint8, device=dev)
    ws[:256].zero_()
    return ws


def _int32(what: str, *numbers: int) -> None:
    """Refuses what an int32 argument would hold as another number."""
    if not all(-0x80000000 <= x <= 0x7fffffff for x in numbers):
        raise DkvError(DKV_ERR_ARG, what)


def dkv_paged_layout(k_pages: torch.Tensor, batch: int, n_q_heads: int, max_pages: int, window: int = 0,
                     sinks: int = 0) -> dkv_paged:
    """Descriptor of a paged cache from one of its pools, fp16 or bf16 [n_pages, Hkv, page_size, d]
    under any strides with adjacent channels (a transposed [n_pages, page_size, Hkv, d], a half of a
    pool that interleaves K and V).  `max_pages`: entries of a page-table row; `window`, `sinks`: a
    query at position p sees token t when t <= p and (window == 0 or t > p - window or t < sinks)."""
    if k_pages.dim() != 4 or k_pages.dtype not in _PAGED_DTYPES or k_pages.stride(3) != 1:
        raise DkvError(DKV_ERR_ARG, "dkv_paged_layout")
    n_pages, hkv, page, d = k_pages.shape
    _int32("dkv_paged_layout", batch, n_q_heads, max_pages, n_pages, hkv, page, d, window, sinks)
    sp, sh, st, _ = k_pages.stride()
    p = dkv_paged(batch, n_q_heads, hkv, d, page, n_pages, max_pages, _PAGED_DTYPES[k_pages.dtype], window, sinks, sp, sh, st)
    _check(lib().dkv_paged_check(ctypes.byref(p)), "dkv_paged_layout")
    return p


def dkv_paged_workspace_bytes(p: dkv_paged, with_weights: bool = False) -> int:
    """Bytes of the workspace of every call below.  A call without one makes its own, and with that goes the
    word that tells of bad lengths and pages (dkv_get_error): keep one where those have to be known."""
    return int(lib().dkv_paged_workspace_bytes(ctypes.byref(p), int(with_weights)))


def dkv_paged_append(p: dkv_paged, K_new: torch.Tensor, V_new: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                     page_table: torch.Tensor, pos: torch.Tensor, counts: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> None:
    """Write K_new, V_new [B, Hkv, n_new, d] (any strides with adjacent channels) into their pages: token
    i < counts[b] of sequence b at position pos[b] + i (counts None: all n_new)."""
    dev = K_new.get_device()
    if _elsewhere(K_new, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_paged_append(p, K_new, V_new, k_pages, v_pages, page_table, pos, counts, workspace)
    g = _geometry(p)
    if K_new.stride() != V_new.stride():
        K_new, V_new = K_new.contiguous(), V_new.contiguous()
    n = K_new.shape[2]
    shape = (g.batch, g.kv_heads, n, g.d)
    s = K_new.stride()
    if K_new.dtype is not g.dtype or K_new.shape != shape or K_new.get_device() != dev or s[-1] != 1:
        _wrong_rows("K_new", K_new, g.dtype, shape, dev)
    if V_new.dtype is not g.dtype or V_new.shape != shape or V_new.get_device() != dev:
        _wrong_rows("V_new", V_new, g.dtype, shape, dev)
    if pos.dtype is not _I32 or pos.shape != g.each or pos.get_device() != dev or not pos.is_contiguous():
        _wrong("pos", pos, _I32, g.each, dev)
    if counts is not None and (counts.dtype is not _I32 or counts.shape != g.each or counts.get_device() != dev or not counts.is_contiguous()):
        _wrong("counts", counts, _I32, g.each, dev)
    if k_pages.dtype is not g.dtype or k_pages.stride() != g.strides or k_pages.shape != g.pool or k_pages.get_device() != dev:
        _check_pool(g, k_pages, dev)
    if v_pages.dtype is not g.dtype or v_pages.stride() != g.strides or v_pages.shape != g.pool or v_pages.get_device() != dev:
        _check_pool(g, v_pages, dev)
    if page_table.dtype is not _I32 or page_table.shape != g.table or page_table.get_device() != dev or not page_table.is_contiguous():
        _wrong("page_table", page_table, _I32, g.table, dev)
    ws = _paged_ws(p, workspace, dev)
    st = g.lib.dkv_paged_append(
        g.ref, K_new.data_ptr(), V_new.data_ptr(), _strides(s[0], s[1], s[2]), n, pos.data_ptr(),
        None if counts is None else counts.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
        ws.data_ptr(), ws.numel(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_paged_append")


def dkv_paged_decode(p: dkv_paged, q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                     lens: torch.Tensor, out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = True,
                     weights: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """One new token per sequence: q [B, Hq, d] at position lens[b] - 1 -> (out [B, Hq, d] in q's type,
    lse fp32 [B, Hq] or None).  `weights` fp32 [B, Hkv, max_pages * page_size]: every visible token's
    softmax weight, summed over its KV head's query heads, is added."""
    dev = q.get_device()
    if _elsewhere(q, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_paged_decode(p, q, k_pages, v_pages, page_table, lens, out, lse, weights, workspace)
    g = _geometry(p)
    s = q.stride()
    if q.dtype is not g.dtype or q.shape != g.q1 or q.get_device() != dev or s[-1] != 1:
        _wrong_rows("q", q, g.dtype, g.q1, dev)
    if k_pages.dtype is not g.dtype or k_pages.stride() != g.strides or k_pages.shape != g.pool or k_pages.get_device() != dev:
        _check_pool(g, k_pages, dev)
    if v_pages.dtype is not g.dtype or v_pages.stride() != g.strides or v_pages.shape != g.pool or v_pages.get_device() != dev:
        _check_pool(g, v_pages, dev)
    if page_table.dtype is not _I32 or page_table.shape != g.table or page_table.get_device() != dev or not page_table.is_contiguous():
        _wrong("page_table", page_table, _I32, g.table, dev)
    if lens.dtype is not _I32 or lens.shape != g.each or lens.get_device() != dev or not lens.is_contiguous():
        _wrong("lens", lens, _I32, g.each, dev)
    if out is None:
        out = torch.empty(g.q1, dtype=g.dtype, device=dev)
    elif out.dtype is not g.dtype or out.shape != g.q1 or out.get_device() != dev or not out.is_contiguous():
        _wrong("out", out, g.dtype, g.q1, dev)
    if lse is True:
        lse = torch.empty(g.lse1, dtype=_F32, device=dev)
    elif lse is False:
        lse = None
    elif lse is not None and (lse.dtype is not _F32 or lse.shape != g.lse1 or lse.get_device() != dev or not lse.is_contiguous()):
        _wrong("lse", lse, _F32, g.lse1, dev)
    if weights is not None and (weights.dtype is not _F32 or weights.shape != g.weights or weights.get_device() != dev or not weights.is_contiguous()):
        _wrong("weights", weights, _F32, g.weights, dev)
    ws = _paged_ws(p, workspace, dev, weights is not None)
    st = g.lib.dkv_paged_decode(
        g.ref, q.data_ptr(), _strides(s[0], s[1], 0), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
        lens.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
        None if weights is None else weights.data_ptr(), ws.data_ptr(), ws.numel(),
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_paged_decode")
    return out, lse


def dkv_paged_prefill(p: dkv_paged, q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                      lens: torch.Tensor, q_lens: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      lse: torch.Tensor | bool | None = True, workspace: torch.Tensor | None = None, stream=None):
    """The last tokens of each sequence: q [B, Hq, Tq, d], query i < q_lens[b] (None: Tq) at position
    lens[b] - q_lens[b] + i -> (out [B, Hq, Tq, d] in q's type, lse fp32 [B, Hq, Tq] or None).  Rows from
    q_lens[b] on are left as they were (zeros in outputs allocated here)."""
    dev = q.get_device()
    if _elsewhere(q, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_paged_prefill(p, q, k_pages, v_pages, page_table, lens, q_lens, out, lse, workspace)
    g, Tq = _geometry(p), q.shape[2]
    shape = (g.batch, g.heads, Tq, g.d)
    s = q.stride()
    if q.dtype is not g.dtype or q.shape != shape or q.get_device() != dev or s[-1] != 1:
        _wrong_rows("q", q, g.dtype, shape, dev)
    if k_pages.dtype is not g.dtype or k_pages.stride() != g.strides or k_pages.shape != g.pool or k_pages.get_device() != dev:
        _check_pool(g, k_pages, dev)
    if v_pages.dtype is not g.dtype or v_pages.stride() != g.strides or v_pages.shape != g.pool or v_pages.get_device() != dev:
        _check_pool(g, v_pages, dev)
    if page_table.dtype is not _I32 or page_table.shape != g.table or page_table.get_device() != dev or not page_table.is_contiguous():
        _wrong("page_table", page_table, _I32, g.table, dev)
    if lens.dtype is not _I32 or lens.shape != g.each or lens.get_device() != dev or not lens.is_contiguous():
        _wrong("lens", lens, _I32, g.each, dev)
    if q_lens is not None and (q_lens.dtype is not _I32 or q_lens.shape != g.each or q_lens.get_device() != dev or not q_lens.is_contiguous()):
        _wrong("q_lens", q_lens, _I32, g.each, dev)
    new = torch.empty if q_lens is None else torch.zeros
    if out is None:
        out = new(shape, dtype=g.dtype, device=dev)
    o = out.stride()
    if out.dtype is not g.dtype or out.shape != shape or out.get_device() != dev or o[-1] != 1:
        _wrong_rows("out", out, g.dtype, shape, dev)
    if lse is True:
        lse = new(shape[:3], dtype=_F32, device=dev)
    elif lse is False:
        lse = None
    elif lse is not None and (lse.dtype is not _F32 or lse.shape != shape[:3] or lse.get_device() != dev or not lse.is_contiguous()):
        _wrong("lse", lse, _F32, shape[:3], dev)
    ws = _paged_ws(p, workspace, dev)
    st = g.lib.dkv_paged_prefill(
        g.ref, q.data_ptr(), _strides(s[0], s[1], s[2]), Tq, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
        lens.data_ptr(), None if q_lens is None else q_lens.data_ptr(), out.data_ptr(), _strides(o[0], o[1], o[2]),
        None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(),
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_paged_prefill")
    return out, lse


def dkv_paged_weights(p: dkv_paged, q: torch.Tensor, lse: torch.Tensor, k_pages: torch.Tensor, page_table: torch.Tensor,
                      lens: torch.Tensor, weights: torch.Tensor, q_lens: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Add the softmax weights that the queries (as in dkv_paged_prefill, with the lse it gave) give every
    token, summed over queries and a KV head's query heads, to weights fp32 [B, Hkv, max_pages * page_size]."""
    dev = q.get_device()
    if _elsewhere(q, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_paged_weights(p, q, lse, k_pages, page_table, lens, weights, q_lens, workspace)
    g, Tq = _geometry(p), q.shape[2]
    shape = (g.batch, g.heads, Tq, g.d)
    s = q.stride()
    if q.dtype is not g.dtype or q.shape != shape or q.get_device() != dev or s[-1] != 1:
        _wrong_rows("q", q, g.dtype, shape, dev)
    if lse.dtype is not _F32 or lse.shape != shape[:3] or lse.get_device() != dev or not lse.is_contiguous():
        _wrong("lse", lse, _F32, shape[:3], dev)
    if k_pages.dtype is not g.dtype or k_pages.stride() != g.strides or k_pages.shape != g.pool or k_pages.get_device() != dev:
        _check_pool(g, k_pages, dev)
    if page_table.dtype is not _I32 or page_table.shape != g.table or page_table.get_device() != dev or not page_table.is_contiguous():
        _wrong("page_table", page_table, _I32, g.table, dev)
    if lens.dtype is not _I32 or lens.shape != g.each or lens.get_device() != dev or not lens.is_contiguous():
        _wrong("lens", lens, _I32, g.each, dev)
    if q_lens is not None and (q_lens.dtype is not _I32 or q_lens.shape != g.each or q_lens.get_device() != dev or not q_lens.is_contiguous()):
        _wrong("q_lens", q_lens, _I32, g.each, dev)
    if weights.dtype is not _F32 or weights.shape != g.weights or weights.get_device() != dev or not weights.is_contiguous():
        _wrong("weights", weights, _F32, g.weights, dev)
    ws = _paged_ws(p, workspace, dev)
    st = g.lib.dkv_paged_weights(
        g.ref, q.data_ptr(), _strides(s[0], s[1], s[2]), Tq, lse.data_ptr(), k_pages.data_ptr(), page_table.data_ptr(),
        lens.data_ptr(), None if q_lens is None else q_lens.data_ptr(), weights.data_ptr(), ws.data_ptr(), ws.numel(),
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_paged_weights")
    return weights


def dkv_paged_evict(p: dkv_paged, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                    weights: torch.Tensor, budget: int, first: int, recent: int, new_table: torch.Tensor,
                    kept: torch.Tensor | None = None, new_lens: torch.Tensor | None = None,
                    new_weights: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Cut every sequence to `budget` tokens: the first `first`, the last `recent` and the heaviest between
    them, in order, moved to new_table's pages (int32 [B, n]; page_table itself compacts in place) ->
    (kept int32 [B, Hkv, budget], new_lens int32 [B], new_weights like weights)."""
    dev = k_pages.get_device()
    if _elsewhere(k_pages, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_paged_evict(p, k_pages, v_pages, page_table, lens, weights, budget, first, recent, new_table, kept,
                                   new_lens, new_weights, workspace)
    _int32("dkv_paged_evict", budget, first, recent)
    g, width = _geometry(p), new_table.shape[-1]
    k_shape, t_shape = (g.batch, g.kv_heads, max(budget, 0)), (g.batch, width)
    if k_pages.dtype is not g.dtype or k_pages.stride() != g.strides or k_pages.shape != g.pool or k_pages.get_device() != dev:
        _check_pool(g, k_pages, dev)
    if v_pages.dtype is not g.dtype or v_pages.stride() != g.strides or v_pages.shape != g.pool or v_pages.get_device() != dev:
        _check_pool(g, v_pages, dev)
    if page_table.dtype is not _I32 or page_table.shape != g.table or page_table.get_device() != dev or not page_table.is_contiguous():
        _wrong("page_table", page_table, _I32, g.table, dev)
    if lens.dtype is not _I32 or lens.shape != g.each or lens.get_device() != dev or not lens.is_contiguous():
        _wrong("lens", lens, _I32, g.each, dev)
    if weights.dtype is not _F32 or weights.shape != g.weights or weights.get_device() != dev or not weights.is_contiguous():
        _wrong("weights", weights, _F32, g.weights, dev)
    if new_table.dtype is not _I32 or new_table.shape != t_shape or new_table.get_device() != dev or not new_table.is_contiguous():
        _wrong("new_table", new_table, _I32, t_shape, dev)
    if kept is None:
        kept = torch.empty(k_shape, dtype=_I32, device=dev)
    if kept.dtype is not _I32 or kept.shape != k_shape or kept.get_device() != dev or not kept.is_contiguous():
        _wrong("kept", kept, _I32, k_shape, dev)
    if new_lens is None:
        new_lens = torch.empty(g.each, dtype=_I32, device=dev)
    if new_lens.dtype is not _I32 or new_lens.shape != g.each or new_lens.get_device() != dev or not new_lens.is_contiguous():
        _wrong("new_lens", new_lens, _I32, g.each, dev)
    if new_weights is None:
        new_weights = torch.empty(g.weights, dtype=_F32, device=dev)
    if new_weights.dtype is not _F32 or new_weights.shape != g.weights or new_weights.get_device() != dev or not new_weights.is_contiguous():
        _wrong("new_weights", new_weights, _F32, g.weights, dev)
    ws = _paged_ws(p, workspace, dev)
    st = g.lib.dkv_paged_evict(
        g.ref, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), lens.data_ptr(), weights.data_ptr(), budget,
        first, recent, new_table.data_ptr(), width, kept.data_ptr(), new_lens.data_ptr(), new_weights.data_ptr(),
        ws.data_ptr(), ws.numel(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_paged_evict")
    return kept, new_lens, new_weights


# ---------------------------------------------------------------- pages and slots, norm and rotation

_I64 = torch.int64


def dkv_paged_plan_workspace_bytes(p) -> int:
    """Bytes of dkv_paged_plan's workspace; p: a dkv_paged or dkv_qpaged."""
    return int(lib().dkv_paged_plan_workspace_bytes(p.batch))


def dkv_paged_plan(p, lens: torch.Tensor, news: torch.Tensor, free_pages: torch.Tensor, n_free: torch.Tensor,
                   page_table: torch.Tensor, rows: int, slots: torch.Tensor | None = None,
                   positions: torch.Tensor | None = None, starts: torch.Tensor | None = None,
                   granted: torch.Tensor | None = None, new_lens: torch.Tensor | None = None,
                   new_n_free: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Pages and slots of a step's new tokens: request b has lens[b] tokens and gets news[b] more (below 0:
    drops its last ones), int32 [B] each.  Pages come off and go back to the stack free_pages[:n_free] (int32,
    n_free int32 [1]) and into page_table int32 [B, max_pages], all in place -> (slots int64 [rows], positions
    int32 [rows], starts int32 [B + 1], granted int32 [B], new_lens int32 [B], new_n_free int32 [1]); rows
    behind the last token hold -1.  new_lens may be lens, new_n_free n_free.  `p`: a dkv_paged or dkv_qpaged."""
    dev = lens.get_device()
    if _elsewhere(lens, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_paged_plan(p, lens, news, free_pages, n_free, page_table, rows, slots, positions, starts, granted,
                                  new_lens, new_n_free, workspace)
    if not -0x80000000 <= rows <= 0x7fffffff:
        raise DkvError(DKV_ERR_ARG, "dkv_paged_plan")
    b, width = p.batch, p.max_pages
    each, row = (b,), (rows if rows > 0 else 0,)
    if slots is None:
        slots = torch.empty(row, dtype=_I64, device=dev)
    if positions is None:
        positions = torch.empty(row, dtype=_I32, device=dev)
    if starts is None:
        starts = torch.empty((b + 1,), dtype=_I32, device=dev)
    if granted is None:
        granted = torch.empty(each, dtype=_I32, device=dev)
    if new_lens is None:
        new_lens = torch.empty(each, dtype=_I32, device=dev)
    if new_n_free is None:
        new_n_free = torch.empty((1,), dtype=_I32, device=dev)
    if lens.dtype is not _I32 or lens.shape != each or lens.get_device() != dev or not lens.is_contiguous():
        _wrong("lens", lens, _I32, each, dev)
    if news.dtype is not _I32 or news.shape != each or news.get_device() != dev or not news.is_contiguous():
        _wrong("news", news, _I32, each, dev)
    if free_pages.dtype is not _I32 or free_pages.dim() != 1 or free_pages.get_device() != dev or not free_pages.is_contiguous():
        _wrong("free_pages", free_pages, _I32, (free_pages.numel(),), dev)
    if n_free.dtype is not _I32 or n_free.shape != (1,) or n_free.get_device() != dev:
        _wrong("n_free", n_free, _I32, (1,), dev)
    if page_table.dtype is not _I32 or page_table.shape != (b, width) or page_table.get_device() != dev or not page_table.is_contiguous():
        _wrong("page_table", page_table, _I32, (b, width), dev)
    if slots.dtype is not _I64 or slots.shape != row or slots.get_device() != dev or not slots.is_contiguous():
        _wrong("slots", slots, _I64, row, dev)
    if positions.dtype is not _I32 or positions.shape != row or positions.get_device() != dev or not positions.is_contiguous():
        _wrong("positions", positions, _I32, row, dev)
    if starts.dtype is not _I32 or starts.shape != (b + 1,) or starts.get_device() != dev or not starts.is_contiguous():
        _wrong("starts", starts, _I32, (b + 1,), dev)
    if granted.dtype is not _I32 or granted.shape != each or granted.get_device() != dev or not granted.is_contiguous():
        _wrong("granted", granted, _I32, each, dev)
    if new_lens.dtype is not _I32 or new_lens.shape != each or new_lens.get_device() != dev or not new_lens.is_contiguous():
        _wrong("new_lens", new_lens, _I32, each, dev)
    if new_n_free.dtype is not _I32 or new_n_free.shape != (1,) or new_n_free.get_device() != dev:
        _wrong("new_n_free", new_n_free, _I32, (1,), dev)
    if workspace is None:
        workspace = torch.zeros(max(dkv_paged_plan_workspace_bytes(p), 256), dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous() or workspace.element_size() != 1:
        raise ValueError("workspace: expected contiguous bytes on the tensors' device")
    st = lib().dkv_paged_plan(
        b, p.page_size, p.n_pages, width, lens.data_ptr(), news.data_ptr(), free_pages.data_ptr(), free_pages.shape[0],
        n_free.data_ptr(), page_table.data_ptr(), rows, slots.data_ptr(), positions.data_ptr(), starts.data_ptr(),
        granted.data_ptr(), new_lens.data_ptr(), new_n_free.data_ptr(), workspace.data_ptr(), workspace.numel(),
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_paged_plan")
    return slots, positions, starts, granted, new_lens, new_n_free


@functools.lru_cache(maxsize=256)
def _rotate(rows: int, hq: int, hkv: int, d: int, dtype: int, norm: bool, rope_dims: int, eps: float, base: float, inv_freq):
    r = dkv_rotate(rows, hq, hkv, d, dtype, norm, rope_dims, eps, base, None)
    if inv_freq is not None:
        r.inv_freq = (ctypes.c_double * len(inv_freq))(*inv_freq)
    return r, ctypes.byref(r)


def dkv_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, rope_dims: int, rope_base: float = 1e4,
                     inv_freq=None, q_gain: torch.Tensor | None = None, k_gain: torch.Tensor | None = None,
                     eps: float | None = 1e-6, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     p: dkv_paged | None = None, v: torch.Tensor | None = None, k_pages: torch.Tensor | None = None,
                     v_pages: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """Norm (eps None: none), gain [d] and rotation of q [rows, Hq, d] and k [rows, Hkv, d] (any strides with
    adjacent channels) at positions int32 [rows] -> (q_out, k_out), in place where those are q and k; rows at
    negative positions are left out (zeros in outputs allocated here).  `inv_freq`: rope_dims / 2 numbers, for
    rope_base^(-2j / rope_dims).  With p, v [rows, Hkv, d], k_pages, v_pages and slots int64 [rows] (-1: none) the
    rotated keys and the values also go into a 16-bit paged cache."""
    dev = q.get_device()
    if _elsewhere(q, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_qk_norm_rope(q, k, positions, rope_dims, rope_base, inv_freq, q_gain, k_gain, eps, q_out, k_out, p, v,
                                    k_pages, v_pages, slots, workspace)
    if q.dim() != 3 or k.dim() != 3 or q.dtype not in _PAGED_DTYPES:
        raise DkvError(DKV_ERR_ARG, "dkv_qk_norm_rope")
    dt = q.dtype
    rows, hq, d = q.shape
    hkv = k.shape[1]
    q_shape, k_shape = (rows, hq, d), (rows, hkv, d)
    if not (rows <= 0x7fffffff and -0x80000000 <= rope_dims <= 0x7fffffff):
        raise DkvError(DKV_ERR_ARG, "dkv_qk_norm_rope")
    qs, ks = q.stride(), k.stride()
    if qs[2] != 1:
        _wrong_rows("q", q, dt, q_shape, dev)
    if k.dtype is not dt or k.shape != k_shape or k.get_device() != dev or ks[2] != 1:
        _wrong_rows("k", k, dt, k_shape, dev)
    if positions.dtype is not _I32 or positions.shape != (rows,) or positions.get_device() != dev or not positions.is_contiguous():
        _wrong("positions", positions, _I32, (rows,), dev)
    if q_gain is not None and (q_gain.dtype is not dt or q_gain.shape != (d,) or q_gain.get_device() != dev or not q_gain.is_contiguous()):
        _wrong("q_gain", q_gain, dt, (d,), dev)
    if k_gain is not None and (k_gain.dtype is not dt or k_gain.shape != (d,) or k_gain.get_device() != dev or not k_gain.is_contiguous()):
        _wrong("k_gain", k_gain, dt, (d,), dev)
    if q_out is None:
        q_out = torch.zeros(q_shape, dtype=dt, device=dev)
    if k_out is None:
        k_out = torch.zeros(k_shape, dtype=dt, device=dev)
    qo, ko = q_out.stride(), k_out.stride()
    if q_out.dtype is not dt or q_out.shape != q_shape or q_out.get_device() != dev or qo[2] != 1:
        _wrong_rows("q_out", q_out, dt, q_shape, dev)
    if k_out.dtype is not dt or k_out.shape != k_shape or k_out.get_device() != dev or ko[2] != 1:
        _wrong_rows("k_out", k_out, dt, k_shape, dev)
    pref = vp = vs = sp = kp = vpp = None
    if p is not None or v is not None or k_pages is not None or v_pages is not None or slots is not None:
        if p is None or v is None or k_pages is None or v_pages is None or slots is None:
            raise DkvError(DKV_ERR_ARG, "dkv_qk_norm_rope")
        g = _geometry(p)
        s = v.stride()
        if v.dtype is not dt or v.shape != k_shape or v.get_device() != dev or s[2] != 1:
            _wrong_rows("v", v, dt, k_shape, dev)
        if k_pages.dtype is not g.dtype or k_pages.stride() != g.strides or k_pages.shape != g.pool or k_pages.get_device() != dev:
            _check_pool(g, k_pages, dev)
        if v_pages.dtype is not g.dtype or v_pages.stride() != g.strides or v_pages.shape != g.pool or v_pages.get_device() != dev:
            _check_pool(g, v_pages, dev)
        if slots.dtype is not _I64 or slots.shape != (rows,) or slots.get_device() != dev or not slots.is_contiguous():
            _wrong("slots", slots, _I64, (rows,), dev)
        pref, vp, vs, sp, kp, vpp = g.ref, v.data_ptr(), _strides(0, s[1], s[0]), slots.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr()
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous() or workspace.element_size() != 1):
        raise ValueError("workspace: expected contiguous bytes on the tensors' device")
    if inv_freq is not None:
        inv_freq = tuple(float(x) for x in inv_freq)
        if len(inv_freq) != rope_dims // 2:
            raise DkvError(DKV_ERR_ARG, "dkv_qk_norm_rope")
    _, ref = _rotate(rows, hq, hkv, d, _PAGED_DTYPES[dt], eps is not None, rope_dims, 0.0 if eps is None else float(eps),
                     float(rope_base), inv_freq)
    st = lib().dkv_qk_norm_rope(
        ref, q.data_ptr(), _strides(0, qs[1], qs[0]), k.data_ptr(), _strides(0, ks[1], ks[0]),
        None if q_gain is None else q_gain.data_ptr(), None if k_gain is None else k_gain.data_ptr(), positions.data_ptr(),
        q_out.data_ptr(), _strides(0, qo[1], qo[0]), k_out.data_ptr(), _strides(0, ko[1], ko[0]), pref, vp, vs, sp, kp, vpp,
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_qk_norm_rope")
    return q_out, k_out


# ---------------------------------------------------------------- paged cache in 4 bits

class _QGeometry:
    """What the calls compare their tensors with, from a descriptor's bytes."""

    __slots__ = ("key", "ref", "dtype", "pool", "strides", "batch", "heads", "kv_heads", "d", "each", "table", "q1", "lse1", "lib")

    def __init__(self, p: dkv_qpaged, key: bytes):
        self.key, self.ref = key, ctypes.byref(p)
        self.dtype = torch.bfloat16 if p.dtype == DKV_BF16 else torch.float16
        self.batch, self.heads, self.kv_heads, self.d = p.batch, p.n_q_heads, p.n_kv_heads, p.head_dim
        self.pool = (p.n_pages, p.n_kv_heads, p.page_size * p.head_dim * 9 // 8)
        self.strides = (p.stride_page, p.stride_head, 1)
        self.each, self.table = (p.batch,), (p.batch, p.max_pages)
        self.q1, self.lse1 = (p.batch, p.n_q_heads, p.head_dim), (p.batch, p.n_q_heads)
        self.lib = lib()


def _qgeometry(p: dkv_qpaged) -> _QGeometry:
    key = bytes(p)
    g = p.__dict__.get("_geometry")
    if g is None or g.key != key:
        g = p._geometry = _QGeometry(p, key)
    return g


def _check_cache(g: _QGeometry, t: torch.Tensor, dev: int) -> None:
    if t.dtype is not torch.uint8 or t.shape != g.pool or t.get_device() != dev:
        raise ValueError(f"cache: expected {torch.uint8} {g.pool} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.stride() != g.strides and any(n > 1 and a != b for n, a, b in zip(g.pool, t.stride(), g.strides)):
        raise ValueError(f"cache: strides {t.stride()} are not the descriptor's {g.strides}")


def _qpaged_ws(p: dkv_qpaged, workspace, dev: int) -> torch.Tensor:
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous() or workspace.element_size() != 1:
            raise ValueError("workspace: expected contiguous bytes on the tensors' device")
        return workspace
    ws = torch.empty(dkv_qpaged_workspace_bytes(p), dtype=torch.uint8, device=dev)
    ws[:256].zero_()
    return ws


def dkv_qpaged_layout(cache: torch.Tensor, batch: int, n_q_heads: int, head_dim: int, max_pages: int,
                      dtype: torch.dtype = torch.float16, window: int = 0, sinks: int = 0) -> dkv_qpaged:
    """Descriptor of a paged cache in 4 bits from its pool, uint8 [n_pages, Hkv, page_size * head_dim * 9 / 8]
    (keys and values together; page and head strides may be any multiples of 16).  `dtype`: fp16 or bf16, of
    rows, queries and outputs; `window`, `sinks` as in dkv_paged_layout."""
    if cache.dim() != 3 or cache.dtype is not torch.uint8 or cache.stride(2) != 1 or dtype not in _PAGED_DTYPES or head_dim not in (64, 128):
        raise DkvError(DKV_ERR_ARG if head_dim in (64, 128) else DKV_ERR_UNSUPPORTED, "dkv_qpaged_layout")
    n_pages, hkv, page_bytes = cache.shape
    if page_bytes * 8 % (9 * head_dim):
        raise DkvError(DKV_ERR_SHAPE, "dkv_qpaged_layout")
    page = page_bytes * 8 // (9 * head_dim)
    _int32("dkv_qpaged_layout", batch, n_q_heads, max_pages, n_pages, hkv, page, window, sinks)
    sp, sh, _ = cache.stride()
    p = dkv_qpaged(batch, n_q_heads, hkv, head_dim, page, n_pages, max_pages, _PAGED_DTYPES[dtype], window, sinks, sp, sh)
    _check(lib().dkv_qpaged_check(ctypes.byref(p)), "dkv_qpaged_layout")
    return p


def dkv_qpaged_workspace_bytes(p: dkv_qpaged) -> int:
    """Bytes of the workspace of every call below; a call without one makes its own, and with that goes the
    word that tells of bad lengths, pages, slots and values (dkv_get_error)."""
    return int(lib().dkv_qpaged_workspace_bytes(ctypes.byref(p)))


def dkv_qpaged_append(p: dkv_qpaged, K_new: torch.Tensor, V_new: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
                      workspace: torch.Tensor | None = None, stream=None) -> None:
    """Write rows K_new, V_new [rows, Hkv, d] (any strides with adjacent channels) in 4 bits to their slots,
    int64 [rows] (page * page_size + place in the page, as dkv_paged_plan gives them; -1: left out)."""
    dev = K_new.get_device()
    if _elsewhere(K_new, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_qpaged_append(p, K_new, V_new, cache, slots, workspace)
    g = _qgeometry(p)
    if K_new.stride() != V_new.stride():
        K_new, V_new = K_new.contiguous(), V_new.contiguous()
    rows = K_new.shape[0]
    shape = (rows, g.kv_heads, g.d)
    s = K_new.stride()
    if K_new.dtype is not g.dtype or K_new.shape != shape or K_new.get_device() != dev or s[-1] != 1:
        _wrong_rows("K_new", K_new, g.dtype, shape, dev)
    if V_new.dtype is not g.dtype or V_new.shape != shape or V_new.get_device() != dev:
        _wrong_rows("V_new", V_new, g.dtype, shape, dev)
    if cache.dtype is not torch.uint8 or cache.stride() != g.strides or cache.shape != g.pool or cache.get_device() != dev:
        _check_cache(g, cache, dev)
    if slots.dtype is not _I64 or slots.shape != (rows,) or slots.get_device() != dev or not slots.is_contiguous():
        _wrong("slots", slots, _I64, (rows,), dev)
    ws = _qpaged_ws(p, workspace, dev)
    st = g.lib.dkv_qpaged_append(g.ref, K_new.data_ptr(), V_new.data_ptr(), _strides(0, s[1], s[0]), rows, slots.data_ptr(),
                                 cache.data_ptr(), ws.data_ptr(), ws.numel(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_qpaged_append")


def dkv_qpaged_gather(p: dkv_qpaged, cache: torch.Tensor, page_table: torch.Tensor, first: torch.Tensor, K_out: torch.Tensor,
                      V_out: torch.Tensor, counts: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None):
    """Read tokens back: token i < counts[b] (None: all n) from position first[b] + i of sequence b into K_out, V_out
    [B, Hkv, n, d] (any strides with adjacent channels, both alike) -> (K_out, V_out).  Rows from counts[b] on stay."""
    dev = cache.get_device()
    if _elsewhere(cache, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_qpaged_gather(p, cache, page_table, first, K_out, V_out, counts, workspace)
    g = _qgeometry(p)
    n = K_out.shape[2]
    shape = (g.batch, g.kv_heads, n, g.d)
    s = K_out.stride()
    if K_out.dtype is not g.dtype or K_out.shape != shape or K_out.get_device() != dev or s[-1] != 1:
        _wrong_rows("K_out", K_out, g.dtype, shape, dev)
    if V_out.dtype is not g.dtype or V_out.shape != shape or V_out.get_device() != dev or V_out.stride() != s:
        _wrong_rows("V_out", V_out, g.dtype, shape, dev)
    if cache.dtype is not torch.uint8 or cache.stride() != g.strides or cache.shape != g.pool or cache.get_device() != dev:
        _check_cache(g, cache, dev)
    if page_table.dtype is not _I32 or page_table.shape != g.table or page_table.get_device() != dev or not page_table.is_contiguous():
        _wrong("page_table", page_table, _I32, g.table, dev)
    if first.dtype is not _I32 or first.shape != g.each or first.get_device() != dev or not first.is_contiguous():
        _wrong("first", first, _I32, g.each, dev)
    if counts is not None and (counts.dtype is not _I32 or counts.shape != g.each or counts.get_device() != dev or not counts.is_contiguous()):
        _wrong("counts", counts, _I32, g.each, dev)
    ws = _qpaged_ws(p, workspace, dev)
    st = g.lib.dkv_qpaged_gather(
        g.ref, cache.data_ptr(), page_table.data_ptr(), first.data_ptr(), None if counts is None else counts.data_ptr(), n,
        K_out.data_ptr(), V_out.data_ptr(), _strides(s[0], s[1], s[2]), ws.data_ptr(), ws.numel(),
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_qpaged_gather")
    return K_out, V_out


def dkv_qpaged_decode(p: dkv_qpaged, q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                      out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = True,
                      workspace: torch.Tensor | None = None, stream=None):
    """One new token per sequence: q [B, Hq, d] at position lens[b] - 1 -> (out [B, Hq, d] in q's type, lse fp32
    [B, Hq] or None)."""
    dev = q.get_device()
    if _elsewhere(q, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_qpaged_decode(p, q, cache, page_table, lens, out, lse, workspace)
    g = _qgeometry(p)
    s = q.stride()
    if q.dtype is not g.dtype or q.shape != g.q1 or q.get_device() != dev or s[-1] != 1:
        _wrong_rows("q", q, g.dtype, g.q1, dev)
    if cache.dtype is not torch.uint8 or cache.stride() != g.strides or cache.shape != g.pool or cache.get_device() != dev:
        _check_cache(g, cache, dev)
    if page_table.dtype is not _I32 or page_table.shape != g.table or page_table.get_device() != dev or not page_table.is_contiguous():
        _wrong("page_table", page_table, _I32, g.table, dev)
    if lens.dtype is not _I32 or lens.shape != g.each or lens.get_device() != dev or not lens.is_contiguous():
        _wrong("lens", lens, _I32, g.each, dev)
    if out is None:
        out = torch.empty(g.q1, dtype=g.dtype, device=dev)
    elif out.dtype is not g.dtype or out.shape != g.q1 or out.get_device() != dev or not out.is_contiguous():
        _wrong("out", out, g.dtype, g.q1, dev)
    if lse is True:
        lse = torch.empty(g.lse1, dtype=_F32, device=dev)
    elif lse is False:
        lse = None
    elif lse is not None and (lse.dtype is not _F32 or lse.shape != g.lse1 or lse.get_device() != dev or not lse.is_contiguous()):
        _wrong("lse", lse, _F32, g.lse1, dev)
    ws = _qpaged_ws(p, workspace, dev)
    st = g.lib.dkv_qpaged_decode(
        g.ref, q.data_ptr(), _strides(s[0], s[1], 0), cache.data_ptr(), page_table.data_ptr(), lens.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_qpaged_decode")
    return out, lse


def dkv_qpaged_prefill(p: dkv_qpaged, q: torch.Tensor, starts: torch.Tensor, max_q: int, cache: torch.Tensor,
                       page_table: torch.Tensor, lens: torch.Tensor, out: torch.Tensor | None = None,
                       lse: torch.Tensor | bool | None = True, workspace: torch.Tensor | None = None, stream=None):
    """The last tokens of each sequence, rows one behind the other: q [rows, Hq, d], sequence b's queries rows
    starts[b] .. starts[b + 1] - 1 (int32 [B + 1]; at most max_q each), the last at position lens[b] - 1 ->
    (out [rows, Hq, d] in q's type, lse fp32 [Hq, rows] or None).  Rows outside every span stay (zeros in outputs
    allocated here)."""
    dev = q.get_device()
    if _elsewhere(q, dev) or stream is not None:
        with _place(dev, stream):
            return dkv_qpaged_prefill(p, q, starts, max_q, cache, page_table, lens, out, lse, workspace)
    if not -0x80000000 <= max_q <= 0x7fffffff:
        raise DkvError(DKV_ERR_ARG, "dkv_qpaged_prefill")
    g, rows = _qgeometry(p), q.shape[0]
    shape = (rows, g.heads, g.d)
    s = q.stride()
    if q.dtype is not g.dtype or q.shape != shape or q.get_device() != dev or s[-1] != 1:
        _wrong_rows("q", q, g.dtype, shape, dev)
    if starts.dtype is not _I32 or starts.shape != (g.batch + 1,) or starts.get_device() != dev or not starts.is_contiguous():
        _wrong("starts", starts, _I32, (g.batch + 1,), dev)
    if cache.dtype is not torch.uint8 or cache.stride() != g.strides or cache.shape != g.pool or cache.get_device() != dev:
        _check_cache(g, cache, dev)
    if page_table.dtype is not _I32 or page_table.shape != g.table or page_table.get_device() != dev or not page_table.is_contiguous():
        _wrong("page_table", page_table, _I32, g.table, dev)
    if lens.dtype is not _I32 or lens.shape != g.each or lens.get_device() != dev or not lens.is_contiguous():
        _wrong("lens", lens, _I32, g.each, dev)
    if out is None:
        out = torch.zeros(shape, dtype=g.dtype, device=dev)
    o = out.stride()
    if out.dtype is not g.dtype or out.shape != shape or out.get_device() != dev or o[-1] != 1:
        _wrong_rows("out", out, g.dtype, shape, dev)
    l_shape = (g.heads, rows)
    if lse is True:
        lse = torch.zeros(l_shape, dtype=_F32, device=dev)
    elif lse is False:
        lse = None
    elif lse is not None and (lse.dtype is not _F32 or lse.shape != l_shape or lse.get_device() != dev or not lse.is_contiguous()):
        _wrong("lse", lse, _F32, l_shape, dev)
    ws = _qpaged_ws(p, workspace, dev)
    st = g.lib.dkv_qpaged_prefill(
        g.ref, q.data_ptr(), _strides(0, s[1], s[0]), rows, max_q, starts.data_ptr(), cache.data_ptr(), page_table.data_ptr(),
        lens.data_ptr(), out.data_ptr(), _strides(0, o[1], o[0]), None if lse is None else lse.data_ptr(), ws.data_ptr(),
        ws.numel(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, "dkv_qpaged_prefill")
    return out, lse


def dkv_debug_set_limits(stop_after_chunks: int = -1, wait_polls: int = 0) -> None:
    """Failure-path diagnostics: producers of the fragment layout's attention CTAs stop
    after `stop_after_chunks` chunks, bounded waits give up after `wait_polls` polls;
    (-1, 0) restores the defaults."""
    _check(lib().dkv_debug_set_limits(int(stop_after_chunks), int(wait_polls)), "dkv_debug_set_limits")


def dkv_debug_set_launch(programmatic: bool = True) -> None:
    """Timing aid: False launches the decode grids in plain stream order (no programmatic
    overlap with the grid before them); True restores the default."""
    _check(lib().dkv_debug_set_launch(1 if programmatic else 0), "dkv_debug_set_launch")


def dkv_get_error(workspace: torch.Tensor, stream=None) -> tuple[int, int]:
    """(status, device error word); clears the word."""
    w = ctypes.c_uint32(0)
    st = lib().dkv_get_error(_ptr(workspace), _stream(stream), ctypes.byref(w))
    return st, int(w.value)
