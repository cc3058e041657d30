"""ctypes binding of libmla_paged_fp8.so (argument marshalling only).

Every step of the decode runs in the library's CUDA kernels; this module only
turns torch tensors into pointers and shapes.  It raises if the compiled
library is missing: there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmla_paged_fp8.so")

MLA_OK = 0
STATUS_NAMES = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_CUDA",
                4: "MLA_ERR_WORKSPACE", 5: "MLA_ERR_TIMEOUT", 6: "MLA_ERR_DEVICE_BOUNDS"}

# every symbol include/mla_paged_fp8.h declares
EXPORTED = ["mla_decode_paged_fp8", "mla_gather_dequant_bf16", "mla_set_num_clusters",
            "mla_get_num_clusters", "mla_last_error_string", "mla_get_device_status",
            "mla_release_workspace", "mla_version", "mla_set_timing_events", "mla_decode_paged_fp8_noalloc",
            "mla_kv_store_fp8", "mla_decode_paged_fp8_scale_folded", "mla_merge_lse_parts_bf16",
            "mla_set_wait_limit_ns", "mla_debug_withhold_arrival_once", "mla_decode_paged_fp8_e4m3_pv",
            "mla_decode_paged_fp8_host", "mla_accumulate_weights_fp8", "mla_accumulate_workspace_bytes", "mla_select_keys", "mla_compact_paged",
            "mla_mha_kv_store", "mla_mha_decode_paged", "mla_mha_decode_workspace_bytes"]

VARIANT_DECODE, VARIANT_SCALE_FOLDED, VARIANT_E4M3_PV = 0, 1, 2


class MlaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class PagedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_q_heads", "head_dim", "v_dim", "num_blocks", "kv_dim", "num_layers", "page_size",
        "num_kv_heads", "num_scale_blocks", "head_dim_granularity", "max_pages")]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (once).  Raises FileNotFoundError when it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with `python -m paged_fp8_kv_mla_b200.build`")
    lib = ctypes.CDLL(path)
    vp, u32, f32, i32 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_float, ctypes.c_int32
    lib.mla_decode_paged_fp8.argtypes = [vp, vp, vp, vp, vp, vp, u32, u32, u32, f32,
                                         ctypes.POINTER(PagedShape), vp, vp, vp]
    lib.mla_decode_paged_fp8.restype = ctypes.c_int
    lib.mla_merge_lse_parts_bf16.argtypes = [vp, vp, ctypes.c_int32, ctypes.c_int64, vp, vp, vp]
    lib.mla_merge_lse_parts_bf16.restype = ctypes.c_int
    lib.mla_decode_paged_fp8_scale_folded.argtypes = lib.mla_decode_paged_fp8.argtypes
    lib.mla_decode_paged_fp8_scale_folded.restype = ctypes.c_int
    lib.mla_decode_paged_fp8_e4m3_pv.argtypes = lib.mla_decode_paged_fp8.argtypes
    lib.mla_decode_paged_fp8_e4m3_pv.restype = ctypes.c_int
    lib.mla_decode_paged_fp8_host.argtypes = [vp, vp, vp, vp, vp, vp, u32, u32, u32, f32,
                                              ctypes.POINTER(PagedShape), vp, vp, i32, i32, vp]
    lib.mla_decode_paged_fp8_host.restype = ctypes.c_int
    lib.mla_decode_paged_fp8_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, u32, u32, u32, f32,
                                                 ctypes.POINTER(PagedShape), vp, vp, vp]
    lib.mla_decode_paged_fp8_noalloc.restype = ctypes.c_int
    lib.mla_gather_dequant_bf16.argtypes = [vp, vp, vp, vp, vp, u32, u32, u32,
                                            ctypes.POINTER(PagedShape), vp, u32, vp]
    lib.mla_gather_dequant_bf16.restype = ctypes.c_int
    lib.mla_kv_store_fp8.argtypes = [vp, vp, vp, vp, u32, u32, ctypes.POINTER(PagedShape), vp, vp, vp]
    lib.mla_kv_store_fp8.restype = ctypes.c_int
    shp, i64, u64 = ctypes.POINTER(PagedShape), ctypes.c_int64, ctypes.c_uint64
    lib.mla_accumulate_weights_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, u32, u32, u32, f32, shp, vp, i64, vp, i64,
                                               vp, u64, vp]
    lib.mla_accumulate_weights_fp8.restype = ctypes.c_int
    lib.mla_accumulate_workspace_bytes.argtypes = [u32, shp, ctypes.POINTER(u64)]
    lib.mla_accumulate_workspace_bytes.restype = ctypes.c_int
    lib.mla_select_keys.argtypes = [vp, i64, vp, i32, u32, i32, i32, i32, vp, i64, vp, vp]
    lib.mla_select_keys.restype = ctypes.c_int
    lib.mla_compact_paged.argtypes = [vp, i64, i32, vp, vp, vp, u32, i32, shp, vp, vp, vp, i64, i32, vp]
    lib.mla_compact_paged.restype = ctypes.c_int
    lib.mla_mha_kv_store.argtypes = [vp, vp, vp, vp, vp, u32, u32, i32, shp, vp, vp, vp]
    lib.mla_mha_kv_store.restype = ctypes.c_int
    lib.mla_mha_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, u32, u32, u32, f32, i32, shp, vp, vp, vp, u64, vp]
    lib.mla_mha_decode_paged.restype = ctypes.c_int
    lib.mla_mha_decode_workspace_bytes.argtypes = [u32, u32, i32, shp, ctypes.POINTER(u64)]
    lib.mla_mha_decode_workspace_bytes.restype = ctypes.c_int
    lib.mla_set_num_clusters.argtypes = [i32]
    lib.mla_set_num_clusters.restype = ctypes.c_int
    lib.mla_get_num_clusters.argtypes = []
    lib.mla_get_num_clusters.restype = i32
    lib.mla_last_error_string.argtypes = []
    lib.mla_last_error_string.restype = ctypes.c_char_p
    lib.mla_get_device_status.argtypes = [vp]
    lib.mla_get_device_status.restype = ctypes.c_int
    lib.mla_release_workspace.argtypes = []
    lib.mla_release_workspace.restype = ctypes.c_int
    lib.mla_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.mla_set_wait_limit_ns.restype = ctypes.c_int
    lib.mla_debug_withhold_arrival_once.argtypes = []
    lib.mla_debug_withhold_arrival_once.restype = ctypes.c_int
    lib.mla_set_timing_events.argtypes = [vp, vp]
    lib.mla_set_timing_events.restype = ctypes.c_int
    lib.mla_version.argtypes = []
    lib.mla_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(st: int):
    if st != MLA_OK:
        raise MlaError(st, load().mla_last_error_string().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def paged_shape(batch, num_q_heads, blocks: torch.Tensor, scales: torch.Tensor, lookup_table: torch.Tensor) -> PagedShape:
    """Shape record from the 6-D blocks / scales tensors and the 2-D page table."""
    NB, KVD, NL, P, NKV, D = blocks.shape
    return PagedShape(batch=batch, num_q_heads=num_q_heads, head_dim=D, v_dim=512, num_blocks=NB, kv_dim=KVD,
                      num_layers=NL, page_size=P, num_kv_heads=NKV, num_scale_blocks=scales.shape[0],
                      head_dim_granularity=scales.shape[-1], max_pages=lookup_table.shape[1])


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


_U32 = (torch.int32,) + ((torch.uint32,) if hasattr(torch, "uint32") else ())
_CODES = (torch.uint8,) + ((torch.float8_e4m3fn,) if hasattr(torch, "float8_e4m3fn") else ())


def _expect(name, t, dtypes, ndim=None, last=None, optional=False):
    """The C ABI takes untyped pointers, so the binding checks what it passes: dtype, rank, last dim
    and contiguity (the device is checked last, by _same_device)."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D (got shape {tuple(t.shape)})")
    if last is not None and t.shape[-1] != last:
        raise ValueError(f"{name} must have last dim {last} (got shape {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _same_device(*ts):
    devs = {t.device for t in ts if t is not None}
    if any(d.type != "cuda" for d in devs):
        raise ValueError("all tensors must be CUDA tensors")
    if len(devs) > 1:
        raise ValueError(f"all tensors must be on one CUDA device (got {sorted(str(d) for d in devs)})")


def _check_cache(blocks, scales, cache_lengths, lookup_table, scales_lookup_table, batch):
    _expect("blocks", blocks, _CODES, ndim=6)
    _expect("scales", scales, (torch.float32,), ndim=6)
    _expect("cache_lengths", cache_lengths, _U32, ndim=1)
    _expect("lookup_table", lookup_table, _U32, ndim=2)
    _expect("scales_lookup_table", scales_lookup_table, _U32, ndim=2, optional=True)
    if cache_lengths.shape[0] != batch or lookup_table.shape[0] != batch:
        raise ValueError(f"cache_lengths and lookup_table must have {batch} rows (one per request)")
    if scales_lookup_table is not None and tuple(scales_lookup_table.shape) != tuple(lookup_table.shape):
        raise ValueError("scales_lookup_table must have the shape of lookup_table")


def _check_decode(q, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, out, lse):
    _expect("q", q, (torch.bfloat16,), ndim=4, last=576)
    B, T, H, _ = q.shape
    _check_cache(blocks, scales, cache_lengths, lookup_table, scales_lookup_table, B)
    _expect("out", out, (torch.bfloat16,), ndim=4, last=512, optional=True)
    _expect("lse", lse, (torch.float32,), ndim=3, optional=True)
    if out is not None and tuple(out.shape) != (B, T, H, 512):
        raise ValueError(f"out must be {(B, T, H, 512)} (got {tuple(out.shape)})")
    if lse is not None and tuple(lse.shape) != (B, T, H):
        raise ValueError(f"lse must be {(B, T, H)} (got {tuple(lse.shape)})")
    _same_device(q, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, out, lse)


def decode(q, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, max_prompt_length: int,
           max_cache_length: int, layer_idx: int, softmax_scale: float, out=None, lse=None, stream=None,
           want_lse: bool = True, fold_scales: bool = False, e4m3_pv: bool = False):
    """mla_decode_paged_fp8 on torch tensors (all on the current CUDA device).

    q bf16 [B, T, H, 576]; blocks uint8 [NB, kv_dim, L, P, 1, 576]; scales fp32 [NSB, kv_dim, L, P, 1, g];
    cache_lengths / lookup_table / scales_lookup_table int32 tensors holding uint32 values.
    fold_scales=True calls mla_decode_paged_fp8_scale_folded instead, e4m3_pv=True
    mla_decode_paged_fp8_e4m3_pv (g = 1 only, at most one of the two).
    Returns (out bf16 [B, T, H, 512], lse fp32 [B, T, H] or None).
    """
    if fold_scales and e4m3_pv:
        raise ValueError("fold_scales and e4m3_pv select different kernels: pass at most one")
    _check_decode(q, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, out, lse)
    lib = load()
    B, T, H, D = q.shape
    if out is None:
        out = torch.empty((B, T, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    shp = paged_shape(B, H, blocks, scales, lookup_table)
    fn = (lib.mla_decode_paged_fp8_scale_folded if fold_scales else
          lib.mla_decode_paged_fp8_e4m3_pv if e4m3_pv else lib.mla_decode_paged_fp8)
    st = fn(_ptr(q), _ptr(blocks), _ptr(scales), _ptr(cache_lengths), _ptr(lookup_table), _ptr(scales_lookup_table),
            int(max_prompt_length), int(max_cache_length), int(layer_idx), float(softmax_scale), ctypes.byref(shp),
            _ptr(out), _ptr(lse), _stream(stream))
    _check(st)
    return out, lse


def decode_host(q, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, max_prompt_length: int,
                max_cache_length: int, layer_idx: int, softmax_scale: float, out, lse=None, variant: int = 0,
                num_chunks: int = 0, stream=None):
    """mla_decode_paged_fp8_host: q, cache_lengths, the page tables, out and lse are CPU tensors (best
    pinned), blocks and scales CUDA tensors on the current device.  Asynchronous on `stream`: out and
    lse are complete after that stream is synchronised.  variant: VARIANT_DECODE, VARIANT_SCALE_FOLDED
    or VARIANT_E4M3_PV; num_chunks 0 = automatic."""
    _expect("q", q, (torch.bfloat16,), ndim=4, last=576)
    B, T, H, _ = q.shape
    _expect("blocks", blocks, _CODES, ndim=6)
    _expect("scales", scales, (torch.float32,), ndim=6)
    _expect("cache_lengths", cache_lengths, _U32, ndim=1)
    _expect("lookup_table", lookup_table, _U32, ndim=2)
    _expect("scales_lookup_table", scales_lookup_table, _U32, ndim=2, optional=True)
    _expect("out", out, (torch.bfloat16,), ndim=4, last=512)
    _expect("lse", lse, (torch.float32,), ndim=3, optional=True)
    if cache_lengths.shape[0] != B or lookup_table.shape[0] != B:
        raise ValueError(f"cache_lengths and lookup_table must have {B} rows (one per request)")
    if scales_lookup_table is not None and tuple(scales_lookup_table.shape) != tuple(lookup_table.shape):
        raise ValueError("scales_lookup_table must have the shape of lookup_table")
    if tuple(out.shape) != (B, T, H, 512) or (lse is not None and tuple(lse.shape) != (B, T, H)):
        raise ValueError("out / lse shapes do not match q")
    host = [t for t in (q, cache_lengths, lookup_table, scales_lookup_table, out, lse) if t is not None]
    if any(t.device.type != "cpu" for t in host):
        raise ValueError("q, cache_lengths, the page tables, out and lse must be CPU tensors")
    _same_device(blocks, scales)
    lib = load()
    shp = paged_shape(B, H, blocks, scales, lookup_table)
    st = lib.mla_decode_paged_fp8_host(_ptr(q), _ptr(blocks), _ptr(scales), _ptr(cache_lengths), _ptr(lookup_table),
                                       _ptr(scales_lookup_table), int(max_prompt_length), int(max_cache_length),
                                       int(layer_idx), float(softmax_scale), ctypes.byref(shp), _ptr(out), _ptr(lse),
                                       int(variant), int(num_chunks), _stream(stream))
    _check(st)
    return out, lse


def kv_store(latent, cache_lengths, lookup_table, scales_lookup_table, layer_idx: int, blocks, scales,
             stream=None):
    """mla_kv_store_fp8 on torch tensors: quantise latent bf16 [B, T, 576] and write it in place into
    blocks / scales at positions cache_lengths[b] + i (page tables as for decode)."""
    _expect("latent", latent, (torch.bfloat16,), ndim=3, last=576)
    B, T, D = latent.shape
    _check_cache(blocks, scales, cache_lengths, lookup_table, scales_lookup_table, B)
    _same_device(latent, blocks, scales, cache_lengths, lookup_table, scales_lookup_table)
    lib = load()
    shp = paged_shape(B, 0, blocks, scales, lookup_table)
    st = lib.mla_kv_store_fp8(_ptr(latent), _ptr(cache_lengths), _ptr(lookup_table), _ptr(scales_lookup_table),
                              int(T), int(layer_idx), ctypes.byref(shp), _ptr(blocks), _ptr(scales), _stream(stream))
    _check(st)
    return blocks, scales


def decode_noalloc(q, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, max_prompt_length: int,
                   max_cache_length: int, layer_idx: int, softmax_scale: float, out, lse, stream=None):
    """mla_decode_paged_fp8_noalloc: the decode on the library's fixed scratch (no device allocation).

    `out` and `lse` must be preallocated by the caller.
    """
    if out is None or lse is None:
        raise ValueError("decode_noalloc needs preallocated out and lse")
    _check_decode(q, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, out, lse)
    lib = load()
    B, T, H, D = q.shape
    shp = paged_shape(B, H, blocks, scales, lookup_table)
    st = lib.mla_decode_paged_fp8_noalloc(_ptr(q), _ptr(blocks), _ptr(scales), _ptr(cache_lengths),
                                          _ptr(lookup_table), _ptr(scales_lookup_table), int(max_prompt_length),
                                          int(max_cache_length), int(layer_idx), float(softmax_scale),
                                          ctypes.byref(shp), _ptr(out), _ptr(lse), _stream(stream))
    _check(st)
    return out, lse


def merge_parts(outs, lses, out=None, lse=None, stream=None):
    """mla_merge_lse_parts_bf16: outs bf16 [R, ..., 512] and lses fp32 [R, ...] (the parts' decode
    results over disjoint key ranges) -> (out bf16 [..., 512], lse fp32 [...])."""
    _expect("outs", outs, (torch.bfloat16,), last=512)
    _expect("lses", lses, (torch.float32,))
    if outs.dim() < 2 or outs.shape[:-1] != lses.shape:
        raise ValueError("outs must be [R, ..., 512] and lses [R, ...] with the same leading dims")
    _expect("out", out, (torch.bfloat16,), optional=True)
    _expect("lse", lse, (torch.float32,), optional=True)
    _same_device(outs, lses, out, lse)
    lib = load()
    R = outs.shape[0]
    rows = lses[0].numel()
    if out is None:
        out = torch.empty(outs.shape[1:], dtype=torch.bfloat16, device=outs.device)
    if lse is None:
        lse = torch.empty(lses.shape[1:], dtype=torch.float32, device=lses.device)
    _contig(out, lse)
    st = lib.mla_merge_lse_parts_bf16(_ptr(outs), _ptr(lses), int(R), int(rows), _ptr(out), _ptr(lse), _stream(stream))
    _check(st)
    return out, lse


def decode_inputs(inp, **kw):
    """decode() on a workloads.DecodeInputs bundle."""
    return decode(inp.q, inp.blocks, inp.scales, inp.cache_lengths, inp.lookup_table, inp.scales_lookup_table,
                  inp.max_prompt_length, inp.max_cache_length, inp.layer_idx, inp.softmax_scale, **kw)


def gather_dequant(blocks, scales, cache_lengths, lookup_table, scales_lookup_table, batch: int,
                   max_prompt_length: int, max_cache_length: int, layer_idx: int, max_keys: Optional[int] = None,
                   out_k=None, stream=None):
    """mla_gather_dequant_bf16: bf16 [B, max_keys, 576] of every stored key (rows past n_b untouched)."""
    _check_cache(blocks, scales, cache_lengths, lookup_table, scales_lookup_table, batch)
    if max_keys is None:
        max_keys = max_cache_length + max_prompt_length
    _expect("out_k", out_k, (torch.bfloat16,), ndim=3, last=576, optional=True)
    if out_k is not None and tuple(out_k.shape) != (batch, max_keys, 576):
        raise ValueError(f"out_k must be {(batch, max_keys, 576)} (got {tuple(out_k.shape)})")
    _same_device(blocks, scales, cache_lengths, lookup_table, scales_lookup_table, out_k)
    lib = load()
    if out_k is None:
        out_k = torch.zeros((batch, max_keys, 576), dtype=torch.bfloat16, device=blocks.device)
    shp = paged_shape(batch, 1, blocks, scales, lookup_table)
    st = lib.mla_gather_dequant_bf16(_ptr(blocks), _ptr(scales), _ptr(cache_lengths), _ptr(lookup_table),
                                     _ptr(scales_lookup_table), int(max_prompt_length), int(max_cache_length),
                                     int(layer_idx), ctypes.byref(shp), _ptr(out_k), int(max_keys), _stream(stream))
    _check(st)
    return out_k


# ---------------------------------------------------------------- cache operators
# These calls are short, so the binding's own time counts: a tensor that is as expected passes one
# compound test, and only one that is not goes through _expect, which says what is wrong with it.
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _plain(t, dtype, ndim):
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()


def _rows(name, t, dtype, batch, cols):
    """A [batch, >= cols] tensor whose rows are contiguous (the row stride is free); returns the stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype} (got {t.dtype})")
    shape = t.shape
    if len(shape) != 2 or shape[0] != batch or shape[1] < cols:
        raise ValueError(f"{name} must be [{batch}, >= {cols}] (got shape {tuple(shape)})")
    n = shape[1]
    step, inner = t.stride()
    if inner != 1 and n > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if batch <= 1:
        return n
    if step < n:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return step


def _apart(name, t, tstep, other, u, ustep, batch, cols):
    """Refuses two fp32 row buffers that overlap in part (columns of one wide buffer may interleave)."""
    a, b = t.data_ptr(), u.data_ptr()
    if a + 4 * ((batch - 1) * tstep + cols) <= b or b + 4 * ((batch - 1) * ustep + cols) <= a:
        return
    if (a != b or tstep != ustep) and not (tstep == ustep and 4 * cols <= (b - a) % (4 * tstep) <= 4 * (tstep - cols)):
        raise ValueError(f"{name} must be {other} itself or not overlap it")


def _one_device(first, *rest):
    """Index of the one CUDA device that all tensors are on."""
    d = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != d:
            d = -1
    if d < 0:
        _same_device(first, *rest)
        raise ValueError("all tensors must be CUDA tensors")
    return d


def _raw_stream(stream, device):
    """Stream handle: the device's current stream unless `stream` is given."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _run(device, fn, *args):
    """One library call, on the tensors' device whatever the current one."""
    if torch._C._cuda_getDevice() == device:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st != MLA_OK:
        _check(st)


def _adr(t):
    return None if t is None else t.data_ptr()


def _allocating_on(stream, device):
    """Allocations for a call belong to the stream that it runs on."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                             else torch.cuda.ExternalStream(_raw_stream(stream, device), torch.device("cuda", device)))


def _scratch(n, like, device, stream):
    if not n:
        return None
    if stream is None:
        return torch.empty(n, dtype=_U8, device=like.device)
    with _allocating_on(stream, device):
        return torch.empty(n, dtype=_U8, device=like.device)


def _check_tables(cache_lengths, lookup_table, scales_lookup_table, batch):
    if not (_plain(cache_lengths, _I32, 1) and _plain(lookup_table, _I32, 2)):
        _expect("cache_lengths", cache_lengths, _U32, ndim=1)
        _expect("lookup_table", lookup_table, _U32, ndim=2)
    if cache_lengths.shape[0] != batch or lookup_table.shape[0] != batch:
        raise ValueError(f"cache_lengths and lookup_table must have {batch} rows (one per request)")
    _check_scale_table(lookup_table, scales_lookup_table)


def _check_scale_table(lookup_table, scales_lookup_table):
    if scales_lookup_table is not None:
        _expect("scales_lookup_table", scales_lookup_table, _U32, ndim=2)
        if scales_lookup_table.shape != lookup_table.shape:
            raise ValueError("scales_lookup_table must have the shape of lookup_table")


@functools.lru_cache(maxsize=1024)      # a function of the sizes alone, only read by the library
def _shape_record(*sizes):
    return PagedShape(*sizes)


def _cache_shape(blocks, scales, scales_lookup_table, batch, heads, v_dim, lookup_table):
    """Shape record of a cache whose scales, where it has them, hold each token's in the last dim."""
    NB, KVD, NL, P, NKV, D = blocks.shape
    NSB, g = NB, 1
    if scales is not None:
        NSB, sKVD, sNL, sP, sNKV, g = scales.shape
        if sKVD != KVD or sNL != NL or sP != P or sNKV != NKV:
            raise ValueError("scales must match blocks in kv_dim, num_layers, page_size and num_heads")
        if NSB != NB and scales_lookup_table is None:
            raise ValueError("without a scales_lookup_table, scales must have as many blocks as blocks")
    return _shape_record(batch, heads, D, v_dim, NB, KVD, NL, P, NKV, NSB, g, lookup_table.shape[1])


# ctypes wraps a number that its 32-bit argument does not hold: (n + _HALF) >> 32 is 0 for those it does.  (What is
# left of the range is the library's to check.)
_HALF, _MOST = 0x80000000, 0x7FFFFFFF


def _too_wide(**numbers):
    for name, n in numbers.items():
        if (n + _HALF) >> 32:
            raise ValueError(f"{name} does not fit 32 bits (got {n})")


def _token_count(max_prompt_length, tokens):
    if max_prompt_length != tokens:
        raise ValueError(f"max_prompt_length must be q's number of tokens, {tokens} (got {max_prompt_length})")


def accumulate_weights(q, lse, blocks, scales, cache_lengths, lookup_table, scales_lookup_table,
                       max_prompt_length: int, max_cache_length: int, layer_idx: int, softmax_scale: float,
                       scores=None, out=None, stream=None, workspace=None):
    """mla_accumulate_weights_fp8: add to every cached key the softmax weight it received in this step.

    q bf16 [B, T, H, 576] and the cache as for decode(), lse fp32 [B, T, H] as decode() returned it.
    scores fp32 [B, >= max_cache_length + T] (rows may be strided), or None for all zero; entries of the
    step's own tokens start at 0.  Writes out (default: scores itself, or a new tensor) and returns it;
    entries past a request's keys are left as they were.  workspace: a uint8 tensor of
    accumulate_workspace_bytes(B, T, H) bytes; by default one is taken from torch's allocator for the call.
    """
    if not (_plain(q, _BF16, 4) and _plain(lse, _F32, 3)) or q.shape[3] != 576:
        _expect("q", q, (_BF16,), ndim=4, last=576)
        _expect("lse", lse, (_F32,), ndim=3)
    B, T, H, _ = q.shape
    if lse.shape != (B, T, H):
        raise ValueError(f"lse must be {(B, T, H)} (got {tuple(lse.shape)})")
    if not (_plain(blocks, _U8, 6) and _plain(scales, _F32, 6)):
        _expect("blocks", blocks, _CODES, ndim=6)
        _expect("scales", scales, (_F32,), ndim=6)
    _check_tables(cache_lengths, lookup_table, scales_lookup_table, B)
    _token_count(max_prompt_length, T)
    max_cache_length, layer_idx = int(max_cache_length), int(layer_idx)
    if (max_cache_length + _HALF | layer_idx + _HALF) >> 32:
        _too_wide(max_cache_length=max_cache_length, layer_idx=layer_idx)
    shp = _cache_shape(blocks, scales, scales_lookup_table, B, H, 512, lookup_table)
    need = max_cache_length + T
    sstep = 0 if scores is None else _rows("scores", scores, _F32, B, need)
    ostep = 0 if out is None else _rows("out", out, _F32, B, need)
    if workspace is not None:
        _expect("workspace", workspace, (_U8,), ndim=1)
    dev = _one_device(q, lse, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, scores, out, workspace)
    lib = load()
    if out is None:
        if scores is None:
            with _allocating_on(stream, dev):
                out = torch.zeros((B, need), dtype=_F32, device=q.device)
            ostep = need
        else:
            out, ostep = scores, sstep
    elif scores is not None and out is not scores:
        _apart("out", out, ostep, "scores", scores, sstep, B, need)
    if B == 0:
        return out
    if workspace is None:
        workspace = _scratch(accumulate_workspace_bytes(B, T, H), q, dev, stream)
    _run(dev, lib.mla_accumulate_weights_fp8, q.data_ptr(), lse.data_ptr(), blocks.data_ptr(), scales.data_ptr(),
         cache_lengths.data_ptr(), lookup_table.data_ptr(), _adr(scales_lookup_table), T, max_cache_length, layer_idx,
         float(softmax_scale), ctypes.byref(shp), _adr(scores), sstep, out.data_ptr(), ostep, _adr(workspace),
         0 if workspace is None else workspace.numel(), _raw_stream(stream, dev))
    return out


@functools.lru_cache(maxsize=1024)      # a function of the sizes alone
def accumulate_workspace_bytes(batch: int, max_prompt_length: int, num_q_heads: int) -> int:
    """Bytes of workspace that accumulate_weights needs."""
    if (batch + _HALF | max_prompt_length + _HALF | num_q_heads + _HALF) >> 32:
        _too_wide(batch=batch, max_prompt_length=max_prompt_length, num_q_heads=num_q_heads)
    n, shp = ctypes.c_uint64(0), PagedShape(batch, num_q_heads)
    _check(load().mla_accumulate_workspace_bytes(max_prompt_length, ctypes.byref(shp), ctypes.byref(n)))
    return n.value


def select_keys(scores, lengths, max_length: int, budget: int, num_recent: int = 0, num_sink: int = 0, kept=None,
                kept_lengths=None, stream=None):
    """mla_select_keys: the keys each request keeps, as (kept int32 [B, budget], kept_lengths int32 [B]).

    scores fp32 [B, >= max_length] (rows may be strided), lengths int32 [B] keys held, max_length >= all of
    them.  A request over the budget keeps its first num_sink keys, its last num_recent keys and the
    keys with the largest scores between (ties to the lowest index); kept[b, :kept_lengths[b]] ascends
    and later entries are left as they were (0 in a new tensor).  kept_lengths may be lengths itself.
    """
    if not _plain(lengths, _I32, 1):
        _expect("lengths", lengths, _U32, ndim=1)
    B = lengths.shape[0]
    max_length, budget, num_recent, num_sink = int(max_length), int(budget), int(num_recent), int(num_sink)
    if (max_length + _HALF | budget + _HALF | num_recent + _HALF | num_sink + _HALF) >> 32:
        _too_wide(max_length=max_length, budget=budget, num_recent=num_recent, num_sink=num_sink)
    sstep = _rows("scores", scores, _F32, B, max_length)
    kstep = 0 if kept is None else _rows("kept", kept, _I32, B, min(budget, max_length))
    if kept_lengths is not None and (not _plain(kept_lengths, _I32, 1) or kept_lengths.shape[0] != B):
        raise ValueError(f"kept_lengths must be a contiguous int32 tensor of {B} entries")
    dev = _one_device(scores, lengths, kept, kept_lengths)
    lib = load()
    if kept is None or kept_lengths is None:
        with _allocating_on(stream, dev):
            if kept is None:
                kstep = max(budget, 1)
                kept = torch.zeros((B, kstep), dtype=_I32, device=scores.device)
            if kept_lengths is None:
                kept_lengths = torch.empty(B, dtype=_I32, device=scores.device)
    if B == 0:
        return kept, kept_lengths
    _run(dev, lib.mla_select_keys, scores.data_ptr(), sstep, lengths.data_ptr(), B, max_length, budget,
         num_recent, num_sink, kept.data_ptr(), kstep, kept_lengths.data_ptr(), _raw_stream(stream, dev))
    return kept, kept_lengths


def compact_cache(kept, kept_lengths, lookup_table, scales_lookup_table, layer_idx: int, blocks, scales, scores=None,
                  stream=None):
    """mla_compact_paged: move row kept[b, j] of every request to row j, in place, in one layer of blocks
    (uint8 / e4m3 or bf16, 6-D), scales (fp32, 6-D, or None) and scores (fp32 [B, n], or None).

    kept int32 [B, n] and kept_lengths int32 [B] as select_keys() returns them (strictly ascending).
    Returns (blocks, scales, scores)."""
    if not _plain(blocks, _U8, 6):
        _expect("blocks", blocks, _CODES + (_BF16,), ndim=6)
    if not _plain(scales, _F32, 6):
        _expect("scales", scales, (_F32,), ndim=6, optional=True)
    if not (_plain(kept_lengths, _I32, 1) and _plain(lookup_table, _I32, 2)):
        _expect("kept_lengths", kept_lengths, (_I32,), ndim=1)
        _expect("lookup_table", lookup_table, _U32, ndim=2)
    B = kept_lengths.shape[0]
    if lookup_table.shape[0] != B:
        raise ValueError(f"lookup_table must have {B} rows (one per request)")
    _check_scale_table(lookup_table, scales_lookup_table)
    kstep = _rows("kept", kept, _I32, B, 1)
    layer_idx = int(layer_idx)
    if (layer_idx + _HALF) >> 32:
        _too_wide(layer_idx=layer_idx)
    shp = _cache_shape(blocks, scales, scales_lookup_table, B, 0, 0, lookup_table)
    sstep = 0 if scores is None else _rows("scores", scores, _F32, B, 1)
    dev = _one_device(kept, kept_lengths, lookup_table, scales_lookup_table, blocks, scales, scores)
    if B == 0:
        return blocks, scales, scores
    _run(dev, load().mla_compact_paged, kept.data_ptr(), kstep, min(kept.shape[1], _MOST), kept_lengths.data_ptr(),
         lookup_table.data_ptr(), _adr(scales_lookup_table), layer_idx, blocks.element_size(), ctypes.byref(shp),
         blocks.data_ptr(), _adr(scales), _adr(scores), sstep, 0 if scores is None else min(scores.shape[1], _MOST),
         _raw_stream(stream, dev))
    return blocks, scales, scores


def _check_mha(blocks, scales, cache_lengths, lookup_table, scales_lookup_table, batch, heads, kv_heads, dim):
    """Shape record of the 6-D multi-head cache (keys in kv plane 0, values in plane 1)."""
    bf16 = _plain(blocks, _BF16, 6)
    if not bf16 and not _plain(blocks, _U8, 6):
        _expect("blocks", blocks, _CODES + (_BF16,), ndim=6)
    NB, KVD, NL, P, NKV, D = blocks.shape
    if D != dim or (kv_heads and NKV != kv_heads):
        raise ValueError(f"blocks hold {NKV} heads of {D} values, expected {kv_heads or NKV} of {dim}")
    NSB = NB
    if bf16:
        if scales is not None:
            raise ValueError("a bf16 cache takes no scales")
    else:
        if not _plain(scales, _F32, 6):
            _expect("scales", scales, (_F32,), ndim=6)
        if scales.shape[1:] != (KVD, NL, P, NKV, 1):
            raise ValueError(f"scales must be [n, {KVD}, {NL}, {P}, {NKV}, 1] (got {tuple(scales.shape)})")
        NSB = scales.shape[0]
        if scales_lookup_table is None and NSB != NB:
            raise ValueError("without a scales_lookup_table, scales must have as many blocks as blocks")
    _check_tables(cache_lengths, lookup_table, scales_lookup_table, batch)
    return _shape_record(batch, heads, D, D, NB, KVD, NL, P, NKV, NSB, 1, lookup_table.shape[1])


def mha_kv_store(k, v, cache_lengths, lookup_table, scales_lookup_table, layer_idx: int, blocks, scales=None, stream=None):
    """mla_mha_kv_store: write the step's keys and values, bf16 [B, T, HKV, D] each, in place into blocks
    (bf16, or uint8 / e4m3 with scales fp32 [.., HKV, 1]) [NB, kv_dim, L, P, HKV, D] at positions
    cache_lengths[b] + i."""
    if not (_plain(k, _BF16, 4) and _plain(v, _BF16, 4)):
        _expect("k", k, (_BF16,), ndim=4)
        _expect("v", v, (_BF16,), ndim=4)
    B, T, HKV, D = k.shape
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape")
    layer_idx = int(layer_idx)
    if (layer_idx + _HALF) >> 32:
        _too_wide(layer_idx=layer_idx)
    shp = _check_mha(blocks, scales, cache_lengths, lookup_table, scales_lookup_table, B, 0, HKV, D)
    dev = _one_device(k, v, blocks, scales, cache_lengths, lookup_table, scales_lookup_table)
    if B == 0 or T == 0:
        return blocks, scales
    _run(dev, load().mla_mha_kv_store, k.data_ptr(), v.data_ptr(), cache_lengths.data_ptr(), lookup_table.data_ptr(),
         _adr(scales_lookup_table), T, layer_idx, blocks.element_size(), ctypes.byref(shp), blocks.data_ptr(), _adr(scales),
         _raw_stream(stream, dev))
    return blocks, scales


def mha_decode(q, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, max_prompt_length: int,
               max_cache_length: int, layer_idx: int, softmax_scale: float, out=None, lse=None, stream=None,
               want_lse: bool = True, workspace=None):
    """mla_mha_decode_paged: grouped-query decode attention over the multi-head cache.

    q bf16 [B, T, H, D], D 64 or 128; blocks [NB, kv_dim >= 2, L, P, HKV, D] bf16, or uint8 / e4m3 with
    scales fp32 [NSB, kv_dim, L, P, HKV, 1]; H a multiple of HKV.  workspace: a uint8 tensor of
    mha_decode_workspace_bytes(...) bytes; by default one is taken from torch's allocator for the call.
    Returns (out bf16 [B, T, H, D], lse fp32 [B, T, H] or None).
    """
    if not _plain(q, _BF16, 4):
        _expect("q", q, (_BF16,), ndim=4)
    B, T, H, D = q.shape
    _token_count(max_prompt_length, T)
    max_cache_length, layer_idx = int(max_cache_length), int(layer_idx)
    if (max_cache_length + _HALF | layer_idx + _HALF) >> 32:
        _too_wide(max_cache_length=max_cache_length, layer_idx=layer_idx)
    shp = _check_mha(blocks, scales, cache_lengths, lookup_table, scales_lookup_table, B, H, 0, D)
    if out is not None and (not _plain(out, _BF16, 4) or out.shape != q.shape):
        raise ValueError(f"out must be a contiguous bf16 tensor of shape {tuple(q.shape)}")
    if lse is not None and (not _plain(lse, _F32, 3) or lse.shape != (B, T, H)):
        raise ValueError(f"lse must be a contiguous fp32 tensor of shape {(B, T, H)}")
    if workspace is not None:
        _expect("workspace", workspace, (_U8,), ndim=1)
    dev = _one_device(q, blocks, scales, cache_lengths, lookup_table, scales_lookup_table, out, lse, workspace)
    lib = load()
    if out is None or (lse is None and want_lse):
        with _allocating_on(stream, dev):
            if out is None:
                out = torch.empty_like(q)
            if lse is None and want_lse:
                lse = torch.empty((B, T, H), dtype=_F32, device=q.device)
    if B == 0:
        return out, lse
    if workspace is None:
        workspace = _scratch(_mha_workspace(dev, T, max_cache_length, blocks.element_size(), B, H, D, shp.num_kv_heads,
                                            shp.page_size, shp.max_pages), q, dev, stream)
    _run(dev, lib.mla_mha_decode_paged, q.data_ptr(), blocks.data_ptr(), _adr(scales), cache_lengths.data_ptr(),
         lookup_table.data_ptr(), _adr(scales_lookup_table), T, max_cache_length, layer_idx, float(softmax_scale),
         blocks.element_size(), ctypes.byref(shp), out.data_ptr(), _adr(lse), _adr(workspace),
         0 if workspace is None else workspace.numel(), _raw_stream(stream, dev))
    return out, lse


@functools.lru_cache(maxsize=4096)      # a function of the device and the sizes alone
def _mha_workspace(device, T, max_cache_length, element_bytes, B, H, D, HKV, P, max_pages):
    shp = PagedShape(B, H, D, D, 1, 2, 1, P, HKV, 1, 1, max_pages)
    n = ctypes.c_uint64(0)
    _run(device, load().mla_mha_decode_workspace_bytes, T, max_cache_length, element_bytes, ctypes.byref(shp), ctypes.byref(n))
    return n.value


def mha_decode_workspace_bytes(q, blocks, lookup_table, max_cache_length: int) -> int:
    """Bytes of workspace that mha_decode needs for these tensors (0 for short caches)."""
    B, T, H, D = q.shape
    max_cache_length = int(max_cache_length)
    if (max_cache_length + _HALF) >> 32:
        _too_wide(max_cache_length=max_cache_length)
    return _mha_workspace(q.get_device(), T, max_cache_length, blocks.element_size(), B, H, D, blocks.shape[4],
                          blocks.shape[3], lookup_table.shape[1])


def set_num_clusters(n: int):
    _check(load().mla_set_num_clusters(int(n)))


def set_wait_limit_ns(ns: int):
    """Bound of every wait inside the decode kernel (default 2 s)."""
    _check(load().mla_set_wait_limit_ns(int(ns)))


def withhold_arrival_once():
    """Test hook: the next decode call withholds one barrier arrival, so a bounded wait runs out."""
    _check(load().mla_debug_withhold_arrival_once())


def get_num_clusters() -> int:
    return int(load().mla_get_num_clusters())


def device_status(stream=None) -> int:
    """Synchronise, then return and clear the sticky device status (0 = OK)."""
    return int(load().mla_get_device_status(_stream(stream)))


def release_workspace():
    _check(load().mla_release_workspace())


def set_timing_events(before=None, after=None):
    """Record torch.cuda.Event `before`/`after` around every later decode-kernel launch (None, None stops)."""
    if before is not None and (before.cuda_event == 0 or after.cuda_event == 0):
        raise ValueError("record each event once before handing it to the library (torch creates it lazily)")
    b = None if before is None else ctypes.c_void_p(before.cuda_event)
    a = None if after is None else ctypes.c_void_p(after.cuda_event)
    _check(load().mla_set_timing_events(b, a))


def version() -> str:
    return load().mla_version().decode()
