"""MLA over the 576-wide latent KV cache on GB300 (sm_103a): Python binding of libmla.

The functions here only marshal torch tensors (device memory, strides, the current CUDA
stream) into the C ABI of ``include/mla.h``; every step of the computation runs in the
library's CUDA kernels.  There is no fallback: if ``libmla.so`` is missing or fails to load,
importing the binding raises.

Entry points (same names as the C ABI, without the ``mla_`` prefix):

  q_concat_cache_insert  decode epilogue: mqa_q = [ql_nope | q_pe] (+ GPT-J RoPE), latent
                         insert into a bf16 / plain fp8 / fp8_ds_mla / mxfp4 paged cache
  key_concat_cache_insert   prefill epilogue (bf16 / fp8_ds_mla / mxfp4 cache): full key
                         [k_nope | rope(k_pe)], q RoPE in place, latent insert
  qkv_quant_cache_fp8_insert  prefill epilogue (plain fp8 cache): E4M3 q / k / v with their
                         own scales, latent insert with the cache scale
  sparse_fwd             sparse CSR forward over 656-byte fp8_ds_mla records
  paged_decode           paged decode / spec-verify (split-K + LSE merge)
  absorb_q               BMM1: q_nope . W_UK_T per head -> ql_nope (latent query)
  v_up_proj              latent output . W_UV per head (+ sigmoid output gate)
  gather_context         chunked-context gather of paged entries (bf16 values or stored bytes)
  merge_attn_states      prefix / suffix merge of partial attentions by their LSEs
  gather_dequant         paged entries -> exact fp32 values (test aid)

Around a step:

  plan_step              blocks, slots, positions and row offsets of a step from the requests' lengths
  rope                   rotary positions of queries and keys: any width, both layouts, inverse
  rope_table             the table of cosines and sines, plain or scaled for long contexts

The selector in front of sparse attention (an index key of 128 values per cached token):

  index_q_cache_insert   index queries and keys rotated, quantised, keys inserted into the
                         paged index cache (bf16, or E4M3 with a scale per key)
  index_gather           cached index keys read back as bf16
  index_scores           weighted relu scores of every visible token, or of blocks of tokens
  index_select           the topk best blocks of every row (and their cache slots)
  selected_decode        decode over the selected pages of a bf16 / fp8 / fp8_ds_mla / mxfp4 cache

Every tensor argument is checked here before the call (CUDA device, dtype, rank, unit
innermost stride; index tensors contiguous), so that a wrong tensor raises instead of being
read with the wrong layout.  Sparse indices may be int32 or int64.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import warnings

import torch

from . import build as _build

CACHE_BF16, CACHE_FP8, CACHE_FP8_DS_MLA, CACHE_MXFP4 = 0, 1, 2, 3
ENTRY_BYTES = {CACHE_BF16: 1152, CACHE_FP8: 576, CACHE_FP8_DS_MLA: 656, CACHE_MXFP4: 400}
_FMT_NAMES = {"bf16": CACHE_BF16, "auto": CACHE_BF16, "fp8": CACHE_FP8, "fp8_ds_mla": CACHE_FP8_DS_MLA, "mxfp4": CACHE_MXFP4}

_lib = None


class MLAError(RuntimeError):
    pass


def library_path() -> str:
    return _build.LIB


def lib():
    """Load libmla.so (build it first with ``build.build()``).  Raises if it is missing."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise ImportError(f"libmla.so not built ({path}); run mla_latent_cache_attention_gb300.build.build()")
        L = ctypes.CDLL(path)
        vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        L.mla_last_error.restype = ctypes.c_char_p
        L.mla_version.restype = ctypes.c_char_p
        L.mla_read_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
        L.mla_q_concat_cache_insert.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, vp, vp, i32,
                                                i64, i64, i64, i32, vp, vp, vp, vp, vp, i64, i32, i32, vp]
        L.mla_sparse_fwd.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, i64, f32, i32, vp, i64, i64, vp,
                                     i32, i32, vp]
        L.mla_paged_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.mla_paged_decode_workspace_size.restype = sz
        L.mla_paged_decode_workspace_size_for.argtypes = [i32, i32, i32, i32, i32, i32]
        L.mla_paged_decode_workspace_size_for.restype = sz
        L.mla_paged_decode.argtypes = [vp, i64, i64, vp, i32, i64, i64, i64, i32, vp, i64, vp, i32, i32, i32,
                                       i32, f32, f32, f32, vp, i64, i64, vp, vp, sz, vp]
        L.mla_paged_decode_noalloc.argtypes = [vp, i64, i64, vp, i32, i64, i64, i64, i32, vp, i64, vp, i32, i32,
                                               i32, i32, f32, f32, f32, vp, i64, i64, vp, vp]
        L.mla_paged_decode_noalloc.restype = ctypes.c_int
        L.mla_profile_attention_events.argtypes = [vp, vp]
        L.mla_profile_attention_events.restype = None
        L.mla_gather_dequant.argtypes = [vp, i32, i64, i64, i64, i32, vp, i64, vp, vp]
        L.mla_sparse_fwd_staged.argtypes = L.mla_sparse_fwd.argtypes
        L.mla_sparse_fwd_ext_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.mla_sparse_fwd_ext_workspace_size.restype = sz
        L.mla_sparse_fwd_ext.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, i64, vp, i64, i64, vp, vp, i64, vp, i32,
                                         f32, i32, vp, i64, i64, vp, i32, i32, vp, sz, vp]
        L.mla_absorb_q.argtypes = [vp, i64, i64, vp, vp, i64, i64, i32, i32, i32, vp]
        L.mla_v_up_proj.argtypes = [vp, i64, i64, vp, vp, i64, vp, i64, i64, i32, i32, i32, vp]
        L.mla_gather_context.argtypes = [vp, i32, i64, i64, i64, i32, vp, i64, vp, vp, i32, i64, i32, f32, vp, i64, vp]
        L.mla_merge_attn_states.argtypes = [vp, i64, i64, vp, vp, i64, i64, vp, vp, i64, i64, vp, i32, i32, i32, vp]
        L.mla_key_concat_cache_insert.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, vp, vp, i32, i64, i64,
                                                  i64, i32, vp, vp, vp, i64, i32, i32, i32, vp]
        L.mla_qkv_quant_cache_fp8_insert.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, vp, i64, i64, vp,
                                                     vp, vp, vp, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, i64,
                                                     i32, i32, i32, i32, vp]
        L.mla_index_q_cache_insert.argtypes = [vp, i64, i64, vp, i64, vp, i64, f32, vp, vp, vp, i32, i64, i64, i64, vp,
                                               i64, i32, vp, vp, vp, i64, i32, i32, vp]
        L.mla_index_gather.argtypes = [vp, i32, i64, i64, i64, vp, i64, i32, vp, i64, i64, vp, vp, i32, i64, vp, i64, vp]
        L.mla_index_scores.argtypes = [vp, i64, i64, vp, i64, vp, i32, i64, i64, i64, vp, i64, i32, vp, i64, i64, vp, vp,
                                       i32, i32, i32, i32, vp, i64, i64, vp]
        L.mla_index_select.argtypes = [vp, i64, i64, vp, vp, i32, i32, i32, i32, i32, i32, vp, i64, vp, i64, vp, i64,
                                       i64, i32, i64, vp]
        for f in (L.mla_selected_decode_workspace_size, L.mla_selected_decode_workspace_bound):
            f.argtypes = [i32, i32, i32, i32, i32, i32]
            f.restype = sz
        L.mla_selected_decode.argtypes = [vp, i64, i64, vp, i32, i64, i64, i64, i32, vp, i64, i64, vp, vp, vp, i64, i32,
                                          i32, i32, i32, f32, f32, f32, vp, i64, i64, vp, vp, sz, vp]
        f64 = ctypes.c_double
        L.mla_rope.argtypes = [i32, vp, i64, i64, vp, i64, i64, i32, i32, i32, vp, i64, i64, vp, i64, i64, i32, i32, i32, vp, vp, i64,
                               i32, i32, i32, i32, vp]
        L.mla_rope_table.argtypes = [vp, i64, i32, f64, i32, f64, i64, f64, f64, f64, vp]
        L.mla_plan_step.argtypes = [vp, vp, vp, vp, i64, i32, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp]
        L.mla_debug_stall_next_decode.argtypes = [i32]
        L.mla_debug_stall_next_decode.restype = None
        L.mla_debug_ds_cluster.argtypes = [i32]
        L.mla_debug_ds_cluster.restype = None
        for f in ("mla_q_concat_cache_insert", "mla_sparse_fwd", "mla_sparse_fwd_staged", "mla_paged_decode",
                  "mla_gather_dequant", "mla_key_concat_cache_insert", "mla_qkv_quant_cache_fp8_insert",
                  "mla_gather_context", "mla_merge_attn_states", "mla_sparse_fwd_ext", "mla_absorb_q",
                  "mla_v_up_proj", "mla_index_q_cache_insert", "mla_index_gather", "mla_index_scores",
                  "mla_index_select", "mla_selected_decode", "mla_rope", "mla_rope_table", "mla_plan_step"):
            getattr(L, f).restype = ctypes.c_int
        L.mla_read_device_errors.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int):
    if rc != 0:
        raise MLAError(f"libmla error {rc}: {lib().mla_last_error().decode()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        return _FMT_NAMES[fmt]
    return int(fmt)


_BYTE_TYPES = (torch.uint8, torch.int8)
_INT32_MAX = 2 ** 31 - 1


def _need(t, name, dtypes, device, *, ndim=None, contiguous=False, inner=True):
    """Marshalling check of one tensor argument: a CUDA tensor on `device` of one of `dtypes`,
    with `ndim` dimensions, unit innermost stride (inner) or fully contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}; expected one of {', '.join(str(d) for d in dtypes)}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if inner and t.dim() > 0 and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have a unit innermost stride")
    return t


def _cuda_device(t) -> torch.device:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    return t.device


def _index_i32(t, name, device, lo, hi):
    """int32 index tensor for the C ABI.  int64 input (accepted by the sparse forward's
    interface) is narrowed on the device after clamping to [lo, hi], so an id outside int32
    keeps its meaning: below lo stays masked / flagged, above hi stays out of range."""
    _need(t, name, (torch.int32, torch.int64), device, ndim=1, contiguous=True)
    if t.dtype == torch.int64:
        t = t.clamp(lo, hi).to(torch.int32)
    return t


def _cache_geometry(kv_cache: torch.Tensor, fmt=None):
    """[num_blocks, block_size, entry_stride] view of a paged cache (any 1- or 2-byte dtype)."""
    es = kv_cache.element_size()
    if kv_cache.dim() == 4 and kv_cache.shape[1] == 1:      # [nb, 1, bs, entry] (a head axis of size 1)
        kv_cache = kv_cache.squeeze(1)
    if kv_cache.dim() != 3 or kv_cache.stride(2) != 1:
        raise ValueError("kv_cache must be [num_blocks, block_size, entry] with a unit innermost stride")
    if fmt == CACHE_MXFP4 and (es != 1 or kv_cache.shape[2] < ENTRY_BYTES[fmt]):
        raise ValueError(f"mxfp4 records are {ENTRY_BYTES[fmt]} bytes of uint8, kv_cache has {kv_cache.shape[2]} of {kv_cache.dtype}")
    return kv_cache.shape[0], kv_cache.stride(0) * es, kv_cache.stride(1) * es, kv_cache.shape[1]


def version() -> str:
    return lib().mla_version().decode()


def profile_attention_events(start=None, stop=None):
    """Bracket later attention-kernel launches of this thread with two torch.cuda.Events
    (recorded on the call's stream); ``None, None`` turns it off."""
    h = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event)
    lib().mla_profile_attention_events(h(start), h(stop))


def read_device_errors(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device error word."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else torch.device(device).index)
    v = ctypes.c_uint32(0)
    with torch.cuda.device(dev):
        _check(lib().mla_read_device_errors(ctypes.byref(v),
                                            ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)))
    return int(v.value)


def q_concat_cache_insert(ql_nope, q_pe, kv_c_normed, k_pe, kv_cache, slot_mapping, *, fmt,
                          q_scale_inv=None, cache_scale_inv=None, positions=None, cos_sin_cache=None,
                          mqa_q=None):
    """Decode epilogue.  Returns mqa_q [B, H, 576] (bf16, or uint8 E4M3 codes for fp8);
    writes kv_cache in place."""
    fmt = _fmt(fmt)
    done = (_step or _plain_step()).q_concat(ql_nope, q_pe, kv_c_normed, k_pe, kv_cache, slot_mapping, fmt, q_scale_inv, cache_scale_inv,
                                             positions, cos_sin_cache, mqa_q)
    if done is not None:
        return done
    dev = _cuda_device(ql_nope)
    bf = (torch.bfloat16,)
    _need(ql_nope, "ql_nope", bf, dev, ndim=3)
    _need(q_pe, "q_pe", bf, dev, ndim=3)
    _need(kv_c_normed, "kv_c_normed", bf, dev, ndim=2)
    k_pe = _need(k_pe, "k_pe", bf, dev).reshape(k_pe.shape[0], -1)
    _need(slot_mapping, "slot_mapping", (torch.int64,), dev, ndim=1, contiguous=True)
    if positions is not None:
        _need(positions, "positions", (torch.int64,), dev, ndim=1, contiguous=True)
    if cos_sin_cache is not None:
        _need(cos_sin_cache, "cos_sin_cache", (torch.float32,), dev, ndim=2, contiguous=True)
    for n, t in (("q_scale_inv", q_scale_inv), ("cache_scale_inv", cache_scale_inv)):
        if t is not None:
            _need(t, n, (torch.float32,), dev)
    B, H, _ = ql_nope.shape
    if mqa_q is None:
        dt = torch.uint8 if fmt == CACHE_FP8 else torch.bfloat16
        mqa_q = torch.empty((B, H, 576), dtype=dt, device=dev)
    _need(mqa_q, "mqa_q", _BYTE_TYPES if fmt == CACHE_FP8 else bf, dev, ndim=3, contiguous=True)
    _need(kv_cache, "kv_cache", _BYTE_TYPES + bf, dev)
    nb, bstride, estride, bs = _cache_geometry(kv_cache, fmt)
    max_pos = 0 if cos_sin_cache is None else cos_sin_cache.shape[0]
    with torch.cuda.device(dev):
        _check(lib().mla_q_concat_cache_insert(
            _ptr(ql_nope), ql_nope.stride(0), ql_nope.stride(1), _ptr(q_pe), q_pe.stride(0), q_pe.stride(1),
            _ptr(kv_c_normed), kv_c_normed.stride(0), _ptr(k_pe), k_pe.stride(0), _ptr(mqa_q), _ptr(kv_cache),
            fmt, nb, bstride, estride, bs, _ptr(slot_mapping), _ptr(q_scale_inv), _ptr(cache_scale_inv),
            _ptr(positions), _ptr(cos_sin_cache), max_pos, B, H, _stream(ql_nope)))
    return mqa_q


def _prefill_common(q, k_nope, k_pe, kv_c_normed, slot_mapping, positions, cos_sin_cache):
    dev = _cuda_device(q)
    bf = (torch.bfloat16,)
    _need(q, "q", bf, dev, ndim=3)
    _need(k_nope, "k_nope", bf, dev, ndim=3)
    k_pe = _need(k_pe, "k_pe", bf, dev).reshape(k_pe.shape[0], -1)
    _need(kv_c_normed, "kv_c_normed", bf, dev, ndim=2)
    _need(slot_mapping, "slot_mapping", (torch.int64,), dev, ndim=1, contiguous=True)
    if positions is not None:
        _need(positions, "positions", (torch.int64,), dev, ndim=1, contiguous=True)
    if cos_sin_cache is not None:
        _need(cos_sin_cache, "cos_sin_cache", (torch.float32,), dev, ndim=2, contiguous=True)
    Tp, H, dn = k_nope.shape
    if q.shape != (Tp, H, dn + 64):
        raise ValueError(f"q must be [Tp, H, dn + 64] = {(Tp, H, dn + 64)}, got {tuple(q.shape)}")
    return dev, k_pe, Tp, H, dn


def key_concat_cache_insert(q, k_nope, k_pe, kv_c_normed, kv_cache, slot_mapping, *, fmt, positions=None,
                            cos_sin_cache=None, k_out=None):
    """Prefill epilogue for the bf16 / fp8_ds_mla / mxfp4 cache.  Rotates the rope part of q in place
    (when positions are given), writes kv_cache in place and returns k_out [Tp, H, dn + 64]."""
    fmt = _fmt(fmt)
    done = (_step or _plain_step()).key_concat(q, k_nope, k_pe, kv_c_normed, kv_cache, slot_mapping, fmt, positions, cos_sin_cache, k_out)
    if done is not None:
        return done
    dev, k_pe, Tp, H, dn = _prefill_common(q, k_nope, k_pe, kv_c_normed, slot_mapping, positions, cos_sin_cache)
    if k_out is None:
        k_out = torch.empty((Tp, H, dn + 64), dtype=torch.bfloat16, device=dev)
    _need(k_out, "k_out", (torch.bfloat16,), dev, ndim=3, contiguous=True)
    _need(kv_cache, "kv_cache", _BYTE_TYPES + (torch.bfloat16,), dev)
    nb, bstride, estride, bs = _cache_geometry(kv_cache, fmt)
    max_pos = 0 if cos_sin_cache is None else cos_sin_cache.shape[0]
    with torch.cuda.device(dev):
        _check(lib().mla_key_concat_cache_insert(
            _ptr(q), q.stride(0), q.stride(1), _ptr(k_nope), k_nope.stride(0), k_nope.stride(1), _ptr(k_pe),
            k_pe.stride(0), _ptr(kv_c_normed), kv_c_normed.stride(0), _ptr(k_out), _ptr(kv_cache), fmt, nb, bstride,
            estride, bs, _ptr(slot_mapping), _ptr(positions), _ptr(cos_sin_cache), max_pos, Tp, H, dn, _stream(q)))
    return k_out


def qkv_quant_cache_fp8_insert(q, k_nope, k_pe, kv_c_normed, v, kv_cache, slot_mapping, *, q_scale_inv, k_scale_inv,
                               v_scale_inv, cache_scale_inv, positions=None, cos_sin_cache=None):
    """Prefill epilogue for the plain fp8 cache.  Returns (q_fp8, k_fp8, v_fp8) as uint8 E4M3
    codes; writes kv_cache in place.  The four scales are device fp32 scalars (1 / scale)."""
    dev, k_pe, Tp, H, dn = _prefill_common(q, k_nope, k_pe, kv_c_normed, slot_mapping, positions, cos_sin_cache)
    _need(v, "v", (torch.bfloat16,), dev, ndim=3)
    dv = v.shape[2]
    for n, t in (("q_scale_inv", q_scale_inv), ("k_scale_inv", k_scale_inv), ("v_scale_inv", v_scale_inv),
                 ("cache_scale_inv", cache_scale_inv)):
        _need(t, n, (torch.float32,), dev)
    _need(kv_cache, "kv_cache", _BYTE_TYPES, dev)
    q8 = torch.empty((Tp, H, dn + 64), dtype=torch.uint8, device=dev)
    k8 = torch.empty((Tp, H, dn + 64), dtype=torch.uint8, device=dev)
    v8 = torch.empty((Tp, H, dv), dtype=torch.uint8, device=dev)
    nb, bstride, estride, bs = _cache_geometry(kv_cache)
    max_pos = 0 if cos_sin_cache is None else cos_sin_cache.shape[0]
    with torch.cuda.device(dev):
        _check(lib().mla_qkv_quant_cache_fp8_insert(
            _ptr(q), q.stride(0), q.stride(1), _ptr(k_nope), k_nope.stride(0), k_nope.stride(1), _ptr(k_pe),
            k_pe.stride(0), _ptr(kv_c_normed), kv_c_normed.stride(0), _ptr(v), v.stride(0), v.stride(1), _ptr(q8),
            _ptr(k8), _ptr(v8), _ptr(kv_cache), nb, bstride, estride, bs, _ptr(slot_mapping), _ptr(q_scale_inv),
            _ptr(k_scale_inv), _ptr(v_scale_inv), _ptr(cache_scale_inv), _ptr(positions), _ptr(cos_sin_cache), max_pos,
            Tp, H, dn, dv, _stream(q)))
    return q8, k8, v8


def sparse_fwd(q, kv_records, kv_indptr, kv_indices, softmax_scale, *, has_invalid=False, out=None,
               return_lse=False, num_records=None, kernel="gather", attn_sink=None, extra_kv=None, extra_indptr=None,
               extra_indices=None, kv_splits=1, workspace=None, lse=None):
    """Sparse forward over fp8_ds_mla records [N, >=656] (uint8).  Returns (out, lse).

    kv_indptr / kv_indices may be int32 or int64 (int64 is narrowed on the device, keeping
    masked and out-of-range ids as such).  attn_sink (fp32 [H]), a second key segment
    (extra_kv records with extra_indptr / extra_indices) and kv_splits > 1 run
    mla_sparse_fwd_ext.  kernel="staged" runs the test aid mla_sparse_fwd_staged (the second
    kernel design) instead of mla_sparse_fwd."""
    dev = _cuda_device(q)
    _need(q, "q", (torch.bfloat16,), dev, ndim=3)
    _need(kv_records, "kv_records", _BYTE_TYPES, dev)
    T, H, _ = q.shape
    rec = kv_records.reshape(-1, kv_records.shape[-1]) if kv_records.dim() != 2 else kv_records
    n_rec = rec.shape[0] if num_records is None else num_records
    if kv_indptr.numel() != T + 1:
        raise ValueError(f"kv_indptr must have T + 1 = {T + 1} entries, got {kv_indptr.numel()}")
    n_idx = kv_indices.numel()
    kv_indptr = _index_i32(kv_indptr, "kv_indptr", dev, 0, min(n_idx, _INT32_MAX))
    kv_indices = _index_i32(kv_indices, "kv_indices", dev, -1, min(n_rec, _INT32_MAX))
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev)
    _need(out, "out", (torch.bfloat16,), dev, ndim=3)
    if return_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, "lse", (torch.float32,), dev, ndim=2, contiguous=True)
        if tuple(lse.shape) != (T, H):
            raise ValueError(f"lse must be [T, H] = {(T, H)}")
    ext = attn_sink is not None or extra_kv is not None or int(kv_splits) != 1
    if not ext:
        fn = {"gather": lib().mla_sparse_fwd, "staged": lib().mla_sparse_fwd_staged}[kernel]
        with torch.cuda.device(dev):
            _check(fn(
                _ptr(q), q.stride(0), q.stride(1), _ptr(rec), rec.stride(0) * rec.element_size(), n_rec,
                _ptr(kv_indptr), _ptr(kv_indices), n_idx, float(softmax_scale), int(bool(has_invalid)),
                _ptr(out), out.stride(0), out.stride(1), _ptr(lse), T, H, _stream(q)))
        return out, lse
    if kernel != "gather":
        raise ValueError("the sink, second segment and kv_splits are served by the gather kernel only")
    rec2, n_rec2, n_idx2 = None, 0, 0
    if extra_kv is not None:
        _need(extra_kv, "extra_kv", _BYTE_TYPES, dev)
        rec2 = extra_kv.reshape(-1, extra_kv.shape[-1]) if extra_kv.dim() != 2 else extra_kv
        n_rec2 = rec2.shape[0]
        if extra_indptr is None or extra_indices is None or extra_indptr.numel() != T + 1:
            raise ValueError("extra_kv needs extra_indptr [T + 1] and extra_indices")
        n_idx2 = extra_indices.numel()
        extra_indptr = _index_i32(extra_indptr, "extra_indptr", dev, 0, min(n_idx2, _INT32_MAX))
        extra_indices = _index_i32(extra_indices, "extra_indices", dev, -1, min(n_rec2, _INT32_MAX))
    if attn_sink is not None:
        _need(attn_sink, "attn_sink", (torch.float32,), dev, ndim=1, contiguous=True)
        if attn_sink.numel() != H:
            raise ValueError(f"attn_sink must have H = {H} entries")
    with torch.cuda.device(dev):
        need = int(lib().mla_sparse_fwd_ext_workspace_size(T, H, int(kv_splits), int(rec2 is not None),
                                                          int(attn_sink is not None)))
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        _check(lib().mla_sparse_fwd_ext(
            _ptr(q), q.stride(0), q.stride(1), _ptr(rec), rec.stride(0) * rec.element_size(), n_rec,
            _ptr(kv_indptr), _ptr(kv_indices), n_idx, _ptr(rec2), 0 if rec2 is None else rec2.stride(0), n_rec2,
            _ptr(extra_indptr) if rec2 is not None else None, _ptr(extra_indices) if rec2 is not None else None,
            n_idx2, _ptr(attn_sink), int(kv_splits), float(softmax_scale), int(bool(has_invalid)), _ptr(out),
            out.stride(0), out.stride(1), _ptr(lse), T, H, _ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(q)))
    return out, lse


def paged_decode_workspace_size(B, q_len, H, max_context, num_sms=0, fmt=None) -> int:
    """Bytes of workspace of a paged_decode; fmt has to be given for the mxfp4 cache, whose decode splits in its own way."""
    if fmt is None:
        return int(lib().mla_paged_decode_workspace_size(B, q_len, H, max_context, num_sms))
    return int(lib().mla_paged_decode_workspace_size_for(_fmt(fmt), B, q_len, H, max_context, num_sms))


def paged_decode(q, kv_cache, block_table, seq_lens, *, fmt, q_len=1, max_context, softmax_scale,
                 q_scale=1.0, k_scale=1.0, out=None, return_lse=False, workspace=None, lse=None):
    """Paged decode / spec-verify.  q [B*q_len, H, 576] (bf16, or uint8 E4M3 codes for fp8).
    Returns (out [B*q_len, H, 512] bf16, lse or None)."""
    fmt = _fmt(fmt)
    done = (_step or _plain_step()).paged(q, kv_cache, block_table, seq_lens, fmt, q_len, max_context, softmax_scale, q_scale, k_scale,
                                          out, return_lse, workspace, lse)
    if done is not None:
        return done
    dev = _cuda_device(q)
    _need(q, "q", _BYTE_TYPES if fmt == CACHE_FP8 else (torch.bfloat16,), dev, ndim=3)
    _need(kv_cache, "kv_cache", _BYTE_TYPES + (torch.bfloat16,), dev)
    _need(block_table, "block_table", (torch.int32,), dev, ndim=2)
    _need(seq_lens, "seq_lens", (torch.int32,), dev, ndim=1, contiguous=True)
    rows, H, _ = q.shape
    B = seq_lens.numel()
    if rows != B * q_len:
        raise ValueError(f"q has {rows} rows; expected B * q_len = {B * q_len}")
    if out is None:
        out = torch.empty((rows, H, 512), dtype=torch.bfloat16, device=dev)
    _need(out, "out", (torch.bfloat16,), dev, ndim=3)
    if return_lse and lse is None:
        lse = torch.empty((rows, H), dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, "lse", (torch.float32,), dev, ndim=2, contiguous=True)
        if tuple(lse.shape) != (rows, H):
            raise ValueError(f"lse must be [B * q_len, H] = {(rows, H)}")
    with torch.cuda.device(dev):
        need = paged_decode_workspace_size(B, q_len, H, max_context, fmt=fmt)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        if workspace is not None:
            _need(workspace, "workspace", _BYTE_TYPES, dev, contiguous=True)
        nb, bstride, estride, bs = _cache_geometry(kv_cache, fmt)
        _check(lib().mla_paged_decode(
            _ptr(q), q.stride(0), q.stride(1), _ptr(kv_cache), fmt, nb, bstride, estride, bs,
            _ptr(block_table), block_table.stride(0), _ptr(seq_lens), B, q_len, H, int(max_context),
            float(softmax_scale), float(q_scale), float(k_scale), _ptr(out), out.stride(0), out.stride(1),
            _ptr(lse), _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
            _stream(q)))
    return out, lse


def absorb_q(q_nope, w_uk_t, *, ql_nope=None):
    """BMM1: ql_nope[b, h] = q_nope[b, h] . w_uk_t[h]; q_nope bf16 [B, H, P] (unit innermost
    stride), w_uk_t bf16 [H, P, 512].  Returns ql_nope [B, H, 512] bf16."""
    dev = _cuda_device(q_nope)
    _need(q_nope, "q_nope", (torch.bfloat16,), dev, ndim=3)
    _need(w_uk_t, "w_uk_t", (torch.bfloat16,), dev, ndim=3, contiguous=True)
    B, H, P = q_nope.shape
    if tuple(w_uk_t.shape) != (H, P, 512):
        raise ValueError(f"w_uk_t must be [H, P, 512] = {(H, P, 512)}, got {tuple(w_uk_t.shape)}")
    if ql_nope is None:
        ql_nope = torch.empty((B, H, 512), dtype=torch.bfloat16, device=dev)
    _need(ql_nope, "ql_nope", (torch.bfloat16,), dev, ndim=3)
    with torch.cuda.device(dev):
        _check(lib().mla_absorb_q(_ptr(q_nope), q_nope.stride(0), q_nope.stride(1), _ptr(w_uk_t), _ptr(ql_nope),
                                  ql_nope.stride(0), ql_nope.stride(1), B, H, P, _stream(q_nope)))
    return ql_nope


def v_up_proj(latent, w_uv, gate=None, *, out=None):
    """out[b, h] = latent[b, h] . w_uv[h] (times bf16(sigmoid(gate[b, h*V:(h+1)*V])) when a
    gate is given); latent bf16 [B, H, 512], w_uv bf16 [H, 512, V], gate bf16 [B, H * V].
    Returns out [B, H, V] bf16."""
    dev = _cuda_device(latent)
    _need(latent, "latent", (torch.bfloat16,), dev, ndim=3)
    _need(w_uv, "w_uv", (torch.bfloat16,), dev, ndim=3, contiguous=True)
    B, H, L = latent.shape
    if L != 512 or w_uv.shape[0] != H or w_uv.shape[1] != 512:
        raise ValueError("latent must be [B, H, 512] and w_uv [H, 512, V]")
    V = w_uv.shape[2]
    if gate is not None:
        _need(gate, "gate", (torch.bfloat16,), dev, ndim=2)
        if tuple(gate.shape) != (B, H * V):
            raise ValueError(f"gate must be [B, H * V] = {(B, H * V)}")
    if out is None:
        out = torch.empty((B, H, V), dtype=torch.bfloat16, device=dev)
    _need(out, "out", (torch.bfloat16,), dev, ndim=3)
    with torch.cuda.device(dev):
        _check(lib().mla_v_up_proj(_ptr(latent), latent.stride(0), latent.stride(1), _ptr(w_uv), _ptr(gate),
                                   0 if gate is None else gate.stride(0), _ptr(out), out.stride(0), out.stride(1), B, H,
                                   V, _stream(latent)))
    return out


def gather_context(kv_cache, block_table, cu_seq_lens, seq_starts=None, *, fmt, num_tokens, raw=False,
                   scale=1.0, dst=None):
    """Chunked-context gather: rows cu_seq_lens[b] .. cu_seq_lens[b+1]-1 hold request b's context
    positions seq_starts[b] + i.  Returns dst [num_tokens, 576] bf16 (raw=False) or
    [num_tokens, entry bytes] uint8 (raw=True)."""
    fmt = _fmt(fmt)
    done = (_step or _plain_step()).context(kv_cache, block_table, cu_seq_lens, seq_starts, fmt, num_tokens, raw, scale, dst)
    if done is not None:
        return done
    dev = _cuda_device(kv_cache)
    _need(kv_cache, "kv_cache", _BYTE_TYPES + (torch.bfloat16,), dev)
    _need(block_table, "block_table", (torch.int32,), dev, ndim=2)
    _need(cu_seq_lens, "cu_seq_lens", (torch.int32,), dev, ndim=1, contiguous=True)
    if seq_starts is not None:
        _need(seq_starts, "seq_starts", (torch.int32,), dev, ndim=1, contiguous=True)
    batch = cu_seq_lens.numel() - 1
    if block_table.shape[0] < batch or (seq_starts is not None and seq_starts.numel() < batch):
        raise ValueError("block_table and seq_starts need a row per request of the chunk")
    if dst is None:
        dst = (torch.empty((num_tokens, ENTRY_BYTES[fmt]), dtype=torch.uint8, device=dev) if raw else
               torch.empty((num_tokens, 576), dtype=torch.bfloat16, device=dev))
    _need(dst, "dst", _BYTE_TYPES if raw else (torch.bfloat16,), dev, ndim=2)
    nb, bstride, estride, bs = _cache_geometry(kv_cache, fmt)
    with torch.cuda.device(dev):
        _check(lib().mla_gather_context(_ptr(kv_cache), fmt, nb, bstride, estride, bs, _ptr(block_table),
                                        block_table.stride(0), _ptr(cu_seq_lens), _ptr(seq_starts), batch,
                                        int(num_tokens), 1 if raw else 0, float(scale), _ptr(dst),
                                        dst.stride(0) * dst.element_size(), _stream(kv_cache)))
    return dst


def merge_attn_states(prefix_output, prefix_lse, suffix_output, suffix_lse, *, output=None, return_lse=False):
    """Merge of a prefix and a suffix partial attention (bf16 [T, H, D], lse fp32 [H, T]).
    Returns (output [T, H, D] bf16, lse [H, T] or None)."""
    dev = _cuda_device(prefix_output)
    _need(prefix_output, "prefix_output", (torch.bfloat16,), dev, ndim=3)
    _need(suffix_output, "suffix_output", (torch.bfloat16,), dev, ndim=3)
    T, H, D = prefix_output.shape
    if tuple(suffix_output.shape) != (T, H, D):
        raise ValueError("prefix and suffix outputs differ in shape")
    for n, t in (("prefix_lse", prefix_lse), ("suffix_lse", suffix_lse)):
        _need(t, n, (torch.float32,), dev, ndim=2, contiguous=True)
        if tuple(t.shape) != (H, T):
            raise ValueError(f"{n} must be [H, T] = {(H, T)}, got {tuple(t.shape)}")
    if output is None:
        output = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
    _need(output, "output", (torch.bfloat16,), dev, ndim=3)
    lse = torch.empty((H, T), dtype=torch.float32, device=dev) if return_lse else None
    with torch.cuda.device(dev):
        _check(lib().mla_merge_attn_states(
            _ptr(output), output.stride(0), output.stride(1), _ptr(lse), _ptr(prefix_output), prefix_output.stride(0),
            prefix_output.stride(1), _ptr(prefix_lse), _ptr(suffix_output), suffix_output.stride(0),
            suffix_output.stride(1), _ptr(suffix_lse), T, H, D, _stream(prefix_output)))
    return output, lse


# The selector's calls are short on the device.  The plain ones (tensors as documented, on the current
# device) are marshalled in C (csrc/mla_marshal.cpp), which declines every other call with None: the Python
# form below then serves it, or words the refusal.
_BF16, _F32, _I32, _I64 = (torch.bfloat16,), (torch.float32,), (torch.int32,), (torch.int64,)
_INDEX_TYPES = {CACHE_BF16: _BF16, CACHE_FP8: _BYTE_TYPES}
_KV_TYPES = _BYTE_TYPES + _BF16
_KV_BYTES = ENTRY_BYTES
_current_device = torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


_marshal = None
_step = None                # its functions for the cache's and the step's calls, or _DeclinedStep


class _DeclinedStep:
    """In place of the C marshalling of the cache's and the step's calls where it is not built."""
    q_concat = key_concat = paged = context = rope = plan = staticmethod(lambda *args: None)


def _plain_step():
    """The C marshalling of the cache's and the step's calls: _plain's module."""
    global _step
    mod = _plain()
    if hasattr(mod, "init_step"):
        mod.init_step(torch.float16, torch.bool)
        _step = mod
    else:
        _step = _DeclinedStep
    return _step


class _Declined:
    """In place of the C marshalling where it is not built: every call takes its Python form."""
    insert = gather = scores = select = selected = staticmethod(lambda *args: None)


def _plain():
    """The C marshalling of the selector's calls, built with libmla.so for this interpreter (without it, a warning
    and the Python form of every call)."""
    global _marshal
    if _marshal is None:
        lib()
        try:
            loader = importlib.machinery.ExtensionFileLoader("mla_marshal", _build.MARSHAL)
            mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("mla_marshal", loader))
            loader.exec_module(mod)
            mod.init(torch.Tensor, torch.empty, getattr(torch._C, "_cuda_getDevice", _current_device), _raw_stream, _check,
                     torch.bfloat16, torch.uint8, torch.int8, torch.float32, torch.int32, torch.int64)
        except ImportError as e:
            warnings.warn(f"the selector's calls take their Python form: {e}; mla_latent_cache_attention_gb300.build.build() builds "
                          "their C marshalling")
            mod = _Declined
        _marshal = mod
    return _marshal


def _strides(t, name, dtypes, dev, ndim):
    """The strides of a tensor that passes _need's checks (unit innermost stride), for the C entry, which refuses
    rows that overlap (an expanded tensor's do).  The stride of a dimension of one entry means nothing: where it
    is below what the entry spans, that is handed over."""
    try:
        plain = t.dtype in dtypes and t.get_device() == dev.index and t.dim() == ndim and t.stride(-1) == 1
    except AttributeError:
        plain = False           # not a tensor: _need says so
    if not plain:
        _need(t, name, dtypes, dev, ndim=ndim)
    st = list(t.stride())
    for i in range(ndim - 2, -1, -1):
        if t.shape[i] <= 1:
            st[i] = max(st[i], t.shape[i + 1] * st[i + 1])
    return st


def _call(fn, dev, *args):
    """fn(*args, current stream of dev) with dev current."""
    index = dev.index
    if _current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(index))
    if rc:
        _check(rc)


_INDEX_FORMATS = {"bf16": CACHE_BF16, "auto": CACHE_BF16, "fp8": CACHE_FP8, CACHE_BF16: CACHE_BF16, CACHE_FP8: CACHE_FP8}


def _index_format(fmt) -> int:
    found = _INDEX_FORMATS.get(fmt)
    if found is None:
        raise ValueError("the index cache is bf16 or fp8")
    return found


def _index_geometry(index_cache, index_scales, fmt, dev):
    """(num_blocks, block stride and entry stride in bytes, scales' address, their block stride,
    block_size) of an index cache [num_blocks, block_size, 128] and its scales fp32
    [num_blocks, block_size]."""
    st = _strides(index_cache, "index_cache", _INDEX_TYPES[fmt], dev, 3)
    nb, bs, width = index_cache.shape
    if width != 128:
        raise ValueError(f"index keys have 128 values, got {width}")
    if fmt == CACHE_BF16:
        if index_scales is not None:
            raise ValueError("index_scales are only for the fp8 index cache")
        return nb, 2 * st[0], 2 * st[1], None, 0, bs
    ss = _strides(index_scales, "index_scales", _F32, dev, 2)
    if index_scales.shape != (nb, bs):
        raise ValueError(f"index_scales must be [num_blocks, block_size] = {(nb, bs)}, got {tuple(index_scales.shape)}")
    return nb, st[0], st[1], index_scales.data_ptr(), ss[0], bs


def _requests(seq_lens, cu_q_lens, T, dev):
    """The number of requests and cu_q_lens' address (None: one row per request)."""
    _strides(seq_lens, "seq_lens", _I32, dev, 1)
    B = seq_lens.shape[0]
    if cu_q_lens is None:
        if T != B:
            raise ValueError(f"without cu_q_lens there is one row per request: {T} rows, {B} requests")
        return B, None
    _strides(cu_q_lens, "cu_q_lens", _I32, dev, 1)
    if cu_q_lens.shape[0] != B + 1:
        raise ValueError(f"cu_q_lens must have B + 1 = {B + 1} entries, got {cu_q_lens.shape[0]}")
    return B, cu_q_lens.data_ptr()


def _table(block_table, rows, dev):
    """Address, row stride and columns of a block table with a row per request."""
    st = _strides(block_table, "block_table", _I32, dev, 2)
    have, cols = block_table.shape
    if have < rows:
        raise ValueError(f"block_table needs a row per request: {have} rows, {rows} requests")
    return block_table.data_ptr(), st[0], cols


def index_q_cache_insert(q, k, weights, index_cache, index_scales, slot_mapping, *, fmt, weight_scale=1.0,
                         positions=None, cos_sin_cache=None, q_out=None, w_out=None):
    """Index queries [T, Hi, 128] and keys [T, 128] (bf16) rotated, quantised, and the keys written to
    the index cache at slot_mapping.  Returns (q_out [T, Hi, 128]: bf16, or uint8 E4M3 codes;
    w_out fp32 [T, Hi]: weights * weight_scale, times the query's scale for fp8)."""
    fmt = _index_format(fmt)
    done = (_marshal or _plain()).insert(q, k, weights, index_cache, index_scales, slot_mapping, fmt, weight_scale, positions,
                                         cos_sin_cache, q_out, w_out)
    if done is not None:
        return done
    dev = _cuda_device(q)
    qs = _strides(q, "q", _BF16, dev, 3)
    T, Hi, width = q.shape
    if isinstance(k, torch.Tensor) and k.dim() == 3 and k.shape[1] == 1:      # [T, 1, 128]
        k = k.squeeze(1)
    ks = _strides(k, "k", _BF16, dev, 2)
    ws = _strides(weights, "weights", _F32, dev, 2)
    _strides(slot_mapping, "slot_mapping", _I64, dev, 1)
    if width != 128 or k.shape != (T, 128) or weights.shape != (T, Hi) or slot_mapping.shape[0] != T:
        raise ValueError("q must be [T, Hi, 128], k [T, 128], weights [T, Hi] and slot_mapping [T]")
    pos = cs = None
    max_pos = 0
    if positions is not None:
        _strides(positions, "positions", _I64, dev, 1)
        if positions.shape[0] != T:
            raise ValueError(f"positions must have T = {T} entries")
        pos = positions.data_ptr()
    if cos_sin_cache is not None:
        if _strides(cos_sin_cache, "cos_sin_cache", _F32, dev, 2)[0] != 64:
            _need(cos_sin_cache, "cos_sin_cache", _F32, dev, ndim=2, contiguous=True)
        max_pos, half = cos_sin_cache.shape
        if half != 64:
            raise ValueError("cos_sin_cache must be [max_position, 64]")
        cs = cos_sin_cache.data_ptr()
    out_types = _INDEX_TYPES[fmt]
    if q_out is None:
        q_out = torch.empty((T, Hi, 128), dtype=out_types[0], device=dev)
    else:
        _need(q_out, "q_out", out_types, dev, ndim=3, contiguous=True)
        if q_out.shape != (T, Hi, 128):
            raise ValueError("q_out must be [T, Hi, 128]")
    if w_out is None:
        w_out = torch.empty((T, Hi), dtype=torch.float32, device=dev)
    else:
        _need(w_out, "w_out", _F32, dev, ndim=2, contiguous=True)
        if w_out.shape != (T, Hi):
            raise ValueError("w_out must be [T, Hi]")
    nb, bstride, estride, sc, sstride, bs = _index_geometry(index_cache, index_scales, fmt, dev)
    _call(lib().mla_index_q_cache_insert, dev, q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], weights.data_ptr(), ws[0],
          float(weight_scale), q_out.data_ptr(), w_out.data_ptr(), index_cache.data_ptr(), fmt, nb, bstride, estride, sc, sstride,
          bs, slot_mapping.data_ptr(), pos, cs, max_pos, T, Hi)
    return q_out, w_out


def index_gather(index_cache, index_scales, block_table, cu_seq_lens, seq_starts=None, *, fmt, num_tokens, dst=None):
    """Cached index keys as bf16 [num_tokens, 128]: rows cu_seq_lens[b] .. cu_seq_lens[b+1]-1 hold
    request b's positions seq_starts[b] + i.  Rows of no request are not written: a dst that is not handed
    in has there what the allocator left."""
    fmt = _index_format(fmt)
    done = (_marshal or _plain()).gather(index_cache, index_scales, block_table, cu_seq_lens, seq_starts, fmt, num_tokens, dst)
    if done is not None:
        return done
    dev = _cuda_device(index_cache)
    nb, bstride, estride, sc, sstride, bs = _index_geometry(index_cache, index_scales, fmt, dev)
    _strides(cu_seq_lens, "cu_seq_lens", _I32, dev, 1)
    batch = cu_seq_lens.shape[0] - 1
    table, tstride, cols = _table(block_table, batch, dev)
    starts = None
    if seq_starts is not None:
        _strides(seq_starts, "seq_starts", _I32, dev, 1)
        if seq_starts.shape[0] < batch:
            raise ValueError("seq_starts needs an entry per request")
        starts = seq_starts.data_ptr()
    num_tokens = int(num_tokens)
    if dst is None:
        dst = torch.empty((num_tokens, 128), dtype=torch.bfloat16, device=dev)
    ds = _strides(dst, "dst", _BF16, dev, 2)
    if dst.shape != (num_tokens, 128):
        raise ValueError(f"dst must be [num_tokens, 128] = {(num_tokens, 128)}")
    _call(lib().mla_index_gather, dev, index_cache.data_ptr(), fmt, nb, bstride, estride, sc, sstride, bs, table, tstride,
          cols, cu_seq_lens.data_ptr(), starts, batch, num_tokens, dst.data_ptr(), ds[0])
    return dst


def index_scores(q, weights, index_cache, index_scales, block_table, seq_lens, cu_q_lens=None, *, fmt, block_tokens=1,
                 max_context, scores=None):
    """Scores sum_h weights[t, h] * relu(q[t, h] . k[j]) of every visible token (block_tokens = 1), or
    their maximum over blocks of block_tokens.  q [T, Hi, 128] (bf16, or uint8 E4M3 codes with their
    scales in the weights).  Returns scores fp32 [T, >= ceil(max_context / block_tokens)]; only the
    columns of visible blocks are written, and no row outside every request."""
    fmt = _index_format(fmt)
    done = (_marshal or _plain()).scores(q, weights, index_cache, index_scales, block_table, seq_lens, cu_q_lens, fmt, block_tokens,
                                         max_context, scores)
    if done is not None:
        return done
    dev = _cuda_device(q)
    qs = _strides(q, "q", _INDEX_TYPES[fmt], dev, 3)
    T, Hi, width = q.shape
    ws = _strides(weights, "weights", _F32, dev, 2)
    if width != 128 or weights.shape != (T, Hi):
        raise ValueError("q must be [T, Hi, 128] and weights [T, Hi]")
    B, cu = _requests(seq_lens, cu_q_lens, T, dev)
    table, tstride, tcols = _table(block_table, B, dev)
    nb, bstride, estride, sc, sstride, bs = _index_geometry(index_cache, index_scales, fmt, dev)
    block_tokens, max_context = int(block_tokens), int(max_context)
    if not 1 <= block_tokens <= 0x7FFFFFFF or max_context < 0:      # (ctypes would wrap a larger one)
        raise ValueError("block_tokens must be in [1, 2^31) and max_context >= 0")
    cols = -(-max_context // block_tokens)
    if scores is None:
        scores = torch.empty((T, cols), dtype=torch.float32, device=dev)
    ss = _strides(scores, "scores", _F32, dev, 2)
    rows, have = scores.shape
    if rows != T or have < cols:
        raise ValueError(f"scores must be [T, >= {cols}] with T = {T}, got {tuple(scores.shape)}")
    _call(lib().mla_index_scores, dev, q.data_ptr(), qs[0], qs[1], weights.data_ptr(), ws[0], index_cache.data_ptr(), fmt, nb,
          bstride, estride, sc, sstride, bs, table, tstride, tcols, seq_lens.data_ptr(), cu, B, T, Hi, block_tokens,
          scores.data_ptr(), ss[0], cols)
    return scores


def index_select(scores, seq_lens, topk, cu_q_lens=None, *, block_tokens=1, first=0, last=0, block_table=None,
                 page_size=0, num_blocks=0, blocks=None, slots=None):
    """The topk best-scored blocks of every row, ascending, -1 after them; ties go to the lowest index,
    -inf and NaN are never taken, the first `first` and last `last` visible blocks always.  With a
    block_table (and page_size, num_blocks) also the cache slots of their visible tokens, for
    sparse_fwd.  Returns (blocks int32 [T, topk], slots int32 [T, topk * block_tokens] or None).  Rows outside
    every request are not written: for a padded batch whose slots go to sparse_fwd hand in slots filled
    with -1."""
    done = (_marshal or _plain()).select(scores, seq_lens, topk, cu_q_lens, block_tokens, first, last, block_table, page_size,
                                         num_blocks, blocks, slots)
    if done is not None:
        return done
    dev = _cuda_device(scores)
    ss = _strides(scores, "scores", _F32, dev, 2)
    T, width = scores.shape
    B, cu = _requests(seq_lens, cu_q_lens, T, dev)
    topk, block_tokens, first, last, page_size, num_blocks = map(int, (topk, block_tokens, first, last, page_size, num_blocks))
    if topk < 1 or block_tokens < 1:
        raise ValueError("topk and block_tokens must be >= 1")
    if max(topk, block_tokens, abs(first), abs(last), abs(page_size)) > 0x7FFFFFFF:      # ctypes would wrap them
        raise ValueError("topk, block_tokens, first, last and page_size are 32-bit")
    if blocks is None:
        blocks = torch.empty((T, topk), dtype=torch.int32, device=dev)
    bs = _strides(blocks, "blocks", _I32, dev, 2)
    if blocks.shape != (T, topk):
        raise ValueError(f"blocks must be [T, topk] = {(T, topk)}")
    table, tstride, tcols, sl, sl_stride = None, 0, 0, None, 0
    if block_table is not None:
        table, tstride, tcols = _table(block_table, B, dev)
        per_row = topk * block_tokens
        if slots is None:
            slots = torch.empty((T, per_row), dtype=torch.int32, device=dev)
        sl_stride = _strides(slots, "slots", _I32, dev, 2)[0]
        if slots.shape != (T, per_row):
            raise ValueError(f"slots must be [T, topk * block_tokens] = {(T, per_row)}")
        sl = slots.data_ptr()
    elif slots is not None:
        raise ValueError("slots need a block_table")
    _call(lib().mla_index_select, dev, scores.data_ptr(), ss[0], width, seq_lens.data_ptr(), cu, B, T,
          block_tokens, topk, first, last, blocks.data_ptr(), bs[0], sl, sl_stride, table, tstride,
          tcols, page_size, num_blocks)
    return blocks, slots


def selected_decode_workspace_size(fmt, T, topk, block_size, H, num_sms=0) -> int:
    """Bytes of workspace of a selected_decode of exactly T rows (fewer rows may need more)."""
    return int(lib().mla_selected_decode_workspace_size(_fmt(fmt), T, topk, block_size, H, num_sms))


def selected_decode_workspace_bound(fmt, max_T, topk, block_size, H, num_sms=0) -> int:
    """Bytes of workspace that are enough for every selected_decode of 1 .. max_T rows."""
    return int(lib().mla_selected_decode_workspace_bound(_fmt(fmt), max_T, topk, block_size, H, num_sms))


def selected_decode(q, kv_cache, block_table, seq_lens, blocks, cu_q_lens=None, *, fmt, softmax_scale, q_scale=1.0,
                    k_scale=1.0, out=None, return_lse=False, workspace=None, lse=None):
    """Decode over the selected pages: row t of q [T, H, 576] attends the visible tokens of pages
    blocks[t] (int32 [T, topk], negative entries skipped) of its request.  Returns (out [T, H, 512]
    bf16, lse [T, H] or None), as paged_decode."""
    fmt = _fmt(fmt)
    done = (_marshal or _plain()).selected(q, kv_cache, block_table, seq_lens, blocks, cu_q_lens, fmt, softmax_scale, q_scale,
                                           k_scale, out, return_lse, workspace, lse)
    if done is not None:
        return done
    dev = _cuda_device(q)
    qs = _strides(q, "q", _BYTE_TYPES if fmt == CACHE_FP8 else _BF16, dev, 3)
    T, H, width = q.shape
    if width != 576:
        raise ValueError(f"q must be [T, H, 576], got {tuple(q.shape)}")
    if isinstance(kv_cache, torch.Tensor) and kv_cache.dim() == 4 and kv_cache.shape[1] == 1:      # a head axis of size 1
        kv_cache = kv_cache.squeeze(1)
    kvs = _strides(kv_cache, "kv_cache", _KV_TYPES if fmt == CACHE_BF16 else _BYTE_TYPES, dev, 3)
    es = kv_cache.element_size()
    if kv_cache.shape[2] * es < _KV_BYTES.get(fmt, 0):
        raise ValueError(f"entries of this cache format have {_KV_BYTES[fmt]} bytes, kv_cache has {kv_cache.shape[2] * es}")
    B, cu = _requests(seq_lens, cu_q_lens, T, dev)
    table, tstride, tcols = _table(block_table, B, dev)
    ls = _strides(blocks, "blocks", _I32, dev, 2)
    rows, topk = blocks.shape
    if rows != T:
        raise ValueError(f"blocks must be [T, topk] with T = {T}, got {tuple(blocks.shape)}")
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev)
    os_ = _strides(out, "out", _BF16, dev, 3)
    if out.shape[:2] != (T, H) or out.shape[2] < 512:
        raise ValueError(f"out must be [T, H, >= 512], got {tuple(out.shape)}")
    if lse is not None:
        _need(lse, "lse", _F32, dev, ndim=2, contiguous=True)
        if lse.shape != (T, H):
            raise ValueError(f"lse must be [T, H] = {(T, H)}")
    elif return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    if B == 0:              # every row is outside every request
        out[..., :512].zero_()
        if lse is not None:
            lse.fill_(float("-inf"))
        return out, lse
    nb, bs, _ = kv_cache.shape
    L = lib()
    if workspace is None:
        if _current_device() == dev.index:
            need = L.mla_selected_decode_workspace_size(fmt, T, topk, bs, H, 0)
        else:
            with torch.cuda.device(dev):
                need = L.mla_selected_decode_workspace_size(fmt, T, topk, bs, H, 0)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", _BYTE_TYPES, dev, contiguous=True)
    _call(L.mla_selected_decode, dev, q.data_ptr(), qs[0], qs[1], kv_cache.data_ptr(), fmt, nb, es * kvs[0], es * kvs[1], bs,
          table, tstride, tcols, seq_lens.data_ptr(), cu, blocks.data_ptr(), ls[0], topk, B, T, H,
          float(softmax_scale), float(q_scale), float(k_scale), out.data_ptr(), os_[0], os_[1], None if lse is None else lse.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse


def gather_dequant(kv_cache, slots, *, fmt):
    """Exact fp32 values [n, 576] of the entries at `slots` (int64)."""
    fmt = _fmt(fmt)
    dev = _cuda_device(kv_cache)
    _need(slots, "slots", (torch.int64,), dev, ndim=1, contiguous=True)
    nb, bstride, estride, bs = _cache_geometry(kv_cache, fmt)
    out = torch.empty((slots.numel(), 576), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().mla_gather_dequant(_ptr(kv_cache), fmt, nb, bstride, estride, bs, _ptr(slots),
                                        slots.numel(), _ptr(out), _stream(kv_cache)))
    return out


def debug_stall_next_decode(wait_us: int):
    """Test aid (mla_debug_stall_next_decode): the next page-kernel decode on this thread
    issues no loads and its waits give up after wait_us microseconds."""
    lib().mla_debug_stall_next_decode(int(wait_us))


def debug_ds_cluster(size: int = 0) -> None:
    """Without effect, kept for its callers: fp8_ds_mla decodes run one CTA per group of 16 columns,
    with the results that every choice gave."""
    lib().mla_debug_ds_cluster(int(size))


# ------------------------------------------------------------------------------------------ around a step

_ROPE_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ROPE_LAYOUTS = {"interleaved": False, "half": True}
_ROPE_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}


def rope_table(max_position, dim, *, base=10000.0, scaling=None, factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0,
               attn_scale=None, device=None):
    """The table of rope and of the fused epilogues (dim 64 there): fp32 [max_position, dim], dim / 2 cosines, then dim / 2
    sines of every position, from angles in 64 bits.  scaling: None, "linear" (positions interpolated by factor), "ntk"
    (the base raised for factor) or "yarn" (pairs that turn more than beta_fast times over the `original` positions
    as they are, less than beta_slow times interpolated, a ramp between).  attn_scale multiplies the table; None is
    0.1 ln(factor) + 1 for yarn with a factor above 1, else 1."""
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(map(repr, _ROPE_SCALINGS))}, got {scaling!r}")
    max_position, dim, original = int(max_position), int(dim), int(original)
    if not 0 <= max_position < 2 ** 40 or not 2 <= dim <= 512 or dim % 2 or not abs(original) < 2 ** 62:
        raise ValueError("max_position must be >= 0 and dim an even number from 2 to 512")
    factor = float(factor)
    if attn_scale is None:
        attn_scale = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1.0 else 1.0
    dev = torch.device("cuda" if device is None else device)
    if dev.type != "cuda":
        raise ValueError("the table is made on a CUDA device")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    out = torch.empty((max_position, dim), dtype=torch.float32, device=dev)
    _call(lib().mla_rope_table, dev, out.data_ptr(), max_position, dim, float(base), _ROPE_SCALINGS[scaling], factor, original,
          float(beta_fast), float(beta_slow), float(attn_scale))
    return out


def _rope_at(at, width, R, name):
    at = width - R if at is None else int(at)
    if not 0 <= at <= width - R:
        raise ValueError(f"{name}: {R} rotated values from {at} on do not fit {width}")
    return at


def rope(q, positions, cos_sin_cache, k=None, *, layout="interleaved", inverse=False, q_at=None, k_at=None, q_out=None, k_out=None):
    """Rotary positions of q [T, H, D] and k [T, Hk, Dk] (bf16, fp16 or fp32) in one launch.  The R values from q_at / k_at on
    (by default the last R of a head; R is the width of cos_sin_cache, see rope_table) turn by their token's angles, in
    pairs (2i, 2i + 1) ("interleaved") or (i, i + R / 2) ("half"); the others are copied.  inverse=True turns back: the
    transposed rotation, which takes the gradient of the output to the input's.  q_out / k_out: new tensors, or q / k
    themselves (in place, both or neither).  Returns q_out, or (q_out, k_out) where k is given."""
    if layout not in _ROPE_LAYOUTS:
        raise ValueError(f"layout must be 'interleaved' or 'half', got {layout!r}")
    half = _ROPE_LAYOUTS[layout]
    done = (_step or _plain_step()).rope(q, positions, cos_sin_cache, k, half, inverse, -1 if q_at is None else q_at, -1 if k_at is None else k_at,
                                         q_out, k_out) if (q_at is None or q_at >= 0) and (k_at is None or k_at >= 0) else None
    if done is not None:
        return done
    dev = _cuda_device(q)
    types = tuple(_ROPE_TYPES)
    qs = _strides(q, "q", types, dev, 3)
    same = (q.dtype,)
    T, H, D = q.shape
    _strides(positions, "positions", _I64, dev, 1)
    if positions.shape[0] != T:
        raise ValueError(f"positions must have T = {T} entries")
    _need(cos_sin_cache, "cos_sin_cache", _F32, dev, ndim=2, contiguous=True)
    max_pos, R = cos_sin_cache.shape
    if R < 2 or R % 2 or R > 512:
        raise ValueError(f"cos_sin_cache must have an even width from 2 to 512, got {R}")

    def out_of(x, out, name):
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=dev)
        st = _strides(out, name, same, dev, 3)
        if out.shape != x.shape:
            raise ValueError(f"{name} must be {tuple(x.shape)}, got {tuple(out.shape)}")
        return out, st

    q_at = _rope_at(q_at, D, R, "q")
    q_out, qos = out_of(q, q_out, "q_out")
    k_args = [None, 0, 0, None, 0, 0, 0, 0, 0]
    if k is not None:
        ks = _strides(k, "k", same, dev, 3)
        if k.shape[0] != T:
            raise ValueError(f"k must have T = {T} tokens, got {k.shape[0]}")
        k_at = _rope_at(k_at, k.shape[2], R, "k")
        k_out, kos = out_of(k, k_out, "k_out")
        k_args = [k.data_ptr(), ks[0], ks[1], k_out.data_ptr(), kos[0], kos[1], k.shape[1], k.shape[2], k_at]
    elif k_out is not None or k_at is not None:
        raise ValueError("k_out and k_at need k")
    _call(lib().mla_rope, dev, _ROPE_TYPES[q.dtype], q.data_ptr(), qs[0], qs[1], q_out.data_ptr(), qos[0], qos[1], H, D, q_at, *k_args,
          positions.data_ptr(), cos_sin_cache.data_ptr(), max_pos, R, int(half), int(bool(inverse)), T)
    return q_out if k is None else (q_out, k_out)


def plan_step(seq_lens, new_lens, block_table, free_blocks, num_free, *, block_size, num_tokens, finished=None, seq_lens_out=None,
              num_free_out=None, served=None, slot_mapping=None, positions=None, cu_q_lens=None):
    """The blocks and slots of a step, without the host.  seq_lens int32 [B] (cached tokens), new_lens int32 [B] (tokens of the
    step), block_table int32 [B, cols] and free_blocks int32 [capacity] (a stack, its top at num_free - 1; both written in
    place), num_free int32 [1], finished bool [B] or None.  The blocks of finished requests go back to the stack, every
    request takes those that its new tokens need, in order.  Returns (slot_mapping int64 [num_tokens], -1 in rows of no
    request; positions int64 [num_tokens]; cu_q_lens int32 [B + 1]; the new lengths int32 [B]; the new num_free int32 [1]).
    seq_lens_out and num_free_out may be seq_lens and num_free themselves; served (bool [B]) says which requests got
    their blocks: the others keep their length, and their rows have slot -1 (device error 32).  From the first request on that
    finds too few blocks, only those that need no new one are served."""
    done = (_step or _plain_step()).plan(seq_lens, new_lens, block_table, free_blocks, num_free, block_size, num_tokens, finished, seq_lens_out,
                                         num_free_out, served, slot_mapping, positions, cu_q_lens)
    if done is not None:
        return done
    dev = _cuda_device(seq_lens)
    _strides(seq_lens, "seq_lens", _I32, dev, 1)
    B = seq_lens.shape[0]
    T, block_size = int(num_tokens), int(block_size)
    if B < 1 or not 0 <= T <= _INT32_MAX or not 1 <= block_size <= _INT32_MAX:
        raise ValueError("at least one request, num_tokens >= 0 and block_size >= 1 are needed")
    table, tstride, cols = _table(block_table, B, dev)

    def vector(t, name, types, n, new=True):
        if t is None and new:
            t = torch.empty((n,), dtype=types[0], device=dev)
        _strides(t, name, types, dev, 1)
        if t.shape[0] != n:
            raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")
        return t

    vector(new_lens, "new_lens", _I32, B, False)
    vector(num_free, "num_free", _I32, 1, False)
    _strides(free_blocks, "free_blocks", _I32, dev, 1)
    flags = (torch.bool, torch.uint8)
    if finished is not None:
        vector(finished, "finished", flags, B, False)
    slot_mapping = vector(slot_mapping, "slot_mapping", _I64, T)
    positions = vector(positions, "positions", _I64, T)
    cu_q_lens = vector(cu_q_lens, "cu_q_lens", _I32, B + 1)
    seq_lens_out = vector(seq_lens_out, "seq_lens_out", _I32, B)
    num_free_out = vector(num_free_out, "num_free_out", _I32, 1)
    if served is not None or B > 1024:      # (more requests need it inside)
        served = vector(served, "served", flags, B)
    _call(lib().mla_plan_step, dev, seq_lens.data_ptr(), new_lens.data_ptr(), None if finished is None else finished.data_ptr(), table,
          tstride, cols, free_blocks.data_ptr(), free_blocks.shape[0], num_free.data_ptr(), seq_lens_out.data_ptr(),
          num_free_out.data_ptr(), None if served is None else served.data_ptr(), cu_q_lens.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(), B, T, block_size)
    return slot_mapping, positions, cu_q_lens, seq_lens_out, num_free_out
