"""ctypes binding of libmla (include/mla.h): argument marshalling only.

Every step of the decode path runs in the library's CUDA kernels; this module
turns torch tensors into device pointers and the current CUDA stream into a
cudaStream_t, and raises on error codes.  Importing it fails loudly when the
shared library has not been built: there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
from dataclasses import dataclass

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libmla.so is not built ({_LIB_PATH}); run "
                      "`python -m head_latent_attention_04_b200.build`")
_lib = ctypes.CDLL(_LIB_PATH)

MLA_OK, MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED = 0, 1, 2
MLA_ERR_WORKSPACE_TOO_SMALL, MLA_ERR_CUDA, MLA_ERR_TIMEOUT = 3, 4, 5
STATUS_BAD_BLOCK, STATUS_TIMEOUT, STATUS_BAD_SEQLEN, STATUS_BAD_PLAN, STATUS_SCORE_RANGE = 0x1, 0x2, 0x4, 0x8, 0x10
STATUS_CACHE_RANGE, STATUS_NO_SPACE = 0x20, 0x40
CACHE_KINDS = {"bf16": 0, "fp8": 1, "fp4": 2}
EXPORTS = ("mla_version", "mla_last_error_string", "mla_absorb_q", "mla_out_uv",
           "mla_max_clusters", "mla_plan_size", "mla_plan", "mla_decode_attn", "mla_combine",
           "mla_debug_gather_pages", "mla_decode_attn_combine_noalloc", "mla_noalloc_scratch_bytes",
           "mla_quantize_w_uk_fp8", "mla_quantize_w_uv_fp8", "mla_quantize_rows_fp8", "mla_absorb_q_fp8",
           "mla_out_uv_fp8", "mla_set_wait_limit_ns", "mla_decode_attn_tree", "mla_prefill_up_proj",
           "mla_prefill_attn", "mla_qkv_a_proj", "mla_q_up_absorb", "mla_decode_attn_fp8cache",
           "mla_kv_quantize_fp8", "mla_kv_quantize_fp4", "mla_kv_dequantize_fp4", "mla_decode_attn_fp4cache",
           "mla_build_tables", "mla_plan_device", "mla_summarize_pages", "mla_select_pages",
           "mla_decode_attn_sized", "mla_combine_sized", "mla_build_tables_held")


class MlaDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("s_q", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("d_nope", ctypes.c_int32), ("d_rope", ctypes.c_int32), ("d_c", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int32)]


_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_pdims = ctypes.POINTER(MlaDims)
_lib.mla_version.restype = _i32
_lib.mla_last_error_string.restype = ctypes.c_char_p
for _name, _args in {
    "mla_absorb_q": [_vp, _vp, _vp, _i32, _i32, _vp],
    "mla_out_uv": [_vp, _vp, _vp, _i32, _i32, _vp],
    "mla_max_clusters": [ctypes.POINTER(_i32)],
    "mla_plan_size": [_pdims, _i32, ctypes.POINTER(_sz), ctypes.POINTER(_sz), ctypes.POINTER(_sz)],
    "mla_plan": [_pdims, _vp, _i32, _vp, _sz, ctypes.POINTER(_i32)],
    "mla_decode_attn": [_pdims, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp],
    "mla_decode_attn_tree": [_pdims, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp],
    "mla_decode_attn_fp8cache": [_pdims, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp],
    "mla_kv_quantize_fp8": [_vp, _vp, ctypes.c_int64, _vp, _i32, _vp, _vp],
    "mla_decode_attn_sized": [_pdims, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i32, _vp, _sz, _vp, _sz, _vp, _vp, _vp,
                              _vp],
    "mla_combine_sized": [_pdims, _vp, _sz, _vp, _sz, _vp, _sz, _vp, _vp, _vp, _vp],
    "mla_kv_quantize_fp4": [_vp, _vp, ctypes.c_int64, _vp, _i32, _vp, _vp],
    "mla_kv_dequantize_fp4": [_vp, _vp, ctypes.c_int64, _vp, _i32, _vp, _vp],
    "mla_decode_attn_fp4cache": [_pdims, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp],
    "mla_build_tables": [_i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "mla_build_tables_held": [_i32, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "mla_plan_device": [_pdims, _vp, _i32, _vp, _sz, _vp, _vp],
    "mla_summarize_pages": [_vp, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp],
    "mla_select_pages": [_pdims, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _sz, _vp,
                         _vp],
    "mla_combine": [_pdims, _vp, _vp, _vp, _vp, _vp, _vp],
    "mla_debug_gather_pages": [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp],
    "mla_decode_attn_combine_noalloc": [_pdims, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i32, _vp, _vp, _vp, _vp],
    "mla_quantize_w_uk_fp8": [_vp, _i32, _vp, _vp, _vp],
    "mla_quantize_w_uv_fp8": [_vp, _i32, _vp, _vp, _vp],
    "mla_quantize_rows_fp8": [_vp, ctypes.c_int64, _i32, _vp, _vp, _vp],
    "mla_absorb_q_fp8": [_vp, _vp, _vp, _vp, _i32, _i32, _vp],
    "mla_out_uv_fp8": [_vp, _vp, _vp, _vp, _i32, _i32, _vp],
    "mla_prefill_up_proj": [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp],
    "mla_qkv_a_proj": [_vp, _vp, _vp, _vp, _i32, _vp],
    "mla_q_up_absorb": [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp],
    "mla_prefill_attn": [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, ctypes.c_float, _vp, _vp, _vp],
}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _i32


_lib.mla_noalloc_scratch_bytes.argtypes = []
_lib.mla_noalloc_scratch_bytes.restype = _sz
_lib.mla_set_wait_limit_ns.argtypes = [ctypes.c_int64]
_lib.mla_set_wait_limit_ns.restype = None


class MlaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = _lib.mla_last_error_string().decode(errors="replace")
        super().__init__(f"{where}: status {code}: {msg}")


def _check(code: int, where: str):
    if code != MLA_OK:
        raise MlaError(code, where)


def _ptr(t) -> int | None:
    """Device address of a tensor argument.  The library reads raw pointers,
    so a host tensor (a host address handed to a kernel) or a strided view
    (read as if contiguous) is refused here, before anything is launched."""
    if t is None:
        return None
    try:
        if t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        if isinstance(t, int):
            return t
        raise
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    raise ValueError("expected a contiguous tensor (the library assumes row-major layouts)")


# The step's calls are launch-bound at decode sizes, so the checks of a call that
# is right take a few attribute reads per tensor; the messages are made only for
# one that is wrong.
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _arg(t, name: str, dtype, *shape) -> int | None:
    """Device address of a tensor argument of the given type and shape, refused
    here when it is anything else (its device is checked by _on)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name}: expected a contiguous tensor (the library assumes row-major layouts)")


def _vec(t, name: str, dtype) -> int | None:
    """_arg for an array of any shape."""
    if t is None or (t.dtype is dtype and t.is_contiguous()):
        return None if t is None else t.data_ptr()
    return _arg(t, name, dtype, *t.shape)


_SAME_DEVICE = contextlib.nullcontext()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(*tensors):
    """The device of the tensors of one call (None: an argument left out), made
    current for the launch: a launch goes to the current device, and its default
    stream is that device's."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors of one call on {tensors[0].device} and {t.device}")
    if dev < 0:
        raise ValueError(f"expected a CUDA tensor, got one on {tensors[0].device}")
    return _SAME_DEVICE if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def _made_on(stream, device):
    """Context in which a call's own tensors are made: on the stream that the call
    uses, so that their memory and their fills belong to it.  A raw handle is taken
    for a stream of the tensors' device, whichever is current."""
    if stream is None:
        return _SAME_DEVICE
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device))


def _stream(stream=None) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def version() -> int:
    return _lib.mla_version()


def make_dims(B, s_q, n_heads, max_blocks, num_blocks, scale=None, causal=True) -> MlaDims:
    if scale is None:
        scale = 1.0 / math.sqrt(128 + 64)
    return MlaDims(B, s_q, n_heads, 128, 64, 512, 128, 64, max_blocks, num_blocks, float(scale),
                   1 if causal else 0)


def set_wait_limit_ns(ns: int) -> None:
    """Bound on each pipeline wait of decode launches made from now on
    (process-wide; 0 restores the 200 ms default).  A wait past it makes the
    kernel give up cleanly with STATUS_TIMEOUT."""
    _lib.mla_set_wait_limit_ns(int(ns))


def max_clusters() -> int:
    n = _i32(0)
    _check(_lib.mla_max_clusters(ctypes.byref(n)), "mla_max_clusters")
    return n.value


def plan_size(dims: MlaDims, num_clusters: int):
    pb, ob, lb = _sz(0), _sz(0), _sz(0)
    _check(_lib.mla_plan_size(ctypes.byref(dims), num_clusters, ctypes.byref(pb), ctypes.byref(ob),
                              ctypes.byref(lb)), "mla_plan_size")
    return pb.value, ob.value, lb.value


def plan(dims: MlaDims, seq_lens, num_clusters: int):
    """Host plan as an int32 numpy array, and the number of partial slots used."""
    pb, _, _ = plan_size(dims, num_clusters)
    buf = np.zeros(pb // 4, dtype=np.int32)
    sl = np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
    ns = _i32(0)
    _check(_lib.mla_plan(ctypes.byref(dims), sl.ctypes.data, num_clusters, buf.ctypes.data, pb,
                         ctypes.byref(ns)), "mla_plan")
    return buf, ns.value


def absorb_q(q_nope: torch.Tensor, w_uk: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    N, H, _ = q_nope.shape
    if out is None:
        out = torch.empty((N, H, 512), dtype=torch.bfloat16, device=q_nope.device)
    _check(_lib.mla_absorb_q(_ptr(q_nope), _ptr(w_uk), _ptr(out), N, H, _stream(stream)), "mla_absorb_q")
    return out


def out_uv(o_lat: torch.Tensor, w_uv: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    N, H, _ = o_lat.shape
    if out is None:
        out = torch.empty((N, H, 128), dtype=torch.bfloat16, device=o_lat.device)
    _check(_lib.mla_out_uv(_ptr(o_lat), _ptr(w_uv), _ptr(out), N, H, _stream(stream)), "mla_out_uv")
    return out


@dataclass
class Fp8Weight:
    """A projection weight as E4M3 codes (uint8) and fp32 block scales [H][4]."""
    codes: torch.Tensor
    scales: torch.Tensor


def quantize_w_uk_fp8(w_uk: torch.Tensor, stream=None) -> Fp8Weight:
    """W_UK bf16 [512][H][128] -> codes [H][512][128] and scales [H][4]."""
    H = w_uk.shape[1]
    codes = torch.empty((H, 512, 128), dtype=torch.uint8, device=w_uk.device)
    scales = torch.empty((H, 4), dtype=torch.float32, device=w_uk.device)
    _check(_lib.mla_quantize_w_uk_fp8(_ptr(w_uk), H, _ptr(codes), _ptr(scales), _stream(stream)),
           "mla_quantize_w_uk_fp8")
    return Fp8Weight(codes, scales)


def quantize_w_uv_fp8(w_uv: torch.Tensor, stream=None) -> Fp8Weight:
    """W_UV bf16 [512][H][128] -> codes [H][128][512] and scales [H][4]."""
    H = w_uv.shape[1]
    codes = torch.empty((H, 128, 512), dtype=torch.uint8, device=w_uv.device)
    scales = torch.empty((H, 4), dtype=torch.float32, device=w_uv.device)
    _check(_lib.mla_quantize_w_uv_fp8(_ptr(w_uv), H, _ptr(codes), _ptr(scales), _stream(stream)),
           "mla_quantize_w_uv_fp8")
    return Fp8Weight(codes, scales)


def quantize_rows_fp8(x: torch.Tensor, stream=None):
    """bf16 [..., cols] -> (codes uint8 [..., cols], scales fp32 [..., cols / 128])."""
    cols = x.shape[-1]
    rows = x.numel() // cols
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty(tuple(x.shape[:-1]) + (cols // 128,), dtype=torch.float32, device=x.device)
    _check(_lib.mla_quantize_rows_fp8(_ptr(x), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)),
           "mla_quantize_rows_fp8")
    return codes, scales


def absorb_q_fp8(q_nope: torch.Tensor, w: Fp8Weight, out: torch.Tensor | None = None, stream=None):
    N, H, _ = q_nope.shape
    if out is None:
        out = torch.empty((N, H, 512), dtype=torch.bfloat16, device=q_nope.device)
    _check(_lib.mla_absorb_q_fp8(_ptr(q_nope), _ptr(w.codes), _ptr(w.scales), _ptr(out), N, H, _stream(stream)),
           "mla_absorb_q_fp8")
    return out


def out_uv_fp8(o_lat: torch.Tensor, w: Fp8Weight, out: torch.Tensor | None = None, stream=None):
    N, H, _ = o_lat.shape
    if out is None:
        out = torch.empty((N, H, 128), dtype=torch.bfloat16, device=o_lat.device)
    _check(_lib.mla_out_uv_fp8(_ptr(o_lat), _ptr(w.codes), _ptr(w.scales), _ptr(out), N, H, _stream(stream)),
           "mla_out_uv_fp8")
    return out


def _sizes(dims, num_clusters, plan_dev, o_part, lse_part):
    """Bytes of a plan's buffer and of the workspaces: the kernels refuse a plan that
    needs more (STATUS_BAD_PLAN).  Raw addresses are taken to have plan_size's sizes."""
    try:
        return plan_dev.nbytes, o_part.nbytes, lse_part.nbytes
    except AttributeError:          # None or an address among them
        bound = plan_size(dims, num_clusters)
        return tuple(0 if t is None else b if isinstance(t, int) else t.nbytes
                     for t, b in zip((plan_dev, o_part, lse_part), bound))


def _decode_attn(what, cache, dims, q_lat, q_rope, kv_pool, block_table, seq_lens, draft_masks, plan_dev, num_clusters,
                 o_part, lse_part, o_lat, lse_out, status, stream):
    plan_bytes, o_bytes, lse_bytes = _sizes(dims, num_clusters, plan_dev, o_part, lse_part)
    _check(_lib.mla_decode_attn_sized(ctypes.byref(dims), CACHE_KINDS[cache], _ptr(q_lat), _ptr(q_rope), _ptr(kv_pool),
                                      _ptr(block_table), _ptr(seq_lens), _ptr(draft_masks), _ptr(plan_dev), plan_bytes,
                                      num_clusters, _ptr(o_part), o_bytes, _ptr(lse_part), lse_bytes, _ptr(o_lat),
                                      _ptr(lse_out), _ptr(status), _stream(stream)), what)


def decode_attn(dims, q_lat, q_rope, kv_pool, block_table, seq_lens, plan_dev, num_clusters,
                o_part, lse_part, o_lat, lse_out=None, status=None, stream=None):
    _decode_attn("mla_decode_attn", "bf16", dims, q_lat, q_rope, kv_pool, block_table, seq_lens, None, plan_dev,
                 num_clusters, o_part, lse_part, o_lat, lse_out, status, stream)


def decode_attn_tree(dims, q_lat, q_rope, kv_pool, block_table, seq_lens, draft_masks, plan_dev, num_clusters,
                     o_part, lse_part, o_lat, lse_out=None, status=None, stream=None):
    """decode_attn for drafts that form a tree: ``draft_masks`` int32 [B][s_q]
    (device), bit j of row i = draft j visible to query i (dims.causal must be 0)."""
    if draft_masks is None:         # without masks _decode_attn would run the causal kernel
        raise MlaError(MLA_ERR_INVALID_ARG, "mla_decode_attn_tree: draft_masks is None")
    _decode_attn("mla_decode_attn_tree", "bf16", dims, q_lat, q_rope, kv_pool, block_table, seq_lens, draft_masks,
                 plan_dev, num_clusters, o_part, lse_part, o_lat, lse_out, status, stream)


FP8_ROW_BYTES = 656   # 512 E4M3 codes | 4 fp32 block scales | 64 bf16 k_rope


def decode_attn_fp8cache(dims, q_lat, q_rope, kv_pool_fp8, block_table, seq_lens, plan_dev, num_clusters,
                         o_part, lse_part, o_lat, lse_out=None, status=None, stream=None):
    """decode_attn on an FP8 latent cache: ``kv_pool_fp8`` uint8
    [num_blocks][64][656] as :func:`kv_quantize_fp8` writes it."""
    _decode_attn("mla_decode_attn_fp8cache", "fp8", dims, q_lat, q_rope, kv_pool_fp8, block_table, seq_lens, None,
                 plan_dev, num_clusters, o_part, lse_part, o_lat, lse_out, status, stream)


def kv_quantize_fp8(kv, slots, kv_pool_fp8, status=None, stream=None):
    """bf16 cache rows ``kv`` [n][576] -> slots ``slots`` (int32 [n], block * 64 +
    row) of the FP8 pool (uint8 [num_blocks][64][656])."""
    n = kv.numel() // 576
    _check(_lib.mla_kv_quantize_fp8(_ptr(kv), _ptr(slots), n, _ptr(kv_pool_fp8), kv_pool_fp8.shape[0],
                                    _ptr(status), _stream(stream)), "mla_kv_quantize_fp8")
    return kv_pool_fp8


def fp8_pool_from(kv_pool, stream=None):
    """The FP8 copy of a whole bf16 pool [num_blocks][64][576] (every slot quantised)."""
    nb = kv_pool.shape[0]
    pool8 = torch.empty((nb, 64, FP8_ROW_BYTES), dtype=torch.uint8, device=kv_pool.device)
    slots = torch.arange(nb * 64, dtype=torch.int32, device=kv_pool.device)
    return kv_quantize_fp8(kv_pool.reshape(nb * 64, 576), slots, pool8, stream=stream)


FP4_ROW_BYTES = 416   # 256 bytes of E2M1 codes | 16 fp16 group scales | 64 bf16 k_rope


def decode_attn_fp4cache(dims, q_lat, q_rope, kv_pool_fp4, block_table, seq_lens, plan_dev, num_clusters,
                         o_part, lse_part, o_lat, lse_out=None, status=None, stream=None):
    """decode_attn on a 4-bit latent cache: ``kv_pool_fp4`` uint8
    [num_blocks][64][416] as :func:`kv_quantize_fp4` writes it."""
    N, H = dims.B * dims.s_q, dims.n_heads
    with _on(q_lat, q_rope, kv_pool_fp4, block_table, seq_lens, plan_dev, o_part, lse_part, o_lat, lse_out, status):
        _check(_lib.mla_decode_attn_sized(
            ctypes.byref(dims), CACHE_KINDS["fp4"], _arg(q_lat, "q_lat", _BF16, N, H, 512),
            _arg(q_rope, "q_rope", _BF16, N, H, 64),
            _arg(kv_pool_fp4, "kv_pool_fp4", _U8, dims.num_blocks, 64, FP4_ROW_BYTES),
            _arg(block_table, "block_table", _I32, dims.B, dims.max_blocks_per_seq),
            _arg(seq_lens, "seq_lens", _I32, dims.B), None, _vec(plan_dev, "plan_dev", _I32),
            0 if plan_dev is None else plan_dev.nbytes, num_clusters, _vec(o_part, "o_part", _F32),
            0 if o_part is None else o_part.nbytes, _vec(lse_part, "lse_part", _F32),
            0 if lse_part is None else lse_part.nbytes, _arg(o_lat, "o_lat", _BF16, N, H, 512), _arg(lse_out, "lse_out", _F32, N, H),
            _vec(status, "status", _I32), _stream(stream)), "mla_decode_attn_fp4cache")


def kv_quantize_fp4(kv, slots, kv_pool_fp4, status=None, stream=None):
    """bf16 cache rows ``kv`` [n][576] -> slots ``slots`` (int32 [n], block * 64 +
    row; -1 is padding) of the 4-bit pool (uint8 [num_blocks][64][416])."""
    nb, n = kv_pool_fp4.shape[0], slots.shape[0]
    with _on(kv_pool_fp4, kv, slots, status):
        _check(_lib.mla_kv_quantize_fp4(_arg(kv, "kv", _BF16, n, 576), _arg(slots, "slots", _I32, n), n,
                                        _arg(kv_pool_fp4, "kv_pool_fp4", _U8, nb, 64, FP4_ROW_BYTES),
                                        nb, _vec(status, "status", _I32), _stream(stream)), "mla_kv_quantize_fp4")
    return kv_pool_fp4


def kv_dequantize_fp4(kv_pool_fp4, slots, kv=None, status=None, stream=None):
    """Slots of a 4-bit pool -> bf16 rows ``kv`` [n][576] (rows of padding and of
    bad slots are left as they were; zeros when ``kv`` is made here)."""
    nb, n = kv_pool_fp4.shape[0], slots.shape[0]
    if kv is None:
        with _made_on(stream, kv_pool_fp4.device):
            kv = torch.zeros((n, 576), dtype=torch.bfloat16, device=kv_pool_fp4.device)
    with _on(kv_pool_fp4, kv, slots, status):
        _check(_lib.mla_kv_dequantize_fp4(_arg(kv_pool_fp4, "kv_pool_fp4", _U8, nb, 64, FP4_ROW_BYTES),
                                          _arg(slots, "slots", _I32, n), n, _arg(kv, "kv", _BF16, n, 576),
                                          nb, _vec(status, "status", _I32), _stream(stream)),
               "mla_kv_dequantize_fp4")
    return kv


def fp4_pool_from(kv_pool, stream=None):
    """The 4-bit copy of a whole bf16 pool [num_blocks][64][576] (every slot quantised)."""
    nb = kv_pool.shape[0]
    with _made_on(stream, kv_pool.device):
        pool4 = torch.empty((nb, 64, FP4_ROW_BYTES), dtype=torch.uint8, device=kv_pool.device)
        slots = torch.arange(nb * 64, dtype=torch.int32, device=kv_pool.device)
    return kv_quantize_fp4(kv_pool.reshape(nb * 64, 576), slots, pool4, stream=stream)


@dataclass
class BatchTables:
    """What :func:`build_tables` writes beside the block table (all int32, device)."""
    seq_lens: torch.Tensor    # [B]        cached + new
    cu_new: torch.Tensor      # [B + 1]    new tokens before each request
    slots: torch.Tensor       # [max_new]  block * 64 + row of each new token, -1 behind the last
    positions: torch.Tensor   # [max_new]  its position in its request, -1 behind the last
    free_head: torch.Tensor   # [1]        the next free block

    @classmethod
    def empty(cls, B: int, max_new: int, device="cuda") -> "BatchTables":
        buf = torch.empty(2 * B + 2 + 2 * max_new, dtype=torch.int32, device=device)
        lens, cu, slots, pos, head = buf.split([B, B + 1, max_new, max_new, 1])
        return cls(lens, cu, slots, pos, head)


def build_tables(cached_lens, new_lens, block_table, free_blocks, free_head, max_new: int, num_blocks: int,
                 out: BatchTables | None = None, status=None, stream=None, held_pages=None) -> BatchTables:
    """Block tables and slot maps of a step on the GPU, from the requests' lengths.

    ``cached_lens``, ``new_lens`` int32 [B]; ``block_table`` int32 [B][max_blocks]
    gains the new pages' blocks, taken from ``free_blocks[free_head[0]:]`` in
    request order.  ``out.seq_lens`` may be ``cached_lens`` and
    ``out.free_head`` may be ``free_head``: a captured step then moves on by itself.

    ``held_pages`` (int32 [B], updated in place; zeros for new requests) counts the
    pages whose blocks each row of the table holds.  Give it where ``cached_lens`` can
    fall (rejected drafts): without it a request is taken to hold the pages of its
    cached tokens only, and a page that only the rejected tokens reached is given a
    second block while the first is lost.
    """
    B, width = cached_lens.shape[0], block_table.shape[-1]
    i32 = torch.int32
    if out is None:
        with _made_on(stream, block_table.device):
            out = BatchTables.empty(B, max_new, block_table.device)
        at = out.seq_lens.data_ptr()              # the five arrays of empty(), one behind the other
        lens, cu, slots, positions = at, at + 4 * B, at + 8 * B + 4, at + 8 * B + 4 + 4 * max_new
        head_out = positions + 4 * max_new
        device = _on(block_table, cached_lens, new_lens, free_blocks, free_head, status, held_pages)
    else:
        lens, cu = _arg(out.seq_lens, "seq_lens", i32, B), _arg(out.cu_new, "cu_new", i32, B + 1)
        slots, positions = _arg(out.slots, "slots", i32, max_new), _arg(out.positions, "positions", i32, max_new)
        head_out = _arg(out.free_head, "free_head", i32, 1)
        device = _on(block_table, cached_lens, new_lens, free_blocks, free_head, status, held_pages, out.seq_lens,
                     out.cu_new, out.slots, out.positions, out.free_head)
    with device:
        _check(_lib.mla_build_tables_held(
            B, _arg(cached_lens, "cached_lens", i32, B), _arg(new_lens, "new_lens", i32, B), width,
            _arg(block_table, "block_table", i32, B, width), _arg(held_pages, "held_pages", i32, B), _vec(free_blocks, "free_blocks", i32), free_blocks.numel(),
            _arg(free_head, "free_head", i32, 1), num_blocks, max_new, lens, cu, slots, positions, head_out,
            _vec(status, "status", i32), _stream(stream)), "mla_build_tables")
    return out


@functools.lru_cache(maxsize=256)
def _plan_words(rows: int, num_clusters: int) -> int:
    return plan_size(make_dims(rows, 1, 1, 1, 1), num_clusters)[0] // 4


def plan_device(dims: MlaDims, seq_lens, num_clusters: int, plan_dev=None, status=None, stream=None):
    """:func:`plan` made on the GPU from device ``seq_lens`` (int32 [B]; 0 is a
    padded row without work): the same words, as an int32 device tensor."""
    if plan_dev is None:
        with _made_on(stream, seq_lens.device):
            plan_dev = torch.empty(_plan_words(dims.B * dims.s_q, num_clusters), dtype=torch.int32, device=seq_lens.device)
    with _on(seq_lens, plan_dev, status):
        _check(_lib.mla_plan_device(ctypes.byref(dims), _arg(seq_lens, "seq_lens", _I32, dims.B), num_clusters,
                                    _vec(plan_dev, "plan_dev", _I32), 4 * plan_dev.numel(), _vec(status, "status", _I32),
                                    _stream(stream)), "mla_plan_device")
    return plan_dev


_POOL_ROWS = {"bf16": (torch.bfloat16, 576), "fp8": (torch.uint8, FP8_ROW_BYTES), "fp4": (torch.uint8, FP4_ROW_BYTES)}


def summarize_pages(kv_pool, blocks, codes, scales, kv_cache: str = "bf16", status=None, stream=None):
    """8-bit summaries (means) of full pages ``blocks`` (int32 [n]; -1 is
    skipped) of a pool of kind ``kv_cache``, into ``codes`` int8 [num_blocks][576]
    and ``scales`` fp32 [num_blocks]."""
    if kv_cache not in CACHE_KINDS:
        raise ValueError("kv_cache must be 'bf16', 'fp8' or 'fp4'")
    nb, n = kv_pool.shape[0], blocks.shape[0]
    dtype, row = _POOL_ROWS[kv_cache]
    with _on(kv_pool, blocks, codes, scales, status):
        _check(_lib.mla_summarize_pages(_arg(kv_pool, "kv_pool", dtype, nb, 64, row), CACHE_KINDS[kv_cache],
                                        _arg(blocks, "blocks", _I32, n), n, nb,
                                        _arg(codes, "codes", torch.int8, nb, 576),
                                        _arg(scales, "scales", _F32, nb), _vec(status, "status", _I32), _stream(stream)),
               "mla_summarize_pages")
    return codes, scales


def select_pages(dims: MlaDims, q_lat, q_rope, codes, scales, block_table, seq_lens, k: int, scores, sel_table,
                 sel_lens, sel_pages=None, n_first: int = 1, n_recent: int = 1, status=None, stream=None,
                 plan_dev=None, num_clusters: int = 0):
    """The pages each query row attends to: all of its pages if there are at most
    ``k``, else the first ``n_first``, the last ``n_recent`` and the best scores.
    Writes ``sel_table`` int32 [N][k] (a block table with one row per query),
    ``sel_lens`` int32 [N] and, if given, ``sel_pages`` int32 [N][k] and
    ``plan_dev`` (the plan of the selection for ``num_clusters`` clusters)."""
    N, H = dims.B * dims.s_q, dims.n_heads
    i32 = torch.int32
    with _on(q_lat, q_rope, codes, scales, block_table, seq_lens, scores, sel_table, sel_lens, sel_pages, plan_dev,
             status):
        _check(_lib.mla_select_pages(
            ctypes.byref(dims), _arg(q_lat, "q_lat", _BF16, N, H, 512),
            _arg(q_rope, "q_rope", _BF16, N, H, 64), _arg(codes, "codes", torch.int8, dims.num_blocks, 576),
            _arg(scales, "scales", _F32, dims.num_blocks),
            _arg(block_table, "block_table", i32, dims.B, dims.max_blocks_per_seq),
            _arg(seq_lens, "seq_lens", i32, dims.B), k, n_first, n_recent,
            _arg(scores, "scores", _F32, N, dims.max_blocks_per_seq), _arg(sel_table, "sel_table", i32, N, k),
            _arg(sel_lens, "sel_lens", i32, N), _arg(sel_pages, "sel_pages", i32, N, k), num_clusters,
            _vec(plan_dev, "plan_dev", i32), 0 if plan_dev is None else 4 * plan_dev.numel(),
            _vec(status, "status", i32), _stream(stream)), "mla_select_pages")
    return sel_table, sel_lens, sel_pages


def combine(dims, plan_dev, o_part, lse_part, o_lat, lse_out=None, stream=None, status=None):
    plan_bytes, o_bytes, lse_bytes = _sizes(dims, 4096, plan_dev, o_part, lse_part)
    _check(_lib.mla_combine_sized(ctypes.byref(dims), _ptr(plan_dev), plan_bytes, _ptr(o_part), o_bytes, _ptr(lse_part),
                                  lse_bytes, _ptr(o_lat), _ptr(lse_out), _ptr(status), _stream(stream)), "mla_combine")


def qkv_a_proj(x, w_qkv_a, c_q=None, kv_a=None, stream=None):
    """Fused down-projections: x [N][7168] -> c_q [N][1536], kv_a [N][576]."""
    N = x.shape[0]
    if c_q is None:
        c_q = torch.empty((N, 1536), dtype=torch.bfloat16, device=x.device)
    if kv_a is None:
        kv_a = torch.empty((N, 576), dtype=torch.bfloat16, device=x.device)
    _check(_lib.mla_qkv_a_proj(_ptr(x), _ptr(w_qkv_a), _ptr(c_q), _ptr(kv_a), N, _stream(stream)), "mla_qkv_a_proj")
    return c_q, kv_a


def q_up_absorb(c_q, w_uq, w_uk, q_lat=None, q_rope=None, stream=None):
    """c_q [N][1536] -> q_lat [N][h][512] (through W_UQ then W_UK) and q_rope [N][h][64]."""
    N, H = c_q.shape[0], w_uq.shape[1]
    if q_lat is None:
        q_lat = torch.empty((N, H, 512), dtype=torch.bfloat16, device=c_q.device)
    if q_rope is None:
        q_rope = torch.empty((N, H, 64), dtype=torch.bfloat16, device=c_q.device)
    _check(_lib.mla_q_up_absorb(_ptr(c_q), _ptr(w_uq), _ptr(w_uk), _ptr(q_lat), _ptr(q_rope), N, H, _stream(stream)),
           "mla_q_up_absorb")
    return q_lat, q_rope


def prefill_up_proj(kv_pool, block_row, T, w_uk, w_uv, k_out=None, v_out=None, stream=None):
    """K and V [T][h][128] of one sequence's first T cached tokens (order 1)."""
    H = w_uk.shape[1]
    if k_out is None:
        k_out = torch.empty((T, H, 128), dtype=torch.bfloat16, device=kv_pool.device)
    if v_out is None:
        v_out = torch.empty((T, H, 128), dtype=torch.bfloat16, device=kv_pool.device)
    _check(_lib.mla_prefill_up_proj(_ptr(kv_pool), _ptr(block_row), T, kv_pool.shape[0], _ptr(w_uk), _ptr(w_uv), H,
                                    _ptr(k_out), _ptr(v_out), _stream(stream)), "mla_prefill_up_proj")
    return k_out, v_out


def prefill_attn(q_nope, q_rope, k, v, kv_pool, block_row, T, scale=None, out=None, lse=None, stream=None):
    """Causal attention of the last s = q_nope.shape[0] of T cached tokens."""
    s, H, _ = q_nope.shape
    if scale is None:
        scale = 1.0 / math.sqrt(128 + 64)
    if out is None:
        out = torch.empty((s, H, 128), dtype=torch.bfloat16, device=q_nope.device)
    _check(_lib.mla_prefill_attn(_ptr(q_nope), _ptr(q_rope), _ptr(k), _ptr(v), _ptr(kv_pool), _ptr(block_row), T, s,
                                 H, kv_pool.shape[0], float(scale), _ptr(out), _ptr(lse), _stream(stream)),
           "mla_prefill_attn")
    return out


def prefill(q_nope, q_rope, kv_pool, block_row, T, w_uk, w_uv, scale=None, lse=None, stream=None):
    """Prefill (s = T) or a prefill chunk (s < T) of one sequence in order 1."""
    k, v = prefill_up_proj(kv_pool, block_row, T, w_uk, w_uv, stream=stream)
    return prefill_attn(q_nope, q_rope, k, v, kv_pool, block_row, T, scale=scale, lse=lse, stream=stream)


def noalloc_scratch_bytes() -> int:
    """Size of the library-owned device array used by ``decode_attn_combine_noalloc``."""
    return _lib.mla_noalloc_scratch_bytes()


def decode_attn_combine_noalloc(dims, q_lat, q_rope, kv_pool, block_table, seq_lens, plan_host: np.ndarray,
                                num_clusters, o_lat, lse_out=None, status=None, stream=None):
    """Attention + split merge with no caller workspace and no device allocation.

    For callers that may not allocate device memory (e.g. a runtime that has
    pre-reserved HBM for its KV cache): ``plan_host`` is the host plan from
    :func:`plan`; the plan copy and the partial outputs live in a fixed array
    inside the library (see :func:`noalloc_scratch_bytes`).
    """
    pl = np.ascontiguousarray(plan_host, dtype=np.int32)
    _check(_lib.mla_decode_attn_combine_noalloc(ctypes.byref(dims), _ptr(q_lat), _ptr(q_rope), _ptr(kv_pool),
                                                _ptr(block_table), _ptr(seq_lens), pl.ctypes.data, pl.nbytes,
                                                num_clusters, _ptr(o_lat), _ptr(lse_out), _ptr(status),
                                                _stream(stream)), "mla_decode_attn_combine_noalloc")


def debug_gather_pages(kv_pool, block_table, b, n_pages, max_blocks, num_blocks, out, status=None,
                       stream=None):
    _check(_lib.mla_debug_gather_pages(_ptr(kv_pool), _ptr(block_table), b, n_pages, max_blocks,
                                       num_blocks, _ptr(out), _ptr(status), _stream(stream)),
           "mla_debug_gather_pages")


@dataclass
class DecodeOutputs:
    out: torch.Tensor        # bf16 [N][h][128]
    q_lat: torch.Tensor      # bf16 [N][h][512]
    o_lat: torch.Tensor      # bf16 [N][h][512]
    lse: torch.Tensor        # fp32 [N][h]
    status: torch.Tensor     # int32 [1]


class Decoder:
    """One decode batch shape: plan, workspace and output buffers made once, then
    ``run()`` enqueues absorb -> attention -> combine -> out_uv on the stream.

    Buffers are allocated here by torch (the library allocates nothing).
    """

    def __init__(self, seq_lens, s_q: int, n_heads: int, max_blocks: int, num_blocks: int,
                 device="cuda", scale=None, causal=True, num_clusters: int | None = None,
                 kv_cache: str = "bf16"):
        """``kv_cache``: "bf16" (pool [num_blocks][64][576] bf16), "fp8" (pool
        uint8 [num_blocks][64][656], see :func:`kv_quantize_fp8`) or "fp4" (pool
        uint8 [num_blocks][64][416], see :func:`kv_quantize_fp4`)."""
        if kv_cache not in CACHE_KINDS:
            raise ValueError("kv_cache must be 'bf16', 'fp8' or 'fp4'")
        self.kv_cache = kv_cache
        self.seq_lens_host = np.asarray(seq_lens, dtype=np.int32)
        self.B = len(self.seq_lens_host)
        self.s_q, self.H = s_q, n_heads
        self.N = self.B * s_q
        self.dims = make_dims(self.B, s_q, n_heads, max_blocks, num_blocks, scale, causal)
        self.num_clusters = num_clusters or max_clusters()
        self.plan_host, self.num_slots = plan(self.dims, self.seq_lens_host, self.num_clusters)
        dev = torch.device(device)
        self.plan_dev = torch.from_numpy(self.plan_host).to(dev)
        self.seq_lens_dev = torch.from_numpy(self.seq_lens_host).to(dev)
        slots = max(self.num_slots, 1)
        self.o_part = torch.empty(slots * n_heads * 512, dtype=torch.float32, device=dev)   # internal layout
        self.lse_part = torch.empty((slots, n_heads), dtype=torch.float32, device=dev)
        self.q_lat = torch.empty((self.N, n_heads, 512), dtype=torch.bfloat16, device=dev)
        self.o_lat = torch.empty((self.N, n_heads, 512), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((self.N, n_heads), dtype=torch.float32, device=dev)
        self.out = torch.empty((self.N, n_heads, 128), dtype=torch.bfloat16, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.fp8_uk: Fp8Weight | None = None
        self.fp8_uv: Fp8Weight | None = None

    def use_fp8_projections(self, w_uk, w_uv, stream=None):
        """Run the two projections as FP8 block-quantised BMMs from now on:
        W_UK and W_UV are quantised once here (their bf16 copies passed to
        run() are then not read)."""
        self.fp8_uk = quantize_w_uk_fp8(w_uk, stream)
        self.fp8_uv = quantize_w_uv_fp8(w_uv, stream)

    def run(self, q_nope, q_rope, kv_pool, block_table, w_uk, w_uv, stream=None,
            draft_masks=None) -> DecodeOutputs:
        """``draft_masks`` (device int32 [B][s_q], only with causal=False): the
        drafts form a tree, see :func:`decode_attn_tree`."""
        if self.fp8_uk is not None:
            absorb_q_fp8(q_nope, self.fp8_uk, self.q_lat, stream)
        else:
            absorb_q(q_nope, w_uk, self.q_lat, stream)
        if draft_masks is not None and self.kv_cache != "bf16":
            raise ValueError("draft-tree masks need the bf16 cache")
        if self.kv_cache != "bf16":
            attn = decode_attn_fp8cache if self.kv_cache == "fp8" else decode_attn_fp4cache
            attn(self.dims, self.q_lat, q_rope, kv_pool, block_table, self.seq_lens_dev, self.plan_dev,
                 self.num_clusters, self.o_part, self.lse_part, self.o_lat, self.lse, self.status, stream)
        elif draft_masks is not None:
            decode_attn_tree(self.dims, self.q_lat, q_rope, kv_pool, block_table, self.seq_lens_dev, draft_masks,
                             self.plan_dev, self.num_clusters, self.o_part, self.lse_part, self.o_lat,
                             self.lse, self.status, stream)
        else:
            decode_attn(self.dims, self.q_lat, q_rope, kv_pool, block_table, self.seq_lens_dev,
                        self.plan_dev, self.num_clusters, self.o_part, self.lse_part, self.o_lat,
                        self.lse, self.status, stream)
        if self.num_slots > 0:
            combine(self.dims, self.plan_dev, self.o_part, self.lse_part, self.o_lat, self.lse, stream)
        if self.fp8_uv is not None:
            out_uv_fp8(self.o_lat, self.fp8_uv, self.out, stream)
        else:
            out_uv(self.o_lat, w_uv, self.out, stream)
        return DecodeOutputs(self.out, self.q_lat, self.o_lat, self.lse, self.status)

    @property
    def launches_per_step(self) -> int:
        return 4 if self.num_slots > 0 else 3


@dataclass
class SparseOutputs:
    o_lat: torch.Tensor      # bf16 [N][h][512]
    lse: torch.Tensor        # fp32 [N][h], over the chosen pages
    pages: torch.Tensor      # int32 [N][k] page numbers, -1 behind the last
    table: torch.Tensor      # int32 [N][k] their blocks
    lens: torch.Tensor       # int32 [N] keys attended
    status: torch.Tensor     # int32 [1]


class SparseAttention:
    """Attention of each query over the pages a cheap score picks, for one batch
    shape: :func:`select_pages` (which makes the plan of its selection too), the
    decode kernel of the cache's kind and :func:`combine`.

    Lengths stay on the device, so one captured ``run()`` serves a batch as it
    grows, and rows of length 0 (a padded batch) are left as they were.  The
    buffers are made here; one object's runs must not overlap.
    """

    def __init__(self, B: int, s_q: int, n_heads: int, max_blocks: int, num_blocks: int, k: int, n_first: int = 1,
                 n_recent: int = 1, kv_cache: str = "bf16", device="cuda", scale=None, causal=True,
                 num_clusters: int | None = None):
        if kv_cache not in CACHE_KINDS:
            raise ValueError("kv_cache must be 'bf16', 'fp8' or 'fp4'")
        if n_first < 0 or n_recent < 1 or n_first + n_recent > k:
            raise ValueError("n_first >= 0, n_recent >= 1 and n_first + n_recent <= k are needed")
        self.kv_cache, self.k, self.n_first, self.n_recent = kv_cache, k, n_first, n_recent
        self.num_clusters = num_clusters or max_clusters()
        N = B * s_q
        self.dims = make_dims(B, s_q, n_heads, max_blocks, num_blocks, scale, causal)
        self.row_dims = make_dims(N, 1, n_heads, k, num_blocks, scale)   # a row is a sequence of its chosen pages
        plan_bytes, o_bytes, lse_bytes = plan_size(self.row_dims, self.num_clusters)
        dev = torch.device(device)
        new = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device=dev)
        self.scores = new(N, max_blocks, dtype=torch.float32)
        self.table, self.lens, self.pages = new(N, k), new(N), new(N, k)
        self.plan_dev = new(plan_bytes // 4)
        self.o_part, self.lse_part = new(o_bytes // 4, dtype=torch.float32), new(lse_bytes // 4, dtype=torch.float32)
        self.o_lat = new(N, n_heads, 512, dtype=torch.bfloat16)
        self.lse = new(N, n_heads, dtype=torch.float32)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._out = SparseOutputs(self.o_lat, self.lse, self.pages, self.table, self.lens, self.status)
        # the arguments of the three calls that stay the same from run to run
        self._attn = {"bf16": _lib.mla_decode_attn, "fp8": _lib.mla_decode_attn_fp8cache,
                      "fp4": _lib.mla_decode_attn_fp4cache}[kv_cache]
        at = lambda t: t.data_ptr()
        self._refs = ctypes.byref(self.dims), ctypes.byref(self.row_dims)
        self._selection = (k, n_first, n_recent, at(self.scores), at(self.table), at(self.lens), at(self.pages),
                           self.num_clusters, at(self.plan_dev), plan_bytes, at(self.status))
        self._attention = (at(self.table), at(self.lens), at(self.plan_dev), self.num_clusters, at(self.o_part),
                           at(self.lse_part), at(self.o_lat), at(self.lse), at(self.status))
        self._merge = at(self.plan_dev), at(self.o_part), at(self.lse_part), at(self.o_lat), at(self.lse)

    def run(self, q_lat, q_rope, kv_pool, codes, scales, block_table, seq_lens, stream=None) -> SparseOutputs:
        """``codes`` and ``scales``: the summaries of the pool's full pages
        (:func:`summarize_pages`); ``seq_lens`` int32 [B] on the device.  The outputs are the
        object's own buffers."""
        d = self.dims
        N, H, nb = d.B * d.s_q, d.n_heads, d.num_blocks
        dtype, row = _POOL_ROWS[self.kv_cache]
        with _on(self.o_lat, q_lat, q_rope, kv_pool, codes, scales, block_table, seq_lens):
            s = _stream(stream)
            queries = _arg(q_lat, "q_lat", torch.bfloat16, N, H, 512), _arg(q_rope, "q_rope", torch.bfloat16, N, H, 64)
            pool = _arg(kv_pool, "kv_pool", dtype, nb, 64, row)
            whole, rows = self._refs
            _check(_lib.mla_select_pages(
                whole, *queries, _arg(codes, "codes", torch.int8, nb, 576), _arg(scales, "scales", torch.float32, nb),
                _arg(block_table, "block_table", torch.int32, d.B, d.max_blocks_per_seq),
                _arg(seq_lens, "seq_lens", torch.int32, d.B), *self._selection, s), "mla_select_pages")
            _check(self._attn(rows, *queries, pool, *self._attention, s), "attention over the selection")
            _check(_lib.mla_combine(rows, *self._merge, s), "mla_combine")
        return self._out


class GraphedStep:
    """One decode step from host memory to host memory, replayed as a CUDA graph.

    For a serving loop with a fixed batch shape: the step's inputs live in
    pinned host buffers (``q_nope``, ``q_rope``, ``block_table``); ``run()``
    replays one graph that copies them to the device, runs absorb ->
    attention -> combine -> out_uv, and copies ``out`` back to the pinned
    ``out`` buffer.  The graph fixes every pointer, so the cache pool, the
    weights and the decoder's buffers must outlive this object; refill the
    host buffers in place between calls.
    """

    def __init__(self, decoder: Decoder, kv_pool, w_uk, w_uv, stream=None):
        dev = kv_pool.device
        N, H = decoder.N, decoder.H
        self.decoder = decoder
        self.q_nope = torch.zeros((N, H, 128), dtype=torch.bfloat16).pin_memory()
        self.q_rope = torch.zeros((N, H, 64), dtype=torch.bfloat16).pin_memory()
        self.block_table = torch.zeros((decoder.B, decoder.dims.max_blocks_per_seq), dtype=torch.int32).pin_memory()
        self.out = torch.empty((N, H, 128), dtype=torch.bfloat16).pin_memory()
        self._q_nope = torch.empty(self.q_nope.shape, dtype=torch.bfloat16, device=dev)
        self._q_rope = torch.empty(self.q_rope.shape, dtype=torch.bfloat16, device=dev)
        self._bt = torch.empty(self.block_table.shape, dtype=torch.int32, device=dev)
        self._args = (kv_pool, w_uk, w_uv)
        self.graph = torch.cuda.CUDAGraph()
        s = stream or torch.cuda.Stream(device=dev)
        s.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(s):
            self._body()                      # warm-up outside capture (lazy library set-up)
            torch.cuda.synchronize(dev)
            with torch.cuda.graph(self.graph, stream=s):
                self._body()
        torch.cuda.synchronize(dev)

    def _body(self):
        kv_pool, w_uk, w_uv = self._args
        self._q_nope.copy_(self.q_nope, non_blocking=True)
        self._q_rope.copy_(self.q_rope, non_blocking=True)
        self._bt.copy_(self.block_table, non_blocking=True)
        r = self.decoder.run(self._q_nope, self._q_rope, kv_pool, self._bt, w_uk, w_uv)
        self.out.copy_(r.out, non_blocking=True)

    def run(self, sync: bool = True) -> torch.Tensor:
        """Replays the step on the current stream; returns the pinned ``out`` buffer."""
        self.graph.replay()
        if sync:
            torch.cuda.current_stream().synchronize()
        return self.out

    @property
    def h2d_bytes(self) -> int:
        return self.q_nope.nbytes + self.q_rope.nbytes + self.block_table.nbytes

    @property
    def d2h_bytes(self) -> int:
        return self.out.nbytes


class StreamedDecoder:
    """Back-to-back decode steps from pinned host memory to pinned host memory,
    with the copies of one step overlapping the kernels of its neighbours.

    ``depth`` input/output sets rotate: step k uses set i = k % depth.  The user
    fills ``host_in[i]`` (q_nope, q_rope, block_table), calls ``submit()``, and
    reads ``host_out[i]`` once ``ready(i)`` (or ``wait(i)``) says the step's
    device-to-host copy is done.  Three streams carry the work: host-to-device
    copies, the kernels (one CUDA graph per set: absorb -> attention ->
    combine -> out_uv, then a device copy of the output into the set's
    buffer), and device-to-host copies; events keep each set's buffers from
    being overwritten while still in use.  The decoder's scratch buffers are
    shared, so the kernels of consecutive steps run one after another.
    """

    def __init__(self, decoder: Decoder, kv_pool, w_uk, w_uv, depth: int = 2):
        dev = kv_pool.device
        N, H, B = decoder.N, decoder.H, decoder.B
        mb = decoder.dims.max_blocks_per_seq
        self.depth = depth
        self.host_in = [(torch.zeros((N, H, 128), dtype=torch.bfloat16).pin_memory(),
                         torch.zeros((N, H, 64), dtype=torch.bfloat16).pin_memory(),
                         torch.zeros((B, mb), dtype=torch.int32).pin_memory()) for _ in range(depth)]
        self.host_out = [torch.empty((N, H, 128), dtype=torch.bfloat16).pin_memory() for _ in range(depth)]
        self._dev_in = [(torch.empty((N, H, 128), dtype=torch.bfloat16, device=dev),
                         torch.empty((N, H, 64), dtype=torch.bfloat16, device=dev),
                         torch.empty((B, mb), dtype=torch.int32, device=dev)) for _ in range(depth)]
        self._dev_out = [torch.empty((N, H, 128), dtype=torch.bfloat16, device=dev) for _ in range(depth)]
        self._s_in, self._s_cmp, self._s_out = (torch.cuda.Stream(device=dev) for _ in range(3))
        self._ev_in = [torch.cuda.Event() for _ in range(depth)]
        self._ev_cmp = [torch.cuda.Event() for _ in range(depth)]
        self._ev_out = [torch.cuda.Event() for _ in range(depth)]
        self._graphs = []
        self._s_cmp.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(self._s_cmp):
            for i in range(depth):
                qn, qr, bt = self._dev_in[i]
                qn.zero_(); qr.zero_(); bt.zero_()
                decoder.run(qn, qr, kv_pool, bt, w_uk, w_uv)   # warm-up outside capture
                torch.cuda.synchronize(dev)
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=self._s_cmp):
                    r = decoder.run(qn, qr, kv_pool, bt, w_uk, w_uv)
                    self._dev_out[i].copy_(r.out)
                self._graphs.append(g)
        torch.cuda.synchronize(dev)
        self.steps = 0

    def submit(self) -> int:
        """Enqueues the next step on the next set; returns the set index."""
        i = self.steps % self.depth
        reuse = self.steps >= self.depth
        if reuse:   # this set's device inputs are free once its previous step's kernels finished
            self._s_in.wait_event(self._ev_cmp[i])
        with torch.cuda.stream(self._s_in):
            for d, h in zip(self._dev_in[i], self.host_in[i]):
                d.copy_(h, non_blocking=True)
            self._ev_in[i].record(self._s_in)
        self._s_cmp.wait_event(self._ev_in[i])
        if reuse:   # and its device output once its previous copy back finished
            self._s_cmp.wait_event(self._ev_out[i])
        with torch.cuda.stream(self._s_cmp):
            self._graphs[i].replay()
            self._ev_cmp[i].record(self._s_cmp)
        self._s_out.wait_event(self._ev_cmp[i])
        with torch.cuda.stream(self._s_out):
            self.host_out[i].copy_(self._dev_out[i], non_blocking=True)
            self._ev_out[i].record(self._s_out)
        self.steps += 1
        return i

    def input_free(self, i: int) -> bool:
        """``host_in[i]`` may be refilled once its last host-to-device copy is done."""
        return self._ev_in[i].query()

    def ready(self, i: int) -> bool:
        return self._ev_out[i].query()

    def wait(self, i: int) -> torch.Tensor:
        self._ev_out[i].synchronize()
        return self.host_out[i]

    @property
    def streams(self):
        return self._s_in, self._s_cmp, self._s_out


def decode(q_nope, q_rope, kv_pool, block_table, seq_lens, w_uk, w_uv, s_q=1, scale=None,
           causal=True, num_clusters=None) -> DecodeOutputs:
    """One-shot absorbed MLA decode on device tensors (see ``Decoder``)."""
    bt = block_table if isinstance(block_table, torch.Tensor) else torch.as_tensor(block_table)
    bt = bt.to(device=kv_pool.device, dtype=torch.int32).contiguous()
    sl = seq_lens.cpu().numpy() if isinstance(seq_lens, torch.Tensor) else np.asarray(seq_lens)
    d = Decoder(sl, s_q, q_nope.shape[1], bt.shape[1], kv_pool.shape[0], kv_pool.device, scale,
                causal, num_clusters)
    return d.run(q_nope, q_rope, kv_pool, bt, w_uk, w_uv)
