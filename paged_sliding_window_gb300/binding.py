"""Thin ctypes binding of libpsw.so (the C ABI declared in include/psw.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, checks dtypes and shapes, and passes raw pointers, sizes and
the current CUDA stream to the C entry point of the same name. All arithmetic
runs in the CUDA kernels of the library; there is no fallback. If the
library cannot be loaded, every call raises ``RuntimeError``.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

PSW_OK = 0
ERRORS = {
    -1: "PSW_ENULL", -2: "PSW_EINVAL_HEADS", -3: "PSW_EINVAL_HDIM", -4: "PSW_EINVAL_SOFTCAP",
    -5: "PSW_EINVAL_WINDOW", -6: "PSW_EINVAL_BLOCKSIZE", -7: "PSW_EINVAL_KEQV",
    -8: "PSW_EINVAL_SCALE", -9: "PSW_EINVAL_NSEQS", -10: "PSW_EWORKSPACE",
    -11: "PSW_ECAPACITY", -12: "PSW_EALIGN", -13: "PSW_EDEVICE", -14: "PSW_ELAUNCH",
    -15: "PSW_ETENSORMAP", -16: "PSW_ESCRATCH", -17: "PSW_EINVAL_ROPE",
    -18: "PSW_EINVAL_LAYERS", -19: "PSW_ENOBLOCKS", -20: "PSW_EBLOCK",
    -21: "PSW_EINVAL_STRIDE",
}
DEVERR_BLOCK_ID, DEVERR_CAPACITY, DEVERR_LENGTH, DEVERR_PIPELINE = 1, 2, 4, 8
DEVERR_NOBLOCKS = 16
EXPORTED = ("psw_workspace_bytes", "kv_cache_write", "attn_decode_paged",
            "attn_prefill_chunked", "psw_get_error", "psw_strerror",
            "attn_decode_paged_noalloc", "qkv_norm_rope_cache_write", "psw_kv_share_map",
            "psw_block_pool_create", "psw_block_pool_destroy", "psw_block_pool_num_free",
            "psw_block_pool_allocate", "psw_block_pool_free", "psw_block_pool_get_cached",
            "psw_block_pool_cache", "psw_block_pool_ref_count", "psw_block_hash",
            "psw_block_pool_admit", "psw_block_pool_commit", "kv_cache_write_fp8",
            "attn_decode_paged_fp8", "psw_testing_stall", "attn_decode_paged_append",
            "psw_latent_workspace_bytes", "latent_norm_rope_cache_write",
            "latent_norm_rope_cache_write_fp8", "attn_decode_latent", "attn_decode_latent_fp8",
            "latent_kv_expand", "latent_kv_expand_fp8", "attn_prefill_latent",
            "block_table_extend", "kv_cache_write_fp4", "kv_cache_read_fp4",
            "psw_fp4_workspace_bytes", "attn_decode_paged_fp4")


class PswLayer(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("window", ctypes.c_int32),
                ("softcap", ctypes.c_float), ("scale", ctypes.c_float),
                ("k_eq_v", ctypes.c_int32), ("block_size", ctypes.c_int32)]


class PswPages(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_blocks", ctypes.c_int64)]


class PswNormRope(ctypes.Structure):
    _fields_ = [("theta", ctypes.c_float), ("partial_rotary_factor", ctypes.c_float),
                ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("v_weight", ctypes.c_void_p)]


class PswLatent(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("latent_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("nope_dim", ctypes.c_int32),
                ("v_dim", ctypes.c_int32), ("window", ctypes.c_int32),
                ("softcap", ctypes.c_float), ("scale", ctypes.c_float),
                ("block_size", ctypes.c_int32)]


class PswLatentNorm(ctypes.Structure):
    _fields_ = [("theta", ctypes.c_float), ("eps", ctypes.c_float),
                ("latent_weight", ctypes.c_void_p)]


class PswError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({strerror(code)})")
        self.code = code


_lib = None
_lock = threading.Lock()


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Loads libpsw.so (building it first if asked and missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(f"libpsw.so not built ({path})")
            path = _build.build()
        lib = ctypes.CDLL(path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        lp = ctypes.POINTER(PswLayer)
        pp = ctypes.POINTER(PswPages)
        lib.psw_workspace_bytes.argtypes = [lp, i32, i32, ctypes.POINTER(sz)]
        lib.kv_cache_write.argtypes = [lp, vp, vp, vp, vp, i32, pp, vp, vp, vp]
        lib.attn_decode_paged.argtypes = [lp, vp, vp, vp, pp, vp, i32, vp, vp, vp, sz, vp]
        lib.attn_prefill_chunked.argtypes = [lp, vp, vp, vp, i32, i32, i32, vp, vp, pp, vp, vp,
                                             vp, sz, vp]
        lib.attn_decode_paged_noalloc.argtypes = [lp, vp, vp, vp, pp, vp, i32, vp, vp, vp]
        lib.attn_decode_paged_noalloc.restype = ctypes.c_int
        lib.qkv_norm_rope_cache_write.argtypes = [lp, ctypes.POINTER(PswNormRope), vp, vp, vp,
                                                  vp, vp, i32, pp, vp, vp, vp, vp]
        lib.qkv_norm_rope_cache_write.restype = ctypes.c_int
        lib.psw_kv_share_map.argtypes = [i32, i32, i32, ctypes.POINTER(i32),
                                         ctypes.POINTER(i32)]
        lib.psw_kv_share_map.restype = ctypes.c_int
        i32p, u64 = ctypes.POINTER(i32), ctypes.c_uint64
        lib.psw_block_pool_create.argtypes = [i64, i32, ctypes.POINTER(vp)]
        lib.psw_block_pool_destroy.argtypes = [vp]
        lib.psw_block_pool_destroy.restype = None
        lib.psw_block_pool_num_free.argtypes = [vp]
        lib.psw_block_pool_num_free.restype = i64
        lib.psw_block_pool_allocate.argtypes = [vp, i32, i32p]
        lib.psw_block_pool_free.argtypes = [vp, i32p, i32]
        lib.psw_block_pool_get_cached.argtypes = [vp, u64, i32p]
        lib.psw_block_pool_cache.argtypes = [vp, i32, u64]
        lib.psw_block_pool_ref_count.argtypes = [vp, i32, i32p]
        lib.psw_block_hash.argtypes = [u64, i32p, i32]
        lib.psw_block_hash.restype = u64
        lib.psw_block_pool_admit.argtypes = [vp, i32p, i32, i32p, i32, i32p]
        lib.psw_block_pool_commit.argtypes = [vp, i32p, i32, i32p]
        for name in ("psw_block_pool_create", "psw_block_pool_allocate", "psw_block_pool_free",
                     "psw_block_pool_get_cached", "psw_block_pool_cache",
                     "psw_block_pool_ref_count", "psw_block_pool_admit",
                     "psw_block_pool_commit"):
            getattr(lib, name).restype = ctypes.c_int
        lib.kv_cache_write_fp8.argtypes = [lp, vp, vp, vp, vp, i32, pp, vp, vp, vp, vp, vp]
        lib.kv_cache_write_fp8.restype = ctypes.c_int
        lib.attn_decode_paged_fp8.argtypes = [lp, vp, vp, vp, vp, vp, pp, vp, i32, vp, vp, vp, sz,
                                              vp]
        lib.attn_decode_paged_fp8.restype = ctypes.c_int
        lib.attn_decode_paged_append.argtypes = [lp, vp, vp, vp, vp, vp, pp, vp, i32, vp, vp, vp,
                                                 sz, vp]
        lib.attn_decode_paged_append.restype = ctypes.c_int
        zp, zn = ctypes.POINTER(PswLatent), ctypes.POINTER(PswLatentNorm)
        lib.psw_latent_workspace_bytes.argtypes = [zp, i32, ctypes.POINTER(sz)]
        write = [zp, zn, vp, i64, vp, i64, i64, vp, vp, i32, i32, pp, vp, i64, i64, vp]
        lib.latent_norm_rope_cache_write.argtypes = write + [vp]
        lib.latent_norm_rope_cache_write_fp8.argtypes = write + [vp, vp]
        lib.attn_decode_latent.argtypes = [zp, vp, vp, pp, vp, i32, vp, vp, vp, sz, vp]
        lib.attn_decode_latent_fp8.argtypes = [zp, vp, vp, vp, pp, vp, i32, vp, vp, vp, sz, vp]
        lib.latent_kv_expand.argtypes = [zp, vp, pp, vp, vp, i32, i32, vp, vp, vp, vp]
        lib.latent_kv_expand_fp8.argtypes = [zp, vp, vp, pp, vp, vp, i32, i32, vp, vp, vp, vp]
        lib.attn_prefill_latent.argtypes = [zp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, i32, vp,
                                            vp, vp]
        for name in ("psw_latent_workspace_bytes", "latent_norm_rope_cache_write",
                     "latent_norm_rope_cache_write_fp8", "attn_decode_latent",
                     "attn_decode_latent_fp8", "latent_kv_expand", "latent_kv_expand_fp8",
                     "attn_prefill_latent"):
            getattr(lib, name).restype = ctypes.c_int
        f32 = ctypes.c_float
        lib.block_table_extend.argtypes = [vp, i32, vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, i32,
                                           vp]
        lib.kv_cache_write_fp4.argtypes = [lp, vp, vp, vp, vp, i32, i32, pp, vp, vp, f32, f32, vp]
        lib.kv_cache_read_fp4.argtypes = [lp, vp, vp, pp, vp, vp, i32, pp, vp, vp, f32, f32, vp]
        lib.psw_fp4_workspace_bytes.argtypes = [lp, i32, ctypes.POINTER(sz)]
        lib.attn_decode_paged_fp4.argtypes = [lp, vp, vp, vp, pp, vp, i32, vp, vp, vp, sz, f32, f32,
                                              vp]
        for name in ("block_table_extend", "kv_cache_write_fp4", "kv_cache_read_fp4",
                     "psw_fp4_workspace_bytes", "attn_decode_paged_fp4"):
            getattr(lib, name).restype = ctypes.c_int
        lib.psw_testing_stall.argtypes = [i32, i32, i32]
        lib.psw_testing_stall.restype = ctypes.c_int
        lib.psw_get_error.argtypes = [vp, ctypes.POINTER(i32)]
        lib.psw_strerror.argtypes = [ctypes.c_int]
        lib.psw_strerror.restype = ctypes.c_char_p
        for name in ("psw_workspace_bytes", "kv_cache_write", "attn_decode_paged",
                     "attn_prefill_chunked", "psw_get_error"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def strerror(code: int) -> str:
    try:
        return load(build_if_missing=False).psw_strerror(int(code)).decode()
    except Exception:
        return ERRORS.get(code, str(code))


def make_layer(layer) -> PswLayer:
    """From any object with the psw_layer_t fields (e.g. workloads.Layer)."""
    return PswLayer(int(layer.n_q_heads), int(layer.n_kv_heads), int(layer.head_dim),
                    int(layer.window), float(layer.softcap), float(layer.scale),
                    int(bool(layer.k_eq_v)), int(getattr(layer, "block_size", 16)))


def make_pages(block_table: torch.Tensor, num_blocks: int) -> PswPages:
    _check(block_table, torch.int32, "block_table")
    pages = PswPages(block_table.data_ptr(), int(block_table.shape[1]), int(num_blocks))
    pages.table = block_table  # keeps the tensor alive as long as its address is held
    return pages


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, dtype, name):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _raise(rc, what):
    if rc != PSW_OK:
        raise PswError(rc, what)


def workspace_bytes(layer, n_seqs: int, max_seq_len: int) -> int:
    out = ctypes.c_size_t(0)
    _raise(load().psw_workspace_bytes(ctypes.byref(make_layer(layer)), int(n_seqs),
                                      int(max_seq_len), ctypes.byref(out)), "psw_workspace_bytes")
    return int(out.value)


WORKSPACE_COUNTER_BYTES = 2048  # PSW_WORKSPACE_COUNTER_BYTES


def alloc_workspace(layer, n_seqs: int, max_seq_len: int, device="cuda") -> torch.Tensor:
    """A caller-owned workspace of the size the library asks for, zero-filled
    once (its counter block must start at zero; calls keep it zero)."""
    return torch.zeros(max(workspace_bytes(layer, n_seqs, max_seq_len), 256), dtype=torch.uint8,
                       device=device)


def kv_cache_write(layer, k, v, cu_new, past_lens, pages: PswPages, k_pool, v_pool,
                   stream=None) -> None:
    for t, n in ((k, "k"), (v, "v"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _check(t, torch.bfloat16, n)
    _check(cu_new, torch.int32, "cu_new")
    _check(past_lens, torch.int32, "past_lens")
    rc = load().kv_cache_write(ctypes.byref(make_layer(layer)), _ptr(k), _ptr(v), _ptr(cu_new),
                               _ptr(past_lens), int(past_lens.shape[0]), ctypes.byref(pages),
                               _ptr(k_pool), _ptr(v_pool), _stream(stream))
    _raise(rc, "kv_cache_write")


def attn_decode_paged(layer, q, k_pool, v_pool, pages: PswPages, seq_lens, out, lse=None,
                      ws=None, stream=None) -> None:
    _check(q, torch.bfloat16, "q")
    _check(k_pool, torch.bfloat16, "k_pool")
    _check(v_pool, torch.bfloat16, "v_pool")
    _check(seq_lens, torch.int32, "seq_lens")
    _check(out, torch.float32, "out")
    _check(lse, torch.float32, "lse")
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = load().attn_decode_paged(ctypes.byref(make_layer(layer)), _ptr(q), _ptr(k_pool),
                                  _ptr(v_pool), ctypes.byref(pages), _ptr(seq_lens),
                                  int(seq_lens.shape[0]), _ptr(out), _ptr(lse), _ptr(ws),
                                  ws_bytes, _stream(stream))
    _raise(rc, "attn_decode_paged")


def attn_prefill_chunked(layer, q, cu_q, past_lens, max_q_len: int, k_pool, v_pool,
                         pages: PswPages, out, lse=None, ws=None, stream=None) -> None:
    _check(q, torch.bfloat16, "q")
    _check(cu_q, torch.int32, "cu_q")
    _check(past_lens, torch.int32, "past_lens")
    _check(k_pool, torch.bfloat16, "k_pool")
    _check(v_pool, torch.bfloat16, "v_pool")
    _check(out, torch.float32, "out")
    _check(lse, torch.float32, "lse")
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = load().attn_prefill_chunked(ctypes.byref(make_layer(layer)), _ptr(q), _ptr(cu_q),
                                     _ptr(past_lens), int(past_lens.shape[0]), int(q.shape[0]),
                                     int(max_q_len),
                                     _ptr(k_pool), _ptr(v_pool), ctypes.byref(pages), _ptr(out),
                                     _ptr(lse), _ptr(ws), ws_bytes, _stream(stream))
    _raise(rc, "attn_prefill_chunked")


def attn_decode_paged_noalloc(layer, q, k_pool, v_pool, pages: PswPages, seq_lens, out,
                              lse=None, stream=None) -> None:
    """attn_decode_paged without a workspace, for callers that cannot allocate
    device memory: the library uses its own static device buffer (see
    include/psw.h for the size limit and the rule that overlapping calls race)."""
    _check(q, torch.bfloat16, "q")
    _check(k_pool, torch.bfloat16, "k_pool")
    _check(v_pool, torch.bfloat16, "v_pool")
    _check(seq_lens, torch.int32, "seq_lens")
    _check(out, torch.float32, "out")
    _check(lse, torch.float32, "lse")
    rc = load().attn_decode_paged_noalloc(ctypes.byref(make_layer(layer)), _ptr(q),
                                          _ptr(k_pool), _ptr(v_pool), ctypes.byref(pages),
                                          _ptr(seq_lens), int(seq_lens.shape[0]), _ptr(out),
                                          _ptr(lse), _stream(stream))
    _raise(rc, "attn_decode_paged_noalloc")


def attn_decode_paged_append(layer, q, k_new, v_new, k_pool, v_pool, pages: PswPages, seq_lens,
                             out, lse=None, ws=None, stream=None) -> None:
    """One decode step in one launch: each sequence's new K/V row written at
    position seq_len - 1 and attended to (kv_cache_write + attn_decode_paged)."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_pool, "k_pool"),
                 (v_pool, "v_pool")):
        _check(t, torch.bfloat16, n)
    _check(seq_lens, torch.int32, "seq_lens")
    _check(out, torch.float32, "out")
    _check(lse, torch.float32, "lse")
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = load().attn_decode_paged_append(ctypes.byref(make_layer(layer)), _ptr(q), _ptr(k_new),
                                         _ptr(v_new), _ptr(k_pool), _ptr(v_pool),
                                         ctypes.byref(pages), _ptr(seq_lens),
                                         int(seq_lens.shape[0]), _ptr(out), _ptr(lse), _ptr(ws),
                                         ws_bytes, _stream(stream))
    _raise(rc, "attn_decode_paged_append")


def kv_cache_write_fp8(layer, k, v, cu_new, past_lens, pages: PswPages, k_pool8, v_pool8,
                       k_scale, v_scale, stream=None) -> None:
    """kv_cache_write into FP8 pools (uint8 codes, fp32 per-row scales)."""
    _check(k, torch.bfloat16, "k")
    _check(v, torch.bfloat16, "v")
    _check(k_pool8, torch.uint8, "k_pool8")
    _check(v_pool8, torch.uint8, "v_pool8")
    _check(k_scale, torch.float32, "k_scale")
    _check(v_scale, torch.float32, "v_scale")
    _check(cu_new, torch.int32, "cu_new")
    _check(past_lens, torch.int32, "past_lens")
    rc = load().kv_cache_write_fp8(ctypes.byref(make_layer(layer)), _ptr(k), _ptr(v),
                                   _ptr(cu_new), _ptr(past_lens), int(past_lens.shape[0]),
                                   ctypes.byref(pages), _ptr(k_pool8), _ptr(v_pool8),
                                   _ptr(k_scale), _ptr(v_scale), _stream(stream))
    _raise(rc, "kv_cache_write_fp8")


def attn_decode_paged_fp8(layer, q, k_pool8, v_pool8, k_scale, v_scale, pages: PswPages,
                          seq_lens, out, lse=None, ws=None, stream=None) -> None:
    """attn_decode_paged over FP8 pools."""
    _check(q, torch.bfloat16, "q")
    _check(k_pool8, torch.uint8, "k_pool8")
    _check(v_pool8, torch.uint8, "v_pool8")
    _check(k_scale, torch.float32, "k_scale")
    _check(v_scale, torch.float32, "v_scale")
    _check(seq_lens, torch.int32, "seq_lens")
    _check(out, torch.float32, "out")
    _check(lse, torch.float32, "lse")
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    rc = load().attn_decode_paged_fp8(ctypes.byref(make_layer(layer)), _ptr(q), _ptr(k_pool8),
                                      _ptr(v_pool8), _ptr(k_scale), _ptr(v_scale),
                                      ctypes.byref(pages), _ptr(seq_lens),
                                      int(seq_lens.shape[0]), _ptr(out), _ptr(lse), _ptr(ws),
                                      ws_bytes, _stream(stream))
    _raise(rc, "attn_decode_paged_fp8")


STALL_OFF, STALL_DECODE, STALL_PREFILL = 0, 1, 2


def testing_stall(kernel: int, cta: int = -1, tile: int = -1) -> None:
    """Testing hook: CTA `cta` of the next launches of `kernel` leaves its
    tile copy `tile` unissued, so a bounded wait runs out (STALL_OFF: off)."""
    _raise(load().psw_testing_stall(kernel, cta, tile), "psw_testing_stall")


def make_norm_rope(theta: float, partial_rotary_factor: float = 1.0, eps: float = 1e-6,
                   q_weight=None, k_weight=None, v_weight=None) -> PswNormRope:
    """psw_norm_rope_t from device fp32 weight tensors (or None)."""
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight"), (v_weight, "v_weight")):
        _check(t, torch.float32, n)
    return PswNormRope(float(theta), float(partial_rotary_factor), float(eps),
                       None if q_weight is None else q_weight.data_ptr(),
                       None if k_weight is None else k_weight.data_ptr(),
                       None if v_weight is None else v_weight.data_ptr())


def qkv_norm_rope_cache_write(layer, rn: PswNormRope, q, k, v, cu_new, past_lens,
                              pages: PswPages | None, q_out, k_pool, v_pool,
                              stream=None) -> None:
    """The fused pre-attention step (per-head RMS-norm, proportional RoPE of q
    and k, cache write of k and v). k = v = pools = None processes q only."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (q_out, "q_out"), (k_pool, "k_pool"),
                 (v_pool, "v_pool")):
        _check(t, torch.bfloat16, n)
    _check(cu_new, torch.int32, "cu_new")
    _check(past_lens, torch.int32, "past_lens")
    rc = load().qkv_norm_rope_cache_write(
        ctypes.byref(make_layer(layer)), ctypes.byref(rn), _ptr(q), _ptr(k), _ptr(v),
        _ptr(cu_new), _ptr(past_lens), int(past_lens.shape[0]),
        None if pages is None else ctypes.byref(pages), _ptr(q_out), _ptr(k_pool), _ptr(v_pool),
        _stream(stream))
    _raise(rc, "qkv_norm_rope_cache_write")


# ---------------------------------------------------------------- latent attention
class _SharedLatent(PswLatent):
    """A layer's struct that every caller with the same fields is given: its fields stay."""

    def __setattr__(self, name, value):
        raise AttributeError(f"{name}: this struct is shared by all layers of the same fields; "
                             "make a PswLatent (or a layer) with the fields wanted")


_LATENT_STRUCTS: dict = {}


def make_latent_layer(layer) -> PswLatent:
    """From any object with the psw_latent_t fields (e.g. workloads.LatentLayer). The struct is
    read-only, one for all layers of the same fields; a PswLatent is returned as it is."""
    if isinstance(layer, PswLatent):
        return layer
    key = (int(layer.n_heads), int(layer.latent_dim), int(layer.rope_dim), int(layer.nope_dim),
           int(layer.v_dim), int(layer.window), float(layer.softcap), float(layer.scale),
           int(getattr(layer, "block_size", 16)))
    got = _LATENT_STRUCTS.get(key)
    if got is None:
        if len(_LATENT_STRUCTS) >= 1024:
            _LATENT_STRUCTS.clear()
        got = _LATENT_STRUCTS[key] = _SharedLatent.from_buffer_copy(PswLatent(*key))
    return got


def make_latent_norm(theta: float = 1e4, eps: float = 1e-6, latent_weight=None) -> PswLatentNorm:
    """psw_latent_norm_t from a device fp32 weight of latent_dim values (or None)."""
    _check(latent_weight, torch.float32, "latent_weight")
    norm = PswLatentNorm(float(theta), float(eps),
                         None if latent_weight is None else latent_weight.data_ptr())
    norm.weight = latent_weight  # keeps the tensor alive as long as its address is held
    return norm


def latent_workspace_bytes(layer, n_seqs: int) -> int:
    out = ctypes.c_size_t(0)
    _raise(load().psw_latent_workspace_bytes(ctypes.byref(make_latent_layer(layer)), int(n_seqs),
                                             ctypes.byref(out)), "psw_latent_workspace_bytes")
    return int(out.value)


def alloc_latent_workspace(layer, n_seqs: int, device="cuda") -> torch.Tensor:
    """A caller-owned workspace for attn_decode_latent(_fp8); it needs no zeroing."""
    return torch.empty(max(latent_workspace_bytes(layer, n_seqs), 256), dtype=torch.uint8,
                       device=device)


def _want(t, dtype, shape, name, device, strided=False):
    """Checks one tensor: dtype, device, shape, contiguity (`strided`: the last dimension
    alone)."""
    if (t.dtype is dtype and t.get_device() == device and t.shape == shape
            and (t.is_contiguous() or (strided and (t.stride(-1) == 1 or shape[-1] <= 1)))):
        return  # (a serving step makes several of these checks per launch)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on device {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous" + (" in its last dimension" if strided else ""))


def _want_rows(pages, n_seqs, device):
    """The page table has a row for every sequence (where it came from make_pages)."""
    table = getattr(pages, "table", None)
    if table is not None and (table.shape[0] < n_seqs or table.get_device() != device):
        raise ValueError(f"the block table must have {n_seqs} rows or more on device {device}, "
                         f"got {tuple(table.shape)} on {table.device}")


def _stream_of(device, stream):
    """The stream of a call on `device`, which must be the current device (as for every call:
    the library launches there)."""
    if device != torch.cuda.current_device():
        raise ValueError(f"the tensors are on device {device}, the current device is "
                         f"{torch.cuda.current_device()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream


def _strides(t):
    """Strides of all but the last dimension; a dimension of extent 1 gets that of packed rows
    (torch leaves any number there)."""
    st = t.stride()
    if 1 in t.shape:
        st, packed = list(st), 1
        for d in range(t.dim() - 1, -1, -1):
            if t.shape[d] == 1:
                st[d] = packed
            packed = max(packed, st[d] * t.shape[d])
    return st[:-1]


_I32, _F32, _BF16, _U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8


def _latent_write(name, layer, norm, ckv, q_rope, cu_new, past_lens, pages, q_rope_out, pool,
                  row_scale, stream):
    z = make_latent_layer(layer)
    row, dev = z.latent_dim + z.rope_dim, ckv.get_device()
    n_seqs, n_tok = past_lens.shape[0], ckv.shape[0]
    _want(ckv, _BF16, (n_tok, row), "ckv", dev, strided=True)
    _want(cu_new, _I32, (n_seqs + 1,), "cu_new", dev)
    _want(past_lens, _I32, (n_seqs,), "past_lens", dev)
    _want(pool, _BF16 if row_scale is None else _U8, (pages.num_blocks, 16, row), "pool", dev)
    if norm.latent_weight and getattr(norm, "weight", None) is not None:
        _want(norm.weight, _F32, (z.latent_dim,), "latent_weight", dev)
    if (q_rope is None) != (q_rope_out is None):
        raise ValueError("q_rope and q_rope_out go together")
    q_args, qo_args = (None, 0, 0), (None, 0, 0)
    if q_rope is not None:
        shape = (n_tok, z.n_heads, z.rope_dim)
        _want(q_rope, _BF16, shape, "q_rope", dev, strided=True)
        _want(q_rope_out, _BF16, shape, "q_rope_out", dev, strided=True)
        q_args = (q_rope.data_ptr(), *_strides(q_rope))
        qo_args = (q_rope_out.data_ptr(), *_strides(q_rope_out))
    tail = [pool.data_ptr()]
    if row_scale is not None:
        _want(row_scale, _F32, (pages.num_blocks, 16), "row_scale", dev)
        tail.append(row_scale.data_ptr())
    _want_rows(pages, n_seqs, dev)
    if n_tok == 0 or n_seqs == 0:
        return
    rc = getattr(load(), name)(ctypes.byref(z), ctypes.byref(norm), ckv.data_ptr(), *_strides(ckv),
                               *q_args, cu_new.data_ptr(), past_lens.data_ptr(), n_seqs, n_tok,
                               ctypes.byref(pages), *qo_args, *tail, _stream_of(dev, stream))
    if rc:
        _raise(rc, name)


def latent_norm_rope_cache_write(layer, norm: PswLatentNorm, ckv, q_rope, cu_new, past_lens,
                                 pages: PswPages, q_rope_out, pool, stream=None) -> None:
    """Norm, rotation and cache write of new latent rows. ckv bf16 [n, latent_dim + 64] (rows may
    be strided); q_rope and q_rope_out bf16 [n, heads, 64] views of
    any token and head stride (in place is fine), or both None."""
    _latent_write("latent_norm_rope_cache_write", layer, norm, ckv, q_rope, cu_new, past_lens,
                  pages, q_rope_out, pool, None, stream)


def latent_norm_rope_cache_write_fp8(layer, norm: PswLatentNorm, ckv, q_rope, cu_new, past_lens,
                                     pages: PswPages, q_rope_out, pool8, row_scale,
                                     stream=None) -> None:
    """The same into FP8 pages: pool8 uint8 [num_blocks, 16, latent_dim + 64] of E4M3 codes,
    row_scale fp32 [num_blocks, 16]."""
    if row_scale is None:
        raise ValueError("row_scale is required")
    _latent_write("latent_norm_rope_cache_write_fp8", layer, norm, ckv, q_rope, cu_new, past_lens,
                  pages, q_rope_out, pool8, row_scale, stream)


def _latent_decode(name, layer, q, pool, row_scale, pages, seq_lens, out, lse, ws, stream):
    z = make_latent_layer(layer)
    row, dev, n_seqs = z.latent_dim + z.rope_dim, q.get_device(), seq_lens.shape[0]
    _want(q, _BF16, (n_seqs, z.n_heads, row), "q", dev)
    _want(pool, _BF16 if row_scale is None else _U8, (pages.num_blocks, 16, row), "pool", dev)
    _want(seq_lens, _I32, (n_seqs,), "seq_lens", dev)
    _want(out, _BF16, (n_seqs, z.n_heads, z.latent_dim), "out", dev)
    if lse is not None:
        _want(lse, _F32, (n_seqs, z.n_heads), "lse", dev)
    pools = [pool.data_ptr()]
    if row_scale is not None:
        _want(row_scale, _F32, (pages.num_blocks, 16), "row_scale", dev)
        pools.append(row_scale.data_ptr())
    ws_ptr, ws_bytes = None, 0
    if ws is not None:
        if not ws.is_cuda or ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be a contiguous CUDA tensor on device {dev}")
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _want_rows(pages, n_seqs, dev)
    if n_seqs == 0:
        return
    rc = getattr(load(), name)(ctypes.byref(z), q.data_ptr(), *pools, ctypes.byref(pages),
                               seq_lens.data_ptr(), n_seqs, out.data_ptr(),
                               None if lse is None else lse.data_ptr(), ws_ptr, ws_bytes,
                               _stream_of(dev, stream))
    if rc:
        _raise(rc, name)


def attn_decode_latent(layer, q, pool, pages: PswPages, seq_lens, out, lse=None, ws=None,
                       stream=None) -> None:
    """Absorbed latent attention of one token per sequence: q bf16 [n, heads, latent_dim + 64],
    out bf16 [n, heads, latent_dim], lse fp32 [n, heads] or None; ws from
    alloc_latent_workspace (calls that may overlap on the GPU need one each)."""
    _latent_decode("attn_decode_latent", layer, q, pool, None, pages, seq_lens, out, lse, ws,
                   stream)


def attn_decode_latent_fp8(layer, q, pool8, row_scale, pages: PswPages, seq_lens, out, lse=None,
                           ws=None, stream=None) -> None:
    """attn_decode_latent over FP8 pages."""
    if row_scale is None:
        raise ValueError("row_scale is required")
    _latent_decode("attn_decode_latent_fp8", layer, q, pool8, row_scale, pages, seq_lens, out,
                   lse, ws, stream)


def _latent_expand(name, layer, pool, row_scale, pages, cu_k, w, kv, k_rope, k_first, stream):
    z = make_latent_layer(layer)
    row, dev = z.latent_dim + z.rope_dim, pool.get_device()
    n_seqs, n_k, e = cu_k.shape[0] - 1, kv.shape[0], z.nope_dim + z.v_dim
    _want(pool, _BF16 if row_scale is None else _U8, (pages.num_blocks, 16, row), "pool", dev)
    _want(cu_k, _I32, (n_seqs + 1,), "cu_k", dev)
    _want(w, _BF16, (z.n_heads, e, z.latent_dim), "w", dev)
    _want(kv, _BF16, (n_k, z.n_heads, e), "kv", dev)
    _want(k_rope, _BF16, (n_k, z.rope_dim), "k_rope", dev)
    if k_first is not None:
        _want(k_first, _I32, (n_seqs,), "k_first", dev)
    pools = [pool.data_ptr()]
    if row_scale is not None:
        _want(row_scale, _F32, (pages.num_blocks, 16), "row_scale", dev)
        pools.append(row_scale.data_ptr())
    _want_rows(pages, n_seqs, dev)
    if n_k == 0 or n_seqs == 0:
        return
    rc = getattr(load(), name)(ctypes.byref(z), *pools, ctypes.byref(pages), cu_k.data_ptr(),
                               None if k_first is None else k_first.data_ptr(), n_seqs, n_k,
                               w.data_ptr(), kv.data_ptr(), k_rope.data_ptr(),
                               _stream_of(dev, stream))
    if rc:
        _raise(rc, name)


def latent_kv_expand(layer, pool, pages: PswPages, cu_k, w, kv, k_rope, k_first=None,
                     stream=None) -> None:
    """Expands cached rows: kv bf16 [n_k, heads, 256] (128 key, 128 value components) from
    w bf16 [heads, 256, latent_dim], k_rope bf16 [n_k, 64]; row cu_k[b] + j of sequence b is
    position k_first[b] + j (k_first None: j)."""
    _latent_expand("latent_kv_expand", layer, pool, None, pages, cu_k, w, kv, k_rope, k_first,
                   stream)


def latent_kv_expand_fp8(layer, pool8, row_scale, pages: PswPages, cu_k, w, kv, k_rope,
                         k_first=None, stream=None) -> None:
    """latent_kv_expand from FP8 pages."""
    if row_scale is None:
        raise ValueError("row_scale is required")
    _latent_expand("latent_kv_expand_fp8", layer, pool8, row_scale, pages, cu_k, w, kv, k_rope,
                   k_first, stream)


def attn_prefill_latent(layer, q, cu_q, past_lens, max_q_len: int, kv, k_rope, cu_k, out,
                        lse=None, k_first=None, stream=None) -> None:
    """Expanded latent attention of a chunk per sequence: q bf16 [n_q, heads, 192], kv and k_rope
    from latent_kv_expand, out bf16 [n_q, heads, 128], lse fp32 [n_q, heads] or None."""
    z = make_latent_layer(layer)
    dev, n_seqs, n_q, n_k = q.get_device(), past_lens.shape[0], q.shape[0], kv.shape[0]
    _want(q, _BF16, (n_q, z.n_heads, z.nope_dim + z.rope_dim), "q", dev)
    _want(cu_q, _I32, (n_seqs + 1,), "cu_q", dev)
    _want(past_lens, _I32, (n_seqs,), "past_lens", dev)
    _want(kv, _BF16, (n_k, z.n_heads, z.nope_dim + z.v_dim), "kv", dev)
    _want(k_rope, _BF16, (n_k, z.rope_dim), "k_rope", dev)
    _want(cu_k, _I32, (n_seqs + 1,), "cu_k", dev)
    _want(out, _BF16, (n_q, z.n_heads, z.v_dim), "out", dev)
    if lse is not None:
        _want(lse, _F32, (n_q, z.n_heads), "lse", dev)
    if k_first is not None:
        _want(k_first, _I32, (n_seqs,), "k_first", dev)
    if n_q == 0 or n_seqs == 0:
        return
    rc = load().attn_prefill_latent(ctypes.byref(z), q.data_ptr(), cu_q.data_ptr(),
                                    past_lens.data_ptr(), n_seqs, n_q, int(max_q_len),
                                    kv.data_ptr() or None, k_rope.data_ptr() or None,
                                    cu_k.data_ptr(),
                                    None if k_first is None else k_first.data_ptr(), n_k,
                                    out.data_ptr(), None if lse is None else lse.data_ptr(),
                                    _stream_of(dev, stream))
    if rc:
        _raise(rc, "attn_prefill_latent")


# ---------------------------------------------------------------- 4-bit pages
_LAYER_STRUCTS: dict = {}


def _layer_struct(layer):
    """(reference to make_layer's struct, n_q_heads, n_kv_heads, head_dim, k_eq_v), one for all
    layers of the same fields (never handed out)."""
    key = (layer.n_q_heads, layer.n_kv_heads, layer.head_dim, layer.window, layer.softcap,
           layer.scale, layer.k_eq_v, getattr(layer, "block_size", 16))
    got = _LAYER_STRUCTS.get(key)
    if got is None:
        if len(_LAYER_STRUCTS) >= 1024:
            _LAYER_STRUCTS.clear()
        z = make_layer(layer)
        got = _LAYER_STRUCTS[key] = (ctypes.byref(z), z.n_q_heads, z.n_kv_heads, z.head_dim,
                                     bool(z.k_eq_v))
    return got


def _stream_here(device, stream):
    """_stream_of for tensors that exist, so that CUDA is up."""
    if device != torch._C._cuda_getDevice():
        return _stream_of(device, stream)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream


def fp4_page_bytes(layer) -> int:
    """Bytes of one page of one KV head in a 4-bit pool (PSW_FP4_PAGE_BYTES)."""
    return 9 * int(layer.head_dim)


def alloc_fp4_pool(layer, num_blocks: int, device="cuda") -> torch.Tensor:
    """A zero-filled 4-bit pool, uint8 [num_blocks, n_kv_heads, fp4_page_bytes]."""
    return torch.zeros(int(num_blocks), int(layer.n_kv_heads), fp4_page_bytes(layer),
                       dtype=torch.uint8, device=device)


def fp4_workspace_bytes(layer, n_seqs: int) -> int:
    out = ctypes.c_size_t(0)
    _raise(load().psw_fp4_workspace_bytes(_layer_struct(layer)[0], int(n_seqs),
                                          ctypes.byref(out)), "psw_fp4_workspace_bytes")
    return int(out.value)


def alloc_fp4_workspace(layer, n_seqs: int, device="cuda") -> torch.Tensor:
    """A caller-owned workspace for attn_decode_paged_fp4, its counters zeroed (calls keep them
    zero); the rest of it needs no zeroing."""
    ws = torch.empty(fp4_workspace_bytes(layer, n_seqs), dtype=torch.uint8, device=device)
    ws[:FP4_COUNTER_BYTES].zero_()
    return ws


FP4_COUNTER_BYTES = 16384  # PSW_FP4_COUNTER_BYTES


def _want_v(v, k_eq_v, name):
    if (v is None) != k_eq_v:
        raise PswError(-7, f"{name} (k_eq_v is {k_eq_v})")


def block_table_extend(block_table, past_lens, new_lens, free_ids, free_pos, free_next, cu_new,
                       seq_lens, slots=None, stream=None) -> None:
    """The tables of a step, built on the device: block_table int32 [n, max_blocks] gets entries
    for the pages that new_lens int32 [n] tokens after past_lens [n] begin, from free_ids int32
    [n_free] at the cursor free_pos int32 [1] on; free_next [1] (may be free_pos), cu_new [n + 1],
    seq_lens [n] and slots int64 [rows] or None are written (n 0: the cursor, where it is not in
    place, and cu_new with it). No other two may overlap: seq_lens is copied to past_lens for the
    next step, not written there."""
    dev, n = block_table.get_device(), past_lens.shape[0]
    if block_table.dim() != 2 or block_table.shape[0] < n:
        raise ValueError(f"block_table must have {n} rows or more, got {tuple(block_table.shape)}")
    one, each = (1,), (n,)
    # (what _want looks at in one expression, and by _want where something is wrong: 1 us)
    if not (block_table.dtype is _I32 and block_table.is_contiguous()
            and past_lens.dtype is _I32 and past_lens.shape == each and past_lens.is_contiguous()
            and new_lens.dtype is _I32 and new_lens.shape == each and new_lens.is_contiguous()
            and free_ids.dtype is _I32 and free_ids.dim() == 1 and free_ids.is_contiguous()
            and free_pos.dtype is _I32 and free_pos.shape == one
            and free_next.dtype is _I32 and free_next.shape == one
            and cu_new.dtype is _I32 and cu_new.shape == (n + 1,) and cu_new.is_contiguous()
            and seq_lens.dtype is _I32 and seq_lens.shape == each and seq_lens.is_contiguous()
            and past_lens.get_device() == new_lens.get_device() == free_ids.get_device()
            == free_pos.get_device() == free_next.get_device() == cu_new.get_device()
            == seq_lens.get_device() == dev):
        _want(block_table, _I32, block_table.shape, "block_table", dev)
        _want(past_lens, _I32, each, "past_lens", dev)
        _want(new_lens, _I32, each, "new_lens", dev)
        _want(free_ids, _I32, (free_ids.numel(),), "free_ids", dev)
        _want(free_pos, _I32, one, "free_pos", dev)
        _want(free_next, _I32, one, "free_next", dev)
        _want(cu_new, _I32, (n + 1,), "cu_new", dev)
        _want(seq_lens, _I32, each, "seq_lens", dev)
    slot_args = (None, 0)
    if slots is not None:
        _want(slots, torch.int64, (slots.numel(),), "slots", dev)
        slot_args = (slots.data_ptr(), slots.shape[0])
    if n == 0:  # (empty tensors have no address, and none of theirs is used)
        at = cu_new.data_ptr()
        rc = load().block_table_extend(at, max(1, block_table.shape[1]), at, at, 0,
                                       free_ids.data_ptr() or None, free_ids.shape[0],
                                       free_pos.data_ptr(), free_next.data_ptr(), at, at,
                                       *slot_args, _stream_here(dev, stream))
        if rc:
            _raise(rc, "block_table_extend")
        return
    rc = load().block_table_extend(block_table.data_ptr(), block_table.shape[1],
                                   past_lens.data_ptr(), new_lens.data_ptr(), n,
                                   free_ids.data_ptr() or None, free_ids.shape[0],
                                   free_pos.data_ptr(), free_next.data_ptr(), cu_new.data_ptr(),
                                   seq_lens.data_ptr(), *slot_args, _stream_here(dev, stream))
    if rc:
        _raise(rc, "block_table_extend")


def kv_cache_write_fp4(layer, k, v, cu_new, past_lens, pages: PswPages, k_pool4, v_pool4,
                       k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """kv_cache_write into 4-bit pools (alloc_fp4_pool): k, v bf16 [n_new, n_kv, head_dim], v and
    v_pool4 None with k_eq_v; k_scale and v_scale are the pools' own, the same in every call."""
    z_ref, n_q, n_kv, hd, k_eq_v = _layer_struct(layer)
    dev, n, rows = k.get_device(), past_lens.shape[0], k.shape[0]
    shape, pool = (rows, n_kv, hd), (pages.num_blocks, n_kv, 9 * hd)
    _want_v(v, k_eq_v, "v")
    _want_v(v_pool4, k_eq_v, "v_pool4")
    # (what _want looks at in one expression, and by _want where something is wrong: 0.4 us)
    if not (k.dtype is _BF16 and k.shape == shape and k.is_contiguous()
            and cu_new.dtype is _I32 and cu_new.shape == (n + 1,) and cu_new.is_contiguous()
            and past_lens.dtype is _I32 and past_lens.shape == (n,) and past_lens.is_contiguous()
            and k_pool4.dtype is _U8 and k_pool4.shape == pool and k_pool4.is_contiguous()
            and cu_new.get_device() == past_lens.get_device() == k_pool4.get_device() == dev):
        _want(k, _BF16, shape, "k", dev)
        _want(cu_new, _I32, (n + 1,), "cu_new", dev)
        _want(past_lens, _I32, (n,), "past_lens", dev)
        _want(k_pool4, _U8, pool, "k_pool4", dev)
    if not (k_eq_v or (
            v.dtype is _BF16 and v.shape == shape and v.is_contiguous()
            and v_pool4.dtype is _U8 and v_pool4.shape == pool and v_pool4.is_contiguous()
            and v.get_device() == v_pool4.get_device() == dev)):
        _want(v, _BF16, shape, "v", dev)
        _want(v_pool4, _U8, pool, "v_pool4", dev)
    _want_rows(pages, n, dev)
    if n == 0 or rows == 0:
        return
    rc = load().kv_cache_write_fp4(z_ref, k.data_ptr(),
                                   None if v is None else v.data_ptr(), cu_new.data_ptr(),
                                   past_lens.data_ptr(), n, rows, ctypes.byref(pages),
                                   k_pool4.data_ptr(), None if v is None else v_pool4.data_ptr(),
                                   k_scale, v_scale, _stream_here(dev, stream))
    if rc:
        _raise(rc, "kv_cache_write_fp4")


def kv_cache_read_fp4(layer, k_pool4, v_pool4, pages: PswPages, first, seq_lens,
                      out_pages: PswPages, k_pool, v_pool, k_scale: float = 1.0,
                      v_scale: float = 1.0, stream=None) -> None:
    """Rows of 4-bit pages into bf16 pages: positions first[b] (int32 [n], or None: 0) to
    seq_lens[b] of every sequence, from pages into the pools of out_pages (for the attention of a
    chunk, attn_prefill_chunked)."""
    z_ref, n_q, n_kv, hd, k_eq_v = _layer_struct(layer)
    dev, n = k_pool4.get_device(), seq_lens.shape[0]
    pool, wide = (pages.num_blocks, n_kv, 9 * hd), (out_pages.num_blocks, 16, n_kv, hd)
    _want_v(v_pool4, k_eq_v, "v_pool4")
    _want_v(v_pool, k_eq_v, "v_pool")
    _want(k_pool4, _U8, pool, "k_pool4", dev)
    _want(k_pool, _BF16, wide, "k_pool", dev)
    _want(seq_lens, _I32, (n,), "seq_lens", dev)
    if first is not None:
        _want(first, _I32, (n,), "first", dev)
    if v_pool is not None:
        _want(v_pool4, _U8, pool, "v_pool4", dev)
        _want(v_pool, _BF16, wide, "v_pool", dev)
    _want_rows(pages, n, dev)
    _want_rows(out_pages, n, dev)
    if n == 0:
        return
    rc = load().kv_cache_read_fp4(z_ref, k_pool4.data_ptr(),
                                  None if v_pool is None else v_pool4.data_ptr(),
                                  ctypes.byref(pages), None if first is None else first.data_ptr(),
                                  seq_lens.data_ptr(), n, ctypes.byref(out_pages),
                                  k_pool.data_ptr(), None if v_pool is None else v_pool.data_ptr(),
                                  k_scale, v_scale, _stream_here(dev, stream))
    if rc:
        _raise(rc, "kv_cache_read_fp4")


def attn_decode_paged_fp4(layer, q, k_pool4, v_pool4, pages: PswPages, seq_lens, out, lse=None,
                          ws=None, k_scale: float = 1.0, v_scale: float = 1.0,
                          stream=None) -> None:
    """attn_decode_paged over 4-bit pools; out is bf16 [n, n_q, head_dim] and must not overlap q, ws from
    alloc_fp4_workspace (calls that may overlap on the GPU need one each)."""
    z_ref, n_q, n_kv, hd, k_eq_v = _layer_struct(layer)
    dev, n = q.get_device(), seq_lens.shape[0]
    rows, pool = (n, n_q, hd), (pages.num_blocks, n_kv, 9 * hd)
    _want_v(v_pool4, k_eq_v, "v_pool4")
    _want(q, _BF16, rows, "q", dev)
    _want(k_pool4, _U8, pool, "k_pool4", dev)
    if v_pool4 is not None:
        _want(v_pool4, _U8, pool, "v_pool4", dev)
    _want(seq_lens, _I32, (n,), "seq_lens", dev)
    _want(out, _BF16, rows, "out", dev)
    if lse is not None:
        _want(lse, _F32, (n, n_q), "lse", dev)
    ws_ptr, ws_bytes = None, 0
    if ws is not None:
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be a contiguous CUDA tensor on device {dev}")
        ws_ptr, ws_bytes = ws.data_ptr(), ws.nbytes
    _want_rows(pages, n, dev)
    if n == 0:
        return
    rc = load().attn_decode_paged_fp4(z_ref, q.data_ptr(), k_pool4.data_ptr(),
                                      None if v_pool4 is None else v_pool4.data_ptr(),
                                      ctypes.byref(pages), seq_lens.data_ptr(), n, out.data_ptr(),
                                      None if lse is None else lse.data_ptr(), ws_ptr, ws_bytes,
                                      k_scale, v_scale, _stream_here(dev, stream))
    if rc:
        _raise(rc, "attn_decode_paged_fp4")


def kv_share_map(n_layers: int, pattern: int, n_shared: int = 0):
    """(is_full, target) lists of a hybrid stack (psw_kv_share_map): layer i is
    full when (i + 1) % pattern == 0; the last n_shared layers read the cache of
    the last cache-owning layer of their type."""
    full = (ctypes.c_int32 * n_layers)()
    tgt = (ctypes.c_int32 * n_layers)()
    _raise(load().psw_kv_share_map(int(n_layers), int(pattern), int(n_shared), full, tgt),
           "psw_kv_share_map")
    return [bool(x) for x in full], [int(x) for x in tgt]


def _i32_array(values):
    arr = (ctypes.c_int32 * max(1, len(values)))(*[int(v) for v in values])
    return arr


def block_hash(parent: int, tokens) -> int:
    """psw_block_hash: chained FNV-1a hash of one page's tokens."""
    return int(load().psw_block_hash(int(parent), _i32_array(tokens), len(tokens)))


class BlockPool:
    """Host page allocator with prefix caching (psw_block_pool_*): ctypes
    marshalling only; the pool lives in libpsw."""

    def __init__(self, num_blocks: int, prefix_cache: bool = True):
        self._lib = load()
        h = ctypes.c_void_p()
        _raise(self._lib.psw_block_pool_create(int(num_blocks), int(bool(prefix_cache)),
                                               ctypes.byref(h)), "psw_block_pool_create")
        self._h = h

    def close(self):
        if self._h:
            self._lib.psw_block_pool_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def num_free(self) -> int:
        return int(self._lib.psw_block_pool_num_free(self._h))

    def allocate(self, n: int):
        """(status, ids)."""
        out = (ctypes.c_int32 * max(1, n))()
        rc = self._lib.psw_block_pool_allocate(self._h, int(n), out)
        return rc, (list(out[:n]) if rc == PSW_OK else [])

    def release(self, ids) -> int:
        return self._lib.psw_block_pool_free(self._h, _i32_array(ids), len(ids))

    def get_cached(self, h: int) -> int:
        out = ctypes.c_int32(-1)
        _raise(self._lib.psw_block_pool_get_cached(self._h, int(h), ctypes.byref(out)),
               "psw_block_pool_get_cached")
        return int(out.value)

    def cache(self, block: int, h: int) -> int:
        return self._lib.psw_block_pool_cache(self._h, int(block), int(h))

    def ref_count(self, block: int) -> int:
        out = ctypes.c_int32(0)
        _raise(self._lib.psw_block_pool_ref_count(self._h, int(block), ctypes.byref(out)),
               "psw_block_pool_ref_count")
        return int(out.value)

    def admit(self, tokens, max_blocks: int):
        """(status, block-table row, tokens whose KV is already cached)."""
        row = (ctypes.c_int32 * max(1, max_blocks))()
        cached = ctypes.c_int32(0)
        rc = self._lib.psw_block_pool_admit(self._h, _i32_array(tokens), len(tokens), row,
                                            int(max_blocks), ctypes.byref(cached))
        return rc, (list(row[:max_blocks]) if rc == PSW_OK else None), int(cached.value)

    def commit(self, tokens, row) -> int:
        return self._lib.psw_block_pool_commit(self._h, _i32_array(tokens), len(tokens),
                                               _i32_array(row))


def get_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error word."""
    val = ctypes.c_int32(0)
    _raise(load().psw_get_error(_stream(stream), ctypes.byref(val)), "psw_get_error")
    return int(val.value)
