"""Python binding of librlk_logp.so: deterministic selected-token logp on MI355X.

Argument marshalling only.  Every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/rlk_logp.h``; PyTorch supplies
device memory and the stream.  There is no fallback: if the library is not
built, importing this package raises.

Functions with the C names take caller-allocated tensors and mirror the C
signatures.  ``forward`` / ``backward`` are conveniences that allocate the
outputs and workspace with torch and call them.
"""
from __future__ import annotations

import contextlib
import ctypes
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "librlk_logp.so"

RLK_OK = 0
RLK_ERR_NULL_POINTER = 1
RLK_ERR_BAD_SHAPE = 2
RLK_ERR_BAD_TILING = 3
RLK_ERR_ALIGNMENT = 4
RLK_ERR_WORKSPACE = 5
RLK_ERR_DTYPE = 6
RLK_ERR_TARGET_RANGE = 7
RLK_ERR_NONFINITE_LSE = 8
RLK_ERR_HIP = 9

RLK_DTYPE_F32 = 0
RLK_DTYPE_BF16 = 1
RLK_DTYPE_F16 = 2
RLK_FLAG_VALIDATE = 1

EXPORTED = ("rlk_logp_workspace_bytes", "rlk_logp_fwd", "rlk_logp_bwd",
            "rlk_logp_ex_workspace_bytes", "rlk_logp_fwd_ex", "rlk_logp_bwd_ex",
            "rlk_logp_fwd_bwd_workspace_bytes", "rlk_logp_fwd_bwd",
            "rlk_logp_fwd_bwd_ex_workspace_bytes", "rlk_logp_fwd_bwd_ex",
            "rlk_logp_fused_lmhead_workspace_bytes", "rlk_logp_fused_lmhead",
            "rlk_logp_fused_lmhead_bwd_workspace_bytes", "rlk_logp_fused_lmhead_bwd",
            "rlk_fp8_quantize", "rlk_lmhead_logits_fp8",
            "rlk_logp_fused_lmhead_fp8_workspace_bytes", "rlk_logp_fused_lmhead_fp8",
            "rlk_logits_process", "rlk_logp_processed_workspace_bytes",
            "rlk_logp_processed_fwd", "rlk_logp_processed_bwd",
            "rlk_linear_fwd", "rlk_linear_bwd_workspace_bytes", "rlk_linear_bwd",
            "rlk_logp_tile_geometry", "rlk_status_string", "rlk_last_error_detail",
            "rlk_logp_fwd_noalloc")


class rlk_logp_desc(ctypes.Structure):  # noqa: N801 - mirrors the C struct name
    _fields_ = [("num_tokens", ctypes.c_int64), ("real_vocab", ctypes.c_int64),
                ("padded_vocab", ctypes.c_int64), ("ld_logits", ctypes.c_int64),
                ("num_vocab_tiles", ctypes.c_int32), ("num_virtual_shards", ctypes.c_int32),
                ("ignore_index", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class rlk_fp8_matrix(ctypes.Structure):  # noqa: N801 - mirrors the C struct name
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("scale_row_stride", ctypes.c_int64), ("scale_col_stride", ctypes.c_int64)]


class rlk_logit_rules(ctypes.Structure):  # noqa: N801
    _fields_ = [("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
                ("history", ctypes.c_void_p), ("history_len", ctypes.c_int64),
                ("history_begin", ctypes.c_void_p), ("history_split", ctypes.c_void_p),
                ("history_end", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("bias_rows", ctypes.c_int64), ("ld_bias", ctypes.c_int64),
                ("bias_index", ctypes.c_void_p), ("allow", ctypes.c_void_p),
                ("allow_rows", ctypes.c_int64), ("ld_allow", ctypes.c_int64),
                ("allow_index", ctypes.c_void_p)]


class rlk_linear_desc(ctypes.Structure):  # noqa: N801
    _fields_ = [("tokens", ctypes.c_int64), ("in_dim", ctypes.c_int64),
                ("out_dim", ctypes.c_int64), ("padded_out", ctypes.c_int64),
                ("ld_out", ctypes.c_int64), ("ld_residual", ctypes.c_int64),
                ("ld_saved", ctypes.c_int64), ("activation", ctypes.c_int32),
                ("bias_dtype", ctypes.c_int32), ("saved_dtype", ctypes.c_int32),
                ("cap", ctypes.c_float)]


class RlkError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.detail = detail
        super().__init__(f"{_lib.rlk_status_string(status).decode()}: {detail}")


def _load() -> ctypes.CDLL:
    if not LIB_PATH.exists():
        raise ImportError(f"{LIB_PATH} is not built; run vocab_selected_token_amd.build_lib "
                          "(there is no fallback path)")
    lib = ctypes.CDLL(str(LIB_PATH))
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    dp = ctypes.POINTER(rlk_logp_desc)
    lib.rlk_logp_workspace_bytes.argtypes = [dp]
    lib.rlk_logp_workspace_bytes.restype = sz
    lib.rlk_logp_fwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.rlk_logp_fwd.restype = ctypes.c_int
    lib.rlk_logp_fwd_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp]
    lib.rlk_logp_fwd_noalloc.restype = ctypes.c_int
    lib.rlk_logp_bwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, i64, ctypes.c_int, vp, sz, vp]
    lib.rlk_logp_bwd.restype = ctypes.c_int
    lib.rlk_logp_ex_workspace_bytes.argtypes = [dp]
    lib.rlk_logp_ex_workspace_bytes.restype = sz
    lib.rlk_logp_fwd_ex.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.rlk_logp_fwd_ex.restype = ctypes.c_int
    lib.rlk_logp_bwd_ex.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, ctypes.c_int, vp,
                                    sz, vp]
    lib.rlk_logp_bwd_ex.restype = ctypes.c_int
    lib.rlk_logp_fwd_bwd_workspace_bytes.argtypes = [dp]
    lib.rlk_logp_fwd_bwd_workspace_bytes.restype = sz
    lib.rlk_logp_fwd_bwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i64, ctypes.c_int, vp, sz,
                                     vp]
    lib.rlk_logp_fwd_bwd.restype = ctypes.c_int
    lib.rlk_logp_fwd_bwd_ex_workspace_bytes.argtypes = [dp]
    lib.rlk_logp_fwd_bwd_ex_workspace_bytes.restype = sz
    lib.rlk_logp_fwd_bwd_ex.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64,
                                        ctypes.c_int, vp, sz, vp]
    lib.rlk_logp_fwd_bwd_ex.restype = ctypes.c_int
    lib.rlk_logp_fused_lmhead_workspace_bytes.argtypes = [dp]
    lib.rlk_logp_fused_lmhead_workspace_bytes.restype = sz
    lib.rlk_logp_fused_lmhead.argtypes = [dp, vp, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.rlk_logp_fused_lmhead.restype = ctypes.c_int
    lib.rlk_logp_fused_lmhead_bwd_workspace_bytes.argtypes = [dp, i64, i32, i32]
    lib.rlk_logp_fused_lmhead_bwd_workspace_bytes.restype = sz
    lib.rlk_logp_fused_lmhead_bwd.argtypes = [dp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                              vp]
    lib.rlk_logp_fused_lmhead_bwd.restype = ctypes.c_int
    mp = ctypes.POINTER(rlk_fp8_matrix)
    lib.rlk_fp8_quantize.argtypes = [i64, i64, vp, i64, i32, vp, vp, i64, i64, vp]
    lib.rlk_fp8_quantize.restype = ctypes.c_int
    lib.rlk_lmhead_logits_fp8.argtypes = [dp, mp, mp, i64, vp, vp]
    lib.rlk_lmhead_logits_fp8.restype = ctypes.c_int
    lib.rlk_logp_fused_lmhead_fp8_workspace_bytes.argtypes = [dp]
    lib.rlk_logp_fused_lmhead_fp8_workspace_bytes.restype = sz
    lib.rlk_logp_fused_lmhead_fp8.argtypes = [dp, mp, mp, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.rlk_logp_fused_lmhead_fp8.restype = ctypes.c_int
    rp, lp = ctypes.POINTER(rlk_logit_rules), ctypes.POINTER(rlk_linear_desc)
    lib.rlk_logits_process.argtypes = [dp, vp, rp, vp, i64, ctypes.c_int, vp]
    lib.rlk_logits_process.restype = ctypes.c_int
    lib.rlk_logp_processed_workspace_bytes.argtypes = [dp]
    lib.rlk_logp_processed_workspace_bytes.restype = sz
    lib.rlk_logp_processed_fwd.argtypes = [dp, vp, rp, vp, vp, vp, vp, vp, sz, vp]
    lib.rlk_logp_processed_fwd.restype = ctypes.c_int
    lib.rlk_logp_processed_bwd.argtypes = [dp, vp, rp, vp, vp, vp, vp, vp, vp, i64, ctypes.c_int,
                                           vp, sz, vp]
    lib.rlk_logp_processed_bwd.restype = ctypes.c_int
    lib.rlk_linear_fwd.argtypes = [lp, vp, vp, vp, vp, vp, vp, vp]
    lib.rlk_linear_fwd.restype = ctypes.c_int
    lib.rlk_linear_bwd_workspace_bytes.argtypes = [lp]
    lib.rlk_linear_bwd_workspace_bytes.restype = sz
    lib.rlk_linear_bwd.argtypes = [lp, vp, vp, vp, vp, i64, vp, vp, vp, vp, sz, vp]
    lib.rlk_linear_bwd.restype = ctypes.c_int
    lib.rlk_logp_tile_geometry.argtypes = [i64, i32, i32, vp, vp]
    lib.rlk_logp_tile_geometry.restype = ctypes.c_int
    lib.rlk_status_string.argtypes = [ctypes.c_int]
    lib.rlk_status_string.restype = ctypes.c_char_p
    lib.rlk_last_error_detail.argtypes = []
    lib.rlk_last_error_detail.restype = ctypes.c_char_p
    return lib


_lib = _load()


def _check(status: int) -> None:
    if status != RLK_OK:
        raise RlkError(status, _lib.rlk_last_error_detail().decode())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


# The handle alone: a Stream object takes ten times as long to make.  It is not part of
# torch's documented interface, so there may be none.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def make_desc(num_tokens: int, real_vocab: int, padded_vocab: int, ld_logits: int,
              num_vocab_tiles: int = 64, num_virtual_shards: int = 1, ignore_index: int = -100,
              validate: bool = False) -> rlk_logp_desc:
    """The rlk_logp_desc of a call: ld_logits is the row stride of the logits in
    elements; validate sets RLK_FLAG_VALIDATE."""
    return rlk_logp_desc(num_tokens, real_vocab, padded_vocab, ld_logits, num_vocab_tiles,
                         num_virtual_shards, ignore_index,
                         RLK_FLAG_VALIDATE if validate else 0)


# -- the C entry points --------------------------------------------------------
# Each function below calls the C function of the same name (include/rlk_logp.h)
# with the same arguments in the same order: tensors go as their data pointers
# (None as NULL), a workspace tensor also gives its size in bytes, `stream`
# defaults to torch's current stream, and a status other than RLK_OK raises
# RlkError with the library's detail text.
def rlk_logp_workspace_bytes(desc: rlk_logp_desc) -> int:
    return int(_lib.rlk_logp_workspace_bytes(ctypes.byref(desc)))


def rlk_logp_fwd(desc, logits, targets, active_mask, logp, lse, workspace, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_fwd(ctypes.byref(desc), _ptr(logits), _ptr(targets), _ptr(active_mask),
                             _ptr(logp), _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)))


def rlk_logp_fwd_noalloc(desc, logits, targets, active_mask, logp, lse, stream=None) -> None:
    _check(_lib.rlk_logp_fwd_noalloc(ctypes.byref(desc), _ptr(logits), _ptr(targets),
                                     _ptr(active_mask), _ptr(logp), _ptr(lse), _stream(stream)))


def rlk_logp_bwd(desc, logits, targets, active_mask, lse, grad_logp, dlogits, ld_dlogits: int,
                 dlogits_dtype: int, workspace, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_bwd(ctypes.byref(desc), _ptr(logits), _ptr(targets), _ptr(active_mask),
                             _ptr(lse), _ptr(grad_logp), _ptr(dlogits), ld_dlogits,
                             dlogits_dtype, _ptr(workspace), ws_bytes, _stream(stream)))


def rlk_logp_ex_workspace_bytes(desc: rlk_logp_desc) -> int:
    return int(_lib.rlk_logp_ex_workspace_bytes(ctypes.byref(desc)))


def rlk_logp_fwd_ex(desc, logits, targets, active_mask, logp, lse, entropy, workspace,
                    stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_fwd_ex(ctypes.byref(desc), _ptr(logits), _ptr(targets),
                                _ptr(active_mask), _ptr(logp), _ptr(lse), _ptr(entropy),
                                _ptr(workspace), ws_bytes, _stream(stream)))


def rlk_logp_bwd_ex(desc, logits, targets, active_mask, lse, entropy, grad_logp, grad_lse,
                    grad_ent, dlogits, ld_dlogits: int, dlogits_dtype: int, workspace,
                    stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_bwd_ex(ctypes.byref(desc), _ptr(logits), _ptr(targets),
                                _ptr(active_mask), _ptr(lse), _ptr(entropy), _ptr(grad_logp),
                                _ptr(grad_lse), _ptr(grad_ent), _ptr(dlogits), ld_dlogits,
                                dlogits_dtype, _ptr(workspace), ws_bytes, _stream(stream)))


def rlk_logp_fwd_bwd_workspace_bytes(desc: rlk_logp_desc) -> int:
    return int(_lib.rlk_logp_fwd_bwd_workspace_bytes(ctypes.byref(desc)))


def rlk_logp_fwd_bwd(desc, logits, targets, active_mask, grad_logp, logp, lse, dlogits,
                     ld_dlogits: int, dlogits_dtype: int, workspace, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_fwd_bwd(ctypes.byref(desc), _ptr(logits), _ptr(targets),
                                 _ptr(active_mask), _ptr(grad_logp), _ptr(logp), _ptr(lse),
                                 _ptr(dlogits), ld_dlogits, dlogits_dtype, _ptr(workspace),
                                 ws_bytes, _stream(stream)))


def rlk_logp_fwd_bwd_ex_workspace_bytes(desc: rlk_logp_desc) -> int:
    return int(_lib.rlk_logp_fwd_bwd_ex_workspace_bytes(ctypes.byref(desc)))


def rlk_logp_fwd_bwd_ex(desc, logits, targets, active_mask, grad_logp, grad_lse, grad_ent, logp,
                        lse, entropy, dlogits, ld_dlogits: int, dlogits_dtype: int, workspace,
                        stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_fwd_bwd_ex(ctypes.byref(desc), _ptr(logits), _ptr(targets),
                                    _ptr(active_mask), _ptr(grad_logp), _ptr(grad_lse),
                                    _ptr(grad_ent), _ptr(logp), _ptr(lse), _ptr(entropy),
                                    _ptr(dlogits), ld_dlogits, dlogits_dtype, _ptr(workspace),
                                    ws_bytes, _stream(stream)))


def rlk_logp_fused_lmhead_workspace_bytes(desc: rlk_logp_desc) -> int:
    return int(_lib.rlk_logp_fused_lmhead_workspace_bytes(ctypes.byref(desc)))


def rlk_logp_fused_lmhead(desc, hidden, weight, hidden_dim: int, targets, active_mask, logp, lse,
                          workspace, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_fused_lmhead(ctypes.byref(desc), _ptr(hidden), _ptr(weight), hidden_dim,
                                      _ptr(targets), _ptr(active_mask), _ptr(logp), _ptr(lse),
                                      _ptr(workspace), ws_bytes, _stream(stream)))


def rlk_logp_fused_lmhead_bwd_workspace_bytes(desc: rlk_logp_desc, hidden_dim: int,
                                              want_dhidden: bool, want_dweight: bool) -> int:
    return int(_lib.rlk_logp_fused_lmhead_bwd_workspace_bytes(ctypes.byref(desc), hidden_dim,
                                                              int(want_dhidden),
                                                              int(want_dweight)))


def rlk_logp_fused_lmhead_bwd(desc, hidden, weight, hidden_dim: int, targets, active_mask, lse,
                              grad_logp, grad_lse, dhidden, dweight, workspace,
                              stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_fused_lmhead_bwd(ctypes.byref(desc), _ptr(hidden), _ptr(weight),
                                          hidden_dim, _ptr(targets), _ptr(active_mask), _ptr(lse),
                                          _ptr(grad_logp), _ptr(grad_lse), _ptr(dhidden),
                                          _ptr(dweight), _ptr(workspace), ws_bytes,
                                          _stream(stream)))


def make_fp8_matrix(q, scale) -> rlk_fp8_matrix:
    """The rlk_fp8_matrix of a pair of tensors (either may be None): values [rows, cols],
    scales [row blocks, column blocks] with any positive strides."""
    # the stride of a dimension of one does not matter, and need not be positive
    rs, cs = (1, 1) if scale is None else scale.stride()
    if scale is not None and 1 in scale.shape:
        rs, cs = (st if n > 1 else 1 for n, st in zip(scale.shape, (rs, cs)))
    return rlk_fp8_matrix(_ptr(q), _ptr(scale), rs, cs)


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def rlk_fp8_quantize(rows: int, cols: int, x, ld_x: int, block_rows: int, q, scale,
                     scale_row_stride: int, scale_col_stride: int, stream=None) -> None:
    _check(_lib.rlk_fp8_quantize(rows, cols, _ptr(x), ld_x, block_rows, _ptr(q), _ptr(scale),
                                 scale_row_stride, scale_col_stride, _stream(stream)))


def rlk_lmhead_logits_fp8(desc, hidden, weight, hidden_dim: int, logits, stream=None) -> None:
    _check(_lib.rlk_lmhead_logits_fp8(ctypes.byref(desc), _ref(hidden), _ref(weight), hidden_dim,
                                      _ptr(logits), _stream(stream)))


def rlk_logp_fused_lmhead_fp8_workspace_bytes(desc: rlk_logp_desc) -> int:
    return int(_lib.rlk_logp_fused_lmhead_fp8_workspace_bytes(ctypes.byref(desc)))


def rlk_logp_fused_lmhead_fp8(desc, hidden, weight, hidden_dim: int, targets, active_mask, logp,
                              lse, workspace, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_fused_lmhead_fp8(ctypes.byref(desc), _ref(hidden), _ref(weight),
                                          hidden_dim, _ptr(targets), _ptr(active_mask),
                                          _ptr(logp), _ptr(lse), _ptr(workspace), ws_bytes,
                                          _stream(stream)))


def rlk_logits_process(desc, logits, rules, out, ld_out: int, out_dtype: int,
                       stream=None) -> None:
    _check(_lib.rlk_logits_process(ctypes.byref(desc), _ptr(logits), _ref(rules), _ptr(out),
                                   ld_out, out_dtype, _stream(stream)))


def rlk_logp_processed_workspace_bytes(desc: rlk_logp_desc) -> int:
    return int(_lib.rlk_logp_processed_workspace_bytes(ctypes.byref(desc)))


def rlk_logp_processed_fwd(desc, logits, rules, targets, active_mask, logp, lse, workspace,
                           stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_processed_fwd(ctypes.byref(desc), _ptr(logits), _ref(rules),
                                       _ptr(targets), _ptr(active_mask), _ptr(logp), _ptr(lse),
                                       _ptr(workspace), ws_bytes, _stream(stream)))


def rlk_logp_processed_bwd(desc, logits, rules, targets, active_mask, lse, grad_logp, grad_lse,
                           dlogits, ld_dlogits: int, dlogits_dtype: int, workspace,
                           stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_logp_processed_bwd(ctypes.byref(desc), _ptr(logits), _ref(rules),
                                       _ptr(targets), _ptr(active_mask), _ptr(lse),
                                       _ptr(grad_logp), _ptr(grad_lse), _ptr(dlogits),
                                       ld_dlogits, dlogits_dtype, _ptr(workspace), ws_bytes,
                                       _stream(stream)))


def rlk_linear_fwd(desc: rlk_linear_desc, x, weight, bias, residual, out, saved,
                   stream=None) -> None:
    _check(_lib.rlk_linear_fwd(ctypes.byref(desc), _ptr(x), _ptr(weight), _ptr(bias),
                               _ptr(residual), _ptr(out), _ptr(saved), _stream(stream)))


def rlk_linear_bwd_workspace_bytes(desc: rlk_linear_desc) -> int:
    return int(_lib.rlk_linear_bwd_workspace_bytes(ctypes.byref(desc)))


def rlk_linear_bwd(desc: rlk_linear_desc, x, weight, saved, grad_out, ld_grad: int, dx, dweight,
                   dbias, workspace, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.rlk_linear_bwd(ctypes.byref(desc), _ptr(x), _ptr(weight), _ptr(saved),
                               _ptr(grad_out), ld_grad, _ptr(dx), _ptr(dweight), _ptr(dbias),
                               _ptr(workspace), ws_bytes, _stream(stream)))


def rlk_logp_tile_geometry(padded_vocab: int, num_vocab_tiles: int, num_virtual_shards: int = 1):
    """Host-only: (tile bounds [T+1] int64, shard first tiles [S+1] int32) as lists."""
    b = (ctypes.c_int64 * (num_vocab_tiles + 1))() if num_vocab_tiles >= 1 else None
    f = (ctypes.c_int32 * (num_virtual_shards + 1))() if num_virtual_shards >= 1 else None
    _check(_lib.rlk_logp_tile_geometry(padded_vocab, num_vocab_tiles, num_virtual_shards,
                                       ctypes.cast(b, ctypes.c_void_p) if b else None,
                                       ctypes.cast(f, ctypes.c_void_p) if f else None))
    return list(b), list(f)


def rlk_status_string(status: int) -> str:
    return _lib.rlk_status_string(status).decode()


def rlk_last_error_detail() -> str:
    return _lib.rlk_last_error_detail().decode()


# -- conveniences: allocate outputs with torch, then call the C entry points ----
# The C entry points take bare pointers and cannot see dtypes, so the conveniences
# check every tensor first (shape and dtype, then device) and raise before anything
# is enqueued.  Targets must already be int32: an int64 tensor would be read as
# pairs of int32 words, and narrowing it here could turn an out-of-range target
# into a valid column.
def _check_logits(logits, name="logits"):
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    if logits.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {logits.dtype}")
    if logits.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")


def _check_rows(name, t, n, dtypes):
    """A per-row vector: 1-D, n elements, contiguous, of one of `dtypes`."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        hint = " (convert with .to(torch.int32))" if name == "targets" else ""
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, "
                        f"got {t.dtype}{hint}")
    if t.dim() != 1 or t.numel() != n:
        raise ValueError(f"{name} must be 1-D with {n} elements, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_device(base, **tensors):
    if base.device.type != "cuda":
        raise ValueError(f"the inputs must be in GPU memory, got {base.device}")
    for name, t in tensors.items():
        if t is not None and t.device != base.device:
            raise ValueError(f"{name} is on {t.device}, the logits on {base.device}")


def _check_workspace(workspace, base):
    """The caller's own: the C entry points see no more than its address and size."""
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != base.device:
        raise ValueError(f"workspace is on {workspace.device}, the inputs on {base.device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


_F32 = (torch.float32,)
_I32 = (torch.int32,)
_MASK = (torch.uint8, torch.bool)


def _check_inputs(logits, targets, active_mask, **vectors):
    """logits bf16 [N, ld]; targets int32 [N]; mask uint8/bool [N] or None; every other
    keyword an fp32 [N] vector or None.  All on the logits' GPU."""
    _check_logits(logits)
    n = logits.shape[0]
    _check_rows("targets", targets, n, _I32)
    if targets is None:
        raise TypeError("targets must be a torch.Tensor")
    _check_rows("active_mask", active_mask, n, _MASK)
    for name, t in vectors.items():
        _check_rows(name, t, n, _F32)
    _check_device(logits, targets=targets, active_mask=active_mask, **vectors)


def _check_vocab(logits, real_vocab, padded_vocab):
    """The kernels read columns [0, V_pad) of every row (V_pad = padded_vocab, or the
    logits' width): a view narrower than that would let them read past it."""
    import operator
    _check_logits(logits)
    v_pad = operator.index(padded_vocab) if padded_vocab else logits.shape[1]
    if operator.index(real_vocab) < 1:
        raise ValueError(f"real_vocab must be positive, got {real_vocab!r}")
    if v_pad > logits.shape[1]:
        raise ValueError(f"padded_vocab={v_pad} exceeds the {logits.shape[1]} columns of the "
                         "logits")
    if real_vocab > v_pad:
        raise ValueError(f"real_vocab={real_vocab} exceeds padded_vocab={v_pad}")
    return v_pad


def _u8_mask(mask):
    if mask is None:
        return None
    return mask.view(torch.uint8) if mask.dtype == torch.bool else mask


# A convenience given a `stream` other than the current one launches there, and takes the
# memory of its results and workspace there too: the allocator hands a freed block out
# again to the stream it was taken on, whose own work is through with it by then, and to no
# other.  (Taken on the current stream, a block could still be in use by work queued there
# that `stream` does not wait for.)  The inputs are the caller's to order: ready on `stream`
# when the call is made, and kept until it is done.
def _torch_stream(stream, device):
    """`stream` as torch knows it; anything with a cuda_stream handle will do."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream.cuda_stream, device=device)


def _call_on(t: torch.Tensor, stream):
    """The context in which memory for a call on t's GPU and `stream` is taken and the call
    is made (none where both are the current ones)."""
    if stream is not None:
        return torch.cuda.stream(_torch_stream(stream, t.device))
    if t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _handed_over(t: torch.Tensor, stream, *results):
    """Records what a call on `stream` returns (Nones apart) on the current stream, where it is
    read: freed, it goes back to the pool of `stream` once the work queued here is through."""
    if stream is None:
        return
    current = torch.cuda.current_stream(t.device)
    if current.cuda_stream != stream.cuda_stream:
        for r in results:
            if r is not None:
                r.record_stream(current)


def _bytes_for(nbytes: int, device) -> torch.Tensor:
    """A workspace of nbytes (0: the descriptor was refused)."""
    if nbytes == 0:
        raise ValueError(f"invalid rlk_logp_desc: {rlk_last_error_detail()}")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def workspace_for(desc: rlk_logp_desc, device) -> torch.Tensor:
    """A fresh workspace of rlk_logp_workspace_bytes(desc) bytes for rlk_logp_fwd
    (its contents on entry do not matter)."""
    return _bytes_for(rlk_logp_workspace_bytes(desc), device)


def forward(logits: torch.Tensor, targets: torch.Tensor, active_mask=None, *, real_vocab: int,
            padded_vocab: int | None = None, num_vocab_tiles: int = 64,
            num_virtual_shards: int = 1, ignore_index: int = -100, validate: bool = False,
            workspace: torch.Tensor | None = None, stream=None):
    """(logp, lse), fp32 [N] each.  logits: bf16 [N, ld] with unit column stride."""
    _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask)
    n = logits.shape[0]
    desc = make_desc(n, real_vocab, padded_vocab or logits.shape[1], logits.stride(0),
                     num_vocab_tiles, num_virtual_shards, ignore_index, validate)
    with _call_on(logits, stream):
        logp = torch.empty(n, dtype=torch.float32, device=logits.device)
        lse = torch.empty(n, dtype=torch.float32, device=logits.device)
        if workspace is None:
            workspace = workspace_for(desc, logits.device)
        else:
            _check_workspace(workspace, logits)
        rlk_logp_fwd(desc, logits, targets, _u8_mask(active_mask), logp, lse, workspace, stream)
    _handed_over(logits, stream, logp, lse)
    return logp, lse


def backward(logits: torch.Tensor, targets: torch.Tensor, active_mask, lse: torch.Tensor,
             grad_logp: torch.Tensor, *, real_vocab: int, padded_vocab: int | None = None,
             out_dtype=torch.float32, ignore_index: int = -100, validate: bool = False,
             num_vocab_tiles: int | None = None, workspace: torch.Tensor | None = None,
             stream=None):
    """dlogits [N, V_pad] (fp32 or bf16)."""
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dlogits dtype must be torch.float32 or torch.bfloat16")
    _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask, lse=lse, grad_logp=grad_logp)
    n = logits.shape[0]
    v_pad = padded_vocab or logits.shape[1]
    tiles = num_vocab_tiles if num_vocab_tiles is not None else min(64, v_pad)
    desc = make_desc(n, real_vocab, v_pad, logits.stride(0), tiles, 1, ignore_index, validate)
    ld_d = (v_pad + 7) // 8 * 8
    code = RLK_DTYPE_BF16 if out_dtype == torch.bfloat16 else RLK_DTYPE_F32
    with _call_on(logits, stream):
        dl = torch.empty((n, ld_d), dtype=out_dtype, device=logits.device)
        if workspace is None:
            workspace = workspace_for(desc, logits.device)
        else:
            _check_workspace(workspace, logits)
        rlk_logp_bwd(desc, logits, targets, _u8_mask(active_mask), lse, grad_logp, dl, ld_d,
                     code, workspace, stream)
    _handed_over(logits, stream, dl)
    return dl[:, :v_pad]


def forward_ex(logits: torch.Tensor, targets: torch.Tensor, active_mask=None, *,
               real_vocab: int, padded_vocab: int | None = None, num_vocab_tiles: int = 64,
               num_virtual_shards: int = 1, ignore_index: int = -100, validate: bool = False,
               workspace: torch.Tensor | None = None, stream=None):
    """(logp, lse, entropy), fp32 [N] each."""
    _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask)
    n = logits.shape[0]
    desc = make_desc(n, real_vocab, padded_vocab or logits.shape[1], logits.stride(0),
                     num_vocab_tiles, num_virtual_shards, ignore_index, validate)
    with _call_on(logits, stream):
        logp = torch.empty(n, dtype=torch.float32, device=logits.device)
        lse = torch.empty(n, dtype=torch.float32, device=logits.device)
        ent = torch.empty(n, dtype=torch.float32, device=logits.device)
        if workspace is None:
            workspace = _bytes_for(rlk_logp_ex_workspace_bytes(desc), logits.device)
        else:
            _check_workspace(workspace, logits)
        rlk_logp_fwd_ex(desc, logits, targets, _u8_mask(active_mask), logp, lse, ent, workspace,
                        stream)
    _handed_over(logits, stream, logp, lse, ent)
    return logp, lse, ent


def backward_ex(logits: torch.Tensor, targets: torch.Tensor, active_mask, lse: torch.Tensor,
                entropy=None, grad_logp=None, grad_lse=None, grad_ent=None, *, real_vocab: int,
                padded_vocab: int | None = None, out_dtype=torch.float32,
                ignore_index: int = -100, validate: bool = False,
                num_vocab_tiles: int | None = None, workspace: torch.Tensor | None = None,
                stream=None):
    """dlogits [N, V_pad] of a loss on (logp, lse, entropy); absent gradients are zero."""
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dlogits dtype must be torch.float32 or torch.bfloat16")
    _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask, lse=lse, entropy=entropy, grad_logp=grad_logp,
                  grad_lse=grad_lse, grad_ent=grad_ent)
    n = logits.shape[0]
    v_pad = padded_vocab or logits.shape[1]
    tiles = num_vocab_tiles if num_vocab_tiles is not None else min(64, v_pad)
    desc = make_desc(n, real_vocab, v_pad, logits.stride(0), tiles, 1, ignore_index, validate)
    ld_d = (v_pad + 7) // 8 * 8
    code = RLK_DTYPE_BF16 if out_dtype == torch.bfloat16 else RLK_DTYPE_F32
    with _call_on(logits, stream):
        dl = torch.empty((n, ld_d), dtype=out_dtype, device=logits.device)
        if workspace is None:
            workspace = workspace_for(desc, logits.device)
        else:
            _check_workspace(workspace, logits)
        rlk_logp_bwd_ex(desc, logits, targets, _u8_mask(active_mask), lse, entropy, grad_logp,
                        grad_lse, grad_ent, dl, ld_d, code, workspace, stream)
    _handed_over(logits, stream, dl)
    return dl[:, :v_pad]


class _SelectedTokenLogprob(torch.autograd.Function):
    """(logp, lse, entropy) of bf16 logits, differentiable in all three; the forward
    and the backward are rlk_logp_fwd_ex and rlk_logp_bwd_ex."""

    @staticmethod
    def forward(ctx, logits, targets, active_mask, real_vocab, padded_vocab, num_vocab_tiles,
                ignore_index):
        logp, lse, ent = forward_ex(logits, targets, active_mask, real_vocab=real_vocab,
                                    padded_vocab=padded_vocab, num_vocab_tiles=num_vocab_tiles,
                                    ignore_index=ignore_index)
        ctx.save_for_backward(logits, targets, lse, ent)
        ctx.active_mask = active_mask
        ctx.cfg = (real_vocab, padded_vocab, num_vocab_tiles, ignore_index)
        return logp, lse, ent

    @staticmethod
    def backward(ctx, g_logp, g_lse, g_ent):
        logits, targets, lse, ent = ctx.saved_tensors
        real_vocab, padded_vocab, num_vocab_tiles, ignore_index = ctx.cfg

        def vec(t):
            return None if t is None else t.contiguous().float()
        g_logp, g_lse, g_ent = vec(g_logp), vec(g_lse), vec(g_ent)
        if g_logp is None and g_lse is None and g_ent is None:
            return (None,) * 7
        v_pad = padded_vocab or logits.shape[1]
        d = backward_ex(logits, targets, ctx.active_mask, lse, ent, g_logp, g_lse, g_ent,
                        real_vocab=real_vocab, padded_vocab=v_pad, out_dtype=logits.dtype,
                        ignore_index=ignore_index, num_vocab_tiles=num_vocab_tiles)
        if d.shape == logits.shape and d.is_contiguous():
            grad = d
        else:
            grad = torch.zeros_like(logits)
            grad[:, :v_pad] = d
        return grad, None, None, None, None, None, None


def selected_token_logprob(logits: torch.Tensor, targets: torch.Tensor, active_mask=None, *,
                           real_vocab: int, padded_vocab: int | None = None,
                           num_vocab_tiles: int = 64, ignore_index: int = -100):
    """The op as a differentiable torch function: returns (logp, lse, entropy), fp32 [N].

    This is the interface a loss built on the selected-token log-probability
    consumes (a policy-gradient loss on logp, a penalty on LSE, an entropy bonus):
    autograd hands the three upstream gradients to rlk_logp_bwd_ex.  logits is
    bf16 [N, ld] with unit column stride; its gradient has its dtype.
    """
    _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask)
    return _SelectedTokenLogprob.apply(logits, targets, active_mask, real_vocab, padded_vocab,
                                       num_vocab_tiles, ignore_index)


def forward_backward(logits: torch.Tensor, targets: torch.Tensor, active_mask,
                     grad_logp: torch.Tensor, *, real_vocab: int, padded_vocab: int | None = None,
                     num_vocab_tiles: int = 64, num_virtual_shards: int = 1,
                     out_dtype=torch.float32, ignore_index: int = -100, validate: bool = False,
                     workspace: torch.Tensor | None = None, stream=None):
    """(logp, lse, dlogits [N, V_pad]) in one launch, with g known up front.

    Bitwise the outputs of forward() then backward().  With the default workspace
    (rlk_logp_fwd_bwd_workspace_bytes) the unit schedule runs where the geometry
    takes it (T <= 64 tiles of 8 to about 2,500 columns): blocks of 8 tiles keep
    their logits on chip and exchange partials through the workspace; a
    256-byte workspace selects one block per row."""
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dlogits dtype must be torch.float32 or torch.bfloat16")
    if grad_logp is None:
        raise TypeError("grad_logp must be a torch.Tensor")
    _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask, grad_logp=grad_logp)
    n = logits.shape[0]
    v_pad = padded_vocab or logits.shape[1]
    desc = make_desc(n, real_vocab, v_pad, logits.stride(0), num_vocab_tiles, num_virtual_shards,
                     ignore_index, validate)
    ld_d = (v_pad + 7) // 8 * 8
    code = RLK_DTYPE_BF16 if out_dtype == torch.bfloat16 else RLK_DTYPE_F32
    with _call_on(logits, stream):
        logp = torch.empty(n, dtype=torch.float32, device=logits.device)
        lse = torch.empty(n, dtype=torch.float32, device=logits.device)
        dl = torch.empty((n, ld_d), dtype=out_dtype, device=logits.device)
        if workspace is None:
            workspace = _bytes_for(rlk_logp_fwd_bwd_workspace_bytes(desc), logits.device)
        else:
            _check_workspace(workspace, logits)
        rlk_logp_fwd_bwd(desc, logits, targets, _u8_mask(active_mask), grad_logp, logp, lse, dl,
                         ld_d, code, workspace, stream)
    _handed_over(logits, stream, logp, lse, dl)
    return logp, lse, dl[:, :v_pad]


def forward_backward_ex(logits: torch.Tensor, targets: torch.Tensor, active_mask,
                        grad_logp=None, grad_lse=None, grad_ent=None, *, real_vocab: int,
                        padded_vocab: int | None = None, num_vocab_tiles: int = 64,
                        num_virtual_shards: int = 1, out_dtype=torch.float32,
                        ignore_index: int = -100, validate: bool = False,
                        workspace: torch.Tensor | None = None, stream=None):
    """(logp, lse, entropy, dlogits [N, V_pad]): forward_ex() then backward_ex() in one
    launch where the unit schedule takes the geometry (the same bits either way);
    absent gradients are zero, at least one must be given."""
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dlogits dtype must be torch.float32 or torch.bfloat16")
    _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask, grad_logp=grad_logp, grad_lse=grad_lse,
                  grad_ent=grad_ent)
    n = logits.shape[0]
    v_pad = padded_vocab or logits.shape[1]
    desc = make_desc(n, real_vocab, v_pad, logits.stride(0), num_vocab_tiles, num_virtual_shards,
                     ignore_index, validate)
    ld_d = (v_pad + 7) // 8 * 8
    code = RLK_DTYPE_BF16 if out_dtype == torch.bfloat16 else RLK_DTYPE_F32
    with _call_on(logits, stream):
        logp = torch.empty(n, dtype=torch.float32, device=logits.device)
        lse = torch.empty(n, dtype=torch.float32, device=logits.device)
        ent = torch.empty(n, dtype=torch.float32, device=logits.device)
        dl = torch.empty((n, ld_d), dtype=out_dtype, device=logits.device)
        if workspace is None:
            workspace = _bytes_for(rlk_logp_fwd_bwd_ex_workspace_bytes(desc), logits.device)
        else:
            _check_workspace(workspace, logits)
        rlk_logp_fwd_bwd_ex(desc, logits, targets, _u8_mask(active_mask), grad_logp, grad_lse,
                            grad_ent, logp, lse, ent, dl, ld_d, code, workspace, stream)
    _handed_over(logits, stream, logp, lse, ent, dl)
    return logp, lse, ent, dl[:, :v_pad]


def _check_lmhead(hidden, weight, targets, active_mask, real_vocab, **vectors):
    """hidden bf16 [N, K], weight bf16 [>= real_vocab, K], both contiguous; targets, mask and
    vectors as in _check_inputs.  All on the hidden states' GPU."""
    for name, t in (("hidden", hidden), ("weight", weight)):
        _check_logits(t, name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if weight.shape[1] != hidden.shape[1]:
        raise ValueError(f"weight has {weight.shape[1]} columns, hidden {hidden.shape[1]}")
    if weight.shape[0] < real_vocab:
        raise ValueError(f"weight has {weight.shape[0]} rows, fewer than real_vocab={real_vocab}")
    n = hidden.shape[0]
    _check_rows("targets", targets, n, _I32)
    if targets is None:
        raise TypeError("targets must be a torch.Tensor")
    _check_rows("active_mask", active_mask, n, _MASK)
    for name, t in vectors.items():
        _check_rows(name, t, n, _F32)
    _check_device(hidden, weight=weight, targets=targets, active_mask=active_mask, **vectors)


def fused_lmhead(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                 active_mask=None, *, real_vocab: int, padded_vocab: int | None = None,
                 num_vocab_tiles: int = 64, num_virtual_shards: int = 1,
                 ignore_index: int = -100, validate: bool = False,
                 workspace: torch.Tensor | None = None, stream=None):
    """(logp, lse) of z = hidden . weight^T without materialising z.
    hidden: bf16 [N, K] contiguous; weight: bf16 [V_pad, K] contiguous."""
    _check_lmhead(hidden, weight, targets, active_mask, real_vocab)
    v_pad = padded_vocab or weight.shape[0]
    desc = make_desc(hidden.shape[0], real_vocab, v_pad, v_pad, num_vocab_tiles,
                     num_virtual_shards, ignore_index, validate)
    return _run_lmhead(desc, hidden, weight, targets, active_mask, workspace, stream)


def _run_lmhead(desc, hidden, weight, targets, active_mask, workspace=None, stream=None):
    n, k = hidden.shape
    with _call_on(hidden, stream):
        logp = torch.empty(n, dtype=torch.float32, device=hidden.device)
        lse = torch.empty(n, dtype=torch.float32, device=hidden.device)
        if workspace is None:
            workspace = _bytes_for(rlk_logp_fused_lmhead_workspace_bytes(desc), hidden.device)
        else:
            _check_workspace(workspace, hidden)
        rlk_logp_fused_lmhead(desc, hidden, weight, k, targets, _u8_mask(active_mask), logp, lse,
                              workspace, stream)
    _handed_over(hidden, stream, logp, lse)
    return logp, lse


def fused_lmhead_backward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                          active_mask, lse: torch.Tensor, grad_logp=None, grad_lse=None, *,
                          real_vocab: int, want_hidden: bool = True, want_weight: bool = True,
                          ignore_index: int = -100, validate: bool = False,
                          workspace: torch.Tensor | None = None, stream=None):
    """(dhidden, dweight) in bf16, with the shapes of hidden and weight, of a loss on
    fused_lmhead's logp and LSE; absent gradients are zero.  The one that is not wanted
    is not computed and comes back as None."""
    if lse is None:
        raise TypeError("lse must be a torch.Tensor")
    if grad_logp is None and grad_lse is None:
        raise TypeError("at least one of grad_logp and grad_lse must be a torch.Tensor")
    if not (want_hidden or want_weight):
        raise ValueError("at least one of want_hidden and want_weight must be true")
    _check_lmhead(hidden, weight, targets, active_mask, real_vocab, lse=lse, grad_logp=grad_logp,
                  grad_lse=grad_lse)
    rows = weight.shape[0]
    desc = make_desc(hidden.shape[0], real_vocab, rows, rows, 1, 1, ignore_index, validate)
    return _run_lmhead_backward(desc, hidden, weight, targets, active_mask, lse, grad_logp,
                                grad_lse, want_hidden, want_weight, workspace, stream)


def _run_lmhead_backward(desc, hidden, weight, targets, active_mask, lse, grad_logp, grad_lse,
                         want_hidden, want_weight, workspace=None, stream=None):
    k = hidden.shape[1]
    with _call_on(hidden, stream):
        dh = torch.empty_like(hidden) if want_hidden else None
        dw = torch.empty_like(weight) if want_weight else None
        if workspace is None:
            workspace = _bytes_for(rlk_logp_fused_lmhead_bwd_workspace_bytes(
                desc, k, want_hidden, want_weight), hidden.device)
        else:
            _check_workspace(workspace, hidden)
        rlk_logp_fused_lmhead_bwd(desc, hidden, weight, k, targets, _u8_mask(active_mask), lse,
                                  grad_logp, grad_lse, dh, dw, workspace, stream)
    _handed_over(hidden, stream, dh, dw)
    return dh, dw


class _LmheadSelectedTokenLogprob(torch.autograd.Function):
    """(logp, lse) of bf16 hidden states and weight, differentiable in both; the forward
    and the backward are rlk_logp_fused_lmhead and rlk_logp_fused_lmhead_bwd."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, active_mask, real_vocab, padded_vocab,
                num_vocab_tiles, ignore_index):
        n, rows = hidden.shape[0], weight.shape[0]
        v_pad = padded_vocab or rows
        logp, lse = _run_lmhead(make_desc(n, real_vocab, v_pad, v_pad, num_vocab_tiles, 1,
                                          ignore_index),
                                hidden, weight, targets, active_mask)
        ctx.save_for_backward(hidden, weight, targets, active_mask, lse)
        ctx.desc = make_desc(n, real_vocab, rows, rows, 1, 1, ignore_index)
        ctx.set_materialize_grads(False)
        return logp, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logp, g_lse):
        # What was saved has been checked, and the gradients have the outputs' shape and
        # device: nothing is checked again.  Autograd's own thread runs this with cold
        # caches, where the checks took as long as two launches (64 tokens x 128 x 2000,
        # forward and backward: 147 -> 132 us with a forward that checks once).
        want_hidden, want_weight = ctx.needs_input_grad[:2]
        if (g_logp is None and g_lse is None) or not (want_hidden or want_weight):
            return (None,) * 8

        def vec(t):
            return None if t is None else t.contiguous().float()
        # (hooks on saved tensors may hand back another layout)
        hidden, weight, targets, active_mask, lse = (
            None if t is None else t.contiguous() for t in ctx.saved_tensors)
        dh, dw = _run_lmhead_backward(ctx.desc, hidden, weight, targets, active_mask, lse,
                                      vec(g_logp), vec(g_lse), want_hidden, want_weight)
        return dh, dw, None, None, None, None, None, None


def lmhead_selected_token_logprob(hidden: torch.Tensor, weight: torch.Tensor,
                                  targets: torch.Tensor, active_mask=None, *, real_vocab: int,
                                  padded_vocab: int | None = None, num_vocab_tiles: int = 64,
                                  ignore_index: int = -100):
    """fused_lmhead as a differentiable torch function: returns (logp, lse), fp32 [N].

    The logits z = hidden . weight^T are never kept: the backward takes them again in
    pieces of the vocabulary.  The softmax cross entropy of a token is -logp; a loss
    on logp and LSE hands its gradients to rlk_logp_fused_lmhead_bwd, which computes
    only the gradients that autograd asks for.  hidden: bf16 [N, K] contiguous;
    weight: bf16 [V_pad, K] contiguous; their gradients are bf16.  Where a training step is
    captured into a HIP graph, no eager autograd graph of the same leaves may be alive: torch
    ends the process.
    """
    _check_lmhead(hidden, weight, targets, active_mask, real_vocab)
    return _LmheadSelectedTokenLogprob.apply(hidden, weight, targets, active_mask, real_vocab,
                                             padded_vocab, num_vocab_tiles, ignore_index)


# -- the LM-head in 8-bit floating point ----------------------------------------
FP8_BLOCK = 128  # columns (and weight rows) that share a scale


def quantize_fp8(x: torch.Tensor, block_rows: int = 1, *, stream=None):
    """(q, scale): bf16 x [R, K] as e4m3 values [R, K] and the fp32 scales
    [ceil(R / block_rows), K / 128] of its block_rows x 128 blocks, so that q * scale stands
    for x.  block_rows is 1 for hidden states and 128 for a weight (its real rows alone, where
    the padding may hold anything: they would share a scale).  The scales of 1 x 128
    blocks lie with the tokens contiguous (a transposed view), as the products read them."""
    _check_logits(x, "x")
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError(f"block_rows must be 1 or {FP8_BLOCK}, got {block_rows!r}")
    n, k = x.shape
    if k == 0 or k % FP8_BLOCK:
        raise ValueError(f"x must have a multiple of {FP8_BLOCK} columns, got {k}")
    _check_device(x)
    col_blocks = k // FP8_BLOCK
    with _call_on(x, stream):
        q = torch.empty((n, k), dtype=torch.float8_e4m3fn, device=x.device)
        if block_rows == 1:
            strides = 1, n or 1
            scale = torch.empty_strided((n, col_blocks), strides, device=x.device)
        else:
            strides = col_blocks, 1
            scale = torch.empty((-(-n // block_rows), col_blocks), device=x.device)
        if n:
            rlk_fp8_quantize(n, k, x, x.stride(0) if n > 1 else k, block_rows, q, scale, *strides,
                             stream)
    _handed_over(x, stream, q, scale)
    return q, scale


def _check_fp8(name, q, scale, block_rows):
    """An e4m3 matrix [R, K], contiguous, and its fp32 scales [ceil(R / block_rows), K / 128]."""
    if not isinstance(q, torch.Tensor) or not isinstance(scale, torch.Tensor):
        raise TypeError(f"{name} and its scales must be torch.Tensors")
    if q.dtype != torch.float8_e4m3fn:
        raise TypeError(f"{name} must be float8_e4m3fn, got {q.dtype}")
    if scale.dtype != torch.float32:
        raise TypeError(f"the scales of {name} must be float32, got {scale.dtype}")
    if q.dim() != 2 or not q.is_contiguous():
        raise ValueError(f"{name} must be 2-D and contiguous")
    if q.shape[1] == 0 or q.shape[1] % FP8_BLOCK:
        raise ValueError(f"{name} must have a multiple of {FP8_BLOCK} columns, got {q.shape[1]}")
    want = (-(-q.shape[0] // block_rows), q.shape[1] // FP8_BLOCK)
    if tuple(scale.shape) != want:
        raise ValueError(f"the scales of {name} must have shape {want}, got {tuple(scale.shape)}")
    if min(scale.stride()) < 1 and any(n > 1 and st < 1 for n, st in
                                       zip(scale.shape, scale.stride())):
        raise ValueError(f"the scales of {name} must have positive strides")


def _check_lmhead_fp8(hidden, weight_q, weight_scale, real_vocab, **rows):
    """hidden: bf16 [N, K], or its (q, scale) pair; rows: targets and active_mask, where there
    are any.  All on one GPU."""
    _check_fp8("weight_q", weight_q, weight_scale, FP8_BLOCK)
    if isinstance(hidden, (tuple, list)):
        _check_fp8("hidden", *hidden, 1)
        q, parts = hidden[0], {"hidden scales": hidden[1]}
    else:
        _check_logits(hidden, "hidden")
        q, parts = hidden, {}
    if weight_q.shape[1] != q.shape[1]:
        raise ValueError(f"weight_q has {weight_q.shape[1]} columns, hidden {q.shape[1]}")
    if weight_q.shape[0] < real_vocab:
        raise ValueError(f"weight_q has {weight_q.shape[0]} rows, fewer than "
                         f"real_vocab={real_vocab}")
    if rows:
        if rows["targets"] is None:
            raise TypeError("targets must be a torch.Tensor")
        _check_rows("targets", rows["targets"], q.shape[0], _I32)
        _check_rows("active_mask", rows["active_mask"], q.shape[0], _MASK)
    _check_device(q, weight_q=weight_q, weight_scale=weight_scale, **parts, **rows)
    return q


def _fp8_operand(hidden, nbytes, stream):
    """(rlk_fp8_matrix of the hidden states, a buffer of at least nbytes): bf16 ones are cast on
    `stream`, behind the nbytes of that buffer (one allocation costs less than three)."""
    if isinstance(hidden, (tuple, list)):
        return make_fp8_matrix(*hidden), _bytes_for(nbytes, hidden[0].device) if nbytes else None
    n, k = hidden.shape
    at = -(-nbytes // 256) * 256
    scales = at + -(-n * k // 256) * 256
    buffer = _bytes_for(scales + n * k // FP8_BLOCK * 4 + 256, hidden.device)
    base = buffer.data_ptr()
    if n:
        _check(_lib.rlk_fp8_quantize(n, k, hidden.data_ptr(), hidden.stride(0) if n > 1 else k,
                                     1, base + at, base + scales, 1, n, _stream(stream)))
    return rlk_fp8_matrix(base + at, base + scales, 1, n or 1), buffer


def lmhead_logits_fp8(hidden, weight_q: torch.Tensor, weight_scale: torch.Tensor, *,
                      real_vocab: int, padded_vocab: int | None = None, stream=None):
    """bf16 logits [N, V_pad] of an 8-bit LM-head, as forward() and its kin take them (their
    rows are padded to a multiple of 8 columns); columns [real_vocab, V_pad) are -inf.

    hidden: bf16 [N, K], cast to e4m3 with one scale per token and 128 columns, or the
    (q, scale) pair of quantize_fp8(x, 1).  weight_q, weight_scale: quantize_fp8(W, 128)."""
    x = _check_lmhead_fp8(hidden, weight_q, weight_scale, real_vocab)
    with _call_on(x, stream):
        matrix, buffer = _fp8_operand(hidden, 0, stream)
        n, k = x.shape
        v_pad = padded_vocab or weight_q.shape[0]
        ld = (v_pad + 7) // 8 * 8
        logits = torch.empty((n, ld), dtype=torch.bfloat16, device=x.device)
        rlk_lmhead_logits_fp8(make_desc(n, real_vocab, v_pad, ld, 1), matrix,
                              make_fp8_matrix(weight_q, weight_scale), k, logits, stream)
    _handed_over(x, stream, logits)
    return logits if ld == v_pad else logits[:, :v_pad]


def fused_lmhead_fp8(hidden, weight_q: torch.Tensor, weight_scale: torch.Tensor,
                     targets: torch.Tensor, active_mask=None, *, real_vocab: int,
                     padded_vocab: int | None = None, num_vocab_tiles: int = 64,
                     num_virtual_shards: int = 1, ignore_index: int = -100,
                     validate: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """fused_lmhead with an 8-bit weight: (logp, lse) of the logits of lmhead_logits_fp8,
    taken before their rounding and never written.  hidden, weight_q and weight_scale as
    there; the rest as for fused_lmhead."""
    x = _check_lmhead_fp8(hidden, weight_q, weight_scale, real_vocab, targets=targets,
                          active_mask=active_mask)
    n = x.shape[0]
    v_pad = padded_vocab or weight_q.shape[0]
    desc = make_desc(n, real_vocab, v_pad, v_pad, num_vocab_tiles, num_virtual_shards,
                     ignore_index, validate)
    with _call_on(x, stream):
        nbytes = rlk_logp_fused_lmhead_fp8_workspace_bytes(desc)
        if nbytes == 0:
            raise ValueError(f"invalid rlk_logp_desc: {rlk_last_error_detail()}")
        if workspace is not None:
            _check_workspace(workspace, x)
        matrix, buffer = _fp8_operand(hidden, nbytes if workspace is None else 0, stream)
        if workspace is None:
            workspace = buffer
        logp = torch.empty(n, dtype=torch.float32, device=x.device)
        lse = torch.empty(n, dtype=torch.float32, device=x.device)
        rlk_logp_fused_lmhead_fp8(desc, matrix,
                                  make_fp8_matrix(weight_q, weight_scale), x.shape[1], targets,
                                  _u8_mask(active_mask), logp, lse, workspace, stream)
    _handed_over(x, stream, logp, lse)
    return logp, lse


# -- what a sampler does to logits -------------------------------------------------
class LogitRules:
    """The rules of a call's N rows: penalties for repeated tokens, a bias, a temperature and a
    grammar's mask.  For row r and column j, with s = j occurs in the row's history and c = how
    often in the generated part of it,

        x1 = (x / repetition if x > 0 else x * repetition) if s else x
        x2 = x1 - frequency c - (presence if c > 0 else 0)
        y  = (x2 + bias_j) / temperature,  -inf where the grammar bars j

    in this order (an engine that adds its bias or divides by its temperature first draws from
    another distribution).

    Every rule may be absent.  repetition, presence, frequency, temperature: fp32 [N].
    history: int32 [H] tokens; row r's are history[history_begin[r]:history_end[r]] (int64 [N]
    each), of which those in front of history_split[r] are its prompt (none without it); rows may
    share tokens, and tokens outside the vocabulary count for nothing.  bias: fp32 [rows, >= V],
    allow: int32 bits [rows, >= ceil(V / 32)], bit j % 32 of word j / 32 set where column j is
    allowed; either with one row (or 1-D) for all, with N, or with an int32 [N] index of the row
    to take (outside the table: none).

    The tensors are checked here, once, and have to stay as they are made: contents may change
    between calls.  They are constants: no gradient reaches them."""

    __slots__ = ("tensors", "names", "rows", "device", "struct", "bias_columns", "allow_words")

    def __init__(self, *, repetition=None, presence=None, frequency=None, temperature=None,
                 history=None, history_begin=None, history_split=None, history_end=None,
                 bias=None, bias_index=None, allow=None, allow_index=None):
        if history is None:
            if not (history_begin is history_split is history_end is None):
                raise TypeError("history_begin, history_split and history_end need a history")
        elif history_begin is None or history_end is None:
            raise TypeError("a history needs history_begin and history_end")
        if bias is None and bias_index is not None:
            raise TypeError("bias_index needs a bias")
        if allow is None and allow_index is not None:
            raise TypeError("allow_index needs allow")
        f32, i32, i64 = torch.float32, torch.int32, torch.int64
        rows = where = None
        kept, names, ptrs = [], [], []
        for name, t, dtype in (("repetition", repetition, f32), ("presence", presence, f32),
                               ("frequency", frequency, f32), ("temperature", temperature, f32),
                               ("history", history, i32), ("history_begin", history_begin, i64),
                               ("history_split", history_split, i64),
                               ("history_end", history_end, i64),
                               ("bias_index", bias_index, i32), ("allow_index", allow_index, i32)):
            if t is None:
                ptrs.append(None)
                continue
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.dtype is not dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            if t.dim() != 1 or not t.is_contiguous():
                raise ValueError(f"{name} must be 1-D and contiguous")
            if name != "history":  # (whose tensor may be an index too)
                if rows is None:
                    rows = t.numel()
                elif t.numel() != rows:
                    raise ValueError(f"{name} has {t.numel()} elements, other rules {rows}")
            if where is None:
                where = t.get_device()
            elif t.get_device() != where:
                raise ValueError(f"{name} is on {t.device}, another rule on {kept[0].device}")
            kept.append(t)
            names.append(name)
            ptrs.append(t.data_ptr())
        tables = []
        for name, t, dtype, index in (("bias", bias, f32, bias_index),
                                      ("allow", allow, i32, allow_index)):
            if t is None:
                tables.append((None, 0, 0, None))
                continue
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.dtype is not dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            if t.dim() not in (1, 2) or (t.shape[-1] > 1 and t.stride(-1) != 1):
                raise ValueError(f"{name} must be 1-D or 2-D with unit column stride")
            n, width = (1, t.shape[0]) if t.dim() == 1 else t.shape
            ld = width if n <= 1 else t.stride(0)
            if n < 1 or ld < width:
                raise ValueError(f"{name} must have a row, and rows that do not overlap")
            if index is None and n > 1:
                if rows is None:
                    rows = n
                elif n != rows:
                    raise ValueError(f"{name} without an index has {n} rows, other rules {rows}")
            if where is None:
                where = t.get_device()
            elif t.get_device() != where:
                raise ValueError(f"{name} is on {t.device}, another rule on {kept[0].device}")
            kept.append(t)
            names.append(name)
            tables.append((t.data_ptr(), n, ld, width))
        (bias_ptr, bias_rows, ld_bias, self.bias_columns), \
            (allow_ptr, allow_rows, ld_allow, self.allow_words) = tables
        self.tensors, self.names, self.rows = tuple(kept), tuple(names), rows
        self.device = kept[0].device if kept else None
        self.struct = rlk_logit_rules(
            *ptrs[:5], 0 if history is None else history.numel(), *ptrs[5:8], bias_ptr, bias_rows,
            ld_bias, ptrs[8], allow_ptr, allow_rows, ld_allow, ptrs[9])


def _check_rules(rules, logits, real_vocab):
    if not isinstance(rules, LogitRules):
        raise TypeError("rules must be LogitRules")
    if rules.rows is not None and rules.rows != logits.shape[0]:
        raise ValueError(f"the rules have {rules.rows} rows, the logits {logits.shape[0]}")
    if rules.bias_columns is not None and rules.bias_columns < real_vocab:
        raise ValueError(f"bias has {rules.bias_columns} columns, fewer than "
                         f"real_vocab={real_vocab}")
    if rules.allow_words is not None and rules.allow_words * 32 < real_vocab:
        raise ValueError(f"allow has {rules.allow_words} words, fewer than "
                         f"real_vocab={real_vocab} needs")
    if rules.device is not None and rules.device != logits.device:
        raise ValueError(f"the rules are on {rules.device}, the logits on {logits.device}")


def process_logits(logits: torch.Tensor, rules: LogitRules, *, real_vocab: int,
                   padded_vocab: int | None = None, out_dtype=torch.bfloat16,
                   out: torch.Tensor | None = None, stream=None):
    """The processed logits [N, V_pad] (bf16 or fp32; rows padded to a multiple of 8 columns,
    columns [real_vocab, V_pad) -inf).  logits: bf16 [N, ld] with unit column stride.  With `out`
    they are written there, a tensor of out_dtype with at least V_pad columns, whose rows lie
    beside those of the logits or are the logits themselves; what lies behind V_pad stays.  No
    gradient: processed_selected_token_logprob has one."""
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    v_pad = _check_vocab(logits, real_vocab, padded_vocab)
    _check_rules(rules, logits, real_vocab)
    n = logits.shape[0]
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.dtype != out_dtype:
            raise TypeError(f"out must be a tensor of {out_dtype}")
        if out.dim() != 2 or out.shape[0] != n or out.shape[1] < v_pad or out.stride(1) != 1:
            raise ValueError(f"out must have {n} rows of at least {v_pad} columns, of unit "
                             "stride")
        if out.requires_grad and torch.is_grad_enabled():
            raise ValueError("out requires a gradient, and process_logits has none")
    _check_device(logits, out=out)
    code = RLK_DTYPE_BF16 if out_dtype == torch.bfloat16 else RLK_DTYPE_F32
    desc = make_desc(n, real_vocab, v_pad, logits.stride(0), 1)
    with _call_on(logits, stream):
        if out is None:
            ld = (v_pad + 7) // 8 * 8
            y = torch.empty((n, ld), dtype=out_dtype, device=logits.device)
        else:
            y, ld = out, out.stride(0)
        rlk_logits_process(desc, logits, rules.struct, y, ld, code, stream)
    if out is not None:
        # (autograd refuses a backward pass that has saved what was there)
        if not out.is_inference():
            torch.autograd.graph.increment_version(out)
        return out
    _handed_over(logits, stream, y)
    return y if ld == v_pad else y[:, :v_pad]


def processed_forward(logits: torch.Tensor, targets: torch.Tensor, rules: LogitRules,
                      active_mask=None, *, real_vocab: int, padded_vocab: int | None = None,
                      ignore_index: int = -100, validate: bool = False,
                      workspace: torch.Tensor | None = None, stream=None):
    """(logp, lse), fp32 [N] each, of the processed logits (see LogitRules), which are not
    written: forward() of process_logits(), but for the rounding."""
    v_pad = _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask)
    _check_rules(rules, logits, real_vocab)
    desc = make_desc(logits.shape[0], real_vocab, v_pad, logits.stride(0), 1, 1, ignore_index,
                     validate)
    return _run_processed(desc, logits, targets, rules, active_mask, workspace, stream)


def _run_processed(desc, logits, targets, rules, active_mask, workspace=None, stream=None):
    n = logits.shape[0]
    with _call_on(logits, stream):
        logp = torch.empty(n, dtype=torch.float32, device=logits.device)
        lse = torch.empty(n, dtype=torch.float32, device=logits.device)
        if workspace is None:
            workspace = _bytes_for(rlk_logp_processed_workspace_bytes(desc), logits.device)
        else:
            _check_workspace(workspace, logits)
        rlk_logp_processed_fwd(desc, logits, rules.struct, targets, _u8_mask(active_mask), logp,
                               lse, workspace, stream)
    _handed_over(logits, stream, logp, lse)
    return logp, lse


def processed_backward(logits: torch.Tensor, targets: torch.Tensor, rules: LogitRules,
                       active_mask, lse: torch.Tensor, grad_logp=None, grad_lse=None, *,
                       real_vocab: int, padded_vocab: int | None = None,
                       out_dtype=torch.float32, ignore_index: int = -100,
                       validate: bool = False, workspace: torch.Tensor | None = None,
                       stream=None):
    """dlogits [N, V_pad] (fp32 or bf16), to the raw logits, of a loss on processed_forward's
    logp and LSE; absent gradients are zero."""
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dlogits dtype must be torch.float32 or torch.bfloat16")
    if lse is None:
        raise TypeError("lse must be a torch.Tensor")
    if grad_logp is None and grad_lse is None:
        raise TypeError("at least one of grad_logp and grad_lse must be a torch.Tensor")
    v_pad = _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask, lse=lse, grad_logp=grad_logp, grad_lse=grad_lse)
    _check_rules(rules, logits, real_vocab)
    desc = make_desc(logits.shape[0], real_vocab, v_pad, logits.stride(0), 1, 1, ignore_index,
                     validate)
    return _run_processed_backward(desc, logits, targets, rules, active_mask, lse, grad_logp,
                                   grad_lse, out_dtype, workspace, stream)


def _run_processed_backward(desc, logits, targets, rules, active_mask, lse, grad_logp, grad_lse,
                            out_dtype, workspace=None, stream=None):
    v_pad = desc.padded_vocab
    ld = (v_pad + 7) // 8 * 8
    code = RLK_DTYPE_BF16 if out_dtype == torch.bfloat16 else RLK_DTYPE_F32
    with _call_on(logits, stream):
        dl = torch.empty((logits.shape[0], ld), dtype=out_dtype, device=logits.device)
        if workspace is None:
            workspace = _bytes_for(256, logits.device)
        else:
            _check_workspace(workspace, logits)
        rlk_logp_processed_bwd(desc, logits, rules.struct, targets, _u8_mask(active_mask), lse,
                               grad_logp, grad_lse, dl, ld, code, workspace, stream)
    _handed_over(logits, stream, dl)
    return dl if ld == v_pad else dl[:, :v_pad]


class _ProcessedSelectedTokenLogprob(torch.autograd.Function):
    """(logp, lse) of bf16 logits under the rules, differentiable in the logits; the forward
    and the backward are rlk_logp_processed_fwd and rlk_logp_processed_bwd."""

    @staticmethod
    def forward(ctx, logits, targets, rules, active_mask, real_vocab, v_pad, ignore_index):
        desc = make_desc(logits.shape[0], real_vocab, v_pad, logits.stride(0), 1, 1, ignore_index)
        logp, lse = _run_processed(desc, logits, targets, rules, active_mask)
        # (the rules' tensors too: one that is changed in between is refused by autograd)
        ctx.save_for_backward(logits, targets, active_mask, lse, *rules.tensors)
        ctx.rules = rules
        # every column of the gradient is written: +0 from real_vocab on
        ctx.desc = make_desc(logits.shape[0], real_vocab, logits.shape[1], logits.stride(0), 1, 1,
                             ignore_index)
        ctx.set_materialize_grads(False)
        return logp, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logp, g_lse):
        if g_logp is None and g_lse is None:
            return (None,) * 7

        def vec(t):
            return None if t is None else t.contiguous().float()
        logits, targets, active_mask, lse, *of_rules = ctx.saved_tensors
        desc, rules = ctx.desc, ctx.rules
        # Hooks on saved tensors hand back others (copies from host memory, for instance), in
        # any layout, and the rules as they were: checked as the call's own were.
        if logits.stride() != (desc.ld_logits, 1) or \
                any(a is not b for a, b in zip(of_rules, rules.tensors)):
            rules = LogitRules(**{k: t.contiguous() for k, t in zip(rules.names, of_rules)})
            if logits.stride() != (desc.ld_logits, 1):
                wide = logits.new_empty((logits.shape[0], desc.ld_logits))
                logits = wide[:, :logits.shape[1]].copy_(logits)
            _check_inputs(logits, targets, active_mask, lse=lse)
            _check_rules(rules, logits, desc.real_vocab)
        d = _run_processed_backward(desc, logits, targets, rules, active_mask, lse, vec(g_logp),
                                    vec(g_lse), logits.dtype)
        return d, None, None, None, None, None, None


def processed_selected_token_logprob(logits: torch.Tensor, targets: torch.Tensor,
                                     rules: LogitRules, active_mask=None, *, real_vocab: int,
                                     padded_vocab: int | None = None, ignore_index: int = -100):
    """processed_forward as a differentiable torch function: returns (logp, lse), fp32 [N].

    The log-probability under the distribution that a sampler with these rules draws from,
    and its gradient to the raw logits (bf16 [N, ld] with unit column stride; the gradient has
    their shape and dtype).  The rules are constants.  Where a training step is captured into a
    HIP graph, no eager autograd graph of the same leaves may be alive: torch ends the process."""
    v_pad = _check_vocab(logits, real_vocab, padded_vocab)
    _check_inputs(logits, targets, active_mask)
    _check_rules(rules, logits, real_vocab)
    for t in rules.tensors:
        if t.requires_grad:
            raise ValueError("the rules are constants: none of their tensors may require a "
                             "gradient")
    return _ProcessedSelectedTokenLogprob.apply(logits, targets, rules, active_mask, real_vocab,
                                                v_pad, ignore_index)


# -- dense products with their epilogue -----------------------------------------------
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "softcap": 5}


_SAVED = {torch.float32: RLK_DTYPE_F32, torch.float16: RLK_DTYPE_F16}


def _check_activation(activation, cap):
    code = ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, "
                         f"got {activation!r}")
    if (cap is not None) != (activation == "softcap"):
        raise ValueError("cap goes with the activation softcap, and with no other")
    if cap is not None and not 1e-30 <= cap <= 1e30:
        raise ValueError(f"cap must be finite and in [1e-30, 1e30], got {cap!r}")
    return code, 0.0 if cap is None else float(cap)


def _check_linear(x, weight, out_dim, bias, **others):
    """x bf16 [M, K] and weight bf16 [>= out_dim, K], contiguous; bias bf16 or fp32, out_dim or
    more; others: bf16 [M, out_dim] with unit column stride.  Nones apart; all on x's GPU."""
    for name, t in (("x", x), ("weight", weight)):
        _check_logits(t, name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if weight.shape[1] != x.shape[1]:
        raise ValueError(f"weight has {weight.shape[1]} columns, x {x.shape[1]}")
    if weight.shape[0] < out_dim:
        raise ValueError(f"weight has {weight.shape[0]} rows, fewer than {out_dim}")
    if bias is not None:
        if not isinstance(bias, torch.Tensor):
            raise TypeError("bias must be a torch.Tensor")
        if bias.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"bias must be torch.bfloat16 or torch.float32, got {bias.dtype}")
        if bias.dim() != 1 or bias.shape[0] < out_dim or not bias.is_contiguous():
            raise ValueError(f"bias must be 1-D and contiguous with {out_dim} elements, got "
                             f"shape {tuple(bias.shape)}")
    for name, t in others.items():
        if t is not None:
            _check_logits(t, name)
            if tuple(t.shape) != (x.shape[0], out_dim):
                raise ValueError(f"{name} must have shape {(x.shape[0], out_dim)}, got "
                                 f"{tuple(t.shape)}")
    _check_device(x, weight=weight, bias=bias, **others)


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _bias_code(dtype):
    return RLK_DTYPE_BF16 if dtype == torch.bfloat16 else RLK_DTYPE_F32


def _run_linear(x, weight, bias, residual, act, cap, out_dim, padded, save, stream=None):
    m, k = x.shape
    ld, ld_saved = (padded + 7) // 8 * 8, (out_dim + 7) // 8 * 8
    with _call_on(x, stream):
        y = torch.empty((m, ld), dtype=torch.bfloat16, device=x.device)
        if ld != padded:
            # (not a view: torch refuses to change one in place that a function returns)
            y.as_strided_((m, padded), (ld, 1))
        # (a bias in fp32 has a gradient in fp32, as exact as what is kept of z)
        exact = bias is not None and bias.dtype == torch.float32
        saved = torch.empty((m, ld_saved), dtype=torch.float32 if exact else torch.float16,
                            device=x.device) if save else None
        desc = rlk_linear_desc(m, k, out_dim, padded, ld,
                               0 if residual is None else _row_stride(residual), ld_saved, act,
                               0 if bias is None else _bias_code(bias.dtype),
                               RLK_DTYPE_F32 if exact else RLK_DTYPE_F16, cap)
        rlk_linear_fwd(desc, x, weight, bias, residual, y, saved, stream)
    _handed_over(x, stream, y, saved)
    return y, saved


def linear_forward(x: torch.Tensor, weight: torch.Tensor, bias=None, residual=None, *,
                   activation: str = "none", cap: float | None = None, save: bool = False,
                   stream=None):
    """(out, saved): out = residual + act(x . weight^T + bias) in bf16 [M, N], rounded once.

    x: bf16 [M, K], weight: bf16 [N, K], both contiguous, K a multiple of 64; bias: bf16 or fp32
    [N]; residual: bf16 [M, N] with unit column stride.  activation: none, relu, gelu, gelu_tanh,
    silu or softcap (cap tanh(z / cap)).  out's rows are padded to a multiple of 8 columns.  With
    `save`, saved is what linear_backward needs (z in fp16, or in fp32 with a bias in fp32; None
    for no activation).  fp16 moves the activation's slope by 2^-11.6 at most, which shows beside
    the rounding of dz to bf16 only where the slope is below 0.05.  No gradient: head_linear has
    them."""
    act, cap = _check_activation(activation, cap)
    _check_logits(weight, "weight")
    n = weight.shape[0]
    _check_linear(x, weight, n, bias, residual=residual)
    return _run_linear(x, weight, bias, residual, act, cap, n, n, save and act != 0, stream)


def linear_backward(x: torch.Tensor, weight: torch.Tensor, grad_out: torch.Tensor, saved=None, *,
                    activation: str = "none", cap: float | None = None, want_x: bool = True,
                    want_weight: bool = True, want_bias: bool = False,
                    bias_dtype=torch.float32, workspace: torch.Tensor | None = None,
                    stream=None):
    """(dx, dweight, dbias) of linear_forward, in bf16 (dbias in bias_dtype), from its `saved` and
    grad_out, bf16 [M, N] with unit column stride (which is the residual's gradient).  What is not
    wanted is not computed and comes back as None."""
    act, cap = _check_activation(activation, cap)
    if bias_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("bias_dtype must be torch.float32 or torch.bfloat16")
    if not (want_x or want_weight or want_bias):
        raise ValueError("at least one of want_x, want_weight and want_bias must be true")
    _check_logits(weight, "weight")
    n = weight.shape[0]
    if grad_out is None:
        raise TypeError("grad_out must be a torch.Tensor")
    _check_linear(x, weight, n, None, grad_out=grad_out)
    if act != 0:
        if not isinstance(saved, torch.Tensor) or saved.dtype not in _SAVED:
            raise TypeError(f"{activation}: the gradient needs what linear_forward saved")
        if tuple(saved.shape) != (x.shape[0], (n + 7) // 8 * 8) or not saved.is_contiguous():
            raise ValueError("saved is not what linear_forward saved for this call")
        _check_device(x, saved=saved)
    return _run_linear_backward(x, weight, grad_out, saved, act, cap, want_x, want_weight,
                                bias_dtype if want_bias else None, workspace, stream)


def _run_linear_backward(x, weight, grad_out, saved, act, cap, want_x, want_weight, bias_dtype,
                         workspace=None, stream=None):
    m, k = x.shape
    n = weight.shape[0]
    desc = rlk_linear_desc(m, k, n, n, n, n, (n + 7) // 8 * 8, act,
                           0 if bias_dtype is None else _bias_code(bias_dtype),
                           RLK_DTYPE_F16 if saved is None else _SAVED[saved.dtype], cap)
    with _call_on(x, stream):
        dx = torch.empty_like(x) if want_x else None
        dw = torch.empty_like(weight) if want_weight else None
        db = None if bias_dtype is None else torch.empty(n, dtype=bias_dtype, device=x.device)
        if workspace is None:
            nbytes = rlk_linear_bwd_workspace_bytes(desc)
            if nbytes == 0:
                raise ValueError(f"invalid rlk_linear_desc: {rlk_last_error_detail()}")
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        else:
            _check_workspace(workspace, x)
        rlk_linear_bwd(desc, x, weight, saved, grad_out, _row_stride(grad_out), dx, dw, db,
                       workspace, stream)
    _handed_over(x, stream, dx, dw, db)
    return dx, dw, db


def _forward_mode():
    """Whether tensors may have tangents.  The level is not part of torch's documented interface;
    where it is gone, they may."""
    return getattr(torch.autograd.forward_ad, "_current_level", 0) >= 0


class _HeadLinear(torch.autograd.Function):
    """residual + act(x . weight^T + bias), differentiable in all four; the forward and the
    backward are rlk_linear_fwd and rlk_linear_bwd."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, act, cap):
        n = weight.shape[0]
        save = act != 0 and any(ctx.needs_input_grad[:3])
        y, saved = _run_linear(x, weight, bias, residual, act, cap, n, n, save)
        ctx.save_for_backward(x, weight, saved)
        ctx.cfg = act, cap, None if bias is None else bias.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        # what was saved has been checked; the gradient has the output's shape, dtype and device
        act, cap, bias_dtype = ctx.cfg
        want_x, want_weight, want_bias, want_residual = ctx.needs_input_grad[:4]
        dx = dw = db = None
        if want_x or want_weight or want_bias:
            # (hooks on saved tensors may hand back another layout)
            x, weight, saved = (None if t is None else t.contiguous() for t in ctx.saved_tensors)
            if grad.stride(1) != 1 or grad.stride(0) < grad.shape[1]:
                grad = grad.contiguous()
            dx, dw, db = _run_linear_backward(x, weight, grad, saved, act, cap, want_x,
                                              want_weight, bias_dtype if want_bias else None)
        return dx, dw, db, grad if want_residual else None, None, None


def head_linear(x: torch.Tensor, weight: torch.Tensor, bias=None, residual=None, *,
                activation: str = "none", cap: float | None = None):
    """linear_forward as a differentiable torch function: returns residual + act(x . weight^T +
    bias), bf16 [M, N], with gradients for the inputs that ask for one (dx, dweight in bf16,
    the bias' in its dtype, the residual's is the upstream one).

    This is a prediction head's dense or residual block, in front of the LM-head.  The backward
    keeps z in 16 bits (32 with a bias in fp32, which may be zeros; see linear_forward) and rounds
    dz to bf16 once.  Where a training step
    is captured into a HIP graph, no eager autograd graph of the same leaves may be alive: torch
    ends the process."""
    act, cap = _check_activation(activation, cap)
    _check_logits(weight, "weight")
    n = weight.shape[0]
    _check_linear(x, weight, n, bias, residual=residual)
    if bias is not None and bias.shape[0] != n:
        raise ValueError(f"bias must have {n} elements, got {bias.shape[0]}")
    # (forward mode is torch's to refuse: a tensor with a tangent need not require a gradient)
    if not _forward_mode() and (not torch.is_grad_enabled() or not (
            x.requires_grad or weight.requires_grad or (bias is not None and bias.requires_grad)
            or (residual is not None and residual.requires_grad))):
        return _run_linear(x, weight, bias, residual, act, cap, n, n, False)[0]
    return _HeadLinear.apply(x, weight, bias, residual, act, cap)


def lmhead_logits(hidden: torch.Tensor, weight: torch.Tensor, bias=None, *, real_vocab: int,
                  padded_vocab: int | None = None, cap: float | None = None, stream=None):
    """bf16 logits [N, V_pad] of an LM-head, z = hidden . weight^T + bias or, with a cap,
    cap tanh(z / cap), rounded once, as forward() and its kin take them (their rows are padded to
    a multiple of 8 columns); columns [real_vocab, V_pad) are -inf.

    hidden: bf16 [N, K] contiguous; weight: bf16 [>= real_vocab, K] contiguous; bias: bf16 or fp32
    [>= real_vocab].  No gradient: fused_lmhead and head_linear have theirs."""
    act, cap = _check_activation("none" if cap is None else "softcap", cap)
    _check_linear(hidden, weight, real_vocab, bias)
    v_pad = padded_vocab or weight.shape[0]
    if not 1 <= real_vocab <= v_pad:
        raise ValueError(f"real_vocab={real_vocab} outside [1, padded_vocab={v_pad}]")
    return _run_linear(hidden, weight, bias, None, act, cap, real_vocab, v_pad, False, stream)[0]
