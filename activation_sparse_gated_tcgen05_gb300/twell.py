"""Thin ctypes binding of libtwell.so (the C ABI in include/twell.h).

Argument marshalling only: every step of the FFN runs in the library's CUDA
kernels.  Functions carry the C names and take torch tensors that already
live on the GPU; they pass raw device pointers and the current CUDA stream.
A non-zero status raises TwellError.  There is no fallback: if the library
is missing or a call fails, the call raises.

Helpers ``alloc_tiles`` / ``alloc_hybrid`` allocate the packed-format
buffers with torch (device memory is the caller's in the C ABI), and
``alloc_adamw_state`` an optimizer's moments.  ``TwellLogits``,
``TwellPolicy``, ``TwellPreference`` and ``TwellParams`` check and describe
their tensors once; a call then passes the description on.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

from . import _build

_lib = None

STATUS = {
    0: "TWELL_OK", 1: "TWELL_ERR_INVALID_ARG", 2: "TWELL_ERR_UNSUPPORTED",
    3: "TWELL_ERR_ALIGNMENT", 4: "TWELL_ERR_CAPACITY", 5: "TWELL_ERR_CUDA",
    6: "TWELL_ERR_DEVICE_TIMEOUT", 7: "TWELL_ERR_WORKSPACE", 8: "TWELL_ERR_INDEX",
}
EXPORTS = (
    "twell_pack", "twell_pack_dense", "hybrid_route", "twell_workspace_bytes",
    "twell_workspace_bytes_capped",
    "twell_tiles_workspace_bytes", "twell_set_split_gathers", "twell_set_pair_gemm",
    "twell_ffn_fwd",
    "twell_ffn_bwd", "twell_dense_workspace_bytes", "twell_dense_ffn_fwd", "twell_dense_ffn_bwd",
    "twell_dense_ffn_fwd_act", "twell_dense_ffn_bwd_act",
    "twell_gemm_bf16", "twell_get_device_status", "twell_status_string", "twell_num_sms",
    "twell_launch_count", "twell_profile_begin", "twell_profile_end", "twell_profile_entry",
    "twell_ffn_fwd_noalloc", "twell_selftest_wait_timeout",
    "twell_token_logp", "twell_policy_loss", "twell_preference_loss", "twell_logp_bwd",
    "twell_grad_norm_workspace_bytes", "twell_grad_norm", "twell_adamw_step",
)


class TwellError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__("%s failed: %s (%d)" % (fn, STATUS.get(status, "?"), status))
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("tile_cap", ctypes.c_int32)]


class Tiles(ctypes.Structure):
    _fields_ = [("val", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("cnt", ctypes.c_void_p),
                ("row_nnz", ctypes.c_void_p)]


class Hybrid(ctypes.Structure):
    _fields_ = [("ell_val", ctypes.c_void_p), ("ell_col", ctypes.c_void_p),
                ("ell_nnz", ctypes.c_void_p), ("ell_width", ctypes.c_int32),
                ("dense_rows", ctypes.c_void_p), ("n_dense", ctypes.c_void_p),
                ("dense_cap", ctypes.c_int32)]


class Logits(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("target", ctypes.c_void_p), ("stride", ctypes.c_int64),
                ("rows", ctypes.c_int32), ("vocab", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("target_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class Policy(ctypes.Structure):
    _fields_ = [("advantage", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("old_logp", ctypes.c_void_p), ("ref_logp", ctypes.c_void_p),
                ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
                ("kl_coeff", ctypes.c_float)]


class Preference(ctypes.Structure):
    _fields_ = [("seq_start", ctypes.c_void_p), ("ref_logp", ctypes.c_void_p),
                ("pairs", ctypes.c_int32), ("beta", ctypes.c_float),
                ("label_smoothing", ctypes.c_float)]


class Param(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64)]


class AdamW(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint64),
                ("grad_scale", ctypes.c_void_p), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("skipped", ctypes.c_void_p)]


def library_path() -> str:
    """libtwell.so, or the checked (bounds-checking debug) build
    libtwell_checked.so when the environment sets TWELL_CHECKED=1."""
    return _build.CHECKED_LIB if os.environ.get("TWELL_CHECKED") == "1" else _build.LIB


def load():
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError("libtwell.so not found at %s: run __graft_entry__.build() "
                           "(or python -m activation_sparse_gated_tcgen05_gb300._build)" % path)
    lib = ctypes.CDLL(path)
    P, I32, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    SP, TP, HP = ctypes.POINTER(Shape), ctypes.POINTER(Tiles), ctypes.POINTER(Hybrid)
    LP, I64 = ctypes.POINTER(Logits), ctypes.c_int64
    sig = {
        "twell_pack": (I32, [P, P, SP, TP, P]),
        "twell_pack_dense": (I32, [P, I32, SP, TP, P]),
        "hybrid_route": (I32, [TP, SP, HP, P]),
        "twell_workspace_bytes": (SZ, [SP, I32, I32]),
        "twell_workspace_bytes_capped": (SZ, [SP, I32, I32, I32]),
        "twell_tiles_workspace_bytes": (SZ, [SP]),
        "twell_set_split_gathers": (I32, [I32]),
        "twell_set_pair_gemm": (I32, [I32]),
        "twell_ffn_fwd": (I32, [P, P, P, P, SP, TP, HP, P, P, SZ, P]),
        "twell_ffn_bwd": (I32, [P, P, P, P, P, SP, HP, F, P, P, P, P, P, SZ, P]),
        "twell_ffn_fwd_noalloc": (I32, [P, P, P, P, SP, HP, P, P]),
        "twell_selftest_wait_timeout": (I32, [I32, P]),
        "twell_dense_workspace_bytes": (SZ, [SP, I32]),
        "twell_dense_ffn_fwd": (I32, [P, P, P, P, SP, P, I32, P, SZ, P]),
        "twell_dense_ffn_bwd": (I32, [P, P, P, P, P, SP, F, P, P, P, P, P, SZ, P]),
        "twell_dense_ffn_fwd_act": (I32, [P, P, P, P, SP, I32, P, I32, P, SZ, P]),
        "twell_dense_ffn_bwd_act": (I32, [P, P, P, P, P, SP, I32, F, P, P, P, P, P, SZ, P]),
        "twell_gemm_bf16": (I32, [P, P, P, I32, I32, I32, I32, I32, I32, I32, P]),
        "twell_get_device_status": (I32, [P, ctypes.POINTER(I32)]),
        "twell_status_string": (ctypes.c_char_p, [I32]),
        "twell_num_sms": (I32, []),
        "twell_launch_count": (ctypes.c_uint64, []),
        "twell_profile_begin": (I32, [ctypes.c_char_p]),
        "twell_profile_end": (I32, []),
        "twell_token_logp": (I32, [LP, P, P, P]),
        "twell_policy_loss": (I32, [LP, ctypes.POINTER(Policy), P, P, P, P, P, P, I64, P]),
        "twell_preference_loss": (I32, [LP, ctypes.POINTER(Preference), P, P, P, P, P, P, P]),
        "twell_logp_bwd": (I32, [LP, P, P, P, P, I64, P]),
        "twell_grad_norm_workspace_bytes": (SZ, []),
        "twell_grad_norm": (I32, [ctypes.POINTER(Param), I32, I32, F, P, P, SZ, P]),
        "twell_adamw_step": (I32, [ctypes.POINTER(Param), I32, ctypes.POINTER(AdamW), P]),
        "twell_profile_entry": (I32, [I32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(I32),
                                      ctypes.POINTER(ctypes.c_double)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        # the raw handle: a Stream object would cost more than most of these calls; PyTorch does not
        # promise the call that gives it, so the object is there for one without
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return torch.cuda.current_stream().cuda_stream if raw is None else raw(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(name: str, status: int):
    if status != 0:
        raise TwellError(name, status)


@dataclass
class TwellTiles:
    val: torch.Tensor      # bf16 [M][T][C]
    idx: torch.Tensor      # uint8 [M][T][C]
    cnt: torch.Tensor      # uint8 [M][T]
    row_nnz: torch.Tensor  # int32 [M]

    def c(self) -> Tiles:
        return Tiles(_ptr(self.val), _ptr(self.idx), _ptr(self.cnt), _ptr(self.row_nnz))


@dataclass
class TwellHybrid:
    ell_val: torch.Tensor     # bf16 [M][W]
    ell_col: torch.Tensor     # uint16 stored as int16 [M][W]
    ell_nnz: torch.Tensor     # int32 [M]
    ell_width: int
    dense_rows: torch.Tensor  # int32 [M]
    n_dense: torch.Tensor     # int32 [1]
    dense_cap: int            # routed rows the workspace holds (host value)

    def c(self) -> Hybrid:
        return Hybrid(_ptr(self.ell_val), _ptr(self.ell_col), _ptr(self.ell_nnz), int(self.ell_width),
                      _ptr(self.dense_rows), _ptr(self.n_dense), int(self.dense_cap))


def make_shape(M: int, d_model: int, d_ff: int, tile_n: int = 128, tile_cap: int = 32) -> Shape:
    return Shape(int(M), int(d_model), int(d_ff), int(tile_n), int(tile_cap))


def _pad16(n: int) -> int:
    return max(16, (n + 15) // 16 * 16)


def alloc_tiles(shape: Shape, device="cuda") -> TwellTiles:
    M, T, C = shape.M, shape.d_ff // shape.tile_n, shape.tile_cap
    # flat buffers padded to 16 bytes so every pointer handed over stays aligned
    val = torch.empty(_pad16(M * T * C * 2) // 2, dtype=torch.bfloat16, device=device)
    idx = torch.empty(_pad16(M * T * C), dtype=torch.uint8, device=device)
    cnt = torch.empty(_pad16(M * T), dtype=torch.uint8, device=device)
    nnz = torch.empty(_pad16(M * 4) // 4, dtype=torch.int32, device=device)
    return TwellTiles(val, idx, cnt, nnz)


def tiles_view(t: TwellTiles, shape: Shape):
    """(val, idx, cnt, row_nnz) reshaped to [M][T][C], [M][T][C], [M][T], [M]."""
    M, T, C = shape.M, shape.d_ff // shape.tile_n, shape.tile_cap
    return (t.val[: M * T * C].view(M, T, C), t.idx[: M * T * C].view(M, T, C),
            t.cnt[: M * T].view(M, T), t.row_nnz[:M])


def alloc_hybrid(shape: Shape, ell_width: int, device="cuda",
                 dense_cap: Optional[int] = None) -> TwellHybrid:
    """Routing buffers; dense_cap (default M, every row) is the routed-row
    capacity the workspace will be sized for."""
    M, W = shape.M, int(ell_width)
    ev = torch.empty(_pad16(M * W * 2) // 2, dtype=torch.bfloat16, device=device)
    ec = torch.empty(_pad16(M * W * 2) // 2, dtype=torch.int16, device=device)
    en = torch.empty(_pad16(M * 4) // 4, dtype=torch.int32, device=device)
    dr = torch.empty(_pad16(M * 4) // 4, dtype=torch.int32, device=device)
    nd = torch.zeros(4, dtype=torch.int32, device=device)
    return TwellHybrid(ev, ec, en, W, dr, nd, M if dense_cap is None else int(dense_cap))


def hybrid_view(h: TwellHybrid, shape: Shape):
    M, W = shape.M, h.ell_width
    return (h.ell_val[: M * W].view(M, W), h.ell_col[: M * W].view(M, W), h.ell_nnz[:M],
            h.dense_rows[:M], h.n_dense[:1])


# ------------------------------------------------------------------ entry points
def twell_pack(x, wgT, shape: Shape, out: TwellTiles, stream=None):
    t = out.c()
    _check("twell_pack", load().twell_pack(_ptr(x), _ptr(wgT), ctypes.byref(shape),
                                           ctypes.byref(t), _stream(stream)))


def twell_pack_dense(a, shape: Shape, out: TwellTiles, stream=None):
    if a.dtype == torch.float32:
        dt = 1
    elif a.dtype == torch.bfloat16:
        dt = 0
    else:
        raise ValueError("a must be float32 or bfloat16")
    t = out.c()
    _check("twell_pack_dense", load().twell_pack_dense(_ptr(a), dt, ctypes.byref(shape),
                                                       ctypes.byref(t), _stream(stream)))


def hybrid_route(tiles: TwellTiles, shape: Shape, out: TwellHybrid, stream=None):
    t, h = tiles.c(), out.c()
    _check("hybrid_route", load().hybrid_route(ctypes.byref(t), ctypes.byref(shape),
                                               ctypes.byref(h), _stream(stream)))


def twell_workspace_bytes(shape: Shape, ell_width: int, training: bool,
                          dense_cap: Optional[int] = None) -> int:
    """Workspace bytes of the sparse forward (and backward, training); room for
    dense_cap routed rows (default: every row)."""
    if dense_cap is None:
        return int(load().twell_workspace_bytes(ctypes.byref(shape), int(ell_width),
                                                int(training)))
    return int(load().twell_workspace_bytes_capped(ctypes.byref(shape), int(ell_width),
                                                   int(dense_cap), int(training)))


def twell_tiles_workspace_bytes(shape: Shape) -> int:
    return int(load().twell_tiles_workspace_bytes(ctypes.byref(shape)))


def twell_set_split_gathers(enable: bool) -> bool:
    """Split (True, the default) or fused (False) gathers for rows wider than
    1024; returns the previous setting."""
    return bool(load().twell_set_split_gathers(int(bool(enable))))


def twell_set_pair_gemm(enable: bool) -> bool:
    """CTA-pair 256 x 256 GEMM tiles (True, the default) or single-CTA
    128 x 256 tiles (False); returns the previous setting."""
    return bool(load().twell_set_pair_gemm(int(bool(enable))))


def twell_ffn_fwd(x, wgT, wuT, wd, shape: Shape, y, tiles: Optional[TwellTiles] = None,
                  route: Optional[TwellHybrid] = None, ws=None, stream=None):
    t = tiles.c() if tiles is not None else None
    h = route.c() if route is not None else None
    _check("twell_ffn_fwd", load().twell_ffn_fwd(
        _ptr(x), _ptr(wgT), _ptr(wuT), _ptr(wd), ctypes.byref(shape),
        ctypes.byref(t) if t is not None else None, ctypes.byref(h) if h is not None else None,
        _ptr(y), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def twell_ffn_fwd_noalloc(x, wgT, wuT, wd, shape: Shape, y, route: TwellHybrid, stream=None):
    """Hybrid forward whose scratch lives in the library's static device array
    (no workspace argument, nothing allocated); see include/twell.h."""
    h = route.c()
    _check("twell_ffn_fwd_noalloc", load().twell_ffn_fwd_noalloc(
        _ptr(x), _ptr(wgT), _ptr(wuT), _ptr(wd), ctypes.byref(shape), ctypes.byref(h), _ptr(y),
        _stream(stream)))


def twell_ffn_bwd(x, wgT, wuT, wd, dy, shape: Shape, route: TwellHybrid, l1_coeff: float, dx,
                  dwgT, dwuT, dwd, ws, stream=None):
    h = route.c()
    _check("twell_ffn_bwd", load().twell_ffn_bwd(
        _ptr(x), _ptr(wgT), _ptr(wuT), _ptr(wd), _ptr(dy), ctypes.byref(shape), ctypes.byref(h),
        float(l1_coeff), _ptr(dx), _ptr(dwgT), _ptr(dwuT), _ptr(dwd), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def twell_dense_workspace_bytes(shape: Shape, training: bool) -> int:
    return int(load().twell_dense_workspace_bytes(ctypes.byref(shape), int(training)))


def twell_dense_ffn_fwd(x, wgT, wuT, wd, shape: Shape, y, training: bool, ws, stream=None):
    _check("twell_dense_ffn_fwd", load().twell_dense_ffn_fwd(
        _ptr(x), _ptr(wgT), _ptr(wuT), _ptr(wd), ctypes.byref(shape), _ptr(y), int(training),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def twell_dense_ffn_bwd(x, wgT, wuT, wd, dy, shape: Shape, l1_coeff: float, dx, dwgT, dwuT, dwd,
                        ws, stream=None):
    _check("twell_dense_ffn_bwd", load().twell_dense_ffn_bwd(
        _ptr(x), _ptr(wgT), _ptr(wuT), _ptr(wd), _ptr(dy), ctypes.byref(shape), float(l1_coeff),
        _ptr(dx), _ptr(dwgT), _ptr(dwuT), _ptr(dwd), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


ACT_RELU, ACT_SILU = 0, 1


def twell_dense_ffn_fwd_act(x, wgT, wuT, wd, shape: Shape, activation: int, y, training: bool, ws,
                            stream=None):
    _check("twell_dense_ffn_fwd_act", load().twell_dense_ffn_fwd_act(
        _ptr(x), _ptr(wgT), _ptr(wuT), _ptr(wd), ctypes.byref(shape), int(activation), _ptr(y),
        int(training), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def twell_dense_ffn_bwd_act(x, wgT, wuT, wd, dy, shape: Shape, activation: int, l1_coeff: float,
                            dx, dwgT, dwuT, dwd, ws, stream=None):
    _check("twell_dense_ffn_bwd_act", load().twell_dense_ffn_bwd_act(
        _ptr(x), _ptr(wgT), _ptr(wuT), _ptr(wd), _ptr(dy), ctypes.byref(shape), int(activation),
        float(l1_coeff), _ptr(dx), _ptr(dwgT), _ptr(dwuT), _ptr(dwd), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def twell_gemm_bf16(A, B, C, M: int, N: int, K: int, a_mn_major: bool, b_mn_major: bool,
                    accumulate: bool = False, stream=None):
    c_dtype = 1 if C.dtype == torch.float32 else 0
    _check("twell_gemm_bf16", load().twell_gemm_bf16(
        _ptr(A), _ptr(B), _ptr(C), int(M), int(N), int(K), int(a_mn_major), int(b_mn_major),
        c_dtype, int(accumulate), _stream(stream)))


# ------------------------------------------------------- the step around the FFN
_DTYPE = {torch.bfloat16: 0, torch.float32: 1}
_INDEX = {torch.int32: 0, torch.int64: 1}
BLOCK = 256  # elements that share one scale of an 8-bit state


def _vec(t: Optional[torch.Tensor], n: int, name: str, dtype=torch.float32):
    """Pointer of a contiguous `dtype` tensor of n elements on the GPU (None stays None)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    if t.numel() != n:
        raise ValueError("%s must have %d elements, not %d" % (name, n, t.numel()))
    return _ptr(t)


def _row_view(t: torch.Tensor, name: str):
    """(pointer, stride) of a 2-D tensor whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s must be [rows][vocab] with contiguous rows" % name)
    stride = t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))
    if stride < t.shape[1]:
        raise ValueError("the rows of %s must not overlap" % name)
    return t.data_ptr(), stride


class TwellLogits:
    """Logits [rows][vocab] (bf16 or fp32, rows contiguous, any row stride) and the token each
    row is scored for (int32 or int64 [rows], negative = ignored); scale = 1 / temperature."""

    def __init__(self, data: torch.Tensor, target: torch.Tensor, scale: float = 1.0):
        if data.dtype not in _DTYPE:
            raise ValueError("logits must be float32 or bfloat16")
        if target.dtype not in _INDEX:
            raise ValueError("target must be int32 or int64")
        ptr, stride = _row_view(data, "logits")
        self.data, self.target = data, target
        self.rows, self.vocab = data.shape
        self.c = Logits(ptr, _vec(target, self.rows, "target", target.dtype), stride, self.rows,
                        self.vocab, _DTYPE[data.dtype], _INDEX[target.dtype], float(scale))
        self.ref = ctypes.byref(self.c)

    def grad_ptr(self, dlogits: Optional[torch.Tensor]):
        """(pointer, stride) of a gradient of these logits."""
        if dlogits is None:
            return None, 0
        if dlogits.dtype != self.data.dtype or dlogits.shape != self.data.shape:
            raise ValueError("dlogits must have the type and shape of the logits")
        return _row_view(dlogits, "dlogits")


class TwellPolicy:
    """Arguments of the clipped policy loss, fp32 [rows] each; weight None = 1, old_logp None =
    on-policy, ref_logp is needed with kl_coeff > 0."""

    def __init__(self, advantage, weight=None, old_logp=None, ref_logp=None, clip_low: float = 0.2,
                 clip_high: float = 0.2, kl_coeff: float = 0.0):
        n = advantage.numel()
        self.rows, self.tensors = n, (advantage, weight, old_logp, ref_logp)
        names = ("advantage", "weight", "old_logp", "ref_logp")
        self.c = Policy(*(_vec(t, n, k) for t, k in zip(self.tensors, names)), float(clip_low),
                        float(clip_high), float(kl_coeff))
        self.ref = ctypes.byref(self.c)


class TwellPreference:
    """Arguments of the preference loss: seq_start int64 [2 pairs + 1] on the GPU (sequence 2 p is
    the chosen answer of pair p, 2 p + 1 the rejected one), ref_logp fp32 [rows] or None."""

    def __init__(self, seq_start, ref_logp=None, beta: float = 0.1, label_smoothing: float = 0.0):
        n = seq_start.numel()
        if n % 2 != 1:
            raise ValueError("seq_start must have 2 * pairs + 1 elements")
        self.pairs = n // 2
        self.rows = None if ref_logp is None else ref_logp.numel()
        self.tensors = (seq_start, ref_logp)
        self.c = Preference(_vec(seq_start, n, "seq_start", torch.int64),
                            None if ref_logp is None else _vec(ref_logp, self.rows, "ref_logp"),
                            self.pairs, float(beta), float(label_smoothing))
        self.ref = ctypes.byref(self.c)


def twell_token_logp(logits: TwellLogits, logp, lse=None, stream=None):
    n = logits.rows
    _check("twell_token_logp", load().twell_token_logp(
        logits.ref, _vec(logp, n, "logp"), _vec(lse, n, "lse"), _stream(stream)))


def twell_policy_loss(logits: TwellLogits, policy: TwellPolicy, loss, tok_loss, logp, lse, coef,
                      dlogits=None, stream=None):
    n = logits.rows
    if policy.rows != n:
        raise ValueError("advantage must have %d elements, not %d" % (n, policy.rows))
    d, stride = logits.grad_ptr(dlogits)
    _check("twell_policy_loss", load().twell_policy_loss(
        logits.ref, policy.ref, _vec(loss, 1, "loss"), _vec(tok_loss, n, "tok_loss"),
        _vec(logp, n, "logp"), _vec(lse, n, "lse"), _vec(coef, n, "coef"), d, stride,
        _stream(stream)))


def twell_preference_loss(logits: TwellLogits, preference: TwellPreference, loss, pair_loss,
                          seq_gain, logp, lse, coef, stream=None):
    n, pairs = logits.rows, preference.pairs
    if preference.rows is not None and preference.rows != n:
        raise ValueError("ref_logp must have %d elements, not %d" % (n, preference.rows))
    _check("twell_preference_loss", load().twell_preference_loss(
        logits.ref, preference.ref, _vec(loss, 1, "loss"), _vec(pair_loss, pairs, "pair_loss"),
        _vec(seq_gain, 2 * pairs, "seq_gain"), _vec(logp, n, "logp"), _vec(lse, n, "lse"),
        _vec(coef, n, "coef"), _stream(stream)))


def twell_logp_bwd(logits: TwellLogits, lse, coef, dlogits, dloss=None, stream=None):
    n = logits.rows
    d, stride = logits.grad_ptr(dlogits)
    _check("twell_logp_bwd", load().twell_logp_bwd(
        logits.ref, _vec(lse, n, "lse"), _vec(coef, n, "coef"), _vec(dloss, 1, "dloss"), d, stride,
        _stream(stream)))


def alloc_adamw_state(param: torch.Tensor, state_bits: int = 32) -> dict:
    """Zero moments of one parameter tensor: m, v (and with 8 bits m_scale, v_scale)."""
    n, dev = param.numel(), param.device
    if state_bits == 32:
        return {k: torch.zeros(n, dtype=torch.float32, device=dev) for k in ("m", "v")}
    if state_bits != 8:
        raise ValueError("state_bits must be 8 or 32")
    st = {k: torch.zeros(n, dtype=torch.float8_e4m3fn, device=dev) for k in ("m", "v")}
    for k in ("m_scale", "v_scale"):
        st[k] = torch.zeros((n + BLOCK - 1) // BLOCK, dtype=torch.float32, device=dev)
    return st


class TwellParams:
    """The tensors of an optimizer step, described once: params (all fp32 or all bf16), grads (all
    fp32 or all bf16), moments m and v (fp32, or float8_e4m3fn with m_scale and v_scale) and, for
    those that have one, the bf16 copies (None entries = none).  Every tensor is contiguous; the
    list keeps them alive.  Give a step's new gradient tensors with set_grads."""

    def __init__(self, params, grads, m, v, copies=None, m_scale=None, v_scale=None):
        n = len(params)
        if grads is None:
            grads = [None] * n
        copies = [None] * n if copies is None else copies
        if (m_scale is None) != (v_scale is None):
            raise ValueError("m_scale and v_scale belong together")
        self.state_bits = 32 if m_scale is None else 8
        scales = [([None] * n if x is None else x) for x in (m_scale, v_scale)]
        lists = (params, copies, grads, m, v, *scales)
        if any(len(x) != n for x in lists):
            raise ValueError("every list must have %d entries" % n)
        self.tensors = [list(x) for x in lists]
        self.count = n
        self.param_dtype = self._dtype("params", params)
        self.grad_dtype = None
        self.c = (Param * max(1, n))()
        state = torch.float32 if self.state_bits == 32 else torch.float8_e4m3fn
        for e, p, c, mm, vv, ms, vs in zip(self.c, params, copies, m, v, *scales):
            e.n = k = p.numel()
            e.param = _vec(p, k, "param", p.dtype)
            e.copy = _vec(c, k, "copy", torch.bfloat16)
            e.m, e.v = _vec(mm, k, "m", state), _vec(vv, k, "v", state)
            blocks = (k + BLOCK - 1) // BLOCK
            e.m_scale, e.v_scale = _vec(ms, blocks, "m_scale"), _vec(vs, blocks, "v_scale")
        self.set_grads(grads)

    @staticmethod
    def _dtype(name, tensors):
        kinds = {t.dtype for t in tensors if t is not None}
        if len(kinds) > 1 or not kinds <= set(_DTYPE):
            raise ValueError("%s must be all float32 or all bfloat16" % name)
        return _DTYPE[kinds.pop()] if kinds else 1

    def set_grads(self, grads):
        """The gradients of the next steps, one for each parameter."""
        if len(grads) != self.count:
            raise ValueError("grads must have %d entries" % self.count)
        dtype = self._dtype("grads", grads)
        for e, g in zip(self.c, grads):
            e.grad = None if g is None else _vec(g, e.n, "grad", g.dtype)
        self.tensors[2], self.grad_dtype = list(grads), dtype

    def drop_grads(self):
        """Lets go of the gradients; set_grads gives the next ones."""
        self.tensors[2], self.grad_dtype = [None] * self.count, None


class TwellGrads:
    """Gradients alone (all fp32 or all bf16, contiguous), for twell_grad_norm."""

    def __init__(self, grads):
        self.count = len(grads)
        self.grad_dtype = TwellParams._dtype("grads", grads)
        self.tensors = list(grads)
        self.c = (Param * max(1, self.count))()
        for e, g in zip(self.c, grads):
            e.n = g.numel()
            e.grad = _vec(g, g.numel(), "grad", g.dtype)


def _has_grads(params):
    if params.grad_dtype is None:
        raise ValueError("the list's gradients were dropped: set_grads gives new ones")


def twell_grad_norm_workspace_bytes() -> int:
    return int(load().twell_grad_norm_workspace_bytes())


def twell_grad_norm(params, max_norm: float, out, ws, stream=None):
    """out (fp32 [2]) = the global norm of the gradients of a TwellParams or TwellGrads, and
    min(1, max_norm / norm)."""
    _has_grads(params)
    _check("twell_grad_norm", load().twell_grad_norm(
        params.c, params.count, params.grad_dtype, float(max_norm), _vec(out, 2, "out"), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def twell_adamw_step(params: TwellParams, step: int, lr: float = 1e-3, beta1: float = 0.9,
                     beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
                     seed: int = 0, grad_scale=None, stream=None, skipped=None):
    """One AdamW step; step counts from 1, grad_scale (fp32 [1] on the GPU) multiplies the
    gradients, seed and step choose the random numbers of 8-bit states, skipped (int32 [1] on the
    GPU) counts the steps that changed nothing, for the bias corrections."""
    _has_grads(params)
    h = AdamW(lr, beta1, beta2, eps, weight_decay, int(step), int(seed) & 0xFFFFFFFFFFFFFFFF,
              _vec(grad_scale, 1, "grad_scale"), params.param_dtype, params.grad_dtype,
              params.state_bits, _vec(skipped, 1, "skipped", torch.int32))
    _check("twell_adamw_step", load().twell_adamw_step(params.c, params.count, ctypes.byref(h),
                                                       _stream(stream)))


def twell_get_device_status(stream=None) -> int:
    out = ctypes.c_int32(0)
    _check("twell_get_device_status", load().twell_get_device_status(_stream(stream),
                                                                     ctypes.byref(out)))
    return int(out.value)


def twell_num_sms() -> int:
    return int(load().twell_num_sms())


def twell_selftest_wait_timeout(limit_us: int, stream=None):
    _check("twell_selftest_wait_timeout",
           load().twell_selftest_wait_timeout(int(limit_us), _stream(stream)))


def twell_launch_count() -> int:
    return int(load().twell_launch_count())


def twell_profile_begin(kernel: Optional[str]):
    _check("twell_profile_begin",
           load().twell_profile_begin(kernel.encode() if kernel else None))


def twell_profile_end() -> dict:
    """Stop profiling; {family: (launches, total_ms)} of the recorded launches."""
    lib = load()
    n = lib.twell_profile_end()
    if n < 0:
        raise TwellError("twell_profile_end", 5)
    out = {}
    for i in range(n):
        name, cnt, ms = ctypes.c_char_p(), ctypes.c_int32(), ctypes.c_double()
        _check("twell_profile_entry", lib.twell_profile_entry(i, ctypes.byref(name),
                                                              ctypes.byref(cnt), ctypes.byref(ms)))
        out[name.value.decode()] = (int(cnt.value), float(ms.value))
    return out
