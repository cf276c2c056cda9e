"""Python binding of libspax.so: argument marshalling only, every step runs in the CUDA library.

The functions carry the names of the C entry points in ``include/spax.h`` and take torch tensors
(device memory and the current CUDA stream come from PyTorch). They raise ``SpaxError`` on a
non-OK status. Importing this module fails loudly when ``libspax.so`` is missing: there is no
CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspax.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"libspax.so not found at {_LIB_PATH}; build it with "
        "`python -m tiered_weight_gemv_b200.build` (nvcc, sm_100a)")
_lib = ctypes.CDLL(_LIB_PATH)

OK = 0
ERR_ARG, ERR_SHAPE, ERR_WORKSPACE, ERR_CUDA, ERR_NONFINITE, ERR_TIMEOUT, ERR_INDEX = 1, 2, 3, 4, 5, 6, 7
FULL_BF16, FULL_INT4_G128 = 0, 1
MASK_THRESHOLD, MASK_TOPK, MASK_GUIDED, MASK_TOPK_SCALED = 0, 1, 2, 3
OP_TIERED_GEMV, OP_DENSE_GEMV, OP_CALIBRATE = 0, 1, 2
MASK_MAX_DIN = 32768
KV_BF16, KV_E4M3 = 0, 1
NORM_RMS, NORM_LAYER = 0, 1


class SpaxError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


class spax_mask_params(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("t_skip", ctypes.c_float), ("t_full", ctypes.c_float),
                ("k_full", ctypes.c_int32), ("k_approx", ctypes.c_int32),
                ("s_skip_bp", ctypes.c_int32), ("s_below_full_bp", ctypes.c_int32),
                ("delta_bp", ctypes.c_int32)]


class spax_packed(ctypes.Structure):
    _fields_ = [("d_out", ctypes.c_int32), ("d_in", ctypes.c_int32), ("full_fmt", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("d_full", ctypes.c_void_p),
                ("d_approx", ctypes.c_void_p)]


class spax_kv_cache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("d_k", ctypes.c_void_p),
                ("d_v", ctypes.c_void_p)]


class spax_rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("d_inv_freq", ctypes.c_void_p)]


class spax_attn_params(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("window", ctypes.c_int32)]


class spax_norm(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("d_weight", ctypes.c_void_p), ("d_bias", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


_P, _I, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_L = ctypes.c_int64
_SIGS = {
    "spax_abi_version": ([], _I),
    "spax_status_string": ([_I], ctypes.c_char_p),
    "spax_pack_bytes": ([_I, _I, _I, _P, _P], _Z),
    "spax_pack_weights": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "spax_calibrate_thresholds": ([_P, _I, _I, _I, _I, _P, _P, _P, _Z, _P], _I),
    "spax_build_mask": ([_P, _I, ctypes.POINTER(spax_mask_params), _P, _P, _P, _P, _P, _P], _I),
    "spax_tiered_gemv": ([ctypes.POINTER(spax_packed), _P, _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "spax_dense_gemv": ([_P, _P, _P, _I, _I, _P, _P, _Z, _P], _I),
    "spax_masked_gemv": ([ctypes.POINTER(spax_packed), _P, ctypes.POINTER(spax_mask_params), _P,
                          _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "spax_masked_gemv_wina": ([ctypes.POINTER(spax_packed), _P, _P,
                               ctypes.POINTER(spax_mask_params), _P, _P, _P, _P, _P, _P, _P, _Z,
                               _P], _I),
    "spax_column_norms": ([_P, _I, _I, _P, _P], _I),
    "spax_masked_gemv_swiglu": ([ctypes.POINTER(spax_packed), _P, ctypes.POINTER(spax_mask_params),
                                 _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "spax_tiered_gemv_fixed_scratch": ([ctypes.POINTER(spax_packed), _P, _P, _P, _P, _P, _P, _P],
                                       _I),
    "spax_fixed_scratch_bytes": ([], _Z),
    "spax_fixed_scratch_reset": ([_P], _I),
    "spax_output_change": ([_P, _P, _I, _P, _P], _I),
    "spax_probe_sensitivity": ([ctypes.POINTER(spax_packed), _P, _I, _I, _P, _P, _P, _P, _Z, _P],
                               _I),
    "spax_test_tiered_gemv_timeout": ([ctypes.POINTER(spax_packed), _P, _P, _P, _P, _P, _P, _P, _Z,
                                      ctypes.c_uint64, _P], _I),
    "spax_workspace_bytes": ([_I, _I, _I], _Z),
    "spax_gemv_plan": ([_I, _I, _I, _I, _P, _P], _I),
    "spax_gemv_plan_sms": ([_I, _I, _I, _I, _I, _P, _P, _P], _I),
    "spax_block_budgets": ([_P, _I, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                            ctypes.c_double, _P], _I),
    "spax_weight_bytes": ([_I, _I, ctypes.c_int64, ctypes.c_int64], ctypes.c_uint64),
    "spax_greedy_allocation": ([_P, _I, ctypes.c_double, ctypes.c_double, ctypes.c_double, _P, _P,
                                _I, _P, _P, _P], _I),
    "spax_kv_append": ([_P, _P, _L, _P, _L, _P, _L, _I, _I, _P, _P, _P, _I, _I, _P, _P, _L, _P,
                        _P], _I),
    "spax_paged_attention": ([_P, _P, _L, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "spax_attention_workspace_bytes": ([_I, _I, _I], _Z),
    "spax_attention_plan_sms": ([_I, _I, _I, _I, _I, _L, _I, _I, _P, _P], _I),
    "spax_residual_norm": ([_P, _P, _I, _I, _P, _P, _L, _F, _F, _P, _P, _P, _P], _I),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_SIGS)


def status_string(status: int) -> str:
    return _lib.spax_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != OK:
        raise SpaxError(fn, status)


def _dev(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _dev_or_pinned(t, name="tensor"):
    """A weight pool: device memory, or page-locked host memory (mapped into the device)."""
    if isinstance(t, torch.Tensor) and not t.is_cuda and t.is_pinned() and t.is_contiguous():
        return ctypes.c_void_p(t.data_ptr())
    return _dev(t, None, name)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# ------------------------------------------------------------------------------ host-only calls

def spax_abi_version() -> int:
    return int(_lib.spax_abi_version())


def spax_pack_bytes(d_out: int, d_in: int, full_fmt: int):
    fb, ab = ctypes.c_size_t(0), ctypes.c_size_t(0)
    tot = _lib.spax_pack_bytes(d_out, d_in, full_fmt, ctypes.byref(fb), ctypes.byref(ab))
    if tot == 0:
        raise SpaxError("spax_pack_bytes", ERR_SHAPE)
    return int(fb.value), int(ab.value)


def spax_workspace_bytes(op: int, d_out: int, d_in: int) -> int:
    return int(_lib.spax_workspace_bytes(op, d_out, d_in))


def spax_gemv_plan(op: int, d_out: int, d_in: int, full_fmt: int = FULL_BF16):
    s, r = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("spax_gemv_plan", _lib.spax_gemv_plan(op, d_out, d_in, full_fmt, ctypes.byref(s),
                                                 ctypes.byref(r)))
    return int(s.value), int(r.value)


def spax_gemv_plan_sms(op: int, d_out: int, d_in: int, full_fmt: int, sm_count: int):
    """Host-only: (splits, row_tile, workspace bytes) of op's plan on a GPU with sm_count SMs."""
    sp, r, w = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_size_t(0)
    _check("spax_gemv_plan_sms", _lib.spax_gemv_plan_sms(op, d_out, d_in, full_fmt, sm_count,
                                                         ctypes.byref(sp), ctypes.byref(r),
                                                         ctypes.byref(w)))
    return int(sp.value), int(r.value), int(w.value)


def spax_block_budgets(sens, s: float, lam: float, lo: float = 0.05, hi: float = 0.95):
    sens = np.ascontiguousarray(sens, dtype=np.float64)
    out = np.zeros_like(sens)
    _check("spax_block_budgets", _lib.spax_block_budgets(
        sens.ctypes.data_as(_P), sens.size, s, lam, lo, hi, out.ctypes.data_as(_P)))
    return out


BLOCK_ERROR_FN = ctypes.CFUNCTYPE(ctypes.c_double, ctypes.POINTER(ctypes.c_double), ctypes.c_int,
                                  ctypes.c_void_p)


def spax_greedy_allocation(params, alpha: float, p_target: float, err, p_max: float = 1.0,
                           max_steps: int = 100000):
    """Per-matrix sparsities of one block (the library's greedy allocation). err(p) -> block
    error for a numpy array of per-matrix sparsities. Returns (p, order)."""
    f = np.ascontiguousarray(params, dtype=np.float64)
    n = f.size
    cb = BLOCK_ERROR_FN(lambda pp, nn, ctx: float(err(np.ctypeslib.as_array(pp, (nn,)).copy())))
    p = np.zeros(n, np.float64)
    order = np.zeros(max(1, max_steps), np.int32)
    steps = ctypes.c_int32(0)
    _check("spax_greedy_allocation", _lib.spax_greedy_allocation(
        f.ctypes.data_as(_P), n, alpha, p_target, p_max, ctypes.cast(cb, _P), None, max_steps,
        p.ctypes.data_as(_P), order.ctypes.data_as(_P), ctypes.byref(steps)))
    return p, order[: steps.value].copy()


def spax_weight_bytes(d_out: int, full_fmt: int, n_full: int, n_approx: int) -> int:
    return int(_lib.spax_weight_bytes(d_out, full_fmt, int(n_full), int(n_approx)))


# ------------------------------------------------------------------------------ device calls

@dataclass
class PackedMatrix:
    """Both pools of a packed d_out x d_in matrix (device uint8 tensors) and its C descriptor."""
    d_out: int
    d_in: int
    full_fmt: int
    full: torch.Tensor
    approx: torch.Tensor

    def desc(self) -> spax_packed:
        return spax_packed(self.d_out, self.d_in, self.full_fmt, 0, self.full.data_ptr(),
                           self.approx.data_ptr())


def alloc_packed(d_out: int, d_in: int, full_fmt: int, device="cuda") -> PackedMatrix:
    fb, ab = spax_pack_bytes(d_out, d_in, full_fmt)
    return PackedMatrix(d_out, d_in, full_fmt,
                        torch.empty(fb, dtype=torch.uint8, device=device),
                        torch.empty(ab, dtype=torch.uint8, device=device))


def packed_to_host(pm: PackedMatrix) -> PackedMatrix:
    """A copy of a packed matrix in page-locked host memory. Unified addressing maps such memory
    into the device address space, so the GEMV kernels read the pools straight over the host
    link (the offloaded-weights setting); the descriptor's pointers are the host pointers."""
    full = torch.empty(pm.full.numel(), dtype=torch.uint8, pin_memory=True)
    approx = torch.empty(pm.approx.numel(), dtype=torch.uint8, pin_memory=True)
    full.copy_(pm.full)
    approx.copy_(pm.approx)
    return PackedMatrix(pm.d_out, pm.d_in, pm.full_fmt, full, approx)


def spax_pack_weights(W: torch.Tensor, full_fmt: int, dst: PackedMatrix, stream=None) -> None:
    d_out, d_in = W.shape
    if (dst.d_out, dst.d_in, dst.full_fmt) != (d_out, d_in, full_fmt):
        raise ValueError("destination descriptor does not match W")
    fb, ab = spax_pack_bytes(d_out, d_in, full_fmt)
    if dst.full.numel() < fb or dst.approx.numel() < ab:
        raise ValueError("destination pools too small")
    _check("spax_pack_weights", _lib.spax_pack_weights(
        _dev(W, torch.bfloat16, "W"), d_out, d_in, full_fmt, _dev(dst.full, torch.uint8, "full"),
        _dev(dst.approx, torch.uint8, "approx"), _stream(stream)))


def spax_calibrate_thresholds(calib_x: torch.Tensor, s_skip_bp: int, s_below_full_bp: int,
                              t_out: torch.Tensor, status: torch.Tensor, ws: torch.Tensor,
                              stream=None) -> None:
    n_tok, d_in = calib_x.shape
    _check("spax_calibrate_thresholds", _lib.spax_calibrate_thresholds(
        _dev(calib_x, torch.float32, "calib_x"), n_tok, d_in, s_skip_bp, s_below_full_bp,
        _dev(t_out, torch.float32, "t_out"), _dev(status, torch.int32, "status"),
        _dev(ws, None, "ws"), ws.numel() * ws.element_size(), _stream(stream)))


def mask_params(mode: int, *, t_skip=0.0, t_full=0.0, k_full=0, k_approx=0, s_skip_bp=0,
                s_below_full_bp=0, delta_bp=0) -> spax_mask_params:
    """The rule's parameters (spax.h, spax_mask_params). In MASK_TOPK mode t_full / t_skip may
    carry a guess of the |x| at rank k_full / k_full + k_approx (calibrated quantiles); it only
    speeds the selection up when it holds, and 0 means no guess. MASK_TOPK_SCALED is the same
    rule with the guesses given as multiples of the token's mean |x|."""
    return spax_mask_params(mode, t_skip, t_full, k_full, k_approx, s_skip_bp, s_below_full_bp,
                            delta_bp)


def spax_build_mask(x: torch.Tensor, params: spax_mask_params, tier: torch.Tensor,
                    full_idx: torch.Tensor, approx_idx: torch.Tensor, counts: torch.Tensor,
                    status: torch.Tensor, stream=None) -> None:
    d_in = x.numel()
    for t, n in ((tier, d_in), (full_idx, d_in), (approx_idx, d_in), (counts, 4)):
        if t.numel() < n:
            raise ValueError("mask output too small")
    _check("spax_build_mask", _lib.spax_build_mask(
        _dev(x, torch.float32, "x"), d_in, ctypes.byref(params), _dev(tier, torch.uint8, "tier"),
        _dev(full_idx, torch.int32, "full_idx"), _dev(approx_idx, torch.int32, "approx_idx"),
        _dev(counts, torch.int32, "counts"), _dev(status, torch.int32, "status"),
        _stream(stream)))


def spax_tiered_gemv(W: PackedMatrix, x: torch.Tensor, full_idx: torch.Tensor,
                     approx_idx: torch.Tensor, counts: torch.Tensor, y: torch.Tensor,
                     status: torch.Tensor, ws: torch.Tensor, stream=None, desc=None) -> None:
    if x.numel() != W.d_in or y.numel() != W.d_out:
        raise ValueError("x / y sizes do not match W")
    d = W.desc() if desc is None else desc
    _check("spax_tiered_gemv", _lib.spax_tiered_gemv(
        ctypes.byref(d), _dev(x, torch.float32, "x"), _dev(full_idx, torch.int32, "full_idx"),
        _dev(approx_idx, torch.int32, "approx_idx"), _dev(counts, torch.int32, "counts"),
        _dev(y, torch.float32, "y"), _dev(status, torch.int32, "status"), _dev(ws, None, "ws"),
        ws.numel() * ws.element_size(), _stream(stream)))


def spax_masked_gemv(W: PackedMatrix, x: torch.Tensor, params: spax_mask_params, y: torch.Tensor,
                     status: torch.Tensor, ws: torch.Tensor, tier=None, full_idx=None,
                     approx_idx=None, counts=None, stream=None, desc=None) -> None:
    """The mask and the tiered GEMV in one launch; tier / lists / counts are optional outputs."""
    if x.numel() != W.d_in or y.numel() != W.d_out:
        raise ValueError("x / y sizes do not match W")
    for t, n in ((tier, W.d_in), (full_idx, W.d_in), (approx_idx, W.d_in), (counts, 4)):
        if t is not None and t.numel() < n:
            raise ValueError("mask output too small")
    d = W.desc() if desc is None else desc
    _check("spax_masked_gemv", _lib.spax_masked_gemv(
        ctypes.byref(d), _dev(x, torch.float32, "x"), ctypes.byref(params),
        _dev(y, torch.float32, "y"), _dev(tier, torch.uint8, "tier"),
        _dev(full_idx, torch.int32, "full_idx"), _dev(approx_idx, torch.int32, "approx_idx"),
        _dev(counts, torch.int32, "counts"), _dev(status, torch.int32, "status"),
        _dev(ws, None, "ws"), ws.numel() * ws.element_size(), _stream(stream)))


def spax_column_norms(W: torch.Tensor, norms: torch.Tensor, stream=None) -> None:
    """Per-column Euclidean norms of the row-major bf16 W (for the WINA score)."""
    d_out, d_in = W.shape
    if norms.numel() < d_in:
        raise ValueError("norms too small")
    _check("spax_column_norms", _lib.spax_column_norms(
        _dev(W, torch.bfloat16, "W"), d_out, d_in, _dev(norms, torch.float32, "norms"),
        _stream(stream)))


def spax_masked_gemv_wina(W: PackedMatrix, x: torch.Tensor, norms: torch.Tensor,
                          params: spax_mask_params, y: torch.Tensor, status: torch.Tensor,
                          ws: torch.Tensor, tier=None, full_idx=None, approx_idx=None, counts=None,
                          stream=None, desc=None) -> None:
    """spax_masked_gemv ranking columns by the WINA score |x_j| * norms[j]."""
    if x.numel() != W.d_in or norms.numel() != W.d_in or y.numel() != W.d_out:
        raise ValueError("x / norms / y sizes do not match W")
    for t, n in ((tier, W.d_in), (full_idx, W.d_in), (approx_idx, W.d_in), (counts, 4)):
        if t is not None and t.numel() < n:
            raise ValueError("mask output too small")
    d = W.desc() if desc is None else desc
    _check("spax_masked_gemv_wina", _lib.spax_masked_gemv_wina(
        ctypes.byref(d), _dev(x, torch.float32, "x"), _dev(norms, torch.float32, "norms"),
        ctypes.byref(params), _dev(y, torch.float32, "y"), _dev(tier, torch.uint8, "tier"),
        _dev(full_idx, torch.int32, "full_idx"), _dev(approx_idx, torch.int32, "approx_idx"),
        _dev(counts, torch.int32, "counts"), _dev(status, torch.int32, "status"),
        _dev(ws, None, "ws"), ws.numel() * ws.element_size(), _stream(stream)))


def spax_masked_gemv_swiglu(W: PackedMatrix, gu: torch.Tensor, params: spax_mask_params,
                            y: torch.Tensor, status: torch.Tensor, ws: torch.Tensor, x_out=None,
                            tier=None, full_idx=None, approx_idx=None, counts=None, stream=None,
                            desc=None) -> None:
    """spax_masked_gemv on x = silu(g) * u formed in the kernel from gu = [g; u] (2 * d_in)."""
    if gu.numel() != 2 * W.d_in or y.numel() != W.d_out:
        raise ValueError("gu / y sizes do not match W")
    for t, n in ((x_out, W.d_in), (tier, W.d_in), (full_idx, W.d_in), (approx_idx, W.d_in),
                 (counts, 4)):
        if t is not None and t.numel() < n:
            raise ValueError("output too small")
    d = W.desc() if desc is None else desc
    _check("spax_masked_gemv_swiglu", _lib.spax_masked_gemv_swiglu(
        ctypes.byref(d), _dev(gu, torch.float32, "gu"), ctypes.byref(params),
        _dev(y, torch.float32, "y"), _dev(x_out, torch.float32, "x_out"),
        _dev(tier, torch.uint8, "tier"), _dev(full_idx, torch.int32, "full_idx"),
        _dev(approx_idx, torch.int32, "approx_idx"), _dev(counts, torch.int32, "counts"),
        _dev(status, torch.int32, "status"), _dev(ws, None, "ws"),
        ws.numel() * ws.element_size(), _stream(stream)))


def spax_tiered_gemv_fixed_scratch(W: PackedMatrix, x: torch.Tensor, full_idx: torch.Tensor,
                                   approx_idx: torch.Tensor, counts: torch.Tensor, y: torch.Tensor,
                                   status: torch.Tensor, stream=None, desc=None) -> None:
    """spax_tiered_gemv without a workspace argument: the library's own per-device scratch array
    is used, so nothing is allocated. Calls on one device must not overlap."""
    if x.numel() != W.d_in or y.numel() != W.d_out:
        raise ValueError("x / y sizes do not match W")
    d = W.desc() if desc is None else desc
    _check("spax_tiered_gemv_fixed_scratch", _lib.spax_tiered_gemv_fixed_scratch(
        ctypes.byref(d), _dev(x, torch.float32, "x"), _dev(full_idx, torch.int32, "full_idx"),
        _dev(approx_idx, torch.int32, "approx_idx"), _dev(counts, torch.int32, "counts"),
        _dev(y, torch.float32, "y"), _dev(status, torch.int32, "status"), _stream(stream)))


def spax_fixed_scratch_bytes() -> int:
    return int(_lib.spax_fixed_scratch_bytes())


def spax_fixed_scratch_reset(stream=None) -> None:
    """Zero the current device's fixed scratch array (after a fixed-scratch call reported a
    device error such as ERR_TIMEOUT)."""
    _check("spax_fixed_scratch_reset", _lib.spax_fixed_scratch_reset(_stream(stream)))


def spax_test_tiered_gemv_timeout(W: PackedMatrix, x: torch.Tensor, full_idx: torch.Tensor,
                                  approx_idx: torch.Tensor, counts: torch.Tensor, y: torch.Tensor,
                                  status: torch.Tensor, ws=None, wait_limit_ns: int = 20_000_000,
                                  stream=None) -> None:
    """Failure-detection test hook: the list-driven GEMV with the last split of every row tile
    left out, so its waits run out after wait_limit_ns and status becomes ERR_TIMEOUT. ws None
    selects the fixed scratch array."""
    d = W.desc()
    _check("spax_test_tiered_gemv_timeout", _lib.spax_test_tiered_gemv_timeout(
        ctypes.byref(d), _dev(x, torch.float32, "x"), _dev(full_idx, torch.int32, "full_idx"),
        _dev(approx_idx, torch.int32, "approx_idx"), _dev(counts, torch.int32, "counts"),
        _dev(y, torch.float32, "y"), _dev(status, torch.int32, "status"),
        None if ws is None else _dev(ws, None, "ws"),
        0 if ws is None else ws.numel() * ws.element_size(), int(wait_limit_ns),
        _stream(stream)))


def spax_output_change(y: torch.Tensor, y_ref: torch.Tensor, acc: torch.Tensor,
                       stream=None) -> None:
    """acc[0] += sum (y - y_ref)^2, acc[1] += sum y_ref^2 (fp64 device accumulators)."""
    if y.numel() != y_ref.numel() or acc.numel() < 2:
        raise ValueError("sizes do not match")
    _check("spax_output_change", _lib.spax_output_change(
        _dev(y, torch.float32, "y"), _dev(y_ref, torch.float32, "y_ref"), y.numel(),
        _dev(acc, torch.float64, "acc"), _stream(stream)))


def spax_probe_sensitivity(W: PackedMatrix, X: torch.Tensor, s_probe_bp: int, y2: torch.Tensor,
                           acc: torch.Tensor, status: torch.Tensor, ws: torch.Tensor, stream=None,
                           desc=None) -> None:
    """Output change of one matrix at probe sparsity s_probe_bp / 1e4 over the calibration
    tokens X [n_tok, d_in], accumulated into acc (two fp64 on the device)."""
    n_tok, d_in = X.shape
    if d_in != W.d_in or y2.numel() < 2 * W.d_out or acc.numel() < 2:
        raise ValueError("sizes do not match W")
    d = W.desc() if desc is None else desc
    _check("spax_probe_sensitivity", _lib.spax_probe_sensitivity(
        ctypes.byref(d), _dev(X, torch.float32, "X"), n_tok, s_probe_bp,
        _dev(y2, torch.float32, "y2"), _dev(acc, torch.float64, "acc"),
        _dev(status, torch.int32, "status"), _dev(ws, None, "ws"), ws.numel() * ws.element_size(),
        _stream(stream)))


def spax_dense_gemv(Wt: torch.Tensor, x: torch.Tensor, y: torch.Tensor, d_out: int, d_in: int,
                    status: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    if x.numel() != d_in or y.numel() != d_out or Wt.numel() * Wt.element_size() < 2 * d_in * d_out:
        raise ValueError("sizes do not match")
    _check("spax_dense_gemv", _lib.spax_dense_gemv(
        _dev_or_pinned(Wt, "Wt"), _dev(x, torch.float32, "x"), _dev(y, torch.float32, "y"), d_out,
        d_in, _dev(status, torch.int32, "status"), _dev(ws, None, "ws"),
        ws.numel() * ws.element_size(), _stream(stream)))


def alloc_workspace(op: int, d_out: int, d_in: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace (the GEMV's flagged partial sums must start at zero)."""
    n = spax_workspace_bytes(op, d_out, d_in)
    if n == 0:
        raise SpaxError("spax_workspace_bytes", ERR_SHAPE)
    return torch.zeros(n, dtype=torch.uint8, device=device)


# ------------------------------------------------------------- the decode layer between projections

# These calls stand between kernels of a few microseconds, so their argument checks are kept short:
# each tensor's type, device and layout in place, the wording of an error only where one fails
# (_refuse), and the stream's handle without its object.
_f32, _i32, _u8 = torch.float32, torch.int32, torch.uint8
_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _refuse(dtype, dev: int, **tensors):
    """Words the error of the first of these tensors that is not of the type, on the device and (rows
    with a name in capitals may be strided) contiguous."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name.lower()} must be a CUDA tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name.lower()} must be {dtype}, got {t.dtype}")
        if t.get_device() != dev:
            raise ValueError(f"{name.lower()} is on cuda:{t.get_device()}, the current device is "
                             f"cuda:{dev}")
        if name.islower() and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _row_stride(t: torch.Tensor, n: int, heads: int, d: int, name: str) -> int:
    """The tokens' stride of [n, heads, d] whose heads are contiguous."""
    if t.shape != (n, heads, d):
        raise ValueError(f"{name} must be [{n}, {heads}, {d}], got {list(t.shape)}")
    row, head, entry = t.stride()
    if entry != 1 or (head != d and heads > 1 and n > 0):
        raise ValueError(f"{name}'s heads must be contiguous within a token")
    return row


class _Described:
    """What a call's descriptor is formed from. It is formed once, so its attributes are fixed with it; a
    tensor whose storage is replaced under it (t.data = ..., a module moved or cast) is seen by its
    address at the next call, and the descriptor is formed again, with its checks."""

    _fixed = frozenset()  # the attributes of a formed object; a caller's own are free

    def __init__(self, **given):
        self._put(given)
        formed = self._form()
        self._put(formed)
        self._put({"_fixed": frozenset((*given, *formed, "_fixed"))})

    def _put(self, values):
        for name, value in values.items():  # not through __dict__, whose use slows later reads
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        if name in self._fixed:
            raise AttributeError(f"{type(self).__name__}.{name} is fixed; make a new {type(self).__name__}")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        if name in self._fixed:
            self.__setattr__(name, None)
        super().__delattr__(name)

    def _again(self):
        self._put(self._form())


class KvCache(_Described):
    """A paged key-value cache of one layer: keys and values as [n_pages, page_size, n_kv_heads,
    head_dim] tensors of bfloat16 or float8_e4m3fn, views with any order of the outer dimensions
    (both with the same strides). An 8-bit element stands for its value times k_scale / v_scale."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: float = 1.0,
                 v_scale: float = 1.0):
        super().__init__(k=k, v=v, k_scale=k_scale, v_scale=v_scale)

    def _form(self):
        k, v = self.k, self.v
        kinds = {torch.bfloat16: KV_BF16, torch.float8_e4m3fn: KV_E4M3}
        if not k.is_cuda or not v.is_cuda or k.device != v.device:
            raise TypeError("the cache's pools must be CUDA tensors of one device")
        if k.dtype not in kinds or k.dtype != v.dtype:
            raise TypeError("the cache's pools must both be bfloat16 or both float8_e4m3fn")
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("the cache's pools must be [n_pages, page_size, n_kv_heads, head_dim] "
                             "with the same strides, the last of them 1")
        dtype, at = kinds[k.dtype], (k.data_ptr(), v.data_ptr())
        desc = spax_kv_cache(*k.shape, dtype, self.k_scale, self.v_scale, 0, *k.stride()[:3], *at)
        return dict(zip(("n_pages", "page_size", "n_kv_heads", "head_dim"), k.shape), dtype=dtype,
                    device=k.device, _dev=k.get_device(), _k_at=at[0], _v_at=at[1], _k_now=k.data_ptr,
                    _v_now=v.data_ptr, _desc=desc, _ref=ctypes.byref(desc))

    def _for(self, dev: int):
        if self._k_now() != self._k_at or self._v_now() != self._v_at:
            self._again()
        if self._dev != dev:
            raise ValueError(f"the cache is on cuda:{self._dev}, the current device is cuda:{dev}")
        return self._ref

    def desc(self) -> spax_kv_cache:
        self._for(self._dev)
        return self._desc


def alloc_kv_cache(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                   dtype: int = KV_BF16, heads_first: bool = False, k_scale: float = 1.0,
                   v_scale: float = 1.0, device="cuda") -> KvCache:
    """A zeroed cache; heads_first lays a page out as [n_kv_heads][page_size][head_dim]."""
    t = {KV_BF16: torch.bfloat16, KV_E4M3: torch.float8_e4m3fn}[dtype]
    shape = ((n_pages, n_kv_heads, page_size, head_dim) if heads_first
             else (n_pages, page_size, n_kv_heads, head_dim))
    k, v = (torch.zeros(shape, dtype=torch.uint8 if dtype == KV_E4M3 else t,
                        device=device).view(t) for _ in range(2))
    if heads_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return KvCache(k, v, k_scale, v_scale)


class Rope(_Described):
    """Rotation by position: inv_freq, fp64 [rot_dim / 2] on the device, the radians per position
    of each pair; pairs (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved."""

    def __init__(self, inv_freq: torch.Tensor, interleaved: bool = False):
        super().__init__(inv_freq=inv_freq, interleaved=bool(interleaved))

    def _form(self):
        f = self.inv_freq
        dev = f.get_device()
        _refuse(torch.float64, dev, inv_freq=f)
        desc = spax_rope(2 * f.numel(), int(self.interleaved), f.data_ptr())
        return dict(_dev=dev, _at=f.data_ptr(), _now=f.data_ptr, _desc=desc, _ref=ctypes.byref(desc))

    def _for(self, dev: int):
        if self._now() != self._at:
            self._again()
        if self._dev != dev:
            raise ValueError(f"the rope is on cuda:{self._dev}, the current device is cuda:{dev}")
        return self._ref


class Norm(_Described):
    """A norm's kind (NORM_RMS or NORM_LAYER), eps, and its weight and bias ([d], both fp32 or both
    bf16; None: none)."""

    def __init__(self, weight=None, bias=None, eps: float = 1e-5, kind: int = NORM_RMS):
        super().__init__(weight=weight, bias=bias, eps=eps, kind=kind)

    def _form(self):
        given = [t for t in (self.weight, self.bias) if t is not None]
        types = {t.dtype for t in given} or {torch.float32}
        if len(types) != 1 or not types <= {torch.float32, torch.bfloat16}:
            raise TypeError("weight and bias must both be float32 or both bfloat16")
        if len({t.numel() for t in given}) > 1:
            raise ValueError("weight and bias must have the same size")
        d = given[0].numel() if given else None
        device = given[0].get_device() if given else None
        dt = types.pop()
        _refuse(dt, device, weight=self.weight, bias=self.bias)
        now = [int if t is None else t.data_ptr for t in (self.weight, self.bias)]  # int(): 0, no address
        at = [f() for f in now]
        desc = spax_norm(self.kind, int(dt == torch.bfloat16), *at, self.eps)
        return dict(d=d, device=device, _w_at=at[0], _b_at=at[1], _w_now=now[0], _b_now=now[1], _desc=desc,
                    _ref=ctypes.byref(desc))

    def _for(self, d: int, dev: int):
        if self._w_now() != self._w_at or self._b_now() != self._b_at:
            self._again()
        if self.d is not None and (self.d != d or self.device != dev):
            raise ValueError(f"the norm's weight has {self.d} entries on cuda:{self.device}, "
                             f"the rows {d} on cuda:{dev}")
        return self._ref


def spax_kv_append(cache: KvCache, q, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                   page_table: torch.Tensor, status: torch.Tensor, rope=None, seq=None, q_out=None,
                   stream=None) -> None:
    """Rotate q and k by pos and write k and v into the cache. q [tokens, heads, head_dim], k and v
    [tokens, n_kv_heads, head_dim], fp32, the tokens' strides free (parts of one qkv row); q None:
    keys and values alone. q_out None: q is rotated in place. pos, seq int32 [tokens] (seq None:
    token t is of sequence t), page_table int32 [sequences, pages]; pos < 0 marks padding."""
    dev = _device()
    ref = cache._for(dev)
    d, heads_kv, n = cache.head_dim, cache.n_kv_heads, pos.numel()
    ks = _row_stride(k, n, heads_kv, d, "k")
    vs = _row_stride(v, n, heads_kv, d, "v")
    heads = qs = os_ = 0
    qp = op = sq = None
    if q is not None:
        heads = q.shape[1] if q.dim() == 3 else 0
        os_ = qs = _row_stride(q, n, heads, d, "q")
        qp = op = q.data_ptr()
        if q.dtype is not _f32 or q.get_device() != dev:
            _refuse(_f32, dev, Q=q)
        if q_out is not None:
            os_ = _row_stride(q_out, n, heads, d, "q_out")
            op = q_out.data_ptr()
            if q_out.dtype is not _f32 or q_out.get_device() != dev:
                _refuse(_f32, dev, Q_OUT=q_out)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if (k.dtype is not _f32 or v.dtype is not _f32 or k.get_device() != dev
            or v.get_device() != dev):
        _refuse(_f32, dev, K=k, V=v)
    if (pos.dtype is not _i32 or page_table.dtype is not _i32 or status.dtype is not _i32
            or pos.get_device() != dev or page_table.get_device() != dev
            or status.get_device() != dev or not pos.is_contiguous()
            or not page_table.is_contiguous()):
        _refuse(_i32, dev, pos=pos, page_table=page_table, status=status)
    n_seq, max_pages = page_table.shape
    if seq is not None:
        sq = seq.data_ptr()
        if (seq.dtype is not _i32 or seq.get_device() != dev or not seq.is_contiguous()
                or seq.numel() != n):
            _refuse(_i32, dev, seq=seq)
            raise ValueError("seq's size does not match pos")
    elif n_seq < n:
        raise ValueError("page_table has fewer rows than there are tokens")
    st = _lib.spax_kv_append(
        ref, qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, n, heads, sq, pos.data_ptr(),
        page_table.data_ptr(), n_seq, max_pages, None if rope is None else rope._for(dev), op, os_,
        status.data_ptr(), _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise SpaxError("spax_kv_append", st)


def spax_attention_workspace_bytes(n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(_lib.spax_attention_workspace_bytes(n_heads, n_kv_heads, head_dim))


def spax_attention_plan_sms(n_seq: int, n_heads: int, n_kv_heads: int, head_dim: int, kv_dtype: int,
                            max_positions: int, window: int, sm_count: int):
    """(CTAs, workspace bytes) of spax_paged_attention on a GPU with sm_count SMs; no CUDA call."""
    ctas, ws = ctypes.c_int32(), ctypes.c_size_t()
    _check("spax_attention_plan_sms", _lib.spax_attention_plan_sms(
        n_seq, n_heads, n_kv_heads, head_dim, kv_dtype, max_positions, window, sm_count,
        ctypes.byref(ctas), ctypes.byref(ws)))
    return ctas.value, ws.value


def alloc_attention_workspace(cache: KvCache, n_heads: int) -> torch.Tensor:
    """A zeroed workspace of spax_paged_attention for this cache's layout, any lengths."""
    with torch.cuda.device(cache.device):
        n = spax_attention_workspace_bytes(n_heads, cache.n_kv_heads, cache.head_dim)
    if n == 0:
        raise SpaxError("spax_attention_workspace_bytes", ERR_SHAPE)
    return torch.zeros(n, dtype=torch.uint8, device=cache.device)


def spax_paged_attention(cache: KvCache, q: torch.Tensor, page_table: torch.Tensor,
                         seq_lens: torch.Tensor, out: torch.Tensor, status: torch.Tensor,
                         ws: torch.Tensor, scale: float, window: int = 0, softcap: float = 0.0,
                         lse=None, stream=None) -> None:
    """Attention of one new token of each sequence over the cache: q fp32 [sequences, heads,
    head_dim] (the sequences' stride free), seq_lens int32 [sequences] counting the new token, out
    fp32 as q, contiguous; lse (optional) fp32 [sequences, heads]."""
    dev = _device()
    ref = cache._for(dev)
    d, n = cache.head_dim, seq_lens.numel()
    heads = q.shape[1] if q.dim() == 3 else 0
    qs = _row_stride(q, n, heads, d, "q")
    n_seq, max_pages = page_table.shape
    if out.shape != q.shape or n_seq < n or (lse is not None and lse.numel() != n * heads):
        raise ValueError("out / page_table / lse sizes do not match q and seq_lens")
    if (q.dtype is not _f32 or out.dtype is not _f32 or q.get_device() != dev
            or out.get_device() != dev or not out.is_contiguous()):
        _refuse(_f32, dev, Q=q, out=out)
    if lse is not None and (lse.dtype is not _f32 or lse.get_device() != dev
                            or not lse.is_contiguous()):
        _refuse(_f32, dev, lse=lse)
    if (page_table.dtype is not _i32 or seq_lens.dtype is not _i32 or status.dtype is not _i32
            or page_table.get_device() != dev or seq_lens.get_device() != dev
            or status.get_device() != dev or not page_table.is_contiguous()
            or not seq_lens.is_contiguous()):
        _refuse(_i32, dev, page_table=page_table, seq_lens=seq_lens, status=status)
    if not -1 << 31 <= window < 1 << 31:  # the structure's field would keep its low 32 bits
        raise ValueError(f"window must be at least 0 and below 2^31, got {window}")
    if ws.dtype is not _u8 or ws.get_device() != dev or not ws.is_contiguous():
        _refuse(_u8, dev, ws=ws)
    st = _lib.spax_paged_attention(
        ref, q.data_ptr(), qs, n, heads, page_table.data_ptr(), max_pages,
        seq_lens.data_ptr(), ctypes.byref(spax_attn_params(scale, softcap, window)),
        out.data_ptr(), None if lse is None else lse.data_ptr(), status.data_ptr(), ws.data_ptr(),
        ws.numel(), _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise SpaxError("spax_paged_attention", st)


def spax_residual_norm(h: torch.Tensor, y, r, x, pre=None, post=None, gate=None,
                       res_scale: float = 1.0, out_scale: float = 1.0, stream=None) -> None:
    """r = res_scale h + out_scale gate N_post(y), x = N_pre(r) by rows: h, y, r, x fp32
    [..., d] of the same size (y None: r = res_scale h; r or x None: not written; r and x may be h
    or y), gate fp32 [d] for all rows or one row each, pre and post a Norm or None."""
    dev = _device()
    shape = h.shape
    d = shape[-1] if len(shape) else 0
    if d == 0:
        raise ValueError("rows must have entries")
    n = h.numel() // d
    yp = rp = xp = gp = None
    gs = 0
    if h.dtype is not _f32 or h.get_device() != dev or not h.is_contiguous():
        _refuse(_f32, dev, h=h)
    if y is not None:
        yp = y.data_ptr()
        if (y.dtype is not _f32 or y.get_device() != dev or not y.is_contiguous()
                or y.shape != shape):
            _refuse(_f32, dev, y=y)
            raise ValueError("y's size does not match h")
    if r is not None:
        rp = r.data_ptr()
        if (r.dtype is not _f32 or r.get_device() != dev or not r.is_contiguous()
                or r.shape != shape):
            _refuse(_f32, dev, r=r)
            raise ValueError("r's size does not match h")
    if x is not None:
        xp = x.data_ptr()
        if (x.dtype is not _f32 or x.get_device() != dev or not x.is_contiguous()
                or x.shape != shape):
            _refuse(_f32, dev, x=x)
            raise ValueError("x's size does not match h")
    if gate is not None:
        gp = gate.data_ptr()
        if gate.dtype is not _f32 or gate.get_device() != dev or not gate.is_contiguous():
            _refuse(_f32, dev, gate=gate)
        if gate.dim() == 0 or gate.shape[-1] != d or gate.numel() not in (d, n * d):
            raise ValueError("gate must be [d] or of h's size")
        gs = d if gate.numel() == n * d and gate.dim() > 1 else 0
    st = _lib.spax_residual_norm(
        h.data_ptr(), yp, n, d, None if post is None else post._for(d, dev), gp, gs, res_scale,
        out_scale, None if pre is None else pre._for(d, dev), rp, xp,
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise SpaxError("spax_residual_norm", st)
