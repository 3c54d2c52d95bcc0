"""Python binding of the B200 transposable N:M mask library (include/tsenor.h).

Argument marshalling only: every step of the solver runs in the CUDA kernels
of libtsenor_b200.so.  PyTorch provides device memory and streams.  There is
no CPU fallback: if the library is missing, importing a function raises.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os
from typing import NamedTuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtsenor_b200.so")

TSENOR_F32, TSENOR_BF16 = 0, 1
BLOCKS = {"row": 0, "column": 1, "tile": 2}
FORMS = {"nt": 0, "nn": 1, "tn": 2}
STATUS = {0: "TSENOR_OK", -1: "TSENOR_ERR_ARG", -2: "TSENOR_ERR_SHAPE", -3: "TSENOR_ERR_UNSUPPORTED_M",
          -4: "TSENOR_ERR_CUDA", -5: "TSENOR_ERR_DEVICE", -6: "TSENOR_ERR_TOO_LARGE"}
NOALLOC_MAX_PARAMS = 16 * 1024 * 1024
DISTILL_MAX_TOP, DISTILL_MAX_VOCAB = 1024, 262144
MAX_TAU = 80.0            # TSENOR_MAX_TAU: larger tau is rejected (TSENOR_ERR_ARG)
EXPORTS = ("tsenor_mask", "tsenor_plan", "tsenor_round", "tsenor_objective", "tsenor_error_count",
           "tsenor_status_string", "tsenor_last_error", "tsenor_mask_noalloc", "tsenor_mask_safeguard",
           "tsenor_mask_padded", "tsenor_mask_warm", "tsenor_plan_warm", "tsenor_mask_scores", "tsenor_mask_host",
           "tsenor_scale_bytes", "tsenor_quantize", "tsenor_quantize_pair", "tsenor_dequantize", "tsenor_matmul",
           "tsenor_distill_loss", "tsenor_distill_step", "tsenor_distill_grad")

_lib = None


class TsenorError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


def lib() -> C.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m sparse_mask_search_b200.build` (nvcc, sm_100a)")
        L = C.CDLL(LIB_PATH)
        p, i64, i32, f32 = C.c_void_p, C.c_int64, C.c_int, C.c_float
        L.tsenor_mask.argtypes = [p, i32, i64, i64, i32, i32, f32, i32, i32, p, p]
        L.tsenor_mask_noalloc.argtypes = [p, i32, i64, i64, i32, i32, f32, i32, i32, p, p]
        L.tsenor_plan.argtypes = [p, i32, i64, i64, i32, i32, f32, i32, p, p]
        L.tsenor_mask_padded.argtypes = [p, i32, i64, i64, i32, i32, f32, i32, i32, p, p]
        L.tsenor_mask_safeguard.argtypes = [p, i32, i64, i64, i32, i32, f32, i32, i32, p, p, p, p]
        L.tsenor_mask_scores.argtypes = [p, i64, i64, i32, i32, f32, i32, i32, p, p]
        L.tsenor_mask_host.argtypes = [p, i32, i64, i64, i32, i32, f32, i32, i32, p, p]
        L.tsenor_mask_warm.argtypes = [p, i32, i64, i64, i32, i32, f32, i32, i32, f32, i32, p, p, p, p]
        L.tsenor_plan_warm.argtypes = [p, i32, i64, i64, i32, i32, f32, i32, f32, i32, p, p, p, p]
        L.tsenor_round.argtypes = [p, p, i32, i64, i64, i32, i32, i32, p, p]
        L.tsenor_objective.argtypes = [p, i32, i64, i64, p, i32, i32, p, p]
        L.tsenor_error_count.argtypes = [p, C.POINTER(C.c_int64)]
        L.tsenor_scale_bytes.argtypes = [i64, i64]
        L.tsenor_scale_bytes.restype = i64
        L.tsenor_quantize.argtypes = [p, i32, i64, i64, i64, i32, p, p, i64, p, p, p]
        L.tsenor_quantize_pair.argtypes = [p, i32, i64, i64, i64, p, i64, p, p, i64, p, p]
        L.tsenor_dequantize.argtypes = [p, i64, i64, i64, p, i32, p, i32, i64, p]
        L.tsenor_matmul.argtypes = [i32, p, i64, p, p, i64, p, i64, i64, i64, p, p, i32, i64, p]
        L.tsenor_distill_loss.argtypes = [p, i32, i64, i64, i64, p, p, i32, p, f32, p, p, p]
        L.tsenor_distill_step.argtypes = [p, i32, i64, i64, i64, p, p, i32, p, f32, p, p, p, i64, p]
        L.tsenor_distill_grad.argtypes = [p, i32, i64, i64, i64, p, p, i32, p, f32, p, p, p, i64, p]
        L.tsenor_status_string.argtypes = [i32]
        L.tsenor_status_string.restype = C.c_char_p
        L.tsenor_last_error.restype = C.c_char_p
        for name in EXPORTS:
            getattr(L, name).restype = getattr(L, name).restype or C.c_int
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != 0:
        L = lib()
        msg = L.tsenor_status_string(status).decode()
        if status == -4:
            msg += ": " + L.tsenor_last_error().decode()
        raise TsenorError(status, msg)


def _stream_handle(stream) -> int | None:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(W) -> int:
    import torch
    if W.dtype == torch.bfloat16:
        return TSENOR_BF16
    if W.dtype == torch.float32:
        return TSENOR_F32
    raise TypeError(f"W must be bfloat16 or float32, got {W.dtype}")


def words_per_row(cols: int) -> int:
    return (cols + 31) // 32


def _check_2d_cuda(t, name):
    if not t.is_cuda or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D CUDA tensor")


def tsenor_mask(W, N: int, M: int, tau: float, iters: int, sweeps: int, out=None, stream=None):
    """Transposable N:M mask of W; returns (rows, ceil(cols/32)) int32 words (bit patterns)."""
    import torch
    _check_2d_cuda(W, "W")
    rows, cols = W.shape
    if out is None:
        out = torch.empty((rows, words_per_row(cols)), dtype=torch.int32, device=W.device)
    _check(lib().tsenor_mask(W.data_ptr(), _dtype_code(W), rows, cols, N, M, float(tau), iters, sweeps,
                             out.data_ptr(), _stream_handle(stream)))
    return out


def tsenor_mask_noalloc(W, N: int, M: int, tau: float, iters: int, sweeps: int, out=None, stream=None):
    """tsenor_mask without any device allocation by the library.

    For callers whose device memory is reserved by another allocator or who
    run under a fixed memory budget.  The plan between the two kernels lives
    in a 64 MiB array inside the library (rows*cols <= NOALLOC_MAX_PARAMS).
    All calls on a device share that array: calls that overlap on the GPU
    race.  The first call on a device looks up the array's address; make it
    before any stream capture.  Only ``out`` is allocated here (by torch)
    when it is not given.
    """
    import torch
    _check_2d_cuda(W, "W")
    rows, cols = W.shape
    if out is None:
        out = torch.empty((rows, words_per_row(cols)), dtype=torch.int32, device=W.device)
    _check(lib().tsenor_mask_noalloc(W.data_ptr(), _dtype_code(W), rows, cols, N, M, float(tau), iters,
                                     sweeps, out.data_ptr(), _stream_handle(stream)))
    return out


def tsenor_mask_safeguard(W, prev_mask, N: int, M: int, tau: float, iters: int, sweeps: int, out=None,
                          kept=None, stream=None):
    """tsenor_mask that keeps, per block, prev_mask where it is valid and keeps more |W|.

    ``kept`` (optional int64 CUDA tensor of one element) receives the count of
    blocks that kept prev_mask (added to its value).
    """
    import torch
    _check_2d_cuda(W, "W")
    rows, cols = W.shape
    if out is None:
        out = torch.empty((rows, words_per_row(cols)), dtype=torch.int32, device=W.device)
    _check(lib().tsenor_mask_safeguard(W.data_ptr(), _dtype_code(W), rows, cols, N, M, float(tau), iters, sweeps,
                                       prev_mask.data_ptr(), out.data_ptr(),
                                       kept.data_ptr() if kept is not None else None, _stream_handle(stream)))
    return out


def tsenor_mask_scores(scores, N: int, M: int, tau: float, iters: int, sweeps: int, out=None, stream=None):
    """Transposable N:M mask of an importance-score matrix (float32; magnitudes are used)."""
    import torch
    _check_2d_cuda(scores, "scores")
    if scores.dtype != torch.float32:
        raise TypeError("scores must be float32")
    rows, cols = scores.shape
    if out is None:
        out = torch.empty((rows, words_per_row(cols)), dtype=torch.int32, device=scores.device)
    _check(lib().tsenor_mask_scores(scores.data_ptr(), rows, cols, N, M, float(tau), iters, sweeps, out.data_ptr(),
                                    _stream_handle(stream)))
    return out


def tsenor_mask_host(W_host, N: int, M: int, tau: float, iters: int, sweeps: int, out=None, stream=None):
    """tsenor_mask of a HOST matrix into a HOST mask, the copies overlapped with the solve.

    W_host: contiguous 2-D CPU tensor (bfloat16 or float32), ideally pinned.
    Returns the (rows, ceil(cols/32)) int32 mask on the host (pinned when
    allocated here).  The result is complete once ``stream`` (default: the
    current CUDA stream) reaches this point, e.g. after its synchronize().
    """
    import torch
    if W_host.is_cuda or W_host.dim() != 2 or not W_host.is_contiguous():
        raise ValueError("W_host must be a contiguous 2-D CPU tensor")
    rows, cols = W_host.shape
    if out is None:
        out = torch.empty((rows, words_per_row(cols)), dtype=torch.int32, pin_memory=True)
    elif out.is_cuda or not out.is_contiguous() or out.numel() < rows * words_per_row(cols):
        raise ValueError("out must be a contiguous CPU int32 tensor of (rows, ceil(cols/32))")
    _check(lib().tsenor_mask_host(W_host.data_ptr(), _dtype_code(W_host), rows, cols, N, M, float(tau), iters,
                                  sweeps, out.data_ptr(), _stream_handle(stream)))
    return out


def tsenor_mask_padded(W, N: int, M: int, tau: float, iters: int, sweeps: int, out=None, stream=None):
    """tsenor_mask for any shape: W is zero-padded to multiples of M, the mask cropped back."""
    import torch
    _check_2d_cuda(W, "W")
    rows, cols = W.shape
    if out is None:
        out = torch.empty((rows, words_per_row(cols)), dtype=torch.int32, device=W.device)
    _check(lib().tsenor_mask_padded(W.data_ptr(), _dtype_code(W), rows, cols, N, M, float(tau), iters, sweeps,
                                    out.data_ptr(), _stream_handle(stream)))
    return out


def _warm_buffers(W, M, potentials, iters_used):
    import torch
    rows, cols = W.shape
    nb = (rows // M) * (cols // M) if M > 0 and rows % M == 0 and cols % M == 0 else 0
    if potentials is None:
        potentials = torch.empty((nb, 2 * M), dtype=torch.float32, device=W.device)
    elif (potentials.dtype != torch.float32 or not potentials.is_cuda or not potentials.is_contiguous()
          or potentials.numel() < nb * 2 * M):
        raise ValueError("potentials must be a contiguous float32 CUDA tensor of (n_blocks, 2M)")
    if iters_used is None:
        iters_used = torch.empty((nb,), dtype=torch.int32, device=W.device)
    elif (iters_used.dtype != torch.int32 or not iters_used.is_cuda or not iters_used.is_contiguous()
          or iters_used.numel() < nb):
        raise ValueError("iters_used must be a contiguous int32 CUDA tensor of n_blocks")
    return potentials, iters_used


def tsenor_mask_warm(W, N: int, M: int, tau: float, iters: int, sweeps: int, tol: float = 0.0, potentials=None,
                     warm: bool = False, iters_used=None, out=None, stream=None):
    """tsenor_mask with warm start and adaptive stopping.

    potentials: (n_blocks, 2M) float32 CUDA tensor, U then V per block
    (natural-log units), read when ``warm`` and overwritten with the final
    state (allocated when None; then ``warm`` must be False).  ``tol`` > 0
    stops a block after the first iteration whose row and column potentials
    are all within tol.  Returns (mask, potentials, iters_used).
    """
    import torch
    _check_2d_cuda(W, "W")
    rows, cols = W.shape
    if warm and potentials is None:
        raise ValueError("warm start needs potentials")
    potentials, iters_used = _warm_buffers(W, M, potentials, iters_used)
    if out is None:
        out = torch.empty((rows, words_per_row(cols)), dtype=torch.int32, device=W.device)
    _check(lib().tsenor_mask_warm(W.data_ptr(), _dtype_code(W), rows, cols, N, M, float(tau), iters, sweeps,
                                  float(tol), int(bool(warm)), potentials.data_ptr(), iters_used.data_ptr(),
                                  out.data_ptr(), _stream_handle(stream)))
    return out, potentials, iters_used


def tsenor_plan_warm(W, N: int, M: int, tau: float, iters: int, tol: float = 0.0, potentials=None,
                     warm: bool = False, iters_used=None, out=None, stream=None):
    """The plan of tsenor_mask_warm; returns (plan, potentials, iters_used)."""
    import torch
    _check_2d_cuda(W, "W")
    rows, cols = W.shape
    if warm and potentials is None:
        raise ValueError("warm start needs potentials")
    potentials, iters_used = _warm_buffers(W, M, potentials, iters_used)
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=W.device)
    _check(lib().tsenor_plan_warm(W.data_ptr(), _dtype_code(W), rows, cols, N, M, float(tau), iters, float(tol),
                                  int(bool(warm)), potentials.data_ptr(), iters_used.data_ptr(), out.data_ptr(),
                                  _stream_handle(stream)))
    return out, potentials, iters_used


def tsenor_plan(W, N: int, M: int, tau: float, iters: int, out=None, stream=None):
    """Fractional plan S (fp32, same shape as W) after `iters` Dykstra iterations."""
    import torch
    _check_2d_cuda(W, "W")
    rows, cols = W.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=W.device)
    _check(lib().tsenor_plan(W.data_ptr(), _dtype_code(W), rows, cols, N, M, float(tau), iters,
                             out.data_ptr(), _stream_handle(stream)))
    return out


def tsenor_round(plan, W, N: int, M: int, sweeps: int, out=None, stream=None):
    """Rounding of a given fp32 plan into a mask (int32 words)."""
    import torch
    _check_2d_cuda(W, "W")
    _check_2d_cuda(plan, "plan")
    rows, cols = W.shape
    if plan.shape != W.shape or plan.dtype != torch.float32:
        raise ValueError("plan must be float32 with the shape of W")
    if out is None:
        out = torch.empty((rows, words_per_row(cols)), dtype=torch.int32, device=W.device)
    _check(lib().tsenor_round(plan.data_ptr(), W.data_ptr(), _dtype_code(W), rows, cols, N, M, sweeps,
                              out.data_ptr(), _stream_handle(stream)))
    return out


def tsenor_objective(W, mask, N: int, M: int, out=None, stream=None):
    """Per-block kept sum of |W| (fp64), NaN where a block row/column is not N:M."""
    import torch
    _check_2d_cuda(W, "W")
    rows, cols = W.shape
    if out is None:
        out = torch.empty(((rows // M) * (cols // M),), dtype=torch.float64, device=W.device)
    _check(lib().tsenor_objective(W.data_ptr(), _dtype_code(W), rows, cols, mask.data_ptr(), N, M,
                                  out.data_ptr(), _stream_handle(stream)))
    return out


class QuantizedMatrix(NamedTuple):
    """A matrix in 8 bits: e4m3 codes with one power-of-two scale per block of 128.

    values: torch.float8_e4m3fn (rows, cols), row stride a multiple of 16.
    scales: uint8 (ceil(cols/512), ceil(rows/128), 512), one byte per row and 128
    columns, for products that sum over the columns; scales_t: uint8
    (ceil(rows/512), ceil(cols/128), 512), for products that sum over the rows
    (the layout stands in include/tsenor.h).  Either may be None.
    """
    values: object
    scales: object = None
    scales_t: object = None

    @property
    def shape(self):
        return tuple(self.values.shape)


def scale_shape(rows: int, cols: int) -> tuple[int, int, int]:
    """Shape of ``scales`` of a rows x cols matrix (of ``scales_t``: with rows and cols exchanged)."""
    return (cols + 511) // 512, (rows + 127) // 128, 512


def _strided(t, name, types):
    """Row stride of a 2-D CUDA tensor whose rows are dense."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} must be {' or '.join(str(x) for x in types)}, got {t.dtype}")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have dense rows")
    if ld < cols:
        if rows > 1:
            raise ValueError(f"{name} must have rows that do not overlap")
        return cols
    return ld


def _dense(t, name, dtype, shape, device):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}")


def _mask_pointer(mask, rows, cols, device):
    import torch
    if mask is None:
        return None
    _dense(mask, "mask", torch.int32, (rows, words_per_row(cols)), device)
    return mask.data_ptr()


@contextlib.contextmanager
def _on(device, stream):
    """The device and the stream of a call: what it allocates belongs to that stream."""
    import torch
    if stream is not None and not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _launch(fn, device, *args):
    """fn(*args, stream) on the device's current stream."""
    import torch
    status = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if status:
        _check(status)


def _needs_guard(device, stream):
    import torch
    return stream is not None or torch.cuda.current_device() != device.index


def _new_codes(rows, cols, device):
    import torch
    return torch.empty_strided((rows, cols), ((cols + 15) // 16 * 16, 1), dtype=torch.float8_e4m3fn, device=device)


def _codes(t, name, device, shape=None):
    """(pointer, row stride) of a codes tensor."""
    import torch
    ld = _strided(t, name, (torch.float8_e4m3fn,))
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {(rows, cols)}")
    if rows <= 1 or cols == 0:
        ld = (cols + 15) // 16 * 16
    if ld % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name} must have rows that start on 16 bytes (a row stride that is a multiple of 16)")
    return t.data_ptr(), ld


def _new_scales(rows, cols, device):
    import torch
    k, t = (cols + 511) // 512, (rows + 127) // 128
    return torch.empty_strided((k, t, 512), (t * 512, 512, 1), dtype=torch.uint8, device=device)


def _new_row_values(rows, device):
    import torch
    return torch.empty_strided((rows,), (1,), dtype=torch.float32, device=device)


def _float_types():
    import torch
    return torch.bfloat16, torch.float32


def tsenor_quantize(X, block: str = "row", mask=None, out=None, stream=None):
    """X (bfloat16 or float32, dense rows) in 8 bits; returns a QuantizedMatrix.

    block: "row" (a scale per 128 entries of a row: ``scales``), "column" (per 128
    entries of a column: ``scales_t``) or "tile" (per 128 x 128 entries: both;
    weights, which both a layer's product and its transposed one read).
    mask: (rows, ceil(cols/32)) int32 words as tsenor_mask returns them; an entry
    whose bit is 0 counts as 0.  out: a QuantizedMatrix to write into.
    """
    import torch
    ldx = _strided(X, "X", _float_types())
    if block not in BLOCKS:
        raise ValueError(f"block must be one of {', '.join(BLOCKS)}, got {block!r}")
    if _needs_guard(X.device, stream):
        with _on(X.device, stream):
            return tsenor_quantize(X, block, mask, out)
    rows, cols = X.shape
    device = X.device
    mask_ptr = _mask_pointer(mask, rows, cols, device)
    if out is None:
        out = QuantizedMatrix(_new_codes(rows, cols, device),
                              _new_scales(rows, cols, device) if block != "column" else None,
                              _new_scales(cols, rows, device) if block != "row" else None)
        values, ldv = out.values.data_ptr(), (cols + 15) // 16 * 16
    else:
        values, ldv = _codes(out.values, "out.values", device, (rows, cols))
        if block != "column":
            _dense(out.scales, "out.scales", torch.uint8, scale_shape(rows, cols), device)
        if block != "row":
            _dense(out.scales_t, "out.scales_t", torch.uint8, scale_shape(cols, rows), device)
    _launch(lib().tsenor_quantize, device, X.data_ptr(), _dtype_code(X), rows, cols, ldx, BLOCKS[block], mask_ptr,
            values, ldv, out.scales.data_ptr() if block != "column" else None,
            out.scales_t.data_ptr() if block != "row" else None)
    return out


def tsenor_quantize_pair(X, stream=None):
    """(tsenor_quantize(X, "row"), tsenor_quantize(X, "column")) from one read of X."""
    ldx = _strided(X, "X", _float_types())
    if _needs_guard(X.device, stream):
        with _on(X.device, stream):
            return tsenor_quantize_pair(X)
    rows, cols = X.shape
    q = QuantizedMatrix(_new_codes(rows, cols, X.device), _new_scales(rows, cols, X.device), None)
    t = QuantizedMatrix(_new_codes(rows, cols, X.device), None, _new_scales(cols, rows, X.device))
    ldv = (cols + 15) // 16 * 16
    _launch(lib().tsenor_quantize_pair, X.device, X.data_ptr(), _dtype_code(X), rows, cols, ldx, q.values.data_ptr(),
            ldv, q.scales.data_ptr(), t.values.data_ptr(), ldv, t.scales_t.data_ptr())
    return q, t


def tsenor_dequantize(Q, dtype=None, out=None, stream=None):
    """What a QuantizedMatrix stands for, in bfloat16 or float32 (default); by ``scales`` where it has them."""
    import torch
    device = Q.values.device
    rows, cols = Q.shape
    ldv = _strided(Q.values, "Q.values", (torch.float8_e4m3fn,))
    if Q.scales is not None:
        _dense(Q.scales, "Q.scales", torch.uint8, scale_shape(rows, cols), device)
    elif Q.scales_t is not None:
        _dense(Q.scales_t, "Q.scales_t", torch.uint8, scale_shape(cols, rows), device)
    else:
        raise ValueError("Q has no scales")
    if _needs_guard(device, stream):
        with _on(device, stream):
            return tsenor_dequantize(Q, dtype, out)
    out, ldo = _output(out, rows, cols, dtype or torch.float32, device)
    scales = Q.scales if Q.scales is not None else Q.scales_t
    _launch(lib().tsenor_dequantize, device, Q.values.data_ptr(), rows, cols, ldv, scales.data_ptr(),
            int(Q.scales is None), out.data_ptr(), _dtype_code(out), ldo)
    return out


def _output(out, rows, cols, dtype, device):
    """(out, row stride): a given output checked, or a new one."""
    import torch
    if out is None:
        if dtype not in _float_types():
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
        return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device), cols
    ldo = _strided(out, "out", _float_types())
    if out.device != device:
        raise ValueError(f"out must be on {device}")
    if tuple(out.shape) != (rows, cols):
        raise ValueError(f"out must have shape {(rows, cols)}, got {tuple(out.shape)}")
    return out, ldo


def tsenor_matmul(A, B, form: str = "nt", mask=None, dtype=None, out=None, stream=None):
    """Product of two QuantizedMatrix operands, summed in fp32.

    form "nt": A (m, k) @ B (n, k).T by A.scales and B.scales;
    "nn": A (m, k) @ B (k, n) by A.scales and B.scales_t;
    "tn": A (k, m).T @ B (k, n) by A.scales_t and B.scales_t.
    mask: optional (m, ceil(n/32)) int32 words; entries whose bit is 0 are written
    as 0.  dtype: torch.bfloat16 (default) or torch.float32, that of ``out`` when it is given.
    """
    import torch
    if form not in FORMS:
        raise ValueError(f"form must be one of {', '.join(FORMS)}, got {form!r}")
    device = A.values.device
    if not A.values.is_cuda:
        raise ValueError("A must be on a CUDA device")
    if _needs_guard(device, stream):
        with _on(device, stream):
            return tsenor_matmul(A, B, form, mask, dtype, out)
    a, lda = _codes(A.values, "A.values", device)
    b, ldb = _codes(B.values, "B.values", device)
    (ra, ca), (rb, cb) = A.values.shape, B.values.shape
    m, k = (ca, ra) if form == "tn" else (ra, ca)
    n, kb = (rb, cb) if form == "nt" else (cb, rb)
    if k != kb:
        raise ValueError(f"the operands sum over {k} and {kb} entries")
    sa, sb = (A.scales_t if form == "tn" else A.scales), (B.scales if form == "nt" else B.scales_t)
    if sa is None or sb is None:
        raise ValueError(f'form "{form}" needs {"A.scales_t" if form == "tn" else "A.scales"} and '
                         f'{"B.scales" if form == "nt" else "B.scales_t"}')
    _dense(sa, "A's scales", torch.uint8, scale_shape(m, k), device)
    _dense(sb, "B's scales", torch.uint8, scale_shape(n, k), device)
    mask_ptr = _mask_pointer(mask, m, n, device)
    if dtype is not None and out is not None and out.dtype != dtype:
        raise TypeError(f"out is {out.dtype}, dtype {dtype}")
    out, ldo = _output(out, m, n, dtype or torch.bfloat16, device)
    _launch(lib().tsenor_matmul, device, FORMS[form], a, lda, sa.data_ptr(), b, ldb, sb.data_ptr(), m, n, k, mask_ptr,
            out.data_ptr(), _dtype_code(out), ldo)
    return out


def _distill_args(logits, index, top_logits, temperature, teacher_lse):
    """The arguments the distillation calls share, checked."""
    import torch
    ld = _strided(logits, "logits", _float_types())
    rows, vocab = logits.shape
    if index.dim() != 2 or index.shape[0] != rows:
        raise ValueError(f"index must have shape ({rows}, top), got {tuple(index.shape)}")
    top = index.shape[1]
    _dense(index, "index", torch.int32, (rows, top), logits.device)
    _dense(top_logits, "top_logits", torch.float32, (rows, top), logits.device)
    if teacher_lse is not None:
        _dense(teacher_lse, "teacher_lse", torch.float32, (rows,), logits.device)
    return (logits.data_ptr(), _dtype_code(logits), rows, vocab, ld, index.data_ptr(), top_logits.data_ptr(), top,
            teacher_lse.data_ptr() if teacher_lse is not None else None, float(temperature))


def _distill_grad_args(logits, weight, grad):
    import torch
    rows, vocab = logits.shape
    if weight is not None:
        _dense(weight, "weight", torch.float32, (rows,), logits.device)
    if grad is None:
        grad, ldg = torch.empty_strided((rows, vocab), (vocab, 1), dtype=logits.dtype, device=logits.device), vocab
    else:
        ldg = _strided(grad, "grad", (logits.dtype,))
        if grad.shape != logits.shape or grad.device != logits.device:
            raise ValueError(f"grad must have shape {tuple(logits.shape)} on {logits.device}")
    return grad, (weight.data_ptr() if weight is not None else None), ldg


def tsenor_distill_loss(logits, index, top_logits, temperature: float = 1.0, teacher_lse=None, stream=None):
    """Distillation loss of each row from the teacher's top logits; returns (loss, lse), fp32 (rows,).

    logits: (rows, vocab) bfloat16 or float32 of the student.  index: (rows, top)
    int32, negative where a row has fewer entries; top_logits: (rows, top) float32.
    loss = T^2 sum_j p_j (log p_j - log softmax(logits / T)[index_j]) with p the
    softmax of top_logits / T over the row's entries, or, with teacher_lse (rows,)
    float32, exp(top_logits / T - teacher_lse).  lse is what tsenor_distill_grad takes.
    """
    if logits.is_cuda and _needs_guard(logits.device, stream):
        with _on(logits.device, stream):
            return tsenor_distill_loss(logits, index, top_logits, temperature, teacher_lse)
    args = _distill_args(logits, index, top_logits, temperature, teacher_lse)
    loss, lse = _new_row_values(logits.shape[0], logits.device), _new_row_values(logits.shape[0], logits.device)
    _launch(lib().tsenor_distill_loss, logits.device, *args, loss.data_ptr(), lse.data_ptr())
    return loss, lse


def tsenor_distill_step(logits, index, top_logits, temperature: float = 1.0, teacher_lse=None, weight=None, grad=None,
                        stream=None):
    """Loss of each row and weight * d loss / d logits from one read of the logits; returns (loss, grad).

    weight: (rows,) float32, default 1: the upstream gradient of each row's loss.
    grad: optional output like the logits, which may be the logits themselves.
    """
    if logits.is_cuda and _needs_guard(logits.device, stream):
        with _on(logits.device, stream):
            return tsenor_distill_step(logits, index, top_logits, temperature, teacher_lse, weight, grad)
    args = _distill_args(logits, index, top_logits, temperature, teacher_lse)
    grad, weight_ptr, ldg = _distill_grad_args(logits, weight, grad)
    loss = _new_row_values(logits.shape[0], logits.device)
    _launch(lib().tsenor_distill_step, logits.device, *args, weight_ptr, loss.data_ptr(), grad.data_ptr(), ldg)
    return loss, grad


def tsenor_distill_grad(logits, index, top_logits, lse, temperature: float = 1.0, teacher_lse=None, weight=None,
                        grad=None, stream=None):
    """weight * d loss / d logits, by the lse that tsenor_distill_loss gave for these logits; returns grad."""
    import torch
    if logits.is_cuda and _needs_guard(logits.device, stream):
        with _on(logits.device, stream):
            return tsenor_distill_grad(logits, index, top_logits, lse, temperature, teacher_lse, weight, grad)
    args = _distill_args(logits, index, top_logits, temperature, teacher_lse)
    _dense(lse, "lse", torch.float32, (logits.shape[0],), logits.device)
    grad, weight_ptr, ldg = _distill_grad_args(logits, weight, grad)
    _launch(lib().tsenor_distill_grad, logits.device, *args, lse.data_ptr(), weight_ptr, grad.data_ptr(), ldg)
    return grad


def tsenor_error_count(stream=None) -> int:
    """Blocks (and rows of the distillation calls) that failed since the previous call (synchronises the stream).

    The C call reports a nonzero count with TSENOR_ERR_DEVICE; here the count
    itself is the result, so that status is not raised.
    """
    n = C.c_int64(0)
    status = lib().tsenor_error_count(_stream_handle(stream), C.byref(n))
    if status != -5:
        _check(status)
    return int(n.value)


__all__ = ["tsenor_mask", "tsenor_mask_host", "tsenor_mask_scores", "tsenor_mask_noalloc", "tsenor_mask_safeguard", "tsenor_mask_padded", "tsenor_mask_warm",
           "tsenor_plan", "tsenor_plan_warm", "tsenor_round", "tsenor_objective", "tsenor_error_count",
           "QuantizedMatrix", "scale_shape", "tsenor_quantize", "tsenor_quantize_pair", "tsenor_dequantize",
           "tsenor_matmul", "tsenor_distill_loss", "tsenor_distill_step", "tsenor_distill_grad",
           "TsenorError", "lib", "words_per_row", "EXPORTS", "LIB_PATH"]
