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


# Helpers of the calls below.  They are called for every launch of a decoded token, so they read each
# attribute of a tensor once and import nothing that their caller has.

def _rows(t, name, types):
    """(rows, cols, row stride) of a 2-D CUDA tensor whose rows are dense."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} must be {' or '.join(str(x) for x in types)}, got {t.dtype}")
    (rows, cols), (ld, step) = t.shape, t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have dense rows")
    if ld < cols:
        if rows > 1:
            raise ValueError(f"{name} must have rows that do not overlap")
        ld = cols
    return rows, cols, ld


def _dense(t, name, dtype, shape, device):
    """Pointer of a contiguous tensor of this type, shape and device."""
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}")
    return t.data_ptr()


def _codes(t, name, types, device):
    """(rows, cols, row stride, pointer) of a codes tensor."""
    rows, cols, ld = _rows(t, name, types)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if rows <= 1 or cols == 0:
        ld = (cols + 15) // 16 * 16
    ptr = t.data_ptr()
    if ld % 16 or ptr % 16:
        raise ValueError(f"{name} must have rows that start on 16 bytes (a row stride that is a multiple of 16)")
    return rows, cols, ld, ptr


@contextlib.contextmanager
def _on(device, stream):
    """The device and the stream of a call: what it allocates belongs to that stream."""
    import torch
    if stream is not None and not hasattr(stream, "cuda_stream"):
        handle = int(stream)                    # ExternalStream takes 0 for a new stream of its own
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    elif getattr(stream, "device", device) != device:
        raise ValueError(f"stream must be on {device}, is on {stream.device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _new_codes(torch, rows, cols, device):
    return torch.empty_strided((rows, cols), ((cols + 15) // 16 * 16, 1), dtype=torch.float8_e4m3fn, device=device)


def _new_scales(torch, rows, cols, device):
    k, t = (cols + 511) // 512, (rows + 127) // 128
    return torch.empty_strided((k, t, 512), (t * 512, 512, 1), dtype=torch.uint8, device=device)


def tsenor_quantize(X, block: str = "row", mask=None, out=None, stream=None):
    """X (bfloat16 or float32, dense rows) in 8 bits; returns a QuantizedMatrix.

    block: "row" (a scale per 128 entries of a row: ``scales``), "column" (per 128
    entries of a column: ``scales_t``) or "tile" (per 128 x 128 entries: both;
    weights, which both a layer's product and its transposed one read).
    mask: (rows, ceil(cols/32)) int32 words as tsenor_mask returns them; an entry
    whose bit is 0 counts as 0.  out: a QuantizedMatrix to write into.
    """
    import torch
    rows, cols, ldx = _rows(X, "X", (torch.bfloat16, torch.float32))
    code = BLOCKS.get(block)
    if code is None:
        raise ValueError(f"block must be one of {', '.join(BLOCKS)}, got {block!r}")
    device = X.device
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream):
            return tsenor_quantize(X, block, mask, out)
    mask_ptr = None
    if mask is not None:
        mask_ptr = _dense(mask, "mask", torch.int32, (rows, words_per_row(cols)), device)
    along = down = None
    if out is None:
        values, ldv = _new_codes(torch, rows, cols, device), (cols + 15) // 16 * 16
        scales = _new_scales(torch, rows, cols, device) if code != 1 else None
        scales_t = _new_scales(torch, cols, rows, device) if code != 0 else None
        out = QuantizedMatrix(values, scales, scales_t)
        ptr = values.data_ptr()
        along = scales.data_ptr() if code != 1 else None
        down = scales_t.data_ptr() if code != 0 else None
    else:
        orows, ocols, ldv, ptr = _codes(out.values, "out.values", (torch.float8_e4m3fn,), device)
        if (orows, ocols) != (rows, cols):
            raise ValueError(f"out.values must have shape {(rows, cols)}, got {(orows, ocols)}")
        if (code != 1 and out.scales is None) or (code != 0 and out.scales_t is None):
            raise ValueError(f'out lacks the scales of block "{block}"')
        if code != 1:
            along = _dense(out.scales, "out.scales", torch.uint8, scale_shape(rows, cols), device)
        if code != 0:
            down = _dense(out.scales_t, "out.scales_t", torch.uint8, scale_shape(cols, rows), device)
    status = lib().tsenor_quantize(X.data_ptr(), X.dtype == torch.bfloat16, rows, cols, ldx, code, mask_ptr, ptr, ldv, along,
                                   down, torch._C._cuda_getCurrentRawStream(device.index))
    if status:
        _check(status)
    return out


def tsenor_quantize_pair(X, stream=None):
    """(tsenor_quantize(X, "row"), tsenor_quantize(X, "column")) from one read of X."""
    import torch
    rows, cols, ldx = _rows(X, "X", (torch.bfloat16, torch.float32))
    device = X.device
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream):
            return tsenor_quantize_pair(X)
    q = QuantizedMatrix(_new_codes(torch, rows, cols, device), _new_scales(torch, rows, cols, device), None)
    t = QuantizedMatrix(_new_codes(torch, rows, cols, device), None, _new_scales(torch, cols, rows, device))
    ldv = (cols + 15) // 16 * 16
    status = lib().tsenor_quantize_pair(X.data_ptr(), X.dtype == torch.bfloat16, rows, cols, ldx, q[0].data_ptr(), ldv,
                                        q[1].data_ptr(), t[0].data_ptr(), ldv, t[2].data_ptr(),
                                        torch._C._cuda_getCurrentRawStream(device.index))
    if status:
        _check(status)
    return q, t


def tsenor_dequantize(Q, dtype=None, out=None, stream=None):
    """What a QuantizedMatrix stands for, in bfloat16 or float32 (default); by ``scales`` where it has them."""
    import torch
    device = Q.values.device
    rows, cols, ldv = _rows(Q.values, "Q.values", (torch.float8_e4m3fn,))
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream):
            return tsenor_dequantize(Q, dtype, out)
    if Q.scales is not None:
        scales = _dense(Q.scales, "Q.scales", torch.uint8, scale_shape(rows, cols), device)
    elif Q.scales_t is not None:
        scales = _dense(Q.scales_t, "Q.scales_t", torch.uint8, scale_shape(cols, rows), device)
    else:
        raise ValueError("Q has no scales")
    out, ldo = _output(torch, out, rows, cols, dtype, torch.float32, device)
    status = lib().tsenor_dequantize(Q.values.data_ptr(), rows, cols, ldv, scales, Q.scales is None, out.data_ptr(),
                                     out.dtype == torch.bfloat16, ldo, torch._C._cuda_getCurrentRawStream(device.index))
    if status:
        _check(status)
    return out


def _output(torch, out, rows, cols, dtype, default, device):
    """(out, row stride): a given output checked, or a new one."""
    if out is None:
        dtype = dtype or default
        if dtype != torch.bfloat16 and dtype != torch.float32:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
        return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device), cols
    orows, ocols, ldo = _rows(out, "out", (torch.bfloat16, torch.float32))
    if out.device != device:
        raise ValueError(f"out must be on {device}")
    if (orows, ocols) != (rows, cols):
        raise ValueError(f"out must have shape {(rows, cols)}, got {(orows, ocols)}")
    if dtype is not None and out.dtype != dtype:
        raise TypeError(f"out is {out.dtype}, dtype {dtype}")
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
    code = FORMS.get(form)
    if code is None:
        raise ValueError(f"form must be one of {', '.join(FORMS)}, got {form!r}")
    av, bv = A[0], B[0]
    device = av.device
    types = (torch.float8_e4m3fn,)
    ra, ca, lda, a = _codes(av, "A.values", types, device)
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream):
            return tsenor_matmul(A, B, form, mask, dtype, out)
    rb, cb, ldb, b = _codes(bv, "B.values", types, device)
    m, k, sa = (ca, ra, A[2]) if code == 2 else (ra, ca, A[1])
    n, kb, sb = (rb, cb, B[1]) if code == 0 else (cb, rb, B[2])
    if k != kb:
        raise ValueError(f"the operands sum over {k} and {kb} entries")
    if sa is None or sb is None:
        raise ValueError(f'form "{form}" needs {"A.scales_t" if code == 2 else "A.scales"} and '
                         f'{"B.scales" if code == 0 else "B.scales_t"}')
    k4 = (k + 511) // 512
    sa = _dense(sa, "A's scales", torch.uint8, (k4, (m + 127) // 128, 512), device)
    sb = _dense(sb, "B's scales", torch.uint8, (k4, (n + 127) // 128, 512), device)
    mask_ptr = None
    if mask is not None:
        mask_ptr = _dense(mask, "mask", torch.int32, (m, words_per_row(n)), device)
    out, ldo = _output(torch, out, m, n, dtype, torch.bfloat16, device)
    status = lib().tsenor_matmul(code, a, lda, sa, b, ldb, sb, m, n, k, mask_ptr, out.data_ptr(), out.dtype == torch.bfloat16,
                                 ldo, torch._C._cuda_getCurrentRawStream(device.index))
    if status:
        _check(status)
    return out


def _distill_args(torch, logits, index, top_logits, temperature, teacher_lse):
    """The arguments the distillation calls share, checked."""
    rows, vocab, ld = _rows(logits, "logits", (torch.bfloat16, torch.float32))
    device = logits.device
    if index.dim() != 2:
        raise ValueError(f"index must have shape ({rows}, top), got {tuple(index.shape)}")
    top = index.shape[1]
    return (logits.data_ptr(), logits.dtype == torch.bfloat16, rows, vocab, ld,
            _dense(index, "index", torch.int32, (rows, top), device),
            _dense(top_logits, "top_logits", torch.float32, (rows, top), device), top,
            None if teacher_lse is None else _dense(teacher_lse, "teacher_lse", torch.float32, (rows,), device), temperature)


def _distill_grad_args(torch, logits, weight, grad):
    """(grad, its row stride, pointer of weight)."""
    (rows, vocab), device = logits.shape, logits.device
    weight = None if weight is None else _dense(weight, "weight", torch.float32, (rows,), device)
    if grad is None:
        return torch.empty_strided((rows, vocab), (vocab, 1), dtype=logits.dtype, device=device), vocab, weight
    grows, gcols, ldg = _rows(grad, "grad", (logits.dtype,))
    if (grows, gcols) != (rows, vocab) or grad.device != device:
        raise ValueError(f"grad must have shape {(rows, vocab)} on {device}")
    return grad, ldg, weight


def tsenor_distill_loss(logits, index, top_logits, temperature: float = 1.0, teacher_lse=None, stream=None):
    """Distillation loss of each row from the teacher's top logits; returns (loss, lse), fp32 (rows,).

    logits: (rows, vocab) bfloat16 or float32 of the student.  index: (rows, top)
    int32, negative where a row has fewer entries; top_logits: (rows, top) float32.
    loss = T^2 sum_j p_j (log p_j - log softmax(logits / T)[index_j]) with p the
    softmax of top_logits / T over the row's entries, or, with teacher_lse (rows,)
    float32, exp(top_logits / T - teacher_lse).  lse is what tsenor_distill_grad takes.
    """
    import torch
    args = _distill_args(torch, logits, index, top_logits, temperature, teacher_lse)
    device = logits.device
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream):
            return tsenor_distill_loss(logits, index, top_logits, temperature, teacher_lse)
    rows = args[2]
    loss = torch.empty_strided((rows,), (1,), dtype=torch.float32, device=device)
    lse = torch.empty_strided((rows,), (1,), dtype=torch.float32, device=device)
    status = lib().tsenor_distill_loss(*args, loss.data_ptr(), lse.data_ptr(),
                                       torch._C._cuda_getCurrentRawStream(device.index))
    if status:
        _check(status)
    return loss, lse


def tsenor_distill_step(logits, index, top_logits, temperature: float = 1.0, teacher_lse=None, weight=None, grad=None,
                        stream=None):
    """Loss of each row and weight * d loss / d logits in one call; returns (loss, grad).

    weight: (rows,) float32, default 1: the upstream gradient of each row's loss.
    grad: optional output like the logits, which may be the logits themselves.
    """
    import torch
    args = _distill_args(torch, logits, index, top_logits, temperature, teacher_lse)
    device = logits.device
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream):
            return tsenor_distill_step(logits, index, top_logits, temperature, teacher_lse, weight, grad)
    grad, ldg, weight_ptr = _distill_grad_args(torch, logits, weight, grad)
    loss = torch.empty_strided((args[2],), (1,), dtype=torch.float32, device=device)
    status = lib().tsenor_distill_step(*args, weight_ptr, loss.data_ptr(), grad.data_ptr(), ldg,
                                       torch._C._cuda_getCurrentRawStream(device.index))
    if status:
        _check(status)
    return loss, grad


def tsenor_distill_grad(logits, index, top_logits, lse, temperature: float = 1.0, teacher_lse=None, weight=None,
                        grad=None, stream=None):
    """weight * d loss / d logits, by the lse that tsenor_distill_loss gave for these logits; returns grad.

    Rows of |lse| above 64 (low temperatures, logits far from 0) are read once more: one float32 says too little there.
    """
    import torch
    args = _distill_args(torch, logits, index, top_logits, temperature, teacher_lse)
    device = logits.device
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream):
            return tsenor_distill_grad(logits, index, top_logits, lse, temperature, teacher_lse, weight, grad)
    lse_ptr = _dense(lse, "lse", torch.float32, (args[2],), device)
    grad, ldg, weight_ptr = _distill_grad_args(torch, logits, weight, grad)
    status = lib().tsenor_distill_grad(*args, lse_ptr, weight_ptr, grad.data_ptr(), ldg,
                                       torch._C._cuda_getCurrentRawStream(device.index))
    if status:
        _check(status)
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
