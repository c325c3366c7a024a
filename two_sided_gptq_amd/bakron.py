"""Thin ctypes binding of libbakron.so (declared in include/bakron.h).

Argument marshalling only: tensors are allocated with torch on the current
device, their pointers and torch's current HIP stream are passed to the C ABI,
and every step of the computation runs in the library's HIP kernels.  There
is no fallback: without the built library or a GPU the calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbakron.so")

Q_SYM, Q_ASYM, Q_UNIT = 0, 1, 2
ORDER_AUTO, ORDER_LA_FIRST, ORDER_LB_FIRST = 0, 1, 2
FLAG_PHASE_TIMING = 4
FLAG_NO_GRAPH = 8
FLAG_MSE_SCALE = 16
FLAG_SPLIT_COLS = 32
FLAG_SPLIT_ROWS = 64
DEV_NONFINITE, DEV_NOT_PD = 1, 2
DEV_BAD_INDEX = 8
T_F32, T_BF16, T_F16 = 0, 1, 2
SCALE_ROW, SCALE_BLOCK = 0, 1

EXPORTS = (
    "bakron_hessian_workspace_size", "bakron_hessian",
    "bakron_factor_workspace_size", "bakron_factor",
    "bakron_quantize_workspace_size", "bakron_quantize", "bakron_quantize_noalloc",
    "bakron_quantize_antidiag_workspace_size", "bakron_quantize_antidiag",
    "bakron_schedule_info", "bakron_schedule_plan", "bakron_last_phase_ms",
    "bakron_fp8_quantize", "bakron_fp8_from_codes",
    "bakron_fp8_matmul_workspace_size", "bakron_fp8_matmul",
    "bakron_grouped_matmul_workspace_size", "bakron_grouped_matmul", "bakron_grouped_matmul_grad_x",
    "bakron_grouped_matmul_grad_w",
    "bakron_token_logprobs_workspace_size", "bakron_token_logprobs", "bakron_token_logprobs_grad",
    "bakron_group_sort_workspace_size", "bakron_group_sort", "bakron_group_gather", "bakron_group_gather_fp8",
    "bakron_group_combine", "bakron_group_combine_grad",
    "bakron_adapter_matmul_workspace_size", "bakron_adapter_matmul",
    "bakron_adapter_matmul_grad_workspace_size", "bakron_adapter_matmul_grad",
    "bakron_verify_drafts_workspace_size", "bakron_verify_drafts",
    "bakron_status_string", "bakron_last_error",
)

_lib = None


class BakronError(RuntimeError):
    pass


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libbakron.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise BakronError(f"{path} is missing; build it with `python -m two_sided_gptq_amd.build`")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ, F, D = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_float, ctypes.c_double)
    lib.bakron_hessian_workspace_size.argtypes = [I64, I64]
    lib.bakron_hessian_workspace_size.restype = SZ
    lib.bakron_hessian.argtypes = [P, I64, I64, F, P, P, SZ, P]
    lib.bakron_hessian.restype = I32
    lib.bakron_factor_workspace_size.argtypes = [I64]
    lib.bakron_factor_workspace_size.restype = SZ
    lib.bakron_factor.argtypes = [P, I64, P, P, P, SZ, P]
    lib.bakron_factor.restype = I32
    lib.bakron_quantize_workspace_size.argtypes = [I64, I64, I32, I32]
    lib.bakron_quantize_workspace_size.restype = SZ
    lib.bakron_quantize.argtypes = [P, I64, I64, P, P, I32, I32, P, P, P, P, P, P, P, I32, P, SZ, P]
    lib.bakron_quantize.restype = I32
    lib.bakron_quantize_noalloc.argtypes = [P, I64, I64, P, P, I32, I32, P, P, P, P, P, P, P, I32, P]
    lib.bakron_quantize_noalloc.restype = I32
    lib.bakron_quantize_antidiag_workspace_size.argtypes = [I64, I64, I32, I32]
    lib.bakron_quantize_antidiag_workspace_size.restype = SZ
    lib.bakron_quantize_antidiag.argtypes = [P, I64, I64, P, P, I32, I32, P, P, P, P, P, P, P, SZ, P]
    lib.bakron_quantize_antidiag.restype = I32
    lib.bakron_schedule_info.argtypes = [I64, I64, I32, ctypes.POINTER(D)]
    lib.bakron_schedule_info.restype = I32
    lib.bakron_schedule_plan.argtypes = [I64, I64, I32, ctypes.POINTER(I32), I64,
                                         ctypes.POINTER(I64)]
    lib.bakron_schedule_plan.restype = I32
    lib.bakron_last_phase_ms.argtypes = [ctypes.POINTER(D)]
    lib.bakron_last_phase_ms.restype = I32
    lib.bakron_fp8_quantize.argtypes = [P, I32, I64, I64, I64, I32, P, I64, P, P, P]
    lib.bakron_fp8_quantize.restype = I32
    lib.bakron_fp8_from_codes.argtypes = [P, P, I64, I64, I32, I32, P, I64, P]
    lib.bakron_fp8_from_codes.restype = I32
    lib.bakron_fp8_matmul_workspace_size.argtypes = [I64, I64, I64, I32]
    lib.bakron_fp8_matmul_workspace_size.restype = SZ
    lib.bakron_fp8_matmul.argtypes = [P, I64, P, P, I64, P, I32, I64, I64, I64, I32, P, P, I32, I64, P, P,
                                      SZ, P]
    lib.bakron_fp8_matmul.restype = I32
    lib.bakron_grouped_matmul_workspace_size.argtypes = [I64, I64, I64, I32]
    lib.bakron_grouped_matmul_workspace_size.restype = SZ
    for f in (lib.bakron_grouped_matmul, lib.bakron_grouped_matmul_grad_x, lib.bakron_grouped_matmul_grad_w):
        f.argtypes = [P, I32, I64, P, I64, I64, I64, I64, I32, P, P, I32, I64, P, P, SZ, P]
        f.restype = I32
    lib.bakron_token_logprobs_workspace_size.argtypes = [I64, I64, I32]
    lib.bakron_token_logprobs_workspace_size.restype = SZ
    lib.bakron_token_logprobs.argtypes = [P, I32, I64, I64, I64, P, I32, P, P, P, P, P, P, P, SZ, P]
    lib.bakron_token_logprobs.restype = I32
    lib.bakron_token_logprobs_grad.argtypes = [P, I32, I64, I64, I64, P, P, P, P, P, P, I64, P, P]
    lib.bakron_token_logprobs_grad.restype = I32
    lib.bakron_group_sort_workspace_size.argtypes = [I64, I32]
    lib.bakron_group_sort_workspace_size.restype = SZ
    lib.bakron_group_sort.argtypes = [P, I32, I64, I32, P, P, P, P, P, SZ, P]
    lib.bakron_group_sort.restype = I32
    lib.bakron_group_gather.argtypes = [P, I32, I64, I32, I64, I64, P, I32, P, P, I64, P, P]
    lib.bakron_group_gather.restype = I32
    lib.bakron_group_gather_fp8.argtypes = [P, I32, I64, I32, I64, I64, P, I32, P, P, I64, P, P, P]
    lib.bakron_group_gather_fp8.restype = I32
    lib.bakron_group_combine.argtypes = [P, I32, I64, I32, I64, I64, P, I32, P, P, P, I64, P, P]
    lib.bakron_group_combine.restype = I32
    lib.bakron_group_combine_grad.argtypes = [P, I64, P, I32, I64, I32, I64, I64, P, I32, P, P, P, I64, P, P, P]
    lib.bakron_group_combine_grad.restype = I32
    lib.bakron_adapter_matmul_workspace_size.argtypes = [I64, I64, I64, I32, I32]
    lib.bakron_adapter_matmul_workspace_size.restype = SZ
    lib.bakron_adapter_matmul.argtypes = [P, I32, I64, P, P, I64, I64, I64, I32, I32, P, P, P, P, I64, P, I32, I64, P, P,
                                          SZ, P]
    lib.bakron_adapter_matmul.restype = I32
    lib.bakron_adapter_matmul_grad_workspace_size.argtypes = [I64, I64, I64, I32, I32]
    lib.bakron_adapter_matmul_grad_workspace_size.restype = SZ
    lib.bakron_adapter_matmul_grad.argtypes = [P, I64, P, I32, I64, P, P, I64, I64, I64, I32, I32, P, P, P, P, I64, P, I32,
                                               I64, P, P, I32, P, P, SZ, P]
    lib.bakron_adapter_matmul_grad.restype = I32
    lib.bakron_verify_drafts_workspace_size.argtypes = [I64, I32, I64]
    lib.bakron_verify_drafts_workspace_size.restype = SZ
    lib.bakron_verify_drafts.argtypes = [P, I64, P, I64, I32, I64, I32, I64, P, P, P, P, P, P, P, SZ, P]
    lib.bakron_verify_drafts.restype = I32
    lib.bakron_status_string.argtypes = [I32]
    lib.bakron_status_string.restype = ctypes.c_char_p
    lib.bakron_last_error.argtypes = []
    lib.bakron_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int, what: str) -> None:
    if rc != 0:
        lib = load()
        raise BakronError(f"{what}: {lib.bakron_status_string(rc).decode()} "
                          f"({lib.bakron_last_error().decode()})")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _f32_dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()):
        raise BakronError(f"{name} must be a contiguous float32 GPU tensor")
    return t


def _workspace(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def hessian(X: torch.Tensor, damp_rel: float, stream=None) -> torch.Tensor:
    """H = X^T X / N + damp_rel * mean(diag) * I (bakron_hessian)."""
    lib = load()
    X = _f32_dev(X, "X")
    N, d = X.shape
    H = torch.empty((d, d), dtype=torch.float32, device=X.device)
    ws = _workspace(lib.bakron_hessian_workspace_size(N, d), X.device)
    _check(lib.bakron_hessian(_ptr(X), N, d, float(damp_rel), _ptr(H), _ptr(ws), ws.numel(),
                              _stream(stream)), "bakron_hessian")
    return H


def factor(H: torch.Tensor, dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """L with L L^T = H^-1, lower (bakron_factor)."""
    lib = load()
    H = _f32_dev(H, "H")
    d = H.shape[0]
    L = torch.empty((d, d), dtype=torch.float32, device=H.device)
    ws = _workspace(lib.bakron_factor_workspace_size(d), H.device)
    _check(lib.bakron_factor(_ptr(H), d, _ptr(L), _ptr(dev_status), _ptr(ws), ws.numel(),
                             _stream(stream)), "bakron_factor")
    return L


def quantize_workspace_size(m: int, n: int, kind: int, bits: int) -> int:
    return int(load().bakron_quantize_workspace_size(m, n, kind, bits))


def quantize(W, LA, LB, kind=Q_SYM, bits=4, order=ORDER_AUTO, want_V=True, want_E=False,
             want_sum=False, dev_status=None, timing=False, graph=True, workspace=None, out=None,
             stream=None, mse=False, split=None):
    """Run bakron_quantize.  Returns a dict with codes (int8), scales, zeros
    (None unless asymmetric), V, E, sum_e2 (device tensors or None).  split:
    None, "cols" or "rows" (the hybrid schedule, BAKRON_FLAG_SPLIT_*)."""
    lib = load()
    W = _f32_dev(W, "W")
    LA = _f32_dev(LA, "LA")
    LB = _f32_dev(LB, "LB")
    m, n = W.shape
    dev = W.device
    if out is None:
        out = dict(
            codes=torch.empty((m, n), dtype=torch.int8, device=dev),
            scales=torch.empty(m, dtype=torch.float32, device=dev),
            zeros=torch.empty(m, dtype=torch.float32, device=dev) if kind == Q_ASYM else None,
            V=torch.empty((m, n), dtype=torch.float32, device=dev) if want_V else None,
            E=torch.empty((m, n), dtype=torch.float32, device=dev) if want_E else None,
            sum_e2=torch.empty(1, dtype=torch.float64, device=dev) if want_sum else None,
        )
    if workspace is None:
        workspace = _workspace(quantize_workspace_size(m, n, kind, bits), dev)
    if split not in (None, "cols", "rows"):
        raise ValueError(f"split must be None, 'cols' or 'rows', not {split!r}")
    flags = (int(order) | (FLAG_PHASE_TIMING if timing else 0) | (0 if graph else FLAG_NO_GRAPH) |
             (FLAG_MSE_SCALE if mse else 0) | (FLAG_SPLIT_COLS if split == "cols" else 0) |
             (FLAG_SPLIT_ROWS if split == "rows" else 0))
    rc = lib.bakron_quantize(_ptr(W), m, n, _ptr(LA), _ptr(LB), kind, bits, _ptr(out["codes"]),
                             _ptr(out["scales"]), _ptr(out["zeros"]), _ptr(out["V"]),
                             _ptr(out["E"]), _ptr(out["sum_e2"]), _ptr(dev_status), flags,
                             _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "bakron_quantize")
    return out


NOALLOC_SCRATCH_BYTES = 256 << 20  # BAKRON_NOALLOC_SCRATCH_BYTES


def quantize_noalloc(W, LA, LB, kind=Q_SYM, bits=4, order=ORDER_AUTO, want_V=True, want_E=False,
                     want_sum=False, dev_status=None, out=None, stream=None, mse=False, split=None):
    """Run bakron_quantize_noalloc (no workspace: the library's fixed scratch
    array; the plan in order on one stream).  Outputs as for quantize(); pass
    ``out`` to reuse preallocated output tensors."""
    lib = load()
    W = _f32_dev(W, "W")
    LA = _f32_dev(LA, "LA")
    LB = _f32_dev(LB, "LB")
    m, n = W.shape
    dev = W.device
    if out is None:
        out = dict(
            codes=torch.empty((m, n), dtype=torch.int8, device=dev),
            scales=torch.empty(m, dtype=torch.float32, device=dev),
            zeros=torch.empty(m, dtype=torch.float32, device=dev) if kind == Q_ASYM else None,
            V=torch.empty((m, n), dtype=torch.float32, device=dev) if want_V else None,
            E=torch.empty((m, n), dtype=torch.float32, device=dev) if want_E else None,
            sum_e2=torch.empty(1, dtype=torch.float64, device=dev) if want_sum else None,
        )
    if split not in (None, "cols", "rows"):
        raise ValueError(f"split must be None, 'cols' or 'rows', not {split!r}")
    flags = (int(order) | (FLAG_MSE_SCALE if mse else 0) | (FLAG_SPLIT_COLS if split == "cols" else 0) |
             (FLAG_SPLIT_ROWS if split == "rows" else 0))
    rc = lib.bakron_quantize_noalloc(_ptr(W), m, n, _ptr(LA), _ptr(LB), kind, bits, _ptr(out["codes"]),
                                     _ptr(out["scales"]), _ptr(out["zeros"]), _ptr(out["V"]),
                                     _ptr(out["E"]), _ptr(out["sum_e2"]), _ptr(dev_status), flags,
                                     _stream(stream))
    _check(rc, "bakron_quantize_noalloc")
    return out


def quantize_antidiag(W, LA, LB, kind=Q_SYM, bits=4, want_V=True, want_E=False, dev_status=None,
                      stream=None):
    """Run bakron_quantize_antidiag (BaKron-antidiagonal).  Returns a dict with
    codes, scales, zeros (None unless asymmetric), V, E (device tensors or None)."""
    lib = load()
    W = _f32_dev(W, "W")
    LA = _f32_dev(LA, "LA")
    LB = _f32_dev(LB, "LB")
    m, n = W.shape
    dev = W.device
    out = dict(
        codes=torch.empty((m, n), dtype=torch.int8, device=dev),
        scales=torch.empty(m, dtype=torch.float32, device=dev),
        zeros=torch.empty(m, dtype=torch.float32, device=dev) if kind == Q_ASYM else None,
        V=torch.empty((m, n), dtype=torch.float32, device=dev) if want_V else None,
        E=torch.empty((m, n), dtype=torch.float32, device=dev) if want_E else None,
    )
    size = int(lib.bakron_quantize_antidiag_workspace_size(m, n, kind, bits))
    workspace = _workspace(size, dev)
    rc = lib.bakron_quantize_antidiag(_ptr(W), m, n, _ptr(LA), _ptr(LB), kind, bits, _ptr(out["codes"]),
                                      _ptr(out["scales"]), _ptr(out["zeros"]), _ptr(out["V"]),
                                      _ptr(out["E"]), _ptr(dev_status), _ptr(workspace),
                                      workspace.numel(), _stream(stream))
    _check(rc, "bakron_quantize_antidiag")
    return out


SCHEDULE_KEYS = ("tile", "leaf_launches", "band_launches", "leaf_steps", "order",
                 "alg_band_flops", "exec_band_flops", "F", "leaf_flops", "depth",
                 "useful_band_flops", "pull_flops", "pull_leaves", "side_launches",
                 "side_useful_flops")


def schedule_info(m: int, n: int, order: int = ORDER_AUTO) -> dict:
    lib = load()
    buf = (ctypes.c_double * len(SCHEDULE_KEYS))()
    _check(lib.bakron_schedule_info(m, n, order, buf), "bakron_schedule_info")
    return dict(zip(SCHEDULE_KEYS, list(buf)))


PLAN_FIELDS = ("kind", "side", "ev", "K", "flags", "L", "H", "depth", "prod", "lo", "hi",
               "mode", "olo", "cols", "rlo", "rows")


def schedule_plan(m: int, n: int, order: int = ORDER_AUTO) -> list:
    """The ordered steps of an m x n solve (bakron_schedule_plan), one dict each."""
    lib = load()
    count = ctypes.c_int64(0)
    _check(lib.bakron_schedule_plan(m, n, order, None, 0, ctypes.byref(count)), "bakron_schedule_plan")
    buf = (ctypes.c_int32 * (16 * count.value))()
    _check(lib.bakron_schedule_plan(m, n, order, buf, count.value, ctypes.byref(count)),
           "bakron_schedule_plan")
    vals = list(buf)
    return [dict(zip(PLAN_FIELDS, vals[16 * k:16 * k + 16])) for k in range(count.value)]


PHASE_KEYS = ("prep_ms", "leaf_ms", "band_ms", "final_ms", "leaf_launches", "band_launches",
              "side_ms", "side_launches", "band_replay_ms", "side_replay_ms")


def last_phase_ms() -> dict:
    lib = load()
    buf = (ctypes.c_double * len(PHASE_KEYS))()
    _check(lib.bakron_last_phase_ms(buf), "bakron_last_phase_ms")
    return dict(zip(PHASE_KEYS, list(buf)))


# Operators for rounded layers.  Matrices are GPU tensors whose rows may lie apart
# (a row's elements are adjacent); nothing is copied to make them contiguous.
# `stream`: where the call runs, by default torch's current stream; inputs and given
# outputs have to be ready for it.  Inputs of 0 rows (no tokens) give outputs of 0 rows,
# and gradients of weights that are 0, without a call of the library.

_TYPES = {torch.float32: T_F32, torch.bfloat16: T_BF16, torch.float16: T_F16}
_FP8 = torch.float8_e4m3fn
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _rows_of(t, name, dtypes, ndim=2, empty=False):
    """The element distance between t's rows, after the checks that every matrix gets.
    empty: there may be no rows."""
    shape, stride, dev = t.shape, t.stride(), t.get_device()
    if dev < 0 or dev != _device():
        raise BakronError(f"{name} must be on the current GPU")
    if t.dtype not in dtypes:
        raise BakronError(f"{name} must be one of {[str(d) for d in dtypes]}, not {t.dtype}")
    if len(shape) != ndim or 0 in shape and not (empty and shape[-1] and not shape[-2]):
        raise BakronError(f"{name} must have {ndim} dimensions, none of size 0, not {tuple(shape)}")
    n, k = shape[-2], shape[-1]
    if k != 1 and stride[-1] != 1:
        raise BakronError(f"the elements of a row of {name} must be adjacent")
    if n != 1:
        ld = stride[-2]
    else:  # one row, or one in each of several matrices
        ld = stride[0] if ndim == 3 and shape[0] != 1 else max(stride[-2], k)
    if ndim == 3 and shape[0] != 1 and stride[0] != n * ld:
        raise BakronError(f"the matrices of {name} must lie {n} rows apart")
    return ld


def _vector(t, name, dtype, shape):
    """t's pointer if it is a contiguous tensor of this dtype and shape on the current GPU."""
    dev = t.get_device()
    if t.dtype != dtype or t.shape != shape or dev < 0 or dev != _device() or not t.is_contiguous():
        raise BakronError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the current GPU")
    return t.data_ptr()


def _out(out, shape, dtype, device, name):
    """(the output, the element distance between its rows): `out` after checks, or new."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device), shape[-1]
    if out.shape != shape or out.dtype != dtype:
        raise BakronError(f"{name} must be {dtype} of shape {tuple(shape)}")
    return out, _rows_of(out, name, (dtype,), len(shape), 0 in shape)


def _here():
    """The handle of torch's current stream."""
    return _raw_stream(_device())


def _elsewhere(stream):
    return stream is not None and stream.cuda_stream != _here()


def _on(stream, op, *args):
    """op(*args) with `stream` as torch's current one, so that outputs and workspaces come
    from its memory: what other streams still do there is over, or ordered before it.
    The results are marked as used on the caller's stream, which frees them."""
    caller = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        result = op(*args)
    for t in result.values() if isinstance(result, dict) else result if isinstance(result, tuple) else (result,):
        if t is not None:
            t.record_stream(caller)
    return result


def _status(t):
    return None if t is None else _vector(t, "dev_status", torch.int32, (1,))


def fp8_quantize(X, block_rows=1, out=None, scales=None, dev_status=None, stream=None):
    """X in e4m3 with a scale for each row (block_rows 1) or 128 rows (128) and 128
    columns (bakron_fp8_quantize).  Returns (codes as float8_e4m3fn, scales of
    shape (ceil(cols / 128), ceil(rows / block_rows)))."""
    if _elsewhere(stream):
        return _on(stream, fp8_quantize, X, block_rows, out, scales, dev_status)
    lib = load()
    ldx = _rows_of(X, "X", _TYPES, empty=True)
    rows, cols = X.shape
    if block_rows not in (1, 128):
        raise BakronError(f"block_rows must be 1 or 128, not {block_rows}")
    Q, ldq = _out(out, (rows, cols), _FP8, X.device, "out")
    of = (-(-cols // 128), -(-rows // block_rows))
    S = torch.empty(of, dtype=torch.float32, device=X.device) if scales is None else scales
    sp = S.data_ptr() if scales is None else _vector(S, "scales", torch.float32, of)
    if rows == 0:
        return Q, S
    _check(lib.bakron_fp8_quantize(X.data_ptr(), _TYPES[X.dtype], rows, cols, ldx, block_rows, Q.data_ptr(),
                                   ldq, sp, _status(dev_status), _here()), "bakron_fp8_quantize")
    return Q, S


def fp8_from_codes(codes, zeros=None, kind=Q_SYM, bits=4, out=None, stream=None):
    """The codes of a solve (2 to 4 bits) as e4m3 weights, exactly (bakron_fp8_from_codes)."""
    if _elsewhere(stream):
        return _on(stream, fp8_from_codes, codes, zeros, kind, bits, out)
    lib = load()
    if codes.dim() != 2 or codes.numel() == 0:
        raise BakronError(f"codes must have 2 dimensions, none of size 0, not {tuple(codes.shape)}")
    m, n = codes.shape
    cp = _vector(codes, "codes", torch.int8, (m, n))
    zp = None if zeros is None else _vector(zeros, "zeros", torch.float32, (m,))
    Q, ldq = _out(out, (m, n), _FP8, codes.device, "out")
    _check(lib.bakron_fp8_from_codes(cp, zp, m, n, kind, bits, Q.data_ptr(), ldq, _here()),
           "bakron_fp8_from_codes")
    return Q


def _groups(W, offsets):
    groups = W.shape[0] if W.dim() == 3 else 1
    if offsets is None:
        if groups != 1:
            raise BakronError("offsets are needed where W has groups")
        return groups, None
    return groups, _vector(offsets, "offsets", torch.int32, (groups + 1,))


def _space(nbytes, device):
    """A workspace of nbytes, or None for none."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def fp8_matmul(X, sx, W, sw, offsets=None, out_dtype=torch.bfloat16, out=None, dev_status=None, stream=None):
    """Y = X W^T of e4m3 operands with scales (bakron_fp8_matmul).

    X (rows, K) with sx (ceil(K / 128), rows); W (N, K), or (groups, N, K) with
    offsets (int32, groups + 1, on the GPU).  sw has one scale for each row of W,
    of shape (N,) or (groups, N), or one for each block, of shape (ceil(K / 128),
    ceil(N / 128)) or (groups, ...).  out_dtype: bfloat16 or float16."""
    if _elsewhere(stream):
        return _on(stream, fp8_matmul, X, sx, W, sw, offsets, out_dtype, out, dev_status)
    lib = load()
    ldx = _rows_of(X, "X", (_FP8,), empty=True)
    ldw = _rows_of(W, "W", (_FP8,), 3 if W.dim() == 3 else 2)
    rows, K = X.shape
    N = W.shape[-2]
    if W.shape[-1] != K:
        raise BakronError(f"W's rows have {W.shape[-1]} elements, X's {K}")
    groups, op = _groups(W, offsets)
    kb, lead = -(-K // 128), tuple(W.shape[:-2])
    sxp = _vector(sx, "sx", torch.float32, (kb, rows))
    if sw.dim() == W.dim():
        wscale, swp = SCALE_BLOCK, _vector(sw, "sw", torch.float32, (*lead, kb, -(-N // 128)))
    else:
        wscale, swp = SCALE_ROW, _vector(sw, "sw", torch.float32, (*lead, N))
    if out_dtype not in (torch.bfloat16, torch.float16):
        raise BakronError(f"out_dtype must be bfloat16 or float16, not {out_dtype}")
    Y, ldy = _out(out, (rows, N), out_dtype, X.device, "out")
    if rows == 0:
        return Y
    ws = _space(lib.bakron_fp8_matmul_workspace_size(rows, N, K, groups), X.device)
    _check(lib.bakron_fp8_matmul(X.data_ptr(), ldx, sxp, W.data_ptr(), ldw, swp, wscale, rows, N, K, groups,
                                 op, Y.data_ptr(), _TYPES[out_dtype], ldy, _status(dev_status),
                                 None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(),
                                 _here()), "bakron_fp8_matmul")
    return Y


def _grouped(fn, what, A, B, rows, N, K, groups, op, shape, out_dtype, out, dev_status, over_rows=False):
    """over_rows: the sums run over the rows, which both operands have."""
    lib = load()
    lda = _rows_of(A, "the left operand", (torch.bfloat16, torch.float16), empty=True)
    ldb = _rows_of(B, "the right operand", (A.dtype,), B.dim(), over_rows)
    dtype = A.dtype if out_dtype is None else out_dtype
    if dtype not in (A.dtype, torch.float32):
        raise BakronError(f"the output's dtype must be {A.dtype} or float32, not {dtype}")
    Y, ldy = _out(out, shape, dtype, A.device, "out")
    if rows == 0:
        return Y.zero_()  # sums over no rows, or no elements
    ws = _space(lib.bakron_grouped_matmul_workspace_size(rows, N, K, groups), A.device)
    _check(fn(A.data_ptr(), _TYPES[A.dtype], lda, B.data_ptr(), ldb, rows, N, K, groups, op, Y.data_ptr(),
              _TYPES[dtype], ldy, _status(dev_status), None if ws is None else ws.data_ptr(),
              0 if ws is None else ws.numel(), _here()), what)
    return Y


def grouped_matmul(X, W, offsets=None, out_dtype=None, out=None, dev_status=None, stream=None):
    """Y[r] = X[r] W_g(r)^T (bakron_grouped_matmul).  X (rows, K) and W (groups, N, K)
    in bfloat16 or float16, offsets (int32, groups + 1, on the GPU): group g has the
    rows offsets[g] .. offsets[g + 1] - 1.  out_dtype: X's (the default) or float32."""
    if _elsewhere(stream):
        return _on(stream, grouped_matmul, X, W, offsets, out_dtype, out, dev_status)
    groups, op = _groups(W, offsets)
    if X.dim() != 2 or W.dim() not in (2, 3) or W.shape[-1] != X.shape[1]:
        raise BakronError(f"X {tuple(X.shape)} and W {tuple(W.shape)} do not fit")
    rows, K, N = X.shape[0], X.shape[1], W.shape[-2]
    return _grouped(load().bakron_grouped_matmul, "bakron_grouped_matmul", X, W, rows, N, K, groups, op,
                    (rows, N), out_dtype, out, dev_status)


def grouped_matmul_grad(dY, X, W, offsets=None, want_x=True, want_w=True, w_dtype=None, dev_status=None,
                        stream=None):
    """grouped_matmul's gradients (dX, dW) for dY (bakron_grouped_matmul_grad_x and
    _grad_w).  One that is not wanted is None.  w_dtype: X's (the default) or float32."""
    if _elsewhere(stream):
        return _on(stream, grouped_matmul_grad, dY, X, W, offsets, want_x, want_w, w_dtype, dev_status)
    groups, op = _groups(W, offsets)
    if X.dim() != 2 or W.dim() not in (2, 3) or W.shape[-1] != X.shape[1] or \
            tuple(dY.shape) != (X.shape[0], W.shape[-2]):
        raise BakronError(f"dY {tuple(dY.shape)}, X {tuple(X.shape)} and W {tuple(W.shape)} do not fit")
    rows, K, N = X.shape[0], X.shape[1], W.shape[-2]
    lib, dX, dW = load(), None, None
    if want_x:
        dX = _grouped(lib.bakron_grouped_matmul_grad_x, "bakron_grouped_matmul_grad_x", dY, W, rows, N, K,
                      groups, op, (rows, K), None, None, dev_status)
    if want_w:
        dW = _grouped(lib.bakron_grouped_matmul_grad_w, "bakron_grouped_matmul_grad_w", dY, X, rows, N, K,
                      groups, op, tuple(W.shape), w_dtype, None, dev_status, over_rows=True)
    return dX, dW


def token_logprobs(logits, targets, top=0, dev_status=None, stream=None):
    """Log probabilities of the targets (int64, negative: none), with entropy and the
    `top` likeliest tokens (bakron_token_logprobs).  Returns a dict with logprob,
    lse, entropy (rows) and top_logprob, top_ids (rows, top; None for top 0)."""
    if _elsewhere(stream):
        return _on(stream, token_logprobs, logits, targets, top, dev_status)
    lib = load()
    ld = _rows_of(logits, "logits", _TYPES, empty=True)
    rows, vocab = logits.shape
    tp = _vector(targets, "targets", torch.int64, (rows,))
    if not 0 <= top <= min(64, vocab):
        raise BakronError(f"top must be in 0 .. {min(64, vocab)}, not {top}")
    dev = logits.device
    stats = torch.empty((3, rows), dtype=torch.float32, device=dev)
    logprob, lse, entropy = stats.unbind()
    tl = torch.empty((rows, top), dtype=torch.float32, device=dev) if top else None
    ti = torch.empty((rows, top), dtype=torch.int64, device=dev) if top else None
    if rows:
        ws = _space(lib.bakron_token_logprobs_workspace_size(rows, vocab, top), dev)
        sp = stats.data_ptr()
        _check(lib.bakron_token_logprobs(logits.data_ptr(), _TYPES[logits.dtype], rows, vocab, ld, tp, top, sp,
                                         sp + 4 * rows, sp + 8 * rows, tl.data_ptr() if top else None,
                                         ti.data_ptr() if top else None, _status(dev_status),
                                         None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(),
                                         _here()), "bakron_token_logprobs")
    return dict(logprob=logprob, lse=lse, entropy=entropy, top_logprob=tl, top_ids=ti)


def token_logprobs_grad(logits, targets, lse, entropy, g_logprob, g_entropy=None, out=None, dev_status=None,
                        stream=None):
    """The gradient of sum(g_logprob logprob + g_entropy entropy) with respect to the
    logits (bakron_token_logprobs_grad), from the forward call's lse and entropy."""
    if _elsewhere(stream):
        return _on(stream, token_logprobs_grad, logits, targets, lse, entropy, g_logprob, g_entropy, out, dev_status)
    lib = load()
    ld = _rows_of(logits, "logits", _TYPES, empty=True)
    rows, vocab = logits.shape
    f32 = torch.float32
    D, ldd = _out(out, (rows, vocab), logits.dtype, logits.device, "out")
    if g_entropy is not None and entropy is None:
        raise BakronError("g_entropy needs the forward call's entropy")
    vectors = (_vector(targets, "targets", torch.int64, (rows,)), _vector(lse, "lse", f32, (rows,)),
               None if entropy is None else _vector(entropy, "entropy", f32, (rows,)),
               _vector(g_logprob, "g_logprob", f32, (rows,)),
               None if g_entropy is None else _vector(g_entropy, "g_entropy", f32, (rows,)))
    if rows:
        _check(lib.bakron_token_logprobs_grad(logits.data_ptr(), _TYPES[logits.dtype], rows, vocab, ld, *vectors,
                                              D.data_ptr(), ldd, _status(dev_status), _here()),
               "bakron_token_logprobs_grad")
    return D


def verify_drafts(p, q, drafts, u, v, dev_status=None, stream=None):
    """Which drafted tokens the target keeps, and the token after them (bakron_verify_drafts).

    p (batch, n + 1, vocab) the target's probabilities; q (batch, n, vocab) the draft's, or
    None for drafts that were not drawn from any; drafts (batch, n) int64, negative from a
    request's end on; u (batch, n) and v (batch,) float32 in [0, 1).  Returns (accepted
    (batch,) int32, tokens (batch, n + 1) int64: the accepted drafts, the drawn token, -1)."""
    if _elsewhere(stream):
        return _on(stream, verify_drafts, p, q, drafts, u, v, dev_status)
    lib = load()
    if p.dim() != 3 or drafts.dim() != 2 or p.shape[:2] != (drafts.shape[0], drafts.shape[1] + 1):
        raise BakronError(f"p {tuple(p.shape)} and drafts {tuple(drafts.shape)} do not fit")
    (batch, n), vocab, dev = drafts.shape, p.shape[2], p.device
    if batch == 0:
        return (torch.empty(0, dtype=torch.int32, device=dev), torch.empty((0, n + 1), dtype=torch.int64, device=dev))
    ldp, ldq = _rows_of(p, "p", _TYPES, 3), 0
    if n == 0:
        q = None
    if q is not None:
        if q.shape != (batch, n, vocab):
            raise BakronError(f"q must be of shape {(batch, n, vocab)}, not {tuple(q.shape)}")
        ldq = _rows_of(q, "q", (p.dtype,), 3)
    vectors = (_vector(drafts, "drafts", torch.int64, (batch, n)), _vector(u, "u", torch.float32, (batch, n)),
               _vector(v, "v", torch.float32, (batch,)))
    accepted = torch.empty(batch, dtype=torch.int32, device=dev)
    tokens = torch.empty((batch, n + 1), dtype=torch.int64, device=dev)
    ws = _space(lib.bakron_verify_drafts_workspace_size(batch, n, vocab), dev)
    _check(lib.bakron_verify_drafts(p.data_ptr(), ldp, None if q is None else q.data_ptr(), ldq, _TYPES[p.dtype], batch, n,
                                    vocab, *vectors, accepted.data_ptr(), tokens.data_ptr(), _status(dev_status),
                                    None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), _here()),
           "bakron_verify_drafts")
    return accepted, tokens


# Rows by group and back.

def group_sort(ids, groups, dev_status=None, stream=None):
    """A stable sort of ids (int32 or int64, contiguous, negative: no group) by group
    (bakron_group_sort).  Returns int32 tensors (offsets (groups + 1,), order (n,),
    slots of ids' shape): group g has the places offsets[g] .. offsets[g + 1] - 1, order
    is the element at each place, slots the place of each element.  Elements of no group
    come last."""
    if _elsewhere(stream):
        return _on(stream, group_sort, ids, groups, dev_status)
    lib = load()
    if ids.dtype not in (torch.int32, torch.int64):
        raise BakronError(f"ids must be int32 or int64, not {ids.dtype}")
    ip, n, dev = _vector(ids, "ids", ids.dtype, ids.shape), ids.numel(), ids.device
    if not 1 <= groups <= 4096:
        raise BakronError(f"groups must be in 1 .. 4096, not {groups}")
    if n == 0:
        return (torch.zeros(groups + 1, dtype=torch.int32, device=dev),
                torch.empty(0, dtype=torch.int32, device=dev), torch.empty(ids.shape, dtype=torch.int32, device=dev))
    offsets = torch.empty(groups + 1, dtype=torch.int32, device=dev)
    order = torch.empty(n, dtype=torch.int32, device=dev)
    slots = torch.empty(ids.shape, dtype=torch.int32, device=dev)
    ws = _space(lib.bakron_group_sort_workspace_size(n, groups), dev)
    _check(lib.bakron_group_sort(ip, 32 if ids.dtype == torch.int32 else 64, n, groups, offsets.data_ptr(),
                                 order.data_ptr(), slots.data_ptr(), _status(dev_status),
                                 None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), _here()),
           "bakron_group_sort")
    return offsets, order, slots


def _pairs(slots, offsets, tokens):
    """(k, groups, slots' and offsets' pointers) after checks."""
    if slots.dim() == 1:
        k = 1
    elif slots.dim() == 2 and slots.shape[1]:
        k = slots.shape[1]
    else:
        raise BakronError(f"slots must be (tokens, k), not {tuple(slots.shape)}")
    if slots.shape[0] != tokens:
        raise BakronError(f"slots are of {slots.shape[0]} tokens, not {tokens}")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise BakronError(f"offsets must be (groups + 1,), not {tuple(offsets.shape)}")
    return (k, offsets.shape[0] - 1, _vector(slots, "slots", torch.int32, slots.shape),
            _vector(offsets, "offsets", torch.int32, offsets.shape))


def group_gather(X, slots, offsets, out=None, dev_status=None, stream=None):
    """The rows of X (tokens, cols) copied to the places of a group_sort of (tokens, k)
    choices, 0 for choices of no group (bakron_group_gather).  Returns (tokens k, cols).
    The gradient of X is group_combine of the copies' gradients, without weights."""
    if _elsewhere(stream):
        return _on(stream, group_gather, X, slots, offsets, out, dev_status)
    lib = load()
    ldx = _rows_of(X, "X", _TYPES, empty=True)
    tokens, cols = X.shape
    k, groups, sp, op = _pairs(slots, offsets, tokens)
    Y, ldo = _out(out, (tokens * k, cols), X.dtype, X.device, "out")
    if tokens:
        _check(lib.bakron_group_gather(X.data_ptr(), _TYPES[X.dtype], tokens, k, cols, ldx, sp, groups, op, Y.data_ptr(),
                                       ldo, _status(dev_status), _here()), "bakron_group_gather")
    return Y


def group_gather_fp8(X, slots, offsets, out=None, scales=None, dev_status=None, stream=None):
    """group_gather in e4m3 with a scale for each row and 128 columns, as fp8_matmul takes
    them (bakron_group_gather_fp8).  Returns (codes (tokens k, cols), scales
    (ceil(cols / 128), tokens k))."""
    if _elsewhere(stream):
        return _on(stream, group_gather_fp8, X, slots, offsets, out, scales, dev_status)
    lib = load()
    ldx = _rows_of(X, "X", _TYPES, empty=True)
    tokens, cols = X.shape
    k, groups, sp, op = _pairs(slots, offsets, tokens)
    Q, ldq = _out(out, (tokens * k, cols), _FP8, X.device, "out")
    of = (-(-cols // 128), tokens * k)
    S = torch.empty(of, dtype=torch.float32, device=X.device) if scales is None else scales
    cp = S.data_ptr() if scales is None else _vector(S, "scales", torch.float32, of)
    if tokens:
        _check(lib.bakron_group_gather_fp8(X.data_ptr(), _TYPES[X.dtype], tokens, k, cols, ldx, sp, groups, op,
                                           Q.data_ptr(), ldq, cp, _status(dev_status), _here()),
               "bakron_group_gather_fp8")
    return Q, S


def _combined(Y, slots, offsets, weights):
    """(row distance, tokens, k, groups, pointers) of the sorted rows Y, after checks."""
    ldy = _rows_of(Y, "Y", _TYPES, empty=True)
    tokens = slots.shape[0] if slots.dim() else 0
    k, groups, sp, op = _pairs(slots, offsets, tokens)
    if Y.shape[0] != tokens * k:
        raise BakronError(f"Y has {Y.shape[0]} rows, slots {tokens * k}")
    return ldy, tokens, k, groups, sp, op, None if weights is None else _vector(weights, "weights", torch.float32,
                                                                                slots.shape)


def group_combine(Y, slots, offsets, weights=None, out=None, dev_status=None, stream=None):
    """out[t] = sum_j weights[t][j] Y[slots[t][j]] over the choices that have a group
    (bakron_group_combine).  Y (tokens k, cols); weights (tokens, k) in float32, or None
    for 1.  Returns (tokens, cols) in Y's dtype."""
    if _elsewhere(stream):
        return _on(stream, group_combine, Y, slots, offsets, weights, out, dev_status)
    lib = load()
    ldy, tokens, k, groups, sp, op, wp = _combined(Y, slots, offsets, weights)
    cols = Y.shape[1]
    R, ldo = _out(out, (tokens, cols), Y.dtype, Y.device, "out")
    if tokens:
        _check(lib.bakron_group_combine(Y.data_ptr(), _TYPES[Y.dtype], tokens, k, cols, ldy, sp, groups, op, wp,
                                        R.data_ptr(), ldo, _status(dev_status), _here()), "bakron_group_combine")
    return R


def group_combine_grad(dout, Y, slots, offsets, weights, out=None, dev_status=None, stream=None):
    """group_combine's gradients (dY of Y's shape and dtype, dweights (tokens, k) in
    float32) for dout (bakron_group_combine_grad); 0 for choices of no group."""
    if _elsewhere(stream):
        return _on(stream, group_combine_grad, dout, Y, slots, offsets, weights, out, dev_status)
    lib = load()
    if weights is None:
        raise BakronError("weights are needed; without them Y's gradient is group_gather of dout")
    ldy, tokens, k, groups, sp, op, wp = _combined(Y, slots, offsets, weights)
    cols = Y.shape[1]
    ldd = _rows_of(dout, "dout", (Y.dtype,), empty=True)
    if dout.shape != (tokens, cols):
        raise BakronError(f"dout must be of shape {(tokens, cols)}, not {tuple(dout.shape)}")
    dY, lddy = _out(out, (tokens * k, cols), Y.dtype, Y.device, "out")
    dw = torch.empty(slots.shape, dtype=torch.float32, device=Y.device)
    if tokens:
        _check(lib.bakron_group_combine_grad(dout.data_ptr(), ldd, Y.data_ptr(), _TYPES[Y.dtype], tokens, k, cols, ldy,
                                             sp, groups, op, wp, dY.data_ptr(), lddy, dw.data_ptr(),
                                             _status(dev_status), _here()), "bakron_group_combine_grad")
    return dY, dw


# Low-rank adapters beside a shared projection.

def _adapters(A, B, offsets, order, scale, rows, dtype):
    """(N, K, rank, groups, pointers of A, B, offsets, order, scale) after checks."""
    if A.dim() not in (2, 3) or B.dim() != A.dim() or A.shape[:-2] != B.shape[:-2] or A.shape[-2] != B.shape[-1] or \
            A.numel() == 0 or B.numel() == 0:
        raise BakronError(f"A {tuple(A.shape)} and B {tuple(B.shape)} do not fit")
    if dtype not in (torch.bfloat16, torch.float16):
        raise BakronError(f"X, A and B must be bfloat16 or float16, not {dtype}")
    groups, op = _groups(A, offsets)
    return (B.shape[-2], A.shape[-1], A.shape[-2], groups, _vector(A, "A", dtype, A.shape), _vector(B, "B", dtype, B.shape),
            op, None if order is None else _vector(order, "order", torch.int32, (rows,)),
            None if scale is None else _vector(scale, "scale", torch.float32, (groups,)))


def _added(base, out, shape, dtype, want, device):
    """(out, its row distance, base's pointer and row distance): base is of out's dtype, `want`
    or the inputs' dtype."""
    if base is not None:
        if want is not None and base.dtype != want:
            raise BakronError(f"base must be {want}, not {base.dtype}")
        want = base.dtype
    want = dtype if want is None and out is None else out.dtype if want is None else want
    if want not in (dtype, torch.float32):
        raise BakronError(f"the output's dtype must be {dtype} or float32, not {want}")
    Y, ldo = _out(out, shape, want, device, "out")
    if base is None:
        return Y, ldo, None, 0
    if base.shape != shape:
        raise BakronError(f"base must be of shape {tuple(shape)}, not {tuple(base.shape)}")
    return Y, ldo, base.data_ptr(), _rows_of(base, "base", (want,), empty=True)


def adapter_matmul(X, A, B, offsets=None, order=None, scale=None, base=None, out=None, out_dtype=None, dev_status=None,
                   stream=None):
    """out[r] = base[r] + scale_g B_g (A_g X[r]) with each row's adapter g (bakron_adapter_matmul).

    X (rows, K); A (adapters, rank, K) and B (adapters, N, rank), contiguous, or without the
    first dimension for one adapter; all bfloat16 or float16.  offsets and order: group_sort
    of the rows' adapters (order None: rows lie sorted); scale (adapters,) float32 or None.
    base (rows, N), the shared projection's result, of out's dtype, which is X's or float32;
    None counts as 0.  out may be base."""
    if _elsewhere(stream):
        return _on(stream, adapter_matmul, X, A, B, offsets, order, scale, base, out, out_dtype, dev_status)
    lib = load()
    ldx = _rows_of(X, "X", (torch.bfloat16, torch.float16), empty=True)
    rows = X.shape[0]
    N, K, rank, groups, ap, bp, op, rp, cp = _adapters(A, B, offsets, order, scale, rows, X.dtype)
    if X.shape[1] != K:
        raise BakronError(f"X's rows have {X.shape[1]} elements, A's {K}")
    Y, ldo, base_p, ldb = _added(base, out, (rows, N), X.dtype, out_dtype, X.device)
    if rows == 0:
        return Y
    ws = _space(lib.bakron_adapter_matmul_workspace_size(rows, N, K, rank, groups), X.device)
    _check(lib.bakron_adapter_matmul(X.data_ptr(), _TYPES[X.dtype], ldx, ap, bp, rows, N, K, rank, groups, op, rp, cp,
                                     base_p, ldb, Y.data_ptr(), _TYPES[Y.dtype], ldo, _status(dev_status),
                                     None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), _here()),
           "bakron_adapter_matmul")
    return Y


def adapter_matmul_grad(dY, X, A, B, offsets=None, order=None, scale=None, base=None, out=None, want_x=True, want_w=True,
                        x_dtype=None, w_dtype=None, dev_status=None, stream=None):
    """adapter_matmul's gradients (dX, dA, dB) for dY (rows, N) (bakron_adapter_matmul_grad).
    dX is added to base, the gradient that X gets from the shared projection (None: 0), and
    written to out if given (it may be base).  Those that are not wanted are None.  x_dtype
    and w_dtype: X's (the default) or float32."""
    if _elsewhere(stream):
        return _on(stream, adapter_matmul_grad, dY, X, A, B, offsets, order, scale, base, out, want_x, want_w, x_dtype,
                   w_dtype, dev_status)
    lib = load()
    lddy = _rows_of(dY, "dY", (torch.bfloat16, torch.float16), empty=True)
    ldx = _rows_of(X, "X", (dY.dtype,), empty=True)
    rows, dtype, dev = X.shape[0], X.dtype, X.device
    N, K, rank, groups, ap, bp, op, rp, cp = _adapters(A, B, offsets, order, scale, rows, dtype)
    if dY.shape != (rows, N) or X.shape[1] != K:
        raise BakronError(f"dY {tuple(dY.shape)}, X {tuple(X.shape)}, A and B do not fit")
    dX, lddx, base_p, ldb, dA, dB = None, 0, None, 0, None, None
    if want_x:
        dX, lddx, base_p, ldb = _added(base, out, (rows, K), dtype, x_dtype, dev)
    elif base is not None or out is not None:
        raise BakronError("base and out go with want_x")
    if want_w:
        w_dtype = dtype if w_dtype is None else w_dtype
        if w_dtype not in (dtype, torch.float32):
            raise BakronError(f"w_dtype must be {dtype} or float32, not {w_dtype}")
        new = torch.zeros if rows == 0 else torch.empty
        dA, dB = (new(t.shape, dtype=w_dtype, device=dev) for t in (A, B))
    if rows == 0 or not (want_x or want_w):
        return dX, dA, dB
    ws = _space(lib.bakron_adapter_matmul_grad_workspace_size(rows, N, K, rank, groups), dev)
    _check(lib.bakron_adapter_matmul_grad(dY.data_ptr(), lddy, X.data_ptr(), _TYPES[dtype], ldx, ap, bp, rows, N, K, rank,
                                          groups, op, rp, cp, base_p, ldb, None if dX is None else dX.data_ptr(),
                                          _TYPES[dtype if dX is None else dX.dtype], lddx,
                                          None if dA is None else dA.data_ptr(), None if dB is None else dB.data_ptr(),
                                          _TYPES[w_dtype] if want_w else 0, _status(dev_status),
                                          None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), _here()),
           "bakron_adapter_matmul_grad")
    return dX, dA, dB
