"""ctypes binding of libnrm.so (include/nrm.h).

Argument marshalling only: every step of every operator runs in the CUDA
library.  torch provides the device memory and the current stream.  If the
library is missing the first call raises; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnrm.so")

NRM_F32, NRM_F16, NRM_BF16 = 0, 1, 2
PLAN_AUTO, PLAN_GENERIC, PLAN_WARP, PLAN_CTA, PLAN_TMA, PLAN_PERSIST, PLAN_WRAW, PLAN_CLUSTER = range(8)
PLAN_NAMES = {0: "auto", 1: "generic", 2: "warp", 3: "cta", 4: "tma", 5: "persist", 6: "wraw",
              7: "cluster"}

_DT = {torch.float32: NRM_F32, torch.float16: NRM_F16, torch.bfloat16: NRM_BF16}

_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_U64 = ctypes.c_uint64
_F = ctypes.c_float
_D = ctypes.c_double
_SZ = ctypes.c_size_t
_INT = ctypes.c_int


class NrmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


def _declare(lib):
    lib.ln_fwd.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _INT, _P]
    lib.rms_fwd.argtypes = [_P, _P, _P, _P, _I64, _I64, _F, _INT, _P]
    lib.add_rms_fwd.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _INT, _P]
    lib.bn_fwd_train_workspace_size.argtypes = [_I64, _I64, _I64, _INT]
    lib.bn_fwd_train_workspace_size.restype = ctypes.c_size_t
    lib.bn_fwd_train.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, _INT,
                                 _P, ctypes.c_size_t, _P]
    for f in ("ln_fwd", "rms_fwd", "add_rms_fwd", "bn_fwd_train"):
        getattr(lib, f).restype = _INT
    lib.bn_fwd_train_noalloc.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F,
                                         _F, _INT, _P]
    lib.bn_fwd_train_noalloc.restype = _INT
    lib.bn_fwd_infer.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _INT, _P]
    lib.bn_fwd_infer.restype = _INT
    lib.bn_bwd_workspace_size.argtypes = [_I64, _I64, _I64, _INT]
    lib.bn_bwd_workspace_size.restype = ctypes.c_size_t
    lib.bn_bwd.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _INT, _P,
                           ctypes.c_size_t, _P]
    lib.bn_bwd.restype = _INT
    lib.softmax_fwd.argtypes = [_P, _P, _P, _P, _I64, _I64, _INT, _P]
    lib.softmax_fwd.restype = _INT
    lib.ln_fwd_ld.argtypes = [_P, _I64, _P, _P, _P, _I64, _P, _P, _I64, _I64, _F, _INT, _P]
    lib.rms_fwd_ld.argtypes = [_P, _I64, _P, _P, _I64, _P, _I64, _I64, _F, _INT, _P]
    lib.add_rms_fwd_ld.argtypes = [_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _I64,
                                   _F, _INT, _P]
    lib.softmax_fwd_ld.argtypes = [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _INT, _P]
    for f in ("ln_fwd_ld", "rms_fwd_ld", "add_rms_fwd_ld", "softmax_fwd_ld"):
        getattr(lib, f).restype = _INT
    lib.bn_fwd_partial_stats.argtypes = [_P, _P, _I64, _I64, _I64, _INT, _P, ctypes.c_size_t, _P]
    lib.bn_fwd_apply_stats.argtypes = [_P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I64,
                                       _F, _F, _INT, _P]
    lib.bn_bwd_partial_sums.argtypes = [_P, _P, _P, _P, _P, _I64, _I64, _I64, _INT, _P,
                                        ctypes.c_size_t, _P]
    lib.bn_bwd_apply_sums.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _I64, _I64,
                                      _I64, _INT, _P]
    for f in ("bn_fwd_partial_stats", "bn_fwd_apply_stats", "bn_bwd_partial_sums",
              "bn_bwd_apply_sums"):
        getattr(lib, f).restype = _INT
    lib.add_rms_fwd_host_workspace_size.argtypes = [_I64, _INT]
    lib.add_rms_fwd_host_workspace_size.restype = ctypes.c_size_t
    lib.add_rms_fwd_host.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _INT, _P,
                                     ctypes.c_size_t, _P]
    lib.add_rms_fwd_host.restype = _INT
    drop = [_D, _U64, _U64, _P]  # p, seed, offset, offset_dev
    lib.dropout_fwd.argtypes = [_P, _P, _I64, _I64, *drop, _INT, _P]
    lib.dropout_fwd_ld.argtypes = [_P, _I64, _P, _I64, _I64, _I64, *drop, _INT, _P]
    lib.dropout_add_rms_fwd.argtypes = [_P] * 6 + [_I64, _I64, *drop, _F, _INT, _P]
    lib.dropout_add_rms_fwd_ld.argtypes = [_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64,
                                           _I64, *drop, _F, _INT, _P]
    lib.dropout_add_rms_bwd_workspace_size.argtypes = [_I64, _I64, _INT]
    lib.dropout_add_rms_bwd_workspace_size.restype = _SZ
    lib.dropout_add_rms_bwd.argtypes = [_P] * 8 + [_I64, _I64, *drop, _INT, _P, _SZ, _P]
    lib.dropout_add_rms_bwd_ld.argtypes = [_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64, _P,
                                           _I64, _P, _I64, _I64, *drop, _INT, _P, _SZ, _P]
    lib.logprob_fwd.argtypes = [_P] * 4 + [_I64, _I64, _F, _INT, _P]
    lib.logprob_fwd_ld.argtypes = [_P, _I64, _P, _P, _P, _I64, _I64, _F, _INT, _P]
    lib.logprob_fwd_stats.argtypes = [_P] * 5 + [_I64, _I64, _F, _INT, _P]
    lib.logprob_fwd_stats_ld.argtypes = [_P, _I64, _P, _P, _P, _P, _I64, _I64, _F, _INT, _P]
    lib.logprob_bwd.argtypes = [_P] * 5 + [_I64, _I64, _F, _INT, _P]
    lib.logprob_bwd_ld.argtypes = [_P, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _F, _INT, _P]
    lib.logprob_bwd_stats.argtypes = lib.logprob_bwd.argtypes
    lib.logprob_bwd_stats_ld.argtypes = lib.logprob_bwd_ld.argtypes
    lib.policy_loss_workspace_size.argtypes = [_I64]
    lib.policy_loss_workspace_size.restype = _SZ
    lib.policy_loss.argtypes = [_P] * 6 + [_D, _D, _F, _F] + [_P] * 4 + [_I64, _I64, _INT, _P, _SZ, _P]
    lib.policy_loss_ld.argtypes = [_P, _I64] + [_P] * 5 + [_D, _D, _F, _F] + [_P] * 4 + [
        _I64, _I64, _I64, _INT, _P, _SZ, _P]
    for f in ("dropout_fwd", "dropout_add_rms_fwd", "dropout_add_rms_bwd", "logprob_fwd",
              "logprob_fwd_stats", "logprob_bwd", "logprob_bwd_stats", "policy_loss"):
        getattr(lib, f).restype = getattr(lib, f + "_ld").restype = _INT
    heads = [_P, _I64, _I64]  # pointer, token stride, head stride
    lib.qk_norm_rope_fwd.argtypes = heads * 2 + [_P] * 4 + heads * 2 + [_I64] * 6 + [_F, _INT, _INT, _P]
    lib.qk_norm_rope_bwd_workspace_size.argtypes = [_I64] * 4
    lib.qk_norm_rope_bwd_workspace_size.restype = _SZ
    lib.qk_norm_rope_bwd.argtypes = heads * 4 + [_P] * 4 + heads * 2 + [_P] * 2 + [_I64] * 6 + [
        _F, _INT, _INT, _P, _SZ, _P]
    lib.route_fwd.argtypes = [_P, _I64] + [_P] * 4 + [_I64] * 3 + [_INT] + [_I64] * 3 + [_INT, _F, _INT, _P]
    lib.route_bwd.argtypes = [_P, _P, _I64, _P, _P, _P] + [_I64] * 4 + [_INT, _INT, _F, _INT, _P]
    lib.logprob_top_fwd.argtypes = [_P] * 7 + [_I64] * 3 + [_F, _INT, _P]
    lib.logprob_top_fwd_ld.argtypes = [_P, _I64] + [_P] * 6 + [_I64] * 3 + [_F, _INT, _P]
    lib.logprob_top_bwd.argtypes = [_P] * 9 + [_I64] * 3 + [_F, _INT, _P]
    lib.logprob_top_bwd_ld.argtypes = [_P] * 4 + [_I64] + [_P] * 5 + [_I64] * 4 + [_F, _INT, _P]
    for f in ("qk_norm_rope_fwd", "qk_norm_rope_bwd", "route_fwd", "route_bwd", "logprob_top_fwd",
              "logprob_top_fwd_ld", "logprob_top_bwd", "logprob_top_bwd_ld"):
        getattr(lib, f).restype = _INT
    lib.nrm_status_string.argtypes = [_INT]
    lib.nrm_status_string.restype = ctypes.c_char_p
    lib.nrm_force_plan.argtypes = [_INT, _INT, _INT, _INT, _INT]
    lib.nrm_force_plan.restype = _INT
    lib.nrm_last_plan.argtypes = [ctypes.POINTER(_INT)] * 5
    lib.nrm_last_plan.restype = None
    lib.nrm_set_wait_limit.argtypes = [ctypes.c_uint]
    lib.nrm_set_wait_limit.restype = ctypes.c_uint
    lib.nrm_device_fault.argtypes = [ctypes.POINTER(ctypes.c_uint), _INT]
    lib.nrm_device_fault.restype = _INT
    lib.nrm_set_pointer_checks.argtypes = [_INT]
    lib.nrm_set_pointer_checks.restype = _INT
    lib.nrm_set_bn_group_bytes.argtypes = [ctypes.c_size_t]
    lib.nrm_set_bn_group_bytes.restype = ctypes.c_size_t
    return lib


def lib():
    """The loaded libnrm.so (ctypes.CDLL).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"{LIB_PATH} is missing: build it first "
                        "(python -c 'import __graft_entry__ as g; g.build()')")
                _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def status_string(status: int) -> str:
    return lib().nrm_status_string(status).decode()


def _check(status: int, where: str):
    if status != 0:
        raise NrmError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _cuda(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _param(p, n, dtype, device, name):
    if p is None:
        return None
    _cuda(p, name)
    if p.dtype != dtype or p.numel() != n or p.device != device:
        raise ValueError(f"{name} must be [{n}] {dtype} on {device}")
    return p


def _rows_view(x: torch.Tensor):
    n = x.shape[-1]
    return x.numel() // n if n else 0, n


def _rows(t: torch.Tensor, name: str):
    """(rows, N, row stride) of a row-operator tensor: contiguous, or 2-D with
    unit column stride (a column slice or a padded buffer)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    n = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // n if n else 0), n, n
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= n:
        return t.shape[0], n, t.stride(0)
    raise ValueError(f"{name} must be contiguous, or 2-D with unit column stride")


def _same_rows(t, x, name):
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError(f"{name} must match x in shape, dtype and device")
    return _rows(t, name)[2]


# ---------------------------------------------------------------------------
# Operators (same names as the C ABI).
# ---------------------------------------------------------------------------
def ln_fwd(x, gamma=None, beta=None, eps=1e-5, *, out=None, mean=None, rstd=None,
           want_stats=True, stream=None):
    """LayerNorm over the last dimension of x.  Returns (y, mean, rstd).  x
    (and out) may be 2-D views with a row stride (ln_fwd_ld)."""
    rows, n, ldx = _rows(x, "x")
    gamma = _param(gamma, n, x.dtype, x.device, "gamma")
    beta = _param(beta, n, x.dtype, x.device, "beta")
    y = torch.empty(x.shape, device=x.device, dtype=x.dtype) if out is None else out
    ldy = _same_rows(y, x, "out")
    if want_stats:
        mean = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32) if mean is None else mean
        rstd = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32) if rstd is None else rstd
    with torch.cuda.device(x.device):
        st = lib().ln_fwd_ld(_ptr(x), ldx, _ptr(gamma), _ptr(beta), _ptr(y), ldy, _ptr(mean),
                             _ptr(rstd), rows, n, eps, _dtype_code(x),
                             stream if stream is not None else _stream(x.device))
    _check(st, "ln_fwd")
    return y, mean, rstd


def rms_fwd(x, w=None, eps=1e-6, *, out=None, rstd=None, want_stats=False, stream=None):
    """RMSNorm over the last dimension of x.  Returns (y, rstd or None)."""
    rows, n, ldx = _rows(x, "x")
    w = _param(w, n, x.dtype, x.device, "w")
    y = torch.empty(x.shape, device=x.device, dtype=x.dtype) if out is None else out
    ldy = _same_rows(y, x, "out")
    if want_stats and rstd is None:
        rstd = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32)
    with torch.cuda.device(x.device):
        st = lib().rms_fwd_ld(_ptr(x), ldx, _ptr(w), _ptr(y), ldy, _ptr(rstd), rows, n, eps,
                              _dtype_code(x), stream if stream is not None else _stream(x.device))
    _check(st, "rms_fwd")
    return y, rstd


def add_rms_fwd(x, residual, w=None, eps=1e-6, *, residual_out=None, out=None, rstd=None,
                want_stats=False, stream=None):
    """residual_out = x + residual (rounded to x.dtype); y = RMSNorm(residual_out, w).
    Returns (residual_out, y, rstd or None).  Pass residual_out=residual to update
    the residual stream in place."""
    rows, n, ldx = _rows(x, "x")
    ldr = _same_rows(residual, x, "residual")
    w = _param(w, n, x.dtype, x.device, "w")
    ro = torch.empty(x.shape, device=x.device, dtype=x.dtype) if residual_out is None else residual_out
    ldro = _same_rows(ro, x, "residual_out")
    y = torch.empty(x.shape, device=x.device, dtype=x.dtype) if out is None else out
    ldy = _same_rows(y, x, "out")
    if want_stats and rstd is None:
        rstd = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32)
    with torch.cuda.device(x.device):
        st = lib().add_rms_fwd_ld(_ptr(x), ldx, _ptr(residual), ldr, _ptr(w), _ptr(ro), ldro,
                                  _ptr(y), ldy, _ptr(rstd), rows, n, eps, _dtype_code(x),
                                  stream if stream is not None else _stream(x.device))
    _check(st, "add_rms_fwd")
    return ro, y, rstd


def add_rms_fwd_host_workspace(n, dtype, device=None):
    """Device staging buffer for add_rms_fwd_host on rows of length n."""
    nbytes = lib().add_rms_fwd_host_workspace_size(n, _DT[dtype])
    return torch.empty(max(nbytes, 256), dtype=torch.uint8,
                       device=device if device is not None else torch.device("cuda"))


def add_rms_fwd_host(x, residual, w=None, eps=1e-6, *, residual_out=None, out=None, rstd=None,
                     workspace=None, stream=None, synchronize=True):
    """add_rms_fwd on HOST tensors (pinned memory is fastest), streamed through
    the current device in chunks.  w and rstd are device tensors.  Returns
    (residual_out, y); with synchronize=False they are complete only once the
    stream is."""
    if x.is_cuda or residual.is_cuda:
        raise ValueError("x and residual must be host tensors")
    if not (x.is_contiguous() and residual.is_contiguous()):
        raise ValueError("x and residual must be contiguous")
    if residual.shape != x.shape or residual.dtype != x.dtype:
        raise ValueError("residual must match x in shape and dtype")
    rows, n = _rows_view(x)
    device = torch.device("cuda", torch.cuda.current_device())
    w = _param(w, n, x.dtype, device, "w")
    ro = torch.empty_like(x) if residual_out is None else residual_out
    y = torch.empty_like(x) if out is None else out
    for t, name in ((ro, "residual_out"), (y, "out")):
        if t.is_cuda or not t.is_contiguous() or t.shape != x.shape or t.dtype != x.dtype:
            raise ValueError(f"{name} must be a contiguous host tensor like x")
    ws = add_rms_fwd_host_workspace(n, x.dtype, device) if workspace is None else workspace
    s = stream if stream is not None else _stream(device)
    st = lib().add_rms_fwd_host(_ptr(x), _ptr(residual), _ptr(w), _ptr(ro), _ptr(y), _ptr(rstd),
                                rows, n, eps, _dtype_code(x), _ptr(ws),
                                ws.numel() * ws.element_size(), s)
    _check(st, "add_rms_fwd_host")
    if synchronize:
        torch.cuda.current_stream(device).synchronize() if stream is None else \
            torch.cuda.synchronize(device)
    return ro, y


def bn_fwd_train_workspace_size(batch, c, hw, dtype=torch.float32) -> int:
    return lib().bn_fwd_train_workspace_size(batch, c, hw, _DT[dtype])


def _bn_train_tensors(x, gamma, beta, running_mean, running_var, out, save_mean, save_rstd):
    """Checks shared by both training-forward entry points; allocates the
    outputs that are None.  Returns (batch, c, hw, gamma, beta, y, save_mean,
    save_rstd)."""
    _cuda(x, "x")
    if x.dim() < 2:
        raise ValueError("x must be [batch, C, ...]")
    batch, c = x.shape[0], x.shape[1]
    hw = x.numel() // (batch * c) if batch * c else 0
    gamma = _param(gamma, c, x.dtype, x.device, "gamma")
    beta = _param(beta, c, x.dtype, x.device, "beta")
    for t, name in ((running_mean, "running_mean"), (running_var, "running_var"),
                    (save_mean, "save_mean"), (save_rstd, "save_rstd")):
        if t is not None:
            _cuda(t, name)
            if t.dtype != torch.float32 or t.numel() != c or t.device != x.device:
                raise ValueError(f"{name} must be [{c}] float32 on {x.device}")
    if out is not None:
        _cuda(out, "out")
        if out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
            raise ValueError("out must be like x")
    y = torch.empty_like(x) if out is None else out
    save_mean = torch.empty(c, device=x.device, dtype=torch.float32) if save_mean is None else save_mean
    save_rstd = torch.empty(c, device=x.device, dtype=torch.float32) if save_rstd is None else save_rstd
    return batch, c, hw, gamma, beta, y, save_mean, save_rstd


def bn_fwd_train(x, gamma=None, beta=None, running_mean=None, running_var=None, eps=1e-5,
                 momentum=0.1, *, out=None, save_mean=None, save_rstd=None, workspace=None,
                 stream=None):
    """BatchNorm2d training forward over NCHW x.  Returns (y, save_mean, save_rstd);
    running_mean / running_var (binary32) are updated in place when given."""
    batch, c, hw, gamma, beta, y, save_mean, save_rstd = _bn_train_tensors(
        x, gamma, beta, running_mean, running_var, out, save_mean, save_rstd)
    need = lib().bn_fwd_train_workspace_size(batch, c, hw, _dtype_code(x))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=x.device, dtype=torch.uint8)
    with torch.cuda.device(x.device):
        st = lib().bn_fwd_train(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(save_mean),
                                _ptr(save_rstd), _ptr(running_mean), _ptr(running_var), batch, c,
                                hw, eps, momentum, _dtype_code(x), _ptr(workspace),
                                workspace.numel() * workspace.element_size(),
                                stream if stream is not None else _stream(x.device))
    _check(st, "bn_fwd_train")
    return y, save_mean, save_rstd


def bn_fwd_train_noalloc(x, gamma=None, beta=None, running_mean=None, running_var=None,
                         eps=1e-5, momentum=0.1, *, out, save_mean, save_rstd, stream=None):
    """bn_fwd_train for callers that cannot allocate device memory at call time:
    every output is passed in (same checks as bn_fwd_train), and the library
    keeps the partial statistics in a fixed array of its own (batch * C <=
    65536).  Returns (y, save_mean, save_rstd)."""
    if out is None or save_mean is None or save_rstd is None:
        raise ValueError("bn_fwd_train_noalloc allocates nothing: pass out, save_mean and save_rstd")
    batch, c, hw, gamma, beta, y, save_mean, save_rstd = _bn_train_tensors(
        x, gamma, beta, running_mean, running_var, out, save_mean, save_rstd)
    with torch.cuda.device(x.device):
        st = lib().bn_fwd_train_noalloc(
            _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(save_mean), _ptr(save_rstd),
            _ptr(running_mean), _ptr(running_var), batch, c, hw, eps, momentum, _dtype_code(x),
            stream if stream is not None else _stream(x.device))
    _check(st, "bn_fwd_train_noalloc")
    return y, save_mean, save_rstd


def softmax_fwd(x, *, out=None, row_max=None, row_sum=None, want_stats=False, stream=None):
    """Softmax over the last dimension of x.  Returns (y, row_max, row_sum);
    the statistics are None unless requested or passed in."""
    rows, n, ldx = _rows(x, "x")
    y = torch.empty(x.shape, device=x.device, dtype=x.dtype) if out is None else out
    ldy = _same_rows(y, x, "out")
    if want_stats:
        if row_max is None:
            row_max = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32)
        if row_sum is None:
            row_sum = torch.empty(x.shape[:-1], device=x.device, dtype=torch.float32)
    with torch.cuda.device(x.device):
        st = lib().softmax_fwd_ld(_ptr(x), ldx, _ptr(y), ldy, _ptr(row_max), _ptr(row_sum),
                                  rows, n, _dtype_code(x),
                                  stream if stream is not None else _stream(x.device))
    _check(st, "softmax_fwd")
    return y, row_max, row_sum


def _nchw(x):
    _cuda(x, "x")
    if x.dim() < 2:
        raise ValueError("x must be [batch, C, ...]")
    batch, c = x.shape[0], x.shape[1]
    hw = 1
    for d in x.shape[2:]:
        hw *= d
    return batch, c, hw


def _stat(t, c, device, name):
    _cuda(t, name)
    if t.dtype != torch.float32 or t.numel() != c or t.device != device:
        raise ValueError(f"{name} must be [{c}] float32 on {device}")
    return t


def bn_fwd_infer(x, running_mean, running_var, gamma=None, beta=None, eps=1e-5, *, out=None,
                 stream=None):
    """BatchNorm2d inference forward over NCHW x with the running statistics.
    Returns y."""
    batch, c, hw = _nchw(x)
    gamma = _param(gamma, c, x.dtype, x.device, "gamma")
    beta = _param(beta, c, x.dtype, x.device, "beta")
    running_mean = _stat(running_mean, c, x.device, "running_mean")
    running_var = _stat(running_var, c, x.device, "running_var")
    y = torch.empty_like(x) if out is None else out
    with torch.cuda.device(x.device):
        st = lib().bn_fwd_infer(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(running_mean),
                                _ptr(running_var), batch, c, hw, eps, _dtype_code(x),
                                stream if stream is not None else _stream(x.device))
    _check(st, "bn_fwd_infer")
    return y


def bn_bwd_workspace_size(batch, c, hw, dtype=torch.float32) -> int:
    return lib().bn_bwd_workspace_size(batch, c, hw, _DT[dtype])


def bn_bwd(dy, x, save_mean, save_rstd, gamma=None, *, out=None, dgamma=None, dbeta=None,
           workspace=None, stream=None):
    """BatchNorm2d training backward over NCHW tensors, from the statistics the
    training forward saved.  Returns (dx, dgamma, dbeta)."""
    batch, c, hw = _nchw(x)
    _cuda(dy, "dy")
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must match x in shape and dtype")
    gamma = _param(gamma, c, x.dtype, x.device, "gamma")
    save_mean = _stat(save_mean, c, x.device, "save_mean")
    save_rstd = _stat(save_rstd, c, x.device, "save_rstd")
    dx = torch.empty_like(x) if out is None else out
    dgamma = torch.empty(c, device=x.device, dtype=torch.float32) if dgamma is None else dgamma
    dbeta = torch.empty(c, device=x.device, dtype=torch.float32) if dbeta is None else dbeta
    need = lib().bn_bwd_workspace_size(batch, c, hw, _dtype_code(x))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=x.device, dtype=torch.uint8)
    with torch.cuda.device(x.device):
        st = lib().bn_bwd(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(save_mean), _ptr(save_rstd),
                          _ptr(dx), _ptr(dgamma), _ptr(dbeta), batch, c, hw, _dtype_code(x),
                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                          stream if stream is not None else _stream(x.device))
    _check(st, "bn_bwd")
    return dx, dgamma, dbeta


def _scratch(batch, c, hw, dtype, device, workspace):
    need = max(lib().bn_fwd_train_workspace_size(batch, c, hw, _DT[dtype]), 16)
    if workspace is None:
        return torch.empty(need, device=device, dtype=torch.uint8)
    return workspace


def bn_fwd_partial_stats(x, *, out=None, workspace=None, stream=None):
    """Per-channel (count, mean, M2) of this process's batch, [C, 3] float64."""
    batch, c, hw = _nchw(x)
    stats = torch.empty(c, 3, device=x.device, dtype=torch.float64) if out is None else out
    ws = _scratch(batch, c, hw, x.dtype, x.device, workspace)
    with torch.cuda.device(x.device):
        st = lib().bn_fwd_partial_stats(_ptr(x), _ptr(stats), batch, c, hw, _dtype_code(x),
                                        _ptr(ws), ws.numel() * ws.element_size(),
                                        stream if stream is not None else _stream(x.device))
    _check(st, "bn_fwd_partial_stats")
    return stats


def bn_fwd_apply_stats(x, parts, gamma=None, beta=None, running_mean=None, running_var=None,
                       eps=1e-5, momentum=0.1, *, out=None, save_mean=None, save_rstd=None,
                       stream=None):
    """Training forward of the local batch from the exchanged [nparts, C, 3]
    float64 statistics.  Returns (y, save_mean, save_rstd)."""
    batch, c, hw = _nchw(x)
    if parts.dtype != torch.float64 or parts.dim() != 3 or parts.shape[1:] != (c, 3):
        raise ValueError(f"parts must be [nparts, {c}, 3] float64")
    _cuda(parts, "parts")
    gamma = _param(gamma, c, x.dtype, x.device, "gamma")
    beta = _param(beta, c, x.dtype, x.device, "beta")
    y = torch.empty_like(x) if out is None else out
    save_mean = torch.empty(c, device=x.device, dtype=torch.float32) if save_mean is None else save_mean
    save_rstd = torch.empty(c, device=x.device, dtype=torch.float32) if save_rstd is None else save_rstd
    with torch.cuda.device(x.device):
        st = lib().bn_fwd_apply_stats(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(parts),
                                      parts.shape[0], _ptr(save_mean), _ptr(save_rstd),
                                      _ptr(running_mean), _ptr(running_var), batch, c, hw, eps,
                                      momentum, _dtype_code(x),
                                      stream if stream is not None else _stream(x.device))
    _check(st, "bn_fwd_apply_stats")
    return y, save_mean, save_rstd


def bn_bwd_partial_sums(dy, x, save_mean, save_rstd, *, out=None, workspace=None, stream=None):
    """Per-channel (sum dy, sum dy * xhat) of this process's batch, [C, 2] float64."""
    batch, c, hw = _nchw(x)
    _cuda(dy, "dy")
    sums = torch.empty(c, 2, device=x.device, dtype=torch.float64) if out is None else out
    ws = _scratch(batch, c, hw, x.dtype, x.device, workspace)
    with torch.cuda.device(x.device):
        st = lib().bn_bwd_partial_sums(_ptr(dy), _ptr(x), _ptr(save_mean), _ptr(save_rstd),
                                       _ptr(sums), batch, c, hw, _dtype_code(x), _ptr(ws),
                                       ws.numel() * ws.element_size(),
                                       stream if stream is not None else _stream(x.device))
    _check(st, "bn_bwd_partial_sums")
    return sums


def bn_bwd_apply_sums(dy, x, save_mean, save_rstd, parts, count, gamma=None, *, out=None,
                      dgamma=None, dbeta=None, stream=None):
    """Backward of the local batch from the exchanged [nparts, C, 2] float64
    sums and the global count.  Returns (dx, dgamma, dbeta)."""
    batch, c, hw = _nchw(x)
    _cuda(dy, "dy")
    if parts.dtype != torch.float64 or parts.dim() != 3 or parts.shape[1:] != (c, 2):
        raise ValueError(f"parts must be [nparts, {c}, 2] float64")
    gamma = _param(gamma, c, x.dtype, x.device, "gamma")
    dx = torch.empty_like(x) if out is None else out
    dgamma = torch.empty(c, device=x.device, dtype=torch.float32) if dgamma is None else dgamma
    dbeta = torch.empty(c, device=x.device, dtype=torch.float32) if dbeta is None else dbeta
    with torch.cuda.device(x.device):
        st = lib().bn_bwd_apply_sums(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(save_mean),
                                     _ptr(save_rstd), _ptr(parts), parts.shape[0], count,
                                     _ptr(dx), _ptr(dgamma), _ptr(dbeta), batch, c, hw,
                                     _dtype_code(x),
                                     stream if stream is not None else _stream(x.device))
    _check(st, "bn_bwd_apply_sums")
    return dx, dgamma, dbeta


# ---------------------------------------------------------------------------
# Training operators.
# ---------------------------------------------------------------------------
def _on_stream(stream, t):
    """Context in which everything that a call allocates and launches belongs
    to `stream` (a raw stream handle or a torch stream)."""
    if not t.is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=t.device)
    return torch.cuda.stream(stream)


# These calls take 10 to 20 us of kernel at ordinary sizes, so their checks are
# written for few attribute reads (0.1 us each): shape, type and device index
# are taken from the first tensor once.
_F32 = torch.float32
# The current stream's handle and the current device as integers, without
# building Stream and device objects (3 us a call on a Grace core).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _stream
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_fns = {}


def _launch(name, dev, *args):
    """One C call on the current stream of device number `dev`."""
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = getattr(lib(), name)
    if dev == _current():
        st = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = f(*args, _raw_stream(dev))
    if st != 0:
        raise NrmError(st, name)


def _code(dtype):
    code = _DT.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _match(t, shape, dtype, dev, name):
    """Row stride of a tensor that has to be like the first one."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype} on device {dev}")
    return shape[-1] if t.is_contiguous() else _rows(t, name)[2]


def _like(t, x, shape, dtype, dev, name):
    """`t`, or a new contiguous tensor like x; and its row stride."""
    if t is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format), shape[-1]
    return t, _match(t, shape, dtype, dev, name)


def _flat(t, shape, dtype, dev, name):
    """A contiguous tensor of exactly this shape and type."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on device {dev}")
    return t


def _weight(w, n, dtype, dev, name):
    if w is not None and (w.dtype is not dtype or w.get_device() != dev or w.numel() != n or not w.is_contiguous()):
        raise ValueError(f"{name} must be contiguous [{n}] {dtype} on device {dev}")
    return w


def _one_value(t, dtype, dev, name):
    """Address of one value on the device, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.numel() != 1:
        raise ValueError(f"{name} must be one {dtype} value on device {dev}")
    return t.data_ptr()


def _scratch_bytes(workspace, need, x):
    """Address and size of a workspace, and what keeps it alive."""
    if workspace is None:
        workspace = torch.empty(need if need > 16 else 16, dtype=torch.uint8, device=x.device)
    elif workspace.get_device() != x.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the tensors' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


_M64 = 0xFFFFFFFFFFFFFFFF


def dropout_fwd(x, p, seed, offset=0, *, out=None, offset_dev=None, stream=None):
    """Dropout over x as rows of its last dimension: y = x / (1 - p) where the
    mask of (seed, offset, row, column) keeps the element, +0 elsewhere; p is
    rounded to a multiple of 2^-16.  seed and offset are integers (modulo
    2^64); offset_dev, an int64 tensor of one element, is added to offset when
    the kernel runs.  out may be x.  Returns y."""
    if stream is not None:
        with _on_stream(stream, x):
            return dropout_fwd(x, p, seed, offset, out=out, offset_dev=offset_dev)
    rows, n, ldx = _rows(x, "x")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    code = _code(dtype)
    y, ldy = _like(out, x, shape, dtype, dev, "out")
    _launch("dropout_fwd_ld", dev, x.data_ptr(), ldx, y.data_ptr(), ldy, rows, n, p, seed & _M64,
            offset & _M64, _one_value(offset_dev, torch.int64, dev, "offset_dev"), code)
    return y


def dropout_bwd(dy, p, seed, offset=0, *, out=None, offset_dev=None, stream=None):
    """Gradient of dropout_fwd: the same places of dy dropped, the rest scaled.
    Returns dx."""
    return dropout_fwd(dy, p, seed, offset, out=out, offset_dev=offset_dev, stream=stream)


def dropout_add_rms_fwd(x, residual, w=None, p=0.0, seed=0, offset=0, eps=1e-6, *,
                        residual_out=None, out=None, rstd=None, offset_dev=None, stream=None):
    """residual_out = residual + dropout(x) (rounded to x.dtype); y =
    RMSNorm(residual_out, w).  Returns (residual_out, y, rstd); the backward
    takes residual_out and rstd.  Pass residual_out=residual to update the
    residual stream in place."""
    if stream is not None:
        with _on_stream(stream, x):
            return dropout_add_rms_fwd(x, residual, w, p, seed, offset, eps,
                                       residual_out=residual_out, out=out, rstd=rstd,
                                       offset_dev=offset_dev)
    rows, n, ldx = _rows(x, "x")
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    code = _code(dtype)
    ldr = _match(residual, shape, dtype, dev, "residual")
    w = _weight(w, n, dtype, dev, "w")
    ro, ldro = _like(residual_out, x, shape, dtype, dev, "residual_out")
    y, ldy = _like(out, x, shape, dtype, dev, "out")
    if rstd is None:
        rstd = torch.empty(shape[:-1], dtype=_F32, device=x.device)
    else:
        _flat(rstd, shape[:-1], _F32, dev, "rstd")
    _launch("dropout_add_rms_fwd_ld", dev, x.data_ptr(), ldx, residual.data_ptr(), ldr, _ptr(w),
            ro.data_ptr(), ldro, y.data_ptr(), ldy, rstd.data_ptr(), rows, n, p, seed & _M64,
            offset & _M64, _one_value(offset_dev, torch.int64, dev, "offset_dev"), eps, code)
    return ro, y, rstd


def dropout_add_rms_bwd_workspace_size(rows, n, dtype) -> int:
    return lib().dropout_add_rms_bwd_workspace_size(rows, n, _DT[dtype])


def dropout_add_rms_bwd(dy, residual_out, rstd, w=None, p=0.0, seed=0, offset=0, *,
                        dresidual_out=None, dx=None, dresidual=None, dw=None, want_dw=None,
                        workspace=None, offset_dev=None, stream=None):
    """Backward of dropout_add_rms_fwd (with p = 0 of add_rms_fwd and, with
    residual_out = x, of rms_fwd) from dy, the gradient of y, and optionally
    dresidual_out, the gradient of residual_out.  Returns (dx, dresidual, dw):
    dw is binary32, computed when w is given (or want_dw=True), else None.
    Without dropout (p = 0) and without a dx to write to, dx is dresidual, the
    same tensor.  dx=dy and dresidual=dresidual_out work in place."""
    if stream is not None:
        with _on_stream(stream, dy):
            return dropout_add_rms_bwd(dy, residual_out, rstd, w, p, seed, offset,
                                       dresidual_out=dresidual_out, dx=dx, dresidual=dresidual,
                                       dw=dw, want_dw=want_dw, workspace=workspace,
                                       offset_dev=offset_dev)
    rows, n, lddy = _rows(dy, "dy")
    shape, dtype, dev = dy.shape, dy.dtype, dy.get_device()
    code = _code(dtype)
    ldh = _match(residual_out, shape, dtype, dev, "residual_out")
    _flat(rstd, shape[:-1], _F32, dev, "rstd")
    w = _weight(w, n, dtype, dev, "w")
    ldu = n if dresidual_out is None else _match(dresidual_out, shape, dtype, dev, "dresidual_out")
    dresidual, lddr = _like(dresidual, dy, shape, dtype, dev, "dresidual")
    same = dx is None and p == 0
    if not same:
        dx, lddx = _like(dx, dy, shape, dtype, dev, "dx")
    if dw is not None:
        _weight(dw, n, _F32, dev, "dw")
    elif want_dw if want_dw is not None else w is not None:
        dw = torch.empty(n, dtype=_F32, device=dy.device)
    ws, wsb, workspace = _scratch_bytes(workspace, lib().dropout_add_rms_bwd_workspace_size(rows, n, code), dy)
    _launch("dropout_add_rms_bwd_ld", dev, dy.data_ptr(), lddy, residual_out.data_ptr(), ldh,
            rstd.data_ptr(), _ptr(w), _ptr(dresidual_out), ldu, None if same else dx.data_ptr(),
            n if same else lddx, dresidual.data_ptr(), lddr, _ptr(dw), rows, n, p, seed & _M64,
            offset & _M64, _one_value(offset_dev, torch.int64, dev, "offset_dev"), code, ws, wsb)
    return (dresidual if same else dx), dresidual, dw


def logprob_fwd(logits, targets, inv_temp=1.0, *, logp=None, lse=None, stats=None, stream=None):
    """Log-softmax of inv_temp * logits at one target (int64) per row of the
    last dimension.  Returns (logp, lse), binary32, one value per row; rows
    with a target outside [0, V) give 0 and are not read.  stats, a contiguous
    binary32 tensor of targets' shape and 2, takes each row's maximum and log
    sum exp(inv_temp * (logits - maximum)) for logprob_bwd."""
    if stream is not None:
        with _on_stream(stream, logits):
            return logprob_fwd(logits, targets, inv_temp, logp=logp, lse=lse, stats=stats)
    rows, v, ldl = _rows(logits, "logits")
    shape, dev = logits.shape[:-1], logits.get_device()
    code = _code(logits.dtype)
    _flat(targets, shape, torch.int64, dev, "targets")
    logp = torch.empty_like(targets, dtype=_F32) if logp is None else _flat(logp, shape, _F32, dev, "logp")
    lse = torch.empty_like(targets, dtype=_F32) if lse is None else _flat(lse, shape, _F32, dev, "lse")
    if stats is not None:
        _flat(stats, (*shape, 2), _F32, dev, "stats")
    _launch("logprob_fwd_stats_ld", dev, logits.data_ptr(), ldl, targets.data_ptr(), logp.data_ptr(),
            lse.data_ptr(), _ptr(stats), rows, v, inv_temp, code)
    return logp, lse


def logprob_bwd(dlogp, logits, targets, lse, inv_temp=1.0, *, stats=None, out=None, stream=None):
    """Gradient of the logits from dlogp, the gradient of logprob_fwd's logp
    (one binary32 value per row), and its lse, or its stats (then lse is not
    used and may be None).  lse's rounding is a factor of up to |lse| 2^-24 on
    its row (6e-4 at 1e4, and a row masked as a whole by the type's lowest value
    loses log V); stats have no such error.  out may be logits.  Returns
    dlogits."""
    if stream is not None:
        with _on_stream(stream, logits):
            return logprob_bwd(dlogp, logits, targets, lse, inv_temp, stats=stats, out=out)
    rows, v, ldl = _rows(logits, "logits")
    shape, dtype, dev = logits.shape, logits.dtype, logits.get_device()
    code = _code(dtype)
    per_row = shape[:-1]
    _flat(dlogp, per_row, _F32, dev, "dlogp")
    _flat(targets, per_row, torch.int64, dev, "targets")
    if stats is None:
        if lse is None:
            raise ValueError("lse or stats must be given")
        name, from_fwd = "logprob_bwd_ld", _flat(lse, per_row, _F32, dev, "lse")
    else:
        name, from_fwd = "logprob_bwd_stats_ld", _flat(stats, (*per_row, 2), _F32, dev, "stats")
    out, lddl = _like(out, logits, shape, dtype, dev, "out")
    _launch(name, dev, dlogp.data_ptr(), logits.data_ptr(), ldl, targets.data_ptr(),
            from_fwd.data_ptr(), out.data_ptr(), lddl, rows, v, inv_temp, code)
    return out


def policy_loss_workspace_size(rows) -> int:
    return lib().policy_loss_workspace_size(rows)


def policy_loss(logits, targets, old_logp, advantages, weights=None, ref_logp=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, inv_temp=1.0, *, grad_scale=None, want_grad=True,
                out=None, logp=None, workspace=None, stream=None):
    """Clipped policy loss with a KL term over token rows, and the gradient of
    the logits in the same pass.  Per row with a target in [0, V) and a weight
    other than 0, ratio = exp(logp - old_logp):
      max(-A ratio, -A clip(ratio, 1 - clip_low, 1 + clip_high))
        + kl_coef (exp(ref_logp - logp) - (ref_logp - logp) - 1)
    weighted and summed.  grad_scale (one binary32 value on the device)
    multiplies the gradient: the loss scale that binary16 gradients need, most
    of which are below 2^-24 at weights of 1 / rows and a large vocabulary.  out, the gradient's tensor, may be logits;
    want_grad=False computes the loss only.  Returns (loss, logp, dlogits or
    None)."""
    if stream is not None:
        with _on_stream(stream, logits):
            return policy_loss(logits, targets, old_logp, advantages, weights, ref_logp, clip_low,
                               clip_high, kl_coef, inv_temp, grad_scale=grad_scale,
                               want_grad=want_grad, out=out, logp=logp, workspace=workspace)
    rows, v, ldl = _rows(logits, "logits")
    shape, dtype, dev = logits.shape, logits.dtype, logits.get_device()
    code = _code(dtype)
    per_row = shape[:-1]
    _flat(targets, per_row, torch.int64, dev, "targets")
    _flat(old_logp, per_row, _F32, dev, "old_logp")
    _flat(advantages, per_row, _F32, dev, "advantages")
    if weights is not None:
        _flat(weights, per_row, _F32, dev, "weights")
    if ref_logp is not None:
        _flat(ref_logp, per_row, _F32, dev, "ref_logp")
    logp = torch.empty_like(targets, dtype=_F32) if logp is None else _flat(logp, per_row, _F32, dev, "logp")
    loss = torch.empty((), dtype=_F32, device=logits.device)
    lddl = v
    if want_grad or out is not None:
        out, lddl = _like(out, logits, shape, dtype, dev, "out")
    ws, wsb, workspace = _scratch_bytes(workspace, 4 * rows + 16, logits)
    _launch("policy_loss_ld", dev, logits.data_ptr(), ldl, targets.data_ptr(), old_logp.data_ptr(),
            advantages.data_ptr(), _ptr(weights), _ptr(ref_logp), clip_low, clip_high, kl_coef,
            inv_temp, _one_value(grad_scale, _F32, dev, "grad_scale"), loss.data_ptr(),
            logp.data_ptr(), _ptr(out), lddl, rows, v, code, ws, wsb)
    return loss, logp, out


# ---------------------------------------------------------------------------
# Inside a block: head norms with the position rotation.
# ---------------------------------------------------------------------------
def _heads(t, shape, dtype, dev, name):
    """(token stride, head stride) of a tensor [..., heads, D] whose leading
    dimensions have one stride between tokens."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype} on device {dev}")
    st = t.stride()
    if len(st) == 3 and st[2] == 1:
        return st[0], st[1]
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"the entries of a head of {name} must be contiguous")
    if 0 in shape[:-2]:
        return 0, st[-2]  # no tokens: no stride is used
    step, n = None, 1
    for d in range(t.dim() - 3, -1, -1):
        if shape[d] == 1:
            continue
        if step is None:
            step, n = st[d], shape[d]
        elif st[d] == step * n:
            n *= shape[d]
        else:
            raise ValueError(f"the tokens of {name} must have one stride")
    return step or 0, st[-2]


def _qk_sizes(q, k, table, positions, wq, wk):
    """Checks of what both directions take.  Returns (shape of q, shape of k or None,
    dtype code, dtype, device index, tokens, q_heads, k_heads, D, rot, max_pos)."""
    shape, dtype, dev = q.shape, q.dtype, q.get_device()
    if dev < 0:
        raise ValueError("q must be a CUDA tensor")
    code = _code(dtype)
    if len(shape) < 2:
        raise ValueError("q must be [..., heads, D]")
    hq, d = shape[-2:]
    lead = positions.shape
    if lead != shape[:-2]:
        raise ValueError(f"positions must be {tuple(shape[:-2])}")
    if positions.dtype is not torch.int64 or positions.get_device() != dev or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous int64 tensor on device {dev}")
    most = table.shape
    if len(most) != 2 or table.dtype is not _F32 or table.get_device() != dev or not table.is_contiguous():
        raise ValueError(f"table must be a contiguous [positions, rotated entries] float32 tensor on device {dev}")
    _weight(wq, d, dtype, dev, "wq")
    kshape, hk = None, 0
    if k is not None:
        kshape = k.shape
        if len(kshape) != len(shape) or kshape[-1] != d or kshape[:-2] != lead:
            raise ValueError("k must be like q but for its heads")
        hk = kshape[-2]
        _weight(wk, d, dtype, dev, "wk")
    elif wk is not None:
        raise ValueError("wk without k")
    return shape, kshape, code, dtype, dev, positions.numel(), hq, hk, d, most[1], most[0]


def qk_norm_rope_fwd(q, k, table, positions, wq=None, wk=None, eps=1e-6, *, interleaved=False, q_out=None,
                     k_out=None, stream=None):
    """RMSNorm of each head of q [..., heads, D] and k [..., key heads, D] with
    weights wq and wk [D], then the position rotation of the first R entries by
    table [P, R] (binary32: R / 2 cosines, then R / 2 sines) at positions [...]
    (int64).  Pairs are (i, i + R / 2), interleaved (2i, 2i + 1).  q and k may be
    slices of one projection's output, k may be None.  Tokens whose position is
    outside [0, P) are not read and get zeros.  Returns (q_out, k_out); they may
    be q and k in place."""
    if stream is not None:
        with _on_stream(stream, q):
            return qk_norm_rope_fwd(q, k, table, positions, wq, wk, eps, interleaved=interleaved, q_out=q_out,
                                    k_out=k_out)
    shape, kshape, code, dtype, dev, tokens, hq, hk, d, rot, most = _qk_sizes(q, k, table, positions, wq, wk)
    qt, qh = _heads(q, shape, dtype, dev, "q")
    if q_out is None:
        q_out, qot, qoh = torch.empty(shape, dtype=dtype, device=q.device), hq * d, d
    else:
        qot, qoh = _heads(q_out, shape, dtype, dev, "q_out")
    kp = kop = None
    kt = kh = kot = koh = 0
    if kshape is not None:
        kp = k.data_ptr()
        kt, kh = _heads(k, kshape, dtype, dev, "k")
        if k_out is None:
            k_out, kot, koh = torch.empty(kshape, dtype=dtype, device=q.device), hk * d, d
        else:
            kot, koh = _heads(k_out, kshape, dtype, dev, "k_out")
        kop = k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    _launch("qk_norm_rope_fwd", dev, q.data_ptr(), qt, qh, kp, kt, kh, table.data_ptr(), positions.data_ptr(),
            None if wq is None else wq.data_ptr(), None if wk is None else wk.data_ptr(), q_out.data_ptr(), qot, qoh, kop,
            kot, koh, tokens, hq, hk, d, rot, most, eps, 1 if interleaved else 0, code)
    return q_out, k_out


def qk_norm_rope_bwd_workspace_size(tokens, q_heads, k_heads, d) -> int:
    return lib().qk_norm_rope_bwd_workspace_size(tokens, q_heads, k_heads, d)


def qk_norm_rope_bwd(dq_out, dk_out, q, k, table, positions, wq=None, wk=None, eps=1e-6, *, interleaved=False,
                     dq=None, dk=None, dwq=None, dwk=None, want_dw=None, workspace=None, stream=None):
    """Backward of qk_norm_rope_fwd from the gradients of q_out and k_out and
    the forward's other arguments.  Returns (dq, dk, dwq, dwk): the weights'
    gradients are binary32, computed for the weights that are given (want_dw:
    for both, or neither), else None.  dq and dk may be dq_out and dk_out, or q
    and k, in place."""
    if stream is not None:
        with _on_stream(stream, q):
            return qk_norm_rope_bwd(dq_out, dk_out, q, k, table, positions, wq, wk, eps, interleaved=interleaved, dq=dq,
                                    dk=dk, dwq=dwq, dwk=dwk, want_dw=want_dw, workspace=workspace)
    shape, kshape, code, dtype, dev, tokens, hq, hk, d, rot, most = _qk_sizes(q, k, table, positions, wq, wk)
    device = q.device
    qt, qh = _heads(q, shape, dtype, dev, "q")
    gqt, gqh = _heads(dq_out, shape, dtype, dev, "dq_out")
    if dq is None:
        dq, dqt, dqh = torch.empty(shape, dtype=dtype, device=device), hq * d, d
    else:
        dqt, dqh = _heads(dq, shape, dtype, dev, "dq")
    kp = gkp = dkp = None
    kt = kh = gkt = gkh = dkt = dkh = 0
    if kshape is not None:
        kt, kh = _heads(k, kshape, dtype, dev, "k")
        gkt, gkh = _heads(dk_out, kshape, dtype, dev, "dk_out")
        kp, gkp = k.data_ptr(), dk_out.data_ptr()
        if dk is None:
            dk, dkt, dkh = torch.empty(kshape, dtype=dtype, device=device), hk * d, d
        else:
            dkt, dkh = _heads(dk, kshape, dtype, dev, "dk")
        dkp = dk.data_ptr()
    elif dk_out is not None or dk is not None or dwk is not None:
        raise ValueError("gradients of k without k")
    if dwq is not None:
        _weight(dwq, d, _F32, dev, "dwq")
    elif want_dw if want_dw is not None else wq is not None:
        dwq = torch.empty(d, dtype=_F32, device=device)
    if dwk is not None:
        _weight(dwk, d, _F32, dev, "dwk")
    elif kshape is not None and (want_dw if want_dw is not None else wk is not None):
        dwk = torch.empty(d, dtype=_F32, device=device)
    ws, wsb = None, 0
    if dwq is not None or dwk is not None:
        ws, wsb, workspace = _scratch_bytes(workspace, qk_norm_rope_bwd_workspace_size(tokens, hq, hk, d), q)
    _launch("qk_norm_rope_bwd", dev, dq_out.data_ptr(), gqt, gqh, gkp, gkt, gkh, q.data_ptr(), qt, qh, kp, kt, kh,
            table.data_ptr(), positions.data_ptr(), None if wq is None else wq.data_ptr(),
            None if wk is None else wk.data_ptr(), dq.data_ptr(), dqt, dqh, dkp, dkt, dkh,
            None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(), tokens, hq, hk, d, rot, most,
            eps, 1 if interleaved else 0, code, ws, wsb)
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------------------
# Routing to experts.
# ---------------------------------------------------------------------------
_SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score):
    code = _SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {', '.join(_SCORES)}, not {score!r}")
    return code


def route_fwd(logits, k, bias=None, *, score="softmax", groups=1, top_groups=None, group_top=1, renormalize=True,
              scale=1.0, want_scores=False, weights=None, ids=None, scores=None, stream=None):
    """The k experts of each token of logits [..., experts] with the largest
    score + bias (bias binary32 [experts], ties: lowest index), score softmax or
    sigmoid of the logits; with top_groups < groups from the top_groups groups of
    neighbouring experts with the largest sums of their group_top best.  Their
    weights are scale * score, renormalized to a sum of scale.  Experts with a
    logit or bias of -inf are not available (none is where a softmax is NaN);
    places without one get id -1 and weight 0.  Returns (weights, ids, scores or
    None): binary32 and int64 [..., k], all scores in binary32 with want_scores."""
    if stream is not None:
        with _on_stream(stream, logits):
            return route_fwd(logits, k, bias, score=score, groups=groups, top_groups=top_groups, group_top=group_top,
                             renormalize=renormalize, scale=scale, want_scores=want_scores, weights=weights, ids=ids,
                             scores=scores)
    tokens, experts, ldl = _rows(logits, "logits")
    shape, dev = logits.shape, logits.get_device()
    code = _code(logits.dtype)
    _weight(bias, experts, _F32, dev, "bias")
    out = (*shape[:-1], k)
    device = logits.device
    weights = torch.empty(out, dtype=_F32, device=device) if weights is None else _flat(weights, out, _F32, dev, "weights")
    ids = torch.empty(out, dtype=torch.int64, device=device) if ids is None else _flat(ids, out, torch.int64, dev, "ids")
    if scores is not None:
        _flat(scores, shape, _F32, dev, "scores")
    elif want_scores:
        scores = torch.empty(shape, dtype=_F32, device=device)
    _launch("route_fwd", dev, logits.data_ptr(), ldl, _ptr(bias), weights.data_ptr(), ids.data_ptr(), _ptr(scores), tokens,
            experts, k, _score(score), groups, groups if top_groups is None else top_groups, group_top,
            1 if renormalize else 0, scale, code)
    return weights, ids, scores


def route_bwd(dweights, logits, ids, *, score="softmax", renormalize=True, scale=1.0, dscores=None, out=None,
              stream=None):
    """Gradient of the logits from dweights, the gradient of route_fwd's weights
    (binary32), its ids, and optionally dscores, the gradient of its scores
    (binary32, like logits).  out may be logits.  Returns dlogits."""
    if stream is not None:
        with _on_stream(stream, logits):
            return route_bwd(dweights, logits, ids, score=score, renormalize=renormalize, scale=scale, dscores=dscores,
                             out=out)
    tokens, experts, ldl = _rows(logits, "logits")
    shape, dtype, dev = logits.shape, logits.dtype, logits.get_device()
    code = _code(dtype)
    k = ids.shape[-1]
    per_token = (*shape[:-1], k)
    _flat(ids, per_token, torch.int64, dev, "ids")
    _flat(dweights, per_token, _F32, dev, "dweights")
    if dscores is not None:
        _flat(dscores, shape, _F32, dev, "dscores")
    out, lddl = _like(out, logits, shape, dtype, dev, "out")
    _launch("route_bwd", dev, dweights.data_ptr(), logits.data_ptr(), ldl, ids.data_ptr(), _ptr(dscores), out.data_ptr(),
            lddl, tokens, experts, k, _score(score), 1 if renormalize else 0, scale, code)
    return out


# ---------------------------------------------------------------------------
# Rows of logits with entropy and alternatives.
# ---------------------------------------------------------------------------
def logprob_top_fwd(logits, targets, k, inv_temp=1.0, *, logp=None, entropy=None, top_ids=None, top_logp=None,
                    stats=None, stream=None):
    """Log-softmax of inv_temp * logits at one target (int64) per row of the last
    dimension, the row's entropy and its k <= 32 largest logits (ties: lowest
    index first) with their log-probabilities, from one pass.  Returns (logp,
    entropy, top_ids, top_logp, stats): binary32 but for the ids, int64; stats
    [..., 2] is for logprob_top_bwd (and logprob_bwd).  Rows with a target
    outside [0, V) are not read: ids -1, all else 0.  Logits of -inf are no
    alternatives: places without one get id -1 and -inf."""
    if stream is not None:
        with _on_stream(stream, logits):
            return logprob_top_fwd(logits, targets, k, inv_temp, logp=logp, entropy=entropy, top_ids=top_ids,
                                   top_logp=top_logp, stats=stats)
    rows, v, ldl = _rows(logits, "logits")
    shape, dev, device = logits.shape[:-1], logits.get_device(), logits.device
    code = _code(logits.dtype)
    _flat(targets, shape, torch.int64, dev, "targets")
    many, two = (*shape, k), (*shape, 2)
    empty = torch.empty
    logp = empty(shape, dtype=_F32, device=device) if logp is None else _flat(logp, shape, _F32, dev, "logp")
    entropy = empty(shape, dtype=_F32, device=device) if entropy is None else _flat(entropy, shape, _F32, dev, "entropy")
    top_ids = empty(many, dtype=torch.int64, device=device) if top_ids is None else _flat(top_ids, many, torch.int64, dev, "top_ids")
    top_logp = empty(many, dtype=_F32, device=device) if top_logp is None else _flat(top_logp, many, _F32, dev, "top_logp")
    stats = empty(two, dtype=_F32, device=device) if stats is None else _flat(stats, two, _F32, dev, "stats")
    _launch("logprob_top_fwd_ld", dev, logits.data_ptr(), ldl, targets.data_ptr(), logp.data_ptr(), entropy.data_ptr(),
            top_ids.data_ptr(), top_logp.data_ptr(), stats.data_ptr(), rows, v, k, inv_temp, code)
    return logp, entropy, top_ids, top_logp, stats


def logprob_top_bwd(dlogp, dentropy, dtop_logp, logits, targets, stats, entropy=None, top_ids=None, inv_temp=1.0, *,
                    out=None, stream=None):
    """Gradient of the logits from dlogp, dentropy and dtop_logp, the gradients of
    logprob_top_fwd's outputs (binary32; each may be None, not all), and its stats,
    entropy (with dentropy) and top_ids (with dtop_logp; any ids of a row, those
    outside [0, V) have no part).  out may be logits.  Returns dlogits."""
    if stream is not None:
        with _on_stream(stream, logits):
            return logprob_top_bwd(dlogp, dentropy, dtop_logp, logits, targets, stats, entropy, top_ids, inv_temp, out=out)
    rows, v, ldl = _rows(logits, "logits")
    shape, dtype, dev = logits.shape, logits.dtype, logits.get_device()
    code = _code(dtype)
    per_row = shape[:-1]
    _flat(targets, per_row, torch.int64, dev, "targets")
    _flat(stats, (*per_row, 2), _F32, dev, "stats")
    if dlogp is not None:
        _flat(dlogp, per_row, _F32, dev, "dlogp")
    if dentropy is not None:
        if entropy is None:
            raise ValueError("dentropy needs entropy")
        _flat(dentropy, per_row, _F32, dev, "dentropy")
        _flat(entropy, per_row, _F32, dev, "entropy")
    k = 0
    if dtop_logp is not None:
        if top_ids is None:
            raise ValueError("dtop_logp needs top_ids")
        k = top_ids.shape[-1]
        _flat(top_ids, (*per_row, k), torch.int64, dev, "top_ids")
        _flat(dtop_logp, (*per_row, k), _F32, dev, "dtop_logp")
    out, lddl = _like(out, logits, shape, dtype, dev, "out")
    _launch("logprob_top_bwd_ld", dev, _ptr(dlogp), _ptr(dentropy), _ptr(dtop_logp), logits.data_ptr(), ldl,
            targets.data_ptr(), stats.data_ptr(), _ptr(entropy), _ptr(top_ids), out.data_ptr(), lddl, rows, v, k, inv_temp,
            code)
    return out


# ---------------------------------------------------------------------------
# Plan control (tests and measurements).
# ---------------------------------------------------------------------------
def force_plan(plan: int = PLAN_AUTO, threads: int = 0, packs: int = 0, stages: int = 0,
               groups: int = 0):
    _check(lib().nrm_force_plan(plan, threads, packs, stages, groups), "nrm_force_plan")


def last_plan():
    """(plan, threads, packs, stages, groups) of this thread's last row-operator call."""
    v = [_INT() for _ in range(5)]
    lib().nrm_last_plan(*[ctypes.byref(x) for x in v])
    return tuple(x.value for x in v)


def set_wait_limit(tries: int) -> int:
    return lib().nrm_set_wait_limit(tries)


def device_fault(clear: bool = True) -> int:
    """Fault bits recorded by kernels on the current device (synchronizes)."""
    v = ctypes.c_uint()
    _check(lib().nrm_device_fault(ctypes.byref(v), 1 if clear else 0), "nrm_device_fault")
    return v.value


def set_bn_group_bytes(nbytes: int) -> int:
    """Input bytes per channel group of the streaming BatchNorm plans (0: default)."""
    return lib().nrm_set_bn_group_bytes(nbytes)


def set_pointer_checks(enable: bool) -> bool:
    return bool(lib().nrm_set_pointer_checks(1 if enable else 0))
