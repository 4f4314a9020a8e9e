"""Thin ctypes binding of libbstq.so (the C ABI in include/bstq.h).

Argument marshalling only: every step of the solve runs in the CUDA library.
PyTorch supplies device memory and streams.  Importing works without a GPU;
calling into the library without libbstq.so raises, there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbstq.so")

F32, F64, BF16, F16 = 0, 1, 2, 3
JOBZ_N, JOBZ_V = 0, 1
SCHED_AUTO, SCHED_FLAT, SCHED_NESTED = 0, 1, 2
QSTORE_AUTO, QSTORE_REGISTERS, QSTORE_SHARED, QSTORE_GLOBAL, QSTORE_HYBRID, QSTORE_SPLIT, QSTORE_LOG = 0, 1, 2, 3, 4, 5, 6
KERNEL_AUTO, KERNEL_STATIC, KERNEL_DYNAMIC = 0, 1, 2
UPDATE_EXP, UPDATE_PG = 0, 1
ERR_CUDA, ERR_NODEVICE = 1, 2
MAX_N = 128

# Every symbol include/bstq.h declares.
EXPORTS = ("bstq_work_size", "bstq_work_size_ex", "bstq_solve", "bstq_solve_ex",
           "bstq_host_work_size", "bstq_solve_host", "bstq_describe",
           "bstq_status_string", "bstq_version", "bstq_last_error", "bstq_solve_noalloc",
           "bstq_syev_work_size", "bstq_syev", "bstq_stedc_leaves_work_size", "bstq_stedc_leaves",
           "bstq_diag_work_size", "bstq_diag",
           "bstq_recur_work_size", "bstq_recur", "bstq_recur_grad_work_size", "bstq_recur_grad",
           "bstq_recur_step", "bstq_orthogonalize_work_size", "bstq_orthogonalize", "bstq_set_wait_limit")

# Diagnostic ops (bstq_diag): one building block of the solve on a table of
# inputs; values in and out per record.
DIAG_RCP, DIAG_DIV, DIAG_SQRT, DIAG_RSQRT, DIAG_HYP1 = 1, 2, 3, 4, 5
DIAG_LARTG, DIAG_LARTG_FAST, DIAG_SHIFT = 6, 7, 8
DIAG_PASS_STATIC, DIAG_PASS_DYN_EXP, DIAG_PASS_DYN_PG = 20, 21, 22
DIAG_FASTQ = 30
DIAG_SHAPE = {DIAG_RCP: (1, 1), DIAG_DIV: (2, 1), DIAG_SQRT: (1, 1), DIAG_RSQRT: (1, 1), DIAG_HYP1: (1, 1),
              DIAG_LARTG: (2, 3), DIAG_LARTG_FAST: (2, 3), DIAG_SHIFT: (3, 4),
              DIAG_PASS_STATIC: (42, 288), DIAG_PASS_DYN_EXP: (42, 288), DIAG_PASS_DYN_PG: (42, 288)}


class Params(ctypes.Structure):
    """bstq_params; all-zero means the defaults."""
    _fields_ = [("no_sort", ctypes.c_int), ("max_sweeps_per_n", ctypes.c_int),
                ("scheduler", ctypes.c_int), ("qstore", ctypes.c_int),
                ("threads_per_block", ctypes.c_int), ("kernel", ctypes.c_int),
                ("back_transform", ctypes.c_int), ("update_scheme", ctypes.c_int),
                ("log_entries", ctypes.c_int)]


class BstqError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        extra = ""
        if code == ERR_CUDA:
            extra = ": " + load().bstq_last_error().decode()
        super().__init__(f"{where}: {status_string(code)} (code {code}){extra}")


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load libbstq.so (built by symmetric_tridiagonal_eigensolver_gb300.build)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise ImportError(f"libbstq.so not found at {path}; run "
                              "`python -c 'import __graft_entry__ as g; g.build()'` first")
        lib = ctypes.CDLL(path)
        vp, sz, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
        P = ctypes.POINTER(Params)
        lib.bstq_work_size.restype = sz
        lib.bstq_work_size.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64]
        lib.bstq_work_size_ex.restype = sz
        lib.bstq_work_size_ex.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, P]
        lib.bstq_solve.restype = ctypes.c_int
        lib.bstq_solve.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, vp, vp, vp, vp, vp]
        lib.bstq_solve_ex.restype = ctypes.c_int
        lib.bstq_solve_ex.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, vp, vp, vp, vp, vp, P]
        lib.bstq_host_work_size.restype = sz
        lib.bstq_host_work_size.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, P]
        lib.bstq_solve_host.restype = ctypes.c_int
        lib.bstq_solve_host.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, vp, vp, vp, vp,
                                        vp, vp, P]
        lib.bstq_describe.restype = ctypes.c_int
        lib.bstq_describe.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, P,
                                      ctypes.c_char_p, sz]
        lib.bstq_status_string.restype = ctypes.c_char_p
        lib.bstq_status_string.argtypes = [ctypes.c_int]
        lib.bstq_version.restype = ctypes.c_char_p
        lib.bstq_version.argtypes = []
        lib.bstq_last_error.restype = ctypes.c_char_p
        lib.bstq_last_error.argtypes = []
        lib.bstq_syev_work_size.restype = sz
        lib.bstq_syev_work_size.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, P]
        lib.bstq_syev.restype = ctypes.c_int
        lib.bstq_syev.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, vp, vp, vp, vp, vp, P]
        lib.bstq_stedc_leaves_work_size.restype = sz
        lib.bstq_stedc_leaves_work_size.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, P]
        lib.bstq_stedc_leaves.restype = ctypes.c_int
        lib.bstq_stedc_leaves.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, vp, vp, vp,
                                          vp, vp, vp, P]
        lib.bstq_diag_work_size.restype = sz
        lib.bstq_diag_work_size.argtypes = [ctypes.c_int, ctypes.c_int, i64]
        lib.bstq_diag.restype = ctypes.c_int
        lib.bstq_diag.argtypes = [ctypes.c_int, ctypes.c_int, i64, ctypes.c_int, vp, vp, vp, vp]
        lib.bstq_solve_noalloc.restype = ctypes.c_int
        lib.bstq_solve_noalloc.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, vp, vp, vp, vp,
                                           vp, P]
        c_int = ctypes.c_int
        lib.bstq_set_wait_limit.restype = i64
        lib.bstq_set_wait_limit.argtypes = [i64]
        lib.bstq_recur_work_size.restype = sz
        lib.bstq_recur_work_size.argtypes = [c_int, i64, i64, i64]
        lib.bstq_recur.restype = c_int
        lib.bstq_recur.argtypes = [c_int, i64, i64, i64] + [vp] * 10
        lib.bstq_recur_grad_work_size.restype = sz
        lib.bstq_recur_grad_work_size.argtypes = [c_int, i64, i64, i64]
        lib.bstq_recur_grad.restype = c_int
        lib.bstq_recur_grad.argtypes = [c_int, i64, i64, i64] + [vp] * 15
        lib.bstq_recur_step.restype = c_int
        lib.bstq_recur_step.argtypes = [c_int, i64, i64, i64, vp, i64] + [vp] * 7
        lib.bstq_orthogonalize_work_size.restype = sz
        lib.bstq_orthogonalize_work_size.argtypes = [c_int, i64, i64, i64]
        lib.bstq_orthogonalize.restype = c_int
        lib.bstq_orthogonalize.argtypes = [c_int, i64, i64, i64, vp, vp, vp, c_int, vp, vp, vp]
        _lib = lib
        return lib


def _params(no_sort=False, max_sweeps_per_n=0, scheduler=0, qstore=0, threads_per_block=0, kernel=0,
            back_transform=False, update_scheme=0, log_entries=0):
    if isinstance(update_scheme, str):
        update_scheme = {"exp": UPDATE_EXP, "pg": UPDATE_PG}[update_scheme.lower()]
    return Params(int(bool(no_sort)), int(max_sweeps_per_n), int(scheduler), int(qstore),
                  int(threads_per_block), int(kernel), int(bool(back_transform)), int(update_scheme),
                  int(log_entries))


def _dtype_code(dt) -> int:
    import torch
    if dt in (torch.float32, np.float32):
        return F32
    if dt in (torch.float64, np.float64):
        return F64
    raise TypeError(f"bstq: dtype must be float32 or float64, got {dt}")


def status_string(code: int) -> str:
    return load().bstq_status_string(int(code)).decode()


def version() -> str:
    return load().bstq_version().decode()


def work_size(dtype, jobz: bool, n: int, batch: int, **params) -> int:
    code = _dtype_code(dtype)
    p = _params(**params)
    return int(load().bstq_work_size_ex(code, int(bool(jobz)), int(n), int(batch), ctypes.byref(p)))


def describe(dtype, jobz: bool, n: int, batch: int, **params) -> str:
    p = _params(**params)
    buf = ctypes.create_string_buffer(256)
    rc = load().bstq_describe(_dtype_code(dtype), int(bool(jobz)), int(n), int(batch),
                              ctypes.byref(p), buf, 256)
    if rc != 0:
        raise BstqError(rc, "bstq_describe")
    return buf.value.decode()


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def solve(d, e, jobz: bool = True, Q=None, work=None, stream=None, Z=None, **params):
    """Solve on CUDA tensors: ``d`` (batch, n) in/out (eigenvalues on exit),
    ``e`` (batch, n-1).  Returns (d, Q, info) where Q is (batch, n, n) with
    Q[b, :, j] the eigenvector of d[b, j] (None for jobz N) and info (batch,)
    int32.  With ``Z`` (batch, n, n) given, the rotations are right-applied to
    Z (back_transform) and the returned Q is Z times the eigenvectors; ``Q``
    given with ``back_transform=True`` is read as the basis in the library's
    storage layout (memory [b][j][i] = Z_ij).  Work is enqueued on ``stream``
    (default: torch's current stream); nothing is synchronised."""
    import torch
    if Z is not None:
        if not jobz:
            raise ValueError("bstq.solve: Z needs jobz = True")
        # storage layout of the library: memory [b][j][i] = Z_ij
        Q = Z.to(device=d.device, dtype=d.dtype).transpose(1, 2).contiguous()
        params["back_transform"] = True
    if not (d.is_cuda and d.is_contiguous()):
        raise ValueError("bstq.solve: d must be a contiguous CUDA tensor")
    if d.dim() != 2:
        raise ValueError("bstq.solve: d must be (batch, n)")
    batch, n = d.shape
    code = _dtype_code(d.dtype)
    if e is None or e.numel() == 0:
        e_ptr = None
    else:
        if not (e.is_cuda and e.is_contiguous() and e.dtype == d.dtype and e.numel() == batch * (n - 1)):
            raise ValueError("bstq.solve: e must be a contiguous CUDA tensor of d's dtype, (batch, n-1)")
        e_ptr = e.data_ptr()
    p = _params(**params)
    lib = load()
    wbytes = int(lib.bstq_work_size_ex(code, int(bool(jobz)), int(n), int(batch), ctypes.byref(p)))
    if wbytes == 0:
        raise BstqError(-10, "bstq_work_size_ex")
    if work is None:
        work = torch.empty(wbytes, dtype=torch.uint8, device=d.device)
    elif work.numel() * work.element_size() < wbytes:
        raise ValueError(f"bstq.solve: work needs {wbytes} bytes")
    if jobz and Q is None:
        Q = torch.empty((batch, n, n), dtype=d.dtype, device=d.device)
    # the library writes column-major per problem: memory [b][j][i] = Q_ij
    rc = lib.bstq_solve_ex(code, int(bool(jobz)), int(n), int(batch), d.data_ptr(), e_ptr,
                           Q.data_ptr() if jobz else None, work.data_ptr(), _stream_handle(stream),
                           ctypes.byref(p))
    if rc != 0:
        raise BstqError(rc, "bstq_solve_ex")
    info = work[: 4 * batch].view(torch.int32)
    Qout = Q.transpose(1, 2) if jobz else None
    return d, Qout, info


def host_work_size(dtype, jobz: bool, n: int, batch: int, **params) -> int:
    p = _params(**params)
    return int(load().bstq_host_work_size(_dtype_code(dtype), int(bool(jobz)), int(n), int(batch),
                                          ctypes.byref(p)))


def solve_host(h_d, h_e, h_Q, h_info, dev, stream=None, jobz: bool = True, **params):
    """End-to-end call on host buffers (pinned torch CPU tensors): copies in,
    solves and copies out on ``stream``; the caller synchronises."""
    batch, n = h_d.shape
    p = _params(**params)
    rc = load().bstq_solve_host(_dtype_code(h_d.dtype), int(bool(jobz)), int(n), int(batch),
                                h_d.data_ptr(), h_e.data_ptr() if h_e is not None and h_e.numel() else None,
                                h_Q.data_ptr() if jobz else None, h_info.data_ptr(), dev.data_ptr(),
                                _stream_handle(stream), ctypes.byref(p))
    if rc != 0:
        raise BstqError(rc, "bstq_solve_host")


def solve_noalloc(d, e, Q, info, stream=None, **params):
    """bstq_solve_noalloc on CUDA tensors (jobz = V): d (batch, n) in/out,
    e (batch, n-1), Q (batch, n, n) and info (batch,) int32 caller-owned; the
    eigenvector scratch is the library's fixed device array.  Returns
    (d, Q viewed with Q[b, :, j] the j-th eigenvector, info)."""
    batch, n = d.shape
    p = _params(**params)
    e_ptr = e.data_ptr() if e is not None and e.numel() else None
    rc = load().bstq_solve_noalloc(_dtype_code(d.dtype), JOBZ_V, int(n), int(batch), d.data_ptr(), e_ptr,
                                   Q.data_ptr(), info.data_ptr(), _stream_handle(stream), ctypes.byref(p))
    if rc != 0:
        raise BstqError(rc, "bstq_solve_noalloc")
    return d, Q.transpose(1, 2), info


def syev_work_size(dtype, jobz: bool, n: int, batch: int, **params) -> int:
    p = _params(**params)
    return int(load().bstq_syev_work_size(_dtype_code(dtype), int(bool(jobz)), int(n), int(batch),
                                          ctypes.byref(p)))


def syev(A, jobz: bool = True, work=None, stream=None, **params):
    """Fused small-n dense symmetric eigensolver on a CUDA tensor ``A``
    (batch, n, n), n <= 32, of which the lower triangle (A[b, i, j], i >= j)
    is read.  Returns (W, V, info): eigenvalues (batch, n) ascending,
    eigenvectors (batch, n, n) with V[b, :, j] that of W[b, j] (None for
    jobz N), info (batch,) int32.  Nothing is synchronised."""
    import torch
    if not A.is_cuda or A.dim() != 3 or A.shape[1] != A.shape[2]:
        raise ValueError("bstq.syev: A must be a (batch, n, n) CUDA tensor")
    batch, n, _ = A.shape
    code = _dtype_code(A.dtype)
    Ac = A.transpose(1, 2).contiguous()  # library layout: memory [b][j][i] = A_ij
    W = torch.empty((batch, n), dtype=A.dtype, device=A.device)
    Vs = torch.empty((batch, n, n), dtype=A.dtype, device=A.device) if jobz else None
    p = _params(**params)
    lib = load()
    wbytes = int(lib.bstq_syev_work_size(code, int(bool(jobz)), int(n), int(batch), ctypes.byref(p)))
    if wbytes == 0:
        raise BstqError(-10, "bstq_syev_work_size")
    if work is None:
        work = torch.empty(wbytes, dtype=torch.uint8, device=A.device)
    elif work.numel() * work.element_size() < wbytes:
        raise ValueError(f"bstq.syev: work needs {wbytes} bytes")
    rc = lib.bstq_syev(code, int(bool(jobz)), int(n), int(batch), Ac.data_ptr(), W.data_ptr(),
                       Vs.data_ptr() if jobz else None, work.data_ptr(), _stream_handle(stream), ctypes.byref(p))
    if rc != 0:
        raise BstqError(rc, "bstq_syev")
    info = work[: 4 * batch].view(torch.int32)
    return W, (Vs.transpose(1, 2) if jobz else None), info


def leaf_shape(n: int, leaf: int):
    """(L, F, t): the leaf size used, the number of full leaves and the rows
    of the shorter last leaf (0 if none), as bstq_stedc_leaves cuts a
    size-n problem."""
    L = min(int(leaf), int(n))
    return L, n // L, n % L


def stedc_leaves_work_size(dtype, jobz: bool, n: int, leaf: int, batch: int, **params) -> int:
    p = _params(**params)
    return int(load().bstq_stedc_leaves_work_size(_dtype_code(dtype), int(bool(jobz)), int(n), int(leaf),
                                                  int(batch), ctypes.byref(p)))


def stedc_leaves(d, e, leaf: int, jobz: bool = True, work=None, stream=None, **params):
    """Leaf solve of divide and conquer on CUDA tensors: ``d`` (batch, n)
    in/out, ``e`` (batch, n-1).  Each problem is torn into leaves of ``leaf``
    rows (the remainder last) and every leaf solved.  Returns (d, Qf, Qt,
    info): d holds each leaf's eigenvalues at its rows; Qf (batch, F, L, L)
    the full leaves' eigenvectors and Qt (batch, t, t) the last shorter
    leaf's (None if none), both with [..., :, j] the j-th eigenvector (None
    for jobz N); info (batch, leaves) int32.  Nothing is synchronised."""
    import torch
    if not (d.is_cuda and d.is_contiguous() and d.dim() == 2):
        raise ValueError("bstq.stedc_leaves: d must be a contiguous (batch, n) CUDA tensor")
    batch, n = d.shape
    code = _dtype_code(d.dtype)
    L, F, t = leaf_shape(n, leaf)
    e_ptr = None
    if n > 1:
        if not (e.is_cuda and e.is_contiguous() and e.dtype == d.dtype and e.numel() == batch * (n - 1)):
            raise ValueError("bstq.stedc_leaves: e must be a contiguous CUDA tensor of d's dtype, (batch, n-1)")
        e_ptr = e.data_ptr()
    p = _params(**params)
    lib = load()
    wbytes = int(lib.bstq_stedc_leaves_work_size(code, int(bool(jobz)), int(n), int(leaf), int(batch),
                                                 ctypes.byref(p)))
    if wbytes == 0:
        raise BstqError(-10, "bstq_stedc_leaves_work_size")
    if work is None:
        work = torch.empty(wbytes, dtype=torch.uint8, device=d.device)
    elif work.numel() * work.element_size() < wbytes:
        raise ValueError(f"bstq.stedc_leaves: work needs {wbytes} bytes")
    leaves = F + (1 if t else 0)
    info = torch.empty((batch, leaves), dtype=torch.int32, device=d.device)
    Q = torch.empty(batch * (F * L * L + t * t), dtype=d.dtype, device=d.device) if jobz else None
    rc = lib.bstq_stedc_leaves(code, int(bool(jobz)), int(n), int(leaf), int(batch), d.data_ptr(), e_ptr,
                               Q.data_ptr() if jobz else None, info.data_ptr(), work.data_ptr(),
                               _stream_handle(stream), ctypes.byref(p))
    if rc != 0:
        raise BstqError(rc, "bstq_stedc_leaves")
    Qf = Qt = None
    if jobz:
        # library layout: column-major blocks, full leaves first, then tails
        Qf = Q[: batch * F * L * L].view(batch, F, L, L).transpose(2, 3)
        if t:
            Qt = Q[batch * F * L * L:].view(batch, t, t).transpose(1, 2)
    return d, Qf, Qt, info


def diag(op: int, inp, count: int, arg: int = 0, stream=None):
    """bstq_diag on a CUDA tensor ``inp`` (float32 or float64, the records of
    ``count`` inputs back to back).  Returns the (count, values out) result
    tensor.  Nothing is synchronised."""
    import torch
    if not (inp.is_cuda and inp.is_contiguous()):
        raise ValueError("bstq.diag: inp must be a contiguous CUDA tensor")
    code = _dtype_code(inp.dtype)
    out_per = 256 if op == DIAG_FASTQ else DIAG_SHAPE[op][1]
    out = torch.empty((count, out_per), dtype=inp.dtype, device=inp.device)
    lib = load()
    wbytes = int(lib.bstq_diag_work_size(int(op), code, int(count)))
    if wbytes == 0:
        raise BstqError(-1, "bstq_diag_work_size")
    work = torch.empty(wbytes, dtype=torch.uint8, device=inp.device)
    rc = lib.bstq_diag(int(op), code, int(count), int(arg), inp.data_ptr(), out.data_ptr(), work.data_ptr(),
                       _stream_handle(stream))
    if rc != 0:
        raise BstqError(rc, "bstq_diag")
    return out


# ---------------------------------------------------------------------------
# Gated linear recurrence and orthogonalised update (float32, bfloat16 and
# float16 tensors).  A call for one token takes the GPU a few microseconds, so
# these bindings keep to few Python operations: checks compare without building
# objects, and sizes that depend on shapes alone are kept.
# ---------------------------------------------------------------------------
_seq = None  # what these calls use of torch and of the library, looked up once


class _Seq:
    def __init__(self):
        import torch
        lib = load()
        self.torch = torch
        self.codes = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
        self.f32, self.i32, self.u8 = torch.float32, torch.int32, torch.uint8
        self.empty, self.empty_like = torch.empty, torch.empty_like
        self.device = torch.cuda.current_device
        self.device()  # the context
        self.device = getattr(torch._C, "_cuda_getDevice", self.device)
        self.recur, self.recur_grad = lib.bstq_recur, lib.bstq_recur_grad
        self.recur_step, self.orthogonalize = lib.bstq_recur_step, lib.bstq_orthogonalize
        self.sizes = {"recur": lib.bstq_recur_work_size, "recur_grad": lib.bstq_recur_grad_work_size,
                      "orthogonalize": lib.bstq_orthogonalize_work_size}
        self.size = functools.lru_cache(maxsize=1024)(lambda device, where, *shape: int(self.sizes[where](*shape)))
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _seq_calls():
    global _seq
    _seq = _Seq()
    return _seq


class _on_stream:
    """Runs a call's allocations and launches on x's device and on the given
    stream; entered only where either is not the current one."""

    def __init__(self, torch, device, stream):
        self.device = torch.cuda.device(device)
        self.stream = torch.cuda.stream(stream)

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *exc):
        self.stream.__exit__(*exc)
        self.device.__exit__(*exc)


def _elsewhere(call, q, x, stream, args):
    """The call again with x's device and the given stream current.  What it
    reads is kept from reuse until the stream is done with it."""
    with _on_stream(q.torch, x.device, stream):
        out = call(*args)
        if stream is not None:
            for t in args:
                if isinstance(t, q.torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)
    return out


def _not_taken(where, x, dims):
    """Why x is not taken: it has to be a CUDA tensor of these dimensions and of
    a type that the kernels have."""
    if not x.is_cuda or x.dim() not in dims:
        raise ValueError(f"bstq.{where}: the first tensor must be on a CUDA device and have "
                         f"{' or '.join(map(str, dims))} dimensions")
    raise TypeError(f"bstq.{where}: dtype must be float32, bfloat16 or float16, got {x.dtype}")


def _differs(where, name, x):
    raise ValueError(f"bstq.{where}: {name} must be a {x.dtype} tensor of shape {tuple(x.shape)} on {x.device}")


def _dense(where, name, t, dev, shape, dtype):
    """The address of a contiguous tensor of the shape and dtype on the device;
    None stays None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"bstq.{where}: {name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"cuda:{dev}")
    return t.data_ptr()


def _rows(where, *named):
    """Element strides of the axes before the last of tensors that are not all
    dense; the last axis has to have stride 1."""
    out = []
    for name, t in zip(named[::2], named[1::2]):
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"bstq.{where}: {name} must have stride 1 along its last axis")
        out.extend(t.stride()[:-1])
    return (ctypes.c_int64 * len(out))(*out)


def _workspace(q, where, work, x, *shape):
    nbytes = q.size(x.get_device(), where, *shape)
    if nbytes == 0:
        raise BstqError(-10, f"bstq_{where}_work_size")
    if work is None:
        return q.empty((nbytes,), dtype=q.u8, device=x.device)
    if work.get_device() != x.get_device() or work.numel() * work.element_size() < nbytes or not work.is_contiguous():
        raise ValueError(f"bstq.{where}: work needs {nbytes} contiguous bytes on {x.device}")
    return work


def _raise(rc, where):
    if rc < 0:
        raise ValueError(f"bstq_{where}: argument {-rc} is invalid (code {rc})")
    raise BstqError(rc, f"bstq_{where}")


def recur(x, r, rate, h0=None, lengths=None, out=None, work=None, stream=None):
    """Gated linear recurrence on CUDA tensors ``x`` and ``r`` (batch, time,
    dim) with ``rate`` (dim,) float32: s = sigmoid(r), a = exp(-max(rate, 0)
    s), h_t = a_t h_{t-1} + (1 - a_t) x_t from ``h0`` (batch, dim) float32
    (default zero).  ``lengths`` (batch,) int32 ends sequences early: h is
    zero beyond.  Returns (h, hT): h in x's dtype (``out`` if given) and the
    last states (batch, dim) float32.  Work is enqueued on ``stream`` (default:
    torch's current stream); nothing is synchronised.  Should a wait inside the
    kernel run out (two seconds), what depends on it is NaN and the first int32
    of ``work`` is 1.  The result carries no autograd graph: its gradients come
    from :func:`recur_grad`."""
    q = _seq or _seq_calls()
    dtype, shape, dev = x.dtype, x.shape, x.get_device()
    code = q.codes.get(dtype)
    if code is None or dev < 0 or len(shape) != 3:
        _not_taken("recur", x, (3,))
    if stream is not None or dev != q.device():
        return _elsewhere(recur, q, x, stream, (x, r, rate, h0, lengths, out, work))
    batch, time, dim = shape
    if r.shape != shape or r.dtype is not dtype or r.get_device() != dev:
        _differs("recur", "r", x)
    # a vector's checks in place: one call less each
    if rate.numel() != dim or rate.dim() != 1 or rate.dtype is not q.f32 or rate.get_device() != dev \
            or not rate.is_contiguous():
        _dense("recur", "rate", rate, dev, (dim,), q.f32)
    np_ = None
    if lengths is not None:
        if lengths.numel() != batch or lengths.dim() != 1 or lengths.dtype is not q.i32 \
                or lengths.get_device() != dev or not lengths.is_contiguous():
            _dense("recur", "lengths", lengths, dev, (batch,), q.i32)
        np_ = lengths.data_ptr()
    h0p = None if h0 is None else _dense("recur", "h0", h0, dev, (batch, dim), q.f32)
    dense = x.is_contiguous() and r.is_contiguous()
    if out is None:
        h = q.empty_like(x) if dense else q.empty(shape, dtype=dtype, device=x.device)
    else:
        h = out
        if h.shape != shape or h.dtype is not dtype or h.get_device() != dev:
            _differs("recur", "out", x)
        dense = dense and h.is_contiguous()
    hT = q.empty((batch, dim), dtype=q.f32, device=x.device)
    work = _workspace(q, "recur", work, x, code, batch, time, dim)
    rc = q.recur(code, batch, time, dim, x.data_ptr(), r.data_ptr(), rate.data_ptr(), h0p, np_, h.data_ptr(),
                 hT.data_ptr(), None if dense else _rows("recur", "x", x, "r", r, "out", h), work.data_ptr(),
                 q.stream(dev))
    if rc != 0:
        _raise(rc, "recur")
    return h, hT


def recur_grad(x, r, rate, h, dh, dhT=None, h0=None, lengths=None, work=None, stream=None):
    """Gradients of :func:`recur`: ``h`` is its output, ``dh`` (batch, time,
    dim) and ``dhT`` (batch, dim) float32 (default zero) the gradients of h and
    hT.  Returns (dx, dr, drate, dh0): dx and dr in x's dtype, zero beyond a
    sequence's length; drate (dim,) and dh0 (batch, dim) float32.  Sums run in
    a fixed order.  Nothing is synchronised; a wait that runs out leaves NaN, as
    in :func:`recur`."""
    q = _seq or _seq_calls()
    dtype, shape = x.dtype, x.shape
    code = q.codes.get(dtype)
    dev = x.get_device()
    if code is None or dev < 0 or len(shape) != 3:
        _not_taken("recur_grad", x, (3,))
    if stream is not None or dev != q.device():
        return _elsewhere(recur_grad, q, x, stream, (x, r, rate, h, dh, dhT, h0, lengths, work))
    batch, time, dim = shape
    for name, t in (("r", r), ("h", h), ("dh", dh)):
        if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
            _differs("recur_grad", name, x)
    dx = q.empty(shape, dtype=dtype, device=x.device)
    dr = q.empty(shape, dtype=dtype, device=x.device)
    drate = q.empty((dim,), dtype=q.f32, device=x.device)
    dh0 = q.empty((batch, dim), dtype=q.f32, device=x.device)
    lp = _dense("recur_grad", "rate", rate, dev, (dim,), q.f32)
    dTp = _dense("recur_grad", "dhT", dhT, dev, (batch, dim), q.f32)
    h0p = _dense("recur_grad", "h0", h0, dev, (batch, dim), q.f32)
    np_ = _dense("recur_grad", "lengths", lengths, dev, (batch,), q.i32)
    st = None
    if not (x.is_contiguous() and r.is_contiguous() and h.is_contiguous() and dh.is_contiguous()):
        st = _rows("recur_grad", "x", x, "r", r, "h", h, "dh", dh, "dx", dx, "dr", dr)
    work = _workspace(q, "recur_grad", work, x, code, batch, time, dim)
    rc = q.recur_grad(code, batch, time, dim, x.data_ptr(), r.data_ptr(), lp, h.data_ptr(), dh.data_ptr(), dTp, h0p,
                      np_, dx.data_ptr(), dr.data_ptr(), drate.data_ptr(), dh0.data_ptr(), st, work.data_ptr(),
                      q.stream(dev))
    if rc != 0:
        _raise(rc, "recur_grad")
    return dx, dr, drate, dh0


def recur_step(state, x, r, rate, slots=None, out=None, stream=None):
    """One token of :func:`recur` for each row of ``x`` and ``r`` (batch,
    dim), on the cache ``state`` (rows, dim) float32, which is updated in
    place.  ``slots`` (batch,) int32 names each sequence's cache row (default:
    its own index), all distinct; a value outside [0, rows) leaves that
    sequence out: h is zero and no row changes.  Returns h (batch, dim) in x's
    dtype (``out`` if given).  Nothing is synchronised."""
    q = _seq or _seq_calls()
    dtype, shape, dev = x.dtype, x.shape, x.get_device()
    code = q.codes.get(dtype)
    if code is None or dev < 0 or len(shape) != 2:
        _not_taken("recur_step", x, (2,))
    if stream is not None or dev != q.device():
        return _elsewhere(recur_step, q, x, stream, (state, x, r, rate, slots, out))
    batch, dim = shape
    rows, width = state.shape if state.dim() == 2 else (0, -1)
    if width != dim or state.dtype is not q.f32 or state.get_device() != dev or (dim > 1 and state.stride(1) != 1):
        raise ValueError(f"bstq.recur_step: state must be a (rows, {dim}) float32 tensor on {x.device} with stride 1 "
                         "along its last axis")
    if r.shape != shape or r.dtype is not dtype or r.get_device() != dev:
        _differs("recur_step", "r", x)
    # a vector's checks in place: one call less each
    if rate.numel() != dim or rate.dim() != 1 or rate.dtype is not q.f32 or rate.get_device() != dev \
            or not rate.is_contiguous():
        _dense("recur_step", "rate", rate, dev, (dim,), q.f32)
    np_ = None
    if slots is not None:
        if slots.numel() != batch or slots.dim() != 1 or slots.dtype is not q.i32 or slots.get_device() != dev \
                or not slots.is_contiguous():
            _dense("recur_step", "slots", slots, dev, (batch,), q.i32)
        np_ = slots.data_ptr()
    dense = x.is_contiguous() and r.is_contiguous()
    if out is None:
        h = q.empty_like(x) if dense else q.empty(shape, dtype=dtype, device=x.device)
    else:
        h = out
        if h.shape != shape or h.dtype is not dtype or h.get_device() != dev:
            _differs("recur_step", "out", x)
        dense = dense and h.is_contiguous()
    rc = q.recur_step(code, batch, dim, rows, state.data_ptr(), state.stride(0) if rows > 1 else dim, x.data_ptr(),
                      r.data_ptr(), rate.data_ptr(), np_, h.data_ptr(),
                      None if dense else _rows("recur_step", "x", x, "r", r, "out", h), q.stream(dev))
    if rc != 0:
        _raise(rc, "recur_step")
    return h


def orthogonalize(G, steps: int = 5, coefs=None, out=None, work=None, stream=None):
    """Newton-Schulz orthogonalisation of each matrix of the CUDA tensor ``G``
    (m, n) or (batch, m, n): X = G / |G|_F, then ``steps`` times
    X <- a X + (b A + c A A) X with A = X X^T (of the transpose where m > n).
    ``coefs`` is one (a, b, c) for all steps or one for each (default 3.4445,
    -4.7750, 2.0315).  Returns X in G's dtype (``out`` if given; it may be G
    itself).  A G whose columns are contiguous (a transposed view) gives an X
    of the same layout.  Nothing is synchronised; a wait that runs out leaves
    NaN, as in :func:`recur`.  The result carries no autograd graph."""
    q = _seq or _seq_calls()
    dtype, shape = G.dtype, G.shape
    code = q.codes.get(dtype)
    dev = G.get_device()
    if code is None or dev < 0 or len(shape) not in (2, 3):
        _not_taken("orthogonalize", G, (2, 3))
    if stream is not None or dev != q.device():
        return _elsewhere(orthogonalize, q, G, stream, (G, steps, coefs, out, work))
    if out is not None and (out.shape != shape or out.dtype is not dtype or out.get_device() != dev):
        _differs("orthogonalize", "out", G)
    if G.stride(-1) != 1 and G.shape[-1] > 1 and (G.stride(-2) == 1 or G.shape[-2] == 1):
        # the polar factor of a transpose is the transpose of the polar factor
        return orthogonalize(G.transpose(-1, -2), steps, coefs, None if out is None else out.transpose(-1, -2),
                             work).transpose(-1, -2)
    X = q.empty(shape, dtype=dtype, device=G.device) if out is None else out
    batch = shape[0] if len(shape) == 3 else 1
    m, n = shape[-2:]
    st = None
    if not (G.is_contiguous() and X.is_contiguous()):
        if n > 1 and (G.stride(-1) != 1 or X.stride(-1) != 1):
            raise ValueError("bstq.orthogonalize: G and out must have stride 1 along the same of their last two axes")
        gb, xb = (G.stride(0), X.stride(0)) if G.dim() == 3 else (m * n, m * n)
        st = (ctypes.c_int64 * 4)(gb, G.stride(-2), xb, X.stride(-2))
    cs = None
    if coefs is not None:
        flat = np.asarray(coefs, dtype=np.float32)
        if flat.shape == (3,):
            flat = np.tile(flat, (max(int(steps), 0), 1))
        if flat.shape != (steps, 3):
            raise ValueError("bstq.orthogonalize: coefs must be (a, b, c) or one such row for each step")
        cs = (ctypes.c_float * flat.size)(*flat.reshape(-1).tolist())
    work = _workspace(q, "orthogonalize", work, G, code, batch, m, n)
    rc = q.orthogonalize(code, batch, m, n, G.data_ptr(), X.data_ptr(), st, int(steps), cs, work.data_ptr(),
                         q.stream(dev))
    if rc != 0:
        _raise(rc, "orthogonalize")
    return X
