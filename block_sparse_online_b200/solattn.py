"""ctypes binding of libsolattn (the C ABI in include/solattn.h).

Argument marshalling only: every step of the operator runs in the library's
CUDA kernels. PyTorch supplies device memory and the current stream. Loading
fails loudly if ``libsolattn.so`` has not been built; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsolattn.so")
# The build with the kernels' device-side bounds checks (python -m block_sparse_online_b200.build
# --debug): same exports, failed checks reported as SOLATTN_EBOUNDS.
DEBUG_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsolattn_debug.so")

SOLATTN_DENSE = 0
SOLATTN_KEEP_DROP = 1
SOLATTN_KEEP_CORRECT = 2
MODES = {"dense": SOLATTN_DENSE, "keep_drop": SOLATTN_KEEP_DROP, "keep_correct": SOLATTN_KEEP_CORRECT}

SOLATTN_OK = 0
SOLATTN_EINVAL = -1
SOLATTN_EUNSUPPORTED = -2
SOLATTN_ECUDA = -3
SOLATTN_ETIMEOUT = -4
SOLATTN_EWORKSPACE = -5
SOLATTN_EBOUNDS = -6
SOLATTN_ETABLE = -7
MAX_KEY_BLOCKS = 1024

EXPORTS = ("solattn_workspace_size", "solattn_pool", "solattn_forward", "solattn_forward_events",
           "solattn_get_status",
           "solattn_host_workspace_size", "solattn_forward_host", "solattn_watchdog_selftest",
           "solattn_selftest_exp2", "solattn_forward_noalloc", "solattn_forward_gaussian", "solattn_forward_ex",
           "solattn_route_keep", "solattn_proxy_map_bytes", "solattn_route_topk", "solattn_route_topp",
           "solattn_cross_workspace_size", "solattn_cross", "solattn_paged_workspace_size", "solattn_paged_forward",
           "solattn_cache_append", "solattn_cache_read", "solattn_strerror")
DTYPES = {torch.bfloat16: 0, torch.float16: 1}  # solattn_dtype
CACHE_KINDS = {torch.int8: 1, torch.float8_e4m3fn: 2}  # solattn_cache_kind of 8-bit pages (16-bit pages: 0)
GAUSS_VARIANTS = {"exact": 0, "diag": 1}  # solattn_gauss_variant
RULES = {"running_max": 0, "gauss_exact": 1, "gauss_diag": 2}  # solattn_rule
CORRECTIONS = {"block": 0, "token": 1}  # solattn_correction


class SolAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {strerror(status)} ({status})")
        self.status = status


class _Stats(ctypes.Structure):
    _fields_ = [("kept_per_head", ctypes.c_void_p), ("keep_mask", ctypes.c_void_p)]


class _Route(ctypes.Structure):  # solattn_route
    _fields_ = [("rule", ctypes.c_int), ("tau", ctypes.c_float), ("beta", ctypes.c_float), ("n_sink", ctypes.c_int),
                ("correction", ctypes.c_int)]


class _View(ctypes.Structure):  # solattn_view
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_n", ctypes.c_int64)]


class _Cache(ctypes.Structure):  # solattn_cache
    _fields_ = [("k", _View), ("v", _View), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int), ("Hkv", ctypes.c_int), ("page", ctypes.c_int), ("d", ctypes.c_int),
                ("kind", ctypes.c_int)]


class _Seqs(ctypes.Structure):  # solattn_seqs
    _fields_ = [("table", ctypes.c_void_p), ("cu", ctypes.c_void_p), ("len", ctypes.c_void_p), ("B", ctypes.c_int),
                ("width", ctypes.c_int), ("total", ctypes.c_int)]


def _load(path=_LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} is not built ({path}); run "
                          "`python -m block_sparse_online_b200.build`" + (" --debug" if path == DEBUG_LIB_PATH else ""))
    lib = ctypes.CDLL(path)
    i, sz, vp, f = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    lib.solattn_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.solattn_workspace_size.restype = sz
    lib.solattn_host_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.solattn_host_workspace_size.restype = sz
    lib.solattn_pool.argtypes = [vp, vp, i, i, i, i, i, vp]
    lib.solattn_pool.restype = i
    lib.solattn_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, ctypes.POINTER(_Stats), vp, sz, vp]
    lib.solattn_forward.restype = i
    lib.solattn_forward_events.argtypes = lib.solattn_forward.argtypes + [vp, vp]
    lib.solattn_forward_gaussian.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, ctypes.POINTER(_Stats),
                                             vp, sz, vp]
    lib.solattn_forward_gaussian.restype = i
    lib.solattn_forward_ex.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, ctypes.POINTER(_Route), i,
                                       ctypes.POINTER(_Stats), vp, sz, vp]
    lib.solattn_forward_ex.restype = i
    lib.solattn_forward_events.restype = i
    lib.solattn_forward_host.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, vp, sz, vp]
    lib.solattn_forward_host.restype = i
    lib.solattn_get_status.argtypes = [vp, vp]
    lib.solattn_get_status.restype = i
    lib.solattn_watchdog_selftest.argtypes = [vp, sz, ctypes.c_uint64, vp]
    lib.solattn_watchdog_selftest.restype = i
    lib.solattn_forward_noalloc.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, ctypes.POINTER(_Stats), vp]
    lib.solattn_forward_noalloc.restype = i
    lib.solattn_selftest_exp2.argtypes = [vp, vp, i, vp]
    lib.solattn_selftest_exp2.restype = i
    lib.solattn_route_keep.argtypes = [vp, vp, i, i, i, i, i, i, f, vp, vp]
    lib.solattn_route_keep.restype = i
    lib.solattn_proxy_map_bytes.argtypes = [i, i, i, i, i]
    lib.solattn_proxy_map_bytes.restype = sz
    lib.solattn_route_topk.argtypes = [vp, vp, i, i, i, i, i, i, i, vp, sz, vp, vp]
    lib.solattn_route_topk.restype = i
    lib.solattn_route_topp.argtypes = [vp, vp, i, i, i, i, i, i, f, vp, sz, vp, vp]
    lib.solattn_route_topp.restype = i
    pv, pc, ps = ctypes.POINTER(_View), ctypes.POINTER(_Cache), ctypes.POINTER(_Seqs)
    lib.solattn_cross_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.solattn_cross_workspace_size.restype = sz
    lib.solattn_cross.argtypes = [pv, pv, pv, pv, vp, i, i, i, i, i, i, i, vp, sz, vp]
    lib.solattn_cross.restype = i
    lib.solattn_paged_workspace_size.argtypes = [i, i, i, i, i]
    lib.solattn_paged_workspace_size.restype = sz
    lib.solattn_paged_forward.argtypes = [pv, pv, pc, ps, i, i, i, i, vp, sz, vp]
    lib.solattn_paged_forward.restype = i
    lib.solattn_cache_append.argtypes = [pc, pv, pv, ps, i, vp, vp]
    lib.solattn_cache_append.restype = i
    lib.solattn_cache_read.argtypes = [pc, ps, pv, pv, i, vp, vp]
    lib.solattn_cache_read.restype = i
    lib.solattn_strerror.argtypes = [i]
    lib.solattn_strerror.restype = ctypes.c_char_p
    return lib


def _addresses(lib):
    """Addresses of the entry points that the short call path (csrc/fastcall.cpp) calls."""
    return {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
            for n in ("solattn_cross", "solattn_paged_forward", "solattn_cache_append", "solattn_cache_read")}


_lib = _load()
_lib_path = _LIB_PATH
_at = _addresses(_lib)
try:  # host code only: without it the same calls go through ctypes
    from . import _fastcall as _fast
except ImportError:
    _fast = None


def library_path() -> str:
    return _lib_path


def load_library(path: str = _LIB_PATH) -> str:
    """Route every call of this module through the library at `path` (the release build by
    default, or DEBUG_LIB_PATH); returns the path that was active before."""
    global _lib, _lib_path, _at
    lib = _load(path)
    prev = _lib_path
    _lib, _lib_path, _at = lib, path, _addresses(lib)
    return prev


def strerror(status: int) -> str:
    return _lib.solattn_strerror(int(status)).decode()


def _check(status: int, what: str):
    if status != SOLATTN_OK:
        raise SolAttnError(status, what)


def _stream(stream, device=None):
    """The CUDA stream handle to pass to the library: ``stream``, or the current stream
    of ``device`` (the tensors' device). A stream on another device is refused, since the
    library launches on the current device."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif device is not None and stream.device != torch.device(device):
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return ctypes.c_void_p(stream.cuda_stream)


def _on_stream(fn):
    """For a call with a ``stream`` parameter: what it allocates (workspace, outputs) and clears belongs to
    the stream it launches on. Memory taken on another stream could be in use there still, and a
    workspace given back there would be handed out again while the kernels run. Tensors that the call returns
    are marked as used on the caller's stream too, so that dropping them there is safe."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        caller = torch.cuda.current_stream(stream.device)
        if caller == stream:
            return fn(*args, **kw)
        if _current_device() == stream.device.index:  # (the context manager takes twice as long)
            torch.cuda.set_stream(stream)
            try:
                result = fn(*args, **kw)
            finally:
                torch.cuda.set_stream(caller)
        else:
            with torch.cuda.stream(stream):
                result = fn(*args, **kw)
        for t in result if isinstance(result, tuple) else (result,):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(caller)
        return result

    return call


def _check_buffer(t, name, dtypes, numel, device):
    """A caller-provided buffer the library writes or reads through a raw pointer: it must
    be contiguous, of an accepted dtype, hold at least ``numel`` elements and live on the
    inputs' device (the library checks none of this; a short or foreign buffer would be
    written out of bounds)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, {numel} needed")
    if t.device != torch.device(device):
        raise ValueError(f"{name} is on {t.device}, the inputs on {device}")


def _mode(mode) -> int:
    return MODES[mode] if isinstance(mode, str) else int(mode)


def _bhnd(x: torch.Tensor):
    if x.dim() != 4:
        raise ValueError("expected a [B, H, N, d] tensor")
    return tuple(int(s) for s in x.shape)


def solattn_workspace_size(B, H, N, d, Bq, Bk) -> int:
    return int(_lib.solattn_workspace_size(B, H, N, d, Bq, Bk))


def solattn_host_workspace_size(B, H, N, d, Bq, Bk) -> int:
    return int(_lib.solattn_host_workspace_size(B, H, N, d, Bq, Bk))


def alloc_workspace(B, H, N, d, Bq, Bk, device="cuda") -> torch.Tensor:
    n = solattn_workspace_size(B, H, N, d, Bq, Bk)
    if n == 0:
        raise SolAttnError(SOLATTN_EUNSUPPORTED, "solattn_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


@_on_stream
def solattn_pool(x: torch.Tensor, blk: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Block means of a bf16 [B, H, N, d] CUDA tensor -> fp32 [B, H, ceil(N/blk), d]."""
    B, H, N, d = _bhnd(x)
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 CUDA tensor")
    nb = -(-N // blk)
    if out is None:
        out = torch.empty((B, H, nb, d), dtype=torch.float32, device=x.device)
    _check_buffer(out, "out", (torch.float32,), B * H * nb * d, x.device)
    with torch.cuda.device(x.device):
        rc = _lib.solattn_pool(x.data_ptr(), out.data_ptr(), B, H, N, d, blk, _stream(stream, x.device))
    _check(rc, "solattn_pool")
    return out


def _inputs(q, k, v):
    B, H, N, d = _bhnd(q)
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (B, H, N, d):
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors of one shape")
        if t.device != q.device:
            raise ValueError("q, k, v must be on one device")
    return B, H, N, d


def _prepare(q, k, v, Bq, Bk, out, kept_per_head, keep_mask, workspace):
    """Checks the inputs and the buffers the caller passed, and allocates the others."""
    B, H, N, d = _inputs(q, k, v)
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    _check_buffer(out, "out", (torch.bfloat16,), B * H * N * d, dev)
    if kept_per_head is None:
        kept_per_head = torch.empty((B, H), dtype=torch.int64, device=dev)
    _check_buffer(kept_per_head, "kept_per_head", (torch.int64,), B * H, dev)
    mask = None
    nq, nk = -(-N // Bq), -(-N // Bk)
    if isinstance(keep_mask, torch.Tensor):
        mask = keep_mask
        _check_buffer(mask, "keep_mask", (torch.int32, torch.uint32), B * H * nq * (-(-nk // 32)), dev)
    elif keep_mask:
        mask = torch.empty((B, H, nq, -(-nk // 32)), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(B, H, N, d, Bq, Bk, dev)
    _check_buffer(workspace, "workspace", (torch.uint8, torch.int8), 0, dev)
    stats = _Stats(kept_per_head.data_ptr(), mask.data_ptr() if mask is not None else None)
    return B, H, N, d, out, kept_per_head, mask, workspace, stats


@_on_stream
def solattn_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, Bq: int, Bk: int, tau: float,
                    mode="keep_correct", out: torch.Tensor | None = None,
                    kept_per_head: torch.Tensor | None = None, keep_mask: bool | torch.Tensor = False,
                    workspace: torch.Tensor | None = None, stream=None, events=None):
    """Run the Sol-Attn forward operator on bf16 [B, H, N, d] CUDA tensors.

    ``events``: optional pair of ``torch.cuda.Event(enable_timing=True)`` recorded
    around the attention kernel (solattn_forward_events).

    Returns (out bf16 [B, H, N, d], kept_per_head int64 [B, H], keep_mask uint32
    [B, H, nQB, ceil(nKB/32)] or None). Asynchronous on ``stream``; device-side
    errors are reported by :func:`solattn_get_status` on the workspace.
    """
    B, H, N, d, out, kept_per_head, mask, workspace, stats = _prepare(q, k, v, Bq, Bk, out, kept_per_head,
                                                                      keep_mask, workspace)
    with torch.cuda.device(q.device):
        args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, N, d, Bq, Bk,
                ctypes.c_float(float(tau)), _mode(mode), ctypes.byref(stats), workspace.data_ptr(),
                workspace.numel(), _stream(stream, q.device))
        if events is None:
            rc = _lib.solattn_forward(*args)
        else:
            st = stream if stream is not None else torch.cuda.current_stream(q.device)
            for e in events:
                if e.cuda_event == 0:  # torch creates the CUDA event on its first record
                    e.record(st)
            rc = _lib.solattn_forward_events(*args, ctypes.c_void_p(events[0].cuda_event),
                                             ctypes.c_void_p(events[1].cuda_event))
    _check(rc, "solattn_forward")
    return out, kept_per_head, mask


@_on_stream
def solattn_forward_gaussian(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, Bq: int, Bk: int, beta: float,
                             variant="exact", mode="keep_correct", out: torch.Tensor | None = None,
                             kept_per_head: torch.Tensor | None = None, keep_mask: bool | torch.Tensor = False,
                             workspace: torch.Tensor | None = None, stream=None):
    """The forward operator under the query-dependent Gaussian threshold
    (theta_i = mu_i + beta * sigma_i; ``variant`` "exact" or "diag"). Returns what
    :func:`solattn_forward` returns."""
    if variant not in GAUSS_VARIANTS:
        raise ValueError(f"unknown variant {variant!r}")
    B, H, N, d, out, kept_per_head, mask, workspace, stats = _prepare(q, k, v, Bq, Bk, out, kept_per_head,
                                                                      keep_mask, workspace)
    with torch.cuda.device(q.device):
        rc = _lib.solattn_forward_gaussian(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, N, d,
                                           Bq, Bk, ctypes.c_float(float(beta)), GAUSS_VARIANTS[variant],
                                           _mode(mode), ctypes.byref(stats), workspace.data_ptr(),
                                           workspace.numel(), _stream(stream, q.device))
    _check(rc, "solattn_forward_gaussian")
    return out, kept_per_head, mask


@_on_stream
def solattn_forward_ex(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, Bq: int, Bk: int, mode="keep_correct",
                       rule="running_max", tau: float = 0.0, beta: float = 0.0, n_sink: int = 0,
                       correction="block", out: torch.Tensor | None = None,
                       kept_per_head: torch.Tensor | None = None,
                       keep_mask: bool | torch.Tensor = False, workspace: torch.Tensor | None = None, stream=None):
    """The forward operator with every routing option: ``rule`` "running_max" (tau),
    "gauss_exact" or "gauss_diag" (beta), ``n_sink`` leading key tokens kept as sinks, and
    the keep_correct ``correction``: "block" (block proxy) or "token" (token-to-block logit).
    Returns what :func:`solattn_forward` returns."""
    if rule not in RULES:
        raise ValueError(f"unknown rule {rule!r}")
    if correction not in CORRECTIONS:
        raise ValueError(f"unknown correction {correction!r}")
    B, H, N, d, out, kept_per_head, mask, workspace, stats = _prepare(q, k, v, Bq, Bk, out, kept_per_head,
                                                                      keep_mask, workspace)
    route = _Route(RULES[rule], float(tau), float(beta), int(n_sink), CORRECTIONS[correction])
    with torch.cuda.device(q.device):
        rc = _lib.solattn_forward_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, N, d, Bq, Bk,
                                     ctypes.byref(route), _mode(mode), ctypes.byref(stats), workspace.data_ptr(),
                                     workspace.numel(), _stream(stream, q.device))
    _check(rc, "solattn_forward_ex")
    return out, kept_per_head, mask


def solattn_get_status(workspace: torch.Tensor, stream=None) -> int:
    if not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    with torch.cuda.device(workspace.device):
        return int(_lib.solattn_get_status(workspace.data_ptr(), _stream(stream, workspace.device)))


@_on_stream
def solattn_forward_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, Bq: int, Bk: int, tau: float,
                         mode="keep_correct", out: torch.Tensor | None = None,
                         kept_per_head: torch.Tensor | None = None, scratch: torch.Tensor | None = None,
                         stream=None):
    """End-to-end call on HOST (ideally pinned) bf16 tensors: host->device copies,
    the operator, and device->host copies of the output and per-head counts, all
    inside the library call, which returns after the stream is synchronised."""
    B, H, N, d = _bhnd(q)
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (B, H, N, d):
            raise ValueError("q, k, v must be contiguous bf16 host tensors of one shape")
    if out is None:
        out = torch.empty_like(q, pin_memory=True)
    _check_buffer(out, "out", (torch.bfloat16,), B * H * N * d, "cpu")
    if kept_per_head is None:
        kept_per_head = torch.empty((B, H), dtype=torch.int64)
    _check_buffer(kept_per_head, "kept_per_head", (torch.int64,), B * H, "cpu")
    need = solattn_host_workspace_size(B, H, N, d, Bq, Bk)
    if scratch is None:
        scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    if not scratch.is_cuda:
        raise ValueError("scratch must be a CUDA tensor")
    _check_buffer(scratch, "scratch", (torch.uint8, torch.int8), 0, scratch.device)
    with torch.cuda.device(scratch.device):
        rc = _lib.solattn_forward_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, N, d, Bq,
                                       Bk, ctypes.c_float(float(tau)), _mode(mode), kept_per_head.data_ptr(),
                                       scratch.data_ptr(), scratch.numel(), _stream(stream, scratch.device))
    _check(rc, "solattn_forward_host")
    return out, kept_per_head


@_on_stream
def solattn_watchdog_selftest(limit_ns: int = 2_000_000, stream=None) -> int:
    """Run the device watchdog self-test; returns the status the kernel stored
    (SOLATTN_ETIMEOUT when a wait that nobody completes is abandoned on time)."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    with torch.cuda.device(ws.device):
        rc = _lib.solattn_watchdog_selftest(ws.data_ptr(), ws.numel(), int(limit_ns), _stream(stream, ws.device))
    _check(rc, "solattn_watchdog_selftest")
    return solattn_get_status(ws, stream)


NOALLOC_SCRATCH_BYTES = 64 << 20


@_on_stream
def solattn_forward_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, Bq: int, Bk: int, tau: float,
                            mode="keep_correct", out: torch.Tensor | None = None,
                            kept_per_head: torch.Tensor | None = None, stream=None):
    """solattn_forward without a workspace: the library uses its static device scratch
    (for callers that cannot allocate device memory). Output and count tensors are
    allocated here only when not given; the library call itself allocates nothing.
    Calls that overlap on the GPU race on the shared scratch."""
    B, H, N, d = _inputs(q, k, v)
    if out is None:
        out = torch.empty_like(q)
    _check_buffer(out, "out", (torch.bfloat16,), B * H * N * d, q.device)
    if kept_per_head is None:
        kept_per_head = torch.empty((B, H), dtype=torch.int64, device=q.device)
    _check_buffer(kept_per_head, "kept_per_head", (torch.int64,), B * H, q.device)
    stats = _Stats(kept_per_head.data_ptr(), None)
    with torch.cuda.device(q.device):
        rc = _lib.solattn_forward_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, N, d, Bq,
                                          Bk, ctypes.c_float(float(tau)), _mode(mode), ctypes.byref(stats),
                                          _stream(stream, q.device))
    _check(rc, "solattn_forward_noalloc")
    return out, kept_per_head


def _route_args(qbar: torch.Tensor, kbar: torch.Tensor, N: int, Bq: int, Bk: int, keep_mask):
    if qbar.dim() != 4 or kbar.dim() != 4:
        raise ValueError("qbar and kbar must be [B, H, nB, d]")
    B, H, nQB, d = (int(x) for x in qbar.shape)
    nKB = -(-N // Bk)
    if nQB != -(-N // Bq) or tuple(kbar.shape) != (B, H, nKB, d):
        raise ValueError("qbar / kbar do not match N, Bq, Bk")
    for name, t in (("qbar", qbar), ("kbar", kbar)):
        _check_buffer(t, name, (torch.float32,), t.numel(), qbar.device)
    if keep_mask is None:
        keep_mask = torch.empty((B, H, nQB, -(-nKB // 32)), dtype=torch.int32, device=qbar.device)
    _check_buffer(keep_mask, "keep_mask", (torch.int32, torch.uint32), B * H * nQB * (-(-nKB // 32)), qbar.device)
    return B, H, d, keep_mask


@_on_stream
def solattn_route_keep(qbar: torch.Tensor, kbar: torch.Tensor, N: int, Bq: int, Bk: int, tau: float,
                       keep_mask: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The running-maximum routing rule alone on pooled blocks (fp32 [B, H, nB, d]); returns the
    keep bits [B, H, nQB, ceil(nKB/32)] (int32 storage of u32 words)."""
    B, H, d, keep_mask = _route_args(qbar, kbar, N, Bq, Bk, keep_mask)
    with torch.cuda.device(qbar.device):
        rc = _lib.solattn_route_keep(qbar.data_ptr(), kbar.data_ptr(), B, H, N, d, Bq, Bk, ctypes.c_float(float(tau)),
                                     keep_mask.data_ptr(), _stream(stream, qbar.device))
    _check(rc, "solattn_route_keep")
    return keep_mask


def solattn_proxy_map_bytes(B, H, N, Bq, Bk) -> int:
    """Bytes of the fp32 proxy map the top-k and top-p routers write (0 if the shape is invalid)."""
    return int(_lib.solattn_proxy_map_bytes(B, H, N, Bq, Bk))


def _proxy_map(B, H, N, Bq, Bk, proxy_map, device):
    n = solattn_proxy_map_bytes(B, H, N, Bq, Bk)
    if proxy_map is None:
        proxy_map = torch.empty(n // 4, dtype=torch.float32, device=device)
    _check_buffer(proxy_map, "proxy_map", (torch.float32,), n // 4, device)
    return proxy_map


@_on_stream
def solattn_route_topk(qbar: torch.Tensor, kbar: torch.Tensor, N: int, Bq: int, Bk: int, k: int,
                       keep_mask: torch.Tensor | None = None, proxy_map: torch.Tensor | None = None, stream=None):
    """Top-k routing (materialised proxy map, the k largest proxies per query block).
    Returns (keep bits, proxy map)."""
    B, H, d, keep_mask = _route_args(qbar, kbar, N, Bq, Bk, keep_mask)
    proxy_map = _proxy_map(B, H, N, Bq, Bk, proxy_map, qbar.device)
    with torch.cuda.device(qbar.device):
        rc = _lib.solattn_route_topk(qbar.data_ptr(), kbar.data_ptr(), B, H, N, d, Bq, Bk, int(k),
                                     proxy_map.data_ptr(), proxy_map.numel() * 4, keep_mask.data_ptr(),
                                     _stream(stream, qbar.device))
    _check(rc, "solattn_route_topk")
    return keep_mask, proxy_map


@_on_stream
def solattn_route_topp(qbar: torch.Tensor, kbar: torch.Tensor, N: int, Bq: int, Bk: int, p: float,
                       keep_mask: torch.Tensor | None = None, proxy_map: torch.Tensor | None = None, stream=None):
    """Top-p routing (materialised proxy map; the heaviest blocks until their share of the
    row's mass reaches p). Returns (keep bits, proxy map)."""
    B, H, d, keep_mask = _route_args(qbar, kbar, N, Bq, Bk, keep_mask)
    proxy_map = _proxy_map(B, H, N, Bq, Bk, proxy_map, qbar.device)
    with torch.cuda.device(qbar.device):
        rc = _lib.solattn_route_topp(qbar.data_ptr(), kbar.data_ptr(), B, H, N, d, Bq, Bk, ctypes.c_float(float(p)),
                                     proxy_map.data_ptr(), proxy_map.numel() * 4, keep_mask.data_ptr(),
                                     _stream(stream, qbar.device))
    _check(rc, "solattn_route_topp")
    return keep_mask, proxy_map


@_on_stream
def solattn_selftest_exp2(x: torch.Tensor, stream=None) -> torch.Tensor:
    """2^x by the software exp2 of the softmax, for a contiguous fp32 CUDA tensor."""
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous fp32 CUDA tensor")
    y = torch.empty_like(x)
    with torch.cuda.device(x.device):
        rc = _lib.solattn_selftest_exp2(x.data_ptr(), y.data_ptr(), x.numel(), _stream(stream, x.device))
    _check(rc, "solattn_selftest_exp2")
    return y


# ---------------------------------------------------------------- dense attention and the cache

_Tensor, _i32, _u8 = torch.Tensor, torch.int32, torch.uint8
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device


def _bad_rows(x, name, dtype, shape, device):
    """Says what is wrong with a tensor that _rows refused."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, not {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, {tuple(shape)} expected")
    if x.device != device:
        raise ValueError(f"{name} is on {x.device}, the inputs on {device}")
    raise ValueError(f"the last dimension of {name} must be contiguous")


def _rows(x, name, dtype, shape, device):
    """Strides of a tensor of rows of d contiguous elements, checked. The usual case passes on one
    line: these calls take a few microseconds on the GPU."""
    if isinstance(x, _Tensor) and x.dtype is dtype and x.get_device() == device.index and x.shape == shape:
        st = x.stride()
        if st[-1] == 1 or not x.numel():
            return st
    _bad_rows(x, name, dtype, shape, device)


def _view4(x, name, dtype, shape, device):  # [B, heads, n, d]
    st = _rows(x, name, dtype, shape, device)
    return _View(x.data_ptr(), st[0], st[1], st[2])


def _view3(x, name, dtype, shape, device):  # packed rows [n, heads, d]
    st = _rows(x, name, dtype, shape, device)
    return _View(x.data_ptr(), 0, st[1], st[0])


def _int32(x, name, numel, device):
    if not (isinstance(x, _Tensor) and x.dtype is _i32 and x.get_device() == device.index and x.is_contiguous()
            and x.numel() >= numel):
        _check_buffer(x, name, (torch.int32,), numel, device)
    return x.data_ptr()


def _workspace(workspace, need, device, least=0):
    """The caller's workspace of at least ``least`` bytes (of a workspace proper the library checks the size, a status
    word alone it takes by its address), or a new one with its header cleared."""
    if workspace is None:
        workspace = torch.empty(need(), dtype=torch.uint8, device=device)
        workspace[:256].zero_()
    elif not (isinstance(workspace, _Tensor) and workspace.dtype is _u8 and workspace.get_device() == device.index
              and workspace.is_contiguous() and workspace.numel() >= least):
        _check_buffer(workspace, "workspace", (torch.uint8, torch.int8), least, device)
    return workspace


def _on_device(device, stream, call, *args):
    """call(*args, stream) with `device` current; the stream is the caller's or the current one."""
    if stream is not None:
        handle = _stream(stream, device)
    else:
        handle = _raw_stream(device.index)
    if _current_device() == device.index:
        return call(*args, handle)
    with torch.cuda.device(device):
        return call(*args, handle)


def _need(size, what):
    if size == 0:
        raise SolAttnError(SOLATTN_EUNSUPPORTED, what)
    return size


def alloc_status(device="cuda") -> torch.Tensor:
    """A cleared status word (256 bytes) for :func:`solattn_cache_append` and :func:`solattn_cache_read`;
    read it with :func:`solattn_get_status`."""
    return torch.zeros(256, dtype=torch.uint8, device=device)


def solattn_cross_workspace_size(B, H, Hkv, Nq, Nk, d) -> int:
    return int(_lib.solattn_cross_workspace_size(B, H, Hkv, Nq, Nk, d))


def solattn_paged_workspace_size(B, H, Hkv, total, d) -> int:
    return int(_lib.solattn_paged_workspace_size(B, H, Hkv, total, d))


def alloc_cross_workspace(B, H, Hkv, Nq, Nk, d, device="cuda") -> torch.Tensor:
    """Workspace of :func:`solattn_cross`, its status word cleared."""
    return _workspace(None, lambda: _need(solattn_cross_workspace_size(B, H, Hkv, Nq, Nk, d), "solattn_cross_workspace_size"),
                      device)


def solattn_cross(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, key_len: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Softmax attention of q [B, H, Nq, d] to keys and values [B, Hkv, Nk, d] of another length
    (an encoder's states), bf16 or fp16, strided views allowed (rows contiguous).

    ``key_len``: int32 [B] on the device, the keys of each sequence (the rest is padding that
    may hold anything); a sequence of none gives zeros. H is a multiple of Hkv: query head h
    uses key head h // (H // Hkv). Returns out [B, H, Nq, d]. Asynchronous on ``stream``;
    lengths outside [0, Nk] are reported by :func:`solattn_get_status` on the workspace (without
    one given they are cut all the same, and not reported). A workspace that the call takes itself, and
    a new ``out``, belong to ``stream``; order other streams behind it before they use ``out``."""
    if _fast is not None:
        rc = _fast.cross(_at["solattn_cross"], q, k, v, key_len, out, workspace, stream)
        if rc is not None:
            if rc:
                _check(rc, "solattn_cross")
            return out
    return _cross(q, k, v, key_len, out, workspace, stream)


@_on_stream
def _cross(q, k, v, key_len, out, workspace, stream):
    dt = DTYPES.get(getattr(q, "dtype", None))
    if dt is None or not q.is_cuda or q.dim() != 4:
        raise ValueError("q must be a bfloat16 or float16 [B, H, N, d] CUDA tensor")
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a [B, Hkv, Nk, d] tensor")
    dtype, dev, shape = q.dtype, q.device, q.shape
    B, H, Nq, d = shape
    Hkv, Nk = k.shape[1], k.shape[2]
    kshape = (B, Hkv, Nk, d)
    if out is None:
        out = torch.empty_like(q) if 0 not in q.stride() else torch.empty(shape, dtype=dtype, device=dev)
    workspace = _workspace(workspace, lambda: _need(solattn_cross_workspace_size(B, H, Hkv, Nq, Nk, d), "solattn_cross"), dev)
    rc = _on_device(dev, stream, _lib.solattn_cross, _view4(q, "q", dtype, shape, dev), _view4(k, "k", dtype, kshape, dev),
                    _view4(v, "v", dtype, kshape, dev), _view4(out, "out", dtype, shape, dev),
                    None if key_len is None else _int32(key_len, "key_len", B, dev), B, H, Hkv, Nq, Nk, d, dt,
                    workspace.data_ptr(), workspace.numel())
    _check(rc, "solattn_cross")
    return out


class PagedCache:
    """A key/value cache in pages: k_pages and v_pages [num_pages, Hkv, page, d] in bf16 or fp16,
    or as int8 or e4m3 codes with k_scale and v_scale fp32 [num_pages, Hkv, page], one
    scale for each row. page is 16, 32, 64 or 128 tokens. The cache keeps references to the
    tensors, not copies. A table [B, width] int32 names each sequence's pages in order
    (entries behind its last page are not read)."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        P, Hkv, page, d = shape = _bhnd(k_pages)
        dt, dev = k_pages.dtype, k_pages.device
        if dt not in DTYPES and dt not in CACHE_KINDS:
            raise ValueError(f"pages must be bfloat16, float16, int8 or float8_e4m3fn, not {dt}")
        if not k_pages.is_cuda:
            raise ValueError("the pages must be CUDA tensors")
        k, v = _view4(k_pages, "k_pages", dt, shape, dev), _view4(v_pages, "v_pages", dt, shape, dev)
        if (dt in CACHE_KINDS) != (k_scale is not None) or (dt in CACHE_KINDS) != (v_scale is not None):
            raise ValueError("8-bit pages need k_scale and v_scale, 16-bit pages take none")
        for name, sc in (("k_scale", k_scale), ("v_scale", v_scale)):
            if sc is not None:
                _check_buffer(sc, name, (torch.float32,), P * Hkv * page, dev)
                if tuple(sc.shape) != (P, Hkv, page):
                    raise ValueError(f"{name} has shape {tuple(sc.shape)}, {(P, Hkv, page)} expected")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.num_pages, self.Hkv, self.page, self.d, self.dtype, self.device = P, Hkv, page, d, dt, dev
        self._c = _Cache(k, v, None if k_scale is None else k_scale.data_ptr(),
                         None if v_scale is None else v_scale.data_ptr(), P, Hkv, page, d, CACHE_KINDS.get(dt, 0))
        # for the short call path: the structure's address, the device and the 16-bit dtype (or -1)
        self._fast = (ctypes.addressof(self._c), dev.index, DTYPES.get(dt, -1))

    def _seqs(self, table, cu, length, total):
        """The sequences of a call, checked."""
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table must be an int32 [B, width] tensor")
        B, width = table.shape
        dev = self.device
        return _Seqs(_int32(table, "table", 1, dev), _int32(cu, "cu", B + 1, dev), _int32(length, "length", B, dev), B,
                     width, total)

    def _rows_dtype(self, x, name):
        """The 16-bit type of packed rows x [total, heads, d], and how many they are."""
        if not isinstance(x, torch.Tensor) or x.dim() != 3:
            raise ValueError(f"{name} must be a [total, heads, d] tensor")
        dtype = x.dtype
        if dtype not in DTYPES or (self.dtype in DTYPES and dtype is not self.dtype):
            raise ValueError(f"{name} must be " + (str(self.dtype) if self.dtype in DTYPES else "bfloat16 or float16"))
        return dtype, x.shape[0]


def alloc_paged_workspace(cache: PagedCache, B, H, total, device=None) -> torch.Tensor:
    """Workspace of :func:`solattn_paged_forward`, its status word cleared."""
    return _workspace(None, lambda: _need(solattn_paged_workspace_size(B, H, cache.Hkv, total, cache.d),
                                          "solattn_paged_workspace_size"), cache.device if device is None else device)


def solattn_paged_forward(q: torch.Tensor, cache: PagedCache, table: torch.Tensor, cu: torch.Tensor,
                          length: torch.Tensor, max_new: int, causal: bool = True, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Softmax attention of a batch's new tokens over a paged cache that already holds them.

    q [total, H, d] (bf16 or fp16) packs the new tokens: rows cu[b] .. cu[b+1] - 1 are the last
    ones of sequence b, which has length[b] tokens in the cache (table, cu, length: int32 on the
    device). ``causal``: each sees the keys up to its own position; else the whole sequence.
    ``max_new``: the most new tokens of a sequence, as far as the caller knows (it selects the
    kernel, not the result). Rows behind cu[B] are left alone. Returns out [total, H, d].
    Lengths or pages out of range are reported by :func:`solattn_get_status` on the workspace."""
    if not isinstance(cache, PagedCache):
        raise ValueError("cache must be a PagedCache")
    if _fast is not None:
        rc = _fast.paged(_at["solattn_paged_forward"], *cache._fast, q, table, cu, length, max_new, causal, out, workspace,
                         stream)
        if rc is not None:
            if rc:
                _check(rc, "solattn_paged_forward")
            return out
    return _paged(q, cache, table, cu, length, max_new, causal, out, workspace, stream)


@_on_stream
def _paged(q, cache, table, cu, length, max_new, causal, out, workspace, stream):
    dtype, total = cache._rows_dtype(q, "q")
    dev, H = cache.device, q.shape[1]
    shape = (total, H, cache.d)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    seqs = cache._seqs(table, cu, length, total)
    workspace = _workspace(workspace, lambda: _need(solattn_paged_workspace_size(seqs.B, H, cache.Hkv, total, cache.d),
                                                    "solattn_paged_forward"), dev)
    rc = _on_device(dev, stream, _lib.solattn_paged_forward, _view3(q, "q", dtype, shape, dev),
                    _view3(out, "out", dtype, shape, dev), cache._c, seqs, H, int(max_new), 1 if causal else 0, DTYPES[dtype],
                    workspace.data_ptr(), workspace.numel())
    _check(rc, "solattn_paged_forward")
    return out


def solattn_cache_append(cache: PagedCache, new_k: torch.Tensor, new_v: torch.Tensor, table: torch.Tensor,
                         cu: torch.Tensor, length: torch.Tensor, workspace: torch.Tensor | None = None, stream=None):
    """Writes the new tokens' keys and values [total, Hkv, d] (bf16 or fp16) into their pages,
    quantised where the cache is 8-bit: scale = max|x| / TOP, code = nearest(x TOP / max|x|), TOP = 127
    (int8) or 448 (e4m3). table, cu, length as in :func:`solattn_paged_forward` (length counts
    the new tokens). ``workspace``: an :func:`alloc_status` tensor or any workspace."""
    if _fast is not None:
        rc = _fast.cache_rows(_at["solattn_cache_append"], True, *cache._fast, new_k, new_v, table, cu, length, workspace,
                              stream)
        if rc is not None:
            if rc:
                _check(rc, "solattn_cache_append")
            return
    _append(cache, new_k, new_v, table, cu, length, workspace, stream)


@_on_stream
def _append(cache, new_k, new_v, table, cu, length, workspace, stream):
    dtype, total = cache._rows_dtype(new_k, "new_k")
    dev, shape = cache.device, (total, cache.Hkv, cache.d)
    seqs = cache._seqs(table, cu, length, total)
    workspace = _workspace(workspace, lambda: 256, dev, 256)
    rc = _on_device(dev, stream, _lib.solattn_cache_append, cache._c, _view3(new_k, "new_k", dtype, shape, dev),
                    _view3(new_v, "new_v", dtype, shape, dev), seqs, DTYPES[dtype], workspace.data_ptr())
    _check(rc, "solattn_cache_append")


def solattn_cache_read(cache: PagedCache, table: torch.Tensor, cu: torch.Tensor, length: torch.Tensor,
                       k_out: torch.Tensor, v_out: torch.Tensor, workspace: torch.Tensor | None = None, stream=None):
    """Reads the new tokens' rows (the last cu[b+1] - cu[b] of each sequence) back from the pages into
    k_out and v_out [total, Hkv, d] (bf16 or fp16): code * scale, rounded once. Returns them."""
    if _fast is not None:
        rc = _fast.cache_rows(_at["solattn_cache_read"], False, *cache._fast, k_out, v_out, table, cu, length, workspace,
                              stream)
        if rc is not None:
            if rc:
                _check(rc, "solattn_cache_read")
            return k_out, v_out
    return _read(cache, table, cu, length, k_out, v_out, workspace, stream)


@_on_stream
def _read(cache, table, cu, length, k_out, v_out, workspace, stream):
    dtype, total = cache._rows_dtype(k_out, "k_out")
    dev, shape = cache.device, (total, cache.Hkv, cache.d)
    seqs = cache._seqs(table, cu, length, total)
    workspace = _workspace(workspace, lambda: 256, dev, 256)
    rc = _on_device(dev, stream, _lib.solattn_cache_read, cache._c, seqs, _view3(k_out, "k_out", dtype, shape, dev),
                    _view3(v_out, "v_out", dtype, shape, dev), DTYPES[dtype], workspace.data_ptr())
    _check(rc, "solattn_cache_read")
    return k_out, v_out


__all__ = [n for n in globals() if n.startswith("solattn_")] + ["PagedCache"] + ["SolAttnError", "MODES"]
