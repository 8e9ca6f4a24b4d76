"""Python binding of the C-ABI library (argument marshalling only).

Every step of the path runs in the CUDA kernels of ``libcoda.so``; this module
checks tensor dtypes/devices/contiguity, allocates outputs and the workspace
with torch (device memory and streams are all torch is used for), and passes
raw device pointers plus ``torch.cuda.current_stream()`` to the C entry points
of the same names.  There is no CPU fallback: if the library is missing or the
device is not sm_100, calls raise.  Each call into an entry point that enqueues
GPU work is wrapped in an NVTX range of the entry point's name.
"""

from __future__ import annotations

import ctypes
import os
import threading
import types

import torch

from .build import LIB_PATH

_c_void_p = ctypes.c_void_p
_c_int = ctypes.c_int
_c_size_t = ctypes.c_size_t
_c_float = ctypes.c_float

CODA_ERR_INVALID_ARG = 1
CODA_ERR_DEVICE_TIMEOUT = 7


class CodaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {_status_string(status)} (status {status})")


_lib = None
_lib_lock = threading.Lock()


def library() -> ctypes.CDLL:
    """Load libcoda.so (built in-tree by gemm_epilogue_fusion_tmem_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"CUDA library not built ({LIB_PATH}); run `python -m gemm_epilogue_fusion_tmem_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, S, F = _c_void_p, _c_int, _c_size_t, _c_float
        sig = {
            "coda_status_string": (ctypes.c_char_p, [I]),
            "coda_version": (I, []),
            "coda_status_clear": (I, [P, P]),
            "coda_status_query": (I, [P, P, ctypes.POINTER(ctypes.c_uint32)]),
            "coda_shared_status": (I, [ctypes.POINTER(P)]),
            "coda_set_wait_limit_ns": (None, [ctypes.c_uint64]),
            "coda_selftest_wait_timeout": (I, [P, ctypes.c_uint64, P]),
            "coda_selftest_fp8_silence": (I, [I, I]),
            "coda_profile_arm": (I, [I, P, P]),
            "coda_gemm_workspace_bytes": (S, []),
            "coda_gemm": (I, [P, P, P, I, I, I, I, I, P, S, P]),
            "coda_fold_gain": (I, [P, P, P, I, I, P]),
            "coda_gemm_swiglu": (I, [P, P, P, P, P, I, I, I, P, S, P]),
            "coda_grg_fwd_workspace_bytes": (S, [I, I, I, I, I]),
            "coda_grg_fwd": (I, [P, P, P, P, P, P, P, P, P, P, I, I, I, I, F, P, S, P]),
            "coda_grg_bwd_workspace_bytes": (S, [I, I, I, I]),
            "coda_grg_bwd": (I, [P, P, P, P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, P, S, P]),
            "coda_swiglu_fwd_workspace_bytes": (S, [I, I, I]),
            "coda_swiglu_fwd": (I, [P, P, P, P, P, P, I, I, I, P, S, P]),
            "coda_swiglu_bwd_workspace_bytes": (S, [I, I, I]),
            "coda_swiglu_bwd": (I, [P, P, P, P, P, P, P, P, P, I, I, I, P, S, P]),
            "coda_grg_fwd_hg_workspace_bytes": (S, [I, I, I, I, I]),
            "coda_grg_fwd_hg": (I, [P] * 10 + [I, I, I, I, F, P, S, P]),
            "coda_xent_fwd_workspace_bytes": (S, [I, I, I]),
            "coda_xent_fwd": (I, [P, P, P, P, P, I, I, I, P, S, P]),
            "coda_xent_bwd_workspace_bytes": (S, [I, I, I]),
            "coda_xent_bwd": (I, [P, P, P, P, P, P, P, I, I, I, P, S, P]),
            "coda_qkv_rope_fwd": (I, [P, P, P, I, I, I, I, I, I, F, P, S, P]),
            "coda_qkv_rope_bwd_workspace_bytes": (S, [I, I, I, I, I]),
            "coda_qkv_rope_bwd": (I, [P, P, P, P, P, I, I, I, I, I, I, F, P, S, P]),
            "coda_mlp_block_fwd_workspace_bytes": (S, [I, I, I, I]),
            "coda_mlp_block_fwd": (I, [P] * 11 + [I, I, I, I, F, P, S, P]),
            "coda_mlp_block_bwd_workspace_bytes": (S, [I, I, I, I]),
            "coda_mlp_block_bwd": (I, [P] * 16 + [I, I, I, I, P, S, P]),
            "coda_swiglu_fwd_unfused": (I, [P, P, P, P, P, P, I, I, I, P, S, P]),
            "coda_swiglu_bwd_unfused_workspace_bytes": (S, [I, I, I]),
            "coda_swiglu_bwd_unfused": (I, [P, P, P, P, P, P, P, P, P, I, I, I, P, S, P]),
            "coda_grg_fwd_unfused_workspace_bytes": (S, [I, I, I, I]),
            "coda_grg_fwd_unfused": (I, [P] * 10 + [I, I, I, I, F, P, S, P]),
            "coda_grg_bwd_unfused_workspace_bytes": (S, [I, I, I, I]),
            "coda_grg_bwd_unfused": (I, [P] * 15 + [I, I, I, I, P, S, P]),
            "coda_grg_fwd_prefolded_static": (I, [P] * 8 + [I, I, I, I, F, P]),
            "coda_static_status_query": (I, [P, ctypes.POINTER(ctypes.c_uint32)]),
            "coda_quant_fp8": (I, [P] * 7 + [I, I, I, P]),
            "coda_quant_fp8_blocks": (I, [P, P, P, I, I, I, P]),
            "coda_gemm_fp8": (I, [P] * 5 + [I] * 10 + [P, S, P]),
            "coda_gemm_fp8_parts": (I, [I] * 7 + [ctypes.POINTER(I)] * 2),
            "coda_gemm_swiglu_fp8": (I, [P] * 8 + [I, I, I, P, S, P]),
            "coda_swiglu_fp8_bwd": (I, [P] * 9 + [I, I, I, P]),
            "coda_rmsnorm_fp8_fwd": (I, [P] * 7 + [I, I, F, P]),
            "coda_rmsnorm_fp8_bwd_workspace_bytes": (S, [I, I]),
            "coda_rmsnorm_fp8_bwd": (I, [P] * 7 + [I, I, P, S, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
            if name not in _UNRANGED and not name.endswith("_workspace_bytes"):
                setattr(lib, name, _Ranged(fn, name))
        _lib = lib
        return lib


# Host-side entry points that enqueue no GPU work get no NVTX range.
_UNRANGED = {"coda_status_string", "coda_version", "coda_set_wait_limit_ns", "coda_profile_arm",
             "coda_status_query", "coda_static_status_query", "coda_selftest_fp8_silence",
             "coda_shared_status", "coda_gemm_fp8_parts"}


class _Ranged:
    """A C entry point called inside an NVTX range of its own name, so profilers
    (ncu --nvtx, Nsight Systems) attribute each call's kernels to it.  Without
    a profiler attached the push and pop do nothing."""

    __slots__ = ("_fn", "_name")

    def __init__(self, fn, name):
        self._fn, self._name = fn, name

    def __call__(self, *args):
        torch.cuda.nvtx.range_push(self._name)
        try:
            return self._fn(*args)
        finally:
            torch.cuda.nvtx.range_pop()

    def __getattr__(self, key):
        return getattr(self._fn, key)

    def __setattr__(self, key, value):
        # restype / argtypes set by a caller go to the ctypes function itself
        if key in self.__slots__:
            object.__setattr__(self, key, value)
        else:
            setattr(self._fn, key, value)


def _status_string(status: int) -> str:
    try:
        return library().coda_status_string(int(status)).decode()
    except Exception:  # pragma: no cover - only when the library cannot load
        return "unknown"


def _check(status: int, where: str) -> None:
    if status != 0:
        raise CodaError(status, where)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _req(t: torch.Tensor, name: str, dtype=torch.bfloat16, shape=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


# ------------------------------------------------------------------ workspace

class Workspace:
    """A caller-owned device workspace whose first 256 bytes are the status word."""

    def __init__(self, nbytes: int, device=None):
        self.buf = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")

    @property
    def nbytes(self) -> int:
        return self.buf.numel()

    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    def clear(self) -> None:
        _check(library().coda_status_clear(self.ptr(), _stream()), "coda_status_clear")

    def query(self) -> tuple[int, int]:
        """Synchronise the current stream and return (status, detail)."""
        detail = ctypes.c_uint32(0)
        st = library().coda_status_query(self.ptr(), _stream(), ctypes.byref(detail))
        return int(st), int(detail.value)


_ws_cache: dict = {}


def workspace(nbytes: int, device=None) -> Workspace:
    """Per-device cached workspace grown on demand (zeroed when (re)allocated)."""
    dev = torch.device(device or "cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    ws = _ws_cache.get(dev)
    if ws is None or ws.nbytes < nbytes:
        ws = Workspace(nbytes, dev)
        _ws_cache[dev] = ws
    return ws


def set_wait_limit_ns(ns: int) -> None:
    library().coda_set_wait_limit_ns(int(ns))


# Kernel ids of the timing hook (coda_profile_arm): GEMMs by epilogue, light passes from 16,
# the 8-bit operators from 32.
EPI_STORE, EPI_RESID_RMS, EPI_SWIGLU, EPI_DN, EPI_SWIGLU_BWD, EPI_XENT, EPI_XENT_BWD, EPI_ROPE = range(8)
(KERNEL_FOLD_GAIN, KERNEL_RMS_ROWREDUCE, KERNEL_SWIGLU_BWD_ROWSTAT, KERNEL_COL_REDUCE, KERNEL_ROWCOEF_REDUCE,
 KERNEL_XENT_REDUCE, KERNEL_ROPE_UNROTATE) = range(16, 23)
(KERNEL_GEMM_FP8, KERNEL_GEMM_SWIGLU_FP8, KERNEL_QUANT_FP8, KERNEL_SWIGLU_FP8_BWD, KERNEL_RMSNORM_FP8_FWD,
 KERNEL_RMSNORM_FP8_BWD) = range(32, 38)


def profile_arm(kernel: int, start=None, stop=None) -> None:
    """Arm a one-shot torch.cuda.Event pair around the next launch, from this
    thread, of the kernel `kernel` names (EPI_* or KERNEL_*); pairs armed for
    the same kernel fire on its successive launches.  No events disarms all."""
    def handle(ev):
        if ev is None:
            return None
        if ev.cuda_event == 0:  # torch creates the CUDA event at its first record
            ev.record()
        return ctypes.c_void_p(ev.cuda_event)

    _check(library().coda_profile_arm(int(kernel), handle(start), handle(stop)), "coda_profile_arm")


def selftest_wait_timeout(ws: Workspace, limit_ns: int) -> None:
    """Launch the bounded-wait self-test (a wait that must time out) on the current stream."""
    _check(library().coda_selftest_wait_timeout(ws.ptr(), int(limit_ns), _stream()), "coda_selftest_wait_timeout")


FP8_ROLE_LOADS, FP8_ROLE_MMA, FP8_ROLE_SCALES = 1, 2, 3


def selftest_fp8_silence(role: int, cta: int = 0) -> None:
    """Keep one role of block `cta` silent in this thread's next 8-bit product, so that its waits run out
    (role 0 disarms); see coda_selftest_fp8_silence."""
    _check(library().coda_selftest_fp8_silence(int(role), int(cta)), "coda_selftest_fp8_silence")


# ------------------------------------------------------------------ entry points

def gemm(A: torch.Tensor, B: torch.Tensor, M: int, N: int, K: int, a_mn_major: bool = False,
         b_mn_major: bool = False, out: torch.Tensor | None = None, ws: Workspace | None = None) -> torch.Tensor:
    """C[M,N] = op(A) op(B)^T (bf16 out, fp32 accumulate); see coda_gemm in include/coda.h."""
    lib = library()
    _req(A, "A", shape=(K, M) if a_mn_major else (M, K))
    _req(B, "B", shape=(K, N) if b_mn_major else (N, K))
    C = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=A.device)
    _req(C, "C", shape=(M, N))
    ws = ws or workspace(lib.coda_gemm_workspace_bytes(), A.device)
    _check(lib.coda_gemm(_ptr(A), _ptr(B), _ptr(C), M, N, K, int(a_mn_major), int(b_mn_major),
                         ws.ptr(), ws.nbytes, _stream()), "coda_gemm")
    return C


def gemm_swiglu(A, Wgu, r=None, save_ab: bool = True, out: dict | None = None,
                ws: Workspace | None = None) -> dict:
    """Y = silu(r*(A Wgu^T)_gate) * (r*(A Wgu^T)_up), AB = [a | b]; see coda_gemm_swiglu."""
    lib = library()
    M, K = A.shape
    F = Wgu.shape[0] // 2
    _req(A, "A"), _req(Wgu, "Wgu", shape=(2 * F, K))
    if r is not None:
        _req(r, "r", torch.float32, (M,))
    o = dict(out or {})
    if "Y" not in o:
        o["Y"] = torch.empty(M, F, dtype=torch.bfloat16, device=A.device)
    if save_ab:
        if "AB" not in o:
            o["AB"] = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=A.device)
    ws = ws or workspace(lib.coda_gemm_workspace_bytes(), A.device)
    _check(lib.coda_gemm_swiglu(_ptr(A), _ptr(Wgu), _ptr(r), _ptr(o["Y"]), _ptr(o.get("AB") if save_ab else None),
                                M, K, F, ws.ptr(), ws.nbytes, _stream()), "coda_gemm_swiglu")
    return o


def fold_gain(W2: torch.Tensor, g: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """W2g = W2 * g (per column), bf16; see coda_fold_gain."""
    N, d = W2.shape
    _req(W2, "W2")
    _req(g, "g", shape=(d,))
    W2g = out if out is not None else torch.empty_like(W2)
    _req(W2g, "W2g", shape=(N, d))
    _check(library().coda_fold_gain(_ptr(W2), _ptr(g), _ptr(W2g), d, N, _stream()), "coda_fold_gain")
    return W2g


def grg_fwd(X, W1, R, g, W2, eps: float, W2g=None, save_ab: bool = True, out: dict | None = None,
            ws: Workspace | None = None) -> dict:
    """Fused GEMM-Residual-PartialRMS-GEMM-SwiGLU forward; returns H, r, Y, AB."""
    lib = library()
    M, K = X.shape
    d = W1.shape[0]
    N = W2.shape[0]
    F = N // 2
    _req(X, "X"), _req(W1, "W1", shape=(d, K)), _req(R, "R", shape=(M, d))
    _req(g, "g", shape=(d,)), _req(W2, "W2", shape=(N, d))
    if W2g is not None:
        _req(W2g, "W2g", shape=(N, d))
    o = dict(out or {})
    dev = X.device
    if "H" not in o:
        o["H"] = torch.empty(M, d, dtype=torch.bfloat16, device=dev)
    if "r" not in o:
        o["r"] = torch.empty(M, dtype=torch.float32, device=dev)
    if "Y" not in o:
        o["Y"] = torch.empty(M, F, dtype=torch.bfloat16, device=dev)
    if save_ab and "AB" not in o:
        o["AB"] = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    _req(o["H"], "H", shape=(M, d)), _req(o["r"], "r", torch.float32, (M,)), _req(o["Y"], "Y", shape=(M, F))
    AB = o.get("AB") if save_ab else None
    if AB is not None:
        _req(AB, "AB", shape=(M, N))
    need = lib.coda_grg_fwd_workspace_bytes(M, K, d, N, int(W2g is not None))
    ws = ws or workspace(need, dev)
    _check(lib.coda_grg_fwd(_ptr(X), _ptr(W1), _ptr(R), _ptr(g), _ptr(W2), _ptr(W2g), _ptr(o["H"]),
                            _ptr(o["r"]), _ptr(o["Y"]), _ptr(AB), M, K, d, N, float(eps),
                            ws.ptr(), ws.nbytes, _stream()), "coda_grg_fwd")
    return o


def grg_fwd_prefolded_static(X, W1, R, W2g, eps: float, save_ab: bool = True, out: dict | None = None) -> dict:
    """The forward for callers that cannot allocate device memory: the same
    kernels as grg_fwd given a pre-folded W2g, with the scratch in the
    library's static device array (no workspace).  Outputs are allocated here
    unless passed in `out`; a caller that must not allocate passes them all.
    Calls that overlap on the GPU share the static array and must be
    serialised.  Returns H, r, Y, AB."""
    lib = library()
    M, K = X.shape
    d = W1.shape[0]
    N = W2g.shape[0]
    F = N // 2
    _req(X, "X"), _req(W1, "W1", shape=(d, K)), _req(R, "R", shape=(M, d)), _req(W2g, "W2g", shape=(N, d))
    o = dict(out or {})
    dev = X.device
    for k, shape, dt in (("H", (M, d), torch.bfloat16), ("r", (M,), torch.float32), ("Y", (M, F), torch.bfloat16)):
        if k not in o:
            o[k] = torch.empty(*shape, dtype=dt, device=dev)
        _req(o[k], k, dt, shape)
    if save_ab and "AB" not in o:
        o["AB"] = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    AB = o.get("AB") if save_ab else None
    if AB is not None:
        _req(AB, "AB", shape=(M, N))
    _check(lib.coda_grg_fwd_prefolded_static(_ptr(X), _ptr(W1), _ptr(R), _ptr(W2g), _ptr(o["H"]), _ptr(o["r"]),
                                             _ptr(o["Y"]), _ptr(AB), M, K, d, N, float(eps), _stream()),
           "coda_grg_fwd_prefolded_static")
    return o


def static_status() -> tuple[int, int]:
    """Synchronise the current stream and return (status, detail) of the last
    grg_fwd_prefolded_static call on the current device."""
    detail = ctypes.c_uint32(0)
    st = library().coda_static_status_query(_stream(), ctypes.byref(detail))
    return int(st), int(detail.value)


def grg_fwd_hg(X, W1, R, g, W2, eps: float, save_ab: bool = True, keep_hg: bool = False, out: dict | None = None,
               ws: Workspace | None = None) -> dict:
    """Forward with the gain on the activation side (Hg = H*g from GEMM1's epilogue); returns H, r, Y, AB (, Hg)."""
    lib = library()
    M, K = X.shape
    d = W1.shape[0]
    N = W2.shape[0]
    F = N // 2
    _req(X, "X"), _req(W1, "W1", shape=(d, K)), _req(R, "R", shape=(M, d))
    _req(g, "g", shape=(d,)), _req(W2, "W2", shape=(N, d))
    o = dict(out or {})
    dev = X.device
    want = [("H", (M, d), torch.bfloat16), ("r", (M,), torch.float32), ("Y", (M, F), torch.bfloat16)]
    if save_ab:
        want.append(("AB", (M, N), torch.bfloat16))
    if keep_hg:
        want.append(("Hg", (M, d), torch.bfloat16))
    for k, shape, dt in want:
        if k not in o:
            o[k] = torch.empty(*shape, dtype=dt, device=dev)
        _req(o[k], k, dt, shape)
    Hg = o.get("Hg") if keep_hg else None
    ws = ws or workspace(lib.coda_grg_fwd_hg_workspace_bytes(M, K, d, N, int(Hg is not None)), dev)
    _check(lib.coda_grg_fwd_hg(_ptr(X), _ptr(W1), _ptr(R), _ptr(g), _ptr(W2), _ptr(o["H"]), _ptr(Hg), _ptr(o["r"]),
                               _ptr(o["Y"]), _ptr(o.get("AB") if save_ab else None), M, K, d, N, float(eps),
                               ws.ptr(), ws.nbytes, _stream()), "coda_grg_fwd_hg")
    return o


def grg_bwd(dY, X, W1, H, r, AB, g, W2, dH_in=None, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Fused backward of the block; returns dX, dR, dW1, dW2, dg."""
    lib = library()
    M, K = X.shape
    d = W1.shape[0]
    N = W2.shape[0]
    F = N // 2
    _req(dY, "dY", shape=(M, F)), _req(X, "X"), _req(W1, "W1", shape=(d, K)), _req(H, "H", shape=(M, d))
    _req(r, "r", torch.float32, (M,)), _req(AB, "AB", shape=(M, N)), _req(g, "g", shape=(d,))
    _req(W2, "W2", shape=(N, d))
    if dH_in is not None:
        _req(dH_in, "dH_in", shape=(M, d))
    o = dict(out or {})
    dev = X.device
    for k, shape, dt in (("dX", (M, K), torch.bfloat16), ("dR", (M, d), torch.bfloat16),
                         ("dW1", (d, K), torch.bfloat16), ("dW2", (N, d), torch.bfloat16),
                         ("dg", (d,), torch.float32)):
        if k not in o:
            o[k] = torch.empty(*shape, dtype=dt, device=dev)
    ws = ws or workspace(lib.coda_grg_bwd_workspace_bytes(M, K, d, N), dev)
    _check(lib.coda_grg_bwd(_ptr(dY), _ptr(dH_in), _ptr(X), _ptr(W1), _ptr(H), _ptr(r), _ptr(AB), _ptr(g),
                            _ptr(W2), _ptr(o["dX"]), _ptr(o["dR"]), _ptr(o["dW1"]), _ptr(o["dW2"]), _ptr(o["dg"]),
                            M, K, d, N, ws.ptr(), ws.nbytes, _stream()), "coda_grg_bwd")
    return o


def swiglu_fwd(X, Wgu, Wdown, save_ab: bool = True, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """SwiGLU MLP forward; returns Y, AB, Out."""
    lib = library()
    M, d = X.shape
    F = Wgu.shape[0] // 2
    _req(X, "X"), _req(Wgu, "Wgu", shape=(2 * F, d)), _req(Wdown, "Wdown", shape=(d, F))
    o = dict(out or {})
    dev = X.device
    if "Y" not in o:
        o["Y"] = torch.empty(M, F, dtype=torch.bfloat16, device=dev)
    if save_ab:
        if "AB" not in o:
            o["AB"] = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=dev)
    if "Out" not in o:
        o["Out"] = torch.empty(M, d, dtype=torch.bfloat16, device=dev)
    ws = ws or workspace(lib.coda_swiglu_fwd_workspace_bytes(M, d, F), dev)
    _check(lib.coda_swiglu_fwd(_ptr(X), _ptr(Wgu), _ptr(Wdown), _ptr(o["Y"]), _ptr(o.get("AB") if save_ab else None),
                               _ptr(o["Out"]), M, d, F, ws.ptr(), ws.nbytes, _stream()), "coda_swiglu_fwd")
    return o


def swiglu_bwd(dOut, X, Wgu, Wdown, Y, AB, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """SwiGLU MLP backward; returns dX, dWgu, dWdown."""
    lib = library()
    M, d = X.shape
    F = Wgu.shape[0] // 2
    _req(dOut, "dOut", shape=(M, d)), _req(X, "X"), _req(Wgu, "Wgu", shape=(2 * F, d))
    _req(Wdown, "Wdown", shape=(d, F)), _req(Y, "Y", shape=(M, F)), _req(AB, "AB", shape=(M, 2 * F))
    o = dict(out or {})
    dev = X.device
    if "dX" not in o:
        o["dX"] = torch.empty(M, d, dtype=torch.bfloat16, device=dev)
    if "dWgu" not in o:
        o["dWgu"] = torch.empty(2 * F, d, dtype=torch.bfloat16, device=dev)
    if "dWdown" not in o:
        o["dWdown"] = torch.empty(d, F, dtype=torch.bfloat16, device=dev)
    ws = ws or workspace(lib.coda_swiglu_bwd_workspace_bytes(M, d, F), dev)
    _check(lib.coda_swiglu_bwd(_ptr(dOut), _ptr(X), _ptr(Wgu), _ptr(Wdown), _ptr(Y), _ptr(AB), _ptr(o["dX"]),
                               _ptr(o["dWgu"]), _ptr(o["dWdown"]), M, d, F, ws.ptr(), ws.nbytes, _stream()),
           "coda_swiglu_bwd")
    return o


# ------------------------------------------------------------------ unfused comparison sequence

def grg_fwd_unfused(X, W1, R, g, W2, eps: float, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Operator-by-operator forward (measurement/comparison only); returns H, r, Y, AB, U."""
    lib = library()
    M, K = X.shape
    d = W1.shape[0]
    N = W2.shape[0]
    F = N // 2
    _req(X, "X"), _req(W1, "W1", shape=(d, K)), _req(R, "R", shape=(M, d))
    _req(g, "g", shape=(d,)), _req(W2, "W2", shape=(N, d))
    o = dict(out or {})
    dev = X.device
    for k, shape, dt in (("H", (M, d), torch.bfloat16), ("r", (M,), torch.float32), ("Y", (M, F), torch.bfloat16),
                         ("AB", (M, N), torch.bfloat16), ("U", (M, d), torch.bfloat16)):
        if k not in o:
            o[k] = torch.empty(*shape, dtype=dt, device=dev)
        _req(o[k], k, dt, shape)
    ws = ws or workspace(lib.coda_grg_fwd_unfused_workspace_bytes(M, K, d, N), dev)
    _check(lib.coda_grg_fwd_unfused(_ptr(X), _ptr(W1), _ptr(R), _ptr(g), _ptr(W2), _ptr(o["H"]), _ptr(o["r"]),
                                    _ptr(o["Y"]), _ptr(o["AB"]), _ptr(o["U"]), M, K, d, N, float(eps),
                                    ws.ptr(), ws.nbytes, _stream()), "coda_grg_fwd_unfused")
    return o


def grg_bwd_unfused(dY, X, W1, H, r, AB, U, g, W2, dH_in=None, out: dict | None = None,
                    ws: Workspace | None = None) -> dict:
    """Operator-by-operator backward (measurement/comparison only); returns dX, dR, dW1, dW2, dg."""
    lib = library()
    M, K = X.shape
    d = W1.shape[0]
    N = W2.shape[0]
    F = N // 2
    _req(dY, "dY", shape=(M, F)), _req(X, "X"), _req(W1, "W1", shape=(d, K)), _req(H, "H", shape=(M, d))
    _req(r, "r", torch.float32, (M,)), _req(AB, "AB", shape=(M, N)), _req(U, "U", shape=(M, d))
    _req(g, "g", shape=(d,)), _req(W2, "W2", shape=(N, d))
    if dH_in is not None:
        _req(dH_in, "dH_in", shape=(M, d))
    o = dict(out or {})
    dev = X.device
    for k, shape, dt in (("dX", (M, K), torch.bfloat16), ("dR", (M, d), torch.bfloat16),
                         ("dW1", (d, K), torch.bfloat16), ("dW2", (N, d), torch.bfloat16),
                         ("dg", (d,), torch.float32)):
        if k not in o:
            o[k] = torch.empty(*shape, dtype=dt, device=dev)
    ws = ws or workspace(lib.coda_grg_bwd_unfused_workspace_bytes(M, K, d, N), dev)
    _check(lib.coda_grg_bwd_unfused(_ptr(dY), _ptr(dH_in), _ptr(X), _ptr(W1), _ptr(H), _ptr(r), _ptr(AB), _ptr(U),
                                    _ptr(g), _ptr(W2), _ptr(o["dX"]), _ptr(o["dR"]), _ptr(o["dW1"]), _ptr(o["dW2"]),
                                    _ptr(o["dg"]), M, K, d, N, ws.ptr(), ws.nbytes, _stream()),
           "coda_grg_bwd_unfused")
    return o


# ------------------------------------------------------------------ cross-entropy on the LM head

def xent_fwd(X, W, targets, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Per-row cross-entropy of X W^T without materialising the logits; returns loss, lse (fp32 [M])."""
    lib = library()
    M, d = X.shape
    V = W.shape[0]
    _req(X, "X"), _req(W, "W", shape=(V, d)), _req(targets, "targets", torch.int32, (M,))
    o = dict(out or {})
    for k in ("loss", "lse"):
        if k not in o:
            o[k] = torch.empty(M, dtype=torch.float32, device=X.device)
        _req(o[k], k, torch.float32, (M,))
    ws = ws or workspace(lib.coda_xent_fwd_workspace_bytes(M, d, V), X.device)
    _check(lib.coda_xent_fwd(_ptr(X), _ptr(W), _ptr(targets), _ptr(o["loss"]), _ptr(o["lse"]), M, d, V,
                             ws.ptr(), ws.nbytes, _stream()), "coda_xent_fwd")
    return o


def xent_bwd(X, W, targets, lse, dloss, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Gradients of sum_i dloss_i loss_i; returns dX [M,d], dW [V,d] (bf16)."""
    lib = library()
    M, d = X.shape
    V = W.shape[0]
    _req(X, "X"), _req(W, "W", shape=(V, d)), _req(targets, "targets", torch.int32, (M,))
    _req(lse, "lse", torch.float32, (M,)), _req(dloss, "dloss", torch.float32, (M,))
    o = dict(out or {})
    if "dX" not in o:
        o["dX"] = torch.empty(M, d, dtype=torch.bfloat16, device=X.device)
    if "dW" not in o:
        o["dW"] = torch.empty(V, d, dtype=torch.bfloat16, device=X.device)
    ws = ws or workspace(lib.coda_xent_bwd_workspace_bytes(M, d, V), X.device)
    _check(lib.coda_xent_bwd(_ptr(X), _ptr(W), _ptr(targets), _ptr(lse), _ptr(dloss), _ptr(o["dX"]), _ptr(o["dW"]),
                             M, d, V, ws.ptr(), ws.nbytes, _stream()), "coda_xent_bwd")
    return o


# ------------------------------------------------------------------ QKV projection with RoPE

def qkv_rope_fwd(X, Wqkv, n_q: int, n_kv: int, head_dim: int, seq_len: int, base: float = 10000.0,
                 out: torch.Tensor | None = None, ws: Workspace | None = None) -> torch.Tensor:
    """QKV = X Wqkv^T with RoPE on the q and k heads applied in the GEMM epilogue."""
    lib = library()
    M, d = X.shape
    ncols = (n_q + 2 * n_kv) * head_dim
    _req(X, "X"), _req(Wqkv, "Wqkv", shape=(ncols, d))
    Q = out if out is not None else torch.empty(M, ncols, dtype=torch.bfloat16, device=X.device)
    _req(Q, "QKV", shape=(M, ncols))
    ws = ws or workspace(lib.coda_gemm_workspace_bytes(), X.device)
    _check(lib.coda_qkv_rope_fwd(_ptr(X), _ptr(Wqkv), _ptr(Q), M, d, n_q, n_kv, head_dim, seq_len, float(base),
                                 ws.ptr(), ws.nbytes, _stream()), "coda_qkv_rope_fwd")
    return Q


def qkv_rope_bwd(dQKV, X, Wqkv, n_q: int, n_kv: int, head_dim: int, seq_len: int, base: float = 10000.0,
                 out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Backward of qkv_rope_fwd; returns dX, dW."""
    lib = library()
    M, d = X.shape
    ncols = (n_q + 2 * n_kv) * head_dim
    _req(dQKV, "dQKV", shape=(M, ncols)), _req(X, "X"), _req(Wqkv, "Wqkv", shape=(ncols, d))
    o = dict(out or {})
    if "dX" not in o:
        o["dX"] = torch.empty(M, d, dtype=torch.bfloat16, device=X.device)
    if "dW" not in o:
        o["dW"] = torch.empty(ncols, d, dtype=torch.bfloat16, device=X.device)
    ws = ws or workspace(lib.coda_qkv_rope_bwd_workspace_bytes(M, d, n_q, n_kv, head_dim), X.device)
    _check(lib.coda_qkv_rope_bwd(_ptr(dQKV), _ptr(X), _ptr(Wqkv), _ptr(o["dX"]), _ptr(o["dW"]), M, d, n_q, n_kv,
                                 head_dim, seq_len, float(base), ws.ptr(), ws.nbytes, _stream()), "coda_qkv_rope_bwd")
    return o


# ------------------------------------------------------------------ full MLP block

def mlp_block_fwd(X, W1, R, g, W2, Wdown, eps: float, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Block forward plus the down projection with the residual epilogue; returns H, r, Y, AB, Out."""
    lib = library()
    M, K = X.shape
    d = W1.shape[0]
    N = W2.shape[0]
    F = N // 2
    _req(X, "X"), _req(W1, "W1", shape=(d, K)), _req(R, "R", shape=(M, d)), _req(g, "g", shape=(d,))
    _req(W2, "W2", shape=(N, d)), _req(Wdown, "Wdown", shape=(d, F))
    o = dict(out or {})
    for k, shape, dt in (("H", (M, d), torch.bfloat16), ("r", (M,), torch.float32), ("Y", (M, F), torch.bfloat16),
                         ("AB", (M, N), torch.bfloat16), ("Out", (M, d), torch.bfloat16)):
        if k not in o:
            o[k] = torch.empty(*shape, dtype=dt, device=X.device)
        _req(o[k], k, dt, shape)
    ws = ws or workspace(lib.coda_mlp_block_fwd_workspace_bytes(M, K, d, F), X.device)
    _check(lib.coda_mlp_block_fwd(_ptr(X), _ptr(W1), _ptr(R), _ptr(g), _ptr(W2), _ptr(Wdown), _ptr(o["H"]),
                                  _ptr(o["r"]), _ptr(o["Y"]), _ptr(o["AB"]), _ptr(o["Out"]), M, K, d, F, float(eps),
                                  ws.ptr(), ws.nbytes, _stream()), "coda_mlp_block_fwd")
    return o


def mlp_block_bwd(dOut, X, W1, H, r, AB, Y, g, W2, Wdown, out: dict | None = None,
                  ws: Workspace | None = None) -> dict:
    """Backward of the full block; returns dX, dR, dW1, dW2, dg, dWdown."""
    lib = library()
    M, K = X.shape
    d = W1.shape[0]
    N = W2.shape[0]
    F = N // 2
    _req(dOut, "dOut", shape=(M, d)), _req(X, "X"), _req(W1, "W1", shape=(d, K)), _req(H, "H", shape=(M, d))
    _req(r, "r", torch.float32, (M,)), _req(AB, "AB", shape=(M, N)), _req(Y, "Y", shape=(M, F))
    _req(g, "g", shape=(d,)), _req(W2, "W2", shape=(N, d)), _req(Wdown, "Wdown", shape=(d, F))
    o = dict(out or {})
    for k, shape, dt in (("dX", (M, K), torch.bfloat16), ("dR", (M, d), torch.bfloat16),
                         ("dW1", (d, K), torch.bfloat16), ("dW2", (N, d), torch.bfloat16),
                         ("dg", (d,), torch.float32), ("dWdown", (d, F), torch.bfloat16)):
        if k not in o:
            o[k] = torch.empty(*shape, dtype=dt, device=X.device)
    ws = ws or workspace(lib.coda_mlp_block_bwd_workspace_bytes(M, K, d, F), X.device)
    _check(lib.coda_mlp_block_bwd(_ptr(dOut), _ptr(X), _ptr(W1), _ptr(H), _ptr(r), _ptr(AB), _ptr(Y), _ptr(g),
                                  _ptr(W2), _ptr(Wdown), _ptr(o["dX"]), _ptr(o["dR"]), _ptr(o["dW1"]), _ptr(o["dW2"]),
                                  _ptr(o["dg"]), _ptr(o["dWdown"]), M, K, d, F, ws.ptr(), ws.nbytes, _stream()),
           "coda_mlp_block_bwd")
    return o


def swiglu_fwd_unfused(X, Wgu, Wdown, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """The SwiGLU MLP forward operator by operator (measurement only); returns Y, AB, Out."""
    lib = library()
    M, d = X.shape
    F = Wgu.shape[0] // 2
    _req(X, "X"), _req(Wgu, "Wgu", shape=(2 * F, d)), _req(Wdown, "Wdown", shape=(d, F))
    o = dict(out or {})
    for k, shape in (("Y", (M, F)), ("AB", (M, 2 * F)), ("Out", (M, d))):
        if k not in o:
            o[k] = torch.empty(*shape, dtype=torch.bfloat16, device=X.device)
    ws = ws or workspace(lib.coda_gemm_workspace_bytes(), X.device)
    _check(lib.coda_swiglu_fwd_unfused(_ptr(X), _ptr(Wgu), _ptr(Wdown), _ptr(o["Y"]), _ptr(o["AB"]), _ptr(o["Out"]),
                                       M, d, F, ws.ptr(), ws.nbytes, _stream()), "coda_swiglu_fwd_unfused")
    return o


def swiglu_bwd_unfused(dOut, X, Wgu, Wdown, Y, AB, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """The SwiGLU MLP backward operator by operator (measurement only); returns dX, dWgu, dWdown."""
    lib = library()
    M, d = X.shape
    F = Wgu.shape[0] // 2
    _req(dOut, "dOut", shape=(M, d)), _req(Y, "Y", shape=(M, F)), _req(AB, "AB", shape=(M, 2 * F))
    o = dict(out or {})
    for k, shape in (("dX", (M, d)), ("dWgu", (2 * F, d)), ("dWdown", (d, F))):
        if k not in o:
            o[k] = torch.empty(*shape, dtype=torch.bfloat16, device=X.device)
    ws = ws or workspace(lib.coda_swiglu_bwd_unfused_workspace_bytes(M, d, F), X.device)
    _check(lib.coda_swiglu_bwd_unfused(_ptr(dOut), _ptr(X), _ptr(Wgu), _ptr(Wdown), _ptr(Y), _ptr(AB), _ptr(o["dX"]),
                                       _ptr(o["dWgu"]), _ptr(o["dWdown"]), M, d, F, ws.ptr(), ws.nbytes, _stream()),
           "coda_swiglu_bwd_unfused")
    return o


# ------------------------------------------------------------------ 8-bit operands

_FP8 = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}


def _cdiv(a: int, b: int) -> int:
    return -(-a // b)


def _fp8(dtype, name: str) -> int:
    if dtype not in _FP8:
        raise TypeError(f"{name} must be torch.float8_e4m3fn or torch.float8_e5m2, got {dtype}")
    return _FP8[dtype]


def _no_int(*sizes) -> None:
    """Refuse sizes of which one is no C int (ctypes would cut it down to one)."""
    raise ValueError(f"sizes must be from 0 to 2^31 - 1, got {sizes}")


def _req2(t, name: str) -> tuple:
    """Rows and columns of the matrix that fixes an entry point's sizes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {t.dim()}")
    R, C = t.shape
    if (R | C) >> 31:
        _no_int(R, C)
    return R, C


def _in(t, name: str, dtype, shape, dev=None):
    """The device address of an argument, after _req's checks; it must lie on `dev`."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.shape == shape
            and t.is_contiguous()):
        _req(t, name, dtype, shape)  # says what is wrong
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    return t.data_ptr()


def _ws_on(ws: Workspace, dev) -> Workspace:
    if ws.buf.device != dev:
        raise ValueError(f"ws is on {ws.buf.device}, the tensors on {dev}")
    return ws


def _new(shape: tuple, dtype, dev):
    """A new dense vector or matrix (empty_strided: a third less host time than new_empty)."""
    return torch.empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=dev)


def _out(o: dict, key: str, shape, dtype, dev):
    """The device address of the caller's output o[key], checked, or of a new one on `dev`."""
    t = o.get(key)
    if t is None:
        t = o[key] = _new(shape, dtype, dev)
        return t.data_ptr()
    return _in(t, key, dtype, shape, dev)


def _call(name: str, dev, *args) -> None:
    """Call an entry point on `dev`'s current stream (the device need not be the current one)."""
    if torch._C._cuda_getDevice() == dev.index:
        _check(getattr(_lib, name)(*args, torch._C._cuda_getCurrentRawStream(dev.index)), name)
    else:
        with torch.cuda.device(dev):
            _check(getattr(_lib, name)(*args, torch._C._cuda_getCurrentRawStream(dev.index)), name)


class _SharedStatus(Workspace):
    """The library's own status word of a device (coda_shared_status)."""

    def __init__(self, dev):
        ptr = _c_void_p()
        with torch.cuda.device(dev):
            _check(library().coda_shared_status(ctypes.byref(ptr)), "coda_shared_status")
            word = {"shape": (256,), "typestr": "|u1", "data": (ptr.value, False), "version": 2}
            self.buf = torch.as_tensor(types.SimpleNamespace(__cuda_array_interface__=word), device=dev)


_status_ws: dict = {}   # by device index, from the first call outside a capture on


def _status_workspace(dev) -> Workspace:
    """The device's status word for calls that need no other scratch: the same
    memory in every call, thread and captured graph, zero from the start."""
    ws = _status_ws.get(dev.index)
    if ws is None:
        ws = _SharedStatus(dev)
        if not torch.cuda.is_current_stream_capturing():
            _status_ws[dev.index] = ws
    return ws


def fp8_status(device=None, clear: bool = False) -> tuple[int, int]:
    """Synchronise the current stream and return (status, detail) of the 8-bit
    products that were given no workspace on this device.  An error stays until
    `clear`."""
    dev = torch.device("cuda" if device is None else device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        ws = _status_workspace(dev)
        status = ws.query()
        if clear:
            ws.clear()
        return status


def quant_fp8(X, rows: bool = True, cols: bool = False, rowvec=None, colvec=None, fmt=torch.float8_e4m3fn,
              out: dict | None = None) -> dict:
    """X (bf16 [R, C], optionally scaled by rowvec fp32 [R] and colvec bf16 [C])
    in 8 bits with a scale per 128 values, in one pass; see coda_quant_fp8.

    rows: Qr [R, C], Sr [ceil(C/128), R], one scale per row and 128 columns;
    cols: Qc [R, C], Sc [ceil(R/128), C], one scale per column and 128 rows."""
    library()
    R, C = _req2(X, "X")
    x = _in(X, "X", torch.bfloat16, (R, C))
    f = _fp8(fmt, "fmt")
    if not rows and not cols:
        raise ValueError("rows or cols (or both) must be asked for")
    dev = X.device
    rv = None if rowvec is None else _in(rowvec, "rowvec", torch.float32, (R,), dev)
    cv = None if colvec is None else _in(colvec, "colvec", torch.bfloat16, (C,), dev)
    o = dict(out or {})
    qr = sr = qc = sc = None
    if rows:
        qr, sr = _out(o, "Qr", (R, C), fmt, dev), _out(o, "Sr", (_cdiv(C, 128), R), torch.float32, dev)
    if cols:
        qc, sc = _out(o, "Qc", (R, C), fmt, dev), _out(o, "Sc", (_cdiv(R, 128), C), torch.float32, dev)
    _call("coda_quant_fp8", dev, x, rv, cv, qr, sr, qc, sc, R, C, f)
    return o


def quant_fp8_blocks(W, fmt=torch.float8_e4m3fn, out: dict | None = None) -> dict:
    """A weight W (bf16 [R, C]) in 8 bits with a scale per 128 x 128 block: Q, S
    [ceil(R/128), ceil(C/128)]; see coda_quant_fp8_blocks."""
    library()
    R, C = _req2(W, "W")
    w = _in(W, "W", torch.bfloat16, (R, C))
    f = _fp8(fmt, "fmt")
    o, dev = dict(out or {}), W.device
    _call("coda_quant_fp8_blocks", dev, w, _out(o, "Q", (R, C), fmt, dev),
          _out(o, "S", (_cdiv(R, 128), _cdiv(C, 128)), torch.float32, dev), R, C, f)
    return o


def gemm_fp8(A, SA, B, SB, M: int, N: int, K: int, a_mn_major: bool = False, b_mn_major: bool = False,
             b_blocks: bool = True, out_dtype=torch.bfloat16, accumulate: bool = False,
             out: torch.Tensor | None = None, ws: Workspace | None = None) -> torch.Tensor:
    """C[M,N] = op(A) op(B)^T over 8-bit operands; see coda_gemm_fp8.

    A [M, K] with row scales, or [K, M] (a_mn_major) with column scales: SA
    [ceil(K/128), M].  B [N, K] or [K, N] (b_mn_major), SB in 128 x 128 blocks of
    B as stored, or (b_blocks=False) [ceil(K/128), N].  out_dtype bf16 or fp32;
    accumulate adds to an fp32 `out`.  Without `ws`, fp8_status() reads the
    status word."""
    library()
    if not (isinstance(A, torch.Tensor) and isinstance(B, torch.Tensor)):
        raise TypeError("A and B must be torch.Tensors")
    fa, fb = _fp8(A.dtype, "A"), _fp8(B.dtype, "B")
    if (M | N | K) >> 31:
        _no_int(M, N, K)
    dev = A.device
    kb, nb = _cdiv(K, 128), _cdiv(N, 128)
    a = _in(A, "A", A.dtype, (K, M) if a_mn_major else (M, K))
    b = _in(B, "B", B.dtype, (K, N) if b_mn_major else (N, K), dev)
    sa = _in(SA, "SA", torch.float32, (kb, M), dev)
    sb = _in(SB, "SB", torch.float32, ((kb, nb) if b_mn_major else (nb, kb)) if b_blocks else (kb, N), dev)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")
    if accumulate and (out is None or out_dtype != torch.float32):
        raise ValueError("accumulate adds to an fp32 `out`: give one, with out_dtype=torch.float32")
    if out is None:
        C = _new((M, N), out_dtype, dev)
        c = C.data_ptr()
    else:
        C, c = out, _in(out, "C", out_dtype, (M, N), dev)
    ws = _status_workspace(dev) if ws is None else _ws_on(ws, dev)
    _call("coda_gemm_fp8", dev, a, sa, b, sb, c, M, N, K, int(a_mn_major), int(b_mn_major), fa, fb, int(b_blocks),
          int(out_dtype == torch.float32), int(accumulate), ws.buf.data_ptr(), ws.nbytes)
    return C


def gemm_fp8_parts(M: int, N: int, K: int, a_mn_major: bool = False, b_mn_major: bool = False, b_blocks: bool = True,
                   out_dtype=torch.bfloat16) -> tuple[bool, int]:
    """(few rows' kernel, CTAs or CTA pairs that share each tile's reduction) of such a product on the current
    device; see coda_gemm_fp8_parts."""
    few, parts = _c_int(0), _c_int(0)
    if (M | N | K) >> 31:
        _no_int(M, N, K)
    _check(library().coda_gemm_fp8_parts(M, N, K, int(a_mn_major), int(b_mn_major), int(b_blocks),
                                         int(out_dtype == torch.float32), ctypes.byref(few), ctypes.byref(parts)),
           "coda_gemm_fp8_parts")
    return bool(few.value), parts.value


def gemm_swiglu_fp8(A, SA, Wgu, SW, save_ab: bool = True, out: dict | None = None,
                    ws: Workspace | None = None) -> dict:
    """Gate/up product with SwiGLU on 8-bit operands (e4m3): Y [M, F] with SY
    [F/128, M] and, with save_ab, the checkpoint AB = [a | b] [M, 2F] with SAB
    [2F/128, M]; see coda_gemm_swiglu_fp8."""
    library()
    e4m3 = torch.float8_e4m3fn
    M, K = _req2(A, "A")
    F = _req2(Wgu, "Wgu")[0] // 2
    dev = A.device
    kb, fb = _cdiv(K, 128), F // 128
    a = _in(A, "A", e4m3, (M, K))
    w = _in(Wgu, "Wgu", e4m3, (2 * F, K), dev)
    if F % 128 != 0:
        raise CodaError(2, "coda_gemm_swiglu_fp8")
    sa, sw = _in(SA, "SA", torch.float32, (kb, M), dev), _in(SW, "SW", torch.float32, (2 * fb, kb), dev)
    o = dict(out or {})
    y, sy = _out(o, "Y", (M, F), e4m3, dev), _out(o, "SY", (fb, M), torch.float32, dev)
    ab = sab = None
    if save_ab:
        ab, sab = _out(o, "AB", (M, 2 * F), e4m3, dev), _out(o, "SAB", (2 * fb, M), torch.float32, dev)
    ws = _status_workspace(dev) if ws is None else _ws_on(ws, dev)
    _call("coda_gemm_swiglu_fp8", dev, a, sa, w, sw, y, sy, ab, sab, M, K, F, ws.buf.data_ptr(), ws.nbytes)
    return o


def swiglu_fp8_bwd(dY, AB, SAB, cols: bool = True, fmt=torch.float8_e4m3fn, out: dict | None = None) -> dict:
    """SwiGLU backward from the 8-bit checkpoint: dA = [da | db] (rows form, SdA)
    and, with cols, dAc, SdAc and Yc, SYc (columns form, the operands of the
    weight gradients); see coda_swiglu_fp8_bwd.  fmt is dA's and dAc's type."""
    library()
    e4m3 = torch.float8_e4m3fn
    M, F = _req2(dY, "dY")
    dev = dY.device
    fb, mb = F // 128, _cdiv(M, 128)
    dy = _in(dY, "dY", torch.bfloat16, (M, F))
    ab = _in(AB, "AB", e4m3, (M, 2 * F), dev)
    f = _fp8(fmt, "fmt")
    if F % 128 != 0:
        raise CodaError(2, "coda_swiglu_fp8_bwd")
    sab = _in(SAB, "SAB", torch.float32, (2 * fb, M), dev)
    o = dict(out or {})
    da, sda = _out(o, "dA", (M, 2 * F), fmt, dev), _out(o, "SdA", (2 * fb, M), torch.float32, dev)
    dac = sdac = yc = syc = None
    if cols:
        dac, sdac = _out(o, "dAc", (M, 2 * F), fmt, dev), _out(o, "SdAc", (mb, 2 * F), torch.float32, dev)
        yc, syc = _out(o, "Yc", (M, F), e4m3, dev), _out(o, "SYc", (mb, F), torch.float32, dev)
    _call("coda_swiglu_fp8_bwd", dev, dy, ab, sab, da, sda, dac, sdac, yc, syc, M, F, f)
    return o


def rmsnorm_fp8_fwd(X, g, eps: float, R=None, out: dict | None = None) -> dict:
    """H = X + R (when R is given), r = rsqrt(mean H^2 + eps), and H r g in 8
    bits: Q [M, d] e4m3, S [ceil(d/128), M]; returns H (with R), r, Q, S; see
    coda_rmsnorm_fp8_fwd."""
    library()
    M, d = _req2(X, "X")
    dev = X.device
    x, gp = _in(X, "X", torch.bfloat16, (M, d)), _in(g, "g", torch.bfloat16, (d,), dev)
    o = dict(out or {})
    rp = hp = None
    if R is not None:
        rp, hp = _in(R, "R", torch.bfloat16, (M, d), dev), _out(o, "H", (M, d), torch.bfloat16, dev)
    _call("coda_rmsnorm_fp8_fwd", dev, x, rp, gp, hp, _out(o, "r", (M,), torch.float32, dev),
          _out(o, "Q", (M, d), torch.float8_e4m3fn, dev), _out(o, "S", (_cdiv(d, 128), M), torch.float32, dev),
          M, d, float(eps))
    return o


def rmsnorm_fp8_bwd(dN, H, r, g, dH_in=None, out: dict | None = None, ws: Workspace | None = None) -> dict:
    """Backward of rmsnorm_fp8_fwd (the rounding to 8 bits passes gradients
    through): returns dH (bf16, the gradient of X and of R) and dg (fp32); see
    coda_rmsnorm_fp8_bwd.  Without `ws` the scratch is this call's own."""
    lib = library()
    bf16 = torch.bfloat16
    M, d = _req2(dN, "dN")
    dev = dN.device
    dn, h = _in(dN, "dN", bf16, (M, d)), _in(H, "H", bf16, (M, d), dev)
    rp, gp = _in(r, "r", torch.float32, (M,), dev), _in(g, "g", bf16, (d,), dev)
    hi = None if dH_in is None else _in(dH_in, "dH_in", bf16, (M, d), dev)
    o = dict(out or {})
    dh, dg = _out(o, "dH", (M, d), bf16, dev), _out(o, "dg", (d,), torch.float32, dev)
    buf = _ws_on(ws, dev).buf if ws is not None else _new((lib.coda_rmsnorm_fp8_bwd_workspace_bytes(M, d),), torch.uint8, dev)
    _call("coda_rmsnorm_fp8_bwd", dev, dn, h, rp, gp, hi, dh, dg, M, d, buf.data_ptr(), buf.numel())
    return o
