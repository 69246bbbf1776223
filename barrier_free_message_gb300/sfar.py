"""Thin binding of libsfar (``include/sfar.h``, ``include/sfar_decode.h``,
``include/sfar_kv.h``, ``include/sfar_fp8.h``, ``include/sfar_rope.h``,
``include/sfar_latent.h``, ``include/sfar_test.h``): ctypes, and for the calls
on whole tensors (``SfarKv``, ``SfarLatent``, ``Sfar.quantize_fp8``,
``Sfar.rowpar_gemm_fp8``, ``Sfar.rope``) the module built from ``csrc/sfar_tensors.cpp``.

Argument marshalling only: every step of the AllReduce runs in the library's
CUDA kernels.  The functions keep the C names; pointers are plain integers
(``tensor.data_ptr()``) and streams are CUDA stream handles as integers
(``torch.cuda.current_stream().cuda_stream``; ``None`` means the current
torch stream).  The library must have been built (``_build.build()``);
loading it otherwise raises, and there is no CPU fallback.
"""
import ctypes
import importlib.machinery
import importlib.util
import os

from . import _build

SFAR_BF16, SFAR_FP32 = 0, 1
SFAR_BASELINE, SFAR_DB, SFAR_LL, SFAR_LL128, SFAR_SENTINEL, SFAR_TWOSHOT, SFAR_TWOSHOT_TMA, \
    SFAR_LL128_ATOMIC, SFAR_TWOSHOT_SENTINEL = range(9)
PROTOS = {"baseline": SFAR_BASELINE, "db": SFAR_DB, "ll": SFAR_LL, "ll128": SFAR_LL128,
          "sentinel": SFAR_SENTINEL, "twoshot": SFAR_TWOSHOT, "twoshot_tma": SFAR_TWOSHOT_TMA,
          "ll128_atomic": SFAR_LL128_ATOMIC, "twoshot_sent": SFAR_TWOSHOT_SENTINEL}
# every protocol but ll128_atomic returns the rank-order fold bit for bit
EXACT_PROTOS = [p for p in PROTOS if p != "ll128_atomic"]
DTYPES = {"bf16": SFAR_BF16, "fp32": SFAR_FP32}
SFAR_OK, SFAR_ERR_INVALID, SFAR_ERR_CUDA, SFAR_ERR_OOM, SFAR_ERR_TIMEOUT, SFAR_ERR_UNSUPPORTED, \
    SFAR_ERR_POISONED = range(7)
SFAR_LAUNCH_SERIAL, SFAR_LAUNCH_OVERLAP, SFAR_LAUNCH_PLAIN, SFAR_LAUNCH_COOPERATIVE = 0, 1, 2, 3
SFAR_ROPE_HALF, SFAR_ROPE_INTERLEAVED = 0, 1
ROPE_LAYOUTS = {"half": SFAR_ROPE_HALF, "interleaved": SFAR_ROPE_INTERLEAVED}
ROPE_SCALINGS = {None: 0, "linear": 1, "wavelength": 2, "ramp": 3}
MODES = {"serial": SFAR_LAUNCH_SERIAL, "overlap": SFAR_LAUNCH_OVERLAP, "plain": SFAR_LAUNCH_PLAIN,
         "cooperative": SFAR_LAUNCH_COOPERATIVE}
WAIT_NAMES = {1: "done", 2: "ll", 3: "sentinel", 4: "ready", 5: "bottom", 6: "ll128", 7: "rs", 8: "ag",
              9: "arrive", 10: "complete", 11: "copy", 12: "counter",
              13: "cluster",
              32: "page", 33: "length", 34: "slot", 35: "tokens", 36: "ring"}


class SfarFault(ctypes.Structure):
    _fields_ = [("code", ctypes.c_int), ("rank", ctypes.c_int), ("cta", ctypes.c_int), ("peer", ctypes.c_int),
                ("epoch", ctypes.c_uint32), ("where", ctypes.c_int)]


class SfarError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})" if what else f"{strerror(code)} ({code})")


_lib = None

# (name, restype, argtypes) of every exported entry point
_SIGS = [
    ("sfar_create", ctypes.c_void_p, [ctypes.c_int, ctypes.c_size_t, ctypes.c_int]),
    ("sfar_last_error", ctypes.c_int, []),
    ("sfar_allreduce", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_int, ctypes.c_void_p]),
    ("sfar_status_get", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(SfarFault)]),
    ("sfar_reset", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    ("sfar_destroy", None, [ctypes.c_void_p]),
    ("sfar_strerror", ctypes.c_char_p, [ctypes.c_int]),
    ("sfar_query_launch", ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    ("sfar_max_bytes", ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int]),
    ("sfar_allreduce_noalloc", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t,
                                              ctypes.c_int, ctypes.c_void_p]),
    ("sfar_noalloc_status", ctypes.c_int, [ctypes.POINTER(SfarFault), ctypes.c_int]),
    ("sfar_test_noalloc_record_failure", ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    ("sfar_allreduce_add_rmsnorm", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                                  ctypes.c_size_t, ctypes.c_float, ctypes.c_void_p]),
    ("sfar_add_rmsnorm", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_size_t,
                                        ctypes.c_float, ctypes.c_void_p]),
    ("sfar_test_set_straggler", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int,
                                               ctypes.c_int, ctypes.c_void_p]),
    ("sfar_test_drop_rank", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    ("sfar_test_set_timeout", ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]),
    ("sfar_test_force_single_buffer", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    ("sfar_set_launch_mode", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    ("sfar_test_set_geometry", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]),
    ("sfar_test_set_trace", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32]),
    ("sfar_rowpar_gemv", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_size_t, ctypes.c_size_t, ctypes.c_void_p]),
    ("sfar_test_query_norm_launch", ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_size_t, ctypes.c_int,
                                                   ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                                                   ctypes.POINTER(ctypes.c_int)]),
    ("sfar_test_set_fused_path", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    ("sfar_test_query_fused_path", ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_size_t,
                                                  ctypes.POINTER(ctypes.c_int)]),
    ("sfar_quantize_fp8", ctypes.c_int, [ctypes.c_void_p] * 4 + [ctypes.c_size_t] * 4 + [ctypes.c_void_p]),
    ("sfar_rowpar_gemm_fp8", ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_size_t] * 5 + [ctypes.c_void_p]),
    ("sfar_kv_create", ctypes.c_void_p, [ctypes.c_int] * 5 + [ctypes.c_size_t] + [ctypes.c_void_p] * 4),
    ("sfar_kv_destroy", None, [ctypes.c_void_p]),
    ("sfar_kv_plan", ctypes.c_int, [ctypes.c_void_p] * 11 + [ctypes.c_size_t] * 3 + [ctypes.c_void_p]),
    ("sfar_kv_append", ctypes.c_int, [ctypes.c_void_p] * 4 + [ctypes.c_size_t] * 5 + [ctypes.c_void_p]),
    ("sfar_kv_attention", ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_size_t] * 8 +
     [ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p]),
    ("sfar_kv_status_get", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(SfarFault)]),
    ("sfar_kv_reset", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    ("sfar_rope", ctypes.c_int, [ctypes.c_void_p] * 7 + [ctypes.c_size_t] * 12 + [ctypes.c_int, ctypes.c_float, ctypes.c_void_p]),
    ("sfar_rope_frequencies", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_double, ctypes.c_int] +
     [ctypes.c_double] * 4),
    ("sfar_latent_create", ctypes.c_void_p, [ctypes.c_int] * 5 + [ctypes.c_size_t, ctypes.c_void_p]),
    ("sfar_latent_destroy", None, [ctypes.c_void_p]),
    ("sfar_latent_plan", ctypes.c_int, [ctypes.c_void_p] * 11 + [ctypes.c_size_t] * 3 + [ctypes.c_void_p]),
    ("sfar_latent_append", ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_size_t] * 2 +
     [ctypes.c_float, ctypes.c_int, ctypes.c_float, ctypes.c_void_p]),
    ("sfar_latent_gather", ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_size_t] * 4 + [ctypes.c_void_p]),
    ("sfar_latent_attention", ctypes.c_int, [ctypes.c_void_p] * 6 + [ctypes.c_size_t] * 8 + [ctypes.c_float, ctypes.c_void_p]),
    ("sfar_latent_prompt", ctypes.c_int, [ctypes.c_void_p] * 8 + [ctypes.c_size_t] * 14 + [ctypes.c_float, ctypes.c_void_p]),
    ("sfar_latent_status_get", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(SfarFault)]),
    ("sfar_latent_reset", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    ("sfar_test_kv_record_failure", ctypes.c_int, [ctypes.c_void_p]),
    ("sfar_test_latent_record_failure", ctypes.c_int, [ctypes.c_void_p]),
    ("sfar_probe_empty", ctypes.c_int, [ctypes.c_void_p]),
    ("sfar_probe_pingpong", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           ctypes.c_void_p, ctypes.c_void_p]),
]


def library_path() -> str:
    return _build.LIB


def lib():
    """The loaded libsfar (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libsfar is not built ({path} missing); run barrier_free_message_gb300._build.build()")
        L = ctypes.CDLL(path)
        for name, res, args in _SIGS:
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def strerror(code: int) -> str:
    if _lib is None:
        return f"status {code}"
    return _lib.sfar_strerror(code).decode()


_current = None


def _stream(stream):
    """The stream's handle; None: torch's current stream of the current device (read without building a Stream
    object, which costs more than a launch)."""
    global _current
    if stream is not None:
        return int(stream)
    if _current is None:
        import torch
        raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        if raw is None or device is None or not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream
        _current = lambda: raw(device())                       # noqa: E731
    return _current()


def _ptr_array(ptrs):
    return (ctypes.c_void_p * len(ptrs))(*[int(p) for p in ptrs])


_native = None


def _tensors():
    """The module that reads the tensors of a call and makes it (raises if it has not been built)."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (the libraries the module is linked with)
        L = lib()
        if not os.path.exists(_build.TENSORS):
            raise RuntimeError(f"{_build.TENSORS} is missing ({_build.tensors_error()}); run barrier_free_message_gb300._build.build()")
        loader = importlib.machinery.ExtensionFileLoader("sfar_tensors", _build.TENSORS)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("sfar_tensors", loader))
        loader.exec_module(module)
        module.bind(*[ctypes.cast(getattr(L, n), ctypes.c_void_p).value
                      for n in ("sfar_kv_plan", "sfar_kv_append", "sfar_kv_attention", "sfar_quantize_fp8", "sfar_rowpar_gemm_fp8",
                                "sfar_rope", "sfar_latent_plan", "sfar_latent_append", "sfar_latent_gather", "sfar_latent_attention",
                                "sfar_latent_prompt")])
        _native = module
    return _native


def _check(code, what):
    if code != SFAR_OK:
        raise SfarError(code, what)


def _layout(layout):
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout: need one of {', '.join(ROPE_LAYOUTS)}, not {layout!r}")
    return ROPE_LAYOUTS[layout]


def rope_frequencies(rot: int, base: float = 10000.0, scaling=None, factor: float = 1.0, trained: float = 4096.0, low: float = 1.0,
                     high: float = 32.0, device="cuda"):
    """(frequencies, scale) of ``Sfar.rope`` and ``SfarLatent.append``: a float32 tensor [rot / 2] on ``device`` and a
    float.  scaling: None, "linear", "wavelength" or "ramp" (``include/sfar_rope.h`` has the formulas)."""
    import torch
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling: need None, \"linear\", \"wavelength\" or \"ramp\", not {scaling!r}")
    if rot < 2:
        raise ValueError(f"rot: need an even number of at least 2, not {rot}")
    freq, scale = (ctypes.c_float * (rot // 2))(), ctypes.c_float()
    _check(lib().sfar_rope_frequencies(freq, ctypes.byref(scale), rot, base, ROPE_SCALINGS[scaling], factor, trained, low, high),
           "sfar_rope_frequencies")
    return torch.tensor(list(freq), dtype=torch.float32, device=device), scale.value


# ------------------------------------------------------------- C-named calls
def sfar_create(R: int, max_bytes: int, dtype="bf16"):
    dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    h = lib().sfar_create(R, max_bytes, dt)
    if not h:
        raise SfarError(lib().sfar_last_error(), "sfar_create")
    return h


def sfar_allreduce(h, in_ptrs, out_ptrs, n: int, proto="ll", stream=None) -> int:
    p = PROTOS[proto] if isinstance(proto, str) else int(proto)
    return lib().sfar_allreduce(h, _ptr_array(in_ptrs), _ptr_array(out_ptrs), n, p, _stream(stream))


def sfar_allreduce_add_rmsnorm(h, in_ptrs, res_ptrs, weight_ptr: int, out_ptrs, res_out_ptrs, rows: int,
                               hidden: int, eps: float, stream=None) -> int:
    return lib().sfar_allreduce_add_rmsnorm(h, _ptr_array(in_ptrs), _ptr_array(res_ptrs), int(weight_ptr),
                                            _ptr_array(out_ptrs), _ptr_array(res_out_ptrs), rows, hidden, eps,
                                            _stream(stream))


def sfar_add_rmsnorm(h, a_ptrs, res_ptrs, weight_ptr: int, out_ptrs, res_out_ptrs, rows: int, hidden: int,
                     eps: float, stream=None) -> int:
    return lib().sfar_add_rmsnorm(h, _ptr_array(a_ptrs), _ptr_array(res_ptrs), int(weight_ptr),
                                  _ptr_array(out_ptrs), _ptr_array(res_out_ptrs), rows, hidden, eps, _stream(stream))


def sfar_rowpar_gemv(h, x_ptrs, w_ptrs, y_ptrs, k: int, hidden: int, prefetch_rows: int = 0, stream=None) -> int:
    return lib().sfar_rowpar_gemv(h, _ptr_array(x_ptrs), _ptr_array(w_ptrs), _ptr_array(y_ptrs), k, hidden,
                                  prefetch_rows, _stream(stream))


def sfar_test_query_norm_launch(h, rows: int, hidden: int, allreduce: bool = True):
    """(status, ctas_per_rank, cluster_size, threads_per_cta) of a fused call."""
    k, cl, t = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    code = lib().sfar_test_query_norm_launch(h, rows, hidden, 1 if allreduce else 0, ctypes.byref(k),
                                             ctypes.byref(cl), ctypes.byref(t))
    return code, k.value, cl.value, t.value


FUSED_PATHS = {"auto": 0, "oneshot": 1, "twoshot": 2}


def sfar_test_set_fused_path(h, path="auto") -> int:
    return lib().sfar_test_set_fused_path(h, FUSED_PATHS[path] if isinstance(path, str) else int(path))


def sfar_test_query_fused_path(h, rows: int, hidden: int):
    """(status, path) of sfar_allreduce_add_rmsnorm: 1 one-shot, 2 two-shot."""
    p = ctypes.c_int(0)
    code = lib().sfar_test_query_fused_path(h, rows, hidden, ctypes.byref(p))
    return code, p.value


def sfar_allreduce_noalloc(in_ptrs, out_ptrs, R: int, n: int, dtype="bf16", stream=None) -> int:
    dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    return lib().sfar_allreduce_noalloc(_ptr_array(in_ptrs), _ptr_array(out_ptrs), R, n, dt, _stream(stream))


def sfar_noalloc_status(clear: bool = False):
    """(code, fault) of sfar_allreduce_noalloc on the current device; clear
    erases a recorded failure."""
    f = SfarFault()
    code = lib().sfar_noalloc_status(ctypes.byref(f), 1 if clear else 0)
    return code, f


def sfar_test_noalloc_record_failure(rank: int, peer: int, where: int) -> int:
    return lib().sfar_test_noalloc_record_failure(rank, peer, where)


def sfar_status_get(h):
    f = SfarFault()
    code = lib().sfar_status_get(h, ctypes.byref(f))
    return code, f


def sfar_reset(h, stream=None) -> int:
    return lib().sfar_reset(h, _stream(stream))


def sfar_destroy(h) -> None:
    if h:
        lib().sfar_destroy(h)


def sfar_query_launch(h, n: int, proto="ll"):
    p = PROTOS[proto] if isinstance(proto, str) else int(proto)
    k, t = ctypes.c_int(), ctypes.c_int()
    _check(lib().sfar_query_launch(h, n, p, ctypes.byref(k), ctypes.byref(t)), "sfar_query_launch")
    return k.value, t.value


def sfar_max_bytes(h, proto="ll") -> int:
    p = PROTOS[proto] if isinstance(proto, str) else int(proto)
    return lib().sfar_max_bytes(h, p)


def sfar_test_set_straggler(h, delays_ptr: int, length: int, rank: int = -1, phase: int = 0, stream=None) -> int:
    return lib().sfar_test_set_straggler(h, delays_ptr, length, rank, phase, _stream(stream))


def sfar_test_drop_rank(h, rank: int, stream=None) -> int:
    return lib().sfar_test_drop_rank(h, rank, _stream(stream))


def sfar_test_set_timeout(h, ns: int, stream=None) -> int:
    return lib().sfar_test_set_timeout(h, ns, _stream(stream))


def sfar_test_force_single_buffer(h, on: bool, stream=None) -> int:
    return lib().sfar_test_force_single_buffer(h, 1 if on else 0, _stream(stream))


def sfar_set_launch_mode(h, mode) -> int:
    m = MODES.get(mode, mode)
    return lib().sfar_set_launch_mode(h, int(m))


def sfar_test_set_geometry(h, ctas_per_rank: int = 0, threads_per_cta: int = 0) -> int:
    return lib().sfar_test_set_geometry(h, ctas_per_rank, threads_per_cta)


def sfar_test_set_trace(h, trace_ptr: int, calls: int) -> int:
    return lib().sfar_test_set_trace(h, trace_ptr, calls)


def sfar_probe_empty(stream=None) -> int:
    return lib().sfar_probe_empty(_stream(stream))


def sfar_probe_pingpong(flags_ptr: int, trips: int, out_ptr: int, relaxed: bool = False, partner: int = 1,
                        stream=None) -> int:
    return lib().sfar_probe_pingpong(flags_ptr, trips, 1 if relaxed else 0, partner, out_ptr, _stream(stream))


# --------------------------------------------------------- convenience class
class Sfar:
    """A handle for R simulated ranks; ``allreduce`` takes lists of CUDA tensors."""

    def __init__(self, R: int, max_bytes: int, dtype: str = "bf16"):
        self.R, self.max_bytes, self.dtype = R, max_bytes, dtype
        self.h = sfar_create(R, max_bytes, dtype)

    def allreduce(self, ins, outs, proto="ll", n=None, stream=None) -> None:
        if len(ins) != self.R or len(outs) != self.R:
            raise ValueError(f"need {self.R} inputs and outputs")
        if n is None:
            n = ins[0].numel()
        code = sfar_allreduce(self.h, [t.data_ptr() for t in ins], [t.data_ptr() for t in outs], n, proto, stream)
        _check(code, "sfar_allreduce")

    def allreduce_add_rmsnorm(self, ins, residuals, weight, outs, residual_outs, hidden: int, eps: float,
                              stream=None) -> None:
        """Tensors of rows * hidden elements per rank; weight of hidden elements."""
        rows = ins[0].numel() // hidden
        code = sfar_allreduce_add_rmsnorm(self.h, [t.data_ptr() for t in ins], [t.data_ptr() for t in residuals],
                                          weight.data_ptr(), [t.data_ptr() for t in outs],
                                          [t.data_ptr() for t in residual_outs], rows, hidden, eps, stream)
        _check(code, "sfar_allreduce_add_rmsnorm")

    def add_rmsnorm(self, a, residuals, weight, outs, residual_outs, hidden: int, eps: float, stream=None) -> None:
        rows = a[0].numel() // hidden
        code = sfar_add_rmsnorm(self.h, [t.data_ptr() for t in a], [t.data_ptr() for t in residuals],
                                weight.data_ptr(), [t.data_ptr() for t in outs], [t.data_ptr() for t in residual_outs],
                                rows, hidden, eps, stream)
        _check(code, "sfar_add_rmsnorm")

    def rowpar_gemv(self, x, w, y, prefetch_rows: int = 0, stream=None) -> None:
        """x: R tensors of k; w: R tensors of k x hidden; y: R tensors of hidden (bf16, on the device)."""
        k, hidden = w[0].shape[0], w[0].shape[1]
        code = sfar_rowpar_gemv(self.h, [t.data_ptr() for t in x], [t.data_ptr() for t in w],
                                [t.data_ptr() for t in y], k, hidden, prefetch_rows, stream)
        _check(code, "sfar_rowpar_gemv")

    def quantize_fp8(self, x, x8, sx, stream=None) -> None:
        """x: [m, k] bf16 per rank -> x8: [m, k] e4m3 and sx: [ceil(k / 128), m] fp32 per rank (lists of R
        tensors, or one tensor [R, ...] each; rows of x and x8 may be strided)."""
        code = (_native or _tensors()).quantize_fp8(self.h, self.R, x, x8, sx, stream)
        if code:
            _check(code, "sfar_quantize_fp8")

    def rowpar_gemm_fp8(self, x8, sx, w8, sw, y, stream=None) -> None:
        """x8 [m, k], sx [ceil(k / 128), m] (as quantize_fp8 gives them), w8 [hidden, k] e4m3 and sw
        [ceil(hidden / 128), ceil(k / 128)] fp32 -> y [m, hidden] bf16, per rank (lists of R tensors, or one
        tensor [R, ...] each; rows of x8 and w8 may be strided by multiples of 16)."""
        code = (_native or _tensors()).rowpar_gemm_fp8(self.h, self.R, x8, sx, w8, sw, y, stream)
        if code:
            _check(code, "sfar_rowpar_gemm_fp8")

    def rope(self, q, q_out, pos, freq, k=None, k_out=None, layout="half", scale: float = 1.0, stream=None) -> None:
        """Rotary positions: q, q_out: [tokens, heads, rotated part] of the handle's type per rank, views of whole heads
        or tensors of their own; k, k_out the same with their own heads (lists of R tensors, or one tensor [R, ...]
        each).  An output may be its input.  pos: [tokens] int32, freq: [rotated part / 2] fp32 (``rope_frequencies``);
        layout "half" or "interleaved"; rows of a negative position are left as they are."""
        code = (_native or _tensors()).rope(self.h, self.R, DTYPES.get(self.dtype, self.dtype) == SFAR_FP32, q, q_out, k, k_out, pos, freq, _layout(layout), scale, stream)
        if code:
            _check(code, "sfar_rope")

    def status(self):
        return sfar_status_get(self.h)

    def reset(self, stream=None) -> None:
        _check(sfar_reset(self.h, stream), "sfar_reset")

    def set_mode(self, mode) -> None:
        _check(sfar_set_launch_mode(self.h, mode), "sfar_set_launch_mode")

    def launch(self, n: int, proto="ll"):
        return sfar_query_launch(self.h, n, proto)

    def close(self) -> None:
        if self.h:
            sfar_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SfarKv:
    """A paged key/value cache in e4m3 with a scale for each page and head, for R simulated ranks
    (``include/sfar_kv.h``).

    ``k_cache``, ``v_cache``: [pages, kv_heads, page_tokens, head_dim] e4m3 (or its bytes) per rank; ``k_scale``,
    ``v_scale``: [pages, kv_heads] fp32 per rank -- lists of R contiguous tensors, or one tensor [R, ...] each.
    The tensors stay the caller's and are kept alive by this object.
    """

    def __init__(self, k_cache, v_cache, k_scale, v_scale, q_heads: int):
        self.h = None
        native, R = _tensors(), len(k_cache)
        pk, k, dense_k = native.ranks(k_cache, R, 4, "byte", "k_cache")
        pv, v, dense_v = native.ranks(v_cache, R, 4, "byte", "v_cache")
        pks, ks, dense_ks = native.ranks(k_scale, R, 2, "fp32", "k_scale")
        pvs, vs, dense_vs = native.ranks(v_scale, R, 2, "fp32", "v_scale")
        if v != k or ks != k[:2] or vs != k[:2] or \
                not (dense_k and dense_v and dense_ks and dense_vs):
            raise ValueError("SfarKv: need contiguous caches [pages, kv_heads, page_tokens, head_dim] and scales "
                             "[pages, kv_heads]")
        self.R, self.q_heads = R, q_heads
        self.pages, self.kv_heads, self.page_tokens, self.head_dim = k
        self.tensors = (k_cache, v_cache, k_scale, v_scale)
        h = lib().sfar_kv_create(R, q_heads, self.kv_heads, self.head_dim, self.page_tokens, self.pages,
                                 *[_ptr_array(p) for p in (pk, pv, pks, pvs)])
        if not h:
            raise SfarError(lib().sfar_last_error(), "sfar_kv_create")
        self.h = h

    def plan(self, lens, delta, table, ring, state, lens_out, state_out, starts, slots, taken, stream=None) -> None:
        """Pages, slots and offsets of a step from the requests' lengths; every tensor int32.  lens, delta,
        lens_out, taken: [requests]; table: [requests, width]; ring: [pages]; state, state_out: [2]; starts:
        [requests + 1]; slots: [tokens].  lens_out may be lens, state_out may be state."""
        code = (_native or _tensors()).plan(self.h, self.pages, lens, delta, table, ring, state, lens_out, state_out, starts, slots,
                                            taken, stream)
        if code:
            _check(code, "sfar_kv_plan")

    def append(self, k, v, slots, stream=None) -> None:
        """k, v: [tokens, kv_heads, head_dim] bf16 per rank (token and head strides multiples of 8); slots: [tokens]."""
        code = (_native or _tensors()).append(self.h, self.R, self.kv_heads, self.head_dim, k, v, slots, stream)
        if code:
            _check(code, "sfar_kv_append")

    def attention(self, q, out, table, lens, starts, max_q: int, scale=None, window: int = 0, stream=None) -> None:
        """q, out: [tokens, q_heads, head_dim] bf16 per rank (token and head strides multiples of 8); table:
        [requests, width], lens: [requests], starts: [requests + 1].  scale: 1 / sqrt(head_dim) if None."""
        if scale is None:
            scale = self.head_dim ** -0.5
        code = (_native or _tensors()).attention(self.h, self.R, self.q_heads, self.head_dim, q, out, table, lens, starts, max_q, scale,
                                                 window, stream)
        if code:
            _check(code, "sfar_kv_attention")

    def status(self):
        f = SfarFault()
        code = lib().sfar_kv_status_get(self.h, ctypes.byref(f))
        return code, f

    def reset(self, stream=None) -> None:
        _check(lib().sfar_kv_reset(self.h, _stream(stream)), "sfar_kv_reset")

    def close(self) -> None:
        if self.h:
            lib().sfar_kv_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SfarLatent:
    """A paged cache of latents and rotated keys in bf16, for R simulated ranks (``include/sfar_latent.h``).

    ``cache``: [pages, page_tokens, latent_dim + rope_dim] bf16 per rank -- a list of R contiguous tensors, or one
    tensor [R, ...].  The tensors stay the caller's and are kept alive by this object.
    """

    def __init__(self, cache, q_heads: int, rope_dim: int = 64):
        self.h = None
        R = len(cache)
        pointers, shape, dense = _tensors().ranks(cache, R, 3, "bf16", "cache")
        if not dense:
            raise ValueError("SfarLatent: need contiguous caches [pages, page_tokens, latent_dim + rope_dim]")
        self.R, self.q_heads, self.rope_dim = R, q_heads, rope_dim
        self.pages, self.page_tokens, self.row = shape
        self.latent_dim = self.row - rope_dim
        self.tensors = cache
        h = lib().sfar_latent_create(R, q_heads, self.latent_dim, rope_dim, self.page_tokens, self.pages, _ptr_array(pointers))
        if not h:
            raise SfarError(lib().sfar_last_error(), "sfar_latent_create")
        self.h = h

    def plan(self, lens, delta, table, ring, state, lens_out, state_out, starts, slots, taken, stream=None) -> None:
        """As ``SfarKv.plan``, for this cache's pages."""
        code = (_native or _tensors()).latent_plan(self.h, self.pages, lens, delta, table, ring, state, lens_out, state_out, starts, slots,
                                                   taken, stream)
        if code:
            _check(code, "sfar_latent_plan")

    def append(self, x, weight, pos, freq, slots, eps: float = 1e-6, layout="interleaved", scale: float = 1.0, stream=None) -> None:
        """x: [tokens, latent_dim + rope_dim] bf16 per rank (token stride a multiple of 8): latents, which are normalised
        (weight: [latent_dim] bf16), and keys, which are turned (pos: [tokens] int32, freq: [rope_dim / 2] fp32, layout
        and scale as in ``Sfar.rope``); slots: [tokens] int32."""
        code = (_native or _tensors()).latent_append(self.h, self.R, self.latent_dim, self.rope_dim, x, weight, pos, freq, slots, eps,
                                                     _layout(layout), scale, stream)
        if code:
            _check(code, "sfar_latent_append")

    def gather(self, out, table, lens, starts, stream=None) -> None:
        """out: [rows, latent_dim + rope_dim] bf16 per rank: row starts[b] + i becomes token i of request b; table:
        [requests, width], lens: [requests], starts: [requests + 1] int32."""
        code = (_native or _tensors()).latent_gather(self.h, self.R, self.row, out, table, lens, starts, stream)
        if code:
            _check(code, "sfar_latent_gather")

    def attention(self, q, out, table, lens, starts, max_q: int, scale: float, stream=None) -> None:
        """Absorbed form.  q: [tokens, q_heads, latent_dim + rope_dim], out: [tokens, q_heads, latent_dim] bf16 per rank
        (token and head strides multiples of 8); table: [requests, width], lens: [requests], starts: [requests + 1]."""
        code = (_native or _tensors()).latent_attention(self.h, self.R, self.q_heads, self.latent_dim, self.rope_dim, q, out, table, lens,
                                                        starts, max_q, scale, stream)
        if code:
            _check(code, "sfar_latent_attention")

    def prompt(self, q, k, v, kr, out, starts, k_starts, max_q: int, scale=None, stream=None) -> None:
        """Expanded form.  q: [tokens, q_heads, head_dim + rope_dim], k, v: [context rows, q_heads, head_dim], kr:
        [context rows, rope_dim], out: [tokens, q_heads, head_dim] bf16 per rank (strides multiples of 8); starts,
        k_starts: [requests + 1].  scale: 1 / sqrt(head_dim + rope_dim) if None."""
        if scale is None:
            scale = q[0].shape[-1] ** -0.5
        code = (_native or _tensors()).latent_prompt(self.h, self.R, self.q_heads, self.rope_dim, q, k, v, kr, out, starts, k_starts, max_q,
                                                     scale, stream)
        if code:
            _check(code, "sfar_latent_prompt")

    def status(self):
        f = SfarFault()
        code = lib().sfar_latent_status_get(self.h, ctypes.byref(f))
        return code, f

    def reset(self, stream=None) -> None:
        _check(lib().sfar_latent_reset(self.h, _stream(stream)), "sfar_latent_reset")

    def close(self) -> None:
        if self.h:
            lib().sfar_latent_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
