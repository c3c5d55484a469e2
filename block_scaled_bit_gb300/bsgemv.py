"""ctypes binding to ``libbsgemv.so`` (the C ABI of include/bsgemv.h).

Argument marshalling only: every step of the GEMV runs in the library's CUDA kernels.  Tensors
are torch tensors (device memory and streams are torch's); their data pointers are passed as
plain addresses.  Importing this module loads the library and raises if it has not been built
(``python -c "import __graft_entry__ as g; g.build()"``) -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

FORMATS = {"int4": 1, "int8": 2, "fp8": 3, "nvfp4": 4}
ACT_BF16 = 0x100
VARIANTS = {"auto": 0, "mma": 1, "cuda_core": 2}
SPLITS = {"auto": 0, "stream_k": 1, "cluster": 2}
MOE_RENORMALIZE, MOE_LOGITS_F32 = 1, 2

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_MISALIGNED = -3
ERR_M_TOO_LARGE = -4
ERR_CUDA = -5
ERR_WRONG_DEVICE = -6
ERR_DEVICE_TIMEOUT = -7
ERR_SCRATCH_LIMIT = -8

# Every extern "C" entry point of include/bsgemv.h.
EXPORTS = ("bsgemv_plan", "bsgemv_run", "bsgemv_run_bias", "bsgemv_run_host",
           "bsgemv_run_host_async", "bsgemv_destroy",
           "bsgemv_status_string", "bsgemv_debug_dequant", "bsgemv_plan_set_override",
           "bsgemv_plan_describe", "bsgemv_geometry_for", "bsgemv_device_status",
           "bsgemv_run_noalloc", "bsgemv_plan_set_split", "bsgemv_plan_autotune",
           "bsgemv_plan_set_test_fault",
           "bsgemv_dense_plan", "bsgemv_dense_run", "bsgemv_dense_describe",
           "bsgemv_dense_geometry_for", "bsgemv_dense_device_status", "bsgemv_dense_destroy",
           "bsgemv_moe_plan", "bsgemv_moe_run", "bsgemv_moe_run_routed",
           "bsgemv_moe_device_status", "bsgemv_moe_set_test_fault", "bsgemv_moe_destroy",
           "bsgemv_attn_plan", "bsgemv_attn_run", "bsgemv_attn_device_status",
           "bsgemv_attn_set_test_fault", "bsgemv_attn_destroy",
           "bsgemv_cache_plan", "bsgemv_cache_copy", "bsgemv_cache_fork", "bsgemv_cache_free",
           "bsgemv_cache_extend", "bsgemv_cache_write", "bsgemv_cache_compact",
           "bsgemv_cache_destroy",
           "bsgemv_version")


class Geometry(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int), ("rows_per_tile", ctypes.c_int),
                ("k_per_stage", ctypes.c_int), ("stages", ctypes.c_int),
                ("consumer_warps", ctypes.c_int), ("ctas", ctypes.c_int),
                ("ctas_per_sm", ctypes.c_int), ("sm_count", ctypes.c_int),
                ("tiles", ctypes.c_int64), ("stages_per_tile", ctypes.c_int64),
                ("total_stages", ctypes.c_int64), ("smem_bytes", ctypes.c_int),
                ("workspace_bytes", ctypes.c_int64), ("cluster", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class BsgemvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_LIB = None


def lib_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build the CUDA library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(path)
        vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.bsgemv_plan.argtypes = [ctypes.POINTER(vp), ci, ci, ci, i64, i64, ci]
        L.bsgemv_run.argtypes = [vp, vp, vp, vp, vp, vp, ci, vp]
        L.bsgemv_run_bias.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, vp]
        L.bsgemv_run_host.argtypes = [vp, vp, vp, vp, vp, vp, ci, vp]
        L.bsgemv_run_host_async.argtypes = [vp, vp, vp, vp, vp, vp, ci, vp]
        L.bsgemv_destroy.argtypes = [vp]
        L.bsgemv_status_string.argtypes = [ci]
        L.bsgemv_status_string.restype = ctypes.c_char_p
        L.bsgemv_debug_dequant.argtypes = [vp, vp, vp, vp, vp, vp]
        L.bsgemv_plan_set_override.argtypes = [vp, ci, ci, ci, ci]
        L.bsgemv_plan_set_split.argtypes = [vp, ci, ci]
        L.bsgemv_plan_autotune.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, vp]
        L.bsgemv_dense_plan.argtypes = [ctypes.POINTER(vp), ci, i64, i64, ci]
        L.bsgemv_dense_run.argtypes = [vp, vp, vp, vp, ci, vp]
        L.bsgemv_dense_describe.argtypes = [vp, ctypes.POINTER(Geometry)]
        L.bsgemv_dense_geometry_for.argtypes = [ci, i64, i64, ci, ci, ctypes.POINTER(Geometry)]
        L.bsgemv_dense_device_status.argtypes = [vp, vp]
        L.bsgemv_dense_destroy.argtypes = [vp]
        L.bsgemv_plan_describe.argtypes = [vp, ctypes.POINTER(Geometry)]
        L.bsgemv_geometry_for.argtypes = [ci, ci, ci, i64, i64, ci, ci, ctypes.POINTER(Geometry)]
        L.bsgemv_device_status.argtypes = [vp, vp]
        L.bsgemv_run_noalloc.argtypes = [ci, ci, ci, i64, i64, vp, vp, vp, vp, vp, ci, vp]
        L.bsgemv_plan_set_test_fault.argtypes = [vp, ci, i64]
        f32 = ctypes.c_float
        L.bsgemv_moe_plan.argtypes = [ctypes.POINTER(vp), ci, ci, ci, i64, i64, ci, ci, ci, ci]
        L.bsgemv_moe_run.argtypes = [vp] * 10 + [ci, vp]
        L.bsgemv_moe_run_routed.argtypes = [vp] * 11 + [ci, vp]
        L.bsgemv_moe_device_status.argtypes = [vp, vp]
        L.bsgemv_moe_set_test_fault.argtypes = [vp, ci, ci, i64]
        L.bsgemv_moe_destroy.argtypes = [vp]
        L.bsgemv_attn_plan.argtypes = [ctypes.POINTER(vp)] + [ci] * 6
        L.bsgemv_attn_run.argtypes = [vp, vp, i64, vp, vp, i64, i64, i64, ci, vp, ci, vp, i64, vp,
                                      ci, f32, vp, vp, vp]
        L.bsgemv_attn_device_status.argtypes = [vp, vp]
        L.bsgemv_attn_set_test_fault.argtypes = [vp, ci, ci, i64]
        L.bsgemv_attn_destroy.argtypes = [vp]
        L.bsgemv_cache_plan.argtypes = [ctypes.POINTER(vp), ci, ci, i64, ci, ci, ci]
        L.bsgemv_cache_copy.argtypes = [vp, vp, vp, vp, ci, vp]
        L.bsgemv_cache_fork.argtypes = [vp] * 8 + [ci, vp]
        L.bsgemv_cache_free.argtypes = [vp] * 5 + [ci, vp]
        L.bsgemv_cache_extend.argtypes = [vp] * 7 + [ci, vp]
        L.bsgemv_cache_write.argtypes = [vp] * 7 + [i64, ci, ci, i64, i64, ci, ci, ci, vp]
        L.bsgemv_cache_compact.argtypes = [vp] * 9
        L.bsgemv_cache_destroy.argtypes = [vp]
        for name in EXPORTS:
            if name != "bsgemv_status_string":
                getattr(L, name).restype = ci
        _LIB = L
    return _LIB


def status_string(status: int) -> str:
    return lib().bsgemv_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != OK:
        raise BsgemvError(status, what)


def format_code(fmt: str, act: str) -> int:
    return FORMATS[fmt] | (ACT_BF16 if act == "bf16" else 0)


def geometry_for(fmt: str, act: str, block_size: int, has_zp: bool, N: int, K: int, max_M: int,
                 sm_count: int) -> dict:
    """The launch geometry a plan would take on a device with `sm_count` SMs (no GPU needed)."""
    g = Geometry()
    _check(lib().bsgemv_geometry_for(format_code(fmt, act), block_size, int(has_zp), N, K,
                                     max_M, sm_count, ctypes.byref(g)), "bsgemv_geometry_for")
    return g.as_dict()


def run_noalloc_status(fmt: str, act: str, block_size: int, has_zp: bool, N: int, K: int, A, W,
                       scales, zp, y, M: int | None = None, stream=None) -> int:
    """One GEMV through bsgemv_run_noalloc (no plan, no allocation); returns the status."""
    M = A.shape[0] if M is None else M
    return lib().bsgemv_run_noalloc(format_code(fmt, act), block_size, int(has_zp), N, K, _ptr(A),
                                    _ptr(W), _ptr(scales), _ptr(zp), _ptr(y), int(M),
                                    _stream(stream))


def noalloc_device_status(stream=None) -> int:
    """Read and clear bsgemv_run_noalloc's error word on the current device (after a stream
    synchronisation): bsgemv_device_status(NULL, stream)."""
    return lib().bsgemv_device_status(None, _stream(stream))


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current = None


def _stream(stream) -> int | None:
    if stream is None:
        # the current stream's handle without a Stream object for it: 0.2 us a call instead of 3
        global _current
        if _current is None:
            import torch
            torch.cuda.current_device()  # (initialises the device)
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
            _current = (lambda: torch.cuda.current_stream().cuda_stream) if raw is None else \
                (lambda: raw(device()))
        return _current()
    return getattr(stream, "cuda_stream", stream)


class Plan:
    """A plan for one weight shape: y[M, N] = A[M, K] . deq(W)[N, K]^T for M <= max_M."""

    def __init__(self, fmt: str, act: str, block_size: int, has_zp: bool, N: int, K: int,
                 max_M: int = 16):
        self.fmt, self.act, self.block_size, self.has_zp = fmt, act, block_size, bool(has_zp)
        self.N, self.K, self.max_M = N, K, max_M
        h = ctypes.c_void_p()
        _check(lib().bsgemv_plan(ctypes.byref(h), format_code(fmt, act), block_size,
                                 int(has_zp), N, K, max_M), "bsgemv_plan")
        self._h = h

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().bsgemv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def handle(self) -> int:
        return self._h.value

    def run_status(self, A, W, scales, zp, y, M: int | None = None, stream=None,
                   bias=None) -> int:
        """Enqueue the GEMV (plus `bias` [N] if given); returns the library status instead of
        raising."""
        M = A.shape[0] if M is None and hasattr(A, "shape") else M
        if bias is not None:
            return lib().bsgemv_run_bias(self._h, _ptr(A), _ptr(W), _ptr(scales), _ptr(zp),
                                         _ptr(bias), _ptr(y), int(M), _stream(stream))
        return lib().bsgemv_run(self._h, _ptr(A), _ptr(W), _ptr(scales), _ptr(zp), _ptr(y),
                                int(M), _stream(stream))

    def run(self, A, W, scales, zp, y, M: int | None = None, stream=None, bias=None) -> None:
        _check(self.run_status(A, W, scales, zp, y, M, stream, bias),
               "bsgemv_run" if bias is None else "bsgemv_run_bias")

    def run_host(self, A_host, W, scales, zp, y_host, M: int | None = None, stream=None) -> None:
        """A and y in host memory (pinned for asynchronous copies); returns when y is ready."""
        M = A_host.shape[0] if M is None else M
        _check(lib().bsgemv_run_host(self._h, _ptr(A_host), _ptr(W), _ptr(scales), _ptr(zp),
                                     _ptr(y_host), int(M), _stream(stream)), "bsgemv_run_host")

    def run_host_async(self, A_host, W, scales, zp, y_host, M: int | None = None,
                       stream=None) -> None:
        """As run_host, but only enqueued: y_host is ready after the stream is synchronised."""
        M = A_host.shape[0] if M is None else M
        _check(lib().bsgemv_run_host_async(self._h, _ptr(A_host), _ptr(W), _ptr(scales), _ptr(zp),
                                           _ptr(y_host), int(M), _stream(stream)),
               "bsgemv_run_host_async")

    def debug_dequant(self, W, scales, zp, out, stream=None) -> None:
        _check(lib().bsgemv_debug_dequant(self._h, _ptr(W), _ptr(scales), _ptr(zp), _ptr(out),
                                          _stream(stream)), "bsgemv_debug_dequant")

    def set_override(self, variant: int = 0, ctas: int = 0, stages: int = 0,
                     rows_per_tile: int = 0) -> int:
        return lib().bsgemv_plan_set_override(self._h, variant, ctas, rows_per_tile, stages)

    def set_split(self, split: str = "auto", cluster: int = 0) -> int:
        """K split of the tiles: "auto", "stream_k" or "cluster" (cluster = CTAs per tile)."""
        return lib().bsgemv_plan_set_split(self._h, SPLITS[split], cluster)

    def autotune_status(self, A, W, scales, zp, y, M: int | None = None, reps: int = 4,
                        stream=None) -> int:
        """Time the plan's candidate geometries on the device (back-to-back calls over weight
        copies that keep L2 cold) and keep the fastest; returns the library status."""
        M = A.shape[0] if M is None and hasattr(A, "shape") else M
        return lib().bsgemv_plan_autotune(self._h, _ptr(A), _ptr(W), _ptr(scales), _ptr(zp),
                                          _ptr(y), int(M), int(reps), _stream(stream))

    def autotune(self, A, W, scales, zp, y, M: int | None = None, reps: int = 4,
                 stream=None) -> dict:
        _check(self.autotune_status(A, W, scales, zp, y, M, reps, stream), "bsgemv_plan_autotune")
        return self.describe()

    def describe(self) -> dict:
        g = Geometry()
        _check(lib().bsgemv_plan_describe(self._h, ctypes.byref(g)), "bsgemv_plan_describe")
        return g.as_dict()

    def device_status(self, stream=None) -> int:
        return lib().bsgemv_device_status(self._h, _stream(stream))

    def set_test_fault(self, skip_stage: int = -1, wait_ns: int = 0) -> int:
        """Test hook of the bounded waits (bsgemv_plan_set_test_fault): CTA 0's copy warp leaves
        out stage `skip_stage` of its range, the waits give up after `wait_ns`; (-1, 0) undoes it."""
        return lib().bsgemv_plan_set_test_fault(self._h, int(skip_stage), int(wait_ns))


def dense_geometry_for(act: str, N: int, K: int, max_M: int, sm_count: int) -> dict:
    """The geometry a dense plan would take on a device with `sm_count` SMs (no GPU needed)."""
    g = Geometry()
    _check(lib().bsgemv_dense_geometry_for(1 if act == "bf16" else 0, N, K, max_M, sm_count,
                                           ctypes.byref(g)), "bsgemv_dense_geometry_for")
    return g.as_dict()


class DensePlan:
    """The dense small-N GEMV y[M, N] = A[M, K] . B[K, N] (B row-major) for M <= max_M <= 8."""

    def __init__(self, act: str, N: int, K: int, max_M: int = 8):
        self.act, self.N, self.K, self.max_M = act, N, K, max_M
        h = ctypes.c_void_p()
        _check(lib().bsgemv_dense_plan(ctypes.byref(h), 1 if act == "bf16" else 0, N, K, max_M),
               "bsgemv_dense_plan")
        self._h = h

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().bsgemv_dense_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def run_status(self, A, B, y, M: int | None = None, stream=None) -> int:
        M = A.shape[0] if M is None and hasattr(A, "shape") else M
        return lib().bsgemv_dense_run(self._h, _ptr(A), _ptr(B), _ptr(y), int(M), _stream(stream))

    def run(self, A, B, y, M: int | None = None, stream=None) -> None:
        _check(self.run_status(A, B, y, M, stream), "bsgemv_dense_run")

    def describe(self) -> dict:
        g = Geometry()
        _check(lib().bsgemv_dense_describe(self._h, ctypes.byref(g)), "bsgemv_dense_describe")
        return g.as_dict()

    def device_status(self, stream=None) -> int:
        return lib().bsgemv_dense_device_status(self._h, _stream(stream))


def _arg(what: str, t, nbytes: int, dtypes=None) -> int | None:
    """The address of a tensor that a kernel takes for `nbytes` bytes in a row; refused if it holds
    fewer, or not in a row, or other types.  None and raw addresses are passed on."""
    if t is None:
        return None
    try:
        if t.nbytes >= nbytes and (dtypes is None or t.dtype in dtypes) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        if isinstance(t, int):
            return t
        raise
    raise BsgemvError(ERR_INVALID_ARG, what)


def _types(act: str):
    """(the activation type or its bits, int32, fp32), as _arg takes them."""
    import torch
    return ({"f16": torch.float16, "bf16": torch.bfloat16}[act], torch.int16, torch.uint16), \
        (torch.int32,), (torch.float32,)


class _Handle:
    """Owner of one library handle: closed by close(), the end of a with block or collection."""

    _destroy = ""

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            getattr(lib(), self._destroy)(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class MoePlan(_Handle):
    """A mixture-of-experts layer for up to max_T <= 32 tokens: top-k routing, the chosen experts'
    gate / up / down products in a block-scaled format, and the weighted sum (bsgemv_moe_plan).
    logits: "act" (the activation dtype) or "f32".  Tensors that are too small for the plan or not
    contiguous are refused (BSGEMV_ERR_INVALID_ARG)."""

    _destroy = "bsgemv_moe_destroy"

    def __init__(self, fmt: str, act: str, block_size: int, has_zp: bool, H: int, I: int, E: int,
                 top_k: int, max_T: int = 32, renormalize: bool = True, logits: str = "act"):
        self.fmt, self.act, self.block_size, self.has_zp = fmt, act, block_size, bool(has_zp)
        self.H, self.I, self.E, self.top_k, self.max_T = H, I, E, top_k, max_T
        flags = (MOE_RENORMALIZE if renormalize else 0) | \
            {"act": 0, "f32": MOE_LOGITS_F32}[logits]
        h = ctypes.c_void_p()
        _check(lib().bsgemv_moe_plan(ctypes.byref(h), format_code(fmt, act), block_size,
                                     int(has_zp), H, I, E, top_k, max_T, flags),
               "bsgemv_moe_plan")
        self._h = h
        self._act, self._i32, self._f32 = _types(act)
        self._logits = (2, self._act) if logits == "act" else (4, self._f32)
        # bytes of each stacked weight, its scales and its zero points (NVFP4: the experts' scales)
        self._bytes = []
        for rows, k in ((2 * I, H), (H, I)):
            n, nb = E * rows, k // block_size
            self._bytes += [n * k // (2 if fmt in ("int4", "nvfp4") else 1),
                            n * nb * {"int4": 2, "int8": 2, "fp8": 4, "nvfp4": 1}[fmt],
                            4 * E if fmt == "nvfp4" else n * ((nb + 1) // 2 if fmt == "int4" else nb)]

    def _weights(self, *tensors):
        return [_arg("W, scales or zp", t, n) for t, n in zip(tensors, self._bytes)]

    def run_status(self, x, logits, W13, scales13, zp13, W2, scales2, zp2, y,
                   T: int | None = None, stream=None) -> int:
        T = x.shape[0] if T is None else T
        n = T if 0 < T <= self.max_T else 0  # (other T: the library's to refuse)
        size, types = self._logits
        try:
            return lib().bsgemv_moe_run(
                self._h, _arg("x", x, 2 * n * self.H, self._act),
                _arg("logits", logits, size * n * self.E, types),
                *self._weights(W13, scales13, zp13, W2, scales2, zp2),
                _arg("y", y, 2 * n * self.H, self._act), int(T), _stream(stream))
        except BsgemvError as e:
            return e.status

    def run(self, x, logits, W13, scales13, zp13, W2, scales2, zp2, y, T: int | None = None,
            stream=None) -> None:
        """Enqueue y = the layer of x [T, H] under router logits [T, E]."""
        _check(self.run_status(x, logits, W13, scales13, zp13, W2, scales2, zp2, y, T, stream),
               "bsgemv_moe_run")

    def run_routed(self, x, ids, weights, W13, scales13, zp13, W2, scales2, zp2, y,
                   T: int | None = None, stream=None) -> None:
        """The layer with the caller's routing: ids [T, top_k] int32, weights [T, top_k] fp32."""
        T = x.shape[0] if T is None else T
        n = T if 0 < T <= self.max_T else 0
        _check(lib().bsgemv_moe_run_routed(
            self._h, _arg("x", x, 2 * n * self.H, self._act),
            _arg("ids", ids, 4 * n * self.top_k, self._i32),
            _arg("weights", weights, 4 * n * self.top_k, self._f32),
            *self._weights(W13, scales13, zp13, W2, scales2, zp2),
            _arg("y", y, 2 * n * self.H, self._act), int(T), _stream(stream)),
            "bsgemv_moe_run_routed")

    def device_status(self, stream=None) -> int:
        return lib().bsgemv_moe_device_status(self._h, _stream(stream))

    def set_test_fault(self, product: int = 0, skip_stage: int = -1, wait_ns: int = 0) -> int:
        """Test hook of the bounded waits (bsgemv_moe_set_test_fault); (0, -1, 0) undoes it."""
        return lib().bsgemv_moe_set_test_fault(self._h, int(product), int(skip_stage),
                                               int(wait_ns))


class AttnPlan(_Handle):
    """Single-token attention of up to max_B sequences that share a prefix, over a paged cache
    (bsgemv_attn_plan).  Tensors of other shapes, types or orders than run() says are refused
    (BSGEMV_ERR_INVALID_ARG)."""

    _destroy = "bsgemv_attn_destroy"

    def __init__(self, act: str, Hq: int, Hkv: int, D: int, page_size: int, max_B: int):
        self.act, self.Hq, self.Hkv, self.D = act, Hq, Hkv, D
        self.page_size, self.max_B = page_size, max_B
        h = ctypes.c_void_p()
        _check(lib().bsgemv_attn_plan(ctypes.byref(h), int(act == "bf16"), Hq, Hkv, D, page_size,
                                      max_B), "bsgemv_attn_plan")
        self._h = h
        self._act, self._i32, self._f32 = _types(act)
        self._scale = D ** -0.5

    def run(self, q, k, v, prefix_table, prefix_len: int, tables, lens, out, lse=None,
            scale: float | None = None, stream=None) -> None:
        """out [B, Hq, D] from q [B, Hq, D] (any stride between sequences); k and v are views
        [pages, Hkv, page_size, D] of the cache in either layout (strides are passed on);
        prefix_table [pages of the prefix or more], tables [B or more, columns] (any stride between
        rows) and lens [B or more] are int32, lse [B, Hq] fp32; scale defaults to D ** -0.5."""
        B, Hq, D = q.shape
        pages, heads, rows, width = shape = k.shape
        ks, (qs, qh, q1), (ts, t1), act = k.stride(), q.stride(), tables.stride(), self._act
        if ks != v.stride() or shape != v.shape or D != self.D or width != D or ks[3] != 1 or \
                q1 != 1 or t1 != 1 or Hq != self.Hq or qh != D and Hq > 1 or heads != self.Hkv or \
                rows != self.page_size or tables.shape[0] < B or q.dtype not in act or \
                k.dtype not in act or v.dtype not in act or tables.dtype not in self._i32:
            raise BsgemvError(ERR_INVALID_ARG, "bsgemv_attn_run")
        status = lib().bsgemv_attn_run(
            self._h, q.data_ptr(), qs, k.data_ptr(), v.data_ptr(), ks[0], ks[1], ks[2], pages,
            _arg("prefix_table", prefix_table, 4 * -(-prefix_len // rows), self._i32), prefix_len,
            tables.data_ptr(), ts, _arg("lens", lens, 4 * B, self._i32), B,
            self._scale if scale is None else scale, _arg("out", out, 2 * B * Hq * D, act),
            _arg("lse", lse, 4 * B * Hq, self._f32), _stream(stream))
        if status != OK:
            raise BsgemvError(status, "bsgemv_attn_run")

    def run_status(self, *args, **kw) -> int:
        """As run, with the status returned."""
        try:
            self.run(*args, **kw)
        except BsgemvError as e:
            return e.status
        return OK

    def device_status(self, stream=None) -> int:
        return lib().bsgemv_attn_device_status(self._h, _stream(stream))

    def set_test_fault(self, kernel: int = 0, skip_tile: int = -1, wait_ns: int = 0) -> int:
        """Test hook of the bounded waits (bsgemv_attn_set_test_fault); (0, -1, 0) undoes it."""
        return lib().bsgemv_attn_set_test_fault(self._h, int(kernel), int(skip_tile), int(wait_ns))


class PageCache(_Handle):
    """The pages of a cache (bsgemv_cache_plan): pool [planes, num_pages, page_bytes], refs
    [num_pages], tables [max_seqs, max_pages] and lens [max_seqs] (int32) are the caller's, as the
    lists (int32).  Tensors of fewer elements, of other types or not contiguous are refused
    (BSGEMV_ERR_INVALID_ARG)."""

    _destroy = "bsgemv_cache_destroy"

    def __init__(self, planes: int, num_pages: int, page_bytes: int, page_size: int,
                 max_seqs: int, max_pages: int):
        self.planes, self.num_pages, self.page_bytes = planes, num_pages, page_bytes
        self.page_size, self.max_seqs, self.max_pages = page_size, max_seqs, max_pages
        h = ctypes.c_void_p()
        _check(lib().bsgemv_cache_plan(ctypes.byref(h), planes, num_pages, page_bytes, page_size,
                                       max_seqs, max_pages), "bsgemv_cache_plan")
        self._h = h
        self._i32 = _types("f16")[1]
        # bytes of the state's parts
        self._pool, self._refs = planes * num_pages * page_bytes, 4 * num_pages
        self._tables, self._lens = 4 * max_seqs * max_pages, 4 * max_seqs

    def copy(self, pool, src, dst, stream=None) -> None:
        """Page src[i] to page dst[i] in every plane."""
        n, i32 = src.shape[0], self._i32
        _check(lib().bsgemv_cache_copy(
            self._h, _arg("pool", pool, self._pool), _arg("src", src, 4 * n, i32),
            _arg("dst", dst, 4 * n, i32), n, _stream(stream)), "bsgemv_cache_copy")

    def fork(self, pool, refs, tables, lens, parents, children, new_pages=None,
             stream=None) -> None:
        """Slot children[i] becomes a copy of sequence parents[i]."""
        n, i32 = parents.shape[0], self._i32
        _check(lib().bsgemv_cache_fork(
            self._h, _arg("pool", pool, self._pool), _arg("refs", refs, self._refs, i32),
            _arg("tables", tables, self._tables, i32), _arg("lens", lens, self._lens, i32),
            _arg("parents", parents, 4 * n, i32), _arg("children", children, 4 * n, i32),
            _arg("new_pages", new_pages, 4 * n, i32), n, _stream(stream)), "bsgemv_cache_fork")

    def free(self, refs, tables, lens, seqs, stream=None) -> None:
        """Release the sequences."""
        n, i32 = seqs.shape[0], self._i32
        _check(lib().bsgemv_cache_free(
            self._h, _arg("refs", refs, self._refs, i32), _arg("tables", tables, self._tables, i32),
            _arg("lens", lens, self._lens, i32), _arg("seqs", seqs, 4 * n, i32), n,
            _stream(stream)), "bsgemv_cache_free")

    def extend(self, pool, refs, tables, lens, seqs, grown=None, stream=None) -> None:
        """Room for one more token in each of the sequences."""
        n, i32 = seqs.shape[0], self._i32
        _check(lib().bsgemv_cache_extend(
            self._h, _arg("pool", pool, self._pool), _arg("refs", refs, self._refs, i32),
            _arg("tables", tables, self._tables, i32), _arg("lens", lens, self._lens, i32),
            _arg("seqs", seqs, 4 * n, i32), _arg("grown", grown, 4 * n, i32), n,
            _stream(stream)), "bsgemv_cache_extend")

    def write(self, pool, tables, lens, seqs, k, v, head_stride: int, row_stride: int,
              k_plane: int, v_plane: int, stream=None) -> None:
        """k, v [n, heads, D] (2-byte elements, any stride between sequences) to the sequences' last
        positions."""
        n, (rows, heads, D), ks, i32 = seqs.shape[0], k.shape, k.stride(), self._i32
        if ks != v.stride() or v.shape != k.shape or ks[2] != 1 or ks[1] != D and heads > 1 or \
                k.itemsize != 2 or v.itemsize != 2 or rows < n:
            raise BsgemvError(ERR_INVALID_ARG, "bsgemv_cache_write")
        _check(lib().bsgemv_cache_write(
            self._h, _arg("pool", pool, self._pool), _arg("tables", tables, self._tables, i32),
            _arg("lens", lens, self._lens, i32), _arg("seqs", seqs, 4 * n, i32), k.data_ptr(),
            v.data_ptr(), ks[0], heads, D, head_stride, row_stride, k_plane, v_plane, n,
            _stream(stream)), "bsgemv_cache_write")

    def compact(self, pool, refs, tables, lens, refs_out, tables_out, live_out,
                stream=None) -> None:
        """Live pages to the front; the new state in refs_out, tables_out and live_out [1]."""
        i32 = self._i32
        _check(lib().bsgemv_cache_compact(
            self._h, _arg("pool", pool, self._pool), _arg("refs", refs, self._refs, i32),
            _arg("tables", tables, self._tables, i32), _arg("lens", lens, self._lens, i32),
            _arg("refs_out", refs_out, self._refs, i32),
            _arg("tables_out", tables_out, self._tables, i32), _arg("live_out", live_out, 4, i32),
            _stream(stream)), "bsgemv_cache_compact")


def upload(case, device="cuda"):
    """Copy a host case (numpy arrays in the storage layouts) to device tensors and allocate y.
    Returns an object with A, W, scales, zp (the NVFP4 global scale for nvfp4), bias (None
    without one) and y."""
    import types

    import numpy as np
    import torch

    def t(a):
        if a is None:
            return None
        a = np.ascontiguousarray(a)
        if a.dtype == np.uint16:
            a = a.view(np.int16)
        return torch.from_numpy(a).to(device)

    zp = t(case.gscale) if case.fmt == "nvfp4" else t(case.zp)
    y = torch.empty((case.M, case.N), dtype=torch.int16, device=device)
    return types.SimpleNamespace(A=t(case.A), W=t(case.W), scales=t(case.scales), zp=zp,
                                 bias=t(getattr(case, "bias", None)), y=y)


def y_bits(y) -> "np.ndarray":
    """Device output tensor (int16 storage) -> numpy uint16 bit patterns."""
    return y.cpu().numpy().view("uint16")
