"""ctypes binding of libmigemm.so (include/migemm.h), names unchanged.

Argument marshalling only: every step of the GEMM runs in the HIP library.
Tensors may be passed as torch tensors (their ``data_ptr()`` is used) or as
raw integer addresses; streams as ``torch.cuda.Stream``, raw handles or None
(the current torch stream).  If the library has not been built this module
raises on first use; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmigemm.so")

MIGEMM_BF16 = 1
MIGEMM_FP8_E4M3 = 2
MIGEMM_INT8 = 3
MIGEMM_FP32 = 4

MIGEMM_OK = 0
MIGEMM_ERR_INVALID_ARG = -1
MIGEMM_ERR_UNSUPPORTED = -2
MIGEMM_ERR_MISALIGNED = -3
MIGEMM_ERR_DEVICE = -4
MIGEMM_ERR_LAUNCH = -5
MIGEMM_ERR_TIMEOUT = -6
MIGEMM_ERR_SCRATCH = -7
MIGEMM_NO_ALLOC_SCRATCH_BYTES = 64 << 20

MIGEMM_F_TILE_CONSUMER = 0x1
MIGEMM_F_STREAM_K = 0x2
MIGEMM_F_STREAM_K_FORCE = 0x4
MIGEMM_F_HANDOFF_DEBUG = 0x10
MIGEMM_F_C_IN_EPILOGUE = 0x20
MIGEMM_F_CONSUMER_OVERLAP = 0x8
MIGEMM_F_TILE_M256 = 0x40
MIGEMM_F_TILE_M192 = 0x80
MIGEMM_TILE_M = 256
MIGEMM_TILE_N = 256

EXPORTED = [
    "gemm_desc_validate", "gemm_plan_create", "gemm_plan_destroy", "gemm_plan_get_info",
    "gemm_plan_workspace_size", "gemm_workspace_init", "gemm_run", "gemm_run_with_tile_consumer",
    "gemm_run_no_alloc", "gemm_debug_read", "gemm_status_string",
    "gemm_norm_desc_validate", "gemm_norm_plan_create", "gemm_norm_plan_destroy",
    "gemm_norm_workspace_size", "gemm_norm_plan_get_info", "gemm_norm_run", "gemm_norm_run_backward",
    "gemm_scaled_desc_validate", "gemm_scaled_plan_create", "gemm_scaled_plan_destroy",
    "gemm_scaled_workspace_size", "gemm_scaled_plan_get_info", "gemm_scaled_run",
    "gemm_vocab_loss_desc_validate", "gemm_vocab_loss_plan_create", "gemm_vocab_loss_plan_destroy",
    "gemm_vocab_loss_workspace_size", "gemm_vocab_loss_plan_get_info", "gemm_vocab_loss_run", "gemm_vocab_loss_run_backward",
    "gemm_int8_desc_validate", "gemm_int8_plan_create", "gemm_int8_plan_destroy",
    "gemm_int8_workspace_size", "gemm_int8_plan_get_info", "gemm_int8_run",
    "gemm_quantize_desc_validate", "gemm_quantize_plan_create", "gemm_quantize_plan_destroy",
    "gemm_quantize_workspace_size", "gemm_quantize_plan_get_info", "gemm_quantize_run",
    "gemm_block_norm_desc_validate", "gemm_block_norm_plan_create", "gemm_block_norm_plan_destroy",
    "gemm_block_norm_workspace_size", "gemm_block_norm_plan_get_info", "gemm_block_norm_run",
    "gemm_block_norm_run_backward",
    "gemm_checkpoint_desc_validate", "gemm_checkpoint_plan_create", "gemm_checkpoint_plan_destroy",
    "gemm_checkpoint_size", "gemm_checkpoint_workspace_size", "gemm_checkpoint_plan_get_info",
    "gemm_checkpoint_pack", "gemm_checkpoint_unpack", "gemm_checkpoint_weight_gradient",
]


class migemm_desc(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a_type", ctypes.c_int32), ("b_type", ctypes.c_int32),
        ("c_type", ctypes.c_int32), ("d_type", ctypes.c_int32),
        ("a_rs", ctypes.c_int64), ("a_cs", ctypes.c_int64),
        ("b_rs", ctypes.c_int64), ("b_cs", ctypes.c_int64),
        ("c_rs", ctypes.c_int64), ("c_cs", ctypes.c_int64),
        ("d_rs", ctypes.c_int64), ("d_cs", ctypes.c_int64),
        ("device", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("max_workgroups", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("L", ctypes.c_int64),
        ("a_bs", ctypes.c_int64), ("b_bs", ctypes.c_int64),
        ("c_bs", ctypes.c_int64), ("d_bs", ctypes.c_int64),
        ("debug_wait_ticks", ctypes.c_int64), ("debug_force_wait", ctypes.c_int32),
        ("reserved2", ctypes.c_int32),
    ]


class migemm_debug_info(ctypes.Structure):
    _fields_ = [
        ("waits_given_up", ctypes.c_uint32), ("max_occupancy", ctypes.c_uint32),
        ("trace_offset", ctypes.c_int64),
        ("grid", ctypes.c_int32), ("waves", ctypes.c_int32),
        ("trace_tiles", ctypes.c_int32), ("trace_words", ctypes.c_int32),
    ]


class migemm_plan_info(ctypes.Structure):
    _fields_ = [
        ("tiles_m", ctypes.c_int64), ("tiles_n", ctypes.c_int64), ("num_tiles", ctypes.c_int64),
        ("grid", ctypes.c_int32), ("block_threads", ctypes.c_int32),
        ("lds_bytes", ctypes.c_int32), ("stages", ctypes.c_int32),
        ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32),
        ("swapped", ctypes.c_int32), ("a_kmajor", ctypes.c_int32), ("b_kmajor", ctypes.c_int32),
        ("cu_count", ctypes.c_int32), ("handoff_slots", ctypes.c_int32),
        ("stream_k_tiles", ctypes.c_int64), ("stream_k_units_per_tile", ctypes.c_int32),
        ("c_in_k_loop", ctypes.c_int32), ("batches", ctypes.c_int64),
    ]


class migemm_norm_desc(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
        ("x_rs", ctypes.c_int64), ("y_rs", ctypes.c_int64),
        ("r_rs", ctypes.c_int64), ("h_rs", ctypes.c_int64),
        ("dy_rs", ctypes.c_int64), ("dx_rs", ctypes.c_int64), ("dh_rs", ctypes.c_int64),
        ("eps", ctypes.c_float), ("y_type", ctypes.c_int32),
        ("device", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class migemm_norm_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "forward_waves", "forward_vectors", "backward_waves", "backward_vectors",
        "backward_workgroups", "cu_count")]


class migemm_scaled_desc(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a_rs", ctypes.c_int64), ("b_cs", ctypes.c_int64), ("d_rs", ctypes.c_int64),
        ("device", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class migemm_scaled_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tile_m", "tile_n", "lds_stages", "splits", "exact", "cu_count")]


class migemm_vocab_loss_desc(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("hidden", ctypes.c_int64),
        ("x_rs", ctypes.c_int64), ("w_rs", ctypes.c_int64),
        ("dx_rs", ctypes.c_int64), ("dw_rs", ctypes.c_int64),
        ("device", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class migemm_vocab_loss_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "forward_tile_m", "forward_tile_n", "gradient_tile_m", "gradient_tile_n",
        "dx_tile_m", "dx_tile_n", "dx_splits", "dw_tile_m", "dw_tile_n", "dw_splits",
        "cu_count", "pieces")] + [("piece", ctypes.c_int64)]


class migemm_int8_desc(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a_rs", ctypes.c_int64), ("b_cs", ctypes.c_int64), ("d_rs", ctypes.c_int64),
        ("device", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class migemm_int8_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tile_m", "tile_n", "lds_stages", "splits", "cu_count")]


class migemm_quantize_desc(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
        ("x_rs", ctypes.c_int64), ("q_rs", ctypes.c_int64),
        ("q_type", ctypes.c_int32), ("device", ctypes.c_int32), ("reserved", ctypes.c_int64),
    ]


class migemm_quantize_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("waves", "vectors", "cu_count")]


class migemm_block_norm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "rows", "cols", "x_rs", "r_rs", "h_rs", "y_rs", "z_rs", "dy_rs", "dx_rs", "dr_rs", "dz_rs", "dh_rs")] + [
        ("eps", ctypes.c_float), ("branch_scale", ctypes.c_float), ("residual_scale", ctypes.c_float),
        ("post_norm", ctypes.c_int32), ("y_type", ctypes.c_int32), ("device", ctypes.c_int32),
    ]


class migemm_block_norm_info(ctypes.Structure):
    _fields_ = migemm_norm_info._fields_


class migemm_checkpoint_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "cols", "x_rs", "out_cols", "dy_rs", "dw_rs")] + [
        ("dw_type", ctypes.c_int32), ("accumulate", ctypes.c_int32),
        ("device", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class migemm_checkpoint_info(ctypes.Structure):
    _fields_ = [("code_bytes", ctypes.c_int64), ("scale_bytes", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in ("tile_m", "tile_n", "lds_stages", "splits", "cu_count", "reserved")]


class MigemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gemm_status_string(status)} ({status})")


_lib = None


def load(path: str | None = None):
    """Load libmigemm.so (once; LIB_PATH unless a path is given).  Raises if
    it is missing.

    torch ships its own HIP runtime library.  It is imported first, when it
    is installed, so that libmigemm.so binds that same runtime: with two HIP
    runtimes in one process the second cannot use the device, and torch's
    device pointers and streams would not be valid in it."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run `python -m warp_specialized_pipelined_amd.build`"
                           " (or __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    P = ctypes.POINTER
    lib.gemm_desc_validate.argtypes = [P(migemm_desc)]
    lib.gemm_desc_validate.restype = i32
    lib.gemm_plan_create.argtypes = [P(migemm_desc), P(vp)]
    lib.gemm_plan_create.restype = i32
    lib.gemm_plan_destroy.argtypes = [vp]
    lib.gemm_plan_destroy.restype = i32
    lib.gemm_plan_get_info.argtypes = [vp, P(migemm_plan_info)]
    lib.gemm_plan_get_info.restype = i32
    lib.gemm_plan_workspace_size.argtypes = [vp]
    lib.gemm_plan_workspace_size.restype = ctypes.c_size_t
    lib.gemm_workspace_init.argtypes = [vp, vp, vp]
    lib.gemm_workspace_init.restype = i32
    lib.gemm_run.argtypes = [vp, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp, vp]
    lib.gemm_run.restype = i32
    lib.gemm_run_with_tile_consumer.argtypes = [vp, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float,
                                                vp, vp, vp, vp, vp]
    lib.gemm_run_with_tile_consumer.restype = i32
    lib.gemm_run_no_alloc.argtypes = [vp, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp]
    lib.gemm_run_no_alloc.restype = i32
    lib.gemm_debug_read.argtypes = [vp, vp, vp, P(migemm_debug_info)]
    lib.gemm_debug_read.restype = i32
    _declare_plan_calls(lib, "norm", migemm_norm_desc, migemm_norm_info)
    lib.gemm_norm_run.argtypes = [vp] * 9
    lib.gemm_norm_run.restype = i32
    lib.gemm_norm_run_backward.argtypes = [vp] * 10
    lib.gemm_norm_run_backward.restype = i32
    _declare_plan_calls(lib, "scaled", migemm_scaled_desc, migemm_scaled_info)
    lib.gemm_scaled_run.argtypes = [vp] * 8
    lib.gemm_scaled_run.restype = i32
    _declare_plan_calls(lib, "vocab_loss", migemm_vocab_loss_desc, migemm_vocab_loss_info)
    lib.gemm_vocab_loss_run.argtypes = [vp] * 8
    lib.gemm_vocab_loss_run.restype = i32
    lib.gemm_vocab_loss_run_backward.argtypes = [vp] * 10
    lib.gemm_vocab_loss_run_backward.restype = i32
    _declare_plan_calls(lib, "int8", migemm_int8_desc, migemm_int8_info)
    _declare_plan_calls(lib, "quantize", migemm_quantize_desc, migemm_quantize_info)
    _declare_plan_calls(lib, "block_norm", migemm_block_norm_desc, migemm_block_norm_info)
    _declare_plan_calls(lib, "checkpoint", migemm_checkpoint_desc, migemm_checkpoint_info)
    lib.gemm_checkpoint_size.argtypes = [vp]
    lib.gemm_checkpoint_size.restype = ctypes.c_size_t
    for name, args in (("int8_run", 9), ("quantize_run", 5), ("block_norm_run", 12), ("block_norm_run_backward", 17),
                       ("checkpoint_pack", 4), ("checkpoint_unpack", 4), ("checkpoint_weight_gradient", 6)):
        f = getattr(lib, "gemm_" + name)
        f.argtypes, f.restype = [vp] * args, i32
    lib.gemm_status_string.argtypes = [i32]
    lib.gemm_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _declare_plan_calls(lib, kind, desc, info):
    """The calls every operator's plan has."""
    vp, i32, P = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER
    for name, args, res in (("desc_validate", [P(desc)], i32),
                            ("plan_create", [P(desc), P(vp)], i32),
                            ("plan_destroy", [vp], i32),
                            ("plan_get_info", [vp, P(info)], i32),
                            ("workspace_size", [vp], ctypes.c_size_t)):
        f = getattr(lib, f"gemm_{kind}_{name}")
        f.argtypes, f.restype = args, res


def _ptr(x) -> int | None:
    if x is None:
        return None
    try:
        return x.data_ptr()
    except AttributeError:
        return int(x)


def _ptrs(xs):
    """_ptr of each: tensors and None, the usual arguments, without a call for
    each (a block norm's ten take 0.8 us instead of 1.6, of a call's 5)."""
    try:
        return [None if x is None else x.data_ptr() for x in xs]
    except AttributeError:
        return [_ptr(x) for x in xs]


_current_stream = None


def _find_current_stream():
    """A call that returns the current torch stream's handle.  torch's public
    one makes an object of it first, which takes longer (2.8 us) than a small
    kernel's launch; it is used where torch lacks the short way (0.1 us)."""
    global _current_stream
    import torch
    torch.cuda.current_stream()  # torch's device state exists from here on
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and device is not None:
        _current_stream = lambda: raw(device())  # noqa: E731
    else:
        _current_stream = lambda: int(torch.cuda.current_stream().cuda_stream)  # noqa: E731
    return _current_stream


def _stream(s) -> int | None:
    if s is None:
        return (_current_stream or _find_current_stream())()
    if hasattr(s, "cuda_stream"):
        return int(s.cuda_stream)
    return int(s)


def _plan(plan):
    """A plan handle from a Plan object or a raw handle.  Passing the Plan
    object keeps it (and so the C plan) alive for the whole call; a handle
    taken from a temporary Plan, as in gemm_run(Plan(d).handle, ...), is
    already destroyed when the call starts, which the library then rejects
    with MIGEMM_ERR_INVALID_ARG."""
    return getattr(plan, "handle", plan)


def make_desc(M, N, K, a_type, b_type, a_rs, a_cs, b_rs, b_cs, c_rs, c_cs, d_rs, d_cs,
              device=0, flags=0, max_workgroups=0, c_type=MIGEMM_BF16, d_type=MIGEMM_BF16,
              L=1, a_bs=0, b_bs=0, c_bs=0, d_bs=0, debug_wait_ticks=0, debug_force_wait=0):
    return migemm_desc(M, N, K, a_type, b_type, c_type, d_type, a_rs, a_cs, b_rs, b_cs, c_rs, c_cs,
                       d_rs, d_cs, device, flags, max_workgroups, 0, L, a_bs, b_bs, c_bs, d_bs,
                       debug_wait_ticks, debug_force_wait, 0)


def gemm_status_string(status: int) -> str:
    return load().gemm_status_string(int(status)).decode()


def gemm_desc_validate(desc: migemm_desc) -> int:
    return int(load().gemm_desc_validate(ctypes.byref(desc)))


def gemm_plan_create(desc: migemm_desc) -> int:
    """Returns the plan handle; raises MigemmError on a non-OK status."""
    h = ctypes.c_void_p()
    st = load().gemm_plan_create(ctypes.byref(desc), ctypes.byref(h))
    if st != MIGEMM_OK:
        raise MigemmError(st, "gemm_plan_create")
    return h.value


def gemm_plan_destroy(plan: int) -> int:
    return int(load().gemm_plan_destroy(_plan(plan)))


def gemm_plan_get_info(plan: int) -> migemm_plan_info:
    info = migemm_plan_info()
    st = load().gemm_plan_get_info(_plan(plan), ctypes.byref(info))
    if st != MIGEMM_OK:
        raise MigemmError(st, "gemm_plan_get_info")
    return info


def gemm_plan_workspace_size(plan: int) -> int:
    return int(load().gemm_plan_workspace_size(_plan(plan)))


def gemm_workspace_init(plan, workspace, stream=None, check: bool = True) -> int:
    st = load().gemm_workspace_init(_plan(plan), _ptr(workspace), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_workspace_init")
    return st


def gemm_run(plan, A, B, C, D, alpha: float, beta: float, workspace=None, stream=None,
             check: bool = True) -> int:
    st = load().gemm_run(_plan(plan), _ptr(A), _ptr(B), _ptr(C), _ptr(D), float(alpha), float(beta),
                         _ptr(workspace), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_run")
    return int(st)


def gemm_run_no_alloc(plan, A, B, C, D, alpha: float, beta: float, stream=None,
                      check: bool = True) -> int:
    st = load().gemm_run_no_alloc(_plan(plan), _ptr(A), _ptr(B), _ptr(C), _ptr(D), float(alpha),
                                  float(beta), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_run_no_alloc")
    return int(st)


def gemm_debug_read(plan, workspace, stream=None) -> tuple:
    """(status, migemm_debug_info): synchronizes the stream, reads the debug
    header.  status is MIGEMM_ERR_TIMEOUT when a bounded wait gave up."""
    info = migemm_debug_info()
    st = load().gemm_debug_read(_plan(plan), _ptr(workspace), _stream(stream), ctypes.byref(info))
    return int(st), info


def gemm_run_with_tile_consumer(plan, A, B, C, D, alpha: float, beta: float, row_sum, row_max,
                                D_copy, workspace=None, stream=None, check: bool = True) -> int:
    st = load().gemm_run_with_tile_consumer(_plan(plan), _ptr(A), _ptr(B), _ptr(C), _ptr(D), float(alpha),
                                            float(beta), _ptr(row_sum), _ptr(row_max),
                                            _ptr(D_copy), _ptr(workspace), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_run_with_tile_consumer")
    return int(st)


class Plan:
    """Owns a plan handle; destroys it when garbage-collected."""

    def __init__(self, desc: migemm_desc):
        self.desc = desc
        self.handle = gemm_plan_create(desc)
        self.info = gemm_plan_get_info(self.handle)

    @property
    def workspace_size(self) -> int:
        return gemm_plan_workspace_size(self.handle)

    def run(self, A, B, C, D, alpha=1.0, beta=0.0, stream=None, workspace=None):
        return gemm_run(self.handle, A, B, C, D, alpha, beta, workspace, stream)

    def run_with_tile_consumer(self, A, B, C, D, alpha, beta, row_sum, row_max, D_copy,
                               stream=None):
        return gemm_run_with_tile_consumer(self.handle, A, B, C, D, alpha, beta, row_sum, row_max,
                                           D_copy, None, stream)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            try:
                gemm_plan_destroy(h)
            except Exception:
                pass
            self.handle = None


def gemm_norm_desc_validate(desc: migemm_norm_desc) -> int:
    return int(load().gemm_norm_desc_validate(ctypes.byref(desc)))


def gemm_norm_run(plan, x, r, weight, h, y, scale, rstd, stream=None, check: bool = True) -> int:
    st = (_lib or load()).gemm_norm_run(_plan(plan), _ptr(x), _ptr(r), _ptr(weight), _ptr(h), _ptr(y),
                                        _ptr(scale), _ptr(rstd), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_norm_run")
    return int(st)


def gemm_norm_run_backward(plan, dy, h, weight, rstd, dh, dx, dweight, workspace=None, stream=None,
                           check: bool = True) -> int:
    st = (_lib or load()).gemm_norm_run_backward(_plan(plan), _ptr(dy), _ptr(h), _ptr(weight), _ptr(rstd),
                                       _ptr(dh), _ptr(dx), _ptr(dweight), _ptr(workspace),
                                       _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_norm_run_backward")
    return int(st)


def gemm_scaled_desc_validate(desc: migemm_scaled_desc) -> int:
    return int(load().gemm_scaled_desc_validate(ctypes.byref(desc)))


def gemm_scaled_run(plan, a, a_scale, b, b_scale, d, workspace=None, stream=None,
                    check: bool = True) -> int:
    st = (_lib or load()).gemm_scaled_run(_plan(plan), _ptr(a), _ptr(a_scale), _ptr(b), _ptr(b_scale), _ptr(d),
                                _ptr(workspace), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_scaled_run")
    return int(st)


def gemm_vocab_loss_desc_validate(desc: migemm_vocab_loss_desc) -> int:
    return int(load().gemm_vocab_loss_desc_validate(ctypes.byref(desc)))


def gemm_vocab_loss_run(plan, x, w, target, loss, lse, workspace=None, stream=None,
                        check: bool = True) -> int:
    st = (_lib or load()).gemm_vocab_loss_run(_plan(plan), _ptr(x), _ptr(w), _ptr(target), _ptr(loss), _ptr(lse),
                                    _ptr(workspace), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_vocab_loss_run")
    return int(st)


def gemm_vocab_loss_run_backward(plan, x, w, target, lse, dloss, dx, dw, workspace=None, stream=None,
                                 check: bool = True) -> int:
    st = (_lib or load()).gemm_vocab_loss_run_backward(_plan(plan), _ptr(x), _ptr(w), _ptr(target), _ptr(lse),
                                             _ptr(dloss), _ptr(dx), _ptr(dw), _ptr(workspace),
                                             _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_vocab_loss_run_backward")
    return int(st)


def gemm_int8_desc_validate(desc: migemm_int8_desc) -> int:
    return int(load().gemm_int8_desc_validate(ctypes.byref(desc)))


def gemm_int8_run(plan, a, a_scale, b, b_scale, bias, d, workspace=None, stream=None, check: bool = True) -> int:
    st = (_lib or load()).gemm_int8_run(_plan(plan), *_ptrs((a, a_scale, b, b_scale, bias, d, workspace)),
                                        _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_int8_run")
    return int(st)


def gemm_quantize_desc_validate(desc: migemm_quantize_desc) -> int:
    return int(load().gemm_quantize_desc_validate(ctypes.byref(desc)))


def gemm_quantize_run(plan, x, q, scale, stream=None, check: bool = True) -> int:
    st = (_lib or load()).gemm_quantize_run(_plan(plan), *_ptrs((x, q, scale)), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_quantize_run")
    return int(st)


def gemm_block_norm_desc_validate(desc: migemm_block_norm_desc) -> int:
    return int(load().gemm_block_norm_desc_validate(ctypes.byref(desc)))


def gemm_block_norm_run(plan, x, z, r, post_weight, weight, h, y, scale, post_rstd, rstd, stream=None,
                        check: bool = True) -> int:
    st = (_lib or load()).gemm_block_norm_run(
        _plan(plan), *_ptrs((x, z, r, post_weight, weight, h, y, scale, post_rstd, rstd)), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_block_norm_run")
    return int(st)


def gemm_block_norm_run_backward(plan, dy, dh, x, z, h, post_weight, weight, post_rstd, rstd, dx, dz, dr,
                                 dpost_weight, dweight, workspace=None, stream=None, check: bool = True) -> int:
    st = (_lib or load()).gemm_block_norm_run_backward(
        _plan(plan), *_ptrs((dy, dh, x, z, h, post_weight, weight, post_rstd, rstd, dx, dz, dr, dpost_weight, dweight,
                             workspace)), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_block_norm_run_backward")
    return int(st)


def gemm_checkpoint_desc_validate(desc: migemm_checkpoint_desc) -> int:
    return int(load().gemm_checkpoint_desc_validate(ctypes.byref(desc)))


def gemm_checkpoint_size(plan) -> int:
    return int(load().gemm_checkpoint_size(_plan(plan)))


def gemm_checkpoint_pack(plan, x, kept, stream=None, check: bool = True) -> int:
    st = (_lib or load()).gemm_checkpoint_pack(_plan(plan), *_ptrs((x, kept)), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_checkpoint_pack")
    return int(st)


def gemm_checkpoint_unpack(plan, kept, x, stream=None, check: bool = True) -> int:
    st = (_lib or load()).gemm_checkpoint_unpack(_plan(plan), *_ptrs((kept, x)), _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_checkpoint_unpack")
    return int(st)


def gemm_checkpoint_weight_gradient(plan, dy, kept, dw, workspace=None, stream=None, check: bool = True) -> int:
    st = (_lib or load()).gemm_checkpoint_weight_gradient(_plan(plan), *_ptrs((dy, kept, dw, workspace)),
                                                          _stream(stream))
    if check and st != MIGEMM_OK:
        raise MigemmError(st, "gemm_checkpoint_weight_gradient")
    return int(st)


class _OperatorPlan:
    """Owns an operator's plan handle; destroys it when garbage-collected."""

    kind = ""
    info_type = None

    def __init__(self, desc):
        self.desc = desc
        h = ctypes.c_void_p()
        st = getattr(load(), f"gemm_{self.kind}_plan_create")(ctypes.byref(desc), ctypes.byref(h))
        if st != MIGEMM_OK:
            raise MigemmError(st, f"gemm_{self.kind}_plan_create")
        self.handle = h.value

    @property
    def workspace_size(self) -> int:
        return int(getattr(load(), f"gemm_{self.kind}_workspace_size")(self.handle))

    @property
    def info(self):
        """The kernels the plan has chosen."""
        info = self.info_type()
        st = getattr(load(), f"gemm_{self.kind}_plan_get_info")(self.handle, ctypes.byref(info))
        if st != MIGEMM_OK:
            raise MigemmError(st, f"gemm_{self.kind}_plan_get_info")
        return info

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            try:
                getattr(load(), f"gemm_{self.kind}_plan_destroy")(h)
            except Exception:
                pass
            self.handle = None


class NormPlan(_OperatorPlan):
    """Residual addition and root-mean-square norm of rows x cols, y in bf16
    or e4m3; row strides in elements.  r_rs and h_rs: with a residual; dy_rs
    and dx_rs (and dh_rs): with a backward pass."""

    kind = "norm"
    info_type = migemm_norm_info

    def __init__(self, rows, cols, eps, y_type=MIGEMM_BF16, *, x_rs, y_rs, r_rs=0, h_rs=0, dy_rs=0,
                 dx_rs=0, dh_rs=0, device=0):
        super().__init__(migemm_norm_desc(rows, cols, x_rs, y_rs, r_rs, h_rs, dy_rs, dx_rs, dh_rs,
                                          eps, y_type, device, 0))

    def run(self, x, r, weight, h, y, scale, rstd, stream=None):
        return gemm_norm_run(self, x, r, weight, h, y, scale, rstd, stream)

    def run_backward(self, dy, h, weight, rstd, dh, dx, dweight, workspace=None, stream=None):
        return gemm_norm_run_backward(self, dy, h, weight, rstd, dh, dx, dweight, workspace, stream)


class ScaledPlan(_OperatorPlan):
    """d (M x N bf16) = a (M x K e4m3, a scale per row) times the transpose of
    b (N x K e4m3, a scale per row); row strides in elements."""

    kind = "scaled"
    info_type = migemm_scaled_info

    def __init__(self, M, N, K, *, a_rs, b_cs, d_rs, device=0):
        super().__init__(migemm_scaled_desc(M, N, K, a_rs, b_cs, d_rs, device, 0))

    def run(self, a, a_scale, b, b_scale, d, workspace=None, stream=None):
        return gemm_scaled_run(self, a, a_scale, b, b_scale, d, workspace, stream)


class VocabLossPlan(_OperatorPlan):
    """Softmax cross entropy of rows x hidden states over a vocabulary's
    vocab x hidden weights; row strides in elements.  dx_rs and dw_rs: with
    a backward pass."""

    kind = "vocab_loss"
    info_type = migemm_vocab_loss_info

    def __init__(self, rows, vocab, hidden, *, x_rs, w_rs, dx_rs=0, dw_rs=0, device=0):
        super().__init__(migemm_vocab_loss_desc(rows, vocab, hidden, x_rs, w_rs, dx_rs, dw_rs, device, 0))

    def run(self, x, w, target, loss, lse, workspace=None, stream=None):
        return gemm_vocab_loss_run(self, x, w, target, loss, lse, workspace, stream)

    def run_backward(self, x, w, target, lse, dloss, dx, dw, workspace=None, stream=None):
        return gemm_vocab_loss_run_backward(self, x, w, target, lse, dloss, dx, dw, workspace, stream)


class Int8Plan(_OperatorPlan):
    """d (M x N bf16) = a (M x K int8, a scale per row) times the transpose of
    b (N x K int8, a scale per row), plus a bias per column or None; row
    strides in elements."""

    kind = "int8"
    info_type = migemm_int8_info

    def __init__(self, M, N, K, *, a_rs, b_cs, d_rs, device=0):
        super().__init__(migemm_int8_desc(M, N, K, a_rs, b_cs, d_rs, device, 0))

    def run(self, a, a_scale, b, b_scale, bias, d, workspace=None, stream=None):
        return gemm_int8_run(self, a, a_scale, b, b_scale, bias, d, workspace, stream)


class QuantizePlan(_OperatorPlan):
    """bf16 rows x cols to int8 or e4m3 with a scale per row; row strides in
    elements."""

    kind = "quantize"
    info_type = migemm_quantize_info

    def __init__(self, rows, cols, q_type=MIGEMM_INT8, *, x_rs, q_rs, device=0):
        super().__init__(migemm_quantize_desc(rows, cols, x_rs, q_rs, q_type, device, 0))

    def run(self, x, q, scale, stream=None):
        return gemm_quantize_run(self, x, q, scale, stream)


class BlockNormPlan(_OperatorPlan):
    """Between two blocks of rows x cols: the norm of a block's output x
    (post_norm), its gate sigmoid(z) (z_rs) and scale, the residual's addition
    and the next block's norm, y in bf16, e4m3 or int8; row strides in
    elements.  dy_rs, dx_rs and dr_rs (dz_rs with a gate, and dh_rs): with a
    backward pass."""

    kind = "block_norm"
    info_type = migemm_block_norm_info

    def __init__(self, rows, cols, eps, y_type=MIGEMM_BF16, *, x_rs, r_rs, h_rs, y_rs, z_rs=0, post_norm=True,
                 branch_scale=1.0, residual_scale=1.0, dy_rs=0, dh_rs=0, dx_rs=0, dr_rs=0, dz_rs=0, device=0):
        super().__init__(migemm_block_norm_desc(rows, cols, x_rs, r_rs, h_rs, y_rs, z_rs, dy_rs, dx_rs, dr_rs, dz_rs,
                                                dh_rs, eps, branch_scale, residual_scale, int(post_norm), y_type,
                                                device))

    def run(self, x, z, r, post_weight, weight, h, y, scale, post_rstd, rstd, stream=None):
        return gemm_block_norm_run(self, x, z, r, post_weight, weight, h, y, scale, post_rstd, rstd, stream)

    def run_backward(self, dy, dh, x, z, h, post_weight, weight, post_rstd, rstd, dx, dz, dr, dpost_weight, dweight,
                     workspace=None, stream=None):
        return gemm_block_norm_run_backward(self, dy, dh, x, z, h, post_weight, weight, post_rstd, rstd, dx, dz, dr,
                                            dpost_weight, dweight, workspace, stream)


class CheckpointPlan(_OperatorPlan):
    """tokens x cols activations kept in 8 bits for the backward pass, and the
    gradient (out_cols x cols) of the weights of the product that took them;
    row strides in elements.  out_cols, dy_rs and dw_rs: with that gradient;
    accumulate: added to dw (fp32)."""

    kind = "checkpoint"
    info_type = migemm_checkpoint_info

    def __init__(self, tokens, cols, *, x_rs, out_cols=0, dy_rs=0, dw_rs=0, dw_type=MIGEMM_BF16, accumulate=False,
                 device=0):
        super().__init__(migemm_checkpoint_desc(tokens, cols, x_rs, out_cols, dy_rs, dw_rs, dw_type,
                                                int(accumulate), device, 0))

    @property
    def checkpoint_size(self) -> int:
        """Bytes of the kept form."""
        return gemm_checkpoint_size(self.handle)

    def pack(self, x, kept, stream=None):
        return gemm_checkpoint_pack(self, x, kept, stream)

    def unpack(self, kept, x, stream=None):
        return gemm_checkpoint_unpack(self, kept, x, stream)

    def weight_gradient(self, dy, kept, dw, workspace=None, stream=None):
        return gemm_checkpoint_weight_gradient(self, dy, kept, dw, workspace, stream)
