"""ctypes binding over libmoe_ffn.so (the C ABI declared in include/moe_ffn.h).

Argument marshalling only: every step of the layer runs in the HIP library.
PyTorch supplies device memory and the current stream. If the library has
not been built this module raises on first use; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# The in-tree build; MOE_FFN_LIBRARY names another build of the same sources
# (the host-sanitizer build of the tests, for one).
LIB_PATH = os.environ.get("MOE_FFN_LIBRARY") or os.path.join(_PKG, "libmoe_ffn.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_ffn.h")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_CAPACITY = 3
MOE_ERR_WORKSPACE = 4
MOE_ERR_HIP = 5

MOE_W_INT4_AWQ = 0
MOE_W_MXFP8 = 1

MOE_PATH_AUTO = 0
MOE_PATH_DECODE = 1
MOE_PATH_GROUPED = 2

MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1
MOE_DTYPE_F16 = 2
MOE_DTYPE_MXFP4 = 3

MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1

_c_i32 = ctypes.c_int32
_c_i64 = ctypes.c_int64
_c_size = ctypes.c_size_t
_c_ptr = ctypes.c_void_p
_c_float = ctypes.c_float


class moe_weights(ctypes.Structure):
    _fields_ = [("fmt", _c_i32), ("group", _c_i32), ("q", _c_ptr), ("scale", _c_ptr),
                ("zero", _c_ptr)]


class moe_ffn_desc(ctypes.Structure):
    _fields_ = [("M", _c_i32), ("H", _c_i32), ("I", _c_i32), ("E", _c_i32), ("k", _c_i32),
                ("b", _c_i32), ("w13", moe_weights), ("w2", moe_weights), ("path", _c_i32),
                ("max_workgroups", _c_i32), ("expert_base", _c_i32)]


class moe_grouped_matmul_desc(ctypes.Structure):
    _fields_ = [("rows", _c_i32), ("E", _c_i32), ("N", _c_i32), ("K", _c_i32), ("dtype", _c_i32),
                ("out_dtype", _c_i32)]


class moe_route_desc(ctypes.Structure):
    _fields_ = [("M", _c_i32), ("E", _c_i32), ("k", _c_i32), ("dtype", _c_i32), ("score", _c_i32),
                ("renormalize", _c_i32), ("scale", _c_float), ("groups", _c_i32), ("topk_groups", _c_i32),
                ("group_top", _c_i32)]


class moe_combine_desc(ctypes.Structure):
    _fields_ = [("M", _c_i32), ("k", _c_i32), ("H", _c_i32), ("rows", _c_i32), ("dtype", _c_i32),
                ("y_dtype", _c_i32)]


class moe_matvec_desc(ctypes.Structure):
    _fields_ = [("M", _c_i32), ("k", _c_i32), ("E", _c_i32), ("N", _c_i32), ("K", _c_i32), ("dtype", _c_i32),
                ("out_dtype", _c_i32), ("w", moe_weights)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {status_str(status)} (status {status})")


_SIGNATURES = {
    "moe_align_capacity": (_c_size, [_c_i32, _c_i32, _c_i32, _c_i32]),
    "moe_align": (_c_i32, [_c_ptr, _c_i32, _c_i32, _c_i32, _c_i32, _c_ptr, _c_ptr, _c_ptr,
                           _c_size, _c_ptr]),
    "moe_align_ex": (_c_i32, [_c_ptr, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_ptr, _c_ptr, _c_ptr,
                              _c_size, _c_ptr, _c_size, _c_ptr]),
    "moe_align_ex_workspace_size": (_c_i32, [_c_i32, _c_i32, _c_i32, ctypes.POINTER(_c_size)]),
    "moe_ffn_workspace_size": (_c_i32, [ctypes.POINTER(moe_ffn_desc), ctypes.POINTER(_c_size)]),
    "moe_ffn_forward": (_c_i32, [ctypes.POINTER(moe_ffn_desc), _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                 _c_ptr, _c_size, _c_ptr]),
    "moe_ffn_forward_aligned": (_c_i32, [ctypes.POINTER(moe_ffn_desc), _c_ptr, _c_ptr, _c_ptr,
                                         _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr, _c_ptr,
                                         _c_size, _c_ptr]),
    "moe_ffn_forward_noalloc": (_c_i32, [ctypes.POINTER(moe_ffn_desc), _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                         _c_ptr]),
    "moe_ffn_noalloc_max_bytes": (_c_size, []),
    "moe_ffn_forward_capture": (_c_i32, [ctypes.POINTER(moe_ffn_desc), _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                         _c_ptr, _c_size, _c_ptr, _c_ptr]),
    "moe_ffn_forward_profiled": (_c_i32, [ctypes.POINTER(moe_ffn_desc), _c_ptr, _c_ptr, _c_ptr,
                                          _c_ptr, _c_ptr, _c_size, _c_ptr,
                                          ctypes.POINTER(_c_ptr), _c_i32]),
    "moe_ffn_gate_up": (_c_i32, [ctypes.POINTER(moe_ffn_desc), _c_ptr, _c_ptr, _c_ptr, _c_size,
                                 _c_ptr]),
    "moe_ffn_down_combine": (_c_i32, [ctypes.POINTER(moe_ffn_desc), _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                      _c_size, _c_ptr]),
    "moe_ffn_gate_up_batched": (_c_i32, [ctypes.POINTER(moe_ffn_desc), _c_ptr, _c_ptr, _c_i32, _c_ptr,
                                         _c_ptr, _c_ptr]),
    "moe_ffn_down_batched": (_c_i32, [ctypes.POINTER(moe_ffn_desc), _c_ptr, _c_ptr, _c_ptr, _c_i32,
                                      _c_ptr, _c_ptr]),
    "moe_grouped_matmul": (_c_i32, [ctypes.POINTER(moe_grouped_matmul_desc), _c_ptr, _c_i64, _c_ptr, _c_ptr,
                                    _c_ptr, _c_i64, _c_ptr]),
    "moe_grouped_matmul_dx": (_c_i32, [ctypes.POINTER(moe_grouped_matmul_desc), _c_ptr, _c_i64, _c_ptr, _c_ptr,
                                       _c_ptr, _c_i64, _c_ptr]),
    "moe_grouped_matmul_dw": (_c_i32, [ctypes.POINTER(moe_grouped_matmul_desc), _c_ptr, _c_i64, _c_ptr, _c_i64,
                                       _c_ptr, _c_ptr, _c_ptr]),
    "moe_grouped_matmul_mxfp4": (_c_i32, [ctypes.POINTER(moe_grouped_matmul_desc), _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                          _c_ptr, _c_ptr, _c_i64, _c_ptr]),
    "moe_mxfp4_quantize": (_c_i32, [_c_i32, _c_ptr, _c_i64, _c_i64, _c_i32, _c_ptr, _c_ptr, _c_ptr]),
    "moe_mxfp4_dequantize": (_c_i32, [_c_i32, _c_ptr, _c_ptr, _c_i64, _c_i32, _c_ptr, _c_i64, _c_ptr]),
    "moe_align_offsets": (_c_i32, [_c_ptr, _c_ptr, _c_size, _c_i32, _c_i32, _c_ptr, _c_ptr]),
    "moe_route": (_c_i32, [ctypes.POINTER(moe_route_desc), _c_ptr, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_ptr]),
    "moe_route_grad": (_c_i32, [ctypes.POINTER(moe_route_desc), _c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i32, _c_ptr,
                                _c_i64, _c_ptr]),
    "moe_align_positions": (_c_i32, [_c_ptr, _c_ptr, _c_size, _c_i32, _c_ptr, _c_ptr]),
    "moe_combine": (_c_i32, [ctypes.POINTER(moe_combine_desc), _c_ptr, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_i64,
                             _c_ptr]),
    "moe_combine_grad": (_c_i32, [ctypes.POINTER(moe_combine_desc), _c_ptr, _c_i64, _c_ptr, _c_i64, _c_ptr, _c_ptr,
                                  _c_ptr, _c_i64, _c_ptr, _c_ptr]),
    "moe_matvec_int4": (_c_i32, [ctypes.POINTER(moe_matvec_desc), _c_ptr, _c_i64, _c_ptr, _c_ptr, _c_i64, _c_ptr]),
    "moe_ffn_kernel_count": (_c_i32, [ctypes.POINTER(moe_ffn_desc)]),
    "moe_ffn_kernel_name": (ctypes.c_char_p, [ctypes.POINTER(moe_ffn_desc), _c_i32]),
    "moe_ffn_intermediate": (_c_i32, [ctypes.POINTER(moe_ffn_desc), ctypes.POINTER(_c_size),
                                      ctypes.POINTER(_c_size), ctypes.POINTER(_c_i32)]),
    "moe_ffn_route_outputs": (_c_i32, [ctypes.POINTER(moe_ffn_desc), ctypes.POINTER(_c_size)]),
    "moe_ffn_auto_decode_max_m": (_c_i32, []),
    "moe_ffn_resolved_path": (_c_i32, [ctypes.POINTER(moe_ffn_desc)]),
    "moe_status_str": (ctypes.c_char_p, [_c_i32]),
}

_lib = None
_bench_lib = None
BENCH_LIB_PATH = os.path.join(_PKG, "libmoe_bench.so")
BENCH_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_bench.h")
_BENCH_SIGNATURES = {
    "moe_bench_stream_read": (_c_i32, [_c_ptr, _c_size, _c_ptr, _c_i32, _c_i32, ctypes.POINTER(_c_i32), _c_ptr,
                                       _c_ptr, _c_ptr]),
    "moe_bench_copy": (_c_i32, [_c_ptr, _c_ptr, _c_size, _c_i32, _c_ptr, _c_ptr, _c_ptr]),
    "moe_bench_mfma": (_c_i32, [_c_i32, _c_i32, _c_i32, _c_i32, _c_ptr, ctypes.POINTER(ctypes.c_double), _c_ptr,
                                _c_ptr, _c_ptr]),
}


def lib() -> ctypes.CDLL:
    """The loaded HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m mixture_experts_ffn_align_amd.build` (there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def bench_lib() -> ctypes.CDLL:
    """The measurement kernels (include/moe_bench.h); raises if not built."""
    global _bench_lib
    if _bench_lib is None:
        if not os.path.exists(BENCH_LIB_PATH):
            raise RuntimeError(f"{BENCH_LIB_PATH} is missing: build it with "
                               "`python -m mixture_experts_ffn_align_amd.build`")
        L = ctypes.CDLL(BENCH_LIB_PATH)
        for name, (res, args) in _BENCH_SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _bench_lib = L
    return _bench_lib


def declared_symbols(header: str = HEADER_PATH, macro: str = "MOE_API") -> list[str]:
    """Entry points a header declares (include/moe_ffn.h by default)."""
    with open(header) as f:
        text = f.read()
    return re.findall(macro + r"\s+[\w\s\*]+?\b(moe_\w+)\s*\(", text)


def status_str(status: int) -> str:
    return lib().moe_status_str(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _expect(name, t, dtype, shape, device=None):
    """Check that tensor ``t`` is a contiguous ``dtype`` tensor of ``shape`` on a
    GPU (on ``device`` when given) before its pointer goes to the library: the
    kernels read raw memory, so a wrong dtype or a short buffer would misread
    or run past its end instead of failing."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be on a GPU, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    return t.device


def _check_layer_io(desc, x=None, topk_ids=None, topk_w=None, y=None, ws=None):
    """dtype / shape checks of a layer call's tensors against ``desc``, then
    the device checks (all on one GPU)."""
    import torch
    M, H, k = desc.M, desc.H, desc.k
    specs = [("x", x, torch.bfloat16, (M, H)), ("topk_ids", topk_ids, torch.int32, (M, k)),
             ("topk_w", topk_w, torch.float32, (M, k)), ("y", y, torch.float32, (M, H)),
             ("ws", ws, torch.uint8, None)]
    specs = [s for s in specs if s[1] is not None]
    for name, t, dtype, shape in specs:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.dtype != dtype:
            raise TypeError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    for name, t, dtype, shape in specs:
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
    dev = None
    for name, t, dtype, shape in specs:
        dev = _expect(name, t, dtype, tuple(t.shape), dev)


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def moe_align_capacity(M: int, k: int, E: int, b: int) -> int:
    return int(lib().moe_align_capacity(M, k, E, b))


def moe_align(topk_ids, E: int, b: int, sorted_route_ids, expert_block_ids, num_padded,
              stream=None, check: bool = True) -> int:
    M, k = topk_ids.shape
    st = lib().moe_align(_ptr(topk_ids), M, k, E, b, _ptr(sorted_route_ids),
                         _ptr(expert_block_ids), _ptr(num_padded),
                         sorted_route_ids.numel(), _stream(stream))
    if check:
        _check(st, "moe_align")
    return st


def moe_align_ex_workspace_size(M: int, k: int, E: int) -> int:
    n = _c_size(0)
    _check(lib().moe_align_ex_workspace_size(M, k, E, ctypes.byref(n)), "moe_align_ex_workspace_size")
    return int(n.value)


def moe_align_ex(topk_ids, E: int, expert_base: int, b: int, sorted_route_ids, expert_block_ids,
                 num_padded, ws=None, stream=None, check: bool = True) -> int:
    M, k = topk_ids.shape
    st = lib().moe_align_ex(_ptr(topk_ids), M, k, E, expert_base, b, _ptr(sorted_route_ids),
                            _ptr(expert_block_ids), _ptr(num_padded), sorted_route_ids.numel(),
                            _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                            _stream(stream))
    if check:
        _check(st, "moe_align_ex")
    return st


def weights_struct(fmt: int, group: int, q, scale, zero) -> moe_weights:
    return moe_weights(fmt, group, _ptr(q), _ptr(scale), _ptr(zero))


def make_desc(M: int, H: int, I: int, E: int, k: int, b: int, w13: moe_weights,
              w2: moe_weights, path: int = MOE_PATH_AUTO, max_workgroups: int = 0,
              expert_base: int = 0) -> moe_ffn_desc:
    return moe_ffn_desc(M, H, I, E, k, b, w13, w2, path, max_workgroups, expert_base)


def moe_ffn_workspace_size(desc: moe_ffn_desc, check: bool = True):
    n = _c_size(0)
    st = lib().moe_ffn_workspace_size(ctypes.byref(desc), ctypes.byref(n))
    if check:
        _check(st, "moe_ffn_workspace_size")
        return int(n.value)
    return st, int(n.value)


def moe_ffn_forward(desc: moe_ffn_desc, x, topk_ids, topk_w, y, ws, stream=None,
                    check: bool = True) -> int:
    _check_layer_io(desc, x, topk_ids, topk_w, y, ws)
    st = lib().moe_ffn_forward(ctypes.byref(desc), _ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(y),
                               _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                               _stream(stream))
    if check:
        _check(st, "moe_ffn_forward")
    return st


def moe_ffn_forward_noalloc(desc: moe_ffn_desc, x, topk_ids, topk_w, y, stream=None,
                            check: bool = True) -> int:
    """moe_ffn_forward on the library's static per-GPU scratch (no workspace)."""
    _check_layer_io(desc, x, topk_ids, topk_w, y)
    st = lib().moe_ffn_forward_noalloc(ctypes.byref(desc), _ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(y),
                                       _stream(stream))
    if check:
        _check(st, "moe_ffn_forward_noalloc")
    return st


def moe_ffn_noalloc_max_bytes() -> int:
    return int(lib().moe_ffn_noalloc_max_bytes())


def moe_ffn_forward_aligned(desc: moe_ffn_desc, x, topk_ids, topk_w, sorted_route_ids,
                            expert_block_ids, num_padded, y, ws, stream=None,
                            check: bool = True) -> int:
    import torch
    _check_layer_io(desc, x, topk_ids, topk_w, y, ws)
    cap = sorted_route_ids.numel()
    _expect("sorted_route_ids", sorted_route_ids, torch.int32, (cap,), x.device)
    _expect("expert_block_ids", expert_block_ids, torch.int32, (cap // max(desc.b, 1),), x.device)
    _expect("num_padded", num_padded, torch.int32, (1,), x.device)
    st = lib().moe_ffn_forward_aligned(
        ctypes.byref(desc), _ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(sorted_route_ids),
        _ptr(expert_block_ids), _ptr(num_padded), sorted_route_ids.numel(), _ptr(y), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream))
    if check:
        _check(st, "moe_ffn_forward_aligned")
    return st


def moe_ffn_forward_capture(desc: moe_ffn_desc, x, topk_ids, topk_w, y, ws, w13_out, stream=None) -> None:
    """moe_ffn_forward that also writes the W13 outputs (gate, up) of every valid
    route into w13_out, fp32 [M*k, 2I]."""
    import torch
    _check_layer_io(desc, x, topk_ids, topk_w, y, ws)
    _expect("w13_out", w13_out, torch.float32, (desc.M * desc.k, 2 * desc.I), x.device)
    _check(lib().moe_ffn_forward_capture(ctypes.byref(desc), _ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(y),
                                         _ptr(ws), ws.numel() * ws.element_size(), _ptr(w13_out),
                                         _stream(stream)), "moe_ffn_forward_capture")


def moe_ffn_forward_profiled(desc: moe_ffn_desc, x, topk_ids, topk_w, y, ws, events,
                             stream=None) -> None:
    """``events`` are torch.cuda.Event(enable_timing=True) objects, two per
    kernel: events[2i] and events[2i + 1] take kernel i's start and end."""
    _check_layer_io(desc, x, topk_ids, topk_w, y, ws)
    for e in events:
        if int(e.cuda_event) == 0:   # torch creates the HIP event on first record
            e.record()
    handles = (_c_ptr * len(events))(*[int(e.cuda_event) for e in events])
    st = lib().moe_ffn_forward_profiled(ctypes.byref(desc), _ptr(x), _ptr(topk_ids), _ptr(topk_w),
                                        _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                                        _stream(stream), handles, len(events))
    _check(st, "moe_ffn_forward_profiled")


def moe_ffn_gate_up(desc: moe_ffn_desc, x, topk_ids, ws, stream=None) -> None:
    _check_layer_io(desc, x, topk_ids, None, None, ws)
    _check(lib().moe_ffn_gate_up(ctypes.byref(desc), _ptr(x), _ptr(topk_ids), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream)), "moe_ffn_gate_up")


def moe_ffn_down_combine(desc: moe_ffn_desc, topk_ids, topk_w, y, ws, stream=None) -> None:
    _check_layer_io(desc, None, topk_ids, topk_w, y, ws)
    _check(lib().moe_ffn_down_combine(ctypes.byref(desc), _ptr(topk_ids), _ptr(topk_w), _ptr(y),
                                      _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_ffn_down_combine")


def moe_ffn_gate_up_batched(desc: moe_ffn_desc, xb, counts, a16, a_scale, stream=None) -> None:
    """xb [E, capacity, H] bf16, counts [E] int32 (device), a16 [E, capacity, I]
    fp16 and a_scale [E, capacity, ceil(I/128), 4] fp32 (intermediate format 2)."""
    import torch
    E, cap = desc.E, xb.shape[1] if xb.dim() == 3 else -1
    dev = _expect("xb", xb, torch.bfloat16, (E, cap, desc.H))
    _expect("counts", counts, torch.int32, (E,), dev)
    _expect("a16", a16, torch.float16, (E, cap, desc.I), dev)
    _expect("a_scale", a_scale, torch.float32, (E, cap, -(-desc.I // 128), 4), dev)
    _check(lib().moe_ffn_gate_up_batched(ctypes.byref(desc), _ptr(xb), _ptr(counts), xb.shape[1],
                                         _ptr(a16), _ptr(a_scale), _stream(stream)),
           "moe_ffn_gate_up_batched")


def moe_ffn_down_batched(desc: moe_ffn_desc, a16, a_scale, counts, yb, stream=None) -> None:
    """a16 [E, capacity, I] fp16 and a_scale [E, capacity, ceil(I/128), 4] fp32, counts [E]
    int32, yb [E, capacity, H] fp32."""
    import torch
    E, cap = desc.E, a16.shape[1] if a16.dim() == 3 else -1
    dev = _expect("a16", a16, torch.float16, (E, cap, desc.I))
    _expect("a_scale", a_scale, torch.float32, (E, cap, -(-desc.I // 128), 4), dev)
    _expect("counts", counts, torch.int32, (E,), dev)
    _expect("yb", yb, torch.float32, (E, cap, desc.H), dev)
    _check(lib().moe_ffn_down_batched(ctypes.byref(desc), _ptr(a16), _ptr(a_scale), _ptr(counts),
                                      a16.shape[1], _ptr(yb), _stream(stream)),
           "moe_ffn_down_batched")


def moe_ffn_kernel_count(desc: moe_ffn_desc) -> int:
    return int(lib().moe_ffn_kernel_count(ctypes.byref(desc)))


def moe_ffn_kernel_name(desc: moe_ffn_desc, i: int) -> str | None:
    r = lib().moe_ffn_kernel_name(ctypes.byref(desc), i)
    return None if r is None else r.decode()


def moe_ffn_intermediate(desc: moe_ffn_desc) -> tuple[int, int, int]:
    """(offset, aux_offset, format) of the intermediate in the workspace."""
    off, aux, fmt = _c_size(0), _c_size(0), _c_i32(0)
    _check(lib().moe_ffn_intermediate(ctypes.byref(desc), ctypes.byref(off), ctypes.byref(aux),
                                      ctypes.byref(fmt)), "moe_ffn_intermediate")
    return int(off.value), int(aux.value), int(fmt.value)


def moe_ffn_route_outputs(desc: moe_ffn_desc) -> int:
    """Offset of the grouped path's routed-W2 rows (fp32 [M*k][H]) in the workspace."""
    off = _c_size(0)
    _check(lib().moe_ffn_route_outputs(ctypes.byref(desc), ctypes.byref(off)), "moe_ffn_route_outputs")
    return int(off.value)


def moe_ffn_auto_decode_max_m() -> int:
    return int(lib().moe_ffn_auto_decode_max_m())


def moe_ffn_resolved_path(desc: moe_ffn_desc) -> int:
    """The path moe_ffn_forward takes for `desc` (-1 if it is rejected)."""
    return int(lib().moe_ffn_resolved_path(ctypes.byref(desc)))


# ---------------------------------------------------------------------------
# Products on rows grouped by expert with ragged counts, MXFP4, row offsets
# ---------------------------------------------------------------------------

# These calls take a few microseconds on the GPU for a single token, so their
# checks are one expression per tensor; which rule failed is worked out only
# then.

_dtype_codes = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16}


def _dtype_code(name, t, allowed) -> int:
    """moe_dtype of tensor ``t``; TypeError unless it is one of ``allowed``."""
    code = _dtype_codes.get(getattr(t, "dtype", None))
    if code not in allowed:
        if not hasattr(t, "data_ptr"):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        raise TypeError(f"{name}: unexpected dtype {t.dtype}")
    return code


def _expect_like(name, t, dtype, shape, device):
    """_expect for a device that is known to be a GPU."""
    if not (getattr(t, "dtype", None) is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        _expect(name, t, dtype, shape, device)


def _expect_rows(name, t, shape, device=None):
    """Check a row operand of a known dtype: a 2-d tensor of ``shape`` on a GPU
    (on ``device`` when given) whose rows are contiguous. Returns its row stride
    in elements (the library checks the stride's own rules)."""
    rows, cols = shape
    if t.shape == shape and (t.is_cuda if device is None else t.device == device):
        ld, step = t.stride()
        if step == 1 or cols == 1:
            return ld if rows > 1 else -(-cols // 8) * 8
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be on a GPU, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    raise ValueError(f"{name}: rows must be contiguous, got strides {t.stride()}")


def _call_on(device, stream, fn, *args) -> int:
    """fn(*args, stream) with ``device`` current; ``stream`` None is the
    device's current stream."""
    index = device.index
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else getattr(stream, "cuda_stream", stream)
    if index == torch.cuda.current_device():
        return fn(*args, raw)
    with torch.cuda.device(device):
        return fn(*args, raw)


_I32_MAX = 2 ** 31 - 1


def _expect_i32(**sizes):
    """ValueError for the first size that does not fit the C ABI's int32 (ctypes
    drops its upper bits instead of failing)."""
    for name, v in sizes.items():
        if not -_I32_MAX <= v <= _I32_MAX:
            raise ValueError(f"{name}: {v} does not fit 32 bits")


def _gmm_desc(rows, E, N, K, dtype, out_dtype):
    if rows > _I32_MAX or E > _I32_MAX or N > _I32_MAX or K > _I32_MAX:
        _expect_i32(rows=rows, E=E, N=N, K=K)
    return moe_grouped_matmul_desc(rows, E, N, K, dtype, out_dtype)


_GMM_TYPES = (MOE_DTYPE_BF16, MOE_DTYPE_F16)
_ALL_TYPES = (MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_F16)


def _expect_3d(name, t):
    if not hasattr(t, "data_ptr"):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dim() != 3:
        raise ValueError(f"{name}: expected [E, N, K], got shape {tuple(t.shape)}")
    return t.shape


def moe_grouped_matmul(x, w, offsets, y, stream=None, check: bool = True) -> int:
    """y[r] = w[e] x[r] for the rows r of every expert e.

    x [rows, K] and w [E, N, K] bf16 or fp16, offsets [E + 1] int32 (expert e owns
    rows offsets[e] .. offsets[e + 1] - 1), y [rows, N] of x's dtype or fp32. x and
    y may have a row stride. Rows no expert owns are left as they were. Autograd
    does not see the call: its gradients are moe_grouped_matmul_dx and _dw."""
    E, N, K = _expect_3d("w", w)
    dt = _dtype_code("x", x, _GMM_TYPES)
    out = _dtype_code("y", y, (dt, MOE_DTYPE_F32))
    rows = x.shape[0] if x.dim() == 2 else -1
    ldx = _expect_rows("x", x, (rows, K))
    dev = x.device
    _expect_like("w", w, x.dtype, (E, N, K), dev)
    _expect_like("offsets", offsets, torch.int32, (E + 1,), dev)
    ldy = _expect_rows("y", y, (rows, N), dev)
    d = _gmm_desc(rows, E, N, K, dt, out)
    st = _call_on(dev, stream, lib().moe_grouped_matmul, ctypes.byref(d), x.data_ptr(), ldx, w.data_ptr(),
                  offsets.data_ptr(), y.data_ptr(), ldy)
    if check:
        _check(st, "moe_grouped_matmul")
    return st


def moe_grouped_matmul_dx(dy, w, offsets, dx, stream=None, check: bool = True) -> int:
    """Gradient of moe_grouped_matmul with respect to x: dx[r] = w[e]^T dy[r].

    dy [rows, N] and w [E, N, K] bf16 or fp16, offsets as there, dx [rows, K] of
    dy's dtype or fp32."""
    E, N, K = _expect_3d("w", w)
    dt = _dtype_code("dy", dy, _GMM_TYPES)
    out = _dtype_code("dx", dx, (dt, MOE_DTYPE_F32))
    rows = dy.shape[0] if dy.dim() == 2 else -1
    lddy = _expect_rows("dy", dy, (rows, N))
    dev = dy.device
    _expect_like("w", w, dy.dtype, (E, N, K), dev)
    _expect_like("offsets", offsets, torch.int32, (E + 1,), dev)
    lddx = _expect_rows("dx", dx, (rows, K), dev)
    d = _gmm_desc(rows, E, N, K, dt, out)
    st = _call_on(dev, stream, lib().moe_grouped_matmul_dx, ctypes.byref(d), dy.data_ptr(), lddy, w.data_ptr(),
                  offsets.data_ptr(), dx.data_ptr(), lddx)
    if check:
        _check(st, "moe_grouped_matmul_dx")
    return st


def moe_grouped_matmul_dw(dy, x, offsets, dw, stream=None, check: bool = True) -> int:
    """Gradient of moe_grouped_matmul with respect to w: dw[e] = sum of
    dy[r] x[r]^T over e's rows (zero for an expert without rows).

    dy [rows, N] and x [rows, K] bf16 or fp16, offsets as there, dw [E, N, K] of
    their dtype or fp32."""
    E, N, K = _expect_3d("dw", dw)
    dt = _dtype_code("dy", dy, _GMM_TYPES)
    out = _dtype_code("dw", dw, (dt, MOE_DTYPE_F32))
    rows = dy.shape[0] if dy.dim() == 2 else -1
    lddy = _expect_rows("dy", dy, (rows, N))
    dev = dy.device
    _dtype_code("x", x, (dt,))
    ldx = _expect_rows("x", x, (rows, K), dev)
    _expect_like("offsets", offsets, torch.int32, (E + 1,), dev)
    _expect_like("dw", dw, dw.dtype, (E, N, K), dev)
    d = _gmm_desc(rows, E, N, K, dt, out)
    st = _call_on(dev, stream, lib().moe_grouped_matmul_dw, ctypes.byref(d), dy.data_ptr(), lddy, x.data_ptr(),
                  ldx, offsets.data_ptr(), dw.data_ptr())
    if check:
        _check(st, "moe_grouped_matmul_dw")
    return st


def moe_grouped_matmul_mxfp4(xq, x_scale, wq, w_scale, offsets, y, stream=None, check: bool = True) -> int:
    """moe_grouped_matmul on MXFP4 operands (moe_mxfp4_quantize's layout).

    xq [rows, K/2], x_scale [rows, K/32], wq [E, N, K/2], w_scale [E, N, K/32] uint8,
    offsets as there, y [rows, N] bf16, fp16 or fp32."""
    E, N, half = _expect_3d("wq", wq)
    K = 2 * half
    out = _dtype_code("y", y, _ALL_TYPES)
    if not hasattr(xq, "data_ptr"):
        raise TypeError(f"xq: expected a torch.Tensor, got {type(xq).__name__}")
    rows = xq.shape[0] if xq.dim() == 2 else -1
    dev = xq.device
    if not (xq.is_cuda and xq.dtype is torch.uint8 and xq.shape == (rows, half) and xq.is_contiguous()):
        _expect("xq", xq, torch.uint8, (rows, half))
    _expect_like("x_scale", x_scale, torch.uint8, (rows, K // 32), dev)
    _expect_like("wq", wq, torch.uint8, (E, N, half), dev)
    _expect_like("w_scale", w_scale, torch.uint8, (E, N, K // 32), dev)
    _expect_like("offsets", offsets, torch.int32, (E + 1,), dev)
    ldy = _expect_rows("y", y, (rows, N), dev)
    d = _gmm_desc(rows, E, N, K, MOE_DTYPE_MXFP4, out)
    st = _call_on(dev, stream, lib().moe_grouped_matmul_mxfp4, ctypes.byref(d), xq.data_ptr(), x_scale.data_ptr(),
                  wq.data_ptr(), w_scale.data_ptr(), offsets.data_ptr(), y.data_ptr(), ldy)
    if check:
        _check(st, "moe_grouped_matmul_mxfp4")
    return st


def _mxfp4_rows(name, t, q, scale):
    """(rows, K, row stride) of the values ``t`` [.., K] beside codes ``q`` [.., K/2]
    and exponents ``scale`` [.., K/32]."""
    if t.dim() < 2:
        raise ValueError(f"{name}: expected [.., K], got shape {tuple(t.shape)}")
    *lead, K = t.shape
    if len(lead) == 1:
        rows = lead[0]
        ld = _expect_rows(name, t, (rows, K))
    else:
        _expect(name, t, t.dtype, t.shape)
        ld, rows = K, 1
        for n in lead:
            rows *= n
    if K > _I32_MAX:
        _expect_i32(K=K)
    dev = t.device
    _expect_like("q", q, torch.uint8, (*lead, K // 2), dev)
    _expect_like("scale", scale, torch.uint8, (*lead, K // 32), dev)
    return rows, K, ld


def moe_mxfp4_quantize(x, q, scale, stream=None, check: bool = True) -> int:
    """Values x [.., K] (bf16, fp16 or fp32; K a multiple of 32; a 2-d x may have a
    row stride) to MXFP4: codes q [.., K/2] and E8M0 exponents scale [.., K/32], uint8."""
    dt = _dtype_code("x", x, _ALL_TYPES)
    rows, K, ld = _mxfp4_rows("x", x, q, scale)
    st = _call_on(x.device, stream, lib().moe_mxfp4_quantize, dt, x.data_ptr(), ld, rows, K, q.data_ptr(),
                  scale.data_ptr())
    if check:
        _check(st, "moe_mxfp4_quantize")
    return st


def moe_mxfp4_dequantize(q, scale, y, stream=None, check: bool = True) -> int:
    """The values MXFP4 codes q [.., K/2] and exponents scale [.., K/32] stand for,
    exact: y [.., K] bf16 or fp32 (a 2-d y may have a row stride)."""
    dt = _dtype_code("y", y, (MOE_DTYPE_F32, MOE_DTYPE_BF16))
    rows, K, ld = _mxfp4_rows("y", y, q, scale)
    st = _call_on(y.device, stream, lib().moe_mxfp4_dequantize, dt, q.data_ptr(), scale.data_ptr(), rows, K,
                  y.data_ptr(), ld)
    if check:
        _check(st, "moe_mxfp4_dequantize")
    return st


def moe_align_offsets(expert_block_ids, num_padded, E: int, b: int, offsets, stream=None,
                      check: bool = True) -> int:
    """Row offsets [E + 1] int32 of moe_align's blocks, as moe_grouped_matmul takes
    them; with b == 1 expert e's routes are sorted_route_ids[offsets[e]:offsets[e + 1]]."""
    if not hasattr(expert_block_ids, "data_ptr"):
        raise TypeError(f"expert_block_ids: expected a torch.Tensor, got {type(expert_block_ids).__name__}")
    n = expert_block_ids.numel()
    dev = expert_block_ids.device
    if dev.type != "cuda":
        _expect("expert_block_ids", expert_block_ids, torch.int32, (n,))
    _expect_like("expert_block_ids", expert_block_ids, torch.int32, (n,), dev)
    _expect_like("num_padded", num_padded, torch.int32, (1,), dev)
    _expect_like("offsets", offsets, torch.int32, (E + 1,), dev)
    if E > _I32_MAX or not -_I32_MAX <= b <= _I32_MAX:
        _expect_i32(E=E, b=b)
    st = _call_on(dev, stream, lib().moe_align_offsets, expert_block_ids.data_ptr(), num_padded.data_ptr(), n, E, b,
                  offsets.data_ptr())
    if check:
        _check(st, "moe_align_offsets")
    return st


# ---------------------------------------------------------------------------
# Routing, the weighted sum of routes, products with packed 4-bit weights
# ---------------------------------------------------------------------------

def _expect_2d(name, t):
    if not hasattr(t, "data_ptr"):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected 2 dimensions, got shape {tuple(t.shape)}")
    return t.shape


def _expect_logits(name, t, shape, device=None):
    """_expect_rows without its rule for one row: any stride from the row's length on."""
    ld = _expect_rows(name, t, shape, device)
    return ld if shape[0] > 1 else shape[1]


def _route_desc(M, E, k, dtype, score, renormalize, scale, groups, topk_groups, group_top):
    if not 0 <= groups | topk_groups | group_top | score | M | E | k <= _I32_MAX:
        _expect_i32(M=M, E=E, k=k, score=score, groups=groups, topk_groups=topk_groups, group_top=group_top)
    return moe_route_desc(M, E, k, dtype, score, 1 if renormalize else 0, scale, groups, topk_groups, group_top)


def moe_route(logits, topk_ids, topk_w, bias=None, score: int = MOE_SCORE_SOFTMAX, renormalize: bool = True,
              scale: float = 1.0, groups: int = 1, topk_groups: int = 1, group_top: int = 1, stream=None,
              check: bool = True) -> int:
    """Routes tokens to experts: topk_ids [M, k] int32 and topk_w [M, k] fp32 of logits
    [M, E] (bf16, fp16 or fp32; may have a row stride).

    The score is softmax or sigmoid (MOE_SCORE_*), the choice by score + bias ([E] fp32,
    or None), within the topk_groups of `groups` groups whose group_top largest values
    sum highest; weights are scale * score, divided by the chosen scores' sum with
    renormalize. Ties go to the lowest index; experts at -inf are never chosen, and
    where fewer than k are left the rest is expert -1 with weight 0."""
    M, E = _expect_2d("logits", logits)
    dt = _dtype_code("logits", logits, _ALL_TYPES)
    ld = _expect_logits("logits", logits, (M, E))
    dev = logits.device
    k = topk_ids.shape[1] if hasattr(topk_ids, "data_ptr") and topk_ids.dim() == 2 else -1
    _expect_like("topk_ids", topk_ids, torch.int32, (M, k), dev)
    _expect_like("topk_w", topk_w, torch.float32, (M, k), dev)
    b = None
    if bias is not None:
        _expect_like("bias", bias, torch.float32, (E,), dev)
        b = bias.data_ptr()
    d = _route_desc(M, E, k, dt, score, renormalize, scale, groups, topk_groups, group_top)
    st = _call_on(dev, stream, lib().moe_route, ctypes.byref(d), logits.data_ptr(), ld, b, topk_ids.data_ptr(),
                  topk_w.data_ptr())
    if check:
        _check(st, "moe_route")
    return st


def moe_route_grad(logits, topk_ids, dtopk_w, dlogits, score: int = MOE_SCORE_SOFTMAX, renormalize: bool = True,
                   scale: float = 1.0, stream=None, check: bool = True) -> int:
    """Gradient of moe_route's weights with respect to the logits: dlogits [M, E] (the
    logits' dtype or fp32; may have a row stride) from topk_ids as moe_route wrote them
    and dtopk_w [M, k] fp32. The choice has no gradient, so bias and groups have no part
    in it."""
    M, E = _expect_2d("logits", logits)
    dt = _dtype_code("logits", logits, _ALL_TYPES)
    out = _dtype_code("dlogits", dlogits, (dt, MOE_DTYPE_F32))
    ld = _expect_logits("logits", logits, (M, E))
    dev = logits.device
    k = topk_ids.shape[1] if hasattr(topk_ids, "data_ptr") and topk_ids.dim() == 2 else -1
    _expect_like("topk_ids", topk_ids, torch.int32, (M, k), dev)
    _expect_like("dtopk_w", dtopk_w, torch.float32, (M, k), dev)
    ldd = _expect_logits("dlogits", dlogits, (M, E), dev)
    d = _route_desc(M, E, k, dt, score, renormalize, scale, 1, 1, 1)
    st = _call_on(dev, stream, lib().moe_route_grad, ctypes.byref(d), logits.data_ptr(), ld, topk_ids.data_ptr(),
                  dtopk_w.data_ptr(), out, dlogits.data_ptr(), ldd)
    if check:
        _check(st, "moe_route_grad")
    return st


def moe_align_positions(sorted_route_ids, num_padded, positions, stream=None, check: bool = True) -> int:
    """The inverse of an alignment: positions [M, k] int32, the row of each route in
    moe_align's sorted_route_ids (-1 for a route without one)."""
    if not hasattr(sorted_route_ids, "data_ptr"):
        raise TypeError(f"sorted_route_ids: expected a torch.Tensor, got {type(sorted_route_ids).__name__}")
    n = sorted_route_ids.numel()
    dev = sorted_route_ids.device
    if dev.type != "cuda":
        _expect("sorted_route_ids", sorted_route_ids, torch.int32, (n,))
    _expect_like("sorted_route_ids", sorted_route_ids, torch.int32, (n,), dev)
    _expect_like("num_padded", num_padded, torch.int32, (1,), dev)
    _expect_like("positions", positions, torch.int32, _expect_2d("positions", positions), dev)
    routes = positions.numel()
    if routes > _I32_MAX:
        _expect_i32(routes=routes)
    st = _call_on(dev, stream, lib().moe_align_positions, sorted_route_ids.data_ptr(), num_padded.data_ptr(), n,
                  routes, positions.data_ptr())
    if check:
        _check(st, "moe_align_positions")
    return st


def _slots(positions, topk_w, M, rows, device):
    """(k, pointers of positions and topk_w) of a combine call. Without both, each
    token has the rows' share of it: rows / M routes."""
    if positions is not None:
        k = positions.shape[1] if hasattr(positions, "data_ptr") and positions.dim() == 2 else -1
        _expect_like("positions", positions, torch.int32, (M, k), device)
    elif topk_w is not None:
        k = topk_w.shape[1] if hasattr(topk_w, "data_ptr") and topk_w.dim() == 2 else -1
    else:
        k = rows // M if M > 0 else 1
    if topk_w is not None:
        _expect_like("topk_w", topk_w, torch.float32, (M, k), device)
    if positions is None and rows != M * k:
        raise ValueError(f"positions: needed for {rows} rows of {M} x {k} routes")
    return k, None if positions is None else positions.data_ptr(), None if topk_w is None else topk_w.data_ptr()


def moe_combine(rows, positions, topk_w, y, stream=None, check: bool = True) -> int:
    """y[t] = sum_j topk_w[t, j] rows[positions[t, j]].

    rows [R, H] and y [M, H] bf16, fp16 or fp32 (each may have a row stride), positions
    [M, k] int32 (moe_align_positions; outside [0, R): no row) or None (route t * k + j is
    that row), topk_w [M, k] fp32 or None (ones)."""
    R, H = _expect_2d("rows", rows)
    dt = _dtype_code("rows", rows, _ALL_TYPES)
    out = _dtype_code("y", y, _ALL_TYPES)
    ldr = _expect_rows("rows", rows, (R, H))
    dev = rows.device
    M = y.shape[0] if y.dim() == 2 else -1
    ldy = _expect_rows("y", y, (M, H), dev)
    k, pos, w = _slots(positions, topk_w, M, R, dev)
    if M > _I32_MAX or k > _I32_MAX or R > _I32_MAX or H > _I32_MAX:
        _expect_i32(M=M, k=k, rows=R, H=H)
    d = moe_combine_desc(M, k, H, R, dt, out)
    st = _call_on(dev, stream, lib().moe_combine, ctypes.byref(d), rows.data_ptr(), ldr, pos, w, y.data_ptr(), ldy)
    if check:
        _check(st, "moe_combine")
    return st


def moe_combine_grad(dy, rows, positions, topk_w, drows, dtopk_w, stream=None, check: bool = True) -> int:
    """Gradient of moe_combine: drows[positions[t, j]] = topk_w[t, j] dy[t] and
    dtopk_w[t, j] = rows[positions[t, j]] . dy[t].

    dy [M, H], drows [R, H] of the rows' dtype, dtopk_w [M, k] fp32 or None (rows are not
    read then and may be None). With topk_w and dtopk_w None it gathers tokens into their
    routes' rows. Rows no slot names are left as they were."""
    R, H = _expect_2d("drows", drows)
    dt = _dtype_code("drows", drows, _ALL_TYPES)
    ydt = _dtype_code("dy", dy, _ALL_TYPES)
    lddr = _expect_rows("drows", drows, (R, H))
    dev = drows.device
    M = dy.shape[0] if dy.dim() == 2 else -1
    lddy = _expect_rows("dy", dy, (M, H), dev)
    k, pos, w = _slots(positions, topk_w, M, R, dev)
    ldr, src, dw = 0, None, None
    if dtopk_w is not None:
        _dtype_code("rows", rows, (dt,))
        ldr = _expect_rows("rows", rows, (R, H), dev)
        src = rows.data_ptr()
        _expect_like("dtopk_w", dtopk_w, torch.float32, (M, k), dev)
        dw = dtopk_w.data_ptr()
    if M > _I32_MAX or k > _I32_MAX or R > _I32_MAX or H > _I32_MAX:
        _expect_i32(M=M, k=k, rows=R, H=H)
    d = moe_combine_desc(M, k, H, R, dt, ydt)
    st = _call_on(dev, stream, lib().moe_combine_grad, ctypes.byref(d), dy.data_ptr(), lddy, src, ldr, pos, w,
                  drows.data_ptr(), lddr, dw)
    if check:
        _check(st, "moe_combine_grad")
    return st


def moe_matvec_int4(x, w, y, topk_ids=None, stream=None, check: bool = True) -> int:
    """Products of a few rows with packed 4-bit weights: y[t] = W x[t], or with topk_ids
    [M, k] int32 y[t, j] = W[topk_ids[t, j]] x[t] (zero for an ID outside [0, E)).

    x [M, K] bf16 or fp16 (may have a row stride), w a DeviceProjection of int4 weights
    (q int32 [E, N, K / 8], scale fp16 or its int16 bits [E, N, K / group], zero uint8 as
    scale or None: 8), y of x's dtype or fp32: [M, N] (may have a row stride), or
    [M, k, N]."""
    M, K = _expect_2d("x", x)
    dt = _dtype_code("x", x, _GMM_TYPES)
    out = _dtype_code("y", y, (dt, MOE_DTYPE_F32))
    ldx = _expect_rows("x", x, (M, K))
    dev = x.device
    if not hasattr(w, "zero"):
        raise TypeError(f"w: expected a DeviceProjection, got {type(w).__name__}")
    q, scale, zero, group = w.q, w.scale, w.zero, w.group
    E, N, words = _expect_3d("q", q)
    if words * 8 != K:
        raise ValueError(f"q: expected shape {(E, N, K // 8)}, got {tuple(q.shape)}")
    _expect_like("q", q, torch.int32, (E, N, words), dev)
    parts = (E, N, K // group if group > 0 else 0)
    _expect_like("scale", scale, torch.float16 if getattr(scale, "dtype", None) is torch.float16 else torch.int16,
                 parts, dev)
    z = None
    if zero is not None:
        _expect_like("zero", zero, torch.uint8, parts, dev)
        z = zero.data_ptr()
    if topk_ids is None:
        k, ids = 1, None
        ldy = _expect_rows("y", y, (M, N), dev)
        ldy = ldy if M > 1 else N
    else:
        k = topk_ids.shape[1] if hasattr(topk_ids, "data_ptr") and topk_ids.dim() == 2 else -1
        _expect_like("topk_ids", topk_ids, torch.int32, (M, k), dev)
        ids, ldy = topk_ids.data_ptr(), N
        _expect_like("y", y, y.dtype, (M, k, N), dev)
    if M > _I32_MAX or k > _I32_MAX or K > _I32_MAX or N > _I32_MAX or E > _I32_MAX or group > _I32_MAX:
        _expect_i32(M=M, k=k, K=K, N=N, E=E, group=group)
    d = moe_matvec_desc(M, k, E, N, K, dt, out, moe_weights(w.fmt, group, q.data_ptr(), scale.data_ptr(), z))
    st = _call_on(dev, stream, lib().moe_matvec_int4, ctypes.byref(d), x.data_ptr(), ldx, ids, y.data_ptr(), ldy)
    if check:
        _check(st, "moe_matvec_int4")
    return st
