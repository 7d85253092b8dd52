"""ctypes binding of libpagedweight (C ABI in include/pagedweight.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Functions carry the C names.  Tensor arguments are torch tensors on
the GPU (their data_ptr() is passed); `stream` is a torch.cuda.Stream, a raw
hipStream_t integer, or None for torch's current stream.

The library must have been built (python -m any_precision_bitplane_amd.build);
loading fails loudly otherwise -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_char_p, c_float, c_int32, c_int64, c_size_t, c_uint32, c_void_p
from typing import Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpagedweight.so")

PW_OK = 0
PW_ERR_INVALID_ARG = -1
PW_ERR_UNSUPPORTED_SHAPE = -2
PW_ERR_BITWIDTH = -3
PW_ERR_WORKSPACE = -4
PW_ERR_ALIGNMENT = -5
PW_ERR_HIP = -6
PW_ERR_UNSUPPORTED = -7
PW_ERR_OUT_OF_MEMORY = -8

PW_PAGE_CPU = 0
PW_PAGE_GPU = 1
PW_PAGE_IN_TRANSFER = 2

PW_DEV_BAD_EXPERT_ID = 0x1
PW_DEV_BAD_BITWIDTH = 0x2

PW_PATH_AUTO = 0
PW_PATH_GEMV = 1
PW_PATH_MFMA = 2
PW_PATH_MGEMV = 3

PW_STAGE_ROUTE = 0
PW_STAGE_GATE_UP = 1
PW_STAGE_DOWN = 2
PW_STAGE_COMBINE = 3
PW_NUM_STAGES = 4

PW_EVENTS_STAGES = 0
PW_EVENTS_KERNELS = 1

PW_F32 = 0
PW_F16 = 1
PW_BF16 = 2
PW_E4M3 = 3

PW_ACT_NONE = 0
PW_ACT_SILU = 1
PW_ACT_GELU = 2


class PwMoeShape(ctypes.Structure):
    _fields_ = [("hidden", c_int32), ("inter", c_int32), ("num_experts", c_int32), ("top_k", c_int32)]


class PwBlockDesc(ctypes.Structure):
    _fields_ = [("planes", c_void_p), ("lut_all", c_void_p)]


class PwMoeOptions(ctypes.Structure):
    _fields_ = [("path", c_int32), ("mfma_min_tokens", c_int32),
                ("stage_events", c_void_p * (PW_NUM_STAGES + 1)),
                ("mgemv_min_tokens", c_int32), ("event_mode", c_int32)]


class PwPageInfo(ctypes.Structure):
    _fields_ = [("desired", c_int32), ("committed", c_int32), ("resident", c_int32), ("pending", c_int32),
                ("state", c_int32), ("reserved", c_int32), ("arena_offset", ctypes.c_uint64)]


class PwPathInfo(ctypes.Structure):
    _fields_ = [("gemv", c_int32), ("mgemv", c_int32), ("mfma", c_int32), ("mgemv_from", c_int32),
                ("mfma_from", c_int32), ("inline_route", c_int32), ("down_kparts", c_int32), ("launches", c_int32),
                ("mfma_tail", c_int32)]


class PwPlanProblem(ctypes.Structure):
    _fields_ = [("num_blocks", c_int32), ("num_experts", c_int32), ("expert_of", c_void_p),
                ("plane_bytes", c_void_p), ("sensitivity", c_void_p), ("correction", c_void_p),
                ("routing_mass", c_void_p), ("hot_fraction", ctypes.c_double), ("floor_cold", c_int32),
                ("floor_hot", c_int32), ("hot_multiplier", ctypes.c_float), ("reserved", c_int32)]


class PwError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {pw_status_str(status)} ({status})")


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libpagedweight.so (once) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m any_precision_bitplane_amd.build`")
    lib = ctypes.CDLL(path)
    sig = {
        "pw_abi_version": (c_int32, []),
        "pw_status_str": (c_char_p, [c_int32]),
        "pw_plane_words": (c_size_t, [c_int32, c_int32]),
        "pw_lut_elems": (c_size_t, [c_int32]),
        "pw_lut_offset": (c_size_t, [c_int32, c_int32]),
        "pw_check_shape": (c_int32, [POINTER(PwMoeShape), c_int32]),
        "pw_workspace_bytes": (c_size_t, [POINTER(PwMoeShape), c_int32]),
        "pw_workspace_init": (c_int32, [c_void_p, c_size_t, c_void_p]),
        "pw_moe_forward": (c_int32, [POINTER(PwMoeShape), c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_size_t, POINTER(PwMoeOptions), c_void_p]),
        "pw_moe_forward_noalloc": (c_int32, [POINTER(PwMoeShape), c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                             c_void_p, c_void_p, c_void_p, POINTER(PwMoeOptions), c_void_p]),
        "pw_moe_path_info": (c_int32, [POINTER(PwMoeShape), c_int32, POINTER(PwMoeOptions), POINTER(PwPathInfo)]),
        "pw_planes_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
        "pw_pack_planes": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_int32, c_void_p, c_void_p]),
        "pw_dequant_block": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_void_p,
                                       c_void_p]),
        "pw_get_device_status": (c_int32, [c_void_p, POINTER(c_uint32), c_void_p]),
        "pw_router_topk": (c_int32, [POINTER(PwMoeShape), c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
        "pw_moe_forward_routed": (c_int32, [POINTER(PwMoeShape), c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                            c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                            POINTER(PwMoeOptions), c_void_p]),
        "pw_moe_forward_layers": (c_int32, [POINTER(PwMoeShape), c_int32, c_int32, c_void_p, c_void_p, c_void_p,
                                            c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                            POINTER(PwMoeOptions), c_void_p]),
        "pw_plan_bitwidths": (c_int32, [POINTER(PwPlanProblem), c_void_p, ctypes.c_int64, c_void_p,
                                        POINTER(ctypes.c_int64), POINTER(c_int32)]),
        "pw_pager_create": (c_int32, [c_int32, POINTER(c_int32), POINTER(c_int32), c_void_p, c_size_t, c_void_p,
                                      c_void_p, POINTER(c_void_p)]),
        "pw_pager_destroy": (c_int32, [c_void_p]),
        "pw_pager_set_block": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p]),
        "pw_pager_request": (c_int32, [c_void_p, c_int32, c_int32]),
        "pw_pager_execute": (c_int32, [c_void_p, c_void_p]),
        "pw_pager_commit": (c_int32, [c_void_p, c_void_p, c_int32, POINTER(c_int32)]),
        "pw_pager_info": (c_int32, [c_void_p, c_int32, POINTER(PwPageInfo)]),
        "pw_pager_arena_used": (c_size_t, [c_void_p]),
        "pw_rmsnorm": (c_int32, [c_int32, c_int32, c_int32, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64,
                                 c_void_p, c_float, c_int32, c_void_p, c_int64, c_void_p, c_int32, c_void_p]),
        "pw_rmsnorm_backward_workspace_bytes": (c_size_t, [c_int32, c_int32]),
        "pw_rmsnorm_backward": (c_int32, [c_int32, c_int32, c_int32, c_void_p, c_int64, c_void_p, c_int64, c_void_p,
                                          c_float, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_size_t,
                                          c_void_p]),
        "pw_moe_permute_workspace_bytes": (c_size_t, [POINTER(PwMoeShape), c_int32]),
        "pw_moe_permute": (c_int32, [POINTER(PwMoeShape), c_int32, c_int32, c_void_p, c_int64, c_void_p, c_int32,
                                     c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_size_t, c_void_p]),
        "pw_moe_permute_backward": (c_int32, [POINTER(PwMoeShape), c_int32, c_int32, c_void_p, c_int64, c_void_p,
                                              c_void_p, c_int64, c_void_p]),
        "pw_moe_unpermute": (c_int32, [POINTER(PwMoeShape), c_int32, c_int32, c_void_p, c_int64, c_void_p, c_void_p,
                                       c_void_p, c_int64, c_void_p]),
        "pw_moe_unpermute_backward": (c_int32, [POINTER(PwMoeShape), c_int32, c_int32, c_void_p, c_int64, c_void_p,
                                                c_int64, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p]),
        "pw_router_backward_workspace_bytes": (c_size_t, [POINTER(PwMoeShape), c_int32]),
        "pw_router_backward": (c_int32, [POINTER(PwMoeShape), c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
        "pw_moe_forward_block": (c_int32, [POINTER(PwMoeShape), c_int32, c_void_p, c_void_p, c_void_p, c_float,
                                           c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                           c_size_t, POINTER(PwMoeOptions), c_void_p]),
        "pw_moe_product_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32, c_int32]),
        "pw_moe_product_backward_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32, c_int32]),
        "pw_moe_product": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, c_void_p, c_int64, c_void_p, c_void_p,
                                     c_void_p, c_int32, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64,
                                     c_void_p, c_size_t, c_void_p]),
        "pw_moe_product_backward": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, c_void_p, c_int64, c_void_p,
                                              c_int64, c_void_p, c_void_p, c_int32, c_void_p, c_int64, c_void_p,
                                              c_int64, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
        "pw_moe_ffn_workspace_bytes": (c_size_t, [POINTER(PwMoeShape), c_int32]),
        "pw_moe_ffn_backward_workspace_bytes": (c_size_t, [POINTER(PwMoeShape), c_int32]),
        "pw_moe_ffn": (c_int32, [POINTER(PwMoeShape), c_int32, c_int32, c_void_p, c_int64, c_void_p, c_void_p, c_void_p,
                                 c_int32, c_int32, c_void_p, c_int64, c_void_p, c_void_p, c_int64, c_void_p, c_size_t,
                                 c_void_p]),
        "pw_moe_ffn_backward": (c_int32, [POINTER(PwMoeShape), c_int32, c_int32, c_void_p, c_int64, c_void_p, c_int64,
                                          c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_int64, c_void_p,
                                          c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def exported_symbols() -> Sequence[str]:
    return ["pw_abi_version", "pw_status_str", "pw_plane_words", "pw_lut_elems", "pw_lut_offset",
            "pw_check_shape", "pw_workspace_bytes", "pw_workspace_init", "pw_moe_forward", "pw_moe_forward_noalloc",
            "pw_moe_path_info",
            "pw_dequant_block", "pw_planes_bytes", "pw_pack_planes", "pw_get_device_status", "pw_pager_create", "pw_pager_destroy",
            "pw_pager_set_block", "pw_pager_request", "pw_pager_execute", "pw_pager_commit", "pw_pager_info",
            "pw_pager_arena_used", "pw_router_topk", "pw_moe_forward_routed", "pw_moe_forward_layers",
            "pw_plan_bitwidths", "pw_rmsnorm", "pw_rmsnorm_backward_workspace_bytes", "pw_rmsnorm_backward",
            "pw_moe_permute_workspace_bytes", "pw_moe_permute", "pw_moe_permute_backward", "pw_moe_unpermute",
            "pw_moe_unpermute_backward", "pw_router_backward_workspace_bytes", "pw_router_backward",
            "pw_moe_forward_block", "pw_moe_product_workspace_bytes", "pw_moe_product_backward_workspace_bytes",
            "pw_moe_product", "pw_moe_product_backward", "pw_moe_ffn_workspace_bytes",
            "pw_moe_ffn_backward_workspace_bytes", "pw_moe_ffn", "pw_moe_ffn_backward"]


# ---------------------------------------------------------------------------
def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != PW_OK:
        raise PwError(status, what)


def shape(H: int, I: int, E: int, k: int) -> PwMoeShape:
    return PwMoeShape(H, I, E, k)


def pw_abi_version() -> int:
    return load().pw_abi_version()


def pw_status_str(status: int) -> str:
    return load().pw_status_str(status).decode()


def pw_plane_words(N: int, K: int) -> int:
    return load().pw_plane_words(N, K)


def pw_lut_elems(N: int) -> int:
    return load().pw_lut_elems(N)


def pw_lut_offset(N: int, b: int) -> int:
    return load().pw_lut_offset(N, b)


def pw_check_shape(shp: PwMoeShape, T: int) -> int:
    return load().pw_check_shape(ctypes.byref(shp), T)


def pw_workspace_bytes(shp: PwMoeShape, T_max: int) -> int:
    return load().pw_workspace_bytes(ctypes.byref(shp), T_max)


def pw_workspace_init(workspace, stream=None) -> None:
    _check(load().pw_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "pw_workspace_init")


def make_options(path: int = PW_PATH_AUTO, mfma_min_tokens: int = 0, events=None,
                 mgemv_min_tokens: int = 0, event_mode: int = 0) -> PwMoeOptions:
    o = PwMoeOptions()
    o.path = path
    o.mfma_min_tokens = mfma_min_tokens
    o.mgemv_min_tokens = mgemv_min_tokens
    o.event_mode = event_mode
    if events is not None:
        for i, ev in enumerate(events):
            o.stage_events[i] = ev
    return o


def pw_moe_forward(shp: PwMoeShape, T: int, x, ids, w, blocks, q, y, workspace,
                   opts: Optional[PwMoeOptions] = None, stream=None, check: bool = True) -> int:
    ws_bytes = workspace.numel() * workspace.element_size()
    st = load().pw_moe_forward(ctypes.byref(shp), T, _ptr(x), _ptr(ids), _ptr(w), _ptr(blocks), _ptr(q),
                               _ptr(y), _ptr(workspace), ws_bytes,
                               ctypes.byref(opts) if opts is not None else None, _stream(stream))
    if check:
        _check(st, "pw_moe_forward")
    return st


PW_NOALLOC_SCRATCH_BYTES = 64 << 20


def pw_moe_forward_noalloc(shp: PwMoeShape, T: int, x, ids, w, blocks, q, y, status=None,
                           opts: Optional[PwMoeOptions] = None, stream=None, check: bool = True) -> int:
    st = load().pw_moe_forward_noalloc(ctypes.byref(shp), T, _ptr(x), _ptr(ids), _ptr(w), _ptr(blocks), _ptr(q),
                                       _ptr(y), _ptr(status), ctypes.byref(opts) if opts is not None else None,
                                       _stream(stream))
    if check:
        _check(st, "pw_moe_forward_noalloc")
    return st


def pw_moe_path_info(shp: PwMoeShape, T: int, opts: Optional[PwMoeOptions] = None) -> PwPathInfo:
    info = PwPathInfo()
    _check(load().pw_moe_path_info(ctypes.byref(shp), T, ctypes.byref(opts) if opts is not None else None,
                                   ctypes.byref(info)), "pw_moe_path_info")
    return info


def pw_planes_bytes(N: int, K: int, nplanes: int) -> int:
    return load().pw_planes_bytes(N, K, nplanes)


def pw_pack_planes(canon, N: int, K: int, nplanes: int, module: int, dev_layout, stream=None,
                   check: bool = True) -> int:
    st = load().pw_pack_planes(_ptr(canon), N, K, nplanes, module, _ptr(dev_layout), _stream(stream))
    if check:
        _check(st, "pw_pack_planes")
    return st


def pw_dequant_block(planes, lut_all, N: int, K: int, q: int, w_out, module: int = 0, stream=None,
                     check: bool = True) -> int:
    st = load().pw_dequant_block(_ptr(planes), _ptr(lut_all), N, K, q, module, _ptr(w_out), _stream(stream))
    if check:
        _check(st, "pw_dequant_block")
    return st


def pw_get_device_status(workspace, stream=None) -> int:
    flags = c_uint32(0)
    _check(load().pw_get_device_status(_ptr(workspace), ctypes.byref(flags), _stream(stream)),
           "pw_get_device_status")
    return flags.value


# --- router ----------------------------------------------------------------
def pw_router_topk(shp: PwMoeShape, T: int, x, router_w, ids, w, stat_count=None, stat_mass=None, workspace=None,
                   stream=None, check: bool = True) -> int:
    ws_bytes = workspace.numel() * workspace.element_size()
    st = load().pw_router_topk(ctypes.byref(shp), T, _ptr(x), _ptr(router_w), _ptr(ids), _ptr(w), _ptr(stat_count),
                               _ptr(stat_mass), _ptr(workspace), ws_bytes, _stream(stream))
    if check:
        _check(st, "pw_router_topk")
    return st


def pw_moe_forward_routed(shp: PwMoeShape, T: int, x, router_w, blocks, q, y, stat_count, stat_mass, workspace,
                          opts: Optional[PwMoeOptions] = None, stream=None, check: bool = True) -> int:
    ws_bytes = workspace.numel() * workspace.element_size()
    st = load().pw_moe_forward_routed(ctypes.byref(shp), T, _ptr(x), _ptr(router_w), _ptr(blocks), _ptr(q), _ptr(y),
                                      _ptr(stat_count), _ptr(stat_mass), _ptr(workspace), ws_bytes,
                                      ctypes.byref(opts) if opts is not None else None, _stream(stream))
    if check:
        _check(st, "pw_moe_forward_routed")
    return st


def pw_moe_forward_layers(shp: PwMoeShape, T: int, x, router_ws, blocks, qs, y, stat_count, stat_mass, workspace,
                          opts: Optional[PwMoeOptions] = None, stream=None, check: bool = True) -> int:
    """router_ws, blocks, qs: sequences of device tensors, one per layer."""
    L = len(router_ws)
    arr = lambda ts: (c_void_p * L)(*[_ptr(t) for t in ts])
    ws_bytes = workspace.numel() * workspace.element_size()
    st = load().pw_moe_forward_layers(ctypes.byref(shp), L, T, _ptr(x), arr(router_ws), arr(blocks), arr(qs), _ptr(y),
                                      _ptr(stat_count), _ptr(stat_mass), _ptr(workspace), ws_bytes,
                                      ctypes.byref(opts) if opts is not None else None, _stream(stream))
    if check:
        _check(st, "pw_moe_forward_layers")
    return st


# --- around the layer ------------------------------------------------------
# These calls take torch tensors: types and row strides come from them.  What
# the library cannot see in a pointer is checked here first (device, type, a
# contiguous last dimension, sizes) and refused as the library would refuse it.
_torch = None
_current_stream = None   # GPU index -> raw handle of torch's current stream there
_current_device = None   # -> index of the current GPU
_DTYPES: dict = {}


def _load_ops() -> ctypes.CDLL:
    global _torch, _current_stream, _current_device
    if _torch is None:
        import torch
        # the handle alone, without a Stream object around it (1.0 us less a call), where torch offers that
        _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _DTYPES.update({torch.float32: PW_F32, torch.float16: PW_F16, torch.bfloat16: PW_BF16,
                        torch.float8_e4m3fn: PW_E4M3})
        _torch = torch
    return _lib or load()


class _Refused(Exception):
    pass


def _gpu(t) -> int:
    """The GPU of the call's first tensor."""
    if t is None:
        raise _Refused("a tensor is missing")
    dev = t.get_device()
    if dev < 0:
        raise _Refused("tensors must be on a GPU")
    return dev


def _rows(t, name, n, H, dev, dtype):
    """(pointer, row stride) of a matrix of at least n rows of H elements of dtype."""
    if t is None:
        return None, 0
    shape = t.shape
    if t.get_device() != dev:
        raise _Refused(f"{name} must be on the GPU of the other tensors")
    if len(shape) != 2 or shape[1] != H or shape[0] < n or t.dtype is not dtype:
        raise _Refused(f"{name} must have at least {n} rows of {H} elements of {dtype}")
    stride, inner = t.stride()
    if inner != 1 and H > 1:
        raise _Refused(f"the elements of a row of {name} must lie next to each other")
    return t.data_ptr(), stride if n > 1 else H


def _array(t, name, n, dev, dtype):
    """Pointer of a contiguous tensor of at least n elements of dtype."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise _Refused(f"{name} must be on the GPU of the other tensors")
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise _Refused(f"{name} must be {n} contiguous elements of {dtype}")
    return t.data_ptr()


def _words(t, name, n, dev):
    """Pointer of n contiguous 32-bit words: the library's are unsigned, torch code mostly keeps them in int32."""
    unsigned = t is not None and t.dtype is _torch.uint32
    return _array(t, name, n, dev, _torch.uint32 if unsigned else _torch.int32)


def _scratch(t, dev):
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise _Refused("workspace must be contiguous and on the GPU of the other tensors")
    return t.data_ptr(), t.numel() * t.element_size()


def _table(t, name, nbytes, dev):
    """Pointer of a contiguous tensor of at least nbytes bytes of any type; an address stays as it is."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() != dev:
        raise _Refused(f"{name} must be on the GPU of the other tensors")
    if t.numel() * t.element_size() < nbytes or not t.is_contiguous():
        raise _Refused(f"{name} must be {nbytes} contiguous bytes")
    return t.data_ptr()


def _handle(stream, dev) -> int:
    """Raw handle of a stream of the tensors' GPU; None: torch's current one there."""
    if stream is None:
        return _current_stream(dev)
    if isinstance(stream, int):
        return stream
    if stream.device.index != dev:
        raise _Refused("stream must be one of the tensors' GPU")
    return stream.cuda_stream


def _call(name, check, dev, fn, args) -> int:
    """fn(*args) with the tensors' GPU as the current one."""
    if _current_device() == dev:
        st = fn(*args)
    else:
        with _torch.cuda.device(dev):
            st = fn(*args)
    if st and check:
        raise PwError(st, name)
    return st


def _refuse(name, check, e) -> int:
    if check:
        raise PwError(PW_ERR_INVALID_ARG, f"{name}: {e}") from None
    return PW_ERR_INVALID_ARG


def pw_rmsnorm(T: int, H: int, x, weight, eps: float, y, residual=None, residual_out=None, scale=None, group: int = 0,
               stream=None, check: bool = True) -> int:
    """y: x's type, or torch.float8_e4m3fn with scale fp32 [T][groups]."""
    lib = _load_ops()
    try:
        dev, dt = _gpu(x), x.dtype
        if y is None:
            raise _Refused("a tensor is missing")
        px, sx = _rows(x, "x", T, H, dev, dt)
        pr, sr = _rows(residual, "residual", T, H, dev, dt)
        po, so = _rows(residual_out, "residual_out", T, H, dev, dt)
        py, sy = _rows(y, "y", T, H, dev, y.dtype)
        pc = None if scale is None else _array(scale, "scale", T * ((H + 127) // 128 if group else 1), dev,
                                               _torch.float32)
        return _call("pw_rmsnorm", check, dev, lib.pw_rmsnorm, (
            T, H, _DTYPES.get(dt, -1), px, sx, pr, sr, po, so, _array(weight, "weight", H, dev, dt), eps,
            _DTYPES.get(y.dtype, -1), py, sy, pc, group, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_rmsnorm", check, e)


def pw_rmsnorm_backward_workspace_bytes(T_max: int, H: int) -> int:
    return load().pw_rmsnorm_backward_workspace_bytes(T_max, H)


def pw_rmsnorm_backward(T: int, H: int, dy, r, weight, eps: float, dx, dweight=None, workspace=None, dresidual=None,
                        stream=None, check: bool = True) -> int:
    lib = _load_ops()
    try:
        dev, dt = _gpu(dy), dy.dtype
        pd, sd = _rows(dy, "dy", T, H, dev, dt)
        pr, sr = _rows(r, "r", T, H, dev, dt)
        pa, sa = _rows(dresidual, "dresidual", T, H, dev, dt)
        px, sx = _rows(dx, "dx", T, H, dev, dt)
        pw, nw = _scratch(workspace, dev)
        return _call("pw_rmsnorm_backward", check, dev, lib.pw_rmsnorm_backward, (
            T, H, _DTYPES.get(dt, -1), pd, sd, pr, sr, _array(weight, "weight", H, dev, dt), eps, pa, sa, px, sx,
            _array(dweight, "dweight", H, dev, _torch.float32), pw, nw, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_rmsnorm_backward", check, e)


def pw_moe_permute_workspace_bytes(shp: PwMoeShape, T_max: int) -> int:
    return load().pw_moe_permute_workspace_bytes(ctypes.byref(shp), T_max)


def pw_moe_permute(shp: PwMoeShape, T: int, x, ids, xs, offsets, inv, perm, workspace, x_scale=None, xs_scale=None,
                   status=None, stream=None, check: bool = True) -> int:
    """perm, x_scale with xs_scale, and status may be None."""
    lib = _load_ops()
    try:
        dev, dt = _gpu(x), x.dtype
        H, S, i32, f32 = shp.hidden, T * shp.top_k, _torch.int32, _torch.float32
        groups = 0
        if x_scale is not None:
            if x_scale.dim() != 2:
                raise _Refused("x_scale must have a row of scales per token")
            groups = x_scale.shape[1]
        px, sx = _rows(x, "x", T, H, dev, dt)
        ps, ss = _rows(xs, "xs", S, H, dev, dt)
        pw, nw = _scratch(workspace, dev)
        return _call("pw_moe_permute", check, dev, lib.pw_moe_permute, (
            ctypes.byref(shp), T, _DTYPES.get(dt, -1), px, sx, _array(x_scale, "x_scale", T * groups, dev, f32),
            groups, _array(ids, "ids", S, dev, i32), ps, ss, _array(xs_scale, "xs_scale", S * groups, dev, f32),
            _array(offsets, "offsets", shp.num_experts + 1, dev, i32), _array(inv, "inv", S, dev, i32),
            _array(perm, "perm", S, dev, i32), _words(status, "status", 1, dev), pw, nw, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_moe_permute", check, e)


def pw_moe_permute_backward(shp: PwMoeShape, T: int, dxs, inv, dx, stream=None, check: bool = True) -> int:
    lib = _load_ops()
    try:
        dev, dt, H, S = _gpu(dxs), dxs.dtype, shp.hidden, T * shp.top_k
        ps, ss = _rows(dxs, "dxs", S, H, dev, dt)
        px, sx = _rows(dx, "dx", T, H, dev, dt)
        return _call("pw_moe_permute_backward", check, dev, lib.pw_moe_permute_backward, (
            ctypes.byref(shp), T, _DTYPES.get(dt, -1), ps, ss, _array(inv, "inv", S, dev, _torch.int32), px, sx,
            _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_moe_permute_backward", check, e)


def pw_moe_unpermute(shp: PwMoeShape, T: int, rows, inv, w, y, stream=None, check: bool = True) -> int:
    """w: fp32 [T][k], or None for ones."""
    lib = _load_ops()
    try:
        dev, dt, H, S = _gpu(rows), rows.dtype, shp.hidden, T * shp.top_k
        pr, sr = _rows(rows, "rows", S, H, dev, dt)
        py, sy = _rows(y, "y", T, H, dev, dt)
        return _call("pw_moe_unpermute", check, dev, lib.pw_moe_unpermute, (
            ctypes.byref(shp), T, _DTYPES.get(dt, -1), pr, sr, _array(inv, "inv", S, dev, _torch.int32),
            _array(w, "w", S, dev, _torch.float32), py, sy, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_moe_unpermute", check, e)


def pw_moe_unpermute_backward(shp: PwMoeShape, T: int, dy, rows, inv, w, drows, dw=None, stream=None,
                              check: bool = True) -> int:
    """dw None: not wanted (rows may then be None)."""
    lib = _load_ops()
    try:
        dev, dt, H, S = _gpu(dy), dy.dtype, shp.hidden, T * shp.top_k
        pd, sd = _rows(dy, "dy", T, H, dev, dt)
        pr, sr = _rows(rows, "rows", S, H, dev, dt)
        po, so = _rows(drows, "drows", S, H, dev, dt)
        return _call("pw_moe_unpermute_backward", check, dev, lib.pw_moe_unpermute_backward, (
            ctypes.byref(shp), T, _DTYPES.get(dt, -1), pd, sd, pr, sr, _array(inv, "inv", S, dev, _torch.int32),
            _array(w, "w", S, dev, _torch.float32), po, so, _array(dw, "dw", S, dev, _torch.float32),
            _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_moe_unpermute_backward", check, e)


def pw_router_backward_workspace_bytes(shp: PwMoeShape, T_max: int) -> int:
    return load().pw_router_backward_workspace_bytes(ctypes.byref(shp), T_max)


def pw_router_backward(shp: PwMoeShape, T: int, x, router_w, ids, w, dw, dx, drouter_w, workspace, dx_add=None,
                       stream=None, check: bool = True) -> int:
    lib = _load_ops()
    try:
        dev, n, S, E = _gpu(x), T * shp.hidden, T * shp.top_k, shp.num_experts * shp.hidden
        f16, f32 = _torch.float16, _torch.float32
        pw, nw = _scratch(workspace, dev)
        return _call("pw_router_backward", check, dev, lib.pw_router_backward, (
            ctypes.byref(shp), T, _array(x, "x", n, dev, f16), _array(router_w, "router_w", E, dev, f16),
            _array(ids, "ids", S, dev, _torch.int32), _array(w, "w", S, dev, f32), _array(dw, "dw", S, dev, f32),
            _array(dx_add, "dx_add", n, dev, f16), _array(dx, "dx", n, dev, f16),
            _array(drouter_w, "drouter_w", E, dev, f32), pw, nw, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_router_backward", check, e)


def pw_moe_forward_block(shp: PwMoeShape, T: int, x, residual, norm_w, eps: float, router_w, blocks, q, y, stat_count,
                         stat_mass, workspace, opts: Optional[PwMoeOptions] = None, stream=None,
                         check: bool = True) -> int:
    """blocks and q: tensors, or raw addresses of tables that live elsewhere."""
    lib = _load_ops()
    try:
        dev, H, E, f16 = _gpu(x), shp.hidden, shp.num_experts, _torch.float16
        pw, nw = _scratch(workspace, dev)
        return _call("pw_moe_forward_block", check, dev, lib.pw_moe_forward_block, (
            ctypes.byref(shp), T, _array(x, "x", T * H, dev, f16), _array(residual, "residual", T * H, dev, f16),
            _array(norm_w, "norm_w", H, dev, f16), eps, _array(router_w, "router_w", E * H, dev, f16),
            _table(blocks, "blocks", 2 * E * ctypes.sizeof(PwBlockDesc), dev), _table(q, "q", 2 * E, dev),
            _array(y, "y", T * H, dev, f16), _words(stat_count, "stat_count", E, dev),
            _array(stat_mass, "stat_mass", E, dev, _torch.float32), pw, nw,
            ctypes.byref(opts) if opts is not None else None, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_moe_forward_block", check, e)


# --- expert products in 16 bits ---------------------------------------------
def pw_moe_product_workspace_bytes(E: int, S_max: int, N: int, K: int) -> int:
    return load().pw_moe_product_workspace_bytes(E, S_max, N, K)


def pw_moe_product_backward_workspace_bytes(E: int, S_max: int, N: int, K: int) -> int:
    return load().pw_moe_product_backward_workspace_bytes(E, S_max, N, K)


def pw_moe_product(E: int, S: int, N: int, K: int, x, w, y, workspace, offsets=None, bias=None, act: int = PW_ACT_NONE,
                   residual=None, pre=None, stream=None, check: bool = True) -> int:
    """offsets: int32 [E+1], or None for one expert with all rows."""
    lib = _load_ops()
    try:
        dev, dt = _gpu(x), x.dtype
        px, sx = _rows(x, "x", S, K, dev, dt)
        pr, sr = _rows(residual, "residual", S, N, dev, dt)
        pp, sp = _rows(pre, "pre", S, N, dev, dt)
        py, sy = _rows(y, "y", S, N, dev, dt)
        pw, nw = _scratch(workspace, dev)
        return _call("pw_moe_product", check, dev, lib.pw_moe_product, (
            E, S, N, K, _DTYPES.get(dt, -1), px, sx, _array(offsets, "offsets", E + 1, dev, _torch.int32),
            _array(w, "w", E * N * K, dev, dt), _array(bias, "bias", E * N, dev, dt), act, pr, sr, pp, sp, py, sy, pw,
            nw, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_moe_product", check, e)


def pw_moe_product_backward(E: int, S: int, N: int, K: int, dy, x, w, workspace, offsets=None, act: int = PW_ACT_NONE,
                            pre=None, dx=None, dw=None, dbias=None, stream=None, check: bool = True) -> int:
    """dx, dw, dbias None: not wanted (without dx, w may be None; without dw, x may be)."""
    lib = _load_ops()
    try:
        dev, dt = _gpu(dy), dy.dtype
        pd, sd = _rows(dy, "dy", S, N, dev, dt)
        px, sx = _rows(x, "x", S, K, dev, dt)
        pp, sp = _rows(pre, "pre", S, N, dev, dt)
        po, so = _rows(dx, "dx", S, K, dev, dt)
        pw, nw = _scratch(workspace, dev)
        return _call("pw_moe_product_backward", check, dev, lib.pw_moe_product_backward, (
            E, S, N, K, _DTYPES.get(dt, -1), pd, sd, px, sx, _array(offsets, "offsets", E + 1, dev, _torch.int32),
            _array(w, "w", E * N * K, dev, dt), act, pp, sp, po, so, _array(dw, "dw", E * N * K, dev, dt),
            _array(dbias, "dbias", E * N, dev, dt), pw, nw, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_moe_product_backward", check, e)


def pw_moe_ffn_workspace_bytes(shp: PwMoeShape, S_max: int) -> int:
    return load().pw_moe_ffn_workspace_bytes(ctypes.byref(shp), S_max)


def pw_moe_ffn_backward_workspace_bytes(shp: PwMoeShape, S_max: int) -> int:
    return load().pw_moe_ffn_backward_workspace_bytes(ctypes.byref(shp), S_max)


def _kept(z, z_scale, S, I, dev, dt):
    """(type, pointer, row stride, pointer of the scales) of the checkpoint of gate and up."""
    if z is None:
        return _DTYPES.get(dt, -1), None, 0, _array(z_scale, "z_scale", 0, dev, _torch.float32)
    pz, sz = _rows(z, "z", S, 2 * I, dev, z.dtype)
    return _DTYPES.get(z.dtype, -1), pz, sz, _array(z_scale, "z_scale", S * 2 * ((I + 127) // 128), dev, _torch.float32)


def pw_moe_ffn(shp: PwMoeShape, S: int, x, w_gate_up, w_down, y, workspace, offsets=None, act: int = PW_ACT_SILU,
               z=None, z_scale=None, stream=None, check: bool = True) -> int:
    """z: checkpoint [S][2I] in x's type, or torch.float8_e4m3fn with z_scale fp32 [S][2 ceil(I / 128)]."""
    lib = _load_ops()
    try:
        dev, dt, E, H, I = _gpu(x), x.dtype, shp.num_experts, shp.hidden, shp.inter
        px, sx = _rows(x, "x", S, H, dev, dt)
        py, sy = _rows(y, "y", S, H, dev, dt)
        zt, pz, sz, pc = _kept(z, z_scale, S, I, dev, dt)
        pw, nw = _scratch(workspace, dev)
        return _call("pw_moe_ffn", check, dev, lib.pw_moe_ffn, (
            ctypes.byref(shp), S, _DTYPES.get(dt, -1), px, sx, _array(offsets, "offsets", E + 1, dev, _torch.int32),
            _array(w_gate_up, "w_gate_up", E * 2 * I * H, dev, dt), _array(w_down, "w_down", E * H * I, dev, dt), act,
            zt, pz, sz, pc, py, sy, pw, nw, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_moe_ffn", check, e)


def pw_moe_ffn_backward(shp: PwMoeShape, S: int, dy, x, w_gate_up, w_down, z, workspace, offsets=None,
                        act: int = PW_ACT_SILU, z_scale=None, dx=None, dw_gate_up=None, dw_down=None, stream=None,
                        check: bool = True) -> int:
    """dx, dw_gate_up, dw_down None: not wanted (without dx, w_gate_up may be None; without dw_gate_up, x may be)."""
    lib = _load_ops()
    try:
        dev, dt, E, H, I = _gpu(dy), dy.dtype, shp.num_experts, shp.hidden, shp.inter
        pd, sd = _rows(dy, "dy", S, H, dev, dt)
        px, sx = _rows(x, "x", S, H, dev, dt)
        po, so = _rows(dx, "dx", S, H, dev, dt)
        zt, pz, sz, pc = _kept(z, z_scale, S, I, dev, dt)
        pw, nw = _scratch(workspace, dev)
        return _call("pw_moe_ffn_backward", check, dev, lib.pw_moe_ffn_backward, (
            ctypes.byref(shp), S, _DTYPES.get(dt, -1), pd, sd, px, sx,
            _array(offsets, "offsets", E + 1, dev, _torch.int32),
            _array(w_gate_up, "w_gate_up", E * 2 * I * H, dev, dt), _array(w_down, "w_down", E * H * I, dev, dt), act,
            zt, pz, sz, pc, po, so, _array(dw_gate_up, "dw_gate_up", E * 2 * I * H, dev, dt),
            _array(dw_down, "dw_down", E * H * I, dev, dt), pw, nw, _handle(stream, dev)))
    except _Refused as e:
        return _refuse("pw_moe_ffn_backward", check, e)


# --- planner ----------------------------------------------------------------
def pw_plan_bitwidths(q_cur, plane_bytes, expert_of, sensitivity, correction=None, routing_mass=None,
                      hot_fraction: float = 0.0, floor_cold: int = 3, floor_hot: int = 3,
                      hot_multiplier: float = 1.0, budget_bytes: int = 0, check: bool = True):
    """Host arrays (numpy) in, (status, q_out int32 [B], plane bytes, fits) out."""
    import numpy as np
    q_cur = np.ascontiguousarray(q_cur, dtype=np.int32)
    pb = np.ascontiguousarray(plane_bytes, dtype=np.int64)
    eo = np.ascontiguousarray(expert_of, dtype=np.int32)
    S = np.ascontiguousarray(sensitivity, dtype=np.float32).reshape(len(q_cur), 6)
    R = None if correction is None else np.ascontiguousarray(correction, dtype=np.float32).reshape(len(q_cur), 6)
    M = None if routing_mass is None else np.ascontiguousarray(routing_mass, dtype=np.float32)
    E = int(eo.max()) + 1 if M is None else len(M)
    prob = PwPlanProblem(len(q_cur), E, eo.ctypes.data, pb.ctypes.data, S.ctypes.data,
                         None if R is None else R.ctypes.data, None if M is None else M.ctypes.data,
                         float(hot_fraction), int(floor_cold), int(floor_hot), float(hot_multiplier), 0)
    out = np.zeros(len(q_cur), dtype=np.int32)
    used = ctypes.c_int64(0)
    fits = c_int32(0)
    st = load().pw_plan_bitwidths(ctypes.byref(prob), q_cur.ctypes.data, int(budget_bytes), out.ctypes.data,
                                  ctypes.byref(used), ctypes.byref(fits))
    if check:
        _check(st, "pw_plan_bitwidths")
    return st, out, used.value, bool(fits.value)


# --- weight pager ----------------------------------------------------------
def pw_pager_create(rows: Sequence[int], cols: Sequence[int], arena, arena_bytes: int, blocks, q) -> int:
    n = len(rows)
    r = (c_int32 * n)(*rows)
    c = (c_int32 * n)(*cols)
    out = c_void_p(0)
    _check(load().pw_pager_create(n, r, c, _ptr(arena), arena_bytes, _ptr(blocks), _ptr(q), ctypes.byref(out)),
           "pw_pager_create")
    return out.value


def pw_pager_destroy(pager: int) -> None:
    _check(load().pw_pager_destroy(pager), "pw_pager_destroy")


def pw_pager_set_block(pager: int, b: int, host_planes, lut_all) -> None:
    _check(load().pw_pager_set_block(pager, b, _ptr(host_planes), _ptr(lut_all)), "pw_pager_set_block")


def pw_pager_request(pager: int, b: int, desired: int, check: bool = True) -> int:
    st = load().pw_pager_request(pager, b, desired)
    if check:
        _check(st, "pw_pager_request")
    return st


def pw_pager_execute(pager: int, copy_stream=None, check: bool = True) -> int:
    st = load().pw_pager_execute(pager, _stream(copy_stream))
    if check:
        _check(st, "pw_pager_execute")
    return st


def pw_pager_commit(pager: int, stream=None, wait: bool = True) -> int:
    n = c_int32(0)
    _check(load().pw_pager_commit(pager, _stream(stream), 1 if wait else 0, ctypes.byref(n)), "pw_pager_commit")
    return n.value


def pw_pager_info(pager: int, b: int) -> PwPageInfo:
    info = PwPageInfo()
    _check(load().pw_pager_info(pager, b, ctypes.byref(info)), "pw_pager_info")
    return info


def pw_pager_arena_used(pager: int) -> int:
    return load().pw_pager_arena_used(pager)
