"""Python binding of libswz.so: swizzled LDS tile movement on gfx950.

Argument marshalling only.  Every step of the path runs in the HIP kernels of
libswz.so; there is no Python or CPU fallback, and importing this package
raises if the library has not been built (``python tiled_movement_amd/build.py``).

Functions take torch tensors (or raw device addresses as ints) and the
library's enum values; they run on the current torch stream of their tensors'
device unless a stream is given (a call of addresses alone on the NULL
stream), and raise ``SwzError`` on a negative status.
"""

from __future__ import annotations

import array
import ctypes
import operator
import os
from typing import Optional, Tuple

_dtype = operator.attrgetter("dtype")
_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libswz.so")

# enum values of include/swz.h
SWZ_OK, SWZ_EINVAL, SWZ_EUNSUPPORTED, SWZ_EHIP = 0, -1, -2, -3
LAYOUT_SWIZZLE, LAYOUT_PAD, LAYOUT_PLAIN, LAYOUT_SWIZZLE_DIRECT = 0, 1, 2, 3
READ_AUTO, READ_SCALAR_COL, READ_B64_4X4, READ_B128_8X8, READ_MFMA_16X16X32, READ_B64_TR16, READ_B64_TR8 = (
    -1, 0, 1, 2, 3, 4, 5)
READ_NARROW1, READ_NARROW2, READ_NARROW4, READ_NARROW8, READ_NARROW16 = 6, 7, 8, 9, 10
READ_HNARROW1, READ_HNARROW2, READ_HNARROW4, READ_HNARROW8, READ_HNARROW16, READ_HNARROW32 = 11, 12, 13, 14, 15, 16
READ_BNARROW1, READ_BNARROW2, READ_BNARROW4, READ_BNARROW8, READ_BNARROW16, READ_BNARROW32, READ_BNARROW64 = (
    17, 18, 19, 20, 21, 22, 23)
READ_ROWS = 24
FRAG_MFMA_F32_16X16X32_BF16 = 0
ORDER_DIAGONAL, ORDER_HALF_DIAGONAL, ORDER_COLUMNS, ORDER_STEEP_DIAGONAL = 0, 1, 2, 3
ORDER_SLOPE_8, ORDER_SLOPE_16, ORDER_SLOPE_32 = 4, 5, 6
ORDERS = tuple(range(7))
C_F32, C_BF16 = 0, 1
X_BF16, X_F16, X_F32 = 0, 1, 2
F8_E4M3, F8_E5M2 = 0, 1
BLOCK_1X128, BLOCK_128X128 = 0, 1
SCALE_F32, SCALE_E8M0 = 0, 1
ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2
LAYOUTS = {"swizzle": LAYOUT_SWIZZLE, "pad": LAYOUT_PAD, "plain": LAYOUT_PLAIN, "direct": LAYOUT_SWIZZLE_DIRECT}

EXPORTS = (
    "swz_map",
    "swz_map_batch",
    "swz_transpose",
    "swz_convert_layout",
    "swz_set_tile_order",
    "swz_get_tile_order",
    "swz_tune_tile_order",
    "swz_stage_operand",
    "swz_stage_operands",
    "swz_gemm_frag",
    "swz_gemm",
    "swz_gemm_ex",
    "swz_quant_f8",
    "swz_gemm_f8",
    "swz_linear_loss_workspace",
    "swz_linear_ce",
    "swz_linear_ce_grad",
    "swz_linear_distill",
    "swz_linear_distill_grad",
    "swz_gated",
    "swz_gated_workspace",
    "swz_gated_grad",
    "swz_quant_w4",
    "swz_dequant_w4",
    "swz_gemm_w4",
    "swz_gated_w4",
    "swz_grad_norm_workspace",
    "swz_grad_norm",
    "swz_clip_grads",
    "swz_fold",
    "swz_choose",
    "swz_predict_conflicts",
    "swz_kernel_accesses",
    "swz_bank_model_get",
    "swz_plan",
    "swz_strerror",
    "swz_lds_probe",
    "swz_copy",
)


class SwzError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call}: {strerror(status)} ({status})")
        self.status = status


class Params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("M", ctypes.c_int32), ("S", ctypes.c_int32)]

    def tuple(self) -> Tuple[int, int, int]:
        return (self.B, self.M, self.S)


class BankModelInfo(ctypes.Structure):
    _fields_ = [
        ("n_banks", (ctypes.c_int32 * 3) * 2),
        ("bank_bytes", (ctypes.c_int32 * 3) * 2),
        ("phase", ((ctypes.c_uint8 * 64) * 3) * 2),
    ]


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("read_kind", ctypes.c_int32),
        ("tile_rows", ctypes.c_int32),
        ("tile_cols", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("params", Params),
        ("pad_elems", ctypes.c_int32),
        ("lds_bytes", ctypes.c_int32),
        ("vec_bytes", ctypes.c_int32),
        ("aligned", ctypes.c_int32),
        ("threads", ctypes.c_int32),
        ("interior_tiles", ctypes.c_int32),
    ]

    def as_dict(self):
        return {
            "read_kind": self.read_kind,
            "tile": (self.tile_rows, self.tile_cols),
            "layout": self.layout,
            "params": self.params.tuple(),
            "pad_elems": self.pad_elems,
            "lds_bytes": self.lds_bytes,
            "vec_bytes": self.vec_bytes,
            "aligned": bool(self.aligned),
            "threads": self.threads,
            "interior_tiles": self.interior_tiles,
        }


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python tiled_movement_amd/build.py` "
            "(there is no fallback path)"
        )
    try:  # bind to the HIP runtime torch already loaded, if torch is present
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(LIB_PATH)
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    P = ctypes.POINTER
    lib.swz_map.argtypes = [vp, vp, i64, Params, vp]
    lib.swz_map_batch.argtypes = [vp, vp, i64, vp, i32, vp]
    lib.swz_transpose.argtypes = [vp, vp, i64, i64, i32, i32, i32, P(Params), vp]
    lib.swz_convert_layout.argtypes = [vp, vp, i64, i64, i64, i32, i32, i32, P(Params), vp]
    lib.swz_set_tile_order.argtypes = [i64, i64, i64, i32, i32, i32]
    lib.swz_get_tile_order.argtypes = [i64, i64, i64, i32, i32, P(ctypes.c_int32)]
    lib.swz_tune_tile_order.argtypes = [vp, vp, i64, i64, i64, i32, i32, i32, P(Params), i32, P(ctypes.c_int32), vp]
    lib.swz_stage_operand.argtypes = [vp, vp, i64, i64, i32, i32, i32, P(Params), vp]
    lib.swz_stage_operands.argtypes = [vp, vp, i64, vp, vp, i64, i64, i32, i32, i32, P(Params), vp]
    lib.swz_gemm_frag.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp]
    lib.swz_gemm.argtypes = [vp, vp, vp, i64, i64, i64, i32, P(Params), vp]
    lib.swz_gemm_ex.argtypes = [vp, vp, vp, i64, i64, i64, i32, P(Params), i32, vp]
    lib.swz_fold.argtypes = [P(Params), ctypes.c_uint32, ctypes.c_uint32, P(ctypes.c_uint32), P(ctypes.c_uint32),
                             P(i64)]
    lib.swz_choose.argtypes = [i32, i32, i32, i32, i32, P(Params)]
    lib.swz_predict_conflicts.argtypes = [i32, i32, P(Params), P(i64), P(i64)]
    lib.swz_kernel_accesses.argtypes = [i32, i32, P(Params), i32, P(i32), i32, P(i32), P(i32)]
    lib.swz_bank_model_get.argtypes = [P(BankModelInfo)]
    lib.swz_plan.argtypes = [i32, i64, i64, i32, i32, i32, P(Params), P(PlanInfo)]
    lib.swz_strerror.argtypes = [ctypes.c_int]
    lib.swz_strerror.restype = ctypes.c_char_p
    lib.swz_copy.argtypes = [vp, vp, i64, vp]
    lib.swz_lds_probe.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp]
    lib.swz_quant_f8.argtypes = [vp, i32, i64, i64, i64, i32, i32, i32, vp, vp, i64, vp, vp, i64, vp]
    lib.swz_gemm_f8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, i32, i32, i32, i32, i32, vp]
    f32 = ctypes.c_float
    lib.swz_linear_loss_workspace.argtypes = [i64, i64, i64, i32, i32, P(i64)]
    lib.swz_linear_ce.argtypes = [vp, vp, i32, vp, vp, vp, vp, i64, i64, i64, vp, i64, vp]
    lib.swz_linear_ce_grad.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, i64, vp]
    lib.swz_linear_distill.argtypes = [vp, vp, i32, vp, vp, i32, f32, vp, vp, vp, i64, i64, i64, vp, i64, vp]
    lib.swz_linear_distill_grad.argtypes = [vp, vp, i32, vp, vp, i32, f32, vp, vp, vp, vp, vp, i64, i64, i64, vp, i64, vp]
    feed_forward = {
        "swz_gated": [vp, vp, vp, i32, i32, vp, vp, i64, i64, i64, vp],
        "swz_gated_workspace": [i64, i64, i64, P(i64)],
        "swz_gated_grad": [vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, i64, i64, i64, vp, i64, vp],
        "swz_quant_w4": [vp, i32, i64, i64, i32, i32, vp, vp, vp, vp],
        "swz_dequant_w4": [vp, vp, vp, i64, i64, i32, i32, vp, vp],
        "swz_gemm_w4": [vp, i32, vp, vp, vp, i32, vp, i64, i64, i64, vp],
        "swz_gated_w4": [vp, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp, i64, i64, i64, vp],
        "swz_grad_norm_workspace": [i32, P(i64)],
        "swz_grad_norm": [vp, vp, vp, i32, vp, vp, i64, vp],
        "swz_clip_grads": [vp, vp, vp, vp, i32, f32, vp, vp, i64, vp],
    }
    for name, types in feed_forward.items():
        getattr(lib, name).argtypes = types
    for name in EXPORTS:
        if name != "swz_strerror":
            getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()


def strerror(status: int) -> str:
    return lib.swz_strerror(status).decode()


def _check(status: int, call: str) -> None:
    if status != SWZ_OK:
        raise SwzError(status, call)


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _buf(call: str, **bufs) -> None:
    """Check the device buffers of one call before it reaches the library:
    every tensor is a contiguous CUDA tensor, all on the current device, and
    holds at least the bytes the call reads or writes there, in elements of the
    type it reads (name=(tensor, bytes) or name=(tensor, bytes, type)).
    Raw integer addresses and None pass unchecked (the library checks what
    it can: NULL, alignment, overlap).  Raises ValueError."""
    _bufs(call, [(name, *spec) if len(spec) == 3 else (name, *spec, None) for name, spec in bufs.items()])


def _bufs(call: str, specs) -> None:
    """_buf of (name, tensor, bytes, type or None)."""
    device, other = None, None
    for name, t, need, kind in specs:
        if t is None or isinstance(t, int):
            continue
        if not getattr(t, "is_cuda", False):
            raise ValueError(f"{call}: {name} must be a CUDA tensor (got {type(t).__name__} on "
                             f"{getattr(t, 'device', 'the host')})")
        if not t.is_contiguous():
            raise ValueError(f"{call}: {name} must be contiguous (a strided view is not its own bytes)")
        here = t.device
        if device is None:
            device = here
        elif here != device:
            raise ValueError(f"{call}: {name} is on {here}, the other buffers on {device}")
        have = t.numel() * t.element_size()
        if have < need:
            raise ValueError(f"{call}: {name} holds {have} bytes, the call needs {int(need)}")
        if kind is not None and getattr(t, "dtype", None) not in kind.seen:
            other = other or []
            other.append((name, t, kind))
    for name, t, kind in other or ():
        kind.check(call, name, t)
    if device is not None and device.index is not None:
        import torch

        # the library launches on, and creates its events on, the current device
        cur = torch.cuda.current_device()
        if device.index != cur:
            raise ValueError(f"{call}: the buffers are on {device}, the current device is cuda:{cur} "
                             f"(call inside torch.cuda.device({device.index}))")


_raw_stream = None  # torch's current stream of a device index as an address


def _stream(stream, *tensors):
    global _raw_stream
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    for t in tensors:
        if hasattr(t, "is_cuda") and t.is_cuda:
            if _raw_stream is None:
                import torch

                # the address alone: a stream object costs as much as a launch
                _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
                    lambda index: torch.cuda.current_stream(index).cuda_stream)
            return _raw_stream(t.device.index)
    return None


def _params(p) -> Optional[ctypes.pointer]:
    if p is None:
        return None
    if isinstance(p, Params):
        return ctypes.pointer(p)
    B, M, S = p
    return ctypes.pointer(Params(B, M, S))


def _layout(layout) -> int:
    return LAYOUTS[layout] if isinstance(layout, str) else int(layout)


def swz_map(inp, out, n: int, params, stream=None) -> None:
    B, M, S = params
    _buf("swz_map", inp=(inp, 4 * n), out=(out, 4 * n))
    _check(lib.swz_map(_ptr(inp), _ptr(out), n, Params(B, M, S), _stream(stream, inp, out)), "swz_map")


def swz_set_tile_order(batch: int, rows: int, cols: int, elem_bytes: int, read_kind: int = READ_AUTO,
                       order: int = ORDER_DIAGONAL) -> None:
    _check(lib.swz_set_tile_order(batch, rows, cols, elem_bytes, read_kind, order), "swz_set_tile_order")


def swz_get_tile_order(batch: int, rows: int, cols: int, elem_bytes: int, read_kind: int = READ_AUTO) -> int:
    order = ctypes.c_int32(-1)
    _check(lib.swz_get_tile_order(batch, rows, cols, elem_bytes, read_kind, ctypes.byref(order)),
           "swz_get_tile_order")
    return order.value


def swz_tune_tile_order(src, dst, batch: int, rows: int, cols: int, elem_bytes: int, layout="swizzle",
                        read_kind: int = READ_AUTO, params=None, reps: int = 10, stream=None) -> int:
    """Time every tile order on this conversion, pin the fastest and return it."""
    chosen = ctypes.c_int32(-1)
    nbytes = batch * rows * cols * elem_bytes
    _buf("swz_tune_tile_order", src=(src, nbytes), dst=(dst, nbytes))
    _check(lib.swz_tune_tile_order(_ptr(src), _ptr(dst), batch, rows, cols, elem_bytes, _layout(layout), read_kind,
                                   _params(params), reps, ctypes.byref(chosen), _stream(stream, src, dst)),
           "swz_tune_tile_order")
    return chosen.value


def swz_map_batch(inp, out, n: int, params_list, stream=None) -> None:
    """out[j][i] = Swizzle(params_list[j])(inp[i]); out holds len(params_list) rows of n."""
    arr = (Params * max(len(params_list), 1))(*[Params(*p) for p in params_list])
    _buf("swz_map_batch", inp=(inp, 4 * n), out=(out, 4 * n * len(params_list)))
    _check(lib.swz_map_batch(_ptr(inp), _ptr(out), n, ctypes.addressof(arr), len(params_list),
                             _stream(stream, inp, out)), "swz_map_batch")


def swz_transpose(src, dst, rows: int, cols: int, elem_bytes: int, layout="swizzle", read_kind: int = READ_AUTO,
                  params=None, stream=None) -> None:
    _buf("swz_transpose", src=(src, rows * cols * elem_bytes), dst=(dst, rows * cols * elem_bytes))
    _check(lib.swz_transpose(_ptr(src), _ptr(dst), rows, cols, elem_bytes, _layout(layout), read_kind,
                             _params(params), _stream(stream, src, dst)), "swz_transpose")


def swz_convert_layout(src, dst, batch: int, rows: int, cols: int, elem_bytes: int, layout="swizzle",
                       read_kind: int = READ_AUTO, params=None, stream=None) -> None:
    nbytes = batch * rows * cols * elem_bytes
    _buf("swz_convert_layout", src=(src, nbytes), dst=(dst, nbytes))
    _check(lib.swz_convert_layout(_ptr(src), _ptr(dst), batch, rows, cols, elem_bytes, _layout(layout), read_kind,
                                  _params(params), _stream(stream, src, dst)), "swz_convert_layout")


def swz_stage_operand(src, frag, mn: int, k: int, elem_bytes: int = 2, frag_kind: int = FRAG_MFMA_F32_16X16X32_BF16,
                      layout="swizzle", params=None, stream=None) -> None:
    _buf("swz_stage_operand", src=(src, mn * k * elem_bytes), frag=(frag, mn * k * elem_bytes))
    _check(lib.swz_stage_operand(_ptr(src), _ptr(frag), mn, k, elem_bytes, frag_kind, _layout(layout),
                                 _params(params), _stream(stream, src, frag)), "swz_stage_operand")


def swz_stage_operands(a, fa, m: int, bt, fb, n: int, k: int, elem_bytes: int = 2,
                       frag_kind: int = FRAG_MFMA_F32_16X16X32_BF16, layout="swizzle", params=None,
                       stream=None) -> None:
    """Stage A [m][k] into fa and B^T [n][k] into fb in one launch."""
    _buf("swz_stage_operands", a=(a, m * k * elem_bytes), fa=(fa, m * k * elem_bytes), bt=(bt, n * k * elem_bytes),
         fb=(fb, n * k * elem_bytes))
    _check(lib.swz_stage_operands(_ptr(a), _ptr(fa), m, _ptr(bt), _ptr(fb), n, k, elem_bytes, frag_kind,
                                  _layout(layout), _params(params), _stream(stream, a, fa, bt, fb)),
           "swz_stage_operands")


def swz_gemm_frag(fa, fb, c, m: int, n: int, k: int, frag_kind: int = FRAG_MFMA_F32_16X16X32_BF16,
                  stream=None) -> None:
    _buf("swz_gemm_frag", fa=(fa, 2 * m * k), fb=(fb, 2 * n * k), c=(c, 4 * m * n))
    _check(lib.swz_gemm_frag(_ptr(fa), _ptr(fb), _ptr(c), m, n, k, frag_kind, _stream(stream, fa, fb, c)),
           "swz_gemm_frag")


def swz_gemm(a, bt, c, m: int, n: int, k: int, layout: str = "swizzle", params=None, stream=None) -> None:
    _buf("swz_gemm", a=(a, 2 * m * k), bt=(bt, 2 * n * k), c=(c, 4 * m * n))
    _check(lib.swz_gemm(_ptr(a), _ptr(bt), _ptr(c), m, n, k, _layout(layout), _params(params),
                        _stream(stream, a, bt, c)), "swz_gemm")


def swz_gemm_ex(a, bt, c, m: int, n: int, k: int, layout: str = "swizzle", params=None, c_type: int = C_F32,
                stream=None) -> None:
    _buf("swz_gemm_ex", a=(a, 2 * m * k), bt=(bt, 2 * n * k), c=(c, (2 if c_type == C_BF16 else 4) * m * n))
    _check(lib.swz_gemm_ex(_ptr(a), _ptr(bt), _ptr(c), m, n, k, _layout(layout), _params(params), c_type,
                           _stream(stream, a, bt, c)), "swz_gemm_ex")


class _Type:
    """An element type that a call reads.  Whole numbers of its size pass as its raw bits."""

    def __init__(self, size: int, name: str):
        self.size, self.name = size, name
        self.seen = set()  # torch types found right: a call's own time counts

    def check(self, call: str, name: str, t) -> None:
        if t.element_size() != self.size:
            raise ValueError(f"{call}: {name} has {t.element_size()}-byte elements, the call reads {self.size}-byte ones")
        dtype = getattr(t, "dtype", None)
        if dtype is None:
            return
        if (dtype.is_floating_point or dtype.is_complex) and str(dtype) != f"torch.{self.name}":
            raise ValueError(f"{call}: {name} holds {dtype}, the call reads {self.name}")
        self.seen.add(dtype)


# By the calls' enums; a value that the library does not know leaves its
# buffers to the library, which refuses it.
_FLOAT, _BF16, _BYTE_SCALE, _INDEX = _Type(4, "float32"), _Type(2, "bfloat16"), _Type(1, "float8_e8m0fnu"), _Type(8, "int64")
_X = {X_BF16: _BF16, X_F16: _Type(2, "float16"), X_F32: _FLOAT}
_F8 = {F8_E4M3: _Type(1, "float8_e4m3fn"), F8_E5M2: _Type(1, "float8_e5m2")}
_SCALE = {SCALE_F32: _FLOAT, SCALE_E8M0: _BYTE_SCALE}
_C = {C_F32: _FLOAT, C_BF16: _BF16}


def _span(rows: int, cols: int, ld: int) -> int:
    """Elements from the first of [rows][ld] to the last row's last of `cols`."""
    return (rows - 1) * ld + cols if rows > 0 and cols > 0 else 0


def _f8_scale_bytes(rows: int, cols: int, block: int, scale_type: int) -> int:
    return (-(-rows // 128) if block == BLOCK_128X128 else rows) * -(-cols // 128) * (1 if scale_type == SCALE_E8M0 else 4)


def swz_quant_f8(x, q, scale, rows: int, cols: int, x_type: int = X_BF16, f8_type: int = F8_E4M3,
                 block: int = BLOCK_1X128, scale_type: int = SCALE_E8M0, ld_x: Optional[int] = None,
                 ld_q: Optional[int] = None, qt=None, scale_t=None, ld_qt: Optional[int] = None, stream=None) -> None:
    """x [rows][cols] to 8-bit values q with power-of-two scales, and its transpose qt [cols][rows].

    Pitches default to tight rows (ld_x) and to tight rows rounded up to 16 bytes (ld_q, ld_qt)."""
    ld_x = cols if ld_x is None else ld_x
    ld_q = -(-cols // 16) * 16 if ld_q is None else ld_q
    ld_qt = -(-rows // 16) * 16 if ld_qt is None else ld_qt
    f8, sc = _F8.get(f8_type), _SCALE.get(scale_type)
    _buf("swz_quant_f8", x=(x, _span(rows, cols, ld_x) * (4 if x_type == X_F32 else 2), _X.get(x_type)),
         q=(q, _span(rows, cols, ld_q), f8), scale=(scale, _f8_scale_bytes(rows, cols, block, scale_type), sc),
         qt=(qt, _span(cols, rows, ld_qt), f8), scale_t=(scale_t, _f8_scale_bytes(cols, rows, block, scale_type), sc))
    _check(lib.swz_quant_f8(_ptr(x), x_type, rows, cols, ld_x, f8_type, block, scale_type, _ptr(q), _ptr(scale), ld_q,
                            _ptr(qt), _ptr(scale_t), ld_qt, _stream(stream, x, q, scale, qt, scale_t)), "swz_quant_f8")


def swz_gemm_f8(a, scale_a, b, scale_b, c, m: int, n: int, k: int, lda: Optional[int] = None,
                ldb: Optional[int] = None, a_type: int = F8_E4M3, b_type: int = F8_E4M3, a_block: int = BLOCK_1X128,
                b_block: int = BLOCK_128X128, scale_type: int = SCALE_E8M0, c_type: int = C_BF16, stream=None) -> None:
    """C [m][n] = A B^T of 8-bit operands with scales (pitches default to k rounded up to 16 bytes)."""
    lda = -(-k // 16) * 16 if lda is None else lda
    ldb = -(-k // 16) * 16 if ldb is None else ldb
    k16, sc = -(-k // 16) * 16, _SCALE.get(scale_type)
    _buf("swz_gemm_f8", a=(a, _span(m, k16, lda), _F8.get(a_type)),
         scale_a=(scale_a, _f8_scale_bytes(m, k, a_block, scale_type), sc),
         b=(b, _span(n, k16, ldb), _F8.get(b_type)), scale_b=(scale_b, _f8_scale_bytes(n, k, b_block, scale_type), sc),
         c=(c, (2 if c_type == C_BF16 else 4) * m * n, _C.get(c_type)))
    _check(lib.swz_gemm_f8(_ptr(a), _ptr(scale_a), _ptr(b), _ptr(scale_b), _ptr(c), m, n, k, lda, ldb, a_type, b_type,
                           a_block, b_block, scale_type, c_type, _stream(stream, a, b, c, scale_a, scale_b)), "swz_gemm_f8")


def swz_linear_loss_workspace(n: int, v: int, k: int, top: int = 1, grad: bool = False) -> int:
    """Bytes of workspace for the losses below (grad: for their gradients too)."""
    out = ctypes.c_int64()
    _check(lib.swz_linear_loss_workspace(n, v, k, top, 1 if grad else 0, ctypes.byref(out)), "swz_linear_loss_workspace")
    return out.value


def _ws_bytes(ws, need: int) -> int:
    """Bytes of a workspace tensor (a raw address is taken to hold what the call needs)."""
    return need if ws is None or isinstance(ws, int) else ws.numel() * ws.element_size()


def swz_linear_ce(h, w, target, loss, lse, zt, n: int, v: int, k: int, ws, x_type: int = X_BF16, stream=None) -> None:
    """loss[i] = lse[i] - zt[i] of the logits h w^T, which are not kept (target: int64)."""
    need = swz_linear_loss_workspace(n, v, k)
    xt = _X.get(x_type)
    _buf("swz_linear_ce", h=(h, 2 * n * k, xt), w=(w, 2 * v * k, xt), target=(target, 8 * n, _INDEX),
         loss=(loss, 4 * n, _FLOAT), lse=(lse, 4 * n, _FLOAT), zt=(zt, 4 * n, _FLOAT), ws=(ws, need))
    _check(lib.swz_linear_ce(_ptr(h), _ptr(w), x_type, _ptr(target), _ptr(loss), _ptr(lse), _ptr(zt), n, v, k, _ptr(ws),
                             _ws_bytes(ws, need), _stream(stream, h, w, target, loss, lse, zt, ws)), "swz_linear_ce")


def swz_linear_ce_grad(h, w, target, lse, zt, upstream, dh, dw, n: int, v: int, k: int, ws, x_type: int = X_BF16,
                       stream=None) -> None:
    """dh [n][k] and dw [v][k] of sum(upstream * loss); either may be None."""
    need = swz_linear_loss_workspace(n, v, k, grad=True)
    xt = _X.get(x_type)
    _buf("swz_linear_ce_grad", h=(h, 2 * n * k, xt), w=(w, 2 * v * k, xt), target=(target, 8 * n, _INDEX),
         lse=(lse, 4 * n, _FLOAT), zt=(zt, 4 * n, _FLOAT), upstream=(upstream, 4 * n, _FLOAT), dh=(dh, 2 * n * k, xt),
         dw=(dw, 2 * v * k, xt), ws=(ws, need))
    _check(lib.swz_linear_ce_grad(_ptr(h), _ptr(w), x_type, _ptr(target), _ptr(lse), _ptr(zt), _ptr(upstream), _ptr(dh),
                                  _ptr(dw), n, v, k, _ptr(ws), _ws_bytes(ws, need),
                                  _stream(stream, h, w, target, lse, zt, upstream, dh, dw, ws)),
           "swz_linear_ce_grad")


def swz_linear_distill(h, w, index, teacher, loss, lse, zt, n: int, v: int, k: int, top: int, tau: float, ws,
                       x_type: int = X_BF16, stream=None) -> None:
    """tau^2 KL(teacher's top logits || softmax(h w^T / tau)) per row (index: int64 [n][top], teacher: fp32)."""
    need = swz_linear_loss_workspace(n, v, k, top)
    xt = _X.get(x_type)
    _buf("swz_linear_distill", h=(h, 2 * n * k, xt), w=(w, 2 * v * k, xt), index=(index, 8 * n * top, _INDEX),
         teacher=(teacher, 4 * n * top, _FLOAT), loss=(loss, 4 * n, _FLOAT), lse=(lse, 4 * n, _FLOAT),
         zt=(zt, 4 * n * top, _FLOAT), ws=(ws, need))
    _check(lib.swz_linear_distill(_ptr(h), _ptr(w), x_type, _ptr(index), _ptr(teacher), top, tau, _ptr(loss), _ptr(lse),
                                  _ptr(zt), n, v, k, _ptr(ws), _ws_bytes(ws, need),
                                  _stream(stream, h, w, index, teacher, loss, lse, zt, ws)),
           "swz_linear_distill")


def swz_linear_distill_grad(h, w, index, teacher, lse, zt, upstream, dh, dw, n: int, v: int, k: int, top: int, tau: float,
                            ws, x_type: int = X_BF16, stream=None) -> None:
    """dh [n][k] and dw [v][k] of sum(upstream * loss); either may be None."""
    need = swz_linear_loss_workspace(n, v, k, top, grad=True)
    xt = _X.get(x_type)
    _buf("swz_linear_distill_grad", h=(h, 2 * n * k, xt), w=(w, 2 * v * k, xt), index=(index, 8 * n * top, _INDEX),
         teacher=(teacher, 4 * n * top, _FLOAT), lse=(lse, 4 * n, _FLOAT), zt=(zt, 4 * n * top, _FLOAT),
         upstream=(upstream, 4 * n, _FLOAT), dh=(dh, 2 * n * k, xt), dw=(dw, 2 * v * k, xt), ws=(ws, need))
    _check(lib.swz_linear_distill_grad(_ptr(h), _ptr(w), x_type, _ptr(index), _ptr(teacher), top, tau, _ptr(lse), _ptr(zt),
                                       _ptr(upstream), _ptr(dh), _ptr(dw), n, v, k, _ptr(ws), _ws_bytes(ws, need),

                                       _stream(stream, h, w, index, teacher, lse, zt, upstream, dh, dw, ws)), "swz_linear_distill_grad")


def swz_gated(x, wg, wu, y, n: int, f: int, k: int, x_type: int = X_BF16, act: int = ACT_SILU, pre=None, stream=None) -> None:
    """y [n][f] = act(x wg^T) * (x wu^T); pre (fp32 [2][n][f]), if given, keeps both products for the gradients."""
    xt = _X.get(x_type)
    _bufs("swz_gated", (("x", x, 2 * n * k, xt), ("wg", wg, 2 * f * k, xt), ("wu", wu, 2 * f * k, xt), ("y", y, 2 * n * f, xt),
                        ("pre", pre, 8 * n * f, _FLOAT)))
    _check(lib.swz_gated(_ptr(x), _ptr(wg), _ptr(wu), x_type, act, _ptr(y), _ptr(pre), n, f, k, _stream(stream, x, wg, wu, y, pre)),
           "swz_gated")


def swz_gated_workspace(n: int, f: int, k: int) -> int:
    """Bytes of workspace for swz_gated_grad."""
    out = ctypes.c_int64()
    _check(lib.swz_gated_workspace(n, f, k, ctypes.byref(out)), "swz_gated_workspace")
    return out.value


def swz_gated_grad(x, wg, wu, dy, dx, dwg, dwu, n: int, f: int, k: int, ws, x_type: int = X_BF16, act: int = ACT_SILU,
                   pre=None, stream=None) -> None:
    """dx [n][k], dwg and dwu [f][k] of sum(dy * y); each may be None (not all).  Without pre the products are made again."""
    need = swz_gated_workspace(n, f, k)
    xt = _X.get(x_type)
    _bufs("swz_gated_grad", (("x", x, 2 * n * k, xt), ("wg", wg, 2 * f * k, xt), ("wu", wu, 2 * f * k, xt), ("dy", dy, 2 * n * f, xt),
                             ("pre", pre, 8 * n * f, _FLOAT), ("dx", dx, 2 * n * k, xt), ("dwg", dwg, 2 * f * k, xt),
                             ("dwu", dwu, 2 * f * k, xt), ("ws", ws, need, None)))
    _check(lib.swz_gated_grad(_ptr(x), _ptr(wg), _ptr(wu), x_type, act, _ptr(dy), _ptr(pre), _ptr(dx), _ptr(dwg), _ptr(dwu), n,
                              f, k, _ptr(ws), _ws_bytes(ws, need),
                              _stream(stream, x, wg, wu, dy, pre, dx, dwg, dwu, ws)), "swz_gated_grad")


_CODES = _Type(1, "uint8")


def _w4_groups(n: int, k: int, group: int) -> int:
    return n * -(-k // group) if group > 0 else 0


def swz_quant_w4(w, q, scale, n: int, k: int, group: int = 128, w_type: int = X_BF16, x_type: int = X_BF16, zero=None,
                 stream=None) -> None:
    """w [n][k] to 4-bit codes q [n][k / 2] with scales of x_type per group (and zero points, uint8, if zero is given)."""
    groups = _w4_groups(n, k, group)
    _bufs("swz_quant_w4", (("w", w, n * k * (4 if w_type == X_F32 else 2), _X.get(w_type)), ("q", q, n * (k // 2), _CODES),
                           ("scale", scale, 2 * groups, _X.get(x_type)), ("zero", zero, groups, _CODES)))
    _check(lib.swz_quant_w4(_ptr(w), w_type, n, k, group, x_type, _ptr(q), _ptr(scale), _ptr(zero),
                            _stream(stream, w, q, scale, zero)),
           "swz_quant_w4")


def swz_dequant_w4(q, scale, w, n: int, k: int, group: int = 128, x_type: int = X_BF16, zero=None, stream=None) -> None:
    """w [n][k] (x_type) = (code - zero) * scale."""
    xt, groups = _X.get(x_type), _w4_groups(n, k, group)
    _bufs("swz_dequant_w4", (("w", w, 2 * n * k, xt), ("q", q, n * (k // 2), _CODES), ("scale", scale, 2 * groups, xt),
                             ("zero", zero, groups, _CODES)))
    _check(lib.swz_dequant_w4(_ptr(q), _ptr(scale), _ptr(zero), n, k, group, x_type, _ptr(w), _stream(stream, q, w, scale, zero)),
           "swz_dequant_w4")


def swz_gemm_w4(x, q, scale, c, m: int, n: int, k: int, group: int = 128, x_type: int = X_BF16, zero=None, stream=None) -> None:
    """c [m][n] = x [m][k] W^T of 4-bit weights, for few rows of x."""
    xt, groups = _X.get(x_type), _w4_groups(n, k, group)
    _bufs("swz_gemm_w4", (("x", x, 2 * m * k, xt), ("c", c, 2 * m * n, xt), ("q", q, n * (k // 2), _CODES),
                          ("scale", scale, 2 * groups, xt), ("zero", zero, groups, _CODES)))
    _check(lib.swz_gemm_w4(_ptr(x), x_type, _ptr(q), _ptr(scale), _ptr(zero), group, _ptr(c), m, n, k,
                           _stream(stream, x, q, scale, c, zero)),
           "swz_gemm_w4")


def swz_gated_w4(x, qg, scale_g, qu, scale_u, c, m: int, n: int, k: int, group: int = 128, x_type: int = X_BF16,
                 act: int = ACT_SILU, zero_g=None, zero_u=None, stream=None) -> None:
    """c [m][n] = act(x Wg^T) * (x Wu^T) of 4-bit weights, for few rows of x."""
    xt, groups, codes = _X.get(x_type), _w4_groups(n, k, group), n * (k // 2)
    _bufs("swz_gated_w4", (("x", x, 2 * m * k, xt), ("c", c, 2 * m * n, xt), ("q_g", qg, codes, _CODES),
                           ("scale_g", scale_g, 2 * groups, xt), ("zero_g", zero_g, groups, _CODES), ("q_u", qu, codes, _CODES),
                           ("scale_u", scale_u, 2 * groups, xt), ("zero_u", zero_u, groups, _CODES)))
    _check(lib.swz_gated_w4(_ptr(x), x_type, act, _ptr(qg), _ptr(scale_g), _ptr(zero_g), _ptr(qu), _ptr(scale_u), _ptr(zero_u),
                            group, _ptr(c), m, n, k,
                            _stream(stream, x, qg, scale_g, qu, scale_u, c, zero_g, zero_u)), "swz_gated_w4")


_X_OF = {}  # torch element types of the norm calls, filled by their first call


def _check_tensor(call: str, i: int, t, device) -> None:
    """What is wrong with one of a norm call's tensors, if anything."""
    if getattr(t, "dtype", None) not in _X_OF:
        raise ValueError(f"{call}: tensor {i} is not a bfloat16, float16 or float32 tensor")
    if not t.is_cuda:
        raise ValueError(f"{call}: tensor {i} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{call}: tensor {i} must be contiguous (a strided view is not its own bytes)")
    if t.device.index != device:
        raise ValueError(f"{call}: tensor {i} is on {t.device}, the current device is cuda:{device} "
                         f"(call inside torch.cuda.device({t.device.index}))")


def _tensors(call: str, tensors):
    """A list of tensors as the norm calls read it: (addresses, sizes, types) as arrays of the host, their types and the
    device.  Attributes are asked for list by list, which takes half as long as tensor by tensor."""
    import torch

    if not _X_OF:
        _X_OF.update({torch.bfloat16: X_BF16, torch.float16: X_F16, torch.float32: X_F32})
    device = torch.cuda.current_device() if tensors else None
    alike = {type(t) for t in tensors} <= {torch.Tensor, torch.nn.Parameter}
    if not (alike and set(map(torch.Tensor.get_device, tensors)) <= {device} and all(map(torch.Tensor.is_contiguous, tensors))
            and all(map(_X_OF.__contains__, map(_dtype, tensors)))):
        for i, t in enumerate(tensors):
            _check_tensor(call, i, t, device)
    if alike:
        at, numel = map(torch.Tensor.data_ptr, tensors), map(torch.Tensor.numel, tensors)
    else:
        at, numel = (t.data_ptr() for t in tensors), (t.numel() for t in tensors)
    kinds = list(map(_dtype, tensors))
    return array.array("Q", at), array.array("q", numel), array.array("i", map(_X_OF.__getitem__, kinds)), kinds, device


def _at(a) -> int:
    return a.buffer_info()[0]


def swz_grad_norm_workspace(tensors) -> int:
    """Bytes of workspace for the norm of these tensors."""
    return _norm_workspace("swz_grad_norm_workspace", len(tensors))


def _norm_workspace(call: str, count: int) -> int:
    out = ctypes.c_int64()
    _check(lib.swz_grad_norm_workspace(count, ctypes.byref(out)), call)
    return out.value


def _norm_buffers(call: str, device, norm, floats: int, ws, need: int) -> None:
    here = getattr(norm, "device", None)
    if device is not None and here is not None and here.index != device:
        raise ValueError(f"{call}: norm is on {here}, the tensors on cuda:{device}")
    _bufs(call, (("norm", norm, 4 * floats, _FLOAT), ("ws", ws, need, None)))


def swz_grad_norm(tensors, norm, ws, stream=None) -> None:
    """norm[0] (fp32) = sqrt of the sum of all the tensors' squares."""
    tensors = list(tensors)
    at, numel, types, _, device = _tensors("swz_grad_norm", tensors)
    need = _norm_workspace("swz_grad_norm", len(at))
    _norm_buffers("swz_grad_norm", device, norm, 1, ws, need)
    _check(lib.swz_grad_norm(_at(at), _at(numel), _at(types), len(at), _ptr(norm), _ptr(ws), _ws_bytes(ws, need),
                             _stream(stream, norm, ws, *tensors[:1])), "swz_grad_norm")


def swz_clip_grads(tensors, max_norm: float, norm, ws, out=None, stream=None) -> None:
    """The tensors scaled so that their norm together is at most max_norm, in place or into the tensors of `out`;
    norm (fp32 [2]): the norm before, and the factor."""
    tensors = list(tensors)
    at, numel, types, kinds, device = _tensors("swz_clip_grads", tensors)
    to = None
    if out is not None:
        to, to_numel, _, to_kinds, _ = _tensors("swz_clip_grads", list(out))
        if len(to) != len(at):
            raise ValueError(f"swz_clip_grads: {len(to)} tensors to write, {len(at)} to read")
        if to_numel != numel or to_kinds != kinds:
            i = next(i for i in range(len(at)) if to_numel[i] != numel[i] or to_kinds[i] != kinds[i])
            raise ValueError(f"swz_clip_grads: tensor {i} to write differs from the one to read in size or type")
    need = _norm_workspace("swz_clip_grads", len(at))
    _norm_buffers("swz_clip_grads", device, norm, 2, ws, need)
    _check(lib.swz_clip_grads(_at(at), None if to is None else _at(to), _at(numel), _at(types), len(at), max_norm, _ptr(norm),
                              _ptr(ws), _ws_bytes(ws, need), _stream(stream, norm, ws, *tensors[:1])), "swz_clip_grads")


def swz_fold(params, base: int, active: int):
    """(collision, folded_base or None, strides dict {bit: stride} or None)."""
    c, fb = ctypes.c_uint32(), ctypes.c_uint32()
    st = (ctypes.c_int64 * 32)()
    rc = lib.swz_fold(ctypes.byref(Params(*params)), base, active, ctypes.byref(c), ctypes.byref(fb), st)
    if rc == SWZ_EUNSUPPORTED:
        return c.value, None, None
    _check(rc, "swz_fold")
    return c.value, fb.value, {b: st[b] for b in range(32) if (active >> b) & 1}


def swz_choose(elem_bytes: int, vec_bytes: int, tile_rows: int, tile_cols: int, read_kind: int) -> Tuple[int, int, int]:
    out = Params()
    _check(lib.swz_choose(elem_bytes, vec_bytes, tile_rows, tile_cols, read_kind, ctypes.byref(out)), "swz_choose")
    return out.tuple()


def swz_predict_conflicts(read_kind: int, layout="swizzle", params=None) -> Tuple[int, int]:
    w, r = ctypes.c_int64(), ctypes.c_int64()
    _check(lib.swz_predict_conflicts(read_kind, _layout(layout), _params(params), ctypes.byref(w), ctypes.byref(r)),
           "swz_predict_conflicts")
    return w.value, r.value


def swz_kernel_accesses(read_kind: int, layout="swizzle", params=None, is_write: int = 0):
    """List of (addresses[64], width) for one tile of the kernel; -1 = idle lane."""
    n, w = ctypes.c_int32(), ctypes.c_int32()
    _check(lib.swz_kernel_accesses(read_kind, _layout(layout), _params(params), is_write, None, 0, ctypes.byref(n),
                                   ctypes.byref(w)), "swz_kernel_accesses")
    buf = (ctypes.c_int32 * (64 * max(n.value, 1)))()
    _check(lib.swz_kernel_accesses(read_kind, _layout(layout), _params(params), is_write, buf, n.value,
                                   ctypes.byref(n), ctypes.byref(w)), "swz_kernel_accesses")
    flat = list(buf)
    return [(flat[64 * i:64 * i + 64], w.value) for i in range(n.value)]


def swz_bank_model_get() -> dict:
    """The built-in bank model, keyed by (direction, bytes per lane) with
    direction "read" or "write": banks, bytes per bank and the phase number
    of every lane."""
    m = BankModelInfo()
    _check(lib.swz_bank_model_get(ctypes.byref(m)), "swz_bank_model_get")
    out = {}
    for d, dname in enumerate(("read", "write")):
        for w, width in enumerate((4, 8, 16)):
            out[(dname, width)] = {
                "n_banks": m.n_banks[d][w],
                "bank_bytes": m.bank_bytes[d][w],
                "phase": list(m.phase[d][w]),
            }
    return out


def swz_plan(op: int, rows: int, cols: int, elem_bytes: int, layout="swizzle", read_kind: int = READ_AUTO,
             params=None) -> dict:
    out = PlanInfo()
    _check(lib.swz_plan(op, rows, cols, elem_bytes, _layout(layout), read_kind, _params(params), ctypes.byref(out)),
           "swz_plan")
    return out.as_dict()


def swz_strerror(status: int) -> str:
    return strerror(status)


def swz_lds_probe(addrs, masks, n_patterns: int, width_bytes: int, is_write: int, iters: int, waves: int, cycles,
                  stream=None) -> None:
    _buf("swz_lds_probe", addrs=(addrs, 4 * 64 * n_patterns), masks=(masks, 8 * n_patterns),
         cycles=(cycles, 8 * n_patterns * waves))
    _check(lib.swz_lds_probe(_ptr(addrs), _ptr(masks), n_patterns, width_bytes, is_write, iters, waves,
                             _ptr(cycles), _stream(stream, addrs, masks, cycles)), "swz_lds_probe")


def swz_copy(src, dst, nbytes: int, stream=None) -> None:
    _buf("swz_copy", src=(src, nbytes), dst=(dst, nbytes))
    _check(lib.swz_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream, src, dst)), "swz_copy")


# Status-returning raw entry points, for callers that test error paths.
raw = lib
