"""Python binding of libconv3d (MI355X / gfx950 fp16 implicit-GEMM conv3d).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libconv3d.so``.  The functions carry the C names of
``include/conv3d.h``.  Tensor arguments may be torch tensors (their
``data_ptr()`` is passed) or raw device addresses (ints); the stream defaults
to torch's current stream on the current device.  There is no CPU fallback:
if the library is missing, importing a function raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libconv3d.so")

CONV3D_OK = 0
CONV3D_ERR_INVALID_ARG = 1
CONV3D_ERR_UNSUPPORTED = 2
CONV3D_ERR_WORKSPACE = 3
CONV3D_ERR_NO_DEVICE = 4
CONV3D_ERR_HIP = 5

CONV3D_TPAD_ZERO = 0
CONV3D_TPAD_REPLICATE = 1

CONV3D_F_BIAS = 1
CONV3D_F_RESIDUAL = 2
CONV3D_F_NO_T1_FASTPATH = 4
CONV3D_F_BF16 = 8
CONV3D_F_CHUNK = 16
CONV3D_F_GN_STATS = 32
CONV3D_F_PREACT = 64
CONV3D_F_POSITIONS = 128
CONV3D_F_LENGTHS = 256
CONV3D_F_TAIL = 512
CONV3D_F_STATE8 = 1024
CONV3D_F_GRAD32 = 2048

CONV3D_ACT_NONE = 0
CONV3D_ACT_SILU = 1
CONV3D_ACT_GELU = 2
CONV3D_ACT_GELU_TANH = 3

ROPE3D_PAIR_ADJACENT = 0
ROPE3D_PAIR_HALVES = 1

CONV3D_PATH_GENERAL = 0
CONV3D_PATH_T1_FOLD = 1
CONV3D_PATH_POINTWISE = 2

EXPORTED = ("conv3d_plan", "conv3d_plan_query", "conv3d_plan_destroy", "conv3d_forward",
            "conv3d_forward_chunk",
            "groupnorm_silu_workspace", "groupnorm_silu", "groupnorm_silu_bf16",
            "groupnorm_silu_from_stats_workspace", "groupnorm_silu_from_stats", "groupnorm_silu_from_stats_bf16",
            "groupnorm_silu_noalloc_max_bytes", "groupnorm_silu_noalloc",
            "linear_plan", "linear_plan_query", "linear_plan_destroy", "linear_forward",
            "linear_backward_workspace", "linear_backward",
            "layernorm", "layernorm_bf16", "layernorm_backward_workspace", "layernorm_backward",
            "layernorm_backward_bf16",
            "rope3d_plan", "rope3d_plan_destroy", "rope3d_forward", "rope3d_backward",
            "attention_plan", "attention_plan_query", "attention_plan_destroy", "attention_forward",
            "attention_backward_workspace", "attention_backward",
            "adamw_plan", "adamw_plan_destroy", "adamw_hyper_pack", "adamw_step",
            "conv3d_calibrate_scratch_bytes",
            "conv3d_calibrate_mfma", "conv3d_calibrate_hbm", "conv3d_clock_stamp_bytes",
            "conv3d_clock_stamp", "conv3d_status_str",
            "conv3d_last_error", "conv3d_version", "conv3d_selftest")


class conv3d_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("n", "t", "h", "w", "c_in", "c_out", "kt", "kh", "kw",
                 "pad_t_front", "pad_t_back", "pad_h", "pad_w", "t_pad_mode")] + \
               [("flags", ctypes.c_uint32)]


class conv3d_plan_info(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("t_out", ctypes.c_int32), ("h_out", ctypes.c_int32),
                ("w_out", ctypes.c_int32), ("gemm_m", ctypes.c_int64), ("gemm_n", ctypes.c_int64),
                ("gemm_k", ctypes.c_int64), ("flops", ctypes.c_double), ("tile_m", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("grid", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_size_t), ("kernel_name", ctypes.c_char * 64),
                ("split_tiles", ctypes.c_int32), ("split_pieces", ctypes.c_int32),
                ("gn_stats_slots", ctypes.c_int32), ("gn_stats_offset", ctypes.c_size_t)]


class linear_desc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("act", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64)]


class linear_plan_info(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("grid", ctypes.c_int64), ("split_tiles", ctypes.c_int32),
                ("split_pieces", ctypes.c_int32), ("workspace_bytes", ctypes.c_size_t),
                ("backward_workspace_bytes", ctypes.c_size_t), ("kernel_name", ctypes.c_char * 64)]


class rope3d_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("n", "t", "h", "w", "heads_q", "heads_k", "head_dim", "dim_t", "dim_h", "dim_w", "pairing")] + \
               [("flags", ctypes.c_uint32), ("base", ctypes.c_double)] + \
               [(n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")]


class attention_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "heads_q", "heads_k", "head_dim", "tq", "tk", "frame", "window")] + \
               [("scale", ctypes.c_float), ("flags", ctypes.c_uint32)] + \
               [(n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "v_stride", "o_stride")]


class attention_plan_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tile_rows", "tile_keys", "threads", "splits")] + \
               [("grid", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t),
                ("backward_workspace_bytes", ctypes.c_size_t), ("kernel_name", ctypes.c_char * 64)]


class adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + \
               [("count", ctypes.c_int64), ("decay", ctypes.c_float)]


class adamw_hyper(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale")] + \
               [("step", ctypes.c_int64)]


ADAMW_DEVICE_HYPER = 9
ADAMW_BLOCK = 128


class Conv3dError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s (status %d): %s" % (_status_name(status), status, message))
        self.status = status


def _status_name(s):
    return {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "WORKSPACE", 4: "NO_DEVICE",
            5: "HIP"}.get(s, "UNKNOWN")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libconv3d.so (raises OSError if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError("libconv3d.so not built at %s: run python -m convolution_implicit_gemm_amd.build"
                      % path)
    lib = ctypes.CDLL(path)
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
    lib.conv3d_plan.argtypes = [ctypes.POINTER(conv3d_desc), ctypes.POINTER(vp), ctypes.POINTER(sz)]
    lib.conv3d_plan.restype = ctypes.c_int
    lib.conv3d_plan_query.argtypes = [vp, ctypes.POINTER(conv3d_plan_info)]
    lib.conv3d_plan_query.restype = ctypes.c_int
    lib.conv3d_plan_destroy.argtypes = [vp]
    lib.conv3d_plan_destroy.restype = None
    lib.conv3d_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.conv3d_forward_chunk.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.conv3d_forward_chunk.restype = ctypes.c_int
    lib.conv3d_forward.restype = ctypes.c_int
    lib.groupnorm_silu_workspace.argtypes = [i32, i64, i32, i32]
    lib.groupnorm_silu_workspace.restype = sz
    lib.groupnorm_silu.argtypes = [vp, vp, vp, vp, i32, i64, i32, i32, ctypes.c_float, i32, vp, sz, vp]
    lib.groupnorm_silu_bf16.argtypes = lib.groupnorm_silu.argtypes
    lib.groupnorm_silu_bf16.restype = ctypes.c_int
    lib.groupnorm_silu.restype = ctypes.c_int
    lib.groupnorm_silu_from_stats_workspace.argtypes = [i32, i32, i32]
    lib.groupnorm_silu_from_stats_workspace.restype = sz
    lib.groupnorm_silu_from_stats.argtypes = [vp, vp, vp, vp, i32, i64, i32, i32, ctypes.c_float, i32, vp, i32,
                                              vp, sz, vp]
    lib.groupnorm_silu_from_stats.restype = ctypes.c_int
    lib.groupnorm_silu_from_stats_bf16.argtypes = lib.groupnorm_silu_from_stats.argtypes
    lib.groupnorm_silu_from_stats_bf16.restype = ctypes.c_int
    lib.groupnorm_silu_noalloc_max_bytes.argtypes = []
    lib.groupnorm_silu_noalloc_max_bytes.restype = sz
    lib.groupnorm_silu_noalloc.argtypes = [vp, vp, vp, vp, i32, i64, i32, i32, ctypes.c_float, i32, vp]
    lib.groupnorm_silu_noalloc.restype = ctypes.c_int
    lib.conv3d_status_str.argtypes = [ctypes.c_int]
    lib.conv3d_status_str.restype = ctypes.c_char_p
    lib.conv3d_last_error.argtypes = []
    lib.conv3d_last_error.restype = ctypes.c_char_p
    lib.conv3d_version.argtypes = []
    lib.conv3d_version.restype = i32
    lib.conv3d_selftest.argtypes = []
    lib.conv3d_selftest.restype = i32
    f32 = ctypes.c_float
    for fn, args, res in (
            ("linear_plan", [ctypes.POINTER(linear_desc), ctypes.POINTER(vp), ctypes.POINTER(sz)], ctypes.c_int),
            ("linear_plan_query", [vp, ctypes.POINTER(linear_plan_info)], ctypes.c_int),
            ("linear_plan_destroy", [vp], None),
            ("linear_forward", [vp] * 8 + [sz, vp], ctypes.c_int),
            ("linear_backward_workspace", [vp], sz),
            ("linear_backward", [vp] * 9 + [sz, vp], ctypes.c_int),
            ("layernorm", [vp] * 5 + [i64, i32, i64, i64, f32, vp], ctypes.c_int),
            ("layernorm_bf16", [vp] * 5 + [i64, i32, i64, i64, f32, vp], ctypes.c_int),
            ("layernorm_backward_workspace", [i64, i32], sz),
            ("layernorm_backward", [vp] * 8 + [i64, i32, i64, i64, vp, sz, vp], ctypes.c_int),
            ("layernorm_backward_bf16", [vp] * 8 + [i64, i32, i64, i64, vp, sz, vp], ctypes.c_int),
            ("rope3d_plan", [ctypes.POINTER(rope3d_desc), ctypes.POINTER(vp)], ctypes.c_int),
            ("rope3d_plan_destroy", [vp], None),
            ("rope3d_forward", [vp] * 6 + [i32, vp], ctypes.c_int),
            ("rope3d_backward", [vp] * 6 + [i32, vp], ctypes.c_int),
            ("attention_plan", [ctypes.POINTER(attention_desc), ctypes.POINTER(vp), ctypes.POINTER(sz)], ctypes.c_int),
            ("attention_plan_query", [vp, ctypes.POINTER(attention_plan_info)], ctypes.c_int),
            ("attention_plan_destroy", [vp], None),
            ("attention_forward", [vp] * 7 + [i64, vp, sz, vp], ctypes.c_int),
            ("attention_backward_workspace", [vp], sz),
            ("attention_backward", [vp] * 11 + [i64, vp, sz, vp], ctypes.c_int),
            ("adamw_plan", [ctypes.POINTER(adamw_tensor), i32, ctypes.c_uint32, ctypes.POINTER(vp)], ctypes.c_int),
            ("adamw_plan_destroy", [vp], None),
            ("adamw_hyper_pack", [ctypes.POINTER(adamw_hyper), ctypes.POINTER(f32)], ctypes.c_int),
            ("adamw_step", [vp, ctypes.POINTER(adamw_hyper), vp, vp], ctypes.c_int)):
        getattr(lib, fn).argtypes = args
        getattr(lib, fn).restype = res
    dp = ctypes.POINTER(ctypes.c_double)
    lib.conv3d_calibrate_scratch_bytes.argtypes = []
    lib.conv3d_calibrate_scratch_bytes.restype = sz
    lib.conv3d_calibrate_mfma.argtypes = [vp, sz, dp, dp, vp]
    lib.conv3d_calibrate_mfma.restype = ctypes.c_int
    lib.conv3d_calibrate_hbm.argtypes = [vp, vp, sz, dp, dp, vp]
    lib.conv3d_calibrate_hbm.restype = ctypes.c_int
    lib.conv3d_clock_stamp_bytes.argtypes = []
    lib.conv3d_clock_stamp_bytes.restype = sz
    lib.conv3d_clock_stamp.argtypes = [vp, sz, vp]
    lib.conv3d_clock_stamp.restype = ctypes.c_int
    _lib = lib
    return lib


def _check(status):
    if status != CONV3D_OK:
        raise Conv3dError(status, load_library().conv3d_last_error().decode())


def _addr(t, what="tensor", elems=None, dtype=None):
    """Device address of a torch tensor (or an int address, passed as is).

    A tensor must be contiguous and on a GPU; with ``elems`` / ``dtype`` it
    must also hold at least that many elements of that dtype (the C layer
    sees only the address and cannot check any of this).  Raises Conv3dError
    (INVALID_ARG) otherwise, before anything is enqueued.
    """
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, "%s is not contiguous (pass .contiguous())" % what)
    if not t.is_cuda:
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, "%s is on %s, not on a GPU" % (what, t.device))
    if dtype is not None and t.dtype != dtype:
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, "%s is %s, the plan expects %s" % (what, t.dtype, dtype))
    if elems is not None and t.numel() < elems:
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, "%s holds %d elements, %d needed" % (what, t.numel(), elems))
    return t.data_ptr()


# What calls need of torch, bound at the first one that needs it (importing this
# module does not import torch).  The name that callers test is assigned last:
# another thread that finds it set finds the others set too.
_F16 = _BF16 = _F32 = _I32 = _raw_stream = _current_device = None


def _bind_torch():
    global _F16, _BF16, _F32, _I32
    import torch
    _BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
    _F16 = torch.float16


def _bind_streams():
    # the raw handle of the current stream, without building a Stream object
    # (2.8 us of a small call's host time)
    global _raw_stream, _current_device
    import torch
    torch.cuda.current_device()  # initialises the device
    _current_device = torch._C._cuda_getDevice
    _raw_stream = torch._C._cuda_getCurrentRawStream


def _elem_dtype(bf16):
    if _F16 is None:
        _bind_torch()
    return _BF16 if bf16 else _F16


def _conv_sizes(desc, chunk_t=None):
    """(x, x_prev, weight, bias, y) element counts of a plan's descriptor."""
    d = desc
    to = d.t if chunk_t else d.t + d.pad_t_front + d.pad_t_back - d.kt + 1
    ho = d.h + 2 * d.pad_h - d.kh + 1
    wo = d.w + 2 * d.pad_w - d.kw + 1
    return (d.n * d.t * d.h * d.w * d.c_in, d.n * max(d.kt - 1, 0) * d.h * d.w * d.c_in,
            d.c_out * d.kt * d.kh * d.kw * d.c_in, d.c_out, d.n * to * ho * wo * d.c_out)


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            _bind_streams()
        return _raw_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Plan:
    """Owns a conv3d_plan_t; destroyed with the object."""

    def __init__(self, handle, workspace_bytes, desc):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.desc = desc

    def info(self) -> conv3d_plan_info:
        return conv3d_plan_query(self)

    def __del__(self):
        if self.handle and _lib is not None:
            _lib.conv3d_plan_destroy(self.handle)
            self.handle = None


def weight_from_ncdhw(weight):
    """A torch Conv3d weight [Cout][Cin][kt][kh][kw] in this library's layout
    [Cout][kt][kh][kw][Cin] (a contiguous copy).  A load-time conversion, done
    once per weight, off the forward path."""
    return weight.permute(0, 2, 3, 4, 1).contiguous()


def make_desc(n, t, h, w, c_in, c_out, kt=3, kh=3, kw=3, pad_t_front=1, pad_t_back=1, pad_h=1,
              pad_w=1, t_pad_mode=CONV3D_TPAD_ZERO, flags=0) -> conv3d_desc:
    return conv3d_desc(n, t, h, w, c_in, c_out, kt, kh, kw, pad_t_front, pad_t_back, pad_h, pad_w,
                       t_pad_mode, flags)


def conv3d_plan(desc: conv3d_desc) -> Plan:
    lib = load_library()
    h = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(lib.conv3d_plan(ctypes.byref(desc), ctypes.byref(h), ctypes.byref(ws)))
    return Plan(h.value, ws.value, desc)


def conv3d_plan_query(plan: Plan) -> conv3d_plan_info:
    info = conv3d_plan_info()
    _check(load_library().conv3d_plan_query(plan.handle, ctypes.byref(info)))
    return info


def conv3d_plan_destroy(plan: Plan) -> None:
    if plan.handle:
        load_library().conv3d_plan_destroy(plan.handle)
        plan.handle = None


def conv3d_forward(plan: Plan, x, weight, bias, residual, y, workspace=None, workspace_bytes=None,
                   stream=None) -> None:
    """Enqueue y = conv3d(x, weight) (+bias) (+residual) on ``stream``."""
    if workspace_bytes is None:
        if workspace is None:
            workspace_bytes = 0
        elif isinstance(workspace, int):
            workspace_bytes = plan.workspace_bytes
        else:
            workspace_bytes = workspace.numel() * workspace.element_size()
    nx, _, nw, nb, ny = _conv_sizes(plan.desc)
    dt = _elem_dtype(plan.desc.flags & CONV3D_F_BF16)
    _check(load_library().conv3d_forward(plan.handle, _addr(x, "x", nx, dt), _addr(weight, "weight", nw, dt),
                                         _addr(bias, "bias", nb, dt), _addr(residual, "residual", ny, dt),
                                         _addr(y, "y", ny, dt), _addr(workspace, "workspace"),
                                         workspace_bytes, _stream(stream)))


def conv3d_forward_chunk(plan: Plan, x_prev, x, weight, bias, residual, y, workspace,
                         workspace_bytes=None, stream=None) -> None:
    """Enqueue one chunk of a chunked causal decode (plan made with CONV3D_F_CHUNK)."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    nx, nxp, nw, nb, ny = _conv_sizes(plan.desc, chunk_t=True)
    dt = _elem_dtype(plan.desc.flags & CONV3D_F_BF16)
    _check(load_library().conv3d_forward_chunk(plan.handle, _addr(x_prev, "x_prev", nxp, dt), _addr(x, "x", nx, dt),
                                               _addr(weight, "weight", nw, dt), _addr(bias, "bias", nb, dt),
                                               _addr(residual, "residual", ny, dt), _addr(y, "y", ny, dt),
                                               _addr(workspace, "workspace"),
                                               workspace_bytes, _stream(stream)))


def groupnorm_silu_workspace(n, thw, c, groups) -> int:
    return load_library().groupnorm_silu_workspace(n, thw, c, groups)


def groupnorm_silu(x, gamma, beta, y, n, thw, c, groups, eps, apply_silu, workspace,
                   workspace_bytes=None, stream=None, bf16=False) -> None:
    """Enqueue y = [SiLU](GroupNorm(x)) on ``stream``."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    lib = load_library()
    fn = lib.groupnorm_silu_bf16 if bf16 else lib.groupnorm_silu
    dt, ne = _elem_dtype(bf16), n * thw * c
    _check(fn(_addr(x, "x", ne, dt), _addr(gamma, "gamma", c, dt), _addr(beta, "beta", c, dt), _addr(y, "y", ne, dt),
              n, thw, c, groups, float(eps), 1 if apply_silu else 0, _addr(workspace, "workspace"),
              workspace_bytes, _stream(stream)))


def groupnorm_silu_from_stats_workspace(n, c, groups) -> int:
    return load_library().groupnorm_silu_from_stats_workspace(n, c, groups)


def gn_stats_view(plan: Plan, workspace):
    """(address, slots) of the GroupNorm partials a CONV3D_F_GN_STATS plan's
    forward leaves in ``workspace`` (a device tensor of the planned size)."""
    info = conv3d_plan_query(plan)
    if not info.gn_stats_slots:
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, "the plan was made without CONV3D_F_GN_STATS")
    if workspace.numel() * workspace.element_size() < plan.workspace_bytes:
        raise Conv3dError(CONV3D_ERR_WORKSPACE, "workspace smaller than the plan's")
    return workspace.data_ptr() + info.gn_stats_offset, info.gn_stats_slots


def groupnorm_silu_from_stats(x, gamma, beta, y, n, thw, c, groups, eps, apply_silu, stats, stats_slots,
                              workspace, workspace_bytes=None, stream=None, bf16=False) -> None:
    """Enqueue y = [SiLU](GroupNorm(x)) with x's statistics merged from the partials
    ``stats`` (an address, see gn_stats_view) that the conv producing x wrote."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    lib = load_library()
    fn = lib.groupnorm_silu_from_stats_bf16 if bf16 else lib.groupnorm_silu_from_stats
    dt, ne = _elem_dtype(bf16), n * thw * c
    _check(fn(_addr(x, "x", ne, dt), _addr(gamma, "gamma", c, dt), _addr(beta, "beta", c, dt), _addr(y, "y", ne, dt),
              n, thw, c, groups, float(eps), 1 if apply_silu else 0, _addr(stats, "stats"), int(stats_slots),
              _addr(workspace, "workspace"), workspace_bytes, _stream(stream)))


def groupnorm_silu_noalloc_max_bytes() -> int:
    return load_library().groupnorm_silu_noalloc_max_bytes()


def groupnorm_silu_noalloc(x, gamma, beta, y, n, thw, c, groups, eps, apply_silu, stream=None) -> None:
    """groupnorm_silu (fp16) with the library's static device scratch instead of a workspace."""
    dt, ne = _elem_dtype(False), n * thw * c
    _check(load_library().groupnorm_silu_noalloc(_addr(x, "x", ne, dt), _addr(gamma, "gamma", c, dt),
                                                 _addr(beta, "beta", c, dt), _addr(y, "y", ne, dt), n, thw, c,
                                                 groups, float(eps), 1 if apply_silu else 0, _stream(stream)))


# ---- the token operators

def _strided_addr(t, what, sizes, strides, dtype):
    """Device address of a tensor that holds the elements at the given sizes and
    strides (in elements, outermost first) from its first one: a view laid out so
    and at least as large, or a contiguous tensor of any shape with as many
    elements.  What its storage holds behind it does not count."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, "%s is on %s, not on a GPU" % (what, t.device))
    if t.dtype != dtype:
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, "%s is %s, %s expected" % (what, t.dtype, dtype))
    have, shape = t.stride(), t.shape
    if have == strides and shape == sizes:
        return t.data_ptr() or None  # a view laid out as the call reads it
    if 0 in sizes:
        return t.data_ptr() or None
    if len(have) >= 2 and len(have) == len(sizes):
        # a size of one may have any stride
        for n, st, want in zip(shape, have, strides):
            if n > 1 and st != want:
                raise Conv3dError(CONV3D_ERR_INVALID_ARG, "%s has strides %s, the call reads %s"
                                  % (what, tuple(have), tuple(strides)))
        if all(n >= size for n, size in zip(shape, sizes)):
            return t.data_ptr()
    if not t.is_contiguous():
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, "%s is %s and not contiguous, the call reads %s"
                          % (what, tuple(shape), tuple(sizes)))
    last = sum((n - 1) * st for n, st in zip(sizes, strides))
    if last >= t.numel():
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, "%s holds %d elements, %d needed" % (what, t.numel(), last + 1))
    return t.data_ptr()


def _rows_addr(t, what, rows, cols, stride, dtype):
    return None if t is None else _strided_addr(t, what, (rows, cols), (stride or cols, 1), dtype)


def _workspace_bytes(workspace, workspace_bytes, planned=0):
    if workspace_bytes is not None:
        return workspace_bytes
    if workspace is None:
        return 0
    return planned if isinstance(workspace, int) else workspace.numel() * workspace.element_size()


class LinearPlan:
    """Owns a linear_plan_t; destroyed with the object."""

    def __init__(self, handle, workspace_bytes, desc):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.desc = desc
        d = desc
        self.sizes = (d.m, d.n, d.k, d.x_stride, d.y_stride, d.residual_stride, _elem_dtype(d.flags & CONV3D_F_BF16))

    def info(self) -> linear_plan_info:
        return linear_plan_query(self)

    def __del__(self):
        if self.handle and _lib is not None:
            _lib.linear_plan_destroy(self.handle)
            self.handle = None


def make_linear_desc(m, n, k, act=CONV3D_ACT_NONE, flags=0, x_stride=0, y_stride=0, residual_stride=0) -> linear_desc:
    return linear_desc(m, n, k, act, flags, x_stride, y_stride, residual_stride)


def linear_plan(desc: linear_desc) -> LinearPlan:
    lib = load_library()
    h = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(lib.linear_plan(ctypes.byref(desc), ctypes.byref(h), ctypes.byref(ws)))
    return LinearPlan(h.value, ws.value, desc)


def linear_plan_query(plan: LinearPlan) -> linear_plan_info:
    info = linear_plan_info()
    _check(load_library().linear_plan_query(plan.handle, ctypes.byref(info)))
    return info


def linear_plan_destroy(plan: LinearPlan) -> None:
    if plan.handle:
        load_library().linear_plan_destroy(plan.handle)
        plan.handle = None


def linear_forward(plan: LinearPlan, x, w, bias, residual, y, preact=None, workspace=None, workspace_bytes=None,
                   stream=None) -> None:
    """Enqueue y = act(x w^T + bias) + residual (and preact, the value before act) on ``stream``."""
    m, n, k, xs, ys, rs, dt = plan.sizes
    _check((_lib or load_library()).linear_forward(
        plan.handle, _rows_addr(x, "x", m, k, xs, dt), _addr(w, "w", n * k, dt), _addr(bias, "bias", n, dt),
        _rows_addr(residual, "residual", m, n, rs, dt), _rows_addr(y, "y", m, n, ys, dt),
        _rows_addr(preact, "preact", m, n, 0, dt), _addr(workspace, "workspace"),
        _workspace_bytes(workspace, workspace_bytes, plan.workspace_bytes), _stream(stream)))


def linear_backward_workspace(plan: LinearPlan) -> int:
    return load_library().linear_backward_workspace(plan.handle)


def linear_backward(plan: LinearPlan, dy, x, w, preact, dx, dw, dbias, workspace, workspace_bytes=None,
                    stream=None) -> None:
    """Enqueue the gradients dx, dw and dbias (each may be None) of one product on ``stream``."""
    m, n, k, xs, ys, _, dt = plan.sizes
    if workspace_bytes is None and isinstance(workspace, int):
        workspace_bytes = linear_backward_workspace(plan)
    _check((_lib or load_library()).linear_backward(
        plan.handle, _rows_addr(dy, "dy", m, n, ys, dt), _rows_addr(x, "x", m, k, xs, dt), _addr(w, "w", n * k, dt),
        _rows_addr(preact, "preact", m, n, 0, dt), _rows_addr(dx, "dx", m, k, xs, dt), _addr(dw, "dw", n * k, dt),
        _addr(dbias, "dbias", n, dt), _addr(workspace, "workspace"), _workspace_bytes(workspace, workspace_bytes),
        _stream(stream)))


def layernorm(x, gamma, beta, y, stats, rows, c, eps, x_stride=0, y_stride=0, stream=None, bf16=False) -> None:
    """Enqueue y = LayerNorm(x) over the c channels of each row on ``stream``;
    gamma, beta and stats (fp32 [rows][2]: mean, 1 / sqrt(var + eps)) may be None."""
    lib, dt = _lib or load_library(), _elem_dtype(bf16)
    fn = lib.layernorm_bf16 if bf16 else lib.layernorm
    _check(fn(_rows_addr(x, "x", rows, c, x_stride, dt), _addr(gamma, "gamma", c, dt), _addr(beta, "beta", c, dt),
              _rows_addr(y, "y", rows, c, y_stride, dt), _addr(stats, "stats", 2 * rows, _F32), rows, c,
              x_stride, y_stride, float(eps), _stream(stream)))


def layernorm_bf16(x, gamma, beta, y, stats, rows, c, eps, x_stride=0, y_stride=0, stream=None) -> None:
    """layernorm with bf16 x, gamma, beta and y."""
    layernorm(x, gamma, beta, y, stats, rows, c, eps, x_stride, y_stride, stream, bf16=True)


def layernorm_backward_workspace(rows, c) -> int:
    return load_library().layernorm_backward_workspace(rows, c)


def layernorm_backward(dy, x, gamma, stats, dres, dx, dgamma, dbeta, rows, c, workspace, x_stride=0, y_stride=0,
                       workspace_bytes=None, stream=None, bf16=False) -> None:
    """Enqueue dx (+ dres), dgamma and dbeta of layernorm on ``stream``; gamma,
    dres, dgamma and dbeta may be None."""
    lib, dt = _lib or load_library(), _elem_dtype(bf16)
    if workspace_bytes is None and isinstance(workspace, int):
        workspace_bytes = layernorm_backward_workspace(rows, c)
    fn = lib.layernorm_backward_bf16 if bf16 else lib.layernorm_backward
    _check(fn(_rows_addr(dy, "dy", rows, c, y_stride, dt), _rows_addr(x, "x", rows, c, x_stride, dt),
              _addr(gamma, "gamma", c, dt), _addr(stats, "stats", 2 * rows, _F32),
              _rows_addr(dres, "dres", rows, c, x_stride, dt), _rows_addr(dx, "dx", rows, c, x_stride, dt),
              _addr(dgamma, "dgamma", c, dt), _addr(dbeta, "dbeta", c, dt), rows, c, x_stride, y_stride,
              _addr(workspace, "workspace"), _workspace_bytes(workspace, workspace_bytes), _stream(stream)))


def layernorm_backward_bf16(dy, x, gamma, stats, dres, dx, dgamma, dbeta, rows, c, workspace, x_stride=0, y_stride=0,
                            workspace_bytes=None, stream=None) -> None:
    """layernorm_backward with bf16 tensors (stats and workspace fp32 as before)."""
    layernorm_backward(dy, x, gamma, stats, dres, dx, dgamma, dbeta, rows, c, workspace, x_stride, y_stride,
                       workspace_bytes, stream, bf16=True)


class RopePlan:
    """Owns a rope3d_plan_t; destroyed with the object."""

    def __init__(self, handle, desc):
        self.handle = handle
        self.desc = desc
        d = desc
        tokens = d.t * d.h * d.w

        def layout(heads, stride):
            stride = tuple(stride)
            if not any(stride):
                stride = (tokens * heads * d.head_dim, heads * d.head_dim, d.head_dim)
            return (d.n, tokens, heads, d.head_dim), stride + (1,)

        # (sizes, strides) of q, k, q_out and k_out
        self.layouts = (layout(d.heads_q, d.q_stride), layout(d.heads_k, d.k_stride),
                        layout(d.heads_q, d.q_out_stride), layout(d.heads_k, d.k_out_stride))
        self.positions = d.n * tokens * 3 if d.flags & CONV3D_F_POSITIONS else 0
        self.dtype = _elem_dtype(d.flags & CONV3D_F_BF16)

    def __del__(self):
        if self.handle and _lib is not None:
            _lib.rope3d_plan_destroy(self.handle)
            self.handle = None


def make_rope3d_desc(n, t, h, w, heads_q, heads_k, head_dim, dims, base=10000.0, pairing=ROPE3D_PAIR_ADJACENT,
                     flags=0, q_stride=(0, 0, 0), k_stride=(0, 0, 0), q_out_stride=(0, 0, 0),
                     k_out_stride=(0, 0, 0)) -> rope3d_desc:
    """dims: the elements of a head that turn with time, height and width;
    strides: elements between samples, tokens and heads (all 0: contiguous)."""
    arr = ctypes.c_int64 * 3
    return rope3d_desc(n, t, h, w, heads_q, heads_k, head_dim, *dims, pairing, flags, base, arr(*q_stride),
                       arr(*k_stride), arr(*q_out_stride), arr(*k_out_stride))


def rope3d_plan(desc: rope3d_desc) -> RopePlan:
    h = ctypes.c_void_p()
    _check(load_library().rope3d_plan(ctypes.byref(desc), ctypes.byref(h)))
    return RopePlan(h.value, desc)


def rope3d_plan_destroy(plan: RopePlan) -> None:
    if plan.handle:
        load_library().rope3d_plan_destroy(plan.handle)
        plan.handle = None


def _rope_call(fn, plan, q, k, q_out, k_out, positions, t_offset, stream, layouts):
    lq, lk, lqo, lko = layouts
    dt = plan.dtype
    if lk[0][2] == 0:
        k = k_out = None
    given = positions if plan.positions else None
    _check(fn(plan.handle, _strided_addr(q, "q", *lq, dt), _strided_addr(k, "k", *lk, dt),
              _strided_addr(q_out, "q_out", *lqo, dt), _strided_addr(k_out, "k_out", *lko, dt),
              _addr(given, "positions", plan.positions, _I32), t_offset, _stream(stream)))


def rope3d_forward(plan: RopePlan, q, k, q_out, k_out, positions=None, t_offset=0, stream=None) -> None:
    """Enqueue the rotation of q into q_out and k into k_out on ``stream``."""
    _rope_call((_lib or load_library()).rope3d_forward, plan, q, k, q_out, k_out, positions, t_offset, stream, plan.layouts)


def rope3d_backward(plan: RopePlan, dq_out, dk_out, dq, dk, positions=None, t_offset=0, stream=None) -> None:
    """Enqueue the gradient of rope3d_forward (strides: those of the outputs, then of the inputs)."""
    lq, lk, lqo, lko = plan.layouts
    _rope_call((_lib or load_library()).rope3d_backward, plan, dq_out, dk_out, dq, dk, positions, t_offset, stream,
               (lqo, lko, lq, lk))


class AttentionPlan:
    """Owns an attention_plan_t; destroyed with the object."""

    def __init__(self, handle, workspace_bytes, desc):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.desc = desc
        d = desc

        def layout(tokens, heads, stride):
            stride = tuple(stride)
            if not any(stride):
                stride = (tokens * heads * d.head_dim, heads * d.head_dim, d.head_dim)
            return (d.n, tokens, heads, d.head_dim), stride + (1,)

        # (sizes, strides) of q, k, v and o
        self.layouts = (layout(d.tq, d.heads_q, d.q_stride), layout(d.tk, d.heads_k, d.k_stride),
                        layout(d.tk, d.heads_k, d.v_stride), layout(d.tq, d.heads_q, d.o_stride))
        self.lse = d.n * d.heads_q * d.tq
        self.lengths = 2 * d.n if d.flags & CONV3D_F_LENGTHS else 0
        self.dtype = _elem_dtype(d.flags & CONV3D_F_BF16)

    def info(self) -> attention_plan_info:
        return attention_plan_query(self)

    def __del__(self):
        if self.handle and _lib is not None:
            _lib.attention_plan_destroy(self.handle)
            self.handle = None


def make_attention_desc(n, tq, tk, heads_q, heads_k, head_dim, frame=0, window=0, scale=0.0, flags=0,
                        q_stride=(0, 0, 0), k_stride=(0, 0, 0), v_stride=(0, 0, 0),
                        o_stride=(0, 0, 0)) -> attention_desc:
    """frame: tokens of a frame (0: every query sees every key); window: the frames that a query sees, its
    own and those before it (0: all); scale 0: 1 / sqrt(head_dim); strides: elements between samples,
    tokens and heads (all 0: contiguous)."""
    arr = ctypes.c_int64 * 3
    return attention_desc(n, heads_q, heads_k, head_dim, tq, tk, frame, window, scale, flags, arr(*q_stride),
                          arr(*k_stride), arr(*v_stride), arr(*o_stride))


def attention_plan(desc: attention_desc) -> AttentionPlan:
    lib = load_library()
    h = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(lib.attention_plan(ctypes.byref(desc), ctypes.byref(h), ctypes.byref(ws)))
    return AttentionPlan(h.value, ws.value, desc)


def attention_plan_query(plan: AttentionPlan) -> attention_plan_info:
    info = attention_plan_info()
    _check(load_library().attention_plan_query(plan.handle, ctypes.byref(info)))
    return info


def attention_plan_destroy(plan: AttentionPlan) -> None:
    if plan.handle:
        load_library().attention_plan_destroy(plan.handle)
        plan.handle = None


def attention_forward(plan: AttentionPlan, q, k, v, o, lse=None, lengths=None, q_offset=0, workspace=None,
                      workspace_bytes=None, stream=None) -> None:
    """Enqueue o = softmax(scale q k^T) v over the keys that each query sees (and lse, the logarithm of its
    exponentials' sum, fp32 [n, heads_q, tq]) on ``stream``; lengths: int32 [n, 2] (queries, keys)."""
    lq, lk, lv, lo = plan.layouts
    dt = plan.dtype
    given = lengths if plan.lengths else None
    _check((_lib or load_library()).attention_forward(
        plan.handle, _strided_addr(q, "q", *lq, dt), _strided_addr(k, "k", *lk, dt), _strided_addr(v, "v", *lv, dt),
        _strided_addr(o, "o", *lo, dt), _addr(lse, "lse", plan.lse, _F32), _addr(given, "lengths", plan.lengths, _I32),
        q_offset, _addr(workspace, "workspace"), _workspace_bytes(workspace, workspace_bytes, plan.workspace_bytes),
        _stream(stream)))


def attention_backward_workspace(plan: AttentionPlan) -> int:
    return load_library().attention_backward_workspace(plan.handle)


def attention_backward(plan: AttentionPlan, dout, q, k, v, o, lse, dq, dk, dv, lengths=None, q_offset=0,
                       workspace=None, workspace_bytes=None, stream=None) -> None:
    """Enqueue the gradients dq, dk and dv (each may be None) of attention_forward on ``stream``."""
    lq, lk, lv, lo = plan.layouts
    dt = plan.dtype
    given = lengths if plan.lengths else None
    if workspace_bytes is None and isinstance(workspace, int):
        workspace_bytes = attention_backward_workspace(plan)
    _check((_lib or load_library()).attention_backward(
        plan.handle, _strided_addr(dout, "dout", *lo, dt), _strided_addr(q, "q", *lq, dt),
        _strided_addr(k, "k", *lk, dt), _strided_addr(v, "v", *lv, dt), _strided_addr(o, "o", *lo, dt),
        _addr(lse, "lse", plan.lse, _F32), _strided_addr(dq, "dq", *lq, dt), _strided_addr(dk, "dk", *lk, dt),
        _strided_addr(dv, "dv", *lv, dt), _addr(given, "lengths", plan.lengths, _I32), q_offset,
        _addr(workspace, "workspace"), _workspace_bytes(workspace, workspace_bytes), _stream(stream)))


class AdamwList:
    """The tensors of an AdamW step: owns an adamw_plan_t and keeps the tensors alive."""

    def __init__(self, handle, tensors):
        self.handle = handle
        self.tensors = tensors

    def __del__(self):
        if self.handle and _lib is not None:
            _lib.adamw_plan_destroy(self.handle)
            self.handle = None


def adamw_list(params, grads, m, v, master=None, m_scale=None, v_scale=None, decay=None) -> AdamwList:
    """The tensors that adamw_step updates, as lists of equal length.

    params: fp16 or bf16 weights, or None; master: fp32 weights, or None (their entries
    too may be None, one of the two is needed for every tensor); grads: of params' type (with
    params None, any of fp16 and bf16) or fp32; m and v: fp32, or float8_e4m3fn / uint8 with m_scale and
    v_scale, uint8 with one scale for each 128 elements; decay: a factor of the weight
    decay for each tensor (1).  The tensors have to stay where they are as long as the list is used."""
    _elem_dtype(False)
    import torch
    grads = list(grads)
    count = len(grads)
    none = [None] * count

    def bad(message):
        raise Conv3dError(CONV3D_ERR_INVALID_ARG, message)

    lists = [none if x is None else list(x) for x in (params, master, grads, m, v, m_scale, v_scale)]
    decay = [1.0] * count if decay is None else list(decay)
    if any(len(x) != count for x in lists + [decay]):
        bad("the lists have different lengths")
    kinds = {t.dtype for t in lists[0] if t is not None}
    if len(kinds) > 1 or not kinds <= {_F16, _BF16}:
        bad("params are %s, all fp16 or all bf16 expected" % sorted(map(str, kinds)))
    for i, t in enumerate(lists[2]):
        if t is None:
            bad("grads[%d] is missing" % i)
    grad_kinds = {t.dtype for t in lists[2]}
    if len(grad_kinds) > 1:
        bad("grads are of different types")
    grad32 = grad_kinds == {_F32}
    half = kinds or (grad_kinds - {_F32}) or {_F16}
    half, = half
    byte = torch.uint8
    state8 = m_scale is not None or v_scale is not None
    state = ({byte, getattr(torch, "float8_e4m3fn", byte)} if state8 else {_F32})
    wanted = ({half}, {_F32}, {_F32} if grad32 else {half}, state, state, {byte}, {byte})
    names = ("params", "master", "grads", "m", "v", "m_scale", "v_scale")
    array = (adamw_tensor * max(count, 1))()
    device = None
    for i in range(count):
        g = lists[2][i]
        n = g.numel()
        for name, kind, tensors, field in zip(names, wanted, lists, ("param", "master", "grad", "m", "v", "m_scale",
                                                                     "v_scale")):
            t = tensors[i]
            if t is None:
                if name in ("m", "v") or (state8 and name.endswith("scale")):
                    bad("%s[%d] is missing" % (name, i))
                continue
            what = "%s[%d]" % (name, i)
            if t.dtype not in kind:
                bad("%s is %s, %s expected" % (what, t.dtype, " or ".join(sorted(map(str, kind)))))
            need = -(-n // ADAMW_BLOCK) if name.endswith("scale") else n
            if t.numel() != need:
                bad("%s holds %d elements, %d expected" % (what, t.numel(), need))
            address = _addr(t, what)
            device = t.device if device is None else device
            if t.device != device:
                bad("%s is on %s, others on %s" % (what, t.device, device))
            setattr(array[i], field, address or None)
        array[i].count = n
        array[i].decay = float(decay[i])
    flags = (CONV3D_F_BF16 if half == _BF16 else 0) | (CONV3D_F_STATE8 if state8 else 0) | \
        (CONV3D_F_GRAD32 if grad32 else 0)
    h = ctypes.c_void_p()
    _check(load_library().adamw_plan(array, count, flags, ctypes.byref(h)))
    return AdamwList(h.value, lists)


def make_adamw_hyper(lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, grad_scale=1.0) -> adamw_hyper:
    return adamw_hyper(lr, beta1, beta2, eps, weight_decay, grad_scale, step)


def adamw_hyper_pack(hyper: adamw_hyper):
    """The floats that a device tensor of hyperparameters holds, as a list."""
    out = (ctypes.c_float * ADAMW_DEVICE_HYPER)()
    _check(load_library().adamw_hyper_pack(ctypes.byref(hyper), out))
    return list(out)


def adamw_step(tensors: AdamwList, hyper, stream=None) -> None:
    """Enqueue one AdamW step over ``tensors`` on ``stream``.  hyper: an adamw_hyper, or a
    device fp32 tensor that holds adamw_hyper_pack's numbers when the step runs."""
    lib = _lib or load_library()
    if isinstance(hyper, adamw_hyper):
        _check(lib.adamw_step(tensors.handle, ctypes.byref(hyper), None, _stream(stream)))
    else:
        _elem_dtype(False)
        _check(lib.adamw_step(tensors.handle, None, _addr(hyper, "hyper", ADAMW_DEVICE_HYPER, _F32), _stream(stream)))


def conv3d_calibrate_scratch_bytes() -> int:
    return load_library().conv3d_calibrate_scratch_bytes()


def conv3d_calibrate_mfma(scratch, scratch_bytes=None, stream=None):
    """(TFLOP/s, shader MHz) of dense fp16 MFMA chains on random operands; synchronises."""
    if scratch_bytes is None:
        scratch_bytes = scratch.numel() * scratch.element_size()
    tf, mhz = ctypes.c_double(), ctypes.c_double()
    _check(load_library().conv3d_calibrate_mfma(_addr(scratch), scratch_bytes, ctypes.byref(tf),
                                                ctypes.byref(mhz), _stream(stream)))
    return tf.value, mhz.value


def conv3d_calibrate_hbm(src, dst, nbytes, stream=None):
    """(read GB/s, copy GB/s, read + write counted) of 16-byte streams; synchronises."""
    rd, cp = ctypes.c_double(), ctypes.c_double()
    _check(load_library().conv3d_calibrate_hbm(_addr(src), _addr(dst), nbytes, ctypes.byref(rd),
                                               ctypes.byref(cp), _stream(stream)))
    return rd.value, cp.value


def conv3d_clock_stamp_bytes() -> int:
    return load_library().conv3d_clock_stamp_bytes()


def conv3d_clock_stamp(out, out_bytes=None, stream=None) -> None:
    """Enqueue a shader-clock stamp into device buffer ``out`` (see conv3d.h)."""
    if out_bytes is None:
        out_bytes = out.numel() * out.element_size()
    _check(load_library().conv3d_clock_stamp(_addr(out), out_bytes, _stream(stream)))


def sclk_between(before, after):
    """Mean shader clock (MHz) per XCD between two stamps (host uint64 arrays
    of conv3d_clock_stamp's layout): {xcd: MHz}.  Stamps are paired by the CU
    they ran on, since the counters of different CUs are not aligned; an XCD's
    figure is the median over its CUs stamped both times."""
    import numpy as np
    b = np.asarray(before, dtype=np.uint64).reshape(-1, 3)
    a = np.asarray(after, dtype=np.uint64).reshape(-1, 3)
    per_xcd = {}
    for loc in sorted(set(b[:, 2].tolist()) & set(a[:, 2].tolist())):
        bb, aa = b[b[:, 2] == loc], a[a[:, 2] == loc]
        dc = aa[:, 0].astype(np.float64).mean() - bb[:, 0].astype(np.float64).mean()
        dr = aa[:, 1].astype(np.float64).mean() - bb[:, 1].astype(np.float64).mean()
        if dr > 0:
            per_xcd.setdefault(int(loc) & 0xF, []).append(100.0 * dc / dr)
    return {x: float(np.median(v)) for x, v in sorted(per_xcd.items())}


def groupnorm_silu_bf16(x, gamma, beta, y, n, thw, c, groups, eps, apply_silu, workspace,
                        workspace_bytes=None, stream=None) -> None:
    """groupnorm_silu with bf16 x, gamma, beta and y."""
    groupnorm_silu(x, gamma, beta, y, n, thw, c, groups, eps, apply_silu, workspace, workspace_bytes,
                   stream, bf16=True)


def conv3d_status_str(status: int) -> str:
    return load_library().conv3d_status_str(status).decode()


def conv3d_last_error() -> str:
    return load_library().conv3d_last_error().decode()


def conv3d_version() -> int:
    return load_library().conv3d_version()


def conv3d_selftest() -> int:
    """Run the library's start-up self-test on the current device (0 = pass)."""
    return load_library().conv3d_selftest()


def selftest_in_subprocess(timeout: float = 300.0) -> int:
    """conv3d_selftest() in a child process, so that a broken driver or device
    cannot take this process down.  Returns the child's exit status: 0 = pass,
    a conv3d_status or 16 + case number as conv3d_selftest documents,
    negative for a child killed by a signal."""
    import subprocess
    import sys
    code = ("import sys; sys.path.insert(0, %r); import convolution_implicit_gemm_amd as c; "
            "rc = c.conv3d_selftest(); sys.stderr.write(c.conv3d_last_error() + '\\n'); sys.exit(rc)"
            % os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    return subprocess.run([sys.executable, "-c", code], timeout=timeout).returncode
