"""Python binding of libconvmi.so, the gfx950 conv2d training-layer library.

Argument marshalling only: every function below passes device pointers (torch tensors'
``data_ptr()``), sizes and the current HIP stream straight to the C ABI declared in
include/convmi.h, whose entry points have the same names.  All computation happens in
the library's HIP kernels.  If the library is not built, importing this package raises
ImportError: there is no fallback path.

Tensors must be CUDA (HIP) tensors, contiguous, in the layouts of convmi.h: x/dx NHWC
[N,H,W,IC], w/dw OHWI [OC,KH,KW,IC], z/y/dy/dz NHWC [N,OH,OW,OC]; data tensors are
float32 or bfloat16 per ``desc.dtype``; bias, gamma, beta, running and saved statistics,
dw, db, dgamma, dbeta are float32.

Beside the convolution layer: ``rms_norm_*`` and ``layer_norm_*`` (norms with the residual's
addition), ``causal_conv_*`` and ``selective_scan_*`` (along sequences that lie one behind the
other in the rows), ``linear_*`` (matrix product with bias, activation and residual) and ``mx8_*`` /
``conv2d_backward_full_mx8`` (activations kept in 8 bits and read by the backward pass).
Their tensors may have any shape with the right number of elements, rows first; weights
turned round (a [K, N] matrix for w or dw [N, K]) are refused.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libconvmi.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_MISALIGNED, ERR_HIP = range(6)
F32, BF16 = 0, 1
ACT_IDENTITY, ACT_RELU, ACT_TANH, ACT_SIGMOID, ACT_GELU, ACT_SILU = 0, 1, 2, 3, 4, 5  # SILU: causal_conv_* only
NORM_NONE, NORM_BATCH, NORM_LAYER, NORM_GROUP = 0, 1, 2, 3
MODE_TRAIN, MODE_EVAL = 0, 1
OP_FORWARD, OP_BACKWARD_DATA, OP_BACKWARD_WEIGHT, OP_BN_STATS, OP_ACTIVATION_BACKWARD, OP_BACKWARD_FULL = range(6)
OP_BACKWARD_FULL_MX8 = 6
LINEAR_FORWARD, LINEAR_BACKWARD_DATA, LINEAR_BACKWARD_WEIGHT = range(3)
SCAN_FORWARD, SCAN_BACKWARD = range(2)
MX8_BLOCK = 32  # values of a row that share a scale byte

STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "WORKSPACE", 4: "MISALIGNED", 5: "HIP"}

# Every symbol include/convmi.h declares.
EXPORTS = ("convmi_output_dims", "convmi_workspace_size", "conv2d_forward", "conv2d_forward_noalloc",
           "conv2d_backward_data",
           "conv2d_backward_weight", "bn_stats_training", "activation_backward", "conv2d_backward_full",
           "convmi_plan_name", "convmi_last_error",
           "convmi_version",
           "mx8_pack", "mx8_unpack", "conv2d_backward_full_mx8",
           "rms_norm_workspace_size", "rms_norm_forward", "rms_norm_backward",
           "layer_norm_workspace_size", "layer_norm_forward", "layer_norm_backward",
           "selective_scan_workspace_size", "selective_scan_saved_size", "selective_scan_forward",
           "selective_scan_backward", "selective_scan_step",
           "causal_conv_workspace_size", "causal_conv_forward", "causal_conv_backward", "causal_conv_step",
           "linear_workspace_size", "linear_plan_name", "linear_forward", "linear_activation_backward",
           "linear_backward_data", "linear_backward_weight")


class ConvDesc(C.Structure):
    """Mirror of convmi_desc."""
    _fields_ = [("N", C.c_int64), ("H", C.c_int64), ("W", C.c_int64), ("IC", C.c_int64), ("OC", C.c_int64),
                ("KH", C.c_int64), ("KW", C.c_int64),
                ("stride_h", C.c_int32), ("stride_w", C.c_int32), ("pad_h", C.c_int32), ("pad_w", C.c_int32),
                ("activation", C.c_int32), ("normalization", C.c_int32), ("mode", C.c_int32),
                ("dtype", C.c_int32), ("momentum", C.c_float), ("eps", C.c_float), ("groups", C.c_int32)]


class RmsDesc(C.Structure):
    """Mirror of convmi_rms_desc."""
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("dtype", C.c_int32), ("eps", C.c_float)]


LayerNormDesc = RmsDesc  # convmi_layer_norm_desc is the same structure


class CausalConvDesc(C.Structure):
    """Mirror of convmi_causal_conv_desc."""
    _fields_ = [("rows", C.c_int64), ("channels", C.c_int64), ("batch", C.c_int64), ("taps", C.c_int32),
                ("activation", C.c_int32), ("dtype", C.c_int32), ("x_pitch", C.c_int64)]


class ScanDesc(C.Structure):
    """Mirror of convmi_scan_desc."""
    _fields_ = [("rows", C.c_int64), ("channels", C.c_int64), ("batch", C.c_int64), ("states", C.c_int32),
                ("groups", C.c_int32), ("dtype", C.c_int32), ("delta_softplus", C.c_int32), ("x_pitch", C.c_int64),
                ("dt_pitch", C.c_int64), ("z_pitch", C.c_int64), ("bc_pitch", C.c_int64)]


class LinearDesc(C.Structure):
    """Mirror of convmi_linear_desc."""
    _fields_ = [("M", C.c_int64), ("K", C.c_int64), ("N", C.c_int64), ("activation", C.c_int32),
                ("dtype", C.c_int32), ("x_mx8", C.c_int32), ("z_mx8", C.c_int32)]


class ConvmiError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"convmi status {status} ({STATUS_NAMES.get(status, '?')}): {message}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                          "(python convolution_layer_amd/build.py)")
    L = C.CDLL(LIB_PATH)
    vp, i32, sz = C.c_void_p, C.c_int32, C.c_size_t
    dp = C.POINTER(ConvDesc)
    L.convmi_last_error.restype = C.c_char_p
    L.convmi_version.restype = C.c_char_p
    L.convmi_output_dims.argtypes = [dp, C.POINTER(C.c_int64), C.POINTER(C.c_int64)]
    L.convmi_workspace_size.argtypes = [dp, i32, C.POINTER(sz)]
    L.conv2d_forward.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.conv2d_forward_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.conv2d_backward_data.argtypes = [dp, vp, vp, vp, vp, sz, vp]
    L.conv2d_backward_weight.argtypes = [dp, vp, vp, vp, vp, i32, vp, sz, vp]
    L.bn_stats_training.argtypes = [dp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.activation_backward.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    L.conv2d_backward_full.argtypes = [dp, vp, vp, vp, i32, vp, vp, vp, vp, i32, vp, sz, vp]
    L.convmi_plan_name.argtypes = [dp, i32, C.c_char_p, sz]
    rp, lp, i64 = C.POINTER(RmsDesc), C.POINTER(LinearDesc), C.c_int64
    L.mx8_pack.argtypes = [i64, i64, i32, vp, vp, vp, vp]
    L.mx8_unpack.argtypes = [i64, i64, i32, vp, vp, vp, vp]
    L.conv2d_backward_full_mx8.argtypes = [dp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, i32, vp, sz, vp]
    L.rms_norm_workspace_size.argtypes = [rp, C.POINTER(sz)]
    L.rms_norm_forward.argtypes = [rp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.rms_norm_backward.argtypes = [rp, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    L.layer_norm_workspace_size.argtypes = [rp, C.POINTER(sz)]
    L.layer_norm_forward.argtypes = [rp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.layer_norm_backward.argtypes = [rp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    cp = C.POINTER(CausalConvDesc)
    L.causal_conv_workspace_size.argtypes = [cp, C.POINTER(sz)]
    L.causal_conv_forward.argtypes = [cp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.causal_conv_backward.argtypes = [cp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    L.causal_conv_step.argtypes = [cp, vp, vp, vp, vp, i64, vp, vp, vp]
    np_ = C.POINTER(ScanDesc)
    L.selective_scan_workspace_size.argtypes = [np_, i32, C.POINTER(sz)]
    L.selective_scan_saved_size.argtypes = [np_, C.POINTER(sz)]
    L.selective_scan_forward.argtypes = [np_] + [vp] * 14 + [sz, vp]
    L.selective_scan_backward.argtypes = [np_] + [vp] * 21 + [i32, vp, sz, vp]
    L.selective_scan_step.argtypes = [np_] + [vp] * 9 + [i64, vp, vp, vp]
    L.linear_workspace_size.argtypes = [lp, i32, C.POINTER(sz)]
    L.linear_plan_name.argtypes = [lp, i32, C.c_char_p, sz]
    L.linear_forward.argtypes = [lp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.linear_activation_backward.argtypes = [lp, vp, vp, vp, vp, vp]
    L.linear_backward_data.argtypes = [lp, vp, vp, vp, vp, sz, vp]
    L.linear_backward_weight.argtypes = [lp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    for name in EXPORTS:
        if name not in ("convmi_last_error", "convmi_version"):
            getattr(L, name).restype = C.c_int
    return L


lib = _load()


def version() -> str:
    return lib.convmi_version().decode()


def make_desc(N, H, W, IC, OC, KH, KW, stride=(1, 1), pad=(0, 0), activation=ACT_IDENTITY,
              normalization=NORM_NONE, mode=MODE_TRAIN, dtype=F32, momentum=0.1, eps=1e-5, groups=1) -> ConvDesc:
    return ConvDesc(N, H, W, IC, OC, KH, KW, stride[0], stride[1], pad[0], pad[1], activation, normalization,
                    mode, dtype, momentum, eps, groups)


def stat_count(desc: ConvDesc) -> int:
    """Entries of save_mean / save_inv_std: OC (batch norm) or N * groups (layer, group)."""
    if desc.normalization == NORM_BATCH:
        return desc.OC
    return desc.N * (desc.groups if desc.normalization == NORM_GROUP else 1)


def _check(status: int):
    if status != OK:
        raise ConvmiError(status, lib.convmi_last_error().decode())


def output_dims(desc: ConvDesc):
    oh, ow = C.c_int64(), C.c_int64()
    _check(lib.convmi_output_dims(C.byref(desc), C.byref(oh), C.byref(ow)))
    return oh.value, ow.value


def workspace_size(desc: ConvDesc, op: int) -> int:
    n = C.c_size_t()
    _check(lib.convmi_workspace_size(C.byref(desc), op, C.byref(n)))
    return n.value


def plan_name(desc: ConvDesc, op: int) -> str:
    """Kernel plan of the forward or the input gradient for this descriptor (host only)."""
    buf = C.create_string_buffer(128)
    _check(lib.convmi_plan_name(C.byref(desc), op, buf, len(buf)))
    return buf.value.decode()


def _ptr(t):
    """Device pointer of a contiguous GPU tensor, or None."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("convmi needs device (HIP) tensors")
    if not t.is_contiguous():
        raise ValueError("convmi needs contiguous tensors")
    return t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def workspace(desc: ConvDesc, op: int, device="cuda"):
    """Allocate the caller-owned workspace one operation needs (None when 0 bytes)."""
    import torch
    n = workspace_size(desc, op)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def conv2d_forward(desc, x, w, bias, gamma, beta, running_mean, running_var, save_mean, save_inv_std, z, y,
                   workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(lib.conv2d_forward(C.byref(desc), _ptr(x), _ptr(w), _ptr(bias), _ptr(gamma), _ptr(beta),
                              _ptr(running_mean), _ptr(running_var), _ptr(save_mean), _ptr(save_inv_std),
                              _ptr(z), _ptr(y), wp, wn, _stream(stream)))


def conv2d_forward_noalloc(desc, x, w, bias, gamma, beta, running_mean, running_var, save_mean, save_inv_std, z,
                           y, stream=None):
    _check(lib.conv2d_forward_noalloc(C.byref(desc), _ptr(x), _ptr(w), _ptr(bias), _ptr(gamma), _ptr(beta),
                                      _ptr(running_mean), _ptr(running_var), _ptr(save_mean), _ptr(save_inv_std),
                                      _ptr(z), _ptr(y), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 8 << 20  # CONVMI_NOALLOC_SCRATCH_BYTES


def conv2d_backward_data(desc, dz, w, dx, workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(lib.conv2d_backward_data(C.byref(desc), _ptr(dz), _ptr(w), _ptr(dx), wp, wn, _stream(stream)))


def conv2d_backward_weight(desc, x, dz, dw, db, accumulate=0, workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(lib.conv2d_backward_weight(C.byref(desc), _ptr(x), _ptr(dz), _ptr(dw), _ptr(db), int(accumulate),
                                      wp, wn, _stream(stream)))


def bn_stats_training(desc, z, save_mean, save_inv_std, running_mean=None, running_var=None, workspace=None,
                      stream=None):
    wp, wn = _ws(workspace)
    _check(lib.bn_stats_training(C.byref(desc), _ptr(z), _ptr(save_mean), _ptr(save_inv_std),
                                 _ptr(running_mean), _ptr(running_var), wp, wn, _stream(stream)))


def activation_backward(desc, z, dy, gamma, beta, save_mean, save_inv_std, dz, dgamma=None, dbeta=None,
                        accumulate=0, workspace=None, stream=None):
    wp, wn = _ws(workspace)
    _check(lib.activation_backward(C.byref(desc), _ptr(z), _ptr(dy), _ptr(gamma), _ptr(beta), _ptr(save_mean),
                                   _ptr(save_inv_std), _ptr(dz), _ptr(dgamma), _ptr(dbeta), int(accumulate),
                                   wp, wn, _stream(stream)))


def conv2d_backward_full(desc, x, w, saved, saved_is_output, dy, dx, dw, db, accumulate=0, workspace=None,
                         stream=None):
    wp, wn = _ws(workspace)
    _check(lib.conv2d_backward_full(C.byref(desc), _ptr(x), _ptr(w), _ptr(saved), int(saved_is_output), _ptr(dy),
                                    _ptr(dx), _ptr(dw), _ptr(db), int(accumulate), wp, wn, _stream(stream)))


# ---------------------------------------------------------------- MX8, RMS norm, linear layer
# These entry points check each tensor's type, size and device before its pointer is
# passed on, and run on the tensors' own device whatever the current one is.  A small call
# takes about as long on the host as on the GPU, so the checks are kept short: one line
# per tensor in the good case.
def _p(name, t, dtypes, n, dev):
    """Pointer of a contiguous tensor on device `dev` with one of the dtypes and n elements, or None."""
    if t is None:
        return None
    if t.get_device() == dev and t.dtype in dtypes and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"convmi needs device (HIP) tensors: {name} is on {t.device}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, others on cuda:{dev}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    raise ValueError(f"convmi needs contiguous tensors: {name} is not")


def _device(name, t):
    """Index of the device the call runs on: that of its first tensor."""
    if t is None:
        raise ValueError(f"{name} is None")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"convmi needs device (HIP) tensors: {name} is on {t.device}")
    return dev


def _w(workspace, dev):
    """(pointer, bytes) of a caller-owned workspace or None."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != dev:
        raise ValueError(f"the workspace is on {workspace.device}, the tensors on cuda:{dev}")
    return _ws(workspace)


def _call(fn, dev, stream, *args):
    """fn(*args, stream) with device `dev` current, on `stream` or that device's current one."""
    raw_stream, current_device, device_guard = _TORCH["run"]
    if stream is None:
        handle = raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        handle = stream.cuda_stream
    if current_device() == dev:
        status = fn(*args, handle)
    else:
        with device_guard(dev):
            status = fn(*args, handle)
    if status != OK:
        _check(status)


_TORCH = {}  # torch's types and calls, looked up once: importing this package does not import torch


def _types(dtype: int):
    """(data, fp32, codes, scales) torch dtypes accepted for a CONVMI dtype."""
    types = _TORCH.get(dtype)
    if types is not None:
        return types
    if not _TORCH:
        import torch
        f32, codes = (torch.float32,), (torch.uint8, torch.float8_e4m3fn)
        scales = (torch.uint8, torch.float8_e8m0fnu)
        _TORCH.update({F32: (f32, f32, codes, scales), BF16: ((torch.bfloat16,), f32, codes, scales),
                       "ids": {torch.float32: F32, torch.bfloat16: BF16}, "int32": (torch.int32,),
                       # current_stream(dev).cuda_stream without the Stream object, current_device() of a
                       # process that has device tensors
                       "run": (torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice, torch.cuda.device)})
    if dtype not in (F32, BF16):
        raise ConvmiError(ERR_INVALID_ARG, f"unknown dtype {dtype}")
    return _TORCH[dtype]


def mx8_blocks(cols: int) -> int:
    """Scale bytes of a row of `cols` values."""
    return -(-cols // MX8_BLOCK)


def _mx8_tensor(x):
    """(rows, cols, CONVMI dtype, accepted dtypes) of the dense side of a packed tensor."""
    types = _types(F32)
    dt = _TORCH["ids"].get(x.dtype)
    if dt is None:
        raise ValueError(f"x has dtype {x.dtype}, expected float32 or bfloat16")
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("convmi MX8 needs a tensor with a last axis")
    cols = x.shape[-1]
    return x.numel() // cols, cols, dt, types


def mx8_pack(x, codes, scales, stream=None):
    """Keep x [..., cols] as MX8: codes (uint8 or float8_e4m3fn, x's size) and scales
    (uint8 or float8_e8m0fnu, [..., ceil(cols/32)])."""
    rows, cols, dt, (_, _, ct, st) = _mx8_tensor(x)
    dev, n = _device("x", x), rows * cols
    _call(lib.mx8_pack, dev, stream, rows, cols, dt, _p("x", x, (x.dtype,), n, dev), _p("codes", codes, ct, n, dev),
          _p("scales", scales, st, rows * mx8_blocks(cols), dev))


def mx8_unpack(codes, scales, x, stream=None):
    """The values of codes and scales into x [..., cols] (float32 or bfloat16)."""
    rows, cols, dt, (_, _, ct, st) = _mx8_tensor(x)
    dev, n = _device("x", x), rows * cols
    _call(lib.mx8_unpack, dev, stream, rows, cols, dt, _p("codes", codes, ct, n, dev),
          _p("scales", scales, st, rows * mx8_blocks(cols), dev), _p("x", x, (x.dtype,), n, dev))


def conv2d_backward_full_mx8(desc, x, x_scales, w, saved, saved_scales, saved_is_output, dy, dx, dw, db,
                             accumulate=0, workspace=None, stream=None):
    """conv2d_backward_full with x and / or saved kept as MX8 (their scales not None)."""
    data, f32, ct, st = _types(desc.dtype)
    oh, ow = output_dims(desc)
    ic, oc = desc.IC, desc.OC
    xr, yr, nw = desc.N * desc.H * desc.W, desc.N * oh * ow, oc * desc.KH * desc.KW * ic
    dev = _device("x", x)
    _call(lib.conv2d_backward_full_mx8, dev, stream, C.byref(desc),
          _p("x", x, data if x_scales is None else ct, xr * ic, dev),
          _p("x_scales", x_scales, st, xr * mx8_blocks(ic), dev), _p("w", w, data, nw, dev),
          _p("saved", saved, data if saved_scales is None else ct, yr * oc, dev),
          _p("saved_scales", saved_scales, st, yr * mx8_blocks(oc), dev), int(saved_is_output),
          _p("dy", dy, data, yr * oc, dev), _p("dx", dx, data, xr * ic, dev), _p("dw", dw, f32, nw, dev),
          _p("db", db, f32, oc, dev), int(accumulate), *_w(workspace, dev))


def make_rms_desc(rows, cols, dtype=F32, eps=1e-5) -> RmsDesc:
    return RmsDesc(rows, cols, dtype, eps)


def rms_workspace_size(desc: RmsDesc) -> int:
    n = C.c_size_t()
    _check(lib.rms_norm_workspace_size(C.byref(desc), C.byref(n)))
    return n.value


def rms_workspace(desc: RmsDesc, device="cuda"):
    """Allocate the caller-owned workspace of rms_norm_backward."""
    import torch
    return torch.empty(rms_workspace_size(desc), dtype=torch.uint8, device=device)


def rms_norm_forward(desc, x, residual, gamma, h, y, save_inv_rms, y8=None, y8_scales=None, stream=None):
    """h = x + residual; y = gamma * h / rms(h), dense in y and / or as MX8 in y8, y8_scales."""
    data, f32, ct, st = _types(desc.dtype)
    rows, cols = desc.rows, desc.cols
    n, dev = rows * cols, _device("x", x)
    _call(lib.rms_norm_forward, dev, stream, C.byref(desc), _p("x", x, data, n, dev),
          _p("residual", residual, data, n, dev), _p("gamma", gamma, f32, cols, dev), _p("h", h, data, n, dev),
          _p("y", y, data, n, dev), _p("y8", y8, ct, n, dev),
          _p("y8_scales", y8_scales, st, rows * mx8_blocks(cols), dev),
          _p("save_inv_rms", save_inv_rms, f32, rows, dev))


def rms_norm_backward(desc, h, gamma, save_inv_rms, dy, dh, dx, dgamma=None, accumulate=0, workspace=None,
                      stream=None):
    """dx = dh + inv_rms (g - hhat mean(g hhat)), g = gamma dy; dgamma (+)= sum of dy hhat."""
    data, f32, _, _ = _types(desc.dtype)
    rows, cols = desc.rows, desc.cols
    n, dev = rows * cols, _device("h", h)
    _call(lib.rms_norm_backward, dev, stream, C.byref(desc), _p("h", h, data, n, dev),
          _p("gamma", gamma, f32, cols, dev), _p("save_inv_rms", save_inv_rms, f32, rows, dev),
          _p("dy", dy, data, n, dev), _p("dh", dh, data, n, dev), _p("dx", dx, data, n, dev),
          _p("dgamma", dgamma, f32, cols, dev), int(accumulate), *_w(workspace, dev))


def make_layer_norm_desc(rows, cols, dtype=F32, eps=1e-5) -> LayerNormDesc:
    return LayerNormDesc(rows, cols, dtype, eps)


def layer_norm_workspace_size(desc: LayerNormDesc) -> int:
    n = C.c_size_t()
    _check(lib.layer_norm_workspace_size(C.byref(desc), C.byref(n)))
    return n.value


def layer_norm_workspace(desc: LayerNormDesc, device="cuda"):
    """Allocate the caller-owned workspace of layer_norm_backward."""
    import torch
    return torch.empty(layer_norm_workspace_size(desc), dtype=torch.uint8, device=device)


def layer_norm_forward(desc, x, residual, gamma, beta, h, y, save_mean, save_inv_std, y8=None, y8_scales=None,
                       stream=None):
    """h = x + residual; y = gamma * (h - mean) * inv_std + beta, dense in y and / or as MX8 in y8, y8_scales."""
    data, f32, ct, st = _types(desc.dtype)
    rows, cols = desc.rows, desc.cols
    n, dev = rows * cols, _device("x", x)
    _call(lib.layer_norm_forward, dev, stream, C.byref(desc), _p("x", x, data, n, dev),
          _p("residual", residual, data, n, dev), _p("gamma", gamma, f32, cols, dev), _p("beta", beta, f32, cols, dev),
          _p("h", h, data, n, dev), _p("y", y, data, n, dev), _p("y8", y8, ct, n, dev),
          _p("y8_scales", y8_scales, st, rows * mx8_blocks(cols), dev), _p("save_mean", save_mean, f32, rows, dev),
          _p("save_inv_std", save_inv_std, f32, rows, dev))


def layer_norm_backward(desc, h, gamma, save_mean, save_inv_std, dy, dh, dx, dgamma=None, dbeta=None, accumulate=0,
                        workspace=None, stream=None):
    """dx = dh + inv_std (g - mean(g) - hhat mean(g hhat)), g = gamma dy; dgamma (+)= sum of dy hhat,
    dbeta (+)= sum of dy."""
    data, f32, _, _ = _types(desc.dtype)
    rows, cols = desc.rows, desc.cols
    n, dev = rows * cols, _device("h", h)
    _call(lib.layer_norm_backward, dev, stream, C.byref(desc), _p("h", h, data, n, dev),
          _p("gamma", gamma, f32, cols, dev), _p("save_mean", save_mean, f32, rows, dev),
          _p("save_inv_std", save_inv_std, f32, rows, dev), _p("dy", dy, data, n, dev), _p("dh", dh, data, n, dev),
          _p("dx", dx, data, n, dev), _p("dgamma", dgamma, f32, cols, dev), _p("dbeta", dbeta, f32, cols, dev),
          int(accumulate), *_w(workspace, dev))


# ---------------------------------------------------------------- operators along sequences
def _cols(name, t, dtypes, rows, cols, pitch, dev):
    """Pointer of a tensor of `rows` rows of `cols` elements that begin `pitch` apart (0: a
    contiguous tensor), or None."""
    if t is None or pitch == 0 or pitch == cols:
        return _p(name, t, dtypes, rows * cols, dev)
    if (t.stride() == (pitch, 1) and t.size(1) == cols and t.size(0) == rows and t.dtype in dtypes
            and t.get_device() == dev):
        return t.data_ptr()
    if t.get_device() != dev or t.dtype not in dtypes or t.numel() != rows * cols or t.dim() == 0 or t.shape[-1] != cols:
        _p(name, t, dtypes, rows * cols, dev)  # says what is wrong, if not only the last axis
        if rows:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected rows of {cols} elements")
    step = pitch
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size > 1 and stride != step:
            raise ValueError(f"{name}: rows are {stride} elements apart in places, the descriptor says {step}")
        step *= size
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: elements of a row are not side by side")
    return t.data_ptr()


def _starts(seq_starts, batch, dev):
    return None if seq_starts is None else _p("seq_starts", seq_starts, _TORCH["int32"], batch + 1, dev)


def _slots(slots, rows, dev):
    return None if slots is None else _p("slots", slots, _TORCH["int32"], rows, dev)


def _pool(name, state, dtypes, per, dev):
    """(pointer, number) of states of `per` elements."""
    if state is None:
        return None, 0
    n = state.shape[0] if state.dim() else 0
    return _p(name, state, dtypes, n * per, dev), n


# All fields of a descriptor at once: a field of a ctypes structure costs as much as a tensor's check.
_SCAN_FIELDS = struct.Struct("@3q4i4q").unpack_from
_CONV_FIELDS = struct.Struct("@3q3iq").unpack_from


def make_causal_conv_desc(rows, channels, taps, batch=1, activation=ACT_IDENTITY, dtype=F32,
                          x_pitch=0) -> CausalConvDesc:
    return CausalConvDesc(rows, channels, batch, taps, activation, dtype, x_pitch)


def causal_conv_workspace_size(desc: CausalConvDesc) -> int:
    n = C.c_size_t()
    _check(lib.causal_conv_workspace_size(C.byref(desc), C.byref(n)))
    return n.value


def causal_conv_workspace(desc: CausalConvDesc, device="cuda"):
    """Allocate the caller-owned workspace of causal_conv_backward (None when 0 bytes)."""
    import torch
    n = causal_conv_workspace_size(desc)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def causal_conv_forward(desc, x, w, bias, y, seq_starts=None, initial_state=None, final_state=None, stream=None):
    """y_t = act(bias + sum_k w[:, k] x_(t - taps + 1 + k)) within each sequence."""
    rows, D, batch, W, _, dtype, xp = _CONV_FIELDS(desc)
    data, f32, _, _ = _types(dtype)
    _upright("w", w, D, W)
    dev, ns = _device("x", x), batch * (W - 1) * D
    _call(lib.causal_conv_forward, dev, stream, C.byref(desc), _cols("x", x, data, rows, D, xp, dev),
          _starts(seq_starts, batch, dev), _p("w", w, data, D * W, dev), _p("bias", bias, f32, D, dev),
          _p("initial_state", initial_state, data, ns, dev), _p("y", y, data, rows * D, dev),
          _p("final_state", final_state, data, ns, dev))


def causal_conv_backward(desc, x, w, bias, dy, dx, dw=None, db=None, accumulate=0, workspace=None, seq_starts=None,
                         initial_state=None, d_final_state=None, d_initial_state=None, stream=None):
    """dx, dw, db and d_initial_state from dy (and d_final_state); z is formed again from x."""
    rows, D, batch, W, _, dtype, xp = _CONV_FIELDS(desc)
    data, f32, _, _ = _types(dtype)
    _upright("w", w, D, W)
    _upright("dw", dw, D, W)
    dev, ns = _device("x", x), batch * (W - 1) * D
    _call(lib.causal_conv_backward, dev, stream, C.byref(desc), _cols("x", x, data, rows, D, xp, dev),
          _starts(seq_starts, batch, dev), _p("w", w, data, D * W, dev), _p("bias", bias, f32, D, dev),
          _p("initial_state", initial_state, data, ns, dev), _p("dy", dy, data, rows * D, dev),
          _p("d_final_state", d_final_state, data, ns, dev), _cols("dx", dx, data, rows, D, xp, dev),
          _p("d_initial_state", d_initial_state, data, ns, dev), _p("dw", dw, f32, D * W, dev),
          _p("db", db, f32, D, dev), int(accumulate), *_w(workspace, dev))


def causal_conv_step(desc, x, w, bias, state, y, slots=None, stream=None):
    """One token of each of desc.rows sequences: y from x and its state in the pool `state`
    [slots, taps - 1, channels] (with one tap it may be None: as many as rows), which moves by one row
    in place."""
    rows, D, _, W, _, dtype, xp = _CONV_FIELDS(desc)
    data, f32, _, _ = _types(dtype)
    _upright("w", w, D, W)
    dev = _device("x", x)
    at, n = _pool("state", state, data, (W - 1) * D, dev)
    _call(lib.causal_conv_step, dev, stream, C.byref(desc), _cols("x", x, data, rows, D, xp, dev),
          _p("w", w, data, D * W, dev), _p("bias", bias, f32, D, dev), at, rows if W == 1 and state is None else n,
          _slots(slots, rows, dev), _p("y", y, data, rows * D, dev))


def make_scan_desc(rows, channels, states, batch=1, groups=1, dtype=F32, delta_softplus=True, x_pitch=0, dt_pitch=0,
                   z_pitch=0, bc_pitch=0) -> ScanDesc:
    return ScanDesc(rows, channels, batch, states, groups, dtype, int(delta_softplus), x_pitch, dt_pitch, z_pitch,
                    bc_pitch)


def scan_workspace_size(desc: ScanDesc, op: int) -> int:
    n = C.c_size_t()
    _check(lib.selective_scan_workspace_size(C.byref(desc), op, C.byref(n)))
    return n.value


def scan_workspace(desc: ScanDesc, op: int, device="cuda"):
    """Allocate the caller-owned workspace of SCAN_FORWARD or SCAN_BACKWARD (None when 0 bytes)."""
    import torch
    n = scan_workspace_size(desc, op)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def scan_saved_size(desc: ScanDesc) -> int:
    n = C.c_size_t()
    _check(lib.selective_scan_saved_size(C.byref(desc), C.byref(n)))
    return n.value


def scan_saved_states(desc: ScanDesc, device="cuda"):
    """Allocate the states that selective_scan_forward keeps for the backward pass."""
    import torch
    return torch.empty(scan_saved_size(desc) // 4, dtype=torch.float32, device=device)


def _scan_inputs(desc, x, dt, dt_bias, A, B, C_, D, z):
    """((rows, channels, batch, states, B's columns), device, data types, fp32, pitches, input pointers)."""
    rows, ch, batch, N, G, dtype, _, xp, dtp, zp, bcp = _SCAN_FIELDS(desc)
    data, f32, _, _ = _types(dtype)
    dev, bc = _device("x", x), G * N
    _upright("A", A, ch, N)
    return (rows, ch, batch, N, bc), dev, data, f32, (xp, dtp, zp, bcp), (
        _cols("x", x, data, rows, ch, xp, dev), _cols("dt", dt, data, rows, ch, dtp, dev),
        _p("dt_bias", dt_bias, f32, ch, dev), _p("A", A, f32, ch * N, dev), _cols("B", B, data, rows, bc, bcp, dev),
        _cols("C", C_, data, rows, bc, bcp, dev), _p("D", D, f32, ch, dev), _cols("z", z, data, rows, ch, zp, dev))


def selective_scan_forward(desc, x, dt, dt_bias, A, B, C_, D, z, y, seq_starts=None, initial_state=None,
                           final_state=None, saved_states=None, workspace=None, stream=None):
    """h_t = exp(delta A) h_(t-1) + delta x B_t; y_t = (sum_n C_t h_t + D x) silu(z) within each sequence."""
    (rows, ch, batch, N, _), dev, data, f32, _, ins = _scan_inputs(desc, x, dt, dt_bias, A, B, C_, D, z)
    ns = batch * ch * N
    _call(lib.selective_scan_forward, dev, stream, C.byref(desc), *ins, _starts(seq_starts, batch, dev),
          _p("initial_state", initial_state, f32, ns, dev), _p("y", y, data, rows * ch, dev),
          _p("final_state", final_state, f32, ns, dev),
          None if saved_states is None else _p("saved_states", saved_states, f32, scan_saved_size(desc) // 4, dev),
          *_w(workspace, dev))


def selective_scan_backward(desc, x, dt, dt_bias, A, B, C_, D, z, saved_states, dy, dx, ddt, dB, dC, dz=None,
                            d_dt_bias=None, dA=None, dD=None, accumulate=0, workspace=None, seq_starts=None,
                            d_final_state=None, d_initial_state=None, stream=None):
    """Gradients of every input from dy (and d_final_state), with the states that the forward kept."""
    (rows, ch, batch, N, bc), dev, data, f32, (xp, dtp, zp, bcp), ins = _scan_inputs(desc, x, dt, dt_bias, A, B, C_, D, z)
    ns = batch * ch * N
    _upright("dA", dA, ch, N)
    _call(lib.selective_scan_backward, dev, stream, C.byref(desc), *ins, _starts(seq_starts, batch, dev),
          _p("saved_states", saved_states, f32, scan_saved_size(desc) // 4, dev), _p("dy", dy, data, rows * ch, dev),
          _p("d_final_state", d_final_state, f32, ns, dev), _cols("dx", dx, data, rows, ch, xp, dev),
          _cols("ddt", ddt, data, rows, ch, dtp, dev), _cols("dB", dB, data, rows, bc, bcp, dev),
          _cols("dC", dC, data, rows, bc, bcp, dev), _cols("dz", dz, data, rows, ch, zp, dev),
          _p("d_dt_bias", d_dt_bias, f32, ch, dev), _p("dA", dA, f32, ch * N, dev), _p("dD", dD, f32, ch, dev),
          _p("d_initial_state", d_initial_state, f32, ns, dev), int(accumulate), *_w(workspace, dev))


def selective_scan_step(desc, x, dt, dt_bias, A, B, C_, D, z, state, y, slots=None, stream=None):
    """One token of each of desc.rows sequences: its state in the pool `state` [slots, channels,
    states] is updated in place."""
    (rows, ch, _, N, _), dev, data, f32, _, ins = _scan_inputs(desc, x, dt, dt_bias, A, B, C_, D, z)
    at, n = _pool("state", state, f32, ch * N, dev)
    _call(lib.selective_scan_step, dev, stream, C.byref(desc), *ins, at, n, _slots(slots, rows, dev),
          _p("y", y, data, rows * ch, dev))


def make_linear_desc(M, K, N, activation=ACT_IDENTITY, dtype=F32, x_mx8=False, z_mx8=False) -> LinearDesc:
    return LinearDesc(M, K, N, activation, dtype, int(x_mx8), int(z_mx8))


def linear_workspace_size(desc: LinearDesc, op: int) -> int:
    n = C.c_size_t()
    _check(lib.linear_workspace_size(C.byref(desc), op, C.byref(n)))
    return n.value


def linear_workspace(desc: LinearDesc, op: int, device="cuda"):
    """Allocate the caller-owned workspace one linear operation needs (None when 0 bytes)."""
    import torch
    n = linear_workspace_size(desc, op)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def linear_plan_name(desc: LinearDesc, op: int) -> str:
    """Kernel plan of a linear operation for this descriptor (host only)."""
    buf = C.create_string_buffer(128)
    _check(lib.linear_plan_name(C.byref(desc), op, buf, len(buf)))
    return buf.value.decode()


def _upright(name, t, rows, cols):
    """Refuse a matrix with its axes turned round: it has the right number of elements in the wrong order."""
    if rows != cols and rows > 1 < cols and t is not None and t.dim() == 2 and t.shape[0] == cols:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({rows}, {cols})")


def linear_forward(desc, x, w, bias, residual, z, y, workspace=None, x_scales=None, w_scales=None, z_scales=None,
                   stream=None):
    """z = x w^T + bias; y = act(z) + residual.  Scales go with tensors kept as MX8."""
    data, f32, ct, st = _types(desc.dtype)
    M, K, N = desc.M, desc.K, desc.N
    _upright("w", w, N, K)
    xt, zt = ct if desc.x_mx8 else data, ct if desc.z_mx8 else data
    n, kb, dev = M * N, mx8_blocks(K), _device("x", x)
    _call(lib.linear_forward, dev, stream, C.byref(desc), _p("x", x, xt, M * K, dev),
          _p("x_scales", x_scales, st, M * kb, dev), _p("w", w, xt, N * K, dev),
          _p("w_scales", w_scales, st, N * kb, dev), _p("bias", bias, f32, N, dev),
          _p("residual", residual, data, n, dev), _p("z", z, zt, n, dev),
          _p("z_scales", z_scales, st, M * mx8_blocks(N), dev), _p("y", y, data, n, dev), *_w(workspace, dev))


def linear_activation_backward(desc, z, dy, dz, z_scales=None, stream=None):
    """dz = act'(z) * dy at z as kept."""
    data, _, ct, st = _types(desc.dtype)
    M, N = desc.M, desc.N
    n, dev = M * N, _device("z", z)
    _call(lib.linear_activation_backward, dev, stream, C.byref(desc), _p("z", z, ct if desc.z_mx8 else data, n, dev),
          _p("z_scales", z_scales, st, M * mx8_blocks(N), dev), _p("dy", dy, data, n, dev), _p("dz", dz, data, n, dev))


def linear_backward_data(desc, dz, w, dx, workspace=None, stream=None):
    """dx = dz w."""
    data = _types(desc.dtype)[0]
    M, K, N = desc.M, desc.K, desc.N
    _upright("w", w, N, K)
    dev = _device("dz", dz)
    _call(lib.linear_backward_data, dev, stream, C.byref(desc), _p("dz", dz, data, M * N, dev),
          _p("w", w, data, N * K, dev), _p("dx", dx, data, M * K, dev), *_w(workspace, dev))


def linear_backward_weight(desc, x, dz, dw, db, accumulate=0, workspace=None, x_scales=None, stream=None):
    """dw (+)= dz^T x; db (+)= column sums of dz.  x_scales goes with an x kept as MX8."""
    data, f32, ct, st = _types(desc.dtype)
    M, K, N = desc.M, desc.K, desc.N
    _upright("dw", dw, N, K)
    dev = _device("x", x)
    _call(lib.linear_backward_weight, dev, stream, C.byref(desc), _p("x", x, ct if desc.x_mx8 else data, M * K, dev),
          _p("x_scales", x_scales, st, M * mx8_blocks(K), dev), _p("dz", dz, data, M * N, dev),
          _p("dw", dw, f32, N * K, dev), _p("db", db, f32, N, dev), int(accumulate), *_w(workspace, dev))
