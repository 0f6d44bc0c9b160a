"""Python binding of the gfx950 selective-scan library (libssm_amd.so).

A thin ctypes layer over the C ABI declared in include/ssm.h: every function
here has the name of the C entry point it calls and only marshals arguments
(torch tensors -> device pointers, the current HIP stream, descriptors).
PyTorch supplies device memory and streams; all arithmetic runs in the HIP
kernels.  Outputs that are not passed in are allocated with torch.empty, on the
stream that the call runs on.

The library must have been built (selective_state_space_ssm_amd/build.py);
importing the binding never falls back to any other implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssm_amd.so")

SSM_OK = 0
SSM_ERR_NULL_ARG = 1
SSM_ERR_BAD_SHAPE = 2
SSM_ERR_UNSUPPORTED = 3
SSM_ERR_WORKSPACE = 4
SSM_ERR_ALIGNMENT = 5
SSM_ERR_ALIAS = 6
SSM_ERR_HIP = 7
SSM_ERR_SCRATCH_LIMIT = 8
SSM_ERR_HOST_MEMORY = 9
SSM_STATIC_SCRATCH_BYTES = 16 << 20   # the library's static device buffer (ssm_scan_fwd_static)

SSM_F32 = 0
SSM_BF16 = 1
SSM_DISC_DELTA_B = 0
SSM_DISC_ZOH = 1
SSM_REDUCE_MEAN = 0
SSM_REDUCE_SUM = 1
SSM_DECAY_CONST = 2   # decay fixed per (channel, state); no step size, dt_raw may be None

EXPORTED_SYMBOLS = (
    "ssm_version", "ssm_status_string", "conv1d_causal", "ssm_scan_fwd_workspace_size",
    "ssm_scan_fwd", "ssm_scan_bwd_workspace_size", "ssm_scan_bwd", "ssm_step",
    "ssm_model_decode_workspace_size", "ssm_model_decode_step", "ssm_scan_fwd_static",
    "ssm_layer_norm_fwd", "ssm_layer_norm_bwd_workspace_size", "ssm_layer_norm_bwd", "ssm_token_logp_fwd",
    "ssm_token_logp_bwd", "ssm_policy_loss_workspace_size", "ssm_policy_loss",
    "ssm_clip_grad_norm_workspace_size", "ssm_clip_grad_norm",
)


class SSMError(RuntimeError):
    def __init__(self, fn, code):
        self.code = int(code)
        super().__init__("%s failed: %s (status %d)" % (fn, ssm_status_string(code), code))


class ssm_scan_desc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("conv_width", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("disc", ctypes.c_int32), ("chunk_len", ctypes.c_int32)]


class ssm_step_desc(ctypes.Structure):
    _fields_ = [("nblocks", ctypes.c_int64), ("nstreams", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("conv_width", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("disc", ctypes.c_int32), ("state_dtype", ctypes.c_int32)]


class ssm_conv_desc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("width", ctypes.c_int32), ("fuse_silu", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ssm_model_desc(ctypes.Structure):
    _fields_ = [("nstreams", ctypes.c_int64), ("vocab", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("n_layers", ctypes.c_int32), ("d_inner", ctypes.c_int32), ("d_state", ctypes.c_int32),
                ("dt_rank", ctypes.c_int32), ("conv_width", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ssm_norm_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("r_stride", ctypes.c_int64), ("s_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class ssm_logp_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("logits_stride", ctypes.c_int64),
                ("dlogits_stride", ctypes.c_int64), ("io_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ssm_policy_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("logits_stride", ctypes.c_int64),
                ("dlogits_stride", ctypes.c_int64), ("clip_low", ctypes.c_double), ("clip_high", ctypes.c_double),
                ("kl_beta", ctypes.c_double), ("grad_scale", ctypes.c_double), ("io_dtype", ctypes.c_int32),
                ("reduction", ctypes.c_int32)]


class ssm_grad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


LAYER_FIELDS = ("norm_w", "norm_b", "in_proj", "conv_w", "conv_b", "x_proj", "dt_proj_w", "dt_proj_b",
                "A_log", "Dskip", "out_proj")


class ssm_layer_weights(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in LAYER_FIELDS]


_lib = None


def lib():
    """The loaded library with argument types set (raises if not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libssm_amd.so is not built; run selective_state_space_ssm_amd/build.py "
                              "(or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        p, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        L.ssm_version.restype = i32
        L.ssm_version.argtypes = []
        L.ssm_status_string.restype = ctypes.c_char_p
        L.ssm_status_string.argtypes = [i32]
        L.conv1d_causal.restype = i32
        L.conv1d_causal.argtypes = [ctypes.POINTER(ssm_conv_desc)] + [p] * 7
        L.ssm_scan_fwd_workspace_size.restype = i32
        L.ssm_scan_fwd_workspace_size.argtypes = [ctypes.POINTER(ssm_scan_desc), ctypes.POINTER(sz)]
        L.ssm_scan_fwd.restype = i32
        L.ssm_scan_fwd.argtypes = [ctypes.POINTER(ssm_scan_desc)] + [p] * 16 + [sz, p]
        L.ssm_scan_fwd_static.restype = i32
        L.ssm_scan_fwd_static.argtypes = [ctypes.POINTER(ssm_scan_desc)] + [p] * 16
        L.ssm_scan_bwd_workspace_size.restype = i32
        L.ssm_scan_bwd_workspace_size.argtypes = [ctypes.POINTER(ssm_scan_desc), ctypes.POINTER(sz)]
        L.ssm_scan_bwd.restype = i32
        L.ssm_scan_bwd.argtypes = [ctypes.POINTER(ssm_scan_desc)] + [p] * 27 + [sz, p]
        L.ssm_step.restype = i32
        L.ssm_step.argtypes = [ctypes.POINTER(ssm_step_desc)] + [p] * 14
        L.ssm_model_decode_workspace_size.restype = i32
        L.ssm_model_decode_workspace_size.argtypes = [ctypes.POINTER(ssm_model_desc), ctypes.POINTER(sz)]
        L.ssm_model_decode_step.restype = i32
        L.ssm_model_decode_step.argtypes = [ctypes.POINTER(ssm_model_desc), p, p, p,
                                            ctypes.POINTER(ssm_layer_weights), p, p, p, p, p, sz, p]
        L.ssm_layer_norm_fwd.restype = i32
        L.ssm_layer_norm_fwd.argtypes = [ctypes.POINTER(ssm_norm_desc)] + [p] * 9
        L.ssm_layer_norm_bwd_workspace_size.restype = i32
        L.ssm_layer_norm_bwd_workspace_size.argtypes = [ctypes.POINTER(ssm_norm_desc), ctypes.POINTER(sz)]
        L.ssm_layer_norm_bwd.restype = i32
        L.ssm_layer_norm_bwd.argtypes = [ctypes.POINTER(ssm_norm_desc)] + [p] * 10 + [sz, p]
        L.ssm_token_logp_fwd.restype = i32
        L.ssm_token_logp_fwd.argtypes = [ctypes.POINTER(ssm_logp_desc)] + [p] * 5
        L.ssm_token_logp_bwd.restype = i32
        L.ssm_token_logp_bwd.argtypes = [ctypes.POINTER(ssm_logp_desc)] + [p] * 6
        L.ssm_policy_loss_workspace_size.restype = i32
        L.ssm_policy_loss_workspace_size.argtypes = [ctypes.POINTER(ssm_policy_desc), ctypes.POINTER(sz)]
        L.ssm_policy_loss.restype = i32
        L.ssm_policy_loss.argtypes = [ctypes.POINTER(ssm_policy_desc)] + [p] * 10 + [sz, p]
        L.ssm_clip_grad_norm_workspace_size.restype = i32
        L.ssm_clip_grad_norm_workspace_size.argtypes = [p, ctypes.c_int64, ctypes.POINTER(sz)]
        L.ssm_clip_grad_norm.restype = i32
        L.ssm_clip_grad_norm.argtypes = [p, ctypes.c_int64, ctypes.c_double, p, p, sz, p]
        _lib = L
    return _lib


def ssm_version() -> int:
    return int(lib().ssm_version())


def ssm_status_string(code: int) -> str:
    return lib().ssm_status_string(int(code)).decode()


# ----------------------------------------------------------------- marshalling
def _io_code(t):
    if t.dtype == torch.float32:
        return SSM_F32
    if t.dtype == torch.bfloat16:
        return SSM_BF16
    raise TypeError("io tensors must be float32 or bfloat16, got %s" % t.dtype)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _alloc(shape, dtype, device, stream, returned=True):
    """What a call on `stream` allocates itself: from that stream's memory."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    return _new(shape, dtype, device, stream, _stream(stream).value or 0, returned)


def _check(fn, rc):
    if rc != SSM_OK:
        raise SSMError(fn, rc)


def _f32(t, name):
    return _ptr(t, torch.float32, name)


# --------------------------------------------------------------------- calls
def conv1d_causal(x, w, b=None, state_in=None, state_out=None, y=None, silu=True, stream=None):
    """y = act(causal depthwise conv(x)) for x [B, L, D] (io dtype), w [D, W].
    Returns y."""
    Bn, L, D = x.shape
    W = w.shape[1]
    io = _io_code(x)
    if y is None:
        y = _alloc(x.shape, x.dtype, x.device, stream)
    desc = ssm_conv_desc(Bn, L, D, W, 1 if silu else 0, io, 0)
    _check("conv1d_causal", lib().conv1d_causal(
        ctypes.byref(desc), _ptr(x, x.dtype, "x"), _f32(w, "w"), _f32(b, "b"),
        _f32(state_in, "state_in"), _f32(state_out, "state_out"), _ptr(y, x.dtype, "y"),
        _stream(stream)))
    return y


def _scan_desc(x, N, conv_width, disc, chunk_len):
    Bn, L, D = x.shape
    return ssm_scan_desc(Bn, L, D, N, conv_width, _io_code(x), disc, chunk_len)


def ssm_scan_fwd_workspace_size(desc) -> int:
    n = ctypes.c_size_t(0)
    _check("ssm_scan_fwd_workspace_size", lib().ssm_scan_fwd_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return int(n.value)


def ssm_scan_bwd_workspace_size(desc) -> int:
    n = ctypes.c_size_t(0)
    _check("ssm_scan_bwd_workspace_size", lib().ssm_scan_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return int(n.value)


def _workspace(nbytes, given, device, stream):
    if nbytes == 0:
        return given
    if given is not None:
        return given
    return _alloc(nbytes, torch.uint8, device, stream, returned=False)


def ssm_scan_fwd(x, dt_raw, A_log, B, C, dt_bias=None, Dskip=None, z=None, conv_w=None, conv_b=None,
                 conv_state_in=None, conv_state_out=None, h0=None, hT=None, y=None,
                 disc=SSM_DISC_DELTA_B, chunk_len=0, workspace=None, stream=None):
    """Selective scan over x [B, L, D] (u, or the conv input when conv_w is
    given).  Writes hT / conv_state_out when passed; returns y."""
    N = A_log.shape[1]
    W = conv_w.shape[1] if conv_w is not None else 0
    desc = _scan_desc(x, N, W, disc, chunk_len)
    if y is None:
        y = _alloc(x.shape, x.dtype, x.device, stream)
    ws = _workspace(ssm_scan_fwd_workspace_size(desc), workspace, x.device, stream)
    t = x.dtype
    _check("ssm_scan_fwd", lib().ssm_scan_fwd(
        ctypes.byref(desc), _ptr(x, t, "x"), _ptr(dt_raw, t, "dt_raw"), _f32(dt_bias, "dt_bias"),
        _f32(A_log, "A_log"), _ptr(B, t, "B"), _ptr(C, t, "C"), _f32(Dskip, "Dskip"), _ptr(z, t, "z"),
        _f32(conv_w, "conv_w"), _f32(conv_b, "conv_b"), _f32(conv_state_in, "conv_state_in"),
        _f32(conv_state_out, "conv_state_out"), _f32(h0, "h0"), _f32(hT, "hT"), _ptr(y, t, "y"),
        _ptr(ws, None, "workspace"), ctypes.c_size_t(ws.numel() if ws is not None else 0),
        _stream(stream)))
    return y


def ssm_scan_fwd_static(x, dt_raw, A_log, B, C, dt_bias=None, Dskip=None, z=None, conv_w=None, conv_b=None,
                        conv_state_in=None, conv_state_out=None, h0=None, hT=None, y=None,
                        disc=SSM_DISC_DELTA_B, chunk_len=0, stream=None):
    """ssm_scan_fwd without a workspace: a time split keeps its chunk summaries
    in the library's static device buffer (SSM_STATIC_SCRATCH_BYTES per GPU).
    Allocates nothing when y is given.  Calls that overlap on one GPU race on
    that buffer.  Returns y."""
    N = A_log.shape[1]
    W = conv_w.shape[1] if conv_w is not None else 0
    desc = _scan_desc(x, N, W, disc, chunk_len)
    if y is None:
        y = _alloc(x.shape, x.dtype, x.device, stream)
    t = x.dtype
    _check("ssm_scan_fwd_static", lib().ssm_scan_fwd_static(
        ctypes.byref(desc), _ptr(x, t, "x"), _ptr(dt_raw, t, "dt_raw"), _f32(dt_bias, "dt_bias"),
        _f32(A_log, "A_log"), _ptr(B, t, "B"), _ptr(C, t, "C"), _f32(Dskip, "Dskip"), _ptr(z, t, "z"),
        _f32(conv_w, "conv_w"), _f32(conv_b, "conv_b"), _f32(conv_state_in, "conv_state_in"),
        _f32(conv_state_out, "conv_state_out"), _f32(h0, "h0"), _f32(hT, "hT"), _ptr(y, t, "y"),
        _stream(stream)))
    return y


def ssm_scan_bwd(x, dt_raw, A_log, B, C, dy, dt_bias=None, Dskip=None, z=None, conv_w=None, conv_b=None,
                 conv_state_in=None, h0=None, dhT=None, disc=SSM_DISC_DELTA_B, chunk_len=0,
                 want=("dx", "d_dt_raw", "d_dt_bias", "dA_log", "dB", "dC", "dD", "dz", "dh0",
                       "dconv_w", "dconv_b", "dconv_state"),
                 out=None, workspace=None, stream=None):
    """Gradients of ssm_scan_fwd for the loss sum(y*dy) + sum(hT*dhT).
    x is u, or the conv input when conv_w is given (then dx flows through
    the conv + SiLU prologue).  Returns a dict of the requested gradients
    (allocated unless given in `out`); the conv ones only with conv_w, dz only
    with z, the dt ones not with SSM_DECAY_CONST."""
    Bn, L, D = x.shape
    N = A_log.shape[1]
    W = conv_w.shape[1] if conv_w is not None else 0
    desc = _scan_desc(x, N, W, disc, chunk_len)
    t = x.dtype
    out = dict(out or {})
    f32 = torch.float32
    shapes = dict(dx=((Bn, L, D), t), d_dt_raw=((Bn, L, D), t), d_dt_bias=((D,), f32),
                  dA_log=((D, N), f32), dB=((Bn, L, N), t), dC=((Bn, L, N), t),
                  dD=((D,), f32), dz=((Bn, L, D), t), dh0=((Bn, D, N), f32),
                  dconv_w=((D, W), f32), dconv_b=((D,), f32), dconv_state=((Bn, max(W - 1, 0), D), f32))
    for k in want:
        if k == "dz" and z is None:
            continue
        if k.startswith("dconv") and W == 0:
            continue
        if k in ("d_dt_raw", "d_dt_bias") and disc == SSM_DECAY_CONST:
            continue
        if k not in out:
            shp, dt_ = shapes[k]
            out[k] = _alloc(shp, dt_, x.device, stream)
    ws = _workspace(ssm_scan_bwd_workspace_size(desc), workspace, x.device, stream)
    g = out.get
    _check("ssm_scan_bwd", lib().ssm_scan_bwd(
        ctypes.byref(desc), _ptr(x, t, "x"), _ptr(dt_raw, t, "dt_raw"), _f32(dt_bias, "dt_bias"),
        _f32(A_log, "A_log"), _ptr(B, t, "B"), _ptr(C, t, "C"), _f32(Dskip, "Dskip"), _ptr(z, t, "z"),
        _f32(conv_w, "conv_w"), _f32(conv_b, "conv_b"), _f32(conv_state_in, "conv_state_in"),
        _f32(h0, "h0"), _ptr(dy, t, "dy"), _f32(dhT, "dhT"), _ptr(g("dx"), t, "dx"),
        _ptr(g("d_dt_raw"), t, "d_dt_raw"), _f32(g("d_dt_bias"), "d_dt_bias"), _f32(g("dA_log"), "dA_log"),
        _ptr(g("dB"), t, "dB"), _ptr(g("dC"), t, "dC"), _f32(g("dD"), "dD"), _ptr(g("dz"), t, "dz"),
        _f32(g("dh0"), "dh0"), _f32(g("dconv_w"), "dconv_w"), _f32(g("dconv_b"), "dconv_b"),
        _f32(g("dconv_state") if W > 1 else None, "dconv_state"),
        _ptr(ws, None, "workspace"), ctypes.c_size_t(ws.numel()), _stream(stream)))
    return out


def ssm_step(h, x, dt_raw, A_log, B, C, conv_state=None, z=None, conv_w=None, conv_b=None, dt_bias=None,
             Dskip=None, y=None, disc=SSM_DISC_DELTA_B, stream=None):
    """One streaming token.  h [nblk, S, D, N] (float32, or bfloat16 for a
    bf16-stored state) and conv_state [nblk, S, W-1, D] (float32) are updated
    in place; x/dt_raw/z [nblk, S, D], B/C [nblk, S, N], per-block parameters
    with a leading [nblk] axis.  Returns y [nblk, S, D]."""
    K, S, D, N = h.shape
    W = conv_w.shape[-1] if conv_w is not None else 0
    t = x.dtype
    if h.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("h must be float32 or bfloat16, got %s" % h.dtype)
    desc = ssm_step_desc(K, S, D, N, W, _io_code(x), disc, _io_code(h))
    if y is None:
        y = _alloc(x.shape, x.dtype, x.device, stream)
    _check("ssm_step", lib().ssm_step(
        ctypes.byref(desc), _ptr(h, h.dtype, "h"), _f32(conv_state, "conv_state"), _ptr(x, t, "x"),
        _ptr(dt_raw, t, "dt_raw"), _ptr(B, t, "B"), _ptr(C, t, "C"), _ptr(z, t, "z"), _f32(conv_w, "conv_w"),
        _f32(conv_b, "conv_b"), _f32(dt_bias, "dt_bias"), _f32(A_log, "A_log"), _f32(Dskip, "Dskip"),
        _ptr(y, t, "y"), _stream(stream)))
    return y


def model_desc(cfg, S) -> ssm_model_desc:
    """Descriptor of a model with shape cfg (keys vocab, d_model, n_layers,
    d_inner, d_state, dt_rank, conv_width) decoding S streams."""
    return ssm_model_desc(S, cfg["vocab"], cfg["d_model"], cfg["n_layers"], cfg["d_inner"], cfg["d_state"],
                          cfg["dt_rank"], cfg["conv_width"], 0)


def ssm_model_decode_workspace_size(desc) -> int:
    n = ctypes.c_size_t(0)
    _check("ssm_model_decode_workspace_size",
           lib().ssm_model_decode_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return int(n.value)


class ModelLayers:
    """The host array of per-block weight pointers for ssm_model_decode_step,
    built once from device tensors (keys LAYER_FIELDS) and kept with them."""

    def __init__(self, layers):
        self.tensors = [dict(lay) for lay in layers]
        arr = (ssm_layer_weights * len(layers))()
        for i, lay in enumerate(self.tensors):
            for f in LAYER_FIELDS:
                t = lay.get(f)
                setattr(arr[i], f, None if t is None else _f32(t, f).value)
        self.array = arr


def ssm_model_decode_step(desc, emb, layers, tokens, h, conv_state, logits=None, norm_f_w=None, norm_f_b=None,
                          workspace=None, stream=None):
    """One token for every stream through the whole model.  layers is a
    ModelLayers; tokens int32 [S] on the device; h [n_layers, S, d_inner, N]
    and conv_state [n_layers, S, W-1, d_inner] (float32) are updated in place.
    Returns logits [S, vocab]."""
    S, V = desc.nstreams, desc.vocab
    if logits is None:
        logits = _alloc((S, V), torch.float32, tokens.device, stream)
    ws = workspace
    if ws is None:
        ws = _alloc(ssm_model_decode_workspace_size(desc), torch.uint8, tokens.device, stream, returned=False)
    _check("ssm_model_decode_step", lib().ssm_model_decode_step(
        ctypes.byref(desc), _f32(emb, "emb"), _f32(norm_f_w, "norm_f_w"), _f32(norm_f_b, "norm_f_b"),
        layers.array, _ptr(tokens, torch.int32, "tokens"), _f32(h, "h"), _f32(conv_state, "conv_state"),
        _f32(logits, "logits"), _ptr(ws, None, "workspace"), ctypes.c_size_t(ws.numel()), _stream(stream)))
    return logits


# --------------------------------------------------- training operators
# These calls run on the device of their tensors, whichever device is current;
# `stream` (default: that device's current stream) must belong to it.  What a
# call allocates itself (outputs not passed in, a workspace) is allocated on the
# stream it runs on: memory that was freed on the current stream may still be
# written by work queued there.  A call on a small tensor is all host time, so
# the checks are plain comparisons in a row.
def _bad(t, dev, dtype, shape, name):
    """Raises for a tensor that is not one of `shape`, `dtype` on `dev`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != dev:
        raise ValueError("%s must be on %s, got %s" % (name, dev, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _dev_ptr(t, dev, dtype, shape, name):
    """Device address of a contiguous tensor on `dev` (None: 0, absent)."""
    if t is None:
        return 0
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.device != dev
            or not t.is_contiguous()):
        _bad(t, dev, dtype, shape, name)
    return t.data_ptr()


def _rows_ptr(t, dev, dtype, shape, name):
    """Address and row stride of [.., D]: values of a row contiguous, rows at
    one stride (None: 0, 0; stride 0: contiguous)."""
    if t is None:
        return 0, 0
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.device != dev:
        _bad(t, dev, dtype, shape, name)
    if t.is_contiguous():
        return t.data_ptr(), 0
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("the values of a row of %s must be contiguous" % name)
    stride = None
    span = 1
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * span:
            raise ValueError("the rows of %s must lie at one stride" % name)
        span *= n
    if stride is None:
        return t.data_ptr(), 0
    if stride < t.shape[-1]:
        raise ValueError("the rows of %s must not overlap" % name)
    return t.data_ptr(), stride


def _io_rows(t, name):
    """Device, dtype, io code, shape and row count of the tensor a call goes by."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    dev, shape = t.device, t.shape
    if dev.type != "cuda":
        raise ValueError("%s must be a device tensor" % name)
    if not shape:
        raise ValueError("%s must have at least one dimension" % name)
    return dev, t.dtype, _io_code(t), shape, t.numel() // shape[-1] if shape[-1] else 0


def _on(dev):
    """Makes `dev` current for a call on another device's tensors."""
    return _HERE_ALREADY if dev.index == _current_device() else torch.cuda.device(dev)


_HERE_ALREADY = contextlib.nullcontext()

# The current stream's handle and the current device as plain numbers; the
# public calls build an object each time (1.9 us of a 10 us call).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_stream(dev, stream):
    """The handle of `stream`, of dev's current stream without one."""
    if stream is None:
        return _current_stream(dev.index)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != dev:
            raise ValueError("stream is on %s, the tensors on %s" % (stream.device, dev))
        return stream.cuda_stream
    return int(stream)


def _new(shape, dtype, dev, stream, handle, returned=True):
    """An uninitialised tensor for a call on `stream`, whose handle is `handle`,
    from that stream's own memory.  A returned one is the caller's on the
    current stream too, so its memory is not used again before both are done."""
    if stream is None or handle == _current_stream(dev.index):
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device=dev)
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if returned and t.numel():
        t.record_stream(here)
    return t


def _given_workspace(ws, dev):
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    if ws.device != dev:
        raise ValueError("workspace must be on %s, got %s" % (dev, ws.device))


def ssm_layer_norm_fwd(x, weight=None, bias=None, residual=None, residual_out=None, mean=None, rstd=None, y=None,
                       eps=1e-5, stream=None):
    """LayerNorm of x (+ residual) over the last axis; x [.., D] in the io
    dtype, rows at one stride.  Writes residual_out (the sum), mean and rstd
    (float32, one per row) when passed; returns y."""
    dev, t, io, shape, T = _io_rows(x, "x")
    rows, vec, f32 = shape[:-1], shape[-1:], torch.float32
    with _on(dev):
        handle = _on_stream(dev, stream)
        if y is None:
            y = _new(shape, t, dev, stream, handle)
        px, sx = _rows_ptr(x, dev, t, shape, "x")
        pr, sr = _rows_ptr(residual, dev, t, shape, "residual")
        po, so = _rows_ptr(residual_out, dev, t, shape, "residual_out")
        py, sy = _rows_ptr(y, dev, t, shape, "y")
        desc = ssm_norm_desc(T, shape[-1], sx, sr, so, sy, io, eps)
        _check("ssm_layer_norm_fwd", lib().ssm_layer_norm_fwd(
            desc, px, pr, _dev_ptr(weight, dev, f32, vec, "weight"), _dev_ptr(bias, dev, f32, vec, "bias"), po, py,
            _dev_ptr(mean, dev, f32, rows, "mean"), _dev_ptr(rstd, dev, f32, rows, "rstd"), handle))
    return y


def ssm_layer_norm_bwd_workspace_size(desc) -> int:
    n = ctypes.c_size_t(0)
    _check("ssm_layer_norm_bwd_workspace_size", lib().ssm_layer_norm_bwd_workspace_size(desc, n))
    return n.value


def ssm_layer_norm_bwd(x, dy, mean, rstd, weight=None, dresidual=None, want=("dx", "dweight", "dbias"), out=None,
                       workspace=None, stream=None):
    """Gradients of ssm_layer_norm_fwd at x (its residual_out where it had a
    residual).  dresidual is the upstream gradient of x itself, added to dx.
    Returns a dict of the wanted gradients, allocated unless given in `out`."""
    dev, t, io, shape, T = _io_rows(x, "x")
    rows, vec, f32 = shape[:-1], shape[-1:], torch.float32
    out = dict(out or {})
    for k in out:
        if k not in ("dx", "dweight", "dbias"):
            raise ValueError("no gradient %r" % (k,))
    with _on(dev):
        handle = _on_stream(dev, stream)
        for k in want:
            if k not in ("dx", "dweight", "dbias"):
                raise ValueError("no gradient %r" % (k,))
            if k not in out:
                out[k] = _new(shape if k == "dx" else vec, t if k == "dx" else f32, dev, stream, handle)
        px, sx = _rows_ptr(x, dev, t, shape, "x")
        pdy, sdy = _rows_ptr(dy, dev, t, shape, "dy")
        pr, sr = _rows_ptr(dresidual, dev, t, shape, "dresidual")
        pdx, sdx = _rows_ptr(out.get("dx"), dev, t, shape, "dx")
        desc = ssm_norm_desc(T, shape[-1], sx, sr, sdx, sdy, io, 1.0)
        if workspace is None:
            workspace = _new(ssm_layer_norm_bwd_workspace_size(desc), torch.uint8, dev, stream, handle, returned=False)
        else:
            _given_workspace(workspace, dev)
        _check("ssm_layer_norm_bwd", lib().ssm_layer_norm_bwd(
            desc, px, _dev_ptr(weight, dev, f32, vec, "weight"), _dev_ptr(mean, dev, f32, rows, "mean"),
            _dev_ptr(rstd, dev, f32, rows, "rstd"), pdy, pr, pdx, _dev_ptr(out.get("dweight"), dev, f32, vec, "dweight"),
            _dev_ptr(out.get("dbias"), dev, f32, vec, "dbias"), workspace.data_ptr(), workspace.numel(),
            handle))
    return out


def ssm_token_logp_fwd(logits, targets, stats=None, logp=None, stream=None):
    """Log-probability of each row's target: logits [.., V] in the io dtype,
    rows at one stride; targets int32 [..], a negative one for a row without a
    target (its logp is 0).  Writes stats [.., 2] (what the backward takes) when
    passed; returns logp, float32 [..]."""
    dev, t, io, shape, T = _io_rows(logits, "logits")
    rows, f32 = shape[:-1], torch.float32
    with _on(dev):
        handle = _on_stream(dev, stream)
        if logp is None:
            logp = _new(rows, f32, dev, stream, handle)
        pz, sz = _rows_ptr(logits, dev, t, shape, "logits")
        desc = ssm_logp_desc(T, shape[-1], sz, 0, io, 0)
        _check("ssm_token_logp_fwd", lib().ssm_token_logp_fwd(
            desc, pz, _dev_ptr(targets, dev, torch.int32, rows, "targets"), _dev_ptr(logp, dev, f32, rows, "logp"),
            _dev_ptr(stats, dev, f32, rows + (2,), "stats"), handle))
    return logp


def ssm_token_logp_bwd(logits, targets, stats, dlogp, dlogits=None, stream=None):
    """Gradient of sum(logp * dlogp) with respect to the logits; stats from
    ssm_token_logp_fwd.  dlogits may be logits itself.  Returns dlogits."""
    dev, t, io, shape, T = _io_rows(logits, "logits")
    rows, f32 = shape[:-1], torch.float32
    with _on(dev):
        handle = _on_stream(dev, stream)
        if dlogits is None:
            dlogits = _new(shape, t, dev, stream, handle)
        pz, sz = _rows_ptr(logits, dev, t, shape, "logits")
        pd, sd = _rows_ptr(dlogits, dev, t, shape, "dlogits")
        desc = ssm_logp_desc(T, shape[-1], sz, sd, io, 0)
        _check("ssm_token_logp_bwd", lib().ssm_token_logp_bwd(
            desc, pz, _dev_ptr(targets, dev, torch.int32, rows, "targets"),
            _dev_ptr(stats, dev, f32, rows + (2,), "stats"), _dev_ptr(dlogp, dev, f32, rows, "dlogp"), pd,
            handle))
    return dlogits


def ssm_policy_loss_workspace_size(desc) -> int:
    n = ctypes.c_size_t(0)
    _check("ssm_policy_loss_workspace_size", lib().ssm_policy_loss_workspace_size(desc, n))
    return n.value


def ssm_policy_loss(logits, targets, old_logp, advantages, ref_logp=None, weights=None, clip_low=0.2, clip_high=0.2,
                    kl_beta=0.0, reduction=SSM_REDUCE_MEAN, grad_scale=1.0, logp=None, dlogits=None, loss=None,
                    workspace=None, stream=None):
    """Clipped policy loss with a KL term over logits [.., V] (rows at one
    stride); targets int32 and the float32 old_logp (None: the present policy),
    advantages, ref_logp and weights are [..].  A token with a negative target
    or weight 0 is left out.  Writes logp, and the gradient dlogits (which may
    be logits itself) when passed; returns loss, float32 [4]: the loss, its
    policy term, the KL term, the share of clipped tokens."""
    dev, t, io, shape, T = _io_rows(logits, "logits")
    rows, f32 = shape[:-1], torch.float32
    with _on(dev):
        handle = _on_stream(dev, stream)
        if loss is None:
            loss = _new(4, f32, dev, stream, handle)
        pz, sz = _rows_ptr(logits, dev, t, shape, "logits")
        pd, sd = _rows_ptr(dlogits, dev, t, shape, "dlogits")
        desc = ssm_policy_desc(T, shape[-1], sz, sd, clip_low, clip_high, kl_beta, grad_scale, io, reduction)
        if workspace is None:
            workspace = _new(ssm_policy_loss_workspace_size(desc), torch.uint8, dev, stream, handle, returned=False)
        else:
            _given_workspace(workspace, dev)
        _check("ssm_policy_loss", lib().ssm_policy_loss(
            desc, pz, _dev_ptr(targets, dev, torch.int32, rows, "targets"),
            _dev_ptr(old_logp, dev, f32, rows, "old_logp"), _dev_ptr(ref_logp, dev, f32, rows, "ref_logp"),
            _dev_ptr(advantages, dev, f32, rows, "advantages"), _dev_ptr(weights, dev, f32, rows, "weights"),
            _dev_ptr(loss, dev, f32, (4,), "loss"), _dev_ptr(logp, dev, f32, rows, "logp"), pd,
            workspace.data_ptr(), workspace.numel(), handle))
    return loss


class GradList:
    """The host list of gradients for ssm_clip_grad_norm, built once and kept
    with them (it holds the tensors).  `out` gives a tensor for each clipped
    gradient, float32 or bfloat16 whatever the gradient's own type (None among
    them: that gradient only counts in the norm); without it gradients are
    clipped in place."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = list(self.grads if out is None else out)
        if len(self.out) != len(self.grads):
            raise ValueError("%d outputs for %d gradients" % (len(self.out), len(self.grads)))
        if not self.grads:
            raise ValueError("no gradients")
        for i, t in enumerate(self.grads + self.out):
            if not isinstance(t, torch.Tensor) and (t is not None or i < len(self.grads)):
                raise TypeError("gradients and outputs must be torch.Tensors")
        self.device = self.grads[0].device
        if self.device.type != "cuda":
            raise ValueError("gradients must be device tensors")
        self._read()

    def _read(self):
        arr = (ssm_grad * len(self.grads))()
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            pg = _dev_ptr(g, self.device, g.dtype, g.shape, "grads[%d]" % i)
            po = 0 if o is None else _dev_ptr(o, self.device, o.dtype, g.shape, "out[%d]" % i)
            arr[i] = ssm_grad(pg, po, g.numel(), _io_code(g), _io_code(g if o is None else o))
        n = ctypes.c_size_t(0)
        _check("ssm_clip_grad_norm_workspace_size",
               lib().ssm_clip_grad_norm_workspace_size(arr, len(self.grads), ctypes.byref(n)))
        self.array, self.workspace_size = arr, int(n.value)
        self._tensors = self.grads + [o for g, o in zip(self.grads, self.out) if o is not None and o is not g]
        self._where = [t.data_ptr() for t in self._tensors]
        # held, so that an address found again is still the same memory
        self._memory = [t.untyped_storage() for t in self._tensors]

    def refresh(self):
        """Looks the tensors up again if the memory of one was replaced.  The
        calls do this themselves (60 ns a tensor: 3 us of a 13.6 us call for 25
        gradients with an output each)."""
        if [t.data_ptr() for t in self._tensors] != self._where:
            self._read()


def ssm_clip_grad_norm_workspace_size(grads) -> int:
    """Bytes of workspace for a GradList."""
    grads.refresh()
    return grads.workspace_size


def ssm_clip_grad_norm(grads, max_norm, norm=None, workspace=None, stream=None):
    """Clips the gradients of a GradList by their global norm; max_norm infinite
    only measures it (factor 1).  Returns norm, float32 [2]: the norm before clipping and
    the factor applied."""
    if not isinstance(grads, GradList):
        raise TypeError("grads must be a GradList")
    grads.refresh()
    dev = grads.device
    with _on(dev):
        handle = _on_stream(dev, stream)
        if norm is None:
            norm = _new(2, torch.float32, dev, stream, handle)
        if workspace is None:
            workspace = _new(grads.workspace_size, torch.uint8, dev, stream, handle, returned=False)
        else:
            _given_workspace(workspace, dev)
        _check("ssm_clip_grad_norm", lib().ssm_clip_grad_norm(
            grads.array, len(grads.grads), max_norm, _dev_ptr(norm, dev, torch.float32, (2,), "norm"),
            workspace.data_ptr(), workspace.numel(), handle))
    return norm
