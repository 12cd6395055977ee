"""Python binding of libgc (include/gc.h): argument marshalling only.

Every function here turns torch tensors into device pointers, a descriptor
and the current HIP stream, and calls the C entry point of the same name;
all computation happens in the HIP kernels behind it.  There is no fallback:
if ``libgc.so`` is missing or a call fails, an exception is raised.
"""
import ctypes
import math
import os

import torch
from torch._C._dynamo.guards import TensorGuards

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgc.so")

GC_OK, GC_ERR_INVALID_ARG, GC_ERR_UNSUPPORTED, GC_ERR_WORKSPACE, GC_ERR_HIP = range(5)
GC_F32, GC_BF16 = 0, 1
GC_OP_FWD, GC_OP_BWD_DATA, GC_OP_BWD_WEIGHT, GC_OP_BWD_BIAS, GC_OP_BWD = 0, 1, 2, 3, 4
GC_OP_BWD_WEIGHT_BIAS = 5

EXPORTED = (
    "gc_conv_out_dims", "gc_conv_workspace_bytes", "gc_conv_fwd", "gc_conv_bwd_data",
    "gc_conv_bwd_weight", "gc_status_string", "gc_fastdiv_selfcheck", "gc_version",
    "gc_set_kernel_policy", "gc_conv_fwd_bias", "gc_conv_bwd_bias", "gc_conv_bwd",
    "gc_conv_plan_name", "gc_conv_fwd_noalloc", "gc_conv_bwd_weight_bias",
    "gc_embed_fwd", "gc_embed_bwd", "gc_embed_workspace_bytes", "gc_group_norm_fwd",
    "gc_group_norm_bwd", "gc_group_norm_workspace_bytes", "gc_grad_norm", "gc_grad_clip",
    "gc_grad_clip_workspace_bytes", "gc_group_norm_plan_name", "gc_embed_plan_name",
)
GC_I32, GC_I64, GC_U8 = 0, 1, 2
GC_NCHW, GC_NHWC = 0, 1
GC_ACT_NONE, GC_ACT_RELU, GC_ACT_SILU, GC_ACT_GELU = range(4)
GC_POLICY_AUTO, GC_POLICY_GENERIC = 0, 1


class GcError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)}")


class gc_conv_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "IC", "H", "W", "OC", "KH", "KW", "stride")]


class gc_embed_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("tokens", ctypes.c_int), ("V", ctypes.c_int),
                ("D", ctypes.c_int), ("itype", ctypes.c_int), ("ld", ctypes.c_int64),
                ("ld_tok", ctypes.c_int64)]


class gc_norm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "C", "H", "W", "groups", "layout", "act")] + \
               [("eps", ctypes.c_float)]


class gc_tensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


_lib = None


def lib():
    """The loaded libgc.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libgc.so not found at {LIB_PATH}; run __graft_entry__.build() "
                           "(python -m backward_implicit_gemm_amd.build)")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i, dp = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.POINTER(gc_conv_desc)
    L.gc_conv_out_dims.argtypes = [dp, ctypes.POINTER(i), ctypes.POINTER(i)]
    L.gc_conv_out_dims.restype = i
    L.gc_conv_workspace_bytes.argtypes = [i, dp, i]
    L.gc_conv_workspace_bytes.restype = sz
    L.gc_conv_fwd.argtypes = [vp, vp, vp, vp, sz, dp, i, i, vp]
    L.gc_conv_fwd.restype = i
    L.gc_conv_fwd_noalloc.argtypes = [vp, vp, vp, dp, i, i, vp]
    L.gc_conv_fwd_noalloc.restype = i
    L.gc_conv_fwd_bias.argtypes = [vp, vp, vp, vp, vp, sz, dp, i, i, vp]
    L.gc_conv_fwd_bias.restype = i
    L.gc_conv_bwd_bias.argtypes = [vp, vp, vp, vp, sz, dp, i, i, vp]
    L.gc_conv_bwd_bias.restype = i
    L.gc_conv_bwd_data.argtypes = [vp, vp, vp, vp, vp, sz, dp, i, i, vp]
    L.gc_conv_bwd_data.restype = i
    L.gc_conv_bwd_weight.argtypes = [vp, vp, vp, vp, vp, sz, dp, i, i, vp]
    L.gc_conv_bwd_weight.restype = i
    L.gc_conv_bwd_weight_bias.argtypes = [vp, vp, vp, vp, vp, vp, sz, dp, i, i, vp]
    L.gc_conv_bwd_weight_bias.restype = i
    L.gc_conv_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, dp, i, i, vp]
    L.gc_conv_bwd.restype = i
    L.gc_status_string.argtypes = [i]
    L.gc_status_string.restype = ctypes.c_char_p
    L.gc_fastdiv_selfcheck.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
    L.gc_fastdiv_selfcheck.restype = ctypes.c_int64
    L.gc_conv_plan_name.argtypes = [i, dp, i, ctypes.c_char_p, sz]
    L.gc_conv_plan_name.restype = i
    L.gc_version.argtypes = []
    L.gc_version.restype = i
    L.gc_set_kernel_policy.argtypes = [i]
    L.gc_set_kernel_policy.restype = i
    f, ep, np_ = ctypes.c_float, ctypes.POINTER(gc_embed_desc), ctypes.POINTER(gc_norm_desc)
    L.gc_embed_fwd.argtypes = [vp, vp, vp, ep, f, i, vp]
    L.gc_embed_fwd.restype = i
    L.gc_embed_workspace_bytes.argtypes = [ep, i]
    L.gc_embed_workspace_bytes.restype = sz
    L.gc_embed_bwd.argtypes = [vp, vp, vp, vp, sz, ep, f, i, vp]
    L.gc_embed_bwd.restype = i
    L.gc_group_norm_workspace_bytes.argtypes = [i, np_, i]
    L.gc_group_norm_workspace_bytes.restype = sz
    L.gc_group_norm_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, np_, i, i, vp]
    L.gc_group_norm_fwd.restype = i
    L.gc_group_norm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, np_, i, i, vp]
    L.gc_group_norm_bwd.restype = i
    L.gc_grad_clip_workspace_bytes.argtypes = [i]
    L.gc_grad_clip_workspace_bytes.restype = sz
    L.gc_group_norm_plan_name.argtypes = [i, np_, i, ctypes.c_char_p, sz]
    L.gc_group_norm_plan_name.restype = i
    L.gc_embed_plan_name.argtypes = [ep, i, ctypes.c_char_p, sz]
    L.gc_embed_plan_name.restype = i
    tp = ctypes.POINTER(gc_tensor)
    L.gc_grad_norm.argtypes = [tp, i, f, vp, vp, sz, vp]
    L.gc_grad_norm.restype = i
    L.gc_grad_clip.argtypes = [tp, i, f, f, f, vp, vp, sz, vp]
    L.gc_grad_clip.restype = i
    _lib = L
    return L


def gc_set_kernel_policy(policy):
    """Process-wide kernel selection (GC_POLICY_AUTO or GC_POLICY_GENERIC);
    returns the previous policy."""
    prev = lib().gc_set_kernel_policy(int(policy))
    if prev < 0:
        raise ValueError(f"unknown kernel policy {policy}")
    return prev


def status_string(status):
    return lib().gc_status_string(int(status)).decode()


def make_desc(B, IC, H, W, OC, KH, KW, stride):
    return gc_conv_desc(int(B), int(IC), int(H), int(W), int(OC), int(KH), int(KW), int(stride))


def desc_from(x_shape, w_shape, stride):
    B, IC, H, W = (int(v) for v in x_shape)
    OC, IC2, KH, KW = (int(v) for v in w_shape)
    if IC2 != IC:
        raise ValueError(f"x has {IC} channels but w expects {IC2}")
    return make_desc(B, IC, H, W, OC, KH, KW, stride)


def gc_conv_out_dims(desc):
    oh, ow = ctypes.c_int(0), ctypes.c_int(0)
    st = lib().gc_conv_out_dims(ctypes.byref(desc), ctypes.byref(oh), ctypes.byref(ow))
    if st != GC_OK:
        raise GcError("gc_conv_out_dims", st)
    return oh.value, ow.value


def gc_conv_workspace_bytes(op, desc, dtype):
    return int(lib().gc_conv_workspace_bytes(int(op), ctypes.byref(desc), int(dtype)))


def gc_conv_plan_name(op, desc, dtype):
    """The kernels `op` would run for this problem (host only, enqueues nothing)."""
    buf = ctypes.create_string_buffer(256)
    st = lib().gc_conv_plan_name(int(op), ctypes.byref(desc), int(dtype), buf, len(buf))
    _check("gc_conv_plan_name", st)
    return buf.value.decode()


def _dtype_code(t):
    if t.dtype == torch.float32:
        return GC_F32
    if t.dtype == torch.bfloat16:
        return GC_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; expected float32 or bfloat16")


def _expect(t, name, shape):
    """Raises ValueError unless tensor t (if given) has exactly this shape;
    checked before anything touches the device, so a wrongly sized buffer
    never reaches the kernels."""
    if t is None:
        return
    if tuple(t.shape) != tuple(int(v) for v in shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _y_shape(desc):
    oh, ow = gc_conv_out_dims(desc)
    return (desc.B, desc.OC, oh, ow)


def _dev(t, name, dtype):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if _dtype_code(t) != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, the call uses another")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ws(workspace):
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    return ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()


def _check(fn, st):
    if st != GC_OK:
        raise GcError(fn, st)


def workspace_for(op, desc, dtype, device="cuda"):
    """A device buffer of the size gc_conv_workspace_bytes asks for (or None)."""
    n = gc_conv_workspace_bytes(op, desc, dtype)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device)


def gc_conv_fwd(x, w, y, relu, stride, workspace=None, stream=None):
    """y = relu?(conv(x, w)) via the C entry point gc_conv_fwd."""
    dt = _dtype_code(x)
    desc = desc_from(x.shape, w.shape, stride)
    _expect(y, "y", _y_shape(desc))
    wp, wn = _ws(workspace)
    st = lib().gc_conv_fwd(_dev(x, "x", dt), _dev(w, "w", dt), _dev(y, "y", dt), wp, wn,
                           ctypes.byref(desc), int(relu), dt, _stream(stream))
    _check("gc_conv_fwd", st)
    return y


def gc_conv_fwd_noalloc(x, w, y, relu, stride, stream=None):
    """y = relu?(conv(x, w)) via gc_conv_fwd_noalloc (no workspace: the
    library's static per-GPU scratch)."""
    dt = _dtype_code(x)
    desc = desc_from(x.shape, w.shape, stride)
    _expect(y, "y", _y_shape(desc))
    st = lib().gc_conv_fwd_noalloc(_dev(x, "x", dt), _dev(w, "w", dt), _dev(y, "y", dt),
                                   ctypes.byref(desc), int(relu), dt, _stream(stream))
    _check("gc_conv_fwd_noalloc", st)
    return y


def gc_conv_fwd_bias(x, w, bias, y, relu, stride, workspace=None, stream=None):
    """y = relu?(conv(x, w) + bias) via the C entry point gc_conv_fwd_bias."""
    dt = _dtype_code(x)
    desc = desc_from(x.shape, w.shape, stride)
    _expect(y, "y", _y_shape(desc))
    _expect(bias, "bias", (desc.OC,))
    wp, wn = _ws(workspace)
    st = lib().gc_conv_fwd_bias(_dev(x, "x", dt), _dev(w, "w", dt), _dev(bias, "bias", dt),
                                _dev(y, "y", dt), wp, wn, ctypes.byref(desc), int(relu), dt,
                                _stream(stream))
    _check("gc_conv_fwd_bias", st)
    return y


def gc_conv_bwd_bias(dy, y_mask, db, relu, x_shape, w_shape, stride, workspace, stream=None):
    """db[oc] = sum of dy (masked by y_mask > 0 when relu) via gc_conv_bwd_bias."""
    dt = _dtype_code(dy)
    desc = desc_from(x_shape, w_shape, stride)
    ys = _y_shape(desc)
    _expect(dy, "dy", ys)
    _expect(y_mask, "y_mask", ys)
    _expect(db, "db", (desc.OC,))
    wp, wn = _ws(workspace)
    st = lib().gc_conv_bwd_bias(_dev(dy, "dy", dt), _dev(y_mask, "y_mask", dt), _dev(db, "db", dt),
                                wp, wn, ctypes.byref(desc), int(relu), dt, _stream(stream))
    _check("gc_conv_bwd_bias", st)
    return db


def gc_conv_bwd_data(dy, w, y_mask, dx, relu, stride, workspace=None, stream=None):
    """dx from dy (masked by y_mask > 0 when relu) via gc_conv_bwd_data."""
    dt = _dtype_code(dy)
    desc = desc_from(dx.shape, w.shape, stride)
    ys = _y_shape(desc)
    _expect(dy, "dy", ys)
    _expect(y_mask, "y_mask", ys)
    wp, wn = _ws(workspace)
    st = lib().gc_conv_bwd_data(_dev(dy, "dy", dt), _dev(w, "w", dt), _dev(y_mask, "y_mask", dt),
                                _dev(dx, "dx", dt), wp, wn, ctypes.byref(desc), int(relu), dt,
                                _stream(stream))
    _check("gc_conv_bwd_data", st)
    return dx


def gc_conv_bwd_weight(x, dy, y_mask, dw, relu, stride, workspace, stream=None):
    """dw from x and dy (masked by y_mask > 0 when relu) via gc_conv_bwd_weight."""
    dt = _dtype_code(x)
    desc = desc_from(x.shape, dw.shape, stride)
    ys = _y_shape(desc)
    _expect(dy, "dy", ys)
    _expect(y_mask, "y_mask", ys)
    wp, wn = _ws(workspace)
    st = lib().gc_conv_bwd_weight(_dev(x, "x", dt), _dev(dy, "dy", dt), _dev(y_mask, "y_mask", dt),
                                  _dev(dw, "dw", dt), wp, wn, ctypes.byref(desc), int(relu), dt,
                                  _stream(stream))
    _check("gc_conv_bwd_weight", st)
    return dw


def gc_conv_bwd_weight_bias(x, dy, y_mask, dw, db, relu, stride, workspace, stream=None):
    """dw and db together (dy masked by y_mask > 0 when relu) via gc_conv_bwd_weight_bias."""
    dt = _dtype_code(x)
    desc = desc_from(x.shape, dw.shape, stride)
    ys = _y_shape(desc)
    _expect(dy, "dy", ys)
    _expect(y_mask, "y_mask", ys)
    _expect(db, "db", (desc.OC,))
    wp, wn = _ws(workspace)
    st = lib().gc_conv_bwd_weight_bias(_dev(x, "x", dt), _dev(dy, "dy", dt),
                                       _dev(y_mask, "y_mask", dt), _dev(dw, "dw", dt),
                                       _dev(db, "db", dt), wp, wn, ctypes.byref(desc), int(relu),
                                       dt, _stream(stream))
    _check("gc_conv_bwd_weight_bias", st)
    return dw, db


def gc_conv_bwd(x, w, dy, y_mask, dx, dw, relu, stride, workspace, stream=None):
    """dx and dw together (dy masked by y_mask > 0 when relu) via gc_conv_bwd."""
    dt = _dtype_code(x)
    desc = desc_from(x.shape, w.shape, stride)
    ys = _y_shape(desc)
    _expect(dy, "dy", ys)
    _expect(y_mask, "y_mask", ys)
    _expect(dx, "dx", x.shape)
    _expect(dw, "dw", w.shape)
    wp, wn = _ws(workspace)
    st = lib().gc_conv_bwd(_dev(x, "x", dt), _dev(w, "w", dt), _dev(dy, "dy", dt),
                           _dev(y_mask, "y_mask", dt), _dev(dx, "dx", dt), _dev(dw, "dw", dt),
                           wp, wn, ctypes.byref(desc), int(relu), dt, _stream(stream))
    _check("gc_conv_bwd", st)
    return dx, dw


class Conv:
    """One convolution layer's three passes with their workspaces (torch
    allocates; the library only receives pointers), one each for the stream the helper
    was made on, see _Workspace."""

    def __init__(self, x_shape, w_shape, stride, relu, dtype, device="cuda"):
        self.stride, self.relu = int(stride), int(relu)
        self.dt = {torch.float32: GC_F32, torch.bfloat16: GC_BF16}[dtype]
        self.dtype = dtype
        self.desc = desc_from(x_shape, w_shape, stride)
        self.x_shape, self.w_shape = tuple(x_shape), tuple(w_shape)
        OH, OW = gc_conv_out_dims(self.desc)
        self.y_shape = (x_shape[0], w_shape[0], OH, OW)
        self.device = _device(device)
        self.ws = {op: _Workspace(gc_conv_workspace_bytes(op, self.desc, self.dt), self.device)
                   for op in (GC_OP_FWD, GC_OP_BWD_DATA, GC_OP_BWD_WEIGHT, GC_OP_BWD_BIAS,
                              GC_OP_BWD, GC_OP_BWD_WEIGHT_BIAS)}

    def _scratch(self, op, stream):
        return self.ws[op].on(_raw_stream(stream, self.device))[2]

    def fwd(self, x, w, y, stream=None):
        return gc_conv_fwd(x, w, y, self.relu, self.stride, self._scratch(GC_OP_FWD, stream), stream)

    def bwd_data(self, dy, w, y, dx, stream=None):
        return gc_conv_bwd_data(dy, w, y if self.relu else None, dx, self.relu, self.stride,
                                self._scratch(GC_OP_BWD_DATA, stream), stream)

    def bwd_weight(self, x, dy, y, dw, stream=None):
        return gc_conv_bwd_weight(x, dy, y if self.relu else None, dw, self.relu, self.stride,
                                  self._scratch(GC_OP_BWD_WEIGHT, stream), stream)

    def bwd(self, x, w, dy, y, dx, dw, stream=None):
        return gc_conv_bwd(x, w, dy, y if self.relu else None, dx, dw, self.relu, self.stride,
                           self._scratch(GC_OP_BWD, stream), stream)

    def fwd_bias(self, x, w, bias, y, stream=None):
        return gc_conv_fwd_bias(x, w, bias, y, self.relu, self.stride, self._scratch(GC_OP_FWD, stream), stream)

    def bwd_weight_bias(self, x, dy, y, dw, db, stream=None):
        return gc_conv_bwd_weight_bias(x, dy, y if self.relu else None, dw, db, self.relu,
                                       self.stride, self._scratch(GC_OP_BWD_WEIGHT_BIAS, stream), stream)

    def bwd_bias(self, dy, y, db, stream=None):
        return gc_conv_bwd_bias(dy, y if self.relu else None, db, self.relu, self.x_shape,
                                self.w_shape, self.stride, self._scratch(GC_OP_BWD_BIAS, stream), stream)


# ---------------------------------------------------------------------------
# The operators around the convolutions
#
# A call is enqueued on `stream` (a torch stream or a raw handle), torch's current
# one if None.  Its tensors are the caller's: as with any work on a second stream,
# that stream first has to wait for what fills them, and they have to live (or be
# recorded on it with record_stream) until it is done with them.  What a helper
# allocates by itself follows the call's stream.
# ---------------------------------------------------------------------------
_ACTS = {"none": GC_ACT_NONE, "relu": GC_ACT_RELU, "silu": GC_ACT_SILU, "gelu": GC_ACT_GELU}
_LAYOUTS = {"nchw": (GC_NCHW, torch.contiguous_format), "nhwc": (GC_NHWC, torch.channels_last)}
_DTYPES = {torch.float32: GC_F32, torch.bfloat16: GC_BF16}
_INT_MAX = 2 ** 31 - 1
_INDEX_TYPES = {torch.int32: GC_I32, torch.int64: GC_I64, torch.uint8: GC_U8}


def _code(dtype):
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}; expected float32 or bfloat16")
    return _DTYPES[dtype]


def _named(table, value, what):
    if value not in table:
        raise ValueError(f"unknown {what} {value!r}; expected one of {', '.join(table)}")
    return table[value]


def _arg(t, name, dtype, shape, device, fmt=torch.contiguous_format):
    """Address of tensor t after checking its shape, dtype, layout and device,
    in this order."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous(memory_format=fmt):
        raise ValueError(f"{name} must be dense in {fmt}")
    return _on(t, name, device)


def _on(t, name, device):
    """Address of tensor t, which has to be on this device."""
    if t.device != device or device.type != "cuda":
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        raise ValueError(f"{name} is on {t.device}, the helper is for {device}")
    return t.data_ptr()


def _device(device):
    """The device with its index, where there is one (a helper may be made
    without a GPU; its calls then refuse their tensors)."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None and torch.cuda.is_available():
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _raw_stream(stream, device):
    if stream is None:
        # the handle alone: building a Stream object costs as much host time as a launch
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def gc_group_norm_plan_name(op, desc, dtype):
    """The kernels a group norm would run (host only, enqueues nothing)."""
    buf = ctypes.create_string_buffer(256)
    _check("gc_group_norm_plan_name",
           lib().gc_group_norm_plan_name(int(op), ctypes.byref(desc), int(dtype), buf, len(buf)))
    return buf.value.decode()


def gc_embed_plan_name(desc, dtype):
    """The kernels an embedding's gradient would run (host only, enqueues nothing)."""
    buf = ctypes.create_string_buffer(256)
    _check("gc_embed_plan_name", lib().gc_embed_plan_name(ctypes.byref(desc), int(dtype), buf, len(buf)))
    return buf.value.decode()


def _empty(shape, dtype, device, raw):
    """Memory for work on the stream of this handle: torch's allocator gives it to nobody else
    before that stream's work so far is done, however early it is freed."""
    if raw == torch._C._cuda_getCurrentRawStream(device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class _Workspace:
    """A helper's scratch memory of n bytes: one buffer for the stream that was current when
    the helper was made, and for a call on another stream (a captured one among them) memory
    of that stream's own, so that neither a dropped helper nor two streams share a buffer in use."""

    def __init__(self, n, device):
        self.n, self.device, self.home = n, device, None
        self._kept = self._args(torch.empty(n, dtype=torch.uint8, device=device)) if n else (None, 0, None)
        if device.type == "cuda":
            self.home = torch._C._cuda_getCurrentRawStream(device.index)

    def _args(self, t):
        return t.data_ptr(), self.n, t

    def on(self, raw):
        """(address, bytes, owner) for a call on the stream of this handle; the owner has to live
        until the call returns."""
        if not self.n or raw == self.home:
            return self._kept
        return self._args(_empty(self.n, torch.uint8, self.device, raw))


class Embedding:
    """Embedding lookup with scaling and its gradient (gc_embed_fwd and
    gc_embed_bwd) for tokens of shape (rows, tokens) and a table of shape
    (vocab, dim).

    Tokens are int32, int64 or uint8; a token outside [0, vocab) is empty: zeros
    out, no gradient.  ``out`` and ``dout`` have shape (rows, tokens, dim); the
    rows, and those of the tokens, may lie further apart than they are long
    (a part of a wider feature row)."""

    def __init__(self, rows, tokens, vocab, dim, dtype, scale=1.0, device="cuda"):
        self.dtype, self.dt, self.scale = dtype, _code(dtype), float(scale)
        self.device = _device(device)
        self.tok_shape = torch.Size((int(rows), int(tokens)))
        self.out_shape = torch.Size((int(rows), int(tokens), int(dim)))
        self.table_shape = torch.Size((int(vocab), int(dim)))
        # ctypes would cut off what a descriptor's field does not hold
        if int(vocab) < 1 or int(dim) < 1 or int(rows) < 0 or int(tokens) < 0 or \
                int(rows) >= 2 ** 60 or max(int(vocab), int(tokens), int(dim)) > _INT_MAX:
            raise ValueError(f"invalid embedding: rows {rows}, tokens {tokens}, vocab {vocab}, dim {dim}")
        if not math.isfinite(ctypes.c_float(self.scale).value):
            raise ValueError(f"the scale has to be finite in fp32, not {scale}")
        self.desc = gc_embed_desc(int(rows), int(tokens), int(vocab), int(dim), GC_I32,
                                  int(tokens) * int(dim), int(tokens))
        self._ref = ctypes.byref(self.desc)
        self._ws = _Workspace(int(lib().gc_embed_workspace_bytes(self._ref, self.dt)), self.device)

    def _describe(self, tok, rows_like, name):
        """Fills the descriptor from the tokens' type and both row distances."""
        rows, tokens, dim = self.out_shape
        if tok.shape != self.tok_shape:
            raise ValueError(f"tokens has shape {tuple(tok.shape)}, expected {tuple(self.tok_shape)}")
        if tok.dtype not in _INDEX_TYPES:
            raise TypeError(f"tokens has dtype {tok.dtype}; expected int32, int64 or uint8")
        if rows_like.shape != self.out_shape:
            raise ValueError(f"{name} has shape {tuple(rows_like.shape)}, expected {tuple(self.out_shape)}")
        if rows_like.dtype != self.dtype:
            raise TypeError(f"{name} has dtype {rows_like.dtype}, expected {self.dtype}")
        self.desc.itype = _INDEX_TYPES[tok.dtype]
        self.desc.ld_tok = self._distance(tok, "tokens", tokens, (1,))
        self.desc.ld = self._distance(rows_like, name, tokens * dim, (dim, 1))

    @staticmethod
    def _distance(t, name, length, inner):
        """Elements between rows; a row itself has to be dense."""
        if t.is_contiguous():
            return length
        if any(s != want for s, want, n in zip(t.stride()[1:], inner, t.shape[1:]) if n > 1):
            raise ValueError(f"{name} must be dense within a row")
        ld = t.stride(0) if t.shape[0] > 1 else length
        if ld < length:
            raise ValueError(f"the rows of {name} must not overlap")
        return ld

    def fwd(self, tok, table, out, stream=None):
        self._describe(tok, out, "out")
        tp = _arg(table, "table", self.dtype, self.table_shape, self.device)
        st = lib().gc_embed_fwd(_on(tok, "tokens", self.device), tp, _on(out, "out", self.device), self._ref,
                                self.scale, self.dt, _raw_stream(stream, self.device))
        _check("gc_embed_fwd", st)
        return out

    def bwd(self, tok, dout, dtable, stream=None):
        self._describe(tok, dout, "dout")
        dp = _arg(dtable, "dtable", self.dtype, self.table_shape, self.device)
        tp, op = _on(tok, "tokens", self.device), _on(dout, "dout", self.device)
        raw = _raw_stream(stream, self.device)
        ws, n, _owner = self._ws.on(raw)
        st = lib().gc_embed_bwd(tp, op, dp, ws, n, self._ref, self.scale, self.dt, raw)
        _check("gc_embed_bwd", st)
        return dtable


class GroupNorm:
    """Group norm with an activation (gc_group_norm_fwd and gc_group_norm_bwd)
    over tensors of shape (B, C, H, W), in memory NCHW (layout "nchw", as the
    convolutions have it) or channels last ("nhwc": torch's channels_last
    format).

    act is "none", "relu", "silu" or "gelu"; gamma and beta (C) have
    param_dtype, float32 or the storage type, or are None; mean and rstd are
    float32 (B, groups), in the forward None where they are not wanted."""

    def __init__(self, shape, groups, act, dtype, layout="nchw", eps=1e-5, param_dtype=torch.float32,
                 device="cuda"):
        self.dtype, self.dt = dtype, _code(dtype)
        self.param_dtype, self.pt = param_dtype, _code(param_dtype)
        if self.pt not in (GC_F32, self.dt):
            raise TypeError(f"param_dtype {param_dtype} is neither float32 nor the storage type {dtype}")
        code, self.format = _named(_LAYOUTS, layout, "layout")
        self.device = _device(device)
        B, C, H, W = (int(v) for v in shape)
        self.shape, self.param_shape = torch.Size((B, C, H, W)), torch.Size((C,))
        self.stat_shape = torch.Size((B, int(groups)))
        if min(B, C, H, W, int(groups)) < 1 or max(B, C, H, W) > _INT_MAX or C % int(groups):
            raise ValueError(f"invalid group norm: shape {tuple(self.shape)}, {groups} groups")
        self.desc = gc_norm_desc(B, C, H, W, int(groups), code, _named(_ACTS, act, "act"), float(eps))
        self._ref = ctypes.byref(self.desc)
        need = lib().gc_group_norm_workspace_bytes
        self._ws = _Workspace(max(int(need(op, self._ref, self.dt)) for op in (GC_OP_FWD, GC_OP_BWD)),
                              self.device)

    def _image(self, t, name):
        return _arg(t, name, self.dtype, self.shape, self.device, self.format)

    def _param(self, t, name):
        return None if t is None else _arg(t, name, self.param_dtype, self.param_shape, self.device)

    def _stat(self, t, name):
        return None if t is None else _arg(t, name, torch.float32, self.stat_shape, self.device)

    def fwd(self, x, gamma, beta, y, mean=None, rstd=None, stream=None):
        args = (self._image(x, "x"), self._param(gamma, "gamma"), self._param(beta, "beta"),
                self._image(y, "y"), self._stat(mean, "mean"), self._stat(rstd, "rstd"))
        raw = _raw_stream(stream, self.device)
        ws, n, _owner = self._ws.on(raw)
        st = lib().gc_group_norm_fwd(*args, ws, n, self._ref, self.dt, self.pt, raw)
        _check("gc_group_norm_fwd", st)
        return y, mean, rstd

    def bwd(self, x, gamma, beta, dy, mean, rstd, dx, dgamma=None, dbeta=None, stream=None):
        args = (self._image(x, "x"), self._param(gamma, "gamma"), self._param(beta, "beta"),
                self._image(dy, "dy"), self._stat(mean, "mean"), self._stat(rstd, "rstd"),
                self._image(dx, "dx"), self._param(dgamma, "dgamma"), self._param(dbeta, "dbeta"))
        raw = _raw_stream(stream, self.device)
        ws, n, _owner = self._ws.on(raw)
        st = lib().gc_group_norm_bwd(*args, ws, n, self._ref, self.dt, self.pt, raw)
        _check("gc_group_norm_bwd", st)
        return dx, dgamma, dbeta


class _Tensors:
    """Tensors a call reads or writes by address: their memory may be replaced
    (``t.data = ...``), their size, type, layout and device may not."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self.kinds = [self._kind(t) for t in self.tensors]
        self._guard()

    @staticmethod
    def _kind(t):
        return t.numel(), t.dtype, t.device, t.is_contiguous()

    def _guard(self):
        # dtype, device, sizes and strides of every tensor in one C++ call: read one by one from
        # Python they cost 3 us more a call for 28 tensors (of 13)
        self._as_seen = TensorGuards(*self.tensors, dynamic_dims_sizes=None, dynamic_dims_strides=None).check

    def addresses(self):
        if not self._as_seen(*self.tensors):
            for i, (t, was) in enumerate(zip(self.tensors, self.kinds)):
                now = self._kind(t)
                if now != was:
                    raise ValueError(f"tensor {i} of the list has changed its size, type, device or layout: "
                                     f"(elements, type, device, contiguous) {now}, made for {was}")
            self._guard()      # another shape of as many elements, or a flag like requires_grad
        return list(map(torch.Tensor.data_ptr, self.tensors))


class GradClip:
    """The global norm of a list of gradients and their clipping (gc_grad_norm
    and gc_grad_clip), in place or into `out`.

    Made once for a program's gradient tensors, which it keeps: gradients that a
    program makes anew each step (torch's zero_grad() does, zero_grad(set_to_none=False)
    keeps them) are other tensors, which it does not see.  Each call reads the tensors'
    present addresses, and refuses them (ValueError) where one has another size, type,
    device or layout than it was made for.  The norm comes back as
    a float32 device tensor with one value, in memory of the call's stream; nothing is
    copied to the host.  prescale multiplies the gradients first (the mean over accumulated steps, or
    an undone loss scale)."""

    def __init__(self, grads, out=None, prescale=1.0, eps=1e-6, device="cuda"):
        self.grads, self.out = list(grads), list(grads if out is None else out)
        self.prescale, self.eps = float(prescale), float(eps)
        if len(self.grads) != len(self.out):
            raise ValueError(f"{len(self.grads)} gradients but {len(self.out)} outputs")
        self.device = self.grads[0].device if self.grads else _device(device)
        self._list = (gc_tensor * len(self.grads))()
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            for t, name in ((g, f"gradient {i}"), (o, f"output {i}")):
                if t.numel() != g.numel() or t.dtype != g.dtype:
                    raise ValueError(f"{name} has {t.numel()} elements of {t.dtype}, the gradient "
                                     f"{g.numel()} of {g.dtype}")
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
                if t.device != self.device:
                    raise ValueError(f"{name} is on {t.device}, gradient 0 is on {self.device}")
            self._list[i] = gc_tensor(g.data_ptr(), o.data_ptr(), g.numel(), _code(g.dtype))
        if self.device.type != "cuda":
            raise ValueError("the gradients must be device tensors")
        self._both = _Tensors(self.grads if out is None else self.grads + self.out)
        self._addresses = self._both.addresses()
        self._ws = _Workspace(int(lib().gc_grad_clip_workspace_bytes(len(self.grads))), self.device)

    def _tensors(self):
        addresses = self._both.addresses()
        if addresses != self._addresses:
            n = len(self.grads)
            for item, src, dst in zip(self._list, addresses[:n], addresses[-n:]):
                item.src, item.dst = src, dst
            self._addresses = addresses
        return self._list

    def norm(self, stream=None):
        raw = _raw_stream(stream, self.device)
        norm = _empty((), torch.float32, self.device, raw)
        ws, n, _owner = self._ws.on(raw)
        st = lib().gc_grad_norm(self._tensors(), len(self.grads), self.prescale, norm.data_ptr(), ws, n, raw)
        _check("gc_grad_norm", st)
        return norm

    def clip(self, max_norm, stream=None):
        raw = _raw_stream(stream, self.device)
        norm = _empty((), torch.float32, self.device, raw)
        ws, n, _owner = self._ws.on(raw)
        st = lib().gc_grad_clip(self._tensors(), len(self.grads), float(max_norm), self.prescale, self.eps,
                                norm.data_ptr(), ws, n, raw)
        _check("gc_grad_clip", st)
        return norm
