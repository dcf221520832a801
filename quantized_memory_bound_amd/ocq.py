"""Python binding of the ocq C ABI (include/ocq.h): argument marshalling only.

Every step of the block runs in the HIP library libocq.so built in-tree next
to this file (``python -m quantized_memory_bound_amd.build``).  There is no
fallback: if the library is missing, every call raises.  PyTorch is used only
for device memory and streams.
"""

import ctypes
import os

import numpy as np

# OCQ_LIBRARY names another build of the library (for instance
# libocq_phases.so, built with --phase-stamps); the default is the in-tree
# libocq.so
LIB_PATH = os.environ.get("OCQ_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libocq.so")

PREC_FP8 = 0
PREC_FP8_DOWN_BF16 = 1
PREC_FP4 = 2

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_DEVICE = -3
ERR_BUFFER_TOO_SMALL = -4
ERR_BAD_BLOB = -5

EXPORTS = ("ocq_version", "ocq_packed_bytes", "ocq_pack_weights_host", "ocq_pack_weights",
           "ocq_unpack_weights_host", "ocq_workspace_bytes", "ocq_mlp_forward", "ocq_check_blob",
           "ocq_set_stage_events", "ocq_last_error", "ocq_stack_workspace_bytes", "ocq_mlp_stack_forward",
           "ocq_calibrate_smoothing_host", "ocq_pack_weights_smoothed_host", "ocq_pack_weights_smoothed",
           "ocq_diag_stream_read", "ocq_diag_window_read", "ocq_diag_mfma_rate", "ocq_diag_empty", "ocq_diag_mfma_dot", "ocq_diag_phase_stamps", "ocq_noalloc_scratch_bytes",
           "ocq_mlp_forward_noalloc", "ocq_set_fused_requant", "ocq_last_requant_in_gateup",
           "ocq_add_rmsnorm", "ocq_rope_frequencies", "ocq_rope_append", "ocq_attention_workspace_bytes",
           "ocq_paged_attention")


class OcqError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("ocq status %d: %s" % (status, message))
        self.status = status


class Taps(ctypes.Structure):
    _fields_ = [("x_codes", ctypes.c_void_p), ("x_scales", ctypes.c_void_p),
                ("h_out", ctypes.c_void_p), ("h_scales", ctypes.c_void_p)]


class KVCacheStruct(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_dev", "v_dev", "k_scale_dev", "v_scale_dev")] +
                [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride", "scale_page_stride",
                                               "scale_head_stride", "scale_token_stride")] +
                [(n, ctypes.c_int) for n in ("num_pages", "page_size", "kv_heads", "head_dim", "format")])


class TokenBatchStruct(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q_start_dev", "kv_lens_dev", "page_table_dev")] +
                [("table_stride", ctypes.c_int64)] +
                [(n, ctypes.c_int) for n in ("requests", "tokens", "max_pages", "max_new", "max_kv")] +
                [("counters_dev", ctypes.c_void_p)])


_lib = None


def lib():
    """Load libocq.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libocq.so is not built (%s); run python -m quantized_memory_bound_amd.build" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    L.ocq_version.argtypes, L.ocq_version.restype = [], i
    L.ocq_last_error.argtypes, L.ocq_last_error.restype = [], ctypes.c_char_p
    L.ocq_packed_bytes.argtypes, L.ocq_packed_bytes.restype = [i, i, i], sz
    L.ocq_pack_weights_host.argtypes = [vp, vp, vp, i, i, i, vp, sz]
    L.ocq_pack_weights_host.restype = i
    L.ocq_pack_weights.argtypes = [vp, vp, vp, i, i, i, vp, sz, vp]
    L.ocq_pack_weights.restype = i
    L.ocq_pack_weights_smoothed_host.argtypes = [vp, vp, vp, vp, i, i, i, vp, sz]
    L.ocq_pack_weights_smoothed_host.restype = i
    L.ocq_pack_weights_smoothed.argtypes = [vp, vp, vp, vp, i, i, i, vp, sz, vp]
    L.ocq_pack_weights_smoothed.restype = i
    L.ocq_calibrate_smoothing_host.argtypes = [vp, i, i, vp, vp, i, f, vp]
    L.ocq_calibrate_smoothing_host.restype = i
    L.ocq_unpack_weights_host.argtypes = [vp, sz, i, vp, vp, ctypes.POINTER(f)]
    L.ocq_unpack_weights_host.restype = i
    L.ocq_workspace_bytes.argtypes, L.ocq_workspace_bytes.restype = [i, i, i, i], sz
    L.ocq_mlp_forward.argtypes = [vp, sz, vp, i, i, i, i, vp, vp, sz, ctypes.POINTER(Taps), vp]
    L.ocq_mlp_forward.restype = i
    L.ocq_check_blob.argtypes, L.ocq_check_blob.restype = [vp, sz, i, i, i, vp], i
    L.ocq_set_stage_events.argtypes, L.ocq_set_stage_events.restype = [ctypes.POINTER(vp), i], i
    ip = ctypes.POINTER(i)
    L.ocq_stack_workspace_bytes.argtypes, L.ocq_stack_workspace_bytes.restype = [i, i, i, ip, i], sz
    L.ocq_mlp_stack_forward.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(sz), ip, i, vp, i, i, i, vp, vp, sz, vp]
    L.ocq_mlp_stack_forward.restype = i
    L.ocq_set_fused_requant.argtypes, L.ocq_set_fused_requant.restype = [i], i
    L.ocq_last_requant_in_gateup.argtypes, L.ocq_last_requant_in_gateup.restype = [], i
    L.ocq_noalloc_scratch_bytes.argtypes, L.ocq_noalloc_scratch_bytes.restype = [], sz
    L.ocq_mlp_forward_noalloc.argtypes = [vp, sz, vp, i, i, i, i, vp, ctypes.POINTER(Taps), vp]
    L.ocq_mlp_forward_noalloc.restype = i
    L.ocq_diag_stream_read.argtypes, L.ocq_diag_stream_read.restype = [vp, sz, vp, i, vp], i
    L.ocq_diag_window_read.argtypes, L.ocq_diag_window_read.restype = [vp, sz, i, vp, i, vp], i
    L.ocq_diag_mfma_rate.argtypes, L.ocq_diag_mfma_rate.restype = [i, vp, i, vp, ctypes.POINTER(ctypes.c_double)], i
    L.ocq_diag_empty.argtypes, L.ocq_diag_empty.restype = [vp], i
    L.ocq_diag_mfma_dot.argtypes, L.ocq_diag_mfma_dot.restype = [i, vp, vp, i, i, i, vp, vp], i
    L.ocq_diag_phase_stamps.argtypes, L.ocq_diag_phase_stamps.restype = [i, vp, sz], i
    i64, d = ctypes.c_int64, ctypes.c_double
    cp, bp = ctypes.POINTER(KVCacheStruct), ctypes.POINTER(TokenBatchStruct)
    L.ocq_add_rmsnorm.argtypes = [vp, i64, vp, i64, vp, f, i, i, vp, vp, vp, vp, vp]
    L.ocq_add_rmsnorm.restype = i
    L.ocq_rope_frequencies.argtypes = [i, d, i, d, d, d, d, vp, ctypes.POINTER(f)]
    L.ocq_rope_frequencies.restype = i
    L.ocq_rope_append.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i64, i, vp, i, i, f, vp, cp, bp, vp, vp]
    L.ocq_rope_append.restype = i
    L.ocq_attention_workspace_bytes.argtypes, L.ocq_attention_workspace_bytes.restype = [i, cp, bp, i, i], sz
    L.ocq_paged_attention.argtypes = [vp, i64, i64, i, cp, bp, f, i, i, vp, vp, vp, sz, vp]
    L.ocq_paged_attention.restype = i
    _lib = L
    return L


def _check(status):
    if status != OK:
        raise OcqError(status, lib().ocq_last_error().decode())
    return status


def last_error():
    return lib().ocq_last_error().decode()


def version():
    return lib().ocq_version()


def packed_bytes(hidden, inter, prec_mode):
    return lib().ocq_packed_bytes(hidden, inter, prec_mode)


def workspace_bytes(M, hidden, inter, prec_mode):
    return lib().ocq_workspace_bytes(M, hidden, inter, prec_mode)


def _f32c(a):
    return np.ascontiguousarray(a, dtype=np.float32)


def calibrate_smoothing(x_calib_bits, w_gate, w_up, alpha=0.5):
    """Per-input-channel smoothing factors (float32 [hidden]) from calibration
    activations (bf16 bits [rows, hidden]) and the gate/up weights."""
    xb = np.ascontiguousarray(x_calib_bits, dtype=np.uint16)
    wg, wu = _f32c(w_gate), _f32c(w_up)
    inter, hidden = wg.shape
    s = np.empty(hidden, dtype=np.float32)
    _check(lib().ocq_calibrate_smoothing_host(xb.ctypes.data, xb.shape[0], hidden, wg.ctypes.data, wu.ctypes.data,
                                              inter, float(alpha), s.ctypes.data))
    return s


def pack_weights_host(w_gate, w_up, w_down, prec_mode, smooth=None):
    """Quantize + pack on the host; returns the blob as a uint8 numpy array.
    smooth: None or per-input-channel factors (float32 [hidden])."""
    wg, wu, wd = _f32c(w_gate), _f32c(w_up), _f32c(w_down)
    inter, hidden = wg.shape
    n = packed_bytes(hidden, inter, prec_mode)
    if n == 0:
        raise OcqError(ERR_UNSUPPORTED, "invalid shape or prec_mode")
    out = np.empty(n, dtype=np.uint8)
    sm = None if smooth is None else _f32c(smooth)
    _check(lib().ocq_pack_weights_smoothed_host(wg.ctypes.data, wu.ctypes.data, wd.ctypes.data,
                                                None if sm is None else sm.ctypes.data, hidden, inter,
                                                prec_mode, out.ctypes.data, n))
    return out


def unpack_weights_host(blob, which, hidden, inter, prec_mode):
    """Plain-layout codes / scales of one projection from a host blob."""
    blob = np.ascontiguousarray(blob, dtype=np.uint8)
    rows, cols = (inter, hidden) if which < 2 else (hidden, inter)
    bf16 = prec_mode == PREC_FP8_DOWN_BF16 and which == 2
    if which == 3:
        xm = np.zeros(hidden, dtype=np.float32)
        _check(lib().ocq_unpack_weights_host(blob.ctypes.data, blob.nbytes, 3, None, xm.ctypes.data, None))
        return None, xm, 0.0
    codes = np.zeros((rows, cols), dtype=np.uint16 if bf16 else np.uint8)
    if prec_mode == PREC_FP4:
        scales = np.zeros((rows, cols // 16), dtype=np.uint8)
    elif bf16:
        scales = None
    else:
        scales = np.zeros(rows, dtype=np.float32)
    ts = ctypes.c_float(0.0)
    _check(lib().ocq_unpack_weights_host(blob.ctypes.data, blob.nbytes, which, codes.ctypes.data,
                                         None if scales is None else scales.ctypes.data, ctypes.byref(ts)))
    return codes, scales, ts.value


def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def pack_weights(w_gate, w_up, w_down, prec_mode, device="cuda", stream=None, smooth=None):
    """Quantize + pack and upload; returns a uint8 torch tensor on `device`.
    smooth: None or per-input-channel factors (float32 [hidden])."""
    import torch
    wg, wu, wd = _f32c(w_gate), _f32c(w_up), _f32c(w_down)
    inter, hidden = wg.shape
    n = packed_bytes(hidden, inter, prec_mode)
    if n == 0:
        raise OcqError(ERR_UNSUPPORTED, "invalid shape or prec_mode")
    blob = torch.empty(n, dtype=torch.uint8, device=device)
    sm = None if smooth is None else _f32c(smooth)
    _check(lib().ocq_pack_weights_smoothed(wg.ctypes.data, wu.ctypes.data, wd.ctypes.data,
                                           None if sm is None else sm.ctypes.data, hidden, inter, prec_mode,
                                           blob.data_ptr(), n, _stream_handle(stream)))
    return blob


FUSED_REQUANT_DEFAULT = 1


def set_fused_requant(mode):
    """Process-wide: requantize h inside the gate/up kernel where its grid
    fits the GPU at once (1 or True, the default), or in a second kernel (0
    or False)."""
    _check(lib().ocq_set_fused_requant(int(mode)))


def last_requant_in_gateup():
    """1 if the last forward call on this thread requantized h inside the
    gate/up kernel, 0 if in a separate kernel, -1 before the first call."""
    return lib().ocq_last_requant_in_gateup()


def set_stage_events(events):
    """events: None (disable) or a list of 5 hipEvent_t handles (int or None)."""
    if events is None:
        _check(lib().ocq_set_stage_events(None, 0))
        return
    arr = (ctypes.c_void_p * 5)(*[e if e else None for e in events])
    _check(lib().ocq_set_stage_events(arr, 5))


def check_blob(blob, hidden, inter, prec_mode, stream=None):
    _check(lib().ocq_check_blob(blob.data_ptr(), blob.numel(), hidden, inter, prec_mode, _stream_handle(stream)))


def _need(t, name, dtype, device, shape=None, min_numel=None):
    """Raise OcqError(ERR_INVALID_ARG) unless t is a contiguous tensor of this
    dtype on this device (and shape / size): the C ABI takes raw pointers and
    would read or write past a tensor of another layout."""
    if t is None or not hasattr(t, "data_ptr"):
        raise OcqError(ERR_INVALID_ARG, "%s must be a tensor" % name)
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise OcqError(ERR_INVALID_ARG, "%s has dtype %s" % (name, t.dtype))
    if t.device != device:
        raise OcqError(ERR_INVALID_ARG, "%s is on %s, not %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise OcqError(ERR_INVALID_ARG, "%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise OcqError(ERR_INVALID_ARG, "%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if min_numel is not None and t.numel() < min_numel:
        raise OcqError(ERR_BUFFER_TOO_SMALL, "%s holds %d elements, needs %d" % (name, t.numel(), min_numel))


def _check_x(x, hidden):
    import torch
    if not hasattr(x, "is_cuda") or not x.is_cuda:
        raise OcqError(ERR_INVALID_ARG, "x must be a CUDA tensor")
    if x.dim() != 2 or x.shape[1] != hidden:
        raise OcqError(ERR_INVALID_ARG, "x must be [M, hidden=%d], got %s" % (hidden, tuple(x.shape)))
    _need(x, "x", torch.bfloat16, x.device)


def _taps_struct(taps, M, hidden, inter, prec_mode, dev):
    """Checked Taps structure (or None) from a dict of optional tensors."""
    import torch
    if not taps:
        return None
    spec = {"x_codes": (torch.uint8, (M, hidden)), "x_scales": (torch.float32, (M,)),
            "h_out": ((torch.int16, torch.uint16) if prec_mode == PREC_FP8_DOWN_BF16 else torch.uint8, (M, inter)),
            "h_scales": (torch.float32, (M,))}
    for k, (dt, shp) in spec.items():
        if taps.get(k) is not None:
            _need(taps[k], "taps[%s]" % k, dt, dev, shape=shp)
    return Taps(*(taps[k].data_ptr() if taps.get(k) is not None else None
                  for k in ("x_codes", "x_scales", "h_out", "h_scales")))


def mlp_forward(blob, x, hidden, inter, prec_mode, y=None, workspace=None, taps=None, stream=None):
    """y = block(x) for x a bf16 [M, hidden] CUDA tensor; returns y (bf16 [M, hidden]).

    taps: optional dict with any of x_codes (uint8 [M, hidden]), x_scales
    (float32 [M]), h_out (uint8 [M, inter]; int16 / uint16 bf16 bits in the
    BF16-down mode) and h_scales (float32 [M]) tensors.  Every tensor must be
    contiguous and on x's device; otherwise OcqError is raised before the call.
    """
    import torch
    _check_x(x, hidden)
    M, dev = x.shape[0], x.device
    _need(blob, "blob", torch.uint8, dev, min_numel=packed_bytes(hidden, inter, prec_mode))
    if y is None:
        y = torch.empty((M, hidden), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, dev, shape=(M, hidden))
    if workspace is None:
        workspace = torch.empty(max(1, workspace_bytes(M, hidden, inter, prec_mode)), dtype=torch.uint8,
                                device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    t = _taps_struct(taps, M, hidden, inter, prec_mode, dev)
    _check(lib().ocq_mlp_forward(blob.data_ptr(), blob.numel(), x.data_ptr(), M, hidden, inter, prec_mode,
                                 y.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                 ctypes.byref(t) if t is not None else None, _stream_handle(stream)))
    return y


def mlp_forward_noalloc(blob, x, hidden, inter, prec_mode, y=None, taps=None, stream=None):
    """As mlp_forward, through the entry point that allocates nothing (its
    workspace is the library's fixed per-device scratch array).  y (bf16
    [M, hidden]) must be given by callers that cannot allocate either."""
    import torch
    _check_x(x, hidden)
    M, dev = x.shape[0], x.device
    _need(blob, "blob", torch.uint8, dev, min_numel=packed_bytes(hidden, inter, prec_mode))
    if y is None:
        y = torch.empty((M, hidden), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, dev, shape=(M, hidden))
    t = _taps_struct(taps, M, hidden, inter, prec_mode, dev)
    _check(lib().ocq_mlp_forward_noalloc(blob.data_ptr(), blob.numel(), x.data_ptr(), M, hidden, inter, prec_mode,
                                         y.data_ptr(), ctypes.byref(t) if t is not None else None,
                                         _stream_handle(stream)))
    return y


def noalloc_scratch_bytes():
    return lib().ocq_noalloc_scratch_bytes()


def _int_array(vals):
    return (ctypes.c_int * len(vals))(*[int(v) for v in vals])


def stack_workspace_bytes(M, hidden, inter, prec_modes):
    return lib().ocq_stack_workspace_bytes(M, hidden, inter, _int_array(prec_modes), len(prec_modes))


def mlp_stack_forward(blobs, prec_modes, x, hidden, inter, y=None, workspace=None, stream=None):
    """L blocks in sequence (block l's output is block l+1's input); returns the
    last block's y (bf16 [M, hidden]).  blobs: L uint8 CUDA tensors."""
    import torch
    if len(blobs) != len(prec_modes):
        raise ValueError("one prec_mode per blob")
    _check_x(x, hidden)
    M, dev = x.shape[0], x.device
    for l, (b, m) in enumerate(zip(blobs, prec_modes)):
        _need(b, "blobs[%d]" % l, torch.uint8, dev, min_numel=packed_bytes(hidden, inter, m))
    if y is None:
        y = torch.empty((M, hidden), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, dev, shape=(M, hidden))
    if workspace is None:
        workspace = torch.empty(max(1, stack_workspace_bytes(M, hidden, inter, prec_modes)), dtype=torch.uint8,
                                device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    n = len(blobs)
    ptrs = (ctypes.c_void_p * n)(*[b.data_ptr() for b in blobs])
    sizes = (ctypes.c_size_t * n)(*[b.numel() for b in blobs])
    _check(lib().ocq_mlp_stack_forward(ptrs, sizes, _int_array(prec_modes), n, x.data_ptr(), M, hidden, inter,
                                       y.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                       _stream_handle(stream)))
    return y


class QuantizedMLP:
    """One packed block on the GPU with its workspace, for repeated calls."""

    def __init__(self, w_gate, w_up, w_down, prec_mode, device="cuda"):
        self.inter, self.hidden = np.asarray(w_gate).shape
        self.prec_mode = prec_mode
        self.device = device
        self.blob = pack_weights(w_gate, w_up, w_down, prec_mode, device)
        self._ws = {}

    def workspace(self, M):
        import torch
        if M not in self._ws:
            self._ws[M] = torch.empty(workspace_bytes(M, self.hidden, self.inter, self.prec_mode),
                                      dtype=torch.uint8, device=self.device)
        return self._ws[M]

    def __call__(self, x, y=None, taps=None, stream=None):
        return mlp_forward(self.blob, x, self.hidden, self.inter, self.prec_mode, y=y,
                           workspace=self.workspace(x.shape[0]), taps=taps, stream=stream)


# ---------------------------------------------------------------- the operators around the block

ATTENTION_COUNTERS = 4096
ROPE_SCALINGS = ("none", "linear", "ntk", "yarn")


_INT_MAX = (1 << 31) - 1

_torch = None
_raw_stream = None
_current_device = None


def _gpu(t, name):
    """The device index of the CUDA tensor t, which must be the current device's."""
    global _torch, _raw_stream, _current_device
    if _torch is None:
        import torch
        _torch = torch
        # the handle of the current stream without a Stream object: 0.1 us instead of 2.8
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda i: torch.cuda.current_stream(i).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    i = t.get_device() if hasattr(t, "get_device") else -1
    if i < 0:
        raise OcqError(ERR_INVALID_ARG, "%s must be a CUDA tensor" % name)
    if i != _current_device():
        raise OcqError(ERR_INVALID_ARG, "%s is on cuda:%d, not on the current device" % (name, i))
    return i


def _bf16_rows(t, name, index, shape):
    """Raise unless t is a bf16 tensor of this shape on device `index`, its last axis contiguous."""
    if t is None or not hasattr(t, "get_device"):
        raise OcqError(ERR_INVALID_ARG, "%s must be a tensor" % name)
    if t.dtype is _torch.bfloat16 and t.get_device() == index and t.shape == shape and t.stride(-1) == 1:
        return
    if t.dtype is not _torch.bfloat16 or t.get_device() != index:
        raise OcqError(ERR_INVALID_ARG, "%s must be bfloat16 on cuda:%d, got %s on %s" %
                       (name, index, t.dtype, t.device))
    if t.shape != shape:
        raise OcqError(ERR_INVALID_ARG, "%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise OcqError(ERR_INVALID_ARG, "the last axis of %s must be contiguous" % name)


def _int32(value, name):
    """value as an int, which the C ABI takes in 32 bits (ctypes would cut it off silently)."""
    value = int(value)
    if not -1 << 31 <= value < 1 << 31:
        raise OcqError(ERR_INVALID_ARG, "%s is %d, beyond 32 bits" % (name, value))
    return value


def _empty(shape, dtype, index, stream):
    """A new tensor for a call on `stream`: allocated on it, so that its memory is not reused before the call."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=index)
    cuda = _torch.cuda
    with cuda.stream(stream if hasattr(stream, "cuda_stream") else cuda.ExternalStream(stream, index)):
        return _torch.empty(shape, dtype=dtype, device=index)


def _empty_as(t, shape, dtype, index, stream):
    """_empty of t's shape (the cheapest allocation where t is contiguous)."""
    if stream is None and t.is_contiguous():
        return _torch.empty_like(t, dtype=dtype)
    return _empty(shape, dtype, index, stream)


def _stream_of(stream, index):
    return _raw_stream(index) if stream is None else getattr(stream, "cuda_stream", stream)


def add_rmsnorm(x, weight, eps=1e-6, residual=None, want_y=False, want_codes=True, residual_out=None, y=None,
                codes=None, scales=None, stream=None):
    """RMSNorm of h = x + residual (x, residual: bf16 [rows, hidden] CUDA tensors, rows strided at will; weight: bf16
    [hidden]); returns (residual_out, y, codes, scales).

    residual_out: bf16(h), None without a residual; y: bf16 of the norm if wanted or given; codes (float8_e4m3fn
    [rows, hidden]) and scales (float32 [rows]): its E4M3 quantization if wanted or given.  Outputs that are not
    given are allocated; given codes may be uint8.
    """
    i = _gpu(x, "x")
    if x.dim() != 2:
        raise OcqError(ERR_INVALID_ARG, "x must be [rows, hidden], got %s" % (tuple(x.shape),))
    shape = rows, hidden = x.shape
    if rows > _INT_MAX or hidden > _INT_MAX:
        raise OcqError(ERR_INVALID_ARG, "x is [%d, %d], beyond 32 bits" % shape)
    _bf16_rows(x, "x", i, shape)
    _bf16_rows(weight, "weight", i, (hidden,))
    bf16, res, res_stride = _torch.bfloat16, None, 0
    if residual is not None:
        _bf16_rows(residual, "residual", i, shape)
        res, res_stride = residual.data_ptr(), residual.stride(0)
    if residual_out is not None:
        _need(residual_out, "residual_out", bf16, x.device, shape)
    elif residual is not None:
        residual_out = _empty_as(x, shape, bf16, i, stream)
    if y is not None:
        _need(y, "y", bf16, x.device, shape)
    elif want_y:
        y = _empty_as(x, shape, bf16, i, stream)
    if codes is not None or scales is not None or want_codes:
        if codes is None:
            codes = _empty_as(x, shape, _torch.float8_e4m3fn, i, stream)
        else:
            _need(codes, "codes", (_torch.float8_e4m3fn, _torch.uint8), x.device, shape)
        if scales is None:
            scales = _empty(rows, _torch.float32, i, stream)
        else:
            _need(scales, "scales", _torch.float32, x.device, (rows,))
    _check(lib().ocq_add_rmsnorm(x.data_ptr(), x.stride(0), res, res_stride, weight.data_ptr(), eps, rows, hidden,
                                 None if residual_out is None else residual_out.data_ptr(),
                                 None if y is None else y.data_ptr(), None if codes is None else codes.data_ptr(),
                                 None if scales is None else scales.data_ptr(), _stream_of(stream, i)))
    return residual_out, y, codes, scales


class PagedKVCache:
    """The paged cache of one layer.

    k, v: [num_pages, kv_heads, page_size, head_dim] CUDA tensors, bf16, or float8_e4m3fn (or uint8) codes with
    k_scale, v_scale float32 [num_pages, kv_heads, page_size].  Any order of the first three axes in memory (a
    permuted view of a pool of another layout is fine), the same for k and v.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        self.index = _gpu(k, "k")
        dev = k.device
        if k.dim() != 4 or k.dtype not in (torch.bfloat16, torch.float8_e4m3fn, torch.uint8):
            raise OcqError(ERR_INVALID_ARG, "k must be [pages, kv_heads, page_size, head_dim], bf16 or E4M3 codes")
        if v is None or not hasattr(v, "data_ptr") or v.device != dev or v.dtype != k.dtype or v.shape != k.shape or \
                v.stride() != k.stride():
            raise OcqError(ERR_INVALID_ARG, "v must have k's device, dtype, shape and strides")
        if k.stride(3) != 1:
            raise OcqError(ERR_INVALID_ARG, "the last axis of k and v must be contiguous")
        e4m3 = k.dtype != torch.bfloat16
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise OcqError(ERR_INVALID_ARG, "E4M3 caches have scales, bf16 caches none")
        if e4m3:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if t.device != dev or t.dtype != torch.float32 or t.shape != k.shape[:3] or \
                        t.stride() != k_scale.stride():
                    raise OcqError(ERR_INVALID_ARG, "%s must be float32 %s, k_scale and v_scale of one layout" %
                                   (name, tuple(k.shape[:3])))
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, dev
        for n, name in zip(k.shape, ("pages", "kv_heads", "page_size", "head_dim")):
            _int32(n, name)
        pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        s = k_scale.stride() if e4m3 else (0, 0, 0)
        self.struct = KVCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if e4m3 else None,
                                    v_scale.data_ptr() if e4m3 else None, k.stride(0), k.stride(1), k.stride(2), s[0],
                                    s[1], s[2], pages, self.page_size, self.kv_heads, self.head_dim, int(e4m3))
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def allocate(cls, num_pages, page_size, kv_heads, head_dim, e4m3=False, device="cuda"):
        """A zeroed cache whose pages hold each head's rows side by side."""
        import torch
        shape = (num_pages, kv_heads, page_size, head_dim)
        if not e4m3:
            return cls(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        kv = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        return cls(*kv, *(torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))


class TokenBatch:
    """The new tokens of one step: request r has rows q_start[r] .. q_start[r + 1] of the token axis, kv_lens[r]
    tokens in the cache with the new ones, and pages page_table[r].

    q_start int32 [requests + 1], kv_lens int32 [requests], page_table int32 [requests, max_pages] (its rows max_pages
    entries or more apart): CUDA tensors whose contents may change between calls.  tokens (the rows of q), max_new and
    max_kv are host numbers: bounds of the new tokens and of kv_lens of any request.

    Attention calls over one batch count their finished work in memory of the batch, 0 between calls, apart for every
    stream that they run on.  A captured call counts where calls on the stream that the batch was made on do: its replays
    are ordered with those, and the batch outlives the graph.  The device arrays must not change while a call runs (its
    counts could stay wrong for the next one).
    """

    def __init__(self, q_start, kv_lens, page_table, max_new, max_kv, tokens=None):
        import torch
        self.index = _gpu(kv_lens, "kv_lens")
        dev = kv_lens.device
        requests = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
        _need(kv_lens, "kv_lens", torch.int32, dev, shape=(requests,))
        _need(q_start, "q_start", torch.int32, dev, shape=(requests + 1,))
        if not hasattr(page_table, "data_ptr") or page_table.dtype != torch.int32 or page_table.device != dev or \
                page_table.dim() != 2 or page_table.shape[0] != requests or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise OcqError(ERR_INVALID_ARG, "page_table must be int32 [%d, max_pages], its rows contiguous" % requests)
        stride = page_table.stride(0)
        if requests <= 1:
            stride = max(stride, page_table.shape[1])   # of a row that has no next one: any
        elif stride < page_table.shape[1]:
            raise OcqError(ERR_INVALID_ARG, "rows of page_table are %d entries apart, fewer than their %d (a table "
                           "that requests share has to be copied: .contiguous())" % (stride, page_table.shape[1]))
        self.q_start, self.kv_lens, self.page_table, self.device = q_start, kv_lens, page_table, dev
        self.requests, self.tokens = requests, None
        self.counters = torch.zeros(ATTENTION_COUNTERS, dtype=torch.int32, device=dev)   # of the stream it is made on
        self.stream = _raw_stream(self.index)             # the stream whose counters the struct holds
        self.counters_of = {self.stream: self.counters}
        self.struct = TokenBatchStruct(q_start.data_ptr(), kv_lens.data_ptr(), page_table.data_ptr(),
                                       stride, requests, 0, _int32(page_table.shape[1], "max_pages"),
                                       _int32(max_new, "max_new"), _int32(max_kv, "max_kv"),
                                       self.counters.data_ptr())
        self.ref = ctypes.byref(self.struct)
        if tokens is not None:
            self.of(tokens)

    def of(self, tokens):
        """The batch as an argument for a call over `tokens` rows."""
        if self.tokens is None:
            self.tokens = self.struct.tokens = _int32(tokens, "tokens")
        elif tokens != self.tokens:
            raise OcqError(ERR_INVALID_ARG, "the batch has %d tokens, the tensor %d" % (self.tokens, tokens))
        return self.ref


    def move_to(self, stream):
        """Count the attention calls that follow in memory of this stream (a raw handle): zeroed in its order and not
        reused before what it has queued is done, also if the batch is dropped meanwhile."""
        cuda, counters = _torch.cuda, self.counters_of.get(stream)
        if counters is None:
            with cuda.stream(cuda.ExternalStream(stream, self.index)):
                if cuda.is_current_stream_capturing():    # a fill would be a part of every replay
                    self.struct.counters_dev, self.stream = self.counters.data_ptr(), None
                    return
                counters = _torch.zeros(ATTENTION_COUNTERS, dtype=_torch.int32, device=self.device)
            self.counters_of[stream] = counters
        self.struct.counters_dev, self.stream = counters.data_ptr(), stream


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, context=4096, beta_fast=32.0, beta_slow=1.0):
    """Rotary frequencies (float64 numpy [rot / 2]) and the multiplier of cos and sin; scaling: one of
    ROPE_SCALINGS (none, positions divided by the factor, stretched base, YaRN)."""
    if scaling not in ROPE_SCALINGS:
        raise OcqError(ERR_INVALID_ARG, "scaling must be one of %s" % (ROPE_SCALINGS,))
    inv = np.empty(max(1, int(rot) // 2), dtype=np.float64)
    mult = ctypes.c_float()
    _check(lib().ocq_rope_frequencies(int(rot), float(base), ROPE_SCALINGS.index(scaling), float(factor),
                                      float(context), float(beta_fast), float(beta_slow), inv.ctypes.data,
                                      ctypes.byref(mult)))
    return inv, mult.value


class Rope:
    """Rotary frequencies on the GPU: inv_freq float64 [rot / 2], the multiplier of cos and sin, and whether pairs
    are (2 j, 2 j + 1) (interleaved) or (j, j + rot / 2)."""

    def __init__(self, inv_freq, multiplier=1.0, interleaved=False):
        import torch
        self.index = _gpu(inv_freq, "inv_freq")
        dev = inv_freq.device
        if inv_freq.dim() != 1:
            raise OcqError(ERR_INVALID_ARG, "inv_freq must be [rot / 2]")
        _need(inv_freq, "inv_freq", torch.float64, dev)
        self.inv_freq, self.multiplier, self.interleaved = inv_freq, float(multiplier), int(bool(interleaved))
        self.rot, self.device = 2 * inv_freq.shape[0], dev

    @classmethod
    def make(cls, rot, interleaved=False, device="cuda", **kw):
        """From rope_frequencies(rot, **kw)."""
        import torch
        inv, mult = rope_frequencies(rot, **kw)
        return cls(torch.from_numpy(inv).to(device), mult, interleaved)


def _on(index, *handles):
    for h in handles:
        if h.index != index:
            raise OcqError(ERR_INVALID_ARG, "%s is on %s, not on cuda:%d" % (type(h).__name__, h.device, index))


def rope_append(q, k, v, rope, cache, batch, positions=None, q_out=None, stream=None):
    """Rotate q (bf16 [tokens, heads, head_dim]) and k ([tokens, kv_heads, head_dim]) and append k and v to the
    cache; returns the rotated q (q_out, contiguous, or q itself).  Token and head strides are free.  positions:
    None (each token's place in its request) or int32 [tokens]."""
    i = _gpu(q, "q")
    if q.dim() != 3:
        raise OcqError(ERR_INVALID_ARG, "q must be [tokens, heads, head_dim], got %s" % (tuple(q.shape),))
    shape = tokens, heads, dim = q.shape
    if dim != cache.head_dim:
        raise OcqError(ERR_INVALID_ARG, "q has head size %d, the cache %d" % (dim, cache.head_dim))
    _bf16_rows(q, "q", i, shape)
    kv_shape = (tokens, cache.kv_heads, dim)
    _bf16_rows(k, "k", i, kv_shape)
    _bf16_rows(v, "v", i, kv_shape)
    _on(i, rope, cache, batch)
    if positions is not None:
        _need(positions, "positions", _torch.int32, q.device, (tokens,))
    if q_out is None:
        q_out = _empty_as(q, shape, _torch.bfloat16, i, stream)
    else:
        _need(q_out, "q_out", _torch.bfloat16, q.device, shape)
    _check(lib().ocq_rope_append(q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1),
                                 v.data_ptr(), v.stride(0), v.stride(1), heads, rope.inv_freq.data_ptr(), rope.rot,
                                 rope.interleaved, rope.multiplier, None if positions is None else positions.data_ptr(),
                                 cache.ref, batch.of(tokens), q_out.data_ptr(), _stream_of(stream, i)))
    return q_out


def attention_workspace_bytes(heads, cache, batch, window=0, sinks=0):
    """Workspace of paged_attention for a batch whose tokens are known."""
    return lib().ocq_attention_workspace_bytes(_int32(heads, "heads"), cache.ref, batch.ref, _int32(window, "window"),
                                               _int32(sinks, "sinks"))


def paged_attention(q, cache, batch, scale=None, window=0, sinks=0, want_lse=False, out=None, lse=None,
                    workspace=None, stream=None):
    """Attention of the new tokens q (bf16 [tokens, heads, head_dim], token and head strides free) over the paged
    cache that already holds them; returns (out, lse): bf16 [tokens, heads, head_dim] and, if wanted or given,
    float32 [tokens, heads].

    scale: default head_dim ** -0.5.  window: keys up to window - 1 places back are visible (0: all); sinks: the
    first tokens, which a window leaves visible.  A token that sees nothing has out 0 and lse -inf.  workspace: a
    uint8 tensor of attention_workspace_bytes(...), allocated if None.
    """
    i = _gpu(q, "q")
    if q.dim() != 3:
        raise OcqError(ERR_INVALID_ARG, "q must be [tokens, heads, head_dim], got %s" % (tuple(q.shape),))
    shape = tokens, heads, dim = q.shape
    if dim != cache.head_dim:
        raise OcqError(ERR_INVALID_ARG, "q has head size %d, the cache %d" % (dim, cache.head_dim))
    _bf16_rows(q, "q", i, shape)
    if not (0 <= window <= _INT_MAX and 0 <= sinks <= _INT_MAX):
        raise OcqError(ERR_INVALID_ARG, "window %d and sinks %d must be in [0, 2^31)" % (window, sinks))
    _on(i, cache, batch)
    if out is None:
        out = _empty_as(q, shape, _torch.bfloat16, i, stream)
    else:
        _need(out, "out", _torch.bfloat16, q.device, shape)
    if lse is not None:
        _need(lse, "lse", _torch.float32, q.device, (tokens, heads))
    elif want_lse:
        lse = _empty((tokens, heads), _torch.float32, i, stream)
    ref, L, handle = batch.of(tokens), lib(), _stream_of(stream, i)
    if handle != batch.stream:
        batch.move_to(handle)
    if workspace is None:
        need = L.ocq_attention_workspace_bytes(heads, cache.ref, ref, window, sinks)
        if need:
            workspace = _empty(need, _torch.uint8, i, stream)
    else:
        _need(workspace, "workspace", _torch.uint8, q.device)
        need = workspace.numel()
    _check(L.ocq_paged_attention(q.data_ptr(), q.stride(0), q.stride(1), heads, cache.ref, ref,
                                 dim ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(),
                                 None if lse is None else lse.data_ptr(),
                                 None if workspace is None else workspace.data_ptr(), need, handle))
    return out, lse


# ---------------------------------------------------------------- measurement helpers

def diag_stream_read(src, out, blocks, stream=None):
    """Read the whole uint8 CUDA tensor src with the library's streaming-read
    kernel (out: int32 / uint8 CUDA tensor of >= 4 * blocks bytes)."""
    import torch
    _need(src, "src", torch.uint8, src.device)
    if out.numel() * out.element_size() < 4 * blocks:
        raise OcqError(ERR_BUFFER_TOO_SMALL, "out holds fewer than 4 * blocks bytes")
    _check(lib().ocq_diag_stream_read(src.data_ptr(), src.numel(), out.data_ptr(), blocks, _stream_handle(stream)))


def diag_window_read(src, window_bytes, passes, out, blocks, stream=None):
    """Every one of `blocks` workgroups reads src[:window_bytes] `passes` times
    (src: uint8 CUDA tensor; out: int32 / uint8 CUDA tensor of >= 4 * blocks
    bytes)."""
    import torch
    _need(src, "src", torch.uint8, src.device)
    if window_bytes > src.numel():
        raise OcqError(ERR_BUFFER_TOO_SMALL, "window larger than src")
    if out.numel() * out.element_size() < 4 * blocks:
        raise OcqError(ERR_BUFFER_TOO_SMALL, "out holds fewer than 4 * blocks bytes")
    _check(lib().ocq_diag_window_read(src.data_ptr(), window_bytes, passes, out.data_ptr(), blocks,
                                      _stream_handle(stream)))


def diag_mfma_rate(iters, out, blocks, stream=None):
    """Launch the matrix-core rate kernel (out: float32 CUDA tensor of >= 512 *
    blocks elements); returns the launch's floating-point operations."""
    import torch
    _need(out, "out", torch.float32, out.device)
    if out.numel() < 512 * blocks:
        raise OcqError(ERR_BUFFER_TOO_SMALL, "out holds fewer than 512 * blocks floats")
    fl = ctypes.c_double()
    _check(lib().ocq_diag_mfma_rate(iters, out.data_ptr(), blocks, _stream_handle(stream), ctypes.byref(fl)))
    return fl.value


def diag_empty(stream=None):
    _check(lib().ocq_diag_empty(_stream_handle(stream)))


PHASE_SHAPES = {0: (2, 512, 8, 8), 1: (512, 12, 8), 2: (2, 1024, 2)}


def diag_phase_stamps(kernel):
    """Phase stamp table of the last launch (kernel 0: LDS-tiled GEMMs,
    kernel 1: producer/consumer gate/up, kernel 2: x quantization and
    requantization) as a uint64 array of shape PHASE_SHAPES[kernel]; needs a
    library built with --phase-stamps."""
    if kernel not in PHASE_SHAPES:
        raise OcqError(ERR_INVALID_ARG, "kernel must be 0, 1 or 2")
    out = np.zeros(PHASE_SHAPES[kernel], dtype=np.uint64)
    _check(lib().ocq_diag_phase_stamps(kernel, out.ctypes.data, out.nbytes))
    return out


def diag_mfma_dot(form, a_codes, b_codes, stream=None):
    """c = dec(a) dec(b)^T (float32 [M, N]) over E4M3 code tensors a [M, K],
    b [N, K] (uint8, CUDA) through matrix-core form 0 (f16), 1 (f8f6f4 K=128)
    or 2 (fp8 K=32)."""
    import torch
    M, K = a_codes.shape
    N = b_codes.shape[0]
    _need(a_codes, "a", torch.uint8, a_codes.device)
    _need(b_codes, "b", torch.uint8, a_codes.device, shape=(N, K))
    c = torch.empty((M, N), dtype=torch.float32, device=a_codes.device)
    _check(lib().ocq_diag_mfma_dot(form, a_codes.data_ptr(), b_codes.data_ptr(), M, N, K, c.data_ptr(),
                                   _stream_handle(stream)))
    return c
