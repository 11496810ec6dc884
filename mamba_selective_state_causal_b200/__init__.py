"""Python binding of the B200 SSD layer library (libssd.so, C ABI in include/ssd.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  torch tensors supply device memory and the CUDA stream.  If the
compiled library is missing, importing the binding's functions raises: there
is no fallback implementation.
"""
import ctypes
import math
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libssd.so")

SSD_F32, SSD_BF16 = 0, 1
STATUS = {0: "SSD_OK", 1: "SSD_ERR_NULL", 2: "SSD_ERR_SHAPE", 3: "SSD_ERR_ALIGN",
          4: "SSD_ERR_STRIDE", 5: "SSD_ERR_DTYPE", 6: "SSD_ERR_UNSUPPORTED",
          7: "SSD_ERR_LAUNCH", 8: "SSD_ERR_TIMEOUT", 9: "SSD_ERR_WORKSPACE", 10: "SSD_ERR_INDEX"}

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p


class SSDError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", _i64), ("total_ms", ctypes.c_double)]


class ScanArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("b", ctypes.c_int), ("L", _i64),
                ("H", ctypes.c_int), ("P", ctypes.c_int), ("N", ctypes.c_int),
                ("G", ctypes.c_int), ("Q", ctypes.c_int), ("s", _i64),
                ("x", _vp), ("x_batch_stride", _i64), ("x_row_stride", _i64),
                ("B", _vp), ("B_batch_stride", _i64), ("B_row_stride", _i64),
                ("C", _vp), ("C_batch_stride", _i64), ("C_row_stride", _i64),
                ("dt", _vp), ("A", _vp), ("D", _vp), ("h0", _vp),
                ("y", _vp), ("y_batch_stride", _i64), ("y_row_stride", _i64),
                ("h_final", _vp), ("h_ckpt", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
                ("dt_bias", _vp), ("dt_softplus", ctypes.c_int),
                ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float)]


class StreamArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("b", ctypes.c_int), ("L", _i64),
                ("H", ctypes.c_int), ("P", ctypes.c_int), ("N", ctypes.c_int),
                ("G", ctypes.c_int), ("Q", ctypes.c_int), ("s", _i64),
                ("u", _vp), ("u_batch_stride", _i64), ("u_row_stride", _i64),
                ("conv_w", _vp), ("conv_bias", _vp), ("tail_in", _vp), ("tail_out", _vp),
                ("v", _vp), ("v_batch_stride", _i64), ("v_row_stride", _i64),
                ("dt", _vp), ("A", _vp), ("D", _vp), ("h0", _vp),
                ("y", _vp), ("y_batch_stride", _i64), ("y_row_stride", _i64),
                ("h_final", _vp), ("h_ckpt", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
                ("dt_bias", _vp), ("dt_softplus", ctypes.c_int),
                ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float),
                ("conv_ckpt", _vp)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("b", ctypes.c_int),
                ("H", ctypes.c_int), ("P", ctypes.c_int), ("N", ctypes.c_int), ("G", ctypes.c_int),
                ("u", _vp), ("u_batch_stride", _i64),
                ("conv_w", _vp), ("conv_bias", _vp), ("tail_in", _vp), ("tail_out", _vp),
                ("dt", _vp), ("A", _vp), ("D", _vp), ("h_in", _vp), ("h_out", _vp),
                ("y", _vp), ("y_batch_stride", _i64),
                ("dt_bias", _vp), ("dt_softplus", ctypes.c_int),
                ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float)]


class ScanBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("b", ctypes.c_int), ("L", _i64),
                ("H", ctypes.c_int), ("P", ctypes.c_int), ("N", ctypes.c_int),
                ("G", ctypes.c_int), ("s", _i64),
                ("x", _vp), ("x_batch_stride", _i64), ("x_row_stride", _i64),
                ("B", _vp), ("B_batch_stride", _i64), ("B_row_stride", _i64),
                ("C", _vp), ("C_batch_stride", _i64), ("C_row_stride", _i64),
                ("dt", _vp), ("A", _vp), ("D", _vp), ("h0", _vp), ("h_ckpt", _vp),
                ("dy", _vp), ("dy_batch_stride", _i64), ("dy_row_stride", _i64),
                ("dh_final", _vp),
                ("dx", _vp), ("dB", _vp), ("dC", _vp), ("ddt", _vp), ("dA", _vp), ("dD", _vp),
                ("dh0", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class LayerBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("b", ctypes.c_int), ("L", _i64),
                ("H", ctypes.c_int), ("P", ctypes.c_int), ("N", ctypes.c_int),
                ("G", ctypes.c_int), ("s", _i64),
                ("u", _vp), ("u_batch_stride", _i64), ("u_row_stride", _i64),
                ("conv_w", _vp), ("conv_bias", _vp), ("tail_in", _vp), ("conv_ckpt", _vp),
                ("dt", _vp), ("A", _vp), ("D", _vp), ("h0", _vp), ("h_ckpt", _vp),
                ("dy", _vp), ("dy_batch_stride", _i64), ("dy_row_stride", _i64),
                ("dh_final", _vp), ("dtail_out", _vp),
                ("du", _vp), ("dtail_in", _vp), ("dconv_w", _vp), ("dconv_bias", _vp),
                ("ddt", _vp), ("dA", _vp), ("dD", _vp), ("dh0", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class PackedPlanArgs(ctypes.Structure):
    _fields_ = [("nseq", ctypes.c_int), ("total", _i64), ("cu_seqlens", _vp), ("slots", _vp), ("resume", _vp),
                ("n_slots", ctypes.c_int), ("max_seqlen", _i64), ("plan", _vp), ("plan_bytes", ctypes.c_size_t)]


class PackedConvArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("nseq", ctypes.c_int), ("total", _i64), ("C_ch", ctypes.c_int), ("plan", _vp),
                ("u", _vp), ("u_row_stride", _i64), ("conv_w", _vp), ("conv_bias", _vp), ("tail_in", _vp),
                ("tail_out", _vp), ("v", _vp), ("v_row_stride", _i64)]


class PackedConvBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("nseq", ctypes.c_int), ("total", _i64),
                ("d_inner", ctypes.c_int), ("d_bc", ctypes.c_int), ("plan", _vp),
                ("u", _vp), ("u_row_stride", _i64), ("conv_w", _vp), ("conv_bias", _vp), ("tail_in", _vp),
                ("dx", _vp), ("dB", _vp), ("dC", _vp), ("dtail_out", _vp),
                ("du", _vp), ("dtail_in", _vp), ("dconv_w", _vp), ("dconv_bias", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class PackedScanArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("nseq", ctypes.c_int), ("total", _i64), ("max_seqlen", _i64),
                ("H", ctypes.c_int), ("P", ctypes.c_int), ("N", ctypes.c_int), ("G", ctypes.c_int), ("plan", _vp),
                ("x", _vp), ("x_row_stride", _i64), ("B", _vp), ("B_row_stride", _i64), ("C", _vp),
                ("C_row_stride", _i64), ("dt", _vp), ("A", _vp), ("D", _vp), ("dt_bias", _vp),
                ("dt_softplus", ctypes.c_int), ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float),
                ("h_in", _vp), ("h_out", _vp), ("y", _vp), ("y_row_stride", _i64),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class PackedScanBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("nseq", ctypes.c_int), ("total", _i64),
                ("H", ctypes.c_int), ("P", ctypes.c_int), ("N", ctypes.c_int), ("G", ctypes.c_int), ("plan", _vp),
                ("x", _vp), ("x_row_stride", _i64), ("B", _vp), ("B_row_stride", _i64), ("C", _vp),
                ("C_row_stride", _i64), ("dt", _vp), ("A", _vp), ("D", _vp), ("h_in", _vp),
                ("dy", _vp), ("dy_row_stride", _i64), ("dh_out", _vp),
                ("dx", _vp), ("dB", _vp), ("dC", _vp), ("ddt", _vp), ("dA", _vp), ("dD", _vp), ("dh_in", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class DecodeSlotsArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("b", ctypes.c_int), ("n_slots", ctypes.c_int),
                ("H", ctypes.c_int), ("P", ctypes.c_int), ("N", ctypes.c_int), ("G", ctypes.c_int),
                ("slots", _vp), ("u", _vp), ("u_batch_stride", _i64), ("conv_w", _vp), ("conv_bias", _vp),
                ("tail_in", _vp), ("tail_out", _vp), ("dt", _vp), ("A", _vp), ("D", _vp), ("dt_bias", _vp),
                ("dt_softplus", ctypes.c_int), ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float),
                ("h_in", _vp), ("h_out", _vp), ("y", _vp), ("y_batch_stride", _i64)]


class GatedRmsnormBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("rows", _i64), ("d", ctypes.c_int), ("group_size", ctypes.c_int),
                ("eps", ctypes.c_float), ("dout", _vp), ("dout_row_stride", _i64), ("y", _vp), ("y_row_stride", _i64),
                ("z", _vp), ("z_row_stride", _i64), ("weight", _vp), ("dy", _vp), ("dy_row_stride", _i64),
                ("dz", _vp), ("dz_row_stride", _i64), ("dweight", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


_lib = None


def lib():
    """The loaded libssd.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        L.ssd_conv_forward.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                       ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int, _vp]
        L.ssd_conv_forward.restype = ctypes.c_int
        L.ssd_scan_forward.argtypes = [ctypes.POINTER(ScanArgs), _vp]
        L.ssd_scan_forward.restype = ctypes.c_int
        L.ssd_stream_forward.argtypes = [ctypes.POINTER(StreamArgs), _vp]
        L.ssd_stream_forward.restype = ctypes.c_int
        L.ssd_decode_step.argtypes = [ctypes.POINTER(DecodeArgs), _vp]
        L.ssd_decode_step.restype = ctypes.c_int
        L.ssd_gated_rmsnorm_forward.argtypes = [_vp, _i64, _vp, _i64, _vp, ctypes.c_float, ctypes.c_int, _vp, _i64,
                                                _i64, ctypes.c_int, ctypes.c_int, _vp]
        L.ssd_gated_rmsnorm_forward.restype = ctypes.c_int
        L.ssd_scan_backward.argtypes = [ctypes.POINTER(ScanBwdArgs), _vp]
        L.ssd_scan_backward.restype = ctypes.c_int
        L.ssd_scan_backward_workspace_size.argtypes = [ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int,
                                                       ctypes.c_int]
        L.ssd_scan_backward_workspace_size.restype = ctypes.c_size_t
        L.ssd_layer_backward.argtypes = [ctypes.POINTER(LayerBwdArgs), _vp]
        L.ssd_layer_backward.restype = ctypes.c_int
        L.ssd_layer_backward_workspace_size.argtypes = [ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int,
                                                        ctypes.c_int, ctypes.c_int, ctypes.c_int]
        L.ssd_layer_backward_workspace_size.restype = ctypes.c_size_t
        L.ssd_stream_workspace_size.argtypes = [ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                ctypes.c_int, ctypes.c_int, ctypes.c_int]
        L.ssd_stream_workspace_size.restype = ctypes.c_size_t
        L.ssd_scan_workspace_size.argtypes = [ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int,
                                              ctypes.c_int, ctypes.c_int]
        L.ssd_scan_workspace_size.restype = ctypes.c_size_t
        for name, args in (("ssd_packed_plan", PackedPlanArgs), ("ssd_packed_conv_forward", PackedConvArgs),
                           ("ssd_packed_conv_backward", PackedConvBwdArgs), ("ssd_packed_scan_forward", PackedScanArgs),
                           ("ssd_packed_scan_backward", PackedScanBwdArgs), ("ssd_decode_slots", DecodeSlotsArgs),
                           ("ssd_gated_rmsnorm_backward", GatedRmsnormBwdArgs)):
            getattr(L, name).argtypes = [ctypes.POINTER(args), _vp]
            getattr(L, name).restype = ctypes.c_int
        for name, args in (("ssd_packed_plan_size", [ctypes.c_int, _i64]),
                           ("ssd_packed_conv_backward_workspace_size", [ctypes.c_int, _i64, ctypes.c_int]),
                           ("ssd_packed_scan_workspace_size", [ctypes.c_int, _i64, _i64] + [ctypes.c_int] * 5),
                           ("ssd_packed_scan_backward_workspace_size", [ctypes.c_int, _i64] + [ctypes.c_int] * 3),
                           ("ssd_gated_rmsnorm_backward_workspace_size", [_i64, ctypes.c_int])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = ctypes.c_size_t
        L.ssd_sync_status.argtypes = [_vp]
        L.ssd_sync_status.restype = ctypes.c_int
        L.ssd_last_error_string.argtypes = []
        L.ssd_last_error_string.restype = ctypes.c_char_p
        L.ssd_version.argtypes = []
        L.ssd_version.restype = ctypes.c_int
        L.ssd_scan_forward_static_scratch.argtypes = [ctypes.POINTER(ScanArgs), _vp]
        L.ssd_scan_forward_static_scratch.restype = ctypes.c_int
        L.ssd_profile_begin.argtypes = []
        L.ssd_profile_begin.restype = ctypes.c_int
        L.ssd_profile_end.argtypes = [ctypes.POINTER(KernelStat), ctypes.c_int,
                                      ctypes.POINTER(ctypes.c_int)]
        L.ssd_profile_end.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc):
    if rc != 0:
        raise SSDError(rc, lib().ssd_last_error_string().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    if t.dtype == torch.float32:
        return SSD_F32
    raise TypeError(f"unsupported I/O dtype {t.dtype}")


def _cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")


def _f32(t, name):
    if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous float32 tensor")
    return t


def workspace_size(b, L, H, P, N, Q):
    return int(lib().ssd_scan_workspace_size(b, L, H, P, N, Q))


def stream_workspace_size(b, L, H, P, N, G, Q, dtype):
    """Workspace bytes of stream_forward without the conv output (keep_v=False)."""
    return int(lib().ssd_stream_workspace_size(b, L, H, P, N, G, Q, dtype))


def alloc_workspace(b, L, H, P, N, Q, device=None):
    n = workspace_size(b, L, H, P, N, Q)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device or "cuda")


def profile_begin():
    """Start timing every kernel the library launches from this thread."""
    _check(lib().ssd_profile_begin())


def profile_end():
    """Stop timing; returns {kernel name: {"launches": n, "total_ms": t}}."""
    cap = 32
    arr = (KernelStat * cap)()
    n = ctypes.c_int(0)
    _check(lib().ssd_profile_end(arr, cap, ctypes.byref(n)))
    return {arr[i].name.decode(): {"launches": int(arr[i].launches), "total_ms": float(arr[i].total_ms)}
            for i in range(min(n.value, cap))}


def sync_status(stream=None):
    _check(lib().ssd_sync_status(_stream(stream)))


def conv_forward(u, w, bias=None, tail_in=None, tail_out=None, v=None, stream=None):
    """v = silu(causal_conv1d_k4(u)); returns (v, tail_out)."""
    _cuda(u, w, bias, tail_in, tail_out, v)
    b, L, cch = u.shape
    if v is None:
        v = torch.empty_like(u)
    _f32(w, "w")
    _f32(bias, "bias")
    rc = lib().ssd_conv_forward(_ptr(u), u.stride(0), u.stride(1), _ptr(w), _ptr(bias),
                                _ptr(tail_in), _ptr(tail_out), _ptr(v), v.stride(0), v.stride(1),
                                b, L, cch, _dtype_code(u), _stream(stream))
    _check(rc)
    return v, tail_out



def _set_dt(a, dt_bias, dt_softplus, dt_limit):
    """The optional dt_bias [H] float32 / softplus / (lo, hi) clamp of the arguments."""
    _cuda(dt_bias)
    _f32(dt_bias, "dt_bias")
    a.dt_bias = dt_bias.data_ptr() if dt_bias is not None else None
    a.dt_softplus = 1 if dt_softplus else 0
    lo, hi = dt_limit if dt_limit is not None else (0.0, 0.0)
    a.dt_min, a.dt_max = float(lo), float(hi)

def scan_forward(x, B, C, dt, A, D=None, h0=None, *, H, G=1, Q=128, s=0, y=None,
                 h_final=None, h_ckpt=None, workspace=None, stream=None, dt_bias=None,
                 dt_softplus=False, dt_limit=None):
    """Chunked selective scan; returns (y, h_final, h_ckpt).

    x: [b, L, >=H*P] view (may be a column slice of the conv output),
    B, C: [b, L, >=G*N] views, dt: [b, L, H] float32, A/D: [H] float32,
    h0: [b, H, P, N] float32 or None.  dt_bias [H] / dt_softplus / dt_limit (lo, hi):
    the kernels use clamp(softplus(dt + dt_bias)) instead of dt (each part optional).
    """
    _cuda(x, B, C, dt, A, D, h0, y, h_final, h_ckpt, workspace)
    b, L = x.shape[0], x.shape[1]
    P = x.shape[2] // H
    N = B.shape[2] // G
    dev = x.device
    if y is None:
        y = torch.empty(b, L, H, P, dtype=x.dtype, device=dev)
    if h_final is None:
        h_final = torch.empty(b, H, P, N, dtype=torch.float32, device=dev)
    if h_ckpt is None and s > 0:
        h_ckpt = torch.empty(b, L // s, H, P, N, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(b, L, H, P, N, Q, dev)
    for t, n in ((dt, "dt"), (A, "A"), (D, "D"), (h0, "h0"), (h_final, "h_final"), (h_ckpt, "h_ckpt")):
        _f32(t, n)
    a = ScanArgs()
    a.dtype = _dtype_code(x); a.b = b; a.L = L; a.H = H; a.P = P; a.N = N; a.G = G; a.Q = Q; a.s = s
    a.x = x.data_ptr(); a.x_batch_stride = x.stride(0); a.x_row_stride = x.stride(1)
    a.B = B.data_ptr(); a.B_batch_stride = B.stride(0); a.B_row_stride = B.stride(1)
    a.C = C.data_ptr(); a.C_batch_stride = C.stride(0); a.C_row_stride = C.stride(1)
    a.dt = dt.data_ptr(); a.A = A.data_ptr(); a.D = D.data_ptr() if D is not None else None
    a.h0 = h0.data_ptr() if h0 is not None else None
    y2 = y.view(b, L, H * P)
    a.y = y.data_ptr(); a.y_batch_stride = y2.stride(0); a.y_row_stride = y2.stride(1)
    a.h_final = h_final.data_ptr() if h_final is not None else None
    a.h_ckpt = h_ckpt.data_ptr() if h_ckpt is not None else None
    a.workspace = workspace.data_ptr(); a.workspace_bytes = workspace.numel() * workspace.element_size()
    _set_dt(a, dt_bias, dt_softplus, dt_limit)
    _check(lib().ssd_scan_forward(ctypes.byref(a), _stream(stream)))
    return y, h_final, h_ckpt


def stream_forward(u, conv_w, dt, A, D=None, *, H, P, N, G=1, Q=128, s=0, conv_bias=None,
                   tail_in=None, tail_out=None, h0=None, v=None, y=None, h_final=None,
                   h_ckpt=None, workspace=None, stream=None, dt_bias=None, dt_softplus=False,
                   dt_limit=None, conv_ckpt=None, keep_v=True):
    """One streamed segment: conv (tail_in -> tail_out), then scan (h0 -> h_final).

    conv_ckpt: a [b, L//s, 3, C_ch] tensor (I/O dtype) to receive the conv buffer at
    every checkpoint, True to allocate one, or None.  keep_v=False (and v None):
    the conv output is not returned, and on the tensor-core shapes the conv of x is
    fused into the scan kernels (the workspace is then ssd_stream_workspace_size)."""
    _cuda(u, conv_w, dt, A, D, conv_bias, tail_in, tail_out, h0, v, y, h_final, h_ckpt, workspace)
    b, L, cch = u.shape
    assert cch == H * P + 2 * G * N, "u must hold x|B|C channels"
    dev = u.device
    if v is None and keep_v:
        v = torch.empty_like(u)
    if y is None:
        y = torch.empty(b, L, H, P, dtype=u.dtype, device=dev)
    if h_final is None:
        h_final = torch.empty(b, H, P, N, dtype=torch.float32, device=dev)
    if tail_out is None:
        tail_out = torch.empty(b, 3, cch, dtype=u.dtype, device=dev)
    if h_ckpt is None and s > 0:
        h_ckpt = torch.empty(b, L // s, H, P, N, dtype=torch.float32, device=dev)
    if workspace is None:
        if v is None:
            n = stream_workspace_size(b, L, H, P, N, G, Q, _dtype_code(u))
            workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
        else:
            workspace = alloc_workspace(b, L, H, P, N, Q, dev)
    if conv_ckpt is True:
        conv_ckpt = torch.empty(b, L // s if s > 0 else 0, 3, cch, dtype=u.dtype, device=dev)
    a = StreamArgs()
    a.dtype = _dtype_code(u); a.b = b; a.L = L; a.H = H; a.P = P; a.N = N; a.G = G; a.Q = Q; a.s = s
    a.u = u.data_ptr(); a.u_batch_stride = u.stride(0); a.u_row_stride = u.stride(1)
    a.conv_w = conv_w.data_ptr(); a.conv_bias = conv_bias.data_ptr() if conv_bias is not None else None
    a.tail_in = tail_in.data_ptr() if tail_in is not None else None
    a.tail_out = tail_out.data_ptr()
    if v is not None:
        a.v = v.data_ptr(); a.v_batch_stride = v.stride(0); a.v_row_stride = v.stride(1)
    a.dt = dt.data_ptr(); a.A = A.data_ptr(); a.D = D.data_ptr() if D is not None else None
    a.h0 = h0.data_ptr() if h0 is not None else None
    y2 = y.view(b, L, H * P)
    a.y = y.data_ptr(); a.y_batch_stride = y2.stride(0); a.y_row_stride = y2.stride(1)
    a.h_final = h_final.data_ptr()
    a.h_ckpt = h_ckpt.data_ptr() if h_ckpt is not None else None
    a.workspace = workspace.data_ptr(); a.workspace_bytes = workspace.numel()
    _set_dt(a, dt_bias, dt_softplus, dt_limit)
    a.conv_ckpt = conv_ckpt.data_ptr() if conv_ckpt is not None else None
    _check(lib().ssd_stream_forward(ctypes.byref(a), _stream(stream)))
    return {"v": v, "y": y, "h_final": h_final, "h_ckpt": h_ckpt, "tail_out": tail_out, "conv_ckpt": conv_ckpt}


def decode_step(u, conv_w, dt, A, D=None, *, H, P, N, G=1, conv_bias=None, tail_in=None,
                tail_out=None, h_in=None, h_out=None, y=None, stream=None, dt_bias=None,
                dt_softplus=False, dt_limit=None):
    """One token of b streams: u [b, C_ch] (pre-conv x|B|C), dt [b, H].  Returns
    {"y": [b, H, P], "h_out": [b, H, P, N], "tail_out": [b, 3, C_ch]}; h_out may be h_in
    and tail_out may be tail_in (updated in place)."""
    _cuda(u, conv_w, dt, A, D, conv_bias, tail_in, tail_out, h_in, h_out, y)
    b, cch = u.shape
    assert cch == H * P + 2 * G * N, "u must hold x|B|C channels"
    dev = u.device
    if y is None:
        y = torch.empty(b, H, P, dtype=u.dtype, device=dev)
    if h_out is None:
        h_out = torch.empty(b, H, P, N, dtype=torch.float32, device=dev)
    if tail_out is None:
        tail_out = torch.empty(b, 3, cch, dtype=u.dtype, device=dev)
    a = DecodeArgs()
    a.dtype = _dtype_code(u); a.b = b; a.H = H; a.P = P; a.N = N; a.G = G
    a.u = u.data_ptr(); a.u_batch_stride = u.stride(0)
    a.conv_w = conv_w.data_ptr(); a.conv_bias = conv_bias.data_ptr() if conv_bias is not None else None
    a.tail_in = tail_in.data_ptr() if tail_in is not None else None
    a.tail_out = tail_out.data_ptr()
    a.dt = dt.data_ptr(); a.A = A.data_ptr(); a.D = D.data_ptr() if D is not None else None
    a.h_in = h_in.data_ptr() if h_in is not None else None
    a.h_out = h_out.data_ptr()
    a.y = y.data_ptr(); a.y_batch_stride = y.view(b, H * P).stride(0)
    _set_dt(a, dt_bias, dt_softplus, dt_limit)
    _check(lib().ssd_decode_step(ctypes.byref(a), _stream(stream)))
    return {"y": y, "h_out": h_out, "tail_out": tail_out}


def backward_workspace_size(b, L, H, P, N):
    return int(lib().ssd_scan_backward_workspace_size(b, L, H, P, N))


def scan_backward(x, B, C, dt, A, D, dy, h0=None, h_ckpt=None, dh_final=None, *, H, G=1, s=0,
                  workspace=None, out=None, stream=None):
    """Gradients through scan_forward: returns dict dx, dB, dC, ddt, dA, dD, dh0 (float32).

    x, B, C, dt, A, D, h0: the forward's inputs (views as for scan_forward);
    dy: [b, L, >=H*P] (I/O dtype) = dLoss/dy, dh_final: [b, H, P, N] float32
    or None.  h_ckpt: the forward's checkpoints [b, L//s, H, P, N] with stride
    s, or None to rebuild the states from h0 over the whole sequence.
    ``out`` may hold preallocated outputs under the same keys.
    """
    _cuda(x, B, C, dt, A, D, dy, h0, h_ckpt, dh_final, workspace)
    b, L = x.shape[0], x.shape[1]
    P = x.shape[2] // H
    N = B.shape[2] // G
    dev = x.device
    o = dict(out or {})
    shapes = {"dx": (b, L, H, P), "dB": (b, L, G, N), "dC": (b, L, G, N), "ddt": (b, L, H),
              "dA": (H,), "dD": (H,), "dh0": (b, H, P, N)}
    for k, shp in shapes.items():
        if k not in o:
            o[k] = torch.empty(shp, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(backward_workspace_size(b, L, H, P, N), 1), dtype=torch.uint8, device=dev)
    for t, n in ((dt, "dt"), (A, "A"), (D, "D"), (h0, "h0"), (h_ckpt, "h_ckpt"), (dh_final, "dh_final"),
                 *((o[k], k) for k in shapes)):
        _f32(t, n)
    a = ScanBwdArgs()
    a.dtype = _dtype_code(x); a.b = b; a.L = L; a.H = H; a.P = P; a.N = N; a.G = G
    a.s = s if h_ckpt is not None else 0
    a.x = x.data_ptr(); a.x_batch_stride = x.stride(0); a.x_row_stride = x.stride(1)
    a.B = B.data_ptr(); a.B_batch_stride = B.stride(0); a.B_row_stride = B.stride(1)
    a.C = C.data_ptr(); a.C_batch_stride = C.stride(0); a.C_row_stride = C.stride(1)
    a.dt = dt.data_ptr(); a.A = A.data_ptr(); a.D = D.data_ptr() if D is not None else None
    a.h0 = h0.data_ptr() if h0 is not None else None
    a.h_ckpt = h_ckpt.data_ptr() if h_ckpt is not None else None
    dy3 = dy.reshape(b, L, -1) if dy.dim() == 4 else dy
    a.dy = dy3.data_ptr(); a.dy_batch_stride = dy3.stride(0); a.dy_row_stride = dy3.stride(1)
    a.dh_final = dh_final.data_ptr() if dh_final is not None else None
    a.dx = o["dx"].data_ptr(); a.dB = o["dB"].data_ptr(); a.dC = o["dC"].data_ptr()
    a.ddt = o["ddt"].data_ptr(); a.dA = o["dA"].data_ptr()
    a.dD = o["dD"].data_ptr() if o["dD"] is not None else None
    a.dh0 = o["dh0"].data_ptr() if o["dh0"] is not None else None
    a.workspace = workspace.data_ptr(); a.workspace_bytes = workspace.numel()
    _check(lib().ssd_scan_backward(ctypes.byref(a), _stream(stream)))
    return o


def layer_backward_workspace_size(b, L, H, P, N, G=1, dtype=SSD_BF16):
    return int(lib().ssd_layer_backward_workspace_size(b, L, H, P, N, G, dtype))


def layer_backward(u, conv_w, dt, A, D, dy, *, H, P, N, G=1, s=0, conv_bias=None, tail_in=None, h0=None,
                   h_ckpt=None, conv_ckpt=None, dh_final=None, dtail_out=None, workspace=None, out=None,
                   stream=None):
    """Gradients through the whole layer (conv1d + SiLU, then the scan): returns dict du,
    dtail_in, dconv_w, dconv_bias, ddt, dA, dD, dh0 (float32).

    u, conv_w, conv_bias, tail_in, dt, A, D, h0: the forward's inputs (as for
    stream_forward); dy: [b, L, >=H*P] (I/O dtype); dh_final [b, H, P, N] and
    dtail_out [b, 3, C_ch] float32 or None.  h_ckpt [b, L//s, H, P, N] and conv_ckpt
    [b, L//s, 3, C_ch] (the forward's checkpoints, s a multiple of 64) rebuild each cell
    of s tokens on its own; without them the whole sequence is rebuilt from h0, tail_in.
    """
    _cuda(u, conv_w, dt, A, D, dy, conv_bias, tail_in, h0, h_ckpt, conv_ckpt, dh_final, dtail_out, workspace)
    b, L, cch = u.shape
    assert cch == H * P + 2 * G * N, "u must hold x|B|C channels"
    dev = u.device
    o = dict(out or {})
    shapes = {"du": (b, L, cch), "dtail_in": (b, 3, cch), "dconv_w": (cch, 4), "dconv_bias": (cch,),
              "ddt": (b, L, H), "dA": (H,), "dD": (H,), "dh0": (b, H, P, N)}
    for k, shp in shapes.items():
        if k not in o:
            o[k] = torch.empty(shp, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(layer_backward_workspace_size(b, L, H, P, N, G, _dtype_code(u)), 1),
                                dtype=torch.uint8, device=dev)
    for t, n in ((conv_w, "conv_w"), (conv_bias, "conv_bias"), (dt, "dt"), (A, "A"), (D, "D"), (h0, "h0"),
                 (h_ckpt, "h_ckpt"), (dh_final, "dh_final"), (dtail_out, "dtail_out"),
                 *((o[k], k) for k in shapes if o[k] is not None)):
        _f32(t, n)
    a = LayerBwdArgs()
    a.dtype = _dtype_code(u); a.b = b; a.L = L; a.H = H; a.P = P; a.N = N; a.G = G
    a.s = s if h_ckpt is not None else 0
    a.u = u.data_ptr(); a.u_batch_stride = u.stride(0); a.u_row_stride = u.stride(1)
    a.conv_w = conv_w.data_ptr(); a.conv_bias = _vp_of(conv_bias); a.tail_in = _vp_of(tail_in)
    a.conv_ckpt = _vp_of(conv_ckpt)
    a.dt = dt.data_ptr(); a.A = A.data_ptr(); a.D = _vp_of(D); a.h0 = _vp_of(h0); a.h_ckpt = _vp_of(h_ckpt)
    dy3 = dy.reshape(b, L, -1) if dy.dim() == 4 else dy
    a.dy = dy3.data_ptr(); a.dy_batch_stride = dy3.stride(0); a.dy_row_stride = dy3.stride(1)
    a.dh_final = _vp_of(dh_final); a.dtail_out = _vp_of(dtail_out)
    a.du = o["du"].data_ptr(); a.dtail_in = _vp_of(o["dtail_in"]); a.dconv_w = o["dconv_w"].data_ptr()
    a.dconv_bias = _vp_of(o["dconv_bias"]); a.ddt = o["ddt"].data_ptr(); a.dA = o["dA"].data_ptr()
    a.dD = _vp_of(o["dD"]); a.dh0 = _vp_of(o["dh0"])
    a.workspace = workspace.data_ptr(); a.workspace_bytes = workspace.numel()
    _check(lib().ssd_layer_backward(ctypes.byref(a), _stream(stream)))
    return o


def _vp_of(t):
    return None if t is None else t.data_ptr()


def gated_rmsnorm(y, z, weight, eps=1e-5, group_size=0, out=None, stream=None):
    """out = rmsnorm(y * silu(z)) * weight over groups of ``group_size`` channels (0: all).

    y, z: [..., d] with the same leading shape, rows of d contiguous channels
    (z may be a column slice of a wider tensor); weight: [d] float32.
    """
    _cuda(y, z, weight, out)
    _f32(weight, "weight")
    d = y.shape[-1]
    y2 = y.reshape(-1, d)
    z2 = z.reshape(-1, d) if z.is_contiguous() else z.flatten(0, -2)
    if out is None:
        out = torch.empty_like(y)
    o2 = out.view(-1, d)
    if z2.dtype != y2.dtype or o2.dtype != y2.dtype:
        raise TypeError("y, z and out must share the I/O dtype")
    rc = lib().ssd_gated_rmsnorm_forward(_ptr(y2), y2.stride(0), _ptr(z2), z2.stride(0), _ptr(weight), float(eps),
                                         int(group_size), _ptr(o2), o2.stride(0), y2.shape[0], d, _dtype_code(y2),
                                         _stream(stream))
    _check(rc)
    return out


# ---------------------------------------------------------------- packed sequences and slots
# The checks below run on every call of a decoding loop: each tensor is looked at once.
def _device(t):
    """The CUDA device that a call's first tensor, and hence all of them, must be on."""
    dev = t.device
    if dev.type != "cuda":
        raise ValueError("all tensors must be CUDA tensors")
    return dev


def _ptr_of(t, shape, dtype, dev, name):
    """The data pointer of a contiguous tensor of this shape and type on `dev` (None for None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        _refuse(t, shape, dtype, dev, name)
    return t.data_ptr()


def _refuse(t, shape, dtype, dev, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"all tensors must be on {dev}, {name} is on {t.device}")
    raise TypeError(f"{name} must be a contiguous {dtype} tensor")


def _rows2(t, rows, width, dtype, dev, name):
    """(data pointer, row stride) of a [rows, width] view whose rows are contiguous."""
    if t.shape != (rows, width):
        raise ValueError(f"{name} must be [{rows}, {width}], got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"all tensors must be on {dev}, {name} is on {t.device}")
    rs, cs = t.stride()
    if cs != 1 and width > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    # a tensor of one row (or none) may carry any stride
    return t.data_ptr(), rs if rows > 1 else width


def _rows3(t, rows, H, P, dtype, dev, name):
    """(pointer, row stride) of rows of H*P elements given as [rows, H, P] or [rows, H*P]."""
    if t.dim() != 3:
        return _rows2(t, rows, H * P, dtype, dev, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"all tensors must be on {dev}, {name} is on {t.device}")
    rs, hs, ps = t.stride()
    if t.shape != (rows, H, P) or (P > 1 and ps != 1) or (H > 1 and hs != P):
        raise ValueError(f"{name} must be [{rows}, {H}, {P}] with contiguous rows, got {tuple(t.shape)}")
    return t.data_ptr(), rs if rows > 1 else H * P


# the current stream's handle without making a Stream object of it (2 us of a decoding step's 14 on the host)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _on_stream(f, args):
    """f(**args) with args' stream current, so that what f allocates or clears is ordered on that stream too, not on the
    one that was current (whose next tensors would take a freed workspace's place while the call still runs)."""
    stream = args.pop("stream")
    t = next(iter(args.values()))
    if stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.stream(stream):
        return f(**args)


def _launch(fn, a, dev, stream):
    """Call a C entry point with `dev` current, on `stream` or the device's current stream."""
    if dev.index is not None and dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _launch(fn, a, dev, stream)
    _check(fn(ctypes.byref(a), stream.cuda_stream if stream is not None else _raw_stream(dev.index or 0)))


def _bytes_on(dev, n):
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=dev)


def _memory(t, dev, name):
    """(data pointer, bytes behind it) of a buffer of any type: a view's elements need not all lie there."""
    if t.device != dev:
        raise ValueError(f"all tensors must be on {dev}, {name} is on {t.device}")
    if not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")
    return t.data_ptr(), t.nbytes


def _set_ws(a, workspace, dev):
    a.workspace, a.workspace_bytes = _memory(workspace, dev, "workspace")


def _outputs(out, shapes, dev):
    """The float32 outputs of these shapes: those given in `out`, the others allocated (zero); with their pointers."""
    o, ptr = dict(out or {}), {}
    for k, shp in shapes:
        if k not in o:
            o[k] = torch.zeros(shp, dtype=torch.float32, device=dev)
        ptr[k] = _ptr_of(o[k], shp, torch.float32, dev, k)
    return o, ptr


class PackedPlan:
    """The plan of a packed batch (packed_plan): keep it while calls on the batch are in flight."""

    def __init__(self, buf, nseq, total, n_slots, max_seqlen, has_slots):
        self.buf, self.nseq, self.total, self.n_slots = buf, nseq, total, n_slots
        self.max_seqlen, self.has_slots, self.device = max_seqlen, has_slots, buf.device


def packed_plan(cu_seqlens, total, *, slots=None, resume=None, n_slots=0, max_seqlen=0, buf=None, stream=None):
    """The plan of a batch of sequences laid end to end: sequence i has rows cu_seqlens[i] .. cu_seqlens[i+1]-1
    of tensors with `total` rows.  Made on the device, once per batch, and taken by every packed call.

    cu_seqlens [n+1] int32; slots [n] int32 or None (sequence i has slot i), -1 = not kept; resume [n] int32 or
    None (all): 0 = start from zero; n_slots: slots of the state pools (0 without slots: n); max_seqlen: a
    bound of the lengths (0: total).  buf: the plan's memory (uint8, lib().ssd_packed_plan_size(n, total)
    bytes), to make it again in the same place (under a captured graph).
    """
    if stream is not None:
        return _on_stream(packed_plan, locals())
    dev = _device(cu_seqlens)
    n = cu_seqlens.numel() - 1
    if n < 0:
        raise ValueError("cu_seqlens needs at least one entry")
    if slots is not None and n_slots <= 0 and n > 0:
        raise ValueError("n_slots is needed with slots")
    a = PackedPlanArgs()
    a.nseq = n; a.total = total; a.n_slots = n_slots; a.max_seqlen = max_seqlen
    a.cu_seqlens = _ptr_of(cu_seqlens, (n + 1,), torch.int32, dev, "cu_seqlens")
    a.slots = _ptr_of(slots, (n,), torch.int32, dev, "slots")
    a.resume = _ptr_of(resume, (n,), torch.int32, dev, "resume")
    if buf is None:
        buf = _bytes_on(dev, lib().ssd_packed_plan_size(n, total))
    a.plan, a.plan_bytes = _memory(buf, dev, "buf")
    _launch(lib().ssd_packed_plan, a, dev, stream)
    return PackedPlan(buf, n, int(total), n_slots if slots is not None else max(n_slots, n), int(max_seqlen), slots is not None)


def _plan_args(a, plan, rows, dev):
    if rows != plan.total:
        raise ValueError(f"the plan is for {plan.total} rows, the tensors have {rows}")
    if plan.device != dev:
        raise ValueError(f"the plan is on {plan.device}, the tensors on {dev}")
    a.nseq = plan.nseq; a.total = rows; a.plan = plan.buf.data_ptr()


def packed_conv_forward(u, w, plan, bias=None, tail_in=None, tail_out=None, v=None, stream=None):
    """v = silu(causal_conv1d_k4(u)) on each sequence of the plan; returns (v, tail_out).

    u: [total, C_ch] (a view with any row stride of whole 16 bytes); tail_in, tail_out: [n_slots, 3, C_ch] or
    None, tail_out may be tail_in.  Rows of v that belong to no sequence stay as they were.
    """
    if stream is not None:
        return _on_stream(packed_conv_forward, locals())
    dev = _device(u)
    total, cch = u.shape
    dt = u.dtype
    if v is None:
        v = torch.empty(total, cch, dtype=dt, device=dev)
    a = PackedConvArgs()
    a.dtype = _dtype_code(u); a.C_ch = cch
    _plan_args(a, plan, total, dev)
    a.u, a.u_row_stride = _rows2(u, total, cch, dt, dev, "u")
    a.v, a.v_row_stride = _rows2(v, total, cch, dt, dev, "v")
    a.conv_w = _ptr_of(w, (cch, 4), torch.float32, dev, "w")
    a.conv_bias = _ptr_of(bias, (cch,), torch.float32, dev, "bias")
    a.tail_in = _ptr_of(tail_in, (plan.n_slots, 3, cch), dt, dev, "tail_in")
    a.tail_out = _ptr_of(tail_out, (plan.n_slots, 3, cch), dt, dev, "tail_out")
    _launch(lib().ssd_packed_conv_forward, a, dev, stream)
    return v, tail_out


def packed_conv_backward_workspace(plan, cch):
    """Workspace of packed_conv_backward for this plan and channel count."""
    return _bytes_on(plan.device, lib().ssd_packed_conv_backward_workspace_size(plan.nseq, plan.total, cch))


def packed_conv_backward(u, w, plan, dx, dB, dC, *, bias=None, tail_in=None, dtail_out=None, out=None, workspace=None, stream=None):
    """Gradients through packed_conv_forward: dict du [total, C_ch], dtail_in [n, 3, C_ch], dconv_w, dconv_bias (float32).

    dx [total, (H, P)], dB, dC [total, (G, N)]: float32 gradients of v's columns, as packed_scan_backward returns
    them; dtail_out: [n, 3, C_ch] float32 or None, by sequence.  Without tail_in no sequence resumes: dtail_in is
    zero (a pool of zeros gives the gradient of a start from zeros).  ``out`` may hold outputs under the same keys;
    rows of no sequence stay as they were in them, and are zero in those allocated here.
    """
    if stream is not None:
        return _on_stream(packed_conv_backward, locals())
    dev = _device(u)
    total, cch = u.shape
    hp, gn = math.prod(dx.shape[1:]), math.prod(dB.shape[1:])
    if dx.shape[0] != total or dB.shape[0] != total or dC.shape != dB.shape or hp + 2 * gn != cch:
        raise ValueError(f"dx, dB and dC must be [{total}, ...] with {cch} channels in all")
    n = plan.nseq
    o, ptr = _outputs(out, (("du", (total, cch)), ("dtail_in", (n, 3, cch)), ("dconv_w", (cch, 4)), ("dconv_bias", (cch,))), dev)
    a = PackedConvBwdArgs()
    a.dtype = _dtype_code(u); a.d_inner = hp; a.d_bc = gn
    _plan_args(a, plan, total, dev)
    a.u, a.u_row_stride = _rows2(u, total, cch, u.dtype, dev, "u")
    a.conv_w = _ptr_of(w, (cch, 4), torch.float32, dev, "w")
    a.conv_bias = _ptr_of(bias, (cch,), torch.float32, dev, "bias")
    a.tail_in = _ptr_of(tail_in, (plan.n_slots, 3, cch), u.dtype, dev, "tail_in")
    a.dx = _ptr_of(dx, dx.shape, torch.float32, dev, "dx")
    a.dB = _ptr_of(dB, dB.shape, torch.float32, dev, "dB")
    a.dC = _ptr_of(dC, dC.shape, torch.float32, dev, "dC")
    a.dtail_out = _ptr_of(dtail_out, (n, 3, cch), torch.float32, dev, "dtail_out")
    a.du = ptr["du"]; a.dtail_in = ptr["dtail_in"]; a.dconv_w = ptr["dconv_w"]; a.dconv_bias = ptr["dconv_bias"]
    _set_ws(a, workspace if workspace is not None else packed_conv_backward_workspace(plan, cch), dev)
    _launch(lib().ssd_packed_conv_backward, a, dev, stream)
    return o


def packed_scan_workspace(plan, H, P, N, dtype, G=1):
    """Workspace of packed_scan_forward for this plan, these heads and this I/O dtype."""
    code = SSD_BF16 if dtype == torch.bfloat16 else SSD_F32
    with torch.cuda.device(plan.device):
        n = lib().ssd_packed_scan_workspace_size(plan.nseq, plan.total, plan.max_seqlen, H, P, N, G, code)
    return _bytes_on(plan.device, n)


def _head_dims(x, B, H, G):
    if H <= 0 or G <= 0 or x.dim() != 2 or B.dim() != 2 or x.shape[1] % H or B.shape[1] % G:
        raise ValueError(f"x must be [total, H*P], B and C [total, G*N] (H={H}, G={G}); got {tuple(x.shape)}, {tuple(B.shape)}")
    return x.shape[1] // H, B.shape[1] // G


def _scan_inputs(a, x, B, C, dt, A, D, h_in, plan, H, G, dev):
    """The arguments that the scan and its gradient share; returns (total, P, N)."""
    P, N = _head_dims(x, B, H, G)
    total, io = x.shape[0], x.dtype
    a.dtype = _dtype_code(x); a.H = H; a.P = P; a.N = N; a.G = G
    _plan_args(a, plan, total, dev)
    a.x, a.x_row_stride = _rows2(x, total, H * P, io, dev, "x")
    a.B, a.B_row_stride = _rows2(B, total, G * N, io, dev, "B")
    a.C, a.C_row_stride = _rows2(C, total, G * N, io, dev, "C")
    a.dt = _ptr_of(dt, (total, H), torch.float32, dev, "dt")
    a.A = _ptr_of(A, (H,), torch.float32, dev, "A")
    a.D = _ptr_of(D, (H,), torch.float32, dev, "D")
    a.h_in = _ptr_of(h_in, (plan.n_slots, H, P, N), torch.float32, dev, "h_in")
    return total, P, N


def _dt_args(a, dt_bias, dt_softplus, dt_limit, H, dev):
    a.dt_bias = _ptr_of(dt_bias, (H,), torch.float32, dev, "dt_bias")
    a.dt_softplus = 1 if dt_softplus else 0
    if dt_limit is not None:
        a.dt_min, a.dt_max = dt_limit


def packed_scan_forward(x, B, C, dt, A, D=None, *, plan, H, G=1, h_in=None, h_out=None, y=None, workspace=None,
                        stream=None, dt_bias=None, dt_softplus=False, dt_limit=None):
    """The selective scan on each sequence of the plan; returns (y [total, H, P], h_out).

    x: [total, H*P], B, C: [total, G*N] views (column slices of the conv output), dt: [total, H] float32,
    A, D: [H] float32.  h_in, h_out: [n_slots, H, P, N] float32 or None; h_out may be h_in (updated in place);
    slots that the batch does not name stay as they were.  dt_bias / dt_softplus / dt_limit as in scan_forward.
    Rows of y that belong to no sequence stay as they were.
    """
    if stream is not None:
        return _on_stream(packed_scan_forward, locals())
    dev = _device(x)
    a = PackedScanArgs()
    total, P, N = _scan_inputs(a, x, B, C, dt, A, D, h_in, plan, H, G, dev)
    if y is None:
        y = torch.empty(total, H, P, dtype=x.dtype, device=dev)
    a.max_seqlen = plan.max_seqlen
    a.y, a.y_row_stride = _rows3(y, total, H, P, x.dtype, dev, "y")
    _dt_args(a, dt_bias, dt_softplus, dt_limit, H, dev)
    a.h_out = _ptr_of(h_out, (plan.n_slots, H, P, N), torch.float32, dev, "h_out")
    _set_ws(a, workspace if workspace is not None else packed_scan_workspace(plan, H, P, N, x.dtype, G), dev)
    _launch(lib().ssd_packed_scan_forward, a, dev, stream)
    return y, h_out


def packed_scan_backward_workspace(plan, H, P, N):
    """Workspace of packed_scan_backward for this plan and these heads."""
    with torch.cuda.device(plan.device):
        n = lib().ssd_packed_scan_backward_workspace_size(plan.nseq, plan.total, H, P, N)
    return _bytes_on(plan.device, n)


def packed_scan_backward(x, B, C, dt, A, D, dy, *, plan, H, G=1, h_in=None, dh_out=None, out=None, workspace=None, stream=None):
    """Gradients through packed_scan_forward: dict dx [total, H, P], dB, dC [total, G, N], ddt [total, H], dA, dD [H],
    dh_in [n, H, P, N] (float32).

    x, B, C, dt, A, D, h_in as in the forward (dt the step that the scan used); dy: [total, H*P] or
    [total, H, P]; dh_out: [n, H, P, N] float32 or None.  dh_out and dh_in go by sequence, h_in by slot.
    Without h_in no sequence resumes: dh_in is zero (a pool of zeros gives the gradient of a start from zeros).
    ``out`` may hold outputs under the same keys; rows of no sequence stay as they were in them, and are
    zero in those allocated here.
    """
    if stream is not None:
        return _on_stream(packed_scan_backward, locals())
    dev = _device(x)
    a = PackedScanBwdArgs()
    total, P, N = _scan_inputs(a, x, B, C, dt, A, D, h_in, plan, H, G, dev)
    n = plan.nseq
    o, ptr = _outputs(out, (("dx", (total, H, P)), ("dB", (total, G, N)), ("dC", (total, G, N)), ("ddt", (total, H)), ("dA", (H,)),
                            ("dD", (H,)), ("dh_in", (n, H, P, N))), dev)
    a.dy, a.dy_row_stride = _rows3(dy, total, H, P, x.dtype, dev, "dy")
    a.dh_out = _ptr_of(dh_out, (n, H, P, N), torch.float32, dev, "dh_out")
    a.dx = ptr["dx"]; a.dB = ptr["dB"]; a.dC = ptr["dC"]; a.ddt = ptr["ddt"]
    a.dA = ptr["dA"]; a.dD = ptr["dD"]; a.dh_in = ptr["dh_in"]
    _set_ws(a, workspace if workspace is not None else packed_scan_backward_workspace(plan, H, P, N), dev)
    _launch(lib().ssd_packed_scan_backward, a, dev, stream)
    return o


def decode_slots(u, conv_w, dt, A, D=None, *, slots, tail_in, h_in, H, P, N, G=1, conv_bias=None, tail_out=None, h_out=None,
                 y=None, stream=None, dt_bias=None, dt_softplus=False, dt_limit=None):
    """One token of b streams of a pool: u [b, C_ch], dt [b, H], slots [b] int32 (-1 = an empty row, whose y is
    zero).  tail_in, tail_out: [n_slots, 3, C_ch], h_in, h_out: [n_slots, H, P, N] float32; without tail_out /
    h_out they are updated in place.  Returns {"y": [b, H, P], "h_out", "tail_out"}."""
    if stream is not None:
        return _on_stream(decode_slots, locals())
    dev = _device(u)
    b, cch = u.shape
    io, f32 = u.dtype, torch.float32
    if cch != H * P + 2 * G * N:
        raise ValueError(f"u must hold H*P + 2*G*N = {H * P + 2 * G * N} channels, has {cch}")
    if tail_out is None:
        tail_out = tail_in
    if h_out is None:
        h_out = h_in
    if y is None:
        y = torch.empty(b, H, P, dtype=io, device=dev)
    n = h_in.shape[0]
    a = DecodeSlotsArgs()
    a.dtype = _dtype_code(u); a.b = b; a.n_slots = n; a.H = H; a.P = P; a.N = N; a.G = G
    a.slots = _ptr_of(slots, (b,), torch.int32, dev, "slots")
    a.u, a.u_batch_stride = _rows2(u, b, cch, io, dev, "u")
    a.y, a.y_batch_stride = _rows3(y, b, H, P, io, dev, "y")
    a.conv_w = _ptr_of(conv_w, (cch, 4), f32, dev, "conv_w")
    a.conv_bias = _ptr_of(conv_bias, (cch,), f32, dev, "conv_bias")
    pool = (n, H, P, N)
    a.h_in = _ptr_of(h_in, pool, f32, dev, "h_in")
    a.h_out = a.h_in if h_out is h_in else _ptr_of(h_out, pool, f32, dev, "h_out")
    pool = (n, 3, cch)
    a.tail_in = _ptr_of(tail_in, pool, io, dev, "tail_in")
    a.tail_out = a.tail_in if tail_out is tail_in else _ptr_of(tail_out, pool, io, dev, "tail_out")
    a.dt = _ptr_of(dt, (b, H), f32, dev, "dt")
    a.A = _ptr_of(A, (H,), f32, dev, "A")
    a.D = _ptr_of(D, (H,), f32, dev, "D")
    _dt_args(a, dt_bias, dt_softplus, dt_limit, H, dev)
    _launch(lib().ssd_decode_slots, a, dev, stream)
    return {"y": y, "h_out": h_out, "tail_out": tail_out}


def _norm_rows(t, shape, dtype, dev, name):
    """(pointer, row stride) of a [..., d] tensor whose leading dimensions step through memory evenly."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dim() != 2:
        t = t.view(-1, shape[-1])
    return _rows2(t, t.shape[0], shape[-1], dtype, dev, name)


def gated_rmsnorm_backward_workspace(rows, d, device=None):
    """Workspace of gated_rmsnorm_backward for this many rows of d channels."""
    dev = torch.device(device or "cuda")
    with torch.cuda.device(dev):
        return _bytes_on("cuda", lib().ssd_gated_rmsnorm_backward_workspace_size(rows, d))


def gated_rmsnorm_backward(dout, y, z, weight, eps=1e-5, group_size=0, out=None, workspace=None, stream=None):
    """Gradients through gated_rmsnorm: dict dy, dz (I/O dtype, shaped like y), dweight [d] float32.

    dout, y, z: [..., d] with the same leading shape, rows of d contiguous channels.  ``out`` may hold outputs
    under the same keys; dy may be dout or y, dz may be z (a row is read before it is written).
    """
    if stream is not None:
        return _on_stream(gated_rmsnorm_backward, locals())
    dev = _device(y)
    shape, io = y.shape, y.dtype
    d = shape[-1]
    o = dict(out or {})
    for k in ("dy", "dz"):
        if k not in o:
            o[k] = torch.empty(shape, dtype=io, device=dev)
    if "dweight" not in o:
        o["dweight"] = torch.empty(d, dtype=torch.float32, device=dev)
    a = GatedRmsnormBwdArgs()
    a.dtype = _dtype_code(y); a.d = d; a.rows = y.numel() // d; a.group_size = int(group_size); a.eps = eps
    a.dout, a.dout_row_stride = _norm_rows(dout, shape, io, dev, "dout")
    a.y, a.y_row_stride = _norm_rows(y, shape, io, dev, "y")
    a.z, a.z_row_stride = _norm_rows(z, shape, io, dev, "z")
    a.dy, a.dy_row_stride = _norm_rows(o["dy"], shape, io, dev, "dy")
    a.dz, a.dz_row_stride = _norm_rows(o["dz"], shape, io, dev, "dz")
    a.weight = _ptr_of(weight, (d,), torch.float32, dev, "weight")
    a.dweight = _ptr_of(o["dweight"], (d,), torch.float32, dev, "dweight")
    _set_ws(a, workspace if workspace is not None else gated_rmsnorm_backward_workspace(a.rows, d, dev), dev)
    _launch(lib().ssd_gated_rmsnorm_backward, a, dev, stream)
    return o
