"""Python binding of the C ABI in ``include/gdn.h`` (ctypes; argument marshalling only).

Every step of the prefill runs in the CUDA library ``libgdn.so``; this module only
turns tensors into pointers.  There is no fallback: if the library cannot be loaded
(not built, or no CUDA runtime) the calls raise.

Functions keep the C names: ``gdn_prefill``, ``gdn_prefill_host``,
``gdn_abi_version``, ``gdn_strerror``, ``gdn_last_cuda_error``,
``gdn_workspace_bytes``, ``gdn_scan_segments``, ``gdn_release_workspace``.  ``prefill`` is a convenience
wrapper that allocates the outputs with PyTorch and checks the status, and so are ``causal_conv``,
``causal_conv_step``, ``ssm_scan``, ``ssm_step`` and ``add_norm`` for the operators around the recurrence;
these take tensors with their strides, check types and shapes (``ValueError``), run on the tensors' device, and
write into given output buffers where the caller has them, else into new ones of the stream that the call runs on.
"""

from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

GDN_OK = 0
GDN_ERR_ARG = -1
GDN_ERR_ALIGN = -2
GDN_ERR_ALLOC = -3
GDN_ERR_LAUNCH = -4
GDN_ERR_SCRATCH = -5
GDN_STATIC_SCRATCH_BYTES = 128 << 20
GDN_FLAG_L2NORM_QK = 1
GDN_FLAG_TWO_LEVEL = 2
GDN_FLAG_ONE_LEVEL = 4
GDN_FLAG_SLICE32 = 0x10000
GDN_FLAG_SLICE16 = 0x40000
GDN_FLAG_SLICE64 = 0x20000
GDN_FLAG_WIDE_RANGE = 0x80000
GDN_STATUS_MMA_TIMEOUT = 1
GDN_STATUS_LOAD_TIMEOUT = 2
GDN_STATUS_PREP_LOAD_TIMEOUT = 4
GDN_STATUS_BAD_CU_SEQLENS = 8
GDN_STATUS_NONFINITE_STATE = 16
GDN_STATUS_SMALL_STATE = 32
GDN_CONV_SILU = 1
GDN_SSM_SOFTPLUS = 1
GDN_SSM_DT_F32 = 2
GDN_NORM_E4M3 = 1


def GDN_FLAG_SEGMENTS(n: int) -> int:
    """Segment count for GDN_FLAG_TWO_LEVEL, in flag bits 8..15."""
    return (int(n) & 0xFF) << 8


EXPORTED = ("gdn_abi_version", "gdn_strerror", "gdn_last_cuda_error", "gdn_prefill",
            "gdn_prefill_host", "gdn_prefill_static", "gdn_prefill_ws", "gdn_prefill_ex", "gdn_decode",
            "gdn_set_phase_events", "gdn_workspace_bytes", "gdn_scan_segments", "gdn_release_workspace",
            "gdn_device_status", "gdn_selftest_wait_timeout", "gdn_selftest_static_wait_timeout",
            "gdn_debug_fail_allocations", "gdn_conv", "gdn_conv_step", "gdn_ssm_scan", "gdn_ssm_workspace_bytes",
            "gdn_debug_ssm_wait_polls", "gdn_ssm_step", "gdn_add_norm")

_lock = threading.Lock()
_lib = None
_UNTRIED = object()
_fast = _UNTRIED  # the gdn_torch module (the tensor functions' common case in C++), or None where there is none


class GdnError(RuntimeError):
    def __init__(self, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        super().__init__(f"gdn status {status}: {gdn_strerror(status)}"
                         + (f" (cudaError {cuda_error})" if cuda_error else ""))


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False):
    """Load libgdn.so (optionally building it first) and declare the signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if build_if_missing and _build.needs_build():
            _build.build()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                               "or python -m hybrid_linear_attention_prefill_gb300.build")
        lib = ctypes.CDLL(path)
        vp, fp, ip, i = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        sig = [vp, vp, vp, fp, fp, ip, fp, vp, fp, i, i, i, i, i, i, vp]
        lib.gdn_prefill.argtypes = sig
        lib.gdn_prefill.restype = i
        lib.gdn_prefill_host.argtypes = sig
        lib.gdn_prefill_host.restype = i
        lib.gdn_prefill_static.argtypes = sig
        lib.gdn_prefill_static.restype = i
        lib.gdn_prefill_ws.argtypes = sig[:-1] + [vp, ctypes.c_size_t, vp]
        lib.gdn_prefill_ws.restype = i
        lib.gdn_prefill_ex.argtypes = sig[:-1] + [ctypes.c_uint, vp]
        lib.gdn_prefill_ex.restype = i
        lib.gdn_decode.argtypes = [vp, vp, vp, fp, fp, fp, vp, i, i, i, i, i, vp]
        lib.gdn_decode.restype = i
        lib.gdn_abi_version.argtypes = []
        lib.gdn_abi_version.restype = i
        lib.gdn_strerror.argtypes = [i]
        lib.gdn_strerror.restype = ctypes.c_char_p
        lib.gdn_last_cuda_error.argtypes = []
        lib.gdn_last_cuda_error.restype = i
        lib.gdn_workspace_bytes.argtypes = [i] * 7
        lib.gdn_workspace_bytes.restype = ctypes.c_size_t
        lib.gdn_scan_segments.argtypes = [i] * 7 + [ctypes.c_uint]
        lib.gdn_scan_segments.restype = i
        lib.gdn_set_phase_events.argtypes = [vp, vp, vp]
        lib.gdn_set_phase_events.restype = None
        lib.gdn_device_status.argtypes = [ctypes.POINTER(ctypes.c_int)]
        lib.gdn_device_status.restype = i
        lib.gdn_selftest_wait_timeout.argtypes = [i, ctypes.POINTER(ctypes.c_int)]
        lib.gdn_selftest_wait_timeout.restype = i
        lib.gdn_selftest_static_wait_timeout.argtypes = [i]
        lib.gdn_selftest_static_wait_timeout.restype = i
        lib.gdn_debug_fail_allocations.argtypes = [i]
        lib.gdn_debug_fail_allocations.restype = i
        lib.gdn_debug_ssm_wait_polls.argtypes = [i]
        lib.gdn_debug_ssm_wait_polls.restype = i
        lib.gdn_ssm_workspace_bytes.argtypes = [i] * 7
        lib.gdn_ssm_workspace_bytes.restype = ctypes.c_size_t
        for name in ("gdn_conv", "gdn_conv_step", "gdn_ssm_scan", "gdn_ssm_step", "gdn_add_norm"):
            getattr(lib, name).argtypes = [ctypes.c_char_p]  # the packed argument struct
            getattr(lib, name).restype = i
        lib.gdn_release_workspace.argtypes = []
        lib.gdn_release_workspace.restype = None
        _lib = lib
        return lib


def _shorter():
    """The gdn_torch module, loaded at a tensor function's first call (the other entries need no PyTorch), or None
    where it was not built or does not load: the tensor functions then check in Python."""
    global _fast
    if _fast is _UNTRIED:
        load()
        with _lock:
            if _fast is _UNTRIED:
                _fast = _load_fast()
    return _fast


def _load_fast():
    import importlib.util
    import warnings

    path = _build.torch_lib()  # (PyTorch's libraries have to be there first)
    if not os.path.exists(path):
        return None
    try:
        spec = importlib.util.spec_from_file_location("gdn_torch", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except (ImportError, OSError) as e:
        warnings.warn(f"{path} does not load ({e}): the tensor functions check in Python")
        return None
    return module


def _ptr(x):
    """Device/host address of a tensor, array or integer (None stays NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):  # torch.Tensor
        return x.data_ptr()
    if hasattr(x, "ctypes"):  # numpy.ndarray
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)!r}")


def _stream(s):
    if s is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def gdn_abi_version() -> int:
    return load().gdn_abi_version()


def gdn_strerror(status: int) -> str:
    return load().gdn_strerror(status).decode()


def gdn_last_cuda_error() -> int:
    return load().gdn_last_cuda_error()


def gdn_workspace_bytes(B, T, Hk, Hv, dk, dv, packed) -> int:
    return load().gdn_workspace_bytes(B, T, Hk, Hv, dk, dv, int(bool(packed)))


def gdn_scan_segments(B, T, Hk, Hv, dk, dv, packed, flags=0) -> int:
    """Segments per sequence gdn_prefill(_ex) would use on the current device (1 = single-level)."""
    return load().gdn_scan_segments(B, T, Hk, Hv, dk, dv, int(bool(packed)), int(flags))


def gdn_set_phase_events(ev_begin, ev_mid, ev_end) -> None:
    """Record three CUDA events around the next gdn_prefill's kernels (handles or torch events)."""
    def h(e):
        if e is None or isinstance(e, int):
            return e
        return e.cuda_event
    load().gdn_set_phase_events(h(ev_begin), h(ev_mid), h(ev_end))


def gdn_device_status():
    """(status code, device status bits of the library workspace and the static array); clears them."""
    st = ctypes.c_int(0)
    rc = load().gdn_device_status(ctypes.byref(st))
    return rc, st.value


def gdn_selftest_wait_timeout(max_polls):
    """(status code, recorded bits) of a bounded wait that is made to run out."""
    st = ctypes.c_int(0)
    rc = load().gdn_selftest_wait_timeout(int(max_polls), ctypes.byref(st))
    return rc, st.value


def gdn_selftest_static_wait_timeout(max_polls) -> int:
    """A bounded wait made to run out, recording into gdn_prefill_static's status word."""
    return load().gdn_selftest_static_wait_timeout(int(max_polls))


def gdn_debug_fail_allocations(count) -> int:
    """Make the library's next `count` device allocations fail; returns the pending count."""
    return load().gdn_debug_fail_allocations(int(count))


def gdn_debug_ssm_wait_polls(polls) -> int:
    """How often a wait of the selective scan's kernels looks before it gives up; returns the limit before."""
    return load().gdn_debug_ssm_wait_polls(int(polls))


def gdn_release_workspace() -> None:
    load().gdn_release_workspace()


def gdn_prefill(q, k, v, g, beta, cu_seqlens, init_state, out, final_state,
                B, T, Hk, Hv, dk, dv, stream=None) -> int:
    """Call the C entry point on device buffers; returns the status code."""
    return load().gdn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                              _ptr(init_state), _ptr(out), _ptr(final_state),
                              int(B), int(T), int(Hk), int(Hv), int(dk), int(dv), _stream(stream))


def gdn_prefill_host(q, k, v, g, beta, cu_seqlens, init_state, out, final_state,
                     B, T, Hk, Hv, dk, dv, stream=None) -> int:
    """Call the C entry point on host buffers (synchronises the stream); returns the status."""
    return load().gdn_prefill_host(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                   _ptr(init_state), _ptr(out), _ptr(final_state),
                                   int(B), int(T), int(Hk), int(Hv), int(dk), int(dv), _stream(stream))


def gdn_prefill_static(q, k, v, g, beta, cu_seqlens, init_state, out, final_state,
                       B, T, Hk, Hv, dk, dv, stream=None) -> int:
    """Call the allocation-free entry point (fixed device scratch); returns the status."""
    return load().gdn_prefill_static(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                     _ptr(init_state), _ptr(out), _ptr(final_state),
                                     int(B), int(T), int(Hk), int(Hv), int(dk), int(dv), _stream(stream))


def gdn_prefill_ws(q, k, v, g, beta, cu_seqlens, init_state, out, final_state,
                   B, T, Hk, Hv, dk, dv, workspace, workspace_bytes, stream=None) -> int:
    """Call the caller-workspace entry point (no allocation, no host sync); returns the status."""
    return load().gdn_prefill_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                 _ptr(init_state), _ptr(out), _ptr(final_state),
                                 int(B), int(T), int(Hk), int(Hv), int(dk), int(dv),
                                 _ptr(workspace), int(workspace_bytes), _stream(stream))


def gdn_prefill_ex(q, k, v, g, beta, cu_seqlens, init_state, out, final_state,
                   B, T, Hk, Hv, dk, dv, flags, stream=None) -> int:
    """gdn_prefill with option flags (GDN_FLAG_*); returns the status."""
    return load().gdn_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                 _ptr(init_state), _ptr(out), _ptr(final_state),
                                 int(B), int(T), int(Hk), int(Hv), int(dk), int(dv), int(flags),
                                 _stream(stream))


def gdn_decode(q, k, v, g, beta, state, out, B, Hk, Hv, dk, dv, stream=None) -> int:
    """One token per sequence, state updated in place; returns the status."""
    return load().gdn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(out),
                             int(B), int(Hk), int(Hv), int(dk), int(dv), _stream(stream))


def check(status: int) -> None:
    if status != GDN_OK:
        raise GdnError(status, gdn_last_cuda_error())


def _output(shape, dtype, device, stream):
    """A tensor for a call on `stream` to write, from that stream's memory: what the current stream freed its work
    may still use, and what is freed to it its next tensor may take while the call runs."""
    import torch

    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream if isinstance(stream, int) else stream.cuda_stream
        # 0 and 1 are CUDA's names of the legacy default stream
        stream = torch.cuda.ExternalStream(raw, device) if raw > 1 else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def prefill(q, k, v, g, beta, cu_seqlens=None, init_state=None, *, B=None, want_final=True, stream=None):
    """Allocate outputs and run ``gdn_prefill`` on CUDA tensors.

    q, k: bf16 [Ttot, Hk, dk]; v: bf16 [Ttot, Hv, dv]; g, beta: fp32 [Ttot, Hv];
    cu_seqlens: int32 [B+1] or None; init_state: fp32 [B, Hv, dv, dk] or None.
    Returns (out bf16 [Ttot, Hv, dv], final_state fp32 [B, Hv, dv, dk] or None).
    """
    import torch

    Ttot, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    if cu_seqlens is not None:
        B = cu_seqlens.numel() - 1
        T = Ttot
    else:
        B = 1 if B is None else B
        T = Ttot // B if B else 0
    out = _output((Ttot, Hv, dv), torch.bfloat16, q.device, stream)
    fin = _output((B, Hv, dv, dk), torch.float32, q.device, stream) if want_final else None
    with torch.cuda.device(q.device):
        check(gdn_prefill(q, k, v, g, beta, cu_seqlens, init_state, out, fin, B, T, Hk, Hv, dk, dv, stream))
    return out, fin


# ---- the operators around the recurrence -----------------------------------------------------
#
# Their C entries take a struct: packed here in the C layout (native alignment; P pointer, q long long,
# i int, I unsigned, N size_t, f float).  A call costs about as much as its launch, so the checks are
# written for speed.

_CONV = struct.Struct("@PqPPPPPPiiiiIP")
_CONV_STEP = struct.Struct("@PqPPPPiiiIP")
_SSM_SCAN = struct.Struct("@PqPqPPqPqPPqPPPPPiiiiiiIPNP")
_SSM_STEP = struct.Struct("@PqPqPPqPqPPqPPPiiiiiIP")
_NORM = struct.Struct("@PqPPPPPiiifIP")


def _addr(x) -> int:
    """Address of a tensor, array or integer; 0 for None."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return _ptr(x)


def _raw_stream(stream, device_index) -> int:
    if device_index < 0:
        raise ValueError("CUDA tensors are wanted")
    if stream is None:
        import torch

        return torch._C._cuda_getCurrentRawStream(device_index)
    if isinstance(stream, int):
        return stream
    of = getattr(stream, "device", None)
    _want(of is None or of.index == device_index, f"stream: one of the device of x is wanted, got one of {of}")
    return stream.cuda_stream


def _call(entry, args, device_index) -> None:
    """A C entry with its arguments packed, on this device: the entries launch on the current one."""
    import torch

    with torch.cuda.device(device_index):
        check(entry(args))


def gdn_conv(x, x_stride, weight, bias, cu_seqlens, init_state, out, final_state, B, T, C, K, flags,
             stream=None) -> int:
    """Short causal convolution of a prompt; returns the status."""
    return load().gdn_conv(_CONV.pack(_addr(x), x_stride, _addr(weight), _addr(bias), _addr(cu_seqlens),
                                      _addr(init_state), _addr(out), _addr(final_state), B, T, C, K, flags,
                                      _stream(stream)))


def gdn_conv_step(x, x_stride, weight, bias, state, out, B, C, K, flags, stream=None) -> int:
    """One token per sequence of the convolution, state updated in place; returns the status."""
    return load().gdn_conv_step(_CONV_STEP.pack(_addr(x), x_stride, _addr(weight), _addr(bias), _addr(state),
                                                _addr(out), B, C, K, flags, _stream(stream)))


def gdn_ssm_scan(x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, D, z, z_stride, dt_bias, cu_seqlens,
                 init_state, out, final_state, B, T, Hk, Hv, dk, dv, flags, workspace=None, workspace_bytes=0,
                 stream=None) -> int:
    """Selective state space scan of a prompt; returns the status."""
    return load().gdn_ssm_scan(_SSM_SCAN.pack(
        _addr(x), x_stride, _addr(dt), dt_stride, _addr(A), _addr(Bm), b_stride, _addr(Cm), c_stride, _addr(D),
        _addr(z), z_stride, _addr(dt_bias), _addr(cu_seqlens), _addr(init_state), _addr(out), _addr(final_state), B,
        T, Hk, Hv, dk, dv, flags, _addr(workspace), workspace_bytes, _stream(stream)))


def gdn_ssm_workspace_bytes(B, T, Hk, Hv, dk, dv, packed) -> int:
    return load().gdn_ssm_workspace_bytes(B, T, Hk, Hv, dk, dv, int(bool(packed)))


def gdn_ssm_step(x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, D, z, z_stride, dt_bias, state, out, B,
                 Hk, Hv, dk, dv, flags, stream=None) -> int:
    """One token per sequence of the scan, state updated in place; returns the status."""
    return load().gdn_ssm_step(_SSM_STEP.pack(
        _addr(x), x_stride, _addr(dt), dt_stride, _addr(A), _addr(Bm), b_stride, _addr(Cm), c_stride, _addr(D),
        _addr(z), z_stride, _addr(dt_bias), _addr(state), _addr(out), B, Hk, Hv, dk, dv, flags, _stream(stream)))


def gdn_add_norm(x, x_stride, residual, weight, residual_out, out, scales, rows, D, group, eps, flags,
                 stream=None) -> int:
    """Root-mean-square norm with the residual's addition; returns the status."""
    return load().gdn_add_norm(_NORM.pack(_addr(x), x_stride, _addr(residual), _addr(weight), _addr(residual_out),
                                          _addr(out), _addr(scales), rows, D, group, eps, flags, _stream(stream)))


def _want(cond, what) -> None:
    if not cond:
        raise ValueError(what)


def _plain(t, name, dtype, shape, dev) -> int:
    """The address of a contiguous tensor of this type and shape on device `dev`; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {shape} on the device of x is wanted, "
                         f"got {t.dtype} {tuple(t.shape)}, strides {t.stride()}, on {t.device}")
    return t.data_ptr()


def _rows(t, name, dtype, shape, dev) -> int:
    """Row stride of a tensor of this shape whose rows are contiguous (a slice of a wider one may be)."""
    if max(shape) > 0x7fffffff:
        raise ValueError(f"{name}: sizes are 32-bit, got {tuple(shape)}")
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name}: a {dtype} tensor of shape {shape} on the device of x is wanted, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    st = t.stride()
    if len(shape) == 3:
        n, h, d = shape
        width = h * d
        ok = (st[2] == 1 or d == 1) and (st[1] == d or h == 1)
    else:
        n, width = shape
        ok = st[1] == 1 or width == 1
    if not ok:
        raise ValueError(f"{name}: the elements of a row have to be contiguous (strides {st})")
    return st[0] if n > 1 else width


def _batch(n, cu_seqlens, B, dev):
    """(sequences, tokens per sequence or in all, boundaries' address) of a dense or packed batch of n rows."""
    if cu_seqlens is None:
        B = 1 if B is None else int(B)
        _want(0 <= B <= 0x7fffffff and (n % B == 0 if B else n == 0), "the tokens have to divide into B sequences")
        return B, n // B if B else 0, 0
    import torch

    _want(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 1, "cu_seqlens: B + 1 boundaries")
    b1 = cu_seqlens.numel()
    return b1 - 1, n, _plain(cu_seqlens, "cu_seqlens", torch.int32, (b1,), dev)


def causal_conv(x, weight, bias=None, cu_seqlens=None, init_state=None, *, B=None, silu=True, out=None,
                final_state=None, want_final=True, stream=None):
    """Short causal convolution of a dense batch of B sequences, or a packed one, with silu.

    x: bf16 [Ttot, C] (rows may be a slice of wider ones); weight: bf16 [C, K], K of 2 to 4; bias: bf16 [C];
    init_state: bf16 [B, K-1, C], the inputs before each sequence, oldest first.  Returns (out bf16
    [Ttot, C], final_state bf16 [B, K-1, C] or None), in `out` and `final_state` where given.
    """
    fast = _shorter()
    if fast is not None and out is not None and (final_state is not None or not want_final):
        rc = fast.causal_conv(x, weight, bias, cu_seqlens, init_state, B, silu, out, final_state, stream)
        if rc is not None:
            if rc:
                check(rc)
            return out, final_state
    import torch

    bf16 = torch.bfloat16
    _want(x.dim() == 2 and weight.dim() == 2, "x: [Ttot, C], weight: [C, K]")
    (n, _), (C, K), dev = x.shape, weight.shape, x.get_device()
    xs = _rows(x, "x", bf16, (n, C), dev)
    B, T, cu = _batch(n, cu_seqlens, B, dev)
    if out is None:
        out = _output((n, C), bf16, x.device, stream)
    if final_state is None and want_final:
        final_state = _output((B, K - 1, C), bf16, x.device, stream)
    _call(load().gdn_conv, _CONV.pack(
        x.data_ptr(), xs, _plain(weight, "weight", bf16, (C, K), dev), _plain(bias, "bias", bf16, (C,), dev), cu,
        _plain(init_state, "init_state", bf16, (B, K - 1, C), dev), _plain(out, "out", bf16, (n, C), dev),
        _plain(final_state, "final_state", bf16, (B, K - 1, C), dev), B, T, C, K, GDN_CONV_SILU if silu else 0,
        _raw_stream(stream, dev)), dev)
    return out, final_state


def causal_conv_step(x, weight, state, bias=None, *, silu=True, out=None, stream=None):
    """One token of each of B sequences: x bf16 [B, C]; state bf16 [B, K-1, C], updated in place."""
    fast = _shorter()
    if fast is not None and out is not None:
        rc = fast.causal_conv_step(x, weight, state, bias, silu, out, stream)
        if rc is not None:
            if rc:
                check(rc)
            return out
    import torch

    bf16 = torch.bfloat16
    _want(x.dim() == 2 and weight.dim() == 2, "x: [B, C], weight: [C, K]")
    (B, _), (C, K), dev = x.shape, weight.shape, x.get_device()
    xs = _rows(x, "x", bf16, (B, C), dev)
    if out is None:
        out = _output((B, C), bf16, x.device, stream)
    _call(load().gdn_conv_step, _CONV_STEP.pack(
        x.data_ptr(), xs, _plain(weight, "weight", bf16, (C, K), dev), _plain(bias, "bias", bf16, (C,), dev),
        _plain(state, "state", bf16, (B, K - 1, C), dev), _plain(out, "out", bf16, (B, C), dev), B, C, K,
        GDN_CONV_SILU if silu else 0, _raw_stream(stream, dev)), dev)
    return out


def _ssm_operands(x, dt, A, Bm, Cm, D, z, dt_bias, out, softplus, stream):
    """Of the scan and its step: (device, sizes, the struct's fields up to dt_bias, out, flags)."""
    import torch

    bf16, f32 = torch.bfloat16, torch.float32
    _want(x.dim() == 3 and Bm.dim() == 3, "x: [Ttot, Hv, dv], Bm and Cm: [Ttot, Hk, dk]")
    n, Hv, dv = shape = x.shape
    _, Hk, dk = Bm.shape
    dev = x.get_device()
    kshape = (n, Hk, dk)
    dt32 = dt.dtype is f32
    fields = (x.data_ptr(), _rows(x, "x", bf16, shape, dev), dt.data_ptr(),
              _rows(dt, "dt", f32 if dt32 else bf16, (n, Hv), dev), _plain(A, "A", f32, (Hv,), dev), Bm.data_ptr(),
              _rows(Bm, "Bm", bf16, kshape, dev), Cm.data_ptr(), _rows(Cm, "Cm", bf16, kshape, dev),
              _plain(D, "D", f32, (Hv,), dev), 0 if z is None else z.data_ptr(),
              0 if z is None else _rows(z, "z", bf16, shape, dev), _plain(dt_bias, "dt_bias", f32, (Hv,), dev))
    if out is None:
        out = _output((n, Hv, dv), bf16, x.device, stream)
    else:
        _plain(out, "out", bf16, shape, dev)
    return dev, (n, Hk, Hv, dk, dv), fields, out, (GDN_SSM_DT_F32 if dt32 else 0) | (GDN_SSM_SOFTPLUS if softplus else 0)


def ssm_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, cu_seqlens=None, init_state=None, *, B=None,
             softplus=True, out=None, final_state=None, want_final=True, workspace=None, stream=None):
    """Selective state space scan of a dense batch of B sequences, or a packed one.

    x, z: bf16 [Ttot, Hv, dv]; dt: bf16 or fp32 [Ttot, Hv]; A, D, dt_bias: fp32 [Hv]; Bm, Cm: bf16
    [Ttot, Hk, dk] (token rows may be slices of wider ones); init_state: fp32 [B, Hv, dv, dk].
    `workspace`: a byte tensor of gdn_ssm_workspace_bytes(...) for these sizes (a smaller batch may need more),
    zeroed once, for calls that overlap or are captured.
    Returns (out bf16 [Ttot, Hv, dv], final_state fp32 [B, Hv, dv, dk] or None).
    """
    fast = _shorter()
    if fast is not None and out is not None and (final_state is not None or not want_final):
        rc = fast.ssm_scan(x, dt, A, Bm, Cm, D, z, dt_bias, cu_seqlens, init_state, B, softplus, out, final_state,
                            workspace, stream)
        if rc is not None:
            if rc:
                check(rc)
            return out, final_state
    import torch

    dev, (n, Hk, Hv, dk, dv), fields, out, flags = _ssm_operands(x, dt, A, Bm, Cm, D, z, dt_bias, out, softplus, stream)
    B, T, cu = _batch(n, cu_seqlens, B, dev)
    shape = (B, Hv, dv, dk)
    if workspace is not None and (workspace.device != x.device or not workspace.is_contiguous()):
        raise ValueError(f"workspace: contiguous, on the device of x, is wanted, got strides {workspace.stride()} on "
                         f"{workspace.device}")
    if final_state is None and want_final:
        final_state = _output(shape, torch.float32, x.device, stream)
    _call(load().gdn_ssm_scan, _SSM_SCAN.pack(
        *fields, cu, _plain(init_state, "init_state", torch.float32, shape, dev), out.data_ptr(),
        _plain(final_state, "final_state", torch.float32, shape, dev), B, T, Hk, Hv, dk, dv, flags,
        0 if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _raw_stream(stream, dev)), dev)
    return out, final_state


def ssm_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, *, softplus=True, out=None, stream=None):
    """One token of each of B sequences of the scan: state fp32 [B, Hv, dv, dk], updated in place."""
    fast = _shorter()
    if fast is not None and out is not None:
        rc = fast.ssm_step(x, dt, A, Bm, Cm, state, D, z, dt_bias, softplus, out, stream)
        if rc is not None:
            if rc:
                check(rc)
            return out
    import torch

    dev, (n, Hk, Hv, dk, dv), fields, out, flags = _ssm_operands(x, dt, A, Bm, Cm, D, z, dt_bias, out, softplus, stream)
    _call(load().gdn_ssm_step, _SSM_STEP.pack(
        *fields, _plain(state, "state", torch.float32, (n, Hv, dv, dk), dev), out.data_ptr(), n, Hk, Hv, dk, dv, flags,
        _raw_stream(stream, dev)), dev)
    return out


def add_norm(x, weight, residual=None, *, eps=1e-6, group=0, e4m3=False, out=None, scales=None, residual_out=None,
             stream=None):
    """Root-mean-square norm of x (+ residual), to bf16, or to e4m3 with a scale per row (group 0) or per
    32, 64 or 128 columns.

    x: bf16 [rows, D] (rows may be slices of wider ones); weight: bf16 [D]; residual: bf16 [rows, D].
    `e4m3` follows from `out` where that is given.  Returns (out, scales or None, residual_out or None);
    residual_out may be `residual` itself.
    """
    fast = _shorter()
    if fast is not None and out is not None and (residual is None or residual_out is not None):
        rc = fast.add_norm(x, weight, residual, eps, group, out, scales, residual_out, stream)
        if rc is not None:
            if rc:
                check(rc)
            return out, scales, residual_out
    import torch

    bf16, f8 = torch.bfloat16, torch.float8_e4m3fn
    _want(x.dim() == 2, "x: [rows, D]")
    _want(0 <= group <= 0x7fffffff, "group: 0, 32, 64 or 128 columns")
    rows, D = shape = x.shape
    dev = x.get_device()
    xs = _rows(x, "x", bf16, shape, dev)
    if out is None:
        out = _output(shape, f8 if e4m3 else bf16, x.device, stream)
    else:
        e4m3 = out.dtype is f8
    if not e4m3:
        scales = None
    elif scales is None:
        scales = _output((rows, -(-D // group) if group else 1), torch.float32, x.device, stream)
    if residual is not None and residual_out is None:
        residual_out = _output(shape, bf16, x.device, stream)
    _call(load().gdn_add_norm, _NORM.pack(
        x.data_ptr(), xs, _plain(residual, "residual", bf16, shape, dev), _plain(weight, "weight", bf16, (D,), dev),
        _plain(residual_out, "residual_out", bf16, shape, dev), _plain(out, "out", f8 if e4m3 else bf16, shape, dev),
        _plain(scales, "scales", torch.float32, (rows, -(-D // group) if group else 1), dev), rows, D, group, eps,
        GDN_NORM_E4M3 if e4m3 else 0, _raw_stream(stream, dev)), dev)
    return out, scales, residual_out
