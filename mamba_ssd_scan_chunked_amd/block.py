"""The operators around the scan in a Mamba layer: the short causal convolution, the
selective scan with a decay per channel and state, the gated norm after the scan and
the residual norm before a block, with their gradients and single-token forms, through
the C ABI in ``include/ssd.h``.

    y, final   = causal_conv(x, weight, bias, init_state, seq_idx, nseqs)
    y          = causal_conv_step(x, weight, bias, state)
    y, final   = selective_scan(x, dt, A_log, B, C, D, z, init_state, seq_idx, nseqs)
    y          = selective_step(x, dt, A_log, B, C, D, state, z)
    out        = gated_norm(x, z, weight)
    out, res   = residual_norm(x, residual, weight)

Activations (x, dt, B, C, z, y, out) are bf16 or fp32; parameters, states and gradients are
fp32.  Activations may be slices of a projection's output (channels contiguous, one
distance between all tokens, below 2^31 elements, or 2^25 for the selective scan of a
prompt): they are read in place.  Anything else that is not contiguous is copied first.
A call runs on ``stream`` (a torch stream or a raw
handle; None: the current stream of the tensors' device), and so do the copies and
allocations it makes.
"""
from __future__ import annotations

import contextlib
import ctypes
import sys
from typing import Optional

_pkg = sys.modules[__package__]       # its loader, error and buffer checks
torch = None                          # imported by the first call, as in the rest of the binding

DTYPE_F32 = 0
DTYPE_BF16 = 1
CONV_SILU = 1
NORM_GATE_FIRST = 1


class ConvProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("nseqs", ctypes.c_int64), ("ldx", ctypes.c_int64), ("width", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_int32)]


class SelectiveProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("nseqs", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("lddt", ctypes.c_int64), ("ldz", ctypes.c_int64), ("ldb", ctypes.c_int64),
                ("ldc", ctypes.c_int64), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("segments", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("group_size", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldz", ctypes.c_int64), ("eps", ctypes.c_float),
                ("x_dtype", ctypes.c_int32), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("reserved", ctypes.c_int32)]


def _declare(lib):
    """Argument types of the library's entry points."""
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    conv, norm, sel = (ctypes.POINTER(s) for s in (ConvProblem, NormProblem, SelectiveProblem))
    for name, args, res in (
            ("ssd_conv_forward", [conv] + [vp] * 8, i32),
            ("ssd_conv_backward_workspace_size", [conv], sz),
            ("ssd_conv_backward", [conv] + [vp] * 12 + [sz, vp], i32),
            ("ssd_conv_step", [conv] + [vp] * 7, i32),
            ("ssd_selective_workspace_size", [sel], sz),
            ("ssd_selective_forward", [sel] + [vp] * 13 + [sz, vp], i32),
            ("ssd_selective_step", [sel] + [vp] * 12, i32),
            ("ssd_selective_backward_workspace_size", [sel], sz),
            ("ssd_selective_backward", [sel] + [vp] * 22 + [sz, vp], i32),
            ("ssd_gated_norm_forward", [norm] + [vp] * 5, i32),
            ("ssd_gated_norm_backward_workspace_size", [norm], sz),
            ("ssd_gated_norm_backward", [norm] + [vp] * 8 + [sz, vp], i32),
            ("ssd_residual_norm_forward", [norm] + [vp] * 7, i32),
            ("ssd_residual_norm_backward_workspace_size", [norm, i32], sz),
            ("ssd_residual_norm_backward", [norm] + [vp] * 11 + [sz, vp], i32)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


def _lib():
    return _pkg.load_library()


def _check(code):
    if code:
        raise _pkg.SSDError(code, _lib().ssd_strerror(code).decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """The device and stream a call works on, as a context."""
    if stream is None:
        return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
    elif stream.device != dev:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, dev))
    return torch.cuda.stream(stream)


def _current(dev):
    """The current stream's handle: straight from torch's binding where it has one, since
    the stream object that the public call builds takes as long as the launch."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev.index) if raw else torch.cuda.current_stream(dev).cuda_stream


def _gpu(x):
    global torch
    if torch is None:
        import torch
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    return dev


def _dtype(name, t):
    if t.dtype is torch.bfloat16:
        return DTYPE_BF16
    if t.dtype is torch.float32:
        return DTYPE_F32
    raise TypeError("%s must be bfloat16 or float32" % name)


def _given(name, t, shape, dtype, dev):
    """An argument of this type and shape, dense."""
    if t is None:
        return None
    if t.device != dev:
        raise ValueError("%s is on %s, x on %s" % (name, t.device, dev))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t if t.is_contiguous() else t.contiguous()


def _output(name, t, shape, dtype, dev):
    """A caller's output buffer, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _pkg._check_buffer(name, t, shape, dtype, dev)
    return t


FAR = 1 << 31                         # the library takes distances below this,
FAR_IN_TILE = 1 << 25                 # and below this where a tile has 32-bit offsets


def _rows(t, far=FAR):
    """(t, ld): t (..., channels) as rows ld < ``far`` elements apart, copied if it is not that."""
    D = t.shape[-1]
    if t.is_contiguous():
        return t, D
    if t.stride(-1) == 1 or D == 1:
        ld = step = 0
        for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
            if size == 1:
                continue
            if ld and stride != step:
                break
            ld = ld or stride
            step = stride * size
            if not ld:                          # a broadcast dimension
                break
        else:
            if D <= ld < far:
                return t, ld
    return t.contiguous(), D


def _workspace(ws, nbytes, dev):
    if ws is None and nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _pkg._check_workspace(ws, nbytes, dev)
    return ws, 0 if ws is None else ws.numel()


def _sequences(x, seq_idx, nseqs):
    """(seq_idx, nseqs) of rows x (b,T,...); without ids each row is one sequence."""
    b, T = x.shape[:2]
    if seq_idx is None:
        if nseqs is not None and int(nseqs) != b:
            raise ValueError("nseqs must be the batch without seq_idx")
        return None, b
    if nseqs is None:
        raise ValueError("nseqs is required with seq_idx (it sizes the states)")
    return _given("seq_idx", seq_idx, (b, T), torch.int32, x.device), int(nseqs)


# ------------------------------------------------------------------ causal convolution
def conv_problem(batch, seqlen, channels, width, nseqs=None, dtype=DTYPE_BF16, silu=True, ldx=None) -> ConvProblem:
    return ConvProblem(batch, seqlen, channels, batch if nseqs is None else nseqs, channels if ldx is None else ldx,
                       width, dtype, CONV_SILU if silu else 0, 0)


def conv_backward_workspace_size(p: ConvProblem) -> int:
    return int(_lib().ssd_conv_backward_workspace_size(ctypes.byref(p)))


def _conv_arguments(x, weight, bias, init_state, seq_idx, nseqs, silu):
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be (b,T,D) and weight (D,K)")
    dev, f32 = x.device, torch.float32
    b, T, D = x.shape
    K = weight.shape[1]
    weight = _given("weight", weight, (D, K), f32, dev)
    bias = _given("bias", bias, (D,), f32, dev)
    seq_idx, ns = _sequences(x, seq_idx, nseqs)
    init_state = _given("init_state", init_state, (ns, K - 1, D), f32, dev)
    x, ldx = _rows(x)
    return conv_problem(b, T, D, K, ns, _dtype("x", x), silu, ldx), x, weight, bias, init_state, seq_idx


def causal_conv(x, weight, bias=None, init_state=None, seq_idx=None, nseqs: Optional[int] = None, silu: bool = True,
                y=None, final_state=None, return_final: bool = True, stream=None):
    """The causal convolution of whole rows through ``ssd_conv_forward``.

    x (b,T,D), weight (D,K) with K = 2..4 (the last tap is the token's own), bias (D).
    ``seq_idx`` (b,T) with ``nseqs`` packs sequences into rows as in :func:`forward`.
    ``init_state`` and the final state are (nseqs,K-1,D): the K-1 inputs before and at
    the end of each sequence.  Returns (y like x, final_state or None)."""
    dev = _gpu(x)
    with _on(dev, stream):
        p, x, weight, bias, init_state, seq_idx = _conv_arguments(x, weight, bias, init_state, seq_idx, nseqs, silu)
        y = _output("y", y, x.shape, x.dtype, dev)
        if final_state is not None or return_final:
            final_state = _output("final_state", final_state, (p.nseqs, p.width - 1, p.channels), torch.float32, dev)
        _check(_lib().ssd_conv_forward(ctypes.byref(p), _ptr(x), _ptr(weight), _ptr(bias), _ptr(init_state),
                                       _ptr(seq_idx), _ptr(y), _ptr(final_state), _current(dev)))
    return y, final_state


def causal_conv_backward(x, weight, dy, bias=None, init_state=None, dfinal=None, seq_idx=None,
                         nseqs: Optional[int] = None, silu: bool = True, workspace=None, stream=None):
    """Gradients through ``ssd_conv_backward`` of <dy, y> + <dfinal, final_state> for
    :func:`causal_conv` with the same arguments; dy (b,T,D) and dfinal fp32.  Returns a
    dict of fp32 tensors dx, dweight, dbias, dinit (dbias and dinit at zero when the
    input was not given)."""
    dev = _gpu(x)
    with _on(dev, stream):
        p, x, weight, bias, init_state, seq_idx = _conv_arguments(x, weight, bias, init_state, seq_idx, nseqs, silu)
        f32 = torch.float32
        state = (p.nseqs, p.width - 1, p.channels)
        dy = _given("dy", dy, x.shape, f32, dev)
        dfinal = _given("dfinal", dfinal, state, f32, dev)
        out = {"dx": torch.empty(x.shape, dtype=f32, device=dev),
               "dweight": torch.empty(weight.shape, dtype=f32, device=dev),
               "dbias": torch.empty(p.channels, dtype=f32, device=dev),
               "dinit": torch.empty(state, dtype=f32, device=dev)}
        ws, nbytes = _workspace(workspace, conv_backward_workspace_size(p), dev)
        _check(_lib().ssd_conv_backward(ctypes.byref(p), _ptr(x), _ptr(weight), _ptr(bias), _ptr(init_state),
                                        _ptr(seq_idx), _ptr(dy), _ptr(dfinal), _ptr(out["dx"]), _ptr(out["dweight"]),
                                        _ptr(out["dbias"]), _ptr(out["dinit"]), _ptr(ws), nbytes, _current(dev)))
    return out


def causal_conv_step(x, weight, bias, state, y=None, silu: bool = True, state_out=None, stream=None):
    """One token per row through ``ssd_conv_step``: x (b,D), ``state`` (b,K-1,D) fp32,
    updated in place or, with ``state_out``, left as it was and the new state written
    there.  Returns y (b,D)."""
    dev = _gpu(x)
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be (b,D) and weight (D,K)")
    with _on(dev, stream):
        b, D = x.shape
        K = weight.shape[1]
        weight = _given("weight", weight, (D, K), torch.float32, dev)
        bias = _given("bias", bias, (D,), torch.float32, dev)
        state, state_out = _states(state, state_out, (b, K - 1, D), dev)
        x, ldx = _rows(x)
        y = _output("y", y, (b, D), x.dtype, dev)
        p = conv_problem(b, 1, D, K, b, _dtype("x", x), silu, ldx)
        _check(_lib().ssd_conv_step(ctypes.byref(p), _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(state_out),
                                    _ptr(y), _current(dev)))
    return y


def _states(state, state_out, shape, dev):
    """The state a step reads and the one it writes (the same without ``state_out``)."""
    if state_out is None:
        _pkg._check_buffer("state", state, shape, torch.float32, dev)
        return state, state
    _pkg._check_buffer("state_out", state_out, shape, torch.float32, dev)
    return _given("state", state, shape, torch.float32, dev), state_out


# ------------------------------------------------------------------ selective scan
FLAG_DT_SOFTPLUS = 2


def selective_problem(batch, seqlen, channels, dstate, ngroups=1, nseqs=None, dtype=DTYPE_BF16, dt_softplus=False,
                      segments=0, ldx=None, lddt=None, ldz=None, ldb=None, ldc=None) -> SelectiveProblem:
    """A problem description; ``segments`` > 0 forces the number of segments each row is
    cut into (0: the library's choice); it does not change the result."""
    wide, gn = channels, ngroups * dstate
    return SelectiveProblem(batch, seqlen, channels, dstate, ngroups, batch if nseqs is None else nseqs,
                            wide if ldx is None else ldx, wide if lddt is None else lddt, wide if ldz is None else ldz,
                            gn if ldb is None else ldb, gn if ldc is None else ldc, dtype,
                            FLAG_DT_SOFTPLUS if dt_softplus else 0, segments, 0)


def selective_workspace_size(p: SelectiveProblem) -> int:
    return int(_lib().ssd_selective_workspace_size(ctypes.byref(p)))


def selective_backward_workspace_size(p: SelectiveProblem) -> int:
    return int(_lib().ssd_selective_backward_workspace_size(ctypes.byref(p)))


def _activation(name, t, shape, like, far):
    """An activation of x's type and device as rows: (t, ld)."""
    if t.device != like.device:
        raise ValueError("%s is on %s, x on %s" % (name, t.device, like.device))
    if t.dtype != like.dtype:
        raise TypeError("%s must be %s, got %s" % (name, like.dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return _rows(t, far)


def _grouped(name, t, shape, like, far):
    """The same of B or C, shape (..., G, N): rows of G N channels."""
    if t.is_contiguous() and t.shape == shape and t.dtype is like.dtype and t.device == like.device:
        return t, shape[-2] * shape[-1]           # without a view, which takes as long as all checks
    return _activation(name, t.flatten(-2), (*shape[:-2], shape[-2] * shape[-1]), like, far)


def _selective_arguments(x, dt, A_log, B, C, D, z, init_state, seq_idx, nseqs, dt_bias, dt_softplus, segments):
    """(problem, pointers' tensors in the order of the C call up to seq_idx)."""
    if x.dim() != 3 or B.dim() != 4 or A_log.dim() != 2:
        raise ValueError("x must be (b,T,D), B and C (b,T,G,N) and A_log (D,N)")
    dev, f32 = x.device, torch.float32
    b, T, Dc = x.shape
    G, N = B.shape[2:]
    code = _dtype("x", x)
    A_log = _given("A_log", A_log, (Dc, N), f32, dev)
    D = _given("D", D, (Dc,), f32, dev)
    dt_bias = _given("dt_bias", dt_bias, (Dc,), f32, dev)
    seq_idx, ns = _sequences(x, seq_idx, nseqs)
    init_state = _given("init_state", init_state, (ns, Dc, N), f32, dev)
    if C.shape != B.shape:
        raise ValueError("B and C must have one shape")
    dt, lddt = _activation("dt", dt, x.shape, x, FAR_IN_TILE)
    ldz = Dc
    if z is not None:
        z, ldz = _activation("z", z, x.shape, x, FAR_IN_TILE)
    B, ldb = _grouped("B", B, (b, T, G, N), x, FAR_IN_TILE)
    C, ldc = _grouped("C", C, (b, T, G, N), x, FAR_IN_TILE)
    x, ldx = _rows(x, FAR_IN_TILE)
    p = selective_problem(b, T, Dc, N, G, ns, code, dt_softplus, segments, ldx, lddt, ldz, ldb, ldc)
    return p, (x, dt, dt_bias, A_log, B, C, D, z, init_state, seq_idx)


def selective_scan(x, dt, A_log, B, C, D=None, z=None, init_state=None, seq_idx=None, nseqs: Optional[int] = None,
                   dt_bias=None, dt_softplus: bool = False, y=None, final_state=None, workspace=None,
                   return_final: bool = True, stream=None, segments: int = 0):
    """The selective scan of whole rows through ``ssd_selective_forward``.

    x, dt (b,T,D), B, C (b,T,G,N) and the gate z (b,T,D; None: no gate) in one type;
    A_log (D,N), D, dt_bias (D) fp32; the state (nseqs,D,N) fp32, N one of 8, 16, 32, 64.
    The step size is dt + dt_bias, through softplus with ``dt_softplus``; packed sequences
    and ``segments`` as in :func:`forward`.  Returns (y like x, final_state or None)."""
    dev = _gpu(x)
    with _on(dev, stream):
        p, args = _selective_arguments(x, dt, A_log, B, C, D, z, init_state, seq_idx, nseqs, dt_bias, dt_softplus,
                                       segments)
        y = _output("y", y, x.shape, x.dtype, dev)
        if final_state is not None or return_final:
            final_state = _output("final_state", final_state, (p.nseqs, p.channels, p.dstate), torch.float32, dev)
        ws, nbytes = _workspace(workspace, selective_workspace_size(p), dev)
        _check(_lib().ssd_selective_forward(ctypes.byref(p), *map(_ptr, args), _ptr(y), _ptr(final_state), _ptr(ws),
                                            nbytes, _current(dev)))
    return y, final_state


def selective_scan_backward(x, dt, A_log, B, C, dy, D=None, z=None, init_state=None, dfinal=None, seq_idx=None,
                            nseqs: Optional[int] = None, dt_bias=None, dt_softplus: bool = False, workspace=None,
                            stream=None, segments: int = 0):
    """Gradients through ``ssd_selective_backward`` of <dy, y> + <dfinal, final_state> for
    :func:`selective_scan` with the same arguments; dy (b,T,D) and dfinal fp32.  Returns a
    dict of fp32 tensors dx, ddt, dA_log, dB, dC, dD, dinit, ddt_bias and, with z, dz (dD,
    dinit and ddt_bias at zero when the input was not given)."""
    dev, f32 = _gpu(x), torch.float32
    with _on(dev, stream):
        p, args = _selective_arguments(x, dt, A_log, B, C, D, z, init_state, seq_idx, nseqs, dt_bias, dt_softplus,
                                       segments)
        state = (p.nseqs, p.channels, p.dstate)
        dy = _given("dy", dy, x.shape, f32, dev)
        dfinal = _given("dfinal", dfinal, state, f32, dev)
        shapes = {"dx": x.shape, "ddt": x.shape, "dA_log": A_log.shape, "dB": B.shape, "dC": C.shape,
                  "dD": (p.channels,), "dz": x.shape, "dinit": state, "ddt_bias": (p.channels,)}
        if z is None:
            del shapes["dz"]
        out = {k: torch.empty(s, dtype=f32, device=dev) for k, s in shapes.items()}
        ws, nbytes = _workspace(workspace, selective_backward_workspace_size(p), dev)
        g = out.get
        _check(_lib().ssd_selective_backward(ctypes.byref(p), *map(_ptr, args), _ptr(dy), _ptr(dfinal), _ptr(g("dx")),
                                             _ptr(g("ddt")), _ptr(g("dA_log")), _ptr(g("dB")), _ptr(g("dC")),
                                             _ptr(g("dD")), _ptr(g("dz")), _ptr(g("dinit")), _ptr(g("ddt_bias")),
                                             _ptr(ws), nbytes, _current(dev)))
    return out


def selective_step(x, dt, A_log, B, C, D, state, z=None, y=None, dt_bias=None, dt_softplus: bool = False,
                   state_out=None, stream=None):
    """One token per row through ``ssd_selective_step``: x, dt, z (b,D), B, C (b,G,N),
    ``state`` (b,D,N) fp32, updated in place or, with ``state_out``, left as it was and the
    new state written there.  Returns y (b,D)."""
    dev, f32 = _gpu(x), torch.float32
    if x.dim() != 2 or B.dim() != 3 or A_log.dim() != 2:
        raise ValueError("x must be (b,D), B and C (b,G,N) and A_log (D,N)")
    with _on(dev, stream):
        b, Dc = x.shape
        G, N = B.shape[1:]
        if C.shape != B.shape:
            raise ValueError("B and C must have one shape")
        A_log = _given("A_log", A_log, (Dc, N), f32, dev)
        D = _given("D", D, (Dc,), f32, dev)
        dt_bias = _given("dt_bias", dt_bias, (Dc,), f32, dev)
        state, state_out = _states(state, state_out, (b, Dc, N), dev)
        dt, lddt = _activation("dt", dt, x.shape, x, FAR)
        ldz = Dc
        if z is not None:
            z, ldz = _activation("z", z, x.shape, x, FAR)
        B, ldb = _grouped("B", B, (b, G, N), x, FAR)
        C, ldc = _grouped("C", C, (b, G, N), x, FAR)
        y = _output("y", y, (b, Dc), x.dtype, dev)
        x, ldx = _rows(x)
        p = selective_problem(b, 1, Dc, N, G, b, _dtype("x", x), dt_softplus, 0, ldx, lddt, ldz, ldb, ldc)
        _check(_lib().ssd_selective_step(ctypes.byref(p), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A_log), _ptr(B),
                                         _ptr(C), _ptr(D), _ptr(z), _ptr(state), _ptr(state_out), _ptr(y),
                                         _current(dev)))
    return y


# ------------------------------------------------------------------ norms
def norm_problem(rows, channels, group_size=None, eps=1e-5, x_dtype=DTYPE_F32, dtype=DTYPE_BF16, gate_first=False,
                 ldx=None, ldz=None) -> NormProblem:
    return NormProblem(rows, channels, channels if group_size is None else group_size,
                       channels if ldx is None else ldx, channels if ldz is None else ldz, eps, x_dtype, dtype,
                       NORM_GATE_FIRST if gate_first else 0, 0)


def gated_norm_backward_workspace_size(p: NormProblem) -> int:
    return int(_lib().ssd_gated_norm_backward_workspace_size(ctypes.byref(p)))


def residual_norm_backward_workspace_size(p: NormProblem, scaled: bool) -> int:
    return int(_lib().ssd_residual_norm_backward_workspace_size(ctypes.byref(p), int(scaled)))


def _gated_arguments(x, z, weight, group_size, eps, gate_first):
    dev = x.device
    if x.dim() < 1 or z.shape != x.shape:
        raise ValueError("x and z must have one shape (..., D)")
    if z.device != dev:
        raise ValueError("z is on %s, x on %s" % (z.device, dev))
    D = x.shape[-1]
    weight = _given("weight", weight, (D,), torch.float32, dev)
    x, ldx = _rows(x)
    z, ldz = _rows(z)
    rows = x.numel() // D if D else 0
    return norm_problem(rows, D, group_size, eps, _dtype("x", x), _dtype("z", z), gate_first, ldx, ldz), x, z, weight


def gated_norm(x, z, weight, group_size: Optional[int] = None, eps: float = 1e-5, gate_first: bool = True, out=None,
               stream=None):
    """The root-mean-square norm after the scan with its gate, through
    ``ssd_gated_norm_forward``: with ``gate_first``, x silu(z) normed and times weight;
    else x normed, times weight and silu(z).  x (..., D) fp32 (the scan's y) or the type
    of z; z (..., D); weight (D) fp32; the mean square is taken over each group of
    ``group_size`` consecutive channels (None: all of them).  Returns out, shaped like x
    in z's type."""
    dev = _gpu(x)
    with _on(dev, stream):
        p, x, z, weight = _gated_arguments(x, z, weight, group_size, eps, gate_first)
        out = _output("out", out, z.shape, z.dtype, dev)
        _check(_lib().ssd_gated_norm_forward(ctypes.byref(p), _ptr(x), _ptr(z), _ptr(weight), _ptr(out), _current(dev)))
    return out


def gated_norm_backward(x, z, weight, dout, group_size: Optional[int] = None, eps: float = 1e-5,
                        gate_first: bool = True, workspace=None, stream=None):
    """Gradients of <dout, out> for :func:`gated_norm` through ``ssd_gated_norm_backward``;
    dout fp32.  Returns a dict of fp32 tensors dx, dz, dweight."""
    dev = _gpu(x)
    with _on(dev, stream):
        p, x, z, weight = _gated_arguments(x, z, weight, group_size, eps, gate_first)
        dout = _given("dout", dout, x.shape, torch.float32, dev)
        out = {"dx": torch.empty(x.shape, dtype=torch.float32, device=dev),
               "dz": torch.empty(x.shape, dtype=torch.float32, device=dev),
               "dweight": torch.empty(weight.shape, dtype=torch.float32, device=dev)}
        ws, nbytes = _workspace(workspace, gated_norm_backward_workspace_size(p), dev)
        _check(_lib().ssd_gated_norm_backward(ctypes.byref(p), _ptr(x), _ptr(z), _ptr(weight), _ptr(dout),
                                              _ptr(out["dx"]), _ptr(out["dz"]), _ptr(out["dweight"]), _ptr(ws), nbytes,
                                              _current(dev)))
    return out


def residual_norm(x, residual, weight, scale=None, eps: float = 1e-5, out=None, residual_out=None, stream=None):
    """The norm before a block with its residual addition, through
    ``ssd_residual_norm_forward``: residual_out = residual + scale x, out its
    root-mean-square norm times weight.  x (..., D); residual (..., D) fp32 or None;
    weight, scale (D) fp32 (scale None: 1).  ``residual_out`` may be ``residual`` (in
    place).  Returns (out in x's type, residual_out fp32)."""
    dev, f32 = _gpu(x), torch.float32
    if x.dim() < 1:
        raise ValueError("x must be (..., D)")
    with _on(dev, stream):
        D = x.shape[-1]
        weight = _given("weight", weight, (D,), f32, dev)
        scale = _given("scale", scale, (D,), f32, dev)
        x, ldx = _rows(x)
        ldz = D
        if residual is not None:
            if residual.device != dev or residual.shape != x.shape:
                raise ValueError("residual must have x's shape and device")
            if residual.dtype != f32:
                raise TypeError("residual must be torch.float32, got %s" % residual.dtype)
            residual, ldz = _rows(residual)
        out = _output("out", out, x.shape, x.dtype, dev)
        residual_out = _output("residual_out", residual_out, x.shape, f32, dev)
        code = _dtype("x", x)
        p = norm_problem(x.numel() // D if D else 0, D, D, eps, code, code, False, ldx, ldz)
        _check(_lib().ssd_residual_norm_forward(ctypes.byref(p), _ptr(x), _ptr(residual), _ptr(weight), _ptr(scale),
                                                _ptr(out), _ptr(residual_out), _current(dev)))
    return out, residual_out


def residual_norm_backward(x, residual_out, weight, dout, dresidual_out=None, scale=None, eps: float = 1e-5,
                           workspace=None, stream=None):
    """Gradients of <dout, out> + <dresidual_out, residual_out> for :func:`residual_norm`
    through ``ssd_residual_norm_backward``, from the residual_out it returned; dout and
    dresidual_out fp32.  Returns a dict of fp32 tensors dx, dresidual, dweight and, with
    a scale, dscale.  Without a scale dx and dresidual are the same values and one tensor."""
    dev, f32 = _gpu(x), torch.float32
    if x.dim() < 1:
        raise ValueError("x must be (..., D)")
    with _on(dev, stream):
        D = x.shape[-1]
        code = _dtype("x", x)
        weight = _given("weight", weight, (D,), f32, dev)
        scale = _given("scale", scale, (D,), f32, dev)
        residual_out = _given("residual_out", residual_out, x.shape, f32, dev)
        dout = _given("dout", dout, x.shape, f32, dev)
        dresidual_out = _given("dresidual_out", dresidual_out, x.shape, f32, dev)
        ldx = D
        if scale is not None:
            x, ldx = _rows(x)
        p = norm_problem(x.numel() // D if D else 0, D, D, eps, code, code, False, ldx, D)
        d = torch.empty(x.shape, dtype=f32, device=dev)
        out = {"dx": d, "dresidual": d, "dweight": torch.empty(D, dtype=f32, device=dev)}
        if scale is not None:
            out["dx"] = torch.empty(x.shape, dtype=f32, device=dev)
            out["dscale"] = torch.empty(D, dtype=f32, device=dev)
        ws, nbytes = _workspace(workspace, residual_norm_backward_workspace_size(p, scale is not None), dev)
        _check(_lib().ssd_residual_norm_backward(ctypes.byref(p), _ptr(x) if scale is not None else None,
                                                 _ptr(residual_out), _ptr(weight), _ptr(scale), _ptr(dout),
                                                 _ptr(dresidual_out), _ptr(out["dx"]) if scale is not None else None,
                                                 _ptr(d), _ptr(out["dweight"]), _ptr(out.get("dscale")), _ptr(ws),
                                                 nbytes, _current(dev)))
    return out
