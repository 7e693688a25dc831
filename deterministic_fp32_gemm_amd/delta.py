"""The gated delta rule and the block norm (include/sdm_gdr.h, include/sdm_nrm.h) on torch tensors.

The functions take and return tensors on the current GPU: they allocate outputs and workspaces with torch's allocator,
check types and shapes, and call the C ABI of libsdm_delta on torch's current stream (or ``stream``). Every arithmetic
step runs in the library's HIP kernels; there is no other path. A wrong argument raises TypeError or ValueError before
anything runs. A call with ``stream`` is the call under ``torch.cuda.stream(stream)``: what it allocates is that
stream's, and tensors made on another stream are the caller's to order and keep alive, as for any torch operation.

Where grad mode is on and a tensor of the call requires a gradient, gdr_forward and norm_forward are part of torch's graph
(_delta_autograd.py), and a backward pass that reaches gdr_step, which has no gradient, is an error. The gradients that
gdr_backward and norm_backward return have no graph of their own. There are no forward-mode derivatives: a tensor that carries
a tangent is an error.
"""

from __future__ import annotations

import ctypes
import os
import threading

from ._binding import (SDM_GX_ERR_ALIGN, SDM_GX_ERR_ARG, SDM_GX_ERR_HIP, SDM_GX_ERR_LIMIT, SDM_GX_ERR_NULL,
                       SDM_GX_ERR_OVERLAP, SDM_GX_ERR_SHAPE, SDM_GX_ERR_STRIDE, SDM_GX_OK)
from ._build import DELTA_LIB_PATH

SDM_F32, SDM_BF16, SDM_F16 = 0, 1, 2
ACTS = {"none": 0, "sigmoid": 1, "silu": 2}
EXPORTS = ("sdm_gdr_check", "sdm_gdr_step_check", "sdm_gdr_workspace", "sdm_gdr_forward", "sdm_gdr_backward",
           "sdm_gdr_step", "sdm_nrm_check", "sdm_nrm_workspace", "sdm_nrm_forward", "sdm_nrm_backward",
           "sdm_delta_strerror", "sdm_delta_last_hip_error")

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_ARG_ERRORS = {SDM_GX_ERR_NULL, SDM_GX_ERR_SHAPE, SDM_GX_ERR_ALIGN, SDM_GX_ERR_OVERLAP, SDM_GX_ERR_STRIDE,
               SDM_GX_ERR_ARG, SDM_GX_ERR_LIMIT}


class sdm_rows_t(ctypes.Structure):
    _fields_ = [("data", _vp), ("batch", _i64), ("token", _i64), ("head", _i64)]


class sdm_gdr_args_t(ctypes.Structure):
    _fields_ = ([("dtype", _i32), ("scale", _f32)] + [(n, _i64) for n in ("B", "T", "Hk", "Hv", "dk", "dv", "nseq")] +
                [("cu_seqlens", _vp)] + [(n, sdm_rows_t) for n in ("q", "k", "v", "g", "beta")] + [("s0", _vp)] +
                [("o", sdm_rows_t), ("s_final", _vp), ("d_o", sdm_rows_t), ("ds_final", _vp)] +
                [(n, sdm_rows_t) for n in ("d_q", "d_k", "d_v", "d_g", "d_beta")] + [("ds0", _vp)])


class sdm_gdr_step_args_t(ctypes.Structure):
    _fields_ = ([("dtype", _i32), ("scale", _f32)] + [(n, _i64) for n in ("B", "T", "Hk", "Hv", "dk", "dv", "pool")] +
                [(n, sdm_rows_t) for n in ("q", "k", "v", "g", "beta", "o")] + [("state", _vp), ("slots", _vp)])


class sdm_nrm_args_t(ctypes.Structure):
    _fields_ = ([("dtype", _i32), ("wtype", _i32), ("act", _i32), ("eps", _f32), ("rows", _i64), ("D", _i64)] +
                [(n, _vp) for n in ("x", "o", "z")] + [(n, _i64) for n in ("ld_x", "ld_o", "ld_z")] +
                [(n, _vp) for n in ("w_post", "w_pre", "scale", "x_new", "y")] + [("ld_xn", _i64), ("ld_y", _i64)] +
                [("rstd", _vp)] + [(n, _vp) for n in ("dxn", "dy")] + [("ld_dxn", _i64), ("ld_dy", _i64)] +
                [(n, _vp) for n in ("dx", "d_o", "dz")] + [(n, _i64) for n in ("ld_dx", "ld_do", "ld_dz")] +
                [(n, _vp) for n in ("dw_post", "dw_pre", "dscale")])


_lib = None
_lock = threading.Lock()


def load() -> ctypes.CDLL:
    """Load libsdm_delta (once). Fails loudly if it has not been built: there is no fallback path."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(DELTA_LIB_PATH):
            raise ImportError(f"{DELTA_LIB_PATH} is missing: build it first "
                              "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(DELTA_LIB_PATH)
        g, s, n = (ctypes.POINTER(t) for t in (sdm_gdr_args_t, sdm_gdr_step_args_t, sdm_nrm_args_t))
        sig = {
            "sdm_gdr_check": [g, _i32],
            "sdm_gdr_step_check": [s],
            "sdm_gdr_workspace": [g, _i32],
            "sdm_gdr_forward": [g, _vp, _i64, _vp],
            "sdm_gdr_backward": [g, _vp, _i64, _vp],
            "sdm_gdr_step": [s, _vp],
            "sdm_nrm_check": [n, _i32],
            "sdm_nrm_workspace": [n],
            "sdm_nrm_forward": [n, _vp],
            "sdm_nrm_backward": [n, _vp, _i64, _vp],
            "sdm_delta_strerror": [ctypes.c_int],
            "sdm_delta_last_hip_error": [],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = {"sdm_delta_strerror": ctypes.c_char_p, "sdm_gdr_workspace": _i64,
                          "sdm_nrm_workspace": _i64}.get(name, ctypes.c_int)
        global _raw_stream
        _raw_stream = _find_raw_stream()
        _lib = lib
        return lib


def _raise(code: int, what: str):
    if code == SDM_GX_OK:
        return
    msg = load().sdm_delta_strerror(code).decode()
    if code == SDM_GX_ERR_HIP:
        msg += f" (hipError {load().sdm_delta_last_hip_error()})"
    exc = ValueError if code in _ARG_ERRORS else RuntimeError
    raise exc(f"{what}: {msg} [status {code}]")


# ---- marshalling ----------------------------------------------------------------------------------------------------
_TYPES = {}


def _dtype(t, name: str) -> int:
    if not _TYPES:
        import torch
        _TYPES.update({torch.float32: SDM_F32, torch.bfloat16: SDM_BF16, torch.float16: SDM_F16})
    d = _TYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{name}: float32, bfloat16 or float16 required, got {t.dtype}")
    return d


def _tensor(t, name: str, shape, dtype=None, device=None):
    """t's checks: a plain tensor of the GPU, of this shape (None: any size) and type."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a torch tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: {dtype} required, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(shape)} required, got {tuple(t.shape)}")
    if t.is_neg() or t.is_conj():
        raise ValueError(f"{name}: lazy negative / conjugate views are not supported (materialise them first)")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: must be on {device}, is on {t.device}")
    return t


def _inner(t):
    """t, copied if its last axis is not contiguous."""
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _rows(t, address=True) -> sdm_rows_t:
    st = t.stride()
    return sdm_rows_t(t.data_ptr() if address else 0, st[0], st[1], st[2])


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _find_raw_stream():
    """torch's own call for a current stream's handle, without the Stream object around it (a microsecond)."""
    import torch
    return getattr(torch._C, "_cuda_getCurrentRawStream", None)


_raw_stream = None


def _increment_version(tensors):
    """Counts a write to tensors, by torch's own call without the type checks around it: a graph that has saved one of
    them must not use it any more."""
    global _increment_version
    import torch
    _increment_version = getattr(torch._C, "_increment_version", torch.autograd.graph.increment_version)
    _increment_version(tensors)


def _stream(device) -> int:
    """The handle of torch's current stream on the device."""
    if _raw_stream is None:
        import torch
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def _under(stream, device):
    """Makes the stream a call names (a torch stream or a handle) the current one: its outputs, copies and workspace
    then come from that stream's memory, so none of them is given to another stream while the call's kernels run."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream: one of {device} required, got one of {stream.device}")
    return torch.cuda.stream(stream)


class _Plans(threading.local):
    """Checked argument structs by the layout of a call's tensors, a set for each host thread: a call whose tensors have
    the layout of an earlier one copies its struct and fills in their addresses. Addresses, values and results are never
    kept: the copy is the call's own, since a finaliser, a signal handler or an allocator's callback may enter the same
    function with the same layout before this call's launch."""

    MOST = 256

    def __init__(self):
        self.known = {}

    def get(self, key):
        return self.known.get(key)

    def put(self, key, plan):
        if len(self.known) >= self.MOST:
            self.known.clear()
        self.known[key] = plan
        return plan


_plans = _Plans()


def _layout(t):
    """What of a tensor a plan depends on; None for None. Raises for what is not a tensor."""
    if t is None:
        return None
    try:
        return t.shape, t.stride(), t.dtype, t.get_device(), t.is_neg()
    except AttributeError:
        raise TypeError("a torch tensor is required") from None


class _OnDevice:
    """Makes a device current for a call where it is not."""

    __slots__ = ("guard",)

    def __init__(self, device):
        import torch
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _requires_grad(*tensors) -> bool:
    for t in tensors:
        if t is not None and t.requires_grad:
            return True
    return False


def _no_tangents(what, *tensors):
    """Refuses a tensor that carries a tangent of torch's forward mode, which the outputs would lose in silence (such a tensor
    need not require a gradient)."""
    import torch
    forward = torch.autograd.forward_ad
    if getattr(forward, "_current_level", 0) < 0:       # outside of every dual_level: no tensor has one
        return
    for t in tensors:
        if t is not None and forward.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{what} has no forward-mode derivative: call it on the primal tensors")


def _scale(scale):
    """scale as a number, also where a tensor holds it; none that torch would differentiate."""
    if scale is None or type(scale) is float:
        return scale
    if getattr(scale, "requires_grad", False):
        import torch
        if torch.is_grad_enabled():
            raise ValueError("scale: a number; no gradient is computed for it (detach it, or scale q)")
    return float(scale)


def _workspace(nbytes: int, device):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ---- the gated delta rule -------------------------------------------------------------------------------------------
def _gdr_shapes(q, k, v, g, beta):
    import torch
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: a torch tensor")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k: [B, T, Hk, dk] and v: [B, T, Hv, dv] required")
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2:]
    dt = _dtype(q, "q")
    dev = q.device
    _tensor(q, "q", (B, T, Hk, dk))
    _tensor(k, "k", (B, T, Hk, dk), q.dtype, dev)
    _tensor(v, "v", (B, T, Hv, dv), q.dtype, dev)
    _tensor(g, "g", (B, T, Hv), torch.float32, dev)
    _tensor(beta, "beta", (B, T, Hv), torch.float32, dev)
    return B, T, Hk, Hv, dk, dv, dt, dev


def _gdr_plan(backward, q, k, v, g, beta, scale, s0, cu, do, ds):
    """The checked argument struct of a forward or backward call, without addresses."""
    import torch
    B, T, Hk, Hv, dk, dv, dt, dev = _gdr_shapes(q, k, v, g, beta)
    nseq = B
    if cu is not None:
        if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 2:
            raise ValueError("cu_seqlens: an int32 tensor of one more entry than sequences, two at least")
        if B != 1:
            raise ValueError("cu_seqlens: packed sequences come in one row (B = 1)")
        nseq = cu.shape[0] - 1
        _tensor(cu, "cu_seqlens", (nseq + 1,), torch.int32, dev)
    state = (nseq, Hv, dk, dv)
    for t, name in ((s0, "initial_state"), (ds, "dfinal_state")):
        if t is not None:
            _tensor(t, name, state, torch.float32, dev)
    if backward:
        _tensor(do, "do", v.shape, v.dtype, dev)
    copied = (any(_inner(t) is not t for t in (q, k, v, do) if t is not None) or
              any(not t.is_contiguous() for t in (cu, s0, ds) if t is not None))
    q, k, v = _inner(q), _inner(k), _inner(v)
    a = sdm_gdr_args_t(dtype=dt, scale=dk ** -0.5 if scale is None else float(scale), B=B, T=T, Hk=Hk, Hv=Hv, dk=dk,
                       dv=dv, nseq=nseq, q=_rows(q, False), k=_rows(k, False), v=_rows(v, False), g=_rows(g, False),
                       beta=_rows(beta, False))
    whole = lambda t: _rows(torch.empty(t.shape, device="meta"), False)  # noqa: E731
    if backward:
        a.d_o = _rows(_inner(do), False)
        a.d_q, a.d_k, a.d_v, a.d_g, a.d_beta = whole(q), whole(k), whole(v), whole(g), whole(beta)
    else:
        a.o = whole(v)
    n = 0
    if T and B:
        if cu is not None:
            a.cu_seqlens = 4        # the workspace of packed sequences is another
        n = load().sdm_gdr_workspace(ctypes.byref(a), int(backward))
        if n < 0:
            _raise(n, "gdr_backward" if backward else "gdr_forward")
        a.cu_seqlens = 0
    return a, n, state, dev, copied


def _gdr_operands(plan, a, q, k, v, g, beta, s0, cu):
    """Fills the inputs' addresses in; returns what has to live until the call."""
    copied = plan[4]
    if copied:
        q, k, v = _inner(q), _inner(k), _inner(v)
        cu = None if cu is None else cu.contiguous()
        s0 = None if s0 is None else s0.contiguous()
    a.q.data, a.k.data, a.v.data, a.g.data, a.beta.data = (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                                                           beta.data_ptr())
    a.cu_seqlens = 0 if cu is None else cu.data_ptr()
    a.s0 = 0 if s0 is None else s0.data_ptr()
    return q, k, v, cu, s0


def gdr_forward(q, k, v, g, beta, *, scale=None, initial_state=None, final_state=True, cu_seqlens=None, stream=None):
    """The gated delta rule over whole sequences: ``(o, state after the last token)``, the state None unless asked for.

    q, k [B, T, Hk, dk], v [B, T, Hv, dv] of one type (float32, bfloat16, float16; Hv a multiple of Hk: value heads
    share q/k heads in order), g (log decay) and beta [B, T, Hv] float32, states [sequences, Hv, dk, dv] float32.
    scale: 1/sqrt(dk) unless given. cu_seqlens: int32 [n + 1] on the GPU, n sequences packed into one row; tokens of no
    sequence get zeros. Any strides; a last axis that is not contiguous is copied first.
    """
    import torch
    scale = _scale(scale)
    key = ("fwd", _layout(q), _layout(k), _layout(v), _layout(g), _layout(beta), _layout(initial_state),
           _layout(cu_seqlens), scale)
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _gdr_plan(False, q, k, v, g, beta, scale, initial_state, cu_seqlens, None, None))
    _no_tangents("gdr_forward", q, k, v, g, beta, initial_state)
    kept, n, state, dev, _ = plan
    if stream is not None:
        with _under(stream, dev):
            return gdr_forward(q, k, v, g, beta, scale=scale, initial_state=initial_state, final_state=final_state,
                               cu_seqlens=cu_seqlens)
    if torch.is_grad_enabled() and _requires_grad(q, k, v, g, beta, initial_state):
        from ._delta_autograd import GatedDeltaRule
        return GatedDeltaRule.apply(q, k, v, g, beta, initial_state, scale, final_state, cu_seqlens)
    o = (torch.empty if cu_seqlens is None else torch.zeros)(v.shape, dtype=v.dtype, device=dev)
    s = torch.empty(state, dtype=torch.float32, device=dev) if final_state else None
    if not n:
        if s is not None:
            s.zero_() if initial_state is None else s.copy_(initial_state)
        return o, s
    a = sdm_gdr_args_t.from_buffer_copy(kept)
    keep = _gdr_operands(plan, a, q, k, v, g, beta, initial_state, cu_seqlens)
    ws = _workspace(n, dev)
    a.o.data, a.s_final = o.data_ptr(), 0 if s is None else s.data_ptr()
    with _OnDevice(dev):
        status = load().sdm_gdr_forward(ctypes.byref(a), ws.data_ptr(), n, _stream(dev))
    del keep
    if status:
        _raise(status, "gdr_forward")
    return o, s


def gdr_backward(q, k, v, g, beta, do, *, scale=None, initial_state=None, dfinal_state=None, cu_seqlens=None,
                 stream=None):
    """The gradient of gdr_forward: ``(dq, dk, dv, dg, dbeta, dinitial_state)`` from do, the gradient of o, and
    dfinal_state, that of the last state (None: zero). It recomputes the forward's states and needs nothing saved but
    the inputs. Gradients have their tensors' shapes and types; tokens of no sequence get zeros."""
    import torch
    scale = _scale(scale)
    key = ("bwd", _layout(q), _layout(k), _layout(v), _layout(g), _layout(beta), _layout(initial_state),
           _layout(cu_seqlens), _layout(do), _layout(dfinal_state), scale)
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _gdr_plan(True, q, k, v, g, beta, scale, initial_state, cu_seqlens, do, dfinal_state))
    _no_tangents("gdr_backward", q, k, v, g, beta, do, initial_state, dfinal_state)
    kept, n, state, dev, copied = plan
    if stream is not None:
        with _under(stream, dev):
            return gdr_backward(q, k, v, g, beta, do, scale=scale, initial_state=initial_state,
                                dfinal_state=dfinal_state, cu_seqlens=cu_seqlens)
    make = torch.empty if cu_seqlens is None else torch.zeros
    outs = [make(t.shape, dtype=t.dtype, device=dev) for t in (q, k, v, g, beta)]
    s = torch.empty(state, dtype=torch.float32, device=dev)
    if not n:
        s.zero_() if dfinal_state is None else s.copy_(dfinal_state)
        return (*outs, s)
    a = sdm_gdr_args_t.from_buffer_copy(kept)
    keep = _gdr_operands(plan, a, q, k, v, g, beta, initial_state, cu_seqlens)
    if copied:
        do = _inner(do)
        dfinal_state = None if dfinal_state is None else dfinal_state.contiguous()
    a.d_o.data, a.ds_final, a.ds0 = do.data_ptr(), 0 if dfinal_state is None else dfinal_state.data_ptr(), s.data_ptr()
    a.d_q.data, a.d_k.data, a.d_v.data, a.d_g.data, a.d_beta.data = (t.data_ptr() for t in outs)
    ws = _workspace(n, dev)
    with _OnDevice(dev):
        status = load().sdm_gdr_backward(ctypes.byref(a), ws.data_ptr(), n, _stream(dev))
    del keep
    if status:
        _raise(status, "gdr_backward")
    return (*outs, s)


def gdr_step(q, k, v, g, beta, state, *, slots=None, scale=None, out=None, stream=None):
    """One token, or the few of a draft, of each stream: returns o [B, T, Hv, dv] and updates ``state`` in place.

    state [pool, Hv, dk, dv] float32, contiguous. slots: int32 [B] on the GPU, the state each stream uses (None: its
    own number); a stream whose slot is not in the pool, such as -1, is idle: zeros in o, no state touched. No two
    streams may name one slot. The other tensors as in gdr_forward. It has no gradient: a backward pass that reaches o
    is an error."""
    import torch
    scale = _scale(scale)
    key = ("step", _layout(q), _layout(k), _layout(v), _layout(g), _layout(beta), _layout(state), _layout(slots),
           _layout(out), scale)
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _step_plan(q, k, v, g, beta, state, slots, scale, out))
    _no_tangents("gdr_step", q, k, v, g, beta, state, out)
    kept, shape, dtype, dev, copied = plan
    if stream is not None:
        with _under(stream, dev):
            return gdr_step(q, k, v, g, beta, state, slots=slots, scale=scale, out=out)
    recorded = torch.is_grad_enabled() and _requires_grad(q, k, v, g, beta, state)
    written = (state,) if out is None else (state, out)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    if kept is None:
        return out
    if copied:
        q, k, v = _inner(q), _inner(k), _inner(v)
        slots = None if slots is None else slots.contiguous()
    a = sdm_gdr_step_args_t.from_buffer_copy(kept)
    a.q.data, a.k.data, a.v.data, a.g.data = q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr()
    a.beta.data, a.o.data, a.state = beta.data_ptr(), out.data_ptr(), state.data_ptr()
    if slots is not None:
        a.slots = slots.data_ptr()
    with _OnDevice(dev):
        status = load().sdm_gdr_step(ctypes.byref(a), _stream(dev))
    if status:
        _raise(status, "gdr_step")
    _increment_version(written)
    if recorded:
        from ._delta_autograd import NoGradient
        return NoGradient.apply([out], "gdr_step", q, k, v, g, beta, state)
    return out


def _step_plan(q, k, v, g, beta, state, slots, scale, out):
    """(argument struct or None for nothing to do, o's shape, type, device, whether an operand is copied first)"""
    import torch
    B, T, Hk, Hv, dk, dv, dt, dev = _gdr_shapes(q, k, v, g, beta)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state: [pool, Hv, dk, dv] required")
    pool = state.shape[0]
    _tensor(state, "state", (pool, Hv, dk, dv), torch.float32, dev)
    if not state.is_contiguous():
        raise ValueError("state: must be contiguous (it is updated in place)")
    if slots is not None:
        _tensor(slots, "slots", (B,), torch.int32, dev)
    o = _rows(torch.empty((B, T, Hv, dv), dtype=v.dtype, device="meta"), False)
    if out is not None:
        _tensor(out, "out", (B, T, Hv, dv), v.dtype, dev)
        if out.stride(-1) != 1 and dv > 1:
            raise ValueError("out: the last axis must be contiguous")
        o = _rows(out, False)
    if B == 0 or T == 0:
        return None, (B, T, Hv, dv), v.dtype, dev, False
    copied = any(_inner(t) is not t for t in (q, k, v)) or (slots is not None and not slots.is_contiguous())
    q, k, v = _inner(q), _inner(k), _inner(v)
    a = sdm_gdr_step_args_t(dt, dk ** -0.5 if scale is None else float(scale), B, T, Hk, Hv, dk, dv, pool,
                            _rows(q, False), _rows(k, False), _rows(v, False), _rows(g, False), _rows(beta, False), o, 0, 0)
    return a, (B, T, Hv, dv), v.dtype, dev, copied


# ---- the block norm -------------------------------------------------------------------------------------------------
def _ld(t) -> int:
    return 0 if t is None else max(t.stride(0), t.shape[1])


def _norm_common(first, o, z, w_post, w_pre, scale, act):
    """Checks what both directions share; returns the flattened operands and the argument struct."""
    if act not in ACTS:
        raise ValueError(f"act: one of {tuple(ACTS)}")
    if (act == "none") != (z is None):
        raise ValueError("z: given exactly when act is not 'none'")
    if o is None and (w_pre is None or z is not None or w_post is not None or scale is not None):
        raise ValueError("without o there is only the second norm: w_pre is required, z, w_post and scale are not used")
    if o is not None and (w_post is None or scale is None):
        raise ValueError("o: w_post and scale are required with it")
    if first.dim() < 2:
        raise ValueError("rows: [..., D] with two axes at least")
    D = first.shape[-1]
    dev = first.device
    wd = next(w.dtype for w in (w_post, w_pre) if w is not None)
    for w, name in ((w_post, "w_post"), (w_pre, "w_pre"), (scale, "scale")):
        if w is not None:
            _tensor(w, name, (D,), wd, dev)
    return D, dev, wd


def _flat(t):
    """t as rows of its last axis, copied if they are not contiguous."""
    if t is None:
        return None
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    return t if t.stride(-1) == 1 and t.stride(0) >= t.shape[1] or t.is_contiguous() else t.contiguous()


def _norm_plan(backward, x, o, z, w_post, w_pre, scale, act, eps, dy=None, xn=None, rstd=None):
    """The checked argument struct of a forward or backward call, without addresses. x: dx_new in the backward call."""
    import torch
    first = o if o is not None else xn if backward else x
    if not isinstance(first, torch.Tensor):
        raise TypeError("x, o, x_new: a torch tensor")
    D, dev, wd = _norm_common(first, o, z, w_post, w_pre, scale, act)
    dt = _dtype(first, "o")
    names = ("dx_new" if backward else "x", "o", "z", "dy", "x_new")
    rows_of = [x, o, z, dy, xn]
    for t, name in zip(rows_of, names):
        if t is not None:
            _tensor(t, name, first.shape, first.dtype, dev)
    rows = first.numel() // D if D else 0
    if backward:
        if (dy is None) != (w_pre is None):
            raise ValueError("dy: given exactly when w_pre is")
        if dy is None and x is None:
            raise ValueError("dx_new: required without dy")
        if dy is not None and xn is None:
            raise ValueError("x_new: required with dy")
        _tensor(rstd, "rstd", (rows, 2), torch.float32, dev)
    _tensor(first, "o", first.shape)
    plain = [w_post, w_pre, scale, rstd]
    flat = [_flat(t) for t in rows_of]
    copied = (any(f is not t for f, t in zip(flat, rows_of)) or
              any(t is not None and not t.is_contiguous() for t in plain))
    fx, fo, fz, fy, fn = flat
    wt = _dtype(w_post if w_post is not None else w_pre, "weights")
    a = sdm_nrm_args_t(dtype=dt, wtype=wt, act=ACTS[act], eps=eps, rows=rows, D=D, ld_o=_ld(fo), ld_z=_ld(fz))
    n = 0
    if backward:
        a.ld_dxn, a.ld_dy, a.ld_xn, a.ld_dx, a.ld_do, a.ld_dz = _ld(fx), _ld(fy), _ld(fn), D, D, D
        if rows:
            n = load().sdm_nrm_workspace(ctypes.byref(a))
            if n < 0:
                _raise(n, "norm_backward")
    else:
        a.ld_x, a.ld_xn, a.ld_y = _ld(fx), D, D
    return a, n, rows, D, dev, wd, copied, first.shape, first.dtype


def norm_forward(x, o, z, w_post, w_pre, scale, *, act="silu", eps=1e-6, stream=None):
    """The norm after a block, its gate and residual scale, and the norm before the next block, in one pass:

        x_new = x + scale * rms_norm(o) w_post act(z);   y = rms_norm(x_new) w_pre

    returns ``(x_new, y, rstd)``; rstd [rows, 2] float32 is what norm_backward reads. x, o, z [..., D] of one type;
    w_post, w_pre, scale [D] in that type or float32. x None: no residual. w_pre None: y is None. o None (with z,
    w_post and scale): y = rms_norm(x) w_pre alone, and x_new is x. act: "none" (z None), "sigmoid" or "silu"."""
    import torch
    eps = float(eps)
    key = ("norm", _layout(x), _layout(o), _layout(z), _layout(w_post), _layout(w_pre), _layout(scale), act, eps)
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _norm_plan(False, x, o, z, w_post, w_pre, scale, act, eps))
    _no_tangents("norm_forward", x, o, z, w_post, w_pre, scale)
    kept, _, rows, D, dev, _, copied, shape, dtype = plan
    if stream is not None:
        with _under(stream, dev):
            return norm_forward(x, o, z, w_post, w_pre, scale, act=act, eps=eps)
    if torch.is_grad_enabled() and _requires_grad(x, o, z, w_post, w_pre, scale):
        from ._delta_autograd import BlockNorm
        made = BlockNorm.apply(x, o, z, w_post, w_pre, scale, act, eps)
        return made if o is not None else (x, *made)
    x_new = x if o is None else torch.empty(shape, dtype=dtype, device=dev)
    y = None if w_pre is None else torch.empty(shape, dtype=dtype, device=dev)
    rstd = torch.empty((rows, 2), dtype=torch.float32, device=dev)
    if not rows:
        return x_new, y, rstd
    if copied:
        x, o, z = _flat(x), _flat(o), _flat(z)
        w_post, w_pre, scale = (None if t is None else t.contiguous() for t in (w_post, w_pre, scale))
    a = sdm_nrm_args_t.from_buffer_copy(kept)
    a.x, a.o, a.z, a.rstd = _ptr(x), _ptr(o), _ptr(z), rstd.data_ptr()
    a.w_post, a.w_pre, a.scale = _ptr(w_post), _ptr(w_pre), _ptr(scale)
    a.x_new, a.y = 0 if o is None else x_new.data_ptr(), _ptr(y)
    with _OnDevice(dev):
        status = load().sdm_nrm_forward(ctypes.byref(a), _stream(dev))
    if status:
        _raise(status, "norm_forward")
    return x_new, y, rstd


def norm_backward(dx_new, dy, x_new, o, z, w_post, w_pre, scale, rstd, *, act="silu", stream=None):
    """The gradient of norm_forward: ``(dx, do, dz, dw_post, dw_pre, dscale)``, None in the place of what the call did
    not have. dx_new, the gradient of x_new beside the one through y, may be None; dy is None when w_pre is. x_new and
    rstd are the forward's. dx is the gradient of x (of the residual branch); weights' gradients have their type."""
    import torch
    key = ("norm_bwd", _layout(dx_new), _layout(dy), _layout(x_new), _layout(o), _layout(z), _layout(w_post),
           _layout(w_pre), _layout(scale), _layout(rstd), act)
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _norm_plan(True, dx_new, o, z, w_post, w_pre, scale, act, 0.0, dy, x_new, rstd))
    _no_tangents("norm_backward", dx_new, dy, x_new, o, z, w_post, w_pre, scale, rstd)
    kept, n, rows, D, dev, wd, copied, shape, dtype = plan
    if stream is not None:
        with _under(stream, dev):
            return norm_backward(dx_new, dy, x_new, o, z, w_post, w_pre, scale, rstd, act=act)
    dx = torch.empty(shape, dtype=dtype, device=dev)
    do = None if o is None else torch.empty(shape, dtype=dtype, device=dev)
    dz = None if z is None else torch.empty(shape, dtype=dtype, device=dev)
    make = torch.empty if rows else torch.zeros
    dw_post = None if w_post is None else make(D, dtype=wd, device=dev)
    dw_pre = None if w_pre is None else make(D, dtype=wd, device=dev)
    dscale = None if scale is None else make(D, dtype=wd, device=dev)
    if not rows:
        return dx, do, dz, dw_post, dw_pre, dscale
    if copied:
        dx_new, dy, x_new, o, z = (_flat(t) for t in (dx_new, dy, x_new, o, z))
        w_post, w_pre, scale, rstd = (None if t is None else t.contiguous() for t in (w_post, w_pre, scale, rstd))
    a = sdm_nrm_args_t.from_buffer_copy(kept)
    a.o, a.z, a.dxn, a.dy, a.rstd = _ptr(o), _ptr(z), _ptr(dx_new), _ptr(dy), rstd.data_ptr()
    a.x_new = 0 if dy is None else x_new.data_ptr()
    a.w_post, a.w_pre, a.scale = _ptr(w_post), _ptr(w_pre), _ptr(scale)
    a.dx, a.d_o, a.dz = dx.data_ptr(), _ptr(do), _ptr(dz)
    a.dw_post, a.dw_pre, a.dscale = _ptr(dw_post), _ptr(dw_pre), _ptr(dscale)
    ws = _workspace(n, dev)
    with _OnDevice(dev):
        status = load().sdm_nrm_backward(ctypes.byref(a), ws.data_ptr(), n, _stream(dev))
    if status:
        _raise(status, "norm_backward")
    return dx, do, dz, dw_post, dw_pre, dscale
