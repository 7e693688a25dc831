"""The gated linear recurrence, rows in 8 bits and the gated feed-forward product (include/sdm_glr.h, include/sdm_qnt.h,
include/sdm_ffn.h) on torch tensors.

The functions take and return tensors on the current GPU in the manner of delta.py: outputs and workspaces come from torch's
allocator, types and shapes are checked, and the C ABI of libsdm_block is called on torch's current stream (or ``stream``,
which is the call under ``torch.cuda.stream(stream)``). Every arithmetic step runs in the library's HIP kernels; there is no
other path. A wrong argument raises TypeError or ValueError before anything runs.

Where grad mode is on and a tensor of the call requires a gradient, glr_forward and ffn_forward are part of torch's graph
(_block_autograd.py), and a backward pass that reaches glr_step, norm_quant, quant_rows or a feed-forward product of 8-bit
operands, which have no gradient, is an error. The gradients that glr_backward and ffn_backward return have no graph of
their own. There are no forward-mode derivatives: a tensor that carries a tangent is an error.
"""

from __future__ import annotations

import ctypes
import os
import threading

from . import delta
from ._binding import SDM_GX_ERR_HIP, SDM_GX_OK
from ._build import BLOCK_LIB_PATH
from .delta import (SDM_BF16, SDM_F16, SDM_F32, _ARG_ERRORS, _dtype, _flat, _inner, _layout, _ld, _no_tangents, _Plans,
                    _ptr, _requires_grad, _tensor, _under, _workspace)

SDM_E4M3 = 3
GATES = {"none": 0, "sigmoid": 1, "silu": 2}
ACTS = {**GATES, "gelu": 3}
EXPORTS = ("sdm_glr_check", "sdm_glr_step_check", "sdm_glr_marks", "sdm_glr_workspace", "sdm_glr_forward",
           "sdm_glr_backward", "sdm_glr_step", "sdm_qnt_check", "sdm_qnt_rows", "sdm_ffn_check", "sdm_ffn_workspace",
           "sdm_ffn_forward", "sdm_ffn_backward", "sdm_block_strerror", "sdm_block_last_hip_error")

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class sdm_seq_t(ctypes.Structure):
    _fields_ = [("data", _vp), ("batch", _i64), ("token", _i64)]


class sdm_glr_args_t(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("gtype", _i32), ("act", _i32), ("reserved", _i32), ("B", _i64), ("T", _i64), ("D", _i64),
                ("nseq", _i64), ("cu_seqlens", _vp), ("x", sdm_seq_t), ("g", sdm_seq_t), ("z", sdm_seq_t), ("h0", _vp),
                ("marks", _vp), ("y", sdm_seq_t), ("h_final", _vp), ("dy", sdm_seq_t), ("dh_final", _vp), ("dx", sdm_seq_t),
                ("dg", sdm_seq_t), ("dz", sdm_seq_t), ("dh0", _vp)]


class sdm_glr_step_args_t(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("gtype", _i32), ("act", _i32), ("reserved", _i32), ("B", _i64), ("T", _i64), ("D", _i64),
                ("pool", _i64), ("x", sdm_seq_t), ("g", sdm_seq_t), ("z", sdm_seq_t), ("y", sdm_seq_t), ("state", _vp),
                ("slots", _vp)]


class sdm_qnt_args_t(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("wtype", _i32), ("eps", _f32), ("reserved", _i32), ("rows", _i64), ("D", _i64), ("x", _vp),
                ("r", _vp), ("w", _vp), ("ld_x", _i64), ("ld_r", _i64), ("x_new", _vp), ("q", _vp), ("ld_xn", _i64),
                ("ld_q", _i64), ("scale", _vp)]


class sdm_ffn_args_t(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("otype", _i32), ("act", _i32), ("precise", _i32), ("M", _i64), ("K", _i64), ("F", _i64),
                ("x", _vp), ("wg", _vp), ("wu", _vp), ("ld_x", _i64), ("ld_wg", _i64), ("ld_wu", _i64), ("sx", _vp),
                ("sg", _vp), ("su", _vp), ("h", _vp), ("ld_h", _i64), ("gate", _vp), ("up", _vp), ("ld_gate", _i64),
                ("ld_up", _i64), ("dh", _vp), ("ld_dh", _i64), ("dx", _vp), ("dwg", _vp), ("dwu", _vp), ("ld_dx", _i64),
                ("ld_dwg", _i64), ("ld_dwu", _i64)]


_lib = None
_lock = threading.Lock()


def load() -> ctypes.CDLL:
    """Load libsdm_block (once). Fails loudly if it has not been built: there is no fallback path."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(BLOCK_LIB_PATH):
            raise ImportError(f"{BLOCK_LIB_PATH} is missing: build it first "
                              "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(BLOCK_LIB_PATH)
        r, s, q, f = (ctypes.POINTER(t) for t in (sdm_glr_args_t, sdm_glr_step_args_t, sdm_qnt_args_t, sdm_ffn_args_t))
        sig = {
            "sdm_glr_check": [r, _i32],
            "sdm_glr_step_check": [s],
            "sdm_glr_marks": [r],
            "sdm_glr_workspace": [r, _i32],
            "sdm_glr_forward": [r, _vp, _i64, _vp],
            "sdm_glr_backward": [r, _vp, _i64, _vp],
            "sdm_glr_step": [s, _vp],
            "sdm_qnt_check": [q],
            "sdm_qnt_rows": [q, _vp],
            "sdm_ffn_check": [f, _i32],
            "sdm_ffn_workspace": [f, _i32],
            "sdm_ffn_forward": [f, _vp, _i64, _vp],
            "sdm_ffn_backward": [f, _vp, _i64, _vp],
            "sdm_block_strerror": [ctypes.c_int],
            "sdm_block_last_hip_error": [],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = (ctypes.c_char_p if name == "sdm_block_strerror" else
                          _i64 if name.endswith(("_workspace", "_marks")) else ctypes.c_int)
        delta._raw_stream = delta._find_raw_stream()
        _lib = lib
        return lib


def _raise(code: int, what: str):
    if code == SDM_GX_OK:
        return
    msg = load().sdm_block_strerror(code).decode()
    if code == SDM_GX_ERR_HIP:
        msg += f" (hipError {load().sdm_block_last_hip_error()})"
    exc = ValueError if code in _ARG_ERRORS else RuntimeError
    raise exc(f"{what}: {msg} [status {code}]")


_plans = _Plans()
_stream = delta._stream


def _call(fn, what, dev, *args):
    """fn's call on the device's current stream, with the device made current where it is not; raises for a refusal."""
    import torch
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(dev))
    if status:
        _raise(status, what)


class _New:
    """New contiguous tensors of one shape (torch makes them fastest from sizes and strides)."""

    __slots__ = ("shape", "strides", "device")

    def __init__(self, shape, device):
        self.shape, strides, n = tuple(shape), [], 1
        for s in reversed(self.shape):
            strides.append(n)
            n *= max(s, 1)
        self.strides, self.device = tuple(strides[::-1]), device

    def __call__(self, dtype, zero=False):
        import torch
        t = torch.empty_strided(self.shape, self.strides, dtype=dtype, device=self.device)
        return t.zero_() if zero else t


# ---- the gated linear recurrence ------------------------------------------------------------------------------------
def _seq(t) -> sdm_seq_t:
    return sdm_seq_t(0, t.stride(0), t.stride(1))


def _whole(t) -> sdm_seq_t:
    """The strides of a new tensor of t's shape."""
    return sdm_seq_t(0, t.shape[1] * t.shape[2], t.shape[2])


def _glr_shapes(x, g, z, act):
    """Checks what every form shares; (type, g's type, device)."""
    import torch
    for t, name in ((x, "x"), (g, "g")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: a torch tensor")
    if x.dim() != 3:
        raise ValueError("x: [B, T, D] required")
    if act not in GATES:
        raise ValueError(f"act: one of {tuple(GATES)}")
    if (act == "none") != (z is None):
        raise ValueError("z: given exactly when act is not 'none'")
    dt, dev = _dtype(x, "x"), x.device
    _tensor(x, "x", x.shape)
    if g.dtype != torch.float32 and g.dtype != x.dtype:
        raise TypeError(f"g: float32 or {x.dtype} required, got {g.dtype}")
    _tensor(g, "g", x.shape, g.dtype, dev)
    if z is not None:
        _tensor(z, "z", x.shape, x.dtype, dev)
    if x.shape[2] < 1:
        raise ValueError("x: a channel at least")
    return dt, _dtype(g, "g"), dev


def _glr_plan(backward, x, g, z, act, h0, cu, dy=None, dh=None, marks=None):
    """(argument struct without addresses, workspace bytes, shape of marks, of the states, device, whether to copy)"""
    import torch
    dt, gt, dev = _glr_shapes(x, g, z, act)
    B, T, D = x.shape
    nseq = B
    if cu is not None:
        if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 2:
            raise ValueError("cu_seqlens: an int32 tensor of one more entry than sequences, two at least")
        if B != 1:
            raise ValueError("cu_seqlens: packed sequences come in one row (B = 1)")
        nseq = cu.shape[0] - 1
        _tensor(cu, "cu_seqlens", (nseq + 1,), torch.int32, dev)
    for t, name in ((h0, "initial_state"), (dh, "dfinal_state")):
        if t is not None:
            _tensor(t, name, (nseq, D), torch.float32, dev)
    if backward:
        _tensor(dy, "dy", x.shape, x.dtype, dev)
    copied = (any(_inner(t) is not t for t in (x, g, z, dy) if t is not None) or
              any(not t.is_contiguous() for t in (cu, h0, dh, marks) if t is not None))
    x, g, z = _inner(x), _inner(g), None if z is None else _inner(z)
    a = sdm_glr_args_t(dtype=dt, gtype=gt, act=GATES[act], B=B, T=T, D=D, nseq=nseq, x=_seq(x), g=_seq(g))
    if z is not None:
        a.z = _seq(z)
    if backward:
        a.dy, a.dx, a.dg = _seq(_inner(dy)), _whole(x), _whole(g)
        if z is not None:
            a.dz = _whole(z)
    else:
        a.y = _whole(x)
    n = rows = 0
    if B and T:
        a.cu_seqlens = 0 if cu is None else 4       # whether there is one
        n, rows = load().sdm_glr_workspace(ctypes.byref(a), int(backward)), load().sdm_glr_marks(ctypes.byref(a))
        if n < 0 or rows < 0:
            _raise(min(n, rows), "glr_backward" if backward else "glr_forward")
        a.cu_seqlens = 0
    if backward:
        _tensor(marks, "marks", (rows, D), torch.float32, dev)
    return a, n, _New(x.shape, dev), _New((rows, D), dev), _New((nseq, D), dev), dev, copied


def _glr_operands(copied, a, x, g, z, h0, cu):
    """Fills the inputs' addresses in; returns what has to live until the call."""
    if copied:
        x, g, z = _inner(x), _inner(g), None if z is None else _inner(z)
        cu = None if cu is None else cu.contiguous()
        h0 = None if h0 is None else h0.contiguous()
    a.x.data, a.g.data, a.z.data, a.cu_seqlens, a.h0 = x.data_ptr(), g.data_ptr(), _ptr(z), _ptr(cu), _ptr(h0)
    return x, g, z, cu, h0


def glr_forward(x, g, z=None, *, act="none", initial_state=None, cu_seqlens=None, stream=None):
    """The gated linear recurrence over whole sequences, h_t = exp(g_t) h_{t-1} + x_t and y_t = h_t act(z_t):
    ``(y, state after the last token, marks)``; marks is what glr_backward reads.

    x [B, T, D] float32, bfloat16 or float16; g (log decay), like x or float32; z like x, exactly when act is "sigmoid" or
    "silu" ("none": y is h); states [sequences, D] float32. cu_seqlens: int32 [n + 1] on the GPU, n sequences packed into
    one row; tokens of no sequence get zeros. Any strides; a last axis that is not contiguous is copied first.
    """
    import torch
    key = ("glr", _layout(x), _layout(g), _layout(z), act, _layout(initial_state), _layout(cu_seqlens))
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _glr_plan(False, x, g, z, act, initial_state, cu_seqlens))
    _no_tangents("glr_forward", x, g, z, initial_state)
    kept, n, whole, marks, states, dev, copied = plan
    if stream is not None:
        with _under(stream, dev):
            return glr_forward(x, g, z, act=act, initial_state=initial_state, cu_seqlens=cu_seqlens)
    if torch.is_grad_enabled() and _requires_grad(x, g, z, initial_state):
        from ._block_autograd import GatedLinearRecurrence
        return GatedLinearRecurrence.apply(x, g, z, initial_state, act, cu_seqlens)
    y, h, marks = whole(x.dtype, cu_seqlens is not None), states(torch.float32), marks(torch.float32)
    if not y.numel():
        h.zero_() if initial_state is None else h.copy_(initial_state)
        return y, h, marks
    a = sdm_glr_args_t.from_buffer_copy(kept)
    keep = _glr_operands(copied, a, x, g, z, initial_state, cu_seqlens)
    a.y.data, a.h_final, a.marks = y.data_ptr(), h.data_ptr(), marks.data_ptr()
    ws = _workspace(n, dev) if n else None
    _call(load().sdm_glr_forward, "glr_forward", dev, ctypes.byref(a), _ptr(ws), n)
    del keep
    return y, h, marks


def glr_backward(x, g, z, dy, marks, *, act="none", initial_state=None, dfinal_state=None, cu_seqlens=None, stream=None):
    """The gradient of glr_forward: ``(dx, dg, dz, dinitial_state)`` from dy, the gradient of y, and dfinal_state, that of
    the last state (None: zero); dz is None without z. marks is the forward call's, and the other arguments are its own.
    Gradients have their tensors' shapes and types; tokens of no sequence get zeros."""
    import torch
    key = ("glr_bwd", _layout(x), _layout(g), _layout(z), act, _layout(initial_state), _layout(cu_seqlens), _layout(dy),
           _layout(dfinal_state), _layout(marks))
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _glr_plan(True, x, g, z, act, initial_state, cu_seqlens, dy, dfinal_state, marks))
    _no_tangents("glr_backward", x, g, z, dy, marks, initial_state, dfinal_state)
    kept, n, whole, _, states, dev, copied = plan
    if stream is not None:
        with _under(stream, dev):
            return glr_backward(x, g, z, dy, marks, act=act, initial_state=initial_state, dfinal_state=dfinal_state,
                                cu_seqlens=cu_seqlens)
    zero = cu_seqlens is not None
    dx, dg, dz = whole(x.dtype, zero), whole(g.dtype, zero), None if z is None else whole(x.dtype, zero)
    dh0 = states(torch.float32)
    if not dx.numel():
        dh0.zero_() if dfinal_state is None else dh0.copy_(dfinal_state)
        return dx, dg, dz, dh0
    a = sdm_glr_args_t.from_buffer_copy(kept)
    keep = _glr_operands(copied, a, x, g, z, initial_state, cu_seqlens)
    if copied:
        dy, marks = _inner(dy), marks.contiguous()
        dfinal_state = None if dfinal_state is None else dfinal_state.contiguous()
    a.dy.data, a.marks, a.dh_final = dy.data_ptr(), marks.data_ptr(), _ptr(dfinal_state)
    a.dx.data, a.dg.data, a.dz.data, a.dh0 = dx.data_ptr(), dg.data_ptr(), _ptr(dz), dh0.data_ptr()
    ws = _workspace(n, dev) if n else None
    _call(load().sdm_glr_backward, "glr_backward", dev, ctypes.byref(a), _ptr(ws), n)
    del keep
    return dx, dg, dz, dh0


def glr_step(x, g, z, state, *, act="none", slots=None, stream=None):
    """One token, or the few of a draft, of each stream: returns y [B, T, D] and updates ``state`` in place.

    state [pool, D] float32, contiguous. slots: int32 [B] on the GPU, the state each stream uses (None: its own number); a
    stream whose slot is not in the pool, such as -1, is idle: zeros in y, no state touched. No two streams may name one
    slot. The other tensors as in glr_forward. It has no gradient: a backward pass that reaches y is an error."""
    import torch
    key = ("glr_step", _layout(x), _layout(g), _layout(z), act, _layout(state), _layout(slots))
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _glr_step_plan(x, g, z, state, act, slots))
    _no_tangents("glr_step", x, g, z, state)
    kept, whole, dev, copied = plan
    if stream is not None:
        with _under(stream, dev):
            return glr_step(x, g, z, state, act=act, slots=slots)
    recorded = torch.is_grad_enabled() and _requires_grad(x, g, z, state)
    y = whole(x.dtype)
    if not y.numel():
        return y
    if copied:
        x, g, z = _inner(x), _inner(g), None if z is None else _inner(z)
        slots = None if slots is None else slots.contiguous()
    a = sdm_glr_step_args_t.from_buffer_copy(kept)
    a.x.data, a.g.data, a.z.data, a.y.data = x.data_ptr(), g.data_ptr(), _ptr(z), y.data_ptr()
    a.state, a.slots = state.data_ptr(), _ptr(slots)
    _call(load().sdm_glr_step, "glr_step", dev, ctypes.byref(a))
    delta._increment_version((state,))
    if recorded:
        from ._block_autograd import NoGradient
        return NoGradient.apply([y], "glr_step", x, g, z, state)
    return y


def _glr_step_plan(x, g, z, state, act, slots):
    import torch
    dt, gt, dev = _glr_shapes(x, g, z, act)
    B, T, D = x.shape
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise ValueError("state: [pool, D] required")
    _tensor(state, "state", (state.shape[0], D), torch.float32, dev)
    if not state.is_contiguous():
        raise ValueError("state: must be contiguous (it is updated in place)")
    if slots is not None:
        _tensor(slots, "slots", (B,), torch.int32, dev)
    elif state.shape[0] < B:
        raise ValueError("state: a state for every stream required without slots")
    copied = any(_inner(t) is not t for t in (x, g, z) if t is not None) or (slots is not None and not slots.is_contiguous())
    x, g, z = _inner(x), _inner(g), None if z is None else _inner(z)
    a = sdm_glr_step_args_t(dtype=dt, gtype=gt, act=GATES[act], B=B, T=T, D=D, pool=state.shape[0], x=_seq(x), g=_seq(g),
                            y=_whole(x))
    if z is not None:
        a.z = _seq(z)
    return a, _New(x.shape, dev), dev, copied


# ---- rows in 8 bits -------------------------------------------------------------------------------------------------
def _qnt_plan(what, x, r, w, eps):
    import torch
    if not isinstance(x, torch.Tensor):
        raise TypeError("x: a torch tensor")
    if x.dim() < 2 or x.shape[-1] < 1:
        raise ValueError("x: [..., D] with two axes and a column at least")
    D, dev, dt = x.shape[-1], x.device, _dtype(x, "x")
    _tensor(x, "x", x.shape)
    if r is not None:
        _tensor(r, "residual", x.shape, x.dtype, dev)
    wt = dt
    if w is not None:
        _tensor(w, "w", (D,), None, dev)
        wt = _dtype(w, "w")
        if wt != SDM_F32 and wt != dt:
            raise TypeError(f"w: float32 or {x.dtype} required, got {w.dtype}")
    rows = x.numel() // D
    fx, fr = _flat(x), _flat(r)
    copied = fx is not x or fr is not r or (w is not None and not w.is_contiguous())
    a = sdm_qnt_args_t(dtype=dt, wtype=wt, eps=eps, rows=rows, D=D, ld_x=_ld(fx), ld_r=_ld(fr), ld_xn=D, ld_q=D)
    return a, _New(x.shape, dev), _New(x.shape[:-1], dev), dev, copied


def _qnt(what, x, r, w, eps, stream):
    import torch
    eps = float(eps)
    key = ("qnt", _layout(x), _layout(r), _layout(w), eps)
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _qnt_plan(what, x, r, w, eps))
    _no_tangents(what, x, r, w)
    kept, whole, by_row, dev, copied = plan
    if stream is not None:
        with _under(stream, dev):
            return _qnt(what, x, r, w, eps, None)
    recorded = torch.is_grad_enabled() and _requires_grad(x, r, w)
    inputs = (x, r, w)
    q, scale, x_new = whole(torch.float8_e4m3fn), by_row(torch.float32), x if r is None else whole(x.dtype)
    if kept.rows:
        if copied:
            x, r, w = _flat(x), _flat(r), None if w is None else w.contiguous()
        a = sdm_qnt_args_t.from_buffer_copy(kept)
        a.x, a.r, a.w, a.q, a.scale = x.data_ptr(), _ptr(r), _ptr(w), q.data_ptr(), scale.data_ptr()
        a.x_new = 0 if r is None else x_new.data_ptr()
        _call(load().sdm_qnt_rows, what, dev, ctypes.byref(a))
    if recorded:
        from ._block_autograd import NoGradient
        scale = NoGradient.apply([scale], what, *inputs)
        if r is not None:
            x_new = NoGradient.apply([x_new], what, *inputs)
    return q, scale, x_new


def norm_quant(x, residual, w, *, eps=1e-6, stream=None):
    """The norm before a feed-forward, with the residual's addition and an output in 8 bits:

        x_new = x + residual;   y = rms_norm(x_new) w;   q = e4m3(y / scale),  scale = max |y| / 448 of each row

    returns ``(q, scale, x_new)``: q [..., D] float8_e4m3fn, scale [...] float32; q times its row's scale stands for y. x,
    residual [..., D] of one type (float32, bfloat16, float16); w [D] in that type or float32. residual None: x_new is x. A
    row that holds a value that is not finite gets NaN throughout. It has no gradient: a backward pass that reaches scale or
    x_new is an error (q cannot be part of a graph)."""
    if w is None:
        raise ValueError("w: required (quant_rows rounds without a norm)")
    return _qnt("norm_quant", x, residual, w, eps, stream)


def quant_rows(x, *, stream=None):
    """Rows brought to 8 bits, such as a weight's: ``(q, scale)``, q = e4m3(x / scale) with scale = max |x| / 448 of each
    row. x [..., D] float32, bfloat16 or float16. It has no gradient, as norm_quant."""
    return _qnt("quant_rows", x, None, None, 0.0, stream)[:2]


# ---- the gated feed-forward product ---------------------------------------------------------------------------------
def _ffn_plan(x, wg, wu, act, scales, dtype, dh=None, kept=None):
    """(argument struct without addresses, what makes h, its type, device, whether an operand is copied first)"""
    import torch
    for t, name in ((x, "x"), (wg, "w_gate"), (wu, "w_up")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: a torch tensor")
    if act not in ACTS:
        raise ValueError(f"act: one of {tuple(ACTS)}")
    if x.dim() < 2 or wg.dim() != 2:
        raise ValueError("x: [..., K] with two axes at least, and w_gate, w_up: [F, K] required")
    dev, lead = x.device, tuple(x.shape[:-1])
    F, K = wg.shape
    if F < 1 or K < 1:
        raise ValueError("w_gate: a row and a column at least")
    small = x.dtype == torch.float8_e4m3fn
    dt = SDM_E4M3 if small else _dtype(x, "x")
    _tensor(x, "x", (*lead, K))
    _tensor(wg, "w_gate", (F, K), x.dtype, dev)
    _tensor(wu, "w_up", (F, K), x.dtype, dev)
    for t, name, shape in zip(scales, ("x_scale", "gate_scale", "up_scale"), (lead, (F,), (F,))):
        if small != (t is not None):
            raise ValueError(f"{name}: given exactly when x and the weights are float8_e4m3fn")
        if small:
            _tensor(t, name, shape, torch.float32, dev)
    if small:
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("dtype: bfloat16 or float16")
    elif dtype not in (None, x.dtype):
        raise TypeError("dtype: another than x's is for float8_e4m3fn only")
    dtype = x.dtype if dtype is None else dtype
    ot = {torch.float32: SDM_F32, torch.bfloat16: SDM_BF16, torch.float16: SDM_F16}[dtype]
    M = x.numel() // K
    fx, fg, fu = _flat(x), _flat(wg), _flat(wu)
    copied = (fx is not x or fg is not wg or fu is not wu or any(t is not None and not t.is_contiguous() for t in scales))
    a = sdm_ffn_args_t(dtype=dt, otype=ot, act=ACTS[act], M=M, K=K, F=F, ld_x=_ld(fx), ld_wg=_ld(fg), ld_wu=_ld(fu), ld_h=F,
                       ld_gate=F, ld_up=F, ld_dx=K, ld_dwg=K, ld_dwu=K)
    if dh is not None:
        if small:
            raise TypeError("x: 8-bit operands have no gradient")
        if not isinstance(kept, (tuple, list)) or len(kept) != 2:
            raise TypeError("kept: the pair that ffn_forward(keep=True) returned")
        _tensor(dh, "dh", (*lead, F), x.dtype, dev)
        for t, name in zip(kept, ("kept[0]", "kept[1]")):
            _tensor(t, name, (*lead, F), torch.float32, dev)
        fd, f0, f1 = _flat(dh), _flat(kept[0]), _flat(kept[1])
        copied = copied or fd is not dh or f0 is not kept[0] or f1 is not kept[1]
        a.ld_dh, a.ld_gate, a.ld_up = _ld(fd), _ld(f0), _ld(f1)
    return a, _New((*lead, F), dev), dtype, dev, copied


def ffn_forward(x, w_gate, w_up, *, act="silu", keep=False, x_scale=None, gate_scale=None, up_scale=None, dtype=None,
                precise=False, stream=None):
    """The gated feed-forward product ``h = act(x w_gate^T) * (x w_up^T)``, both projections, the activation and the product
    in one kernel: h [..., F], or with keep ``(h, kept)``, kept the pair of products (float32) that ffn_backward reads.

    x [..., K], w_gate, w_up [F, K] of one type: float32, bfloat16, float16, or float8_e4m3fn with x_scale [...],
    gate_scale and up_scale [F] float32 (what norm_quant and quant_rows return); h has that type, or for 8-bit operands
    ``dtype``, bfloat16 (the default) or float16. act: "none", "sigmoid", "silu" or "gelu" (with the normal distribution's
    integral). precise: ffn_backward's, for the gradient through torch's graph."""
    import torch
    scales = (x_scale, gate_scale, up_scale)
    key = ("ffn", _layout(x), _layout(w_gate), _layout(w_up), act, _layout(x_scale), _layout(gate_scale), _layout(up_scale),
           dtype)
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _ffn_plan(x, w_gate, w_up, act, scales, dtype))
    _no_tangents("ffn_forward", x, w_gate, w_up, *scales)
    struct, whole, otype, dev, copied = plan
    if stream is not None:
        with _under(stream, dev):
            return ffn_forward(x, w_gate, w_up, act=act, keep=keep, x_scale=x_scale, gate_scale=gate_scale, up_scale=up_scale,
                               dtype=dtype, precise=precise)
    recorded = torch.is_grad_enabled() and _requires_grad(x, w_gate, w_up, *scales)
    if recorded and x_scale is None:
        from ._block_autograd import GatedFeedForward
        h, *kept = GatedFeedForward.apply(x, w_gate, w_up, act, precise)
        return (h, tuple(kept)) if keep else h
    h, kept = whole(otype), (whole(torch.float32), whole(torch.float32)) if keep else (None, None)
    inputs = (x, w_gate, w_up, *scales)
    if struct.M:
        if copied:
            x, w_gate, w_up = _flat(x), _flat(w_gate), _flat(w_up)
            x_scale, gate_scale, up_scale = (None if t is None else t.contiguous() for t in scales)
        a = sdm_ffn_args_t.from_buffer_copy(struct)
        a.x, a.wg, a.wu, a.h = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), h.data_ptr()
        a.sx, a.sg, a.su, a.gate, a.up = _ptr(x_scale), _ptr(gate_scale), _ptr(up_scale), _ptr(kept[0]), _ptr(kept[1])
        n = load().sdm_ffn_workspace(ctypes.byref(a), 0)
        if n < 0:
            _raise(n, "ffn_forward")
        ws = _workspace(n, dev) if n else None
        _call(load().sdm_ffn_forward, "ffn_forward", dev, ctypes.byref(a), _ptr(ws), n)
    if recorded:
        from ._block_autograd import NoGradient
        h = NoGradient.apply([h], "ffn_forward of 8-bit operands", *inputs)
    return (h, kept) if keep else h


def ffn_backward(dh, x, w_gate, w_up, kept, *, act="silu", precise=False, stream=None):
    """The gradient of ffn_forward: ``(dx, dw_gate, dw_up)`` from dh and what ffn_forward(keep=True) kept. Gradients have
    their tensors' shapes and types (float32, bfloat16 or float16). 16-bit types: the gradients of both products are rounded to the
    type on their way, which makes the result's error 1.4 times that of its own rounding; with precise they are not, and the
    products take twice as long."""
    import torch
    if not isinstance(kept, (tuple, list)) or len(kept) != 2:
        raise TypeError("kept: the pair that ffn_forward(keep=True) returned")
    if dh is None:
        raise TypeError("dh: a torch tensor")
    key = ("ffn_bwd", _layout(dh), _layout(x), _layout(w_gate), _layout(w_up), _layout(kept[0]), _layout(kept[1]), act)
    plan = _plans.get(key)
    if plan is None:
        plan = _plans.put(key, _ffn_plan(x, w_gate, w_up, act, (None,) * 3, None, dh, kept))
    _no_tangents("ffn_backward", dh, x, w_gate, w_up, *kept)
    struct, _, otype, dev, copied = plan
    if stream is not None:
        with _under(stream, dev):
            return ffn_backward(dh, x, w_gate, w_up, kept, act=act, precise=precise)
    make = torch.empty if struct.M else torch.zeros
    dx = torch.empty(x.shape, dtype=otype, device=dev)
    dwg, dwu = (make(w_gate.shape, dtype=otype, device=dev) for _ in range(2))
    if not struct.M:
        return dx, dwg, dwu
    gate, up = kept
    if copied:
        dh, x, w_gate, w_up, gate, up = (_flat(t) for t in (dh, x, w_gate, w_up, gate, up))
    a = sdm_ffn_args_t.from_buffer_copy(struct)
    a.dh, a.x, a.wg, a.wu, a.gate, a.up = (t.data_ptr() for t in (dh, x, w_gate, w_up, gate, up))
    a.dx, a.dwg, a.dwu, a.precise = dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(), bool(precise)
    n = load().sdm_ffn_workspace(ctypes.byref(a), 1)
    if n < 0:
        _raise(n, "ffn_backward")
    ws = _workspace(n, dev)
    _call(load().sdm_ffn_backward, "ffn_backward", dev, ctypes.byref(a), ws.data_ptr(), n)
    return dx, dwg, dwu
