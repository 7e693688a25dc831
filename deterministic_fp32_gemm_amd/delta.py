"""The gated delta rule and the block norm (include/sdm_gdr.h, include/sdm_nrm.h) on torch tensors.

The functions take and return tensors on the current GPU: they allocate outputs and workspaces with torch's allocator,
check types and shapes, and call the C ABI of libsdm_delta on torch's current stream (or ``stream``). Every arithmetic
step runs in the library's HIP kernels; there is no other path. A wrong argument raises TypeError or ValueError before
anything runs. Tensors used on a stream other than the one they were made on are the caller's to keep alive, as with
any torch operation called under that stream.
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
    """t with its last axis contiguous and no negative or expanded layout the kernels could not address."""
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _rows(t) -> sdm_rows_t:
    st = t.stride()
    return sdm_rows_t(t.data_ptr(), st[0], st[1], st[2])


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream, device) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


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


def _gdr_args(q, k, v, g, beta, scale, initial_state, cu_seqlens):
    import torch
    B, T, Hk, Hv, dk, dv, dt, dev = _gdr_shapes(q, k, v, g, beta)
    nseq = B
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens: an int32 tensor of one more entry than sequences, two at least")
        if B != 1:
            raise ValueError("cu_seqlens: packed sequences come in one row (B = 1)")
        nseq = cu_seqlens.shape[0] - 1
        _tensor(cu_seqlens, "cu_seqlens", (nseq + 1,), torch.int32, dev)
        if not cu_seqlens.is_contiguous():
            cu_seqlens = cu_seqlens.contiguous()
    if initial_state is not None:
        initial_state = _tensor(initial_state, "initial_state", (nseq, Hv, dk, dv), torch.float32, dev).contiguous()
    q, k, v = _inner(q), _inner(k), _inner(v)
    a = sdm_gdr_args_t(dtype=dt, scale=dk ** -0.5 if scale is None else float(scale), B=B, T=T, Hk=Hk, Hv=Hv, dk=dk,
                       dv=dv, nseq=nseq, cu_seqlens=_ptr(cu_seqlens), q=_rows(q), k=_rows(k), v=_rows(v), g=_rows(g),
                       beta=_rows(beta), s0=_ptr(initial_state))
    return a, (q, k, v, cu_seqlens, initial_state), nseq, dev


def gdr_forward(q, k, v, g, beta, *, scale=None, initial_state=None, final_state=True, cu_seqlens=None, stream=None):
    """The gated delta rule over whole sequences: ``(o, state after the last token)``, the state None unless asked for.

    q, k [B, T, Hk, dk], v [B, T, Hv, dv] of one type (float32, bfloat16, float16; Hv a multiple of Hk: value heads
    share q/k heads in order), g (log decay) and beta [B, T, Hv] float32, states [sequences, Hv, dk, dv] float32.
    scale: 1/sqrt(dk) unless given. cu_seqlens: int32 [n + 1] on the GPU, n sequences packed into one row; tokens of no
    sequence get zeros. Any strides; a last axis that is not contiguous is copied first.
    """
    import torch
    a, keep, nseq, dev = _gdr_args(q, k, v, g, beta, scale, initial_state, cu_seqlens)
    make = torch.empty if cu_seqlens is None else torch.zeros
    o = make(v.shape, dtype=v.dtype, device=dev)
    s = torch.empty((nseq, a.Hv, a.dk, a.dv), dtype=torch.float32, device=dev) if final_state else None
    if a.T == 0 or a.B == 0:
        if s is not None:
            s.zero_() if initial_state is None else s.copy_(initial_state)
        return o, s
    a.o, a.s_final = _rows(o), _ptr(s)
    lib = load()
    with torch.cuda.device(dev):
        n = lib.sdm_gdr_workspace(ctypes.byref(a), 0)
        if n < 0:
            _raise(n, "gdr_forward")
        ws = _workspace(n, dev)
        _raise(lib.sdm_gdr_forward(ctypes.byref(a), ws.data_ptr(), n, _stream(stream, dev)), "gdr_forward")
    return o, s


def gdr_backward(q, k, v, g, beta, do, *, scale=None, initial_state=None, dfinal_state=None, cu_seqlens=None,
                 stream=None):
    """The gradient of gdr_forward: ``(dq, dk, dv, dg, dbeta, dinitial_state)`` from do, the gradient of o, and
    dfinal_state, that of the last state (None: zero). It recomputes the forward's states and needs nothing saved but
    the inputs. Gradients have their tensors' shapes and types; tokens of no sequence get zeros."""
    import torch
    a, keep, nseq, dev = _gdr_args(q, k, v, g, beta, scale, initial_state, cu_seqlens)
    do = _inner(_tensor(do, "do", v.shape, v.dtype, dev))
    if dfinal_state is not None:
        dfinal_state = _tensor(dfinal_state, "dfinal_state", (nseq, a.Hv, a.dk, a.dv), torch.float32, dev).contiguous()
    make = torch.empty if cu_seqlens is None else torch.zeros
    outs = [make(t.shape, dtype=t.dtype, device=dev) for t in (q, k, v, g, beta)]
    ds = torch.empty((nseq, a.Hv, a.dk, a.dv), dtype=torch.float32, device=dev)
    if a.T == 0 or a.B == 0:
        ds.zero_() if dfinal_state is None else ds.copy_(dfinal_state)
        return (*outs, ds)
    a.d_o, a.ds_final, a.ds0 = _rows(do), _ptr(dfinal_state), _ptr(ds)
    a.d_q, a.d_k, a.d_v, a.d_g, a.d_beta = (_rows(t) for t in outs)
    lib = load()
    with torch.cuda.device(dev):
        n = lib.sdm_gdr_workspace(ctypes.byref(a), 1)
        if n < 0:
            _raise(n, "gdr_backward")
        ws = _workspace(n, dev)
        _raise(lib.sdm_gdr_backward(ctypes.byref(a), ws.data_ptr(), n, _stream(stream, dev)), "gdr_backward")
    return (*outs, ds)


def gdr_step(q, k, v, g, beta, state, *, slots=None, scale=None, out=None, stream=None):
    """One token, or the few of a draft, of each stream: returns o [B, T, Hv, dv] and updates ``state`` in place.

    state [pool, Hv, dk, dv] float32, contiguous. slots: int32 [B] on the GPU, the state each stream uses (None: its
    own number); a stream whose slot is not in the pool, such as -1, is idle: zeros in o, no state touched. No two
    streams may name one slot. The other tensors as in gdr_forward."""
    import torch
    B, T, Hk, Hv, dk, dv, dt, dev = _gdr_shapes(q, k, v, g, beta)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state: [pool, Hv, dk, dv] required")
    pool = state.shape[0]
    _tensor(state, "state", (pool, Hv, dk, dv), torch.float32, dev)
    if not state.is_contiguous():
        raise ValueError("state: must be contiguous (it is updated in place)")
    if slots is not None:
        slots = _tensor(slots, "slots", (B,), torch.int32, dev).contiguous()
    if out is None:
        out = torch.empty((B, T, Hv, dv), dtype=v.dtype, device=dev)
    else:
        _tensor(out, "out", (B, T, Hv, dv), v.dtype, dev)
        if out.stride(-1) != 1 and dv > 1:
            raise ValueError("out: the last axis must be contiguous")
    if B == 0 or T == 0:
        return out
    q, k, v = _inner(q), _inner(k), _inner(v)
    a = sdm_gdr_step_args_t(dt, dk ** -0.5 if scale is None else float(scale), B, T, Hk, Hv, dk, dv, pool, _rows(q),
                            _rows(k), _rows(v), _rows(g), _rows(beta), _rows(out), state.data_ptr(), _ptr(slots))
    with torch.cuda.device(dev):
        _raise(load().sdm_gdr_step(ctypes.byref(a), _stream(stream, dev)), "gdr_step")
    return out


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


def _flat(t, name, like, dtype, dev):
    if t is None:
        return None
    _tensor(t, name, like.shape, dtype, dev)
    t = t.reshape(-1, like.shape[-1])
    return t if t.stride(-1) == 1 and t.stride(0) >= t.shape[1] or t.is_contiguous() else t.contiguous()


def norm_forward(x, o, z, w_post, w_pre, scale, *, act="silu", eps=1e-6, stream=None):
    """The norm after a block, its gate and residual scale, and the norm before the next block, in one pass:

        x_new = x + scale * rms_norm(o) w_post act(z);   y = rms_norm(x_new) w_pre

    returns ``(x_new, y, rstd)``; rstd [rows, 2] float32 is what norm_backward reads. x, o, z [..., D] of one type;
    w_post, w_pre, scale [D] in that type or float32. x None: no residual. w_pre None: y is None. o None (with z,
    w_post and scale): y = rms_norm(x) w_pre alone, and x_new is x. act: "none" (z None), "sigmoid" or "silu"."""
    import torch
    first = o if o is not None else x
    if not isinstance(first, torch.Tensor):
        raise TypeError("x, o: a torch tensor")
    D, dev, wd = _norm_common(first, o, z, w_post, w_pre, scale, act)
    dt = _dtype(first, "o" if o is not None else "x")
    x2, o2, z2 = (_flat(t, n, first, first.dtype, dev) for t, n in ((x, "x"), (o, "o"), (z, "z")))
    _tensor(first, "o" if o is not None else "x", first.shape)
    rows = first.numel() // D if D else 0
    x_new = x if o is None else torch.empty(first.shape, dtype=first.dtype, device=dev)
    y = None if w_pre is None else torch.empty(first.shape, dtype=first.dtype, device=dev)
    rstd = torch.empty((rows, 2), dtype=torch.float32, device=dev)
    if rows == 0:
        return x_new, y, rstd
    w = [None if t is None else t.contiguous() for t in (w_post, w_pre, scale)]
    a = sdm_nrm_args_t(dtype=dt, wtype=_dtype(w[0] if w[0] is not None else w[1], "weights"), act=ACTS[act], eps=eps,
                       rows=rows, D=D, x=_ptr(x2), o=_ptr(o2), z=_ptr(z2), ld_x=_ld(x2), ld_o=_ld(o2), ld_z=_ld(z2),
                       w_post=_ptr(w[0]), w_pre=_ptr(w[1]), scale=_ptr(w[2]), x_new=0 if o is None else x_new.data_ptr(),
                       y=_ptr(y), ld_xn=D, ld_y=D, rstd=rstd.data_ptr())
    with torch.cuda.device(dev):
        _raise(load().sdm_nrm_forward(ctypes.byref(a), _stream(stream, dev)), "norm_forward")
    return x_new, y, rstd


def norm_backward(dx_new, dy, x_new, o, z, w_post, w_pre, scale, rstd, *, act="silu", stream=None):
    """The gradient of norm_forward: ``(dx, do, dz, dw_post, dw_pre, dscale)``, None in the place of what the call did
    not have. dx_new, the gradient of x_new beside the one through y, may be None; dy is None when w_pre is. x_new and
    rstd are the forward's. dx is the gradient of x (of the residual branch); weights' gradients have their type."""
    import torch
    first = o if o is not None else x_new
    if not isinstance(first, torch.Tensor):
        raise TypeError("x_new, o: a torch tensor")
    D, dev, wd = _norm_common(first, o, z, w_post, w_pre, scale, act)
    dt = _dtype(first, "o" if o is not None else "x_new")
    _tensor(first, "o" if o is not None else "x_new", first.shape)
    if (dy is None) != (w_pre is None):
        raise ValueError("dy: given exactly when w_pre is")
    if dy is None and dx_new is None:
        raise ValueError("dx_new: required without dy")
    if dy is not None and x_new is None:
        raise ValueError("x_new: required with dy")
    rows = first.numel() // D if D else 0
    _tensor(rstd, "rstd", (rows, 2), torch.float32, dev)
    rstd = rstd.contiguous()
    u2, y2, xn2, o2, z2 = (_flat(t, n, first, first.dtype, dev) for t, n in
                           ((dx_new, "dx_new"), (dy, "dy"), (x_new, "x_new"), (o, "o"), (z, "z")))
    like = dict(dtype=first.dtype, device=dev)
    dx = torch.empty(first.shape, **like)
    do = None if o is None else torch.empty(first.shape, **like)
    dz = None if z is None else torch.empty(first.shape, **like)
    make = torch.zeros if rows == 0 else torch.empty
    dw = [None if t is None else make(D, dtype=wd, device=dev) for t in (w_post, w_pre, scale)]
    if rows == 0:
        return dx, do, dz, *dw
    w = [None if t is None else t.contiguous() for t in (w_post, w_pre, scale)]
    a = sdm_nrm_args_t(dtype=dt, wtype=_dtype(w[0] if w[0] is not None else w[1], "weights"), act=ACTS[act], eps=0.0,
                       rows=rows, D=D, o=_ptr(o2), z=_ptr(z2), ld_o=_ld(o2), ld_z=_ld(z2), w_post=_ptr(w[0]),
                       w_pre=_ptr(w[1]), scale=_ptr(w[2]), x_new=0 if dy is None else xn2.data_ptr(), ld_xn=_ld(xn2),
                       rstd=rstd.data_ptr(), dxn=_ptr(u2), dy=_ptr(y2), ld_dxn=_ld(u2), ld_dy=_ld(y2),
                       dx=dx.data_ptr(), d_o=_ptr(do), dz=_ptr(dz), ld_dx=D, ld_do=D, ld_dz=D, dw_post=_ptr(dw[0]),
                       dw_pre=_ptr(dw[1]), dscale=_ptr(dw[2]))
    lib = load()
    with torch.cuda.device(dev):
        n = lib.sdm_nrm_workspace(ctypes.byref(a))
        if n < 0:
            _raise(n, "norm_backward")
        ws = _workspace(n, dev)
        _raise(lib.sdm_nrm_backward(ctypes.byref(a), ws.data_ptr(), n, _stream(stream, dev)), "norm_backward")
    return dx, do, dz, *dw
