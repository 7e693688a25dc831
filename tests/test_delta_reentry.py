"""A call of the delta entry points that is entered again before its launch, by a finaliser, a signal handler or an
allocator's callback on the same thread, with tensors of the same layout (no GPU: the library is replaced by a recorder
of the addresses that each launch gets)."""

import contextlib
import ctypes

import pytest
import torch

from deterministic_fp32_gemm_amd import delta as D


class Recorder:
    def __init__(self):
        self.launches = []

    def __getattr__(self, name):
        def call(args, *rest):
            if name.endswith("_workspace"):
                return 256
            a = args._obj
            got = {}
            for field, kind in a._fields_:
                x = getattr(a, field)
                if kind is D.sdm_rows_t:
                    got[field] = x.data
                elif kind is ctypes.c_void_p:
                    got[field] = x
            self.launches.append(got)
            return 0
        return call


def gdr(seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.rand(*s, generator=gen)  # noqa: E731
    return dict(q=r(1, 4, 1, 8), k=r(1, 4, 1, 8), v=r(1, 4, 2, 8), g=r(1, 4, 2), beta=r(1, 4, 2))


def norm(seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.rand(*s, generator=gen)  # noqa: E731
    return dict(o=r(3, 8), z=r(3, 8), w_post=r(8), w_pre=r(8), scale=r(8))


CALLS = {
    "gdr_forward": (lambda t: D.gdr_forward(**t), gdr, ("q", "k", "v", "g", "beta")),
    "gdr_backward": (lambda t: D.gdr_backward(**t, do=t["v"]), gdr, ("q", "k", "v", "g", "beta")),
    "gdr_step": (lambda t: D.gdr_step(**t, state=torch.zeros(1, 2, 8, 8)), gdr, ("q", "k", "v", "g", "beta")),
    "norm_forward": (lambda t: D.norm_forward(t["o"], **t), norm, ("o", "z", "w_post", "w_pre", "scale")),
    "norm_backward": (lambda t: D.norm_backward(t["o"], t["o"], t["o"], **t, rstd=torch.zeros(3, 2)), norm,
                      ("o", "z", "w_post", "w_pre", "scale")),
}


@pytest.mark.parametrize("name,where", [(n, "_stream") for n in CALLS] +
                         [(n, "_workspace") for n in ("gdr_forward", "gdr_backward", "norm_backward")])
def test_a_call_entered_again_keeps_its_addresses(monkeypatch, name, where):
    call, make, names = CALLS[name]
    lib = Recorder()
    monkeypatch.setattr(D, "load", lambda: lib)
    monkeypatch.setattr(D, "_tensor", lambda t, *rest: t)
    monkeypatch.setattr(D, "_OnDevice", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(D, "_stream", lambda device: 0)
    monkeypatch.setattr(D, "_plans", D._Plans())
    one, two = make(1), make(2)
    call(one)                                   # the layout is known from here on
    real, entered = getattr(D, where), []

    def again(*args):
        if not entered:
            entered.append(True)
            call(two)
        return real(*args)

    monkeypatch.setattr(D, where, again)
    lib.launches.clear()
    call(one)
    inner, outer = lib.launches
    for n in names:
        assert inner[n] == two[n].data_ptr(), ("inner", n)
        assert outer[n] == one[n].data_ptr(), ("outer", n)
    assert not any(inner[k] == outer[k] != 0 for k in inner if inner[k] is not None)
