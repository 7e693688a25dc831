"""The example's gradients, parameter by parameter, against differences of its loss along each gradient.

Tolerance, set before the first run on a GPU: a difference of step 1e-2 has an error of h^2 / 6 of the third derivative,
2e-3 of the slope at the most over the parameters of two such models in the CPU runs of this file's kind, and of the
loss's own rounding over 2 h; the smallest slope is 0.017 and the loss a mean of 188 logarithms of logits that are exact
to 3e-6 of some units, 3e-6 / 188^0.5 / 1e-2 / 0.017 = 1e-3: 1e-2 together. On the CPU the operators are their 64-bit
definitions, and the comparison has to fail by ten times that where one operator's gradient is left out or turned round."""

import importlib.util
import os
import types

import pytest
import torch

from tests import delta_ref as R
from tests.delta_slopes import slope_errors

TOLERANCE = 1e-2


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_block.py")
    spec = importlib.util.spec_from_file_location("delta_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def errors(ex, device):
    torch.manual_seed(4)
    model = ex.Model(D=64, Hk=1, Hv=2, dk=32, dv=32, dtype=torch.float32).to(device)
    tokens = ex.recall(4, 12, torch.Generator().manual_seed(5))
    return slope_errors(dict(model.named_parameters()), lambda: -model(tokens)[0].double().log_softmax(-1)[:, :-1].gather(
        -1, tokens[:, 1:, None]).mean(), 1e-2)


class Scaled(torch.autograd.Function):
    """The tensors themselves, their gradients times a factor."""

    @staticmethod
    def forward(ctx, factor, *tensors):
        ctx.factor = factor
        return tuple(t.clone() for t in tensors)

    @staticmethod
    def backward(ctx, *grads):
        return (None, *(g * ctx.factor for g in grads))


@pytest.fixture
def on_cpu(monkeypatch):
    """The example on the CPU, its operators by their definitions; factors of the operators' gradients."""
    monkeypatch.setattr(torch.Tensor, "cuda", lambda t: t)
    ex = example()
    factor = types.SimpleNamespace(rule=1.0, norm=1.0)

    def gdr_forward(q, k, v, g, beta):
        q, k, v, g, beta = Scaled.apply(factor.rule, q, k, v, g, beta)
        o, s = R.gdr(q, k, v, g, beta, q.shape[-1] ** -0.5)
        return o.to(v.dtype), s.float()

    def norm_forward(x, o, z, w_post, w_pre, scale, act="silu"):
        if o is None:
            return x, R.norm(x, None, None, None, w_pre, None, act, 1e-6, x.dtype)[1].to(x.dtype), None
        o, z, w_post, scale = Scaled.apply(factor.norm, o, z, w_post, scale)
        xn, y, _, _ = R.norm(x, o, z, w_post, w_pre, scale, act, 1e-6, x.dtype)
        return xn.to(x.dtype), y.to(x.dtype), None

    monkeypatch.setattr(ex, "sdm", types.SimpleNamespace(gdr_forward=gdr_forward, norm_forward=norm_forward))
    return ex, factor


def test_right_gradients_pass(on_cpu):
    found = errors(on_cpu[0], "cpu")
    assert len(found) == 14 and max(found.values()) <= TOLERANCE, found


@pytest.mark.parametrize("which", ["rule", "norm"])
@pytest.mark.parametrize("factor", [0.0, -1.0, 0.5])
def test_wrong_gradients_show(on_cpu, which, factor):
    setattr(on_cpu[1], which, factor)
    found = errors(on_cpu[0], "cpu")
    assert max(found.values()) > 10 * TOLERANCE, found


@pytest.mark.gpu
def test_gradients():
    found = errors(example(), "cuda")
    print(found, flush=True)
    assert len(found) == 14 and max(found.values()) <= TOLERANCE, found
