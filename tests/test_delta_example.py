"""The example's model on the GPU: it learns, its gradients hold, and answering token by token is the whole pass.

Tolerances, set before the first run: in float32 a logit is the end of some 20 products and norms of at most 256 terms,
20 * 256 * 2^-24 = 3e-4 of the largest logit."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_block.py")
    spec = importlib.util.spec_from_file_location("delta_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_tokens_one_at_a_time(ex):
    torch.manual_seed(3)
    model = ex.Model(dtype=torch.float32).cuda()
    tokens = ex.recall(5, 20, torch.Generator().manual_seed(2))
    whole, _ = model(tokens)
    for prompt in (1, 40, 79):
        got = ex.answer(model, tokens, prompt)
        off = (got - whole[:, prompt:]).abs().max()
        assert off <= 3e-4 * whole.abs().max(), (prompt, float(off))


def test_gradients_against_differences(ex):
    """Loss along a random direction of all weights; a central difference of step h has its own error of h^2 and 2^-24 / h."""
    torch.manual_seed(4)
    model = ex.Model(D=64, Hk=1, Hv=2, dk=32, dv=32, dtype=torch.float32).cuda()
    tokens = ex.recall(4, 12, torch.Generator().manual_seed(5))
    loss_of = lambda: model(tokens)[0].double().log_softmax(-1)[:, :-1].gather(  # noqa: E731
        -1, tokens[:, 1:, None]).mean().neg()
    loss = loss_of()
    loss.backward()
    params = list(model.parameters())
    way = [torch.randn_like(p) for p in params]
    size = sum(float((w.double() ** 2).sum()) for w in way) ** 0.5
    slope = sum(float((p.grad.double() * w.double()).sum()) for p, w in zip(params, way)) / size
    norm = sum(float((p.grad.double() ** 2).sum()) for p in params) ** 0.5
    h = 1e-2
    ends = []
    with torch.no_grad():
        for s in (1, -1):
            for p, w in zip(params, way):
                p.add_(w, alpha=s * h / size)
            ends.append(float(loss_of()))
            for p, w in zip(params, way):
                p.add_(w, alpha=-s * h / size)
    assert abs((ends[0] - ends[1]) / (2 * h) - slope) <= 1e-2 * norm


@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_it_learns(ex, ty):
    """64 tokens, half of them values: guessing among the values costs ln 32 = 3.5, untrained weights more."""
    torch.manual_seed(0)
    model = ex.Model(dtype=ex.TYPES[ty]).cuda()
    losses = ex.train(model, 100)
    print("losses", losses[::20], flush=True)
    assert sum(losses[-5:]) / 5 < 3.0 < losses[0]
