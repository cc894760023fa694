"""The example's training step: gradients against FP64 autograd, a falling loss, and decoding."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("expert_lm_step",
                                                  os.path.join(ROOT, "examples", "expert_lm_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_against_autograd(cuda_device):
    """The whole step's gradients against FP64 autograd of the same BF16 weights, the choice of
    experts given.  A gradient passes through up to eight BF16 roundings of 2^-8 each on its
    way (activations, upstream gradients, weights' gradients): 2-norms within 8 * 2^-8."""
    m = example()
    model = m.Model(seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    tokens = torch.randint(0, 1003, (700,), generator=g, device="cuda")
    targets = torch.randint(0, 1003, (700,), generator=g, device="cuda")
    targets[::9] = -100
    loss, grads = model.loss_and_gradients(tokens, targets)
    choice = model.forward(tokens)["choice"]
    w = {k: v.double().requires_grad_(True) for k, v in model.w.items()}
    x0 = w["embed"][tokens]
    x1 = torch.nn.functional.gelu(x0 @ w["w1"].t() + w["b1"]) @ w["w2"].t() + w["b2"] + x0
    p = torch.softmax(x1 @ w["router"].t(), 1)
    rows = []
    for r in range(700):
        e = choice[r]
        a = torch.nn.functional.silu(x1[r] @ w["e1"][e].t() + w["c1"][e]) @ w["e2"][e].t()
        rows.append(x1[r] + p[r, e] * a)
    want = torch.nn.functional.cross_entropy(torch.stack(rows) @ w["head"].t(), targets)
    want.backward()
    assert abs(float(loss) - float(want)) <= 8 * 2.0 ** -8 * float(want)
    for name, v in w.items():
        off = float((grads[name].double() - v.grad).norm() / v.grad.norm())
        assert off <= 8 * 2.0 ** -8, (name, off)


def test_loss_falls_and_decoding_follows(cuda_device):
    losses, right = example().train(steps=60)
    assert losses[0] > 6.0                    # log(1003) = 6.9 at the start
    assert losses[-1] < 0.5 * losses[0]
    assert right >= 0.5
