"""The example's training step: its gradients against 64-bit automatic
differentiation of the same model, and that it learns its task.

The step rounds to bf16 at some eight places between a weight and its
gradient (lookup, products, SwiGLU, combine, logits, their gradients and the
sums of paths); each moves a value by at most 2^-9 of it on average, so the
relative 2-norm of each gradient's error is within 8 * 2^-9 = 2^-6."""

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from nvfp4_mixture_experts_counting_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_against_autograd(example):
    from nvfp4_mixture_experts_counting_gb300 import ftmoe
    m = example.Model(V=48, H=128, E=8, k=3, I=64, T=100, bits=32, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    ids = torch.randint(0, m.V, (m.T,), generator=g, device="cuda")
    target = torch.randint(0, m.V, (m.T,), generator=g, device="cuda")
    adv = torch.randn(m.T, generator=g, device="cuda")
    logits = m.forward(ids)
    lp = torch.log_softmax(logits.float(), 1).gather(1, target[:, None])[:, 0]
    old, ref = lp + 0.05, lp - 0.1  # every ratio is 0.951, inside the clip's bounds
    ftmoe.ftmoe_policy_loss(ftmoe.policy_args(logits, target, old, ref, adv, None, m.loss, m.row_loss, m.logp, m.dlogits,
                                              kl_coef=0.5))
    m.backward(ids)
    w = {n: v.double().requires_grad_() for n, v in m.p.items()}
    x = w["table"][ids] * math.sqrt(m.H)
    chosen = torch.softmax((x @ w["router"].t()).gather(1, m.idx.long()), 1)
    y = torch.zeros_like(x)
    for j in range(m.k):
        e = m.idx[:, j].long()
        gate, up = torch.einsum("th,thi->ti", x, w["gate_up"][e]).chunk(2, 1)
        y = y + chosen[:, j:j + 1] * torch.einsum("ti,tih->th", torch.nn.functional.silu(gate) * up, w["down"][e])
    logp = torch.log_softmax((x + y) @ w["out"], 1).gather(1, target[:, None])[:, 0]
    d = ref.double() - logp
    loss = (-torch.exp(logp - old.double()) * adv.double() + 0.5 * (torch.exp(d) - d - 1)).mean()
    loss.backward()
    loss = loss.detach()
    assert abs(float(m.loss) - float(loss)) <= 2.0 ** -6 * (abs(float(loss)) + float(adv.abs().mean()))
    for n in m.p:
        a, b = m.grad[n].double(), w[n].grad
        assert float((a - b).norm() / b.norm()) <= 2.0 ** -6, n


@pytest.mark.parametrize("bits", [8, 32])
def test_the_step_learns(example, bits):
    """From one choice in 64 at random to most of them right."""
    m = example.Model(bits=bits)
    first = float(m.step(1))
    last = [float(m.step(t)) for t in range(2, 151)][-10:]
    assert first < 0.1 and sum(last) / 10 > 0.5
    from nvfp4_mixture_experts_counting_gb300 import ftmoe
    assert ftmoe.ftmoe_ops_status() == 0
