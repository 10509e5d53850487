"""The example's training step, run as a user runs it: its loss falls, and one
step's gradients are those that torch's autograd gives the same model."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("train_lm", os.path.join(ROOT, "examples", "train_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_loss_falls():
    m = _example()
    losses, final = m.main(steps=60, report=0)
    # The first step sees a random model: within 1 of the uniform loss.
    assert abs(losses[0] - math.log(m.VOCAB)) < 1.0
    assert final < 0.7 * losses[0] and all(math.isfinite(v) for v in losses)


def test_the_table_gradient_is_autograds():
    # The tied table's gradient (head, then embedding added into it) against
    # autograd in fp32 on the same bf16 values.  The chain rounds each of about
    # 12 intermediate results to bf16 (2^-8): 5 % of the norm is ample.
    m = _example()
    model, (tokens, targets) = m.Model(), next(m.batches())
    seen = {}
    model.adam.step = lambda grads: seen.update(table=grads[0].clone())
    bf = lambda t: t.bfloat16().float()  # noqa: E731
    table = bf(model.table).requires_grad_()
    w1, w2 = [bf(w) for w in model.w1], [bf(w) for w in model.w2]
    loss = model.step(tokens, targets, lr=0.0)
    x = table[tokens] * math.sqrt(m.DIM)
    for i in range(m.BLOCKS):
        n = torch.nn.functional.layer_norm(x, (m.DIM,))
        x = x + torch.relu(n @ w1[i].t()) @ w2[i].t()
    z = torch.nn.functional.layer_norm(x, (m.DIM,)) @ table.t()
    want = torch.nn.functional.cross_entropy(z, targets, ignore_index=m.IGNORE)
    want.backward()
    assert abs(float(loss) - want.item()) < 0.01 * want.item()
    assert float((seen["table"] - table.grad).norm()) < 0.05 * float(table.grad.norm())
