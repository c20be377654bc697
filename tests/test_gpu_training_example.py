"""The example that runs the training-side operators and the loss-scaled step together:
its gradients against automatic differentiation in fp32, and its loss."""
from __future__ import annotations

import pytest
import torch

from examples import train_blocks

pytestmark = pytest.mark.gpu


def _reference_loss(model, params, inputs, targets):
    """The example's model in plain fp32."""
    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + model.eps) * w

    def last(i):
        return "w_last" if i == model.blocks else f"w_pre{i}"

    h = params["embed"][inputs]
    for i in range(model.blocks):
        a = torch.relu(norm(h, params[last(i)]) @ params[f"w1_{i}"].t()).square()
        y = a @ params[f"w2_{i}"].t()
        h = h + params[f"gate{i}"] * norm(y, params[f"w_post{i}"])
    logits = norm(h, params["w_last"]) @ params["embed"].t()
    return -torch.log_softmax(logits, 1).gather(1, targets[:, None]).mean()


def test_gradients_follow_automatic_differentiation():
    """Every parameter's gradient within 5 % (norm of the difference): the 8-bit checkpoints
    are off by up to 1 % rms (half a step of 1/64 to 1/128 of a block's largest value) and
    each bf16 product by 0.2 %, over a handful of layers."""
    model = train_blocks.BlockStack(vocab=1000, width=192, inner=320, blocks=3)
    g = torch.Generator(device="cuda").manual_seed(3)
    inputs, targets = train_blocks.batch(model, 700, g)
    kept = model.forward(inputs, targets)
    loss = -kept["logprob"].mean()
    grad = model.grads[0]
    model.backward(kept, grad)
    train_blocks.dp.stream_status()
    scale = train_blocks.dp.read_loss_scale(model.scale_state).scale
    params = {n: model.p(n).float().requires_grad_() for n in model.where}
    want = _reference_loss(model, params, inputs, targets)
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) <= 0.02 * want
    for n, p in params.items():
        got = model.view(grad, n).float() / scale
        ref = p.grad.reshape(got.shape)
        err = float((got - ref).norm() / ref.norm())
        assert err <= 0.05, (n, err)


def test_example_trains(capsys):
    losses = train_blocks.main(["--steps", "40", "--tokens", "512"])
    assert losses[-1] < 0.6 * losses[0]
    assert "skipped 0" in capsys.readouterr().out


def test_an_overflow_in_a_checkpoint_skips_the_step():
    """A non-finite activation reaches the gradients through its packed block and the
    loss-scaled step leaves the parameters alone."""
    model = train_blocks.BlockStack(vocab=256, width=128, inner=128, blocks=1)
    g = torch.Generator(device="cuda").manual_seed(3)
    for r, grad in enumerate(model.grads):
        kept = model.forward(*train_blocks.batch(model, 100, g))
        if r == 0:
            kept["blocks"][0]["a8"][1][7, 2] = 255  # as packing an Inf leaves it
        model.backward(kept, grad)
    before = model.master.clone()
    model.update()
    train_blocks.dp.stream_status()
    state = train_blocks.dp.read_loss_scale(model.scale_state)
    assert state.skipped == 1 and state.step == 0
    assert torch.equal(model.master, before)
