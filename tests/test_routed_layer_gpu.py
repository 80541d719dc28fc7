"""The routed-layer example: its gradients against autograd through plain
products in 64 bits, its training loss, and its captured serving step."""
import pytest
import torch

from examples import routed_layer

pytestmark = pytest.mark.gpu


def test_gradients_match_autograd_in_64_bits():
    gen = torch.Generator(device="cuda").manual_seed(3)
    tokens, fan, experts, width, out = 150, 2, 5, 72, 136
    x = (torch.randint(-8, 9, (tokens, width), generator=gen, device="cuda") / 8.0).half()
    w = (torch.randint(-8, 9, (experts, out, width), generator=gen, device="cuda") / 8.0).half()
    ids = torch.randint(-1, experts, (tokens, fan), generator=gen, device="cuda").to(torch.int32)
    gates = torch.randint(1, 5, (tokens, fan), generator=gen, device="cuda") / 4.0
    up = torch.randint(-8, 9, (tokens, out), generator=gen, device="cuda") / 8.0
    a = [t.clone().requires_grad_() for t in (x, w)] + [gates.clone().requires_grad_()]
    y = routed_layer.RoutedLinear.apply(a[0], a[1], ids, a[2])
    y.backward(up)
    b = [t.double().cpu().requires_grad_() for t in (x, w, gates)]
    z = torch.zeros(tokens, out, dtype=torch.float64)
    for t in range(tokens):
        for f in range(fan):
            if ids[t, f] >= 0:
                z[t] = z[t] + b[2][t, f] * (b[1][int(ids[t, f])] @ b[0][t])
    z.backward(up.double().cpu())
    # multiples of 1/2048 at most, exact sums: the gradients' one rounding to fp16 is all
    assert torch.equal(y.double().cpu(), z)
    assert torch.equal(a[0].grad.cpu(), b[0].grad.half())
    assert torch.equal(a[1].grad.cpu(), b[1].grad.half())
    assert torch.equal(a[2].grad.double().cpu(), b[2].grad)


def test_training_loss_falls():
    losses = routed_layer.train(tokens=512, width=128, out=128, steps=4)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_serving_step_replays():
    for got, want in zip(*routed_layer.serve()):
        # y ~ N(0, 2): half a step of fp16 below 8 is 2^-9; the fp32 sums' own error is far below
        assert float((got.float() - want).abs().max()) <= 2.0**-8
