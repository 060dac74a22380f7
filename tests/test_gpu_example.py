"""The training operators together, as the MLP block of examples/ uses them."""

import importlib.util
import os

import pytest
import torch

from tests.helpers import library, require_gpu

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "mlp_block.py")


def example():
    spec = importlib.util.spec_from_file_location("mlp_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,dim,hidden,block", [(2048, 512, 1024, 256), (333, 264, 520, 128)])
def test_block_gradients_match_autograd(tokens, dim, hidden, block):
    """Against float64 autograd of the same block.  An e4m3 code is within 2^-4 of its
    value, on average over a binade 2^-4 / sqrt(3) = 0.036 in the mean square; sqrt(h) has
    half of that.  An int8 code of a normal row has an error of step / sqrt(12), with a step
    of at most amax / 63.5 and amax near 2.1 to 3 in groups of 32: 0.014.  The 16-bit
    roundings of y, h, dz and dW add 2^-9 each.  The errors of different elements are
    independent, so each gradient's relative error in the Frobenius norm is at most
    sqrt(0.036^2 + 0.014^2 + ...) < 0.045."""
    require_gpu()
    dr = library()
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    net = example().MlpBlock(dim, hidden, block, generator=g)
    net.gamma = 1 + 0.2 * torch.randn(dim, device="cuda", generator=g)
    x, res, dout, drr = (torch.randn((tokens, dim), device="cuda", generator=g).bfloat16()
                         for _ in range(4))
    out, r = net.forward(x, res)
    dx, dgamma, dw1, dw2 = net.backward(dout, drr)
    leaf = [t.double().requires_grad_() for t in (r, net.gamma, net.w1.w16, net.w2.w16)]
    r64, g64, a64, b64 = leaf
    y = r64 * (r64.square().mean(1, keepdim=True) + 1e-5).rsqrt() * g64
    o64 = torch.relu(y @ a64.T).square() @ b64.T
    ((o64 * dout.double()).sum() + (r64 * drr.double()).sum()).backward()

    def rel(got, want):
        return float((got.double() - want).norm() / want.norm())

    assert rel(out, o64.detach()) < 0.01
    for got, want, what in ((dx, r64.grad, "dx"), (dgamma, g64.grad, "dgamma"),
                            (dr.unpack_blocks(dw1, hidden, dim), a64.grad, "dW1"),
                            (dr.unpack_blocks(dw2, dim, hidden), b64.grad, "dW2")):
        assert rel(got, want) < 0.045, what
    assert dr.device_status() == 0


def test_block_trains():
    require_gpu()
    library()
    losses = example().train(steps=20, tokens=2048, dim=512, hidden=1024, block=256,
                             log=lambda s: None)
    assert losses[-1] < 0.5 * losses[0], losses
