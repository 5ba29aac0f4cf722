"""The gated MLP example: its gradients against fp32 ones of the same step,
and a short training run."""
import importlib.util
import os

import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_mlp_8bit.py")


@pytest.fixture(scope="module")
def example():
    need_gpu()
    spec = importlib.util.spec_from_file_location("gated_mlp_8bit", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,width,hidden", [(300, 128, 192), (77, 65, 50)])
def test_one_step(example, tokens, width, hidden):
    """A code is off by at most half a step, a 254th of its row's largest
    value: for normal rows (largest value about 3.5 standard deviations)
    0.4 % of a standard deviation, as an rms of a uniform error.  Each product
    has two such operands (0.6 %), its bf16 result 0.2 %; a gradient is at the
    end of a chain of four products and a checkpoint or two, and silu' may
    double what reaches it: below 5 %."""
    m = example.GatedMlp8(tokens, width, hidden, torch.device("cuda"), seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((tokens, width), generator=g, device="cuda").to(torch.bfloat16)
    dy = (torch.randn((tokens, width), generator=g, device="cuda") / tokens).to(torch.bfloat16)
    y = m.forward(x).float().cpu()
    dx = m.backward(dy).float().cpu()
    xr = x.float().cpu().requires_grad_()
    w_in, w_out = m.w_in.cpu().clone().requires_grad_(), m.w_out.cpu().clone().requires_grad_()
    gu = xr @ w_in.t()
    want = (torch.nn.functional.silu(gu[:, :hidden]) * gu[:, hidden:]) @ w_out.t()
    want.backward(dy.float().cpu())
    for got, ref in ((y, want.detach()), (dx, xr.grad), (m.dw_in.cpu(), w_in.grad), (m.dw_out.cpu(), w_out.grad)):
        rel = ((got - ref).norm() / ref.norm()).item()
        assert rel < 0.05, rel


def test_training_reduces_the_loss(example):
    losses = example.train(tokens=512, width=64, hidden=96, steps=25, log=lambda *_: None)
    assert losses[-1] < 0.8 * losses[0]
