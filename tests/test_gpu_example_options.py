"""The gated MLP example with MXFP4 products and with AdamW: that it runs, its
gradients against fp32 ones of the same step, and its weights after a step
against the 64-bit formula."""
import numpy as np
import pytest
import torch

import mx_ref as ref
from test_gpu_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,width,hidden", [(300, 128, 192), (77, 65, 50)])
def test_one_step_on_mxfp4_products(example, tokens, width, hidden):  # noqa: F811
    """A code is off by at most a quarter of its value (half a step at the
    bottom of a power of two), or of the group's 2^E below 2^E: as an rms of a
    uniform error 14 % of the value and less.  A product has two such operands
    (20 %).  The outputs are at the end of two products with silu * up, both of
    whose factors are products, between them: sqrt(20^2 + 20^2 + 20^2) = 35 %; a
    gradient adds two more, and silu' may double what reaches it."""
    m = example.GatedMlp8(tokens, width, hidden, torch.device("cuda"), seed=3, products="mxfp4")
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
    for got, r, bound in ((y, want.detach(), 0.35), (dx, xr.grad, 0.6), (m.dw_in.cpu(), w_in.grad, 0.6),
                          (m.dw_out.cpu(), w_out.grad, 0.35)):
        rel = ((got - r).norm() / r.norm()).item()
        assert rel < bound, rel


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_of_adamw(example, bits):  # noqa: F811
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(7)
    w = [torch.randn(s, generator=g) for s in ((60, 33), (33, 30))]
    weights, grads = [t.to(dev) for t in w], [torch.randn(t.shape, generator=g).to(dev) for t in w]
    adam = example.AdamW(weights, grads, 0.01, bits)
    p = np.concatenate([t.double().numpy().ravel() for t in w])
    dw = np.concatenate([t.double().cpu().numpy().ravel() for t in grads])
    norm = np.sqrt((dw ** 2).sum())
    adam.step()
    want, _, _, upd = ref.adamw(p, dw, 0.0 * p, 0.0 * p, 0.01, 0.9, 0.99, 1e-8, 0.01, 1, scale=1.0 / norm)
    got = torch.cat([t.view(-1) for t in weights]).double().cpu().numpy()
    assert abs(float(adam.norm[0]) / norm - 1) < 2 * ref.U32
    assert (np.abs(got - want) <= ref.U32 * (4 * np.abs(p) + 20 * upd)).all()


@pytest.mark.parametrize("products,optimizer", [("mxfp4", "adamw8"), ("mxfp4", "sgd"), ("int8", "adamw")])
def test_it_runs(example, products, optimizer):  # noqa: F811
    losses = example.train(tokens=256, width=64, hidden=96, steps=6, lr=0.1 if optimizer == "sgd" else 0.002,
                           products=products, optimizer=optimizer, log=lambda *_: None)
    assert len(losses) == 6 and np.isfinite(losses).all()
