"""The MXFP4 product on the GPU at sizes that reach every tile shape, with and
without splits of k, rows of scales that end inside a piece, and whole stages
taken by the loop for them; against a 64-bit product of what the codes stand
for.  Tolerances are those of test_gpu_mxfp4.py."""
import numpy as np
import pytest
import torch

import mx_ref as ref
from gpu_util import need_gpu
from test_gpu_matrix import BF16, F32, Buf, qt
from test_gpu_mxfp4 import EPS, Held, space

pytestmark = pytest.mark.gpu

# (m, n, k): the shapes and parts that they reach are checked on the host
SIZES = [
    (128, 4090, 2100), (33, 4100, 515),
    (100, 4549, 1395), (250, 4090, 4649), (130, 120, 30050), (700, 900, 20001),
    (1003, 1530, 2043), (500, 4090, 4100), (2083, 40, 42219),
    (1000, 4001, 6100), (1010, 4050, 4219), (1052, 69, 55680), (500, 520, 65302),
    (2100, 2050, 5000), (2040, 4090, 3225), (4330, 41, 38264),
    (4090, 4090, 4111), (4096, 4096, 4224), (4000, 3900, 1500), (130, 2938, 65302),
    (257, 255, 512), (300, 520, 1030), (1024, 70, 300), (300, 8847, 385), (162, 19082, 993),
    # blocks that go on to a second and a third tile
    (4300, 4353, 300), (2100, 8500, 3001), (5000, 8200, 33), (8150, 4090, 1500), (4095, 8190, 4000),
    # the longest rows
    (20, 40, 1 << 23), (257, 300, (1 << 22) + 5),
]


@pytest.fixture(scope="module")
def qc():
    return need_gpu()


def values(held, dim):
    """What codes and scales on the GPU stand for, in 64 bits."""
    rows = held.rows
    codes, scales = held.codes.view(rows, -1), held.scales.view(rows, -1)
    table = torch.from_numpy(np.concatenate([ref.VALUES, -ref.VALUES])).cuda()
    wide = torch.stack([codes & 15, codes >> 4], 2).view(rows, -1)
    step = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), scales.int() - 127)
    return (table[wide.int()] * step.repeat_interleave(32, 1)[:, : wide.shape[1]])[:, :dim].contiguous()


def random_held(qc, rows, dim, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = Held(qc, rows, dim)
    codes = torch.randint(0, 256, (rows, h.codes.numel() // rows), generator=g, device="cuda", dtype=torch.uint8)
    if dim % 2:
        codes[:, dim // 2] &= 15
    codes[:, (dim + 1) // 2:] = 0
    scales = torch.randint(110, 136, (rows, h.scales.numel() // rows), generator=g, device="cuda", dtype=torch.uint8)
    scales[:, -(-dim // 32):] = 0
    h.codes.copy_(codes.view(-1))
    h.scales.copy_(scales.view(-1))
    return h


@pytest.mark.parametrize("ctype", [BF16, F32, "added"], ids=str)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(qc, m, n, k, ctype):
    a, b = random_held(qc, m, k, 1), random_held(qc, n, k, 2)
    dtype = BF16 if ctype is BF16 else F32
    ldc = n + 3
    c = Buf(m, n, ldc, dtype, skip=1)
    if ctype == "added":
        c.t[:, :n] = torch.randn((m, n), device="cuda") * 100.0
    c0 = c.t[:, :n].double() if ctype == "added" else 0.0
    w = space(qc.qc_matmul_mxfp4_workspace(m, n, k))
    qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), m, n, k, c.t, qt(qc, dtype), ldc, ctype == "added", w)
    got = c.t[:, :n].double()
    av, bv = values(a, k), values(b, k)
    want = torch.matmul(av, bv.t().contiguous())
    size = torch.matmul(av.abs(), bv.abs().t().contiguous())
    if ctype == "added":
        want, size = want + c0, size + c0.abs()
    tol = size * (k + 2) * 2.0 ** -24 + want.abs() * EPS[dtype]
    # the bound of k additions is wide; their roundings are independent, and the mean error far below it
    assert bool(((got - want).abs() <= tol).all())
    rms = float(((got - want).square().mean() / size.square().mean()).sqrt())
    assert rms <= (k ** 0.5 + 2) * 2.0 ** -24 + EPS[dtype], rms
    c.check()
