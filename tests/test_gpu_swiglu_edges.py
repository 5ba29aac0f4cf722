"""The gated activation where its sigmoid is tiny and where its inputs are
infinities and NaNs.

Tolerances, in half steps of fp32 (the sigmoid s = 1 / (1 + exp(-x))): exp
within 4, its sum with one 1, the reciprocal 1, the product of the two 1: s
and 1 - s within 7 each; h = g s u takes two more products, dU two, dG four
products and one sum: 9, 9 and 12 + 10 |G| half steps.  Below 2^-126 the
sigmoid is a subnormal number, off by half of 2^-149, or by the rounding of
exp and of its product with the reciprocal both: 2^-149 |g u| in h, 2^-149
|dh G| in dU, 2^-149 |dh U| (1 + |G|) in dG."""
import numpy as np
import pytest
import torch

import matrix_ref as ref
from gpu_util import need_gpu
from test_gpu_matrix import BF16, DTYPES, F32, U32, run_swiglu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qc():
    return need_gpu()


def near(got, want, half_steps, floor, dtype):
    off = np.abs(got.double().numpy() - want)
    eps = ref.EPS[dtype]
    # a result below the smallest normal number of its type has steps of their own
    tiny = 2.0 ** -134 if dtype is BF16 else 2.0 ** -150
    bound = (U32 * half_steps * np.abs(want) + floor) * (1 + eps) + (eps * np.abs(want) if dtype is BF16 else 0) + tiny
    assert np.all(off <= bound), (off - bound).max()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("scale", [0, 60, 100])
def test_tiny_sigmoid(qc, scale, dtype):
    """Gates from -80 down to -110: what the other factor makes of a sigmoid around 2^-126 is a normal number."""
    rows, dim = 40, 96
    g = -(80 + 30 * torch.rand((rows, dim), generator=torch.Generator().manual_seed(1))).to(dtype)
    u, dh = (ref.matrix(rows, dim, s, F32, 0.1).mul(2.0 ** scale).to(dtype) for s in (2, 3))
    _, _, h, dg, du = run_swiglu(qc, g, u, dh, 2 * dim, 0)
    gd, ud, dd = g.double().numpy(), u.double().numpy(), dh.double().numpy()
    near(h, gd * ref.sigmoid(gd) * ud, 9, 2.0 ** -149 * np.abs(gd * ud), dtype)
    G, U = ref.held(*ref.ckpt8(g), dim), ref.held(*ref.ckpt8(u), dim)
    s = ref.sigmoid(G)
    near(du, dd * G * s, 9, 2.0 ** -149 * np.abs(dd * G) + 2.0 ** -150 * np.abs(G), dtype)
    factor = 1 + G * (1 - s)
    off = U32 * (12 + 10 * np.abs(G)) * np.abs(dd * U * s)
    floor = (2.0 ** -149 * np.abs(dd * U) + 2.0 ** -150 * np.abs(U)) * (1 + np.abs(G))
    near(dg, dd * U * s * factor, 0, off + floor, dtype)


def run(qc, g, u, dh):
    _, _, h, dg, du = run_swiglu(qc, g, u, dh, 2 * g.shape[1], 0)
    return h, dg, du


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("where", ["gate", "up", "dh"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")], ids=str)
def test_infinities_and_nans(qc, value, where, dtype):
    """An infinity or a NaN shows in the result of its own place, and, where
    it was kept, in the gradients that read its group; everything else has
    the bits that it has without it."""
    rows, dim, at = 5, 200, (2, 70)
    g, u, dh = (ref.matrix(rows, dim, s, dtype) for s in (1, 2, 3))
    for x in (g, u, dh):
        x[at] = 1.5
    clean = run(qc, g, u, dh)
    {"gate": g, "up": u, "dh": dh}[where][at] = value
    got = run(qc, g, u, dh)
    group = torch.zeros((rows, dim), dtype=torch.bool)
    group[2, 64:96] = True
    own = torch.zeros_like(group)
    own[at] = True
    none = torch.zeros_like(group)
    # which places of h, dG and dU are reached
    reached = {"gate": (own, group, group), "up": (own, group, none), "dh": (none, own, own)}[where]
    for name, c, r, spot in zip(("h", "dgate", "dup"), clean, got, reached):
        assert torch.equal(r[~spot], c[~spot]), name
        assert bool(torch.isfinite(c).all()) and not bool(torch.isfinite(r[spot]).any()), name
    h, dg, du = (float(t[at]) for t in got)
    if where in ("gate", "up"):
        # silu(-inf) = -inf / (1 + exp(inf)) has no value
        assert h == value if np.isposinf(value) or (where == "up" and np.isinf(value)) else np.isnan(h)
        assert np.isnan(dg)
    elif np.isinf(value):  # dG and dU are dh times positive numbers: G = U = 1.5, nearly
        assert dg == value and du == value
    else:
        assert np.isnan(dg) and np.isnan(du)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_largest_gates(qc, dtype):
    """Finite gates as large as their type holds: silu(g) is g or 0, and no NaN appears."""
    big = torch.finfo(dtype).max
    g = torch.tensor([[big, -big, big / 2, -big / 2, 200.0, -200.0, 0.0, -0.0]]).to(dtype)
    u, dh = torch.full_like(g, 0.5), torch.full_like(g, 0.25)
    h, dg, du = run(qc, g, u, dh)
    gd = g.double().numpy()
    want = np.where(gd > 0, gd * 0.5, 0.0)
    assert np.array_equal(h.double().numpy(), want)
    assert bool(torch.isfinite(dg).all()) and bool(torch.isfinite(du).all())
