"""Weight gradients on every kernel, tile, split and loop that the sizes can
choose (test_matrix_plan_host.py says which sizes reach which), with bounds
narrow enough to show the loss of an fp32 gradient's third bf16 piece.

Tolerances.  A product is exact, so only the sum's additions round: T =
tokens * pieces of them, at most 64 more where splits are joined.  Two half
steps are allowed for each.  One value is then within 2 (T + 64) half steps
of the sum of its terms' magnitudes; as the errors of single additions are
no conspiracy, and no partial sum is much larger than the largest, the whole
matrix is within 2 sqrt(T + 64) half steps in its norm."""
import numpy as np
import pytest
import torch

import matrix_ref as ref
from gpu_util import need_gpu
from test_gpu_matrix import BF16, F32, U32, run_wgrad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qc():
    return need_gpu()


# (tokens, output channels, input channels)
BF16_SIZES = [(2238, 662, 2853), (2688, 434, 2885), (387, 2803, 2999), (4097, 1021, 1030), (1728, 2063, 1728)]
F32_SIZES = [(1152, 927, 800), (320, 261, 5184), (2233, 129, 2717), (609, 2602, 3601), (300, 4, 200), (300, 5, 200),
             (77, 6, 333), (300, 7, 200)]
SIMPLE_N = {BF16: [1, 3, 7], F32: [1, 3]}
SIMPLE = [(rows, dim) for rows in (65, 200, 9000) for dim in (129, 300)]
ALL = ([(BF16, *s) for s in BF16_SIZES] + [(F32, *s) for s in F32_SIZES] +
       [(t, rows, n, dim) for t in (BF16, F32) for n in SIMPLE_N[t] for rows, dim in SIMPLE])


def gradients(rows, n, dtype):
    """fp32 values with their lowest eight bits set: what a lost third piece would take is as large as it can be."""
    dy = ref.matrix(rows, n, 1, dtype)
    return dy if dtype is BF16 else (dy.view(torch.int32) | 0xFF).view(F32)


def norm_bound(rows, dtype):
    return 2 * U32 * (rows * (3 if dtype is F32 else 1) + 64) ** 0.5


def check(got, want, mag, rows, dtype, out):
    off = np.abs(got.double().numpy() - want)
    terms = rows * (3 if dtype is F32 else 1) + 64
    half = ref.EPS[BF16] if out is BF16 else 0.0
    assert np.all(off <= 2 * U32 * terms * mag * (1 + half) + half * np.abs(want)), off.max()
    # a rounding to bf16 is at most half a step of each value
    rel = np.linalg.norm(off) / np.linalg.norm(want)
    assert rel <= norm_bound(rows, dtype) * (1 + half) + half, rel


@pytest.mark.parametrize("dtype,rows,n,dim", ALL, ids=str)
def test_every_path(qc, dtype, rows, n, dim):
    dy, x = gradients(rows, n, dtype), ref.matrix(rows, dim, 2, dtype)
    start = 8.0 * torch.randn((n, dim), generator=torch.Generator().manual_seed(9))
    got, v = run_wgrad(qc, dy, x)
    d = dy.double().numpy()
    want, mag = d.T @ v, np.abs(d).T @ np.abs(v)
    check(got, want, mag, rows, dtype, F32)
    again, _ = run_wgrad(qc, dy, x, F32, False, n + 1, 1, dim + 3, 1)  # rows that start anywhere
    assert torch.equal(got, again)
    added, _ = run_wgrad(qc, dy, x, F32, True, start=start)
    # the sums as above, then one addition
    assert torch.equal(added, start + got)
    small, _ = run_wgrad(qc, dy, x, BF16)
    assert torch.equal(small, got.to(BF16))
    check(small, want, mag, rows, dtype, BF16)


def one_token_a_channel(rows, n, low, high, seed):
    """Token j modulo rows is channel j's only one; magnitudes 2^low to 2^high, every bit of the mantissa in use."""
    g = torch.Generator().manual_seed(seed)
    bits = torch.randint(0, 1 << 23, (n,), generator=g, dtype=torch.int32) | 0xFF
    bits |= torch.randint(low + 127, high + 127, (n,), generator=g, dtype=torch.int32) << 23
    value = bits.view(F32) * torch.where(torch.rand(n, generator=g) < 0.5, -1.0, 1.0)
    at = torch.arange(n) % rows
    dy = torch.zeros((rows, n))
    dy[at, torch.arange(n)] = value
    return dy, at.numpy(), value.double().numpy()


PIECES = [(1152, 927, 800), (2233, 129, 2717), (609, 2602, 3601), (96, 40, 64), (300, 5, 200), (200, 3, 129)]


@pytest.mark.parametrize("rows,n,dim", PIECES)
def test_fp32_gradients_whole(qc, rows, n, dim):
    """One token a channel: the three pieces' products are exact, so two additions round."""
    dy, at, value = one_token_a_channel(rows, n, -8, 8, 5)
    got, v = run_wgrad(qc, dy, ref.matrix(rows, dim, 2, F32))
    want = value[:, None] * v[at]
    assert np.all(np.abs(got.double().numpy() - want) <= 4 * U32 * np.abs(want))


@pytest.mark.parametrize("rows,n,dim", PIECES)
def test_fp32_gradients_whole_when_small(qc, rows, n, dim):
    """The same where a gradient has bits below 2^-133, the smallest that bf16
    has, and the products are normal numbers: gradients from 2^-126 to 2^-100,
    and activations around 2^60."""
    dy, at, value = one_token_a_channel(rows, n, -126, -100, 6)
    got, v = run_wgrad(qc, dy, ref.matrix(rows, dim, 2, F32) * 2.0 ** 60)
    want = value[:, None] * v[at]
    off = np.abs(got.double().numpy() - want)
    assert np.all(off <= 4 * U32 * np.abs(want)), (off / np.maximum(np.abs(want), 2.0 ** -126)).max()


@pytest.mark.parametrize("rows,n,dim", PIECES)
def test_fp32_gradients_whole_beside_large_ones(qc, rows, n, dim):
    """Both kinds in a wave: sums that the bits below 2^-133 change and sums
    that they do not reach."""
    dy, at, value = one_token_a_channel(rows, n, -126, 8, 7)
    got, v = run_wgrad(qc, dy, ref.matrix(rows, dim, 2, F32) * 2.0 ** 60)
    want = value[:, None] * v[at]
    assert np.all(np.abs(got.double().numpy() - want) <= 4 * U32 * np.abs(want))


@pytest.mark.parametrize("rows,n,dim", PIECES)
def test_small_gradients_among_large_ones(qc, rows, n, dim):
    """Gradients whose last bits no sum shows; channel 1 has no others, and the
    inputs' channel 2 is zero."""
    dy, x = gradients(rows, n, F32), ref.matrix(rows, dim, 2, F32)
    dy[torch.rand((rows, n), generator=torch.Generator().manual_seed(3)) < 0.01] = 1.2345e-37
    dy[:, 1] = 1.2345e-37
    x[:, 2] = 0
    got, v = run_wgrad(qc, dy, x)
    d = dy.double().numpy()
    want, mag = d.T @ v, np.abs(d).T @ np.abs(v)
    off = np.abs(got.double().numpy() - want)
    assert np.all(off <= 2 * U32 * (3 * rows + 64) * mag), off.max()
    for rows_ in (np.arange(n) != 1, np.arange(n) == 1):
        assert np.linalg.norm(off[rows_]) <= norm_bound(rows, F32) * np.linalg.norm(want[rows_])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_no_tokens_added(qc, dtype):
    """Nothing is added: dW keeps its bits, zeros their signs and NaNs theirs."""
    n, dim = 9, 40
    values = torch.tensor([-0.0, 0.0, float("nan"), -float("inf"), 2.0 ** -149, 1.0])
    dw = values.repeat(n * dim // 6).view(n, dim).cuda()
    before = dw.clone()
    none = lambda *shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    qc.qc_ckpt8_wgrad(none(0, n, t=dtype), qc.QC_BF16 if dtype is BF16 else qc.QC_F32, n, none(0, 64, t=torch.int8),
                      none(0, 4, t=torch.uint8), 0, n, dim, dw, qc.QC_F32, dim, True)
    torch.cuda.synchronize()
    assert torch.equal(dw.view(torch.int32), before.view(torch.int32))
