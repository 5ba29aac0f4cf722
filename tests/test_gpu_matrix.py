"""The matrix operators on the GPU against their plain 64-bit forms
(matrix_ref.py): INT8 rows and their product, 8-bit checkpoints, the weight
gradient taken from them, the gated activation.

Tolerances: codes, scales, exponents and restored values are equal.  The
product rounds its exact sum to fp32 and once per scale: three half steps of
fp32, and one of the output's type.  A weight gradient's products are exact;
its fp32 sum of T terms is within T half steps (two allowed for each
addition) of the sum of their magnitudes.  The gated activation's bounds are
stated at its test."""
import numpy as np
import pytest
import torch

import matrix_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = [BF16, F32]
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def qc():
    return need_gpu()


def qt(qc, dtype):
    return qc.QC_BF16 if dtype is BF16 else qc.QC_F32


class Buf:
    """A [rows][ld] buffer of which [rows][cols] is an output, between guards;
    check() asserts that nothing outside was written."""

    def __init__(self, rows, cols, ld, dtype, skip=0):
        self.rows, self.cols, self.ld, self.skip = rows, cols, ld, skip
        self.es = torch.empty((), dtype=dtype).element_size()
        n = (skip + rows * ld + 64) * self.es
        self.raw = torch.full((n,), 0x5C, dtype=torch.uint8, device="cuda")
        self.flat = self.raw.view(dtype)
        self.t = self.flat[skip: skip + rows * ld].view(rows, ld)

    def get(self):
        return self.t[:, : self.cols].cpu()

    def check(self):
        keep = torch.ones(self.raw.numel() // self.es, dtype=torch.bool)
        keep[self.skip: self.skip + self.rows * self.ld].view(self.rows, self.ld)[:, : self.cols] = False
        b = self.raw.cpu().view(-1, self.es)
        assert bool((b[keep] == 0x5C).all()), "a write outside the output"


def strided(x, ld, skip=0):
    """x on the GPU inside a wider matrix, NaN everywhere else (random bytes for codes)."""
    rows, cols = x.shape
    flat = torch.empty(skip + rows * ld, dtype=x.dtype, device="cuda")
    if x.dtype.is_floating_point:
        flat.fill_(float("nan"))
    else:
        flat.random_(-128, 128)
    t = flat[skip:].view(rows, ld)
    t[:, :cols] = x.cuda()
    return t


def same(got, want):
    return np.array_equal(got, want, equal_nan=got.dtype.kind == "f")


# ------------------------------------------------------------- INT8 rows


DIMS = [1, 2, 7, 8, 9, 15, 16, 17, 127, 512, 513, 1024, 1025, 2048, 2049, 4099, 8192, 8200, 16384, 16400, 20001]


def encode_int8(qc, x, ldx, ldq, skip=0):
    rows, dim = x.shape
    q = Buf(rows, ref.up(dim, 16), ldq, torch.int8)
    s = Buf(1, rows, rows, F32)
    qc.qc_encode_int8_rowwise(strided(x, ldx, skip), qt(qc, x.dtype), rows, dim, ldx, q.t, ldq, s.t)
    torch.cuda.synchronize()
    q.check()
    s.check()
    return q.get().numpy(), s.get().numpy()[0]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("dim", DIMS)
def test_int8_rows(qc, dim, dtype):
    x = ref.matrix(7, dim, dim, dtype)
    q, s = encode_int8(qc, x, dim, ref.up(dim, 16))
    wq, ws = ref.int8_rows(x)
    assert same(s, ws)
    assert np.array_equal(q[:, :dim], wq) and not q[:, dim:].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,dim,ldx,ldq,skip", [(5, 100, 131, 128, 1), (33, 1000, 1003, 1024, 3), (1, 40, 64, 48, 0),
                                                    (130, 8, 9, 32, 5), (9, 4097, 4099, 4128, 1)])
def test_int8_rows_strides(qc, rows, dim, ldx, ldq, skip, dtype):
    x = ref.matrix(rows, dim, 3, dtype)
    q, s = encode_int8(qc, x, ldx, ldq, skip)
    wq, ws = ref.int8_rows(x)
    assert same(s, ws) and np.array_equal(q[:, :dim], wq) and not q[:, dim:].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("dim", [96, 300, 700, 5000, 17000])
def test_int8_rows_hard(qc, dim, dtype):
    x = ref.hard_rows(dim, dtype)
    q, s = encode_int8(qc, x, dim, ref.up(dim, 16))
    wq, ws = ref.int8_rows(x)
    assert same(s, ws) and np.array_equal(q[:, :dim], wq)


def test_int8_rows_near_borders(qc):
    """Values within a few steps of the middle between two codes."""
    g = torch.Generator().manual_seed(5)
    rows, dim = 64, 1500
    amax = torch.exp(8 * torch.randn((rows, 1), generator=g)).float()
    s = (amax.double() / 127).float().double()
    c = torch.randint(-126, 126, (rows, dim), generator=g).double() + 0.5
    x = (c * s).float()
    step = torch.randint(-3, 4, (rows, dim), generator=g)
    x = (x.view(torch.int32) + step.int()).view(torch.float32)
    x[:, 7:8] = amax
    q, sc = encode_int8(qc, x, dim, ref.up(dim, 16))
    wq, ws = ref.int8_rows(x)
    assert same(sc, ws) and np.array_equal(q[:, :dim], wq)


# --------------------------------------------------------------- product


def codes_of(rows, k, seed, lo=-127):
    return torch.randint(lo, 128, (rows, k), generator=torch.Generator().manual_seed(seed), dtype=torch.int8)


def run_matmul(qc, a, sa, b, sb, dtype, lda=None, ldb=None, ldc=None, skip=0):
    (m, k), n = a.shape, b.shape[0]
    kp = ref.up(k, 16)
    lda, ldb, ldc = lda or kp, ldb or kp, ldc or n
    c = Buf(m, n, ldc, dtype, skip)
    qc.qc_matmul_int8(strided(a, lda), sa.cuda(), lda, strided(b, ldb), sb.cuda(), ldb, m, n, k, c.t, qt(qc, dtype), ldc)
    torch.cuda.synchronize()
    c.check()
    return c.get().double().numpy()


def check_product(got, a, sa, b, sb, dtype):
    want = ref.matmul(a.numpy(), sa.numpy(), b.numpy(), sb.numpy())
    tol = (1 + ref.EPS[BF16] if dtype is BF16 else 1) * (1 + U32) ** 3 - 1
    off = np.abs(got - want)
    assert np.all(off <= tol * np.abs(want) + 2.0 ** -133), off.max()


MNK = [(1, 16, 16), (1, 1, 1), (1, 17, 15), (1, 300, 4096), (3, 33, 127), (15, 64, 128), (16, 65, 129), (17, 31, 1000),
       (31, 128, 257), (32, 40, 2043), (33, 257, 640), (61, 100, 2048), (64, 64, 64), (65, 70, 130), (100, 130, 100),
       (127, 255, 383), (129, 64, 512), (300, 500, 200), (257, 1000, 1040), (1003, 153, 204)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,n,k", MNK)
def test_matmul(qc, m, n, k, dtype):
    a, b = codes_of(m, k, m), codes_of(n, k, n + 1)
    sa = torch.rand(m, generator=torch.Generator().manual_seed(1)) * 1e-2 + 1e-4
    sb = torch.rand(n, generator=torch.Generator().manual_seed(2)) * 1e-3 + 1e-5
    check_product(run_matmul(qc, a, sa, b, sb, dtype), a, sa, b, sb, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,n,k", [(3700, 3400, 150), (2000, 1900, 333), (1030, 3000, 131)])
def test_matmul_large_tiles(qc, m, n, k, dtype):
    """Enough tiles for the larger tile shapes, none of them full at the edges."""
    a, b = codes_of(m, k, 11), codes_of(n, k, 12)
    sa, sb = torch.full((m,), 0.25), torch.full((n,), 2.0 ** -9)
    c = Buf(m, n, n, dtype)
    kp = ref.up(k, 16)
    qc.qc_matmul_int8(strided(a, kp), sa.cuda(), kp, strided(b, kp), sb.cuda(), kp, m, n, k, c.t, qt(qc, dtype), n)
    torch.cuda.synchronize()
    c.check()
    # power-of-two scales and sums below 2^24: fp32 is exact, bf16 rounds once
    want = (torch.from_numpy(a.numpy().astype(np.float32) @ b.numpy().astype(np.float32).T) * 2.0 ** -11).to(dtype)
    assert torch.equal(c.get(), want)


@pytest.mark.parametrize("m,n,k", [(3700, 3400, 1500), (2000, 1900, 1024), (1500, 2100, 641), (3584, 3840, 448),
                                   (9, 5000, 1333), (30, 4001, 2700), (60, 3900, 1100), (120, 4002, 2900),
                                   (250, 3907, 1300), (500, 4000, 1601), (1000, 4003, 1700), (2000, 4000, 1111),
                                   (256, 4096, 512), (250, 4000, 513), (512, 4096, 1024), (500, 4090, 385),
                                   (1024, 4096, 1152), (1020, 4000, 640), (2048, 4096, 768), (2010, 3900, 897)])
def test_matmul_large_tiles_long_k(qc, m, n, k):
    """The same over enough k for the steady state of the pipeline; codes small
    enough that every sum is below 2^24 and fp32 on the host exact."""
    a, b = codes_of(m, k, 21) // 2, codes_of(n, k, 22) // 2
    c = Buf(m, n, n, BF16)
    kp = ref.up(k, 16)
    sa, sb = torch.full((m,), 0.5), torch.full((n,), 2.0 ** -7)
    qc.qc_matmul_int8(strided(a, kp), sa.cuda(), kp, strided(b, kp), sb.cuda(), kp, m, n, k, c.t, qc.QC_BF16, n)
    torch.cuda.synchronize()
    c.check()
    want = (torch.from_numpy(a.numpy().astype(np.float32) @ b.numpy().astype(np.float32).T) * 2.0 ** -8).to(BF16)
    assert torch.equal(c.get(), want)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("more,skip", [(0, 0), (8, 0), (4, 0), (3, 0), (8, 2)])
@pytest.mark.parametrize("m,n,k", [(250, 4000, 200), (500, 4000, 300), (1000, 4000, 260), (2000, 4000, 130),
                                   (3700, 3400, 70)])
def test_matmul_tile_stores(qc, m, n, k, more, skip, dtype):
    """Whole tiles of C at every alignment of its rows, each row and column
    with a scale of its own (powers of two, so fp32 is exact)."""
    a, b = codes_of(m, k, 31), codes_of(n, k, 32)
    sa = torch.exp2((torch.arange(m) % 7).float())
    sb = torch.exp2(-(torch.arange(n) % 11).float())
    c = Buf(m, n, n + more, dtype, skip)
    kp = ref.up(k, 16)
    qc.qc_matmul_int8(strided(a, kp), sa.cuda(), kp, strided(b, kp), sb.cuda(), kp, m, n, k, c.t, qt(qc, dtype), n + more)
    torch.cuda.synchronize()
    c.check()
    sums = torch.from_numpy(a.numpy().astype(np.float32) @ b.numpy().astype(np.float32).T)
    assert torch.equal(c.get(), ((sums * sa[:, None]) * sb[None, :]).to(dtype))


@pytest.mark.parametrize("m,n,k,lda,ldb,ldc,skip", [(5, 40, 100, 128, 160, 43, 1), (40, 70, 333, 352, 336, 71, 3),
                                                     (200, 130, 77, 96, 80, 132, 2), (300, 300, 300, 320, 304, 304, 0)])
def test_matmul_strides(qc, m, n, k, lda, ldb, ldc, skip):
    a, b = codes_of(m, k, 1), codes_of(n, k, 2)
    sa, sb = torch.rand(m) + 0.5, torch.rand(n) + 0.5
    for dtype in DTYPES:
        check_product(run_matmul(qc, a, sa, b, sb, dtype, lda, ldb, ldc, skip), a, sa, b, sb, dtype)


@pytest.mark.parametrize("m", [1, 70])
def test_matmul_longest_k(qc, m):
    """All codes at -128 and the longest k: the int32 sum is at its limit."""
    k = 131071
    a = torch.full((m, k), -128, dtype=torch.int8)
    b = torch.full((20, k), -128, dtype=torch.int8)
    got = run_matmul(qc, a, torch.ones(m), b, torch.ones(20), F32)
    assert np.all(got == np.float32(k * 16384))


@pytest.mark.parametrize("m", [3, 90])
def test_matmul_scales(qc, m):
    """Zero, tiny and NaN scales: zeros, subnormal results, NaN rows and columns."""
    n, k = 37, 50
    a, b = codes_of(m, k, 4), codes_of(n, k, 5)
    sa, sb = torch.rand(m) + 0.5, torch.rand(n) + 0.5
    sa[0], sa[1], sb[0], sb[1], sb[2] = 0.0, float("nan"), 0.0, float("nan"), 2.0 ** -149
    got = run_matmul(qc, a, sa, b, sb, F32)
    with np.errstate(invalid="ignore"):
        s = (a.numpy().astype(np.int64) @ b.numpy().astype(np.int64).T).astype(np.float32)
        want = (s * sa.numpy()[:, None]) * sb.numpy()[None, :]
    assert same(got.astype(np.float32), want)


# ----------------------------------------------------------- checkpoints


def save(qc, x, ldx, skip=0):
    rows, dim = x.shape
    c, e = Buf(rows, ref.up(dim, 32), ref.up(dim, 32), torch.int8), Buf(rows, ref.up(dim, 128) // 32, ref.up(dim, 128) // 32, torch.uint8)
    qc.qc_encode_ckpt8(strided(x, ldx, skip), qt(qc, x.dtype), rows, dim, ldx, c.t, e.t)
    torch.cuda.synchronize()
    c.check()
    e.check()
    return c, e


CKPT = [(1, 1), (1, 31), (3, 32), (5, 33), (5, 515), (17, 127), (16, 128), (33, 129), (2, 4096), (3, 4097), (300, 8),
        (1, 70000), (1000, 40)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,dim", CKPT)
def test_checkpoint(qc, rows, dim, dtype):
    x = ref.matrix(rows, dim, rows + dim, dtype, 2.0)
    for ldx, skip in ((dim, 0), (dim + 3, 1)):
        c, e = save(qc, x, ldx, skip)
        wc, we = ref.ckpt8(x)
        assert np.array_equal(e.get().numpy(), we) and np.array_equal(c.get().numpy(), wc)
        want = ref.held(wc, we, dim)
        for out in DTYPES:
            y = Buf(rows, dim, dim + skip, out, skip)
            qc.qc_decode_ckpt8(c.t, e.t, rows, dim, y.t, qt(qc, out), dim + skip)
            torch.cuda.synchronize()
            y.check()
            assert same(y.get().double().numpy(), want)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("dim", [32, 100, 513])
def test_checkpoint_hard(qc, dim, dtype):
    x = ref.hard_rows(dim, dtype)
    c, e = save(qc, x, dim)
    wc, we = ref.ckpt8(x)
    assert np.array_equal(e.get().numpy(), we) and np.array_equal(c.get().numpy(), wc)
    y = Buf(x.shape[0], dim, dim, BF16)
    qc.qc_decode_ckpt8(c.t, e.t, x.shape[0], dim, y.t, qc.QC_BF16, dim)
    torch.cuda.synchronize()
    assert same(y.get().double().numpy(), ref.held(wc, we, dim))


# ------------------------------------------------------- weight gradient


def kept(x):
    c, e = ref.ckpt8(x)
    return torch.from_numpy(c).cuda(), torch.from_numpy(e).cuda(), ref.held(c, e, x.shape[1])


def run_wgrad(qc, dy, x, wtype=F32, accumulate=False, ldy=None, skip=0, ldw=None, wskip=0, start=None):
    (rows, n), dim = dy.shape, x.shape[1]
    c, e, v = kept(x)
    ldy, ldw = ldy or n, ldw or dim
    dw = Buf(n, dim, ldw, wtype, wskip)
    if start is not None:
        dw.t[:, :dim] = start.cuda()
    need = qc.qc_ckpt8_wgrad_workspace(rows, n, dim, qt(qc, dy.dtype))
    ws = torch.full((max(need, 16) + 64,), 0x7F, dtype=torch.uint8, device="cuda") if need else None
    qc.qc_ckpt8_wgrad(strided(dy, ldy, skip), qt(qc, dy.dtype), ldy, c, e, rows, n, dim, dw.t, qt(qc, wtype), ldw,
                      accumulate, ws)
    torch.cuda.synchronize()
    dw.check()
    if need:
        assert bool((ws[need:] == 0x7F).all())
    return dw.get(), v


def check_wgrad(got, dy, v, wtype, start=None):
    d = dy.double().numpy()
    want, mag = d.T @ v, np.abs(d).T @ np.abs(v)
    if start is not None:
        want, mag = want + start.double().numpy(), mag + np.abs(start.double().numpy())
    terms = (3 if dy.dtype is F32 else 1) * dy.shape[0] + 600  # the joins of up to 512 splits among them
    tol = 2 * U32 * terms * mag + (ref.EPS[BF16] * np.abs(want) if wtype is BF16 else 0)
    off = np.abs(got.double().numpy() - want)
    assert np.all(off <= tol + 2.0 ** -126), (off.max(), (off - tol).max())
    # and, as its rounding errors are no conspiracy, far closer as a whole
    rel = np.linalg.norm(off) / max(np.linalg.norm(want), 1e-30)
    assert rel <= (4e-3 if wtype is BF16 else 1e-5), rel


WG = [(2049, 64, 130), (4500, 264, 200), (1, 8, 16), (1, 1, 1), (5, 33, 70), (63, 16, 32), (64, 128, 128),
      (65, 130, 127), (130, 250, 500), (200, 64, 257), (257, 384, 129), (1000, 40, 72), (3000, 64, 100), (515, 8, 300)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,n,dim", WG)
def test_wgrad(qc, rows, n, dim, dtype):
    dy, x = ref.matrix(rows, n, 1, dtype), ref.matrix(rows, dim, 2, dtype)
    got, v = run_wgrad(qc, dy, x)
    check_wgrad(got, dy, v, F32)
    again, _ = run_wgrad(qc, dy, x)
    assert torch.equal(got, again)


@pytest.mark.parametrize("rows,n,dim", [(70, 3600, 3700), (129, 3504, 3425), (64, 4095, 3300), (609, 3600, 3601),
                                        (512, 3584, 3840), (289, 3592, 3500)])
def test_wgrad_large_tiles(qc, rows, n, dim):
    dy, x = ref.matrix(rows, n, 1, BF16), ref.matrix(rows, dim, 2, BF16)
    got, v = run_wgrad(qc, dy, x)
    check_wgrad(got, dy, v, F32)


@pytest.mark.parametrize("rows,n,dim", [(1, 2700, 3300), (33, 2701, 3302), (70, 3600, 3700), (129, 3503, 3425),
                                        (190, 2563, 3329), (225, 3000, 4000), (609, 2602, 3601), (2048, 513, 2000)])
def test_wgrad_large_tiles_fp32(qc, rows, n, dim):
    """Stages from one to twenty, the last ones short, over the wide tile."""
    dy, x = ref.matrix(rows, n, 1, F32), ref.matrix(rows, dim, 2, F32)
    got, v = run_wgrad(qc, dy, x)
    check_wgrad(got, dy, v, F32)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,n,dim,ldy,skip,ldw,wskip", [(100, 24, 50, 33, 1, 53, 1), (70, 64, 64, 72, 8, 68, 4),
                                                            (200, 40, 96, 48, 0, 97, 3), (2500, 48, 40, 56, 8, 41, 1)])
def test_wgrad_strides_and_outputs(qc, rows, n, dim, ldy, skip, ldw, wskip, dtype):
    dy, x = ref.matrix(rows, n, 3, dtype), ref.matrix(rows, dim, 4, dtype)
    start = torch.randn((n, dim), generator=torch.Generator().manual_seed(9))
    got, v = run_wgrad(qc, dy, x, F32, True, ldy, skip, ldw, wskip, start)
    check_wgrad(got, dy, v, F32, start)
    got, v = run_wgrad(qc, dy, x, BF16, False, ldy, skip, ldw, wskip)
    check_wgrad(got, dy, v, BF16)


def test_wgrad_no_tokens(qc):
    for acc in (False, True):
        dw = Buf(33, 50, 50, F32)
        dw.t[:, :50] = 3.0
        e = torch.empty((0, 4), dtype=torch.uint8, device="cuda")
        qc.qc_ckpt8_wgrad(torch.empty((0, 33), dtype=BF16, device="cuda"), qc.QC_BF16, 33,
                          torch.empty((0, 64), dtype=torch.int8, device="cuda"), e, 0, 33, 50, dw.t, qc.QC_F32, 50, acc)
        torch.cuda.synchronize()
        dw.check()
        assert bool((dw.get() == (3.0 if acc else 0.0)).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,n,dim", [(70, 16, 96), (130, 13, 96), (65, 272, 160), (77, 2602, 3400)])
def test_wgrad_infinities(qc, rows, n, dim, dtype):
    """An infinite gradient makes its channel infinite (or NaN where values
    of both signs meet it), a NaN group its columns; all else stays finite.
    The last token of a short tile carries them."""
    dy, x = ref.matrix(rows, n, 5, dtype), ref.matrix(rows, dim, 6, dtype).abs() + 0.5
    dy[rows - 1, 2] = float("inf")
    dy[0, 4] = float("nan")
    x[rows - 1, 40] = float("nan")
    got, v = run_wgrad(qc, dy, x)
    got = got.numpy()
    with np.errstate(invalid="ignore"):
        want = dy.double().numpy().T @ v
    cols = np.zeros(dim, bool)
    cols[32:64] = True
    rowsel = np.ones(n, bool)
    rowsel[[2, 4]] = False
    assert np.isnan(got[4]).all() and np.isnan(got[:, cols]).all()
    assert np.isposinf(got[2, ~cols][v[rows - 1, ~cols] > 0]).all()
    assert np.isfinite(got[rowsel][:, ~cols]).all() and np.isfinite(want[rowsel][:, ~cols]).all()


@pytest.mark.parametrize("rows,n,dim", [(96, 40, 64)])
def test_wgrad_fp32_pieces(qc, rows, n, dim):
    """An fp32 gradient is taken whole: with one token a column the products come out as fp32 products."""
    g = torch.Generator().manual_seed(8)
    dy = torch.zeros((rows, n))
    dy[torch.arange(n) % rows, torch.arange(n)] = torch.randn(n, generator=g) * torch.exp(6 * torch.randn(n, generator=g))
    x = ref.matrix(rows, dim, 2, F32)
    got, v = run_wgrad(qc, dy, x)
    want = dy.double().numpy().T @ v  # one term an output
    # three pieces, each product exact: two additions
    assert np.all(np.abs(got.double().numpy() - want) <= 4 * U32 * np.abs(want) + 2.0 ** -126)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("n", [3, 16])
def test_wgrad_every_step(qc, n, dtype):
    """One token a channel and a power of two: dW holds what the checkpoint
    stands for, from the largest step to the smallest, exactly (results below
    the smallest normal number may come out as zero)."""
    x = ref.hard_rows(96, dtype)[:14]  # the finite ones
    dy = torch.zeros((14, n), dtype=dtype)
    for first in range(0, 14, n):
        dy.zero_()
        k = min(n, 14 - first)
        dy[torch.arange(first, first + k), torch.arange(k)] = 2.0 ** -3
        got, v = run_wgrad(qc, dy, x)
        want = v[first: first + k] / 8
        off = np.abs(got[:k].double().numpy() - want)
        assert np.all(off <= np.where(np.abs(want) < 2.0 ** -125, np.abs(want), 0.0)), off.max()


def test_wgrad_is_the_gradient(qc):
    """Against differences of sum(dy * (X W^T)), X as held."""
    rows, n, dim = 90, 12, 40
    dy, x = ref.matrix(rows, n, 1, F32), ref.matrix(rows, dim, 2, F32)
    got, v = run_wgrad(qc, dy, x)
    w, d = np.random.default_rng(0).standard_normal((n, dim)), dy.double().numpy()
    for j, i in ((0, 0), (5, 17), (11, 39)):
        h = np.zeros_like(w)
        h[j, i] = 0.5  # the function is linear: any step will do
        diff = (d * (v @ (w + h).T)).sum() - (d * (v @ (w - h).T)).sum()
        scale = np.abs(d[:, j]) @ np.abs(v[:, i])
        assert abs(got[j, i].item() - diff) <= 2 * U32 * (3 * rows + 600) * scale + 1e-9 * np.abs(d).sum()


# ------------------------------------------------------ gated activation


def hard_gate(dtype):
    v = torch.tensor([0.0, -0.0, 1.0, -1.0, -1.2784645, 20.0, -20.0, 87.0, -87.0, 88.8, -88.8, 100.0, -100.0, 1e4, -1e4,
                      2.0 ** -130, -(2.0 ** -130), 0.5, -0.5, 3.0])
    return v.repeat(20)[: 13 * 30].view(13, 30).to(dtype)


def run_swiglu(qc, g, u, dh, ldx, skip, apart=False):
    rows, dim = g.shape
    t = qt(qc, g.dtype)
    if apart:
        gd, ud = strided(g, ldx, skip), strided(u, ldx, skip)
    else:
        both = strided(torch.cat([g, u], 1), ldx, skip)
        gd, ud = both[:, :dim], both[:, dim: 2 * dim]
    pc, pe = ref.up(dim, 32), ref.up(dim, 128) // 32
    kg, ku = [(Buf(rows, pc, pc, torch.int8), Buf(rows, pe, pe, torch.uint8)) for _ in range(2)]
    h = Buf(rows, dim, dim + skip, g.dtype, skip)
    qc.qc_swiglu_ckpt8(gd, ud, t, ldx, rows, dim, h.t, dim + skip, kg[0].t, kg[1].t, ku[0].t, ku[1].t)
    ldg = 2 * dim + skip
    d = Buf(rows, 2 * dim, ldg, g.dtype, skip)
    qc.qc_swiglu_ckpt8_backward(strided(dh, dim + 1, 1), t, dim + 1, kg[0].t, kg[1].t, ku[0].t, ku[1].t, rows, dim,
                                d.t[:, :dim], d.t[:, dim: 2 * dim], ldg)
    torch.cuda.synchronize()
    for b in (*kg, *ku, h, d):
        b.check()
    return kg, ku, h.get(), d.get()[:, :dim], d.get()[:, dim:]


def close(got, want, tol, dtype, floor):
    off = np.abs(got.double().numpy() - want)
    eps = ref.EPS[dtype]
    bound = tol * (1 + eps) + eps * np.abs(want) + floor + (2.0 ** -133 if dtype is BF16 else 2.0 ** -149)
    assert np.all(off <= bound), (off.max(), np.argmax(off - bound))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,dim", [(1, 1), (7, 1001), (3, 128), (65, 40), (2, 4096), ("hard", 0)])
def test_swiglu(qc, rows, dim, dtype):
    """exp is within 2 ulp (4 half steps of fp32), its sum with one, a
    quotient and two products add one half step each: h within 8 half steps,
    and where exp overflows (g < -88.7) within 2^-120 |u| of a value below
    that.  With s = 1/(1+exp(-G)) within 6 half steps and 1 - s within 7 of
    1: dU within 8 half steps; dG, whose last factor is 1 + G (1 - s), within
    |dh U s| (12 + 10 |G|) half steps."""
    if rows == "hard":
        g = hard_gate(dtype)
        rows, dim = g.shape
        u, dh = ref.matrix(rows, dim, 2, dtype), ref.matrix(rows, dim, 3, dtype)
    else:
        g, u, dh = (ref.matrix(rows, dim, s, dtype) for s in (1, 2, 3))
    for ldx, skip, apart in ((2 * dim, 0, False), (2 * dim + 1, 1, False), (dim + 8, 0, True)):
        kg, ku, h, dg, du = run_swiglu(qc, g, u, dh, ldx, skip, apart)
        for (c, e), x in ((kg, g), (ku, u)):
            wc, we = ref.ckpt8(x)
            assert np.array_equal(c.get().numpy(), wc) and np.array_equal(e.get().numpy(), we)
        gd, ud, dd = g.double().numpy(), u.double().numpy(), dh.double().numpy()
        want = gd * ref.sigmoid(gd) * ud
        close(h, want, 8 * U32 * np.abs(want), dtype, 2.0 ** -120 * np.abs(ud))
        G, U = ref.held(*ref.ckpt8(g), dim), ref.held(*ref.ckpt8(u), dim)
        s = ref.sigmoid(G)
        wu = dd * G * s
        close(du, wu, 8 * U32 * np.abs(wu), dtype, 2.0 ** -120 * np.abs(dd))
        wg = dd * U * s * (1 + G * (1 - s))
        close(dg, wg, np.abs(dd * U * s) * U32 * (12 + 10 * np.abs(G)), dtype,
              2.0 ** -120 * np.abs(dd * U) * (1 + np.abs(G)))


def test_swiglu_backward_is_the_gradient(qc):
    """Against differences of sum(dh * silu(G) U) at values a checkpoint holds
    exactly; the step 2^-10 leaves an error of its square."""
    rows, dim = 5, 64
    gen = torch.Generator().manual_seed(3)
    g, u = (torch.randint(-127, 128, (rows, dim), generator=gen).float() / 32 for _ in range(2))
    g[:, ::32], u[:, ::32] = 127 / 32, 127 / 32
    dh = torch.randn((rows, dim), generator=gen)
    _, _, _, dg, du = run_swiglu(qc, g, u, dh, 2 * dim, 0)
    G, U, d, e = g.double().numpy(), u.double().numpy(), dh.double().numpy(), 2.0 ** -10
    f = lambda a, b: d * a * ref.sigmoid(a) * b  # noqa: E731
    big = np.abs(d) * 5  # |U| <= 4; the third derivative of silu is below 1/2
    assert np.all(np.abs(dg.numpy() - (f(G + e, U) - f(G - e, U)) / (2 * e)) <= big * (e * e + 2.0 ** -18))
    assert np.all(np.abs(du.numpy() - (f(G, U + e) - f(G, U - e)) / (2 * e)) <= big * 2.0 ** -18)


# -------------------------------------------------- streams, graphs, sizes


def layer(qc, s):
    """One pass of everything, as a training step strings it together."""
    t, m, n, k = qc.QC_BF16, s["m"], s["n"], s["k"]
    qc.qc_encode_int8_rowwise(s["x"], t, m, k, k, s["q"], s["q"].shape[1], s["s"])
    qc.qc_matmul_int8(s["q"], s["s"], s["q"].shape[1], s["w"], s["ws"], s["q"].shape[1], m, n, k, s["y"], t, n)
    qc.qc_encode_ckpt8(s["x"], t, m, k, k, s["c"], s["e"])
    qc.qc_ckpt8_wgrad(s["y"], t, n, s["c"], s["e"], m, n, k, s["dw"], qc.QC_F32, k, False, s["work"])
    qc.qc_decode_ckpt8(s["c"], s["e"], m, k, s["r"], t, k)


def layer_state(qc, m, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kp = ref.up(k, 16)
    s = dict(m=m, n=n, k=k)
    s["x"] = torch.randn((m, k), device="cuda", generator=g).to(BF16)
    s["w"] = torch.randint(-127, 128, (n, kp), device="cuda", generator=g, dtype=torch.int8)
    s["ws"] = torch.rand(n, device="cuda", generator=g) * 1e-3
    s["q"], s["s"] = torch.empty((m, kp), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    s["y"], s["dw"] = torch.empty((m, n), dtype=BF16, device="cuda"), torch.empty((n, k), device="cuda")
    cb, eb = qc.ckpt8_bytes(m, k)
    s["c"], s["e"] = torch.empty(cb, dtype=torch.int8, device="cuda"), torch.empty(eb, dtype=torch.uint8, device="cuda")
    s["r"] = torch.empty((m, k), dtype=BF16, device="cuda")
    s["work"] = torch.empty(max(16, qc.qc_ckpt8_wgrad_workspace(m, n, k, qc.QC_BF16)), dtype=torch.uint8, device="cuda")
    return s


OUT = ("q", "s", "y", "c", "e", "dw", "r")


@pytest.mark.parametrize("m,n,k", [(5, 70, 200), (1500, 96, 130)])
def test_streams_and_graph(qc, m, n, k):
    s = layer_state(qc, m, n, k, 1)
    layer(qc, s)
    torch.cuda.synchronize()
    want = {o: s[o].clone() for o in OUT}
    side = torch.cuda.Stream()
    for o in OUT:
        s[o].zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(qc, s)
    side.synchronize()
    assert all(torch.equal(s[o].view(torch.uint8), want[o].view(torch.uint8)) for o in OUT)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(qc, s)
    first = s["x"].clone()
    for turn in range(3):
        s["x"].copy_(first * (turn + 1))
        layer(qc, s)
        torch.cuda.synchronize()
        eager = {o: s[o].clone() for o in OUT}
        for o in OUT:
            s[o].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s[o].view(torch.uint8), eager[o].view(torch.uint8)) for o in OUT)


@pytest.mark.parametrize("m,n", [(4200000, 3), (3, 1100000)])
def test_matmul_many_tiles(qc, m, n):
    """More tiles one way than a grid has in its second dimension."""
    g = torch.Generator(device="cuda").manual_seed(2)
    a = torch.randint(-127, 128, (m, 16), device="cuda", generator=g, dtype=torch.int8)
    b = torch.randint(-127, 128, (n, 16), device="cuda", generator=g, dtype=torch.int8)
    c = torch.empty((m, n), device="cuda")
    one = torch.ones(max(m, n), device="cuda")
    qc.qc_matmul_int8(a, one, 16, b, one, 16, m, n, 16, c, qc.QC_F32, n)
    assert torch.equal(c, a.float() @ b.float().t())  # sums below 2^24: exact


def test_rows_past_the_grid(qc):
    """More rows than blocks of one launch."""
    rows = 4400000
    x = torch.randn((rows, 8), device="cuda").to(BF16)
    q, s = torch.empty((rows, 16), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    c, e = torch.empty((rows, 32), dtype=torch.int8, device="cuda"), torch.empty((rows, 4), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    qc.qc_encode_int8_rowwise(x, qc.QC_BF16, rows, 8, 8, q, 16, s)
    qc.qc_encode_ckpt8(x, qc.QC_BF16, rows, 8, 8, c, e)
    qc.qc_decode_ckpt8(c, e, rows, 8, y, qc.QC_BF16, 8)
    torch.cuda.synchronize()
    for at in (0, 1048570, 4194300, rows - 50):
        part = x[at: at + 50].cpu()
        wq, ws = ref.int8_rows(part)
        wc, we = ref.ckpt8(part)
        assert np.array_equal(q[at: at + 50, :8].cpu().numpy(), wq) and same(s[at: at + 50].cpu().numpy(), ws)
        assert np.array_equal(c[at: at + 50].cpu().numpy(), wc) and np.array_equal(e[at: at + 50].cpu().numpy(), we)
        assert same(y[at: at + 50].cpu().double().numpy(), ref.held(wc, we, 8))


def test_offsets_past_32_bits(qc):
    """Row strides that put the last rows past 2^31 elements."""
    rows, ld, cols = 70000, 32768, 40
    x = torch.zeros((rows, ld), dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[:, :cols] = torch.randn((rows, cols), device="cuda", generator=g).to(BF16)
    small = x[:, :cols].contiguous()
    s = torch.empty((2, rows), device="cuda")
    q = torch.empty((2, rows, 48), dtype=torch.int8, device="cuda")
    c, e = torch.empty((2, rows, 64), dtype=torch.int8, device="cuda"), torch.empty((2, rows, 4), dtype=torch.uint8, device="cuda")
    b, sb = torch.randint(-127, 128, (32, 48), device="cuda", dtype=torch.int8), torch.rand(32, device="cuda")
    dw = torch.empty((2, cols, cols), device="cuda")
    work = torch.empty(qc.qc_ckpt8_wgrad_workspace(rows, cols, cols, qc.QC_BF16), dtype=torch.uint8, device="cuda")
    for i, (t, l) in enumerate(((x, ld), (small, cols))):
        qc.qc_encode_int8_rowwise(t, qc.QC_BF16, rows, cols, l, q[i], 48, s[i])
        qc.qc_encode_ckpt8(t, qc.QC_BF16, rows, cols, l, c[i], e[i])
        qc.qc_ckpt8_wgrad(t, qc.QC_BF16, l, c[i], e[i], rows, cols, cols, dw[i], qc.QC_F32, cols, False, work)
    y = torch.empty((rows, 32), dtype=BF16, device="cuda")
    qc.qc_matmul_int8(q[1], s[1], 48, b, sb, 48, rows, 32, cols, y, qc.QC_BF16, 32)
    qc.qc_matmul_int8(q[1], s[1], 48, b, sb, 48, rows, 32, cols, x, qc.QC_BF16, ld)
    torch.cuda.synchronize()
    for p in (q, s, c, e, dw):
        assert torch.equal(p[0], p[1])
    assert torch.equal(x[:, :32], y) and bool((x[:, cols:] == 0).all())
