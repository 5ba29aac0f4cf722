"""The 4-bit matrix operators on the GPU against their plain 64-bit forms
(mx_ref.py).

Tolerances: codes, scales and decoded values are equal.  A product's terms are
exact; its fp32 sum of k terms is within k + 1 half steps (two allowed for
each addition) of the sum of their magnitudes, and its output rounds once
more to its type; accumulation adds one more fp32 rounding."""
import numpy as np
import pytest
import torch

import mx_ref as ref
from gpu_util import need_gpu
from test_gpu_matrix import BF16, DTYPES, F32, Buf, qt, strided

pytestmark = pytest.mark.gpu
EPS = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def qc():
    return need_gpu()


class Held:
    """Buffers of an MXFP4 matrix between guards, prefilled."""

    def __init__(self, qc, rows, dim):
        self.rows, self.dim = rows, dim
        cb, sb = qc.mxfp4_bytes(rows, dim)
        self.raw = [torch.full((n + 256,), 0x5C, dtype=torch.uint8, device="cuda") for n in (cb, sb)]
        self.codes, self.scales = (r[:n] for r, n in zip(self.raw, (cb, sb)))

    def set(self, codes, scales):
        self.codes.copy_(torch.from_numpy(codes).view(-1))
        self.scales.copy_(torch.from_numpy(scales).view(-1))
        return self

    def host(self):
        for r in self.raw:
            assert bool((r[-256:] == 0x5C).all()), "a write past the end"
        return (self.codes.cpu().numpy().reshape(self.rows, -1), self.scales.cpu().numpy().reshape(self.rows, -1))

    def pair(self):
        return self.codes, self.scales


def matrix(rows, dim, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, dim), generator=g) * torch.exp(torch.randn((1, dim), generator=g))
    return (x * torch.exp(2.0 * torch.randn((rows, 1), generator=g))).to(dtype)


def check_encoding(qc, x, ldx, skip, both):
    rows, dim = x.shape
    a, t = Held(qc, rows, dim), Held(qc, dim, rows)
    kept = {"rows": (*a.pair(), None, None), "columns": (None, None, *t.pair()), "both": (*a.pair(), *t.pair())}[both]
    qc.qc_encode_mxfp4(strided(x, ldx, skip), qt(qc, x.dtype), rows, dim, ldx, *kept)
    for held, want, name in ((a, x, "columns"), (t, x.t(), "rows")):
        if both == name:
            continue
        for got, ref_ in zip(held.host(), ref.encode(want)):
            assert np.array_equal(got, ref_)


@pytest.mark.parametrize("both", ["rows", "columns", "both"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 32), (3, 31), (33, 64), (5, 515), (127, 129), (128, 128), (129, 127),
                                      (64, 4096), (300, 200), (1000, 7), (31, 1001)])
def test_encode(qc, rows, dim, dtype, both):
    check_encoding(qc, matrix(rows, dim, rows + dim, dtype), dim, 0, both)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("ldx,skip", [(131, 0), (136, 8), (200, 3), (131, 1)])
def test_encode_part_of_a_wider_matrix(qc, dtype, ldx, skip):
    check_encoding(qc, matrix(70, 130, 5, dtype), ldx, skip, "both")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("dim", [1, 32, 33, 128, 300])
def test_encode_hard_rows(qc, dim, dtype):
    x = ref.hard_rows(dim, dtype)
    check_encoding(qc, x, dim, 0, "both")
    check_encoding(qc, x.t().contiguous(), x.shape[0], 0, "both")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_every_bf16_number(qc, dtype):
    """All finite bf16 numbers, each beside neighbours of its own size."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(BF16).float()
    x = torch.where(torch.isfinite(x), x, torch.zeros(())).view(-1, 32).to(dtype)
    check_encoding(qc, x, 32, 0, "both")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,dim,ldo", [(1, 1, 1), (16, 32, 32), (7, 131, 140), (64, 515, 515), (255, 256, 256)])
def test_decode_every_code_and_scale(qc, rows, dim, ldo, dtype):
    codes, scales = ref.random_mx(rows, dim, 3, 1, 256)  # 255 among the scales
    scales[scales == 254] = 253  # 6 * 2^127 is no fp32 number
    out = Buf(rows, dim, ldo, dtype, skip=1)
    h = Held(qc, rows, dim).set(codes, scales)
    qc.qc_decode_mxfp4(*h.pair(), rows, dim, out.t, qt(qc, dtype), ldo)
    want = torch.from_numpy(ref.held(codes, scales, dim)).to(dtype)
    got = out.get()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok].float().view(torch.int32), want[ok].float().view(torch.int32))  # signs of zeros too
    out.check()


# ---------------------------------------------------------------- products


def space(need):
    return torch.full((max(16, need),), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs: nothing may rely on zeros


def check_product(got, a, b, c0=None):
    """got against the 64-bit a b^T (+ c0)."""
    dtype, k = got.dtype, a.shape[1]
    got = got.double().numpy()
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    if c0 is not None:
        want, size = want + c0, size + np.abs(c0)
    tol = size * (k + 2) * 2.0 ** -24 + np.abs(want) * EPS[dtype] + 2.0 ** -126
    nan = np.isnan(want)
    assert np.array_equal(nan, np.isnan(got))
    assert (np.abs(got - want)[~nan] <= tol[~nan]).all()


SIZES = [(1, 1, 1), (1, 16, 32), (1, 130, 515), (2, 33, 64), (7, 48, 1000), (16, 64, 128), (17, 100, 300), (33, 31, 65),
         (64, 64, 4096), (61, 200, 2043), (100, 90, 130), (128, 256, 256), (130, 258, 777), (257, 255, 512),
         (300, 520, 1030), (520, 300, 96), (64, 96, 9000)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(qc, m, n, k, dtype):
    (ac, as_), (bc, bs) = ref.random_mx(m, k, 1), ref.random_mx(n, k, 2)
    a, b = Held(qc, m, k).set(ac, as_), Held(qc, n, k).set(bc, bs)
    ldc = n + 5
    c = Buf(m, n, ldc, dtype, skip=3)
    w = space(qc.qc_matmul_mxfp4_workspace(m, n, k))
    qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), m, n, k, c.t, qt(qc, dtype), ldc, False, w)
    check_product(c.get(), ref.held(ac, as_, k), ref.held(bc, bs, k))
    c.check()
    first = c.get().clone()
    qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), m, n, k, c.t, qt(qc, dtype), ldc, False, w)
    assert torch.equal(first.view(torch.uint8), c.get().view(torch.uint8))  # the same bits again


@pytest.mark.parametrize("m,n,k", [(1, 40, 96), (40, 70, 300), (130, 260, 515), (256, 512, 1024), (64, 96, 9000)])
def test_product_added(qc, m, n, k):
    (ac, as_), (bc, bs) = ref.random_mx(m, k, 3), ref.random_mx(n, k, 4)
    a, b = Held(qc, m, k).set(ac, as_), Held(qc, n, k).set(bc, bs)
    c = Buf(m, n, n + 1, F32)
    c0 = torch.randn((m, n)) * 10.0
    c.t[:, :n] = c0.cuda()
    w = space(qc.qc_matmul_mxfp4_workspace(m, n, k))
    for times in (1, 2):
        qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), m, n, k, c.t, qc.QC_F32, n + 1, True, w)
        check_product(c.get(), times * ref.held(ac, as_, k), ref.held(bc, bs, k), c0.double().numpy())
    c.check()


@pytest.mark.parametrize("m,n,k", [(1, 40, 300), (40, 70, 300), (300, 300, 520)])
def test_product_with_nan_groups(qc, m, n, k):
    """A group that stands for NaNs makes its row or column NaN, no other."""
    (ac, as_), (bc, bs) = ref.random_mx(m, k, 5), ref.random_mx(n, k, 6)
    for codes, scales, r, g in ((ac, as_, m // 2, 1), (bc, bs, n - 1, k // 32)):
        scales[r, g] = 255
        codes[r, 16 * g: 16 * g + 16] = 0
    a, b = Held(qc, m, k).set(ac, as_), Held(qc, n, k).set(bc, bs)
    c = Buf(m, n, n, F32)
    w = space(qc.qc_matmul_mxfp4_workspace(m, n, k))
    qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), m, n, k, c.t, qc.QC_F32, n, False, w)
    want = ref.held(ac, as_, k) @ ref.held(bc, bs, k).T
    assert np.isnan(want).sum() == m + n - 1
    check_product(c.get(), ref.held(ac, as_, k), ref.held(bc, bs, k))


def test_scales_at_their_ends(qc):
    """The largest and smallest scales on opposite sides, and sums that overflow."""
    m, n, k = 40, 48, 256
    (ac, _), (bc, _) = ref.random_mx(m, k, 7), ref.random_mx(n, k, 8)
    for sa, sb in ((253, 1), (1, 253), (127, 127), (250, 5)):
        as_, bs = np.full((m, 8), sa, np.uint8), np.full((n, 8), sb, np.uint8)
        a, b = Held(qc, m, k).set(ac, as_), Held(qc, n, k).set(bc, bs)
        c = Buf(m, n, n, F32)
        qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), m, n, k, c.t, qc.QC_F32, n, False,
                           space(qc.qc_matmul_mxfp4_workspace(m, n, k)))
        check_product(c.get(), ref.held(ac, as_, k), ref.held(bc, bs, k))


def test_scales_that_only_others_write(qc):
    """Bytes 0 and 254, 2^-127 and 2^127, which the encoder does not need: decoded
    (6 * 2^127 is no fp32 number) and multiplied."""
    rows, dim = 255, 32
    codes = np.tile(np.arange(16, dtype=np.uint8) * 16 + np.arange(16, dtype=np.uint8)[::-1], (rows, 1))
    scales = np.zeros((rows, 4), np.uint8)
    scales[:, 0] = np.arange(rows)
    h = Held(qc, rows, dim).set(codes, scales)
    for dtype in DTYPES:
        out = torch.empty((rows, dim), dtype=dtype, device="cuda")
        qc.qc_decode_mxfp4(*h.pair(), rows, dim, out, qt(qc, dtype), dim)
        want = torch.from_numpy(ref.held(codes, scales, dim)).to(dtype)
        assert torch.equal(out.cpu(), want)
    m, n, k = 33, 70, 300
    (ac, _), (bc, _) = ref.random_mx(m, k, 7), ref.random_mx(n, k, 8)
    for sa, sb in ((254, 0), (0, 254), (254, 2)):
        as_, bs = (np.zeros((r, 12), np.uint8) for r in (m, n))
        as_[:, :10], bs[:, :10] = sa, sb
        c = Buf(m, n, n, F32)
        a, b = Held(qc, m, k).set(ac, as_), Held(qc, n, k).set(bc, bs)
        qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), m, n, k, c.t, qc.QC_F32, n, False,
                           space(qc.qc_matmul_mxfp4_workspace(m, n, k)))
        check_product(c.get(), ref.held(ac, as_, k), ref.held(bc, bs, k))


WIDE = [(1, 5003, 700), (3, 4100, 1030), (5, 4200, 2043), (8, 8190, 515), (9, 4100, 600)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("m,n,k", SIZES + WIDE + [(4, 48, 4700), (8, 64, 9000), (1, 20, 20000)])
def test_linear(qc, m, n, k, dtype):
    bc, bs = ref.random_mx(n, k, 9)
    x = matrix(m, k, 10, dtype)
    b = Held(qc, n, k).set(bc, bs)
    c = Buf(m, n, n + 2, dtype)
    w = space(qc.qc_linear_mxfp4_workspace(m, n, k, qt(qc, dtype)))
    qc.qc_linear_mxfp4(strided(x, k + 3, 1), qt(qc, dtype), k + 3, *b.pair(), m, n, k, c.t, qt(qc, dtype), n + 2, w)
    check_product(c.get(), ref.held(*ref.encode(x), k), ref.held(bc, bs, k))
    c.check()


@pytest.mark.parametrize("m", [1, 5, 40])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_linear_of_hard_rows(qc, m, dtype):
    """Infinities and NaNs in a token reach that token's outputs only; each
    other row is right, whatever the size of its values."""
    k, n = 300, 50
    rows = ref.hard_rows(k, dtype)
    bc, bs = ref.random_mx(n, k, 11, 120, 130)
    b = Held(qc, n, k).set(bc, bs)
    w = space(qc.qc_linear_mxfp4_workspace(m, n, k, qt(qc, dtype)))
    for at in range(0, rows.shape[0], m):
        x = rows[at: at + m]
        x = torch.cat([x, rows[: m - x.shape[0]]])
        c = Buf(m, n, n, F32)
        qc.qc_linear_mxfp4(x.cuda(), qt(qc, dtype), k, *b.pair(), m, n, k, c.t, qc.QC_F32, n, w)
        with np.errstate(over="ignore"):
            want = ref.held(*ref.encode(x), k) @ ref.held(bc, bs, k).T
        got = c.get().double().numpy()
        big = np.abs(want) > 1e38  # may overflow on the way
        assert np.array_equal(np.isnan(got) | big, np.isnan(want) | big)
        size = np.abs(ref.held(*ref.encode(x), k)) @ np.abs(ref.held(bc, bs, k)).T
        ok = ~np.isnan(want) & ~big & (size < 1e37)
        assert (np.abs(got - want)[ok] <= size[ok] * (k + 2) * 2.0 ** -24 + 2.0 ** -126).all()


def representable(rows, dim, seed):
    """Values that MXFP4 holds exactly, whatever else is in their groups."""
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.choice([-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6], (rows, dim))).float()


@pytest.mark.parametrize("m,n,k", [(40, 70, 100), (130, 96, 200)])
def test_gradients_of_a_layer(qc, m, n, k):
    """Forward and both gradients, of values that encoding leaves as they are,
    against autograd and against differences: the loss <dy, x w^T> is linear
    in each of x and w, so a difference quotient is the gradient, and every sum
    here is a multiple of 1/8 below 2^21: exact in fp32."""
    x, w, dy = representable(m, k, 1), representable(n, k, 2), representable(m, n, 3)

    def layer(x, w, dy):
        held = {}
        for name, t in (("x", x), ("w", w), ("dy", dy)):
            r, d = t.shape
            held[name] = Held(qc, r, d), Held(qc, d, r)
            qc.qc_encode_mxfp4(t.cuda(), qc.QC_F32, r, d, d, *held[name][0].pair(), *held[name][1].pair())
        y, dx, dw = (torch.zeros(s, device="cuda") for s in ((m, n), (m, k), (n, k)))

        def product(a, b, m, n, k, c, add):
            work = space(qc.qc_matmul_mxfp4_workspace(m, n, k))
            qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), m, n, k, c, qc.QC_F32, n, add, work)

        product(held["x"][0], held["w"][0], m, n, k, y, False)
        product(held["dy"][0], held["w"][1], m, k, n, dx, False)
        product(held["dy"][1], held["x"][1], n, k, m, dw, True)
        return y.cpu(), dx.cpu(), dw.cpu()

    y, dx, dw = layer(x, w, dy)
    xr, wr = x.double().requires_grad_(), w.double().requires_grad_()
    out = xr @ wr.t()
    out.backward(dy.double())
    assert torch.equal(y.double(), out.detach())
    assert torch.equal(dx.double(), xr.grad) and torch.equal(dw.double(), wr.grad)
    for r, c in ((0, 0), (n // 2, k // 3), (n - 1, k - 1)):
        w2 = w.clone()
        w2[r, c] = 0.0 if w[r, c] else 1.0
        y2 = layer(x, w2, dy)[0]
        assert (dy * (y2 - y)).sum().double() == float(w2[r, c] - w[r, c]) * dw[r, c].double()
    for r, c in ((0, k - 1), (m - 1, 0)):
        x2 = x.clone()
        x2[r, c] = 0.0 if x[r, c] else 1.0
        y2 = layer(x2, w, dy)[0]
        assert (dy * (y2 - y)).sum().double() == float(x2[r, c] - x[r, c]) * dx[r, c].double()


@pytest.mark.parametrize("m,n,k", [(1, 256, 1024), (40, 200, 600), (300, 260, 900), (64, 64, 9000)])
def test_captured_and_replayed(qc, m, n, k):
    """A captured linear layer and product, replayed with new inputs between
    eager work, and on a stream of its own."""
    bc, bs = ref.random_mx(n, k, 12)
    b = Held(qc, n, k).set(bc, bs)
    x = torch.empty((m, k), dtype=BF16, device="cuda")
    a = Held(qc, m, k)
    c1, c2 = (torch.empty((m, n), device="cuda") for _ in range(2))
    w1, w2 = space(qc.qc_linear_mxfp4_workspace(m, n, k, qc.QC_BF16)), space(qc.qc_matmul_mxfp4_workspace(m, n, k))

    def run():
        qc.qc_linear_mxfp4(x, qc.QC_BF16, k, *b.pair(), m, n, k, c1, qc.QC_F32, n, w1)
        qc.qc_encode_mxfp4(x, qc.QC_BF16, m, k, k, *a.pair())
        qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), m, n, k, c2, qc.QC_F32, n, False, w2)

    x.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            run()
    for seed in range(4):
        xs = matrix(m, k, seed, BF16)
        x.copy_(xs)
        c1.zero_(), c2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = c1.clone(), c2.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(replayed[0], c1) and torch.equal(replayed[1], c2)
        check_product(c1.cpu(), ref.held(*ref.encode(xs), k), ref.held(bc, bs, k))


def test_two_streams_at_once(qc):
    """Calls that run beside each other, each with buffers and a workspace of its own."""
    cases = [(40, 500, 9000), (64, 64, 9000), (1, 300, 700), (1003, 510, 2043)]
    work = []
    for i, (m, n, k) in enumerate(cases):
        bc, bs = ref.random_mx(n, k, 20 + i)
        x, b = matrix(m, k, 30 + i, BF16).cuda(), Held(qc, n, k).set(bc, bs)
        need = qc.qc_linear_mxfp4_workspace(m, n, k, qc.QC_BF16)
        work.append((x, b, m, n, k, torch.empty((m, n), device="cuda"), space(need), torch.cuda.Stream()))

    def call(x, b, m, n, k, c, w):
        qc.qc_linear_mxfp4(x, qc.QC_BF16, k, *b.pair(), m, n, k, c, qc.QC_F32, n, w)

    alone = []
    for *args, _ in work:
        call(*args)
        alone.append(args[5].clone())
        args[5].fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for *args, stream in work:
            with torch.cuda.stream(stream):
                call(*args)
    torch.cuda.synchronize()
    for want, (*args, _) in zip(alone, work):
        assert torch.equal(args[5], want)


def test_more_channels_than_one_launch_encodes_tokens_for(qc):
    """2^27 channels: 16 a block of 512 threads would be a launch of 2^32."""
    m, n, k, period = 2, (1 << 27) + 5, 32, 4099
    (bc, bs), x = ref.random_mx(period, k, 1), matrix(m, k, 2, F32)
    whole = n // period * period
    b = Held(qc, n, k)
    for t, v in ((b.codes.view(n, -1), bc), (b.scales.view(n, -1), bs)):
        v = torch.from_numpy(v).cuda().view(period, -1)
        t[:whole].view(-1, *v.shape)[:] = v
        t[whole:] = v[: n - whole]
    c = torch.full((m, n), float("nan"), device="cuda")
    w = space(qc.qc_linear_mxfp4_workspace(m, n, k, qc.QC_F32))
    qc.qc_linear_mxfp4(x.cuda(), qc.QC_F32, k, *b.pair(), m, n, k, c, qc.QC_F32, n, w)
    check_product(c[:, :period].cpu(), ref.held(*ref.encode(x), k), ref.held(bc, bs, k))
    for row in c:
        assert bool((row[:whole].view(-1, period) == row[:period]).all())
        assert torch.equal(row[whole:], row[: n - whole])


def test_codes_past_32_bit_offsets(qc):
    """A tall matrix: codes of its last rows lie more than 2^32 bytes behind
    its first ones, its values further."""
    rows, dim, n = 140_000, 65_536, 16
    x = torch.zeros((rows, dim), dtype=BF16, device="cuda")  # 17 GiB
    probe = matrix(200, dim, 1, BF16)
    x[-200:] = probe.cuda()
    a = Held(qc, rows, dim)
    assert a.codes.numel() > 1 << 32
    qc.qc_encode_mxfp4(x, qc.QC_BF16, rows, dim, dim, *a.pair())
    want = ref.encode(probe)
    for got, w in zip(a.pair(), want):
        assert np.array_equal(got.view(rows, -1)[-200:].cpu().numpy(), w)
    assert int(a.codes.view(rows, -1)[:-200].max()) == 0
    bc, bs = ref.random_mx(n, dim, 2)
    b = Held(qc, n, dim).set(bc, bs)
    del x
    c = torch.full((rows, n), float("nan"), device="cuda")
    need = qc.qc_matmul_mxfp4_workspace(rows, n, dim)
    qc.qc_matmul_mxfp4(*a.pair(), *b.pair(), rows, n, dim, c, qc.QC_F32, n, False, space(need))
    assert bool((c[:-200] == 0).all())
    check_product(c[-200:].cpu(), ref.held(*want, dim), ref.held(bc, bs, dim))
    out = torch.empty((rows, dim), dtype=BF16, device="cuda")
    qc.qc_decode_mxfp4(*a.pair(), rows, dim, out, qc.QC_BF16, dim)
    assert np.array_equal(out[-200:].double().cpu().numpy(), ref.held(*want, dim))
    assert bool((out[:1000] == 0).all())
