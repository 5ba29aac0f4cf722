"""The optimizer's side of a tensor list on the GPU against its plain 64-bit
form (mx_ref.py): the clipping norm, the AdamW step with fp32 and with 8-bit
states, and those states' codes.

Tolerances, in half steps of fp32 (2^-24 of the value): with x = g * scale
rounded once, m = m * b1 + x * (1 - b1) is off by 4 of its two terms'
magnitudes (x, 1 - b1, the product and the sum round; b1, the product and the
sum); v by 6 of its own (x twice, its square, 1 - b2, the product and the sum);
r = sqrt(v) by 4; the update rate * m / (r * root + eps) by 16 of the update
that |m|'s two terms would give (m 4; rate, root and their products 4; r 4; the
sum with eps 1; a reciprocal within an ulp 2, the product with it 1); p by one for each of its factor, product and
difference.  Where v falls below 2^-126 it may be off by 2^-149, and r with it
by 2^-74."""
import math

import numpy as np
import pytest
import torch

import mx_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
U = ref.U32


@pytest.fixture(scope="module")
def qc():
    return need_gpu()


def qt(qc, dtype):
    return qc.QC_BF16 if dtype is BF16 else qc.QC_F32


class Tensors:
    """Tensors of these sizes in one buffer, `gap` elements of canary before
    each and after the last, so that they start at any alignment."""

    def __init__(self, qc, sizes, dtype, gap):
        self.sizes = sizes
        self.flat = torch.full((sum(sizes) + gap * (len(sizes) + 1),), 77.0, dtype=dtype, device="cuda")
        self.list, at = [], gap
        for s in sizes:
            self.list.append(self.flat[at: at + s])
            at += s + gap
        self.inside = torch.zeros(self.flat.numel(), dtype=torch.bool)
        at = gap
        for s in sizes:
            self.inside[at: at + s] = True
            at += s + gap
        self.table = qc.TensorTable(self.list)

    def set(self, x):
        for t, part in zip(self.list, torch.as_tensor(x).split(self.sizes)):
            t.copy_(part)
        return self

    def host(self):
        h = self.flat.cpu()
        assert bool((h[~self.inside] == 77.0).all()), "a write outside the tensors"
        return h[self.inside].double().numpy()


LISTS = {
    "one": [1], "two_small": [3, 5], "eight": [8], "block": [256], "odd": [257, 255, 1], "empty_ones": [0, 7, 0, 0, 300, 0],
    "segment": [4096], "segments": [4096, 4096, 1], "tiny_many": [1, 2, 3, 4, 5, 6, 7, 8, 9] * 60,
    "mixed": [1000, 3, 4097, 64, 12345, 1, 1, 70000, 33], "large": [1 << 20, 4097, 300001],
    # more tensors in a segment than a block holds at a time (255), ends of such parts and empty ones among them
    "parts": [1] * 254 + [0] * 300 + [3] * 255 + [0] * 255 + [5000, 2, 2] + [1] * 2100 + [0] * 700 + [8],
}


def values(n, seed, spread=2.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal(n) * np.exp(spread * g.standard_normal(n))
    x[g.random(n) < 0.1] = 0.0
    return x.astype(np.float32)


def near(got, want, tol):
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    ok = np.isfinite(want)
    assert (np.abs(got - want)[ok] <= tol[ok]).all(), float((np.abs(got - want)[ok] / tol[ok]).max())


def tolerances(p, g, m, v, new_v, upd, t, scale, hyper=HYPER):
    """(m, v, p) bounds for a step from these 64-bit values."""
    b1, b2 = hyper["beta1"], hyper["beta2"]
    m_size = b1 * np.abs(m) + (1 - b1) * np.abs(g * scale)
    tol_m, tol_v = 4 * U * m_size + 2.0 ** -149, 6 * U * new_v + 2.0 ** -148
    den = np.sqrt(new_v / (1 - b2 ** t)) + hyper["eps"]
    upd_size = hyper["lr"] / (1 - b1 ** t) * m_size / np.maximum(den, 1e-300)
    upd_size = np.where(den > 0, upd_size, 0.0)
    tol_p = 3 * U * np.abs(p) + 16 * U * upd_size + U * upd + 2.0 ** -149
    return tol_m, tol_v, tol_p


@pytest.mark.parametrize("gtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("weights", ["f32", "bf16", "master"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("name", LISTS)
def test_steps(qc, name, bits, weights, gtype):
    """Three steps, each against the 64-bit one from the state before it."""
    sizes = LISTS[name]
    n = sum(sizes)
    ptype = F32 if weights == "f32" else BF16
    params = Tensors(qc, sizes, ptype, gap=5).set(values(n, 1))
    grads = Tensors(qc, sizes, gtype, gap=3)
    master = torch.from_numpy(params.host().astype(np.float32)).cuda() if weights == "master" else None
    pad = lambda count, dtype: torch.full((count + 64,), 77, dtype=dtype, device="cuda")  # noqa: E731
    nb = -(-n // 256)
    if bits == 32:
        store = [pad(n, F32), pad(n, F32)]
        state = [t[:n].zero_() for t in store]
    else:
        store = [pad(n, torch.uint8), pad(nb, F32), pad(n, torch.uint8), pad(nb, F32)]
        state = [t[: (n, nb, n, nb)[k]].zero_() for k, t in enumerate(store)]

    def held():
        s = [t.cpu().numpy() for t in state]
        if bits == 32:
            return s[0].astype(np.float64), s[1].astype(np.float64)
        return ref.state_values(ref.M, s[0], s[1]), ref.state_values(ref.R, s[2], s[3]) ** 2

    scale = torch.tensor([0.75], device="cuda")
    for step in (1, 2, 3):
        grads.set(values(n, 10 + step))
        g = grads.host()
        p = master.cpu().double().numpy() if weights == "master" else params.host()
        m, v = held()
        call = qc.qc_adamw_multi if bits == 32 else qc.qc_adamw8_multi
        t = params.table
        call(t.xs, qt(qc, ptype), grads.table.xs, qt(qc, gtype), t.offsets, t.seg_first, t.ntensors, n, master, *state,
             step=step, grad_scale=scale if step > 1 else None, **HYPER)
        c = 0.75 if step > 1 else 1.0
        p1, m1, v1, upd = ref.adamw(p, g, m, v, step=step, scale=c, **HYPER)
        tol_m, tol_v, tol_p = tolerances(p, g, m, v, v1, upd, step, c)
        got_p = params.host()
        if weights == "master":
            mp = master.cpu().double().numpy()
            near(mp, p1, tol_p)
            assert np.array_equal(got_p, torch.from_numpy(mp).to(BF16).double().numpy())
        else:
            near(got_p, p1, tol_p + (2.0 ** -8 * (np.abs(p1) + tol_p) if ptype is BF16 else 0.0))
        if bits == 32:
            near(state[0].cpu().double().numpy(), m1, tol_m)
            near(state[1].cpu().double().numpy(), v1, tol_v)
        else:
            s = [x.cpu().numpy() for x in state]
            i = np.arange(n, dtype=object) if n < 100 else np.arange(n, dtype=np.int64)
            for kind, x, codes, sc in ((ref.M, m1, s[0], s[1]), (ref.R, np.sqrt(v1), s[2], s[3])):
                want = ref.state_scale(kind, x)
                # the largest magnitude's error, and two roundings of the scale
                err = 4 * U * (ref.blocks(np.abs(m) * 0.9 + 0.1 * np.abs(g * c)).max(1) if kind.signed
                               else ref.blocks(x).max(1)) / kind.largest + 2 * U * want
                near(sc.astype(np.float64), want, err + 2.0 ** -149)
                u = np.asarray(ref.dither(kind, i, step), np.float64)
                if kind.signed:  # m's error is relative to its terms: those near cancellation are left out
                    sure = tol_m <= 16 * U * np.abs(x)
                    check_some(kind, codes, sc, x, u, 16 * U, sure)
                else:
                    check_some(kind, codes, sc, x, u, 4 * U, np.ones(n, bool))
        for buf, part in zip(store, state):
            assert bool((buf[part.numel():] == 77).all()), "a write past the state"


def check_some(kind, codes, scale, x, u, err, sure):
    """check_codes, with elements that are not sure given their own code's value."""
    vals = ref.state_values(kind, codes, scale)
    x = np.where(sure, x, vals)
    if not sure.all():
        u = np.where(sure, u, 0.5)
    ref.check_codes(kind, codes, scale, x, u, err)


def saved(kind, x, step):
    """Codes and scales of fp32 values at a step, in fp32 arithmetic."""
    low, first, top = (20, 896, 127) if kind.signed else (19, 1792, 255)
    b = np.pad(x, (0, -x.size % 256)).reshape(-1, 256)
    largest, least = (np.array([first + c], np.uint32) << low for c in (top, 1))
    rest, least = np.float32(1) / largest.view(np.float32)[0], least.view(np.float32)[0]
    amax = np.abs(b).max(1)
    scale = np.where(amax > 0, np.maximum(amax * rest, np.float32(2.0 ** -100)), np.float32(0))
    with np.errstate(divide="ignore"):
        inv = np.where(scale > 0, np.float32(1) / scale, np.float32(0))
    y = (np.abs(b) * inv[:, None]).reshape(-1)[: x.size]
    u = (0x91E10DA5 * np.arange(x.size, dtype=np.uint64) + 0xC13FA9A9 * step + (0 if kind.signed else 1 << 31)) % (1 << 32)
    code = ((y.view(np.uint32) + (u >> (32 - low))) >> low).astype(np.int64) - first
    under = y > (u >> 8).astype(np.float32) * (least * np.float32(2.0 ** -24)) if kind.signed else y > 0
    code = np.where(y < least, under, np.minimum(code, top))
    return np.where(kind.signed & (x < 0) & (code > 0), code | 128, code).astype(np.uint8), scale


@pytest.mark.parametrize("gtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("bits", [32, 8])
def test_states_are_the_formulas_bits(qc, bits, gtype):
    """Six steps of states, carried on by the host in fp32 on its own: no
    rounding apart, where one code of one block's largest element would show."""
    sizes = [40000, 3, 255, 100001]
    n, nb = sum(sizes), -(-sum(sizes) // 256)
    params, grads = Tensors(qc, sizes, F32, 1).set(values(n, 1)), Tensors(qc, sizes, gtype, 1)
    b1, b2, rest1, rest2 = (np.float32(x) for x in (0.9, 0.999, 1 - 0.9, 1 - 0.999))
    m, v = np.zeros(n, np.float32), np.zeros(n, np.float32)
    if bits == 32:
        state = [torch.zeros(n, device="cuda") for _ in range(2)]
    else:
        state = [torch.zeros(k, dtype=d, device="cuda") for k, d in ((n, torch.uint8), (nb, F32)) * 2]
    call = qc.qc_adamw_multi if bits == 32 else qc.qc_adamw8_multi
    t, c = params.table, torch.tensor([0.37], device="cuda")
    for step in range(1, 7):
        grads.set(values(n, 20 + step))
        call(t.xs, 0, grads.table.xs, qt(qc, gtype), t.offsets, t.seg_first, t.ntensors, n, None, *state, step=step,
             grad_scale=c, **HYPER)
        x = grads.host().astype(np.float32) * np.float32(0.37)
        m, v = m * b1 + x * rest1, v * b2 + x * x * rest2
        got = [s.cpu().numpy() for s in state]
        if bits == 32:
            want = [m, v]
        else:
            want = [*saved(ref.M, m, step), *saved(ref.R, np.sqrt(v), step)]
            back = []
            for kind, (code, scale) in ((ref.M, want[:2]), (ref.R, want[2:])):
                mag = (code & 127 if kind.signed else code).astype(np.uint32)
                f = np.where(mag > 0, ((896 + mag << 20) if kind.signed else (1792 + mag << 19)).view(np.float32), np.float32(0))
                f = np.where(kind.signed & (code > 127), -f, f)
                back.append((np.pad(f, (0, nb * 256 - n)).reshape(nb, 256) * scale[:, None]).reshape(-1)[:n])
            m, v = back[0], back[1] * back[1]
        for g, w in zip(got, want):
            assert np.array_equal(g, w), (step, int((g != w).sum()))


@pytest.mark.parametrize("bits", [32, 8])
def test_nothing_but_zeros(qc, bits):
    """Zero gradients and states, eps 0 or not: 0 / (0 + eps)."""
    n = 700
    params, grads = Tensors(qc, [n], F32, 0).set(np.ones(n, np.float32)), Tensors(qc, [n], F32, 0).set(np.zeros(n, np.float32))
    nb = 3
    state = ([torch.zeros(n, device="cuda") for _ in range(2)] if bits == 32 else
             [torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(nb, device="cuda"),
              torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(nb, device="cuda")])
    call = qc.qc_adamw_multi if bits == 32 else qc.qc_adamw8_multi
    t = params.table
    call(t.xs, 0, grads.table.xs, 0, t.offsets, t.seg_first, 1, n, None, *state, step=1, **HYPER)
    assert (params.host() == np.float32(1 - 1e-3)).all()
    assert all(bool((s == 0).all()) for s in state)


def test_infinities_and_nans_stay_visible(qc):
    """A gradient that is not finite marks its element (fp32 states) or its
    block of states (8 bits), and no other."""
    n = 2000
    g = np.ones(n, np.float32)
    g[300], g[1500] = np.inf, np.nan
    for bits in (32, 8):
        params, grads = Tensors(qc, [n], F32, 1).set(np.ones(n, np.float32)), Tensors(qc, [n], F32, 1).set(g)
        t = params.table
        if bits == 32:
            m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
            qc.qc_adamw_multi(t.xs, 0, grads.table.xs, 0, t.offsets, t.seg_first, 1, n, None, m, v, step=1, **HYPER)
            bad = ~torch.isfinite(m).cpu().numpy()
            assert list(np.nonzero(bad)[0]) == [300, 1500] and np.array_equal(bad, ~torch.isfinite(v).cpu().numpy())
        else:
            mc, rc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
            ms, rs = (torch.zeros(8, device="cuda") for _ in range(2))
            qc.qc_adamw8_multi(t.xs, 0, grads.table.xs, 0, t.offsets, t.seg_first, 1, n, None, mc, ms, rc, rs, step=1,
                               **HYPER)
            out = torch.empty(n, device="cuda")
            for kind, codes, sc in ((qc.QC_STATE_M, mc, ms), (qc.QC_STATE_R, rc, rs)):
                assert list(np.nonzero(torch.isnan(sc).cpu().numpy())[0]) == [1, 5]
                qc.qc_decode_state8(kind, codes, sc, n, out, qc.QC_F32)
                nan = torch.isnan(out).cpu().numpy()
                assert nan[256:512].all() and nan[1280:1536].all() and nan.sum() == 512
        p = params.host()
        assert list(np.nonzero(np.isnan(p))[0]) == [300, 1500] and (p[~np.isnan(p)] < 1).all()


@pytest.mark.parametrize("name", ["one", "odd", "tiny_many", "mixed", "large", "parts"])
@pytest.mark.parametrize("gtype", [F32, BF16], ids=str)
def test_norm(qc, name, gtype):
    sizes = LISTS[name]
    n = sum(sizes)
    grads = Tensors(qc, sizes, gtype, gap=3).set(values(n, 5) + np.float32(0.5))
    want = math.sqrt((grads.host() ** 2).sum())
    t = grads.table
    work = torch.full((qc.qc_grad_norm_workspace(n),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((4,), 77.0, device="cuda")
    for most in (want / 3, want * 3, math.inf):
        qc.qc_grad_norm_multi(t.xs, qt(qc, gtype), t.offsets, t.seg_first, t.ntensors, n, most, work, out)
        norm, c, *rest = out.cpu().double().tolist()
        assert rest == [77.0, 77.0]
        assert abs(norm - want) <= 1.01 * U * want and abs(c - min(1.0, most / want)) <= 1.01 * U * c


def test_norm_of_large_small_and_not_finite_gradients(qc):
    n = 5000
    work = torch.empty(qc.qc_grad_norm_workspace(n), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, device="cuda")
    grads = Tensors(qc, [n], F32, 0)
    t = grads.table

    def norm(g):
        grads.set(g)
        qc.qc_grad_norm_multi(t.xs, 0, t.offsets, t.seg_first, 1, n, 2.0, work, out)
        return out.cpu().double().tolist()

    for value in (1e30, 1e-30, 0.0):  # squares that fp32 cannot hold
        got, c = norm(np.full(n, value, np.float32))
        want = float(np.float32(value)) * math.sqrt(n)
        assert abs(got - want) <= 1.01 * U * want
        assert abs(c - (min(1.0, 2.0 / want) if want else 1.0)) <= 1.01 * U
    for bad in (np.inf, -np.inf, np.nan):
        g = np.ones(n, np.float32)
        g[n - 1] = bad
        got, c = norm(g)
        assert not math.isfinite(got) and math.isnan(c)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_with_a_schedule(qc, bits):
    """Norm, clip and step in one graph, the step's number and rate on the
    device, replayed with new gradients between eager work."""
    sizes = [1000, 3, 4097, 500]
    n = sum(sizes)
    nb = -(-n // 256)
    start = values(n, 1)
    grads = Tensors(qc, sizes, F32, gap=1)
    sides = []
    for _ in range(2):  # the graph's and the eager one
        state = ([torch.zeros(n, device="cuda") for _ in range(2)] if bits == 32 else
                 [torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(nb, device="cuda"),
                  torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(nb, device="cuda")])
        sides.append((Tensors(qc, sizes, F32, gap=2).set(start), state,
                      torch.empty(qc.qc_grad_norm_workspace(n), dtype=torch.uint8, device="cuda"),
                      torch.empty(2, device="cuda")))
    schedule = torch.tensor([0.0, 0.0], device="cuda")
    call = qc.qc_adamw_multi if bits == 32 else qc.qc_adamw8_multi

    def run(side, lr, step, schedule):
        params, state, work, out = side
        t = params.table
        qc.qc_grad_norm_multi(grads.table.xs, 0, t.offsets, t.seg_first, t.ntensors, n, 1.0, work, out)
        call(t.xs, 0, grads.table.xs, 0, t.offsets, t.seg_first, t.ntensors, n, None, *state,
             **(HYPER | dict(lr=lr)), step=step, grad_scale=out[1:], schedule=schedule)

    grads.set(values(n, 2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(sides[0], 1e-2, 1, schedule)
    for step in range(1, 5):
        lr = float(np.float32(1e-2 / step))
        grads.set(values(n, 20 + step))
        schedule.copy_(torch.tensor([lr, float(step)]))
        graph.replay()
        torch.cuda.synchronize()
        run(sides[1], lr, step, None)
        torch.cuda.synchronize()
        (p, s, _, _), (q, r, _, _) = sides
        # the constants of the two ways differ by a rounding: a code may
        a, b = p.host(), q.host()
        assert (np.abs(a - b) <= 8 * U * np.abs(b) + (1e-2 * 16 * U if bits == 32 else 1e-2 * 0.2)).all()
        if bits == 32:
            assert all(torch.equal(x, y) for x, y in zip(s, r))
        else:
            assert (s[0] != r[0]).float().mean() < 1e-3 and (s[2] != r[2]).float().mean() < 1e-3


# ------------------------------------------------------------------- states


@pytest.mark.parametrize("signed", [True, False])
@pytest.mark.parametrize("n", [1, 7, 8, 255, 256, 257, 2048, 5001, 70000])
def test_state_codes(qc, n, signed):
    kind, k = (ref.M, qc.QC_STATE_M) if signed else (ref.R, qc.QC_STATE_R)
    x = values(n, n, spread=4.0)
    x = x if signed else np.abs(x)
    x[:: 97] *= np.float32(1e-30)
    codes = torch.full((n + 64,), 77, dtype=torch.uint8, device="cuda")
    scale = torch.full((-(-n // 256) + 64,), 77.0, device="cuda")
    qc.qc_encode_state8(k, torch.from_numpy(x).cuda(), n, codes, scale)
    nb = -(-n // 256)
    assert bool((codes[n:] == 77).all()) and bool((scale[nb:] == 77).all())
    c, s = codes[:n].cpu().numpy(), scale[:nb].cpu().numpy()
    want = ref.state_scale(kind, x.astype(np.float64))
    near(s.astype(np.float64), want, 2 * U * want)
    ref.check_codes(kind, c, s, x.astype(np.float64), np.full(n, 0.5), 0.0)
    for dtype in (F32, BF16):
        out = torch.full((n + 64,), 77.0, dtype=dtype, device="cuda")
        qc.qc_decode_state8(k, codes, scale, n, out, qt(qc, dtype))
        assert bool((out[n:] == 77).all())
        w = ref.state_values(kind, c, s)
        near(out[:n].double().cpu().numpy(), w, (U if dtype is F32 else U + 2.0 ** -8) * np.abs(w))
    # nearest: off by half a code of the value, or of the first code
    gap = 2.0 ** (kind.low - 23)
    w, s_ = ref.state_values(kind, c, s), np.repeat(s.astype(np.float64), 256)[:n]
    low = np.abs(x) < kind.least * s_
    off = np.abs(w - x)
    assert (off[~low] <= (gap / 2 * (1 + 1e-5)) * np.abs(x[~low]) + 1e-45).all()
    assert (off[low] <= (kind.least * s_ * (0.5 if signed else 1.0) * (1 + 1e-5))[low]).all()
    if not signed:
        assert (c[x > 0] > 0).all()


def test_state_of_every_code(qc):
    """What a code stands for is encoded as that code."""
    for kind, k in ((ref.M, qc.QC_STATE_M), (ref.R, qc.QC_STATE_R)):
        codes = torch.arange(256, dtype=torch.uint8, device="cuda")
        scale = torch.tensor([3.0], device="cuda")
        out = torch.empty(256, device="cuda")
        qc.qc_decode_state8(k, codes, scale, 256, out, qc.QC_F32)
        again, s2 = torch.empty_like(codes), torch.empty_like(scale)
        qc.qc_encode_state8(k, out, 256, again, s2)
        want = codes.clone()
        if kind.signed:
            want[128] = 0  # minus zero
        assert torch.equal(again, want) and abs(float(s2) - 3.0) < 1e-6


def test_states_of_blocks_that_are_zero_tiny_or_not_finite(qc):
    x = np.zeros((6, 256), np.float32)
    x[1] = 1e-40
    x[2, 17] = 2.0 ** -149
    x[3] = 3e38
    x[4, 3] = np.nan
    x[5, 255] = np.inf
    for kind, k in ((ref.M, qc.QC_STATE_M), (ref.R, qc.QC_STATE_R)):
        codes, scale = torch.empty(6 * 256, dtype=torch.uint8, device="cuda"), torch.empty(6, device="cuda")
        qc.qc_encode_state8(k, torch.from_numpy(x).cuda().view(-1), 6 * 256, codes, scale)
        s, c = scale.cpu().numpy(), codes.cpu().numpy().reshape(6, 256)
        assert s[0] == 0 and s[1] == s[2] == np.float32(2.0 ** -100) and np.isnan(s[4:]).all()
        assert not c[0].any() and not c[4:].any() and (c[3] == kind.top).all()
        assert (c[1] == (0 if kind.signed else 1)).all() and c[2].sum() == (0 if kind.signed else 1)


def test_slow_changes_are_followed(qc):
    """The gradient's size falls to a quarter in one element of a block: its r
    follows, though each step moves it by less than a code (v by 0.1 %, half
    a code is 6 % of v).  With steady g, v_t = g^2 + (v_0 - g^2) b2^t; a code
    covers up to 1/16 of r, and the thresholds of 400 steps leave it within
    two codes of that."""
    n = 256
    params = Tensors(qc, [n], F32, 0).set(np.zeros(n, np.float32))
    grads = Tensors(qc, [n], F32, 0)
    t = params.table
    x = np.ones(n, np.float32)
    mc, rc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, rs = (torch.zeros(1, device="cuda") for _ in range(2))
    qc.qc_encode_state8(qc.QC_STATE_R, torch.from_numpy(x).cuda(), n, rc, rs)
    g = x.copy()
    g[1::2] = 0.25
    grads.set(g)
    out = torch.empty(n, device="cuda")
    for step in range(1, 2001):
        qc.qc_adamw8_multi(t.xs, 0, grads.table.xs, 0, t.offsets, t.seg_first, 1, n, None, mc, ms, rc, rs, step=step,
                           **HYPER)
        if step % 500 == 0:
            qc.qc_decode_state8(qc.QC_STATE_R, rc, rs, n, out, qc.QC_F32)
            r = out.cpu().double().numpy()
            want = np.sqrt(g.astype(np.float64) ** 2 + (1 - g.astype(np.float64) ** 2) * 0.999 ** step)
            assert (np.abs(r / want - 1) <= 2 / 16).all()


def test_elements_past_32_bits(qc):
    """A list of more than 2^32 elements: its last tensor's are right."""
    sizes = [1 << 31, (1 << 31) + 77, 5000]
    n = sum(sizes)
    big = torch.zeros(max(sizes), dtype=BF16, device="cuda")  # the gradient of the two long ones: read only
    last_g, last_p = values(5000, 3), values(5000, 4)
    grads = [big[: sizes[0]], big[: sizes[1]], torch.from_numpy(last_g).cuda().to(BF16)]
    params = [torch.zeros(s, dtype=BF16, device="cuda") for s in sizes[:2]] + [torch.from_numpy(last_p).cuda().to(BF16)]
    gt, pt = qc.TensorTable(grads), qc.TensorTable(params)
    nb = -(-n // 256)
    mc, rc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, rs = (torch.zeros(nb, device="cuda") for _ in range(2))
    g, p = grads[2].double().cpu().numpy(), params[2].double().cpu().numpy()
    work, out = torch.empty(qc.qc_grad_norm_workspace(n), dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
    qc.qc_grad_norm_multi(gt.xs, 1, pt.offsets, pt.seg_first, 3, n, 1e9, work, out)
    want = math.sqrt((g ** 2).sum())
    assert abs(float(out[0]) - want) <= 1.01 * U * want
    qc.qc_adamw8_multi(pt.xs, 1, gt.xs, 1, pt.offsets, pt.seg_first, 3, n, None, mc, ms, rc, rs, step=1, **HYPER)
    p1, m1, v1, upd = ref.adamw(p, g, np.zeros(5000), np.zeros(5000), step=1, **HYPER)
    _, _, tol = tolerances(p, g, np.zeros(5000), np.zeros(5000), v1, upd, 1, 1.0)
    near(params[2].double().cpu().numpy(), p1, tol + 2.0 ** -8 * (np.abs(p1) + tol))
    # blocks that hold the last tensor alone
    first = (n - 5000 + 255) // 256 * 256
    at = first - (n - 5000)
    i = np.arange(first, n, dtype=np.uint64).astype(object)
    for kind, x, codes, sc, err in ((ref.M, m1, mc, ms, 4 * U), (ref.R, np.sqrt(v1), rc, rs, 4 * U)):
        u = np.asarray(ref.dither(kind, i, 1), np.float64)
        ref.check_codes(kind, codes[first:].cpu().numpy(), sc[first // 256:].cpu().numpy(), x[at:], u, err)
