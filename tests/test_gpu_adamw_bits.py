"""The AdamW step's 8-bit states bit for bit over every list of
test_gpu_adamw.py, and a step whose rate and number lie on the device against
the one that is given them."""
import numpy as np
import pytest
import torch

import mx_ref as ref
from gpu_util import need_gpu
from test_gpu_adamw import BF16, F32, HYPER, LISTS, U, Tensors, qt, saved, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qc():
    return need_gpu()


def stored(kind, codes, scale):
    """What codes stand for, in fp32 arithmetic."""
    mag = (codes & 127 if kind.signed else codes).astype(np.uint32)
    f = np.where(mag > 0, ((kind.first + mag) << kind.low).astype(np.uint32).view(np.float32), np.float32(0))
    f = np.where(kind.signed & (codes > 127), -f, f)
    return (ref.blocks(f) * scale[:, None]).reshape(-1)[: codes.size]


@pytest.mark.parametrize("gtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("name", LISTS)
def test_states_of_every_list(qc, name, gtype):
    """Three steps, the states carried on by the host: every code and scale is
    equal, those of an m near cancellation among them."""
    sizes = LISTS[name]
    n, nb = sum(sizes), -(-sum(sizes) // 256)
    weights = ("f32", "bf16", "master")[(list(LISTS).index(name) + (gtype is BF16)) % 3]
    ptype = F32 if weights == "f32" else BF16
    params, grads = Tensors(qc, sizes, ptype, 5).set(values(n, 1)), Tensors(qc, sizes, gtype, 3)
    master = torch.from_numpy(params.host().astype(np.float32)).cuda() if weights == "master" else None
    state = [torch.zeros(k, dtype=d, device="cuda") for k, d in ((n, torch.uint8), (nb, F32)) * 2]
    b1, b2, rest1, rest2 = (np.float32(x) for x in (0.9, 0.999, 1 - 0.9, 1 - 0.999))
    m, v = np.zeros(n, np.float32), np.zeros(n, np.float32)
    t, c = params.table, torch.tensor([0.37], device="cuda")
    for step in range(1, 4):
        grads.set(values(n, 40 + step))
        qc.qc_adamw8_multi(t.xs, qt(qc, ptype), grads.table.xs, qt(qc, gtype), t.offsets, t.seg_first, t.ntensors, n,
                           master, *state, step=step, grad_scale=c, **HYPER)
        x = grads.host().astype(np.float32) * np.float32(0.37)
        m, v = m * b1 + x * rest1, v * b2 + x * x * rest2
        want = [*saved(ref.M, m, step), *saved(ref.R, np.sqrt(v), step)]
        for got, w in zip(state, want):
            got = got.cpu().numpy()
            assert np.array_equal(got, w), (step, int((got != w).sum()))
        m, r = stored(ref.M, *want[:2]), stored(ref.R, *want[2:])
        v = r * r


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_from_the_device_is_the_step(qc, bits):
    """The states are equal bit for bit.  The weights' three constants come from
    64 bits that differ by far less than a step of fp32, so each is the same
    or its neighbour (2 half steps).  From the same weights and states p decay
    is apart by 4 of them (the constant, and a rounding on each side), the
    update by 16 (rate 2, its product 2, root 2, the sum with eps 2, two
    reciprocals within an ulp 4, the product 2, and 2 for what this bound
    takes from 64 bits), the difference by 2 of both."""
    sizes = LISTS["mixed"]
    n, nb = sum(sizes), -(-sum(sizes) // 256)
    call = qc.qc_adamw_multi if bits == 32 else qc.qc_adamw8_multi
    kinds = ((n, F32), (n, F32)) if bits == 32 else ((n, torch.uint8), (nb, F32)) * 2
    sides = [(Tensors(qc, sizes, F32, 2), [torch.zeros(k, dtype=d, device="cuda") for k, d in kinds]) for _ in range(2)]
    grads, schedule, p = Tensors(qc, sizes, F32, 1), torch.zeros(2, device="cuda"), values(n, 1)
    m, v = np.zeros(n), np.zeros(n)
    for step in (1, 2, 3, 100, 12345, 1 << 24):
        lr = float(np.float32(1e-2 / np.sqrt(step)))
        grads.set(values(n, step))
        schedule.copy_(torch.tensor([lr, float(step)]))
        for (params, state), on_device in zip(sides, (True, False)):
            params.set(p)
            t = params.table
            given = (0.5, 7) if on_device else (lr, step)  # what the device holds takes their place
            call(t.xs, 0, grads.table.xs, 0, t.offsets, t.seg_first, t.ntensors, n, None, *state,
                 **(HYPER | dict(lr=given[0])), step=given[1], schedule=schedule if on_device else None)
        for x, y in zip(*(s for _, s in sides)):
            assert torch.equal(x, y)
        a, b = (params.host() for params, _ in sides)
        g = grads.host()
        _, _, v1, _ = ref.adamw(p.astype(np.float64), g, m, v, **(HYPER | dict(lr=lr)), step=step)
        den = np.sqrt(v1 / (1 - 0.999 ** step)) + 1e-8
        update = lr / (1 - 0.9 ** step) * (0.9 * np.abs(m) + (1 - 0.9) * np.abs(g)) / den
        size = np.abs(p.astype(np.float64))
        assert (np.abs(a - b) <= U * (4 * size + 16 * update + 2 * (size + update)) + 2.0 ** -149).all()
        s = [x.cpu().numpy() for x in sides[0][1]]
        if bits == 32:
            m, v = (x.astype(np.float64) for x in s)
        else:
            m, v = ref.state_values(ref.M, s[0], s[1]), ref.state_values(ref.R, s[2], s[3]) ** 2
        p = a.astype(np.float32)
