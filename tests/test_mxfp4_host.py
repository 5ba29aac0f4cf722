"""Refusals of the 4-bit matrix operators and of the optimizer's entry points,
on the host: a bad argument is an error status, or an exception of the binding,
before any device work (no GPU is needed); and the 64-bit forms that they are
tested with, against hand-made values."""
import ctypes
import math

import numpy as np
import pytest
import torch

import mx_ref as ref
from test_matrix_binding_host import BF16, F16, F32, F64, I8, I32, U8, OnGpu, Reached
from test_matrix_host import A, qc, status  # noqa: F401

MIS = A + 4
BIG = 1 << 57
OK, ARG, ALIGN, UNSUP = 0, 1, 2, 3


def call(names, defaults):
    def make(**k):
        d = dict(defaults)
        assert set(k) <= set(d), k
        d.update(k)
        return [d[n] for n in names.split()] + [None]

    return make


ENCODE = call("x t rows dim ldx codes scales codes_t scales_t",
              dict(x=A, t=1, rows=3, dim=40, ldx=40, codes=A, scales=A, codes_t=A, scales_t=A))
DECODE = call("codes scales rows dim out t ldo", dict(codes=A, scales=A, rows=3, dim=40, out=A, t=1, ldo=40))
MATMUL = call("a sa b sb m n k c t ldc acc ws wb",
              dict(a=A, sa=A, b=A, sb=A, m=3, n=5, k=40, c=A, t=0, ldc=5, acc=0, ws=None, wb=0))
LINEAR = call("x xt ldx b sb m n k c t ldc ws wb",
              dict(x=A, xt=1, ldx=40, b=A, sb=A, m=3, n=5, k=40, c=A, t=1, ldc=5, ws=None, wb=0))
NORM = call("grads t off seg T n most ws wb out",
            dict(grads=A, t=0, off=A, seg=A, T=2, n=100, most=1.0, ws=A, wb=8, out=A))
HYPER = dict(lr=0.1, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=1, scale=A, sched=A)
LIST = dict(params=A, pt=1, grads=A, gt=0, off=A, seg=A, T=2, n=100, master=A)
ADAMW = call("params pt grads gt off seg T n master m v lr b1 b2 eps wd step scale sched",
             {**LIST, "m": A, "v": A, **HYPER})
ADAMW8 = call("params pt grads gt off seg T n master m ms r rs lr b1 b2 eps wd step scale sched",
              {**LIST, "m": A, "ms": A, "r": A, "rs": A, **HYPER})
ENC8 = call("kind x n codes scale", dict(kind=0, x=A, n=10, codes=A, scale=A))
DEC8 = call("kind codes scale n out t", dict(kind=1, codes=A, scale=A, n=10, out=A, t=0))

REFUSED = {
    ("qc_encode_mxfp4", ENCODE): [
        (ARG, [dict(x=None), dict(codes=None), dict(scales=None), dict(codes_t=None), dict(scales_t=None),
               dict(codes=None, scales=None, codes_t=None, scales_t=None), dict(t=2), dict(t=-1), dict(rows=-1),
               dict(dim=0), dict(ldx=39), dict(rows=BIG), dict(dim=BIG, ldx=BIG),
               dict(rows=1 << 31, dim=1 << 10, ldx=1 << 10), dict(rows=1 << 30, dim=40, ldx=40),
               dict(rows=1 << 31, dim=40, ldx=40, codes_t=None, scales_t=None)]),
        (ALIGN, [dict(x=A + 1), dict(t=0, x=A + 2), dict(codes=MIS), dict(scales=MIS), dict(codes_t=MIS),
                 dict(scales_t=MIS)]),
        (UNSUP, [dict(rows=1, dim=(1 << 34) + 1, ldx=(1 << 34) + 1), dict(rows=(1 << 34) + 1, dim=1, ldx=1)]),
        (OK, [dict(rows=0), dict(rows=0, x=None, codes=None)])],
    ("qc_decode_mxfp4", DECODE): [
        (ARG, [dict(codes=None), dict(scales=None), dict(out=None), dict(t=3), dict(rows=-1), dict(dim=0), dict(ldo=39)]),
        (ALIGN, [dict(codes=MIS), dict(scales=MIS), dict(out=A + 1), dict(t=0, out=A + 2)]),
        (UNSUP, [dict(rows=1, dim=(1 << 34) + 1, ldo=(1 << 34) + 1)]),
        (OK, [dict(rows=0, codes=None, scales=None, out=None)])],
    ("qc_matmul_mxfp4", MATMUL): [
        (ARG, [dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(c=None), dict(t=2), dict(m=-1), dict(n=-1),
               dict(k=0), dict(ldc=4), dict(m=BIG), dict(k=BIG), dict(m=1 << 31, n=1 << 31, ldc=1 << 31),
               dict(m=1, n=1 << 31, ldc=1 << 31), dict(m=130, n=120, ldc=120, k=30050),
               dict(m=130, n=120, ldc=120, k=30050, ws=A, wb=15 * 130 * 120 * 4 - 1)]),
        (ALIGN, [dict(a=MIS), dict(sa=MIS), dict(b=MIS), dict(sb=MIS), dict(c=A + 2), dict(t=1, c=A + 1),
                 dict(m=130, n=120, ldc=120, k=30050, ws=A + 8, wb=1 << 30)]),
        (UNSUP, [dict(t=1, acc=1), dict(k=(1 << 23) + 1)]),
        (OK, [dict(m=0), dict(n=0), dict(m=0, a=None, c=None)])],
    ("qc_linear_mxfp4", LINEAR): [
        (ARG, [dict(x=None), dict(b=None), dict(sb=None), dict(c=None), dict(t=2), dict(xt=2), dict(m=-1), dict(n=-1),
               dict(k=0), dict(ldc=4), dict(ldx=39), dict(m=BIG), dict(m=9), dict(m=9, ws=A, wb=255),
               dict(m=1, n=1 << 31, ldc=1 << 31), dict(m=1 << 26, k=1 << 12, ldx=1 << 12, n=1, ldc=1, ws=A, wb=1 << 60)]),
        (ALIGN, [dict(x=A + 1), dict(xt=0, x=A + 2), dict(b=MIS), dict(sb=MIS), dict(c=A + 1), dict(t=0, c=A + 2),
                 dict(m=9, ws=A + 8, wb=1 << 20)]),
        (UNSUP, [dict(k=(1 << 23) + 1, ldx=(1 << 23) + 1)]),
        (OK, [dict(m=0), dict(n=0), dict(m=0, x=None, c=None)])],
    ("qc_grad_norm_multi", NORM): [
        (ARG, [dict(grads=None), dict(off=None), dict(seg=None), dict(out=None), dict(ws=None), dict(wb=7), dict(t=2),
               dict(n=-1), dict(T=0), dict(most=0.0), dict(most=-1.0), dict(most=math.nan), dict(n=BIG, wb=1 << 62),
               dict(n=5000, wb=16)]),
        (ALIGN, [dict(grads=MIS), dict(off=MIS), dict(seg=A + 2), dict(ws=MIS), dict(out=A + 2)]),
        (OK, [dict(n=0), dict(n=0, grads=None, ws=None, wb=0, out=None)])],
}
STEP = [
    (ARG, [dict(params=None), dict(grads=None), dict(off=None), dict(seg=None), dict(pt=2), dict(gt=-1), dict(n=-1),
           dict(T=0), dict(pt=0), dict(lr=-1.0), dict(lr=math.inf), dict(lr=math.nan), dict(b1=1.0), dict(b1=-0.1),
           dict(b2=1.0), dict(b2=math.nan), dict(eps=-1e-9), dict(eps=math.inf), dict(eps=1e-39), dict(eps=5e-324), dict(wd=-0.1), dict(wd=math.nan),
           dict(step=0), dict(step=-5), dict(n=BIG), dict(m=None)]),
    (ALIGN, [dict(params=MIS), dict(grads=MIS), dict(off=MIS), dict(seg=A + 2), dict(master=MIS), dict(m=MIS),
             dict(scale=A + 2), dict(sched=A + 2)]),
    (OK, [dict(n=0), dict(n=0, params=None, m=None), dict(n=0, eps=0.0), dict(n=0, eps=2.0 ** -126)])]
REFUSED["qc_adamw_multi", ADAMW] = STEP + [(ARG, [dict(v=None)]), (ALIGN, [dict(v=MIS)])]
REFUSED["qc_adamw8_multi", ADAMW8] = STEP + [(ARG, [dict(ms=None), dict(r=None), dict(rs=None)]),
                                             (ALIGN, [dict(ms=MIS), dict(r=MIS), dict(rs=MIS)])]
REFUSED["qc_encode_state8", ENC8] = [
    (ARG, [dict(x=None), dict(codes=None), dict(scale=None), dict(n=-1), dict(n=BIG)]), (UNSUP, [dict(kind=2), dict(kind=-1)]),
    (ALIGN, [dict(x=MIS), dict(codes=MIS), dict(scale=MIS)]), (OK, [dict(n=0, x=None)])]
REFUSED["qc_decode_state8", DEC8] = [
    (ARG, [dict(out=None), dict(codes=None), dict(scale=None), dict(n=-1), dict(t=2)]), (UNSUP, [dict(kind=7)]),
    (ALIGN, [dict(out=MIS), dict(codes=MIS), dict(scale=MIS)]), (OK, [dict(n=0, out=None)])]


@pytest.mark.parametrize("fn,make,want,kw", [(f, m, w, kw) for (f, m), rows in REFUSED.items() for w, kws in rows
                                             for kw in kws], ids=lambda v: str(v) if isinstance(v, (dict, int)) else None)
def test_refused(qc, fn, make, want, kw):  # noqa: F811
    assert status(qc, fn, *make(**kw)) == want


def test_sizes(qc):  # noqa: F811
    for rows, dim, cb, sb in ((3, 1, 16, 4), (3, 32, 16, 4), (3, 33, 32, 4), (3, 128, 64, 4), (3, 129, 80, 8), (0, 7, 16, 4)):
        assert qc.mxfp4_bytes(rows, dim) == (rows * cb, rows * sb)
    c = ctypes.c_int64(-7)
    for rows, dim in ((-1, 8), (1, 0), (1 << 57, 8), (1, 1 << 57)):
        assert qc.lib().qc_mxfp4_bytes(rows, dim, ctypes.byref(c), ctypes.byref(c)) == ARG and c.value == -7
    L = qc.lib()
    for args in ((-1, 8, 8), (8, -1, 8), (8, 8, 0), (BIG, 8, 8), (1, 1 << 31, 8)):
        assert L.qc_matmul_mxfp4_workspace(*args) == -1 and L.qc_linear_mxfp4_workspace(*args, 0) == -1
        with pytest.raises(qc.QcError):
            qc.qc_matmul_mxfp4_workspace(*args)
    assert L.qc_linear_mxfp4_workspace(8, 8, 8, 5) == -1
    assert qc.qc_matmul_mxfp4_workspace(0, 5, 40) == qc.qc_linear_mxfp4_workspace(0, 5, 40, 0) == 0
    assert L.qc_grad_norm_workspace(-1) == -1 and qc.qc_grad_norm_workspace(0) == 0
    assert qc.qc_grad_norm_workspace(1) == qc.qc_grad_norm_workspace(2048) == 8 and qc.qc_grad_norm_workspace(2049) == 16
    assert qc.qc_grad_norm_workspace(1 << 40) <= 8 * 2048


# ----------------------------------------------------------------- binding


class Elsewhere(OnGpu):
    def get_device(self):
        return 0


def test_workspace_of_rows_that_are_too_long(qc):  # noqa: F811
    """As many bytes as the product would refuse to use: none, and no arithmetic on a length past 32 bits."""
    L = qc.lib()
    for k in ((1 << 23) + 1, 1 << 32, 1 << 45, 1 << 56):
        assert L.qc_matmul_mxfp4_workspace(1, 1, k) == L.qc_linear_mxfp4_workspace(1, 1, k, 0) == -1, k
        assert L.qc_matmul_mxfp4_workspace(0, 1, k) == L.qc_linear_mxfp4_workspace(1, 0, k, 0) == 0
    assert L.qc_matmul_mxfp4_workspace(1, 1, 1 << 23) >= 0


def test_one_launch_takes_fewer_than_2_to_the_32_threads(qc):  # noqa: F811
    """A few tokens are encoded by the blocks that multiply them, 512 threads
    for 16 channels, as far as one launch goes; then by a launch of their own."""
    most = 16 * ((1 << 23) - 1)
    for m in (1, 4, 8):
        assert qc.qc_linear_mxfp4_workspace(m, most, 32, 1) == 0
        assert qc.qc_linear_mxfp4_workspace(m, most + 1, 32, 1) == 512


def T(shape, dtype, device=0):
    t = Elsewhere(torch.zeros(shape, dtype=dtype))
    t.get_device = lambda: device
    return t


@pytest.fixture()
def bound(qc, monkeypatch):  # noqa: F811
    class Lib:
        def __getattr__(self, name):
            def reached(*args):
                raise Reached(name)

            return reached

    monkeypatch.setattr(qc.binding, "lib", Lib)
    monkeypatch.setattr(qc.binding, "_now", lambda: 0)
    return qc


def arguments(**k):
    """Tensors that a call of each kind takes, some of them replaced."""
    d = dict(x=T((3, 40), BF16), codes=T(3 * 32, U8), scales=T(3 * 4, U8), codes_t=T(40 * 16, U8), scales_t=T(40 * 4, U8),
             b=T(5 * 32, U8), b_scales=T(5 * 4, U8), c=T((3, 5), BF16), workspace=T(64, U8), params=T(2, torch.int64),
             grads=T(2, torch.int64), offsets=T(3, torch.int64), seg_first=T(2, I32), master=T(100, F32), m=T(100, F32),
             v=T(100, F32), m_codes=T(100, U8), m_scale=T(1, F32), r_codes=T(100, U8), r_scale=T(1, F32),
             grad_scale=T(1, F32), schedule=T(2, F32), out=T(2, F32), flat=T(100, BF16), wide=T(100, F32))
    d.update(k)
    return d


TABLES = lambda d: (d["offsets"], d["seg_first"], 2, 100)  # noqa: E731
RATES = dict(lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1)
CALLS = {
    "encode": (lambda q, d: q.qc_encode_mxfp4(d["x"], 1, 3, 40, 40, d["codes"], d["scales"], d["codes_t"], d["scales_t"],
                                              stream=0), "x codes scales codes_t scales_t"),
    "decode": (lambda q, d: q.qc_decode_mxfp4(d["codes"], d["scales"], 3, 40, d["x"], 1, 40, stream=0), "codes scales x"),
    "matmul": (lambda q, d: q.qc_matmul_mxfp4(d["codes"], d["scales"], d["b"], d["b_scales"], 3, 5, 40, d["c"], 1, 5, False,
                                              d["workspace"], stream=0), "codes scales b b_scales c"),
    "linear": (lambda q, d: q.qc_linear_mxfp4(d["x"], 1, 40, d["b"], d["b_scales"], 3, 5, 40, d["c"], 1, 5, d["workspace"],
                                              stream=0), "x b b_scales c"),
    "norm": (lambda q, d: q.qc_grad_norm_multi(d["grads"], 0, *TABLES(d), 1.0, d["workspace"], d["out"], stream=0),
             "grads offsets seg_first out"),
    "adamw": (lambda q, d: q.qc_adamw_multi(d["params"], 1, d["grads"], 0, *TABLES(d), d["master"], d["m"], d["v"],
                                            grad_scale=d["grad_scale"], schedule=d["schedule"], stream=0, **RATES),
              "params grads offsets seg_first master m v grad_scale schedule"),
    "adamw8": (lambda q, d: q.qc_adamw8_multi(d["params"], 1, d["grads"], 0, *TABLES(d), d["master"], d["m_codes"],
                                              d["m_scale"], d["r_codes"], d["r_scale"], grad_scale=d["grad_scale"],
                                              schedule=d["schedule"], stream=0, **RATES),
               "params grads offsets seg_first master m_codes m_scale r_codes r_scale"),
    "encode8": (lambda q, d: q.qc_encode_state8(0, d["wide"], 100, d["m_codes"], d["m_scale"], stream=0),
                "wide m_codes m_scale"),
    "decode8": (lambda q, d: q.qc_decode_state8(1, d["r_codes"], d["r_scale"], 100, d["flat"], 1, stream=0),
                "r_codes r_scale flat"),
}
ARGUMENTS = [(c, a) for c, (_, names) in CALLS.items() for a in names.split()]
UNTYPED = ("params", "grads", "offsets", "seg_first")  # tables: their bytes are checked


@pytest.mark.parametrize("name", CALLS)
def test_right_tensors_pass(bound, name):
    with pytest.raises(Reached):
        CALLS[name][0](bound, arguments())


@pytest.mark.parametrize("name,arg", ARGUMENTS)
def test_tensor_too_small(bound, name, arg):
    t = arguments()[arg]
    small = T((2, 40) if arg == "x" else (2, 5) if arg == "c" else t.numel() - 1, t.dtype)
    with pytest.raises(ValueError):
        CALLS[name][0](bound, arguments(**{arg: small}))


@pytest.mark.parametrize("name,arg", [p for p in ARGUMENTS if p[1] not in UNTYPED])
@pytest.mark.parametrize("dtype", [F16, F64, I32], ids=str)
def test_tensor_of_another_type(bound, name, arg, dtype):
    with pytest.raises(ValueError, match="is a tensor of"):
        CALLS[name][0](bound, arguments(**{arg: T(arguments()[arg].shape, dtype)}))


@pytest.mark.parametrize("name,arg", ARGUMENTS + [("matmul", "workspace"), ("linear", "workspace"), ("norm", "workspace")])
def test_tensor_of_another_device(bound, name, arg):
    t = arguments()[arg]
    with pytest.raises(ValueError, match="is on GPU 1, the current one is 0"):
        CALLS[name][0](bound, arguments(**{arg: T(t.shape, t.dtype, device=1)}))


@pytest.mark.parametrize("name,arg", ARGUMENTS)
def test_host_tensor(bound, name, arg):
    t = arguments()[arg]
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        CALLS[name][0](bound, arguments(**{arg: torch.zeros(t.shape, dtype=t.dtype)}))


def test_raw_workspace_is_refused(bound):
    for name in ("matmul", "linear", "norm"):
        with pytest.raises(ValueError, match="workspace must be a GPU tensor"):
            CALLS[name][0](bound, arguments(workspace=A))


# -------------------------------------------------------------- references


def test_reference_of_encoding():
    x = torch.tensor([[6.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.1, -0.0, 0.2]])
    codes, scales = ref.encode(x)
    assert scales.tolist() == [[127, 0, 0, 0]]
    nibbles = [v for b in codes[0, :6] for v in (b & 15, b >> 4)]
    assert nibbles == [7, 0, 1, 2, 2, 4, 4, 6, 6, 15, 8, 0] and not codes[0, 6:].any()
    assert ref.held(codes, scales, 12).tolist() == [[6, 0, .5, 1, 1, 2, 2, 4, 4, -6, 0, 0]]
    for top, byte in ((6.99, 127), (7.0, 128), (3.49, 126), (3.5, 127), (0.0, 1), (2.0 ** -140, 1), (3.4e38, 253)):
        assert ref.encode(torch.tensor([[top]]))[1][0, 0] == byte
    assert ref.encode(torch.tensor([[math.inf, 1.0]]))[1][0, 0] == 255


def test_reference_of_states():
    assert ref.M.largest == 1.875 and ref.R.largest == 1.9375
    assert ref.M.least == 1.125 * 2 ** -15 and ref.R.least == 1.0625 * 2 ** -15
    codes = np.array([127, 255, 0, 1, 129], np.uint8)
    assert ref.state_values(ref.M, codes, np.array([2.0], np.float32)).tolist() == [3.75, -3.75, 0, ref.M.least * 2,
                                                                                    -ref.M.least * 2]
    # a planted mistake in a code is found, one at a border is not
    x = np.linspace(0.1, 1.875, 256)
    s = np.array([1.0], np.float32)
    gap = 2.0 ** np.floor(np.log2(x)) / 8
    good = (np.floor(x / gap + 0.5) * gap)
    c = (good.astype(np.float32).view(np.uint32) >> 20).astype(np.int64) - 896
    ref.check_codes(ref.M, np.minimum(c, 127).astype(np.uint8), s, x, np.full(256, 0.5), 1e-7)
    c[100] += 1
    with pytest.raises(AssertionError):
        ref.check_codes(ref.M, np.minimum(c, 127).astype(np.uint8), s, x, np.full(256, 0.5), 1e-7)


def test_thresholds_cover_the_unit_interval():
    """For an element, over steps; and over neighbouring elements."""
    for u in (ref.dither(ref.M, 12345, np.arange(1, 1001, dtype=np.int64)),
              ref.dither(ref.R, np.arange(1000, dtype=np.int64), 7)):
        gaps = np.diff(np.sort(np.concatenate([u, [u.min() + 1]])))
        assert (u >= 0).all() and (u < 1).all() and gaps.max() < 4e-3


def test_reference_of_a_step_against_torch():
    p, g = torch.randn(50, dtype=torch.float64), torch.randn(50, dtype=torch.float64)
    w = p.clone().requires_grad_()
    opt = torch.optim.AdamW([w], lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    q, m, v = p.numpy(), np.zeros(50), np.zeros(50)
    for step in range(1, 5):
        w.grad = g * step
        opt.step()
        q, m, v, _ = ref.adamw(q, g.numpy() * step, m, v, 1e-2, 0.9, 0.99, 1e-8, 0.1, step)
    assert np.allclose(q, w.detach().numpy(), rtol=1e-12, atol=1e-14)
