"""What the binding of the matrix operators refuses of tensors, on the host
(stand-ins carry a tensor's metadata; no call gets as far as the device)."""
import pytest
import torch

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
I8, U8, I16, I32 = torch.int8, torch.uint8, torch.int16, torch.int32


class OnGpu:
    """The metadata of a host tensor, said to be on a GPU."""

    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)


def T(shape, dtype):
    return OnGpu(torch.zeros(shape, dtype=dtype))


class Reached(Exception):
    """The library was called: nothing was refused."""


@pytest.fixture()
def qc(monkeypatch):
    import embedding_communication_codecs_amd as q

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                raise Reached(name)

            return call

    monkeypatch.setattr(q.binding, "lib", Lib)
    return q


def encode_int8(qc, x=F32, codes=I8, scale=F32, t=0):
    qc.qc_encode_int8_rowwise(T((3, 40), x), t, 3, 40, 40, T((3, 48), codes), 48, T(3, scale), stream=0)


def matmul(qc, a=I8, sa=F32, b=I8, sb=F32, c=F32, t=0):
    qc.qc_matmul_int8(T((3, 48), a), T(3, sa), 48, T((5, 48), b), T(5, sb), 48, 3, 5, 40, T((3, 5), c), t, 5, stream=0)


def encode_ckpt(qc, x=F32, codes=I8, exps=U8, t=0):
    qc.qc_encode_ckpt8(T((3, 40), x), t, 3, 40, 40, T((3, 64), codes), T((3, 4), exps), stream=0)


def decode_ckpt(qc, out=F32, codes=I8, exps=U8, t=0):
    qc.qc_decode_ckpt8(T((3, 64), codes), T((3, 4), exps), 3, 40, T((3, 40), out), t, 40, stream=0)


def wgrad(qc, dy=F32, codes=I8, exps=U8, dw=F32, t=0, wt=0):
    qc.qc_ckpt8_wgrad(T((3, 5), dy), t, 5, T((3, 64), codes), T((3, 4), exps), 3, 5, 40, T((5, 40), dw), wt, 40, False,
                      None, stream=0)


def swiglu(qc, gate=F32, up=F32, h=F32, codes=I8, exps=U8, t=0):
    m = lambda d: T((3, 40), d)  # noqa: E731
    kept = lambda: (T((3, 64), codes), T((3, 4), exps))  # noqa: E731
    qc.qc_swiglu_ckpt8(m(gate), m(up), t, 40, 3, 40, m(h), 40, *kept(), *kept(), stream=0)


def swiglu_backward(qc, dh=F32, dgate=F32, dup=F32, codes=I8, exps=U8, t=0):
    m = lambda d: T((3, 40), d)  # noqa: E731
    kept = lambda: (T((3, 64), codes), T((3, 4), exps))  # noqa: E731
    qc.qc_swiglu_ckpt8_backward(m(dh), t, 40, *kept(), *kept(), 3, 40, m(dgate), m(dup), 40, stream=0)


MATRICES = {encode_int8: ["x"], matmul: ["c"], encode_ckpt: ["x"], decode_ckpt: ["out"], wgrad: ["dy"],
            swiglu: ["gate", "up", "h"], swiglu_backward: ["dh", "dgate", "dup"]}
CALLS = list(MATRICES)
NAME = lambda v: v.__name__ if callable(v) else str(v)  # noqa: E731


@pytest.mark.parametrize("call", CALLS, ids=NAME)
def test_right_types_pass(qc, call):
    with pytest.raises(Reached):
        call(qc)
    with pytest.raises(Reached):
        call(qc, **{m: BF16 for m in MATRICES[call]}, t=1)


@pytest.mark.parametrize("said,dtype", [(1, F16), (1, I16), (0, I32), (1, F32), (0, BF16), (0, F64)], ids=NAME)
@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in MATRICES[c]], ids=NAME)
def test_matrix_of_another_type(qc, call, name, said, dtype):
    kw = {m: BF16 if said == 1 else F32 for m in MATRICES[call]}
    kw[name] = dtype
    with pytest.raises(ValueError, match=rf"{name} is a tensor of {dtype}"):
        call(qc, **kw, t=said)


@pytest.mark.parametrize("wt,dtype", [(1, F16), (0, I32)])
def test_wgrad_output_of_another_type(qc, wt, dtype):
    with pytest.raises(ValueError, match="dw is a tensor of"):
        wgrad(qc, dw=dtype, wt=wt)


@pytest.mark.parametrize("call,name", [(encode_int8, "scale"), (matmul, "sa"), (matmul, "sb")], ids=NAME)
@pytest.mark.parametrize("dtype", [F64, I32, F16], ids=NAME)
def test_scales_of_another_type(qc, call, name, dtype):
    with pytest.raises(ValueError, match="scale is a tensor of"):
        call(qc, **{name: dtype})


@pytest.mark.parametrize("call,name", [(encode_int8, "codes"), (matmul, "a"), (matmul, "b"),
                                       *[(c, n) for c in CALLS[2:] for n in ("codes", "exps")]], ids=NAME)
def test_codes_of_another_type(qc, call, name):
    for dtype in (torch.bool, torch.float8_e4m3fn, I16, F32):
        with pytest.raises(ValueError, match="is a tensor of"):
            call(qc, **{name: dtype})
    for dtype in (I8, U8):
        with pytest.raises(Reached):
            call(qc, **{name: dtype})


def out(qc, t, rows=3, dim=40, ldo=40):
    qc.qc_decode_ckpt8(T((rows, 64), I8), T((rows, 4), U8), rows, dim, OnGpu(t), 0, ldo, stream=0)


@pytest.mark.parametrize("view,ldo", [
    (lambda: torch.zeros(9, 40)[:2], 40),             # a row short; there are rows below
    (lambda: torch.zeros(9, 64)[:, :39], 64),         # a column short; there are columns beside
    (lambda: torch.zeros(9, 64)[2:4, 8:48], 64),
    (lambda: torch.zeros(500)[100:219], 40),          # an element short, flat
    (lambda: torch.zeros(500)[100:219].view(1, 119), 40),
    (lambda: torch.zeros(9, 2, 20)[:2], 40),
    (lambda: torch.zeros(500)[:0], 40),
    (lambda: torch.zeros(500)[7], 40),
], ids=str)
def test_views_smaller_than_the_call(qc, view, ldo):
    """What lies beside a view is not the call's to write."""
    with pytest.raises(ValueError, match="out holds"):
        out(qc, view(), ldo=ldo)


@pytest.mark.parametrize("view,ldo", [
    (lambda: torch.zeros(9, 40)[4:7], 40), (lambda: torch.zeros(9, 64)[:3, 8:48], 64),
    (lambda: torch.zeros(500)[100:220], 40), (lambda: torch.zeros(500)[100:268], 64),
    (lambda: torch.zeros(1, 500)[:, :120], 40), (lambda: torch.zeros(3, 2, 20), 40),
], ids=str)
def test_views_large_enough_pass(qc, view, ldo):
    with pytest.raises(Reached):
        out(qc, view(), ldo=ldo)


def test_codes_without_their_padding(qc):
    """Codes may be a view that ends at k, where the padding up to 16 lies behind it in the same rows."""
    a, b = torch.zeros((3, 48), dtype=I8), torch.zeros((5, 64), dtype=I8)

    def args(a, b, m=3):
        return OnGpu(a), T(4, F32), 48, OnGpu(b), T(5, F32), 64, m, 5, 40, T((4, 5), F32), 0, 5

    with pytest.raises(Reached):
        qc.qc_matmul_int8(*args(a[:, :40], b[:, :40]), stream=0)
    with pytest.raises(ValueError, match="a holds"):  # the last row's padding is not there
        qc.qc_matmul_int8(*args(torch.zeros(3 * 48 - 8, dtype=I8).as_strided((3, 40), (48, 1)), b), stream=0)
    with pytest.raises(ValueError, match="a holds"):
        qc.qc_matmul_int8(*args(torch.zeros((9, 48), dtype=I8)[:3, :40], b, 4), stream=0)
    with pytest.raises(ValueError, match="a holds"):
        qc.qc_matmul_int8(*args(a[:, :39], b), stream=0)
