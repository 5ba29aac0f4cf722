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
