"""Refusals of the matrix operators, on the host: a bad argument is an error
status before any device work (no GPU is needed), and the 64-bit reference
they are tested with against hand-made values."""
import ctypes

import numpy as np
import pytest
import torch

import matrix_ref as ref

BIG = 1 << 57


@pytest.fixture(scope="module")
def qc():
    import os

    import embedding_communication_codecs_amd as q

    if not os.path.exists(q.binding.LIB_PATH):
        pytest.skip("libqc.so not built (python -m embedding_communication_codecs_amd.build)")
    q.lib()
    return q


def status(qc, fn, *args):
    return getattr(qc.lib(), fn)(*args)


A = 0x1000  # an aligned address; never read, as every call here is refused or empty


def enc_int8(**k):
    d = dict(x=A, t=1, rows=3, dim=40, ldx=40, codes=A, ldq=48, scale=A)
    d.update(k)
    return [d[n] for n in ("x", "t", "rows", "dim", "ldx", "codes", "ldq", "scale")] + [None]


def matmul(**k):
    d = dict(a=A, sa=A, lda=48, b=A, sb=A, ldb=48, m=3, n=5, k=40, c=A, t=1, ldc=5)
    d.update(k)
    return [d[n] for n in ("a", "sa", "lda", "b", "sb", "ldb", "m", "n", "k", "c", "t", "ldc")] + [None]


def enc_ckpt(**k):
    d = dict(x=A, t=1, rows=3, dim=40, ldx=40, codes=A, exps=A)
    d.update(k)
    return [d[n] for n in ("x", "t", "rows", "dim", "ldx", "codes", "exps")] + [None]


def dec_ckpt(**k):
    d = dict(codes=A, exps=A, rows=3, dim=40, out=A, t=1, ldo=40)
    d.update(k)
    return [d[n] for n in ("codes", "exps", "rows", "dim", "out", "t", "ldo")] + [None]


def wgrad(**k):
    d = dict(dy=A, t=1, ldy=5, codes=A, exps=A, rows=3, n=5, dim=40, dw=A, wt=0, ldw=40, acc=0, ws=None, wb=0)
    d.update(k)
    return [d[n] for n in ("dy", "t", "ldy", "codes", "exps", "rows", "n", "dim", "dw", "wt", "ldw", "acc", "ws",
                           "wb")] + [None]


def swiglu(**k):
    d = dict(g=A, u=A, t=1, ldx=40, rows=3, dim=40, h=A, ldh=40, gc=A, ge=A, uc=A, ue=A)
    d.update(k)
    return [d[n] for n in ("g", "u", "t", "ldx", "rows", "dim", "h", "ldh", "gc", "ge", "uc", "ue")] + [None]


def swiglu_bwd(**k):
    d = dict(dh=A, t=1, lddh=40, gc=A, ge=A, uc=A, ue=A, rows=3, dim=40, dg=A, du=A, ldg=40)
    d.update(k)
    return [d[n] for n in ("dh", "t", "lddh", "gc", "ge", "uc", "ue", "rows", "dim", "dg", "du", "ldg")] + [None]


OK, ARG, ALIGN, UNSUP = 0, 1, 2, 3

REFUSED = [
    *[("qc_encode_int8_rowwise", enc_int8, kw, st) for kw, st in [
        (dict(x=None), ARG), (dict(codes=None), ARG), (dict(scale=None), ARG), (dict(t=2), ARG), (dict(t=-1), ARG),
        (dict(rows=-1), ARG), (dict(dim=0), ARG), (dict(dim=-3), ARG), (dict(ldx=39), ARG), (dict(ldq=32), ARG),
        (dict(ldq=40), ARG), (dict(rows=BIG), ARG), (dict(ldx=BIG), ARG), (dict(rows=0, dim=0), ARG),
        (dict(x=A + 1), ALIGN), (dict(t=0, x=A + 2), ALIGN), (dict(codes=A + 8), ALIGN), (dict(scale=A + 2), ALIGN),
        (dict(rows=0, x=None, codes=None, scale=None), OK)]],
    *[("qc_matmul_int8", matmul, kw, st) for kw, st in [
        (dict(a=None), ARG), (dict(sa=None), ARG), (dict(b=None), ARG), (dict(sb=None), ARG), (dict(c=None), ARG),
        (dict(t=5), ARG), (dict(m=-1), ARG), (dict(n=-1), ARG), (dict(k=0), ARG), (dict(k=-2), ARG),
        (dict(lda=32), ARG), (dict(ldb=40), ARG), (dict(ldc=4), ARG), (dict(m=1 << 50), ARG), (dict(m=1 << 36), ARG),
        (dict(k=131072, lda=131072, ldb=131072), UNSUP), (dict(lda=(1 << 23) + 16), UNSUP),
        (dict(ldb=(1 << 23) + 16), UNSUP), (dict(a=A + 4), ALIGN), (dict(b=A + 8), ALIGN), (dict(sa=A + 1), ALIGN),
        (dict(sb=A + 2), ALIGN), (dict(c=A + 1), ALIGN), (dict(c=A + 2, t=0), ALIGN),
        (dict(m=0, a=None, sa=None, c=None), OK), (dict(n=0, b=None, sb=None, c=None, ldc=0), OK)]],
    *[("qc_encode_ckpt8", enc_ckpt, kw, st) for kw, st in [
        (dict(x=None), ARG), (dict(codes=None), ARG), (dict(exps=None), ARG), (dict(t=3), ARG), (dict(rows=-1), ARG),
        (dict(dim=0), ARG), (dict(ldx=39), ARG), (dict(rows=BIG), ARG), (dict(x=A + 1), ALIGN),
        (dict(x=A + 2, t=0), ALIGN), (dict(codes=A + 4), ALIGN), (dict(exps=A + 4), ALIGN),
        (dict(rows=0, x=None), OK)]],
    *[("qc_decode_ckpt8", dec_ckpt, kw, st) for kw, st in [
        (dict(codes=None), ARG), (dict(exps=None), ARG), (dict(out=None), ARG), (dict(t=3), ARG), (dict(rows=-1), ARG),
        (dict(dim=0), ARG), (dict(ldo=39), ARG), (dict(out=A + 1), ALIGN), (dict(codes=A + 4), ALIGN),
        (dict(exps=A + 4), ALIGN), (dict(rows=0, out=None), OK)]],
    *[("qc_ckpt8_wgrad", wgrad, kw, st) for kw, st in [
        (dict(dy=None), ARG), (dict(codes=None), ARG), (dict(exps=None), ARG), (dict(dw=None), ARG), (dict(t=3), ARG),
        (dict(wt=3), ARG), (dict(rows=-1), ARG), (dict(n=-1), ARG), (dict(dim=0), ARG), (dict(ldy=4), ARG),
        (dict(ldw=39), ARG), (dict(rows=BIG), ARG), (dict(n=BIG), ARG), (dict(dim=BIG, ldw=BIG), ARG),
        (dict(wt=1, acc=1), UNSUP), (dict(ldy=(1 << 23) + 8), UNSUP),
        (dict(dim=(1 << 23) + 32, ldw=(1 << 23) + 32), UNSUP), (dict(dy=A + 1), ALIGN),
        (dict(dw=A + 2), ALIGN), (dict(codes=A + 8), ALIGN), (dict(exps=A + 8), ALIGN),
        (dict(rows=1 << 16), ARG), (dict(rows=1 << 16, ws=A, wb=16), ARG),  # too little workspace
        (dict(rows=1 << 16, ws=A + 8, wb=1 << 40), ALIGN),
        (dict(n=0, dy=None, dw=None, ldy=0), OK)]],
    *[("qc_swiglu_ckpt8", swiglu, kw, st) for kw, st in [
        *[({n: None}, ARG) for n in ("g", "u", "h", "gc", "ge", "uc", "ue")],
        (dict(t=2), ARG), (dict(rows=-1), ARG), (dict(dim=0), ARG), (dict(ldx=39), ARG), (dict(ldh=39), ARG),
        (dict(g=A + 1), ALIGN), (dict(u=A + 1), ALIGN), (dict(h=A + 2, t=0), ALIGN),
        *[({n: A + 8}, ALIGN) for n in ("gc", "ge", "uc", "ue")], (dict(rows=0, g=None), OK)]],
    *[("qc_swiglu_ckpt8_backward", swiglu_bwd, kw, st) for kw, st in [
        *[({n: None}, ARG) for n in ("dh", "gc", "ge", "uc", "ue", "dg", "du")],
        (dict(t=2), ARG), (dict(rows=-1), ARG), (dict(dim=0), ARG), (dict(lddh=39), ARG), (dict(ldg=39), ARG),
        (dict(dh=A + 1), ALIGN), (dict(dg=A + 1), ALIGN), (dict(du=A + 2, t=0), ALIGN),
        *[({n: A + 8}, ALIGN) for n in ("gc", "ge", "uc", "ue")], (dict(rows=0, dh=None), OK)]],
]


@pytest.mark.parametrize("fn,args,kw,want", REFUSED, ids=lambda v: str(v) if isinstance(v, (str, dict)) else "")
def test_refusals(qc, fn, args, kw, want):
    if want == OK:  # empty calls only: nothing may reach the device here
        assert any(kw.get(k) == 0 for k in ("rows", "m", "n"))
    assert status(qc, fn, *args(**kw)) == want


def test_ckpt8_bytes(qc):
    for rows, dim in ((0, 1), (1, 1), (3, 31), (3, 32), (3, 33), (7, 128), (7, 129), (1000, 4097)):
        assert qc.ckpt8_bytes(rows, dim) == (rows * ref.up(dim, 32), rows * ref.up(dim, 128) // 32)
    c = ctypes.c_int64()
    for rows, dim in ((-1, 8), (1, 0), (BIG, 8), (1, BIG)):
        assert qc.lib().qc_ckpt8_bytes(rows, dim, ctypes.byref(c), ctypes.byref(c)) == ARG
    assert qc.lib().qc_ckpt8_bytes(1, 1, None, ctypes.byref(c)) == ARG


def test_wgrad_workspace(qc):
    assert qc.qc_ckpt8_wgrad_workspace(0, 64, 64, qc.QC_BF16) == 0
    assert qc.qc_ckpt8_wgrad_workspace(1, 64, 64, qc.QC_BF16) == 0
    assert qc.qc_ckpt8_wgrad_workspace(4096, 0, 64, qc.QC_BF16) == 0
    few = qc.qc_ckpt8_wgrad_workspace(1 << 16, 64, 65, qc.QC_BF16)
    assert few > 0 and few % (64 * 68 * 4) == 0  # whole fp32 matrices of a pitch of 68
    for bad in ((-1, 8, 8, 0), (8, -1, 8, 0), (8, 8, 0, 0), (8, 8, 8, 7), (BIG, 8, 8, 0)):
        with pytest.raises(qc.QcError):
            qc.qc_ckpt8_wgrad_workspace(*bad)


def test_binding_refuses_small_or_wrong_tensors(qc):
    x = torch.zeros((3, 40))
    with pytest.raises(ValueError, match="GPU"):
        qc.qc_encode_int8_rowwise(x, qc.QC_F32, 3, 40, 40, A, 48, A, stream=0)


# --------------------------------------------------------- the reference


def test_reference_int8_rows():
    q, s = ref.int8_rows(torch.tensor([[127.0, -1.0, 0.5, 1.5, -2.5], [0.0] * 5, [1.0, np.inf, 0, 0, 0]]))
    assert q[0].tolist() == [127, -1, 0, 2, -2] and s[0] == 1.0
    assert q[1].tolist() == [0] * 5 and s[1] == 0.0
    assert q[2].tolist() == [0] * 5 and np.isnan(s[2])


def test_reference_checkpoint():
    x = torch.zeros((1, 160))
    x[0, 0], x[0, 1], x[0, 32], x[0, 64], x[0, 96], x[0, 128] = 127.0, 0.5, 127.5, 2.0 ** -149, 2.0 ** 127, np.nan
    q, e = ref.ckpt8(x)
    assert q.shape == (1, 160) and e.shape == (1, 8)
    assert (q[0, 0], q[0, 1], e[0, 0]) == (127, 0, 127)      # 127 = 127 * 2^0; half a step rounds to even
    assert (q[0, 32], e[0, 1]) == (64, 128)                  # 127.5 needs the step 2: 63.75 rounds to 64
    assert (q[0, 64], e[0, 2]) == (0, 1)                     # below the smallest step
    assert (q[0, 96], e[0, 3]) == (64, 248)
    assert (q[0, 128], e[0, 4]) == (0, 255) and e[0, 5:].tolist() == [0, 0, 0]
    v = ref.held(q, e, 160)
    assert v[0, 0] == 127.0 and v[0, 32] == 128.0 and np.isnan(v[0, 128])
