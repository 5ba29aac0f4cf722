"""Sizes beyond what one launch takes are refused before any device work (no
GPU is needed: a call that went on would end in QC_ERR_LAUNCH here)."""
import ctypes

import pytest

from test_matrix_host import ARG, UNSUP, dec_ckpt, enc_ckpt, matmul, qc, status, swiglu, swiglu_bwd  # noqa: F401


@pytest.mark.parametrize("kw", [dict(m=1, n=1 << 31, ldc=1 << 31), dict(m=1 << 31, n=1, ldc=1),
                                dict(m=1 << 20, n=1 << 19, ldc=1 << 19), dict(m=(1 << 31) - 255, n=256, ldc=256),
                                dict(m=3, n=1 << 34, ldc=1 << 34)], ids=str)
def test_product_of_too_many_tiles(qc, kw):  # noqa: F811
    """2^23 tiles of 256 x 256: a grid has fewer than 2^32 threads, 512 a tile."""
    assert status(qc, "qc_matmul_int8", *matmul(**kw)) == ARG


@pytest.mark.parametrize("fn,args,ld", [
    ("qc_encode_ckpt8", enc_ckpt, ("ldx",)), ("qc_decode_ckpt8", dec_ckpt, ("ldo",)),
    ("qc_swiglu_ckpt8", swiglu, ("ldx", "ldh")), ("qc_swiglu_ckpt8_backward", swiglu_bwd, ("lddh", "ldg"))])
def test_checkpoint_of_too_long_rows(qc, fn, args, ld):  # noqa: F811
    dim = (1 << 34) + 1
    assert status(qc, fn, *args(rows=1, dim=dim, **{n: dim for n in ld})) == UNSUP


def test_sizes_of_long_rows(qc):  # noqa: F811
    c = ctypes.c_int64()
    assert qc.ckpt8_bytes(1, 1 << 34) == (1 << 34, 1 << 29)
    assert qc.lib().qc_ckpt8_bytes(1, 1 << 57, ctypes.byref(c), ctypes.byref(c)) == ARG


def test_sizes_that_are_bad(qc):  # noqa: F811
    """qc_ckpt8_bytes answers with a status and writes nothing; the workspace's size is -1."""
    cb, eb = ctypes.c_int64(-7), ctypes.c_int64(-7)
    for rows, dim in ((-1, 8), (1, 0), (1 << 57, 8), (1, 1 << 57)):
        assert qc.lib().qc_ckpt8_bytes(rows, dim, ctypes.byref(cb), ctypes.byref(eb)) == ARG
        assert (cb.value, eb.value) == (-7, -7)
    for args in ((-1, 8, 8, 0), (8, -1, 8, 0), (8, 8, 0, 0), (8, 8, 8, 7), (1 << 57, 8, 8, 0)):
        assert qc.lib().qc_ckpt8_wgrad_workspace(*args) == -1
