"""The sizes of test_gpu_matrix_paths.py and test_gpu_matrix.py reach every
kernel, tile, split and loop of the weight gradient and every tile of the
INT8 product; and the bounds of test_gpu_matrix_paths.py show a lost piece of
an fp32 gradient."""
import numpy as np
import pytest
import torch

import matrix_plan as plan
import matrix_ref as ref
import test_gpu_matrix as old
import test_gpu_matrix_paths as paths
from test_matrix_host import qc  # noqa: F401

BF16, F32 = torch.bfloat16, torch.float32


def test_plan_is_the_library_s(qc):  # noqa: F811
    """The splits, through the workspace that the library asks for."""
    r = np.random.default_rng(3)
    sizes = [s[1:] for s in paths.ALL] + [tuple(int(v) for v in np.exp(r.uniform(0, 9, 3)) + 1) for _ in range(3000)]
    for rows, n, dim in sizes:
        for bf16 in (True, False):
            splits = plan.wgrad(rows, n, dim, bf16)[2]
            want = splits * n * ref.up(dim, 4) * 4 if splits > 1 else 0
            assert qc.qc_ckpt8_wgrad_workspace(rows, n, dim, qc.QC_BF16 if bf16 else qc.QC_F32) == want, (rows, n, dim)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_every_path_is_reached(dtype):
    bf16 = dtype is BF16
    unit = 8 if bf16 else 4
    reached = set()
    for t, rows, n, dim in paths.ALL:
        if t is dtype:
            kernel, bd, splits, per = plan.wgrad(rows, n, dim, bf16)
            turns = plan.main_loop_turns(rows, n, dim, bf16)
            loop = "twice" if max(turns) >= 2 else "once" if max(turns) else "never"
            reached.add((kernel, bd, splits > 1, loop))
            if kernel == "pipelined":
                reached.add(("short last piece", bd, splits > 1, n % unit != 0))
    for bd in (128, 256):
        for split in (False, True):
            assert ("pipelined", bd, split, "twice") in reached, (bd, split)
            assert ("short last piece", bd, split, True) in reached, (bd, split)
    for split in (False, True):
        assert ("simple", 128, split, "never") in reached


def test_simple_kernel_takes_several_stages_and_tiles():
    for bf16 in (True, False):
        plans = [plan.wgrad(rows, 3, dim, bf16) for rows, dim in paths.SIMPLE]
        assert any(p[3] >= 3 * 64 and p[2] > 1 for p in plans), plans
        assert {p[0] for p in plans} == {"simple"}
    assert any(dim > 2 * 128 for _, dim in paths.SIMPLE)


def test_pieces_are_tested_on_every_fp32_kernel():
    reached = set()
    for rows, n, dim in paths.PIECES:
        kernel, bd, splits, _ = plan.wgrad(rows, n, dim, False)
        reached.add((kernel, bd, splits > 1, max(plan.main_loop_turns(rows, n, dim, False)) > 1))
    assert {("pipelined", 128, True, True), ("pipelined", 256, False, True), ("pipelined", 256, True, True),
            ("simple", 128, True, False)} <= reached


def sizes_of(test):
    """The (m, n, k) that a test is parametrised with."""
    marks = [m for m in test.pytestmark if m.name == "parametrize" and m.args[0] == "m,n,k"]
    return [size for mark in marks for size in mark.args[1]]


def test_every_product_tile_is_reached():
    every = set(range(len(plan.PRODUCT)))
    sizes = sizes_of(old.test_matmul) + sizes_of(old.test_matmul_large_tiles_long_k)
    assert {plan.product(m, n) for m, n, k in sizes if k >= 1024} == every


def first_pieces(x, count):
    """The sum of the first pieces of an fp32 gradient, eight mantissa bits each."""
    total, rest = torch.zeros_like(x), x.clone()
    for _ in range(count):
        piece = (rest.view(torch.int32) & -65536).view(F32)
        total, rest = total + piece, rest - piece
    return total


@pytest.mark.parametrize("rows,n,dim", [s for s in paths.F32_SIZES if s[0] * s[1] * s[2] < 2 ** 30])
def test_a_lost_piece_is_seen(rows, n, dim):
    """A sum of two pieces of three, planted in the reference, breaks the norm's bound; three are exact."""
    dy = paths.gradients(rows, n, F32)
    assert torch.equal(first_pieces(dy, 3), dy)
    v = ref.matrix(rows, dim, 2, F32).double().numpy()
    d = dy.double().numpy()
    want = d.T @ v
    lost = first_pieces(dy, 2).double().numpy().T @ v
    rel = np.linalg.norm(lost - want) / np.linalg.norm(want)
    assert rel > 1.5 * paths.norm_bound(rows, F32), rel


def test_a_lost_piece_is_seen_in_single_products():
    _, _, value = paths.one_token_a_channel(100, 100, -126, -100, 6)
    x = torch.from_numpy(value.astype(np.float32))
    for count in (1, 2):
        off = np.abs(first_pieces(x, count).double().numpy() - value)
        assert np.all(off > 8 * 2.0 ** -24 * np.abs(value))
