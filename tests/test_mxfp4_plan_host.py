"""The sizes of test_gpu_mxfp4_paths.py reach every tile shape of the MXFP4
product, split and not, and the loop over whole stages with rows of scales that
end inside a piece and that do not."""
import numpy as np

import mx_plan as plan
import test_gpu_mxfp4 as small
import test_gpu_mxfp4_paths as paths
from test_matrix_host import qc  # noqa: F401


def test_plan_is_the_library_s(qc):  # noqa: F811
    """The parts of k, through the workspace that the library asks for."""
    r = np.random.default_rng(3)
    for _ in range(5000):
        m, n, k = (int(v) for v in np.exp(r.uniform(0, 11, 3)))
        _, parts, _ = plan.product(m, n, k)
        want = parts * m * (-(-n // 4) * 4) * 4 if parts > 1 else 0
        assert qc.qc_matmul_mxfp4_workspace(m, n, k) == want, (m, n, k)
        x = 0 if m <= plan.FEW else (-(-m * (-(-k // 32) * 16) // 256) + -(-m * (-(-k // 128) * 4) // 256)) * 256 + want
        assert qc.qc_linear_mxfp4_workspace(m, n, k, qc.QC_BF16) == x, (m, n, k)


def test_every_path_is_reached():
    reached, loops = set(), set()
    for m, n, k in paths.SIZES + small.SIZES:
        shape, parts, each = plan.product(m, n, k)
        reached.add((shape, parts > 1))
        if shape >= plan.FIRST_PIPE:
            turns = plan.fast_turns(k, shape, each if parts > 1 else None)
            loops.add((shape, min(turns, 2), -(-k // 128) % 4 != 0))
    for shape in range(len(plan.SHAPES)):
        assert (shape, False) in reached, shape
        if shape >= plan.FIRST_PIPE:
            assert (shape, True) in reached, shape
            assert (shape, 2, True) in loops, shape
            assert any(s == shape and t == 0 for s, t, _ in loops) or any(s == shape and t == 1 for s, t, _ in loops)
    assert any(t == 2 and not ragged for _, t, ragged in loops)
    further = set()
    for m, n, k in paths.SIZES:
        shape, parts, each = plan.product(m, n, k)
        bn, bm = (int(v) for v in plan.SHAPES[shape][:2])
        tiles = -(-n // bn) * -(-m // bm)
        if parts == 1 and tiles > 256:
            further.add((shape, min(-(-tiles // 256), 3), min(plan.fast_turns(k, shape), 1)))
    last = len(plan.SHAPES) - 1
    assert {(last, 2, 1), (last, 3, 0), (last - 1, 3, 0), (last - 1, 3, 1)} <= further, further
    assert {m for m, _, _ in small.SIZES} >= {1, 2, 7}  # encoded by the blocks that multiply them
    assert any(4 < m <= plan.FEW and n > 4096 for m, n, _ in small.WIDE)
