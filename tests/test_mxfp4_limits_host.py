"""Answers of the 4-bit matrix operators and of the optimizer's entry points
for sizes that no call takes (no GPU is needed)."""
import pytest

from test_matrix_host import qc  # noqa: F401


@pytest.mark.parametrize("n", [(1 << 56) + 1, 1 << 62, (1 << 63) - 2048, (1 << 63) - 1])
def test_workspace_of_a_norm_that_is_refused(qc, n):  # noqa: F811
    """No bytes for a list that qc_grad_norm_multi refuses, and no arithmetic
    past 64 bits on its length."""
    assert qc.lib().qc_grad_norm_workspace(n) == -1
    with pytest.raises(qc.QcError):
        qc.qc_grad_norm_workspace(n)


def test_workspace_of_the_longest_norm(qc):  # noqa: F811
    assert 0 < qc.qc_grad_norm_workspace(1 << 56) <= 8 * 2048
