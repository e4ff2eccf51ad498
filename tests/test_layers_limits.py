"""Limits of a decoder layer's operators on both sides, through the C ABI without a GPU:
what is past them is refused on the host."""
import pytest

from test_layers_binding import INVALID, OK, P, lib, run

FAR = 1 << 43          # bytes between addresses that nothing reads
ROWS = 2 ** 32 // 1024 - 1


def norm(rows, dim):
    return lib().rms_norm(0, rows, dim, P, dim, None, dim, 0, P + FAR, 1e-6, 0, P + 2 * FAR, dim, None, 1, None, dim,
                          None, None)


@pytest.mark.parametrize("dim", [64, 1024, 32768])
@pytest.mark.parametrize("rows, status", [(ROWS, OK), (ROWS + 1, (INVALID,)), (1 << 30, (INVALID,))])
def test_rows_of_a_norm(rows, status, dim):
    run(norm, dict(rows=rows, dim=dim), status)


def backward(rows, dim):
    size = lib().rms_norm_backward_workspace(rows, dim)
    return lib().rms_norm_backward(0, rows, dim, P, dim, P + FAR, dim, 0, P + 2 * FAR, P + 3 * FAR, None, dim,
                                   P + 4 * FAR, dim, P + 5 * FAR, P + 6 * FAR, size, None)


@pytest.mark.parametrize("dim", [1, 64, 1024, 32768])
def test_rows_of_a_norms_gradient(dim):
    for rows in (ROWS, ROWS + 1, (1 << 30) if dim < 32768 else 1 << 27):
        run(backward, dict(rows=rows, dim=dim), OK)
        # (sums of workgroups that walk rows)
        assert 0 < lib().rms_norm_backward_workspace(rows, dim) <= 4 * 1024 * dim
    run(backward, dict(rows=(1 << 30) + 1, dim=dim), (INVALID,))
    assert lib().rms_norm_backward_workspace((1 << 30) + 1, dim) == -1
