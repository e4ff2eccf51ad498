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


def grouped(rows, N, groups=1):
    return lib().gemm_grouped(0, groups, rows, N, 0, None, 0, None, N, 0, 0, P, P + FAR, N, 0, None)


def wgrad(groups, N, K):
    return lib().gemm_grouped_wgrad(0, groups, 0, N, K, None, K, None, N, P, P + FAR, N, N * K, 0, None)


def w8a8(rows, N, groups=1):
    return lib().gemm_grouped_w8a8(groups, rows, N, 0, None, 0, P + FAR, None, 0, 0, P + 2 * FAR, N, None, N, P,
                                   P + 3 * FAR, N, None)


# A launch holds 2^32 - 1 threads: 128 x 128 tiles, the most that the rows could need (a tile of
# a group's own for each row up to the groups), and 8 that the shares of the XCDs may round up.
TILES = (2 ** 32 - 1) // 256 - 8


@pytest.mark.parametrize("call", [grouped, w8a8])
@pytest.mark.parametrize("rows, groups, tiles", [(129, 1, 2), (127 * 128, 1, 128), (5, 9, 5), (1000, 60000, 1007)])
def test_tiles_of_grouped_products(rows, groups, tiles, call):
    N = TILES // tiles * 128
    run(call, dict(rows=rows, N=N, groups=groups), OK)
    run(call, dict(rows=rows, N=N + 1, groups=groups), (INVALID,))


def test_tiles_of_a_weights_gradient():
    # (65535 groups; tiles of 128 x 128)
    run(wgrad, dict(groups=65535, N=128 * 16, K=128 * 16), OK)
    run(wgrad, dict(groups=65535, N=128 * 16, K=128 * 16 + 1), (INVALID,))
    run(wgrad, dict(groups=1, N=128 * 4095, K=128 * 4096), OK)
    run(wgrad, dict(groups=1, N=128 * 4096, K=128 * 4096), (INVALID,))
