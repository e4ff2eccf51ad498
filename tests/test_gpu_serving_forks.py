"""cache_fork's rule for parents, and what cache_fork and cache_extend say is
missing, written out from their documentation."""
import pytest
import torch

import mixed_precision_dense_tiled_amd as mp

pytestmark = pytest.mark.gpu
PAGE = 4


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def state(lens, pages, width=4):
    """Row r holds its own pages in ascending order from page 0 on."""
    table, refs, at = [], [0] * pages, 0
    for n in lens:
        k = -(-n // PAGE)
        table.append(list(range(at, at + k)) + [-1] * (width - k))
        refs[at:at + k] = [1] * k
        at += k
    kv = torch.randint(0, 100, (2, pages, PAGE, 8), device="cuda").to(torch.bfloat16)
    return kv, ints(refs), ints(table), ints(lens)


@pytest.mark.parametrize("own", [1, 99, 4], ids=["itself", "out_of_range", "one_past_the_last"])
def test_a_row_that_stays_is_a_parent(gpu_ok, own):
    """Row 1 names itself (or nobody): it is not forked into, and rows 2 and 3 may
    name it."""
    kv, refs, table, lens = state([6, 7, 0, 0], 10)
    before = kv.clone()
    short = mp.cache_fork(kv, refs, table, lens, ints([-1, own, 1, 1]), PAGE)
    assert short.item() == 0
    assert lens.tolist() == [6, 7, 7, 7]
    assert table.tolist() == [[0, 1, -1, -1], [2, 3, -1, -1], [2, 4, -1, -1], [2, 5, -1, -1]]
    assert refs.tolist() == [1, 1, 3, 1, 1, 1, 0, 0, 0, 0]
    assert torch.equal(kv[:, :4], before[:, :4]) and torch.equal(kv[:, 6:], before[:, 6:])
    assert torch.equal(kv[:, 4], before[:, 3]) and torch.equal(kv[:, 5], before[:, 3])


def test_beams_that_name_themselves(gpu_ok):
    """The usual step of a beam search: parents [0, 1, 0, 0]."""
    kv, refs, table, lens = state([8, 4, 0, 0], 6)
    assert mp.cache_fork(kv, refs, table, lens, ints([0, 1, 0, 0]), PAGE).item() == 0
    assert lens.tolist() == [8, 4, 8, 8]
    assert table.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1], [0, 1, -1, -1], [0, 1, -1, -1]]
    assert refs.tolist() == [3, 3, 1, 0, 0, 0]


def test_a_row_that_is_written_is_no_parent(gpu_ok):
    """Two rows that name each other, and one that names a copy: they stay."""
    kv, refs, table, lens = state([6, 7, 3, 0, 0], 10)
    before = [t.clone() for t in (kv, refs, table, lens)]
    assert mp.cache_fork(kv, refs, table, lens, ints([1, 0, -1, -1, -1]), PAGE).item() == 0
    for a, b in zip(before, (kv, refs, table, lens)):
        assert torch.equal(a, b)
    assert mp.cache_fork(kv, refs, table, lens, ints([-1, -1, -1, 2, 3]), PAGE).item() == 0
    assert lens.tolist() == [6, 7, 3, 3, 0] and table[3].tolist() == [5, -1, -1, -1] and refs.sum().item() == 6


@pytest.mark.parametrize("pages, missing", [(9, 0), (8, 1), (4, 5), (3, 6)])
def test_fork_says_how_many_pages_are_missing(gpu_ok, pages, missing):
    """Six copies of a part-filled page; also where they are more than the cache has."""
    kv, refs, table, lens = state([10] + [0] * 6, pages)
    before = [t.clone() for t in (kv, refs, table, lens)]
    assert mp.cache_fork(kv, refs, table, lens, ints([-1] + [0] * 6), PAGE).item() == missing
    if missing:
        for a, b in zip(before, (kv, refs, table, lens)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("pages, missing", [(13, 0), (12, 1), (9, 4), (8, 5), (3, 10), (1, 12)])
def test_extend_says_how_many_pages_are_missing(gpu_ok, pages, missing):
    """Four rows of which one holds a page, each to three or four pages: 12 more."""
    kv, refs, table, lens = state([4, 0, 0, 0], pages)
    before = [t.clone() for t in (refs, table, lens)]
    assert mp.cache_extend(refs, table, lens, ints([12, 12, 9, 11]), PAGE).item() == missing
    if missing:
        for a, b in zip(before, (refs, table, lens)):
            assert torch.equal(a, b)
    else:
        assert lens.tolist() == [16, 12, 9, 11] and refs.tolist() == [1] * 13
