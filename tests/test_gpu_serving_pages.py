"""Page bookkeeping on the GPU against the plain lists of serving_ref.Pages:
forks, extensions, frees and compactions, whole numbers and page contents
equal; nothing changes where pages are missing."""
import random

import pytest
import torch

import mixed_precision_dense_tiled_amd as mp
from serving_ref import Pages

pytestmark = pytest.mark.gpu


def state(rows, lens, pages, page, width, seed, planes=3, dtype=torch.bfloat16, inner=(2, 16), page_major=False):
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table, refs = torch.full((rows, width), -1, dtype=torch.int32), torch.zeros(pages, dtype=torch.int32)
    at = 0
    for r, n in enumerate(lens):
        k = -(-n // page)
        table[r, :k] = order[at:at + k]
        refs[order[at:at + k].long()] = 1
        at += k
    shape = (pages, planes, page, *inner) if page_major else (planes, pages, page, *inner)
    kv = torch.randint(-100, 100, shape, generator=g).to(dtype).cuda()
    if page_major:
        kv = kv.transpose(0, 1)
    lens = torch.tensor(list(lens) + [0] * (rows - len(lens)), dtype=torch.int32)
    return kv, refs.cuda(), table.cuda(), lens.cuda()


def same(ref, refs, table, lens, what):
    assert refs.tolist() == ref.refs, what
    assert table.tolist() == ref.table, what
    assert lens.tolist() == ref.lens, what


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page, seed", [(1, 0), (16, 1), (16, 2), (64, 3), (5, 4)])
@pytest.mark.parametrize("kind", ["plain", "page_major", "odd_bytes"])
def test_random_steps(gpu_ok, page, seed, kind):
    rng = random.Random(seed)
    rows, pages, width = 12, 90, 14
    more = dict(page_major=kind == "page_major")
    if kind == "odd_bytes":
        more = dict(dtype=torch.uint8, inner=(3, 7))
    kv, refs, table, lens = state(rows, [rng.randint(0, 4 * page) for _ in range(5)], pages, page, width, seed, **more)
    ref = Pages(refs, table, lens, page)
    plain = kv.clone()
    for step in range(12):
        what = (step, page, kind)
        parent = [-1] * rows
        empty = [r for r in range(rows) if ref.lens[r] == 0]
        full = [r for r in range(rows) if ref.lens[r]]
        for r in empty:
            if full and rng.random() < 0.5:
                parent[r] = rng.choice(full)
        short = mp.cache_fork(kv, refs, table, lens, ints(parent), page)
        assert short.item() == ref.fork(parent), what
        same(ref, refs, table, lens, what)
        add = [rng.choice([0, 0, 1, 2, page, 2 * page + 1]) for _ in range(rows)]
        short = mp.cache_extend(refs, table, lens, ints(add), page)
        assert short.item() == ref.extend(add), what
        same(ref, refs, table, lens, what)
        drop = [int(rng.random() < 0.35) for _ in range(rows)]
        mp.cache_free(refs, table, lens, ints(drop), page)
        ref.drop(drop)
        same(ref, refs, table, lens, what)
        if step % 3 == 2:
            mp.cache_compact(kv, refs, table, lens, page)
            ref.compact()
            same(ref, refs, table, lens, what)
        for src, dst in ref.copies:
            plain[:, dst] = plain[:, src]
        ref.copies.clear()
        assert torch.equal(kv, plain), what


def test_many_rows_and_pages(gpu_ok):
    """More rows and pages than one pass of the planning workgroup covers."""
    rows, page, pages = 2500, 4, 13000
    lens0 = [(r * 7) % 19 for r in range(1200)]
    kv, refs, table, lens = state(rows, lens0, pages, page, 9, 5, planes=2, inner=(8,))
    ref = Pages(refs, table, lens, page)
    plain = kv.clone()
    parent = [-1] * 1200 + [r % 1200 for r in range(1300)]
    assert mp.cache_fork(kv, refs, table, lens, ints(parent), page).item() == ref.fork(parent) == 0
    add = [r % 6 for r in range(rows)]
    assert mp.cache_extend(refs, table, lens, ints(add), page).item() == ref.extend(add) == 0
    drop = [int(r % 3 == 0) for r in range(rows)]
    mp.cache_free(refs, table, lens, ints(drop), page)
    ref.drop(drop)
    mp.cache_compact(kv, refs, table, lens, page)
    ref.compact()
    same(ref, refs, table, lens, "many")
    for src, dst in ref.copies:
        plain[:, dst] = plain[:, src]
    assert torch.equal(kv, plain)


def test_nothing_changes_where_pages_are_missing(gpu_ok):
    kv, refs, table, lens = state(6, [10, 20, 30], 6, 16, 4, 6)
    before = [t.clone() for t in (kv, refs, table, lens)]
    assert mp.cache_fork(kv, refs, table, lens, ints([-1, -1, -1, 0, 1, 2]), 16).item() == 2      # one page is free
    assert mp.cache_extend(refs, table, lens, ints([40, 0, 0, 0, 0, 0]), 16).item() == 2
    assert mp.cache_extend(refs, table, lens, ints([55, 0, 0, 0, 0, 0]), 16).item() == 4          # past the row's end
    assert mp.cache_extend(refs, table, lens, ints([2 ** 31 - 1] * 6, ), 16).item() > 0
    for a, b in zip(before, (kv, refs, table, lens)):
        assert torch.equal(a, b)


def test_parents_that_are_none(gpu_ok):
    """Itself, out of range, or itself forked into: the row stays."""
    kv, refs, table, lens = state(6, [10, 20, 30], 20, 16, 4, 7)
    before = [t.clone() for t in (kv, refs, table, lens)]
    parent = [-1, -1, -1, 99, 4, 3]
    assert mp.cache_fork(kv, refs, table, lens, ints(parent), 16).item() == 0
    for a, b in zip(before, (kv, refs, table, lens)):
        assert torch.equal(a, b)
    ref = Pages(refs, table, lens, 16)
    parent = [-1, -1, -1, 1, 3, 4]          # 4 and 5 name rows that are written by the same call
    mp.cache_fork(kv, refs, table, lens, ints(parent), 16)
    ref.fork(parent)
    same(ref, refs, table, lens, "chain")
    assert lens.tolist() == [10, 20, 30, 20, 0, 0]


def test_table_entries_out_of_range_are_left_alone(gpu_ok):
    kv, refs, table, lens = state(4, [40, 20], 12, 16, 4, 8)
    table[0, 1] = 500
    mp.cache_fork(kv, refs, table, lens, ints([-1, -1, 0, -1]), 16)
    mp.cache_compact(kv, refs, table, lens, 16)
    assert table[0, 1] == 500 and table[2, 1] == 500
    mp.cache_free(refs, table, lens, ints([1, 0, 1, 0]), 16)
    # row 1 holds two pages, and the page whose entry was written over keeps its holder
    assert (refs >= 0).all() and int(refs.sum()) == 3


def test_strided_tables_and_empty_calls(gpu_ok):
    kv, refs, table, lens = state(4, [40, 20], 12, 16, 4, 9)
    wide = torch.full((4, 9), 77, dtype=torch.int32, device="cuda")
    wide[:, 2:6] = table
    ref = Pages(refs, table, lens, 16)
    mp.cache_fork(kv, refs, wide[:, 2:6], lens, ints([-1, -1, 1, 0]), 16)
    ref.fork([-1, -1, 1, 0])
    same(ref, refs, wide[:, 2:6], lens, "strided")
    assert (wide[:, :2] == 77).all() and (wide[:, 6:] == 77).all()
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    assert mp.cache_fork(kv, refs, none, none[:, 0].contiguous(), none[:, 0].contiguous(), 16).item() == 0
    mp.cache_compact(kv, refs, none, none[:, 0].contiguous(), 16)


def test_captured_into_a_graph(gpu_ok):
    kv, refs, table, lens = state(6, [10, 20, 33], 40, 16, 6, 10)
    ref = Pages(refs, table, lens, 16)
    parent, add, drop = ints([-1, -1, -1, 0, 1, 2]), ints([0, 0, 0, 1, 1, 1]), ints([0, 0, 0, 1, 1, 1])

    def step():
        mp.cache_fork(kv, refs, table, lens, parent, 16)
        mp.cache_extend(refs, table, lens, add, 16)
        seen = refs.clone(), table.clone(), lens.clone()
        mp.cache_free(refs, table, lens, drop, 16)
        mp.cache_compact(kv, refs, table, lens, 16)
        return seen

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()

    def plain():
        ref.fork(parent.tolist())
        ref.extend(add.tolist())
        mid = Pages(torch.tensor(ref.refs), torch.tensor(ref.table), torch.tensor(ref.lens), 16)
        ref.drop(drop.tolist())
        ref.compact()
        return mid

    plain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        seen = step()
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        mid = plain()
        same(mid, *seen, i)
        same(ref, refs, table, lens, i)
