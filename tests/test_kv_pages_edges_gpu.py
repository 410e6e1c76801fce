"""Shared pages where they can go wrong, on the GPU: bad cells and stacks, destinations that several pairs ask for, the
releases' forms for large tables, lengths below what rows share."""
import numpy as np
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests.kv_pages_ref import BAD_INDEX, BAD_LEN, BAD_ROW, NO_PAGES, State
from tests.test_kv_pages_gpu import Device, dev, ones

pytestmark = pytest.mark.gpu


def fork(g, src, dst, lens):
    a, b = (torch.full((len(src),), -5, dtype=torch.int32, device="cuda") for _ in range(2))
    L.gdn_kv_fork(g.kd, dev(src), dev(dst), dev(lens), g.held, g.table, g.free, g.count, g.refs, a, b)
    return a.tolist(), b.tolist(), L.gdn_get_status(clear=True)


@pytest.mark.parametrize("rows", [4, 3000])
@pytest.mark.parametrize("bad", [-1, -2, 40, 1 << 30])
def test_fork_of_a_last_page_outside_the_cache(gdn, bad, rows):
    """The source's partly filled page is no page of the cache: that pair is not made, and takes nothing; others are."""
    st = State(rows, 16, 12, 40)  # (in one cluster, and in two kernels)
    g = Device(st)
    g.plan(0, 200, [0] * rows, [40, 40] + [0] * (rows - 2), ones(rows))
    good = g.table[0, 2].item()
    g.table[0, 2] = bad
    before = [t.clone() for t in (g.held, g.table, g.refs)]
    count, top = g.count.item(), g.free.tolist()
    n = rows - 2
    src, dst, lens = [0] * n, list(range(2, rows)), [40] * n
    a, b, status = fork(g, src, dst, lens)
    assert (a, b, status) == ([-2] * n, [-2] * n, BAD_INDEX)
    assert all(torch.equal(x, y) for x, y in zip(before, (g.held, g.table, g.refs))) and g.count.item() == count
    # a pair of whole pages, and one of another source, go through; the refused one's destination is free for a later pair
    a, b, status = fork(g, [0, 0, 1], [2, 2, 3], [40, 32, 40])
    assert status == BAD_INDEX and a == [-2, -1, g.table[1, 2].item()] and b == [-2, -1, top[count - 1]]
    assert g.held.tolist()[:4] == [3, 3, 2, 3] and g.table[2].tolist()[:3] == before[1][0].tolist()[:2] + [-1]
    assert good != bad


def test_fork_where_the_stack_holds_no_page(gdn):
    """A stack entry outside the cache: its pair is not made, and the entry is dropped."""
    for bad in (-1, -2, 20, 1 << 30):
        st = State(4, 16, 4, 20)
        g = Device(st)
        g.plan(0, 100, [0] * 4, [40, 0, 0, 0], ones(4))
        count = g.count.item()
        g.free[count - 1] = bad
        want = g.free[count - 2].item()
        a, b, status = fork(g, [0, 0, 0], [1, 2, 3], [40, 40, 32])
        assert status == BAD_INDEX and a == [-2, g.table[0, 2].item(), -1] and b == [-2, want, -1]
        assert g.held.tolist() == [3, 0, 3, 2] and g.table[1].tolist() == [-1] * 4 and g.count.item() == count - 2
        refs = [0] * 20
        for p in g.table[0, :2].tolist():
            refs[p] = 3
        refs[g.table[0, 2].item()] = refs[want] = 1
        assert g.refs.tolist() == refs


@pytest.mark.parametrize("M", [4, 2000])
@pytest.mark.parametrize("bad", [-1, -7, 20, (1 << 27) + 3, 1 << 30])
def test_plan_where_the_stack_holds_no_page(gdn, bad, M):
    """A stack entry outside the cache: its place in the table gets -1, its tokens no slots; the row beside is served."""
    st = State(3, 16, M, 20)
    g = Device(st)
    g.free[18] = bad  # the second page taken: row 0's places 16 .. 31
    z = lambda n: torch.full((n,), -5, dtype=torch.int32, device="cuda")
    out = dict(q_start=z(4), q_count=z(3), kv_len=z(3), slots=z(60), positions=z(60))
    L.gdn_kv_plan_shared(g.kd, dev([0] * 3), dev([40, 0, 10]), dev(ones(3), torch.uint8), g.held, g.table, g.free, g.count, g.refs, **out)
    assert L.gdn_get_status(clear=True) == BAD_INDEX
    assert g.table[:, :4].tolist() == [[19, -1, 17, -1], [-1] * 4, [16, -1, -1, -1]] and g.held.tolist() == [3, 0, 1]
    assert g.refs.tolist() == [0] * 16 + [1, 1, 0, 1] and g.count.item() == 16
    slots = [19 * 16 + i for i in range(16)] + [-1] * 16 + [17 * 16 + i for i in range(8)] + [16 * 16 + i for i in range(10)]
    assert out["slots"].tolist() == slots + [-1] * 10
    assert out["positions"].tolist() == list(range(40)) + list(range(10)) + [-1] * 10
