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


def forks_in_order(st, src, dst, lens):
    """The pairs one after the other, as gdn.h has them: a destination is taken once a pair of it is made."""
    before, status, out, P = list(st.held), 0, [], st.P
    for s, d, n in zip(src, dst, lens):
        want, need = -(-n // P), n % P > 0
        rows = 0 <= s < st.B and 0 <= d < st.B and s != d
        pair = (-2, -2)
        if n < 0 or want > st.M or (rows and before[s] < want):
            status |= BAD_LEN
        elif not rows or before[d] or (n and st.held[d]):
            status |= BAD_ROW
        elif n == 0:
            pair = (-1, -1)
        elif need and st.count == 0:
            status |= NO_PAGES
        else:
            pair = (-1, -1)
            for c in range(n // P):
                st.table[d][c] = st.table[s][c]
                st.refs[st.table[s][c]] += 1
            if need:
                st.count -= 1
                pair = (st.table[s][n // P], st.free[st.count])
                st.table[d][n // P] = pair[1]
                st.refs[pair[1]] = 1
            st.held[d] = want
        out.append(pair)
    return [a for a, _ in out], [b for _, b in out], status


@pytest.mark.parametrize("B,M,n,spare", [(6, 6, 2, 0), (6, 6, 5, 1), (6, 6, 9, 2), (40, 8, 60, 7), (40, 8, 400, 0), (300, 12, 1500, 90), (2000, 20, 4000, 300)])
def test_a_destination_goes_to_the_first_pair_that_is_made(gdn, B, M, n, spare):
    """Destinations that several pairs ask for, while pages run out: one whose page is missing leaves its row to a later pair
    that needs none."""
    rng = np.random.default_rng(n)
    for turn in range(4):
        sources = max(2, B // 10)
        need = [int(rng.integers(17, 16 * M + 1)) if b < sources else 0 for b in range(B)]
        used = sum(-(-x // 16) for x in need)
        st = State(B, 16, M, used + spare, rng.permutation(used + spare).tolist())
        g = Device(st)
        g.plan(0, sum(need), [0] * B, need, ones(B))
        src = rng.integers(0, sources + 1, n).tolist()
        dst = rng.integers(sources - 1, min(B, sources + 1 + n // 2), n).tolist()
        lens = [int(rng.choice([need[s], need[s] // 16 * 16, 16, 0, int(rng.integers(0, need[s] + 20))])) for s in src]
        want = forks_in_order(st, src, dst, lens)
        assert fork(g, src, dst, lens) == want
        g.same()
        st.check()


def test_whole_pages_after_the_last_page(gdn):
    """No page is left: a pair of 33 tokens is not made, one of 32 for the same row is, and later ones find the row taken."""
    st = State(5, 16, 4, 3)
    g = Device(st)
    g.plan(0, 40, [0] * 5, [33, 0, 0, 0, 0], ones(5))
    a, b, status = fork(g, [0] * 6, [3, 3, 3, 3, 4, 3], [33, 32, 32, 33, 1, 0])
    assert (a, b) == ([-2, -1, -2, -2, -2, -1],) * 2 and status == NO_PAGES | BAD_ROW
    assert g.held.tolist() == [3, 0, 0, 2, 0] and g.table[3].tolist() == g.table[0].tolist()[:2] + [-1, -1]
    assert g.refs.tolist() == [2 if p in g.table[3].tolist() else 1 for p in range(3)]


def test_a_row_of_a_negative_count_is_not_empty(gdn):
    st = State(4, 16, 4, 20)
    g = Device(st)
    g.plan(0, 40, [0] * 4, [33, 0, 0, 0], ones(4))
    g.held[1], g.held[2] = -1, -100
    a, b, status = fork(g, [0] * 4, [1, 2, 2, 3], [32] * 4)
    assert (a, b) == ([-2, -2, -2, -1],) * 2 and status == BAD_ROW and g.held.tolist() == [3, -1, -100, 2]


@pytest.mark.parametrize("B,M,lo,bad", [(120, 400, 60, False), (120, 400, 60, True), (100, 700, 690, False), (100, 700, 690, True), (3, 1400, 1, True), (1024, 8, 1, True), (1030, 40, 33, True)])
def test_releases_of_large_tables(gdn, B, M, lo, bad):
    """Pages given back where the table has thousands of cells, up to 4 x 8 x 1024 releases in a call (they stay in registers)
    and more (they do not): rows of one prompt, cut to any length and ended, with cells outside the cache and pages that
    nobody holds among them."""
    rng = np.random.default_rng(B * M)
    P, prompts = 16, max(1, B // 5)
    need = [int(rng.integers(lo * P, M * P + 1)) if b < prompts else 0 for b in range(B)]
    n = sum(-(-x // P) for x in need) + B + 10
    st = State(B, P, M, n, rng.permutation(n).tolist())
    g = Device(st)
    g.plan(0, sum(need), [0] * B, need, ones(B))
    dst = list(range(prompts, B))
    src = [d % prompts for d in dst]
    lens = need[:prompts] + [max(1, need[s] - int(rng.integers(0, need[s] // 3 + 1))) for s in src]
    g.fork(src, dst, lens[prompts:])
    st.check()
    if bad:
        for b in rng.permutation(B)[: max(3, B // 9)].tolist():
            st.table[b][int(rng.integers(0, st.held[b]))] = int(rng.choice([-1, -9, n, n + 1000, 1 << 30]))
        for b in rng.permutation(B)[: max(3, B // 9)].tolist():
            page = st.table[b][int(rng.integers(0, st.held[b]))]
            if 0 <= page < n:
                st.refs[page] = 0
        g.upload()
    some = rng.permutation(B)[: B // 2].tolist()
    held = list(st.held)
    for b in some:
        lens[b] = int(rng.choice([0, int(rng.integers(0, lens[b] + 1)), lens[b]]))
    status = lambda new: BAD_INDEX if any(not 0 <= p < n or st.refs[p] == 0 for b in range(B) for p in st.table[b][-(-new[b] // P): st.held[b]]) else 0
    g.plan(1, B, lens, [0] * B, ones(B), status=status(lens))
    assert sum(held) > sum(st.held) or B < 5
    g.plan(1, B, [0] * B, [0] * B, ones(B), status=status([0] * B))
    assert not any(st.held) and (bad or st.count == n)


def plan(g, T, N, lens, add, active=None):
    z = lambda n: torch.full((n,), -5, dtype=torch.int32, device="cuda")
    B = g.st.B
    out = dict(q_start=z(B + 1), q_count=z(B), kv_len=z(B), slots=z(N), positions=z(N))
    L.gdn_kv_plan_shared(g.kd, dev(lens), dev(add), dev(active or ones(B), torch.uint8), g.held, g.table, g.free, g.count, g.refs, **out, T=T)
    return {k: v.tolist() for k, v in out.items()}, L.gdn_get_status(clear=True)


@pytest.mark.parametrize("M", [8, 1500])
@pytest.mark.parametrize("T", [0, 4])
def test_no_row_writes_into_a_page_that_another_holds(gdn, M, T):
    """A row whose next token would stand in a shared page gets no tokens, and a status; the others get theirs.  Row 0 has 70
    tokens, row 1 continues them, row 2 the first 40, row 3 is alone."""
    def start():
        g = Device(State(4, 16, M, 40))
        g.plan(0, 200, [0] * 4, [70, 0, 0, 33], ones(4))
        g.fork([0, 0], [1, 2], [70, 40])
        return g

    # as the header has it: behind what is shared
    g = start()
    g.plan(T, 16, [70, 70, 40, 33], [4] * 4, ones(4))
    g.st.check()
    # rows 0 and 1 both cut: row 1 gives its third page back, so row 0 may go on in it; row 1's second is also row 0's
    g = start()
    out, status = plan(g, T, 16, [34, 20, 40, 33], [4] * 4)
    assert status == BAD_LEN and out["q_count"] == [4, 0, 4, 4] and out["kv_len"] == [38, 20, 44, 37]
    assert g.held.tolist() == [3, 2, 3, 3]
    # row 0 at 34 while row 1 stays
    g = start()
    out, status = plan(g, T, 16, [34, 70, 40, 33], [4] * 4)
    assert status == BAD_LEN and out["q_count"] == [0, 4, 4, 4] and out["kv_len"] == [34, 74, 44, 37] and g.held.tolist() == [3, 5, 3, 3]
    at = out["q_start"][1]
    assert out["slots"][at] == g.table[1, 4].item() * 16 + 70 % 16 and (T == 0 or out["slots"][:4] == [-1] * 4)
    # a row that begins anew while it still holds what it shared; nothing to write, nothing wrong
    g = start()
    out, status = plan(g, T, 16, [0, 70, 40, 33], [4] * 4)
    assert status == BAD_LEN and out["q_count"] == [0, 4, 4, 4]
    out, status = plan(g, T, 16, [0, 74, 44, 37], [0, 4, 4, 4])
    assert status == 0 and g.held.tolist() == [0, 5, 3, 3]
    out, status = plan(g, T, 16, [0, 78, 48, 41], [4, 0, 0, 0])
    assert status == 0 and out["q_count"] == [4, 0, 0, 0] and g.refs[g.table[0, 0]].item() == 1
    # the other holders end in the same call: nobody shares it any more
    g = start()
    out, status = plan(g, T, 16, [34, 0, 0, 33], [4, 0, 0, 4])
    assert status == 0 and out["q_count"] == [4, 0, 0, 4]
    # a fork of more than the source has committed
    g = start()
    out, status = plan(g, T, 16, [70, 70, 0, 20], [0] * 4)  # row 3: 20 committed, in two pages
    assert status == 0 and g.held.tolist() == [5, 5, 0, 2]
    assert fork(g, [3], [2], [32]) == ([-1], [-1], 0)
    out, status = plan(g, T, 16, [70, 70, 32, 20], [0, 0, 4, 4])
    assert status == BAD_LEN and out["q_count"] == [0, 0, 4, 0]
    # inactive rows and rows without new tokens may be of any length
    out, status = plan(g, T, 16, [34, 20, 33, 3], [4, 0, 0, 4], [0, 1, 1, 0])
    assert status == 0


@pytest.mark.parametrize("B", [1030, 2500])
def test_shared_rows_of_many_chunks(gdn, B):
    """The same where rows take more than one look, in the fixed and the packed layout, against a row-by-row reading."""
    rng = np.random.default_rng(B)
    g = Device(State(B, 16, 6, 4 * B))
    need = [int(rng.integers(1, 80)) if b % 3 == 0 else 0 for b in range(B)]
    g.plan(0, sum(need), [0] * B, need, ones(B))
    lens = list(need)
    pairs = [(b - b % 3, b, int(rng.integers(1, need[b - b % 3] + 1))) for b in range(B) if b % 3]
    g.fork(*map(list, zip(*pairs)))
    for s, d, n in pairs:
        lens[d] = n
    cut = [int(rng.integers(1, n + 1)) if rng.random() < 0.3 else n for n in lens]
    add = rng.integers(0, 4, B).tolist()
    st = g.st
    held = [min(st.held[b], -(-(cut[b] + add[b]) // 16)) for b in range(B)]
    left = [0] * st.n
    for b in range(B):
        for c in range(held[b]):
            left[st.table[b][c]] += 1
    bad = [add[b] > 0 and cut[b] // 16 < held[b] and left[st.table[b][cut[b] // 16]] > 1 for b in range(B)]
    assert 20 < sum(bad) < B // 2
    for T in (3, 0):
        g.upload()
        out, status = plan(g, T, 3 * B, cut, add)
        assert status == BAD_LEN
        assert out["q_count"] == [0 if x else a for x, a in zip(bad, add)]
        assert g.held.tolist() == [held[b] if bad[b] else -(-(cut[b] + add[b]) // 16) for b in range(B)]
        seen = [0] * st.n
        for b, (row, k) in enumerate(zip(g.table.tolist(), g.held.tolist())):
            for p in row[:k]:
                seen[p] += 1
        assert seen == g.refs.tolist()
