"""Shared pages of the attention cache on the GPU against plain references:
gdn_kv_plan_shared, gdn_kv_fork, gdn_kv_compact and gdn_kv_copy_pages.  Whole
numbers and copied bytes: equal."""
import numpy as np
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref
from tests.kv_pages_ref import BAD_INDEX, BAD_LEN, BAD_ROW, NO_PAGES, State

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x).tolist(), dtype=dtype, device="cuda")


class Device:
    """A State's arrays on the GPU, and the calls on them, each checked against the State's own."""

    def __init__(self, st, H_kv=1, d=64):
        self.st = st
        self.kd = L.kv4_dims(st.B, H_kv, H_kv, d, st.P, st.M, st.n)
        self.upload()

    def upload(self):
        st = self.st
        self.held, self.table, self.refs = dev(st.held), dev(st.table).view(st.B, st.M), dev(st.refs)
        self.free, self.count = dev(st.free), dev([st.count])

    def same(self):
        st = self.st
        assert self.held.tolist() == st.held and self.table.tolist() == st.table and self.refs.tolist() == st.refs
        assert self.count.item() == st.count and self.free.tolist()[: st.count] == st.free[: st.count]

    def plan(self, T, N, lens, add, active, status=0):
        z = lambda n: torch.full((n,), -5, dtype=torch.int32, device="cuda")
        out = dict(q_start=z(self.st.B + 1), q_count=z(self.st.B), kv_len=z(self.st.B), slots=z(N), positions=z(N))
        L.gdn_kv_plan_shared(self.kd, dev(lens), dev(add), dev(active, torch.uint8), self.held, self.table, self.free, self.count, self.refs, **out, T=T)
        want, bits = self.st.plan(T, N, lens, add, active)
        assert L.gdn_get_status(clear=True) == bits == status
        for k, v in want.items():
            assert out[k].tolist() == v, k
        self.same()

    def fork(self, src, dst, lens, status=0):
        a, b = (torch.full((len(src),), -5, dtype=torch.int32, device="cuda") for _ in range(2))
        L.gdn_kv_fork(self.kd, dev(src), dev(dst), dev(lens), self.held, self.table, self.free, self.count, self.refs, a, b)
        want = self.st.fork(src, dst, lens)
        assert L.gdn_get_status(clear=True) == want[2] == status
        assert (a.tolist(), b.tolist()) == want[:2]
        self.same()
        return a, b

    def compact(self, in_place):
        st, z = self.st, lambda n: torch.full((max(n, 1),), -5, dtype=torch.int32, device="cuda")
        table, refs = (self.table, self.refs) if in_place else (torch.full_like(self.table, -5), z(st.n))
        free, count, page_map, src, dst, copies = z(st.n), z(1), z(st.n), z(st.n // 2), z(st.n // 2), z(1)
        L.gdn_kv_compact(self.kd, self.held, self.table, self.refs, table, refs, free, count, page_map, src, dst, copies)
        new, map_, a, b = st.compact()
        assert L.gdn_get_status(clear=True) == 0
        assert page_map.tolist() == map_ and copies.item() == len(a)
        assert src.tolist()[: len(a)] == a and dst.tolist()[: len(a)] == b
        assert all(x == -5 for x in src.tolist()[len(a):] + dst.tolist()[len(a):])
        assert free.tolist() == new.free
        self.st, self.table, self.refs, self.free, self.count = new, table, refs, free, count
        self.same()
        return src, dst, copies


def ones(n):
    return [1] * n


@pytest.mark.parametrize("B,page,T", [(1, 16, 1), (6, 16, 2), (13, 32, 5), (40, 64, 8), (1500, 16, 3)])
def test_cycles_with_forks_and_ends(gdn, B, page, T):
    """Random cycles: prompts, forks of whole and partly filled pages, drafts, rows that end, compaction; counts agree with the tables throughout."""
    rng = np.random.default_rng(B)
    M = 12
    st = State(B, page, M, B * 7 + 3, rng.permutation(B * 7 + 3).tolist())
    g = Device(st)
    lens = [0] * B
    for cycle in range(8):
        st = g.st
        live = [b for b in range(B) if lens[b]]
        empty = [b for b in range(B) if not lens[b] and not st.held[b]]
        rng.shuffle(empty)
        if cycle % 4 == 0:  # prompts for some
            add = [0] * B
            for b in empty[: max(1, B // 3)]:
                add[b] = int(rng.integers(1, 5 * page))
            N = sum(add) + 3
            g.plan(0, N, lens, add, ones(B))
            lens = [x + y for x, y in zip(lens, add)]
        elif cycle % 4 == 1 and live and empty:
            n = min(len(empty), 2 * len(live))
            src = [int(live[i % len(live)]) for i in range(n)]
            at = [int(rng.choice([lens[s], max(1, lens[s] // page * page), max(1, lens[s] // 2)])) for s in src]
            g.fork(src, empty[:n], at)
            for d, k in zip(empty[:n], at):
                lens[d] = k
        elif cycle % 4 == 2:
            add, active = rng.integers(0, T + 1, B), (rng.random(B) < 0.8).astype(int)
            add = [int(a) if lens[b] and -(-(lens[b] + int(a)) // page) <= M else 0 for b, a in enumerate(add)]
            before = list(lens)
            g.plan(T, B * T + 2, lens, add, active.tolist())
            lens = [before[b] + (int(rng.integers(0, add[b] + 1)) if active[b] else 0) for b in range(B)]
        else:
            for b in range(B):
                if rng.random() < 0.5:
                    lens[b] = 0
            g.plan(1, B, lens, [0] * B, ones(B))
            g.compact(bool(cycle & 4))
        g.st.check()
    g.plan(1, B, [0] * B, [0] * B, ones(B))
    assert g.st.count == g.st.n and not any(g.st.refs)


def test_pages_go_back_where_their_last_holder_does(gdn):
    """Rows that share a prefix end in one call, in two, and in the middle of others."""
    st = State(5, 16, 8, 30)
    g = Device(st)
    g.plan(0, 300, [0] * 5, [70, 0, 33, 0, 16], ones(5))
    g.fork([0, 0], [1, 3], [70, 40])
    lens = [70, 70, 33, 40, 16]
    g.plan(1, 5, [0, 70, 33, 40, 0], [0] * 5, ones(5))  # pages of row 0 stay with 1 and 3
    g.plan(1, 5, [0, 0, 33, 0, 0], [0] * 5, ones(5))    # and go where row 3 has them, not row 1
    g.plan(1, 5, [0, 0, 0, 0, 0], [0] * 5, ones(5))
    assert g.st.count == 30 and lens[0] == 70


def test_plan_shared_is_the_plan_where_nothing_is_shared(gdn):
    rng = np.random.default_rng(3)
    B, T, page, M, n = 20, 4, 32, 9, 120
    st = State(B, page, M, n)
    g = Device(st)
    held, table, free, count = ([0] * B, [[-1] * M for _ in range(B)], list(range(n)), n)
    lens = rng.integers(0, 200, B).tolist()
    for _ in range(4):
        add = rng.integers(0, T + 1, B).tolist()
        z = lambda k: torch.full((k,), -5, dtype=torch.int32, device="cuda")
        t = dict(held=dev(held), table=dev(table), free_list=dev(free), free_count=dev([count]))
        out = dict(q_start=z(B + 1), q_count=z(B), kv_len=z(B), slots=z(B * T), positions=z(B * T))
        L.gdn_kv_plan(g.kd, dev(lens), dev(add), dev(ones(B), torch.uint8), **t, **out, T=T)
        g.plan(T, B * T, lens, add, ones(B))
        held, table, free, count = t["held"].tolist(), t["table"].tolist(), t["free_list"].tolist(), t["free_count"].item()
        assert held == g.st.held and table == g.st.table and free[:count] == g.st.free[:count]
        lens = [x + int(rng.integers(0, a + 1)) for x, a in zip(lens, add)]
        lens = [0 if rng.random() < 0.2 else x for x in lens]


def test_plan_shared_refusals(gdn):
    st = State(4, 16, 4, 6)
    g = Device(st)
    g.plan(0, 100, [0] * 4, [40, 40, 10, 0], ones(4), status=NO_PAGES)  # 3 + 3 pages: row 2 gets none
    g.plan(1, 4, [40, 40, -1, 0], [0] * 4, ones(4), status=BAD_LEN)
    # a cell outside the cache, and a page without a holder: dropped
    g.st.table[0][2], g.st.refs[g.st.table[1][2]] = 77, 0
    g.upload()
    g.plan(1, 4, [0, 0, 0, 0], [0] * 4, ones(4), status=BAD_INDEX)


def test_fork_refusals(gdn):
    st = State(9, 16, 6, 12)
    g = Device(st)
    g.plan(0, 200, [0] * 9, [40, 0, 64, 0, 0, 0, 0, 0, 0], ones(9))  # 3 + 4 pages, 5 free
    g.fork([0, -1, 0, 0, 9], [1, 3, 9, 0, 3], [40, 5, 5, 5, 5], status=BAD_ROW)
    g.fork([0, 0, 0], [3, 4, 5], [49, -1, 1 << 30], status=BAD_LEN)
    g.fork([0, 2, 1], [3, 3, 3], [20, 20, 20], status=BAD_ROW)      # the first that asks has it
    g.fork([3], [2], [5], status=BAD_ROW)                           # not empty
    g.fork([5], [6], [0])                                           # nothing of an empty row
    g.fork([2, 4], [4, 5], [64, 3], status=BAD_LEN)                 # a destination is no source in the same call
    g.fork([0, 0, 2, 0, 2], [5, 6, 7, 8, 0], [17, 33, 48, 1, 0], status=BAD_ROW)
    g.st.check()
    # pages run out: those that need none still go through
    st = State(7, 16, 6, 8)
    g = Device(st)
    g.plan(0, 200, [0] * 7, [33, 35, 0, 0, 0, 0, 0], ones(7))
    g.fork([0, 1, 1, 0, 0], [2, 3, 4, 5, 6], [33, 35, 3, 32, 31], status=NO_PAGES)
    g.st.check()


def test_many_forks_of_long_rows(gdn):
    """More pairs than a CTA has threads, and long tables."""
    B, M = 1300, 40
    st = State(B, 16, M, 1500)
    g = Device(st)
    add = [0] * B
    add[7], add[1299] = 600, 333
    g.plan(0, 1000, [0] * B, add, ones(B))
    dst = [b for b in range(B) if not add[b]]
    g.fork([7 if b % 2 else 1299 for b in dst], dst, [600 - b % 40 if b % 2 else 333 - b % 16 for b in dst])
    g.st.check()
    lens = [0] * B
    g.plan(2, 2 * B, lens, [0] * B, ones(B))
    assert g.st.count == 1500


@pytest.mark.parametrize("n", [1, 2, 5, 127, 128, 129, 4096, 4097, 5001, 20011])
@pytest.mark.parametrize("full", [0.0, 0.3, 0.95, 1.0])
def test_compact_sizes(gdn, n, full):
    """Any number of pages and of gaps, sources and counts at addresses that are no multiple of 16."""
    rng = np.random.default_rng(n)
    st = State(3, 16, max(1, n), n)
    used = [i for i in range(n) if rng.random() < full]
    rng.shuffle(used)
    for i, page in enumerate(used):
        b = i % 3
        st.table[b][st.held[b]] = page
        st.held[b] += 1
        st.refs[page] = 1
    free = [i for i in range(n) if not st.refs[i]]
    st.free, st.count = free + [-1] * (n - len(free)), len(free)
    for in_place in (False, True):
        g = Device(st)
        g.refs = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), g.refs])[1:] if n % 2 else g.refs
        g.compact(in_place)
        g.st.check()


def test_compact_of_bad_cells(gdn):
    st = State(2, 16, 3, 9)
    g = Device(st)
    g.plan(0, 100, [0, 0], [40, 20], ones(2))
    table = g.table.clone()
    g.table[0, 1], g.table[1, 0] = 99, 0  # outside the cache; not in use
    assert g.refs[0].item() == 0
    out = dict(new_table=torch.zeros_like(g.table), new_refs=torch.zeros_like(g.refs), new_free_list=torch.zeros_like(g.free), new_free_count=torch.zeros_like(g.count),
               page_map=torch.zeros_like(g.refs), copy_src=torch.zeros_like(g.refs), copy_dst=torch.zeros_like(g.refs), copy_count=torch.zeros_like(g.count))
    L.gdn_kv_compact(g.kd, g.held, g.table, g.refs, **out)
    assert L.gdn_get_status(clear=True) == BAD_INDEX
    assert out["new_table"][0, 1].item() == -1 and out["new_table"][1, 0].item() == -1
    assert out["new_table"][0, 0].item() == out["page_map"][table[0, 0]].item() >= 0


@pytest.mark.parametrize("d,page,H_kv,layers", [(64, 16, 1, 1), (128, 32, 3, 5), (256, 64, 2, 10), (64, 64, 8, 256)])
def test_copies(gdn, d, page, H_kv, layers):
    """Whole pages in every layer; the count cuts the list, negative pages are skipped, bad ones named."""
    n = 24
    kd = L.kv4_dims(1, H_kv, H_kv, d, page, 4, n)
    size = L.gdn_kv4_page_bytes(kd)
    gen = torch.Generator(device="cuda").manual_seed(layers)
    caches = [torch.randint(0, 256, (n + 1, size), generator=gen, dtype=torch.uint8, device="cuda") for _ in range(layers)]
    src, dst = [3, 5, -1, 0, -2, 23, 9], [4, 6, 2, -1, -2, 22, 10]
    for count in (None, 0, 1, 3, 7, 100, -4):
        want = [c.clone() for c in caches]
        k = 7 if count is None else max(0, min(count, 7))
        for w in want:
            for a, b in list(zip(src, dst))[:k]:
                if a >= 0 and b >= 0:
                    w[b] = w[a]
        L.gdn_kv_copy_pages(kd, caches, dev(src), dev(dst), count=None if count is None else dev([count]))
        assert all(torch.equal(a, b) for a, b in zip(want, caches))
        assert L.gdn_get_status(clear=True) == 0
    before = [c.clone() for c in caches]
    L.gdn_kv_copy_pages(kd, caches, dev([n, 1]), dev([2, n]))
    assert L.gdn_get_status(clear=True) == BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(before, caches))


def test_forked_rows_attend_as_their_source_does(gdn):
    """Append, fork in the middle of a page, copy, append different tokens, attend; then compact and attend again: a row's
    output depends on its own tokens alone."""
    B, P, M, H, d, T = 4, 16, 8, 2, 64, 3
    n = 40
    st = State(B, P, M, n, np.random.default_rng(0).permutation(n).tolist())
    g = Device(st, H, d)
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.zeros(n * L.gdn_kv4_page_bytes(g.kd), dtype=torch.uint8, device="cuda")
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")

    def step(lens, add, T, N, k, v, q):
        out = dict(q_start=z(B + 1), q_count=z(B), kv_len=z(B), slots=z(N), positions=z(N))
        L.gdn_kv_plan_shared(g.kd, dev(lens), dev(add), dev(ones(B), torch.uint8), g.held, g.table, g.free, g.count, g.refs, **out, T=T)
        q_out, o = torch.empty_like(q), torch.zeros_like(q)
        L.gdn_kv4_append(g.kd, q, k, v, out["positions"][None], None, b"", out["slots"], cache, q_out)
        span = max(max(add), 1)
        ws = z(L.gdn_kv4_attend_workspace_bytes(g.kd, N, span), dtype=torch.uint8)
        L.gdn_kv4_attend(g.kd, q_out, cache, g.table, out["q_start"], out["q_count"], out["kv_len"], d ** -0.5, o, ws, span)
        return out, o

    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    n0 = 41
    k, v, q = rand(n0, H, d), rand(n0, H, d), rand(n0, H, d)
    step([0] * B, [n0, 0, 0, 0], 0, n0, k, v, q)
    src, dst = z(3), z(3)
    L.gdn_kv_fork(g.kd, dev([0, 0, 0]), dev([1, 2, 3]), dev([n0, n0, 20]), g.held, g.table, g.free, g.count, g.refs, src, dst)
    L.gdn_kv_copy_pages(g.kd, [cache], src, dst)
    lens = [n0, n0, n0, 20]
    k1, v1, q1 = rand(T, H, d), rand(T, H, d), rand(T, H, d)
    k2, v2, q2 = rand(T, H, d), rand(T, H, d), rand(T, H, d)
    tile = lambda a, b: torch.cat([a, b, a, a])  # rows 0 and 2 go on alike, row 1 otherwise, row 3 from its own length
    out, o = step(lens, [T] * B, T, B * T, tile(k1, k2), tile(v1, v2), tile(q1, q2))
    o = o.view(B, T, H, d)
    assert torch.equal(o[0], o[2]) and not torch.equal(o[0], o[1]) and not torch.equal(o[0], o[3])
    # against plain attention over what the cache stands for
    for b in range(B):
        total = lens[b] + T
        at = g.table[b][torch.arange(total, device="cuda") // P] * P + torch.arange(total, device="cuda") % P
        kr, vr = (torch.empty(total, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        L.gdn_kv4_read(g.kd, at.to(torch.int32), cache, kr, vr)
        for t in range(T):
            s = torch.einsum("hd,nhd->hn", (q2 if b == 1 else q1)[t].double(), kr[: lens[b] + t + 1].double()) * d ** -0.5
            ref = torch.einsum("hn,nhd->hd", s.softmax(-1), vr[: lens[b] + t + 1].double())
            # keys and values read back are rounded to bf16 (2^-9 of magnitudes up to 4 in 64 products), outputs too
            assert (o[b, t].double() - ref).abs().max() < 0.03
    new = dict(new_table=torch.zeros_like(g.table), new_refs=torch.zeros_like(g.refs), new_free_list=torch.zeros_like(g.free), new_free_count=torch.zeros_like(g.count),
               page_map=torch.zeros_like(g.refs), copy_src=z(n // 2), copy_dst=z(n // 2), copy_count=z(1))
    L.gdn_kv_compact(g.kd, g.held, g.table, g.refs, **new)
    L.gdn_kv_copy_pages(g.kd, [cache], new["copy_src"], new["copy_dst"], count=new["copy_count"])
    o2 = torch.zeros_like(o)
    ws = z(L.gdn_kv4_attend_workspace_bytes(g.kd, B * T, T), dtype=torch.uint8)
    for table in (g.table, new["new_table"]):  # the old tables stay valid until something is appended
        L.gdn_kv4_attend(g.kd, tile(q1, q2), cache, table, out["q_start"], out["q_count"], out["kv_len"], d ** -0.5, o2, ws, T)
        assert torch.equal(o, o2)
    assert L.gdn_get_status(clear=True) == 0


def test_captured_cycle(gdn):
    """Fork, copy, plan and end captured into a graph and replayed: the state comes back each time."""
    B, P, M, n = 6, 16, 6, 30
    st = State(B, P, M, n)
    g = Device(st)
    g.plan(0, 200, [0] * B, [50, 0, 0, 0, 0, 0], ones(B))
    size = L.gdn_kv4_page_bytes(g.kd)
    cache = torch.randint(0, 256, (n, size), dtype=torch.uint8, device="cuda")
    z = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")
    args = dict(src=dev([0] * 5), dst=dev([1, 2, 3, 4, 5]), at=dev([50, 33, 16, 50, 1]))
    a, b = z(5), z(5)
    out = dict(q_start=z(B + 1), q_count=z(B), kv_len=z(B), slots=z(B * 2), positions=z(B * 2))
    lens, add, none, back, act = dev([50, 50, 33, 16, 50, 1]), dev([2] * B), dev([0] * B), dev([50, 0, 0, 0, 0, 0]), dev(ones(B), torch.uint8)

    def cycle():
        L.gdn_kv_fork(g.kd, args["src"], args["dst"], args["at"], g.held, g.table, g.free, g.count, g.refs, a, b)
        L.gdn_kv_copy_pages(g.kd, [cache], a, b)
        L.gdn_kv_plan_shared(g.kd, lens, add, act, g.held, g.table, g.free, g.count, g.refs, **out, T=2)

    def end():
        L.gdn_kv_plan_shared(g.kd, back, none, act, g.held, g.table, g.free, g.count, g.refs, out["q_start"], out["q_count"], out["kv_len"], z(B * 2), z(B * 2), T=2)

    cycle(), end()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cycle()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        table, live = g.table.tolist(), [x for x in zip(a.tolist(), b.tolist()) if x[0] >= 0]
        assert len(live) == 4 and all(torch.equal(cache[x], cache[y]) for x, y in live)
        assert all(table[d][: w // P] == table[0][: w // P] for d, w in ((1, 50), (2, 33), (3, 16), (4, 50)))
        end()
        torch.cuda.synchronize()
        assert g.count.item() == n - 4 and g.refs.sum().item() == 4 and L.gdn_get_status() == 0
