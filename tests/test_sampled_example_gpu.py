"""Several sampled continuations of a prompt, end to end: prefill, fork, sampled cycles in a graph, ends, compaction,
cycles again.  What the rows hold stays in step throughout, and the last attention is the one over what the cache
stands for."""
import numpy as np
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref as R
from tests.test_hybrid_example_gpu import load_example

pytestmark = pytest.mark.gpu


def check_pages(m):
    """Every page is held as often as its count says, or free once."""
    held, table, refs = m.held.tolist(), m.table.tolist(), m.refs.tolist()
    seen = [0] * m.kd.n_pages
    for b in range(m.B):
        for c in range(held[b]):
            seen[table[b][c]] += 1
    assert seen == refs
    free = m.free_list.tolist()[: m.free_count.item()]
    assert sorted(free) == [i for i, s in enumerate(seen) if not s]
    return seen


def check_attention(m):
    table, q, o = m.table.cpu().numpy(), m.step["q"].double().cpu().numpy(), m.step["o"].double().cpu().numpy()
    kv_len = m.kv_len.tolist()
    cache = R.Cache(m.kd.n_pages, m.H_kv, m.kd.page, m.d)
    data = m.pages.cpu().numpy().reshape(cache.bytes.shape)
    T, G = m.T, m.H_q // m.H_kv
    for b in range(m.B):
        if not m.active[b]:
            assert (o[b * T:(b + 1) * T] == 0).all()
            continue
        pos = np.arange(kv_len[b])
        k, v = cache.read(table[b, pos // m.kd.page] * m.kd.page + pos % m.kd.page, data)
        for i in range(T):
            see = kv_len[b] - T + i + 1
            for h in range(m.H_q):
                s = k[:see, h // G] @ q[b * T + i, h] * m.d ** -0.5
                p = np.exp(s - s.max())
                p /= p.sum()
                want, size = p @ v[:see, h // G], p @ np.abs(v[:see, h // G])
                # as in the greedy example's test: keys, P and V one fp16 rounding each, the output one of bf16
                terms = (np.abs(k[:see, h // G]) @ np.abs(q[b * T + i, h]) * m.d ** -0.5).max()
                bound = size * (2 * 2 ** -11 * terms + 3 * 2 ** -11 + 2 ** -8) + 2 ** -8 * np.abs(want) + 1e-6
                assert (np.abs(o[b * T + i, h] - want) <= bound).all()


@pytest.mark.parametrize("rows,prompt,cycles,draft,samples", [(2, 77, 9, 1, 3), (1, 64, 12, 3, 5), (3, 31, 4, 0, 2)])
def test_sampled_continuations(gdn, rows, prompt, cycles, draft, samples):
    m, _ = load_example().run(rows=rows, prompt=prompt, cycles=cycles, draft=draft, samples=samples, temperature=1.0)
    B, T, P = rows * samples, draft + 1, m.kd.page
    assert m.B == B
    offsets = m.offsets.cpu().numpy()
    assert (offsets >= prompt + cycles + 1).all() and (offsets <= prompt + (cycles + 1) * T).all()
    # the prompts' full pages stand in all their rows, and nowhere else
    table, whole = m.table.tolist(), prompt // P
    for b in range(B):
        assert table[b][:whole] == table[b % rows][:whole]
    seen = check_pages(m)
    assert all(seen[p] == samples for b in range(rows) for p in table[b][:whole]) and sum(s > 1 for s in seen) == rows * whole
    check_attention(m)
    if prompt > 60:  # rows of one prompt go different ways
        assert len({tuple(m.tokens[b].tolist()) + (int(offsets[b]),) for b in range(0, B, rows)}) > 1 or samples == 1
    # the prompts' own rows end first; what their continuations share stays
    m.end(torch.arange(rows, device="cuda"))
    seen = check_pages(m)
    assert all(seen[p] == samples - 1 for b in range(rows) for p in table[b][:whole])
    before = [m.pages.view(m.kd.n_pages, -1)[m.table[b, : m.held[b]].long()].clone() for b in range(B)]
    used = m.compact()
    assert all(s > 0 for s in check_pages(m)[:used])
    for b in range(B):
        assert torch.equal(before[b], m.pages.view(m.kd.n_pages, -1)[m.table[b, : m.held[b]].long()])
    for _ in range(3):
        m.cycle()
    check_pages(m)
    check_attention(m)
    m.end(torch.arange(B, device="cuda"))
    check_pages(m)
    assert m.free_count.item() == m.kd.n_pages and L.gdn_get_status() == 0
