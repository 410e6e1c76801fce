"""The hybrid decoding example: its cycles leave the cache, the lengths and the
pages in step, and its last attention is the one over what the cache stands for."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref as R
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


def load_example():
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("rows,prompt,cycles,draft", [(3, 77, 9, 1), (1, 1, 5, 0), (2, 40, 40, 3)])
def test_hybrid_decode(gdn, rows, prompt, cycles, draft):
    m, _ = load_example().run(rows=rows, prompt=prompt, cycles=cycles, draft=draft)
    T = draft + 1
    offsets, kv_len, held = (t.cpu().numpy() for t in (m.offsets, m.kv_len, m.held))
    keep = m.keep.cpu().numpy()
    # one cycle runs before the graph, which its capture does not run
    assert (offsets >= prompt + cycles + 1).all() and (offsets <= prompt + (cycles + 1) * T).all()
    assert (kv_len == offsets - keep + T).all() and (held == -(-kv_len // m.kd.page)).all()
    assert m.free_count.item() == m.kd.n_pages - held.sum()
    # the last cycle's attention against the cache's own values in 64 bits
    table, q, o = m.table.cpu().numpy(), m.step["q"].double().cpu().numpy(), m.step["o"].double().cpu().numpy()
    cache = R.Cache(m.kd.n_pages, m.H_kv, m.kd.page, m.d)
    data = m.pages.cpu().numpy().reshape(cache.bytes.shape)
    G = m.H_q // m.H_kv
    for b in range(rows):
        n = int(kv_len[b])
        pos = np.arange(n)
        k, v = cache.read(table[b, pos // m.kd.page] * m.kd.page + pos % m.kd.page, data)
        for i in range(T):
            see = n - T + i + 1
            for h in range(m.H_q):
                s = k[:see, h // G] @ q[b * T + i, h] * m.d ** -0.5
                p = np.exp(s - s.max())
                p /= p.sum()
                want, size = p @ v[:see, h // G], p @ np.abs(v[:see, h // G])
                # q exact in fp16 up to its power of two; keys rounded to fp16 at most once move a score by
                # 2^-11 of its terms' sum, which moves each probability as much; P and V one fp16 rounding
                # each, the output one bf16 rounding
                terms = (np.abs(k[:see, h // G]) @ np.abs(q[b * T + i, h]) * m.d ** -0.5).max()
                bound = size * (2 * 2 ** -11 * terms + 3 * 2 ** -11 + 2 ** -8) + 2 ** -8 * np.abs(want) + 1e-6
                assert (np.abs(o[b * T + i, h] - want) <= bound).all()
