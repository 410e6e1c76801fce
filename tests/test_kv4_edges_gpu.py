"""Edges of the paged 4-bit cache's calls."""
import numpy as np
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref as R
from tests.test_kv4_gpu import append_case, attend_case, bits, run_append, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 32), (256, 256)])
def test_position_outside_does_not_turn(gdn, d, rot, pairs):
    """Channels whose position is outside the table come out as they went in: an infinity in the other channel of the pair
    leaves no NaN, a zero keeps its sign.  The pairs of another axis turn as ever."""
    N, Hq, Hkv, page = 9, 3, 1, 16
    x, pos, axis, n_pages, slots = append_case(N, Hq, Hkv, d, rot, 2, page, pairs)
    half = rot // 2
    axis = bytes([0, 1] * (half // 2))
    a, b = (lambda i: (2 * i, 2 * i + 1) if pairs else (i, i + half))(np.arange(half))
    x[:, 0] = -0.0
    x[:, 1, a[1::2]] = float("inf")
    pos[1, :5], pos[1, 5:] = -1, 5000
    slots[::2] = -1
    cache = R.Cache(n_pages, Hkv, page, d, seed=1)
    q_out, pages, k, v, status = run_append(x, pos, axis, n_pages, slots, Hq, Hkv, d, rot, page, pairs, cache)
    assert status == L.GDN_STATUS_BAD_INDEX and np.array_equal(pages, cache.bytes)
    q = x.float().numpy()[:, :Hq]
    tab = R.rope_table(5000, rot).numpy()
    cs = np.stack([tab[np.clip(pos[axis[i]], 0, 4999), i] for i in range(half)], 1)
    want = R.rotate(q, cs, rot, pairs)
    for c in (a, b):
        want[..., c[1::2]] = q[..., c[1::2]]
    assert torch.equal(bits(q_out), bits(R.bf16(want)))


@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("cell", [-1, -2, -3, -(1 << 31)])
def test_attend_negative_cell_raises_status(gdn, T, cell):
    """Any negative cell where a row has keys is a page outside the cache; not a bit of the other row changes."""
    cache, table, q_start, q_count, kv_len, q = attend_case(8, 2, 128, 16, [(100, T, T), (80, T, T)], seed=1)
    good, *_ = run_attend(cache, table, q_start, q_count, kv_len, q, 0.1, T)
    assert L.gdn_get_status(clear=True) == 0
    table[0, 3] = cell
    out, *_ = run_attend(cache, table, q_start, q_count, kv_len, q, 0.1, T)
    assert L.gdn_get_status(clear=True) == L.GDN_STATUS_BAD_INDEX
    assert torch.equal(bits(out[T:]), bits(good[T:]))
