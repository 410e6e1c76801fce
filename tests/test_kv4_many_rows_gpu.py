"""Cache attention where the line of work is laid by more rows than a CTA has
threads, with wide groups of heads, and with scales of every sign."""
import numpy as np
import pytest

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref as R
from tests.test_kv4_gpu import attend_case, check_attend, run_attend

pytestmark = pytest.mark.gpu


def short_rows(B, T, seed):
    """B rows of up to 40 keys, T tokens each at most: idle ones, empty spans, rows without a key among them."""
    rng = np.random.default_rng(seed)
    rows = []
    for _ in range(B):
        span = int(rng.integers(0, T + 1))
        count = int(rng.integers(0, span + 1))
        rows.append((int(rng.integers(count if rng.random() < 0.8 else 0, 41)), count, span))
    rows[B // 2] = (500, T, T)
    return rows


@pytest.mark.parametrize("B", [700, 1500])
@pytest.mark.parametrize("Hq,Hkv,d,T", [(2, 1, 64, 2), (2, 1, 128, 2), (2, 1, 256, 2),      # few rows: 384, 384 and 256 threads
                                        (8, 1, 64, 6), (8, 1, 128, 6), (4, 1, 256, 6)])      # many rows: 640 threads
def test_more_rows_than_threads(gdn, B, Hq, Hkv, d, T):
    check_attend(Hq, Hkv, d, 16, short_rows(B, T, B + d), pad=3, seed=B)


@pytest.mark.parametrize("G", [16, 33, 50, 64])
@pytest.mark.parametrize("Hkv,d", [(2, 64), (1, 128), (1, 256)])
def test_wide_groups_of_heads(gdn, G, Hkv, d):
    """Up to 64 query heads a key head: tiles of one to eight tokens, cut rows, tokens that see nothing."""
    check_attend(G * Hkv, Hkv, d, 32, [(3, 5, 5), (300, 1, 5), (77, 4, 5), (0, 0, 5), (2000, 3, 5)], seed=G)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (4, 2, 128), (4, 2, 256)])
@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("scale", [-0.1, 0.0, -1e-12])
def test_scales_of_every_sign(gdn, Hq, Hkv, d, T, scale):
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 16, [(200, T, T), (90, T - 1, T)], seed=3)
    out, *_ = run_attend(cache, table, q_start, q_count, kv_len, q, scale, T)
    assert L.gdn_get_status(clear=True) == 0
    want, tol = R.attend(q.double().numpy(), cache, table, q_start, q_count, kv_len, scale)
    assert (np.abs(out.cpu().double().numpy() - want) <= tol).all()


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (4, 2, 128), (4, 2, 256)])
@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("place", [0, 1], ids=["step", "base"])
@pytest.mark.parametrize("which", [0, 1], ids=["key", "value"])
def test_infinite_entry_stays_with_its_queries(gdn, Hq, Hkv, d, T, place, which):
    """The newest token with an infinite step or base: the queries before it are untouched."""
    n = 150
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 16, [(n, T, T), (80, T, T)], seed=6)
    want, tol = R.attend(q.double().numpy(), cache, table, q_start, q_count, kv_len, d ** -0.5)
    at = 2 * cache.a + which * cache.e + ((n - 1) % 16) * (d // 64) * 4 + 2 * place
    cache.bytes[table[0, (n - 1) // 16], :, at: at + 2] = np.frombuffer(np.float16(np.inf).tobytes(), np.uint8)
    out, *_ = run_attend(cache, table, q_start, q_count, kv_len, q, d ** -0.5, T)
    got = out.cpu().double().numpy()
    rest = [t for t in range(2 * T) if t != T - 1]
    assert (np.abs(got - want)[rest] <= tol[rest]).all()
    if which:  # the group's channels, in every head of the query that sees it
        first = [c for c in range(d) if (c // 8) % (d // 64) == 0]
        other = [c for c in range(d) if (c // 8) % (d // 64) != 0]
        assert not np.isfinite(got[T - 1][:, first]).any()
        assert (np.abs(got - want)[T - 1][:, other] <= tol[T - 1][:, other]).all()
