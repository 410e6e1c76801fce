"""Attention over cached groups whose levels pass fp16's largest number.

An entry's step and base are finite fp16 numbers, but the level base + 15 * step
that they stand for may lie anywhere up to 16 * 65504.  Keys and values of such
groups count as what they stand for, in both forms of the call, and a query that
does not see them is not touched by them."""
import numpy as np
import pytest

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref as R
from tests.test_kv4_gpu import attend_case, bits, run_attend

pytestmark = pytest.mark.gpu

# least and largest value of the group: its top level is 65520 (which fp16 rounds to infinity), 65536, 70144, 982560 (base and
# step are held at 65504), 917056, and a group whose large values are negative
SPANS = [(0.0, 65504.0), (-65504.0, 65504.0), (0.0, 70144.0), (0.0, 1e6), (-3e38, 3e38), (-1e6, 0.0)]
SHAPES = [(4, 2, 64), (4, 2, 128), (4, 2, 256)]


def put(cache, table, b, t, which, group, lo, hi):
    """Token t of row b, every head: group `group` of its key (0) or value (1) becomes zeros with one lo and one hi."""
    slot = int(table[b, t // cache.P]) * cache.P + t % cache.P
    k, v = (x[0].astype(np.float32) for x in cache.read([slot]))
    ch = [c for c in range(cache.d) if (c // 8) % (cache.d // 64) == group]
    x = v if which else k
    x[:, ch] = 0
    x[:, ch[0]], x[:, ch[3]] = lo, hi
    cache.write(slot, k, v)
    return ch[0], ch[3]


def check(cache, table, q_start, q_count, kv_len, q, T):
    scale = cache.d ** -0.5
    out, *_ = run_attend(cache, table, q_start, q_count, kv_len, q, scale, T)
    assert L.gdn_get_status(clear=True) == 0
    want, tol = R.attend(q.double().numpy(), cache, table, q_start, q_count, kv_len, scale)
    got = out.cpu().double().numpy()
    assert np.isfinite(got).all()
    # numbers of a tile with such a group may be formed as sixteenths: they keep 16 * 2^-25 of absolute precision
    assert (np.abs(got - want) <= tol + 2.0 ** -20).all()
    return out


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES, ids=lambda v: str(v))
@pytest.mark.parametrize("T,n", [(2, 100), (2, 3000), (70, 100), (70, 1500)])
@pytest.mark.parametrize("span", SPANS, ids=lambda s: f"{s[0]:g}..{s[1]:g}")
def test_value_past_fp16(gdn, Hq, Hkv, d, T, n, span):
    """The newest token's value, which only the last query sees."""
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 16, [(n, T, T), (90, T, T)], seed=3)
    put(cache, table, 0, n - 1, 1, d // 64 - 1, *span)
    check(cache, table, q_start, q_count, kv_len, q, T)


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES, ids=lambda v: str(v))
@pytest.mark.parametrize("T,n", [(2, 100), (2, 3000), (70, 300), (70, 1500)])
def test_values_past_fp16_that_all_see(gdn, Hq, Hkv, d, T, n):
    """Such values among the keys that every query sees, and one behind the first: weights and sums go on over both."""
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 32, [(90, T, T), (n, T, T)], seed=4)
    for i, span in enumerate(SPANS):
        put(cache, table, 1, 7 + i * (n - T - 8) // len(SPANS), 1, i % (d // 64), *span)
    put(cache, table, 1, n - T + 1, 1, 0, 0.0, 1e6)
    check(cache, table, q_start, q_count, kv_len, q, T)


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES, ids=lambda v: str(v))
@pytest.mark.parametrize("T,n", [(2, 100), (2, 3000), (70, 100), (70, 1500)])
@pytest.mark.parametrize("span", SPANS, ids=lambda s: f"{s[0]:g}..{s[1]:g}")
def test_key_past_fp16(gdn, Hq, Hkv, d, T, n, span):
    """Keys of that kind, met by queries that are small in those channels, so that their scores are ordinary numbers."""
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 16, [(n, T, T), (90, T, T)], seed=5)
    for t in (n - 1, (n - T) // 2):
        for c in put(cache, table, 0, t, 0, 0, *span):
            q[..., c] = 2.0 ** -15
    check(cache, table, q_start, q_count, kv_len, q, T)


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES, ids=lambda v: str(v))
@pytest.mark.parametrize("T", [2, 70])
def test_keys_and_values_past_fp16_in_one_tile(gdn, Hq, Hkv, d, T):
    n = 333
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 64, [(n, T, T)], seed=6)
    for t in (20, 21, 200):
        for c in put(cache, table, 0, t, 0, 0, 0.0, 1e6):
            q[..., c] = -(2.0 ** -16)
        put(cache, table, 0, t + (t == 20), 1, d // 64 - 1, -3e38, 3e38)
    check(cache, table, q_start, q_count, kv_len, q, T)


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES, ids=lambda v: str(v))
@pytest.mark.parametrize("T", [2, 70])
def test_places_behind_a_row_do_not_count(gdn, Hq, Hkv, d, T):
    """What the pages hold behind a row's end, NaN or levels past fp16, leaves not a bit of the result different."""
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 64, [(75, T, T), (140, T, T)], seed=7)
    a = check(cache, table, q_start, q_count, kv_len, q, T)
    for b, n in ((0, 75), (1, 140)):
        for t in range(n, -(-n // 64) * 64):
            slot = int(table[b, t // 64]) * 64 + t % 64
            big = np.full((Hkv, d), 3e38, np.float32)
            big[:, ::5] = -1.0
            cache.write(slot, big, big)
    assert bits(check(cache, table, q_start, q_count, kv_len, q, T)).equal(bits(a))
