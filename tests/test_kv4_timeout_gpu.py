"""The bounded-wait failure path of the cache attention, forced without any GPU
fault: gdn_test_kv4_attend_timeout makes the barrier of the first CTA's first
copies expect an arrival that never comes, so that its waits run out.  The
kernel must return, flag GDN_STATUS_TIMEOUT and leave the context usable; on a
zero-filled workspace the next ordinary call gives its usual bits."""
import time

import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests.test_kv4_gpu import attend_case, bits, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (4, 2, 128), (4, 2, 256)], ids=lambda v: str(v))
@pytest.mark.parametrize("rows", [
    [(100, 2, 2)],                                    # one unit, its only copies
    [(5000, 2, 2), (40, 1, 2), (3000, 2, 2)],         # few rows: cut units, the next unit's copies ahead
    [(100, 70, 70)],                                  # many rows: fewer tiles than the ring has places
    [(2500, 90, 90), (90, 90, 90), (1500, 70, 90)],   # more tiles, cut units
    [(300, 60, 60)] * 40,                             # several units a CTA
], ids=["few-one", "few-cut", "many-one", "many-cut", "many-units"])
def test_bounded_wait_runs_out_and_recovers(gdn, Hq, Hkv, d, rows):
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 32, rows, seed=1)
    T = max(s for _, _, s in rows)
    want, ws, kd, args = run_attend(cache, table, q_start, q_count, kv_len, q, 0.1, T)
    torch.cuda.synchronize()
    assert L.gdn_get_status(clear=True) == 0
    for _ in range(2):
        out = torch.empty_like(want)
        t0 = time.perf_counter()
        L.gdn_test_kv4_attend_timeout(kd, *args, 0.1, out, ws, T, wait_limit=4000)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 2, "each wait gives up after some milliseconds"
        assert L.gdn_get_status(clear=True) == L.GDN_STATUS_TIMEOUT
        ws.zero_()
        L.gdn_kv4_attend(kd, *args, 0.1, out, ws, T)
        assert L.gdn_get_status(clear=True) == 0 and torch.equal(bits(out), bits(want))
