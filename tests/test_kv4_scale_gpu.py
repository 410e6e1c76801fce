"""Attention at scales far from 1: tiny ones leave the mean of the visible
values, and rows without a query, or without a visible key, their zeros."""
import numpy as np
import pytest

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref as R
from tests.test_kv4_gpu import attend_case, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (4, 2, 128), (4, 2, 256)], ids=lambda v: str(v))
@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("scale", [1e-12, 1e-20, 1e-30, 1e-40])
def test_tiny_scale(gdn, Hq, Hkv, d, T, scale):
    """Queries of zeros and tokens of a span without a query stand next to ordinary ones."""
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 16, [(100, T - 1, T), (1, T, T), (77, T, T)], seed=2)
    q[::2] = 0
    out, *_ = run_attend(cache, table, q_start, q_count, kv_len, q, scale, T)
    assert L.gdn_get_status(clear=True) == 0
    want, tol = R.attend(q.double().numpy(), cache, table, q_start, q_count, kv_len, scale)
    got = out.cpu().double().numpy()
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (4, 2, 128), (4, 2, 256)], ids=lambda v: str(v))
@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("scale", [0.1, 1e-12, 1e-30])
def test_tiny_queries(gdn, Hq, Hkv, d, T, scale):
    """Queries near the least bf16 numbers, which the kernels scale up before they round."""
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 16, [(100, T - 1, T), (1, T, T), (77, T, T)], seed=2)
    q = (q.float() * 1e-30).bfloat16()
    out, *_ = run_attend(cache, table, q_start, q_count, kv_len, q, scale, T)
    assert L.gdn_get_status(clear=True) == 0
    want, tol = R.attend(q.double().numpy(), cache, table, q_start, q_count, kv_len, scale)
    got = out.cpu().double().numpy()
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()
