"""Shared pages without a GPU: refusals before any launch, and the references' own sense."""
import ctypes

import numpy as np
import pytest

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref
from tests.kv_pages_ref import State

G = 1 << 20  # an aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return L.load()


def kd(**kw):
    return L.kv4_dims(**{**dict(B=8, H_q=16, H_kv=2, d=256, page=64, max_pages=512, n_pages=4096), **kw})


BAD = [dict(B=-1), dict(B=65536), dict(d=32), dict(page=8), dict(H_q=15), dict(H_kv=0), dict(max_pages=0), dict(n_pages=0)]


def layers(*p):
    return (ctypes.c_void_p * max(len(p), 1))(*p)


@pytest.mark.parametrize("kw", BAD, ids=str)
def test_bad_dims(lib, kw):
    d, f = ctypes.byref(kd(**kw)), L.GDN_ERR_UNSUPPORTED
    assert lib.gdn_kv_plan_shared(d, 2, 16, *([G] * 13), None) == f and L.gdn_last_error()
    assert lib.gdn_kv_fork(d, 2, *([G] * 10), None) == f
    assert lib.gdn_kv_compact(d, *([G] * 11), None) == f
    assert lib.gdn_kv_copy_pages(d, 1, layers(G), 2, G, G, None, None) == f


@pytest.mark.parametrize("name,lead,count,bytes_at", [("gdn_kv_plan_shared", (2, 16), 13, 2), ("gdn_kv_fork", (4,), 10, None), ("gdn_kv_compact", (), 11, None)])
def test_pointers(lib, name, lead, count, bytes_at):
    d = ctypes.byref(kd())
    for i in range(count):
        for bad, code in ((None, L.GDN_ERR_INVALID_ARG), (G + 2, L.GDN_ERR_MISALIGNED)):
            if i == bytes_at and bad:
                continue  # active: bytes, any address
            a = [G] * count
            a[i] = bad
            assert getattr(lib, name)(d, *lead, *a, None) == code, i
    assert getattr(lib, name)(None, *lead, *([G] * count), None) == L.GDN_ERR_INVALID_ARG


def test_sizes(lib):
    d = ctypes.byref(kd())
    a = [G] * 13
    assert lib.gdn_kv_plan_shared(d, -1, 16, *a, None) == L.GDN_ERR_INVALID_ARG
    assert lib.gdn_kv_plan_shared(d, 2, 15, *a, None) == L.GDN_ERR_INVALID_ARG
    assert lib.gdn_kv_plan_shared(d, 2, -1, *a, None) == L.GDN_ERR_UNSUPPORTED
    assert lib.gdn_kv_plan_shared(ctypes.byref(kd(B=4096, max_pages=1 << 19)), 0, 16, *a, None) == L.GDN_ERR_UNSUPPORTED
    assert lib.gdn_kv_plan_shared(ctypes.byref(kd(B=0)), 2, 16, *([None] * 13), None) == L.GDN_OK
    assert lib.gdn_kv_fork(d, -1, *([G] * 10), None) == L.GDN_ERR_UNSUPPORTED
    assert lib.gdn_kv_fork(d, 65536, *([G] * 10), None) == L.GDN_ERR_UNSUPPORTED
    assert lib.gdn_kv_fork(d, 0, *([None] * 10), None) == L.GDN_OK


def test_copy_refuses(lib):
    d = ctypes.byref(kd())
    call = lambda n_layers=2, pages=layers(G, G), n=3, src=G, dst=G, count=None: lib.gdn_kv_copy_pages(d, n_layers, pages, n, src, dst, count, None)
    for kw in (dict(n_layers=0), dict(n_layers=257), dict(pages=None), dict(pages=layers(G, None)), dict(n=-1), dict(src=None), dict(dst=None)):
        assert call(**kw) == L.GDN_ERR_INVALID_ARG, kw
    for kw in (dict(pages=layers(G, G + 8)), dict(src=G + 2), dict(dst=G + 2), dict(count=G + 2)):
        assert call(**kw) == L.GDN_ERR_MISALIGNED, kw
    assert call(n=0, src=None, dst=None) == L.GDN_OK


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    k, i = kd(B=1, max_pages=1, n_pages=1), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        L.gdn_kv_fork(k, *([i] * 10))
    with pytest.raises(TypeError, match="src_rows"):
        L.gdn_kv_fork(k, None, *([i] * 9))
    with pytest.raises(ValueError, match="copy_src"):
        L.gdn_kv_compact(kd(), *([i] * 11))
    with pytest.raises(TypeError, match="copy_src"):
        L.gdn_kv_compact(k, *([i] * 8), None, i, i)
    with pytest.raises(TypeError, match="src"):
        L.gdn_kv_copy_pages(k, [], None, i)
    with pytest.raises(TypeError, match="slots"):
        L.gdn_kv_plan_shared(k, *([i] * 11), None, i)


def test_reference_plan_agrees_with_the_plan_where_nothing_is_shared():
    rng = np.random.default_rng(0)
    B, page, M, n, T = 9, 16, 5, 30, 3
    st = State(B, page, M, n)
    lens = [0] * B
    for _ in range(30):
        add, active = rng.integers(-1, T + 2, B).tolist(), (rng.random(B) < 0.8).astype(int).tolist()
        want = kv4_ref.plan(page, M, n, T, B * T, lens, add, active, st.held, st.table, st.free, st.count)
        out, status = st.plan(T, B * T, lens, add, active)
        flat = repr(want)
        for k in ("slots", "positions", "q_count", "kv_len", "q_start"):
            assert repr(list(out[k])) in flat, k
        assert repr(st.held) in flat and repr(st.table) in flat
        st.check()
        lens = [0 if rng.random() < 0.2 else max(0, int(x + rng.integers(0, 20))) for x in lens]


def test_reference_in_small():
    st = State(3, 16, 4, 8)
    st.plan(0, 100, [0, 0, 0], [40, 0, 0], [1, 1, 1])
    assert st.table[0][:3] == [7, 6, 5]
    assert st.fork([0, 0], [1, 2], [40, 16]) == ([5, -1], [4, -1], 0)
    assert st.table[1][:3] == [7, 6, 4] and st.refs == [0, 0, 0, 0, 1, 1, 2, 3]
    st.check()
    new, page_map, src, dst = st.compact()
    assert (src, dst) == ([4, 5, 6, 7], [0, 1, 2, 3]) and new.table[1][:3] == [3, 2, 0]
    new.check()
    st.plan(1, 3, [0, 40, 16], [0, 0, 0], [1, 1, 1])
    assert st.free[: st.count] == [0, 1, 2, 3, 5] and st.refs == [0, 0, 0, 0, 1, 0, 1, 2]
