"""The paged 4-bit cache's calls without a GPU: sizes, refusals before any
launch, and the references' own sense."""
import ctypes

import numpy as np
import pytest

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref as R

G = 1 << 20  # an aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return L.load()


def kd(**kw):
    return L.kv4_dims(**{**dict(B=8, H_q=16, H_kv=2, d=256, page=64, max_pages=512, n_pages=4096), **kw})


def test_page_bytes(lib):
    for d in (64, 128, 256):
        for page in (16, 32, 64):
            # K and V: half a byte a channel and four bytes a group of 64
            assert L.gdn_kv4_page_bytes(kd(d=d, page=page)) == 2 * 2 * page * (d // 2 + d // 64 * 4)
    assert L.gdn_kv4_page_bytes(kd(d=96)) == 0


BAD = [dict(B=-1), dict(B=65536), dict(d=32), dict(d=192), dict(page=8), dict(page=128), dict(page=48), dict(H_q=15),
       dict(H_q=0), dict(H_kv=0), dict(H_q=130, H_kv=2), dict(max_pages=0), dict(max_pages=(1 << 20) + 1), dict(n_pages=0),
       dict(n_pages=1 << 25)]


@pytest.mark.parametrize("kw", BAD, ids=str)
def test_bad_dims(lib, kw):
    d = ctypes.byref(kd(**kw))
    f = L.GDN_ERR_UNSUPPORTED
    assert lib.gdn_kv_plan(d, 2, 16, *([G] * 12), None) == f and L.gdn_last_error()
    assert lib.gdn_kv4_append(d, 4, G, 8192, G, 8192, G, 8192, G, 1, G, 10, 0, b"", 0, G, G, G, None) == f
    assert lib.gdn_kv4_read(d, 4, G, G, G, G, None) == f
    assert lib.gdn_kv4_attend(d, 4, 1, G, G, G, G, G, G, 1.0, G, G, 1 << 40, None) == f
    assert lib.gdn_kv4_attend_workspace_bytes(d, 4, 1) == 0


def test_plan_refuses(lib):
    d = ctypes.byref(kd())
    a = [G] * 12
    for i in range(12):
        for bad, code in ((None, L.GDN_ERR_INVALID_ARG), (G + 2, L.GDN_ERR_MISALIGNED)):
            if i == 2 and bad:
                continue  # active: bytes, any address
            b = list(a)
            b[i] = bad
            assert lib.gdn_kv_plan(d, 2, 16, *b, None) == code, i
    assert lib.gdn_kv_plan(d, -1, 16, *a, None) == L.GDN_ERR_INVALID_ARG
    assert lib.gdn_kv_plan(d, 2, 15, *a, None) == L.GDN_ERR_INVALID_ARG
    assert lib.gdn_kv_plan(d, 2, -1, *a, None) == L.GDN_ERR_UNSUPPORTED
    assert lib.gdn_kv_plan(None, 2, 16, *a, None) == L.GDN_ERR_INVALID_ARG
    assert lib.gdn_kv_plan(ctypes.byref(kd(B=0)), 2, 16, *([None] * 12), None) == L.GDN_OK


def append(lib, d, N=4, q=G, qs=4096, k=G, ks=512, v=G, vs=512, pos=G, axes=3, rope=G, top=100, rot=64, axis=bytes(32), style=0, slots=G, pages=G, out=G):
    return lib.gdn_kv4_append(ctypes.byref(d), N, q, qs, k, ks, v, vs, pos, axes, rope, top, rot, axis, style, slots, pages, out, None)


def test_append_refuses(lib):
    d = kd()
    for name in ("q", "k", "v", "pos", "rope", "slots", "pages", "out", "axis"):
        assert append(lib, d, **{name: None}) == L.GDN_ERR_INVALID_ARG, name
    for name in ("q", "k", "v", "pages", "out"):
        assert append(lib, d, **{name: G + 8}) == L.GDN_ERR_MISALIGNED, name
    for name in ("pos", "rope", "slots"):
        assert append(lib, d, **{name: G + 2}) == L.GDN_ERR_MISALIGNED, name
    for kw in (dict(qs=4088), dict(ks=504), dict(vs=0), dict(qs=4100), dict(ks=516), dict(style=2), dict(axes=0), dict(top=0),
               dict(axis=bytes([3] * 32)), dict(axis=bytes(31) + b"\xff")):
        assert append(lib, d, **kw) == L.GDN_ERR_INVALID_ARG, kw
    for kw in (dict(rot=-16), dict(rot=24), dict(rot=272), dict(N=-1), dict(N=(1 << 24) + 1)):
        assert append(lib, d, **kw) == L.GDN_ERR_UNSUPPORTED, kw
    assert append(lib, d, N=0, q=None, k=None, v=None, slots=None, pages=None, out=None) == L.GDN_OK


def test_read_refuses(lib):
    d = ctypes.byref(kd())
    for i in range(4):
        a = [G] * 4
        a[i] = None
        assert lib.gdn_kv4_read(d, 4, *a, None) == L.GDN_ERR_INVALID_ARG
        a[i] = G + 2
        assert lib.gdn_kv4_read(d, 4, *a, None) == L.GDN_ERR_MISALIGNED
    assert lib.gdn_kv4_read(d, -1, *([G] * 4), None) == L.GDN_ERR_UNSUPPORTED
    assert lib.gdn_kv4_read(d, 0, *([None] * 4), None) == L.GDN_OK


def test_attend_refuses(lib):
    k = kd()
    d = ctypes.byref(k)
    need = L.gdn_kv4_attend_workspace_bytes(k, 16, 2)
    assert need > 0 and L.gdn_kv4_attend_workspace_bytes(k, 16, 0) == 0 and L.gdn_kv4_attend_workspace_bytes(k, -1, 2) == 0

    def call(a=None, N=16, max_q=2, scale=1.0, nbytes=need, dims=d):
        a = [G] * 8 if a is None else a
        return lib.gdn_kv4_attend(dims, N, max_q, *a[:6], scale, a[6], a[7], nbytes, None)

    for i in range(8):
        a = [G] * 8
        a[i] = None
        assert call(a) == L.GDN_ERR_INVALID_ARG, i
        a[i] = G + 2
        assert call(a) == L.GDN_ERR_MISALIGNED, i
    assert call(nbytes=need - 1) == L.GDN_ERR_WORKSPACE
    assert call(scale=float("nan")) == L.GDN_ERR_INVALID_ARG and call(scale=float("inf")) == L.GDN_ERR_INVALID_ARG
    assert call(max_q=0) == L.GDN_ERR_UNSUPPORTED and call(max_q=(1 << 20) + 1) == L.GDN_ERR_UNSUPPORTED
    assert call(N=-1) == L.GDN_ERR_UNSUPPORTED
    assert call([None] * 8, N=0) == L.GDN_OK and call([None] * 8, dims=ctypes.byref(kd(B=0))) == L.GDN_OK


def test_binding_checks_shapes():
    torch = pytest.importorskip("torch")
    d = kd(B=2, max_pages=4, n_pages=8)
    t = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="table"):
        L.gdn_kv_plan(d, t, t, t, t, t, t, t, t, t, t, t, t)
    with pytest.raises(ValueError, match="q: expected a CUDA tensor"):
        L.gdn_kv4_append(d, torch.zeros(1, 16, 256), None, None, None, None, b"", t, t, t)
    with pytest.raises(ValueError, match="q: expected"):
        L.gdn_kv4_attend(d, torch.zeros(3, dtype=torch.bfloat16), t, t, t, t, t, 1.0, t, t, 1)


# ------------------------------------------------------------------ the references themselves
def test_reference_pack_round_trip():
    rng = np.random.default_rng(0)
    for d in (64, 128, 256):
        x = rng.normal(size=(5, d)).astype(np.float32)
        c, e = R.pack(x)
        y = R.values(c, e)
        g = (np.arange(d) // 8) % (d // 64)
        assert (np.abs(x - y) <= 0.51 * e[:, g, 0].astype(np.float64) + 2e-3).all()
        # every group is 64 channels and its extremes are its first and last level
        assert [int((g == i).sum()) for i in range(d // 64)] == [64] * (d // 64)


def test_reference_plan_conserves_pages():
    rng = np.random.default_rng(1)
    st = dict(held=[0] * 7, table=[[-1] * 9 for _ in range(7)], free=list(range(40)), count=40)
    lens = np.zeros(7, int)
    for _ in range(30):
        st = R.plan(16, 9, 40, 0, 300, lens, rng.integers(0, 40, 7), [1] * 7, st["held"], st["table"], st["free"], st["count"])
        pages = [p for b in range(7) for p in st["table"][b][:st["held"][b]]] + st["free"][:st["count"]]
        assert sorted(pages) == list(range(40))
        lens = np.where(rng.random(7) < 0.2, 0, lens + rng.integers(0, 1 + np.array(st["q_count"])))
        lens = np.minimum(lens, 100)


def test_reference_attend_is_softmax():
    """Equal keys: the mean of the values; the first query of a fresh row: its own value."""
    cache = R.Cache(1, 1, 16, 64)
    rng = np.random.default_rng(2)
    for t in range(5):
        cache.write(t, np.ones((1, 64), np.float32), rng.normal(size=(1, 64)).astype(np.float32))
    q = rng.normal(size=(5, 2, 64))
    out, tol = R.attend(q, cache, [[0]], [0, 5], [5], [5], 0.3)
    _, v = cache.read(range(5))
    for i in range(5):
        assert np.allclose(out[i], v[:i + 1].mean(0))


@pytest.mark.parametrize("what", ["table", "q_start", "q_count", "kv_len", "out"])
def test_attend_names_what_is_not_a_tensor(what):
    """Anything but a tensor is refused by its name, whatever else is wrong."""
    torch = pytest.importorskip("torch")
    dims = L.kv4_dims(2, 4, 2, 64, 16, 3, 6)
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype)
    a = dict(q=z(5, 4, 64, dtype=torch.bfloat16), pages=z(6 * 2 * 2 * 16 * 36, dtype=torch.uint8), table=z(2, 3), q_start=z(3),
             q_count=z(2), kv_len=z(2), scale=0.125, out=z(5, 4, 64, dtype=torch.bfloat16), ws=z(16, dtype=torch.uint8), max_q=3)
    with pytest.raises(TypeError, match=what):
        L.gdn_kv4_attend(dims, **{**a, what: None})
    with pytest.raises(ValueError, match="expected"):
        L.gdn_kv4_attend(dims, **{**a, what: a[what][..., :1]})
    with pytest.raises(ValueError, match="CUDA"):
        L.gdn_kv4_attend(dims, **a)
