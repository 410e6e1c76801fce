"""The binding of the paged 4-bit cache's calls without a GPU: what it refuses, and how it names it."""
import ctypes

import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L

G = 1 << 20  # an aligned address that is never dereferenced: validation fails first


def test_timeout_hook_refuses():
    lib = L.load()
    kd = L.kv4_dims(8, 16, 2, 256, 64, 512, 4096)
    need = L.gdn_kv4_attend_workspace_bytes(kd, 16, 2)

    def call(dims=kd, limit=4000, nbytes=need):
        return lib.gdn_test_kv4_attend_timeout(ctypes.byref(dims), 16, 2, *([G] * 6), 1.0, G, G, nbytes, limit, None)

    assert call(limit=0) == L.GDN_ERR_INVALID_ARG and "wait_limit" in L.gdn_last_error()
    assert call(nbytes=need - 1) == L.GDN_ERR_WORKSPACE
    assert call(dims=L.kv4_dims(8, 16, 2, 96, 64, 512, 4096)) == L.GDN_ERR_UNSUPPORTED


def test_cache_size_is_checked_after_a_refused_call(monkeypatch):
    """Dims that were refused once and then set right: the cache's size is checked like any other's."""
    monkeypatch.setattr(L, "_ptr", lambda t, what, dtype=None: G)  # (the tensor stands for one on a GPU)
    kd = L.kv4_dims(2, 0, 2, 64, 16, 4, 8)
    per = 2 * 2 * 16 * (32 + 4)
    pages = torch.zeros(8 * per - 1, dtype=torch.uint8)
    assert L._cache(kd, pages) == G  # H_q = 0: the library refuses the call
    kd.H_q = 4
    with pytest.raises(ValueError, match="pages: "):
        L._cache(kd, pages)
    assert L._cache(kd, torch.zeros(8 * per, dtype=torch.uint8)) == G


@pytest.mark.parametrize("what", ["lens", "slots", "positions", "table"])
def test_plan_names_what_is_not_a_tensor(what):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)
    a = dict(lens=z(2), add=z(2), active=z(2).byte(), held=z(2), table=z(2, 4), free_list=z(8), free_count=z(1), q_start=z(3),
             q_count=z(2), kv_len=z(2), slots=z(5), positions=z(5))
    with pytest.raises(TypeError, match=what):
        L.gdn_kv_plan(L.kv4_dims(2, 1, 1, 64, 16, 4, 8), **{**a, what: [1, 2]})


@pytest.mark.parametrize("what", ["slots", "pages", "k", "v"])
def test_read_names_what_is_not_a_tensor(what, monkeypatch):
    monkeypatch.setattr(L, "_ptrs", as_on_gpu)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    a = dict(slots=torch.zeros(3, dtype=torch.int32), pages=torch.zeros(8 * 2 * 16 * 36, dtype=torch.uint8), k=z(3, 1, 64), v=z(3, 1, 64))
    with pytest.raises(TypeError, match=what):
        L.gdn_kv4_read(L.kv4_dims(2, 1, 1, 64, 16, 4, 8), **{**a, what: None})


@pytest.mark.parametrize("what", ["q", "pages", "ws"])
def test_attend_names_what_else_is_not_a_tensor(what, monkeypatch):
    monkeypatch.setattr(L, "_ptrs", as_on_gpu)
    monkeypatch.setattr(L, "_ptr", lambda t, what, dtype=None: None if t is None else G)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)
    a = dict(q=z(5, 4, 64).bfloat16(), pages=torch.zeros(6 * 2 * 2 * 16 * 36, dtype=torch.uint8), table=z(2, 3), q_start=z(3), q_count=z(2),
             kv_len=z(2), scale=0.125, out=z(5, 4, 64).bfloat16(), ws=torch.zeros(16, dtype=torch.uint8), max_q=3)
    with pytest.raises(TypeError, match=what):
        L.gdn_kv4_attend(L.kv4_dims(2, 4, 2, 64, 16, 3, 6), **{**a, what: None})


@pytest.mark.parametrize("what", ["positions", "rope", "axis", "slots", "q_out", "pages"])
def test_append_names_what_is_not_a_tensor(what, monkeypatch):
    monkeypatch.setattr(L, "_ptrs", as_on_gpu)
    monkeypatch.setattr(L, "_ptr", lambda t, what, dtype=None: None if t is None else G)
    monkeypatch.setattr(L, "_tokens", lambda t, what, heads, d: (G, heads * d))
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    a = dict(q=z(3, 2, 64), k=z(3, 1, 64), v=z(3, 1, 64), positions=torch.zeros(1, 3, dtype=torch.int32), rope=torch.zeros(9, 8, 2),
             axis=bytes(8), slots=torch.zeros(3, dtype=torch.int32), pages=torch.zeros(8 * 2 * 16 * 36, dtype=torch.uint8), q_out=z(3, 2, 64))
    with pytest.raises(TypeError, match=what):
        L.gdn_kv4_append(L.kv4_dims(2, 2, 1, 64, 16, 4, 8), **{**a, what: [0] * 8})


def as_on_gpu(*args):
    """_ptrs with tensors that stand for some on a GPU."""
    for t, what, n, _ in args:
        L._count(t, what, n)
    return [G] * len(args)
