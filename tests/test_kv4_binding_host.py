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
