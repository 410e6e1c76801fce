"""The binding of the paged 4-bit cache's calls without a GPU: what it refuses, and how it names it."""
import ctypes


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
