"""Arrays that a call writes and others that it still reads may not be the same memory: such calls are refused before any
launch.  (Row numbers that a fork's outputs overwrite would send its kernels outside the tables.)"""
import ctypes

import pytest

from speculative_decode_gated_gdn_gb300 import lib as L

G = 1 << 30  # addresses that are never dereferenced: every call below is refused
STEP = 1 << 24


@pytest.fixture(scope="module")
def lib():
    return L.load()


def spread(names):
    return {n: G + i * STEP for i, n in enumerate(names.split())}


def refused(rc, *names):
    message = L.gdn_last_error()
    return rc == L.GDN_ERR_INVALID_ARG and "overlap" in message and all(n in message for n in names)


KD = L.kv4_dims(B=8, H_q=16, H_kv=2, d=256, page=64, max_pages=512, n_pages=4096)


@pytest.mark.parametrize("out,shift", [("token", -44), ("token", 0), ("token", 44), ("keep", -12), ("keep", 44), ("next", 0), ("next", 32), ("ws", 0)])
def test_acceptance(lib, out, shift):
    names = "draft active temperature top_k top_p min_p u keep next token logp ws"
    a = spread(names)
    a[out] = a["draft"] + shift  # draft and token have 48 bytes, keep and next 16
    assert refused(lib.gdn_accept_sampled(4, 3, 100, G - STEP, 100, *(a[n] for n in names.split()), 1 << 12, None), out, "draft")


@pytest.mark.parametrize("out", ["copy_src", "copy_dst"])
@pytest.mark.parametrize("other", ["src_rows", "dst_rows", "lens", "held", "table", "refs", "copy"])
def test_forks(lib, out, other):
    names = "src_rows dst_rows lens held table free_list free_count refs copy_src copy_dst"
    a = spread(names)
    other = {"copy_src": "copy_dst", "copy_dst": "copy_src"}[out] if other == "copy" else other
    a[out] = a[other] + 8
    assert refused(lib.gdn_kv_fork(ctypes.byref(KD), 4, *(a[n] for n in names.split()), None), out, other)


OUTS = ["page_map", "copy_src", "copy_dst", "copy_count", "new_free_list", "new_free_count", "new_table", "new_refs"]


@pytest.mark.parametrize("out,other", [(a, b) for a in OUTS for b in ["held", "table", "refs"] + OUTS if a != b])
def test_compaction(lib, out, other):
    names = "held table refs new_table new_refs new_free_list new_free_count page_map copy_src copy_dst copy_count"
    a = spread(names)
    a[out] = a[other] + (16 if not other.endswith("count") else 0)
    assert refused(lib.gdn_kv_compact(ctypes.byref(KD), *(a[n] for n in names.split()), None), out, other)
    a = spread(names)  # in place, but one of the two into the other's place
    a["new_table"], a["new_refs"] = a["refs"], a["table"]
    assert refused(lib.gdn_kv_compact(ctypes.byref(KD), *(a[n] for n in names.split()), None))


@pytest.mark.parametrize("shift", [0, 28, -28])
def test_shared_plan(lib, shift):
    names = "lens add active held table free_list free_count refs q_start q_count kv_len slots positions"
    a = spread(names)
    a["kv_len"] = a["lens"] + shift
    assert refused(lib.gdn_kv_plan_shared(ctypes.byref(KD), 2, 16, *(a[n] for n in names.split()), None), "kv_len", "lens")
