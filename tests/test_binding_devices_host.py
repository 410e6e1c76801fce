"""The binding without a GPU: tensors of another CUDA device than the current one, in the place of each argument of the
sampling, acceptance and cache calls; and what it asks of torch."""
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L

G = 1 << 20  # an aligned address that is never dereferenced: every call below is refused


class OnGpu(torch.Tensor):
    """Stands for a tensor on the CUDA device `at`."""
    is_cuda = True
    at = 0
    device = property(lambda self: f"cuda:{self.at}")
    get_device = lambda self: self.at
    data_ptr = lambda self: G


def on(at, *shape, dtype=torch.int32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)
    t.at = at
    return t


u8, bf16, f32 = torch.uint8, torch.bfloat16, torch.float32
B, T, V, N, n = 3, 2, 50, 5, 8
KD = dict(B=B, H_q=4, H_kv=2, d=64, page=16, max_pages=4, n_pages=n)
PAGES = dict(pages=((n * 2 * 2 * 16 * 36,), u8))
ROWS = dict(held=((B,),), table=((B, 4),), free_list=((n,),), free_count=((1,),))
PLAN = dict(lens=((B,),), add=((B,),), active=((B,), u8), **ROWS)
OUT = dict(q_start=((B + 1,),), q_count=((B,),), kv_len=((B,),), slots=((N,),), positions=((N,),))
CALLS = {
    "gdn_kv4_append": (dict(q=((N, 4, 64), bf16), k=((N, 2, 64), bf16), v=((N, 2, 64), bf16), positions=((1, N),), rope=((9, 8, 2), f32), slots=((N,),),
                            q_out=((N, 4, 64), bf16), **PAGES), dict(axis=bytes(8))),
    "gdn_kv4_read": (dict(slots=((N,),), k=((N, 2, 64), bf16), v=((N, 2, 64), bf16), **PAGES), {}),
    "gdn_kv4_attend": (dict(q=((N, 4, 64), bf16), table=((B, 4),), q_start=((B + 1,),), q_count=((B,),), kv_len=((B,),), out=((N, 4, 64), bf16), ws=((1 << 16,), u8),
                            **PAGES), dict(scale=1.0, max_q=2)),
    "gdn_kv_plan": (dict(**PLAN, **OUT), {}),
    "gdn_kv_plan_shared": (dict(**PLAN, refs=((n,),), **OUT), {}),
    "gdn_kv_fork": (dict(src_rows=((2,),), dst_rows=((2,),), lens=((2,),), **ROWS, refs=((n,),), copy_src=((2,),), copy_dst=((2,),)), {}),
    "gdn_kv_compact": (dict(held=((B,),), table=((B, 4),), refs=((n,),), new_table=((B, 4),), new_refs=((n,),), new_free_list=((n,),), new_free_count=((1,),),
                            page_map=((n,),), copy_src=((4,),), copy_dst=((4,),), copy_count=((1,),)), {}),
    "gdn_kv_copy_pages": (dict(src=((2,),), dst=((2,),), count=((1,),), caches=PAGES["pages"]), {}),
    "gdn_accept_greedy": (dict(logits=((B, T, V), bf16), draft=((B, T),), active=((B,), u8), keep=((B,),), nxt=((B,),), ws=((4096,), u8)), {}),
    "gdn_sample": (dict(logits=((B, V), bf16), u=((B,), f32), token=((B,),), logp=((B,), f32), temperature=((B,), f32), top_k=((B,),), top_p=((B,), f32),
                        min_p=((B,), f32), active=((B,), u8)), {}),
}


@pytest.mark.parametrize("name,bad", [(name, bad) for name, (sizes, _) in CALLS.items() for bad in sizes])
def test_tensors_of_another_device_are_refused(monkeypatch, name, bad):
    sizes, rest = CALLS[name]
    monkeypatch.setattr(L, "_here", lambda: 0)
    monkeypatch.setattr(L, "_stream", lambda stream: pytest.fail("the call was not refused"))
    args = {k: on(int(k == bad), *v[0], dtype=v[1] if len(v) > 1 else torch.int32) for k, v in sizes.items()}
    if "caches" in args:
        args["caches"] = [on(0, *sizes["caches"][0], dtype=u8), args["caches"]]
    kd = () if name in ("gdn_accept_greedy", "gdn_sample") else (L.kv4_dims(**KD),)
    with pytest.raises(ValueError, match="cuda:1"):
        getattr(L, name)(*kd, **args, **rest)


@pytest.fixture
def bare_torch(monkeypatch):
    """torch without the private names that make the two questions of every call cheap."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    for name in ("_device_number", "_raw_stream"):
        monkeypatch.setattr(L, name, None)
    return monkeypatch


def test_public_device_and_stream_serve_where_the_private_names_are_gone(bare_torch):
    class Stream:
        cuda_stream = 5

    bare_torch.setattr(torch.cuda, "current_device", lambda: 3)
    bare_torch.setattr(torch.cuda, "current_stream", lambda: Stream)
    assert L._here() == 3 and [L._stream(None), L._stream(None)] == [5, 5]
    Stream.cuda_stream = 7
    assert L._stream(None) == 7 and L._stream(9) == 9 and L._stream(Stream) == 7


@pytest.mark.parametrize("error", [RuntimeError, AssertionError])
def test_no_device_is_none(bare_torch, error):
    def none():
        raise error("no CUDA")

    bare_torch.setattr(torch.cuda, "current_device", none)
    assert L._here() == -2
