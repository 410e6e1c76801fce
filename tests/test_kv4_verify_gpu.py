"""A flagged GDN verify directly behind the kernels that take all of an SM's
tensor memory: the cache attention's form for many rows, and another cohort's
prefill.  (Which of them may start when is read in test_tensor_memory_host.py;
these runs show that the calls go together and change no bit.)"""
import numpy as np
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from speculative_decode_gated_gdn_gb300 import synth
from tests.gdn_harness import GpuStack
from tests.test_kv4_gpu import attend_case, bits, run_attend
from tests.test_prefill_gpu import fresh_state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("mode", [L.GDN_COMMIT_RECOMPUTE, L.GDN_COMMIT_DEFERRED], ids=["recompute", "deferred"])
def test_flagged_verify_behind_attend_and_prefill(gdn, mode, d):
    geom = synth.Geometry(B=8, T=2, H_k=16, H_v=32, d=128)
    gpu = GpuStack(geom, synth.layer_state(geom, 3, 3), synth.active_mask(8), mode, 3)
    cy = synth.cycle_inputs(geom, 3, 0, 3)
    x = [torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.bfloat16) for a in cy["x"]]
    g, beta = ([torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in cy[k]] for k in ("g", "beta"))

    def verify(l, flags):
        L.gdn_conv_verify(gpu.dims, mode | flags, x[l], gpu.w[l], g[l], beta[l], gpu.state[l], gpu.ring[l], gpu.offsets,
                          gpu.active, gpu.out[l], gpu.ws[l])

    for l in range(3):
        verify(l, 0)
    torch.cuda.synchronize()
    want = gpu.out.clone()

    rows = [(700, 150, 150), (300, 100, 150)]
    cache, table, q_start, q_count, kv_len, q = attend_case(16, 2, d, 32, rows, seed=1)
    o, ws, kd, args = run_attend(cache, table, q_start, q_count, kv_len, q, d ** -0.5, 150)
    o_want = o.clone()
    small = synth.Geometry(B=1, T=2, H_k=2, H_v=4, d=128)
    prompt = GpuStack(small, fresh_state(small, 5), synth.active_mask(1), mode, 1)
    pr = synth.prompt_inputs(small, 5, 100)
    nbytes = L.gdn_prefill_workspace_bytes(prompt.dims, 100)
    p_ws, p_out = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty(1, 100, 4, 128, dtype=torch.bfloat16, device="cuda")
    p_in = [torch.from_numpy(np.ascontiguousarray(pr["x"]).view(np.int16)).cuda().view(torch.bfloat16), prompt.w[0],
            torch.from_numpy(pr["g"]).cuda(), torch.from_numpy(pr["beta"]).cuda()]
    torch.cuda.synchronize()
    for _ in range(20):
        gpu.out.zero_()
        verify(0, 0)
        L.gdn_kv4_attend(kd, *args, d ** -0.5, o, ws, 150)
        verify(1, L.GDN_VERIFY_OVERLAP)
        L.gdn_prefill_chunked(prompt.dims, 100, *p_in, prompt.state[0], prompt.ring[0], prompt.offsets, p_out, p_ws)
        verify(2, L.GDN_VERIFY_OVERLAP)
        torch.cuda.synchronize()
        assert L.gdn_get_status(clear=True) == 0
        assert torch.equal(bits(gpu.out), bits(want)) and torch.equal(bits(o), bits(o_want))
