"""Sampled decoding where it can go wrong, on the GPU: tokens equal to the 64-bit reference's, logp as in
tests/test_sample_gpu.py."""
import math

import numpy as np
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests.test_sample_gpu import INF, bell, bits_of, check, logits_on

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,v", [(310, 16500), (304, 40001), (16, 151936), (3, 200003)])
def test_largest_logit_behind_the_first_granules(gdn, rows, v):
    """Slices longer than what their bound is taken from, the largest logits behind it and a binade or more above: the same
    outputs on every run, and the reference's."""
    rng = np.random.default_rng(v)
    x = rng.standard_normal((rows, v))
    x[:, -40:] += rng.uniform(4, 200, (rows, 1))
    x[::3, rng.integers(0, v, 30)] *= 50
    bits, u = bits_of(x), rng.random(rows).astype(np.float32)
    check(bits[:16], u[:16], temperature=1.5, top_p=0.95)
    check(bits[:16], u[:16], temperature=20.0, top_k=300)
    logits, uu = logits_on(bits), torch.from_numpy(u).cuda()
    ways = dict(temperature=torch.full((rows,), 3.0, device="cuda"), top_p=torch.full((rows,), 0.97, device="cuda"))
    outs = [(torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, device="cuda")) for _ in range(25)]
    for o in outs:
        L.gdn_sample(logits, uu, *o, **ways)
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, outs[0]))
