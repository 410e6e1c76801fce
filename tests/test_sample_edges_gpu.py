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


@pytest.mark.parametrize("rows,v", [(1, 151936), (3, 60003), (160, 40001), (300, 16500), (6, 3001)])
@pytest.mark.parametrize("temperature", [INF, 1e38, 3e4])
@pytest.mark.parametrize("mask", [0.5, 0.99])
def test_forbidden_tokens_are_never_drawn(gdn, rows, v, temperature, mask):
    """Half of the tokens or nearly all forbidden, at temperatures at which all others weigh the same, in slices longer than
    their first granules and shorter ones: -infinity has no weight, and decides no border either."""
    rng = np.random.default_rng(v)
    n = min(rows, 6)
    x = rng.standard_normal((n, v)) * 2
    x[rng.random((n, v)) < mask] = -INF
    bits = bits_of(x)
    allowed = np.isfinite(x)
    for kw in (dict(), dict(top_p=0.5), dict(top_k=7), dict(min_p=0.5)):
        u = np.linspace(0.03, 0.999, n)
        check(bits, u, temperature=temperature, **kw)
    # all rows of the launch, every place of u
    logits = logits_on(np.tile(bits, (-(-rows // n), 1))[:rows])
    token, logp = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, device="cuda")
    for u in np.linspace(0, 1, 9):
        L.gdn_sample(logits, torch.full((rows,), float(u), device="cuda"), token, logp, temperature=torch.full((rows,), temperature, device="cuda"))
        t, lp = token.cpu().numpy(), logp.double().cpu().numpy()
        for i in range(rows):
            assert allowed[i % n, t[i]]
            if temperature == INF:
                assert abs(lp[i] + math.log(allowed[i % n].sum())) <= 2 ** -22 * (1 + math.log(v))


def test_forbidden_tokens_do_not_decide_an_exact_border(gdn):
    """Two equal maxima, top_p a half, the rest forbidden: one of them is half of the mass, so it is kept alone, whatever the
    temperature; slices whose bins reach the largest magnitudes."""
    x = np.full((6, 151936), -INF)
    x[:, [9, 33000]] = 3.0
    x[3:] = -INF
    x[3:, [9, 33000]] = -2e38
    for temperature in (INF, 1e38, 1.0):
        got = check(bits_of(x), np.linspace(0.05, 0.95, 6), temperature=temperature, top_p=0.5)
        assert set(got.tolist()) == {9}


@pytest.mark.parametrize("min_p,kept", [(1e-15, True), (7.0e-15, True), (1e-30, True), (7.3e-15, False), (1e-13, False), (0.1, False)])
@pytest.mark.parametrize("tops,others,v", [(2, 3, 40), (4, 5, 5000), (2, 900, 20000), (2, 40, 151936)])
def test_min_p_below_the_masses_units(gdn, tops, others, v, min_p, kept):
    """Equal maxima, others of 2^-47 = 7.1e-15 of them, top_p a half: where min_p leaves the others, one maximum more than half of
    them is kept."""
    x = np.full((8, v), -INF)
    x[:, 1:1 + tops] = 3.0
    x[:, 20:20 + others] = -5.0
    temperature = np.float32(8.0 / (47 * math.log(2)))
    got = check(bits_of(x), np.linspace(0.05, 0.95, 8), temperature=temperature, top_p=0.5, min_p=min_p)
    assert len(set(got.tolist())) == (tops // 2 + 1 if kept else tops // 2)
    check(bits_of(x), np.linspace(0.05, 0.95, 8), temperature=temperature, top_p=0.5, min_p=min_p, top_k=tops)
    check(bits_of(x), np.linspace(0.05, 0.95, 8), temperature=temperature, top_p=0.5, min_p=min_p, top_k=tops + 1)


def test_far_below_the_units_is_nothing_at_any_scale(gdn):
    """Two equal maxima near the largest number, another 2^-98 of them: nothing, so top_p of a half keeps one maximum."""
    x = np.full((4, 5000), -INF)
    x[:, [3, 9]], x[:, 40] = 3.3e38, -3.3e38
    got = check(bits_of(x), np.linspace(0.05, 0.95, 4), temperature=1e37, top_p=0.5)
    assert set(got.tolist()) == {3}


@pytest.mark.parametrize("temperature", [2e-42, 9e-41, 1.2e-39, 9e-39, 1.2e-38, 1e-20, 1e19, 2e19, 3e37, 3e38])
def test_temperatures_of_any_size(gdn, temperature):
    """Logits some temperatures apart, at temperatures below the normal numbers and near the largest."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 9001)) * 3 * np.float64(np.float32(temperature))
    bits = bits_of(np.clip(x, -3.3e38, 3.3e38))
    for kw in (dict(), dict(top_p=0.8), dict(top_k=30), dict(min_p=0.1)):
        check(bits, rng.random(4), temperature=temperature, **kw)


@pytest.mark.parametrize("bits,decides", [(52.97, True), (50.0, True), (54.5, False)])
def test_dust_down_to_its_border(gdn, bits, decides):
    """Two equal maxima, top_p a half, others of 2^-bits of them: down to 2^-53 they make the half less than half."""
    x = np.full((8, 300), -INF)
    x[:, [4, 9]], x[:, 20:200] = 3.0, -5.0
    token = torch.zeros(8, dtype=torch.int32, device="cuda")
    full = lambda a: torch.full((8,), a, device="cuda")
    L.gdn_sample(logits_on(bits_of(x)), torch.linspace(0.05, 0.95, 8, device="cuda"), token, temperature=full(8 / (bits * math.log(2))), top_p=full(0.5))
    assert set(token.tolist()) == ({4, 9} if decides else {4})
