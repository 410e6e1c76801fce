"""Sampled decoding on the GPU against a 64-bit reference: gdn_sample and
gdn_accept_sampled.

Tokens are whole numbers and have to be equal.  logp is -log1p(m / w) in fp32 of
integers m, w that hold weights to 2^-37: two conversions and a quotient are off by
3 * 2^-24 relative, which the logarithm passes on at most as such, and its own
rounding is within 2 * 2^-24 of its value, so 2^-22 * (1 + |logp|) holds."""
import math

import numpy as np
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import sample_ref as R

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


def bits_of(x):
    return torch.as_tensor(x, dtype=torch.float32).bfloat16().view(torch.int16).numpy().view(np.uint16)


def logits_on(bits, pad=0, shift=0):
    """The bits [R][V] on the GPU, rows `pad` elements further apart than V, from the `shift`-th element of an allocation;
    what lies between the rows must not matter."""
    r, v = bits.shape
    flat = torch.full((r * (v + pad) + shift + 8,), 30000.0, dtype=torch.bfloat16, device="cuda")
    t = torch.as_strided(flat, (r, v), (v + pad, 1), shift)
    t.copy_(torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16))
    return t


def check(bits, u, pad=0, shift=0, active=None, **kw):
    """Every row of bits [R][V] with its own parameters (arrays or numbers)."""
    r, v = bits.shape
    dev = {}
    host = {}
    for k, dtype in (("temperature", np.float32), ("top_k", np.int32), ("top_p", np.float32), ("min_p", np.float32)):
        if k in kw:
            host[k] = np.broadcast_to(np.asarray(kw[k], dtype), (r,)).copy()
            dev[k] = torch.from_numpy(host[k]).cuda()
    u = np.broadcast_to(np.asarray(u, np.float32), (r,)).copy()
    token = torch.full((r,), -7, dtype=torch.int32, device="cuda")
    logp = torch.full((r,), 9.0, dtype=torch.float32, device="cuda")
    act = None if active is None else torch.from_numpy(active).cuda()
    L.gdn_sample(logits_on(bits, pad, shift), torch.from_numpy(u).cuda(), token, logp, active=act, **dev)
    got, got_logp = token.cpu().numpy(), logp.cpu().numpy().astype(np.float64)
    x = R.values(bits)
    for i in range(r):
        if active is not None and not active[i]:
            assert got[i] == -1 and got_logp[i] == 0
            continue
        t, lp, border = R.draw(x[i], u[i], **{k: a[i].item() for k, a in host.items()})
        assert got[i] == t, (i, got[i], t, border, {k: a[i] for k, a in host.items()}, u[i])
        if math.isinf(lp):
            assert got_logp[i] == lp, i
        else:
            assert abs(got_logp[i] - lp) <= 2 ** -22 * (1 + abs(lp)), (i, got_logp[i], lp)
    assert L.gdn_get_status() == 0
    return got


def bell(rng, r, v, scale=2.2, peaks=8):
    x = rng.standard_normal((r, v)) * scale
    for i in range(r):
        x[i, rng.integers(0, v, min(peaks, v))] = 6 + rng.random(min(peaks, v)) * 9 * rng.random()
    return x


FILTERS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=40), dict(top_k=700), dict(top_p=0.9), dict(min_p=0.05),
           dict(temperature=1.7, top_k=1200, top_p=0.95, min_p=0.001), dict(temperature=0.3, top_k=50, top_p=0.5, min_p=0.2)]


@pytest.mark.parametrize("kw", FILTERS, ids=str)
@pytest.mark.parametrize("shape", [(3, 1), (5, 2), (9, 7), (4, 8), (6, 1003), (5, 32000), (2, 100003), (3, 151936)], ids=str)
def test_filters_and_sizes(gdn, shape, kw):
    rng = np.random.default_rng(sum(shape))
    check(bits_of(bell(rng, *shape)), rng.random(shape[0]), **kw)


@pytest.mark.parametrize("v", [262144, 500001, 1 << 20])
def test_large_vocabularies(gdn, v):
    rng = np.random.default_rng(v)
    bits = bits_of(bell(rng, 2, v))
    check(bits, rng.random(2))
    check(bits, rng.random(2), temperature=0.8, top_k=300, top_p=0.9)


@pytest.mark.parametrize("rows", [1, 20, 75, 151, 153, 310, 700])
def test_many_rows(gdn, rows):
    """Each number of rows has its own share of the GPU."""
    rng = np.random.default_rng(rows)
    check(bits_of(bell(rng, rows, 5003)), rng.random(rows), temperature=rng.choice([0.0, 0.5, 1.0, 2.0], rows),
          top_k=rng.choice([0, 1, 30], rows), top_p=rng.choice([1.0, 0.8], rows), min_p=rng.choice([0.0, 0.1], rows),
          active=(rng.random(rows) < 0.9).astype(np.uint8))


@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 5), (7, 7), (64, 2), (0, 4)])
def test_strides_and_addresses(gdn, pad, shift):
    rng = np.random.default_rng(pad * 8 + shift)
    for v in (1, 6, 17, 4099):
        check(bits_of(bell(rng, 6, v)), rng.random(6), pad, shift, temperature=1.3, top_p=0.97)


def test_equal_values_go_by_index(gdn):
    """Equal logits everywhere: the place of u in the row, exactly; and ties at the border of top_k and top_p."""
    rng = np.random.default_rng(1)
    for v in (1, 8, 1000, 40003):
        bits = np.full((7, v), bits_of(1.5), np.uint16)
        u = np.array([0, 0.25, 0.5, 0.75, 1 - 2 ** -24, 0.123, 0.9], np.float32)
        got = check(bits, u)
        assert np.array_equal(got, np.minimum((u.astype(np.float64) * v).astype(np.int64), v - 1))
        check(bits, u, top_k=5)
        check(bits, u, top_p=0.5)
    x = rng.integers(-3, 4, (6, 20000)).astype(np.float64)  # thousands of equal ones
    for kw in (dict(), dict(top_k=17), dict(top_k=1499), dict(top_k=5000), dict(top_p=0.3), dict(min_p=0.05)):
        check(bits_of(x), rng.random(6), **kw)


def test_the_largest_vocabulary_of_equal_values(gdn):
    """2^20 logits of weight 1: the mass is 2^63 units."""
    v = 1 << 20
    x = torch.full((3, v), -2.5, dtype=torch.bfloat16, device="cuda")
    u = torch.tensor([0.0, 0.5, 1 - 2 ** -24], device="cuda")
    token, logp = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, device="cuda")
    L.gdn_sample(x, u, token, logp)
    assert token.tolist() == [0, v // 2, v - 1]
    assert (logp.double() + math.log(v)).abs().max() <= 2 ** -22 * (1 + math.log(v))
    L.gdn_sample(x, u, token, top_p=torch.full((3,), 0.75, device="cuda"), top_k=torch.full((3,), v - 4, dtype=torch.int32, device="cuda"))
    n = (v - 4) * 3 // 4
    assert token.tolist() == [0, n // 2, int((1 - 2 ** -24) * n)]


def test_most_rows(gdn):
    rng = np.random.default_rng(11)
    bits = bits_of(rng.standard_normal((65535, 40)) * 3)
    u = rng.random(65535).astype(np.float32)
    token = torch.zeros(65535, dtype=torch.int32, device="cuda")
    L.gdn_sample(logits_on(bits), torch.from_numpy(u).cuda(), token)
    got, x = token.cpu().numpy(), R.values(bits)
    for i in range(0, 65535, 331):
        assert got[i] == R.draw(x[i], u[i])[0]


def test_threads_and_repeats(gdn):
    """Calls at once on streams of their own give what one call gives, every time."""
    import threading
    wrong = []

    def work(seed):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                gen = torch.Generator(device="cuda").manual_seed(seed)
                x = (torch.randn(20, 30011, device="cuda", generator=gen) * 2).bfloat16()
                u = torch.rand(20, device="cuda", generator=gen)
                first = torch.zeros(20, dtype=torch.int32, device="cuda"), torch.zeros(20, device="cuda")
                L.gdn_sample(x, u, *first)
                outs = [(torch.zeros_like(first[0]), torch.zeros_like(first[1])) for _ in range(30)]
                for o in outs:
                    L.gdn_sample(x, u, *o)
                stream.synchronize()
                assert all(torch.equal(a, b) for o in outs for a, b in zip(o, first))
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_borders_that_the_mass_meets_exactly(gdn):
    """Two, or four, equal maxima and top_p a half: the first are half of the mass, so they are kept alone only if nothing else
    has any; what is 2^-47 of the largest, and less than a unit of the masses, still decides."""
    for tops, others, v in ((2, 0, 40), (2, 3, 40), (4, 5, 5000), (2, 900, 20000)):
        x = np.full((8, v), -INF)
        x[:, 1:1 + tops] = 3.0
        x[:, 10:10 + others] = 3.0 - 47 * math.log(2) * 0.25  # weights of 2^-47 at a quarter's temperature
        u = np.linspace(0.05, 0.95, 8)
        got = check(bits_of(x), u, temperature=0.25, top_p=0.5)
        assert len(set(got.tolist())) == (tops // 2 + 1 if others else tops // 2)
        check(bits_of(x), u, temperature=0.25, top_p=0.5, top_k=tops)  # only the maxima
        check(bits_of(x), u, temperature=0.25, top_p=0.5, top_k=tops + 1)
        check(bits_of(x), u, temperature=0.25, top_p=0.5, min_p=0.1)


def test_masks(gdn):
    """Forbidden tokens, rows with one allowed token or none, NaN and infinities."""
    rng = np.random.default_rng(2)
    for v in (13, 9001, 40001):
        x = bell(rng, 12, v)
        x[0, rng.random(v) < 0.99] = -INF
        x[1] = -INF
        x[1, v // 2] = -4.0
        x[2] = -INF
        x[3] = NAN
        x[4, :] = np.where(np.arange(v) % 2, -INF, NAN)
        x[5, rng.random(v) < 0.5] = NAN
        x[6, [0, v // 3, v - 1]] = INF
        x[7, 5] = INF
        x[8] = -np.finfo(np.float32).max
        x[9] = 0.0
        x[9, ::2] = -0.0
        x[10] = -1e-38 * (1 + np.arange(v) % 5)
        x[11] = -3e38 * rng.random(v)
        bits = bits_of(x)
        for kw in (dict(), dict(temperature=0.0), dict(temperature=0.5, top_k=3), dict(top_p=0.7), dict(min_p=0.3)):
            check(bits, rng.random(12), **kw)


def test_parameters_out_of_their_range(gdn):
    rng = np.random.default_rng(3)
    bits = bits_of(bell(rng, 14, 3001))
    u = np.full(14, 0.4, np.float32)
    temperature = np.array([1, 1, 1, 1, 1, 1, 1, 1, -1, NAN, INF, 1e-30, 1e-42, 1e30], np.float32)
    top_p = np.array([-1, 0, 2, NAN, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1], np.float32)
    min_p = np.array([0, 0, 0, 0, -1, 2, NAN, 1, 0, 0, 0, 0, 0, 0], np.float32)
    top_k = np.array([0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, -5], np.int32)
    check(bits, u, temperature=temperature, top_p=top_p, min_p=min_p, top_k=top_k)
    check(bits, u, top_k=1 << 30)
    check(bits[:6], np.array([-1, 1, 2, NAN, INF, -INF], np.float32), top_p=0.9)


def test_u_of_one_and_more_is_the_nearest_below(gdn):
    """The largest fp32 below 1 leaves 2^-24 of the mass behind it: a token of 2^-36 is not drawn, one of 2^-20 is."""
    for below, want in ((25.0, 7), (14.0, 40)):
        x = np.full((4, 100), -INF)
        x[:, 7], x[:, 40] = 8.0, 8.0 - below
        check(bits_of(x), np.array([1, 2, INF, 1 - 2.0 ** -24], np.float32))
        token, logp = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
        L.gdn_sample(logits_on(bits_of(x)), torch.tensor([1, 2, INF, 1 - 2.0 ** -24], device="cuda"), token, logp)
        assert token.tolist() == [want] * 4


@pytest.mark.parametrize("name", ["tiny", "huge", "wide", "mixed magnitudes", "far", "near the largest number", "late maximum"])
def test_values_far_from_usual(gdn, name):
    """Logits whose magnitudes are far apart: the values between take more than one look."""
    rng = np.random.default_rng(len(name))
    v = 30011
    x = {"tiny": lambda: rng.standard_normal((4, v)) * 1e-6, "huge": lambda: rng.standard_normal((4, v)) * 1e6,
         "wide": lambda: rng.standard_normal((4, v)) * 300,
         "mixed magnitudes": lambda: np.exp(rng.uniform(-80, 3, (4, v))) * rng.choice([-1, 1], (4, v)),
         "far": lambda: rng.standard_normal((4, v)) * 0.1 - 200,
         "near the largest number": lambda: rng.uniform(-3e38, 3e38, (4, v)),
         "late maximum": lambda: np.where(np.arange(v) > v - 50, 90.0, rng.standard_normal((4, v)) * 1e-3)}[name]()
    bits = bits_of(x)
    for kw in (dict(), dict(temperature=3.0, top_p=0.6), dict(temperature=1e5), dict(temperature=1e38), dict(top_k=900), dict(top_k=20000, top_p=0.99)):
        check(bits, rng.random(4), **kw)


@pytest.mark.parametrize("rows,v", [(160, 40001), (80, 60003), (40, 100003), (3, 200003)])
@pytest.mark.parametrize("name", ["forbidden", "late", "late infinity", "late negative", "every slice its own"])
def test_counts_begin_again(gdn, name, rows, v):
    """Logits far above what a slice's first 16384 show, in slices of one, two, four and eight a row: the counts begin again
    with other bins, in some CTAs and not in others."""
    rng = np.random.default_rng(v)
    x = rng.standard_normal((rows, v))
    kw = dict(temperature=1.0, top_p=0.9)
    if name == "forbidden":  # few allowed, small ones first
        x *= 2.2
        x[rng.random((rows, v)) < 0.99] = -INF
        x[:, 17] = 1.0
        kw = dict(min_p=0.2, top_k=1231, top_p=0.99)
    elif name == "late":
        x[:, :v // 2] *= 1e-3
        x[:, -90:] += 40
        kw = dict(temperature=2.0, top_k=rng.choice([0, 5, 60, 700], rows))
    elif name == "late infinity":
        x[::2, -7] = INF
        x[1::2, -1] = 3e38
    elif name == "late negative":
        x[:, -5000:] = -1e6 * (1 + rng.random((rows, 5000)))
        kw = dict(temperature=1e7)
    else:
        x *= np.exp2(rng.integers(-6, 7, v // 1000 + 1)).repeat(1000)[:v]
        kw = dict(temperature=30.0)
    check(bits_of(x), rng.random(rows), **kw)


@pytest.mark.parametrize("temperature,below", [(1.0, 20.0), (1.0, 24.0), (0.25, 5.5), (8.0, 184.0)])
@pytest.mark.parametrize("v", [3001, 60003])
def test_logp_of_a_rare_token(gdn, v, temperature, below):
    """A token whose weight is a few units of the masses: logp is as near as any other's.  From the logits
    it is (x - max) / temperature - log(mass): two roundings of the first (2^-23 of it), log's of the second
    (2^-23 of it; it is half of |logp| at most), one of the mass (2^-24; the units are 2^-24 of it too)
    and the last one (2^-24 |logp|): below 2^-22 (1 + |logp|)."""
    x = np.full((2, v), 8.0 - below, np.float64)
    x[0, 5], x[1, v - 2] = 8.0, 8.0
    bits = bits_of(x)
    u = np.array([1 - 2.0 ** -23, 1 - 2.0 ** -23], np.float32)
    if not v * math.exp(-below / temperature) > 2.0 ** -22:
        u[:] = 1.0  # the last one
    token, logp = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda")
    L.gdn_sample(logits_on(bits), torch.from_numpy(u).cuda(), token, logp, temperature=torch.full((2,), temperature, device="cuda"))
    for i in range(2):
        assert R.values(bits[i])[int(token[i])] < 8.0
        lp = -below / temperature - math.log1p((v - 1) * math.exp(-below / temperature))
        assert abs(float(logp[i]) - lp) <= 2 ** -22 * (1 + abs(lp)), (i, float(logp[i]), lp)


def run_accept(logits, draft, active, u, ws=None, outputs=True, **kw):
    B, T, V = logits.shape
    z = lambda *s, dtype=torch.int32: torch.full(s, -9, dtype=dtype, device="cuda")
    if ws is None:
        ws = torch.zeros(L.gdn_accept_sampled_workspace_bytes(B, T, V), dtype=torch.uint8, device="cuda")
    keep, nxt = z(B), z(B)
    token, logp = (z(B, T), z(B, T, dtype=torch.float32)) if outputs else (None, None)
    L.gdn_accept_sampled(logits, draft, active, u, keep, nxt, token, logp, ws, **kw)
    return keep, nxt, token, logp, ws


@pytest.mark.parametrize("shape", [(1, 1, 50), (3, 2, 1003), (8, 2, 151936), (5, 64, 33), (64, 8, 3001)], ids=str)
def test_accept(gdn, shape):
    """keep and next follow from the tokens, the tokens are gdn_sample's, and the workspace is ready again."""
    B, T, V = shape
    rng = np.random.default_rng(V)
    bits = bits_of(bell(rng, B * T, V, peaks=1))
    x = logits_on(bits).view(B, T, V)
    active = (rng.random(B) < 0.8).astype(np.uint8)
    u = torch.from_numpy(rng.random((B, T)).astype(np.float32)).cuda()
    temp, top_p = torch.full((B,), 0.8, device="cuda"), torch.full((B,), 0.9, device="cuda")
    draft = rng.integers(0, V, (B, T)).astype(np.int32)
    ref = np.array([[R.draw(R.values(bits[b * T + t]), u[b, t].item(), 0.8, top_p=0.9)[0] for t in range(T)] for b in range(B)])
    for b in range(B):
        n = rng.integers(0, T)
        draft[b, 1:1 + n] = ref[b, :n]
    dev = torch.from_numpy(draft).cuda(), torch.from_numpy(active).cuda()
    ws = None
    for _ in range(3):
        keep, nxt, token, logp, ws = run_accept(x, *dev, u, ws, temperature=temp, top_p=top_p)
        k_ref, n_ref = R.accept(ref, draft, active)
        assert np.array_equal(keep.cpu().numpy(), k_ref) and np.array_equal(nxt.cpu().numpy(), n_ref)
        assert np.array_equal(token.cpu().numpy(), np.where(active[:, None] > 0, ref, -1))
        assert (logp.cpu().numpy()[active == 0] == 0).all()
    keep2, nxt2, _, _, _ = run_accept(x, *dev, u, ws, outputs=False, temperature=temp, top_p=top_p)
    assert torch.equal(keep, keep2) and torch.equal(nxt, nxt2)
    one = torch.zeros(B * T, dtype=torch.int32, device="cuda")
    each = lambda t: t.repeat_interleave(T)
    L.gdn_sample(x.view(B * T, V), u.view(-1), one, temperature=each(temp), top_p=each(top_p), active=each(dev[1]))
    assert torch.equal(one.view(B, T), token)


def test_one_workspace_for_calls_of_other_sizes(gdn):
    """Zeroed once, then used with other B and T, as a host that varies its drafts' depth does; all zero after each call."""
    rng = np.random.default_rng(12)
    ws = torch.zeros(max(L.gdn_accept_sampled_workspace_bytes(B, T, 1003) for B, T in ((200, 8), (700, 1), (3, 64))), dtype=torch.uint8, device="cuda")
    for B, T in ((4, 2), (200, 8), (4, 2), (3, 64), (700, 1), (70, 2), (200, 8), (4, 3)):
        x = torch.from_numpy(bell(rng, B * T, 1003)).bfloat16().cuda().view(B, T, 1003)
        draft = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
        active = torch.from_numpy((rng.random(B) < 0.8).astype(np.uint8)).cuda()
        u = torch.rand(B, T, device="cuda")
        first = torch.zeros(B * T, dtype=torch.int32, device="cuda")
        L.gdn_sample(x.view(B * T, 1003), u.view(-1), first)
        draft[:, 1:] = first.view(B, T)[:, :-1]  # all of them kept
        keep, nxt = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        L.gdn_accept_sampled(x, draft, active, u, keep, nxt, None, None, ws)
        on = active.bool()
        assert torch.equal(keep, torch.where(on, T, 0).int()), (B, T)
        assert torch.equal(nxt, torch.where(on, first.view(B, T)[:, -1], -1)), (B, T)
        assert not ws.any(), (B, T)


def test_accept_at_temperature_0_is_the_greedy_one(gdn):
    B, T, V = 6, 4, 5003
    rng = np.random.default_rng(9)
    bits = bits_of(bell(rng, B * T, V))
    bits[3] = bits_of(NAN)
    bits[5] = bits_of(-INF)
    x = logits_on(bits).view(B, T, V).contiguous()
    draft = torch.from_numpy(rng.integers(0, V, (B, T)).astype(np.int32)).cuda()
    draft[:, 1:3] = x.nan_to_num(nan=-INF, neginf=-INF).argmax(-1)[:, :2]
    active = torch.ones(B, dtype=torch.uint8, device="cuda")
    u = torch.rand(B, T, device="cuda")
    keep, nxt, *_ = run_accept(x, draft, active, u, temperature=torch.zeros(B, device="cuda"))
    k, n = torch.zeros_like(keep), torch.zeros_like(nxt)
    L.gdn_accept_greedy(x, draft, active, k, n, torch.zeros(L.gdn_accept_workspace_bytes(B, T, V), dtype=torch.uint8, device="cuda"))
    assert torch.equal(keep, k) and torch.equal(nxt, n)


def test_draws_follow_the_distribution(gdn):
    """Many draws of one row: with u = (i + 1/2) / n, a token's count is its probability times n to within one a border."""
    rng = np.random.default_rng(4)
    n, v = 4096, 300
    x = rng.standard_normal(v) * 2
    bits = np.broadcast_to(bits_of(x), (n, v)).copy()
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    token = torch.zeros(n, dtype=torch.int32, device="cuda")
    L.gdn_sample(logits_on(bits), torch.from_numpy(u).cuda(), token)
    p = np.exp(R.values(bits[0]))
    p /= p.sum()
    count = np.bincount(token.cpu().numpy(), minlength=v)
    assert np.abs(count - p * n).max() <= 1 + 1e-6


def test_captured_and_on_a_side_stream(gdn):
    """A captured call follows its inputs when it is replayed, beside a call on another stream."""
    B, T, V = 4, 3, 20011
    rng = np.random.default_rng(5)
    x = logits_on(bits_of(bell(rng, B * T, V))).view(B, T, V)
    y = logits_on(bits_of(bell(rng, B * T, V))).view(B, T, V)
    draft = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    u = torch.rand(B, T, device="cuda")
    top_k = torch.full((B,), 30, dtype=torch.int32, device="cuda")
    want = [run_accept(z, draft, None, u, top_k=top_k)[:4] for z in (x, y)]
    buf = x.clone()
    ws = torch.zeros(L.gdn_accept_sampled_workspace_bytes(B, T, V), dtype=torch.uint8, device="cuda")
    out = run_accept(buf, draft, None, u, ws, top_k=top_k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_accept(buf, draft, None, u, ws, top_k=top_k)
    side = torch.cuda.Stream()
    for z, w in zip((y, x, y), (want[1], want[0], want[1])):
        buf.copy_(z)
        graph.replay()
        with torch.cuda.stream(side):
            token = torch.zeros(B * T, dtype=torch.int32, device="cuda")
            L.gdn_sample(x.view(B * T, V), u.view(-1), token, top_k=top_k.repeat_interleave(T))
        torch.cuda.synchronize()
        for a, b in zip(out[:4], w):
            assert torch.equal(a, b)
        assert torch.equal(token.view(B, T), want[0][2])
