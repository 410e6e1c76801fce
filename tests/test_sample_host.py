"""Sampled decoding without a GPU: sizes, refusals before any launch, the reference's own sense, and the weights' arithmetic."""
import math
import os
import re
from fractions import Fraction

import numpy as np
import pytest

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import sample_ref as R
from tests.conftest import ROOT

G = 1 << 20  # an aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return L.load()


def sample(lib, B=4, V=100, logits=G, stride=100, active=G, temp=G, k=G, p=G, m=G, u=G, token=G, logp=G):
    return lib.gdn_sample(B, V, logits, stride, active, temp, k, p, m, u, token, logp, None)


def test_sample_refuses(lib):
    for name in ("logits", "u", "token"):
        assert sample(lib, **{name: None}) == L.GDN_ERR_INVALID_ARG, name
    assert sample(lib, logits=G + 1) == L.GDN_ERR_MISALIGNED
    for name in ("temp", "k", "p", "m", "u", "token", "logp"):
        assert sample(lib, **{name: G + 2}) == L.GDN_ERR_MISALIGNED, name
    for kw in (dict(B=-1), dict(V=0), dict(stride=99), dict(stride=(1 << 40) + 1)):
        assert sample(lib, **kw) == L.GDN_ERR_INVALID_ARG, kw
    for kw in (dict(B=65536), dict(V=(1 << 20) + 1, stride=1 << 21)):
        assert sample(lib, **kw) == L.GDN_ERR_UNSUPPORTED, kw
        assert L.gdn_last_error()
    assert sample(lib, B=0, logits=None, u=None, token=None) == L.GDN_OK


def test_accept_refuses(lib):
    need = L.gdn_accept_sampled_workspace_bytes(4, 3, 100)
    assert need > 0
    for bad in ((-1, 3, 100), (4, 0, 100), (4, 65, 100), (4, 3, 0), (4, 3, (1 << 20) + 1), (65535, 2, 100)):
        assert L.gdn_accept_sampled_workspace_bytes(*bad) == 0

    def call(B=4, T=3, V=100, logits=G, stride=100, draft=G, active=G, temp=G, k=G, p=G, m=G, u=G, keep=G, nxt=G, token=G, logp=G, ws=G, n=need):
        return lib.gdn_accept_sampled(B, T, V, logits, stride, draft, active, temp, k, p, m, u, keep, nxt, token, logp, ws, n, None)

    for name in ("logits", "draft", "u", "keep", "nxt", "ws"):
        assert call(**{name: None}) == L.GDN_ERR_INVALID_ARG, name
    for name in ("draft", "temp", "k", "p", "m", "u", "keep", "nxt", "token", "logp", "ws"):
        assert call(**{name: G + 2}) == L.GDN_ERR_MISALIGNED, name
    assert call(n=need - 1) == L.GDN_ERR_WORKSPACE
    assert call(T=65) == L.GDN_ERR_UNSUPPORTED and call(B=65535, T=2) == L.GDN_ERR_UNSUPPORTED
    assert call(T=0) == L.GDN_ERR_INVALID_ARG and call(stride=99) == L.GDN_ERR_INVALID_ARG
    assert call(B=0, logits=None, draft=None, u=None, keep=None, nxt=None, ws=None, n=0) == L.GDN_OK


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    f, i = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(4, 100, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        L.gdn_sample(x, f, i)
    with pytest.raises(TypeError, match="logits"):
        L.gdn_sample(None, f, i)
    with pytest.raises(TypeError, match="logits"):
        L.gdn_accept_sampled(7, i, i, f, i, i, i, f, i)


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    """A fake tensor of device 1 where device 0 is the current one, in the place of each argument."""
    torch = pytest.importorskip("torch")

    class Fake:
        def __init__(self, shape, dtype, device):
            self.shape, self.dtype, self.at, self.device, self.is_cuda = shape, dtype, device, f"cuda:{device}", True

        numel = lambda self: math.prod(self.shape)
        element_size = lambda self: 4
        get_device = lambda self: self.at
        is_contiguous = lambda self: True
        data_ptr = lambda self: G
        stride = lambda self: tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    monkeypatch.setattr(L, "_here", lambda: 0)
    monkeypatch.setattr(L, "_need", lambda **a: None)
    monkeypatch.setattr(L, "_ptr", lambda t, what, dtype=None: G)
    B, T, V = 3, 2, 50
    i32, f32 = torch.int32, torch.float32
    sizes = dict(u=((B, T), f32), keep=((B,), i32), nxt=((B,), i32), token=((B, T), i32), logp=((B, T), f32), ws=((4096,), torch.uint8),
                 temperature=((B,), f32), top_k=((B,), i32), top_p=((B,), f32), min_p=((B,), f32), logits=((B, T, V), torch.bfloat16),
                 draft=((B, T), i32), active=((B,), torch.uint8))
    for bad in sizes:
        args = {k: Fake(shape, dtype, int(k == bad)) for k, (shape, dtype) in sizes.items()}
        with pytest.raises(ValueError, match="cuda:1"):
            L.gdn_accept_sampled(**args)


def test_reference_in_small():
    x = np.log(np.array([0.1, 0.4, 0.1, 0.3, 0.1]))
    assert [R.draw(x, u)[0] for u in (0.0, 0.39, 0.41, 0.69, 0.71, 0.79, 0.81, 0.95)] == [1, 1, 3, 3, 0, 0, 2, 4]
    assert [R.draw(x, u, top_k=3)[0] for u in (0.49, 0.51, 0.9)] == [1, 3, 0]
    assert [R.draw(x, u, top_p=0.65)[0] for u in (0.5, 0.6, 0.99)] == [1, 3, 3]
    assert R.draw(x, 0.99, min_p=0.5)[0] == 3
    assert abs(R.draw(x, 0.0)[1] - math.log(0.4)) < 1e-12
    assert R.draw([math.nan, -math.inf], 0.5)[0] == 1 and R.draw([math.nan] * 2, 0.5)[0] == 0


def test_table_of_powers():
    """The table's entries are 2^(m/32) in units of 2^-62, to the nearest: entry^32 against 2^(m + 62 * 32) on both sides."""
    text = open(os.path.join(ROOT, "speculative_decode_gated_gdn_gb300", "csrc", "sample.cuh")).read()
    table = [int(x, 16) for x in re.findall(r"0x([0-9a-f]{16})ull", text)]
    assert len(table) == 32
    for m, t in enumerate(table):
        target = Fraction(2) ** (m + 62 * 32)
        assert (t - Fraction(1, 2)) ** 32 <= target <= (t + Fraction(1, 2)) ** 32


def test_weights_arithmetic():
    """The weights' steps in numpy's fp32, against exp in 64 bits: within 2^-37 of the value and 2^-43 of the largest."""
    text = open(os.path.join(ROOT, "speculative_decode_gated_gdn_gb300", "csrc", "sample.cuh")).read()
    table = [int(x, 16) for x in re.findall(r"0x([0-9a-f]{16})ull", text)]
    f = np.float32
    rng = np.random.default_rng(0)

    def fma(a, b, c):
        return f(np.longdouble(a) * np.longdouble(b) + np.longdouble(c))

    worst = 0.0
    for _ in range(4000):
        temp = f(np.exp(rng.uniform(-3, 3)))
        zmax, z = (R.values((np.float32(v).view(np.uint32) >> 16).astype(np.uint16)) for v in (rng.uniform(-5, 30), rng.uniform(-40, 20)))
        zmax, z = max(zmax, z), min(zmax, z)
        if zmax == z or (z - zmax) / float(temp) < -29:
            continue
        c = 2.8853900817779268147 / np.float64(temp)
        hi_c = f(c)
        lo_c = f(c - np.float64(hi_c))
        a, b = f(0.5 * z), f(0.5 * zmax)
        s = f(a - b)
        back = f(s - a)
        err = f(f(a - f(s - back)) + f(f(-b) - back))
        t = f(s * hi_c)
        t_lo = f(fma(s, hi_c, -t) + fma(s, lo_c, f(err * hi_c)))
        k = int(np.rint(f(t * f(32))))
        r = fma(f(k), f(-0.03125), t)
        ln2, ln2_lo = f(0.693147182464599609), f(-1.9046542121259336e-9)
        y = f(r * ln2)
        y_lo = f(fma(r, ln2, -y) + fma(r, ln2_lo, f(t_lo * ln2)))
        hi = f(y + y_lo)
        lo = f(y_lo - f(hi - y))
        q = f(f(hi * hi) * fma(hi, fma(hi, fma(hi, f(1 / 120), f(1 / 24)), f(1 / 6)), f(0.5)))
        F = (1 << 50) + int(np.rint(np.float64(hi) * 2.0 ** 50)) + int(np.rint(np.float64(f(fma(lo, hi, lo) + q)) * 2.0 ** 50))
        w = table[k & 31] * (F << 13) >> 64
        shift = 61 - 43 - (k >> 5)
        w = (w + (1 << (shift - 1))) >> shift
        true = math.exp((z - zmax) / np.float64(temp))
        worst = max(worst, (abs(w * 2.0 ** -43 - true) - 2.0 ** -43) / true)
    assert worst < 2.0 ** -37
