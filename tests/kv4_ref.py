"""Plain references of the paged 4-bit cache's operators, on the CPU: the plan
in Python integers, the append in the fp32 steps its definition names, the
attention in 64 bits.  They share no code with the library."""
import math

import numpy as np
import torch


def pack(x):
    """fp32 [..., d] -> (codes uint8 [..., d/2], entries fp16 [..., d/64, 2])."""
    x = np.asarray(x, np.float32)
    d = x.shape[-1]
    w = d // 64
    codes = np.zeros(x.shape, np.uint8)
    entries = np.zeros(x.shape[:-1] + (w, 2), np.float16)
    with np.errstate(all="ignore"):
        for g in range(w):
            ch = [c for c in range(d) if (c // 8) % w == g]
            y = x[..., ch]
            ok = np.isfinite(y).all(-1)
            base = np.clip(y.min(-1), np.float32(-65504), np.float32(65504)).astype(np.float16)
            step = np.minimum((y.max(-1) - y.min(-1)) / np.float32(15), np.float32(65504)).astype(np.float16)
            base, step = np.where(ok, base, np.float16(np.nan)), np.where(ok, step, np.float16(np.nan))
            b, s = base.astype(np.float32)[..., None], step.astype(np.float32)[..., None]
            c = np.clip(np.rint((y - b) / s), 0, 15)
            codes[..., ch] = np.where((s > 0) & ok[..., None], c, 0).astype(np.uint8)
            entries[..., g, 0], entries[..., g, 1] = step, base
    return codes[..., 0::2] | (codes[..., 1::2] << 4), entries


def values(codes, entries):
    """What codes and entries stand for, fp64 [..., d]."""
    d = codes.shape[-1] * 2
    w = d // 64
    code = np.empty(codes.shape[:-1] + (d,), np.float64)
    code[..., 0::2], code[..., 1::2] = codes & 15, codes >> 4
    g = (np.arange(d) // 8) % w
    e = entries.astype(np.float64)
    return e[..., g, 1] + e[..., g, 0] * code


class Cache:
    """A cache on the host: pages uint8 [n][H_kv][record], unwritten places
    random codes under NaN entries."""

    def __init__(self, n_pages, H_kv, page, d, seed=0):
        rng = np.random.default_rng(seed)
        self.n, self.H, self.P, self.d = n_pages, H_kv, page, d
        a, e = page * d // 2, page * (d // 64) * 4
        self.bytes = np.zeros((n_pages, H_kv, 2 * (a + e)), np.uint8)
        self.bytes[..., :2 * a] = rng.integers(0, 256, (n_pages, H_kv, 2 * a))
        self.bytes[..., 2 * a:] = np.frombuffer(np.full(1, np.nan, np.float16).tobytes(), np.uint8)[None].repeat(e, 0).reshape(-1)
        self.a, self.e = a, e

    def views(self, data=None):
        b = self.bytes if data is None else data
        a, e, w = self.a, self.e, self.d // 64
        ent = b[..., 2 * a:].copy().view(np.float16)
        shape = b.shape[:2]
        return (b[..., :a].reshape(*shape, self.P, -1), b[..., a:2 * a].reshape(*shape, self.P, -1),
                ent[..., :e // 2].reshape(*shape, self.P, w, 2), ent[..., e // 2:].reshape(*shape, self.P, w, 2))

    def write(self, slot, k, v):
        """One token's k, v fp32 [H][d] at a slot."""
        page, off = divmod(slot, self.P)
        a, e, w = self.a, self.e, self.d // 64
        for i, x in enumerate((k, v)):
            c, s = pack(x)
            self.bytes[page, :, i * a + off * self.d // 2: i * a + (off + 1) * self.d // 2] = c
            at = 2 * a + i * e + off * w * 4
            self.bytes[page, :, at: at + w * 4] = s.reshape(self.H, -1).view(np.uint8)

    def read(self, slots, data=None):
        """(k, v) fp64 [len(slots)][H][d]; a negative slot reads as zeros."""
        kc, vc, ke, ve = self.views(data)
        s = np.asarray(slots, np.int64)
        page, off = np.maximum(s, 0) // self.P, np.maximum(s, 0) % self.P
        dead = (s < 0)[:, None, None]
        return (np.where(dead, 0, values(kc[page, :, off], ke[page, :, off])), np.where(dead, 0, values(vc[page, :, off], ve[page, :, off])))


def rotate(x, angles_cs, rot, pairs):
    """fp32 [N][H][d] turned by (cos, sin) fp32 [N][rot/2][2], one rounding a product and a sum."""
    x = np.array(x, np.float32)
    half = rot // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    c, s = angles_cs[:, None, :, 0], angles_cs[:, None, :, 1]
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a] = xa * c - xb * s
    x[..., b] = xb * c + xa * s
    return x


def plan(page, max_pages, n_pages, T, N, lens, add, active, held, table, free, count):
    """The plan's definition, row by row; returns the new state and the outputs."""
    B = len(lens)
    held, table, free = list(held), [list(r) for r in table], list(free)
    status = 0
    a = [max(int(x), 0) if f else 0 for x, f in zip(add, active)]
    want, bad = [], []
    for b in range(B):
        w = -(-(int(lens[b]) + a[b]) // page)
        no = lens[b] < 0 or w > max_pages or (T > 0 and a[b] > T) or not 0 <= held[b] <= max_pages
        bad.append(no)
        if no:
            a[b] = 0
            status |= 32
        want.append(held[b] if no else w)
    for b in range(B):
        for c in range(want[b], held[b]):
            free[count] = table[b][c]
            count += 1
            table[b][c] = -1
        held[b] = min(held[b], want[b])
    need_sum = tok_sum = taken = 0
    top = count
    q_start, q_count, kv_len = [], [], []
    at = 0
    for b in range(B):
        need_sum += want[b] - held[b]
        tok_sum += a[b]
        if need_sum > top or (T == 0 and tok_sum > N):
            if a[b] or want[b] > held[b]:
                status |= 8
            a[b] = 0
        else:
            while held[b] < want[b]:
                count -= 1
                table[b][held[b]] = free[count]
                held[b] += 1
        q_start.append(b * T if T else at)
        q_count.append(a[b])
        kv_len.append(max(int(lens[b]), 0) + a[b])
        at += a[b]
    q_start.append(B * T if T else at)
    slots, pos = [-1] * N, [-1] * N
    for b in range(B):
        for i in range(a[b]):
            x = int(lens[b]) + i
            slots[q_start[b] + i] = table[b][x // page] * page + x % page
            pos[q_start[b] + i] = x
    return dict(held=held, table=table, free=free, count=count, q_start=q_start, q_count=q_count, kv_len=kv_len, slots=slots, positions=pos, status=status)


def attend(q, cache, table, q_start, q_count, kv_len, scale, data=None):
    """fp64 outputs [N][H_q][d] (NaN where no span has the token) and, for each
    value, how far 16-bit operands may move it: with u = 2^-11 (fp16, half a
    step), a key rounded once moves a score by at most u * scale * sum |q k|,
    a query scaled by a power of two by nothing, probabilities and values
    rounded once each by u, and fp32 sums by n 2^-24."""
    N, Hq, d = q.shape
    G = Hq // cache.H
    out = np.full((N, Hq, d), np.nan)
    tol = np.zeros((N, Hq, d))
    u = 2.0 ** -11
    for b in range(len(q_count)):
        s, e = q_start[b], q_start[b + 1]
        out[s:e] = 0
        n, m = kv_len[b], q_count[b]
        slots = [table[b][t // cache.P] * cache.P + t % cache.P for t in range(n)]
        if not n or not m:
            continue
        k, v = cache.read(slots, data)
        for i in range(m):
            seen = n - m + i + 1
            if seen <= 0:
                continue
            for h in range(Hq):
                kk, vv = k[:seen, h // G], v[:seen, h // G]
                x = kk @ q[s + i, h] * scale
                moved = u * abs(scale) * (np.abs(kk) @ np.abs(q[s + i, h]))
                p = np.exp(x - x.max())
                p /= p.sum()
                out[s + i, h] = p @ vv
                spread = np.abs(vv - out[s + i, h])
                tol[s + i, h] = (p * (moved + 2.0 ** -20 * (1 + np.abs(x)))) @ spread * 1.02 + (2 * u + (seen + 64) * 2.0 ** -24) * (p @ np.abs(vv))
    tol = tol + 2.0 ** -8 * np.abs(np.nan_to_num(out)) + 1e-30
    return out, tol


def rope_table(top, rot, base=1e6):
    half = rot // 2
    inv = base ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))
    ang = torch.arange(top, dtype=torch.float64)[:, None] * inv[None]
    return torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


assert math.isnan(float(np.float16(np.nan)))
