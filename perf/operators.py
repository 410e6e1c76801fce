"""What the attention layers of a hybrid model cost next to its GDN layers, operator by operator.

A verify cycle of such a model needs, for its attention layers, pages for the new tokens' keys and values, the rotated
queries and keys, the cache itself and the attention that reads it.  The cases below measure these operators:

  plan     gdn_kv_plan: block tables, slots and positions from the rows' lengths, on the device (a cycle that takes the
           drafts' pages, then one that gives them back)
  append   gdn_kv4_append + gdn_kv4_read: rotary positions with several axes on q and k, k and v into a cache of 4 bits,
           and the appended tokens read back as the values that the cache stands for
  attend   gdn_kv4_attend: causal attention of the new tokens over that cache, from one token to a whole prompt

The cache: a page holds `page` tokens; for each kv head it is one record
  K codes [page][d/2] | V codes [page][d/2] | K scales [page][d/64] | V scales [page][d/64]
with channel 2i in the low and 2i+1 in the high four bits of byte i, and a scale entry = (fp16 step, fp16 base).
Channel c belongs to group (c / 8) mod (d / 64) of its token and stands for base + step * code.
"""
import math

import numpy as np
import torch

own = False

F16_MAX = 65504.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the eight-row cohort with one draft a row, long prompts behind it (13,239 tokens), two rows idle
        dict(name="plan cohort", op="plan", B=8, T=2, fixed=True, page=64, kv=13239, idle=2, chunk=0),
        # a serving batch that mixes single tokens, drafts and chunks of prompts over small pages
        dict(name="plan mixed batch", op="plan", B=768, T=4, fixed=False, page=16, kv=32768, idle=96, chunk=1024),
        # the same cohort's 16 new tokens, a quarter of each head rotated, positions of three axes
        dict(name="append cohort", op="append", B=8, T=2, Hq=16, Hkv=2, d=256, rot=64, axes=3, page=64, idle=2),
        # a prompt with pictures: every channel rotated, half-odd length
        dict(name="append pictures", op="append", B=3, T=1367, Hq=32, Hkv=8, d=128, rot=128, axes=3, page=32, idle=0),
        # the long prompt of the prefill benchmark, text only
        dict(name="append prompt 32768", op="append", B=1, T=32768, Hq=16, Hkv=2, d=256, rot=64, axes=1, page=64, idle=0),
        # the smallest call: one row, one token, a short context
        dict(name="attend one token", op="attend", B=1, T=1, Hq=8, Hkv=8, d=64, page=16, kv=129, spread=0.0, idle=0),
        # the cohort's verify over its long prompts
        dict(name="attend cohort", op="attend", B=8, T=2, Hq=16, Hkv=2, d=256, page=64, kv=13239, spread=0.2, idle=2),
        # one request with a very long context: few rows, one long axis
        dict(name="attend long context", op="attend", B=1, T=2, Hq=32, Hkv=8, d=128, page=64, kv=131001, spread=0.0, idle=0),
        # plain decoding of a ragged batch
        dict(name="attend ragged batch", op="attend", B=64, T=1, Hq=32, Hkv=8, d=128, page=32, kv=8192, spread=0.9, idle=5),
        # deep drafts: eight positions a row
        dict(name="attend deep drafts", op="attend", B=32, T=8, Hq=32, Hkv=4, d=128, page=64, kv=6001, spread=0.5, idle=8),
        # a whole prompt of the prefill benchmark at once
        dict(name="attend prompt 4096", op="attend", B=1, T=4096, Hq=16, Hkv=2, d=256, page=64, kv=4096, spread=0.0, idle=0),
        # a chunk of a prompt behind a long prefix
        dict(name="attend chunk", op="attend", B=1, T=2000, Hq=32, Hkv=8, d=128, page=16, kv=18001, spread=0.0, idle=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64])
    if op == "plan":
        B = _log_int(rng, 1, 768)
        fixed = rng.random() < 0.5
        return dict(op=op, B=B, T=rng.randint(1, 8), fixed=fixed, page=page, kv=_log_int(rng, 1, 32768), idle=rng.randint(0, B // 4),
                    chunk=0 if fixed else _log_int(rng, 16, 1024))
    while True:
        d, Hkv, group = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        if (group + 2) * Hkv * d != 3 * 1024:
            break
    Hq = Hkv * group
    if op == "append":
        B = _log_int(rng, 1, 64)
        T = rng.randint(1, 8) if rng.random() < 0.5 else _log_int(rng, 9, max(9, 120_000_000 // (B * d * (Hq + 2 * Hkv))))
        return dict(op=op, B=B, T=min(T, 32768 // B), Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([0, d // 4, d // 2, d]), axes=rng.choice([1, 3, 4]), page=page, idle=rng.randint(0, B // 4))
    if rng.random() < 0.6:  # verify or decode
        B, T = _log_int(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 8])
        kv = _log_int(rng, T, min(65536, 280_000_000 // (B * Hkv * d)))
    else:  # prompts
        B, T = rng.choice([1, 1, 2, 3]), _log_int(rng, 9, 2500)
        kv = _log_int(rng, T, max(T, min(16384, 130_000_000_000 // (B * Hq * T * d))))
    return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, page=page, kv=kv, spread=rng.choice([0.0, 0.3, 0.9]), idle=rng.randint(0, B // 4))


def _rows(case):
    """The rows' lengths, new tokens and active flags: what the case fixes, whatever the seed."""
    c = case
    r = np.random.RandomState((c["B"] * 7919 + c["T"] * 104729 + c.get("kv", 0) * 31 + c["page"]) % (1 << 31))
    active = np.ones(c["B"], np.uint8)
    if c["idle"]:
        active[r.permutation(c["B"])[: c["idle"]]] = 0
    if c["op"] == "append":
        lens = r.randint(0, 2000, c["B"]).astype(np.int32)
        return lens, np.full(c["B"], c["T"], np.int32), active
    if c["op"] == "attend":  # lens counts the new tokens too
        low = max(c["T"], int(c["kv"] * (1 - c["spread"])))
        lens = r.randint(low, c["kv"] + 1, c["B"]).astype(np.int32) if low < c["kv"] else np.full(c["B"], c["kv"], np.int32)
        lens[r.randint(0, c["B"])] = c["kv"]
        return lens, np.full(c["B"], c["T"], np.int32), active
    lens = np.exp(r.uniform(0, math.log(c["kv"] + 1), c["B"])).astype(np.int32)
    add = r.randint(1, c["T"] + 1, c["B"]).astype(np.int32)
    if c["chunk"]:
        some = r.rand(c["B"]) < 0.1
        add[some] = r.randint(1, c["chunk"] + 1, int(some.sum()))
    return lens, add, active


# ------------------------------------------------------------------ the cache's format
def _groups(d, device):
    return (torch.arange(d, device=device) // 8) % (d // 64)


def _parts(pages, page, d):
    """Views of a cache: codes [n][Hkv][page][d/2] and scale entries [n][Hkv][page][d/64][2] of K and V."""
    n, h = pages.shape[:2]
    a, w = page * d // 2, d // 64
    s = pages[..., 2 * a:].view(torch.float16)
    return (pages[..., :a].unflatten(-1, (page, d // 2)), pages[..., a:2 * a].unflatten(-1, (page, d // 2)),
            s[..., :page * w * 2].unflatten(-1, (page, w, 2)), s[..., page * w * 2:].unflatten(-1, (page, w, 2)))


def _quantise(x):
    """x [..., d] -> codes [..., d/2] uint8, entries [..., d/64, 2] fp16, in x's own precision."""
    d = x.shape[-1]
    g = x.unflatten(-1, (8, d // 64, 8)).transpose(-3, -2).flatten(-2)  # [..., d/64, 64]
    fine = torch.isfinite(g).all(-1)
    base = g.amin(-1).clamp(-F16_MAX, F16_MAX).to(torch.float16)
    step = ((g.amax(-1) - g.amin(-1)) / torch.tensor(15.0, dtype=g.dtype, device=g.device)).clamp(max=F16_MAX).to(torch.float16)
    bad = torch.tensor(math.nan, dtype=torch.float16, device=x.device)
    base, step = torch.where(fine, base, bad), torch.where(fine, step, bad)
    b, s = base.to(g.dtype)[..., None], step.to(g.dtype)[..., None]
    code = torch.where((s > 0) & fine[..., None], ((g - b) / s).round().clamp(0, 15), torch.zeros((), dtype=g.dtype, device=g.device))
    code = code.unflatten(-1, (8, 8)).transpose(-3, -2).flatten(-3).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.stack([step, base], -1)


def _values(codes, entries, dtype=torch.float32):
    d = codes.shape[-1] * 2
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(dtype)
    e = entries.to(dtype)[..., _groups(d, codes.device), :]
    return e[..., 0] * code + e[..., 1]


# ------------------------------------------------------------------ inputs
def _pages(case, lens, gen, dev):
    """A block table of scattered pages, -1 behind each row's own, and an empty cache; unwritten places hold NaN entries."""
    c = case
    held = -(-lens // c["page"])
    n = int(held.sum()) + 3
    width = max(1, int(held.max()))
    order = torch.randperm(n, generator=gen, device=dev).to(torch.int32)
    table = torch.full((c["B"], width), -1, dtype=torch.int32, device=dev)
    col = torch.arange(width, device=dev)
    h = torch.from_numpy(held.astype(np.int64)).to(dev)
    first = torch.cumsum(h, 0) - h
    mine = col[None] < h[:, None]
    table = torch.where(mine, order[(first[:, None] + col[None]).clamp(max=n - 1)], table)
    rec = c["page"] * (c["d"] + c["d"] // 64 * 8)
    cache = torch.empty(n + 1, c["Hkv"], rec, dtype=torch.uint8, device=dev)  # the page behind the last is nobody's
    a = c["page"] * c["d"]
    cache[..., :a] = torch.randint(0, 256, (1, c["Hkv"], a), generator=gen, device=dev).to(torch.uint8)
    cache[..., a:].view(torch.float16).fill_(math.nan)
    return table.contiguous(), cache, n


def _filled(case, lens, gen, dev):
    """The same with keys and values of every row's first lens[b] tokens."""
    c = case
    table, cache, n = _pages(c, lens, gen, dev)
    kc, vc, ke, ve = _parts(cache, c["page"], c["d"])
    # keys have a few channels far from zero, values have not
    offset = torch.randn(c["Hkv"], 1, c["d"], generator=gen, device=dev) * (torch.rand(c["Hkv"], 1, c["d"], generator=gen, device=dev) < 0.05) * 4
    block = max(1, (1 << 25) // (c["Hkv"] * c["page"] * c["d"]))
    of = torch.full((n + 1,), 0, dtype=torch.int64, device=dev)  # tokens in each page
    cnt = (torch.from_numpy(lens.astype(np.int64)).to(dev)[:, None] - torch.arange(table.shape[1], device=dev)[None] * c["page"]).clamp(0, c["page"])
    of.scatter_(0, torch.where(table < 0, n, table).long().flatten(), cnt.flatten())
    of[n] = 0
    tok = torch.arange(c["page"], device=dev)
    for a in range(0, n, block):
        b = min(n, a + block)
        live = (tok[None] < of[a:b, None])[:, None, :, None]
        for codes, entries, off in ((kc, ke, offset), (vc, ve, None)):
            x = torch.randn(b - a, c["Hkv"], c["page"], c["d"], generator=gen, device=dev)
            x = (x + off if off is not None else x).to(torch.bfloat16).float()
            q, e = _quantise(x)
            codes[a:b] = torch.where(live, q, codes[a:b])
            entries[a:b] = torch.where(live[..., None], e, entries[a:b])
    return table, cache, n


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens_h, add_h, active_h = _rows(c)
    s = dict(case=c, lens=torch.from_numpy(lens_h).to(dev), add=torch.from_numpy(add_h).to(dev), active=torch.from_numpy(active_h).to(dev))
    i32 = dict(dtype=torch.int32, device=dev)
    B = c["B"]
    if c["op"] == "plan":
        longest = c["kv"] + max(c["T"], c["chunk"])
        M = -(-longest // c["page"])
        held_h = -(-lens_h // c["page"])
        spare = int((-(-(lens_h + add_h) // c["page"]) - held_h).sum()) + 8
        n = int(held_h.sum()) + spare
        order = torch.randperm(n, generator=gen, device=dev).to(torch.int32)
        held = torch.from_numpy(held_h.astype(np.int32)).to(dev)
        col = torch.arange(M, device=dev)
        first = torch.cumsum(held.long(), 0) - held
        table = torch.where(col[None] < held[:, None], order[(first[:, None] + col[None]).clamp(max=n - 1)], torch.full((), -1, **i32)).contiguous()
        free = torch.cat([order[int(held_h.sum()):], torch.full((int(held_h.sum()),), -1, **i32)]).contiguous()
        N = B * c["T"] if c["fixed"] else int((add_h * active_h).sum()) + 5
        outs = [dict(q_start=torch.zeros(B + 1, **i32), q_count=torch.zeros(B, **i32), kv_len=torch.zeros(B, **i32), slots=torch.zeros(N, **i32), positions=torch.zeros(N, **i32))
                for _ in range(2)]
        s |= dict(N=N, M=M, n=n, held=held, table=table, free=free, free_count=torch.full((1,), spare, **i32), outs=outs, none=torch.zeros(B, **i32))
        if own:
            from speculative_decode_gated_gdn_gb300 import lib as L
            s["kd"] = L.kv4_dims(B, 1, 1, 64, c["page"], M, n)
        return s
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if c["op"] == "append":
        total = lens_h + add_h
        table, cache, n = _pages(c, total, gen, dev)
        N = B * c["T"]
        row = torch.arange(N, device=dev) // c["T"]
        pos = s["lens"].long()[row] + torch.arange(N, device=dev) % c["T"]
        slots = table[row, pos // c["page"]].long() * c["page"] + pos % c["page"]
        slots = torch.where(s["active"][row] > 0, slots, -1).to(torch.int32)
        # one fused projection: q | k | v of a token side by side
        x = torch.randn(N, Hq + 2 * Hkv, d, generator=gen, device=dev)
        x[:, :, :: 37] *= 4.0
        x = x.to(torch.bfloat16)
        # text positions far into a context on the first axis, grid places on the others
        positions = torch.stack([pos + 100_000] + [torch.randint(0, 1000, (N,), generator=gen, device=dev) for _ in range(c["axes"] - 1)]).to(torch.int32).contiguous()
        half = c["rot"] // 2
        axis = [i % c["axes"] for i in range(half)]
        inv = 1e6 ** (-torch.arange(half, device=dev, dtype=torch.float64) / max(half, 1))
        top = 140_000
        ang = torch.arange(top, device=dev, dtype=torch.float64)[:, None] * inv[None]
        rope = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()  # what a program builds once
        s |= dict(N=N, n=n, x=x, q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], positions=positions, axis=bytes(axis), inv=inv, top=top, rope=rope, slots=slots, cache=cache)
        s["axis_t"] = torch.tensor(axis, device=dev, dtype=torch.int64)
        s |= dict(q_out=torch.empty(N, Hq, d, dtype=torch.bfloat16, device=dev), k_out=torch.empty(N, Hkv, d, dtype=torch.bfloat16, device=dev), v_out=torch.empty(N, Hkv, d, dtype=torch.bfloat16, device=dev))
        if own:
            from speculative_decode_gated_gdn_gb300 import lib as L
            s["kd"] = L.kv4_dims(B, Hq, Hkv, d, c["page"], table.shape[1], n)
        return s
    table, cache, n = _filled(c, lens_h, gen, dev)
    N = B * c["T"]
    count = s["add"] * s["active"].to(torch.int32)
    s |= dict(N=N, n=n, table=table, cache=cache, q=torch.randn(N, Hq, d, generator=gen, device=dev).mul_(1.5).to(torch.bfloat16), q_start=(torch.arange(B + 1, device=dev) * c["T"]).to(torch.int32),
              q_count=count, kv_len=s["lens"], scale=d ** -0.5, out=torch.empty(N, Hq, d, dtype=torch.bfloat16, device=dev))
    if own:
        from speculative_decode_gated_gdn_gb300 import lib as L
        s["kd"] = L.kv4_dims(B, Hq, Hkv, d, c["page"], table.shape[1], n)
        s["ws"] = torch.zeros(L.gdn_kv4_attend_workspace_bytes(s["kd"], N, c["T"]), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"plan": _run_plan, "append": _run_append, "attend": _run_attend}[s["case"]["op"]](s)


def _run_plan(s):
    c = s["case"]
    a, b = s["outs"]
    if own:
        from speculative_decode_gated_gdn_gb300 import lib as L
        for o, add in ((a, s["add"]), (b, s["none"])):
            L.gdn_kv_plan(s["kd"], s["lens"], add, s["active"], s["held"], s["table"], s["free"], s["free_count"], o["q_start"], o["q_count"], o["kv_len"], o["slots"], o["positions"],
                          T=c["T"] if c["fixed"] else 0)
        return dict(drafts=a, back=b, held=s["held"], table=s["table"], free=s["free"], free_count=s["free_count"])
    res = []
    for add in (s["add"], s["none"]):
        res.append(_plan(s, add))
    return dict(drafts=res[0], back=res[1], held=s["held"], table=s["table"], free=s["free"], free_count=s["free_count"])


def _plan(s, add):
    """Rows are served in their order; the first that finds no page or no place, and all that add tokens after it, get none."""
    c, dev, N, n, M, P = s["case"], s["lens"].device, s["N"], s["n"], s["M"], s["case"]["page"]
    lens, held = s["lens"].long(), s["held"].long()
    a = torch.where(s["active"] > 0, add.long().clamp(min=0), 0)
    want = (lens + a + P - 1) // P
    bad = (lens < 0) | (want > M) | (a > c["T"] if c["fixed"] else torch.zeros_like(lens, dtype=torch.bool))
    a = torch.where(bad, 0, a)
    want = torch.where(bad, held, want)
    rel = (held - want).clamp(min=0)
    need = (want - held).clamp(min=0)
    count = s["free_count"].long()
    avail = count + rel.sum()
    ends = torch.cumsum(need, 0)
    fits = ends <= avail
    if not c["fixed"]:
        fits &= torch.cumsum(a, 0) <= N
    a = torch.where(fits, a, 0)
    need = torch.where(fits, need, 0)
    col = torch.arange(M, device=dev)[None]
    # pages given back go onto the free list in row order, then pages are taken from its end
    back = (col >= want[:, None]) & (col < held[:, None]) & (rel[:, None] > 0)
    at = count + (torch.cumsum(rel, 0) - rel)[:, None] + col - want[:, None]
    free = torch.cat([s["free"], s["free"][:1]])
    free.scatter_(0, torch.where(back, at, n).flatten(), s["table"].flatten())
    free = free[:n]
    table = torch.where(back, -1, s["table"])
    new = (col >= held[:, None]) & (col < (held + need)[:, None])
    take = avail - 1 - ((ends - (want - held).clamp(min=0))[:, None] + col - held[:, None])
    table = torch.where(new, free[take.clamp(0, n - 1)], table)
    s["free"].copy_(free)
    s["table"].copy_(table)
    s["held"].copy_((held - rel + need).to(torch.int32))
    s["free_count"].copy_((avail - need.sum()).to(torch.int32))
    i = torch.arange(N, device=dev)
    if c["fixed"]:
        start = torch.arange(c["B"] + 1, device=dev) * c["T"]
    else:
        start = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(a, 0)])
    row = (torch.searchsorted(start, i, right=True) - 1).clamp(0, c["B"] - 1)
    k = i - start[row]
    live = (k < a[row]) & (i < start[-1])
    pos = lens[row] + k
    page = table[row, (pos // P).clamp(0, M - 1)].long()
    return dict(q_start=start.to(torch.int32), q_count=a.to(torch.int32), kv_len=(lens.clamp(min=0) + a).to(torch.int32), slots=torch.where(live, page * P + pos % P, -1).to(torch.int32),
                positions=torch.where(live, pos, -1).to(torch.int32))


def _rotate(x, cos, sin):
    """The first 2 * half channels turned: channel i with channel i + half."""
    half = cos.shape[-1]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _run_append(s):
    c, N = s["case"], s["N"]
    if own:
        from speculative_decode_gated_gdn_gb300 import lib as L
        L.gdn_kv4_append(s["kd"], s["q"], s["k"], s["v"], s["positions"], s["rope"] if c["rot"] else None, s["axis"], s["slots"], s["cache"], s["q_out"])
        L.gdn_kv4_read(s["kd"], s["slots"], s["cache"], s["k_out"], s["v_out"])
        return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["rot"]:
        cs = s["rope"][s["positions"].long()[s["axis_t"]].t(), torch.arange(c["rot"] // 2, device=q.device)]
        cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
        q, k = _rotate(q, cos, sin), _rotate(k, cos, sin)
    slots = s["slots"].long()
    live = slots >= 0
    page, off = torch.where(live, slots // c["page"], s["n"]), torch.where(live, slots % c["page"], 0)
    kc, vc, ke, ve = _parts(s["cache"], c["page"], c["d"])
    got = []
    for codes, entries, x in ((kc, ke, k), (vc, ve, v)):
        code, entry = _quantise(x)
        codes[page, :, off] = code
        entries[page, :, off] = entry
        got.append(torch.where(live[:, None, None], _values(codes[page, :, off], entries[page, :, off]), 0).to(torch.bfloat16))
    return dict(q=q.to(torch.bfloat16), k=got[0], v=got[1])


def _run_attend(s):
    c = s["case"]
    if own:
        from speculative_decode_gated_gdn_gb300 import lib as L
        L.gdn_kv4_attend(s["kd"], s["q"], s["cache"], s["table"], s["q_start"], s["q_count"], s["kv_len"], s["scale"], s["out"], s["ws"], max_q=c["T"])
        return s["out"]
    B, T, Hq, Hkv, d = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"]
    pages = s["cache"][s["table"].long().clamp(min=0)]  # [B][pages][Hkv][record]
    kc, vc, ke, ve = _parts(pages.flatten(0, 1), c["page"], d)
    K = s["table"].shape[1] * c["page"]
    key = torch.arange(K, device=pages.device)
    there = (key[None] < s["kv_len"].long()[:, None])[:, None, :, None]

    def rows(codes, entries):  # [B][Hkv][K][d], nothing of what lies behind a row's end
        x = _values(codes, entries).unflatten(0, (B, -1)).transpose(1, 2).flatten(2, 3)
        return torch.where(there, x, 0)

    q = s["q"].float().view(B, T, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B][Hkv][group * T][d]
    score = torch.matmul(q, rows(kc, ke).transpose(-1, -2)).mul_(s["scale"]).unflatten(2, (-1, T))
    i = torch.arange(T, device=q.device)
    place = (s["kv_len"] - s["q_count"]).long()[:, None] + i[None]
    seen = (key[None, None] <= place[..., None]) & (i[None, :, None] < s["q_count"].long()[:, None, None])
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top > -math.inf, top, 0)).exp_()
    den = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), rows(vc, ve)).unflatten(2, (-1, T)) / torch.where(den > 0, den, 1)
    return o.permute(0, 3, 1, 2, 4).reshape(B * T, Hq, d).to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    lens, add, active = _rows(c)
    add = add * active
    if c["op"] == "plan":  # two calls: the small arrays, the slots and positions, the pages that change hands
        moved = int((-(-(lens + add) // c["page"]) + lens // -c["page"]).sum())
        n = c["B"] * c["T"] if c["fixed"] else int(add.sum()) + 5
        return {"bytes": 2 * (4 * c["B"] * 7 + 8 * n) + 16 * moved + 4 * int(add.sum()), "flops": 8 * (c["B"] + n)}
    d, Hq, Hkv = c["d"], c["Hq"], c["Hkv"]
    entry = d // 2 + d // 64 * 4  # a token's bytes of one head, K or V
    if c["op"] == "append":
        N, live = c["B"] * c["T"], int(add.sum())
        turn = 4 * N * c["rot"] * (1 + c["axes"] / 32)
        return {"bytes": 2 * N * d * (2 * Hq + 2 * Hkv) + 2 * live * Hkv * entry + 4 * live * Hkv * d + turn + 4 * N * (c["axes"] + 2), "flops": 3 * N * c["rot"] * (Hq + Hkv) + 16 * N * Hkv * d}
    seen = sum(int(a) * int(n) - int(a) * (int(a) - 1) // 2 for n, a in zip(lens, add))  # pairs of a query and a key
    read = int((lens * (add > 0)).sum())
    return {"bytes": 2 * Hkv * entry * read + 4 * c["B"] * c["T"] * Hq * d + 4 * int((-(-lens // c["page"]) * (add > 0)).sum()), "flops": 4 * d * Hq * seen}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None  # whole numbers only
    s = prepare(c, seed)
    f64 = torch.float64
    if c["op"] == "append":
        half = c["rot"] // 2
        out = {}
        for name, x in (("q", s["q"]), ("k", s["k"]), ("v", s["v"])):
            y = x.to(f64)
            if half and name != "v":
                turn = torch.polar(torch.ones(s["N"], half, dtype=f64, device=y.device), s["positions"][s["axis_t"]].t().to(f64) * s["inv"])[:, None]
                z = torch.complex(y[..., :half], y[..., half:2 * half]) * turn
                y = torch.cat([z.real, z.imag, y[..., 2 * half:]], -1)
            if name != "q":
                y = _nearest(y)
                y[s["slots"] < 0] = 0
            out[name] = y
        return out
    T, G = c["T"], c["Hq"] // c["Hkv"]
    out = torch.zeros(c["B"] * T, c["Hq"], c["d"], dtype=f64, device=s["q"].device)
    half = c["page"] * c["d"] // 2
    for b in range(c["B"]):
        n, m = int(s["kv_len"][b]), int(s["q_count"][b])
        if not m or not n:
            continue
        rec = s["cache"][s["table"][b, : -(-n // c["page"])].long()]
        for h in range(c["Hkv"]):
            k, v = (_decode(rec[:, h], w, half, c)[:n] for w in (0, 1))
            at = torch.arange(n, device=k.device)[None] <= (n - m + torch.arange(m, device=k.device))[:, None]
            for g in range(h * G, (h + 1) * G):
                x = (s["q"][b * T: b * T + m, g].to(f64) @ k.t()) * c["d"] ** -0.5
                x = torch.softmax(x.masked_fill(~at, -math.inf), -1)
                out[b * T: b * T + m, g] = x @ v
    return out


def _decode(rec, which, half, c):
    """Keys (0) or values (1) of one head's records [pages][bytes], token by token in 64 bits."""
    d, w, P = c["d"], c["d"] // 64, c["page"]
    raw = rec[:, which * half:(which + 1) * half].reshape(-1, d // 2)
    lo, hi = raw.remainder(16), raw.div(16, rounding_mode="floor")
    code = torch.empty(raw.shape[0], d, dtype=torch.float64, device=raw.device)
    code[:, 0::2], code[:, 1::2] = lo.double(), hi.double()
    e = rec[:, 2 * half + which * P * w * 4: 2 * half + (which + 1) * P * w * 4].contiguous().view(torch.float16).reshape(-1, 1, w, 1, 2).double()
    return (code.view(-1, 8, w, 8) * e[..., 0] + e[..., 1]).reshape(-1, d)


def _nearest(y):
    """Each value of y [..., d] on its group's sixteen levels."""
    d = y.shape[-1]
    z = y.reshape(*y.shape[:-1], 8, d // 64, 8)
    lo, hi = (f(f(z, -1, keepdim=True), -3, keepdim=True) for f in (torch.amin, torch.amax))
    base, step = lo.to(torch.float16).double(), ((hi - lo) / 15).to(torch.float16).double()
    level = torch.where(step > 0, torch.round((z - base) / step.clamp(min=1e-30)), torch.zeros_like(z)).clamp(0, 15)
    return (base + step * level).reshape(y.shape)
