"""What sampled decoding of several continuations of a prompt costs next to the greedy cycle, operator by operator.

Greedy decoding takes the most likely token of every position.  Sampled decoding draws it, after the usual filters, and
several continuations of one prompt share the prompt's pages of the attention cache until they part.  The cases below
measure these operators:

  sample   gdn_sample: one token a row from its logits, with temperature, min-p, top-k and top-p of the row's own, from a
           given random number, and the logarithm of the probability that it was drawn with
  accept   gdn_accept_sampled: the same for every position of a verify, and the accepted prefix of the drafts
  fork     gdn_kv_fork + gdn_kv_copy_pages: rows that continue other rows' sequences: full pages are shared, the last,
           partly filled one is copied in every layer; then gdn_kv_plan_shared for the next tokens of all rows, and
           once more when the continuations end and give their pages back
  compact  gdn_kv_compact + gdn_kv_copy_pages: the pages in use move to the cache's front

The order in which sample and accept go: values descending, equal ones by index.  From a row's numbers above -infinity
(NaN never takes part) with weights w = exp((x - max) / temperature): those with w >= min_p, of these the first top_k, of
these the shortest beginning that has top_p of their mass, and of these the first whose running sum passes u times their
mass.  temperature 0: the first.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest call: one request, a small vocabulary, all filters on
        dict(name="sample one row", op="sample", B=1, V=32000, temp=0.8, top_k=40, top_p=0.95, min_p=0.02, mixed=False, pad=0, mask=0.0),
        # a vocabulary of no round size: rows that start at any address; a grammar forbids most tokens
        dict(name="sample odd vocabulary", op="sample", B=7, V=100003, temp=1.0, top_k=0, top_p=0.9, min_p=0.0, mixed=False, pad=0, mask=0.9),
        # a serving batch whose rows ask for different things, greedy ones among them, logits padded to a multiple of 128
        dict(name="sample mixed batch", op="sample", B=64, V=151936, temp=0.9, top_k=50, top_p=0.9, min_p=0.05, mixed=True, pad=128, mask=0.0),
        # the whole distribution, as for training data: nothing filtered
        dict(name="sample unfiltered batch", op="sample", B=256, V=151936, temp=1.0, top_k=0, top_p=1.0, min_p=0.0, mixed=False, pad=0, mask=0.0),
        # the benchmark's cohort: eight rows, one draft each, two of them idle
        dict(name="accept cohort", op="accept", B=8, T=2, V=151936, temp=0.7, top_k=20, top_p=0.8, min_p=0.0, mixed=False, pad=0, mask=0.0, idle=2),
        # a small vocabulary and ragged sizes
        dict(name="accept small ragged", op="accept", B=5, T=5, V=1003, temp=1.3, top_k=0, top_p=0.97, min_p=0.01, mixed=False, pad=0, mask=0.0, idle=1),
        # deep drafts of a large cohort
        dict(name="accept deep drafts", op="accept", B=64, T=8, V=151936, temp=0.6, top_k=0, top_p=0.95, min_p=0.0, mixed=False, pad=0, mask=0.0, idle=5),
        # eight continuations of the cohort's long prompt, ten attention layers
        dict(name="fork one prompt", op="fork", S=1, K=8, kv=13239, spread=0.0, Hkv=2, d=256, page=64, layers=10, T=2),
        # many prompts, two continuations each, small pages
        dict(name="fork small pages", op="fork", S=61, K=2, kv=6001, spread=0.9, Hkv=4, d=64, page=16, layers=8, T=5),
        # sixteen continuations of sixteen prompts at once
        dict(name="fork many", op="fork", S=16, K=16, kv=4011, spread=0.3, Hkv=8, d=128, page=64, layers=8, T=2),
        # the cohort with short contexts, after some requests have ended
        dict(name="compact cohort", op="compact", B=8, kv=500, Hkv=2, d=256, page=64, layers=10, full=0.7),
        # a ragged batch whose cache is half empty
        dict(name="compact ragged batch", op="compact", B=64, kv=8192, Hkv=8, d=128, page=32, layers=4, full=0.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "accept", "accept", "fork", "compact"])
    if op in ("sample", "accept"):
        c = dict(op=op, V=_log_int(rng, 300, 262144), temp=rng.choice([0.3, 0.7, 1.0, 1.0, 1.6]), top_k=rng.choice([0, 0, 1, _log_int(rng, 2, 1500)]),
                 top_p=rng.choice([1.0, 0.5, 0.9, 0.99]), min_p=rng.choice([0.0, 0.0, 0.01, 0.2]), mixed=rng.random() < 0.3, pad=rng.choice([0, 0, 8, 128]),
                 mask=rng.choice([0.0, 0.0, 0.5, 0.99]))
        if op == "sample":
            return c | dict(B=_log_int(rng, 1, min(512, 38_000_000 // c["V"])))
        T = rng.randint(1, 8)
        B = _log_int(rng, 1, min(128, 38_000_000 // (c["V"] * T)))
        return c | dict(B=B, T=T, idle=rng.randint(0, B // 4))
    c = dict(op=op, Hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64]), layers=rng.randint(1, 12))
    size = c["Hkv"] * c["page"] * c["d"] * 9 // 8 * c["layers"]  # bytes of a page in all layers
    if op == "fork":
        S = _log_int(rng, 1, 48)
        K = _log_int(rng, 1, max(1, 300 // S))
        kv = _log_int(rng, 1, max(c["page"], min(32768, 1_200_000_000 // size * c["page"] // S)))
        return c | dict(S=S, K=K, kv=kv, spread=rng.choice([0.0, 0.3, 0.9]), T=rng.randint(1, 8))
    B = _log_int(rng, 2, 96)
    return c | dict(B=B, kv=_log_int(rng, 20, max(c["page"], min(16384, 900_000_000 // size * c["page"] // B))), full=rng.choice([0.3, 0.5, 0.9]))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"sample": _prepare_draw, "accept": _prepare_draw, "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, seed, gen, "cuda")


def _prepare_draw(c, seed, gen, dev):
    B, T, V = c["B"], c.get("T", 1), c["V"]
    stride = -(-V // c["pad"]) * c["pad"] if c["pad"] else V
    R = B * T
    # what a language model's head gives: a broad bell, and a few candidates far above it in the rows that are sure
    x = torch.empty(R, stride, dtype=torch.bfloat16, device=dev)
    sure = torch.rand(R, 1, generator=gen, device=dev) * 9
    for a in range(0, R, 64):
        b = min(R, a + 64)
        y = torch.randn(b - a, V, generator=gen, device=dev).mul_(2.2)
        at = torch.randint(0, V, (b - a, 12), generator=gen, device=dev)
        y.scatter_(1, at, 6 + torch.rand(b - a, 12, generator=gen, device=dev) * sure[a:b])
        if c["mask"]:
            y.masked_fill_(torch.rand(b - a, V, generator=gen, device=dev) < c["mask"], -math.inf)
            y[:, 17] = 1.0  # something is always allowed
        x[a:b, :V] = y
    x[:, V:] = -math.inf
    logits = x[:, :V]
    # drafts: the most likely token for a while, then something else
    draft = torch.randint(0, V, (B, T), generator=gen, device=dev)
    if T > 1:
        best = logits.view(B, T, V).argmax(-1) if stride == V else logits.argmax(-1).view(B, T)
        good = torch.randint(0, T, (B, 1), generator=gen, device=dev)
        draft[:, 1:] = torch.where(torch.arange(T - 1, device=dev)[None] < good, best[:, :-1], draft[:, 1:])
    f32 = dict(dtype=torch.float32, device=dev)
    temp, top_p, min_p = (torch.full((B,), c[k], **f32) for k in ("temp", "top_p", "min_p"))
    top_k = torch.full((B,), c["top_k"], dtype=torch.int32, device=dev)
    if c["mixed"]:
        kind = torch.randint(0, 5, (B,), generator=gen, device=dev)  # greedy, all filters, one filter each
        temp = torch.where(kind == 0, 0.0, temp * (0.5 + torch.rand(B, generator=gen, device=dev)))
        top_k = torch.where((kind == 1) | (kind == 2), top_k, 0).to(torch.int32)
        top_p = torch.where((kind == 1) | (kind == 3), top_p, 1.0)
        min_p = torch.where((kind == 1) | (kind == 4), min_p, 0.0)
    active = torch.ones(B, dtype=torch.uint8, device=dev)
    if c.get("idle"):
        active[torch.randperm(B, generator=gen, device=dev)[: c["idle"]]] = 0
    s = dict(case=c, logits=logits, draft=draft.to(torch.int32), temp=temp, top_p=top_p, min_p=min_p, top_k=top_k, active=active, u=torch.rand(R, generator=gen, device=dev))
    s |= dict(token=torch.empty(R, dtype=torch.int32, device=dev), logp=torch.empty(R, **f32))
    if c["op"] == "accept":
        s |= dict(logits=torch.as_strided(x, (B, T, V), (T * stride, stride, 1)), u=s["u"].view(B, T), token=s["token"].view(B, T), logp=s["logp"].view(B, T),
                  keep=torch.empty(B, dtype=torch.int32, device=dev), next=torch.empty(B, dtype=torch.int32, device=dev))
        if own:
            from speculative_decode_gated_gdn_gb300 import lib as L
            s["ws"] = torch.zeros(L.gdn_accept_sampled_workspace_bytes(B, T, V), dtype=torch.uint8, device=dev)
    return s


def _page_bytes(c):
    return c["Hkv"] * 2 * c["page"] * (c["d"] // 2 + c["d"] // 64 * 4)


def _caches(c, n, gen, dev):
    """The layers' caches; copies do not look at what they copy."""
    return [torch.randint(0, 256, (n, _page_bytes(c)), generator=gen, device=dev, dtype=torch.uint8) for _ in range(c["layers"])]


def _dims(c, B, M, n):
    from speculative_decode_gated_gdn_gb300 import lib as L
    return L.kv4_dims(B, c["Hkv"], c["Hkv"], c["d"], c["page"], M, n)


def _fork_rows(c):
    """The prompts' lengths and the rows of prompts and continuations: what the case fixes, whatever the seed."""
    r = np.random.RandomState((c["S"] * 7919 + c["K"] * 104729 + c["kv"] * 31 + c["page"]) % (1 << 31))
    lens = r.randint(max(1, int(c["kv"] * (1 - c["spread"]))), c["kv"] + 1, c["S"]).astype(np.int64)
    lens[0] = c["kv"]
    rows = r.permutation(c["S"] * (1 + c["K"]))
    return lens, rows[: c["S"]], rows[c["S"]:]


def _prepare_fork(c, seed, gen, dev):
    lens_h, src_h, dst_h = _fork_rows(c)
    S, K, P = c["S"], c["K"], c["page"]
    B, M = S * (1 + K), -(-(c["kv"] + c["T"]) // P)
    held_h = -(-lens_h // P)
    whole = lens_h // P
    spare = K * int((held_h - whole).sum()) + (1 + K) * int((-(-(lens_h + c["T"]) // P) - held_h).sum()) + 5
    used = int(held_h.sum())
    n = used + spare
    order = torch.randperm(n, generator=gen, device=dev).to(torch.int32)
    i32 = dict(dtype=torch.int32, device=dev)
    src, dst, lens0, h = (torch.from_numpy(a.astype(np.int64)).to(dev) for a in (src_h, dst_h, lens_h, held_h))
    held, lens = torch.zeros(B, **i32), torch.zeros(B, **i32)
    held[src], lens[src] = h.to(torch.int32), lens0.to(torch.int32)
    table = torch.full((B, M), -1, **i32)
    col = torch.arange(M, device=dev)
    first = torch.cumsum(h, 0) - h
    table[src] = torch.where(col[None] < h[:, None], order[(first[:, None] + col[None]).clamp(max=n - 1)], -1)
    refs = torch.zeros(n, **i32)
    refs[order[:used].long()] = 1
    free = torch.cat([order[used:], torch.full((used,), -1, **i32)]).contiguous()
    pairs = torch.arange(S * K, device=dev) % S  # continuation i is of prompt i mod S
    lens_all = lens.clone()
    lens_all[dst] = lens0[pairs].to(torch.int32)
    N = B * c["T"]
    outs = [dict(q_start=torch.zeros(B + 1, **i32), q_count=torch.zeros(B, **i32), kv_len=torch.zeros(B, **i32), slots=torch.zeros(N, **i32), positions=torch.zeros(N, **i32)) for _ in range(2)]
    s = dict(case=c, B=B, M=M, n=n, N=N, held=held, table=table, free=free, free_count=torch.full((1,), spare, **i32), refs=refs, caches=_caches(c, n, gen, dev), outs=outs,
             src=src[pairs].to(torch.int32), dst=dst.to(torch.int32), at=lens0[pairs].to(torch.int32), lens=lens, lens_all=lens_all, add=torch.full((B,), c["T"], **i32),
             none=torch.zeros(B, **i32), active=torch.ones(B, dtype=torch.uint8, device=dev), copy_src=torch.zeros(S * K, **i32), copy_dst=torch.zeros(S * K, **i32))
    if own:
        s["kd"] = _dims(c, B, M, n)
    return s


def _compact_rows(c):
    r = np.random.RandomState((c["B"] * 7919 + c["kv"] * 31 + c["page"]) % (1 << 31))
    lens = r.randint(1, c["kv"] + 1, c["B"]).astype(np.int64)
    held = -(-lens // c["page"])
    share = np.zeros_like(held)  # every other row begins with pages of the row before it
    share[1::2] = np.minimum(held[1::2], held[0:2 * len(share[1::2]):2]) // 2
    return held, share


def _prepare_compact(c, seed, gen, dev):
    held_h, share_h = _compact_rows(c)
    B, M = c["B"], int(held_h.max()) + 1
    own_h = held_h - share_h
    U = int(own_h.sum())
    n = max(U + 1, int(U / c["full"]))
    order = torch.randperm(n, generator=gen, device=dev).to(torch.int32)
    held, share, mine = (torch.from_numpy(a).to(dev) for a in (held_h, share_h, own_h))
    col = torch.arange(M, device=dev)
    first = torch.cumsum(mine, 0) - mine
    place = first[:, None] + col[None] - share[:, None]
    before = torch.cat([place[:1], place[:-1]])  # a shared page stands where the row before has it
    place = torch.where(col[None] < share[:, None], before, place)
    table = torch.where(col[None] < held[:, None], order[place.clamp(0, n - 1)], -1).to(torch.int32).contiguous()
    refs = torch.zeros(n + 1, dtype=torch.int32, device=dev)
    refs.scatter_add_(0, torch.where(table < 0, n, table).long().flatten(), torch.ones(B * M, dtype=torch.int32, device=dev))
    refs = refs[:n].contiguous()
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(case=c, B=B, M=M, n=n, held=held.to(torch.int32), table=table, refs=refs, caches=_caches(c, n, gen, dev), new_table=torch.zeros(B, M, **i32), new_refs=torch.zeros(n, **i32),
             new_free=torch.zeros(n, **i32), new_count=torch.zeros(1, **i32), page_map=torch.zeros(n, **i32), copy_src=torch.full((n // 2 + 1,), -1, **i32), copy_dst=torch.full((n // 2 + 1,), -1, **i32),
             copies=torch.zeros(1, **i32))
    if own:
        s["kd"] = _dims(c, B, M, n)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"sample": _run_sample, "accept": _run_accept, "fork": _run_fork, "compact": _run_compact}[s["case"]["op"]](s)


def _run_sample(s):
    if own:
        from speculative_decode_gated_gdn_gb300 import lib as L
        L.gdn_sample(s["logits"], s["u"], s["token"], s["logp"], temperature=s["temp"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return dict(token=s["token"], logp=s["logp"])
    token, logp = _draw(s["logits"], s["temp"], s["top_k"], s["top_p"], s["min_p"], s["u"])
    return dict(token=token, logp=logp)


def _run_accept(s):
    if own:
        from speculative_decode_gated_gdn_gb300 import lib as L
        L.gdn_accept_sampled(s["logits"], s["draft"], s["active"], s["u"], s["keep"], s["next"], s["token"], s["logp"], s["ws"], temperature=s["temp"], top_k=s["top_k"], top_p=s["top_p"],
                             min_p=s["min_p"])
        return dict(token=s["token"], logp=s["logp"], keep=s["keep"], next=s["next"])
    B, T, V = s["logits"].shape
    each = lambda x: x.repeat_interleave(T)
    token, logp = _draw(s["logits"].reshape(B * T, V), each(s["temp"]), each(s["top_k"]), each(s["top_p"]), each(s["min_p"]), s["u"].reshape(-1))
    on = s["active"] > 0
    token, logp = token.view(B, T), logp.view(B, T)
    hit = torch.cumprod((s["draft"][:, 1:] == token[:, :-1]).to(torch.int32), 1).sum(1) if T > 1 else torch.zeros_like(s["draft"][:, 0])
    keep = torch.where(on, 1 + hit, 0)
    nxt = torch.where(on, token.gather(1, hit.long()[:, None])[:, 0], -1)
    return dict(token=torch.where(on[:, None], token, -1), logp=torch.where(on[:, None], logp, 0), keep=keep.to(torch.int32), next=nxt.to(torch.int32))


def _draw(x, temp, top_k, top_p, min_p, u):
    """A token of every row and its log-probability.  Sums and what is next to a border in 64 bits."""
    R, V = x.shape
    v, at = torch.sort(torch.nan_to_num(x.float(), nan=-math.inf, posinf=math.inf, neginf=-math.inf) + 0.0, dim=-1, descending=True, stable=True)
    greedy = (temp <= 0)[:, None]
    w = v.double()
    del v
    w -= w[:, :1].clone()
    w /= torch.where(greedy, 1.0, temp[:, None].double())
    w.exp_()
    rank = torch.arange(V, device=x.device)[None]
    k = torch.where(greedy, 1, torch.where(top_k[:, None] > 0, top_k[:, None], V))
    w *= (w >= min_p[:, None].double()) & (rank < k)
    run_ = torch.cumsum(w, -1)
    want = torch.where(top_p < 1, top_p.double().clamp(min=0) * run_[:, -1], math.inf)[:, None]
    stay = torch.ones_like(w, dtype=torch.bool)
    stay[:, 1:] = run_[:, :-1] < want
    w *= stay
    run_ = torch.cumsum(w, -1)
    del stay
    mass = run_[:, -1:]
    n = (w > 0).sum(-1, keepdim=True)
    r = u[:, None].double() * mass
    j = torch.minimum((run_ <= r).sum(-1, keepdim=True), n - 1)
    mine = w.gather(1, j)
    return at.gather(1, j)[:, 0].to(torch.int32), -torch.log1p((mass - mine) / mine)[:, 0].float()


def _run_fork(s):
    c = s["case"]
    a, b = s["outs"]
    if own:
        from speculative_decode_gated_gdn_gb300 import lib as L
        L.gdn_kv_fork(s["kd"], s["src"], s["dst"], s["at"], s["held"], s["table"], s["free"], s["free_count"], s["refs"], s["copy_src"], s["copy_dst"])
        L.gdn_kv_copy_pages(s["kd"], s["caches"], s["copy_src"], s["copy_dst"])
        for o, lens, add in ((a, s["lens_all"], s["add"]), (b, s["lens"], s["none"])):
            L.gdn_kv_plan_shared(s["kd"], lens, add, s["active"], s["held"], s["table"], s["free"], s["free_count"], s["refs"], o["q_start"], o["q_count"], o["kv_len"], o["slots"],
                                 o["positions"], T=c["T"])
        plans = dict(cycle=a, end=b)
    else:
        s["copy_src"], s["copy_dst"] = _fork(s)
        _copy_pages(s)
        plans = dict(cycle=_plan(s, s["lens_all"], s["add"]), end=_plan(s, s["lens"], s["none"]))
    return dict(plans, held=s["held"], table=s["table"], free=s["free"], free_count=s["free_count"], refs=s["refs"], copy_src=s["copy_src"], copy_dst=s["copy_dst"], caches=s["caches"])


def _fork(s):
    """Pages of the first at[i] tokens of row src[i] for the empty row dst[i]: full ones shared, the rest's taken from the stack's end."""
    P, dev = s["case"]["page"], s["table"].device
    src, dst, at = s["src"].long(), s["dst"].long(), s["at"].long()
    whole, rest = at // P, (at % P > 0).long()
    col = torch.arange(s["M"], device=dev)[None]
    mine = s["table"][src]
    shared = col < whole[:, None]
    s["refs"].scatter_add_(0, mine.clamp(min=0).long().flatten(), shared.flatten().to(torch.int32))
    new = s["free"][(s["free_count"].long() - 1 - (torch.cumsum(rest, 0) - rest)).clamp(min=0)]
    s["refs"].scatter_add_(0, new.clamp(min=0).long(), rest.to(torch.int32))
    copied = (col == whole[:, None]) & (rest[:, None] > 0)
    s["table"][dst] = torch.where(shared, mine, torch.where(copied, new[:, None], -1)).to(torch.int32)
    s["held"][dst] = (whole + rest).to(torch.int32)
    s["free_count"] -= rest.sum().to(torch.int32)
    last = mine.gather(1, whole.clamp(max=s["M"] - 1)[:, None])[:, 0]
    return torch.where(rest > 0, last, -1).to(torch.int32), torch.where(rest > 0, new, -1).to(torch.int32)


def _copy_pages(s):
    a, b = s["copy_src"].long(), s["copy_dst"].long()
    live = a >= 0
    a, b = a[live], b[live]
    for x in s["caches"]:
        x[b] = x[a]


def _plan(s, lens, add):
    """Rows that hold more pages than they need give them back, then rows that hold fewer take some.  A page goes onto the
    free list when its last holder gives it back, at that holder's place."""
    c, dev, N, n, M, P = s["case"], lens.device, s["N"], s["n"], s["M"], s["case"]["page"]
    lens, held, a = lens.long(), s["held"].long(), add.long()
    want = (lens + a + P - 1) // P
    count = s["free_count"].long()
    col = torch.arange(M, device=dev)[None]
    back = ((col >= want[:, None]) & (col < held[:, None])).flatten()
    page = torch.where(back, s["table"].flatten().long(), n)
    given = torch.zeros(n + 1, dtype=torch.int32, device=dev).scatter_add_(0, page, torch.ones_like(page, dtype=torch.int32))[:n]
    refs = s["refs"] - given
    i = torch.arange(page.numel(), device=dev)
    last = torch.full((n + 1,), -1, dtype=torch.int64, device=dev).scatter_reduce_(0, page, i, "amax")
    gone = torch.cat([(refs == 0) & (given > 0), torch.zeros(1, dtype=torch.bool, device=dev)])
    push = back & gone[page] & (last[page] == i)
    place = count + torch.cumsum(push.long(), 0) - 1
    free = torch.cat([s["free"], s["free"][:1]]).scatter_(0, torch.where(push, place, n), s["table"].flatten())[:n]
    table = torch.where(back.view(-1, M), -1, s["table"])
    avail = count + push.sum()
    need = (want - held).clamp(min=0)
    ends = torch.cumsum(need, 0)
    fits = ends <= avail
    a, need = torch.where(fits, a, 0), torch.where(fits, need, 0)
    new = (col >= held[:, None]) & (col < (held + need)[:, None])
    take = free[(avail - 1 - ((ends - need)[:, None] + col - held[:, None])).clamp(0, n - 1)]
    table = torch.where(new, take, table)
    refs.scatter_add_(0, torch.where(new, take, 0).long().flatten(), new.flatten().to(torch.int32))
    s["free"].copy_(free)
    s["table"].copy_(table)
    s["refs"].copy_(refs)
    s["held"].copy_((torch.minimum(held, want) + need).to(torch.int32))
    s["free_count"].copy_((avail - need.sum()).to(torch.int32))
    t = torch.arange(N, device=dev)
    row, k = t // c["T"], t % c["T"]
    live = k < a[row]
    pos = lens[row] + k
    at = table[row, (pos // P).clamp(0, M - 1)].long()
    return dict(q_start=(torch.arange(s["B"] + 1, device=dev) * c["T"]).to(torch.int32), q_count=a.to(torch.int32), kv_len=(lens + a).to(torch.int32),
                slots=torch.where(live, at * P + pos % P, -1).to(torch.int32), positions=torch.where(live, pos, -1).to(torch.int32))


def _run_compact(s):
    if own:
        from speculative_decode_gated_gdn_gb300 import lib as L
        L.gdn_kv_compact(s["kd"], s["held"], s["table"], s["refs"], s["new_table"], s["new_refs"], s["new_free"], s["new_count"], s["page_map"], s["copy_src"], s["copy_dst"], s["copies"])
        L.gdn_kv_copy_pages(s["kd"], s["caches"], s["copy_src"], s["copy_dst"], count=s["copies"])
    else:
        _compact(s)
        _copy_pages(s)
    return {k: s[k] for k in ("new_table", "new_refs", "new_free", "new_count", "page_map", "copy_src", "copy_dst", "copies", "caches")}


def _compact(s):
    """The i-th page in use behind the first U places moves to the i-th free one among them."""
    n, dev = s["n"], s["table"].device
    used = s["refs"] > 0
    U = used.sum()
    at = torch.arange(n, device=dev)
    src, dst = used & (at >= U), ~used & (at < U)
    a, b = torch.cumsum(src.long(), 0) - 1, torch.cumsum(dst.long(), 0) - 1
    size = s["copy_src"].numel()
    for out, mask, place in ((s["copy_src"], src, a), (s["copy_dst"], dst, b)):
        out.copy_(torch.cat([out, out[:1]]).scatter_(0, torch.where(mask, place, size), at.to(torch.int32))[:size])
    to = torch.where(src, s["copy_dst"][a.clamp(0, size - 1)].long(), at)
    s["page_map"].copy_(torch.where(used, to, -1).to(torch.int32))
    s["new_refs"].copy_(torch.zeros(n + 1, dtype=torch.int32, device=dev).scatter_(0, torch.where(used, to, n), s["refs"])[:n])
    col = torch.arange(s["M"], device=dev)[None]
    s["new_table"].copy_(torch.where(col < s["held"][:, None], s["page_map"][s["table"].clamp(min=0).long()], s["table"]))
    s["new_free"].copy_(torch.where(at < n - U, n - 1 - at, -1).to(torch.int32))
    s["new_count"].copy_((n - U).to(torch.int32))
    s["copies"].copy_(src.sum().to(torch.int32))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] in ("sample", "accept"):  # every logit read once
        R = c["B"] * c.get("T", 1)
        live = R - c.get("idle", 0) * c.get("T", 1)
        return {"bytes": 2 * live * c["V"] + 16 * c["B"] + 12 * R, "flops": 4 * live * c["V"]}
    if c["op"] == "fork":
        lens, _, _ = _fork_rows(c)
        P, forks = c["page"], c["S"] * c["K"]
        shared, tails = int((lens // P).sum()) * c["K"], int((lens % P > 0).sum()) * c["K"]
        B = c["S"] * (1 + c["K"])
        # a shared page: its cell read and written, its count read and written, when it is taken and when it is given back
        return {"bytes": 2 * tails * _page_bytes(c) * c["layers"] + 32 * shared + 48 * tails + 20 * forks + 2 * B * (7 * 4 + 8 * c["T"]), "flops": 4 * shared}
    held, share = _compact_rows(c)
    U = int((held - share).sum())
    n = max(U + 1, int(U / c["full"]))
    moved = U - U * U // n  # of pages scattered evenly
    return {"bytes": 2 * moved * _page_bytes(c) * c["layers"] + 8 * int(held.sum()) + 16 * n + 8 * moved, "flops": 4 * n}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    c = case
    if c["op"] not in ("sample", "accept"):
        return None  # whole numbers and copied bytes only
    s = prepare(c, seed)
    T = c.get("T", 1)
    x, u = s["logits"].reshape(-1, c["V"]), s["u"].reshape(-1).tolist()
    host = {k: s[k].tolist() for k in ("temp", "top_k", "top_p", "min_p", "active")}
    logp = []
    for i in range(x.shape[0]):
        p = {k: v[i // T] for k, v in host.items()}
        logp.append(_log_probability(x[i], p, u[i]) if p["active"] else 0.0)
    logp = torch.tensor(logp, dtype=torch.float64, device=x.device)
    if c["op"] == "sample":
        return dict(token=None, logp=logp)
    return dict(token=None, logp=logp.view(c["B"], T), keep=None, next=None)


def _log_probability(x, p, u):
    """Of the token that u draws: over the distinct values of a row, each with how many tokens have it."""
    if p["temp"] <= 0:
        return 0.0
    v, n = torch.unique(x.double(), return_counts=True)
    v, n = v.flip(0).cpu().numpy(), n.flip(0).cpu().numpy().astype(np.float64)
    w = np.exp((v - v[0]) / p["temp"])
    keep = (w >= p["min_p"]) & (w > 0)
    w, n = w[keep], n[keep]
    if p["top_k"] > 0:
        n = np.clip(p["top_k"] - (np.cumsum(n) - n), 0, n)
    if p["top_p"] < 1:
        mass = np.cumsum(n * w)
        lack = max(p["top_p"], 0.0) * mass[-1] - (mass - n * w)
        n = np.clip(np.ceil(lack / w), 0, n)
        n[0] = max(n[0], 1.0)
    mass = np.cumsum(n * w)
    j = min(int(np.searchsorted(mass, u * mass[-1], side="right")), int(np.flatnonzero(n)[-1]))
    return float(np.log(w[j] / mass[-1]))
