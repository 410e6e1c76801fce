"""GPU parity of the paged 4-bit cache's operators (plan, append, read, attend)
against plain references: integers, codes and entries bit for bit, attention
within what its 16-bit operands and one bf16 rounding allow."""
import numpy as np
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests import kv4_ref as R

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda().contiguous()


# ------------------------------------------------------------------ plan
def run_plan(page, max_pages, n_pages, T, N, st, lens, add, active):
    B = len(lens)
    kd = L.kv4_dims(B, 1, 1, 64, page, max_pages, n_pages)
    t = dict(held=dev(st["held"]), table=dev(st["table"]), free=dev(st["free"]), count=dev([st["count"]]))
    o = dict(q_start=dev([-7] * (B + 1)), q_count=dev([-7] * B), kv_len=dev([-7] * B), slots=dev([-7] * N), positions=dev([-7] * N))
    L.gdn_kv_plan(kd, dev(lens), dev(add), dev(active, torch.uint8), t["held"], t["table"], t["free"], t["count"],
                  o["q_start"], o["q_count"], o["kv_len"], o["slots"], o["positions"], T=T)
    status = L.gdn_get_status(clear=True)
    got = {k: v.cpu().numpy().tolist() for k, v in {**t, **o}.items()}
    got["count"] = got["count"][0]
    got["status"] = status
    return got


def fresh(B, max_pages, n_pages, seed=0):
    order = np.random.default_rng(seed).permutation(n_pages).tolist()
    return dict(held=[0] * B, table=[[-1] * max_pages for _ in range(B)], free=order, count=n_pages)


def check_plan(page, max_pages, n_pages, T, N, st, lens, add, active):
    want = R.plan(page, max_pages, n_pages, T, N, lens, add, active, st["held"], st["table"], st["free"], st["count"])
    got = run_plan(page, max_pages, n_pages, T, N, st, lens, add, active)
    for k in ("q_start", "q_count", "kv_len", "slots", "positions", "held", "table", "count", "free", "status"):
        assert got[k] == want[k], k
    return want


@pytest.mark.parametrize("B,T,page", [(1, 1, 16), (8, 2, 64), (37, 5, 16), (1024, 3, 32), (1500, 0, 16), (2049, 8, 64)])
def test_plan_cycles(gdn, B, T, page):
    """Growing, rejecting, finishing and joining rows over five cycles."""
    rng = np.random.default_rng(B + T)
    max_pages, n_pages = 24, max(8, B * 9)
    st = fresh(B, max_pages, n_pages)
    lens = np.zeros(B, np.int64)
    for c in range(5):
        add = rng.integers(0, (T if T else 40) + 1, B)
        if c == 0 and not T:
            add = rng.integers(0, 200, B)
        active = (rng.random(B) > 0.2).astype(np.uint8)
        N = B * T if T else int((add * active).sum()) + 3
        st = check_plan(page, max_pages, n_pages, T, max(N, 1), st, lens, add, active)
        lens = lens + np.minimum(rng.integers(0, 9, B), st["q_count"])
        done = rng.random(B) < 0.1
        lens[done] = 0


def test_plan_runs_out_in_row_order(gdn):
    page, M = 16, 8
    st = fresh(6, M, 5)
    # rows need 1, 2, 0 (inactive), 2, 1, 0 pages of 5, then one more than is left
    st = check_plan(page, M, 5, 0, 200, st, [0] * 6, [16, 17, 9, 32, 1, 0], [1, 1, 0, 1, 1, 1])
    assert st["status"] == 8 and st["q_count"] == [16, 17, 0, 32, 0, 0]
    # row 1 finishes: its pages serve row 4 in the same call
    st = check_plan(page, M, 5, 0, 200, st, [16, 0, 0, 32, 0, 0], [0, 0, 0, 0, 20, 0], [1] * 6)
    assert st["status"] == 0 and st["q_count"][4] == 20 and st["held"][1] == 0


def test_plan_refusals(gdn):
    """No place among N, too many pages, negative lengths, more than T: the row keeps what it holds."""
    st = fresh(4, 4, 64)
    st = check_plan(16, 4, 64, 0, 10, st, [0, 0, 0, 0], [4, 4, 4, 1], [1] * 4)
    assert st["q_count"] == [4, 4, 0, 0] and st["status"] == 8
    st = check_plan(16, 4, 64, 0, 100, st, [4, -1, 60, 0], [1, 1, 5, -3], [1] * 4)
    assert st["status"] == 32 and st["q_count"] == [1, 0, 0, 0]
    st = check_plan(16, 4, 64, 2, 8, st, [5, 4, 0, 0], [2, 3, 2, 1], [1] * 4)
    assert st["status"] == 32 and st["q_count"] == [2, 0, 2, 1]


def test_plan_many_tokens(gdn):
    """More tokens than one CTA writes: prompts of thousands of tokens, odd lengths, tokens left over."""
    lens, add = [0, 5, 1000, 0, 77], [20001, 0, 8191, 1, 3000]
    st = fresh(5, 2000, 3000)
    st = check_plan(16, 2000, 3000, 0, sum(add) + 100, st, [0] * 5, lens, [1] * 5)
    check_plan(16, 2000, 3000, 0, sum(add) + 100, st, lens, add, [1] * 5)


# ------------------------------------------------------------------ append and read
APPEND = [  # N, H_q, H_kv, d, rot, axes, page, pairs
    (1, 1, 1, 64, 64, 1, 16, False),
    (16, 16, 2, 256, 64, 3, 64, False),
    (37, 8, 8, 128, 128, 3, 32, False),
    (5, 3, 1, 128, 32, 2, 16, True),
    (301, 5, 1, 256, 256, 4, 16, True),
    (64, 10, 2, 64, 0, 1, 64, False),
    (33, 7, 7, 64, 16, 1, 32, False),
]


def append_case(N, Hq, Hkv, d, rot, axes, page, pairs, seed=0, top=5000):
    rng = np.random.default_rng(seed)
    x = R.bf16(rng.normal(size=(N, Hq + 2 * Hkv, d)) * rng.choice([0.01, 1.0, 30.0], size=(N, Hq + 2 * Hkv, 1)))
    pos = rng.integers(0, top, (axes, N)).astype(np.int32)
    axis = bytes(int(a) for a in rng.integers(0, axes, rot // 2))
    n_pages = N // page + 5
    slots = rng.permutation(n_pages * page)[:N].astype(np.int32)
    return x, pos, axis, n_pages, slots


def run_append(x, pos, axis, n_pages, slots, Hq, Hkv, d, rot, page, pairs, cache, top=5000, table=None):
    N = x.shape[0]
    kd = L.kv4_dims(1, Hq, Hkv, d, page, 1, n_pages)
    xd = x.cuda()
    pages = torch.from_numpy(cache.bytes.copy()).cuda()
    q_out = torch.full((N, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    rope = (R.rope_table(top, rot) if table is None else table).cuda() if rot else None
    L.gdn_kv4_append(kd, xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], dev(pos), rope, axis, dev(slots), pages, q_out,
                     style=L.GDN_ROPE_PAIRS if pairs else L.GDN_ROPE_HALF)
    k = torch.full((N, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full((N, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    L.gdn_kv4_read(kd, dev(slots), pages, k, v)
    status = L.gdn_get_status(clear=True)
    return q_out.cpu(), pages.cpu().numpy(), k.cpu(), v.cpu(), status


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "N{}q{}kv{}d{}r{}a{}p{}{}".format(*c[:7], "x" if c[7] else ""))
def test_append_and_read(gdn, case):
    N, Hq, Hkv, d, rot, axes, page, pairs = case
    x, pos, axis, n_pages, slots = append_case(*case)
    slots[::7] = -1  # tokens that are rotated but not cached
    cache = R.Cache(n_pages, Hkv, page, d, seed=1)
    q_out, pages, k, v, status = run_append(x, pos, axis, n_pages, slots, Hq, Hkv, d, rot, page, pairs, cache)
    assert status == 0
    xf = x.float().numpy()
    q, kk, vv = xf[:, :Hq], xf[:, Hq:Hq + Hkv], xf[:, Hq + Hkv:]
    if rot:
        tab = R.rope_table(5000, rot).numpy()
        cs = np.stack([tab[pos[axis[i]], i] for i in range(rot // 2)], 1)
        q, kk = R.rotate(q, cs, rot, pairs), R.rotate(kk, cs, rot, pairs)
    assert torch.equal(bits(q_out), bits(R.bf16(q)))
    for n in range(N):
        if slots[n] >= 0:
            cache.write(int(slots[n]), kk[n], vv[n])
    assert np.array_equal(pages, cache.bytes), "codes, entries, and every place that was not written"
    rk, rv = cache.read(slots)
    assert torch.equal(bits(k), bits(R.bf16(rk))) and torch.equal(bits(v), bits(R.bf16(rv)))
    # what the cache stands for is within half a step of the value, and what
    # fp16 leaves of the base and of the largest code
    live = slots >= 0
    kc, vc, ke, ve = cache.views()
    for got, y, e in ((rk, kk, ke), (rv, vv, ve)):
        step = e[slots[live] // page, :, slots[live] % page, :, 0].astype(np.float64)
        g = (np.arange(d) // 8) % (d // 64)
        bound = step[..., g] * (0.5 + 15 * 2.0 ** -11) + 2.0 ** -11 * np.abs(y[live]).max(-1, keepdims=True) + 2.0 ** -24
        assert (np.abs(got[live] - y[live]) <= bound * 1.001).all()


def test_append_borders(gdn):
    """Equal values, zeros, subnormal steps, magnitudes over fp16, infinities and NaN."""
    Hq, Hkv, d, page = 1, 1, 64, 16
    x = torch.zeros(10, 3, d)
    x[1, 1:] = 3.140625
    x[2, 1:, :8] = 1e-6
    x[3, 1:, 0] = 3e38
    x[4, 1:, 0], x[4, 1:, 9] = 3e38, -3e38
    x[5, 1:, 63] = float("inf")
    x[6, 1:, 5] = float("nan")
    x[7, 1:, 5] = -70000.0
    x[8, 1:] = torch.arange(64.0) / 15
    x[9, 1:] = torch.arange(64.0) % 16 + 0.5
    x = x.to(torch.bfloat16)
    slots = np.arange(10, dtype=np.int32)
    cache = R.Cache(2, Hkv, page, d)
    q_out, pages, k, v, status = run_append(x, np.zeros((1, 10), np.int32), b"", 2, slots, Hq, Hkv, d, 0, page, False, cache)
    xf = x.float().numpy()
    for n in range(10):
        cache.write(n, xf[n, 1:2], xf[n, 2:3])
    kc, vc, ke, ve = cache.views()
    gk, gv, hke, hve = cache.views(pages)
    assert np.array_equal(gk, kc) and np.array_equal(gv, vc)
    assert np.array_equal(hke, ke, equal_nan=True) and np.array_equal(hve, ve, equal_nan=True)
    assert torch.isnan(k[5]).all() and torch.isnan(v[6]).all() and torch.isfinite(k[4].float()).all()
    assert status == 0


def test_append_out_of_bounds_is_skipped(gdn):
    """A slot or position outside the cache: status, and no byte of the cache changes for that token."""
    N, Hq, Hkv, d, rot, axes, page, pairs = 6, 2, 2, 128, 32, 2, 16, False
    x, pos, axis, n_pages, slots = append_case(N, Hq, Hkv, d, rot, axes, page, pairs)
    axis = bytes([0, 1] * 8)
    slots[1] = n_pages * page
    pos[1, 3] = 5000
    pos[0, 4] = -1
    slots[5] = -1
    pos[:, 5] = -1
    cache = R.Cache(n_pages, Hkv, page, d, seed=1)
    q_out, pages, k, v, status = run_append(x, pos, axis, n_pages, slots, Hq, Hkv, d, rot, page, pairs, cache)
    assert status == L.GDN_STATUS_BAD_INDEX
    xf = x.float().numpy()
    tab = R.rope_table(5000, rot).numpy()
    cs = np.stack([tab[np.clip(pos[axis[i]], 0, 4999), i] for i in range(rot // 2)], 1)
    kk = R.rotate(xf[:, Hq:Hq + Hkv], cs, rot, pairs)
    for n in (0, 2):
        cache.write(int(slots[n]), kk[n], xf[n, Hq + Hkv:])
    assert np.array_equal(pages, cache.bytes)
    assert torch.equal(bits(q_out[5]), bits(x[5, :Hq])), "a token without a position does not turn"
    assert (k[1] == 0).all() and (v[5] == 0).all()


def test_far_positions(gdn):
    """A million tokens into a context the angle is the table's, to the last bit."""
    N, Hq, Hkv, d, rot, page = 3, 1, 1, 64, 64, 16
    x, _, _, n_pages, slots = append_case(N, Hq, Hkv, d, rot, 1, page, False)
    inv = 1e6 ** (-torch.arange(32, dtype=torch.float64) / 32)
    far = 999_990
    ang = (far + torch.arange(10, dtype=torch.float64))[:, None] * inv[None]
    table = torch.zeros(far + 10, 32, 2)
    table[far:] = torch.stack([ang.cos(), ang.sin()], -1).float()
    pos = np.array([[far, far + 4, far + 9]], np.int32)
    cache = R.Cache(n_pages, Hkv, page, d)
    q_out, *_, status = run_append(x, pos, bytes(32), n_pages, slots, Hq, Hkv, d, rot, page, False, cache, table=table)
    q = R.rotate(x.float().numpy()[:, :1], table.numpy()[pos[0]], rot, False)
    assert status == 0 and torch.equal(bits(q_out), bits(R.bf16(q)))


# ------------------------------------------------------------------ attend
def attend_case(Hq, Hkv, d, page, rows, pad=0, seed=0, gain=1.0, spare=2):
    """rows: (kv_len, count, span) of each; scattered pages, NaN entries wherever no row has a token."""
    rng = np.random.default_rng(seed)
    B = len(rows)
    held = [-(-n // page) for n, _, _ in rows]
    n_pages = sum(held) + spare
    order = rng.permutation(n_pages).tolist()
    width = max(1, max(held)) + 1
    table = np.full((B, width), -1, np.int64)
    cache = R.Cache(n_pages, Hkv, page, d, seed)
    far = rng.normal(size=(Hkv, d)) * (rng.random((Hkv, d)) < 0.1) * 5
    for b, (n, _, _) in enumerate(rows):
        table[b, :held[b]] = [order.pop() for _ in range(held[b])]
        k = (rng.normal(size=(n, Hkv, d)) + far).astype(np.float32)
        v = rng.normal(size=(n, Hkv, d)).astype(np.float32)
        kc, ke = R.pack(k)
        vc, ve = R.pack(v)
        for t in range(n):
            pg, off = table[b, t // page], t % page
            for i, (c, e) in enumerate(((kc[t], ke[t]), (vc[t], ve[t]))):
                cache.bytes[pg, :, i * cache.a + off * d // 2: i * cache.a + (off + 1) * d // 2] = c
                at = 2 * cache.a + i * cache.e + off * (d // 64) * 4
                cache.bytes[pg, :, at: at + d // 64 * 4] = e.reshape(Hkv, -1).view(np.uint8)
    q_start = np.concatenate([[pad], pad + np.cumsum([s for _, _, s in rows])]).tolist()
    N = q_start[-1] + pad
    q = R.bf16(rng.normal(size=(N, Hq, d)) * gain * rng.choice([0.05, 1.0, 3.0], size=(N, Hq, 1)))
    return cache, table, q_start, [c for _, c, _ in rows], [n for n, _, _ in rows], q


def run_attend(cache, table, q_start, q_count, kv_len, q, scale, max_q, ws=None, stream=None):
    N, Hq, d = q.shape
    kd = L.kv4_dims(len(q_count), Hq, cache.H, d, cache.P, table.shape[1], cache.n)
    out = torch.full((N, Hq, d), 77.0, dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = torch.zeros(L.gdn_kv4_attend_workspace_bytes(kd, N, max_q), dtype=torch.uint8, device="cuda")
    args = (q.cuda(), torch.from_numpy(cache.bytes).cuda(), dev(table), dev(q_start), dev(q_count), dev(kv_len))
    L.gdn_kv4_attend(kd, *args, scale, out, ws, max_q, stream=stream)
    return out, ws, kd, args


def check_attend(Hq, Hkv, d, page, rows, pad=0, seed=0, gain=1.0):
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, page, rows, pad, seed, gain)
    scale = d ** -0.5
    out, *_ = run_attend(cache, table, q_start, q_count, kv_len, q, scale, max(s for _, _, s in rows))
    status = L.gdn_get_status(clear=True)
    assert status == 0
    want, tol = R.attend(q.double().numpy(), cache, table, q_start, q_count, kv_len, scale)
    got = out.cpu().double().numpy()
    outside = np.isnan(want)
    assert (got[outside] == 77.0).all(), "tokens in no span are not written"
    err = np.abs(got - want)[~outside]
    assert np.isfinite(got).all()
    worst = (err / tol[~outside]).max() if err.size else 0
    assert worst <= 1, f"error {worst:.2f} of what the roundings allow"
    return worst


HEADS = [(1, 1, 64), (8, 8, 64), (10, 2, 64), (8, 2, 128), (5, 1, 128), (32, 4, 128), (16, 2, 256), (2, 2, 256), (8, 1, 256)]


@pytest.mark.parametrize("Hq,Hkv,d", HEADS, ids=lambda v: str(v))
@pytest.mark.parametrize("page", [16, 32, 64])
def test_attend_lengths(gdn, Hq, Hkv, d, page):
    """One and two new tokens over lengths around the edges of pages and tiles; a row without keys, one without queries."""
    rows = [(1, 1, 2), (2, 2, 2), (page - 1, 1, 1), (page, 2, 2), (page + 1, 1, 2), (0, 0, 2), (63, 2, 2), (65, 1, 1),
            (40, 0, 2), (129, 2, 2), (300, 1, 1)]
    check_attend(Hq, Hkv, d, page, rows, pad=1, seed=page + Hq)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 1, 128), (4, 4, 64), (10, 2, 256)], ids=lambda v: str(v))
def test_attend_queries(gdn, T, Hq, Hkv, d):
    """Every number of queries a row: tiles of queries that end inside a token's group of heads."""
    check_attend(Hq, Hkv, d, 16, [(T, T, T), (T + 70, T, T), (200, max(T - 1, 1), T)], seed=T)


def test_attend_queries_before_the_first_key(gdn):
    """A row with more queries than cached tokens: its first ones see nothing and get zeros."""
    for Hq, Hkv, d in ((4, 2, 64), (16, 2, 128), (16, 2, 256)):
        check_attend(Hq, Hkv, d, 16, [(3, 5, 5), (0, 4, 4), (1, 40, 40)], seed=5)


@pytest.mark.parametrize("Hq,Hkv,d,T,n", [(16, 2, 256, 150, 150), (8, 2, 128, 131, 400), (4, 4, 64, 300, 333), (5, 1, 128, 77, 1000)])
def test_attend_prompts(gdn, Hq, Hkv, d, T, n):
    check_attend(Hq, Hkv, d, 32, [(n, T, T), (T // 2, T // 2, T // 2)], seed=T)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 1, 128), (4, 2, 64), (16, 2, 256)], ids=lambda v: str(v))
def test_attend_long_rows(gdn, Hq, Hkv, d):
    """Few rows and a long axis, next to short ones: the work is split over the keys and joined."""
    check_attend(Hq, Hkv, d, 64, [(9000, 1, 1), (5, 1, 1), (4099, 1, 1)], seed=2)


@pytest.mark.parametrize("Hq,Hkv,d,T,n", [(8, 1, 256, 3, 12000), (8, 1, 128, 6, 20000), (8, 1, 64, 10, 20000), (8, 1, 128, 16, 20000),
                                          (1, 1, 64, 1, 20000), (8, 1, 128, 1, 20000), (4, 1, 256, 2, 12000), (8, 2, 128, 3, 9000)])
def test_attend_row_cut_among_many_ctas(gdn, Hq, Hkv, d, T, n):
    """A line long enough that one unit's parts are joined in more than one step, of one to four blocks of query rows; a
    short row on either side."""
    check_attend(Hq, Hkv, d, 32, [(40, T, T), (n, T, T), (7, 1, T)], seed=T)


def test_attend_sharp_and_flat(gdn):
    """Scores far apart (one key takes all) and all equal (gain 0)."""
    for gain in (0.0, 12.0):
        check_attend(8, 2, 128, 16, [(500, 2, 2), (77, 1, 2)], seed=3, gain=gain)
        check_attend(4, 2, 64, 16, [(300, 40, 40)], seed=4, gain=gain)


def test_attend_scales_of_values(gdn):
    """Values of 1e-4 next to values of 1e4, in one row's keys and across groups of channels."""
    for Hq, Hkv, d, T in ((8, 2, 128, 2), (16, 2, 256, 2), (4, 2, 64, 50), (16, 2, 256, 20)):
        cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 16, [(400, T, T)], seed=9)
        rng = np.random.default_rng(1)
        data = cache.bytes
        ent = data[..., 2 * cache.a + cache.e:].copy().view(np.float16)
        f = (10.0 ** rng.integers(-4, 4, ent.shape[:-1] + (ent.shape[-1] // 2, 1))).astype(np.float16)
        ent = (ent.reshape(*ent.shape[:-1], -1, 2).astype(np.float32) * f).astype(np.float16).reshape(ent.shape)
        data[..., 2 * cache.a + cache.e:] = ent.view(np.uint8)
        out, *_ = run_attend(cache, table, q_start, q_count, kv_len, q, d ** -0.5, T)
        want, tol = R.attend(q.double().numpy(), cache, table, q_start, q_count, kv_len, d ** -0.5)
        # values under fp16's normal range keep 2^-25 of absolute precision
        assert (np.abs(out.cpu().double().numpy() - want) <= tol + 2.0 ** -24).all()


def test_attend_nan_key_stays_with_its_queries(gdn):
    """A NaN key or value poisons the queries that see it and no other."""
    for Hq, Hkv, d, T in ((8, 2, 128, 2), (16, 2, 256, 3), (4, 2, 64, 70)):
        cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 16, [(100, T, T), (100, T, T)], seed=6)
        for which in (0, 1):
            data = cache.bytes.copy()
            t = 100 - 1  # the newest token of row 0: seen by its last query only
            at = 2 * cache.a + which * cache.e + (t % 16) * (d // 64) * 4
            data[table[0, t // 16], :, at: at + 2] = np.frombuffer(np.float16(np.nan).tobytes(), np.uint8)
            c2 = R.Cache.__new__(R.Cache)
            c2.__dict__.update(cache.__dict__)
            c2.bytes = data
            out, *_ = run_attend(c2, table, q_start, q_count, kv_len, q, d ** -0.5, T)
            got = out.float().cpu().numpy()
            want, tol = R.attend(q.double().numpy(), cache, table, q_start, q_count, kv_len, d ** -0.5)
            hit = np.isnan(got[T - 1])
            assert hit.any(-1).all() and (which == 1 or hit.all())
            rest = [n for n in range(2 * T) if n != T - 1]
            assert (np.abs(got[rest] - want[rest]) <= tol[rest]).all()


def test_attend_bad_page_and_lengths_raise_status(gdn):
    cache, table, q_start, q_count, kv_len, q = attend_case(8, 2, 128, 16, [(100, 2, 2), (50, 2, 2)], seed=1)
    want, tol = R.attend(q.double().numpy(), cache, table, q_start, q_count, kv_len, 1.0)
    for cell in (-1, cache.n, 1 << 30):
        t2 = table.copy()
        t2[0, 3] = cell
        out, *_ = run_attend(cache, t2, q_start, q_count, kv_len, q, 1.0, 2)
        assert L.gdn_get_status(clear=True) == L.GDN_STATUS_BAD_INDEX
        assert (np.abs(out.cpu().double().numpy() - want)[2:] <= tol[2:]).all(), "the other row is untouched"
    for n in (-5, 10 ** 6):
        out, *_ = run_attend(cache, table, q_start, q_count, [n, 50], q, 1.0, 2)
        assert L.gdn_get_status(clear=True) & L.GDN_STATUS_BAD_LEN
        assert (np.abs(out.cpu().double().numpy() - want)[2:] <= tol[2:]).all()


def test_attend_workspace_is_ready_again_and_repeatable(gdn):
    """The same call twice on one workspace, other shapes between: equal bits each time."""
    rows = [(3000, 2, 2), (64, 1, 2), (777, 2, 2)]
    cache, table, q_start, q_count, kv_len, q = attend_case(16, 2, 256, 64, rows, seed=8)
    a, ws, kd, args = run_attend(cache, table, q_start, q_count, kv_len, q, 0.06, 2)
    for n in ([40, 64, 2], [3000, 64, 777], [0, 1, 64], [3000, 64, 777]):
        out = torch.empty_like(a)
        L.gdn_kv4_attend(kd, *args[:-1], dev(n), 0.06, out, ws, 2)
        if n[0] == 3000:
            assert torch.equal(bits(out), bits(a))


@pytest.mark.parametrize("Hq,Hkv,d,T,n", [(8, 1, 128, 8, 200), (16, 2, 256, 40, 300), (4, 4, 64, 70, 500), (16, 2, 256, 2, 3000), (8, 2, 128, 1, 777)])
def test_attend_gives_equal_bits_call_after_call(gdn, Hq, Hkv, d, T, n):
    """Forty calls without a wait between them: the split and the joins leave nothing to timing."""
    rows = [(T, T, T), (n, T, T), (n // 2, max(1, T - 1), T)]
    cache, table, q_start, q_count, kv_len, q = attend_case(Hq, Hkv, d, 16, rows, seed=11)
    a, ws, kd, args = run_attend(cache, table, q_start, q_count, kv_len, q, 0.09, T)
    outs = [torch.empty_like(a) for _ in range(40)]
    for o in outs:
        L.gdn_kv4_attend(kd, *args, 0.09, o, ws, T)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(o), bits(a)) for o in outs)


def test_attend_on_another_stream_and_in_a_graph(gdn):
    rows = [(2000, 2, 2), (500, 1, 2)]
    cache, table, q_start, q_count, kv_len, q = attend_case(8, 2, 128, 32, rows, seed=8)
    a, ws, kd, args = run_attend(cache, table, q_start, q_count, kv_len, q, 0.1, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(a)
    side.wait_stream(torch.cuda.current_stream())
    L.gdn_kv4_attend(kd, *args, 0.1, out, ws, 2, stream=side)
    side.synchronize()
    assert torch.equal(bits(out), bits(a))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        L.gdn_kv4_attend(kd, *args, 0.1, out, ws, 2)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(a))


def test_cache_beyond_32_bits(gdn):
    """A cache of more than 2^32 bytes: the last pages are written, read and attended."""
    Hq, Hkv, d, page = 4, 2, 64, 64
    per = Hkv * 2 * (page * d // 2 + page * 4)
    n_pages = (1 << 32) // per + 100
    kd = L.kv4_dims(1, Hq, Hkv, d, page, 2, n_pages)
    assert L.gdn_kv4_page_bytes(kd) == per
    pages = torch.zeros(n_pages * per, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(0)
    N = 100
    x = R.bf16(rng.normal(size=(N, Hq + 2 * Hkv, d)))
    table = np.array([[n_pages - 1, n_pages - 70]])
    slots = np.array([table[0][t // page] * page + t % page for t in range(N)], np.int32)
    xd = x.cuda()
    q_out = torch.empty((N, Hq, d), dtype=torch.bfloat16, device="cuda")
    L.gdn_kv4_append(kd, xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], None, None, b"", dev(slots), pages, q_out)
    k = torch.empty((N, Hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    L.gdn_kv4_read(kd, dev(slots), pages, k, v)
    small = R.Cache(2, Hkv, page, d)
    for t in range(N):
        small.write(t, x[t, Hq:Hq + Hkv].float().numpy(), x[t, Hq + Hkv:].float().numpy())
    rk, rv = small.read(np.arange(N))
    assert torch.equal(bits(k.cpu()), bits(R.bf16(rk))) and torch.equal(bits(v.cpu()), bits(R.bf16(rv)))
    out = torch.empty((1, Hq, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(L.gdn_kv4_attend_workspace_bytes(kd, 1, 1), dtype=torch.uint8, device="cuda")
    L.gdn_kv4_attend(kd, q_out[-1:].contiguous(), pages, dev(table), dev([0, 1]), dev([1]), dev([N]), 0.125, out, ws, 1)
    want, tol = R.attend(x[-1:, :Hq].double().numpy(), small, [[0, 1]], [0, 1], [1], [N], 0.125)
    assert (np.abs(out.cpu().double().numpy() - want) <= tol).all()
    assert L.gdn_get_status(clear=True) == 0
