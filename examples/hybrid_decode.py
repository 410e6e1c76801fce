"""Speculative decoding of a two-layer hybrid model: one GDN layer, one attention layer over the paged 4-bit cache.

    python examples/hybrid_decode.py [--rows 8] [--prompt 500] [--cycles 64] [--draft 1]

The weights are random, so the tokens mean nothing; what the script shows is how the calls go together.  The committed
offsets that gdn_commit advances are the attention layer's lengths as well.  A prompt:

    gdn_kv_plan (packed)     pages, slots and positions of the prompt's tokens
    gdn_prefill_chunked      the GDN layer over the prompt, offsets to its length
    gdn_kv4_append           rotate q and k, keys and values into the cache
    gdn_kv4_attend           causal attention of the prompt over the cache

and a cycle of T tokens a row (the last accepted one and T - 1 drafts), captured once into a CUDA graph:

    gdn_kv_plan (fixed T)    also takes back what the last cycle's rejected drafts held
    gdn_conv_verify, gdn_kv4_append, gdn_kv4_attend
    gdn_accept_greedy        keep, and the next token
    gdn_commit               the GDN state of the accepted prefix; offsets += keep
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decode_gated_gdn_gb300 import lib as L  # noqa: E402

MODE = L.GDN_COMMIT_RECOMPUTE


class Model:
    """B rows of the model with their GDN state, conv ring and cache pages."""

    def __init__(self, B, T, max_len, vocab=512, width=256, H_k=2, H_v=4, d_gdn=64, H_q=8, H_kv=2, d=128, rot=64, page=32,
                 seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).bfloat16()
        zeros = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")
        self.B, self.T, self.H_q, self.H_kv, self.d, self.rot, self.vocab = B, T, H_q, H_kv, d, rot, vocab
        self.gdims = L.dims(B=B, T=T, H_k=H_k, H_v=H_v, d=d_gdn)
        C = (2 * H_k + H_v) * d_gdn
        self.H_v, self.d_gdn = H_v, d_gdn
        self.embed = rand(vocab, width)
        self.w_gdn, self.conv_w = rand(width, C, scale=width ** -0.5), rand(C, 4, scale=0.5)
        self.w_gate = rand(width, 2 * H_v, scale=width ** -0.5)
        self.w_qkv = rand(width, (H_q + 2 * H_kv) * d, scale=width ** -0.5)
        self.w_out = rand(H_v * d_gdn + H_q * d, vocab, scale=0.1)
        self.state = zeros(B, H_v, d_gdn, d_gdn, dtype=torch.float32)
        self.ring = zeros(B, 3 + T, C, dtype=torch.bfloat16)
        self.offsets, self.active = zeros(B), torch.ones(B, dtype=torch.uint8, device="cuda")
        self.gdn_ws = zeros(L.gdn_layer_workspace_bytes(self.gdims, MODE), dtype=torch.uint8)

        max_pages = -(-(max_len + T) // page)
        n_pages = B * max_pages
        self.kd = L.kv4_dims(B, H_q, H_kv, d, page, max_pages, n_pages)
        self.pages = zeros(n_pages * L.gdn_kv4_page_bytes(self.kd), dtype=torch.uint8)
        self.held, self.table = zeros(B), torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free_list = torch.arange(n_pages, dtype=torch.int32, device="cuda")
        self.free_count = torch.full((1,), n_pages, dtype=torch.int32, device="cuda")
        self.q_start, self.q_count, self.kv_len = zeros(B + 1), zeros(B), zeros(B)
        # text: the three axes of a position are the same, and the pairs of a head take them in turn
        t = torch.arange(max_len + T, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
        self.rope = torch.stack((t.cos(), t.sin()), -1).float().cuda().contiguous()
        self.axis = bytes(i % 3 for i in range(rot // 2))

        self.add = torch.full((B,), T, dtype=torch.int32, device="cuda")
        self.tokens, self.keep, self.next = zeros(B, T), zeros(B), zeros(B)
        self.accept_ws = zeros(L.gdn_accept_workspace_bytes(B, T, vocab), dtype=torch.uint8)
        self.step = self._buffers(B * T, T)

    def _buffers(self, N, max_q):
        """What a call over N tokens needs besides the model."""
        z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")
        return dict(slots=z(N), positions=z(3, N), q=z(N, self.H_q, self.d, dtype=torch.bfloat16),
                    o=z(N, self.H_q, self.d, dtype=torch.bfloat16), max_q=max_q,
                    ws=z(L.gdn_kv4_attend_workspace_bytes(self.kd, N, max_q), dtype=torch.uint8))

    def _plan(self, buf, add, T):
        L.gdn_kv_plan(self.kd, self.offsets, add, self.active, self.held, self.table, self.free_list, self.free_count,
                      self.q_start, self.q_count, self.kv_len, buf["slots"], buf["positions"][0], T=T)
        buf["positions"][1:] = buf["positions"][0]

    def _attention(self, h, buf):
        """The attention layer over the N tokens with embeddings h [N][width]."""
        qkv = (h @ self.w_qkv).view(h.shape[0], self.H_q + 2 * self.H_kv, self.d)
        q, k, v = qkv.split((self.H_q, self.H_kv, self.H_kv), 1)  # slices: the token stride is the projection's
        L.gdn_kv4_append(self.kd, q, k, v, buf["positions"], self.rope, self.axis, buf["slots"], self.pages, buf["q"])
        L.gdn_kv4_attend(self.kd, buf["q"], self.pages, self.table, self.q_start, self.q_count, self.kv_len, self.d ** -0.5,
                         buf["o"], buf["ws"], buf["max_q"])
        return buf["o"].flatten(1)

    def _gdn_inputs(self, h, n):
        x = (h @ self.w_gdn).view(self.B, n, -1).contiguous()
        g, beta = (h @ self.w_gate).float().view(self.B, n, 2, self.H_v).unbind(2)
        return x, -torch.nn.functional.softplus(g).contiguous(), beta.sigmoid().contiguous()

    def prompt(self, tokens):
        """tokens [B][n]: fills state and cache, and puts the first token to verify in place."""
        n = tokens.shape[1]
        buf = self._buffers(self.B * n, n)
        self._plan(buf, torch.full_like(self.add, n), 0)
        h = self.embed[tokens.reshape(-1)]
        x, g, beta = self._gdn_inputs(h, n)
        o = torch.empty(self.B, n, self.H_v, self.d_gdn, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(L.gdn_prefill_workspace_bytes(self.gdims, n), 16), dtype=torch.uint8, device="cuda")
        a = self._attention(h, buf)
        L.gdn_prefill_chunked(self.gdims, n, x, self.conv_w, g, beta, self.state, self.ring, self.offsets, o, ws)
        last = torch.cat((o[:, -1].flatten(1), a.view(self.B, n, -1)[:, -1]), 1) @ self.w_out
        self._feed(last.argmax(1).int())

    def _feed(self, nxt):
        """The next cycle's tokens: the accepted one, and drafts of it by a rule in place of a draft model."""
        self.tokens[:, 0] = nxt
        for t in range(1, self.T):
            self.tokens[:, t] = (self.tokens[:, t - 1] * 5 + 1) % self.vocab

    def cycle(self):
        """One verify cycle; no host round trip, so it can be captured."""
        buf, T = self.step, self.T
        self._plan(buf, self.add, T)
        h = self.embed[self.tokens.reshape(-1)]
        x, g, beta = self._gdn_inputs(h, T)
        o = torch.empty(self.B, T, self.H_v, self.d_gdn, dtype=torch.bfloat16, device="cuda")
        L.gdn_conv_verify(self.gdims, MODE, x, self.conv_w, g, beta, self.state, self.ring, self.offsets, self.active, o,
                          self.gdn_ws)
        logits = (torch.cat((o.flatten(2).flatten(0, 1), self._attention(h, buf)), 1) @ self.w_out).view(self.B, T, -1)
        L.gdn_accept_greedy(logits, self.tokens, self.active, self.keep, self.next, self.accept_ws)
        L.gdn_commit(self.gdims, MODE, [self.state], [self.ring], [self.gdn_ws], self.keep, self.active, self.offsets)
        self._feed(self.next)


def run(rows=8, prompt=500, cycles=64, draft=1, seed=0):
    """Decodes and returns the model and the seconds a cycle took."""
    m = Model(rows, draft + 1, prompt + (cycles + 3) * (draft + 1), seed=seed)
    m.prompt(torch.randint(0, m.vocab, (rows, prompt), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 1)))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        m.cycle()  # the first calls set kernels up, outside the capture
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.cycle()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(cycles):
        graph.replay()
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t0) / max(cycles, 1)
    status = L.gdn_get_status(clear=True)
    if status:
        raise RuntimeError(f"device status {status}")
    return m, dt


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--cycles", type=int, default=64)
    ap.add_argument("--draft", type=int, default=1)
    a = ap.parse_args()
    m, dt = run(a.rows, a.prompt, a.cycles, a.draft)
    done = (m.offsets - a.prompt).float().mean().item()
    used = m.kd.n_pages - m.free_count.item()
    print(f"{a.rows} rows, prompt {a.prompt}: {done:.1f} tokens a row in {a.cycles + 1} cycles of {a.draft + 1}, "
          f"{dt * 1e6:.0f} us a cycle, {used} pages of {m.kd.page} tokens held ({used * L.gdn_kv4_page_bytes(m.kd)} bytes)")


if __name__ == "__main__":
    main()
