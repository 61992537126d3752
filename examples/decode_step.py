"""Decoding with drafted runs by the operators of one decoder layer's step.  In torch stay the
embedding, the plain products, the draft model and the record of what was said.

One step for B sequences with n drafted tokens each:
  plan_step (pages, slots, positions) -> embed -> q, k, v -> rotary_write (rotated, quantised into
  the cache) -> paged_attention -> forward_few (the expert layer, FP8) -> adjust_logits (penalties,
  biases, mask, temperature) -> verify_draft -> release_pages (what refused drafts had taken).
A sequence that ends gives its pages back, and a waiting one takes its row.  Weights are random; the
draft model is the target without its attention and experts.

    python examples/decode_step.py [--steps N] [--waiting TOKENS]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_forward_gb300 import _lib as L  # noqa: E402
from mixture_experts_forward_gb300 import inputs  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, HEAD_DIM = 512, 8, 2, 64
EXPERTS, TOP_K, INNER, VOCAB, PAGE = 16, 2, 256, 2000, 16


class Server:
    """The weights, the cache and its pages, and the sequences' state."""

    def __init__(self, batch: int, n_draft: int, pages: int, most: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        bf16 = lambda t: t.to(torch.bfloat16).cuda()   # noqa: E731
        zeros = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.n, self.batch, self.pages = n_draft, batch, pages
        self.embed = bf16(rnd(VOCAB, HIDDEN))
        width = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.w_qkv = bf16(rnd(HIDDEN, width) / HIDDEN ** 0.5)
        self.w_o = bf16(rnd(Q_HEADS * HEAD_DIM, HIDDEN) / HIDDEN ** 0.5)
        self.w_out = bf16(rnd(HIDDEN, VOCAB) * 3 / HIDDEN ** 0.5)
        self.w_router = (rnd(HIDDEN, EXPERTS) / HIDDEN ** 0.5).cuda()
        up_q, up_s = inputs.quantize_weights_e4m3(rnd(EXPERTS, 2 * INNER, HIDDEN) / HIDDEN ** 0.5)
        dn_q, dn_s = inputs.quantize_weights_e4m3(rnd(EXPERTS, HIDDEN, INNER) / INNER ** 0.5)
        self.up, self.up_s, self.dn, self.dn_s = up_q.cuda(), up_s.cuda(), dn_q.cuda(), dn_s.cuda()
        self.rope = L.rotary_table(HEAD_DIM, base=10000.0, scaling="turns", factor=4.0, original=4096,
                                   low=1.0, high=4.0)
        self.k, self.v, self.ks, self.vs = L.new_kv_cache(L.DTYPE_FP8, pages, PAGE, KV_HEADS, HEAD_DIM)
        # every page is free; a sequence may hold up to `most` positions
        self.table, self.held = zeros(batch, -(-most // PAGE)) - 1, zeros(batch)
        self.free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
        self.count = torch.tensor([pages], dtype=torch.int32, device="cuda")
        self.len = zeros(batch)                                            # cached positions
        self.history, self.said, self.prompt = zeros(batch, most), zeros(batch), zeros(batch)
        self.ws, self.ctrl = L.new_workspace(L.ATTENTION_WS_BYTES), L.new_workspace(L.CTRL_BYTES)
        few = L.forward_args(dtype=L.DTYPE_FP8, M=L.FEW_TOKENS, K=HIDDEN, N=INNER, E=EXPERTS, top_k=TOP_K, gated=1)
        self.few_ws = L.new_workspace(L.few_workspace_size(few))
        # decoding: one token is never said, one is favoured, and a repetition costs
        self.penalties = dict(repetition=torch.full((batch,), 1.2, device="cuda"),
                              frequency=torch.full((batch,), 0.1, device="cuda"),
                              temperature=torch.full((batch,), 0.7, device="cuda"),
                              bias_tokens=zeros(batch, 1) + 7, bias_values=torch.ones(batch, 1, device="cuda"))
        bits = torch.full((batch, (VOCAB + 31) // 32), -1, dtype=torch.int32, device="cuda")
        bits[:, 0] = ~(1 << 13)
        self.mask = bits

    def experts(self, x):
        """The expert layer, as many tokens a call as it takes."""
        logits, out = x.float() @ self.w_router, torch.empty_like(x)
        for a in range(0, x.shape[0], L.FEW_TOKENS):
            part, lg = x[a:a + L.FEW_TOKENS], logits[a:a + L.FEW_TOKENS]
            args = L.forward_args(dtype=L.DTYPE_FP8, M=part.shape[0], K=HIDDEN, N=INNER, E=EXPERTS, top_k=TOP_K,
                                  logits=lg, x=part, w=self.up, w_scales=self.up_s, w2=self.dn, w2_scales=self.dn_s,
                                  gated=1)
            L.forward_few(args, out[a:a + L.FEW_TOKENS], self.few_ws)
        return out

    def forward(self, tokens, new, most_new):
        """tokens [T]: new[b] of each sequence, packed; returns their logits [T, VOCAB].  Their keys
        and values are cached; self.len is left as it was."""
        T = tokens.shape[0]
        slots, positions, cu, kv = L.plan_step(self.len, new, self.table, self.held, self.free, self.count, T, PAGE,
                                               self.pages, self.ctrl)
        x = self.embed[tokens.long()]
        qkv = (x @ self.w_qkv).view(T, Q_HEADS + 2 * KV_HEADS, HEAD_DIM)
        q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], dim=1)          # strided views
        q = L.rotary_write(q, k, v, positions, slots, self.rope, self.k, self.v, self.ctrl, k_scales=self.ks,
                           v_scales=self.vs)
        a, _ = L.paged_attention(q, self.k, self.v, self.table, cu, kv, self.ws, max_q=most_new, k_scales=self.ks,
                                 v_scales=self.vs)
        x = x + a.view(T, -1) @ self.w_o
        x = x + self.experts(x)
        return (x @ self.w_out).float()

    def drafts(self, last, g):
        """n drafted tokens after `last` [B] and the distributions they came from."""
        tokens, probs = [], []
        for _ in range(self.n):
            q = torch.softmax((self.embed[last.long()] @ self.w_out).float(), -1)
            last = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32)
            tokens.append(last)
            probs.append(q)
        return torch.stack(tokens, 1), torch.stack(probs, 1)

    def step(self, last, g):
        """One step: the last token and n drafts of every sequence; returns (accepted, tokens)."""
        draft, q_probs = self.drafts(last, g)
        m = self.n + 1
        new = torch.full((self.batch,), m, dtype=torch.int32, device="cuda")
        tokens = torch.cat([last[:, None], draft], 1)
        logits = self.forward(tokens.reshape(-1), new, m).view(self.batch, m, VOCAB)
        p = L.adjust_logits(logits, self.ctrl, history=self.history, history_lens=self.said, prompt_lens=self.prompt,
                            draft=draft, mask=self.mask, **self.penalties)
        u = torch.rand(self.batch, self.n, device="cuda", generator=g)
        accepted, out = L.verify_draft(p, q_probs, draft, u, torch.rand(self.batch, device="cuda", generator=g),
                                       self.ctrl)
        self.len = self.len + accepted + 1
        L.release_pages(self.len, self.table, self.held, self.free, self.count, PAGE, self.ctrl)
        # what was said joins the history
        at = self.said.long()[:, None] + torch.arange(m, device="cuda")
        said = torch.arange(m, device="cuda")[None] <= accepted[:, None]
        self.history.scatter_(1, at, torch.where(said, out, self.history.gather(1, at)))
        self.said = self.said + accepted + 1
        return accepted, out

    def end(self, b):
        """Sequence b ends: all of its pages go back."""
        keep = self.len.clone()
        keep[b] = 0
        L.release_pages(keep, self.table, self.held, self.free, self.count, PAGE, self.ctrl)
        self.len, self.said[b], self.prompt[b] = keep, 0, 0

    def admit(self, b, text):
        """A sequence takes row b, which is free: all of its prompt but the last token is cached."""
        n = text.numel()
        new = torch.zeros_like(self.len)
        new[b] = n - 1
        self.forward(text[:-1], new, n - 1)
        self.len, self.said[b], self.prompt[b] = self.len + new, n, n
        self.history[b, :n] = text

    def status(self):
        return [L.get_error(w) for w in (self.ctrl, self.ws, self.few_ws)]


def main(steps: int = 8, batch: int = 4, n_draft: int = 3, prompt: int = 37, seed: int = 0, waiting: int = 0):
    """Decodes `steps` steps of `batch` sequences, then the first ends.  waiting > 0: one with a prompt
    of so many tokens (2 to `prompt`) takes its place, and `steps` steps more are decoded."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    most = prompt + ((2 if waiting else 1) * steps + 1) * (n_draft + 1)
    pages = batch * -(-most // PAGE)
    s = Server(batch, n_draft, pages, most, seed)
    # prompts of ragged lengths, as one packed chunk each
    lens = torch.tensor([prompt - 5 * b for b in range(batch)], dtype=torch.int32, device="cuda")
    text = torch.randint(VOCAB, (batch, prompt), device="cuda", generator=g, dtype=torch.int32)
    real = torch.arange(prompt, device="cuda")[None] < (lens - 1)[:, None]
    s.forward(text[real], lens - 1, prompt - 1)
    s.len = lens - 1
    s.history[:, :prompt] = torch.where(torch.arange(prompt, device="cuda")[None] < lens[:, None], text, 0)
    s.said, s.prompt = lens.clone(), lens.clone()
    last = text.gather(1, (lens - 1).long()[:, None])[:, 0]
    out = [[] for _ in range(batch)]

    def decode(last):
        for _ in range(steps):
            accepted, tokens = s.step(last, g)
            last = tokens.gather(1, accepted.long()[:, None])[:, 0]
            for b, (a, row) in enumerate(zip(accepted.tolist(), tokens.tolist())):
                out[b] += row[:a + 1]
        return last

    last = decode(last)
    lengths, held, free = s.len.tolist(), s.held.tolist(), int(s.count)
    s.end(0)
    r = dict(tokens=out, lengths=lengths, held=held, free=free, pages=pages, after=(s.held.tolist(), int(s.count)),
             server=s)
    if waiting:
        ended, out[0] = out[0], []
        text = torch.randint(VOCAB, (waiting,), device="cuda", generator=g, dtype=torch.int32)
        s.admit(0, text)
        last[0] = text[-1]
        decode(last)
        r.update(ended=ended, lengths=s.len.tolist(), held=s.held.tolist(), free=int(s.count))
    r["status"] = s.status()
    return r


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--waiting", type=int, default=25)
    a = ap.parse_args()
    r = main(a.steps, waiting=a.waiting)
    for b, t in enumerate(r["tokens"]):
        print(f"sequence {b}: {len(t)} tokens {t[:12]}{' ...' if len(t) > 12 else ''}")
    if "ended" in r:
        print(f"(the first row had {len(r['ended'])} tokens of a sequence that ended)")
    print(f"cached positions {r['lengths']}, pages held {r['held']}, free {r['free']} of {r['pages']}, "
          f"status {r['status']}")
