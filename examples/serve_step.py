"""Speculative decoding steps of a one-layer sparse decoder, served from a paged
FP8 cache: the serving operators around the fused expert forward.

One step for B sequences with n drafted tokens each:
  embed -> q, k, v -> kv_write (quantised) -> paged_attention (n + 1 rows a
  sequence) -> moe_forward (FP8 experts) -> probabilities -> verify_draft,
then the accepted tokens and one more extend each sequence; the cached rows of
refused drafts are overwritten by the next step.  At the end one sequence's cache is
read back and written to other pages (as a prefix is handed to another
worker).  Weights are random; the draft model is the target without its
attention and experts; products outside the library's scope are torch matmuls.

    python examples/serve_step.py [--steps N]
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
EXPERTS, TOP_K, VOCAB, PAGE = 16, 2, 2000, 16


class Server:
    """The weights, the cache and the sequences' state."""

    def __init__(self, batch: int, n_draft: int, max_len: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        bf16 = lambda t: t.to(torch.bfloat16).cuda()   # noqa: E731
        self.n, self.batch = n_draft, batch
        self.embed = bf16(rnd(VOCAB, HIDDEN))
        width = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.w_qkv = bf16(rnd(HIDDEN, width) / HIDDEN ** 0.5)
        self.w_o = bf16(rnd(Q_HEADS * HEAD_DIM, HIDDEN) / HIDDEN ** 0.5)
        self.w_out = bf16(rnd(HIDDEN, VOCAB) * 3 / HIDDEN ** 0.5)
        self.w_router = (rnd(HIDDEN, EXPERTS) / HIDDEN ** 0.5).cuda()
        w_q, w_s = inputs.quantize_weights_e4m3(rnd(EXPERTS, HIDDEN, HIDDEN) / HIDDEN ** 0.5)
        self.w_q, self.w_s = w_q.cuda(), w_s.cuda()
        # the cache: every sequence owns max_len positions, in pages of a random order
        per = -(-max_len // PAGE)
        self.k, self.v, self.ks, self.vs = L.new_kv_cache(L.DTYPE_FP8, (batch + 1) * per, PAGE,
                                                          KV_HEADS, HEAD_DIM)
        pages = torch.randperm((batch + 1) * per, generator=g).to(torch.int32).view(batch + 1, per)
        self.table, self.spare = pages[:batch].contiguous().cuda(), pages[batch:].contiguous().cuda()
        self.len = torch.zeros(batch, dtype=torch.int32, device="cuda")   # cached positions
        # one attention workspace and one status block for the small operators
        self.ws, self.ctrl = L.new_workspace(L.ATTENTION_WS_BYTES), L.new_workspace(L.CTRL_BYTES)
        self._moe = {}

    def slots(self, table, first, count):
        """Slots of positions first[b] .. first[b] + count - 1 of each sequence."""
        pos = first.long()[:, None] + torch.arange(count, device="cuda")
        return (table.long().gather(1, pos // PAGE) * PAGE + pos % PAGE).to(torch.int32).reshape(-1)

    def experts(self, x):
        T = x.shape[0]
        logits = (x.float() @ self.w_router).contiguous()
        if T not in self._moe:                        # buffers and arguments kept per row count
            out, lg, xb = torch.empty_like(x), torch.empty_like(logits), torch.empty_like(x)
            args = L.forward_args(dtype=L.DTYPE_FP8, M=T, K=HIDDEN, N=HIDDEN, E=EXPERTS, top_k=TOP_K,
                                  logits=lg, x=xb, w=self.w_q, w_scales=self.w_s)
            self._moe[T] = (args, L.new_workspace(L.workspace_size(args)), out, lg, xb)
        args, ws, out, lg, xb = self._moe[T]
        lg.copy_(logits)
        xb.copy_(x)
        return L.forward(args, out, ws)

    def forward(self, tokens):
        """tokens [B, m]: appends their keys and values and returns their
        next-token probabilities [B, m, VOCAB]; self.len is left as it was."""
        B, m = tokens.shape
        x = self.embed[tokens.reshape(-1).long()]
        qkv = (x @ self.w_qkv).view(B * m, Q_HEADS + 2 * KV_HEADS, HEAD_DIM)
        q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], dim=1)     # strided views
        L.kv_write(k, v, self.slots(self.table, self.len, m), self.k, self.v, self.ctrl,
                   k_scales=self.ks, v_scales=self.vs)
        cu = torch.arange(0, (B + 1) * m, m, dtype=torch.int32, device="cuda")
        a, _ = L.paged_attention(q, self.k, self.v, self.table, cu, self.len + m, self.ws, max_q=m,
                                 k_scales=self.ks, v_scales=self.vs)
        x = x + a.view(B * m, -1) @ self.w_o
        x = x + self.experts(x)
        return torch.softmax((x @ self.w_out).float(), -1).view(B, m, VOCAB)

    def drafts(self, last, g):
        """n drafted tokens after `last` [B] and the distributions they came from."""
        tokens, probs = [], []
        for _ in range(self.n):
            q = torch.softmax((self.embed[last.long()] @ self.w_out).float(), -1)
            last = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32)
            tokens.append(last)
            probs.append(q)
        return torch.stack(tokens, 1), torch.stack(probs, 1)

    def step(self, last, draft, q_probs, u, u_sample):
        """Scores the last token and the drafts, keeps what is accepted."""
        p = self.forward(torch.cat([last[:, None], draft], 1))
        accepted, tokens = L.verify_draft(p, q_probs, draft, u, u_sample, self.ctrl)
        self.len = self.len + accepted + 1
        return accepted, tokens

    def status(self):
        return L.get_error(self.ctrl), L.get_error(self.ws)


def main(steps: int = 8, batch: int = 3, n_draft: int = 4, prompt: int = 37, seed: int = 0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = Server(batch, n_draft, prompt + (steps + 1) * (n_draft + 1), seed)
    text = torch.randint(VOCAB, (batch, prompt), device="cuda", generator=g, dtype=torch.int32)
    s.forward(text[:, :-1])                                           # the prompt, as one chunk
    s.len += prompt - 1
    last = text[:, -1]
    out = [[] for _ in range(batch)]
    for _ in range(steps):
        draft, q_probs = s.drafts(last, g)
        u = torch.rand(batch, n_draft, device="cuda", generator=g)
        u_sample = torch.rand(batch, device="cuda", generator=g)
        accepted, tokens = s.step(last, draft, q_probs, u, u_sample)
        last = tokens.gather(1, accepted.long()[:, None])[:, 0]
        for b, (a, row) in enumerate(zip(accepted.tolist(), tokens.tolist())):
            out[b] += row[:a + 1]
    # hand sequence 0 over: read its cache, write it to other pages
    n = int(s.len[0])
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    k, v = L.kv_read(s.k, s.v, s.table[:1].contiguous(), cu, n, s.ctrl, k_scales=s.ks, v_scales=s.vs)
    L.kv_write(k, v, s.slots(s.spare, torch.zeros(1, dtype=torch.int32, device="cuda"), n), s.k, s.v,
               s.ctrl, k_scales=s.ks, v_scales=s.vs)
    k2, _ = L.kv_read(s.k, s.v, s.spare, cu, n, s.ctrl, k_scales=s.ks, v_scales=s.vs)
    drift = ((k2.float() - k.float()).norm() / k.float().norm()).item()
    status = s.status()
    return dict(tokens=out, lengths=s.len.tolist(), status=status, drift=drift)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    r = main(ap.parse_args().steps)
    for b, t in enumerate(r["tokens"]):
        print(f"sequence {b}: {len(t)} tokens {t[:12]}{' ...' if len(t) > 12 else ''}")
    print(f"cached positions {r['lengths']}, status {r['status']}, "
          f"handed-over cache differs by {r['drift']:.1e}")
