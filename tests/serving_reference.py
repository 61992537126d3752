"""Plain 64-bit forms of the serving operators, and the paged caches their
tests use (no code of the package's operators here)."""
from __future__ import annotations

import math

import torch

NAN_CODE = 0x7F


def quantise_rows(x: torch.Tensor):
    """The row rule on bf16 rows [..., D]: (codes u8, scales f32).  amax/448 and
    1/s are single binary32 roundings, the cast is torch's own."""
    f = x.float()
    amax = f.abs().amax(-1, keepdim=True)
    s = amax / 448.0
    inv = 1.0 / s
    tiny = amax < 448.0 * 2.0 ** -126
    codes = (f * inv).clamp(-448.0, 448.0)
    codes = torch.where(tiny, torch.zeros_like(codes), codes).to(torch.float8_e4m3fn)
    s = torch.where(tiny, torch.zeros_like(s), s)
    return codes.view(torch.uint8), s.squeeze(-1)


class Paged:
    """A cache whose unowned positions are NaN, with ragged sequences in pages
    of a random order.  keys / values: lists of bf16 [n_b, H, D]."""

    def __init__(self, keys, values, page, fp8, seed=0, extra_pages=2, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        H, D = keys[0].shape[1:]
        need = [-(-k.shape[0] // page) for k in keys]
        n_pages = sum(need) + extra_pages
        order = torch.randperm(n_pages, generator=g).tolist()
        width = max(max(need), 1) + 1
        self.table = torch.full((len(keys), width), -1, dtype=torch.int32)   # unused entries: -1
        self.page, self.fp8, self.H, self.D = page, fp8, H, D
        if fp8:
            self.k = torch.full((n_pages, H, page, D), NAN_CODE, dtype=torch.uint8)
            self.ks = torch.full((n_pages, H, page), math.nan)
        else:
            self.k = torch.full((n_pages, H, page, D), math.nan, dtype=torch.bfloat16)
            self.ks = None
        self.v = self.k.clone()
        self.vs = None if self.ks is None else self.ks.clone()
        self.slots = []
        at = 0
        for b, n in enumerate(need):
            ids = order[at:at + n]
            at += n
            self.table[b, :n] = torch.tensor(ids, dtype=torch.int32)
            rows = keys[b].shape[0]
            pos = torch.arange(rows)
            pg = torch.tensor(ids, dtype=torch.int64)[pos // page] if rows else pos
            self.slots.append((pg * page + pos % page).to(torch.int32))
            for src, dst, sc in ((keys[b], self.k, self.ks), (values[b], self.v, self.vs)):
                if rows == 0:
                    continue
                if fp8:
                    c, s = quantise_rows(src)
                    dst[pg, :, pos % page] = c
                    sc[pg, :, pos % page] = s
                else:
                    dst[pg, :, pos % page] = src
        for name in ("k", "v", "ks", "vs", "table"):
            t = getattr(self, name)
            setattr(self, name, None if t is None else t.to(device))

    def rows(self, name, b, n):
        """[n, H, D] float64 of sequence b's first n positions."""
        pages, sc = getattr(self, name), getattr(self, name + "s")
        pos = torch.arange(n, device=pages.device)
        pg = self.table[b].long()[pos // self.page]
        x = pages[pg, :, pos % self.page]
        if self.fp8:
            return x.view(torch.float8_e4m3fn).double() * sc[pg, :, pos % self.page].double()[..., None]
        return x.double()


def attention(q, cache: Paged, q_lens, kv_lens, *, scale=0.0, softcap=0.0, window=0, causal=True):
    """(out, lse, tol_out, tol_lse) in float64 of q bf16 [T, Hq, D].

    The tolerances bound a binary32 computation: delta, the error of a score, is
    at most (D + 8) * 2^-23 * |scale| * sum |q k| (each product exact, every partial
    sum rounded or truncated once), plus c * 2^-20 through a softcap; a weight is
    then off by delta, and once more by its rounding to 8 bits (2^-8, the
    coarsest kernel's); so is the sum, without the rounding; the output is
    rounded to 8 bits (2^-8 of itself).  2^-16 covers the exponentials and sums."""
    T, Hq, D = q.shape
    G = Hq // cache.H
    scale = scale or 1.0 / math.sqrt(D)
    dev = q.device
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    tol_o = torch.zeros_like(out)
    tol_l = torch.zeros_like(lse)
    at = 0
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        if m == 0:
            continue
        k, v = cache.rows("k", b, n), cache.rows("v", b, n)
        i = torch.arange(m, device=dev)[:, None]
        j = torch.arange(n, device=dev)[None, :]
        seen = torch.ones(m, n, dtype=torch.bool, device=dev)
        if causal:
            seen = j <= n - m + i
            if window:
                seen &= j > n - m + i - window
        for h in range(Hq):
            qh, kh, vh = q[at:at + m, h].double(), k[:, h // G], v[:, h // G]
            if n == 0:
                continue
            x = qh @ kh.T * scale
            # scores that nobody sees do not count towards the tolerance
            delta = ((qh.abs() @ kh.abs().T) * abs(scale) * (D + 8) * 2.0 ** -23)
            delta = delta.masked_fill(~seen, 0.0).amax(1, keepdim=True)
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                delta = delta + softcap * 2.0 ** -20
            x = x.masked_fill(~seen, -math.inf)
            any_ = seen.any(1)
            w = torch.where(any_[:, None], torch.softmax(x, 1), torch.zeros_like(x))
            o = w @ vh
            a = w @ vh.abs()
            out[at:at + m, h] = o
            lse[at:at + m, h] = torch.where(any_, torch.logsumexp(x, 1), lse[at:at + m, h])
            tol_o[at:at + m, h] = o.abs() * 2.0 ** -8 + a * (2.0 ** -8 + 2 * delta + 2.0 ** -16)
            tol_l[at:at + m, h] = delta[:, 0] + 2.0 ** -20 * (1 + lse[at:at + m, h].abs().nan_to_num(0, 0, 0))
        at += m
    return out, lse, tol_o, tol_l


def verify(p, q, draft, lens, u, us, fix=38):
    """(accepted, tokens) by Python integers, one sequence at a time."""
    B, n, V = q.shape
    p, q = p.float().cpu(), q.float().cpu()
    acc, tok = [], []
    for b in range(B):
        r = 0
        while r < int(lens[b]):
            x = int(draft[b, r])
            # one binary32 product, as the operator's definition has it
            if not (0 <= x < V) or not bool(u[b, r] * q[b, r, x] < p[b, r, x]):
                break
            r += 1
        pr = p[b, r].nan_to_num(0.0).clamp(0, 1)
        rest = pr - q[b, r] if r < int(lens[b]) else pr.clone()
        rest = rest.nan_to_num(0.0).clamp(0, 1)
        w = (rest.double() * 2.0 ** fix).floor().long()
        if int(w.sum()) == 0:
            w = (pr.double() * 2.0 ** fix).floor().long()
        total = int(w.sum())
        t = (int(float(us[b]) * 2 ** 24) * total) >> 24
        new = int((w.cumsum(0) <= t).sum()) if total else -1
        acc.append(r)
        tok.append([int(draft[b, i]) for i in range(r)] + [new] + [-1] * (n - r))
    return torch.tensor(acc, dtype=torch.int32), torch.tensor(tok, dtype=torch.int32)
