"""What each form of moe_paged_attention may be off by, derived from its own roundings
(include/moe.h), against the 64-bit result.

With A = sum_j w_j |v_j| (w the softmax weights, in 64 bits) and delta a bound of a score's
error, an output is off by at most

    |o| 2^-8 + A (r + 2 delta + 2^-15 + steps 2^-22) + floor

  2^-8 |o|   the output's rounding to bf16 (8 significant bits: half a unit is 2^-8 of 2^e)
  r          the roundings of a weight, and of a value where the form rounds it:
               few rows, BF16    two bf16 terms                        2^-16
               few rows, FP8     binary16, then two E4M3 terms         2^-11 + 2^-8 (1 + 2^-7)
               many rows, BF16   bf16                                  2^-8
               many rows, FP8    binary16; scale and value in binary16 2^-11 + 2^-10
  2 delta    a score's error moves a weight and the sum (as serving_reference.attention has it;
             over an FP8 cache query elements below 2^-13 of their row's largest are rounded to
             2^-21 of it besides)
  2^-15      exponentials and the sum of the weights, once each
  steps      products of the tensor core, whose partial sums are truncated
  floor      where a weight's type ends.  Few rows, FP8: half of 2^-13 in units in which the
             largest weight times value scale of the row in that tile of 128 keys is at least 1, on
             each code.  Many rows, FP8: 2^-25 of the row's largest weight, on each value.

The few-row form takes up to 64 rows (new tokens of the longest sequence x query heads per cache
head), 48 over an FP8 cache."""
from __future__ import annotations

import math

import torch

import serving_reference as R

TILE = 128


def _codes(cache, name, b, n):
    """(codes as numbers [n, H, D], scales [n, H]) in float64."""
    pages, sc = getattr(cache, name), getattr(cache, name + "s")
    pos = torch.arange(n, device=pages.device)
    pg = cache.table[b].long()[pos // cache.page]
    x = pages[pg, :, pos % cache.page].view(torch.float8_e4m3fn).double()
    return x, sc[pg, :, pos % cache.page].double()


def few_rows(rows, fp8):
    return rows <= (48 if fp8 else 64)


def rounding(few, fp8):
    if few:
        return 2.0 ** -11 + 2.0 ** -8 * (1 + 2.0 ** -7) if fp8 else 2.0 ** -16
    return 2.0 ** -11 + 2.0 ** -10 if fp8 else 2.0 ** -8


def attention(q, cache, q_lens, kv_lens, *, scale=0.0, softcap=0.0, window=0, causal=True):
    """(out, lse, tol_out, tol_lse) in float64."""
    T, Hq, D = q.shape
    G = Hq // cache.H
    few = few_rows(max(q_lens) * G, cache.fp8)
    r = rounding(few, cache.fp8)
    scale = scale or 1.0 / math.sqrt(D)
    want, want_l, _, _ = R.attention(q, cache, q_lens, kv_lens, scale=scale, softcap=softcap,
                                     window=window, causal=causal)
    tol_o, tol_l = torch.zeros_like(want), torch.zeros_like(want_l)
    at = 0
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        if m == 0 or n == 0:
            at += m
            continue
        k, v = cache.rows("k", b, n), cache.rows("v", b, n)
        if cache.fp8:
            codes, vs = _codes(cache, "v", b, n)
        i = torch.arange(m, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None, :]
        seen = torch.ones(m, n, dtype=torch.bool, device=q.device)
        if causal:
            seen = j <= n - m + i
            if window:
                seen &= j > n - m + i - window
        steps = -(-n // (32 if cache.fp8 and few else 16)) * (2 if few else 1) + D // 16
        for h in range(Hq):
            qh, kh, vh = q[at:at + m, h].double(), k[:, h // G], v[:, h // G]
            x = qh @ kh.T * scale
            delta = (qh.abs() @ kh.abs().T) * abs(scale) * (D + 8) * 2.0 ** -23
            if cache.fp8:
                top = qh.abs().amax(1, keepdim=True)
                low = torch.where(qh.abs() < top * 2.0 ** -13, top * 2.0 ** -21, 0.0 * top)
                delta = delta + low @ kh.abs().T * abs(scale)
            delta = delta.masked_fill(~seen, 0.0).amax(1, keepdim=True)
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                delta = delta + softcap * 2.0 ** -20
            x = x.masked_fill(~seen, -math.inf)
            w = torch.softmax(x, 1).nan_to_num(0.0)
            a = w @ vh.abs()
            floor = torch.zeros_like(a)
            if cache.fp8 and few:
                wv = torch.nn.functional.pad(w * vs[:, h // G], (0, -n % TILE))
                most = wv.view(m, -1, TILE).amax(2, keepdim=True).expand(-1, -1, TILE).reshape(m, -1)[:, :n]
                floor = 2.0 ** -14 * ((most * seen) @ codes[:, h // G].abs())
            elif cache.fp8:
                floor = 2.0 ** -25 * w.amax(1, keepdim=True) * (seen.double() @ vh.abs())
            o = want[at:at + m, h]
            tol_o[at:at + m, h] = (o.abs() * 2.0 ** -8 +
                                   a * (r + 2 * delta + 2.0 ** -15 + steps * 2.0 ** -22) + floor) * 1.01
            tol_l[at:at + m, h] = delta[:, 0] + 2.0 ** -20 * (
                1 + want_l[at:at + m, h].abs().nan_to_num(0, 0, 0))
        at += m
    return want, want_l, tol_o, tol_l


# ------------------------------------------------------------------ a case whose roundings agree
def weight(few, fp8):
    """A weight that the form's (first) type rounds down by nearly all of half a unit: bf16, or
    E4M3's 4 significant bits."""
    return 0.5 + (2.0 ** -5 - 2.0 ** -10 if few and fp8 else 2.0 ** -9 - 2.0 ** -14)


def same_sign_case(q_len, G, D, fp8, device, n=2001):
    """(q, cache, scale): the first key's weight is 1 of the reference's unit and each other's is
    weight(), whose rounding lowers every term alike; the values are positive, so nothing
    cancels, and their largest is 1.75, so that a quantised row's scale is a power of two."""
    q = torch.zeros(q_len, G, D, dtype=torch.bfloat16, device=device)
    q[..., 0] = 1.0
    k = torch.zeros(n, 1, D, dtype=torch.bfloat16)
    k[1:, :, 0] = -1.0
    g = torch.Generator().manual_seed(0)
    v = (1.0 + 0.75 * torch.rand(1, 1, D, generator=g)).to(torch.bfloat16)
    v[..., 0] = 1.75
    c = R.Paged([k], [v.expand(n, 1, D)], 64, fp8, device=device)
    return q, c, -math.log(weight(few_rows(q_len * G, fp8), fp8))
