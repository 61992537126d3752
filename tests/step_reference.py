"""Plain forms, in 64 bits and on the CPU, of the operators between the serving calls: the step's
plan and the release of pages, rotary positions, the few-token expert layer and the logits.  Written
from the definitions in include/moe.h, token by token."""
import math

import torch


def ceil_div(a, b):
    return -(-a // b)


class Pages:
    """The state of moe_page_state as Python lists."""

    def __init__(self, table, held, free, count):
        self.table, self.held = [list(r) for r in table], list(held)
        self.free, self.count = list(free), count

    def plan(self, lens, news, rows, page, num_pages):
        """(slots, positions, cu_q, kv_lens, faults) of moe_plan_step."""
        room = (len(self.table[0]) if self.table else 0) * page
        slots, positions, cu, kv, faults = [-1] * rows, [0] * rows, [0], [], 0
        count, taken, at, exhausted = self.count, 0, 0, 0
        for b, (n, m) in enumerate(zip(lens, news)):
            bad = (n < 0 or m < 0 or not 0 <= self.held[b] <= len(self.table[b]) or n + m > room or
                   self.held[b] * page < n)
            fits = at + max(m, 0) <= rows or m <= 0
            need = 0 if bad else max(0, ceil_div(n + m, page) - self.held[b])
            exhausted += need                                # (also of one that is past the rows)
            served = not bad and fits and (need == 0 or exhausted <= count)
            faults += bad or not fits
            if served:
                for _ in range(need):
                    taken += 1
                    self.table[b][self.held[b]] = self.free[count - taken]
                    self.held[b] += 1
            for i in range(max(m, 0)):
                if at + i >= rows:
                    break
                positions[at + i] = n + i if n >= 0 else 0
                if served:
                    page_id = self.table[b][(n + i) // page]
                    if 0 <= page_id < num_pages:
                        slots[at + i] = page_id * page + (n + i) % page
                    else:
                        faults += 1
            at = min(rows, at + max(m, 0))
            cu.append(at)
            kv.append(n + m if served else 0)
        self.count = count - taken
        return slots, positions, cu, kv, faults

    def release(self, keep, page):
        out = []
        for b, k in enumerate(keep):
            kept = self.held[b] if k < 0 else min(self.held[b], ceil_div(k, page))
            for j in range(kept, self.held[b]):
                out.append(self.table[b][j])
                self.table[b][j] = -1
            self.held[b] = kept
        for j, page_id in enumerate(reversed(out)):
            self.free[self.count + j] = page_id
        self.count += len(out)


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    out = []
    for i in range(rot // 2):
        t = base ** (-2.0 * i / rot)
        keep = 1.0
        if scaling == "linear":
            keep = 0.0
        elif scaling == "turns":
            keep = (original * t / (2 * math.pi) - low) / (high - low)
        elif scaling == "index":
            def index(turns):
                return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo = max(math.floor(index(high)), 0)
            hi = min(math.ceil(index(low)), rot - 1)
            keep = 1 - (i - lo) / ((hi - lo) if hi > lo else 0.001)
        keep = min(1.0, max(0.0, keep))
        out.append(t * keep + t / factor * (1 - keep))
    return out


def rotated(x, positions, theta, interleaved, amplitude=1.0):
    """(values, |a| + |b| of each element's pair) in 64 bits of x [T, H, D]."""
    x = x.double()
    rot = 2 * len(theta)
    angle = positions.double()[:, None] * torch.tensor(theta, dtype=torch.float64)
    c, s = torch.cos(angle)[:, None] * amplitude, torch.sin(angle)[:, None] * amplitude
    if interleaved:
        first, second = slice(0, rot, 2), slice(1, rot, 2)
    else:
        first, second = slice(0, rot // 2), slice(rot // 2, rot)
    out, size = x.clone(), torch.zeros_like(x)
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * c - b * s, a * s + b * c
    size[..., first] = size[..., second] = (a.abs() + b.abs()) * abs(amplitude)
    return out, size


def few(x, ids, weights, up, down, fp8):
    """(out, bound on the error before the last rounding) in 64 bits.  up [E, 2I, H] and down [E, H, I]
    as values, ids and weights [T, k].  The bound counts: a term of 2^-23 for each 16 products that the
    tensor core adds (and 8 more), the roundings of h (2^-11 of it over FP8 weights, with 2^-39 of
    its block's largest; 2^-16 over BF16), x's own over FP8 (2^-39 of its block's largest), 2^-20 for
    silu and the weights."""
    T, H = x.shape
    I = down.shape[2]
    x = x.double()
    u23 = 2.0 ** -23
    out, err = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        xe = torch.zeros(H, dtype=torch.float64)
        if fp8:
            xe = x[t].abs().view(-1, 128).amax(1).repeat_interleave(128) * 2.0 ** -39
        for j in range(ids.shape[1]):
            e, w = int(ids[t, j]), float(weights[t, j])
            gu = up[e] @ x[t]
            size = up[e].abs() @ x[t].abs() * (H / 16 + 8) * u23 + up[e].abs() @ xe
            g, u, ge, ue = gu[:I], gu[I:], size[:I], size[I:]
            silu = g / (1 + torch.exp(-g))
            h = silu * u
            he = 1.1 * ge * (u.abs() + ue) + silu.abs() * ue + h.abs() * 2.0 ** -20
            if fp8:
                he = he + h.abs() * 2.0 ** -11 + h.abs().view(-1, 128).amax(1).repeat_interleave(128) * 2.0 ** -39
            else:
                he = he + h.abs() * 2.0 ** -16
            out[t] += w * (down[e] @ h)
            err[t] += w * (down[e].abs() @ (he + h.abs() * ((I / 16 + 8) * u23 + 2.0 ** -20)))
    return out, err


def logits(x, history=None, history_lens=None, prompt_lens=None, draft=None, repetition=None,
           presence=None, frequency=None, temperature=None, bias_tokens=None, bias_values=None,
           mask=None, probabilities=True):
    """moe_adjust_logits in 64 bits; x [B, m, V], the rest as lists or CPU tensors."""
    B, m, V = x.shape
    out = torch.zeros(B, m, V, dtype=torch.float64)
    at = lambda v, b, none: none if v is None else float(v[b])  # noqa: E731
    for b in range(B):
        for i in range(m):
            l = x[b, i].double().clone()
            l[torch.isnan(l)] = -math.inf
            said = torch.zeros(V, dtype=torch.float64)
            count = torch.zeros(V, dtype=torch.float64)
            if history is not None:
                n = history.shape[1] if history_lens is None else int(history_lens[b])
                p = 0 if prompt_lens is None else int(prompt_lens[b])
                for place, v in enumerate(history[b, :n].tolist()):
                    if 0 <= v < V:
                        (said if place < p else count)[v] += 1
            if draft is not None:
                for v in draft[b, :i].tolist():
                    if 0 <= v < V:
                        count[v] += 1
            rep = at(repetition, b, 1.0)
            old = (said + count) > 0
            l[old] = torch.where(l[old] > 0, l[old] / rep, l[old] * rep)
            l = l - at(frequency, b, 0.0) * count - at(presence, b, 0.0) * (count > 0)
            if bias_tokens is not None:
                for v, add in zip(bias_tokens[b].tolist(), bias_values[b].tolist()):
                    if 0 <= v < V and l[v] > -math.inf:
                        l[v] += add
            l[torch.isnan(l)] = -math.inf
            if mask is not None:
                words = mask[b, i] if mask.dim() == 3 else mask[b]
                bits = (words[:, None] >> torch.arange(32)) & 1
                l[bits.flatten()[:V] == 0] = -math.inf
            if not probabilities:
                out[b, i] = l
                continue
            top = l.max()
            temp = at(temperature, b, 1.0)
            if top == -math.inf:
                continue
            if temp == 0:
                out[b, i, int((l == top).nonzero()[0])] = 1
            elif top == math.inf:
                out[b, i] = (l == top).double() / (l == top).sum()
            else:
                e = torch.exp((l - top) / temp)
                out[b, i] = e / e.sum()
    return out
