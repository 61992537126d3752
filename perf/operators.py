"""Cases of the serving operators next to the expert layer: the paged key/value
cache (written quantised, read back), the attention of new tokens over it, and
the verification of drafted tokens.

Every case has an "op": "write", "read", "attention" or "verify".  With
``own`` false ``run`` is the plain form (elementary torch operations in binary32);
with ``own`` true it calls the library's entry points.
"""
import math

import torch

own = False

WS_BYTES = 64 << 20        # one zeroed workspace, as a serving process keeps
FIX = 38                   # verification sums its weights in units of 2^-38


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the cache write of one decode step, 32 sequences with a token each
        dict(name="write-step", op="write", T=32, H=8, D=128, fp8=True, page=16),
        # the cache write of a long prompt chunk, k and v as views of a packed projection
        dict(name="write-prompt", op="write", T=16384, H=8, D=128, fp8=True, page=64),
        # one sequence read back (a prefix handed to another worker)
        dict(name="read-one", op="read", B=1, kv=777, H=8, D=128, fp8=True, page=16),
        # a batch of ragged sequences read back
        dict(name="read-batch", op="read", B=24, kv=8192, H=8, D=128, fp8=True, page=64),
        # one decode step of a few short sequences: latency
        dict(name="decode-few", op="attention", B=4, q=1, kv=1000, Hq=32, Hkv=8, D=128, fp8=False,
             page=16, window=0, softcap=0.0, causal=True),
        # one decode step of a full batch at long ragged contexts, quantised cache
        dict(name="decode-many-fp8", op="attention", B=64, q=1, kv=16384, Hq=64, Hkv=8, D=128,
             fp8=True, page=64, window=0, softcap=0.0, causal=True),
        # a drafted run of five tokens scored for 16 sequences, quantised cache
        dict(name="draft-scores-fp8", op="attention", B=16, q=5, kv=8192, Hq=32, Hkv=4, D=128,
             fp8=True, page=32, window=0, softcap=0.0, causal=True),
        # prompts of ragged lengths, computed whole; capped scores, sliding window, small heads
        dict(name="prompts-window", op="attention", B=5, q=2500, kv=2500, Hq=24, Hkv=8, D=64,
             fp8=False, page=16, window=1024, softcap=30.0, causal=True),
        # a long chunk of one prompt over what is cached of it
        dict(name="chunk-long", op="attention", B=1, q=4096, kv=16384, Hq=32, Hkv=8, D=128,
             fp8=False, page=64, window=0, softcap=0.0, causal=True),
        # the same kind of chunk over a quantised cache, odd sizes
        dict(name="chunk-fp8", op="attention", B=2, q=1537, kv=8191, Hq=32, Hkv=8, D=128, fp8=True,
             page=128, window=0, softcap=0.0, causal=True),
        # one sequence's drafted tokens verified: latency
        dict(name="verify-one", op="verify", B=1, n=4, V=32768),
        # a batch of drafted runs over a large, odd vocabulary
        dict(name="verify-batch", op="verify", B=96, n=5, V=131071),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "attention", "verify"])
    if op == "verify":
        return dict(op=op, B=_log(rng, 1, 96), n=rng.randint(1, 8), V=_log(rng, 1000, 131071))
    fp8 = rng.random() < 0.6
    page = rng.choice([16, 32, 64, 128, 256])
    D = rng.choice([64, 128, 128])
    if op == "write":
        return dict(op=op, T=_log(rng, 1, 16384), H=rng.choice([1, 2, 4, 5, 8]), D=D, fp8=fp8,
                    page=page)
    if op == "read":
        return dict(op=op, B=_log(rng, 1, 24), kv=_log(rng, 30, 8192),
                    H=rng.choice([1, 2, 4, 5, 8]), D=D, fp8=fp8, page=page)
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    while Hkv * group > 64:
        group -= 1
    form = rng.choice(["decode", "draft", "chunk"])
    window = 0 if rng.random() < 0.7 else _log(rng, 32, 4000)
    softcap = 0.0 if rng.random() < 0.7 else 30.0
    if form == "decode":
        B, q, kv = _log(rng, 1, 64), 1, _log(rng, 100, 16384)
    elif form == "draft":
        B, q, kv = _log(rng, 1, 32), rng.randint(2, 12), _log(rng, 100, 12000)
    else:
        B = rng.randint(1, 3)
        q = _log(rng, 60, 1500)
        kv = q + _log(rng, 1, 8000)
    # unmasked pairs and cached elements stay below the largest listed cases'
    while B * q * kv * Hkv * group > 4096 * 16384 * 28 or B * kv * Hkv > 64 * 16384 * 8:
        kv = max(q, kv // 2)
        B = max(1, B - 1)
    causal = rng.random() < 0.85
    return dict(op=op, B=B, q=q, kv=kv, Hq=Hkv * group, Hkv=Hkv, D=D, fp8=fp8, page=page,
                window=window if causal else 0, softcap=softcap, causal=causal)


# ------------------------------------------------------------------ inputs
def _lens(case):
    """Ragged lengths: the same for every seed (a case's work is fixed), from
    half of the longest on; the first sequence is the longest."""
    B, kv = case["B"], case["kv"]
    return [kv if b == 0 else max(1, kv - (b * 7919) % (kv // 2 + 1)) for b in range(B)]


def _q_lens(case):
    lens = _lens(case)
    if case["q"] >= 64:            # prompts and chunks are ragged too
        return [min(n, max(1, case["q"] - (b * 611) % (case["q"] // 2))) for b, n in enumerate(lens)]
    return [min(n, case["q"]) for n in lens]


def _quantised(x):
    amax = x.float().abs().amax(-1, keepdim=True)
    s = amax / 448.0
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    return (x.float() * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s.squeeze(-1)


def _pages(g, n_pages, H, page, D, fp8):
    """Keys with a few strong channels, values whose rows differ in size."""
    dev = "cuda"
    k = torch.randn(n_pages, H, page, D, device=dev, generator=g, dtype=torch.bfloat16)
    v = torch.randn(n_pages, H, page, D, device=dev, generator=g, dtype=torch.bfloat16)
    k[..., :4] *= 3
    v *= torch.rand(n_pages, H, page, 1, device=dev, generator=g).to(torch.bfloat16) + 0.5
    if not fp8:
        return dict(k=k, v=v, ks=None, vs=None)
    kq, ks = _quantised(k)
    vq, vs = _quantised(v)
    return dict(k=kq.view(torch.uint8), v=vq.view(torch.uint8), ks=ks, vs=vs)


def _stale(st, lens, page):
    """Past the end of a sequence its last page holds whatever was there (NaN here)."""
    mask = torch.zeros(st["k"].shape[0], page, dtype=torch.bool, device="cuda")
    n = torch.tensor(lens, device="cuda")
    last = (n - 1) // page
    ids = st["table"].gather(1, last[:, None])[:, 0].long()
    mask[ids] = torch.arange(page, device="cuda")[None, :] >= (n - last * page)[:, None]
    for name in ("k", "v"):
        st[name].masked_fill_(mask[:, None, :, None], 0x7f if st["ks"] is not None else math.nan)
        if st["ks"] is not None:
            st[name + "s"].masked_fill_(mask[:, None, :], math.nan)


def _tables(g, lens, page, spare=3):
    """Block tables over pages in a random order, and how many pages there are."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    width = max(need)
    at = torch.zeros(len(lens), width, dtype=torch.int64, device="cuda")
    first = 0
    for b, n in enumerate(need):
        at[b, :n] = torch.arange(first, first + n, device="cuda")
        first += n
    return order[at].contiguous(), total


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    op = case["op"]
    st = dict(case=case)
    if op == "verify":
        B, n, V = case["B"], case["n"], case["V"]
        # a draft distribution and a target near it, both peaked like a model's
        base = torch.randn(B, n + 1, V, device="cuda", generator=g) * 2.5
        st["q"] = torch.softmax(base[:, :n] + 0.5 * torch.randn(B, n, V, device="cuda", generator=g), -1)
        st["p"] = torch.softmax(base, -1)
        st["draft"] = torch.multinomial(st["q"].view(B * n, V), 1, generator=g).view(B, n).to(torch.int32)
        st["u"] = torch.rand(B, n, device="cuda", generator=g)
        st["us"] = torch.rand(B, device="cuda", generator=g)
        # every eighth sequence drafted one token less
        st["n"] = torch.tensor([n - (b % 8 == 7) for b in range(B)], dtype=torch.int32, device="cuda")
        st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    H, D, page, fp8 = case.get("H", case.get("Hkv")), case["D"], case["page"], case["fp8"]
    if op == "write":
        T = case["T"]
        n_pages = -(-T // page) + 1
        dt = torch.uint8 if fp8 else torch.bfloat16
        st["k"] = torch.zeros(n_pages, H, page, D, dtype=dt, device="cuda")
        st["v"] = torch.zeros_like(st["k"])
        st["ks"] = torch.zeros(n_pages, H, page, device="cuda") if fp8 else None
        st["vs"] = torch.zeros(n_pages, H, page, device="cuda") if fp8 else None
        # k and v are views of one packed projection [T, 2, H, D]
        kv = torch.randn(T, 2, H, D, device="cuda", generator=g, dtype=torch.bfloat16)
        kv[..., :4] *= 3
        st["new_k"], st["new_v"] = kv[:, 0], kv[:, 1]
        # a sequence fills its pages one after another, and the pages lie in any order
        order = torch.randperm(n_pages, device="cuda", generator=g)
        t = torch.arange(T, device="cuda")
        st["slots"] = (order[t // page] * page + t % page).to(torch.int32)
        st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    lens = _lens(case)
    st["table"], n_pages = _tables(g, lens, page)
    st.update(_pages(g, n_pages, H, page, D, fp8))
    _stale(st, lens, page)
    if op == "read":
        st["cu"], st["rows"] = _cu(lens), sum(lens)
        st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    ql = _q_lens(case)
    st["cu"], st["max_q"], st["max_kv"] = _cu(ql), max(ql), max(lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["new_q"] = torch.randn(sum(ql), case["Hq"], D, device="cuda", generator=g, dtype=torch.bfloat16)
    st["ws"] = torch.zeros(WS_BYTES, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st, op)
    if op == "write":
        return _plain_write(st)
    if op == "read":
        return _plain_read(st)
    if op == "attention":
        return _plain_attention(st)
    return _plain_verify(st)


def _cache_outputs(st):
    if st["ks"] is None:
        return dict(k=st["k"], v=st["v"])
    return dict(k=st["k"].view(torch.float8_e4m3fn), v=st["v"].view(torch.float8_e4m3fn),
                ks=st["ks"], vs=st["vs"])


def _own(st, op):
    from mixture_experts_forward_gb300 import _lib as L
    if op == "write":
        L.kv_write(st["new_k"], st["new_v"], st["slots"], st["k"], st["v"], st["ws"],
                   k_scales=st["ks"], v_scales=st["vs"])
        return _cache_outputs(st)
    if op == "read":
        k, v = L.kv_read(st["k"], st["v"], st["table"], st["cu"], st["rows"], st["ws"],
                         k_scales=st["ks"], v_scales=st["vs"])
        return dict(k=k, v=v)
    if op == "attention":
        c = st["case"]
        out, lse = L.paged_attention(st["new_q"], st["k"], st["v"], st["table"], st["cu"],
                                     st["lens"], st["ws"], max_q=st["max_q"], max_kv=st["max_kv"],
                                     k_scales=st["ks"], v_scales=st["vs"], softcap=c["softcap"],
                                     window=c["window"], causal=c["causal"], lse=True)
        return dict(out=out, lse=lse)
    accepted, tokens = L.verify_draft(st["p"], st["q"], st["draft"], st["u"], st["us"], st["ws"],
                                      draft_lens=st["n"])
    return dict(accepted=accepted, tokens=tokens)


def _plain_write(st):
    page = st["case"]["page"]
    at = st["slots"].long()
    pg, off = at // page, at % page
    for new, cache, scales in ((st["new_k"], st["k"], st["ks"]), (st["new_v"], st["v"], st["vs"])):
        if scales is None:
            cache[pg, :, off] = new
        else:
            codes, s = _quantised(new)
            cache[pg, :, off] = codes.view(torch.uint8)
            scales[pg, :, off] = s
    return _cache_outputs(st)


def _values(pages, scales):
    """Cached rows [..., D] as binary32."""
    if scales is None:
        return pages.float()
    return pages.view(torch.float8_e4m3fn).float() * scales.unsqueeze(-1)


def _plain_read(st):
    page = st["case"]["page"]
    cu = st["cu"].long()
    r = torch.arange(st["rows"], device="cuda")
    b = torch.searchsorted(cu[1:], r, right=True)
    pos = r - cu[b]
    pg, off = st["table"][b, pos // page].long(), pos % page
    out = []
    for pages, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        out.append(_values(pages[pg, :, off], None if scales is None else scales[pg, :, off])
                   .to(torch.bfloat16))
    return dict(k=out[0], v=out[1])


def _plain_attention(st):
    c = st["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    table, cu, lens = st["table"].long(), st["cu"].long(), st["lens"].long()
    B, L, Q = table.shape[0], st["max_kv"], st["max_q"]
    ql = cu[1:] - cu[:-1]

    def gathered(pages, scales):       # [B, Hkv, L, D] binary32, nothing past a length
        x = _values(pages[table], None if scales is None else scales[table])
        x = x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)[:, :, :L]
        past = torch.arange(L, device="cuda")[None, :] >= lens[:, None]
        return x.masked_fill(past[:, None, :, None], 0.0)

    # query rows padded to the longest: [B, Q, Hq, D]
    i = torch.arange(Q, device="cuda")
    real = i[None, :] < ql[:, None]
    row = (cu[:-1, None] + i[None, :]).clamp(max=st["new_q"].shape[0] - 1)
    q = st["new_q"][row].float().reshape(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    s = torch.matmul(q, gathered(st["k"], st["ks"]).transpose(-1, -2))
    s *= 1.0 / math.sqrt(D)
    if c["softcap"] > 0:
        s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    s = s.view(B, Hkv, G, Q, L)
    j = torch.arange(L, device="cuda")
    pos = lens[:, None] - ql[:, None] + i[None, :]
    seen = (j[None, None, :] < lens[:, None, None]) & real[:, :, None]
    if c["causal"]:
        seen &= j[None, None, :] <= pos[:, :, None]
        if c["window"] > 0:
            seen &= j[None, None, :] > pos[:, :, None] - c["window"]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    s.sub_(m).exp_()
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hkv, G * Q, L), gathered(st["v"], st["vs"])).view(B, Hkv, G, Q, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)[real]
    return dict(out=o.to(torch.bfloat16), lse=lse.permute(0, 3, 1, 2).reshape(B, Q, Hq)[real])


def _plain_verify(st):
    p, q, draft, n = st["p"], st["q"], st["draft"].long(), st["n"].long()
    B, N = draft.shape
    i = torch.arange(N, device="cuda")
    px = p[:, :N].gather(2, draft.unsqueeze(2)).squeeze(2)
    qx = q.gather(2, draft.unsqueeze(2)).squeeze(2)
    ok = (st["u"] * qx < px) & (i[None, :] < n[:, None])
    accepted = ok.int().cumprod(1).sum(1)
    b = torch.arange(B, device="cuda")
    pr = p[b, accepted].clamp(0, 1)
    qr = q[b, accepted.clamp(max=N - 1)]
    rest = (pr - torch.where((accepted < n)[:, None], qr, torch.zeros_like(qr))).clamp(0, 1)
    w = (rest * float(1 << FIX)).long()
    w = torch.where((w.sum(1) > 0)[:, None], w, (pr * float(1 << FIX)).long())
    cum = w.cumsum(1)
    total = cum[:, -1]
    u = (st["us"] * float(1 << 24)).long()
    t = (total >> 24) * u + (((total & ((1 << 24) - 1)) * u) >> 24)
    new = (cum <= t[:, None]).sum(1)
    k = torch.arange(N + 1, device="cuda")[None, :]
    padded = torch.cat([draft, draft[:, :1]], 1)
    tokens = torch.where(k < accepted[:, None], padded, torch.full_like(padded, -1))
    tokens = torch.where(k == accepted[:, None], new[:, None], tokens)
    return dict(accepted=accepted.to(torch.int32), tokens=tokens.to(torch.int32))


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "verify":
        B, n, V = case["B"], case["n"], case["V"]
        # the drafted tokens' two probabilities, then the two rows of the draw
        return dict(bytes=B * (n * 16 + 2 * V * 4 + (n + 2) * 4), flops=3 * B * V)
    H, D, fp8 = case.get("H", case.get("Hkv")), case["D"], case["fp8"]
    row = (D + 4) if fp8 else 2 * D          # one cached row of one head
    if op == "write":
        return dict(bytes=case["T"] * (2 * H * (2 * D + row) + 4), flops=case["T"] * 4 * H * D)
    if op == "read":
        n = sum(_lens(case))
        return dict(bytes=2 * n * H * (row + 2 * D), flops=2 * n * H * D)
    lens, ql = _lens(case), _q_lens(case)
    w, causal = case["window"], case["causal"]
    pairs = cached = 0
    for n, m in zip(lens, ql):
        if not causal:
            pairs, cached = pairs + n * m, cached + n
            continue
        lo = n - m + 1                       # keys that the first new token sees, without a window
        span = w if w > 0 else n
        # sum over the rows of min(span, keys up to the row)
        ragged = min(m, max(0, span - lo))
        pairs += (m - ragged) * span + ragged * lo + ragged * (ragged - 1) // 2
        cached += min(n, m + span - 1)
    T = sum(ql)
    return dict(bytes=2 * cached * H * row + T * case["Hq"] * (4 * D + 4),
                flops=4 * D * case["Hq"] * pairs)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return None                          # whole numbers only
    page = case["page"]
    if op == "write":
        out = {}
        for name, new in (("k", st["new_k"]), ("v", st["new_v"])):
            if not case["fp8"]:
                held = torch.zeros(st[name].shape[0] * page, new.shape[1], case["D"],
                                   dtype=torch.float64, device="cuda")
                held[st["slots"].long()] = new.double()
                out[name] = held.view(-1, page, new.shape[1], case["D"]).permute(0, 2, 1, 3)
                continue
            out[name] = None                 # an 8-bit code has no value of its own
            s = torch.zeros(st["ks"].shape[0] * page, new.shape[1], dtype=torch.float64, device="cuda")
            s[st["slots"].long()] = new.double().abs().max(-1).values / 448.0
            out[name + "s"] = s.view(-1, page, new.shape[1]).permute(0, 2, 1)
        return out

    def sequence(name, b, n):                # [n, H, D] in 64 bits
        ids = st["table"][b, : -(-n // page)].long()
        x = st[name][ids]
        x = x.view(torch.float8_e4m3fn).double() if case["fp8"] else x.double()
        if case["fp8"]:
            x = x * st[name + "s"][ids].double()[..., None]
        return x.transpose(1, 2).flatten(0, 1)[:n]

    lens = _lens(case)
    if op == "read":
        return dict(k=torch.cat([sequence("k", b, n) for b, n in enumerate(lens)]),
                    v=torch.cat([sequence("v", b, n) for b, n in enumerate(lens)]))
    T, Hq, D = st["new_q"].shape
    G = Hq // case["Hkv"]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, m) in enumerate(zip(lens, _q_lens(case))):
        k, v = sequence("k", b, n), sequence("v", b, n)
        place = torch.arange(n - m, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None, :]
        hidden = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= key > place
            if case["window"] > 0:
                hidden |= key <= place - case["window"]
        for h in range(Hq):
            x = st["new_q"][first:first + m, h].double() @ k[:, h // G].T / math.sqrt(D)
            if case["softcap"] > 0:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            x = x.masked_fill(hidden, -math.inf)
            lse[first:first + m, h] = torch.logsumexp(x, 1)
            out[first:first + m, h] = torch.softmax(x, 1) @ v[:, h // G]
        first += m
    return dict(out=out, lse=lse)
