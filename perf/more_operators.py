"""Cases of the serving operators that stand between the cache, the attention, the experts and
the verification of one decode step: the step's plan (block tables and slot maps from request
lengths), rotary positions written into the paged cache, the whole expert layer for a few tokens,
and penalties, biases and grammar masks on logits.

Every case has an "op": "plan", "rotary", "few" or "logits".  With ``own`` false ``run`` is
the plain form (elementary torch operations in binary32, angles of positions in binary64); with
``own`` true it calls the library's entry points.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the plan of one decode step of a few sequences: latency
        dict(name="plan-few", op="plan", B=8, new=1, kv=4000, page=16, short=False),
        # a full batch: prompt chunks beside drafted runs and single tokens
        dict(name="plan-mixed", op="plan", B=1024, new=128, kv=8192, page=64, short=False),
        # one decode step's queries and keys rotated, keys and values cached quantised: latency
        dict(name="rotary-step-fp8", op="rotary", T=32, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, cache="fp8", page=16, scaling="none", far=8192),
        # a long prompt chunk, all three as views of one packed projection
        dict(name="rotary-prompt-fp8", op="rotary", T=16384, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, cache="fp8", page=64, scaling="turns", far=131072),
        # part of small heads, pairs side by side, BF16 cache, positions far beyond the trained ones
        dict(name="rotary-long-bf16", op="rotary", T=5003, Hq=24, Hkv=8, D=64, rot=32,
             interleaved=True, cache="bf16", page=16, scaling="index", far=1000000),
        # one token through a small expert layer: latency
        dict(name="few-one-fp8", op="few", T=1, H=2048, I=512, E=256, k=8, fp8=True, softcap=30.0),
        # a decode batch whose tokens go to about a hundred experts
        dict(name="few-batch-fp8", op="few", T=16, H=2048, I=512, E=256, k=8, fp8=True, softcap=30.0),
        # one token through two large BF16 experts
        dict(name="few-one-bf16", op="few", T=1, H=4096, I=1024, E=8, k=2, fp8=False, softcap=0.0),
        # one drafted run of five tokens, many BF16 experts
        dict(name="few-drafts-bf16", op="few", T=5, H=4096, I=1408, E=48, k=6, fp8=False, softcap=0.0),
        # one sequence's next token: latency
        dict(name="logits-one", op="logits", B=1, n=0, V=32768, hist=700, nb=16, bf16=False, probs=True),
        # the probabilities of a batch of drafted runs over a large, odd vocabulary
        dict(name="logits-drafts", op="logits", B=96, n=5, V=131071, hist=4000, nb=64, bf16=False,
             probs=True),
        # a decode batch's adjusted logits, from BF16
        dict(name="logits-batch-bf16", op="logits", B=200, n=0, V=100003, hist=8000, nb=64, bf16=True,
             probs=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rotary", "few", "logits"])
    if op == "plan":
        B, new = _log(rng, 1, 1024), rng.choice([1, 2, 5, 33, 128])
        return dict(op=op, B=B, new=new, kv=_log(rng, 30, 8192), page=rng.choice([16, 32, 64, 128, 256]),
                    short=rng.random() < 0.3)
    if op == "rotary":
        D, Hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 5, 8])
        return dict(op=op, T=_log(rng, 1, 16384), Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv, D=D,
                    rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= D]),
                    interleaved=rng.random() < 0.4, cache=rng.choice(["fp8", "fp8", "bf16", "none"]),
                    page=rng.choice([16, 32, 64, 128, 256]),
                    scaling=rng.choice(["none", "linear", "turns", "index"]),
                    far=_log(rng, 100, 1000000))
    if op == "few":
        fp8 = rng.random() < 0.6
        H = 128 * rng.randint(4, 32) + (0 if fp8 or rng.random() < 0.5 else 64)
        I, E = 128 * rng.randint(1, 16), _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 16)
        while T * k * 3 * I * H > 30 * 3 * 1408 * 4096 and T > 1:
            T -= 1
        while E * 3 * I * H * (1 if fp8 else 2) > 48 * 3 * 1408 * 4096 * 2 and E > k:
            E = max(k, E // 2)
        return dict(op=op, T=T, H=H, I=I, E=E, k=k, fp8=fp8, softcap=rng.choice([0.0, 30.0]))
    B, n, V = _log(rng, 1, 200), rng.choice([0, 0, 1, 3, 5, 8]), _log(rng, 1000, 131071)
    while B * (n + 1) * V > 96 * 6 * 131071:
        B -= 1
    return dict(op=op, B=B, n=n, V=V, hist=_log(rng, 10, 8000), nb=rng.choice([0, 7, 64, 300]),
                bf16=rng.random() < 0.4, probs=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs
def _plan_lens(case):
    """Ragged lengths, the same for every seed (a case's work is fixed) but for their order: every
    fourth sequence brings up to `new` tokens, the others one or a short run."""
    B, kv, new = case["B"], case["kv"], case["new"]
    lens = [(b * 7919 + 13) % kv for b in range(B)]
    news = [1 + (b * 611) % new if b % 4 == 0 else 1 + b % min(new, 5) for b in range(B)]
    return lens, news


def _pages_of(n, page):
    return -(-n // page)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_plan(case, g, st):
    B, page = case["B"], case["page"]
    lens, news = _plan_lens(case)
    order = torch.randperm(B, device="cuda", generator=g)
    st["lens"], st["new"] = _i32(lens)[order].contiguous(), _i32(news)[order].contiguous()
    held = [_pages_of(n, page) for n in lens]
    st["held"] = _i32(held)[order].contiguous()
    grow = sum(_pages_of(n + m, page) - h for n, m, h in zip(lens, news, held))
    # the free pages are enough, or only for some of the sequences
    free = max(1, grow * 2 // 3) if case["short"] else grow + 5
    total = sum(held) + free
    st["num_pages"] = total
    # whole tables, with room for what a sequence may grow to
    width = max(_pages_of(n + m, page) for n, m in zip(lens, news)) + 2
    ids = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    first = torch.cumsum(st["held"].long(), 0) - st["held"].long()
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col).clamp(max=total - 1)
    st["table"] = torch.where(col < st["held"].long()[:, None], ids[at], torch.full_like(ids[at], -1))
    st["free"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    st["free"][:free] = ids[sum(held):]
    st["count"] = _i32([free])
    # the batch is padded to a multiple of 64 rows
    st["rows"] = -(-sum(news) // 64) * 64
    st["most"] = max(_pages_of(n + m, page) - h for n, m, h in zip(lens, news, held))
    st["keep"] = st["lens"].clone()       # every new token is refused: the pages go back
    st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")


ROPE_FACTOR, ROPE_ORIGINAL, ROPE_LOW, ROPE_HIGH, ROPE_BASE = 8.0, 8192, 1.0, 4.0, 500000.0


def _frequencies(case):
    """Radians a position of each pair, as Python floats."""
    rot, kind = case["rot"], case["scaling"]
    base = 10000.0 if kind == "none" else ROPE_BASE
    theta = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "none":
        return theta
    if kind == "linear":
        return [t / ROPE_FACTOR for t in theta]
    out = []
    if kind == "turns":       # blended by the turns that a pair makes over the trained context
        for t in theta:
            keep = min(1.0, max(0.0, (ROPE_ORIGINAL * t / (2 * math.pi) - ROPE_LOW) / (ROPE_HIGH - ROPE_LOW)))
            out.append(t * keep + t / ROPE_FACTOR * (1 - keep))
        return out
    # blended by the pair's index between those that make ROPE_HIGH and ROPE_LOW turns
    def index(turns):
        return rot * math.log(ROPE_ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(index(ROPE_HIGH)), 0), min(math.ceil(index(ROPE_LOW)), rot - 1)
    hi = hi if hi > lo else lo + 0.001
    for i, t in enumerate(theta):
        keep = 1 - min(1.0, max(0.0, (i - lo) / (hi - lo)))
        out.append(t * keep + t / ROPE_FACTOR * (1 - keep))
    return out


def _prepare_rotary(case, g, st):
    T, Hq, Hkv, D, page = (case[n] for n in ("T", "Hq", "Hkv", "D", "page"))
    # q, k and v are views of one packed projection; a few channels are strong
    packed = torch.randn(T, Hq + 2 * Hkv, D, device="cuda", generator=g, dtype=torch.bfloat16)
    packed[..., :4] *= 3
    st["q"], st["k"], st["v"] = packed.split([Hq, Hkv, Hkv], dim=1)
    theta = _frequencies(case)
    st["theta"] = torch.tensor(theta, dtype=torch.float64, device="cuda")
    # the handle: turns a position, in units of 2^-64
    fixed = [int(t / (2 * math.pi) * 2.0 ** 64) for t in theta]
    st["table"] = torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in fixed], dtype=torch.int64,
                               device="cuda")
    st["amplitude"] = 0.1 * math.log(ROPE_FACTOR) + 1.0 if case["scaling"] == "index" else 1.0
    # chunks of sequences that start anywhere below `far`
    chunk = max(1, T // 5)
    start = torch.randint(0, case["far"], (T // chunk + 1,), device="cuda", generator=g)
    t = torch.arange(T, device="cuda")
    st["positions"] = (start[t // chunk] + t % chunk).to(torch.int32)
    st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    st["ck"] = st["cv"] = st["ks"] = st["vs"] = None
    if case["cache"] == "none":
        return
    n_pages = _pages_of(T, page) + 1
    order = torch.randperm(n_pages, device="cuda", generator=g)
    st["slots"] = (order[t // page] * page + t % page).to(torch.int32)
    if T > 20:
        st["slots"][T - 3:] = -1          # the padded end of a batch
    fp8 = case["cache"] == "fp8"
    dt = torch.uint8 if fp8 else torch.bfloat16
    st["ck"] = torch.zeros(n_pages, Hkv, page, D, dtype=dt, device="cuda")
    st["cv"] = torch.zeros_like(st["ck"])
    if fp8:
        st["ks"] = torch.zeros(n_pages, Hkv, page, device="cuda")
        st["vs"] = torch.zeros(n_pages, Hkv, page, device="cuda")


def _prepare_few(case, g, st):
    T, H, I, E = (case[n] for n in ("T", "H", "I", "E"))

    def weights(rows, cols):
        if not case["fp8"]:
            return torch.randn(E, rows, cols, device="cuda", generator=g, dtype=torch.bfloat16) / cols ** 0.5, None
        w = torch.randn(E, rows, cols, device="cuda", generator=g, dtype=torch.bfloat16)
        w = w.mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s = (torch.rand(E, rows // 128, cols // 128, device="cuda", generator=g) + 0.5) / (100 * cols ** 0.5)
        return w.view(torch.uint8), s

    st["up"], st["up_s"] = weights(2 * I, H)
    st["down"], st["down_s"] = weights(H, I)
    x = torch.randn(T, H, device="cuda", generator=g)
    x[:, :: 97] *= 20                     # a few channels are strong
    st["x"] = x.to(torch.bfloat16)
    # popular experts: the tokens share some
    bias = 1.5 * torch.log(1.0 / torch.arange(1, E + 1, device="cuda").float())
    bias = bias[torch.randperm(E, device="cuda", generator=g)]
    st["logits"] = torch.randn(T, E, device="cuda", generator=g) + 0.3 * bias
    st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    st["ws"] = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")


def _prepare_logits(case, g, st):
    B, m, V = case["B"], case["n"] + 1, case["V"]
    x = torch.randn(B, m, V, device="cuda", generator=g) * 2.5
    st["logits"] = x.to(torch.bfloat16) if case["bf16"] else x
    # tokens come from a peaked distribution, so a history repeats itself
    def tokens(*shape):
        u = torch.rand(*shape, device="cuda", generator=g)
        return (u * u * u * V).to(torch.int32).clamp(max=V - 1)
    b = torch.arange(B, device="cuda")
    st["hist"] = tokens(B, case["hist"])
    st["hist_lens"] = (case["hist"] - (b * 37) % (case["hist"] // 2 + 1)).to(torch.int32)
    st["prompt_lens"] = (st["hist_lens"] * 2 // 3).to(torch.int32)
    st["draft"] = tokens(B, m - 1) if m > 1 else None
    rnd = lambda lo, hi: torch.rand(B, device="cuda", generator=g) * (hi - lo) + lo  # noqa: E731
    st["repetition"], st["presence"], st["frequency"] = rnd(1.0, 1.3), rnd(0.0, 0.6), rnd(0.0, 0.3)
    st["temperature"] = rnd(0.6, 1.2)
    st["temperature"][5::8] = 0.0         # some are decoded greedily
    st["bias_t"] = st["bias_v"] = None
    if case["nb"]:
        st["bias_t"] = tokens(B, case["nb"])
        st["bias_v"] = torch.randn(B, case["nb"], device="cuda", generator=g)
    # a third of the sequences follow a grammar that leaves about one token in 64
    words = (V + 31) // 32
    bits = lambda: torch.randint(-2 ** 31, 2 ** 31, (B, m, words), device="cuda", generator=g)  # noqa: E731
    mask = bits()
    for _ in range(5):
        mask &= bits()
    mask[b % 3 != 1] = -1
    if B > 8:
        mask[7, -1] = 0                   # and one row is left with nothing
    st["mask"] = mask.to(torch.int32)
    st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    st = dict(case=case)
    {"plan": _prepare_plan, "rotary": _prepare_rotary, "few": _prepare_few,
     "logits": _prepare_logits}[case["op"]](case, g, st)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st, op)
    return {"plan": _plain_plan, "rotary": _plain_rotary, "few": _plain_few,
            "logits": _plain_logits}[op](st)


def _own(st, op):
    from mixture_experts_forward_gb300 import _lib as L
    c = st["case"]
    if op == "plan":
        slots, positions, cu, kv = L.plan_step(st["lens"], st["new"], st["table"], st["held"], st["free"],
                                               st["count"], st["rows"], c["page"], st["num_pages"], st["ws"])
        L.release_pages(st["keep"], st["table"], st["held"], st["free"], st["count"], c["page"], st["ws"])
        return _plan_outputs(st, slots, positions, cu, kv)
    if op == "rotary":
        if c["cache"] == "none":
            q, k = L.rotary(st["q"], st["k"], st["positions"], st["table"], interleaved=c["interleaved"],
                            amplitude=st["amplitude"])
            return dict(q=q, k=k)
        q = L.rotary_write(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["table"], st["ck"],
                           st["cv"], st["ws"], k_scales=st["ks"], v_scales=st["vs"],
                           interleaved=c["interleaved"], amplitude=st["amplitude"])
        return _rotary_outputs(st, q)
    if op == "few":
        a = L.forward_args(dtype=L.DTYPE_FP8 if c["fp8"] else L.DTYPE_BF16, M=c["T"], K=c["H"], N=c["I"],
                           E=c["E"], top_k=c["k"], softcap=c["softcap"], logits=st["logits"], x=st["x"],
                           w=st["up"], w_scales=st["up_s"], w2=st["down"], w2_scales=st["down_s"], gated=1)
        return dict(out=L.forward_few(a, st["out"], st["ws"]))
    return dict(out=L.adjust_logits(
        st["logits"], st["ws"], history=st["hist"], history_lens=st["hist_lens"],
        prompt_lens=st["prompt_lens"], draft=st["draft"], repetition=st["repetition"],
        presence=st["presence"], frequency=st["frequency"], temperature=st["temperature"],
        bias_tokens=st["bias_t"], bias_values=st["bias_v"], mask=st["mask"], probabilities=c["probs"]))


def _plan_outputs(st, slots, positions, cu, kv):
    return dict(slots=slots, positions=positions, cu=cu, kv=kv, table=st["table"], held=st["held"],
                free=st["free"], count=st["count"])


def _plain_plan(st):
    page, rows, most = st["case"]["page"], st["rows"], st["most"]
    lens, new, held = st["lens"].long(), st["new"].long(), st["held"].long()
    table, free, count = st["table"], st["free"], st["count"].long()
    B, width = table.shape
    # pages that each sequence needs, and who gets them
    need = ((lens + new + page - 1) // page - held).clamp(min=0)
    upto = torch.cumsum(need, 0)
    served = (need == 0) | (upto <= count)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(new, 0)])
    r = torch.arange(rows, device="cuda")
    b = torch.searchsorted(cu[1:], r, right=True).clamp(max=B - 1)
    real = r < cu[B]
    pos = torch.where(real, lens[b] + r - cu[b], torch.zeros_like(r))
    entry = pos // page
    ranked = upto[b] - need[b] + entry - held[b]
    fresh = free[(count - 1 - ranked).clamp(0, free.shape[0] - 1)].long()
    ids = torch.where(entry < held[b], table[b, entry.clamp(max=width - 1)].long(), fresh)
    slots = torch.where(real & served[b], ids * page + pos % page, torch.full_like(r, -1))
    kv = torch.where(served, lens + new, torch.zeros_like(lens))
    # the new pages enter the tables
    j = torch.arange(max(most, 1), device="cuda")
    taken = (j < need[:, None]) & served[:, None]
    rank = (upto - need)[:, None] + j
    seq, col = torch.nonzero(taken, as_tuple=True)
    table[seq, held[seq] + col] = free[count - 1 - rank[seq, col]]
    held = held + torch.where(served, need, torch.zeros_like(need))
    count = count - torch.where(served, need, torch.zeros_like(need)).sum()
    # what lies past `keep` goes back, the last page first
    kept = torch.minimum(held, (st["keep"].long() + page - 1) // page)
    give = held - kept
    upto = torch.cumsum(give, 0)
    j = torch.arange(width, device="cuda")
    seq, col = torch.nonzero(j < give[:, None], as_tuple=True)
    rank = upto[seq] - give[seq] + col
    free[count + upto[-1] - 1 - rank] = table[seq, kept[seq] + col]
    table[seq, kept[seq] + col] = -1
    st["held"].copy_(kept)
    st["count"].copy_(count + upto[-1])
    i32 = torch.int32
    return _plan_outputs(st, slots.to(i32), pos.to(i32), cu.to(i32), kv.to(i32))


def _quantised(x):
    """E4M3 codes and scales of binary32 rows."""
    s = x.abs().amax(-1, keepdim=True) / 448.0
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    return (x * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s.squeeze(-1)


def _rotary_outputs(st, q):
    if st["ks"] is None:
        return dict(q=q, k=st["ck"], v=st["cv"])
    return dict(q=q, k=st["ck"].view(torch.float8_e4m3fn), v=st["cv"].view(torch.float8_e4m3fn),
                ks=st["ks"], vs=st["vs"])


def _plain_rotary(st):
    c = st["case"]
    rot, half = c["rot"], c["rot"] // 2
    angle = st["positions"].double()[:, None] * st["theta"]
    cos = (torch.cos(angle) * st["amplitude"]).float()[:, None]
    sin = (torch.sin(angle) * st["amplitude"]).float()[:, None]

    def rotated(x):
        x = x.float()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([turned, x[..., rot:]], -1)

    q, k = rotated(st["q"]).to(torch.bfloat16), rotated(st["k"])
    if c["cache"] == "none":
        return dict(q=q, k=k.to(torch.bfloat16))
    real = st["slots"] >= 0
    at = st["slots"][real].long()
    pg, off = at // c["page"], at % c["page"]
    for new, cache, scales in ((k, st["ck"], st["ks"]), (st["v"].float(), st["cv"], st["vs"])):
        if scales is None:
            cache[pg, :, off] = new[real].to(torch.bfloat16)
        else:
            codes, s = _quantised(new[real])
            cache[pg, :, off] = codes.view(torch.uint8)
            scales[pg, :, off] = s
    return _rotary_outputs(st, q)


def _plain_few(st):
    c = st["case"]
    T, H, I, k = c["T"], c["H"], c["I"], c["k"]
    z = st["logits"]
    if c["softcap"] > 0:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    z, ids = torch.sort(z, dim=1, descending=True, stable=True)
    z, ids = z[:, :k], ids[:, :k]
    w = torch.exp(z - z[:, :1])
    w = w / w.sum(1, keepdim=True)

    def chosen(weights, scales):           # [T, k, rows, cols] binary32
        if scales is None:
            return weights[ids].float()
        x = weights[ids].view(torch.float8_e4m3fn).float()
        s = scales[ids]
        return x.view(*x.shape[:2], s.shape[2], 128, s.shape[3], 128).mul_(s[:, :, :, None, :, None]).view(x.shape)

    gu = torch.matmul(chosen(st["up"], st["up_s"]), st["x"].float()[:, None, :, None]).squeeze(-1)
    gate, up = gu[..., :I], gu[..., I:]
    h = gate / (1 + torch.exp(-gate)) * up
    y = torch.matmul(chosen(st["down"], st["down_s"]), h[..., None]).squeeze(-1)
    return dict(out=(w[..., None] * y).sum(1).to(torch.bfloat16))


def _plain_logits(st):
    c = st["case"]
    B, m, V = c["B"], c["n"] + 1, c["V"]
    l = st["logits"].float()
    pos = torch.arange(c["hist"], device="cuda")
    in_prompt = pos < st["prompt_lens"][:, None]
    in_output = ~in_prompt & (pos < st["hist_lens"][:, None])
    hist = st["hist"].long()
    prompt = torch.zeros(B, V, device="cuda").scatter_add_(1, hist, in_prompt.float())
    count = torch.zeros(B, V, device="cuda").scatter_add_(1, hist, in_output.float())
    count = count[:, None].expand(B, m, V)
    if m > 1:
        # position i counts the drafts before it
        i, j = torch.arange(m, device="cuda")[:, None], torch.arange(m - 1, device="cuda")[None, :]
        before = (j < i).float().expand(B, m, m - 1)
        count = count.clone().scatter_add_(2, st["draft"].long()[:, None].expand(B, m, m - 1).contiguous(), before)
    col = lambda t: t[:, None, None]  # noqa: E731
    seen = (prompt[:, None] > 0) | (count > 0)
    l = torch.where(seen, torch.where(l > 0, l / col(st["repetition"]), l * col(st["repetition"])), l)
    l = l - col(st["frequency"]) * count - col(st["presence"]) * (count > 0)
    if st["bias_t"] is not None:
        l = l + torch.zeros(B, V, device="cuda").scatter_add_(1, st["bias_t"].long(), st["bias_v"])[:, None]
    v = torch.arange(V, device="cuda")
    allowed = (st["mask"][..., v // 32] >> (v % 32).to(torch.int32)) & 1
    l = torch.where(allowed > 0, l, torch.full_like(l, -math.inf))
    if not c["probs"]:
        return dict(out=l)
    top = l.amax(-1, keepdim=True)
    some = top > -math.inf
    temp = col(st["temperature"])
    e = torch.exp((l - torch.where(some, top, torch.zeros_like(top))) / torch.where(temp > 0, temp, torch.ones_like(temp)))
    p = e / torch.where(some, e.sum(-1, keepdim=True), torch.ones_like(top))
    # greedy: all on the largest (the lowest token of equals)
    at = torch.where(l == top, v, torch.full_like(v, V)).amin(-1, keepdim=True)
    return dict(out=torch.where(temp > 0, p, ((v == at) & some).float()))


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "plan":
        lens, news = _plan_lens(case)
        B, page = case["B"], case["page"]
        rows = -(-sum(news) // 64) * 64
        held = [_pages_of(n, page) for n in lens]
        grow = sum(_pages_of(n + m, page) - h for n, m, h in zip(lens, news, held))
        # lengths in, rows out, the open pages' entries, the pages taken and given back
        return dict(bytes=4 * (3 * B + 2 * rows + 2 * B + 1 + B + 6 * grow + 4 * B), flops=4 * rows)
    if op == "rotary":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        row = D + 4 if case["cache"] == "fp8" else 2 * D
        n = T * Hq * 4 * D + T * Hkv * (2 * D + row) * (1 if case["cache"] == "none" else 2)
        return dict(bytes=n + 8 * T, flops=T * (Hq + Hkv) * 3 * case["rot"])
    if op == "few":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        # the experts that T tokens reach, were each as likely as the others
        reached = E * (1 - (1 - k / E) ** T)
        return dict(bytes=reached * 3 * I * H * (1 if case["fp8"] else 2) + T * (4 * E + 4 * H),
                    flops=T * k * 6 * I * H)
    rows, V = case["B"] * (case["n"] + 1), case["V"]
    return dict(bytes=rows * V * (6 if case["bf16"] else 8) + rows * ((V + 31) // 32) * 4 +
                case["B"] * (3 * case["hist"] + 8 * case["nb"]), flops=rows * V * 8)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None                          # whole numbers only
    st = prepare(case, seed)
    if op == "rotary":
        return _exact_rotary(case, st)
    if op == "few":
        return _exact_few(case, st)
    return _exact_logits(case, st)


def _exact_rotary(case, st):
    rot, D, page = case["rot"], case["D"], case["page"]
    angle = torch.outer(st["positions"].double(), st["theta"])
    turn = torch.polar(torch.full_like(angle, st["amplitude"]), angle)     # complex [T, rot/2]
    # which elements make a pair
    i = torch.arange(rot // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)

    def rotated(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k, v = rotated(st["q"]), rotated(st["k"]), st["v"].double()
    if case["cache"] == "none":
        return dict(q=q, k=k)
    real = st["slots"] >= 0
    at, n = st["slots"][real].long(), st["ck"].shape[0]

    def placed(rows):                        # [pages, heads, page, ...]
        held = torch.zeros(n * page, *rows.shape[1:], dtype=torch.float64, device="cuda")
        held[at] = rows[real]
        return held.view(n, page, *rows.shape[1:]).transpose(1, 2)

    if case["cache"] == "bf16":
        return dict(q=q, k=placed(k), v=placed(v))
    # an 8-bit code has no value of its own
    return dict(q=q, k=None, v=None, ks=placed(k.abs().amax(-1) / 448), vs=placed(v.abs().amax(-1) / 448))


def _exact_few(case, st):
    T, H, I = case["T"], case["H"], case["I"]
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")

    def expert(weights, scales, e):
        if scales is None:
            return weights[e].double()
        s = scales[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return weights[e].view(torch.float8_e4m3fn).double() * s

    for t in range(T):
        z = st["logits"][t].double()
        if case["softcap"] > 0:
            z = case["softcap"] * torch.tanh(z / case["softcap"])
        order = sorted(range(case["E"]), key=lambda e, v=z.tolist(): (-v[e], e))[:case["k"]]
        w = torch.softmax(z[order], 0)
        for j, e in enumerate(order):
            gu = expert(st["up"], st["up_s"], e) @ st["x"][t].double()
            h = torch.nn.functional.silu(gu[:I]) * gu[I:]
            out[t] += w[j] * (expert(st["down"], st["down_s"], e) @ h)
    return dict(out=out)


def _exact_logits(case, st):
    B, m, V = case["B"], case["n"] + 1, case["V"]
    out = torch.empty(B, m, V, dtype=torch.float64, device="cuda")
    lens, prompts = st["hist_lens"].tolist(), st["prompt_lens"].tolist()
    f64 = lambda name: st[name].double().tolist()  # noqa: E731
    rep, pres, freq, temp = f64("repetition"), f64("presence"), f64("frequency"), f64("temperature")
    place = torch.arange(32, device="cuda")
    for b in range(B):
        said = torch.bincount(st["hist"][b, :prompts[b]].long(), minlength=V)
        count = torch.bincount(st["hist"][b, prompts[b]:lens[b]].long(), minlength=V)
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        if st["bias_t"] is not None:
            bias.index_add_(0, st["bias_t"][b].long(), st["bias_v"][b].double())
        for i in range(m):
            c = count if i == 0 else count + torch.bincount(st["draft"][b, :i].long(), minlength=V)
            l = st["logits"][b, i].double()
            old = (said + c) > 0
            l[old] = torch.where(l[old] > 0, l[old] / rep[b], l[old] * rep[b])
            l = l - freq[b] * c - pres[b] * (c > 0) + bias
            bits = ((st["mask"][b, i][:, None] >> place) & 1).bool().flatten()[:V]
            l[~bits] = -math.inf
            if not case["probs"]:
                out[b, i] = l
            elif not bits.any():
                out[b, i] = 0
            elif temp[b] > 0:
                out[b, i] = torch.softmax(l / temp[b], 0)
            else:
                out[b, i] = 0
                out[b, i, torch.nonzero(l == l.max())[0, 0]] = 1
    return dict(out=out)
