"""The operators between the serving calls against 64-bit forms (tests/step_reference.py)."""
import math
import random

import pytest
import torch

import step_reference as R
from mixture_experts_forward_gb300 import _lib as L
from mixture_experts_forward_gb300 import inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def ctrl():
    return L.new_workspace(L.CTRL_BYTES)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plan and release
def pages_state(lens, extra, free, width, seed, page, capacity=None):
    """(R.Pages, device tensors) of sequences that hold what they need and `extra` pages more."""
    rng = random.Random(seed)
    held = [R.ceil_div(n, page) + e for n, e in zip(lens, extra)]
    ids = list(range(sum(held) + free))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    stack = ids[at:] + [-1] * ((capacity or len(ids)) - free)
    ref = R.Pages(table, held, stack, free)
    dev = dict(block_table=i32(table).view(len(lens), width), held=i32(held), free_pages=i32(stack), free_count=i32([free]))
    return ref, dev, len(ids)


def same_state(ref, dev):
    assert dev["block_table"].tolist() == ref.table
    assert dev["held"].tolist() == ref.held
    assert dev["free_pages"].tolist() == ref.free
    assert dev["free_count"].item() == ref.count


PLANS = [  # lens, new, extra pages, free pages, rows
    ([5], [1], [0], 3, 1),
    ([16], [1], [0], 3, 4),                          # the first token of a new page, padded rows
    ([0], [0], [0], 2, 3),                           # an empty sequence that brings nothing
    ([0, 0, 31, 32, 33], [1, 40, 1, 1, 15], [0] * 5, 9, 64),
    ([16, 16, 16, 5], [1, 1, 1, 2], [0] * 4, 2, 8),  # pages for two of three; the last needs none
    ([16, 0, 16, 5], [1, 100, 1, 0], [0] * 4, 3, 102),   # one that is too long stops those after it
    ([3, 40], [30, 0], [4, 1], 0, 30),               # pages kept from refused drafts are used first
    ([7, 9], [1, 1], [0, 0], 0, 2),                  # nothing free, nothing needed
]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("case", range(len(PLANS)))
def test_plan_and_release(case, page):
    lens, news, extra, free, rows = PLANS[case]
    k = page // 16
    lens = [n * k for n in lens]
    ref, dev, total = pages_state(lens, extra, free, 12, case, page)
    ws = ctrl()
    got = L.plan_step(i32(lens), i32(news), **dev, rows=rows, page_size=page, num_pages=total, ws=ws)
    want = ref.plan(lens, news, rows, page, total)
    for g, w in zip(got, want[:4]):
        assert g.tolist() == w
    same_state(ref, dev)
    assert want[4] == 0 and L.get_error(ws) == L.MOE_OK
    # refused drafts' pages go back, then everything
    for keep in ([n if b % 2 else -1 for b, n in enumerate(lens)], [n - 1 if n else 0 for n in lens], [0] * len(lens)):
        L.release_pages(i32(keep), **dev, page_size=page, ws=ws)
        ref.release(keep, page)
        same_state(ref, dev)
    assert L.get_error(ws) == L.MOE_OK


@pytest.mark.parametrize("B", [1, 31, 1024, 1025, 4099, 8192])
def test_plan_of_many_sequences(B):
    rng = random.Random(B)
    page, width = 32, 9
    lens = [rng.randrange(0, 200) for _ in range(B)]
    news = [rng.choice([0, 1, 1, 5, 60]) for _ in range(B)]
    need = sum(R.ceil_div(n + m, page) - R.ceil_div(n, page) for n, m in zip(lens, news))
    ref, dev, total = pages_state(lens, [0] * B, need * 3 // 4 + 1, width, B, page)
    rows, ws = sum(news) + 77, ctrl()
    for again in range(2):                           # a plan, its release restores the stack, the same plan
        before = list(ref.free[:ref.count])
        got = L.plan_step(i32(lens), i32(news), **dev, rows=rows, page_size=page, num_pages=total, ws=ws)
        want = ref.plan(lens, news, rows, page, total)
        for g, w in zip(got, want[:4]):
            assert g.tolist() == w
        L.release_pages(i32(lens), **dev, page_size=page, ws=ws)
        ref.release(lens, page)
        same_state(ref, dev)
        assert ref.free[:ref.count] == before
    assert L.get_error(ws) == L.MOE_OK


@pytest.mark.parametrize("what", ["length", "new", "held", "few held", "too long", "rows", "free id", "table id", "count"])
def test_plans_of_bad_data(what):
    """Recorded, the sequence not served, and the others as if it were not there."""
    page = 16
    lens, news, rows = [20, 33, 40], [3, 20, 2], 25
    ref, dev, total = pages_state(lens, [0, 0, 0], 5, 6, 3, page)
    ws = ctrl()
    if what == "length":
        lens[1] = -4
    if what == "new":
        news[1] = -1
    if what == "held":
        ref.held[1] = 7
    if what == "few held":
        ref.held[1] = 1
    if what == "too long":
        news[1] = 64
        rows = 69
    if what == "rows":
        rows = 20
    if what == "free id":
        ref.free[:5] = [total] * 5
    if what == "table id":
        ref.table[0][1] = -7
    if what == "count":
        ref.count = len(ref.free) + 3
    dev = dict(block_table=i32(ref.table), held=i32(ref.held), free_pages=i32(ref.free), free_count=i32([ref.count]))
    if what == "count":
        ref.count = len(ref.free)
    got = L.plan_step(i32(lens), i32(news), **dev, rows=rows, page_size=page, num_pages=total, ws=ws)
    assert L.get_error(ws) == L.MOE_ERR_DEVICE_FAULT
    want = ref.plan(lens, news, rows, page, total)
    for g, w in zip(got, want[:4]):
        assert g.tolist() == w
    same_state(ref, dev)


def test_a_stack_without_room_takes_nothing():
    ref, dev, total = pages_state([40, 40], [0, 0], 1, 4, 1, 16, capacity=4)
    ws = ctrl()
    before = [t.clone() for t in dev.values()]
    L.release_pages(i32([0, 0]), **dev, page_size=16, ws=ws)
    assert L.get_error(ws) == L.MOE_ERR_DEVICE_FAULT
    assert all(torch.equal(a, b) for a, b in zip(before, dev.values()))
    L.release_pages(i32([0, -1]), **dev, page_size=16, ws=ws)     # three fit
    assert L.get_error(ws) == L.MOE_OK and dev["free_count"].item() == 4
    dev["held"][0] = 9
    L.release_pages(i32([0, -1]), **dev, page_size=16, ws=ws)
    assert L.get_error(ws) == L.MOE_ERR_DEVICE_FAULT


def test_a_plan_of_no_sequences():
    ws = ctrl()
    e = i32([]).view(0, 3)
    slots, pos, cu, kv = L.plan_step(i32([]), i32([]), e, i32([]), i32([4, 5]), i32([2]), 3, 16, 6, ws)
    assert slots.tolist() == [-1] * 3 and pos.tolist() == [0] * 3 and cu.tolist() == [0] and kv.numel() == 0
    assert L.get_error(ws) == L.MOE_OK


# ------------------------------------------------------------------ rotary
def near(got, want, size, extra=0.0):
    """bf16: half a step (2^-8 of the value), and the arithmetic before it: an angle is off by its
    truncation to 2^-32 turns and by a binary32 rounding of at most half a turn (together
    below 2e-7), sincospi by 2 units of 2^-24, products and sums by 3: 8e-7 of the pair."""
    tol = want.abs() * 2.0 ** -8 + size * 8e-7 + 1e-38 + extra
    bad = (got.double().cpu() - want).abs() > tol
    assert not bad.any(), (got.double().cpu()[bad][:4], want[bad][:4])


ROTARY = [  # T, Hq, Hkv, D, rot, interleaved, scaling, largest position
    (1, 4, 1, 128, 128, False, "none", 100), (1, 1, 1, 64, 64, True, "none", 5),
    (7, 6, 2, 128, 64, False, "linear", 4000), (33, 8, 8, 64, 16, True, "turns", 100000),
    (150, 5, 5, 128, 48, False, "index", 2 ** 31 - 1), (700, 3, 1, 64, 32, True, "none", 2 ** 30),
    (2500, 2, 1, 128, 128, False, "turns", 1000000)]


def rotary_inputs(T, Hq, Hkv, D, rot, scaling, far, seed=0):
    g = torch.Generator().manual_seed(seed + T)
    packed = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(BF16)
    packed[..., 1] *= 30
    pos = torch.randint(0, far + 1, (T,), generator=g).to(torch.int32)
    pos[0] = far
    if T > 2:
        pos[1], pos[2] = 0, -far
    kw = dict(base=500000.0 if scaling == "turns" else 10000.0, scaling=scaling, factor=8.0, original=8192, low=1.0,
              high=4.0)
    return packed, pos, R.frequencies(rot, **kw), L.rotary_table(rot, **kw)


@pytest.mark.parametrize("case", range(len(ROTARY)))
def test_rotary_without_a_cache(case):
    T, Hq, Hkv, D, rot, inter, scaling, far = ROTARY[case]
    packed, pos, theta, table = rotary_inputs(T, Hq, Hkv, D, rot, scaling, far)
    dev, amp = packed.cuda(), 1.25
    q, k = dev[:, :Hq], dev[:, Hq:Hq + Hkv]          # views of a packed projection
    qo, ko = L.rotary(q, k, pos.cuda(), table, interleaved=inter, amplitude=amp)
    for got, x in ((qo, packed[:, :Hq]), (ko, packed[:, Hq:Hq + Hkv])):
        want, size = R.rotated(x, pos, theta, inter, amp)
        near(got, want, size)
        assert torch.equal(got[..., rot:].cpu(), x[..., rot:])
    # one of them alone, in place, and into a wider output: the same bits
    assert torch.equal(L.rotary(None, k, pos.cuda(), table, interleaved=inter, amplitude=amp)[1], ko)
    wide = torch.full((T, Hq, D + 16), 7.0, dtype=BF16, device="cuda")
    L.rotary(q, None, pos.cuda(), table, interleaved=inter, amplitude=amp, q_out=wide[..., :D])
    assert torch.equal(wide[..., :D], qo) and (wide[..., D:] == 7).all()
    L.rotary(q, k, pos.cuda(), table, interleaved=inter, amplitude=amp, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(dev[:, Hq + Hkv:].cpu(), packed[:, Hq + Hkv:])


@pytest.mark.parametrize("D,rot", [(16, 16), (80, 32), (256, 256), (192, 112)])
def test_rotary_of_other_head_sizes(D, rot):
    g = torch.Generator().manual_seed(D)
    x = torch.randn(9, 3, D, generator=g).to(BF16)
    pos = torch.randint(0, 5000, (9,), generator=g).to(torch.int32)
    for inter in (False, True):
        got, _ = L.rotary(x.cuda(), None, pos.cuda(), L.rotary_table(rot), interleaved=inter)
        want, size = R.rotated(x, pos, R.frequencies(rot), inter)
        near(got, want, size)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("case", range(len(ROTARY)))
def test_rotary_into_a_cache(case, page, fp8):
    T, Hq, Hkv, D, rot, inter, scaling, far = ROTARY[case]
    packed, pos, theta, table = rotary_inputs(T, Hq, Hkv, D, rot, scaling, far, seed=5)
    n_pages = R.ceil_div(T, page) + 2
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    if T > 5:
        slots[3] = -1
    dt = L.DTYPE_FP8 if fp8 else L.DTYPE_BF16
    kc, vc, ks, vs = L.new_kv_cache(dt, n_pages, page, Hkv, D)
    k2, v2, ks2, vs2 = L.new_kv_cache(dt, n_pages, page, Hkv, D)
    dev, ws = packed.cuda(), ctrl()
    q, k, v = dev.split([Hq, Hkv, Hkv], dim=1)
    out = L.rotary_write(q, k, v, pos.cuda(), slots.cuda(), table, kc, vc, ws, k_scales=ks, v_scales=vs, interleaved=inter)
    assert L.get_error(ws) == L.MOE_OK
    assert torch.equal(out, L.rotary(q, None, pos.cuda(), table, interleaved=inter)[0])
    # values, and keys at position 0, as moe_kv_write stores them
    L.kv_write(k, v, slots.cuda(), k2, v2, ws, k_scales=ks2, v_scales=vs2)
    assert torch.equal(vc, v2) and (not fp8 or torch.equal(vs, vs2))
    kc3, vc3, ks3, vs3 = L.new_kv_cache(dt, n_pages, page, Hkv, D)
    L.rotary_write(q, k, v, torch.zeros_like(pos).cuda(), slots.cuda(), table, kc3, vc3, ws, k_scales=ks3, v_scales=vs3,
                   interleaved=inter)
    assert torch.equal(kc3, k2) and (not fp8 or torch.equal(ks3, ks2))
    want, size = R.rotated(packed[:, Hq:Hq + Hkv], pos, theta, inter)
    real = slots >= 0
    at = slots[real].long()
    held = kc.cpu()[at // page, :, at % page]
    want, size = want[real], size[real]
    if not fp8:
        near(held, want, size)
    else:
        scale = ks.cpu()[at // page, :, at % page].double()
        top = want.abs().amax(-1) / 448
        assert ((scale - top).abs() <= top * 2.0 ** -20 + size.amax(-1) * 8e-7 / 448).all()
        value = held.view(torch.float8_e4m3fn).double() * scale[..., None]
        # half a step of the code (2^-4 of it, or of the smallest normal one), and the arithmetic before
        tol = torch.maximum(want.abs() * 2.0 ** -4, 2.0 ** -10 * scale[..., None]) * 1.0001 + size * 8e-7
        assert ((value - want).abs() <= tol).all()
    touched = torch.zeros(n_pages, page, dtype=torch.bool)
    touched[at // page, at % page] = True
    assert (kc.cpu().float().abs().amax(dim=(1, 3))[~touched] == 0).all()


def test_rotary_slots_out_of_range_and_odd_values():
    T, table = 6, L.rotary_table(64)
    x = torch.randn(T, 6, 64, device="cuda").to(BF16)
    q, k, v = x.split([2, 2, 2], dim=1)
    k = k.clone()
    k[0, 0, 3], k[1, 0, 5], k[2] = math.nan, math.inf, 0
    kc, vc, ks, vs = L.new_kv_cache(L.DTYPE_FP8, 2, 16, 2, 64)
    ws = ctrl()
    L.rotary_write(q, k, v, i32([0] * T), i32([0, 1, 2, 32, -2, 31]), table, kc, vc, ws, k_scales=ks, v_scales=vs)
    assert L.get_error(ws) == L.MOE_ERR_DEVICE_FAULT
    codes = kc.view(torch.float8_e4m3fn).float()
    assert codes[0, 0, 0, 3].isnan() and not codes[0, 1, 0].isnan().any()
    assert ks[0, 0, 1] == math.inf and ks[0, 0, 2] == 0 and (codes[0, :, 2] == 0).all()
    assert (ks[1, :, 15] > 0).all() and (ks > 0).sum() == 2 * 3 - 0      # slots 0, 1 and 31 (2 heads each)
    L.rotary_write(q[:0], k[:0], v[:0], i32([]), i32([]), table, kc, vc, ws, k_scales=ks, v_scales=vs)


# ------------------------------------------------------------------ few tokens
def few_case(fp8, T, H, I, E, k, seed=0, softcap=0.0, renorm=1, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    up = torch.randn(E, 2 * I, H, generator=g) / H ** 0.5
    down = torch.randn(E, H, I, generator=g) / I ** 0.5
    x = torch.randn(T, H, generator=g)
    x[:, ::61] *= 40
    x = x.to(BF16)
    logits = torch.randn(T, E, generator=g) * spread
    if fp8:
        up, up_s = inputs.quantize_weights_e4m3(up)
        down, dn_s = inputs.quantize_weights_e4m3(down)
        wide = lambda w, s: (w.view(torch.float8_e4m3fn).double() *  # noqa: E731
                             s.double().repeat_interleave(128, 1).repeat_interleave(128, 2))
        values = wide(up, up_s), wide(down, dn_s)
    else:
        up, down, up_s, dn_s = up.to(BF16), down.to(BF16), None, None
        values = up.double(), down.double()
    dev = dict(logits=logits, x=x, w=up, w_scales=up_s, w2=down, w2_scales=dn_s)
    dev = {n: None if t is None else t.cuda().contiguous() for n, t in dev.items()}
    args = L.forward_args(dtype=L.DTYPE_FP8 if fp8 else L.DTYPE_BF16, M=T, K=H, N=I, E=E, top_k=k, softcap=softcap,
                          renorm=renorm, gated=1, **dev)
    return args, dev, x, values


def check_few(args, dev, x, values, fp8):
    T, H, k = args.M, args.K, args.top_k
    ws = L.new_workspace(L.few_workspace_size(args))
    out = torch.full((T, H), math.nan, dtype=BF16, device="cuda")
    L.forward_few(args, out, ws)
    assert L.get_error(ws) == L.MOE_OK
    ids, w = L.route(dev["logits"], k, softcap=args.softcap, renorm=args.renorm)
    want, err = R.few(x, ids.cpu(), w.cpu(), *values, fp8)
    tol = err + (want.abs() + err) * 2.0 ** -8 + 1e-38
    diff = (out.cpu().double() - want).abs()
    assert (diff <= tol).all(), (diff / tol).max()
    again = torch.empty_like(out)
    L.forward_few(args, again, ws)
    assert torch.equal(out, again)                   # the same bits: no order depends on the schedule
    return out


FEW = [  # T, H, I, E, k, softcap, renorm, spread of the logits
    (1, 128, 128, 1, 1, 0.0, 1, 1.0), (1, 256, 128, 8, 2, 30.0, 1, 1.0), (2, 384, 256, 5, 5, 0.0, 0, 1.0),
    (5, 512, 384, 16, 4, 0.0, 1, 1.0), (8, 640, 128, 40, 3, 30.0, 1, 4.0), (9, 256, 256, 300, 8, 0.0, 1, 1.0),
    (16, 1152, 128, 12, 6, 0.0, 1, 0.01), (16, 256, 640, 4, 4, 0.0, 0, 1.0), (13, 128, 128, 70, 32, 0.0, 1, 1.0)]


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("case", range(len(FEW)))
def test_few_tokens(case, fp8):
    T, H, I, E, k, cap, renorm, spread = FEW[case]
    check_few(*few_case(fp8, T, H, I, E, k, seed=case, softcap=cap, renorm=renorm, spread=spread), fp8)


@pytest.mark.parametrize("fp8,T,H,I", [(True, 16, 5120, 128), (False, 16, 4160, 128), (True, 3, 24576, 128),
                                       (False, 1, 320, 3200), (True, 2, 9856, 256), (True, 11, 5888, 384)])
def test_few_tokens_of_long_rows(fp8, T, H, I):
    """x that fits a launch by halves, odd numbers of blocks, more rows of h than are staged at once."""
    check_few(*few_case(fp8, T, H, I, 3, 2, seed=T), fp8)


@pytest.mark.parametrize("fp8", [True, False])
def test_few_tokens_that_share_all_experts(fp8):
    args, dev, x, values = few_case(fp8, 16, 256, 1024, 6, 6, seed=3)
    check_few(args, dev, x, values, fp8)


@pytest.mark.parametrize("fp8", [True, False])
def test_few_tokens_of_odd_values(fp8):
    """A token of zeros, one of very large and one of very small elements, a NaN and an infinity: each
    stays with its token."""
    args, dev, x, values = few_case(fp8, 6, 256, 128, 8, 2, seed=9)
    plain = check_few(args, dev, x, values, fp8)
    dev["x"][1] = 0
    dev["x"][2] *= 2.0 ** 100
    dev["x"][3] *= 2.0 ** -110
    dev["x"][4, 7] = math.nan
    dev["x"][5, 9] = math.inf
    ws = L.new_workspace(L.few_workspace_size(args))
    out = L.forward_few(args, torch.empty_like(plain), ws)
    assert torch.equal(out[0], plain[0]) and (out[1] == 0).all()
    assert out[4].isnan().all() and not out[5].isfinite().any()
    assert (out[3].float().abs() < 1e-30).all()
    assert not torch.isfinite(out[2].float()).all() or out[2].float().abs().max() > 1e28


def test_few_tokens_beside_the_forward():
    """The FP8 forward quantises its activations, the few-token form does not: they differ by that, a
    few E4M3 half steps (2^-4) averaged over hundreds of terms."""
    args, dev, x, values = few_case(True, 8, 512, 256, 16, 4, seed=11)
    few = check_few(args, dev, x, values, True).float()
    out = torch.empty_like(few, dtype=BF16)
    L.forward(args, out, L.new_workspace(L.workspace_size(args)))
    assert ((out.float() - few).norm() / few.norm()) < 2.0 ** -4


# ------------------------------------------------------------------ logits
def logits_case(B, m, V, hist, nb, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, m, V, generator=g) * 3).to(dtype)
    tok = lambda *s: (torch.rand(*s, generator=g) ** 2 * V).to(torch.int32).clamp(max=V - 1)  # noqa: E731
    kw = dict(history=tok(B, hist), draft=tok(B, m - 1) if m > 1 else None,
              history_lens=torch.tensor([max(0, hist - 7 * b) for b in range(B)], dtype=torch.int32),
              repetition=1 + torch.rand(B, generator=g) * 0.5, presence=torch.randn(B, generator=g),
              frequency=torch.rand(B, generator=g) * 0.5, temperature=0.5 + torch.rand(B, generator=g))
    kw["prompt_lens"] = kw["history_lens"] // 2
    if nb:
        kw["bias_tokens"], kw["bias_values"] = tok(B, nb), torch.randn(B, nb, generator=g) * 2
    bits = torch.randint(-2 ** 31, 2 ** 31, (B, m, (V + 31) // 32), generator=g)
    kw["mask"] = (bits | torch.randint(-2 ** 31, 2 ** 31, bits.shape, generator=g)).to(torch.int32)
    return x, kw


def run_logits(x, kw, **more):
    dev = {n: t.cuda() if torch.is_tensor(t) else t for n, t in {**kw, **more}.items()}
    ws = ctrl()
    out = L.adjust_logits(x.cuda(), ws, **dev)
    return out.cpu(), L.get_error(ws)


def check_logits(x, kw, **more):
    out, status = run_logits(x, kw, **more)
    want = R.logits(x, **kw, **more)
    assert status == L.MOE_OK
    assert torch.equal(out == -math.inf, want == -math.inf)
    if more.get("probabilities") is False:
        fine = torch.isfinite(want)
        # six roundings to binary32, each of at most 2^-24 of what has been added up till then (below 60)
        assert ((out.double() - want)[fine].abs() <= 6 * 2.0 ** -24 * 60).all()
    else:
        # the adjusted logits' error (below 6 * 2^-24 * 60) over a temperature of 0.5, the exponent's own
        # (2^-22 of at most 120), a sum of up to 2^18 terms by threads and warps (2^-17)
        rel = 6 * 2.0 ** -24 * 60 / 0.5 + 2.0 ** -22 * 120 + 2.0 ** -17 + 2.0 ** -20
        assert ((out.double() - want).abs() <= want * rel + 1e-36).all()
    return out


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("B,m,V,hist,nb", [(1, 1, 1, 3, 1), (1, 1, 33, 0, 0), (3, 1, 4097, 50, 5), (2, 3, 8192, 700, 40),
                                           (4, 5, 1003, 64, 1024), (2, 2, 20011, 3000, 64), (1, 4, 70001, 200, 3),
                                           (1, 2, 131072, 100, 8), (1, 1, 262144, 5000, 30), (1, 33, 300, 20, 7)])
def test_logits(B, m, V, hist, nb, dtype, probs):
    x, kw = logits_case(B, m, V, max(hist, 1), nb, V + B, dtype)
    if hist == 0:
        for n in ("history", "history_lens", "prompt_lens"):
            kw[n] = None
    check_logits(x, kw, probabilities=probs)


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("B,m,V,hist", [(200, 5, 4000, 100), (200, 5, 4000, 9000), (38, 2, 70001, 2000),
                                        (38, 2, 131072, 60000)])
def test_logits_of_sequences_whose_rows_share_their_counts(B, m, V, hist, probs):
    """So many rows that some of a sequence's go together; of the long histories a CTA's tokens are
    mostly named, too many for a list."""
    x, kw = logits_case(B, m, V, hist, 7, seed=V + hist)
    g = torch.Generator().manual_seed(hist)
    kw["history"] = torch.randint(0, V, (B, hist), generator=g, dtype=torch.int32)
    kw["draft"][::2, 1:] = kw["draft"][::2, :1]                       # the same draft again
    kw["draft"][1::2] = kw["history"][1::2, : m - 1]                  # and one that is in the prompt
    check_logits(x, kw, probabilities=probs)


def test_logits_one_thing_at_a_time():
    x, kw = logits_case(2, 3, 5001, 300, 20, 4)
    plain = check_logits(x, {})
    assert (plain.sum(-1) - 1).abs().max() < 1e-5
    for names in (["mask"], ["temperature"], ["bias_tokens", "bias_values"], ["draft", "frequency"],
                  ["history", "repetition"], ["history", "presence"], ["history", "prompt_lens", "frequency"],
                  ["history", "history_lens", "draft", "presence", "frequency"]):
        check_logits(x, {n: kw[n] for n in names})
        check_logits(x, {n: kw[n] for n in names}, probabilities=False)
    check_logits(x, dict(mask=kw["mask"][:, 0].contiguous()))          # one mask for a sequence's rows


def test_logits_greedy_takes_the_lowest_of_equals():
    x = torch.zeros(3, 2, 40000)
    x[0, 0, [39999, 20000, 31]] = 5.0
    x[0, 1, 39999] = 1.0
    x[1, 0, 7], x[1, 0, 6] = math.inf, math.nan
    x[1, 1] = -math.inf
    x[2, 0, 100:] = -1.0                                               # ties of all from 0 on
    out, status = run_logits(x, dict(temperature=torch.zeros(3)))
    assert status == L.MOE_OK
    assert out[0, 0].nonzero().flatten().tolist() == [31] and out[0, 1].nonzero().flatten().tolist() == [39999]
    assert out[1, 0].nonzero().flatten().tolist() == [7] and (out[1, 1] == 0).all()
    assert out[2, 0].nonzero().flatten().tolist() == [0]
    assert out.max() == 1


def test_logits_at_the_ends_of_the_type():
    V = 9000
    big = torch.finfo(torch.float32).max
    x = torch.zeros(6, 1, V)
    x[0] = -big                                     # masks of the lowest value: the same for all
    x[1, 0, :] = -big
    x[1, 0, 8] = 3.0
    x[2, 0, [4, 8999]] = math.inf                   # share all of it
    x[3] = -math.inf                                # nothing left
    x[4, 0, 10:20] = math.nan
    x[5, 0, 5] = big
    out, _ = run_logits(x, dict(temperature=torch.tensor([0.5, 1.0, 2.0, 1.0, 1.0, 1e-30])))
    assert torch.allclose(out[0], torch.full((1, V), 1 / V), rtol=1e-5)
    assert out[1, 0, 8] == 1 and out[1].sum() == 1
    assert out[2, 0, 4] == 0.5 and out[2, 0, 8999] == 0.5 and out[2].sum() == 1
    assert (out[3] == 0).all()
    assert (out[4, 0, 10:20] == 0).all() and torch.allclose(out[4].sum(), torch.tensor(1.0), rtol=1e-5)
    assert out[5, 0, 5] == 1 and out[5].sum() == 1
    # a token at -inf stays there whatever is added; an infinite bias takes all
    kw = dict(bias_tokens=torch.tensor([[3, 4, 4, -1]], dtype=torch.int32),
              bias_values=torch.tensor([[math.inf, 1.0, 2.0, 9.0]]))
    y = torch.zeros(1, 1, 100)
    y[0, 0, 3] = -math.inf
    out, status = run_logits(y, kw, probabilities=False)
    assert status == L.MOE_OK and out[0, 0, 3] == -math.inf and out[0, 0, 4] == 3 and out[0, 0, 5] == 0
    y[0, 0, 3] = 0
    assert run_logits(y, kw)[0][0, 0, 3] == 1


@pytest.mark.parametrize("probs", [True, False])
def test_logits_of_strided_rows_and_in_place(probs):
    x, kw = logits_case(3, 2, 3001, 90, 9, 8)
    want = check_logits(x, kw, probabilities=probs)
    dev = {n: t.cuda() for n, t in kw.items()}
    wide = torch.full((3, 4, 3005), 77.0, device="cuda")
    view = wide[:, 1:3, 2:3003]
    view.copy_(x)
    got = L.adjust_logits(view, ctrl(), **dev, probabilities=probs, out=view)
    assert torch.equal(got.cpu(), want)
    assert (wide[:, 0] == 77).all() and (wide[:, 3] == 77).all() and (wide[:, :, :2] == 77).all() and (wide[:, :, 3003:] == 77).all()


@pytest.mark.parametrize("bad", ["history", "draft", "bias", "lens", "prompt", "repetition", "temperature"])
def test_logits_of_bad_data(bad):
    x, kw = logits_case(2, 2, 500, 30, 4, 2)
    fine = dict(kw)
    if bad == "history":
        kw["history"][1, 2], fine["history"] = 500, kw["history"].clone()
        fine["history"][1, 2] = -1
    if bad == "draft":
        kw["draft"][0, 0], fine["draft"] = -2, kw["draft"].clone()
        fine["draft"][0, 0] = -1
    if bad == "bias":
        kw["bias_tokens"][1, 1], fine["bias_tokens"] = 2 ** 31 - 1, kw["bias_tokens"].clone()
        fine["bias_tokens"][1, 1] = -1
    if bad == "lens":
        fine["history_lens"] = torch.tensor([30, 0], dtype=torch.int32)
        kw["history_lens"] = torch.tensor([31, -5], dtype=torch.int32)
        kw["prompt_lens"] = fine["prompt_lens"] = torch.zeros(2, dtype=torch.int32)
    if bad == "prompt":
        fine["prompt_lens"] = kw["history_lens"]
        kw["prompt_lens"] = kw["history_lens"] + 1
    if bad == "repetition":
        kw["repetition"] = torch.tensor([0.0, math.nan])
        fine["repetition"] = torch.ones(2)
    if bad == "temperature":
        kw["temperature"] = torch.tensor([-1.0, math.nan])
        fine["temperature"] = torch.ones(2)
    out, status = run_logits(x, kw)
    assert status == L.MOE_ERR_DEVICE_FAULT
    want, status = run_logits(x, fine)
    assert status == L.MOE_OK and torch.equal(out, want)


def test_the_same_logits_give_the_same_bits():
    x, kw = logits_case(5, 6, 30011, 2000, 64, 1)
    dev = {n: t.cuda() for n, t in kw.items()}
    x, ws = x.cuda(), ctrl()
    first = L.adjust_logits(x, ws, **dev)
    for _ in range(5):
        assert torch.equal(first, L.adjust_logits(x, ws, **dev))


# ------------------------------------------------------------------ graphs and streams
def small_calls():
    """name -> a call that returns what it computed, on inputs of its own."""
    _, dev, total = pages_state([20, 33], [0, 0], 6, 6, 2, 16)
    lens, news, ws = i32([20, 33]), i32([15, 3]), ctrl()
    packed, pos, _, table = rotary_inputs(40, 2, 1, 64, 64, "none", 300)
    packed, pos = packed.cuda(), pos.cuda()
    cache, slots = L.new_kv_cache(L.DTYPE_FP8, 4, 16, 1, 64), i32(range(40))
    q, k, v = packed.split([2, 1, 1], dim=1)
    args, few, _, _ = few_case(True, 3, 256, 128, 8, 2)
    few_ws, out = L.new_workspace(L.few_workspace_size(args)), torch.empty(3, 256, dtype=BF16, device="cuda")
    x, kw = logits_case(2, 2, 9001, 100, 5, 3)
    x, kw = x.cuda(), {n: t.cuda() for n, t in kw.items()}

    def plan(stream=None):
        got = L.plan_step(lens, news, **dev, rows=20, page_size=16, num_pages=total, ws=ws, stream=stream)
        L.release_pages(lens, **dev, page_size=16, ws=ws, stream=stream)
        return [*got, *dev.values()]

    def write(stream=None):
        o = L.rotary_write(q, k, v, pos, slots, table, cache[0], cache[1], ws, k_scales=cache[2], v_scales=cache[3],
                           stream=stream)
        return [o, *cache]

    return dict(plan=plan, rotary=lambda stream=None: list(L.rotary(q, k, pos, table, stream=stream)), write=write,
                few=lambda stream=None: [L.forward_few(args, out, few_ws, stream=stream), few["x"]],
                logits=lambda stream=None: [L.adjust_logits(x, ws, **kw, stream=stream)])


@pytest.mark.parametrize("name", ["plan", "rotary", "write", "few", "logits"])
def test_in_a_graph_and_on_another_stream(name):
    call = small_calls()[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = call()
    for _ in range(3):
        for t in outs[:1]:
            t.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_two_captured_calls_with_workspaces_of_their_own():
    """Two graphs of the few-token layer that run at the same time."""
    cases = [few_case(fp8, 7, 512, 256, 16, 4, seed=s) for s, fp8 in ((1, True), (2, False))]
    runs = []
    for args, dev, x, values in cases:
        ws, out = L.new_workspace(L.few_workspace_size(args)), torch.empty(7, 512, dtype=BF16, device="cuda")
        want = L.forward_few(args, out, ws).clone()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            L.forward_few(args, out, ws)
        runs.append((g, s, out, want, ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s, out, _, _ in runs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, out, want, ws in runs:
        assert torch.equal(out, want) and L.get_error(ws) == L.MOE_OK
