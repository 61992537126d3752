"""The serving operators on the GPU: the paged cache (bit-exact), attention over
it (against 64 bits, with derived tolerances) and draft verification (exact)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import serving_reference as R
from gpu_helpers import bits, ensure_built
from mixture_experts_forward_gb300 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def ctrl():
    return L.new_workspace(L.CTRL_BYTES)


_ws = {}


def attention_ws():
    if "ws" not in _ws:
        _ws["ws"] = L.new_workspace(L.ATTENTION_WS_BYTES)
    return _ws["ws"]


def cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand_bf16(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


# ------------------------------------------------------------------ cache
@pytest.mark.parametrize("T", [0, 1, 2, 33, 500])
@pytest.mark.parametrize("H,D", [(1, 64), (3, 128), (8, 128), (5, 64)])
@pytest.mark.parametrize("fp8", [True, False])
def test_kv_write_is_bit_exact(T, H, D, fp8):
    page = 16
    n_pages = T // page + 3
    packed = rand_bf16(max(T, 1), 2, H, D, seed=T + H).cuda()[:T]
    packed[:, :, :, :2] *= 40
    if T > 2:
        packed[1] = 0                                     # a row of zeros
        packed[2] = -0.0
        packed[0, 0, 0] = 1e-39                           # 1/s would overflow
        packed[0, 1, 0, 3] = math.nan                     # keeps its place
    k, v = packed[:, 0], packed[:, 1]                     # strided views
    kc, vc, ks, vs = L.new_kv_cache(L.DTYPE_FP8 if fp8 else L.DTYPE_BF16, n_pages, page, H, D)
    slots = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(1))[:T].to(torch.int32)
    if T > 4:
        slots[4] = -1                                     # skipped
    ws = ctrl()
    L.kv_write(k, v, slots.cuda(), kc, vc, ws, k_scales=ks, v_scales=vs)
    assert L.get_error(ws) == L.MOE_OK
    keep = (slots >= 0).nonzero()[:, 0]
    at = slots[keep].long()
    for new, cache, scales in ((k, kc, ks), (v, vc, vs)):
        want = torch.zeros(n_pages * page, H, D, dtype=cache.dtype)
        new = new.cpu()[keep]
        if fp8:
            nan = new.float().isnan()
            codes, s = R.quantise_rows(new.nan_to_num(0.0))
            codes[nan] = R.NAN_CODE
            want[at] = codes
            want_s = torch.zeros(n_pages * page, H)
            want_s[at] = s
            got_s = scales.cpu().permute(0, 2, 1).reshape(-1, H)
            assert torch.equal(got_s, want_s)
            got = cache.cpu().permute(0, 2, 1, 3).reshape(-1, H, D)
            same = (got == want) | (((got & 0x7f) == 0) & ((want & 0x7f) == 0))   # +0 and -0
            assert bool(same.all())
        else:
            want[at] = new
            got = cache.cpu().permute(0, 2, 1, 3).reshape(-1, H, D)
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_kv_write_matches_the_oracle_quantiser():
    T, H, D = 37, 4, 128
    x = rand_bf16(T * H, D, seed=5)
    kc, vc, ks, vs = L.new_kv_cache(L.DTYPE_FP8, 3, 16, H, D)
    xg = x.cuda().view(T, H, D)
    ws = ctrl()
    L.kv_write(xg, xg, torch.arange(T, dtype=torch.int32, device="cuda"), kc, vc, ws, k_scales=ks,
               v_scales=vs)
    q, s = oracle.quant_gather(bits(x), 1, np.arange(T * H, dtype=np.int32))
    got = kc.cpu().permute(0, 2, 1, 3).reshape(-1, H, D)[:T].reshape(T * H, D).numpy()
    assert np.array_equal(got, np.asarray(q).view(np.uint8))
    assert np.array_equal(ks.cpu().permute(0, 2, 1).reshape(-1, H)[:T].reshape(-1).numpy(),
                          np.asarray(s).reshape(-1))
    assert torch.equal(kc, vc) and torch.equal(ks, vs)


@pytest.mark.parametrize("page,H,D,fp8", [(16, 3, 128, True), (64, 8, 64, True), (256, 1, 128, False),
                                         (32, 5, 64, False)])
def test_kv_read_is_bit_exact(page, H, D, fp8):
    lens = [1, 0, 77, page, 300]
    keys = [rand_bf16(n, H, D, seed=n) for n in lens]
    vals = [rand_bf16(n, H, D, seed=n + 1) for n in lens]
    c = R.Paged(keys, vals, page, fp8)
    ws = ctrl()
    k, v = L.kv_read(c.k, c.v, c.table, cu(lens), sum(lens), ws, k_scales=c.ks, v_scales=c.vs)
    for got, name in ((k, "k"), (v, "v")):
        want = torch.cat([c.rows(name, b, n) for b, n in enumerate(lens)])
        # code * scale has at most 28 bits: binary32 rounds it once before bf16 does
        assert torch.equal(got, want.float().to(torch.bfloat16))
    # a middle piece of each sequence
    starts = [0, 0, 20, page - 1, 123]
    part = [n - s for n, s in zip(lens, starts)]
    k, _ = L.kv_read(c.k, c.v, c.table, cu(part), sum(part), ws, k_scales=c.ks, v_scales=c.vs,
                     starts=i32(starts))
    want = torch.cat([c.rows("k", b, n)[s:] for b, (n, s) in enumerate(zip(lens, starts))])
    assert torch.equal(k, want.float().to(torch.bfloat16))
    assert L.get_error(ws) == L.MOE_OK


def test_cache_reports_what_is_out_of_range():
    H, D = 2, 64
    kc, vc, ks, vs = L.new_kv_cache(L.DTYPE_FP8, 2, 16, H, D)
    x = rand_bf16(3, H, D).cuda()
    for bad in (32, -2, 1 << 30):
        ws = ctrl()
        L.kv_write(x, x, i32([0, bad, 31]), kc, vc, ws, k_scales=ks, v_scales=vs)
        assert L.get_error(ws) == L.MOE_ERR_DEVICE_FAULT
    for table, n in (([[0, 2]], 20), ([[0, -1]], 20), ([[0, 1]], 33)):
        ws = ctrl()
        k, _ = L.kv_read(kc, vc, i32(table), cu([n]), n, ws, k_scales=ks, v_scales=vs)
        assert L.get_error(ws) == L.MOE_ERR_DEVICE_FAULT
        assert bool((k[32 if n == 33 else 16:] == 0).all())


# ------------------------------------------------------------------ attention
def check_attention(q_lens, kv_lens, Hq, Hkv, D, page, fp8, *, scale=0.0, softcap=0.0, window=0,
                    causal=True, seed=0, spread=1.0, packed=False, max_kv=None, ws=None, stream=None):
    keys = [rand_bf16(n, Hkv, D, seed=seed + 10 * b + n, scale=spread) for b, n in enumerate(kv_lens)]
    vals = [rand_bf16(n, Hkv, D, seed=seed + 10 * b + n + 1) for b, n in enumerate(kv_lens)]
    c = R.Paged(keys, vals, page, fp8, seed=seed)
    T = sum(q_lens)
    if packed:      # a view of a packed projection, and a strided output
        q = rand_bf16(T, Hq + 2 * Hkv, D, seed=seed + 7).cuda()[:, :Hq]
        out = torch.full((T, Hq + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    else:
        q = rand_bf16(T, Hq, D, seed=seed + 7).cuda()
        out = None
    ws = attention_ws() if ws is None else ws
    got, lse = L.paged_attention(q, c.k, c.v, c.table, cu(q_lens), i32(kv_lens), ws,
                                 max_q=max(q_lens), max_kv=max(kv_lens) if max_kv is None else max_kv,
                                 k_scales=c.ks, v_scales=c.vs, scale=scale, softcap=softcap,
                                 window=window, causal=causal,
                                 out=None if out is None else out[:, :Hq], lse=True, stream=stream)
    if stream is not None:
        stream.synchronize()
    assert L.get_error(ws) == L.MOE_OK
    assert not bool(ws[L.CTRL_BYTES:L.ATTENTION_CTRL_BYTES].any()), "counters left behind"
    want, want_l, tol, tol_l = R.attention(q, c, q_lens, kv_lens, scale=scale, softcap=softcap,
                                           window=window, causal=causal)
    got = got.double()
    assert bool(torch.isfinite(got).all())
    over = ((got - want).abs() - tol).amax().item() if T else -1
    assert over <= 0, f"out: {over:.3e} over its tolerance"
    none = torch.isinf(want_l)
    assert torch.equal(torch.isinf(lse), none) and bool((lse[none] < 0).all())
    assert bool((got[none] == 0).all())
    d = ((lse.double() - want_l).abs() - tol_l)[~none]
    assert d.numel() == 0 or d.amax().item() <= 0, f"lse: {d.amax().item():.3e} over its tolerance"
    if out is not None:
        assert bool((out[:, Hq] == 7).all())
    return got


FORMS = [(64, False), (64, True), (128, False), (128, True)]


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (5, 1), (16, 16), (32, 1), (7, 7)])
def test_single_tokens(D, fp8, Hq, Hkv):
    check_attention([1, 1, 1, 1, 1, 1], [1, 2, 17, 64, 255, 1000], Hq, Hkv, D, 16, fp8)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages_that_end_inside_a_tile(D, fp8, page):
    check_attention([1, 3, 40, 0, 129], [page + 1, 2 * page - 1, 300, 5, 513], 6, 2, D, page, fp8)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_lens,kv_lens", [([5, 2, 7], [900, 31, 7]), ([17, 130], [17, 700]),
                                            ([257, 64], [300, 64]), ([1, 300], [3000, 1500])])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (9, 3), (2, 2)])
def test_chunks(D, fp8, q_lens, kv_lens, Hq, Hkv):
    check_attention(q_lens, kv_lens, Hq, Hkv, D, 64, fp8, packed=True)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("window", [1, 16, 100, 1000])
def test_windows(D, fp8, window):
    check_attention([1, 4, 150, 260], [800, 999, 150, 1100], 4, 2, D, 32, fp8, window=window)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [3, 9, 2], [140, 129, 20]])
def test_softcap_and_scale(D, fp8, q_lens):
    check_attention(q_lens, [700, 333, 140], 8, 2, D, 16, fp8, softcap=5.0, scale=0.3)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [3, 9, 2], [140, 300, 20]])
def test_without_the_causal_mask(D, fp8, q_lens):
    """Cross attention to cached states of another length."""
    check_attention(q_lens, [1, 333, 1025], 8, 2, D, 16, fp8, causal=False)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_rows_that_see_nothing(D, fp8):
    """No cached positions at all, and more new tokens than positions."""
    check_attention([1, 2, 5, 150], [0, 0, 3, 100], 4, 2, D, 16, fp8)
    check_attention([3, 140], [0, 0], 4, 2, D, 16, fp8, causal=False)
    check_attention([0, 0, 1], [5, 0, 0], 4, 2, D, 16, fp8)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_lens", [[1], [6], [200]])
def test_sharp_scores(D, fp8, q_lens):
    """Scores far apart: the running maximum moves often and far."""
    check_attention(q_lens, [1777], 4, 1, D, 64, fp8, spread=12.0)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("q_len,window", [(1, 0), (150, 0), (300, 70), (300, 1)])
def test_scores_far_from_zero(D, fp8, sign, q_len, window):
    """Every score near +-230 (log2 units): nothing may lean on a reference of 0,
    in rows whose first keys come late neither."""
    n = 400
    base = rand_bf16(1, 1, D, seed=3).abs() + 0.5
    q = base.expand(q_len, 4, D).contiguous().cuda() + rand_bf16(q_len, 4, D, seed=4, scale=0.02).cuda()
    k = (base * sign).expand(n, 2, D) + rand_bf16(n, 2, D, seed=5, scale=0.05)
    v = rand_bf16(n, 2, D, seed=6)
    c = R.Paged([k.to(torch.bfloat16)], [v], 16, fp8)
    ws = attention_ws()
    scale = 160.0 / float((base.double() ** 2).sum())
    got, lse = L.paged_attention(q, c.k, c.v, c.table, cu([q_len]), i32([n]), ws, max_q=q_len,
                                 k_scales=c.ks, v_scales=c.vs, scale=scale, window=window, lse=True)
    assert L.get_error(ws) == L.MOE_OK
    want, want_l, tol, tol_l = R.attention(q, c, [q_len], [n], scale=scale, window=window)
    assert bool(((got.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - want_l).abs() <= tol_l).all())


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len", [1, 6, 13])
@pytest.mark.parametrize("gap,at,size", [(12.3, 0, 1.0), (13.5, 0, 1.0), (13.5, 0, 2.0 ** -6),
                                         (13.5, 5000, 1.0)])
def test_many_small_weights_beside_a_large_one(D, fp8, q_len, gap, at, size):
    """One key takes most of the weight, and 131071 others share the rest with equal weights
    (so that roundings do not cancel): what they add up to must not be lost.  One CTA has
    them all: the workspace has no room for a split."""
    n = 131072
    q = torch.ones(q_len, 8, D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(n, 1, D, dtype=torch.bfloat16)
    k[at] = gap / math.sqrt(D)
    v = (rand_bf16(1, 1, D, seed=2).abs() + 0.5).to(torch.bfloat16).expand(n, 1, D).clone()
    v[at] = (rand_bf16(1, D, seed=3) * size).to(torch.bfloat16)
    c = R.Paged([k], [v], 256, fp8)
    ws = L.new_workspace(L.ATTENTION_CTRL_BYTES)
    got, lse = L.paged_attention(q, c.k, c.v, c.table, cu([q_len]), i32([n]), ws, max_q=q_len,
                                 k_scales=c.ks, v_scales=c.vs, causal=False, lse=True)
    assert L.get_error(ws) == L.MOE_OK
    want, want_l, tol, tol_l = R.attention(q, c, [q_len], [n], causal=False)
    assert bool(((got.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - want_l).abs() <= tol_l).all())


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len", [1, 9, 40])
@pytest.mark.parametrize("at", [0, 200])
@pytest.mark.parametrize("small", [10, 14, 18])
def test_all_weight_on_a_small_value(D, fp8, q_len, at, small):
    """The key that takes (1 - e^-18 of) the weight has a value 2^-small of its neighbours':
    the output is that value, to the output's own rounding."""
    if fp8 and q_len * 4 > 64 and small == 18:
        pytest.skip("binary16 weights end at 2^-28 of the row's largest: the neighbours, with weights "
                    "of 2^-34.6, count as nothing, which shows in channels where the value is 0")
    n = 300
    q = torch.ones(q_len, 4, D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(n, 1, D, dtype=torch.bfloat16)
    k[at] = 24.0 / math.sqrt(D)
    v = rand_bf16(n, 1, D, seed=1)
    v[at] = (v[at].float() * 2.0 ** -small).to(torch.bfloat16)
    c = R.Paged([k], [v], 64, fp8)
    ws = attention_ws()
    got, lse = L.paged_attention(q, c.k, c.v, c.table, cu([q_len]), i32([n]), ws, max_q=q_len,
                                 k_scales=c.ks, v_scales=c.vs, causal=False, lse=True)
    assert L.get_error(ws) == L.MOE_OK
    want, want_l, tol, tol_l = R.attention(q, c, [q_len], [n], causal=False)
    assert bool(((got.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - want_l).abs() <= tol_l).all())


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len", [1, 9, 40])
@pytest.mark.parametrize("span", [3, 6, 10])
def test_value_rows_of_very_different_sizes(D, fp8, q_len, span):
    """Value rows of sizes 2^-span to 2^span in any order under sharp scores: a row whose
    weight lies on a small value, beside large ones of no weight, keeps its bits."""
    n = 3000
    for seed in range(2):
        g = torch.Generator().manual_seed(seed)
        k = torch.randn(n, 1, D, generator=g).to(torch.bfloat16)
        size = torch.exp2((torch.rand(n, 1, 1, generator=g) * 2 - 1) * span)
        v = (torch.randn(n, 1, D, generator=g) * size).to(torch.bfloat16)
        q = (torch.randn(q_len, 4, D, generator=g) * 3).to(torch.bfloat16).cuda()
        c = R.Paged([k], [v], 64, fp8, seed=seed)
        for ws in (attention_ws(), L.new_workspace(L.ATTENTION_CTRL_BYTES)):
            got, lse = L.paged_attention(q, c.k, c.v, c.table, cu([q_len]), i32([n]), ws,
                                         max_q=q_len, k_scales=c.ks, v_scales=c.vs, lse=True)
            assert L.get_error(ws) == L.MOE_OK
            want, want_l, tol, tol_l = R.attention(q, c, [q_len], [n])
            assert bool(((got.double() - want).abs() <= tol).all())
            assert bool(((lse.double() - want_l).abs() <= tol_l).all())


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("q_len", [1, 9, 40])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_pages_before_the_window_may_be_gone(D, fp8, page, q_len, softcap):
    """Pages wholly before the first token's window have left the table, and the positions
    of a page that are before it are NaN."""
    n, window = 1100, 300
    first = n - q_len - window + 1
    keys, vals = rand_bf16(n, 2, D, seed=1), rand_bf16(n, 2, D, seed=2)
    q = rand_bf16(q_len, 4, D, seed=3).cuda()
    c = R.Paged([keys], [vals], page, fp8)
    want, want_l, tol, tol_l = R.attention(q, c, [q_len], [n], window=window, softcap=softcap)
    for pos in range(first):
        pg = int(c.table[0, pos // page])
        for x in (c.k, c.v):
            x[pg, :, pos % page] = R.NAN_CODE if fp8 else math.nan
        for x in (c.ks, c.vs) if fp8 else ():
            x[pg, :, pos % page] = math.nan
    c.table[0, :first // page] = -1
    ws = attention_ws()
    got, lse = L.paged_attention(q, c.k, c.v, c.table, cu([q_len]), i32([n]), ws, max_q=q_len,
                                 k_scales=c.ks, v_scales=c.vs, window=window, softcap=softcap,
                                 lse=True)
    assert L.get_error(ws) == L.MOE_OK
    assert bool(((got.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - want_l).abs() <= tol_l).all())


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len", [1, 9, 40])
def test_an_infinite_value_leaves_lse_alone(D, fp8, q_len):
    n = 500
    k, v = rand_bf16(n, 1, D, seed=1), rand_bf16(n, 1, D, seed=2)
    v[200, 0, 3] = math.inf
    q = rand_bf16(q_len, 4, D, seed=3).cuda()
    c = R.Paged([k], [v], 16, fp8)
    ws = attention_ws()
    got, lse = L.paged_attention(q, c.k, c.v, c.table, cu([q_len]), i32([n]), ws, max_q=q_len,
                                 k_scales=c.ks, v_scales=c.vs, lse=True)
    assert L.get_error(ws) == L.MOE_OK
    _, want_l, _, tol_l = R.attention(q, c, [q_len], [n])
    assert not bool(torch.isfinite(got[..., 3].float()).any())
    assert bool(((lse.double() - want_l).abs() <= tol_l).all())


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len", [2, 150])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_a_nan_reaches_its_rows_and_no_others(D, fp8, q_len, softcap):
    """A NaN in one query row, and in a key that only the last rows see: those rows
    are NaN, the rows before it are not (scores are masked before they meet a sum)."""
    n = 300
    k, v = rand_bf16(n, 1, D, seed=1), rand_bf16(n, 1, D, seed=2)
    k[n - 1, 0, 5] = math.nan
    q = rand_bf16(q_len, 2, D, seed=3)
    q[0, 1, 7] = math.nan
    c = R.Paged([k.nan_to_num(0.0)], [v], 16, fp8)
    last = R.Paged([k], [v], 16, False) if not fp8 else None
    if fp8:                                   # the NaN code in the last key
        pos = n - 1
        c.k[c.table[0, pos // 16], 0, pos % 16, 5] = R.NAN_CODE
    else:
        c = last
    ws = attention_ws()
    out, lse = L.paged_attention(q.cuda(), c.k, c.v, c.table, cu([q_len]), i32([n]), ws, max_q=q_len,
                                 k_scales=c.ks, v_scales=c.vs, softcap=softcap, lse=True)
    assert L.get_error(ws) == L.MOE_OK
    bad = torch.isnan(out.float()).all(-1).cpu()
    some = torch.isnan(out.float()).any(-1).cpu()
    want = torch.zeros(q_len, 2, dtype=torch.bool)
    want[0, 1] = True
    want[q_len - 1] = True
    assert torch.equal(some, want) and torch.equal(bad, want)
    assert torch.equal(torch.isnan(lse).cpu(), want)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_negative_scale(D, fp8):
    check_attention([3, 200], [300, 333], 4, 2, D, 32, fp8, scale=-0.11)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_long_caches_are_split(D, fp8):
    check_attention([1], [40000], 8, 1, D, 64, fp8)
    check_attention([2, 1, 20], [20000, 13, 9000], 8, 2, D, 64, fp8)


@pytest.mark.parametrize("q_lens", [[1, 1], [30, 30], [200, 200]])
def test_hint_and_workspace_do_not_change_the_result(q_lens):
    """A hint far off, a small workspace, another stream."""
    args = (q_lens, [3001, 700], 8, 2, 128, 64, True)
    a = check_attention(*args)
    small = L.new_workspace(L.ATTENTION_CTRL_BYTES)
    for kw in (dict(max_kv=1), dict(max_kv=0), dict(ws=small), dict(stream=torch.cuda.Stream())):
        torch.cuda.synchronize()
        b = check_attention(*args, **kw)
        assert (a - b).abs().max().item() <= 2.0 ** -6 * a.abs().max().item()
    assert torch.equal(a, check_attention(*args)), "the same call again gives other bits"


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("q", [1, 40])
def test_offsets_past_32_bits(fp8, q):
    """The used pages lie beyond the first 4 GiB of each of k and v."""
    D, H, page = 128, 4, 64
    per_page = H * page * D * (1 if fp8 else 2)
    n_pages = (5 << 30) // per_page
    k = torch.empty(n_pages, H, page, D, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ks = torch.empty(n_pages, H, page, device="cuda") if fp8 else None
    vs = torch.empty(n_pages, H, page, device="cuda") if fp8 else None
    n = 200
    ids = [n_pages - 1, n_pages - 7, n_pages - 3, n_pages - 5]
    new_k, new_v = rand_bf16(n, H, D, seed=1).cuda(), rand_bf16(n, H, D, seed=2).cuda()
    table = i32([ids])
    pos = torch.arange(n, device="cuda")
    slots = (table[0].long()[pos // page] * page + pos % page).to(torch.int32)
    ws = attention_ws()
    L.kv_write(new_k, new_v, slots, k, v, ws, k_scales=ks, v_scales=vs)
    qq = rand_bf16(q, 8, D, seed=3).cuda()
    out, lse = L.paged_attention(qq, k, v, table, cu([q]), i32([n]), ws, max_q=q, k_scales=ks,
                                 v_scales=vs, lse=True)
    back, _ = L.kv_read(k, v, table, cu([n]), n, ws, k_scales=ks, v_scales=vs)
    assert L.get_error(ws) == L.MOE_OK
    c = R.Paged([new_k.cpu()], [new_v.cpu()], page, fp8)
    assert torch.equal(back, c.rows("k", 0, n).float().to(torch.bfloat16))
    want, want_l, tol, tol_l = R.attention(qq, c, [q], [n])
    assert bool(((out.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - want_l).abs() <= tol_l).all())


@pytest.mark.parametrize("q", [1, 64])
def test_attention_reports_what_is_out_of_range(q):
    D, H, page = 128, 1, 16
    k = [rand_bf16(64, H, D)]
    c = R.Paged(k, k, page, True)
    x = rand_bf16(q, 4, D).cuda()

    def status(table, cu_q, lens):
        ws = attention_ws()
        L.paged_attention(x, c.k, c.v, table, cu_q, lens, ws, max_q=q, k_scales=c.ks, v_scales=c.vs)
        return L.get_error(ws)

    good = c.table[:, :4].contiguous()
    assert status(good, cu([q]), i32([64])) == L.MOE_OK
    bad = good.clone()
    bad[0, 2] = c.k.shape[0]
    assert status(bad, cu([q]), i32([64])) == L.MOE_ERR_DEVICE_FAULT
    bad[0, 2] = -5
    assert status(bad, cu([q]), i32([64])) == L.MOE_ERR_DEVICE_FAULT
    assert status(good, cu([q]), i32([65])) == L.MOE_ERR_DEVICE_FAULT
    assert status(good, cu([q]), i32([-1])) == L.MOE_ERR_DEVICE_FAULT
    assert status(good, i32([0, q + 1]), i32([64])) == L.MOE_ERR_DEVICE_FAULT
    assert status(good, i32([-1, q - 1]), i32([64])) == L.MOE_ERR_DEVICE_FAULT
    assert status(good, i32([1, 0]), i32([64])) == L.MOE_ERR_DEVICE_FAULT
    assert status(good, cu([q]), i32([64])) == L.MOE_OK


# ------------------------------------------------------------------ verification
def draft_case(B, n, V, dtype, seed=0, near=0.5):
    g = torch.Generator().manual_seed(seed)
    base = torch.randn(B, n + 1, V, generator=g) * 2
    p = torch.softmax(base, -1).to(dtype)
    q = torch.softmax(base[:, :n] + near * torch.randn(B, n, V, generator=g), -1).to(dtype)
    draft = torch.multinomial(q.float().view(-1, V), 1, generator=g).view(B, n).to(torch.int32)
    u = torch.rand(B, n, generator=g)
    us = torch.rand(B, generator=g)
    lens = torch.tensor([n - (b % 3) if n > 2 else n for b in range(B)], dtype=torch.int32)
    return p, q, draft, lens, u, us


def run_verify(p, q, draft, lens, u, us, ws=None):
    ws = ctrl() if ws is None else ws
    dev = [t.cuda() for t in (p, q, draft, u, us)]
    a, t = L.verify_draft(*dev[:3], dev[3], dev[4], ws,
                          draft_lens=None if lens is None else lens.cuda())
    return a.cpu(), t.cpu(), L.get_error(ws)


@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (2, 3, 2), (3, 4, 31), (5, 2, 33), (7, 8, 1000),
                                   (40, 5, 4099), (2, 32, 20001), (1, 4, 65536)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_is_exact(B, n, V, dtype):
    case = draft_case(B, n, V, dtype, seed=V)
    p, q, draft, lens, u, us = case
    a, t, status = run_verify(*case)
    wa, wt = R.verify(*case)
    assert status == L.MOE_OK
    assert torch.equal(a, wa) and torch.equal(t, wt)


def test_verify_edges():
    B, n, V = 9, 3, 500
    p, q, draft, lens, u, us = draft_case(B, n, V, torch.float32, seed=3)
    lens = torch.tensor([0, 1, 2, 3, 3, 3, 3, 3, 3], dtype=torch.int32)
    q[3] = p[3, :n]                                       # equal: all accepted
    us[3] = 0.0
    us[4], u[4] = 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -24
    p[5, 0, int(draft[5, 0])] = 0.0                       # refused at once
    p[6] = 0.0                                            # no weight anywhere
    p[7, 0, 17] = math.nan
    u[7, 0] = 1.0 - 2.0 ** -24
    q[8, 0] = 2.0 * p[8, 0]                               # no residual weight: drawn from p itself
    u[8, 0] = 0.75
    a, t, status = run_verify(p, q, draft, lens, u, us)
    wa, wt = R.verify(p, q, draft, lens, u, us)
    assert status == L.MOE_OK
    assert torch.equal(a, wa) and torch.equal(t, wt)
    assert int(a[0]) == 0 and int(a[3]) == 3 and int(a[5]) == 0 and int(t[6, 0]) == -1


def test_verify_strides_and_streams():
    B, n, V = 6, 4, 777
    p, q, draft, lens, u, us = draft_case(B, n, V, torch.float32, seed=9)
    both = torch.full((B, 2 * n + 2, V + 3), math.nan).cuda()
    both[:, :n + 1, 1:V + 1] = p.cuda()
    both[:, n + 1:2 * n + 1, 2:V + 2] = q.cuda()
    ws = ctrl()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, t = L.verify_draft(both[:, :n + 1, 1:V + 1], both[:, n + 1:2 * n + 1, 2:V + 2], draft.cuda(),
                          u.cuda(), us.cuda(), ws, draft_lens=lens.cuda(), stream=s)
    s.synchronize()
    wa, wt = R.verify(p, q, draft, lens, u, us)
    assert torch.equal(a.cpu(), wa) and torch.equal(t.cpu(), wt)


def test_verify_draws_by_the_residual_distribution():
    """Over many given random numbers the output's first token follows p."""
    V, N = 8, 20000
    g = torch.Generator().manual_seed(0)
    p1, q1 = torch.softmax(torch.randn(V, generator=g), 0), torch.softmax(torch.randn(V, generator=g), 0)
    p = p1.expand(N, 2, V).contiguous()
    q = q1.expand(N, 1, V).contiguous()
    draft = torch.multinomial(q1, N, replacement=True, generator=g).view(N, 1).to(torch.int32)
    a, t, _ = run_verify(p, q, draft, None, torch.rand(N, 1, generator=g), torch.rand(N, generator=g))
    freq = torch.bincount(t[:, 0].long(), minlength=V).double() / N
    # five standard deviations of a frequency
    assert bool(((freq - p1.double()).abs() < 5 * (p1 * (1 - p1) / N).sqrt()).all())


def test_verify_reports_bad_tokens():
    case = list(draft_case(2, 2, 100, torch.float32))
    for bad in (-1, 100):
        case[2] = case[2].clone()
        case[2][1, 0] = bad
        a, t, status = run_verify(*case)
        assert status == L.MOE_ERR_DEVICE_FAULT and int(a[1]) == 0
    case = list(draft_case(2, 2, 100, torch.float32))
    case[3] = torch.tensor([3, 1], dtype=torch.int32)
    assert run_verify(*case)[2] == L.MOE_ERR_DEVICE_FAULT
