"""Attention over the paged cache where it can go wrong: rows of the dispatch's edges, calls in
which the groups of the few-row form disagree about a second pass, windows and values at the ends
of their types, batches of unlike sequences (against 64 bits)."""
import math

import pytest
import torch

import serving_reference as R
from gpu_helpers import ensure_built
from mixture_experts_forward_gb300 import _lib as L

pytestmark = pytest.mark.gpu

FORMS = [(64, False), (64, True), (128, False), (128, True)]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.fixture(scope="module")
def ws(built):
    return L.new_workspace(L.ATTENTION_WS_BYTES)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return i32(at)


def rand_bf16(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def attend(q, c, q_lens, kv_lens, ws, **kw):
    """(out, lse) of a call that records no fault and leaves its counters zero."""
    got = L.paged_attention(q, c.k, c.v, c.table, cu(q_lens), i32(kv_lens), ws, max_q=max(q_lens),
                            k_scales=c.ks, v_scales=c.vs, lse=True, **kw)
    assert L.get_error(ws) == L.MOE_OK
    assert not bool(ws[L.CTRL_BYTES:L.ATTENTION_CTRL_BYTES].any()), "counters left behind"
    return got


def within(got, want, tol):
    """got is within tol of want, and as infinite as want."""
    got = got.double()
    inf = torch.isinf(want)
    return torch.equal(got[inf], want[inf]) and bool(((got - want).abs() <= tol)[~inf].all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,Hq", [(1, 16), (5, 8), (12, 4), (15, 4)])
def test_groups_that_disagree_about_a_second_pass(D, q_len, Hq, ws):
    """FP8, few rows: key tiles whose weights are small for some rows and large for others, in
    an order that changes from tile to tile, so that some warps take a second pass in nearly every
    tile and others in none.  Repeated calls give the same bits."""
    n = 128 * 60 + 17
    g = torch.Generator().manual_seed(D + q_len)
    k = torch.randn(n, 1, D, generator=g) * 0.3
    # channel x is strong in some key tiles, and query row x looks at channel x
    level = torch.randn(60 + 1, D, generator=g) * 3
    k += level.repeat_interleave(128, 0)[:n, None, :]
    q = torch.randn(q_len, Hq, D, generator=g) * 0.05
    for r in range(q_len * Hq):
        q[r // Hq, r % Hq, r % D] += 12.0
    c = R.Paged([k.to(torch.bfloat16)], [rand_bf16(n, 1, D, seed=3)], 64, True)
    q = q.to(torch.bfloat16).cuda()
    want, want_l, tol, tol_l = R.attention(q, c, [q_len], [n])
    one = L.new_workspace(L.ATTENTION_CTRL_BYTES)             # no room for a split: one CTA
    for w in (one, ws):
        first = attend(q, c, [q_len], [n], w)
        assert within(first[0], want, tol) and within(first[1], want_l, tol_l)
        for _ in range(50):
            again = attend(q, c, [q_len], [n], w)
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len", [1, 9, 70])
@pytest.mark.parametrize("fp8", [True, False])
def test_small_query_elements_beside_a_large_one(D, q_len, fp8, ws):
    """The scores come from elements between 2^-10.3 and 2^-6.9 of their row's largest, which
    meets keys of 0: the query's terms hold them exactly."""
    n = 300
    g = torch.Generator().manual_seed(q_len)
    q = (torch.rand(q_len, 4, D, generator=g) * 0.09 + 0.01) * (torch.randint(0, 2, (q_len, 4, D), generator=g) * 2 - 1)
    q[..., 5] = 12.0
    k = 1.0 + 0.1 * torch.randn(n, 1, D, generator=g)
    k[..., 5] = 0.0
    c = R.Paged([k.to(torch.bfloat16)], [rand_bf16(n, 1, D, seed=3)], 64, fp8)
    q = q.to(torch.bfloat16).cuda()
    want, want_l, tol, tol_l = R.attention(q, c, [q_len], [n])
    out, lse = attend(q, c, [q_len], [n], ws)
    assert within(out, want, tol) and within(lse, want_l, tol_l)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len,Hq", [(12, 2), (15, 8), (150, 2), (300, 4)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100])
def test_a_window_as_wide_as_it_can_be(D, fp8, q_len, Hq, window, ws):
    """Wider than any cache: the rows see what they see without one, where a sequence has more
    new tokens than positions too."""
    kv = [8, 100, 700]
    lens = [q_len, q_len, min(q_len, 20)]
    c = R.Paged([rand_bf16(n, 2, D, seed=n) for n in kv], [rand_bf16(n, 2, D, seed=n + 1) for n in kv],
                32, fp8)
    q = rand_bf16(sum(lens), Hq, D, seed=3).cuda()
    out, lse = attend(q, c, lens, kv, ws, window=window)
    want, want_l, tol, tol_l = R.attention(q, c, lens, kv)
    assert within(out, want, tol) and within(lse, want_l, tol_l)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_lens,kv,Hq,page", [([1], [40000], 8, 64), ([30, 3], [9000, 40], 4, 16),
                                               ([150, 20], [6000, 700], 4, 32), ([12, 12], [8, 100], 2, 32),
                                               ([300, 20], [100, 700], 4, 32)])
def test_a_window_wider_than_the_cache_is_none(D, fp8, q_lens, kv, Hq, page, ws):
    """The same split as without a window, so the same bits: 2^31 - 1, and just as wide as the
    table's positions."""
    c = R.Paged([rand_bf16(n, 1, D, seed=n) for n in kv], [rand_bf16(n, 1, D, seed=n + 1) for n in kv],
                page, fp8)
    q = rand_bf16(sum(q_lens), Hq, D, seed=3).cuda()
    plain, plain_lse = attend(q, c, q_lens, kv, ws)
    for window in (2 ** 31 - 1, 2 ** 31 - 100, c.table.shape[1] * page):
        out, lse = attend(q, c, q_lens, kv, ws, window=window)
        assert torch.equal(out, plain) and torch.equal(lse, plain_lse)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("q_len,Hq", [(15, 2), (15, 8), (40, 2), (120, 2), (300, 2)])
def test_rows_that_see_nothing_beside_a_bad_value(D, fp8, bad, q_len, Hq, ws):
    """More new tokens than positions, and a value row that is not finite: the rows that see no
    key give 0 and -inf, whatever lies in a value."""
    n = 9
    k, v = rand_bf16(n, 1, D, seed=1), rand_bf16(n, 1, D, seed=2)
    c = R.Paged([k], [v], 16, fp8)
    pg, at = int(c.table[0, 0]), 4
    if fp8:
        c.v[pg, 0, at, 5] = R.NAN_CODE if math.isnan(bad) else 0x7e
        c.vs[pg, 0, at] = bad
    else:
        c.v[pg, 0, at, 5] = bad
    q = rand_bf16(q_len, Hq, D, seed=3).cuda()
    for w in (ws, L.new_workspace(L.ATTENTION_CTRL_BYTES)):
        out, lse = attend(q, c, [q_len], [n], w)
        assert bool((out[:q_len - n] == 0).all()) and bool((lse[:q_len - n] == -math.inf).all())
        assert bool(torch.isfinite(lse[q_len - n:]).all())
        assert not bool(torch.isfinite(out[-1, :, 5]).any())


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len,Hq", [(1, 4), (6, 4), (13, 4), (40, 4), (300, 1)])
@pytest.mark.parametrize("n,low", [(700, 100), (700, 300), (9000, 6000)])
@pytest.mark.parametrize("value", [-3e38, -math.inf])
def test_first_keys_as_low_as_their_type_goes(D, fp8, q_len, Hq, n, low, value, ws):
    """The first `low` keys score -inf in binary32 (weight 0), and all others near -160: nothing
    may lean on a reference of 0, neither in one CTA nor where parts are joined.  The result is
    that of the other keys alone."""
    if fp8 and math.isinf(value):
        pytest.skip("a row with an infinity has an infinite scale and reads back as NaN")
    base = rand_bf16(1, 1, D, seed=3).abs() + 0.5
    base[..., 0] = 0
    q = base.expand(q_len, Hq, D) + rand_bf16(q_len, Hq, D, seed=4, scale=0.02)
    q[..., 0] = 12.0
    k = -base.expand(n, 1, D) + rand_bf16(n, 1, D, seed=5, scale=0.05)
    k[..., 0] = 0
    k[:low, 0, 0] = value
    k, v, q = k.to(torch.bfloat16), rand_bf16(n, 1, D, seed=6), q.to(torch.bfloat16).cuda()
    scale = 160.0 / float((base.double() ** 2).sum())
    c, rest = R.Paged([k], [v], 64, fp8), R.Paged([k[low:]], [v[low:]], 64, fp8)
    want, want_l, tol, tol_l = R.attention(q, rest, [q_len], [n - low], scale=scale, causal=False)
    for w in (ws, L.new_workspace(L.ATTENTION_CTRL_BYTES)):
        out, lse = attend(q, c, [q_len], [n], w, scale=scale, causal=False)
        assert within(out, want, tol) and within(lse, want_l, tol_l)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len", [1, 9, 150])
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_an_infinite_query_element(D, fp8, q_len, bad, softcap, ws):
    """Its scores are infinities of both signs: without a cap the row is NaN.  (Capped, BF16
    scores of +-c are numbers; over an FP8 cache the row is NaN either way.)  Other rows are not
    touched, and a row that sees nothing stays 0."""
    n, at = 300, q_len - 1
    k, v = rand_bf16(n, 1, D, seed=1), rand_bf16(n, 1, D, seed=2)
    q = rand_bf16(q_len, 2, D, seed=3)
    c = R.Paged([k], [v], 16, fp8)
    want, want_l, tol, tol_l = R.attention(q.cuda(), c, [q_len], [n], softcap=softcap)
    q[at, 1, 7] = bad
    out, lse = attend(q.cuda(), c, [q_len], [n], ws, softcap=softcap)
    others = torch.ones(q_len, 2, dtype=torch.bool)
    others[at, 1] = False
    assert within(out[others], want[others], tol[others])
    assert within(lse[others], want_l[others], tol_l[others])
    if fp8 or not softcap:
        assert bool(torch.isnan(out[at, 1]).all()) and bool(torch.isnan(lse[at, 1]))
    out, lse = attend(q.cuda(), c, [q_len], [0], ws, softcap=softcap)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len", [1, 9, 40, 150])
@pytest.mark.parametrize("small", [0.0, 1e-25])
@pytest.mark.parametrize("tiles", [(0,), (2,), (1, 3), (4,)])
def test_a_key_tile_of_zero_values_beside_large_ones(D, fp8, q_len, small, tiles, ws):
    """Values near 1e20, but for whole key tiles of (nearly) zero ones: their weights count in
    the sum all the same."""
    n = 128 * 5
    k, v = rand_bf16(n, 1, D, seed=1), rand_bf16(n, 1, D, seed=2).float() * 1e20
    for t in tiles:
        v[128 * t:128 * t + 128] *= small / 1e20
    q = rand_bf16(q_len, 4, D, seed=3).cuda()
    c = R.Paged([k], [v.to(torch.bfloat16)], 64, fp8)
    for causal in (True, False):
        want, want_l, tol, tol_l = R.attention(q, c, [q_len], [n], causal=causal)
        for w in (ws, L.new_workspace(L.ATTENTION_CTRL_BYTES)):
            out, lse = attend(q, c, [q_len], [n], w, causal=causal)
            assert within(out, want, tol) and within(lse, want_l, tol_l)


@pytest.mark.parametrize("B", [0, 2])
def test_a_call_without_rows(B, ws):
    c = R.Paged([rand_bf16(20, 1, 64)] * 2, [rand_bf16(20, 1, 64)] * 2, 16, True)
    out, lse = L.paged_attention(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), c.k, c.v,
                                 c.table[:B], cu([0] * B), i32([20] * B), ws, max_q=0,
                                 k_scales=c.ks, v_scales=c.vs, lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4) and L.get_error(ws) == L.MOE_OK


@pytest.mark.parametrize("name", ["write", "read", "attention", "verify"])
def test_each_tensor_must_be_on_the_gpu(name):
    """One tensor at a time left in host memory, and a workspace without room for its status."""
    from test_serving_binding import all_calls
    call, host = all_calls()[name]
    on = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in host.items()}
    if name == "verify":
        on["q"] = on["p"][:, :3]
    call(**on)
    assert L.get_error(on["ws"]) in (L.MOE_OK, L.MOE_ERR_DEVICE_FAULT)   # (lengths of 0: no rows)
    for key, v in host.items():
        if isinstance(v, torch.Tensor):
            with pytest.raises(L.MoeError, match="on one GPU"):
                call(**dict(on, **{key: v}))
    with pytest.raises(L.MoeError) as e:
        call(**dict(on, ws=torch.zeros(128, dtype=torch.uint8, device="cuda")))
    assert e.value.code == L.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("fp8", [True, False])
def test_dimensions_of_one_have_any_stride(fp8, ws):
    """One token, or one head: views whose stride there is no multiple of 8."""
    D, n = 64, 40
    k, v = rand_bf16(n, 1, D, seed=1), rand_bf16(n, 1, D, seed=2)
    c = R.Paged([k], [v], 16, fp8)
    q = rand_bf16(1, 4, D, seed=3).cuda()
    want, want_l = attend(q, c, [1], [n], ws)

    def odd(x, dim):                                    # the same values, a stride of 12 at dim
        shape, stride = list(x.shape), list(x.stride())
        stride[dim] = 12
        return x.as_strided(shape, stride)
    out, lse = attend(odd(q, 0), c, [1], [n], ws, out=odd(torch.empty_like(q), 0))
    assert torch.equal(out, want) and torch.equal(lse, want_l)
    one = q[:, :1].contiguous()
    out, lse = attend(odd(one, 1), c, [1], [n], ws, out=odd(torch.empty_like(one), 1))
    assert torch.equal(out, want[:, :1]) and torch.equal(lse, want_l[:, :1])
    for T, dim in ((1, 0), (5, 1)):
        new = rand_bf16(T, 1, D, seed=4).cuda()
        slots = torch.arange(T, dtype=torch.int32, device="cuda")
        pages = [L.new_kv_cache(L.DTYPE_FP8 if fp8 else L.DTYPE_BF16, 1, 16, 1, D) for _ in range(2)]
        for x, (kc, vc, ks, vs) in zip((new, odd(new, dim)), pages):
            L.kv_write(x, x, slots, kc, vc, ws, k_scales=ks, v_scales=vs)
        assert all(torch.equal(a, b) for a, b in zip(*pages) if a is not None)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("q_lens", [[1, 3], [1, 90]])
def test_block_tables_that_are_columns_of_a_wider_one(fp8, q_lens, ws):
    kv, D = [300, 211], 64
    c = R.Paged([rand_bf16(n, 1, D, seed=n) for n in kv], [rand_bf16(n, 1, D, seed=n + 1) for n in kv],
                16, fp8)
    q = rand_bf16(sum(q_lens), 4, D, seed=3).cuda()
    want = attend(q, c, q_lens, kv, ws)
    rows = L.kv_read(c.k, c.v, c.table, cu(kv), sum(kv), ws, k_scales=c.ks, v_scales=c.vs)
    w = c.table.shape[1]
    wide = torch.full((3, w + 9), -1, dtype=torch.int32, device="cuda")
    wide[:2, :w] = c.table
    c.table = wide[:2, :w]
    got = attend(q, c, q_lens, kv, ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    back = L.kv_read(c.k, c.v, c.table, cu(kv), sum(kv), ws, k_scales=c.ks, v_scales=c.vs)
    assert torch.equal(back[0], rows[0]) and torch.equal(back[1], rows[1])
    # rows that would run past the storage, that overlap, or that are not contiguous
    for bad in (wide[1:, 1:w + 1], c.table[:1].expand(2, w), wide[:2, :2 * (w // 2):2]):
        with pytest.raises(L.MoeError):
            L.paged_attention(q, c.k, c.v, bad, cu(q_lens), i32(kv), ws, max_q=max(q_lens),
                              k_scales=c.ks, v_scales=c.vs)


@pytest.mark.parametrize("q_lens", [[1, 2], [90, 1]])
@pytest.mark.parametrize("D,fp8", FORMS)
def test_a_block_table_without_entries(D, fp8, q_lens, ws):
    """Sequences with no cached position at all (states that are still empty)."""
    c = R.Paged([rand_bf16(20, 1, D)], [rand_bf16(20, 1, D)], 16, fp8)
    q = rand_bf16(sum(q_lens), 4, D, seed=3).cuda()
    c.table = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    out, lse = attend(q, c, q_lens, [0, 0], ws, causal=False)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    L.paged_attention(q, c.k, c.v, c.table, cu(q_lens), i32([0, 1]), ws, max_q=max(q_lens),
                      k_scales=c.ks, v_scales=c.vs)
    assert L.get_error(ws) == L.MOE_ERR_DEVICE_FAULT
    k, _ = L.kv_read(c.k, c.v, c.table, cu([0, 2]), 2, ws, k_scales=c.ks, v_scales=c.vs)
    assert L.get_error(ws) == L.MOE_ERR_DEVICE_FAULT and bool((k == 0).all())


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len", [1, 6, 12, 40])
@pytest.mark.parametrize("zeros", [128, 256, 300])
@pytest.mark.parametrize("size", [1.0, 4000.0, 1e30])
def test_first_values_of_zero_and_later_ones_of_no_weight(D, fp8, q_len, zeros, size, ws):
    """All weight is on the first keys, whose values are 0; the others score 200 lower.  The
    output is 0 and lse that of the first keys, however large the other values are."""
    n = 700
    k = torch.zeros(n, 1, D)
    k[:zeros, 0, 0] = 200.0 / math.sqrt(D)
    v = rand_bf16(n, 1, D, seed=2).float() * size
    v[:zeros] = 0
    q = torch.zeros(q_len, 4, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = float(D)
    c = R.Paged([k.to(torch.bfloat16)], [v.to(torch.bfloat16)], 64, fp8)
    for causal in (True, False):
        _, want_l, _, tol_l = R.attention(q, c, [q_len], [n], causal=causal)
        for w in (ws, L.new_workspace(L.ATTENTION_CTRL_BYTES)):
            out, lse = attend(q, c, [q_len], [n], w, causal=causal)
            assert bool((out == 0).all()) and within(lse, want_l, tol_l)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len", [1, 6, 12, 40, 150])
@pytest.mark.parametrize("rise", [10.0, 20.0, 38.0, 100.0])
def test_large_values_under_rising_scores(D, fp8, q_len, rise, ws):
    """Values near 1e23 whose keys score `rise` more after the first tile, and as much again after
    the second: sums of weights times values stay finite."""
    n = 128 * 5
    k, v = rand_bf16(n, 1, D, seed=1).float() * 0.3, rand_bf16(n, 1, D, seed=2).float() * 1e23
    k[..., 0] = 0
    k[128:256, 0, 0] = 1.0
    k[256:, 0, 0] = 2.0
    q = rand_bf16(q_len, 4, D, seed=3)
    q[..., 0] = rise * math.sqrt(D)
    c = R.Paged([k.to(torch.bfloat16)], [v.to(torch.bfloat16)], 64, fp8)
    q = q.cuda()
    for causal in (True, False):
        want, want_l, tol, tol_l = R.attention(q, c, [q_len], [n], causal=causal)
        for w in (ws, L.new_workspace(L.ATTENTION_CTRL_BYTES)):
            out, lse = attend(q, c, [q_len], [n], w, causal=causal)
            assert within(out, want, tol) and within(lse, want_l, tol_l)
