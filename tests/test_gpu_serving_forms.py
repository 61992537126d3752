"""Attention over the paged cache against the bounds of each form's own roundings, at the sizes
where one form ends and the next begins: 1 to 64 rows (tiles of 16, 32, 48 and 64), 65 and more."""
import pytest
import torch

import serving_forms as F
import serving_reference as R
from gpu_helpers import ensure_built
from mixture_experts_forward_gb300 import _lib as L
from test_gpu_serving_edges import FORMS, attend, i32, cu, rand_bf16, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.fixture(scope="module")
def workspaces(built):
    """Room for every split, and for none."""
    return L.new_workspace(L.ATTENTION_WS_BYTES), L.new_workspace(L.ATTENTION_CTRL_BYTES)


# (new tokens of the longest sequence, query heads per cache head): their product is the rows
ROWS = {1: (1, 1), 16: (4, 4), 17: (17, 1), 32: (8, 4), 33: (11, 3), 48: (12, 4), 49: (7, 7),
        50: (10, 5), 63: (9, 7), 64: (16, 4), 65: (13, 5), 96: (24, 4), 129: (43, 3)}


def check(q_lens, kv_lens, G, Hkv, D, page, fp8, workspaces, **kw):
    c = R.Paged([rand_bf16(n, Hkv, D, seed=n) for n in kv_lens],
                [rand_bf16(n, Hkv, D, seed=n + 1) for n in kv_lens], page, fp8)
    packed = rand_bf16(sum(q_lens), G * Hkv + 2, D, seed=7).cuda()
    q = packed[:, 1:G * Hkv + 1]
    want, want_l, tol, tol_l = F.attention(q, c, q_lens, kv_lens, **kw)
    for ws in workspaces:
        out, lse = attend(q, c, q_lens, kv_lens, ws, **kw)
        assert within(out, want, tol) and within(lse, want_l, tol_l)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kw", [dict(), dict(window=100), dict(softcap=5.0, scale=0.3),
                                dict(causal=False)], ids=["causal", "window", "cap", "full"])
def test_rows_at_the_edges_of_the_forms(D, fp8, rows, kw, workspaces):
    """One sequence of so many rows, then shorter ones (whole groups of rows idle), one with
    fewer positions than tokens and one of none."""
    n, G = ROWS[rows]
    check([n, 1, max(1, n // 2), n, 0], [900, 130, 511, 3, 40], G, 2, D, 32, fp8, workspaces, **kw)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("rows", [49, 64, 65])
def test_long_caches_at_the_edges_of_the_forms(D, fp8, rows, workspaces):
    n, G = ROWS[rows]
    check([n, 2], [9000, 3333], G, 1, D, 64, fp8, workspaces)
    check([1], [5000], rows, 1, D, 16, fp8, workspaces)          # one token, so many query heads


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len,G", [(1, 4), (5, 4), (10, 4), (16, 4), (33, 4), (70, 4)])
def test_roundings_that_agree(D, fp8, q_len, G, workspaces):
    """Every weight is rounded the same way, so a form that dropped its low term would be a whole
    unit off (test_serving_bounds.py shows that the bounds see it)."""
    q, c, scale = F.same_sign_case(q_len, G, D, fp8, "cuda")
    want, want_l, tol, tol_l = F.attention(q, c, [q_len], [2001], scale=scale, causal=False)
    for ws in workspaces:
        out, lse = attend(q, c, [q_len], [2001], ws, scale=scale, causal=False)
        assert within(out, want, tol) and within(lse, want_l, tol_l)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_len,G", [(7, 7), (16, 4)])
def test_a_stalled_pipeline_of_the_64_row_form(D, fp8, q_len, G, workspaces):
    """No loads are issued: every wait runs out, the status says so, the next call is right.  (Over
    an FP8 cache these rows go to the 256-row tiles.)"""
    n = 2000
    c = R.Paged([rand_bf16(n, 1, D, seed=1)], [rand_bf16(n, 1, D, seed=2)], 16, fp8)
    q = rand_bf16(q_len, G, D, seed=3).cuda()
    for ws in workspaces:
        good = attend(q, c, [q_len], [n], ws)
        try:
            L.debug_set_pipeline_fault(True, 2_000_000)
            L.paged_attention(q, c.k, c.v, c.table, cu([q_len]), i32([n]), ws, max_q=q_len,
                              k_scales=c.ks, v_scales=c.vs)
            assert L.get_error(ws) == L.MOE_ERR_TIMEOUT
        finally:
            L.debug_set_pipeline_fault(False)
        again = attend(q, c, [q_len], [n], ws)
        assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("q_lens,kv_lens", [([700, 1], [700, 9000]), ([1, 1, 1, 600, 5], [5000, 77, 8000, 900, 4000]),
                                            ([300, 1, 0, 130], [8192, 8192, 100, 130])])
def test_chunks_and_single_tokens_in_one_call(D, fp8, q_lens, kv_lens, workspaces):
    """Single tokens over long caches beside a chunk: all are taken in the chunk's form."""
    for kw in (dict(), dict(window=1000), dict(max_kv=max(kv_lens))):
        hint = kw.pop("max_kv", 0)
        c = R.Paged([rand_bf16(n, 2, D, seed=n) for n in kv_lens],
                    [rand_bf16(n, 2, D, seed=n + 1) for n in kv_lens], 64, fp8)
        q = rand_bf16(sum(q_lens), 8, D, seed=7).cuda()
        want, want_l, tol, tol_l = F.attention(q, c, q_lens, kv_lens, **kw)
        for ws in workspaces:
            out, lse = attend(q, c, q_lens, kv_lens, ws, max_kv=hint, **kw)
            assert within(out, want, tol) and within(lse, want_l, tol_l)
