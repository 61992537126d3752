"""The serving operators' refusals, on the host before any CUDA call (CPU only)."""
import ctypes
import math

import pytest
import torch

from mixture_experts_forward_gb300 import _lib as L
from mixture_experts_forward_gb300 import build as moe_build

FAKE = 1 << 20   # a non-null, aligned fake device address; never dereferenced
INV, UNS, WS, OK = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE, L.MOE_OK


@pytest.fixture(scope="module", autouse=True)
def built():
    moe_build.build()


def cache(**kw):
    base = dict(dtype=L.DTYPE_FP8, num_pages=4, page_size=16, heads=2, head_dim=64, k=FAKE, v=FAKE,
                k_scales=FAKE, v_scales=FAKE)
    base.update(kw)
    return L.KvCache(*[base[n] for n, _ in L.KvCache._fields_])


BAD_CACHES = [(dict(k=None), INV), (dict(v=None), INV), (dict(k=FAKE + 8), INV),
              (dict(k_scales=None), INV), (dict(v_scales=FAKE + 2), INV), (dict(dtype=2), INV),
              (dict(num_pages=0), INV), (dict(heads=0), INV), (dict(page_size=0), INV),
              (dict(page_size=8), UNS), (dict(page_size=48), UNS), (dict(page_size=512), UNS),
              (dict(head_dim=96), UNS), (dict(head_dim=256), UNS),
              (dict(num_pages=1 << 30, page_size=256), UNS)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_caches_that_are_refused(kw, code):
    P = ctypes.c_void_p(FAKE)
    c = cache(**kw)
    assert L.lib().moe_kv_write(c, P, P, 1, 128, 64, 128, 64, P, P, None) == code
    assert L.lib().moe_kv_read(c, P, 4, P, None, 1, 1, P, P, P, None) == code
    assert L.lib().moe_paged_attention(attention(cache=c), P, L.ATTENTION_WS_BYTES, None) == code


def test_cache_calls():
    P, f, c = ctypes.c_void_p, ctypes.c_void_p(FAKE), cache()
    w, r = L.lib().moe_kv_write, L.lib().moe_kv_read
    assert w(c, f, f, 0, 128, 64, 128, 64, f, f, None) == OK            # no tokens
    assert w(c, f, f, -1, 128, 64, 128, 64, f, f, None) == INV
    assert w(c, None, f, 1, 128, 64, 128, 64, f, f, None) == INV
    assert w(c, f, f, 1, 128, 64, 128, 64, None, f, None) == INV
    assert w(c, P(FAKE + 8), f, 1, 128, 64, 128, 64, f, f, None) == INV
    assert w(c, f, f, 1, 132, 64, 128, 64, f, f, None) == INV            # a stride of 8n + 4
    assert w(c, f, f, 1, 128, 64, 128, 68, f, f, None) == INV
    assert w(c, f, f, 1, 128, 64, 128, 64, f, None, None) == WS
    assert w(c, f, f, 1, 128, 64, 128, 64, f, P(FAKE + 16), None) == WS
    assert r(c, f, 4, f, None, 1, 0, f, f, f, None) == OK                # no rows
    assert r(c, f, 4, f, None, 0, 3, f, f, f, None) == INV
    assert r(c, f, 4, None, None, 1, 3, f, f, f, None) == INV
    assert r(c, f, 4, f, None, 1, 3, P(FAKE + 4), f, f, None) == INV
    assert r(c, f, -1, f, None, 1, 3, f, f, f, None) == INV
    assert r(c, f, 4, f, None, 1, 3, f, f, None, None) == WS


def attention(**kw):
    base = dict(cache=cache(), B=1, T=2, q_heads=4, max_q=2, max_kv=0, table_stride=4, q=FAKE,
                q_stride_t=256, q_stride_h=64, out=FAKE, out_stride_t=256, out_stride_h=64, lse=FAKE,
                cu_q=FAKE, kv_lens=FAKE, block_table=FAKE, scale=0.0, softcap=0.0, window=0, causal=1)
    base.update(kw)
    return L.AttentionArgs(*[base[n] for n, _ in L.AttentionArgs._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), OK), (dict(B=0), OK), (dict(max_q=0), OK),
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(q_heads=0), INV), (dict(q_heads=5), INV),
    (dict(max_q=-1), INV), (dict(max_kv=-1), INV), (dict(table_stride=-1), INV),
    (dict(window=-1), INV), (dict(window=4, causal=0), INV), (dict(causal=2), INV),
    (dict(softcap=-1.0), INV), (dict(softcap=math.nan), INV), (dict(softcap=math.inf), INV),
    (dict(scale=math.nan), INV), (dict(scale=math.inf), INV),
    (dict(q=None), INV), (dict(out=None), INV), (dict(cu_q=None), INV), (dict(kv_lens=None), INV),
    (dict(block_table=None), INV), (dict(q=FAKE + 8), INV), (dict(out=FAKE + 8), INV),
    (dict(lse=FAKE + 2), INV), (dict(q_stride_t=260), INV), (dict(out_stride_h=65), INV),
    (dict(table_stride=1 << 28), UNS), (dict(max_q=1 << 30), UNS), (dict(T=1 << 30), UNS),
])
def test_attention_arguments(kw, code):
    assert L.lib().moe_paged_attention(attention(**kw), ctypes.c_void_p(FAKE), L.ATTENTION_WS_BYTES,
                                       None) == code


def test_attention_workspace():
    P = ctypes.c_void_p
    call = L.lib().moe_paged_attention
    assert call(attention(), None, L.ATTENTION_WS_BYTES, None) == WS
    assert call(attention(), P(FAKE + 128), L.ATTENTION_WS_BYTES, None) == WS
    assert call(attention(), P(FAKE), L.ATTENTION_CTRL_BYTES - 1, None) == WS
    assert call(None, P(FAKE), L.ATTENTION_WS_BYTES, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), OK), (dict(B=-1), INV), (dict(n=0), INV), (dict(V=0), INV), (dict(n=33), UNS),
    (dict(V=1 << 24), UNS), (dict(dtype=L.DTYPE_FP8), INV), (dict(p=None), INV), (dict(q=None), INV),
    (dict(draft=None), INV), (dict(u_accept=None), INV), (dict(u_sample=None), INV),
    (dict(accepted=None), INV), (dict(tokens=None), INV), (dict(p=FAKE + 2), INV),
    (dict(dtype=L.DTYPE_BF16, q=FAKE + 1), INV),
])
def test_verify_arguments(kw, code):
    base = dict(dtype=L.DTYPE_F32, B=1, n=2, V=100, p=FAKE, p_stride_b=300, p_stride_i=100, q=FAKE,
                q_stride_b=200, q_stride_i=100, draft=FAKE, draft_lens=None, u_accept=FAKE,
                u_sample=FAKE, accepted=FAKE, tokens=FAKE)
    base.update(kw)
    a = L.VerifyArgs(*[base[n] for n, _ in L.VerifyArgs._fields_])
    assert L.lib().moe_verify_draft(a, ctypes.c_void_p(FAKE), None) == code
    if code == OK:
        base["B"] = 1
        a = L.VerifyArgs(*[base[n] for n, _ in L.VerifyArgs._fields_])
        assert L.lib().moe_verify_draft(a, None, None) == WS


def test_the_binding_refuses_tensors_that_do_not_fit():
    """Types, shapes and strides are checked before a pointer is taken."""
    def zeros(*s, dtype=torch.float32):
        return torch.zeros(*s, dtype=dtype)
    k = zeros(4, 2, 16, 64, dtype=torch.uint8)
    sc = zeros(4, 2, 16)
    x = zeros(3, 2, 64, dtype=torch.bfloat16)
    slots, ws = zeros(3, dtype=torch.int32), zeros(256, dtype=torch.uint8)
    for bad in (dict(k=x.float()), dict(k=x[:, :1]), dict(slots=slots.long()), dict(slots=slots[:2]),
                dict(k_cache=k.transpose(1, 2)), dict(k_scales=None), dict(k_scales=sc.double()),
                dict(v_scales=sc[:2]), dict(k=zeros(3, 2, 128, dtype=torch.bfloat16)[:, :, ::2]),
                dict(k_cache=k.to(torch.int8), v_cache=k.to(torch.int8))):
        a = dict(k=x, v=x, slots=slots, k_cache=k, v_cache=k, ws=ws, k_scales=sc, v_scales=sc)
        a.update(bad)
        with pytest.raises(L.MoeError):
            L.kv_write(**a)
    table, cu = zeros(1, 4, dtype=torch.int32), zeros(2, dtype=torch.int32)
    for bad in (dict(cu_rows=cu.long()), dict(block_table=table.long()), dict(cu_rows=zeros(3, dtype=torch.int32)),
                dict(starts=cu)):
        a = dict(k_cache=k, v_cache=k, block_table=table, cu_rows=cu, rows=3, ws=ws, k_scales=sc,
                 v_scales=sc)
        a.update(bad)
        with pytest.raises(L.MoeError):
            L.kv_read(**a)
    q = zeros(3, 4, 64, dtype=torch.bfloat16)
    for bad in (dict(q=q.float()), dict(q=zeros(3, 4, 128, dtype=torch.bfloat16)),
                dict(q=q.transpose(1, 2)), dict(kv_lens=cu), dict(cu_q=cu.long()),
                dict(block_table=table.t()), dict(out=q.float()), dict(out=q[:2])):
        a = dict(q=q, k_cache=k, v_cache=k, block_table=table, cu_q=cu,
                 kv_lens=zeros(1, dtype=torch.int32), ws=ws, max_q=3, k_scales=sc, v_scales=sc)
        a.update(bad)
        with pytest.raises(L.MoeError):
            L.paged_attention(**a)
    p, qd, d = zeros(2, 4, 50), zeros(2, 3, 50), zeros(2, 3, dtype=torch.int32)
    for bad in (dict(p=p.double()), dict(p=p[:, :3]), dict(q=zeros(2, 3, 100)[:, :, ::2]),
                dict(draft=d.long()), dict(u_accept=zeros(2, 2)), dict(u_sample=zeros(3)),
                dict(draft_lens=zeros(2))):
        a = dict(p=p, q=qd, draft=d, u_accept=zeros(2, 3), u_sample=zeros(2), ws=ws)
        a.update(bad)
        with pytest.raises(L.MoeError):
            L.verify_draft(**a)


def test_an_empty_call_needs_no_gpu():
    c = L.new_kv_cache(L.DTYPE_BF16, 2, 16, 2, 64, device="cpu")
    assert c[0].shape == (2, 2, 16, 64) and c[2] is None
