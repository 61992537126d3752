"""The refusals of the operators between the serving calls, and what needs no GPU of them."""
import ctypes
import math

import pytest
import torch

import step_reference as R
from mixture_experts_forward_gb300 import _lib as L
from mixture_experts_forward_gb300 import build as moe_build

FAKE = 1 << 20   # a non-null, aligned fake device address; never dereferenced
INV, UNS, WS, OK = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE, L.MOE_OK
P = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def built():
    moe_build.build()


def struct(cls, base, **kw):
    base = {**base, **kw}
    return cls(*[base[n] for n, _ in cls._fields_])


def pages(**kw):
    return struct(L.PageState, dict(B=2, table_stride=4, page_size=16, free_capacity=9, block_table=FAKE,
                                    held=FAKE, free_pages=FAKE, free_count=FAKE), **kw)


BAD_PAGES = [(dict(B=-1), INV), (dict(table_stride=-1), INV), (dict(page_size=0), INV),
             (dict(free_capacity=-1), INV), (dict(block_table=None), INV), (dict(held=None), INV),
             (dict(free_pages=None), INV), (dict(free_count=None), INV), (dict(held=FAKE + 2), INV),
             (dict(block_table=FAKE + 1), INV), (dict(free_pages=FAKE + 2), INV),
             (dict(page_size=8), UNS), (dict(page_size=48), UNS), (dict(page_size=512), UNS),
             (dict(B=8193), UNS), (dict(B=8192, table_stride=1 << 18), UNS),
             (dict(table_stride=1 << 28), UNS)]


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_page_states_that_are_refused(kw, code):
    f = P(FAKE)
    assert L.lib().moe_plan_step(pages(**kw), f, f, 3, 9, f, f, f, f, f, None) == code
    assert L.lib().moe_release_pages(pages(**kw), f, f, None) == code


def test_plan_calls():
    f, plan, release = P(FAKE), L.lib().moe_plan_step, L.lib().moe_release_pages
    assert plan(None, f, f, 3, 9, f, f, f, f, f, None) == INV
    assert plan(pages(), None, f, 3, 9, f, f, f, f, f, None) == INV
    assert plan(pages(), f, None, 3, 9, f, f, f, f, f, None) == INV
    assert plan(pages(), f, f, -1, 9, f, f, f, f, f, None) == INV
    assert plan(pages(), f, f, 3, -1, f, f, f, f, f, None) == INV
    assert plan(pages(), f, f, 3, 9, None, f, f, f, f, None) == INV
    assert plan(pages(), f, f, 3, 9, f, None, f, f, f, None) == INV
    assert plan(pages(), f, f, 3, 9, f, f, None, f, f, None) == INV
    assert plan(pages(), f, f, 3, 9, f, f, f, None, f, None) == INV
    assert plan(pages(), P(FAKE + 2), f, 3, 9, f, f, f, f, f, None) == INV
    assert plan(pages(), f, f, (1 << 30) + 1, 9, f, f, f, f, f, None) == UNS
    assert plan(pages(), f, f, 3, 1 << 27, f, f, f, f, f, None) == UNS
    assert plan(pages(), f, f, 3, 9, f, f, f, f, None, None) == WS
    assert plan(pages(), f, f, 3, 9, f, f, f, f, P(FAKE + 8), None) == WS
    assert release(pages(B=0), None, None, None) == OK
    assert release(pages(), None, f, None) == INV
    assert release(pages(), f, None, None) == WS


ROPE = [dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0),
        dict(base=500000.0, scaling="turns", factor=8.0, original=8192, low=1.0, high=4.0),
        dict(scaling="index", factor=16.0, original=4096, low=1.0, high=32.0),
        dict(scaling="index", factor=2.0, original=7, low=1.0, high=32.0),      # no pair makes a turn
        dict(scaling="linear", factor=0.01)]


@pytest.mark.parametrize("rot", [2, 16, 96, 128])
@pytest.mark.parametrize("kw", ROPE)
def test_rotary_table(rot, kw):
    table = L.rotary_table(rot, device="cpu", **kw).tolist()
    want = [t / (2 * math.pi) for t in R.frequencies(rot, **kw)]
    assert len(table) == rot // 2
    for got, turns in zip(table, want):
        got = (got + (1 << 64)) % (1 << 64) / 2.0 ** 64
        # two 64-bit evaluations: a few units in their last place, and one of the table's
        assert abs(got - turns % 1.0) <= 1e-14 * max(turns, 1e-300) + 2.0 ** -63 + (1e-14 if turns >= 1 else 0)


def test_rotary_tables_that_are_refused():
    out = (ctypes.c_uint64 * 64)()
    call = L.lib().moe_rotary_table
    for args, code in [((0, 1e4, 0, 1, 0, 1, 32), INV), ((15, 1e4, 0, 1, 0, 1, 32), INV),
                       ((514, 1e4, 0, 1, 0, 1, 32), UNS), ((64, 1.0, 0, 1, 0, 1, 32), INV),
                       ((64, math.nan, 0, 1, 0, 1, 32), INV), ((64, 1e4, 4, 1, 9, 1, 32), INV),
                       ((64, 1e4, 1, 0.0, 0, 1, 32), INV), ((64, 1e4, 2, 2.0, 0, 1, 4), INV),
                       ((64, 1e4, 2, 2.0, 99, 4, 4), INV), ((64, 1e4, 3, 2.0, 99, 0, 4), INV),
                       ((64, 1e4, 3, math.inf, 99, 1, 4), INV)]:
        assert call(*args, out) == code, args
    assert call(64, 1e4, 0, 1, 0, 1, 32, None) == INV
    with pytest.raises(L.MoeError, match="scaling is one of"):
        L.rotary_table(64, scaling="other", device="cpu")


def cache(**kw):
    return struct(L.KvCache, dict(dtype=L.DTYPE_FP8, num_pages=4, page_size=16, heads=2, head_dim=64, k=FAKE,
                                  v=FAKE, k_scales=FAKE, v_scales=FAKE), **kw)


def rotary(**kw):
    return struct(L.RotaryArgs, dict(
        T=3, q_heads=4, kv_heads=2, head_dim=64, rotary_dim=32, interleaved=0, amplitude=1.0, table=FAKE,
        positions=FAKE, q=FAKE, q_stride_t=256, q_stride_h=64, q_out=FAKE, q_out_stride_t=256,
        q_out_stride_h=64, k=FAKE, k_stride_t=128, k_stride_h=64, k_out=FAKE, k_out_stride_t=128,
        k_out_stride_h=64, v=FAKE, v_stride_t=128, v_stride_h=64, slots=FAKE, cache=cache()), **kw)


NONE = dict(k=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), OK), (dict(q_heads=0, kv_heads=0, cache=cache(k=None)), OK),
    (dict(T=-1), INV), (dict(q_heads=-1), INV), (dict(rotary_dim=0), INV), (dict(rotary_dim=80), INV),
    (dict(interleaved=2), INV), (dict(amplitude=math.nan), INV), (dict(rotary_dim=24), UNS),
    (dict(head_dim=72, cache=cache(k=None)), UNS), (dict(head_dim=272, cache=cache(k=None)), UNS),
    (dict(kv_heads=3), INV), (dict(head_dim=128, rotary_dim=32), INV), (dict(table=None), INV),
    (dict(table=FAKE + 4), INV), (dict(positions=None), INV), (dict(positions=FAKE + 2), INV),
    (dict(q=None), INV), (dict(q_out=None), INV), (dict(q=FAKE + 8), INV), (dict(q_out=FAKE + 8), INV),
    (dict(q_stride_t=260), INV), (dict(q_out_stride_h=4), INV), (dict(k=None), INV), (dict(k=FAKE + 2), INV),
    (dict(k_stride_h=4), INV), (dict(v=None), INV), (dict(v=FAKE + 4), INV), (dict(v_stride_t=7), INV),
    (dict(slots=None), INV), (dict(slots=FAKE + 1), INV), (dict(cache=cache(page_size=8)), UNS),
    (dict(cache=cache(head_dim=96), head_dim=96), UNS), (dict(cache=cache(v=None)), INV),
    (dict(cache=cache(k=None), k_out=None), INV), (dict(cache=cache(k=None), k_out=FAKE + 4), INV),
    (dict(cache=cache(k=None), k_out_stride_t=9), INV), (dict(q_heads=1 << 21), UNS),
])
def test_rotary_arguments(kw, code):
    assert L.lib().moe_rotary(rotary(**kw), P(FAKE), None) == code


def test_rotary_workspace():
    assert L.lib().moe_rotary(None, P(FAKE), None) == INV
    assert L.lib().moe_rotary(rotary(), None, None) == WS
    assert L.lib().moe_rotary(rotary(), P(FAKE + 16), None) == WS


def few_args(**kw):
    base = dict(dtype=L.DTYPE_FP8, M=4, K=256, N=128, E=8, top_k=2, softcap=0.0, renorm=1, logits=FAKE,
                x=FAKE, w=FAKE, w_scales=FAKE, w2=FAKE, block_m=0, sched=0, k_splits=0, use_graph=1,
                gather_rows=0, gated=1, w2_scales=FAKE, cta_pairs=0)
    return struct(L.ForwardArgs, base, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(M=0), INV), (dict(M=17), UNS), (dict(K=0), INV), (dict(K=192), UNS), (dict(N=64), UNS),
    (dict(K=32896), UNS), (dict(N=32896), UNS), (dict(E=0), INV), (dict(E=1025), UNS), (dict(top_k=0), INV),
    (dict(top_k=9), UNS), (dict(E=64, top_k=33), UNS), (dict(softcap=-1.0), INV), (dict(softcap=math.nan), INV),
    (dict(softcap=math.inf), INV), (dict(dtype=L.DTYPE_F32), INV), (dict(gated=0), UNS), (dict(gated=2), INV),
    (dict(dtype=L.DTYPE_BF16, K=224), UNS)])
def test_few_shapes(kw, code):
    a = few_args(**kw)
    assert L.lib().moe_forward_few(a, P(FAKE), P(FAKE), 1 << 20, None) == code
    assert L.lib().moe_few_workspace_size(a) == 0
    with pytest.raises(L.MoeError):
        L.few_workspace_size(a)


@pytest.mark.parametrize("kw", [dict(logits=None), dict(x=None), dict(w=None), dict(w2=None), dict(w_scales=None),
                                dict(w2_scales=None), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(w2=FAKE + 4),
                                dict(logits=FAKE + 2), dict(w_scales=FAKE + 1)])
def test_few_pointers(kw):
    assert L.lib().moe_forward_few(few_args(**kw), P(FAKE), P(FAKE), 1 << 20, None) == INV


def test_few_workspace():
    a = few_args()
    n = L.few_workspace_size(a)
    assert n >= 256 + 4 * 2 * 128 * 4 and n % 256 == 0
    call = L.lib().moe_forward_few
    assert call(a, None, P(FAKE), n, None) == INV
    assert call(a, P(FAKE + 1), P(FAKE), n, None) == INV
    assert call(a, P(FAKE), None, n, None) == WS
    assert call(a, P(FAKE), P(FAKE + 128), n, None) == WS
    assert call(a, P(FAKE), P(FAKE), 255, None) == WS
    assert call(None, P(FAKE), P(FAKE), n, None) == INV
    assert L.few_workspace_size(few_args(dtype=L.DTYPE_BF16, K=192, gated=0)) > 0


def logits_args(**kw):
    base = dict(dtype=L.DTYPE_F32, B=2, m=3, V=100, logits=FAKE, logits_stride_b=300, logits_stride_i=100, out=FAKE,
                out_stride_b=300, out_stride_i=100, probabilities=1, history=FAKE, history_stride=7,
                history_lens=FAKE, prompt_lens=FAKE, draft=FAKE, repetition=FAKE, presence=FAKE, frequency=FAKE,
                temperature=FAKE, biases=4, bias_tokens=FAKE, bias_values=FAKE, mask=FAKE, mask_stride_b=12,
                mask_stride_i=4)
    return struct(L.LogitsArgs, base, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), OK), (dict(B=-1), INV), (dict(m=0), INV), (dict(V=0), INV), (dict(m=34), UNS), (dict(V=262145), UNS),
    (dict(biases=-1), INV), (dict(biases=1025), UNS), (dict(history_stride=-1), INV), (dict(dtype=0), INV),
    (dict(probabilities=2), INV), (dict(logits=None), INV), (dict(out=None), INV), (dict(logits=FAKE + 2), INV),
    (dict(dtype=L.DTYPE_BF16, logits=FAKE + 1), INV), (dict(bias_tokens=None), INV), (dict(bias_values=None), INV),
    (dict(out=FAKE + 2), INV), (dict(history=FAKE + 2), INV), (dict(mask=FAKE + 1), INV), (dict(draft=FAKE + 3), INV),
    (dict(temperature=FAKE + 2), INV), (dict(B=1 << 25), UNS)])
def test_logits_arguments(kw, code):
    a = logits_args(**kw)
    assert L.lib().moe_adjust_logits(a, P(FAKE), None) == code
    if code == OK:
        assert L.lib().moe_adjust_logits(logits_args(), None, None) == WS
        assert L.lib().moe_adjust_logits(logits_args(), P(FAKE + 4), None) == WS
        assert L.lib().moe_adjust_logits(None, P(FAKE), None) == INV


# ------------------------------------------------------------------ the binding
def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def all_calls():
    """name -> (entry point, arguments that are valid but for their place, wrong ones)."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8)
    state = dict(block_table=i32(2, 4), held=i32(2), free_pages=i32(9), free_count=i32(1), page_size=16, ws=ws)
    cu8 = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    sc = torch.zeros(4, 2, 16)
    turn = dict(positions=i32(3), table=torch.zeros(16, dtype=torch.int64))
    write = dict(turn, q=bf(3, 4, 64), k=bf(3, 2, 64), v=bf(3, 2, 64), slots=i32(3), k_cache=cu8, v_cache=cu8,
                 ws=ws, k_scales=sc, v_scales=sc)
    lg = dict(logits=torch.zeros(2, 3, 50), ws=ws, history=i32(2, 7), history_lens=i32(2), prompt_lens=i32(2),
              draft=i32(2, 2), repetition=torch.zeros(2), presence=torch.zeros(2), frequency=torch.zeros(2),
              temperature=torch.zeros(2), bias_tokens=i32(2, 5), bias_values=torch.zeros(2, 5), mask=i32(2, 3, 2),
              out=torch.zeros(2, 3, 50))
    return dict(
        plan=(L.plan_step, dict(state, lens=i32(2), new_lens=i32(2), rows=5, num_pages=9),
              [dict(lens=i32(3)), dict(new_lens=i32(2).long()), dict(held=i32(3)), dict(free_count=i32(2)),
               dict(free_pages=i32(9).long()), dict(block_table=i32(4, 2).t()), dict(block_table=i32(2, 4).long()),
               dict(rows=-1)]),
        release=(L.release_pages, dict(state, keep=i32(2)), [dict(keep=i32(3)), dict(keep=i32(2).float())]),
        rotary=(L.rotary, dict(turn, q=bf(3, 4, 64), k=bf(3, 2, 64)),
                [dict(q=None, k=None), dict(q=torch.zeros(3, 4, 64)), dict(k=bf(2, 2, 64)), dict(k=bf(3, 2, 128)),
                 dict(positions=i32(2)), dict(positions=i32(3).long()), dict(table=torch.zeros(16)),
                 dict(table=torch.zeros(2, 8, dtype=torch.int64)), dict(q_out=bf(3, 4, 32)),
                 dict(k_out=torch.zeros(3, 2, 64)), dict(q=bf(3, 64, 4).transpose(1, 2))]),
        write=(L.rotary_write, write,
               [dict(k=bf(3, 3, 64)), dict(v=bf(3, 1, 64)), dict(q=bf(2, 4, 64)), dict(q=bf(3, 4, 128)),
                dict(slots=i32(2)), dict(k_scales=None), dict(q_out=bf(3, 2, 64)), dict(v=torch.zeros(3, 2, 64))]),
        few=(lambda out, ws: L.forward_few(few_args(), out, ws), dict(out=bf(4, 256), ws=ws),
             [dict(out=bf(4, 128)), dict(out=torch.zeros(4, 256)), dict(out=bf(256, 4).t())]),
        logits=(L.adjust_logits, lg,
                [dict(logits=torch.zeros(2, 3, 50, dtype=torch.float64)), dict(logits=torch.zeros(2, 3, 100)[:, :, ::2]),
                 dict(history=i32(2, 7).long()), dict(history=None), dict(history_lens=i32(3)), dict(prompt_lens=i32(1)),
                 dict(draft=i32(2, 3)), dict(repetition=torch.zeros(3)), dict(presence=torch.zeros(2).double()),
                 dict(frequency=i32(2)), dict(temperature=torch.zeros(1)), dict(bias_tokens=None),
                 dict(bias_values=None), dict(bias_values=torch.zeros(2, 4)), dict(mask=i32(2, 3, 1)),
                 dict(mask=i32(2, 2, 2)), dict(mask=i32(2, 3, 2).long()), dict(out=torch.zeros(2, 3, 49)),
                 dict(out=torch.zeros(2, 3, 50, dtype=torch.bfloat16))]))


@pytest.mark.parametrize("name", ["plan", "release", "rotary", "write", "few", "logits"])
def test_what_the_binding_refuses(name):
    call, args, wrong = all_calls()[name]
    with pytest.raises(L.MoeError, match="on one GPU"):        # host tensors, before an address is passed on
        call(**args)
    for kw in wrong:
        with pytest.raises(L.MoeError) as e:
            call(**{**args, **kw})
        assert "on one GPU" not in str(e.value), kw


def test_sizes_past_the_types_are_refused():
    out = (ctypes.c_uint64 * 64)()
    # theta / factor is no number
    assert L.lib().moe_rotary_table(64, 1e4, 1, 5e-324, 0, 1, 32, out) == INV
    # a token's count and its other marks share 32 bits
    most = (1 << 20) - 64
    assert L.lib().moe_adjust_logits(logits_args(history_stride=most + 1), P(FAKE), None) == UNS
    assert L.lib().moe_adjust_logits(logits_args(history_stride=most + 1, history=None, B=0), P(FAKE), None) == OK
    assert L.lib().moe_adjust_logits(logits_args(history_stride=most), None, None) == WS
