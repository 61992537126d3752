"""The operators between the serving calls where their sizes and values end (64-bit forms of
tests/step_reference.py)."""
import math
import os
import subprocess
import sys

import pytest
import torch

import step_reference as R
from gpu_helpers import ensure_built
from mixture_experts_forward_gb300 import _lib as L
from mixture_experts_forward_gb300 import inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


# ------------------------------------------------------------------ logits
FRESH = """
import sys
sys.path.insert(0, {here!r})
sys.path.insert(0, {root!r})
import test_gpu_step as S
x, kw = S.logits_case(1, 1, {V}, 40, {nb}, 5)
for probs in (True, False):
    S.check_logits(x, kw, probabilities=probs)
print("fine")
"""


@pytest.mark.parametrize("V,nb", [(50257, 286), (50257, 300), (50257, 341), (65536, 342), (32769, 1024)])
def test_biases_that_end_near_the_default_limit_of_shared_memory(V, nb):
    """16 values a thread and 286 to 341 biases ask for just less than 48 KB.  Each in a process of
    its own: a larger call before would have raised the kernel's limit for good."""
    code = FRESH.format(here=HERE, root=os.path.dirname(HERE), V=V, nb=nb)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------ few tokens
class Alike:
    """n experts' values of which the same few repeat."""

    def __init__(self, values, n):
        self.values, self.shape = values, (n, *values.shape[1:])

    def __getitem__(self, e):
        return self.values[e % len(self.values)]


def many_experts(fp8, T, H, I, E, k, seed, distinct=4):
    """(args, tensors, x, values) of a layer of E experts of which `distinct` differ."""
    g = torch.Generator().manual_seed(seed)
    up = torch.randn(distinct, 2 * I, H, generator=g) / H ** 0.5
    down = torch.randn(distinct, H, I, generator=g) / I ** 0.5
    x = torch.randn(T, H, generator=g).to(BF16)
    if fp8:
        (up, up_s), (down, dn_s) = inputs.quantize_weights_e4m3(up), inputs.quantize_weights_e4m3(down)
        wide = lambda w, s: (w.view(torch.float8_e4m3fn).double() *  # noqa: E731
                             s.double().repeat_interleave(128, 1).repeat_interleave(128, 2))
        values = wide(up, up_s), wide(down, dn_s)
    else:
        up, down, up_s, dn_s = up.to(BF16), down.to(BF16), None, None
        values = up.double(), down.double()
    dev = dict(w=up, w_scales=up_s, w2=down, w2_scales=dn_s)
    dev = {n: None if t is None else t.cuda().repeat(E // distinct, 1, 1) for n, t in dev.items()}
    dev.update(logits=torch.randn(T, E, generator=g).cuda(), x=x.cuda())
    args = L.forward_args(dtype=L.DTYPE_FP8 if fp8 else L.DTYPE_BF16, M=T, K=H, N=I, E=E, top_k=k, gated=1, **dev)
    return args, dev, x, [Alike(v, E) for v in values]


@pytest.mark.parametrize("fp8,T,H,E,k", [(True, 16, 4096, 1024, 32), (False, 16, 4096, 1024, 32),
                                         (True, 16, 4096, 512, 28), (True, 13, 4992, 1024, 32),
                                         (False, 15, 4352, 1024, 32), (True, 16, 3968, 1024, 32)])
def test_many_routes_and_long_rows(fp8, T, H, E, k):
    """The routes' tables and x of these do not fit shared memory together: two passes."""
    args, dev, x, values = many_experts(fp8, T, H, 128, E, k, seed=T + k)
    ws = L.new_workspace(L.few_workspace_size(args))
    out = torch.full((T, H), math.nan, dtype=BF16, device="cuda")
    L.forward_few(args, out, ws)
    assert L.get_error(ws) == L.MOE_OK
    ids, w = L.route(dev["logits"], k)
    want, err = R.few(x, ids.cpu(), w.cpu(), *values, fp8)
    tol = err + (want.abs() + err) * 2.0 ** -8 + 1e-38
    diff = (out.cpu().double() - want).abs()
    assert (diff <= tol).all(), (diff / tol).max()


@pytest.mark.parametrize("T", [6, 13])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("fp8", [True, False])
def test_weights_that_are_not_finite_stay_with_their_expert(fp8, bad, T):
    """Tokens that are not routed to the expert keep their bits (FP8's infinity is a scale's)."""
    H, E = 256, 8
    args, dev, x, _ = many_experts(fp8, T, H, 128, E, 2, seed=T, distinct=8)
    dev["logits"][:, 3] = -50.0
    mine = torch.arange(T, device="cuda") % 3 == 1
    dev["logits"][mine, 3] = 50.0                    # tokens 1, 4, .. go to expert 3
    ws = L.new_workspace(L.few_workspace_size(args))
    clean = L.forward_few(args, torch.empty(T, H, dtype=BF16, device="cuda"), ws)
    assert clean.isfinite().all()
    if fp8 and math.isinf(bad):
        dev["w_scales"][3], dev["w2_scales"][3] = bad, bad
    else:
        for w in ("w", "w2"):
            dev[w][3, ::5, ::3] = 0x7f if fp8 else bad
    out = L.forward_few(args, torch.empty_like(clean), ws)
    assert L.get_error(ws) == L.MOE_OK
    assert torch.equal(out[~mine], clean[~mine])
    assert not out[mine].isfinite().all(1).any()


@pytest.mark.parametrize("fp8", [True, False])
def test_an_infinite_h_is_an_infinite_output(fp8):
    """h past binary32 over positive weights: the sum is +inf, not NaN."""
    H = 128
    one = torch.ones(2, 256, H)
    if fp8:
        up = torch.full((2, 256, H), 0x38, dtype=torch.uint8, device="cuda")          # 1.0
        kw = dict(w=up, w2=up[:, :128].contiguous(), w_scales=torch.ones(2, 2, 1, device="cuda"),
                  w2_scales=torch.ones(2, 1, 1, device="cuda"))
    else:
        kw = dict(w=one.to(BF16).cuda(), w2=one[:, :128].to(BF16).cuda())
    x = torch.full((2, H), 2.0 ** 70, dtype=BF16, device="cuda")
    x[1] = 1.0
    args = L.forward_args(dtype=L.DTYPE_FP8 if fp8 else L.DTYPE_BF16, M=2, K=H, N=128, E=2, top_k=1, gated=1, x=x,
                          logits=torch.zeros(2, 2, device="cuda"), **kw)
    ws = L.new_workspace(L.few_workspace_size(args))
    out = L.forward_few(args, torch.empty(2, H, dtype=BF16, device="cuda"), ws)
    assert (out[0] == math.inf).all()
    # silu(128) * 128 = 2^14, 128 of them
    assert (out[1] == 2.0 ** 21).all()


# ------------------------------------------------------------------ rotary
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base,factor", [(10000.0, 1.0), (500000.0, 8.0), (1e6, 40.0), (1e7, 1000.0)])
def test_slow_pairs_at_small_positions(base, factor, interleaved):
    """One element of each pair is 0, so that the other's sine stands alone.  What may be off: bf16's
    half step and, relative to the result, sincospi (2 units of 2^-24), the product and the
    amplitude's (one each); the angle within its turn by 2^-24 of it, by 2^-64 turns a position (the
    table's step) and by 2^-50 of the whole angle (two evaluations in 64 bits)."""
    rot, T = 128, 40
    pos = torch.cat([torch.arange(-7, 25), torch.tensor([100, 1000, 30011, 131071, -100, -1000, 1 << 20, 77])])
    kw = dict(base=base, scaling="linear", factor=factor)
    theta, table = R.frequencies(rot, **kw), L.rotary_table(rot, **kw)
    angle = pos.double()[:, None] * torch.tensor(theta, dtype=torch.float64)
    within = torch.remainder(angle + math.pi, 2 * math.pi) - math.pi
    off = within.abs() * 2.0 ** -24 + pos.double().abs()[:, None] * 2 * math.pi * 2.0 ** -64 + angle.abs() * 2.0 ** -50
    off = (off.repeat_interleave(2, 1) if interleaved else torch.cat([off, off], 1))[:, None]
    for zero in (0, 1):
        x = torch.ones(T, 1, rot)
        if interleaved:
            x[..., zero::2] = 0
        else:
            x[..., zero * rot // 2:(zero + 1) * rot // 2] = 0
        got, _ = L.rotary(x.to(BF16).cuda(), None, pos.to(torch.int32).cuda(), table, interleaved=interleaved)
        want, _ = R.rotated(x, pos, theta, interleaved)
        tol = want.abs() * (2.0 ** -8 + 4 * 2.0 ** -24) + off * 1.01
        bad = (got.double().cpu() - want).abs() > tol
        assert not bad.any(), (bad.sum(), got.double().cpu()[bad][:4], want[bad][:4])


# ------------------------------------------------------------------ faults
def test_a_shared_control_block_says_which_operator_saw_the_fault():
    """The control block's fourth word, after one bad call of each operator on a block of their own."""
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = L.new_kv_cache(L.DTYPE_BF16, 2, 16, 1, 64)[:2]
    x = torch.ones(1, 1, 64, dtype=BF16, device="cuda")
    p = torch.full((1, 2, 8), 0.125, device="cuda")
    u = torch.zeros(1, device="cuda")
    state = lambda: dict(block_table=i32(0, 1).view(1, 2), held=i32(2), free_pages=i32(3, 4, 5),  # noqa: E731
                         free_count=i32(3), page_size=16)
    bad = dict(
        write=lambda ws: L.kv_write(x, x, i32(32), *cache, ws),
        read=lambda ws: L.kv_read(*cache, i32(9).view(1, 1), i32(0, 1), 1, ws),
        attention=lambda ws: L.paged_attention(x, *cache, i32(0).view(1, 1), i32(0, 1), i32(17), ws, max_q=1),
        verify=lambda ws: L.verify_draft(p, p[:, :1].contiguous(), i32(8).view(1, 1), u.view(1, 1), u, ws),
        plan=lambda ws: L.plan_step(i32(-1), i32(1), **state(), rows=1, num_pages=6, ws=ws),
        plan_page=lambda ws: L.plan_step(i32(20), i32(1), **state(), rows=1, num_pages=1, ws=ws),
        plan_count=lambda ws: L.plan_step(i32(20), i32(1), **{**state(), "free_count": i32(4)}, rows=1, num_pages=6,
                                          ws=ws),
        release_held=lambda ws: L.release_pages(i32(0), **{**state(), "held": i32(3)}, ws=ws),
        release_count=lambda ws: L.release_pages(i32(-1), **{**state(), "free_count": i32(-1)}, ws=ws),
        release_room=lambda ws: L.release_pages(i32(0), **state(), ws=ws),
        rotary=lambda ws: L.rotary_write(x, x, x, i32(0), i32(32), L.rotary_table(64), *cache, ws),
        token=lambda ws: L.adjust_logits(p, ws, draft=i32(8).view(1, 1)),
        lengths=lambda ws: L.adjust_logits(p, ws, history=i32(1, 2).view(1, 2), history_lens=i32(3)),
        number=lambda ws: L.adjust_logits(p, ws, temperature=torch.full((1,), -1.0, device="cuda")))
    places = {}
    for name, call in bad.items():
        ws = L.new_workspace(L.ATTENTION_WS_BYTES if name == "attention" else L.CTRL_BYTES)
        call(ws)
        places[name] = ws[12:16].view(torch.int32).item()
        assert L.get_error(ws) == L.MOE_ERR_DEVICE_FAULT, name
    assert len(set(places.values())) == len(bad), places


# ------------------------------------------------------------------ the binding
@pytest.mark.parametrize("name", ["logits", "x", "w", "w_scales", "w2", "w2_scales"])
def test_one_host_tensor_among_the_experts_arguments(name):
    """Refused, before its address is passed on."""
    args, dev, _, _ = many_experts(True, 2, 256, 128, 4, 2, seed=1)
    ws, out = L.new_workspace(L.few_workspace_size(args)), torch.zeros(2, 256, dtype=BF16, device="cuda")
    dev[name] = dev[name].cpu()
    args = L.forward_args(dtype=L.DTYPE_FP8, M=2, K=256, N=128, E=4, top_k=2, gated=1, **dev)
    with pytest.raises(L.MoeError, match="on one GPU"):
        L.forward_few(args, out, ws)
    assert (out == 0).all()


# ------------------------------------------------------------------ the exponential
@pytest.mark.parametrize("temperature", [1.0, 0.3, 7.0])
@pytest.mark.parametrize("V", [4000, 50257, 262144])
def test_probabilities_far_below_the_largest(V, temperature):
    """Relative to themselves off by (d + 40) 2^-22, d = (max - l) / temperature: 2^-22 of d for the
    difference, the rate's two roundings and the product, twice 2^-22 for the exponentials, the mean of d
    under the distribution (at most ln V, 12.5) and 81 additions of 2^-24 for the sum."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn(2, 1, V, generator=g) * 14 * temperature
    x[1] = torch.rand(1, V, generator=g) * 60 * temperature
    out = L.adjust_logits(x.cuda(), L.new_workspace(L.CTRL_BYTES),
                          temperature=torch.full((2,), temperature, device="cuda")).cpu().double()
    t = float(torch.tensor(temperature))
    d = (x.double().amax(-1, keepdim=True) - x.double()) / t
    want = torch.softmax(-d, -1)
    seen = want > 2.0 ** -120
    assert ((out - want).abs() <= want * (d + 40) * 2.0 ** -22)[seen].all()
