"""Results of calls on a stream of the caller's: they come from that stream's memory, so that work
still queued on the current stream keeps what it reads."""
import pytest
import torch

from gpu_helpers import ensure_built
from mixture_experts_forward_gb300 import _lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def pool_of(t):
    """The stream whose memory t lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls():
    """name -> a call that takes a stream and returns its results (inputs ready on the device)."""
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    ctrl, ws = L.new_workspace(L.CTRL_BYTES), L.new_workspace(L.ATTENTION_WS_BYTES)
    kc, vc, _, _ = L.new_kv_cache(L.DTYPE_BF16, 64, 16, 2, 64)
    table, q = torch.arange(64, dtype=torch.int32, device="cuda").view(1, -1), torch.zeros(3, 4, 64, **bf16)
    p = torch.full((2, 4, 100), 0.01, device="cuda")
    draft, u = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, device="cuda")
    M, E, k = 8, 4, 2
    logits, x = torch.zeros(M, E, device="cuda"), torch.zeros(M, 256, **bf16)
    ids, w = L.route(logits, k)
    lay_ws = L.new_workspace(1 << 20)
    lay = L.layout(ids, E, 16, lay_ws)
    rows, gu = torch.zeros(M * k, 256, device="cuda"), torch.zeros(16, 512, device="cuda")
    cu_rows, cu_q, lens, us = i32([0, 1000]), i32([0, 3]), i32([900]), torch.zeros(2, device="cuda")
    out = dict(
        read=lambda s: L.kv_read(kc, vc, table, cu_rows, 1000, ctrl, stream=s),
        attention=lambda s: L.paged_attention(q, kc, vc, table, cu_q, lens, ws, max_q=3, lse=True,
                                              stream=s),
        verify=lambda s: L.verify_draft(p, p[:, :3], draft, u, us, ctrl, stream=s),
        route=lambda s: L.route(logits, k, stream=s),
        layout=lambda s: list(L.layout(ids, E, 16, lay_ws, stream=s).values()),
        quant=lambda s: L.quant_gather(x, k, lay["route_slot"], stream=s),
        scatter=lambda s: [L.scatter(rows, lay["route_slot"], w, ctrl, stream=s)],
        swiglu=lambda s: L.swiglu_quant(gu, stream=s))
    torch.cuda.synchronize()
    return out


NAMES = ["read", "attention", "verify", "route", "layout", "quant", "scatter", "swiglu"]


@pytest.mark.parametrize("name", NAMES)
def test_results_lie_in_their_streams_memory(name):
    call, s = calls()[name], torch.cuda.Stream()
    for t in call(s):
        assert pool_of(t) == s.cuda_stream
    s.synchronize()
    for stream in (None, torch.cuda.current_stream()):       # the current one: as without
        for t in call(stream):
            assert pool_of(t) == torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()


def test_work_queued_on_the_current_stream_keeps_its_inputs():
    """A tensor is copied late on the current stream and freed at once; a call on another stream
    whose results have its size must not write into it."""
    H, D, rows = 2, 64, 4096
    kc, vc, _, _ = L.new_kv_cache(L.DTYPE_BF16, rows // 16, 16, H, D)
    table = torch.arange(rows // 16, dtype=torch.int32, device="cuda").view(1, -1)
    cu, ctrl, s = i32([0, rows]), L.new_workspace(L.CTRL_BYTES), torch.cuda.Stream()
    L.kv_read(kc, vc, table, cu, rows, ctrl, stream=s)       # (whatever a first call sets up)
    torch.cuda.synchronize()
    x = [torch.full((rows, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(100_000_000)                           # about 50 ms
    late = [t.clone() for t in x]
    del x
    k, v = L.kv_read(kc, vc, table, cu, rows, ctrl, stream=s)
    torch.cuda.synchronize()
    assert all(bool((t == 7.0).all()) for t in late)
    assert bool((k == 0).all()) and bool((v == 0).all())
