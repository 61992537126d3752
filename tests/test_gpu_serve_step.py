"""The serving operators around the expert forward, as a program uses them
(examples/serve_step.py): chunks and single tokens agree, and the steps' bookkeeping holds."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import serve_step  # noqa: E402
from gpu_helpers import ensure_built  # noqa: E402
from mixture_experts_forward_gb300 import _lib as L  # noqa: E402

pytestmark = pytest.mark.gpu


def test_steps_extend_the_sequences():
    ensure_built()
    r = serve_step.main(steps=5, batch=3, n_draft=4, prompt=21)
    assert r["status"] == (L.MOE_OK, L.MOE_OK)
    for tokens, length in zip(r["tokens"], r["lengths"]):
        assert 5 <= len(tokens) <= 25 and all(0 <= t < serve_step.VOCAB for t in tokens)
        assert length == 20 + len(tokens)
    # a row quantised again from its own values moves by about bf16's and E4M3's rounding
    assert r["drift"] < 0.05


def test_a_chunk_equals_its_tokens_one_by_one():
    """The chunk form (many rows), the drafted form and the single-token form read
    the same cache: their probabilities differ by roundings only."""
    ensure_built()
    tokens = torch.randint(serve_step.VOCAB, (2, 70), dtype=torch.int32,
                           generator=torch.Generator().manual_seed(1)).cuda()
    runs = []
    for cut in (70, 7, 1):
        s = serve_step.Server(2, 4, 80, seed=5)
        p = []
        for i in range(0, 70, cut):
            p.append(s.forward(tokens[:, i:i + cut]))
            s.len = s.len + cut
        assert s.status() == (L.MOE_OK, L.MOE_OK)
        runs.append(torch.cat(p, 1))
    for other in runs[1:]:
        assert (other - runs[0]).norm() / runs[0].norm() < 2e-2


def test_the_operators_run_inside_a_graph():
    """Captured on a stream of the caller's, replayed on new inputs."""
    ensure_built()
    k, v, _, _ = L.new_kv_cache(L.DTYPE_BF16, 8, 16, 2, 64)
    new = torch.randn(3, 2, 2, 64, device="cuda").to(torch.bfloat16)
    q = torch.randn(3, 8, 64, device="cuda").to(torch.bfloat16)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    slots = table[:, 0] * 16
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    lens = torch.ones(3, dtype=torch.int32, device="cuda")
    ws, ctrl = L.new_workspace(L.ATTENTION_WS_BYTES), L.new_workspace(L.CTRL_BYTES)

    def step():
        L.kv_write(new[:, 0], new[:, 1], slots, k, v, ctrl)
        return L.paged_attention(q, k, v, table, cu, lens, ws, max_q=1)[0]

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    new.copy_(torch.randn_like(new))
    g.replay()
    torch.cuda.synchronize()
    # one cached position: its weight is 1, the output its value row
    got_k, got_v = L.kv_read(k, v, table, cu, 3, ctrl)
    assert torch.equal(got_v, new[:, 1]) and torch.equal(got_k, new[:, 0])
    assert torch.equal(out.view(3, 2, 4, 64), got_v[:, :, None, :].expand(3, 2, 4, 64))
    assert L.get_error(ws) == L.MOE_OK and L.get_error(ctrl) == L.MOE_OK


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("q_len,heads", [(1, 4), (10, 4), (100, 4)])
def test_a_stalled_pipeline_ends_with_a_status(fp8, q_len, heads):
    """No loads are issued: every wait runs out, the kernel ends, the status says
    so, and the next call is right (the counters of split tiles too)."""
    ensure_built()
    n = 2000
    k, v, ks, vs = L.new_kv_cache(L.DTYPE_FP8 if fp8 else L.DTYPE_BF16, n // 16, 16, 1, 128)
    new = torch.randn(n, 2, 1, 128, device="cuda").to(torch.bfloat16)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    ws, ctrl = L.new_workspace(L.ATTENTION_WS_BYTES), L.new_workspace(L.CTRL_BYTES)
    L.kv_write(new[:, 0], new[:, 1], slots, k, v, ctrl, k_scales=ks, v_scales=vs)
    q = torch.randn(q_len, heads, 128, device="cuda").to(torch.bfloat16)
    args = (q, k, v, torch.arange(n // 16, dtype=torch.int32, device="cuda").view(1, -1),
            torch.tensor([0, q_len], dtype=torch.int32, device="cuda"),
            torch.tensor([n], dtype=torch.int32, device="cuda"), ws)
    good, _ = L.paged_attention(*args, max_q=q_len, k_scales=ks, v_scales=vs)
    assert L.get_error(ws) == L.MOE_OK
    try:
        L.debug_set_pipeline_fault(True, 2_000_000)
        L.paged_attention(*args, max_q=q_len, k_scales=ks, v_scales=vs)
        assert L.get_error(ws) == L.MOE_ERR_TIMEOUT
    finally:
        L.debug_set_pipeline_fault(False)
    assert not bool(ws[L.CTRL_BYTES:L.ATTENTION_CTRL_BYTES].any())
    again, _ = L.paged_attention(*args, max_q=q_len, k_scales=ks, v_scales=vs)
    assert L.get_error(ws) == L.MOE_OK and torch.equal(good, again)
