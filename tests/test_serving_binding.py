"""What the serving operators' Python entry points refuse, and what they take (CPU only)."""
import pytest
import torch

from mixture_experts_forward_gb300 import _lib as L
from mixture_experts_forward_gb300 import build as moe_build


@pytest.fixture(scope="module", autouse=True)
def built():
    moe_build.build()


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def attention_args(B=1, T=3, Hq=4, entries=4):
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    sc = torch.zeros(4, 2, 16)
    return dict(q=torch.zeros(T, Hq, 64, dtype=torch.bfloat16), k_cache=pages, v_cache=pages,
                block_table=i32(B, entries), cu_q=i32(B + 1), kv_lens=i32(B),
                ws=torch.zeros(L.ATTENTION_CTRL_BYTES, dtype=torch.uint8), max_q=T, k_scales=sc,
                v_scales=sc)


@pytest.mark.parametrize("B,max_q", [(1, 0), (0, 3), (0, 0)])
@pytest.mark.parametrize("out", [None, torch.zeros(3, 4, 64, dtype=torch.bfloat16)])
def test_rows_that_no_sequence_would_write(B, max_q, out):
    a = attention_args(B=B)
    a.update(max_q=max_q, out=out)
    with pytest.raises(L.MoeError, match="nothing would write out"):
        L.paged_attention(**a)


def all_calls():
    """name -> (entry point, valid arguments but for their place)."""
    a = attention_args(T=3)
    cache = {n: a[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales", "ws")}
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    p = torch.zeros(2, 4, 50)
    return dict(
        write=(L.kv_write, dict(cache, k=x, v=x, slots=i32(3))),
        read=(L.kv_read, dict(cache, block_table=i32(1, 4), cu_rows=i32(2), starts=i32(1), rows=3)),
        attention=(L.paged_attention, dict(a, out=torch.zeros_like(a["q"]))),
        verify=(L.verify_draft, dict(p=p, q=p[:, :3], draft=i32(2, 3), u_accept=p[:, 0, :3].contiguous(),
                                     u_sample=p[:, 0, 0].contiguous(), draft_lens=i32(2), ws=a["ws"])))


@pytest.mark.parametrize("name", ["write", "read", "attention", "verify"])
def test_tensors_in_host_memory(name):
    """Refused by the binding, before an address is passed on."""
    call, args = all_calls()[name]
    with pytest.raises(L.MoeError, match="on one GPU"):
        call(**args)
