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
