"""What forward_few refuses of the tensors behind its arguments, before an address is passed on
(CPU only)."""
import pytest
import torch

from mixture_experts_forward_gb300 import _lib as L
from mixture_experts_forward_gb300 import build as moe_build

M, K, N, E = 3, 256, 128, 4


@pytest.fixture(scope="module", autouse=True)
def built():
    moe_build.build()


def tensors(fp8):
    bf, u8 = torch.bfloat16, torch.uint8
    t = dict(logits=torch.zeros(M, E), x=torch.zeros(M, K, dtype=bf),
             w=torch.zeros(E, 2 * N, K, dtype=u8 if fp8 else bf), w2=torch.zeros(E, K, N, dtype=u8 if fp8 else bf))
    if fp8:
        t.update(w_scales=torch.zeros(E, 2 * N // 128, K // 128), w2_scales=torch.zeros(E, K // 128, N // 128))
    return t


def call(fp8, **kw):
    a = L.forward_args(dtype=L.DTYPE_FP8 if fp8 else L.DTYPE_BF16, M=M, K=K, N=N, E=E, top_k=2, gated=1,
                       **{**tensors(fp8), **kw})
    L.forward_few(a, torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8))


def wrong():
    bf = torch.bfloat16
    z = torch.zeros
    every = [dict(logits=z(M, E, dtype=bf)), dict(logits=z(M, E - 1)), dict(logits=z(E, M).t()),
             dict(logits=None), dict(x=z(M, K)), dict(x=z(M - 1, K, dtype=bf)), dict(x=None),
             dict(x=z(M, 2 * K, dtype=bf)[:, :K]), dict(w=None), dict(w2=None), dict(w=z(E, 2 * N, K))]
    fp8 = [dict(w=z(E, 2 * N, K, dtype=bf)), dict(w=z(E, N, K, dtype=torch.uint8)),
           dict(w2=z(E, N, K, dtype=torch.uint8).transpose(1, 2)), dict(w_scales=None),
           dict(w2_scales=z(E, 2, 1, dtype=bf)), dict(w_scales=z(E, 1, 2)), dict(w2_scales=z(E, 2, 2)[:, :, :1])]
    b16 = [dict(w=z(E, 2 * N, K, dtype=torch.uint8)), dict(w2=z(E - 1, K, N, dtype=bf)),
           dict(w=z(E, 2 * N, K, dtype=torch.float16))]
    return [(True, kw) for kw in every + fp8] + [(False, kw) for kw in every + b16]


@pytest.mark.parametrize("case", range(len(wrong())))
def test_tensors_of_other_types_and_sizes(case):
    fp8, kw = wrong()[case]
    with pytest.raises(L.MoeError) as e:
        call(fp8, **kw)
    assert "on one GPU" not in str(e.value)


@pytest.mark.parametrize("fp8", [True, False])
def test_tensors_in_host_memory(fp8):
    with pytest.raises(L.MoeError, match="on one GPU"):
        call(fp8)
    w = torch.zeros(E, 2 * N, K, dtype=torch.float8_e4m3fn)        # codes under their own type
    with pytest.raises(L.MoeError, match="on one GPU"):
        call(True, w=w, x=torch.zeros(M + 4, K, dtype=torch.bfloat16))


def test_addresses_that_the_caller_fills_in():
    """Not the tensors that forward_args was given (if any): those are not looked at."""
    kw = dict(dtype=L.DTYPE_FP8, M=M, K=K, N=N, E=E, top_k=2, gated=1)
    one = torch.zeros(1, K, dtype=torch.bfloat16)
    other = L.forward_args(**{**kw, "M": 1}, **{**tensors(True), "x": one})
    empty = L.forward_args(**kw)
    t = tensors(True)
    for a in (other, empty):
        a.M = M
        for name in t:
            setattr(a, name, t[name].data_ptr())
        with pytest.raises(L.MoeError, match="on one GPU"):        # of out and ws
            L.forward_few(a, torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8))
    small = L.forward_args(**{**kw, "M": 1}, **{**t, "x": one})
    small.M = M                                                    # more tokens than x has
    with pytest.raises(L.MoeError, match="x is bf16"):
        L.forward_few(small, torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8))
