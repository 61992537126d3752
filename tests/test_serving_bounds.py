"""The bounds of serving_forms.py tell a form from one with a term left out (CPU): the forms'
roundings of weights and values are imitated in 64 bits, with and without a mistake."""
import pytest
import torch

import serving_forms as F


def e4m3(x):
    return x.float().clamp(-448, 448).to(torch.float8_e4m3fn).double()


def rounded(x, dtype):
    return x.float().to(dtype).double()


def imitated(few, fp8, q_len, G, D, mistake):
    """(over, under): is some output over its bound, is none."""
    q, c, scale = F.same_sign_case(q_len, G, D, fp8, "cpu")
    n = 2001
    want, _, tol, _ = F.attention(q, c, [q_len], [n], scale=scale, causal=False)
    x = q.view(-1, D).double() @ c.rows("k", 0, n)[:, 0].T * scale
    w = torch.exp(x)                                       # the first key's score is 0
    v = c.rows("v", 0, n)[:, 0]
    if few and not fp8:
        hi = rounded(w, torch.bfloat16)
        p = hi if mistake else hi + rounded(w - hi, torch.bfloat16)
    elif few:
        p = 16.0 * w                                       # the value scales are all the same
        hi = e4m3(p)
        p = (hi if mistake else hi + e4m3(16.0 * (rounded(p, torch.float16) - hi)) / 16.0) / 16.0
    elif fp8:
        p = rounded(8.0 * w, torch.bfloat16 if mistake else torch.float16) / 8.0
        v = rounded(v, torch.float16)
    else:
        p = rounded(w, torch.bfloat16)
        p = rounded(p * (1 - 2.0 ** -8), torch.bfloat16) if mistake else p
    o = rounded(p @ v / w.sum(1, keepdim=True), torch.bfloat16).view(q_len, G, D)
    return bool(((o - want).abs() > tol).any())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("few,fp8", [(True, False), (True, True), (False, False), (False, True)])
def test_the_bounds_pass_the_form_and_not_a_dropped_term(few, fp8, D):
    q_len, G = (9, 4) if few else (70, 4)
    assert not imitated(few, fp8, q_len, G, D, False)
    assert imitated(few, fp8, q_len, G, D, True)
