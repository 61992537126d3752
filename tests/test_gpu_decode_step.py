"""The step's operators together, as examples/decode_step.py runs them."""
import math
import os
import sys

import pytest
import torch

import step_reference as R
from mixture_experts_forward_gb300 import _lib as L

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_step as E  # noqa: E402

pytestmark = pytest.mark.gpu


def test_decoding_runs_and_keeps_its_books():
    a, b = E.main(steps=6), E.main(steps=6)
    assert a["tokens"] == b["tokens"] and a["status"] == [L.MOE_OK] * 3
    for r in (a, b):
        # every page is held or free, and a sequence holds what its positions fill
        assert sum(r["held"]) + r["free"] == r["pages"]
        assert r["held"] == [-(-n // E.PAGE) for n in r["lengths"]]
        held, free = r["after"]
        assert held == [0] + r["held"][1:] and free == r["free"] + r["held"][0]
        assert all(13 not in t for t in r["tokens"])                 # the token that the mask forbids
        s = r["server"]
        ids = s.table[s.table >= 0].tolist() + s.free[:free].tolist()
        assert sorted(ids) == list(range(r["pages"]))                # each once


def test_a_step_against_the_plain_form():
    """The logits of one step, through pages, rotary positions, cache, attention and experts, against
    the same layer without a cache in 64 bits.  What is rounded on the way: bf16 products and sums of
    the residual stream (2^-8 each, a dozen of them), E4M3 keys and values (2^-4 of an element, averaged
    over 64 to 512 of them)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    s = E.Server(2, 1, 12, 64, seed=4)
    n = [21, 34]
    text = [torch.randint(E.VOCAB, (k,), device="cuda", generator=g, dtype=torch.int32) for k in n]
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    s.forward(torch.cat([t[:-2] for t in text]), lens - 2, max(n) - 2)
    s.len = lens - 2
    got = s.forward(torch.cat([t[-2:] for t in text]), torch.full_like(lens, 2), 2).double().cpu()
    assert s.status() == [L.MOE_OK] * 3
    theta = R.frequencies(E.HEAD_DIM, scaling="turns", factor=4.0, original=4096, low=1.0, high=4.0)
    d = lambda t: t.double().cpu()  # noqa: E731
    wide = lambda w, sc: (w.view(torch.float8_e4m3fn).double() *  # noqa: E731
                          sc.double().repeat_interleave(128, 1).repeat_interleave(128, 2)).cpu()
    up, down = wide(s.up, s.up_s), wide(s.dn, s.dn_s)
    want = []
    for t in text:
        T = t.numel()
        x = d(s.embed[t.long()])
        qkv = (x @ d(s.w_qkv)).view(T, -1, E.HEAD_DIM)
        q, k, v = qkv.split([E.Q_HEADS, E.KV_HEADS, E.KV_HEADS], 1)
        pos = torch.arange(T)
        q, k = R.rotated(q, pos, theta, False)[0], R.rotated(k, pos, theta, False)[0]
        rep = E.Q_HEADS // E.KV_HEADS
        sc = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(rep, 1)) / math.sqrt(E.HEAD_DIM)
        sc = sc.masked_fill(torch.ones(T, T).triu(1).bool(), -math.inf)
        a = torch.einsum("hij,jhd->ihd", torch.softmax(sc, -1), v.repeat_interleave(rep, 1)).reshape(T, -1)
        x = (x + a @ d(s.w_o))[-2:]
        z = x @ d(s.w_router)
        top, ids = torch.topk(z, E.TOP_K, 1)
        x = x + R.few(x, ids, torch.softmax(top, 1), up, down, True)[0]
        want.append(x @ d(s.w_out))
    want = torch.cat(want)
    assert ((got - want).norm() / want.norm()) < 12 * 2.0 ** -8
