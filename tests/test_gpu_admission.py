"""Pages that one sequence gave back and another took: through plan, rotary positions, cache and
attention, as examples/decode_step.py runs them."""
import os
import sys

import pytest
import torch

from mixture_experts_forward_gb300 import _lib as L

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_step as E  # noqa: E402

pytestmark = pytest.mark.gpu


def books(s, held, free, pages):
    """Every page is held once or free."""
    ids = s.table[s.table >= 0].tolist() + s.free[:free].tolist()
    assert sorted(ids) == list(range(pages)) and sum(held) + free == pages


def test_a_waiting_sequence_takes_an_ended_ones_row():
    a, b = (E.main(steps=4, waiting=29) for _ in range(2))
    assert a["tokens"] == b["tokens"] and a["ended"] == b["ended"] and a["status"] == [L.MOE_OK] * 3
    assert a["ended"] == E.main(steps=4, waiting=0)["tokens"][0]
    assert a["held"] == [-(-n // E.PAGE) for n in a["lengths"]]
    assert a["lengths"][0] == 29 - 1 + len(a["tokens"][0]) and len(a["tokens"][0]) >= 4
    assert all(13 not in t for t in a["tokens"])                     # the token that the mask forbids
    books(a["server"], a["held"], a["free"], a["pages"])


def test_logits_over_pages_that_others_had():
    """The same sequence on a server that has served others and on a fresh one: the same calls but
    for the pages, so the same bits."""
    g = torch.Generator(device="cuda").manual_seed(5)
    text = lambda n: torch.randint(E.VOCAB, (n,), device="cuda", generator=g, dtype=torch.int32)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    used, fresh = E.Server(2, 1, 6, 64, seed=4), E.Server(2, 1, 6, 64, seed=4)
    used.forward(text(35 + 47), i32(35, 47), 47)                     # six pages: all
    used.len = i32(35, 47)
    assert int(used.count) == 0
    had = used.table[:, :3].tolist()
    used.end(0)
    used.end(1)
    books(used, [0, 0], 6, 6)
    mine, two = text(61), text(2)
    logits = []
    for s in (used, fresh):
        s.admit(1, mine)
        new = i32(0, 2)
        logits.append(s.forward(two, new, 2))
        assert s.status() == [L.MOE_OK] * 3
    took = used.table[1].tolist()
    assert set(took) & set(had[0]) and set(took) & set(had[1]) and took != fresh.table[1].tolist()
    assert torch.equal(*logits)
