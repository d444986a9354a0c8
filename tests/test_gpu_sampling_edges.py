"""Sampling where little weight decides, on the GPU against 64-bit arithmetic (GB300)."""
import math

import numpy as np
import pytest
import torch

from oracle import sampling as so

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("vocab", [262144, 250001])
def test_weights_of_a_few_units_are_rounded_to_the_nearest(vocab, given):
    """A rejected draft leaves tokens of 4.9 and 4.1 units of 2^-44 of its own weight, half of them each: 54.4% of what is
    left are the larger ones', 55.6% once both are whole numbers next to them.  By u = 0.52 the next token is a
    larger one; cut to four units both would hold one half, and it would be a smaller one."""
    from prefix_reused_prefill_gb300 import kvr_accept
    logits = torch.empty(2, vocab)
    half = (vocab - 1) // 2
    logits[:, 0] = 0.0
    logits[:, 1:1 + half] = math.log(4.9) - 44 * math.log(2)
    logits[:, 1 + half:] = math.log(4.1) - 44 * math.log(2)
    u, u_next = torch.tensor([1 - 2.0 ** -24, 0.5]), torch.tensor([0.52])
    tokens, q = torch.tensor([7, 0], dtype=torch.int32), None
    if given:
        q = torch.zeros(2, vocab)
        q[:, 0] = 1.0
    share = torch.softmax(logits[0].double(), 0)
    assert share[0] < u[0].double()                     # (so the draft does not stay)
    kept, following = kvr_accept(logits.to(DEV), tokens.to(DEV), torch.tensor([0, 2], dtype=torch.int32, device=DEV), u.to(DEV),
                                 u_next.to(DEV), draft_probs=None if q is None else q.to(DEV))
    want = so.accept(logits.double().numpy(), tokens.tolist(), u.double().numpy(), 0.52,
                     q=None if q is None else q.double().numpy())
    assert want[0] == 0 and 1 <= want[1] <= half
    assert kept.item() == 0 and 1 <= following.item() <= half, (kept.item(), following.item(), half)
