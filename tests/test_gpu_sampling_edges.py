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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("levels", [[(3.0, 1), (1.0, 2000)], [(3.0, 200), (1.0, 70), (0.998, 70), (-2.0, 1700)],
                                    [(1.0, 129)], [(2.0, 3), (1.0, 126)], [(2.0, 1), (1.0, 64), (0.5, 65)], [(9.0, 47), (1.0, 2001)]])
def test_lists_of_many_equal_logits_beside_others(levels, dtype):
    """In the order of their index, wherever the run ends; the rest of the vocabulary far below."""
    from prefix_reused_prefill_gb300 import kvr_sample
    vocab, n = 40000, sum(m for _, m in levels)
    g = torch.Generator().manual_seed(n)
    row = torch.full((vocab,), -60.0)
    at, i = torch.randperm(vocab, generator=g), 0
    for x, m in levels:
        row[at[i:i + m]] = x
        i += m
    u = torch.cat([torch.rand(10, generator=g), torch.tensor([0.0, 1 - 2.0 ** -24])])
    rows = row.repeat(len(u), 1).to(dtype)
    for s in (dict(top_p=0.9999), dict(top_k=n), dict(top_k=max(n - 5, 1), top_p=0.7), dict(temperature=2.0, min_p=0.001, top_k=n)):
        token, prob = kvr_sample(rows.to(DEV), u.to(DEV), **s)
        exact = {k: v if k == "top_k" else float(np.float32(v)) for k, v in s.items()}
        for r in range(len(u)):
            want = so.sample(rows[r].double().numpy(), u[r].double().item(), **exact)
            assert token[r].item() == want[0], (s, r)
            assert abs(prob[r].double().item() - want[1]) <= 2.0 ** -23 * want[1], (s, r)
