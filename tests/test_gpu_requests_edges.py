"""Adapters and sampling at the ends of what their calls allow (GB300): buffers of more than 2^31 elements, and a process's
first call inside a capture."""
import subprocess
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("rows,k,cols", [(530001, 4096, [64]), (262200, 64, [8192, 8])])
def test_adapters_over_more_elements_than_31_bits_count(rows, k, cols):
    """The last rows of x, or of base and out, are theirs as if alone."""
    from prefix_reused_prefill_gb300 import Adapters
    g = torch.Generator(device=DEV).manual_seed(rows)
    n = sum(cols)
    site = Adapters([((torch.randn(16 * len(cols), k, generator=g, device=DEV) * k ** -0.5).to(BF),
                      torch.randn(n, 16, generator=g, device=DEV).to(BF), 1.0)], cols)
    assert rows * max(k, n) > 2 ** 31
    x = torch.full((rows, k), 0.5, dtype=BF, device=DEV)
    base = torch.full((rows, n), -1.0, dtype=BF, device=DEV)
    last = 300
    x[-last:] = torch.randn(last, k, generator=g, device=DEV).to(BF)
    base[-last:] = torch.randn(last, n, generator=g, device=DEV).to(BF)
    ends = base[-last:].float()
    added = site.kvr_adapt(x[-last:].contiguous(), i32([0, last]), i32([0]), out=torch.empty(last, n, device=DEV))
    same = site.kvr_adapt(x[:1].contiguous(), i32([0, 1]), i32([0]), out=torch.empty(1, n, device=DEV))
    got = site.kvr_adapt(x, i32([0, 5, rows]), i32([-1, 0]), base, out=base)
    assert (got[:5] == -1).all()
    # (half a step of bf16, and 32-bit sums in two orders)
    near = lambda a, b: ((a.float() - b).abs() <= 2.0 ** -8 * b.abs() + 1e-4).all()
    assert near(got[-last:], ends + added)
    for r in range(5, rows - last, 1 << 16):
        assert near(got[r:min(r + (1 << 16), rows - last)], same - 1.0)


def test_sampling_over_more_elements_than_31_bits_count():
    from prefix_reused_prefill_gb300 import kvr_accept, kvr_sample
    rows, vocab = 8200, 262144
    g = torch.Generator(device=DEV).manual_seed(1)
    logits = torch.zeros(rows, vocab, dtype=BF, device=DEV)
    logits[-8:] = (torch.randn(8, vocab, generator=g, device=DEV) * 3).to(BF)
    u = torch.rand(rows, generator=g, device=DEV)
    token, prob = kvr_sample(logits, u)
    want = kvr_sample(logits[-8:].contiguous(), u[-8:].contiguous())
    assert torch.equal(token[-8:], want[0]) and torch.equal(prob[-8:], want[1])
    assert torch.equal(token[:-8].double(), (u[:-8].double() * vocab).floor())
    tokens = token.roll(1).contiguous()
    cu = i32(list(range(0, rows + 1, 4)))
    kept, following = kvr_accept(logits, tokens, cu, u, u[::4].contiguous(), temperature=1.0)
    tail = kvr_accept(logits[-8:].contiguous(), tokens[-8:].contiguous(), i32([0, 4, 8]), u[-8:].contiguous(),
                      u[::4][-2:].contiguous(), temperature=1.0)
    assert torch.equal(kept[-2:], tail[0]) and torch.equal(following[-2:], tail[1])


FIRST = """
import torch
from prefix_reused_prefill_gb300 import Adapters, kvr_accept, kvr_sample
g = torch.Generator().manual_seed(1)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
bf = lambda *n: torch.randn(*n, generator=g).bfloat16().cuda()
site = Adapters([(bf(16, 256), bf(64, 16), 1.0)], [64])
x, cu, which = bf(300, 256), i32([0, 300]), i32([0])
logits, u = torch.randn(8, 1000, generator=g).cuda(), torch.rand(8, generator=g).cuda()
tokens, cu2, un = i32(list(range(8))), i32([0, 4, 8]), torch.rand(2, generator=g).cuda()
calls = dict(adapt=lambda: (site.kvr_adapt(x, cu, which),), sample=lambda: kvr_sample(logits, u, dist=True),
             accept=lambda: kvr_accept(logits, tokens, cu2, u, un))
call = calls["{name}"]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, call()))
print("as outside")
"""


@pytest.mark.parametrize("name", ["adapt", "sample", "accept"])
def test_the_first_call_of_a_process_in_a_capture(name):
    r = subprocess.run([sys.executable, "-c", FIRST.replace("{name}", name)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as outside" in r.stdout, r.stderr[-2000:]
