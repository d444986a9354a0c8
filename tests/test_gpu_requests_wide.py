"""Conversations with adapters through a layer of real widths, more rows than one block of tokens (GB300).

The oracle runs each conversation on weights that its adapter is merged into.  K and V, and rows of the small shapes, are
held to the stated bar, 1e-2 + 2e-2 |oracle|.  At 7B widths the chain of bf16 rounding points alone moves a row's elements
by 0.0034 of its rms (root mean square, measured without any adapter; 39 of 10^6 elements are then beyond 1e-2 of it, as 3
of their deviations are passed by 0.3% of a normal distribution): there a row's rms error is held to 1e-2 of its rms.  An
adapter left out moves rows by a tenth of their rms and more."""
import dataclasses

import numpy as np
import pytest
import torch

import workloads
from conftest import oracle_dims, oracle_weights
from oracle import model as om
from test_gpu_requests import ATOL, close, make_adapters

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("name,lens,which", [("qwen7b", [280, 21], [1, 0]),          # 301 rows: two blocks of tokens
                                              ("small", [300, 1, 260], [0, -1, 1]),   # three
                                              ("small_bf16", [300, 1, 260], [0, 1, 1]), ("small_q4k", [270, 40], [1, 0])])
def test_batch_of_more_than_one_block(name, lens, which):
    from prefix_reused_prefill_gb300 import Kvr, config_for_shape
    shape = dataclasses.replace(workloads.SHAPES[name], n_layers=1)
    lws = workloads.stack_weights(shape, 7)
    kv = Kvr(config_for_shape(shape, 4, 1024, 640), device="cuda")
    w, W = kv.weights(workloads.weights_to(lws, "cuda")), [oracle_weights(shape, lw) for lw in lws]
    ad, merged = make_adapters(kv, shape, W, [16, 64], 4)
    seqs = [list(range(1000 * j, 1000 * j + m)) for j, m in enumerate(lens)]
    xs = [workloads.hidden_for_tokens(s, shape.hidden, 5 + j) for j, s in enumerate(seqs)]
    out = kv.kvr_prefill_batch_adapted(list(range(len(lens))), seqs, torch.cat(xs).cuda(), w, ad, which)
    kv.kvr_sync_status()
    if name == "qwen7b":
        plain = workloads.bf16_to_f64(kv.kvr_prefill_batch([3], [seqs[0]], xs[0].cuda(), w))
        moved = workloads.bf16_to_f64(out[:lens[0]]) - plain
        assert (np.mean(moved ** 2, axis=1) > 1e-2 * np.mean(plain ** 2, axis=1)).all()
    at = 0
    for j, m in enumerate(lens):
        cache = om.SlotKV(1, shape.n_kv_heads, 1024, shape.head_dim)
        ref = om.prefill(oracle_dims(shape), merged[which[j]] if which[j] >= 0 else W, cache, workloads.bf16_to_f64(xs[j]), 0)
        got = workloads.bf16_to_f64(out[at:at + m])
        if name == "qwen7b":
            off = np.sqrt(np.mean((got - ref) ** 2, axis=1) / np.mean(ref ** 2, axis=1))
            assert (off <= ATOL).all(), (j, off.max())
        else:
            close(got, ref, f"conversation {j} rows")
        k, v = kv.kvr_slot_kv(j, 0)
        close(workloads.bf16_to_f64(k[:, :m]), cache.K[0][:, :m], f"conversation {j} K")
        close(workloads.bf16_to_f64(v[:, :, :m].transpose(1, 2)), cache.V[0][:, :m], f"conversation {j} V")
        at += m
