"""Pins of the paged cache's float64 oracle, and the host side of the C ABI (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import pages as op


def test_tables_by_hand():
    t = op.Tables(6, 3, 256)
    # 65 tokens take pages 0 and 1, one token takes page 2
    assert t.plan([0, 0], [65, 1], 80)
    assert t.pages == [[0, 1], [2], []] and t.free == [5, 4, 3] and t.lens == [65, 1, 0]
    assert t.rows[63:66] == [(0, 63, 63), (0, 64, 64), (1, 0, 128)]
    # the first gives pages 0 and 1 back (0 on top), the second takes them in order
    assert t.plan([0, 1], [0, 128], 128)
    assert t.pages == [[], [2, 0, 1], []] and t.free == [5, 4, 3]
    assert t.rows[0] == (1, 1, 129) and t.rows[63] == (1, 64, 0) and t.rows[-1] == (1, 128, 64)
    # refused: more than there is, more than kept, more rows than the buffers, a longer step than promised
    for keep, add, rows, most in [([0, 129], [256, 0], 256, 0), ([1, 129], [0, 0], 8, 0), ([0, 129], [5, 4], 8, 0),
                                  ([0, 129], [5, 0], 8, 4), ([0, 129], [-1, 0], 8, 0), ([0, 129], [0, 128], 128, 0)]:
        assert not t.plan(keep, add, rows, most)
        assert t.pages == [[], [2, 0, 1], []] and t.lens == [0, 129, 0] and t.rows == []


def test_quantiser_by_hand():
    x = np.zeros((1, 32))
    x[0, :6] = [7.0, 0.5, 1.5, -2.5, -0.5, 3.4999]       # s = 1: halves go to the even code
    c, s = op.quantise(x)
    assert s.item() == 1.0 and list(c[0, 0, :6]) == [7, 0, 2, -2, 0, 3]
    c, s = op.quantise(np.full((1, 32), 1e6))             # beyond the largest scale: clipped to 7 * 8188
    assert s.item() == 8188.0 and (c == 7).all()
    c, s = op.quantise(np.full((1, 32), 2.0 ** -23))      # 2^-23 / 7 is below half of the least fp16 number
    assert s.item() == 0.0 and (c == 0).all()
    x = np.ones((1, 64))
    x[0, 40] = np.inf
    assert np.isnan(op.values(x)[0, 32:]).all() and np.allclose(op.values(x)[0, :32], 1.0, rtol=2 ** -11)


def test_norm_rotate_by_hand():
    x = np.zeros((1, 64))
    x[0, 0] = 3.0
    y = op.norm_rotate(x, 1, 1.0)                          # theta = 1: every pair turns by one radian
    assert np.allclose(y[0, [0, 32]], [3 * np.cos(1), 3 * np.sin(1)]) and np.count_nonzero(y) == 2
    y = op.norm_rotate(x, 0, 1e6, gain=np.full(64, 2.0))   # x / rms = sqrt(64), times the gain
    assert np.isclose(y[0, 0], 16.0)


def test_attend_by_hand():
    k = np.zeros((1, 3, 64))
    v = np.stack([np.full(64, x) for x in (1.0, 2.0, 6.0)])[None]
    o, mag = op.attend(np.ones((2, 64)), k, v, 1.0)        # equal scores: the mean
    assert np.allclose(o, 3.0) and np.allclose(mag, 3.0)


# --------------------------------------------------------------------------- host side
@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from prefix_reused_prefill_gb300 import kvr
    return kvr.load_library()


def config(**kw):
    from prefix_reused_prefill_gb300 import paged_config
    base = dict(n_pages=10, n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=64, max_seqs=4, max_len=300, max_rows=64)
    return paged_config(**{**base, **kw})


def test_sizes(lib):
    for d in (64, 128):
        cfg = config(head_dim=d)
        # per token and KV head: d / 2 bytes of codes and d / 32 scales, for k and for v
        assert lib.kvr_pages_pool_bytes(ctypes.byref(cfg)) == 2 * 10 * 2 * 64 * 2 * (d // 2 + d // 32 * 2)
        assert lib.kvr_pages_work_bytes(ctypes.byref(cfg)) > 300 * d // 2 * 8


@pytest.mark.parametrize("field,value", [
    ("n_pages", 0), ("n_pages", (1 << 24) + 1), ("n_layers", 0), ("n_kv_heads", 0), ("n_q_heads", 7),
    ("n_q_heads", 130), ("head_dim", 96), ("max_seqs", 0), ("max_seqs", 2049), ("max_len", 0),
    ("max_len", (1 << 22) + 1), ("max_rows", 0), ("max_rows", (1 << 22) + 1), ("act", 2), ("rope_theta", 0.0),
    ("rope_theta", float("nan")), ("norm_eps", -1.0), ("norm_eps", float("inf"))])
def test_invalid_configurations_are_refused(lib, field, value):
    cfg = config()
    setattr(cfg, field, value)
    assert lib.kvr_pages_pool_bytes(ctypes.byref(cfg)) == 0 and lib.kvr_pages_work_bytes(ctypes.byref(cfg)) == 0
    out = ctypes.c_void_p()
    assert lib.kvr_pages_create(ctypes.byref(cfg), 256, 1 << 40, 256, 1 << 40, ctypes.byref(out)) == -1
    assert not out.value


def test_pools_beyond_any_card_are_refused(lib):
    cfg = config(n_pages=1 << 23, n_kv_heads=16, n_q_heads=16)   # 2^27 page heads
    assert lib.kvr_pages_pool_bytes(ctypes.byref(cfg)) == 0


def test_create_checks_its_memory(lib):
    cfg = config()
    pb, wb = lib.kvr_pages_pool_bytes(ctypes.byref(cfg)), lib.kvr_pages_work_bytes(ctypes.byref(cfg))
    out = ctypes.c_void_p()
    for pool, work, p, w, code in [(None, 256, pb, wb, -1), (256, None, pb, wb, -1), (128, 256, pb, wb, -1),
                                   (256, 128, pb, wb, -1), (256, 256, pb - 1, wb, -2), (256, 256, pb, wb - 1, -2)]:
        assert lib.kvr_pages_create(ctypes.byref(cfg), pool, p, work, w, ctypes.byref(out)) == code
        assert not out.value
    assert lib.kvr_pages_create(ctypes.byref(cfg), 256, pb, 256, wb, None) == -1


def test_null_handle(lib):
    assert lib.kvr_pages_destroy(None) == -1 and lib.kvr_pages_sync(None, None) == -1
    assert lib.kvr_page_plan(None, 1, None, None, 1, 1, None) == -1
    assert lib.kvr_page_append(None, 0, None, 0, None, 0, None, 0, None, None, 1, None, 1, None) == -1
    assert lib.kvr_page_read(None, 0, None, None, 1, None) == -1
    assert lib.kvr_page_attend(None, 0, None, 0, None, 0, 1.0, 1, None) == -1
    assert lib.kvr_pages_tables(None, None) == -1
    assert lib.kvr_pages_error(None) == b"null handle"
