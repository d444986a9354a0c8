"""Refusals of sampling and adapters that need no GPU: checks of arguments come before anything of the device."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from prefix_reused_prefill_gb300 import kvr
    return kvr.load_library()


A, B, C, D, E = (1 << 32) * 1, (1 << 32) * 2, (1 << 32) * 3, (1 << 32) * 4, (1 << 32) * 5   # addresses that nobody reads


def call(fn, default, **change):
    assert set(change) <= set(default)
    return fn(*{**default, **change}.values())


def test_sample(lib):
    good = dict(x=A, type=2, stride=64, rows=4, vocab=64, s=None, u=B, token=C, prob=D, dist=E, ds=64, st=None)
    for bad in (dict(type=3), dict(type=-1), dict(stride=63), dict(rows=-1), dict(rows=(1 << 20) + 1), dict(vocab=0),
                dict(vocab=262145), dict(x=None), dict(x=A + 2), dict(u=None), dict(u=B + 1), dict(token=None), dict(token=C + 2),
                dict(prob=D + 1), dict(dist=E + 3), dict(ds=63), dict(token=A + 1020), dict(prob=C + 8), dict(dist=A + 4),
                dict(dist=B - 16)):
        assert call(lib.kvr_sample, good, **bad) == -1, bad
        assert lib.kvr_batch_error()
    assert call(lib.kvr_sample, good, rows=0, x=None, u=None) == 0


def test_accept(lib):
    good = dict(x=A, type=2, stride=64, rows=4, vocab=64, s=None, n=2, cu=B, tokens=B + 64, q=E, qs=64, u=B + 128, un=B + 192,
                acc=C, nxt=C + 64, work=D, wb=16, st=None)
    assert lib.kvr_accept_work_bytes(-1) == 0 and lib.kvr_accept_work_bytes(4) == 16
    for bad in (dict(n=0), dict(n=65537), dict(cu=None), dict(tokens=None), dict(u=None), dict(un=None), dict(acc=None),
                dict(nxt=None), dict(qs=63), dict(q=E + 2), dict(acc=C + 1), dict(nxt=C + 4), dict(work=B + 64), dict(acc=D + 8)):
        assert call(lib.kvr_accept, good, **bad) == -1, bad
    for bad in (dict(work=None), dict(work=D + 8), dict(wb=15)):
        assert call(lib.kvr_accept, good, **bad) == -2, bad


def test_adapt(lib):
    from prefix_reused_prefill_gb300.kvr import KvrAdapterSite
    sites = []

    def site(**k):
        f = {**dict(table=E, n=2, rank=16, k=64, parts=2, cols=(32, 8, 0), type=0), **k}
        sites.append(KvrAdapterSite(f["table"], f["n"], f["rank"], f["k"], f["parts"], (ctypes.c_int * 3)(*f["cols"]), f["type"]))
        return ctypes.byref(sites[-1])

    for bad in (dict(table=None), dict(table=E + 4), dict(n=0), dict(rank=0), dict(rank=12), dict(rank=136), dict(k=0), dict(k=60),
                dict(parts=0), dict(parts=4), dict(cols=(32, 4, 0)), dict(cols=(0, 8, 0)), dict(type=2), dict(type=-1)):
        assert lib.kvr_adapt_work_bytes(site(**bad), 4) == 0, bad
    s = site()
    wb = lib.kvr_adapt_work_bytes(s, 4)
    assert wb > 0 and lib.kvr_adapt_work_bytes(s, -1) == 0 and lib.kvr_adapt_work_bytes(s, (1 << 22) + 1) == 0
    good = dict(site=s, x=A, xs=64, cu=B, which=B + 64, n=2, rows=4, base=C, bs=40, out=C, os=40, type=2, work=D, wb=wb, st=None)
    for bad in (dict(site=site(k=60)), dict(xs=56), dict(xs=68), dict(cu=None), dict(which=None), dict(n=0), dict(n=2049),
                dict(rows=-1), dict(rows=(1 << 22) + 1), dict(x=None), dict(x=A + 8), dict(base=C + 8), dict(out=None), dict(os=32),
                dict(os=44), dict(bs=48), dict(type=1), dict(out=C + 160), dict(out=A), dict(out=E - 16), dict(work=A),
                dict(work=C + 16), dict(cu=D)):
        assert call(lib.kvr_adapt, good, **bad) == -1, bad
    for bad in (dict(work=None), dict(work=D + 8), dict(wb=wb - 1)):
        assert call(lib.kvr_adapt, good, **bad) == -2, bad
    assert call(lib.kvr_adapt, good, rows=0) == 0
