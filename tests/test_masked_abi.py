"""Refusals of the windowed, tree, key weight and eviction calls: every check
runs before any CUDA call, so they are tested with fake device addresses, and
only where no GPU can be reached."""
import ctypes

import pytest
import torch

from scaled_dot_product_05_gb300 import _abi
from scaled_dot_product_05_gb300 import build as cuda_build


@pytest.fixture(scope="module")
def fake():
    if torch.cuda.is_available():
        pytest.skip("fake device addresses are passed only where no GPU can be reached")
    cuda_build.build()
    return _abi.lib()


OK = (8, 10)              # every check passed: no device here
F = ctypes.c_float
A = [0x100000000 * i for i in range(1, 20)]


def lay(l):
    return None if l is None else ctypes.byref(_abi.Layout(*l))


def cache(k=A[0], v=A[1], ks=A[2], vs=A[3], n=100, page=64, kl=None, vl=None):
    c = _abi.Cache(k, v, ks, vs, n, page, None if kl is None else ctypes.pointer(_abi.Layout(*kl)),
                   None if vl is None else ctypes.pointer(_abi.Layout(*vl)))
    return ctypes.byref(c)


def check(got, want):
    assert got in want if isinstance(want, tuple) else got == want


def fwd(lib, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], o=A[3], lse=A[4], B=2, Hq=8, Hkv=2, Sq=100, Skv=100, D=128, ol=None, scale=0.1, win=10,
             sinks=4, dt=0)
    a.update(kw)
    return lib.sdpa_fwd_window(a["q"], a["k"], a["v"], a["o"], a["lse"], a["B"], a["Hq"], a["Hkv"], a["Sq"], a["Skv"], a["D"],
                               None, None, None, lay(a["ol"]), F(a["scale"]), a["win"], a["sinks"], a["dt"], None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(sinks=0), OK), (dict(win=2 ** 31 - 1, sinks=2 ** 31 - 1), OK), (dict(D=32), OK), (dict(lse=None), OK), (dict(dt=1), OK),
    (dict(win=0), 3), (dict(win=-5), 3), (dict(sinks=-1), 3), (dict(Sq=0), 3), (dict(Hkv=3), 4), (dict(D=96), 5), (dict(dt=2), 6),
    (dict(dt=3), 6), (dict(scale=0.0), 7), (dict(q=None), 1), (dict(o=A[3] + 8), 2), (dict(o=A[0]), 9), (dict(lse=A[3] + 64), 9),
    (dict(ol=(100 * 8 * 128, 8 * 128, 64)), 11),
], ids=str)
def test_fwd_window(fake, kw, status):
    check(fwd(fake, **kw), status)


def bwd(lib, **kw):
    a = dict(b=A[:10], B=2, Hq=8, Hkv=2, Sq=100, Skv=100, D=128, win=10, sinks=4, dt=0, ws_bytes=1 << 30)
    a.update(kw)
    return lib.sdpa_bwd_window(*a["b"][:9], a["B"], a["Hq"], a["Hkv"], a["Sq"], a["Skv"], a["D"], F(0.1), a["win"], a["sinks"],
                               a["dt"], a["b"][9], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(D=64), OK), (dict(D=32), 5), (dict(win=0), 3), (dict(sinks=-1), 3), (dict(dt=2), 6), (dict(ws_bytes=1000), 12),
    (dict(b=A[:5] + [None] + A[6:10]), 1), (dict(b=A[:6] + [A[0]] + A[7:10]), 9),
], ids=str)
def test_bwd_window(fake, kw, status):
    check(bwd(fake, **kw), status)


def paged(lib, tree=False, **kw):
    a = dict(q=A[4], c=cache(), table=A[5], start=A[6], count=A[7], mask=A[8], o=A[9], lse=A[10], B=2, Hq=8, Hkv=2, Sq=5, D=128,
             width=10, scale=0.1, win=10, sinks=4, dt=0, ws=A[11], ws_bytes=1 << 30)
    a.update(kw)
    head = [a["q"], a["c"], a["table"], a["start"], a["count"]]
    size = [a["o"], a["lse"], a["B"], a["Hq"], a["Hkv"], a["Sq"], a["D"], a["width"], None, None, F(a["scale"])]
    if tree:
        return lib.sdpa_fwd_paged_tree(*head, a["mask"], *size, a["dt"], a["ws"], a["ws_bytes"], None)
    return lib.sdpa_fwd_paged_window(*head, *size, a["win"], a["sinks"], a["dt"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(sinks=0, win=1), OK), (dict(win=0), 3), (dict(sinks=-1), 3), (dict(D=32), 5), (dict(Hq=9), 4), (dict(dt=2), 6),
    (dict(scale=float("inf")), 7), (dict(ws=None), 1), (dict(ws_bytes=16), 12), (dict(o=A[0]), 9), (dict(ws=A[5]), 9), (dict(c=None), 1),
    (dict(c=cache(page=48)), 3),
    (dict(tree=True), OK), (dict(tree=True, Sq=33), OK), (dict(tree=True, mask=None), 1), (dict(tree=True, mask=A[8] + 2), 2),
    (dict(tree=True, o=A[8]), 9), (dict(tree=True, lse=A[8] + 4), 9), (dict(tree=True, dt=5), 6),
], ids=str)
def test_paged(fake, kw, status):
    check(paged(fake, **kw), status)


@pytest.mark.parametrize("rows,nr", [(1, 8), (8, 8), (9, 16), (17, 64), (64, 64), (65, 128), (5000, 128)])
def test_paged_workspace(fake, rows, nr):
    ctas = 304 if nr <= 16 else 152
    assert fake.sdpa_paged_workspace_bytes(3, 2, 2, rows, 64) == ctas * (2 * nr * 65 * 4 + 16)


def weights(lib, **kw):
    a = dict(q=A[4], c=cache(), table=A[5], start=A[6], count=A[7], lse=A[8], score=A[9], out=A[10], B=2, Hq=8, Hkv=2, Sq=5, D=128,
             width=10, stride=640, scale=0.1, causal=1, dt=0)
    a.update(kw)
    return lib.sdpa_cache_weights(a["q"], a["c"], a["table"], a["start"], a["count"], a["lse"], a["score"], a["out"], a["B"], a["Hq"],
                                  a["Hkv"], a["Sq"], a["D"], a["width"], a["stride"], None, F(a["scale"]), a["causal"], a["dt"], None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(score=None), OK), (dict(out=A[9]), OK), (dict(count=None), OK), (dict(Sq=500), OK), (dict(Hq=300), OK),
    (dict(lse=None), 1), (dict(out=None), 1), (dict(out=A[10] + 2), 2), (dict(stride=0), 3), (dict(stride=1 << 31), 3), (dict(Sq=0), 3),
    (dict(Hq=9), 4), (dict(D=32), 5), (dict(dt=2), 6), (dict(scale=-1.0), 7), (dict(out=A[9] + 64), 9), (dict(out=A[0]), 9),
    (dict(out=A[8]), 9), (dict(out=A[4]), 9),
], ids=str)
def test_weights(fake, kw, status):
    check(weights(fake, **kw), status)


def evict(lib, **kw):
    a = dict(c=cache(), table=A[5], length=A[6], score=A[7], new=A[8], kept=A[9], ks=A[10], B=2, Hkv=2, D=128, width=10, new_width=4,
             stride=640, sinks=4, recent=10, budget=256)
    a.update(kw)
    return lib.sdpa_cache_evict(a["c"], a["table"], a["length"], a["score"], a["new"], a["kept"], a["ks"], a["B"], a["Hkv"], a["D"],
                                a["width"], a["new_width"], a["stride"], a["sinks"], a["recent"], a["budget"], None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(ks=None), OK), (dict(sinks=0, recent=0, budget=1), OK), (dict(sinks=128, recent=128), OK), (dict(D=64), OK),
    (dict(score=None), 1), (dict(new=None), 1), (dict(kept=None), 1), (dict(length=None), 1), (dict(kept=A[9] + 1), 2),
    (dict(budget=0), 3), (dict(budget=257), 3), (dict(sinks=-1), 3), (dict(recent=-1), 3), (dict(sinks=128, recent=129), 3),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), 3), (dict(new_width=0), 3), (dict(stride=0), 3), (dict(B=0), 3), (dict(D=32), 5),
    (dict(c=cache(v=A[0])), 9), (dict(c=cache(kl=(0, 128, 128))), 11), (dict(kept=A[7]), 9), (dict(ks=A[9] + 4), 9), (dict(kept=A[0]), 9),
    (dict(kept=A[2]), 9),
], ids=str)
def test_evict(fake, kw, status):
    check(evict(fake, **kw), status)
