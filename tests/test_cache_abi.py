"""Refusals of the norm / rotation, cache append and cached attention calls:
every check runs before any CUDA call, so they are tested with fake device
addresses, and only where no GPU can be reached."""
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
A = [0x10000000 * i for i in range(1, 16)]


def lay(l):
    return None if l is None else ctypes.byref(_abi.Layout(*l))


def rope(table=A[8], n_pos=4096, rot=128, inter=0):
    return ctypes.byref(_abi.Rope(table, n_pos, rot, inter))


def norm_rope(lib, **kw):
    a = dict(q=A[0], k=A[1], qo=A[2], ko=A[3], B=2, S=100, Hq=8, Hkv=2, D=128, ql=None, kl=None, qol=None, kol=None, norm=1,
             qw=A[4], kw=A[5], wd=3, eps=1e-6, rope=rope(), pos=A[6], dt=0)
    a.update(kw)
    return lib.sdpa_qk_norm_rope(a["q"], a["k"], a["qo"], a["ko"], a["B"], a["S"], a["Hq"], a["Hkv"], a["D"], lay(a["ql"]),
                                 lay(a["kl"]), lay(a["qol"]), lay(a["kol"]), a["norm"], a["qw"], a["kw"], a["wd"],
                                 F(a["eps"]), a["rope"], a["pos"], a["dt"], None)


W = 12 * 128              # a fused row of 8 + 2 + 2 heads
FQ, FK = (100 * W, W, 128), (100 * W, W, 128)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(rope=None, pos=None), OK), (dict(norm=0, qw=None, kw=None), OK), (dict(wd=0), OK),
    (dict(k=None, ko=None, Hkv=0, kw=None), OK), (dict(rope=rope(rot=24)), OK), (dict(rope=rope(table=None)), OK),
    (dict(qo=A[0], ko=A[1]), OK),                                                  # in place
    (dict(q=A[0], k=A[0] + 8 * 256, ql=FQ, kl=FK), OK),                            # a fused projection
    (dict(q=A[0], k=A[0] + 8 * 256, ql=FQ, kl=FK, qo=A[0], ko=A[0] + 8 * 256, qol=FQ, kol=FK), OK),
    (dict(qo=A[2], ko=A[2] + 8 * 256, qol=FQ, kol=FK), OK),
    (dict(q=None), 1), (dict(ko=None), 1), (dict(k=None), 1),
    (dict(q=A[0] + 8), 2), (dict(qw=A[4] + 2), 2), (dict(pos=A[6] + 2), 2), (dict(rope=rope(table=A[8] + 4)), 2),
    (dict(B=0), 3), (dict(S=0), 3), (dict(Hq=0), 3), (dict(Hkv=-1), 3), (dict(Hkv=0), 3), (dict(B=1 << 20, S=1 << 12), 3),
    (dict(rope=rope(n_pos=0)), 3),
    (dict(D=96), 5), (dict(D=256), 5), (dict(rope=rope(rot=136)), 5), (dict(rope=rope(rot=12)), 5), (dict(rope=rope(rot=4)), 5),
    (dict(dt=2), 6), (dict(dt=3), 6), (dict(wd=1), 6), (dict(wd=2), 6),
    (dict(eps=-1.0), 7), (dict(eps=float("nan")), 7), (dict(eps=float("inf")), 7),
    (dict(ql=(100 * 1024, 1024, 4)), 11), (dict(kl=(0, 256, 128)), 11), (dict(qol=(100 * 1024, 128, 128)), 11),
    (dict(qo=A[0] + 256), 9), (dict(qo=A[1]), 9), (dict(ko=A[2]), 9), (dict(qo=A[4]), 9), (dict(ko=A[6]), 9), (dict(qo=A[8]), 9),
    # heads that reach into the neighbour's part of the row; in place with other strides
    (dict(qo=A[2], ko=A[2] + 7 * 256, qol=FQ, kol=FK), 9), (dict(qo=A[0], qol=FQ), 9),
])
def test_norm_rope(fake, kw, status):
    st = norm_rope(fake, **kw)
    assert st in status if isinstance(status, tuple) else st == status


def norm_rope_bwd(lib, **kw):
    a = dict(q=A[0], k=A[1], gq=A[2], gk=A[3], dq=A[4], dk=A[5], dwq=A[6], dwk=A[7], B=2, S=100, Hq=8, Hkv=2, D=128, norm=1,
             qw=A[9], kw=A[10], wd=3, ws=A[11], n=None, dql=None, dkl=None, pos=A[12], dt=1)
    a.update(kw)
    n = a["n"] if a["n"] is not None else lib.sdpa_qk_norm_rope_bwd_workspace_bytes(2, 100, 8, 2, 128)
    return lib.sdpa_qk_norm_rope_bwd(a["q"], a["k"], a["gq"], a["gk"], a["dq"], a["dk"], a["dwq"], a["dwk"], a["B"], a["S"],
                                     a["Hq"], a["Hkv"], a["D"], None, None, None, None, lay(a["dql"]), lay(a["dkl"]),
                                     a["norm"], a["qw"], a["kw"], a["wd"], F(1e-6), rope(), a["pos"], a["dt"], a["ws"], n,
                                     None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(norm=0, ws=None, n=0), OK), (dict(dwq=None, dwk=None), OK),
    (dict(k=None, gk=None, dk=None, dwk=None, Hkv=0), OK),
    (dict(dq=A[4], dk=A[4] + 8 * 256, dql=FQ, dkl=FK), OK),
    (dict(gq=None), 1), (dict(gk=None), 1), (dict(ws=None), 1), (dict(dq=None), 1),
    (dict(gq=A[2] + 8), 2), (dict(dwq=A[6] + 2), 2),
    (dict(n=64), 12), (dict(ws=A[11] + 8), 12),
    (dict(dq=A[0]), 9), (dict(dq=A[2]), 9), (dict(dk=A[4]), 9), (dict(dwq=A[0]), 9), (dict(dwk=A[6]), 9), (dict(ws=A[2]), 9),
    (dict(ws=A[9]), 9), (dict(dwq=A[10]), 9), (dict(dq=A[11]), 9), (dict(dk=A[12]), 9), (dict(dwq=A[8]), 9),
    (dict(D=48), 5), (dict(dt=2), 6),
])
def test_norm_rope_bwd(fake, kw, status):
    st = norm_rope_bwd(fake, **kw)
    assert st in status if isinstance(status, tuple) else st == status


def test_norm_rope_bwd_workspace(fake):
    f = fake.sdpa_qk_norm_rope_bwd_workspace_bytes
    assert f(1, 1, 1, 1, 128) == 2 * 128 * 4 and f(1, 1, 1, 0, 64) == 64 * 4
    assert f(8, 100000, 32, 8, 128) <= 760 * 128 * 4
    assert f(0, 1, 1, 1, 128) == f(1, 1, 1, 1, 96) == f(1, 1, 1, -1, 64) == 0


def cache(k=A[0], v=A[1], ks=A[2], vs=A[3], n_pages=50, page=64, kl=None, vl=None):
    keep = [_abi.Layout(*l) if l else None for l in (kl, vl)]
    c = _abi.Cache(k, v, ks, vs, n_pages, page, *(ctypes.pointer(l) if l else None for l in keep))
    c.keep = keep
    return c


CACHE_REFUSALS = [
    (dict(cache=dict(k=None)), 1), (dict(cache=dict(v=None)), 1), (dict(cache=dict(ks=None)), 1), (dict(cache=dict(vs=None)), 1),
    (dict(table=None), 1), (dict(start=None), 1),
    (dict(cache=dict(k=A[0] + 8)), 2), (dict(cache=dict(vs=A[3] + 2)), 2), (dict(table=A[4] + 2), 2), (dict(start=A[5] + 1), 2),
    (dict(count=A[6] + 2), 2),
    (dict(cache=dict(page=8)), 3), (dict(cache=dict(page=48)), 3), (dict(cache=dict(page=256)), 3), (dict(cache=dict(n_pages=0)), 3),
    (dict(width=0), 3), (dict(width=1 << 30), 3), (dict(B=0), 3), (dict(Hkv=0), 3), (dict(S=0), 3),
    (dict(D=32), 5), (dict(D=96), 5), (dict(dt=2), 6), (dict(dt=3), 6),
    (dict(cache=dict(kl=(64 * 256, 256, 8))), 11), (dict(cache=dict(vl=(0, 256, 128))), 11),
]


def append(lib, **kw):
    a = dict(x=A[8], y=A[9], cache={}, table=A[4], start=A[5], count=A[6], B=3, S=20, Hkv=2, D=128, width=10, xl=None,
             rope=rope(table=A[10]), dt=0)
    a.update(kw)
    c = cache(**a["cache"])
    return lib.sdpa_cache_append(a["x"], a["y"], ctypes.byref(c), a["table"], a["start"], a["count"], a["B"], a["S"], a["Hkv"],
                                 a["D"], a["width"], lay(a["xl"]), None, a["rope"], a["dt"], None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    ({}, OK), (dict(count=None, rope=None), OK), (dict(cache=dict(page=16)), OK),
    (dict(cache=dict(v=A[0] + 128, kl=(64 * 512, 512, 256), vl=(64 * 512, 512, 256))), OK),    # K and V side by side
    (dict(cache=dict(kl=(64 * 256, 128, 64 * 128))), OK),
    (dict(x=None), 1), (dict(y=A[9] + 4), 2), (dict(xl=(20 * 256, 256, 12)), 11), (dict(rope=rope(table=A[10], rot=20)), 5),
    (dict(cache=dict(kl=(64 * 256, 128, 128))), 11),                                # two slots at one address
    (dict(cache=dict(v=A[0])), 9), (dict(cache=dict(vs=A[2])), 9), (dict(x=A[0] + 256), 9), (dict(y=A[3]), 9),
    (dict(cache=dict(v=A[4] - 256)), 9), (dict(start=A[2] + 16), 9), (dict(rope=rope(table=A[1])), 9),
    (dict(cache=dict(ks=A[0])), 9), (dict(B=1 << 16, S=1 << 20), 3),
])
def test_append(fake, kw, status):
    st = append(fake, **kw)
    assert st in status if isinstance(status, tuple) else st == status


def read(lib, **kw):
    a = dict(q=A[8], o=A[9], lse=A[10], cache={}, table=A[4], start=A[5], count=A[6], B=3, Hq=8, Hkv=2, S=20, D=128, width=10,
             ql=None, ol=None, scale=0.1, causal=1, dt=0, ws=A[11], n=1 << 27)
    a.update(kw)
    c = cache(**a["cache"])
    return lib.sdpa_fwd_paged(a["q"], ctypes.byref(c), a["table"], a["start"], a["count"], a["o"], a["lse"], a["B"], a["Hq"],
                              a["Hkv"], a["S"], a["D"], a["width"], lay(a["ql"]), lay(a["ol"]), F(a["scale"]), a["causal"],
                              a["dt"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    ({}, OK), (dict(count=None, lse=None), OK), (dict(causal=0, S=1), OK),
    (dict(q=None), 1), (dict(o=None), 1), (dict(ws=None), 1), (dict(q=A[8] + 8), 2), (dict(lse=A[10] + 2), 2),
    (dict(Hq=0), 3), (dict(Hq=9), 4), (dict(B=1 << 16, S=1 << 16), 3),
    (dict(scale=0.0), 7), (dict(scale=float("nan")), 7), (dict(scale=float("inf")), 7),
    (dict(ol=(20 * 1024, 1024, 64)), 11), (dict(ql=(20 * 1024, 1024, 4)), 11),
    (dict(ws=A[11] + 8), 12), (dict(n=8), 12),
    (dict(o=A[8] + 256), 9), (dict(lse=A[9]), 9), (dict(o=A[0]), 9), (dict(lse=A[5]), 9), (dict(ws=A[9]), 9), (dict(ws=A[1]), 9),
    (dict(lse=A[3]), 9),
])
def test_attention(fake, kw, status):
    st = read(fake, **kw)
    assert st in status if isinstance(status, tuple) else st == status


def test_attention_workspace(fake):
    f = fake.sdpa_paged_workspace_bytes
    assert f(0, 8, 2, 1, 128) == f(1, 8, 3, 1, 128) == f(1, 8, 2, 0, 128) == f(1, 8, 2, 1, 32) == 0
    assert f(1, 8, 2, 1, 128) > 0


def test_binding_rejects():
    import scaled_dot_product_05_gb300 as lib
    x = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.sdpa_qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        lib.sdpa_qk_norm_rope_bwd(x, x, x, x)
    codes, scale = torch.zeros((3, 16, 2, 64), dtype=torch.uint8), torch.zeros((3, 2))
    with pytest.raises(ValueError):
        lib.PagedCache(codes, codes, scale, scale)


def test_rope_table():
    import scaled_dot_product_05_gb300 as lib
    t = lib.rope_table(70000, 64, base=5e5, device="cpu")
    assert t.shape == (70000, 32, 2) and t.dtype == torch.float32
    a = 69999 * 5e5 ** (-2 * 5 / 64)
    assert abs(t[69999, 5, 0].item() - torch.tensor(a, dtype=torch.float64).cos().item()) < 2.0 ** -24


@pytest.mark.parametrize("kw,status", [(dict(Hq=9), 4), (dict(B=0), 3), (dict(S=0), 3), (dict(scale=-1.0), 7), ({}, 1)])
def test_attention_names_the_fault_that_leaves_no_workspace_size(fake, kw, status):
    """The workspace of sizes that are refused is of 0 bytes, which PyTorch allocates as a null pointer."""
    assert read(fake, ws=None, n=0, **kw) == status


@pytest.mark.parametrize("scale,status", [(2.3e38, OK), (2.4e38, 7), (3.4e38, 7), (1e-45, OK)])
def test_attention_scale_stays_finite_in_base_two(fake, scale, status):
    st = read(fake, scale=scale)
    assert st in status if isinstance(status, tuple) else st == status
