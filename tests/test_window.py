"""Attention with a sliding window and first keys that stay visible, and its
gradient, against the definition in 64 bits.

Tolerances, element by element.  u is half a step of the 16-bit type
(finfo.eps / 2).  The weights p are rounded to it before they meet V, and O
once more: |O - ref| <= u sum_j p_j |v_j| + u |ref|.  What is computed in 32
bits (scores, exponentials, sums over at most 2048 keys) is within 2^-13 of the
same sums: a score of magnitude 30 at most is off by 30 * 2^-20, an exponential
by 2^-22, sums of products by 2048 * 2^-24.  The gradients count alike: dV
rounds p and itself, dQ and dK round ds = p (dp - delta) and themselves.  The
LSE is within 2^-13 absolutely.  Differences: the second-order term of the
central difference with step h is h^2 / 6 times the third derivative, below
1e-4 of the gradient's norm at h = 1e-3; the 16-bit gradients are off by 2 u of
their terms.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
F32 = 2.0 ** -13


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from scaled_dot_product_05_gb300 import build
    build.build()
    torch.cuda.set_device(0)
    yield
    from scaled_dot_product_05_gb300 import sdpa_device_error
    assert sdpa_device_error() == 0


def lib():
    import scaled_dot_product_05_gb300 as m
    return m


def seen(Sq, Skv, window, sinks):
    i = torch.arange(Sq, device=DEV)[:, None]
    j = torch.arange(Skv, device=DEV)
    return (j <= i) & ((i - j < window) | (j < sinks))


def inputs(B, Sq, Skv, Hq, Hkv, D, dtype, seed=0, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = TYPES[dtype]
    q = (scale * torch.randn(B, Sq, Hq, D, generator=g, device=DEV)).to(dt)
    k = torch.randn(B, Skv, Hkv, D, generator=g, device=DEV).to(dt)
    v = torch.randn(B, Skv, Hkv, D, generator=g, device=DEV).to(dt)
    return q, k, v


def heads(x, G=1):
    """[B, S, H, D] as [B, H * G, S, D] in 64 bits, each head G times."""
    return x.double().transpose(1, 2).repeat_interleave(G, 1)


def reference(q, k, v, window, sinks):
    """(O, LSE, sum p |v|) by the definition; a row without keys is 0 and -inf."""
    G = q.shape[2] // k.shape[2]
    m = seen(q.shape[1], k.shape[1], window, sinks)
    s = heads(q) @ heads(k, G).transpose(2, 3) / math.sqrt(q.shape[3])
    s = s.masked_fill(~m, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(m, (s - lse[..., None]).exp(), torch.zeros_like(s))
    return (p @ heads(v, G)).transpose(1, 2), lse, (p @ heads(v, G).abs()).transpose(1, 2)


def check_forward(o, lse, q, k, v, window, sinks):
    ref, z, mass = reference(q, k, v, window, sinks)
    u = torch.finfo(q.dtype).eps / 2
    assert ((o.double() - ref).abs() <= u * mass + u * ref.abs() + F32 * mass + 1e-30).all()
    empty = z == -math.inf
    assert (lse.double()[empty] == -math.inf).all()
    assert ((lse.double() - z)[~empty].abs() <= F32).all()


CASES = [
    # B, Sq, Skv, Hq, Hkv, D, window, sinks
    (1, 1, 1, 1, 1, 64, 1, 0),
    (1, 5, 5, 2, 1, 32, 2, 1),
    (2, 128, 128, 2, 2, 64, 128, 0),           # the causal mask of one tile
    (1, 129, 129, 3, 1, 128, 1, 0),            # each row sees itself alone
    (1, 300, 300, 4, 2, 128, 77, 3),
    (2, 511, 511, 4, 4, 64, 200, 130),         # first keys over two tiles
    (1, 1000, 1000, 2, 1, 128, 129, 0),        # the lower edge moves through every tile
    (1, 1000, 1000, 2, 1, 128, 128, 4),
    (1, 1000, 1000, 2, 2, 32, 127, 1),
    (1, 900, 900, 8, 1, 64, 5000, 7),          # a window wider than the rows: the causal mask
    (1, 700, 300, 2, 2, 64, 50, 0),            # rows 350 .. see no key
    (1, 700, 300, 2, 2, 128, 50, 2),           # and here two
    (1, 300, 700, 2, 2, 128, 64, 1),           # keys 300 .. are seen by none
    (1, 1500, 1500, 2, 1, 128, 300, 1400),     # nearly everything stays
    (40, 256, 256, 16, 16, 64, 100, 1),        # many small units: two Q tiles a CTA at D = 64
    (1, 2048, 2048, 2, 2, 128, 2 ** 31 - 1, 2 ** 31 - 1),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, dtype):
    B, Sq, Skv, Hq, Hkv, D, window, sinks = case
    q, k, v = inputs(B, Sq, Skv, Hq, Hkv, D, dtype)
    lse = torch.full((B, Hq, Sq), math.nan, device=DEV)
    o = lib().sdpa_fwd_window(q, k, v, lse=lse, window=window, sinks=sinks)
    check_forward(o, lse, q, k, v, window, sinks)


def test_forward_large_scores_in_late_tiles():
    """Maxima that grow from tile to tile, and rows whose first tile is wholly masked."""
    q, k, v = inputs(1, 900, 900, 2, 1, 128, "bf16", scale=1.0)
    k = (k.float() * torch.linspace(0.1, 2.5, 900, device=DEV)[None, :, None, None]).to(k.dtype)
    for window, sinks in ((129, 0), (300, 2), (40, 0)):
        lse = torch.empty((1, 2, 900), device=DEV)
        o = lib().sdpa_fwd_window(q, k, v, lse=lse, window=window, sinks=sinks)
        check_forward(o, lse, q, k, v, window, sinks)


def test_forward_infinite_masked_keys():
    """Infinite scores of keys that a row does not see do not reach it."""
    q, k, v = inputs(1, 400, 400, 2, 2, 64, "bf16")
    q = q.abs()                                 # (so that no score of the infinite key is NaN)
    k[0, 60] = math.inf
    o = lib().sdpa_fwd_window(q, k, v, window=100)
    rows = torch.ones(400, dtype=torch.bool, device=DEV)
    rows[60:160] = False
    ref, _, mass = reference(q, torch.nan_to_num(k, posinf=0.0), v, 100, 0)
    u = torch.finfo(q.dtype).eps / 2
    assert ((o.double() - ref).abs() <= u * mass + u * ref.abs() + F32 * mass)[:, rows].all()


def test_forward_equals_causal():
    """A window that covers everything: the causal pass, bit for bit."""
    q, k, v = inputs(2, 777, 777, 4, 2, 128, "bf16")
    lse, lse2 = torch.empty((2, 4, 777), device=DEV), torch.empty((2, 4, 777), device=DEV)
    o2 = torch.empty_like(q)
    lib().sdpa_fwd_ex(q, k, v, o2, lse2, causal=True)
    o = lib().sdpa_fwd_window(q, k, v, lse=lse, window=777, sinks=0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_forward_layouts():
    """Heads in front, a padded buffer around O: nothing beside O is written."""
    B, S, Hq, Hkv, D = 2, 333, 4, 2, 64
    q, k, v = inputs(B, S, S, Hq, Hkv, D, "fp16")
    qt, kt, vt = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v))
    buf = torch.full((B, S + 3, Hq + 1, D), 7.0, dtype=q.dtype, device=DEV)
    o = buf[:, :S, :Hq]
    lse = torch.empty((B, Hq, S), device=DEV)
    lib().sdpa_fwd_window(qt, kt, vt, o, lse, window=100, sinks=2)
    check_forward(o, lse, q, k, v, 100, 2)
    assert (buf[:, S:] == 7).all() and (buf[:, :, Hq:] == 7).all()


def backward_reference(q, k, v, o, do, lse, window, sinks):
    """Gradients by the formulas in 64 bits, and for each the sum of its terms' magnitudes."""
    G = q.shape[2] // k.shape[2]
    Hkv, scale = k.shape[2], 1 / math.sqrt(q.shape[3])
    m = seen(q.shape[1], k.shape[1], window, sinks)
    Q, K, V, O, dO = heads(q), heads(k, G), heads(v, G), heads(o), heads(do)
    p = (Q @ K.transpose(2, 3) * scale - lse.double()[..., None]).exp()
    p = torch.where(m, p, torch.zeros_like(p))
    dp, delta = dO @ V.transpose(2, 3), (dO * O).sum(-1, keepdim=True)
    ds = p * (dp - delta) * scale
    wide = p * (dO.abs() @ V.abs().transpose(2, 3) + (dO * O).abs().sum(-1, keepdim=True)) * scale

    def fold(x):                                # the heads of a group share their key head
        return x.unflatten(1, (Hkv, G)).sum(2).transpose(1, 2)
    T = lambda x: x.transpose(2, 3)
    return ((ds @ K).transpose(1, 2), fold(T(ds) @ Q), fold(T(p) @ dO),
            (ds.abs() @ K.abs()).transpose(1, 2), fold(T(ds.abs()) @ Q.abs()), fold(T(p) @ dO.abs()),
            (wide @ K.abs()).transpose(1, 2), fold(T(wide) @ Q.abs()))


def check_backward(grads, ref, u):
    dq, dk, dv, aq, ak, av, wq, wk = ref
    for got, want, terms, wide in zip(grads, (dq, dk, dv), (aq, ak, av), (wq, wk, av)):
        assert torch.isfinite(got).all()
        assert ((got.double() - want).abs() <= u * terms + u * want.abs() + F32 * wide + 1e-6).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", [c for c in CASES if c[5] != 32 and c[0] < 40], ids=str)
def test_backward(case, dtype):
    B, Sq, Skv, Hq, Hkv, D, window, sinks = case
    q, k, v = inputs(B, Sq, Skv, Hq, Hkv, D, dtype, seed=1)
    do = inputs(B, Sq, Skv, Hq, Hkv, D, dtype, seed=2)[0]
    lse = torch.empty((B, Hq, Sq), device=DEV)
    o = lib().sdpa_fwd_window(q, k, v, lse=lse, window=window, sinks=sinks)
    grads = lib().sdpa_bwd_window(q, k, v, o, do, lse, window=window, sinks=sinks)
    check_backward(grads, backward_reference(q, k, v, o, do, lse, window, sinks), torch.finfo(q.dtype).eps / 2)


def test_backward_against_differences():
    """The directional derivative of sum(dO * O), O by the definition in 64 bits."""
    window, sinks = 40, 2
    q, k, v = inputs(1, 200, 200, 4, 2, 64, "fp16", seed=3)
    do = inputs(1, 200, 200, 4, 2, 64, "fp16", seed=4)[0]
    lse = torch.empty((1, 4, 200), device=DEV)
    o = lib().sdpa_fwd_window(q, k, v, lse=lse, window=window, sinks=sinks)
    grads = lib().sdpa_bwd_window(q, k, v, o, do, lse, window=window, sinks=sinks)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    u = torch.finfo(torch.float16).eps / 2
    for which, grad in enumerate(grads):
        step = torch.randn(grad.shape, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-3

        def at(e):
            x = [t.double() for t in (q, k, v)]
            x[which] = x[which] + e * step
            return (reference(*x, window, sinks)[0] * do.double()).sum()
        slope = (at(h) - at(-h)) / (2 * h)
        got = (grad.double() * step).sum()
        # grad's elements are off by a few u of their terms, in random directions under a random step
        assert abs(slope - got) <= 8 * u * grad.double().norm() + 1e-4 * grad.double().norm()


def test_graph_replays_and_streams():
    q, k, v = inputs(1, 600, 600, 4, 2, 128, "bf16")
    do = inputs(1, 600, 600, 4, 2, 128, "bf16", seed=9)[0]
    m = lib()
    lse, o = torch.empty((1, 4, 600), device=DEV), torch.empty_like(q)
    m.sdpa_fwd_window(q, k, v, o, lse, window=200, sinks=4)
    ws = torch.empty(m.bwd_workspace_bytes(1, 4, 600, 128), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        m.sdpa_fwd_window(q, k, v, o2, lse2, window=200, sinks=4)
        m.sdpa_bwd_window(q, k, v, o2, do, lse2, *grads, window=200, sinks=4, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_backward(grads, backward_reference(q, k, v, o, do, lse, 200, 4), torch.finfo(q.dtype).eps / 2)


def test_refusals():
    m = lib()
    q, k, v = inputs(1, 64, 64, 2, 2, 64, "bf16")
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(m.SdpaError):
            m.sdpa_fwd_window(q, k, v, window=window, sinks=sinks)
    with pytest.raises(m.SdpaError):
        m.sdpa_fwd_window(q.float(), k.float(), v.float(), window=4)
    with pytest.raises(ValueError):
        m.sdpa_fwd_window(q, k[..., :32], v, window=4)
    with pytest.raises(ValueError):
        m.sdpa_bwd_window(q, k, v, q.clone(), q.clone(), None, window=4)
