"""Norm and rotation of queries and keys (sdpa_qk_norm_rope) and its gradient
against plain formulas in 64 bits.

Tolerances.  The result is computed in fp32 and rounded once: half a step of
the type (bf16 2^-8, fp16 2^-11 relative, fp16 subnormals 2^-25) plus the fp32
arithmetic.  That is at most 16 roundings of 2^-24 relative to the largest
magnitude that enters a value (the norm's factor: the sum of squares 5, the
root 2, two products; the rotation 3; the inputs are exact): 2^-20 of the
row's largest term, doubled for the gradient, whose projection adds two more
sums over the row."""
import math

import pytest
import torch

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


# ------------------------------------------------------ the formulas, 64 bits --

def table64(n_pos, rot, base=10000.0):
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.stack((a.cos(), a.sin()), -1)


def rotate64(x, table, pos, inter, sign=1.0):
    """x [B, S, H, D]; table [n, rot / 2, 2] in 64 bits; pos [B, S]."""
    if table is None:
        return x.clone()
    half = table.shape[1]
    c, s = table[pos][:, :, None, :, 0], sign * table[pos][:, :, None, :, 1]
    y = x.clone()
    ia = torch.arange(half) * 2 if inter else torch.arange(half)
    ib = ia + 1 if inter else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def forward64(x, w, table, pos, inter, norm, eps):
    if norm:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        x = x * w if w is not None else x
    return rotate64(x, table, pos, inter)


def backward64(x, g, w, table, pos, inter, norm, eps):
    """(dx, dw, the largest term of each row of dx, the sum of magnitudes behind dw)."""
    h = rotate64(g, table, pos, inter, -1.0)
    if not norm:
        return h, None, h.abs().amax(-1, keepdim=True), None
    r = 1 / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    n = x * r
    u = h * w if w is not None else h
    along = (u * n).mean(-1, keepdim=True)
    big = r * (u.abs().amax(-1, keepdim=True) + n.abs().amax(-1, keepdim=True) * (u * n).abs().mean(-1, keepdim=True))
    return r * (u - n * along), (h * n).sum((0, 1, 2)), big, (h * n).abs().sum((0, 1, 2))


def test_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(5)
    x = torch.randn((2, 3, 2, 32), generator=g, dtype=torch.float64)
    up = torch.randn(x.shape, generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(32, generator=g, dtype=torch.float64)
    table, pos = table64(50, 16), torch.tensor([[4, 9, 0], [49, 7, 7]])
    for inter in (False, True):
        dx, dw, _, _ = backward64(x, up, w, table, pos, inter, True, 1e-3)
        f = lambda x, w: (up * forward64(x, w, table, pos, inter, True, 1e-3)).sum()   # noqa: E731
        e = 1e-5
        for idx in [(0, 0, 0, 0), (1, 2, 1, 31), (0, 1, 1, 8), (1, 0, 0, 15)]:
            d = torch.zeros_like(x)
            d[idx] = e
            # central differences: third derivatives times e^2 / 6, and 1e-16 / e
            assert abs((f(x + d, w) - f(x - d, w)).item() / (2 * e) - dx[idx].item()) < 1e-7
        for i in (0, 9, 31):
            d = torch.zeros_like(w)
            d[i] = e
            assert abs((f(x, w + d) - f(x, w - d)).item() / (2 * e) - dw[i].item()) < 1e-7


# -------------------------------------------------------------------- inputs --

def make(seed, B, S, Hq, Hkv, D, dt, fused):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, S, Hq + 2 * max(Hkv, 1), D), generator=g).to(DT[dt])
    x[0, 0, 0] *= 2.0 ** -6                      # a row of small values, where eps counts
    x[-1, -1, 0] = 0                             # a row of zeros
    up = torch.randn((B, S, Hq + max(Hkv, 1), D), generator=g).to(DT[dt])
    w = [(1 + 0.3 * torch.randn(D, generator=g)) for _ in range(2)]
    xd, ud = x.to(DEV), up.to(DEV)
    q, k = xd[:, :, :Hq], xd[:, :, Hq:Hq + Hkv]
    gq, gk = ud[:, :, :Hq], ud[:, :, Hq:Hq + Hkv]
    if not fused:
        q, k, gq, gk = (t.contiguous() for t in (q, k, gq, gk))
    return q, k, gq, gk, w


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from scaled_dot_product_05_gb300 import build
    build.build()
    torch.cuda.set_device(0)
    yield
    from scaled_dot_product_05_gb300 import sdpa_device_error
    assert sdpa_device_error() == 0


# B, S, Hq, Hkv, D, rot, dtype, norm, interleaved, fused, weights ("f32", "x", None)
CASES = [
    (2, 5, 4, 2, 128, 128, "bf16", True, False, False, "f32"),
    (1, 1, 1, 1, 128, 128, "bf16", True, False, False, "f32"),
    (3, 7, 6, 3, 128, 64, "bf16", True, False, True, "x"),
    (2, 33, 5, 1, 64, 64, "fp16", True, True, True, "f32"),
    (2, 9, 3, 3, 64, 24, "fp16", True, False, False, "x"),
    (1, 130, 7, 7, 32, 32, "bf16", True, True, False, None),
    (2, 17, 9, 2, 32, 8, "fp16", True, False, True, "f32"),
    (2, 11, 8, 8, 128, 128, "bf16", False, True, False, None),
    (1, 300, 3, 1, 64, 0, "bf16", True, False, True, "f32"),
    (4, 3, 5, 0, 128, 128, "fp16", True, False, False, "f32"),
]
IDS = lambda c: "-".join(map(str, c))      # noqa: E731


def setup(case, seed=11):
    import scaled_dot_product_05_gb300 as lib
    B, S, Hq, Hkv, D, rot, dt, norm, inter, fused, wt = case
    q, k, gq, gk, w = make(seed, B, S, Hq, Hkv, D, dt, fused)
    if wt == "x":
        w = [t.to(DT[dt]) for t in w]
    elif wt is None:
        w = [None, None]
    n_pos = 4 * S + 7
    rope = lib.rope_table(n_pos, rot, device=DEV) if rot else None
    pos = torch.randint(0, n_pos, (B, S), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    pos[0, 0] = n_pos - 1
    kw = dict(norm=norm, q_weight=None if w[0] is None else w[0].to(DEV), rope=rope, positions=pos.to(DEV),
              k_weight=None if w[1] is None or not Hkv else w[1].to(DEV), interleaved=inter, eps=1e-4)
    ref = dict(table=None if rope is None else rope.cpu().double(), pos=pos.long(), inter=inter, norm=norm, eps=1e-4)
    return q, k if Hkv else None, gq, gk if Hkv else None, w, kw, ref


def w64(w):
    return None if w is None else w.double()


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(gpu, case):
    import scaled_dot_product_05_gb300 as lib
    dt = case[6]
    q, k, _, _, w, kw, ref = setup(case)
    outs = lib.sdpa_qk_norm_rope(q, k, **kw)
    torch.cuda.synchronize()
    for x, y, wt in zip((q, k), outs, w):
        if x is None:
            assert y is None
            continue
        r = forward64(x.cpu().double(), w64(wt), **ref)
        tol = HALF[dt] * r.abs() + 2.0 ** -20 * r.abs().amax(-1, keepdim=True) + 2.0 ** -25
        assert y.dtype == DT[dt] and y.is_contiguous()
        assert ((y.cpu().double() - r).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(gpu, case):
    import scaled_dot_product_05_gb300 as lib
    dt = case[6]
    q, k, gq, gk, w, kw, ref = setup(case)
    dq, dk, dwq, dwk = lib.sdpa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    again = lib.sdpa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    torch.cuda.synchronize()
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert a is None and b is None or torch.equal(a, b)
    for x, g, dx, dw, wt in ((q, gq, dq, dwq, w[0]), (k, gk, dk, dwk, w[1])):
        if x is None:
            assert dx is None and dw is None
            continue
        rx, rw, big, mag = backward64(x.cpu().double(), g.cpu().double(), w64(wt), **ref)
        assert ((dx.cpu().double() - rx).abs() <= HALF[dt] * rx.abs() + 2.0 ** -19 * big + 2.0 ** -25).all()
        if rw is None:
            assert dw is None
        else:
            # 16 roundings of a term; a lane adds a few rows in order, then at most 64 groups, 20 blocks and 32 slices
            assert ((dw.cpu().double() - rw).abs() <= 2.0 ** -24 * (16 + 128) * mag + 1e-30).all()


@pytest.mark.gpu
def test_long_weight_gradient(gpu):
    # enough rows that every block walks several items, on both sides
    import scaled_dot_product_05_gb300 as lib
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn((2, 3001, 32, 64), generator=g, device=DEV).to(torch.bfloat16)
    k = torch.randn((2, 3001, 5, 64), generator=g, device=DEV).to(torch.bfloat16)
    gq, gk = torch.randn(q.shape, generator=g, device=DEV).bfloat16(), torch.randn(k.shape, generator=g, device=DEV).bfloat16()
    rope = lib.rope_table(3001, 64, device=DEV)
    _, _, dwq, dwk = lib.sdpa_qk_norm_rope_bwd(q, k, gq, gk, rope=rope)
    pos = torch.arange(3001).expand(2, -1)
    for x, up, dw in ((q, gq, dwq), (k, gk, dwk)):
        _, rw, _, mag = backward64(x.cpu().double(), up.cpu().double(), None, rope.cpu().double(), pos, False, True, 1e-6)
        # 16 roundings of a term; in order: 192064 rows over 400 blocks of 32 groups at least, 16 of a lane; then
        # 32 groups, 20 blocks, 32 slices: < 150 additions behind a term
        assert ((dw.cpu().double() - rw).abs() <= 2.0 ** -24 * 166 * mag).all()


@pytest.mark.gpu
def test_writes_only_its_rows_and_strided_outputs(gpu):
    import scaled_dot_product_05_gb300 as lib
    case = (2, 6, 4, 2, 64, 64, "bf16", True, False, True, "f32")
    q, k, gq, gk, _, kw, _ = setup(case)
    plain = lib.sdpa_qk_norm_rope(q, k, **kw)
    buf = torch.full((2, 6, 4 + 2 * 2, 64), 7.0, dtype=q.dtype, device=DEV)
    lib.sdpa_qk_norm_rope(q, k, buf[:, :, :4], buf[:, :, 4:6], **kw)
    torch.cuda.synchronize()
    assert torch.equal(buf[:, :, :4], plain[0]) and torch.equal(buf[:, :, 4:6], plain[1]) and (buf[:, :, 6:] == 7).all()
    # the gradient into the rows of one buffer
    ref = lib.sdpa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    buf.fill_(7.0)
    lib.sdpa_qk_norm_rope_bwd(q, k, gq, gk, buf[:, :, :4], buf[:, :, 4:6], **kw)
    torch.cuda.synchronize()
    assert torch.equal(buf[:, :, :4], ref[0]) and torch.equal(buf[:, :, 4:6], ref[1]) and (buf[:, :, 6:] == 7).all()


@pytest.mark.gpu
def test_in_place(gpu):
    import scaled_dot_product_05_gb300 as lib
    case = (2, 6, 4, 2, 128, 128, "bf16", True, False, True, "f32")
    q, k, _, _, _, kw, _ = setup(case)
    ref = lib.sdpa_qk_norm_rope(q, k, **kw)
    lib.sdpa_qk_norm_rope(q, k, q, k, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])


@pytest.mark.gpu
def test_default_positions_and_bhsd(gpu):
    import scaled_dot_product_05_gb300 as lib
    q = torch.randn((2, 9, 3, 64), device=DEV).half()
    rope = lib.rope_table(9, 64, device=DEV)
    pos = torch.arange(9, dtype=torch.int32, device=DEV).expand(2, -1).contiguous()
    a, _ = lib.sdpa_qk_norm_rope(q, rope=rope)
    b, _ = lib.sdpa_qk_norm_rope(q, rope=rope, positions=pos)
    qt = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    ot = torch.empty((2, 3, 9, 64), dtype=q.dtype, device=DEV).permute(0, 2, 1, 3)
    c, _ = lib.sdpa_qk_norm_rope(qt, q_out=ot, rope=rope)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.gpu
def test_position_outside_the_table(gpu):
    # the kernel checks each position before it forms an address: nothing is written for such a row
    import scaled_dot_product_05_gb300 as lib
    q = torch.randn((1, 4, 2, 64), device=DEV).bfloat16()
    rope = lib.rope_table(10, 64, device=DEV)
    pos = torch.tensor([[3, 10, -1, 9]], dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 7.0)
    lib.sdpa_qk_norm_rope(q, q_out=out, rope=rope, positions=pos)
    assert lib.sdpa_device_error() == 0x701
    assert (out[:, 1:3] == 7).all() and not (out[:, 0] == 7).all() and not (out[:, 3] == 7).all()
    g = torch.randn_like(q)
    dq = torch.full_like(q, 7.0)
    _, _, dw, _ = lib.sdpa_qk_norm_rope_bwd(q, None, g, None, dq, rope=rope, positions=pos)
    assert lib.sdpa_device_error() == 0x701
    good = [0, 3]
    ref = lib.sdpa_qk_norm_rope_bwd(q[:, good].contiguous(), None, g[:, good].contiguous(), None, rope=rope,
                                    positions=pos[:, good].contiguous())
    assert (dq[:, 1:3] == 7).all() and torch.equal(dq[:, good], ref[0])
    assert torch.allclose(dw, ref[2], rtol=1e-5, atol=1e-6) and lib.sdpa_device_error() == 0


@pytest.mark.gpu
def test_nan_stays_in_its_row(gpu):
    import scaled_dot_product_05_gb300 as lib
    q = torch.randn((1, 5, 2, 128), device=DEV).bfloat16()
    rope = lib.rope_table(5, 128, device=DEV)
    a, _ = lib.sdpa_qk_norm_rope(q, rope=rope)
    q2 = q.clone()
    q2[0, 2, 1, 5] = float("nan")
    q2[0, 4, 0, 0] = float("inf")
    b, _ = lib.sdpa_qk_norm_rope(q2, rope=rope)
    torch.cuda.synchronize()
    hit = torch.zeros((5, 2), dtype=torch.bool, device=DEV)
    hit[2, 1] = hit[4, 0] = True
    assert torch.equal(a[0][~hit], b[0][~hit]) and b[0][2, 1].isnan().all()


@pytest.mark.gpu
def test_other_stream_and_graph(gpu):
    import scaled_dot_product_05_gb300 as lib
    case = (2, 40, 4, 2, 128, 128, "bf16", True, False, False, "f32")
    q, k, gq, gk, _, kw, _ = setup(case)
    ref = lib.sdpa_qk_norm_rope(q, k, **kw) + lib.sdpa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ws = torch.empty(lib.qk_norm_rope_bwd_workspace_bytes(2, 40, 4, 2, 128), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(t) for t in ref]
    torch.cuda.synchronize()

    def both(**extra):
        lib.sdpa_qk_norm_rope(q, k, outs[0], outs[1], **kw, **extra)
        lib.sdpa_qk_norm_rope_bwd(q, k, gq, gk, outs[2], outs[3], dq_weight=outs[4], dk_weight=outs[5], workspace=ws,
                                  **kw, **extra)
    both(stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for o in outs:
        o.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, outs))


@pytest.mark.gpu
def test_training_step_against_autograd(gpu):
    """Norm and rotation, attention, attention's gradient, the gradient of the norm and rotation: gradients of the
    projections' outputs against autograd in 64 bits.  Errors of the bf16 chain: q, k, o, dq and dk are each rounded
    once (half a step, 2^-8 at most, 2^-9 in the mean at most), and the attention's own gradients are tested to 4 units of 2^-9 relative RMS:
    4 + 5 units."""
    import scaled_dot_product_05_gb300 as lib
    B, S, Hq, Hkv, D = 2, 150, 4, 2, 64
    q, k, _, _, w = make(21, B, S, Hq, Hkv, D, "bf16", True)
    g = torch.Generator(device=DEV).manual_seed(4)
    v = torch.randn((B, S, Hkv, D), generator=g, device=DEV).bfloat16()
    up = torch.randn((B, S, Hq, D), generator=g, device=DEV).bfloat16()
    rope = lib.rope_table(S, D, device=DEV)
    kw = dict(q_weight=w[0].to(DEV), k_weight=w[1].to(DEV), rope=rope, eps=1e-4)
    qr, kr = lib.sdpa_qk_norm_rope(q, k, **kw)
    o, lse = torch.empty_like(qr), torch.empty((B, Hq, S), device=DEV)
    lib.sdpa_fwd_ex(qr, kr, v, o, lse, causal=True)
    dqr, dkr, dv = lib.sdpa_bwd(qr, kr, v, o, up, lse, causal=True)
    got = lib.sdpa_qk_norm_rope_bwd(q, k, dqr, dkr, **kw)
    leaves = [t.detach().cpu().double().requires_grad_() for t in (q, k, w[0], w[1])]
    pos = torch.arange(S).expand(B, -1)
    a = forward64(leaves[0], leaves[2], rope.cpu().double(), pos, False, True, 1e-4)
    b = forward64(leaves[1], leaves[3], rope.cpu().double(), pos, False, True, 1e-4).repeat_interleave(Hq // Hkv, 2)
    sc = torch.einsum("bihd,bjhd->bhij", a, b) / math.sqrt(D)
    sc = sc.masked_fill(torch.ones(S, S, dtype=torch.bool).triu(1), -math.inf)
    ref = torch.einsum("bhij,bjhd->bihd", sc.softmax(-1), v.cpu().double().repeat_interleave(Hq // Hkv, 2))
    ref.backward(up.cpu().double())
    for t, x in zip(got, leaves):
        err = (t.cpu().double() - x.grad).norm() / x.grad.norm()
        assert err <= 9 * 2.0 ** -9
