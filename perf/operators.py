"""Measured cases of the cache and rotation operators: the normalisation and
position rotation of queries and keys (forward and backward), the append to a
paged 8-bit key / value cache, and the attention that reads that cache.

A case is a dict of plain sizes.  `prepare` makes what a program has in hand
before the call, `run` is one call, in elementary torch operations or, where
`own` is set, through the library, and `exact` states the definition in 64
bits."""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # queries and keys of one training step: the causal GQA headline shape
        dict(name="norm-rope train 4096", op="norm_rope", B=2, S=4096, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16",
             norm=True, inter=False, fused=False, ctx=8192),
        # one token of 64 requests, each at its own position, read out of the fused projection
        dict(name="norm-rope decode b64", op="norm_rope", B=64, S=1, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16",
             norm=True, inter=False, fused=True, ctx=32768),
        # the gradient of the training step above
        dict(name="norm-rope bwd 4096", op="norm_rope_bwd", B=2, S=4096, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16",
             norm=True, inter=False, fused=False, ctx=8192),
        # a small training batch: 16 heads of 64, odd length, half of each head rotated in adjacent pairs
        dict(name="norm-rope bwd mha 999", op="norm_rope_bwd", B=4, S=999, Hq=16, Hkv=16, D=64, rot=32, dtype="fp16",
             norm=True, inter=True, fused=False, ctx=2048),
        # prompts of four requests, padded to 2000 tokens, two of them continuing an earlier turn
        dict(name="append prompts 2000", op="append", B=4, S=2000, Hkv=8, D=128, page=64, rot=128, dtype="bf16",
             inter=False, ctx=6000),
        # one new token of each of 128 requests
        dict(name="append decode b128", op="append", B=128, S=1, Hkv=8, D=128, page=64, rot=128, dtype="bf16",
             inter=False, ctx=1024),
        # one short request: the smallest call, where latency counts
        dict(name="paged b1 500", op="paged", B=1, S=1, Hq=32, Hkv=8, D=128, page=16, dtype="bf16", ctx=500,
             ragged=False),
        # a served batch: 64 requests of unlike lengths, one token each
        dict(name="paged b64 ragged 8k", op="paged", B=64, S=1, Hq=32, Hkv=8, D=128, page=64, dtype="bf16", ctx=8192,
             ragged=True),
        # the decode workload of the benchmark: 8 sequences of 32768 keys
        dict(name="paged b8 32k", op="paged", B=8, S=1, Hq=32, Hkv=8, D=128, page=64, dtype="bf16", ctx=32768,
             ragged=False),
        # five drafted tokens checked at once, one KV head for 32 query heads, fp16
        dict(name="paged draft mqa", op="paged", B=16, S=5, Hq=32, Hkv=1, D=128, page=32, dtype="fp16", ctx=20001,
             ragged=True),
        # 16 query heads each with its own KV head of 64, one token
        dict(name="paged mha d64", op="paged", B=16, S=1, Hq=16, Hkv=16, D=64, page=128, dtype="bf16", ctx=4097,
             ragged=True),
        # a chunk of two long prompts behind what the cache already holds
        dict(name="paged chunk 512", op="paged", B=2, S=512, Hq=32, Hkv=8, D=128, page=64, dtype="bf16", ctx=8192,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "paged", "paged"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("norm_rope", "norm_rope_bwd"):
        D = rng.choice([32, 64, 128])
        B = _log(rng, 1, 64)
        S = max(1, min(_log(rng, 1, 8192), 2 * 4096 * 40 * 128 // (B * (Hq + Hkv) * D)))
        return dict(op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2]), dtype=dtype,
                    norm=rng.random() < 0.75, inter=rng.random() < 0.3, fused=rng.random() < 0.5,
                    ctx=S + rng.randrange(4096))
    if op == "append":
        B = _log(rng, 1, 128)
        S = 1 if rng.random() < 0.5 else max(1, min(_log(rng, 1, 4096), 4 * 2000 * 8 * 128 // (B * Hkv * D)))
        return dict(op=op, B=B, S=S, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), rot=rng.choice([0, D, D, D // 2]),
                    dtype=dtype, inter=rng.random() < 0.3, ctx=S + rng.randrange(1024))
    B = _log(rng, 1, 64)
    S = rng.choice([1, 1, 1, _log(rng, 1, 16), _log(rng, 1, 300)])
    ctx = S + min(_log(rng, 1, 40000), 8 * 32768 * 8 * 128 // (B * Hkv * D))
    if S * B * ctx * Hq * D > 2 * 512 * 8192 * 32 * 128:
        ctx = S + 2 * 512 * 8192 * 32 * 128 // (S * B * Hq * D)
    return dict(op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), dtype=dtype, ctx=ctx,
                ragged=rng.random() < 0.7)


# -------------------------------------------------------------- the inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _lengths(case, seed):
    """(tokens in the cache before the call, new tokens) of each sequence, on the host."""
    g = torch.Generator()
    g.manual_seed(1000 + int(seed))
    B, S, ctx = case["B"], case["S"], case["ctx"]
    top = max(0, ctx - S)
    if case["op"] == "append":
        start = torch.randint(0, top + 1, (B,), generator=g)
        if S > 1:
            start = torch.where(torch.arange(B) % 2 == 0, torch.zeros_like(start), start)
        count = torch.randint((S + 1) // 2, S + 1, (B,), generator=g)
    else:
        start = torch.full((B,), top, dtype=torch.int64)
        if case["ragged"]:
            start = torch.randint(top // 4, top + 1, (B,), generator=g)
        count = torch.full((B,), S, dtype=torch.int64)
    return start, count


def _table(n_pos, rot):
    """cos and sin of position * 10000^(-2 i / rot), angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float()


def _cache(case, seed, g):
    """A page pool with a page table: twice the pages that the sequences need, handed out in random order."""
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    width = -(-case["ctx"] // page)
    n_pages = B * width + 7
    h = torch.Generator()
    h.manual_seed(2000 + int(seed))
    table = torch.randperm(n_pages, generator=h)[:B * width].reshape(B, width).to(torch.int32).to(DEV)
    out = []
    for part in range(2):
        codes = torch.empty((n_pages, page, Hkv, D), dtype=torch.float8_e4m3fn, device=DEV)
        scale = torch.empty((n_pages, Hkv), dtype=torch.float32, device=DEV)
        step = max(1, (1 << 26) // (page * Hkv * D))
        for p in range(0, n_pages, step):
            x = torch.randn((min(step, n_pages - p), page, Hkv, D), generator=g, device=DEV)
            x *= 0.5 + torch.rand((x.shape[0], 1, Hkv, 1), generator=g, device=DEV)
            s = _pow2_scale(x.abs().amax((1, 3)))
            codes[p:p + step] = (x / s[:, None, :, None]).to(torch.float8_e4m3fn)
            scale[p:p + step] = s
        out += [codes, scale]
    k, ks, v, vs = out
    return k, v, ks, vs, table


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], _TYPES[case["dtype"]]
    B, S, Hkv, D = case["B"], case["S"], case["Hkv"], case["D"]
    st = dict(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if op in ("norm_rope", "norm_rope_bwd"):
        Hq = case["Hq"]
        # the channels of a projection differ in size; the weights of a norm lie around one
        x = normal(B, S, Hq + 2 * Hkv, D) * (0.5 + torch.rand(D, generator=g, device=DEV))
        x = x.to(dt)
        q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
        if not case["fused"]:
            q, k = q.contiguous(), k.contiguous()
        st.update(q=q, k=k, wq=None, wk=None)
        if case["norm"]:
            st.update(wq=1 + 0.2 * normal(D), wk=1 + 0.2 * normal(D))
        st["rope"] = _table(case["ctx"], case["rot"])
        first = torch.randint(0, case["ctx"] - S + 1, (B, 1), generator=g, device=DEV)
        st["pos"] = (first + torch.arange(S, device=DEV)).to(torch.int32)
        if op == "norm_rope_bwd":
            st.update(gq=normal(B, S, Hq, D).to(dt), gk=normal(B, S, Hkv, D).to(dt))
        if own:
            import scaled_dot_product_05_gb300 as lib
            st["lib"] = lib
            if op == "norm_rope_bwd":
                st["ws"] = torch.empty(lib.qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hkv, D), dtype=torch.uint8,
                                       device=DEV)
        return st

    start, count = _lengths(case, seed)
    st["start"], st["count"] = start.to(torch.int32).to(DEV), count.to(torch.int32).to(DEV)
    st["kc"], st["vc"], st["ks"], st["vs"], st["table"] = _cache(case, seed, g)
    if op == "append":
        st["k"], st["v"] = (2 * normal(B, S, Hkv, D)).to(dt), normal(B, S, Hkv, D).to(dt)
        st["rope"] = _table(case["ctx"], case["rot"]) if case["rot"] else None
    else:
        st["q"] = normal(B, S, case["Hq"], D).to(dt)
    if own:
        import scaled_dot_product_05_gb300 as lib
        st["lib"] = lib
        st["cache"] = lib.PagedCache(st["kc"], st["vc"], st["ks"], st["vs"])
        if op == "paged":
            st["ws"] = torch.empty(lib.paged_workspace_bytes(B, case["Hq"], Hkv, S, D), dtype=torch.uint8, device=DEV)
    return st


# --------------------------------------------------------- the plain forms --

def _rotate(x, rope, pos, inter):
    """x [B, S, H, D] with the first 2 * rope.shape[1] channels rotated by the angles of pos [B, S]."""
    half = rope.shape[1]
    c = rope[pos.long()][:, :, None]
    cos, sin = c[..., 0], c[..., 1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([r, rest], -1)


def _norm_rope_plain(x, w, s):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
    return _rotate(y, s["rope"], s["pos"], s["inter"]).to(x.dtype)


def _norm_rope_bwd_plain(x, w, g, s):
    back = torch.stack([s["rope"][..., 0], -s["rope"][..., 1]], -1)      # the inverse rotation
    g = _rotate(g.float(), back, s["pos"], s["inter"])
    if w is None:
        return g.to(x.dtype), None
    y = x.float()
    r = torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
    n = y * r
    dw = (g * n).sum((0, 1, 2), dtype=torch.float64).float()
    g = g * w
    return ((g - n * (g * n).mean(-1, keepdim=True)) * r).to(x.dtype), dw


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (1/2^60 at least)."""
    m, e = torch.frexp((amax / E4M3_MAX).clamp(min=2.0 ** -60))
    e = torch.where(m == 0.5, e - 1, e).clamp(-60, 60)
    return torch.ldexp(torch.ones_like(amax), e)


def _append_plain(x, codes, scale, s):
    B, S, H, D = x.shape
    n_pages, page = codes.shape[:2]
    i = torch.arange(S, device=DEV)
    live = i < s["count"][:, None]
    pos = s["start"][:, None] + i
    slot = (pos % page).long()
    width = s["table"].shape[1]
    pid = s["table"].long().gather(1, (pos // page).clamp(max=width - 1).long())
    row, pid_l, slot_l = x[live], pid[live], slot[live]
    amax = torch.zeros((n_pages, H), device=DEV)
    amax.scatter_reduce_(0, pid_l[:, None].expand(-1, H), row.abs().amax(-1), "amax")
    touched = torch.zeros(n_pages, dtype=torch.bool, device=DEV).index_fill_(0, pid_l, True)
    # the page in which a sequence goes on keeps at least its scale
    lo = s["start"] % page
    first = s["table"].long().gather(1, (s["start"] // page).clamp(max=width - 1).long()[:, None])[:, 0]
    goes_on = first[(lo > 0) & (s["count"] > 0)]
    fresh = _pow2_scale(amax)
    new = fresh.index_copy(0, goes_on, torch.maximum(fresh[goes_on], scale[goes_on]))
    new = torch.where(touched[:, None], new, scale)
    # the earlier tokens of such a page are rounded to the scale that it has now
    f = (scale[goes_on] / new[goes_on])[:, None, :, None]
    earlier = torch.arange(page, device=DEV) < lo[(lo > 0) & (s["count"] > 0)][:, None]
    was = codes[goes_on].float()
    codes[goes_on] = torch.where(earlier[:, :, None, None], was * f, was).to(torch.float8_e4m3fn)
    scale.copy_(new)
    codes[pid_l, slot_l] = (row / new[pid_l][:, :, None]).to(torch.float8_e4m3fn)


def _paged_plain(s):
    q, B, S, Hq, Hkv, D = s["q"], s["B"], s["S"], s["Hq"], s["Hkv"], s["D"]
    page = s["page"]
    width = s["table"].shape[1]
    L = width * page
    t = s["table"].long()

    def gather(codes, scale):
        x = codes[t].float() * scale[t][:, :, None, :, None]             # [B, pages, page, Hkv, D]
        return x.reshape(B, L, Hkv, D).permute(0, 2, 1, 3)               # [B, Hkv, L, D]

    k, v = gather(s["kc"], s["ks"]), gather(s["vc"], s["vs"])
    qf = q.float().reshape(B, S, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, S * (Hq // Hkv), D)
    sc = torch.matmul(qf, k.transpose(2, 3)) * (1 / math.sqrt(D))
    pos = s["start"][:, None] + torch.arange(S, device=DEV)              # a new token's position: it sees keys 0..pos
    seen = torch.arange(L, device=DEV) <= pos[:, :, None]
    seen = seen[:, None, :, None].expand(B, 1, S, Hq // Hkv, L).reshape(B, 1, S * (Hq // Hkv), L)
    sc = sc.masked_fill(~seen, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / l
    lse = (m + l.log())[..., 0]
    G = Hq // Hkv
    o = o.reshape(B, Hkv, S, G, D).permute(0, 2, 1, 3, 4).reshape(B, S, Hq, D).to(q.dtype)
    return o, lse.reshape(B, Hkv, S, G).permute(0, 1, 3, 2).reshape(B, Hq, S)


def run(s):
    op = s["op"]
    if op == "norm_rope":
        if own:
            return s["lib"].sdpa_qk_norm_rope(s["q"], s["k"], norm=s["norm"], q_weight=s["wq"], k_weight=s["wk"],
                                              rope=s["rope"], positions=s["pos"], interleaved=s["inter"])
        return _norm_rope_plain(s["q"], s["wq"], s), _norm_rope_plain(s["k"], s["wk"], s)
    if op == "norm_rope_bwd":
        if own:
            return s["lib"].sdpa_qk_norm_rope_bwd(s["q"], s["k"], s["gq"], s["gk"], norm=s["norm"], q_weight=s["wq"],
                                                  k_weight=s["wk"], rope=s["rope"], positions=s["pos"],
                                                  interleaved=s["inter"], workspace=s["ws"])
        dq, dwq = _norm_rope_bwd_plain(s["q"], s["wq"], s["gq"], s)
        dk, dwk = _norm_rope_bwd_plain(s["k"], s["wk"], s["gk"], s)
        return dq, dk, dwq, dwk
    if op == "append":
        if own:
            s["lib"].sdpa_cache_append(s["k"], s["v"], s["cache"], s["table"], s["start"], s["count"], rope=s["rope"],
                                       interleaved=s["inter"])
        else:
            k = s["k"].float()
            if s["rope"] is not None:
                pos = (s["start"][:, None] + torch.arange(s["S"], device=DEV)).clamp(max=s["ctx"] - 1)
                k = _rotate(k, s["rope"], pos, s["inter"])
            _append_plain(k, s["kc"], s["ks"], s)
            _append_plain(s["v"].float(), s["vc"], s["vs"], s)
        return s["kc"], s["vc"], s["ks"], s["vs"]
    if own:
        lse = torch.empty((s["B"], s["Hq"], s["S"]), dtype=torch.float32, device=DEV)
        o = s["lib"].sdpa_fwd_paged(s["q"], s["cache"], s["table"], s["start"], s["count"], lse=lse,
                                    workspace=s["ws"])
        return o, lse
    return _paged_plain(s)


# ------------------------------------------------- the definition, 64 bits --

def _e4m3(x):
    """The nearest E4M3 value, ties to the even code, |x| <= 448."""
    _, e = torch.frexp(x)
    unit = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / unit) * unit


def _turned(x, table, pos, inter):
    """x [T, H, D] in 64 bits, its rotated channels as complex numbers times cos + i sin."""
    half = table.shape[1]
    z = torch.complex(table[pos, :, 0].double(), table[pos, :, 1].double())[:, None, :]
    r = x[..., :2 * half]
    if inter:
        r = torch.view_as_real(torch.view_as_complex(r.reshape(*r.shape[:-1], half, 2).contiguous()) * z).flatten(-2)
    else:
        t = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * z
        r = torch.cat([t.real, t.imag], -1)
    return torch.cat([r, x[..., 2 * half:]], -1)


def _exact_norm_rope(s):
    outs = []
    for name in ("q", "k"):
        x = s[name].double()
        if s["norm"]:
            x = x / (x.pow(2).sum(-1, keepdim=True) / s["D"] + 1e-6).sqrt() * s["w" + name].double()
        y = _turned(x.flatten(0, 1), s["rope"], s["pos"].long().flatten(), s["inter"])
        outs.append(y.reshape(x.shape))
    return outs[0], outs[1]


def _exact_norm_rope_bwd(s):
    """The gradient by its Jacobian: with x^ = x / rms, d x^_j / d x_i = (delta_ij - x^_i x^_j / D) / rms."""
    grads, weights = [], []
    back = s["rope"] * torch.tensor([1.0, -1.0], device=DEV)
    for name in ("q", "k"):
        x, g = s[name].double(), s["g" + name].double()
        g = _turned(g.flatten(0, 1), back, s["pos"].long().flatten(), s["inter"]).reshape(x.shape)
        if not s["norm"]:
            grads.append(g)
            weights.append(None)
            continue
        rms = (x.pow(2).sum(-1, keepdim=True) / s["D"] + 1e-6).sqrt()
        weights.append(torch.einsum("bshd,bshd->d", g, x / rms))
        u = g * s["w" + name].double()
        along = torch.einsum("bshd,bshd->bsh", u, x)[..., None]
        grads.append(u / rms - x * along / (s["D"] * rms.pow(3)))
    return grads[0], grads[1], weights[0], weights[1]


def _exact_append(s):
    state = {}
    start, count = s["start"].tolist(), s["count"].tolist()
    table = s["table"].tolist()
    page = s["page"]
    for name in ("k", "v"):
        codes, scale = s[name + "c"].double(), s[name + "s"].double()
        for b in range(s["B"]):
            x = s[name][b, :count[b]].double()
            if name == "k" and s["rope"] is not None:
                x = _turned(x, s["rope"], torch.arange(start[b], start[b] + count[b], device=DEV), s["inter"])
            at = start[b]
            while at < start[b] + count[b]:
                end = min((at // page + 1) * page, start[b] + count[b])
                p, rows = table[b][at // page], x[at - start[b]:end - start[b]]
                lo = at % page
                top = rows.abs().amax((0, 2)) / E4M3_MAX
                new = torch.pow(2.0, torch.log2(top).ceil().clamp(-60, 60))
                if lo:
                    new = torch.maximum(new, scale[p])
                    codes[p, :lo] = _e4m3(codes[p, :lo] * (scale[p] / new)[:, None])
                codes[p, lo:lo + end - at] = _e4m3(rows / new[:, None])
                scale[p] = new
                at = end
        state[name] = (codes, scale)
    return state["k"][0], state["v"][0], state["k"][1], state["v"][1]


def _exact_paged(s):
    B, S, Hq, Hkv, D, page = (s[n] for n in ("B", "S", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    o = torch.empty((B, S, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((B, Hq, S), dtype=torch.float64, device=DEV)
    for b, st in enumerate(s["start"].tolist()):
        n = st + S
        p = s["table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            k = (s["kc"][p, :, h].double() * s["ks"][p, h].double()[:, None, None]).reshape(-1, D)[:n]
            v = (s["vc"][p, :, h].double() * s["vs"][p, h].double()[:, None, None]).reshape(-1, D)[:n]
            a = torch.einsum("sgd,ld->gsl", s["q"][b, :, h * G:(h + 1) * G].double(), k) / math.sqrt(D)
            late = torch.ones((S, n), dtype=torch.bool, device=DEV).triu(st + 1)
            a[:, late] = -math.inf
            z = torch.logsumexp(a, -1)
            o[b, :, h * G:(h + 1) * G] = torch.einsum("gsl,ld->sgd", (a - z[..., None]).exp(), v)
            lse[b, h * G:(h + 1) * G] = z
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "norm_rope_bwd": _exact_norm_rope_bwd, "append": _exact_append,
            "paged": _exact_paged}[case["op"]](s)


# --------------------------------------------------------------------- work --

def work(case):
    B, S, Hkv, D = case["B"], case["S"], case["Hkv"], case["D"]
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        n = B * S * (case["Hq"] + Hkv) * D
        back = case["op"] == "norm_rope_bwd"
        # x (and the gradient) read, the result written, 16 bits each; the positions and at most their rows of the table
        rows = min(B * S, case["ctx"])
        passes = 2 if not back else (3 if case["norm"] else 2)
        return {"bytes": 2 * passes * n + 4 * B * S + 4 * rows * case["rot"] + 16 * D, "flops": (18 if back else 9) * n}
    start, count = _lengths(case, 0)
    if case["op"] == "append":
        n = int(count.sum()) * Hkv * D
        pages = sum(-(-(a + c) // case["page"]) - a // case["page"] for a, c in zip(start.tolist(), count.tolist()))
        return {"bytes": 2 * n * (2 + 1) + 8 * pages * Hkv + 8 * B + 4 * pages, "flops": 8 * n}
    Hq = case["Hq"]
    ends = (start + count).tolist()
    keys = sum(ends)
    pages = sum(-(-n // case["page"]) for n in ends)
    seen = sum(sum(range(a + 1, a + S + 1)) for a in start.tolist())
    return {"bytes": 2 * keys * Hkv * D + pages * (4 + 8 * Hkv) + 4 * B * S * Hq * D + 4 * B * S * Hq,
            "flops": 4 * seen * Hq * D}
