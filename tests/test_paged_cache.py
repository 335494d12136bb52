"""The paged 8-bit cache: sdpa_cache_append and sdpa_fwd_paged against plain
implementations in 64 bits, alone and as a serving loop.

Tolerances.  Append: E4M3 rounds to half a step, 2^-4 relative (2^-10 scales
for subnormal codes), of a key rotated in fp32 (three roundings of 2^-24);
values, and keys that are not rotated, have to match bit for bit.  Attention:
scores are sums of D exact products in fp32 (each addition rounds by 2^-24 of
the magnitude that has been summed: D 2^-24 sum |q k| at most, taken as
2^-17 for D = 128); a weight may be off by 2^-8 of itself (two E4M3 parts of
half a step 2^-4 each) and, where it is small, by 2^-13 / 112 of its row's largest
(the smaller part's subnormal step); the output rounds once."""
import math

import pytest
import torch

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


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


# ------------------------------------------------------- plain definitions --

def e4m3(x):
    """Nearest E4M3 value of a 64-bit tensor (saturating, NaN kept)."""
    return x.clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn).double()


def pow2_scale(amax):
    if amax == 0:
        return 2.0 ** -60
    m, e = math.frexp(amax / 448)
    return 2.0 ** max(-60, min(60, e - 1 if m == 0.5 else e))


def rotate64(x, table, pos, inter):
    """x [n, H, D] rotated by the 64-bit table rows of pos [n]."""
    half = table.shape[1]
    c, s = table[pos][:, None, :, 0], table[pos][:, None, :, 1]
    y = x.clone()
    ia = torch.arange(half) * 2 if inter else torch.arange(half)
    ib = ia + 1 if inter else ia + half
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y


class PlainCache:
    """The cache as values: codes and scales in 64 bits on the host."""

    def __init__(self, cache):
        self.page = cache.page_size
        self.codes = [t.cpu().double() for t in (cache.k.view(torch.float8_e4m3fn), cache.v.view(torch.float8_e4m3fn))]
        self.scale = [t.cpu().double() for t in (cache.k_scale, cache.v_scale)]

    def append(self, which, x, table, start, count):
        """x [B, S, H, D] in 64 bits, rotated already."""
        for b in range(x.shape[0]):
            at, end = start[b], start[b] + count[b]
            while at < end:
                stop = min((at // self.page + 1) * self.page, end)
                p, lo = table[b][at // self.page], at % self.page
                for h in range(x.shape[2]):
                    rows = x[b, at - start[b]:stop - start[b], h]
                    fin = rows.abs()[rows.isfinite()]
                    new = pow2_scale(fin.max().item() if fin.numel() else 0.0)
                    if lo:
                        old = self.scale[which][p, h].item()
                        new = max(old, new)
                        self.codes[which][p, :lo, h] = e4m3(self.codes[which][p, :lo, h] * (old / new))
                    self.codes[which][p, lo:lo + stop - at, h] = e4m3(rows / new)
                    self.scale[which][p, h] = new
                at = stop

    def rows(self, which, pages, n):
        x = self.codes[which][pages] * self.scale[which][pages][:, None, :, None]
        return x.reshape(-1, *x.shape[2:])[:n]


def attention64(q, k, v, first, causal, total, scale):
    """q [S, Hq, D] at positions first .., k and v [n, Hkv, D]: (O, LSE, sum p |v|, score magnitude, the largest
    weight times sum |v|)."""
    S, Hq, D = q.shape
    G = Hq // k.shape[1]
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("shd,nhd->hsn", q, kk) * scale
    mag = torch.einsum("shd,nhd->hsn", q.abs(), kk.abs()) * scale
    pos = torch.arange(k.shape[0])
    last = first + torch.arange(S) if causal else torch.full((S,), total - 1)
    hide = pos[None] > last[:, None]
    s = s.masked_fill(hide, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(hide, 0.0, (s - torch.where(lse.isinf(), 0.0, lse)[..., None]).exp())
    o = torch.einsum("hsn,nhd->shd", p, vv)
    spread = torch.einsum("hsn,nhd->shd", p, vv.abs())
    floor = p.amax(-1).T[..., None] * torch.einsum("hsn,nhd->shd", (~hide).double().expand_as(p), vv.abs())
    return o, lse, spread, mag.masked_fill(hide, 0).amax(-1), floor


def make_cache(n_pages, page, H, D, layout, seed=1, filled=True):
    import scaled_dot_product_05_gb300 as lib
    g = torch.Generator().manual_seed(seed)
    if layout == "heads":
        c = lib.PagedCache.empty(n_pages, page, H, D, device=DEV)
    elif layout == "tokens":
        t = [torch.zeros((n_pages, page, H, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
        c = lib.PagedCache(*t, *(torch.ones((n_pages, H), device=DEV) for _ in range(2)))
    else:                                           # K and V of a slot side by side in one buffer
        t = torch.zeros((n_pages, page, H, 2, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        c = lib.PagedCache(t[:, :, :, 0], t[:, :, :, 1], *(torch.ones((n_pages, H), device=DEV) for _ in range(2)))
    if filled:
        for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
            x = torch.randn((n_pages, page, H, D), generator=g) * (0.5 + torch.rand((n_pages, 1, H, 1), generator=g))
            s = 2.0 ** torch.ceil(torch.log2(x.abs().amax((1, 3)) / 448))
            codes.view(torch.uint8).copy_((x / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV))
            scale.copy_(s)
    return c


def tables(n_pages, B, width, seed):
    p = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))[:B * width]
    return p.reshape(B, width).to(torch.int32)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# -------------------------------------------------------------------- append --

# page, Hkv, D, S, rot, interleaved, dtype, layout, starts, counts
APPENDS = [
    (16, 2, 128, 1, 128, False, "bf16", "heads", [0, 5, 15, 16, 47], None),
    (64, 3, 64, 1, 64, True, "fp16", "tokens", [0, 63, 64, 127, 1], [1, 1, 0, 1, 1]),
    (128, 1, 128, 1, 0, False, "bf16", "pairs", [0, 100, 127, 128, 300], None),
    (32, 2, 128, 7, 64, False, "fp16", "heads", [0, 30, 31, 60, 3], [7, 7, 1, 5, 0]),
    (16, 1, 64, 40, 64, False, "bf16", "tokens", [0, 9, 15, 16, 31], [40, 39, 17, 16, 1]),
    (128, 2, 128, 300, 128, True, "bf16", "heads", [0, 1, 127, 200, 64], [300, 255, 129, 300, 64]),
    (64, 2, 64, 131, 24, False, "fp16", "pairs", [0, 60, 1, 64, 33], [131, 4, 130, 64, 31]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(map(str, c[:8])))
def test_append(gpu, case):
    import scaled_dot_product_05_gb300 as lib
    page, H, D, S, rot, inter, dt, layout, start, count = case
    B, width = len(start), (max(start) + S) // page + 1
    cache = make_cache(B * width + 3, page, H, D, layout)
    plain = PlainCache(cache)
    table = tables(B * width + 3, B, width, 4)
    g = torch.Generator().manual_seed(6)
    k = (3 * torch.randn((B, S, H, D), generator=g)).to(DT[dt])
    v = torch.randn((B, S, H, D), generator=g).to(DT[dt])
    v[0] = 0                                        # a page of zeros
    k[1, 0] *= 40                                   # a scale that grows
    rope = lib.rope_table(max(start) + S, rot, device=DEV) if rot else None
    lib.sdpa_cache_append(k.to(DEV), v.to(DEV), cache, table.to(DEV), i32(start), None if count is None else i32(count),
                          rope=rope, interleaved=inter)
    assert lib.sdpa_device_error() == 0
    n = [S] * B if count is None else count
    kr = k.double()
    if rot:
        for b in range(B):
            kr[b] = rotate64(kr[b], rope.cpu().double(), torch.arange(start[b], start[b] + S), inter)
    plain.append(0, kr, table.tolist(), start, n)
    plain.append(1, v.double(), table.tolist(), start, n)
    got = PlainCache(cache)
    assert torch.equal(got.scale[0], plain.scale[0]) and torch.equal(got.scale[1], plain.scale[1])
    assert torch.equal(got.codes[1], plain.codes[1])
    if not rot:
        assert torch.equal(got.codes[0], plain.codes[0])
        return
    # a key next to the border between two codes may go to either: one step apart, and few of them
    a, b = got.codes[0], plain.codes[0]
    assert ((a - b).abs() <= 2.0 ** -3 * torch.maximum(a.abs(), b.abs()) + 2.0 ** -9).all()
    assert (a != b).double().mean() <= 1e-3


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_rotated_keys_get_the_codes_of_the_exact_product(gpu, inter):
    """A rotation in fp32 is off by an ulp or so, which would send some of a few million keys to the code on the other
    side of a border: codes have to be those of the exact product, wherever it is not the rest of terms more than
    eight times as large, and not subnormal."""
    import scaled_dot_product_05_gb300 as lib
    page, H, D, S = 128, 16, 128, 4000
    cache = make_cache(S // page + 1, page, H, D, "heads", filled=False)
    k = torch.randn((1, S, H, D), generator=torch.Generator().manual_seed(11)).bfloat16()
    rope = lib.rope_table(S, D, device=DEV)
    table = torch.arange(S // page + 1, dtype=torch.int32, device=DEV)[None]
    lib.sdpa_cache_append(k.to(DEV), k.to(DEV), cache, table, i32([0]), rope=rope, interleaved=inter)
    x = rotate64(k[0].double(), rope.cpu().double(), torch.arange(S), inter)
    # the sum of the magnitudes of the two terms
    terms = rotate64(k[0].double().abs(), torch.stack((rope[..., 0].abs(), -rope[..., 1].abs()), -1).cpu().double(),
                     torch.arange(S), inter)
    if inter:
        other = rotate64(k[0].double().abs(), rope.abs().cpu().double(), torch.arange(S), inter)
        terms[..., 1::2] = other[..., 1::2]
    else:
        other = rotate64(k[0].double().abs(), rope.abs().cpu().double(), torch.arange(S), inter)
        terms[..., D // 2:] = other[..., D // 2:]
    got = PlainCache(cache)
    pages = table[0].cpu().long()
    codes = got.codes[0][pages].reshape(-1, H, D)[:S]
    scale = got.scale[0][pages].repeat_interleave(page, 0)[:S, :, None]
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)      # (to 32 bits first would round twice)
    want = torch.round(y / step) * step
    sure = (x.abs() * 8 >= terms) & (y.abs() >= 2.0 ** -6)
    assert sure.double().mean() > 0.7
    assert torch.equal(codes[sure], want[sure])


@pytest.mark.gpu
def test_append_special_values(gpu):
    import scaled_dot_product_05_gb300 as lib
    cache = make_cache(4, 16, 1, 64, "heads", filled=False)
    x = torch.randn((1, 3, 1, 64), generator=torch.Generator().manual_seed(1)).bfloat16()
    x[0, 0, 0, 0], x[0, 1, 0, 1], x[0, 2, 0, 2] = float("inf"), -float("inf"), float("nan")
    table = i32([[2, 0]])
    lib.sdpa_cache_append(x.to(DEV), x.to(DEV), cache, table, i32([0]))
    s = pow2_scale(x[x.isfinite()].abs().max().item())
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert scale[2, 0].item() == s
        c = codes[2, :3, 0].cpu().float()
        assert c[0, 0] == 448 and c[1, 1] == -448 and c[2, 2].isnan()
        ok = x[0, :, 0].isfinite()
        assert torch.equal(c[ok].double(), e4m3(x[0, :, 0][ok].double() / s))
        raw = codes.view(torch.uint8)
        assert (raw[2, 3:] == 0).all() and (raw[[0, 1, 3]] == 0).all()
    # the largest finite values and the smallest: the scale stays in [2^-60, 2^60]
    for big, want in ((3e38, 2.0 ** 60), (2.0 ** -70, 2.0 ** -60)):
        y = torch.full((1, 1, 1, 64), big, device=DEV).bfloat16()
        lib.sdpa_cache_append(y, y, cache, table, i32([0]))
        assert cache.k_scale[2, 0].item() == want


@pytest.mark.gpu
def test_append_goes_on_under_a_scale_that_is_no_power_of_two(gpu):
    import scaled_dot_product_05_gb300 as lib
    cache = make_cache(2, 32, 2, 64, "heads")
    cache.k_scale.fill_(0.3)
    cache.v_scale.fill_(1e-3)
    plain = PlainCache(cache)
    x = torch.randn((1, 4, 2, 64), generator=torch.Generator().manual_seed(1)).half()
    lib.sdpa_cache_append(x.to(DEV), x.to(DEV), cache, i32([[1]]), i32([9]))
    for which in (0, 1):
        # the quotient of two fp32 numbers, rounded to fp32 and then to E4M3, as the kernel forms it
        old = torch.tensor([0.3, 1e-3][which])
        got = PlainCache(cache)
        for h in range(2):
            fresh = pow2_scale(x[0, :, h].float().abs().max().item())
            s = old if old.item() >= fresh else torch.tensor(fresh)
            assert got.scale[which][1, h].item() == s.item()
            assert torch.equal(got.codes[which][1, 9:13, h], e4m3((x[0, :, h].float() / s).double()))
            if s is not old:
                assert torch.equal(got.codes[which][1, :9, h], e4m3((plain.codes[which][1, :9, h].float() * (old / s)).double()))
            else:
                assert torch.equal(got.codes[which][1, :9, h], plain.codes[which][1, :9, h])
        assert torch.equal(got.codes[which][0], plain.codes[which][0])
        assert torch.equal(got.codes[which][1, 13:], plain.codes[which][1, 13:])


@pytest.mark.gpu
def test_append_bad_indexes(gpu):
    """Indexes that lie outside are checked before an address is formed."""
    import scaled_dot_product_05_gb300 as lib
    x = torch.randn((4, 20, 1, 64), device=DEV).bfloat16()
    table = i32([[0, 99], [-1, 1], [2, 3], [4, 5]])     # pages of a pool of 8
    cache = make_cache(8, 16, 1, 64, "heads")
    before = cache.k.view(torch.uint8).clone()
    lib.sdpa_cache_append(x, x, cache, table, i32([0, 0, 0, 0]))
    assert lib.sdpa_device_error() == 0x601
    changed = (cache.k.view(torch.uint8) != before).flatten(1).any(1).tolist()
    assert changed == [True, True, True, True, True, True, False, False]
    # behind the end of the table, and before its beginning
    before = cache.k.view(torch.uint8).clone()
    lib.sdpa_cache_append(x[2:], x[2:], cache, table[2:], i32([30, -5]))
    assert lib.sdpa_device_error() == 0x602
    changed = (cache.k.view(torch.uint8) != before).flatten(1).any(1).tolist()
    assert changed == [False, False, False, True, False, False, False, False]
    # a position outside the rotation table: that key is not written, its value is
    rope = lib.rope_table(3, 64, device=DEV)
    bk, bv = cache.k.view(torch.uint8).clone(), cache.v.view(torch.uint8).clone()
    y = x[:1, :5].contiguous()
    lib.sdpa_cache_append(y, y, cache, i32([[6]]), i32([0]), rope=rope)
    assert lib.sdpa_device_error() == 0x701
    assert torch.equal(cache.k.view(torch.uint8)[6, 3:], bk[6, 3:]) and not torch.equal(cache.k.view(torch.uint8)[6, :3], bk[6, :3])
    assert not torch.equal(cache.v.view(torch.uint8)[6, 3:5], bv[6, 3:5])


# ----------------------------------------------------------------- attention --

# page, Hq, Hkv, D, Sq, dtype, layout, causal, starts, counts, scale
READS = [
    (16, 4, 1, 128, 1, "bf16", "heads", True, [0, 15, 16, 127, 128, 1000], None, None),
    (64, 8, 2, 128, 1, "fp16", "tokens", True, [0, 63, 64, 2047, 5000, 129], None, None),
    (128, 3, 3, 64, 1, "bf16", "pairs", False, [0, 127, 128, 3000, 1, 255], None, 0.3),
    (32, 10, 2, 64, 3, "fp16", "heads", True, [0, 29, 30, 126, 127, 700], [3, 3, 2, 3, 1, 0], None),
    (64, 32, 1, 128, 5, "bf16", "heads", True, [0, 250, 123, 4000, 60, 1], [5, 5, 4, 5, 1, 5], None),
    (16, 14, 2, 128, 40, "bf16", "tokens", True, [0, 100, 88, 7, 1, 500], [40, 17, 40, 1, 40, 40], 0.125),
    (128, 6, 2, 64, 200, "fp16", "heads", True, [0, 56, 700, 57, 128, 1], [200, 200, 143, 1, 200, 64], None),
    (32, 4, 4, 128, 130, "bf16", "pairs", False, [0, 3, 126, 300, 0, 1], [130, 64, 130, 128, 1, 127], None),
]


def read_case(case, seed=9):
    page, Hq, Hkv, D, Sq, dt, layout, causal, start, count, scale = case
    B, width = len(start), (max(start) + Sq) // page + 2
    cache = make_cache(B * width + 5, page, Hkv, D, layout, seed)
    table = tables(B * width + 5, B, width, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    q = torch.randn((B, Sq, Hq, D), generator=g).to(DT[dt])
    return cache, table, q


def check(case, cache, table, q, o, lse, fill=None):
    page, Hq, Hkv, D, Sq, dt, layout, causal, start, count, scale = case
    plain = PlainCache(cache)
    scale = scale or 1 / math.sqrt(D)
    for b in range(len(start)):
        n = Sq if count is None else count[b]
        total = start[b] + n
        pages = table[b, :-(-total // page)].long()
        if n:
            ref, z, spread, mag, floor = attention64(q[b, :n].double(), plain.rows(0, pages, total),
                                                     plain.rows(1, pages, total), start[b], causal, total, scale)
            ds = 2.0 ** -17 * mag + 1e-6                        # a score's error
            tol = (HALF[dt] * ref.abs() + (2.0 ** -8 + 2 * ds.T[..., None]) * spread + 2.0 ** -13 / 112 * floor + 2.0 ** -25)
            err = (o[b, :n].cpu().double() - ref).abs()
            assert (err <= tol).all(), (b, (err / tol).max().item())
            assert ((lse[b, :, :n].cpu().double() - z).abs() <= ds + 2.0 ** -22 * z.abs()).all(), b
        if fill is not None:
            assert (o[b, n:] == fill).all() and (lse[b, :, n:] == fill).all()


def launch(case, cache, table, q, **kw):
    import scaled_dot_product_05_gb300 as lib
    page, Hq, Hkv, D, Sq, dt, layout, causal, start, count, scale = case
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full((q.shape[0], Hq, Sq), 7.0, device=DEV)
    lib.sdpa_fwd_paged(q.to(DEV), cache, table.to(DEV), i32(start), None if count is None else i32(count), o, lse,
                       causal=causal, scale=scale, **kw)
    assert lib.sdpa_device_error() == 0
    return o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("case", READS, ids=lambda c: "-".join(map(str, c[:8])))
def test_attention(gpu, case):
    cache, table, q = read_case(case)
    o, lse = launch(case, cache, table, q)
    check(case, cache, table, q, o, lse, fill=7.0)
    again = launch(case, cache, table, q)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Sq", [1, 4, 70])
def test_stale_slots_and_pages_do_not_count(gpu, Sq, causal):
    """NaN codes in every slot behind a sequence's end, NaN scales in every page that it does not use, and page
    indexes behind its end that point nowhere."""
    import scaled_dot_product_05_gb300 as lib
    case = (16, 4, 2, 128, Sq, "bf16", "heads", causal, [0, 13, 14, 130, 255 - Sq], None, None)
    cache, table, q = read_case(case)
    good = launch(case, cache, table, q)
    keep = torch.zeros((cache.n_pages, 16), dtype=torch.bool)
    for b, s in enumerate(case[8]):
        for pos in range(s + Sq):
            keep[table[b, pos // 16].long(), pos % 16] = True
    for codes in (cache.k, cache.v):
        raw = codes.view(torch.uint8)
        raw[~keep.to(DEV)] = 0x7F
    for scale in (cache.k_scale, cache.v_scale):
        scale[~keep.any(1).to(DEV)] = float("nan")
    bad = table.clone()
    for b, s in enumerate(case[8]):
        bad[b, -(-(s + Sq) // 16):] = torch.tensor(-7 if b % 2 else 1 << 30, dtype=torch.int32)
    o, lse = launch(case, cache, bad, q)
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
    assert lib.sdpa_device_error() == 0


@pytest.mark.gpu
def test_nan_value_of_a_later_token_stays_out_of_earlier_rows(gpu):
    case = (16, 4, 2, 64, 6, "bf16", "heads", True, [0, 12, 124, 300], None, None)
    cache, table, q = read_case(case)
    good = launch(case, cache, table, q)
    for b, s in enumerate(case[8]):
        cache.v.view(torch.uint8)[table[b, (s + 4) // 16].long(), (s + 4) % 16, 1, 9] = 0xFF
    o, lse = launch(case, cache, table, q)
    assert torch.equal(o[:, :4], good[0][:, :4]) and torch.equal(lse, good[1])
    assert torch.equal(o[:, 4:, :2], good[0][:, 4:, :2])                 # the other KV head
    assert o[:, 4:, 2:, 9].isnan().all()
    rest = [d for d in range(64) if d != 9]
    assert torch.equal(o[:, 4:, 2:][..., rest], good[0][:, 4:, 2:][..., rest])


@pytest.mark.gpu
def test_nan_key_reaches_the_rows_that_see_it(gpu):
    case = (32, 2, 1, 128, 3, "fp16", "heads", True, [40, 126], None, None)
    cache, table, q = read_case(case)
    good = launch(case, cache, table, q)
    for b, s in enumerate(case[8]):
        cache.k.view(torch.uint8)[table[b, (s + 1) // 32].long(), (s + 1) % 32, 0, 0] = 0x7F
    o, lse = launch(case, cache, table, q)
    assert torch.equal(o[:, 0], good[0][:, 0]) and o[:, 1:].isnan().all() and lse[:, :, 1:].isnan().all()


@pytest.mark.gpu
def test_rows_that_see_no_key(gpu):
    # a start before the beginning: the rows whose position is negative see nothing
    case = (16, 4, 2, 128, 3, "bf16", "heads", True, [-2, 5, -9], None, None)
    import scaled_dot_product_05_gb300 as lib
    cache = make_cache(12, 16, 2, 128, "heads")
    table = tables(12, 3, 2, 3)
    q = torch.randn((3, 3, 4, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    o, lse = launch(case, cache, table, q)
    assert (o[0, :2] == 0).all() and (lse[0, :, :2] == -math.inf).all()
    assert (o[2] == 0).all() and (lse[2] == -math.inf).all()
    plain = PlainCache(cache)
    v0 = plain.rows(1, table[0, :1].long(), 1)[0].repeat_interleave(2, 0)
    # position 0 sees one key: its value, which 4 bits hold and so do 8
    assert torch.equal(o[0, 2].cpu().double(), v0)
    assert lib.sdpa_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [1, 40])
def test_attention_bad_pages(gpu, Sq):
    """Pages outside the pool and positions outside the table are left out."""
    import scaled_dot_product_05_gb300 as lib
    cache = make_cache(9, 32, 1, 64, "heads")
    table = i32([[1, 50, 3, -1, 4], [2, 0, 5, 6, 7]])
    q = torch.randn((2, Sq, 2, 64), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    o = torch.empty_like(q)
    lse = torch.empty((2, 2, Sq), device=DEV)
    lib.sdpa_fwd_paged(q, cache, table, i32([149, 100]), None, o, lse, causal=False)
    assert lib.sdpa_device_error() in (0x601, 0x602)
    plain = PlainCache(cache)
    n = 149 + Sq
    keys = [p * 32 + t for p in (0, 2, 4) for t in range(32) if p * 32 + t < n]
    full = table[0].cpu().long().clamp(0, 8)
    k, v = plain.rows(0, full, 160)[keys], plain.rows(1, full, 160)[keys]
    ref, z, spread, mag, floor = attention64(q[0].cpu().double(), k, v, 0, False, len(keys), 1 / 8)
    tol = HALF["bf16"] * ref.abs() + (2.0 ** -8 + 2.0 ** -15 * mag.T[..., None]) * spread + 2.0 ** -13 / 112 * floor + 2.0 ** -25
    assert ((o[0].cpu().double() - ref).abs() <= tol).all()
    assert o.isfinite().all() and lse.isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_wide_range_of_scores_and_scales(gpu, dt):
    """Pages whose scales differ by 2^12, queries with large and small channels."""
    case = (16, 4, 1, 128, 2, dt, "heads", True, [3000, 700], None, 0.05)
    cache, table, q = read_case(case)
    g = torch.Generator().manual_seed(2)
    cache.v_scale.mul_((2.0 ** torch.randint(-6, 7, cache.v_scale.shape, generator=g)).to(DEV))
    cache.k_scale.mul_((2.0 ** torch.randint(-3, 2, cache.k_scale.shape, generator=g)).to(DEV))
    q[..., ::7] *= 2.0 ** -9
    q[..., 1::7] *= 2.0 ** 3
    o, lse = launch(case, cache, table, q)
    check(case, cache, table, q, o, lse)


@pytest.mark.gpu
def test_attention_sink(gpu):
    """One token far above the others, whose many small weights still make most of the sum.  The whole output: half a
    step of bf16, and 2^-8 for the weights."""
    n, D = 40000, 128
    cache = make_cache(n // 64, 64, 1, D, "heads")
    cache.k.view(torch.uint8)[:, :, :, 0] = 0
    cache.k.view(torch.uint8)[0, 5, 0, 0] = 0x7E                       # 448
    q = torch.randn((1, 1, 4, D), generator=torch.Generator().manual_seed(1)).bfloat16() * 0.25
    table = torch.arange(n // 64, dtype=torch.int32)[None]
    q[..., 0] = 9.0 / (448 * cache.k_scale[0, 0].item()) * math.sqrt(D)  # its score: about 9 above the rest
    case = (64, 4, 1, D, 1, "bf16", "heads", True, [n - 1], None, None)
    o, lse = launch(case, cache, table, q)
    check(case, cache, table, q, o, lse)
    plain = PlainCache(cache)
    ref = attention64(q[0].double(), plain.rows(0, table[0].long(), n), plain.rows(1, table[0].long(), n), n - 1, True,
                      n, 1 / math.sqrt(D))[0]
    assert ((o[0].cpu().double() - ref).norm() / ref.norm()).item() <= 2.0 ** -8 + HALF["bf16"]


@pytest.mark.gpu
def test_strided_queries_and_outputs(gpu):
    import scaled_dot_product_05_gb300 as lib
    case = (32, 8, 2, 128, 3, "bf16", "heads", True, [90, 17], None, None)
    cache, table, q = read_case(case)
    ref, lse = launch(case, cache, table, q)
    wide = torch.randn((2, 3, 12, 128), device=DEV).bfloat16()
    wide[:, :, :8] = q.to(DEV)
    out = torch.full((2, 8, 3, 128), 7.0, device=DEV).bfloat16().permute(0, 2, 1, 3)
    lib.sdpa_fwd_paged(wide[:, :, :8], cache, table.to(DEV), i32([90, 17]), o=out)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


@pytest.mark.gpu
def test_streams_graphs_and_chained_calls(gpu):
    import scaled_dot_product_05_gb300 as lib
    case = (16, 8, 2, 128, 1, "bf16", "heads", True, [500, 17, 1023], None, None)
    cache, table, q = read_case(case)
    t, qd = table.to(DEV), q.to(DEV)
    start = i32(case[8])
    x = torch.randn((3, 1, 2, 128), device=DEV).bfloat16()
    ref_cache = [a.clone() for a in (cache.k, cache.v, cache.k_scale, cache.v_scale)]

    def step(o, lse, ws, c, **kw):
        lib.sdpa_cache_append(x, x, c, t, start, **kw)
        lib.sdpa_fwd_paged(qd, c, t, start, o=o, lse=lse, workspace=ws, **kw)

    def bufs():
        return (torch.zeros_like(qd), torch.zeros((3, 8, 1), device=DEV),
                torch.empty(lib.paged_workspace_bytes(3, 8, 2, 1, 128), dtype=torch.uint8, device=DEV))

    a = bufs()
    step(*a, cache)
    torch.cuda.synchronize()
    # another stream, a cache as it was
    other = lib.PagedCache(*[s.clone(memory_format=torch.preserve_format) for s in ref_cache])
    b, st = bufs(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    step(*b, other, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(cache.k.view(torch.uint8), other.k.view(torch.uint8))
    # two captured graphs that share a workspace, replayed in turn
    graphs = []
    for _ in range(2):
        c = bufs()
        c = (c[0], c[1], b[2])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(*c, other)
        graphs.append((g, c))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, c in graphs:
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    # the lengths are read on the device: the same graph on another position
    start.fill_(40)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    d = bufs()
    step(*d, other)
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], d[0]) and not torch.equal(d[0], a[0])


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_memory_of_a_call_on_another_stream(gpu, raw, monkeypatch):
    """What a call allocates comes from its stream's memory: the workspace that it drops must not go to an allocation
    of the current stream, whose kernels would not wait for the call's."""
    import scaled_dot_product_05_gb300 as lib
    from scaled_dot_product_05_gb300 import cache as module
    n_pages, page, B, Hkv, Hq, D = 12, 16, 1, 2, 8, 64
    c = lib.PagedCache.empty(n_pages, page, Hkv, D, device=DEV)
    g = torch.Generator(DEV).manual_seed(5)
    q = torch.randn((B, 1, Hq, D), generator=g, device=DEV).to(torch.bfloat16)
    k = torch.randn((B, 150, Hkv, D), generator=g, device=DEV).to(torch.bfloat16)
    table = torch.arange(n_pages, dtype=torch.int32, device=DEV)[None]
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    lib.sdpa_cache_append(k, k, c, table, zero)
    start = zero + 149
    want = lib.sdpa_fwd_paged(q, c, table, start)
    w = torch.ones(D, device=DEV)
    grads = lib.sdpa_qk_norm_rope_bwd(k, None, k, None, q_weight=w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    spans = []
    orig = module._workspace

    def spy(t, device):
        spans.append((t.data_ptr(), t.data_ptr() + t.numel()))
        return orig(t, device)
    monkeypatch.setattr(module, "_workspace", spy)
    stream = side.cuda_stream if raw else side
    got = lib.sdpa_fwd_paged(q, c, table, start, stream=stream)
    gots = lib.sdpa_qk_norm_rope_bwd(k, None, k, None, q_weight=w, stream=stream)
    assert len(spans) == 2
    kept = [torch.empty(b - a, dtype=torch.uint8, device=DEV) for a, b in spans for _ in range(4)]
    for t in kept:
        for a, b in spans:
            assert t.data_ptr() >= b or t.data_ptr() + t.numel() <= a
    side.synchronize()
    assert torch.equal(got, want)
    for x, y in zip(gots, grads):
        assert (x is None and y is None) or torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_serving_loop(gpu, dt):
    """Prompts of unlike lengths, then single tokens: norm and rotation of q and k, append, attention, against the
    plain cache in 64 bits."""
    import scaled_dot_product_05_gb300 as lib
    B, Hq, Hkv, D, page, width = 3, 4, 2, 128, 16, 5
    cache = make_cache(B * width + 1, page, Hkv, D, "heads", filled=False)
    table = tables(B * width + 1, B, width, 8)
    td = table.to(DEV)
    rope = lib.rope_table(page * width, D, device=DEV)
    g = torch.Generator().manual_seed(13)
    start = [0, 0, 0]
    for S, count in ((45, [45, 16, 3]), (1, [1, 1, 1]), (1, [1, 0, 1]), (2, [2, 1, 2])):
        x = torch.randn((B, S, Hq + 2 * Hkv, D), generator=g).to(DT[dt]).to(DEV)
        pos = (torch.tensor(start)[:, None] + torch.arange(S)).to(torch.int32).to(DEV)
        q, k = lib.sdpa_qk_norm_rope(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], rope=rope, positions=pos)
        lib.sdpa_cache_append(k, x[:, :, Hq + Hkv:], cache, td, i32(start), i32(count))
        o, lse = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV), torch.full((B, Hq, S), 7.0, device=DEV)
        lib.sdpa_fwd_paged(q, cache, td, i32(start), i32(count), o, lse)
        assert lib.sdpa_device_error() == 0
        case = (page, Hq, Hkv, D, S, dt, "heads", True, start, count, None)
        check(case, cache, table, q.cpu(), o, lse, fill=7.0)
        # and what the cache holds is what was put there, within E4M3's half step
        plain = PlainCache(cache)
        for b in range(B):
            if count[b]:
                n = start[b] + count[b]
                rows = plain.rows(1, table[b, :-(-n // page)].long(), n)[start[b]:]
                want = x[b, :count[b], Hq + Hkv:].cpu().double()
                assert ((rows - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * plain.scale[1][table[b].long()].max()).all()
        start = [a + c for a, c in zip(start, count)]


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu):
    """A pool whose far pages lie more than 2^32 bytes from its base."""
    import scaled_dot_product_05_gb300 as lib
    H, page, D = 8, 128, 128
    n_pages = (1 << 32) // (H * page * D) + 40
    cache = lib.PagedCache.empty(n_pages, page, H, D, device=DEV)
    table = torch.tensor([[n_pages - 1, n_pages - 9], [3, n_pages - 5]], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((2, 200, H, D), generator=g).bfloat16()
    lib.sdpa_cache_append(x.to(DEV), x.to(DEV), cache, table.to(DEV), i32([0, 0]), i32([200, 150]))
    q = torch.randn((2, 1, H, D), generator=g).bfloat16()
    o, lse = torch.empty_like(q, device=DEV), torch.empty((2, H, 1), device=DEV)
    lib.sdpa_fwd_paged(q.to(DEV), cache, table.to(DEV), i32([199, 149]), None, o, lse)
    assert lib.sdpa_device_error() == 0
    at = table.flatten().long().to(DEV)
    small = lib.PagedCache(*(t.view(torch.uint8)[at] for t in (cache.k, cache.v)), cache.k_scale[at], cache.v_scale[at])
    o2 = lib.sdpa_fwd_paged(q.to(DEV), small, i32([[0, 1], [2, 3]]), i32([199, 149]))
    torch.cuda.synchronize()
    assert torch.equal(o, o2)
    check((page, H, H, D, 1, "bf16", "heads", True, [199, 149], None, None), small,
          torch.tensor([[0, 1], [2, 3]], dtype=torch.int32), q, o, lse)
