"""Attention over the paged cache with a sliding window and for trees of
drafted tokens, against the definition in 64 bits.

Tolerances.  Scores are sums of D exact products in 32 bits (2^-17 of the sum
of their magnitudes for D = 128); a weight is rounded to f16: by 2^-11 of
itself, or, where it is small, by 2^-32 of its row's largest; the output rounds
once (half a step of its type).  The LSE has the scores' error and that of a
logarithm in 32 bits."""
import math

import pytest
import torch

from tests.test_paged_cache import DEV, DT, HALF, PlainCache, gpu, i32, make_cache, tables  # noqa: F401

FILL = 7.0


def attention64(q, k, v, seen, scale):
    """q [S, Hq, D], k and v [n, Hkv, D], seen [S, n]: (O, LSE, sum p |v|, magnitude of the scores, largest weight's
    share of small ones)."""
    G = q.shape[1] // k.shape[1]
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("shd,nhd->hsn", q, kk) * scale
    mag = (torch.einsum("shd,nhd->hsn", q.abs(), kk.abs()) * scale).masked_fill(~seen, 0)
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:2], -math.inf, dtype=s.dtype)
    p = torch.where(seen, (s - torch.where(lse.isinf(), 0.0, lse)[..., None]).exp(), torch.zeros_like(s))
    o = torch.einsum("hsn,nhd->shd", p, vv)
    spread = torch.einsum("hsn,nhd->shd", p, vv.abs())
    if not s.shape[-1]:
        return o, lse, spread, torch.zeros_like(lse), spread
    floor = p.amax(-1).T[..., None] * torch.einsum("hsn,nhd->shd", seen.double().expand_as(p), vv.abs())
    return o, lse, spread, mag.amax(-1), floor


def check(cache, table, q, start, count, sees, o, lse, dt):
    """sees(b, n, total) gives the mask [n, total] of a sequence."""
    plain = PlainCache(cache)
    Sq, D = q.shape[1], q.shape[3]
    for b, st in enumerate(start):
        n = Sq if count is None else count[b]
        total = max(0, st + n)
        if n:
            pages = table[b, :-(-total // cache.page_size)].long()
            ref, z, spread, mag, floor = attention64(q[b, :n].double(), plain.rows(0, pages, total),
                                                     plain.rows(1, pages, total), sees(b, n, total), 1 / math.sqrt(D))
            ds = 2.0 ** -17 * mag + 1e-6
            tol = HALF[dt] * ref.abs() + (2.0 ** -11 + 2 * ds.T[..., None]) * spread + 2.0 ** -32 * floor + 2.0 ** -25
            err = (o[b, :n].cpu().double() - ref).abs()
            assert (err <= tol).all(), (b, (err / tol).max().item())
            got = lse[b, :, :n].cpu().double()
            none = z == -math.inf
            assert (got[none] == -math.inf).all() and (o[b, :n].cpu().double().transpose(0, 1)[none] == 0).all()
            assert ((got - z).abs()[~none] <= (ds + 2.0 ** -22 * z.abs())[~none]).all(), b
        assert (o[b, n:] == FILL).all() and (lse[b, :, n:] == FILL).all()


def case_data(page, Hq, Hkv, D, Sq, dt, layout, start, seed=3):
    B, width = len(start), (max(0, max(start)) + Sq) // page + 2
    cache = make_cache(B * width + 5, page, Hkv, D, layout, seed)
    table = tables(B * width + 5, B, width, seed + 1)
    q = torch.randn((B, Sq, Hq, D), generator=torch.Generator().manual_seed(seed + 2)).to(DT[dt])
    return cache, table, q


def outputs(q):
    B, Sq, Hq, _ = q.shape
    return torch.full(q.shape, FILL, dtype=q.dtype, device=DEV), torch.full((B, Hq, Sq), FILL, device=DEV)


# -------------------------------------------------------------------- window --

def window_sees(start, window, sinks):
    def sees(b, n, total):
        i = start[b] + torch.arange(n)[:, None]
        j = torch.arange(total)
        return (j <= i) & ((j > i - window) | (j < sinks))
    return sees


def give_back(cache, table, start, count, Sq, window, sinks):
    """A table whose pages without a visible position point nowhere, those behind the end too."""
    t, page = table.clone(), cache.page_size
    for b, st in enumerate(start):
        n = Sq if count is None else count[b]
        for p in range(t.shape[1]):
            if p * page >= st + n or (p * page >= sinks and (p + 1) * page <= st - window + 1):
                t[b, p] = -5 if p % 2 else 1 << 29
    return t


# page, Hq, Hkv, D, Sq, dtype, layout, starts, counts, window, sinks
WINDOWS = [
    (16, 4, 1, 128, 1, "bf16", "heads", [0, 15, 16, 127, 128, 1000, 333], None, 100, 4),
    (64, 8, 2, 128, 1, "fp16", "tokens", [0, 63, 64, 2047, 5000, 129], None, 64, 0),
    (128, 3, 3, 64, 1, "bf16", "pairs", [0, 127, 128, 3000, 1, 255], None, 1, 1),
    (128, 3, 3, 64, 1, "fp16", "heads", [0, 127, 128, 3000, 1, 255], None, 1, 0),       # each sees itself alone
    (32, 10, 2, 64, 3, "fp16", "heads", [0, 29, 30, 126, 127, 700], [3, 3, 2, 3, 1, 0], 60, 130),
    (64, 16, 2, 64, 2, "bf16", "heads", [0, 250, 123, 4000, 60, 1], None, 1 << 30, 0),   # everything
    (64, 32, 1, 128, 5, "bf16", "heads", [0, 250, 123, 4000, 60, 1], [5, 5, 4, 5, 1, 5], 3, 1),
    (16, 14, 2, 128, 40, "bf16", "tokens", [0, 100, 88, 7, 1, 500], [40, 17, 40, 1, 40, 40], 33, 2),
    (128, 6, 2, 64, 200, "fp16", "heads", [0, 56, 700, 57, 128, 1], [200, 200, 143, 1, 200, 64], 70, 0),
    (32, 4, 4, 128, 300, "fp16", "pairs", [0, 3, 126, 900, 0, 1], [300, 64, 300, 128, 1, 127], 500, 200),
    (16, 4, 2, 128, 20, "bf16", "heads", [-3, -30, 0, 5], None, 8, 2),                   # rows before the first position
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(map(str, c)))
def test_window(gpu, case):  # noqa: F811
    import scaled_dot_product_05_gb300 as lib
    page, Hq, Hkv, D, Sq, dt, layout, start, count, window, sinks = case
    cache, table, q = case_data(page, Hq, Hkv, D, Sq, dt, layout, start)
    freed = give_back(cache, table, start, count, Sq, window, sinks)
    for t in (table, freed):
        o, lse = outputs(q)
        lib.sdpa_fwd_paged_window(q.to(DEV), cache, t.to(DEV), i32(start), None if count is None else i32(count), o, lse,
                                  window=window, sinks=sinks)
        assert lib.sdpa_device_error() == 0
        check(cache, table, q, start, count, window_sees(start, window, sinks), o, lse, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [1, 4, 70])
def test_window_masked_nan(gpu, Sq):  # noqa: F811
    """NaN in every slot that no row sees, and in one that only some rows see."""
    import scaled_dot_product_05_gb300 as lib
    window, sinks, start = 50, 3, [0, 13, 200, 400 - Sq]
    cache, table, q = case_data(32, 4, 2, 128, Sq, "bf16", "heads", start)

    def go():
        o, lse = outputs(q)
        lib.sdpa_fwd_paged_window(q.to(DEV), cache, table.to(DEV), i32(start), None, o, lse, window=window, sinks=sinks)
        assert lib.sdpa_device_error() == 0
        return o, lse
    good = go()
    keep = torch.zeros((cache.n_pages, 32), dtype=torch.bool)
    for b, s in enumerate(start):
        for pos in range(s + Sq):
            if pos < sinks or pos > s - window:
                keep[table[b, pos // 32].long(), pos % 32] = True
    for codes in (cache.k, cache.v):
        codes.view(torch.uint8)[~keep.to(DEV)] = 0x7F
    again = go()
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
    if Sq == 1:
        return
    # a value that the first rows see and the last do not (behind the window's lower edge), and the other way round
    for shift, first, last in ((-window + 1, 0, 1), (Sq - 1, Sq - 1, Sq)):
        saved = cache.v.view(torch.uint8).clone()
        for b in (2, 3):
            pos = start[b] + shift
            cache.v.view(torch.uint8)[table[b, pos // 32].long(), pos % 32, 1, 9] = 0xFF
        o, lse = go()
        for b in (2, 3):
            bad = o[b].isnan()
            want = torch.zeros_like(bad)
            want[first:last, 2:, 9] = True
            assert torch.equal(bad, want)
            assert torch.equal(o[b][~bad], good[0][b][~bad])
        cache.v.view(torch.uint8).copy_(saved)


@pytest.mark.gpu
def test_window_bad_page(gpu):  # noqa: F811
    """A page that some row sees and that is none is left out and reported."""
    import scaled_dot_product_05_gb300 as lib
    cache, table, q = case_data(16, 4, 2, 64, 1, "bf16", "heads", [100, 40])
    table[0, 5] = 9999
    o, lse = outputs(q)
    lib.sdpa_fwd_paged_window(q.to(DEV), cache, table.to(DEV), i32([100, 40]), None, o, lse, window=30, sinks=0)
    assert lib.sdpa_device_error() == 0x601

    def sees(b, n, total):
        m = window_sees([100, 40], 30, 0)(b, n, total)
        if b == 0:
            m[:, 80:96] = False
        return m
    table[0, 5] = 0
    check(cache, table, q, [100, 40], None, sees, o, lse, "bf16")


# ---------------------------------------------------------------------- tree --

def random_tree(B, T, seed):
    g = torch.Generator().manual_seed(seed)
    parents = torch.full((B, T), -1, dtype=torch.int64)
    for i in range(1, T):
        parents[:, i] = torch.randint(-1, i, (B,), generator=g)
    return parents


def ancestors(parents):
    B, T = parents.shape
    m = torch.zeros((B, T, T), dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            j = i
            while j >= 0:
                m[b, i, j] = True
                j = int(parents[b, j])
    return m


def pack(m):
    """[B, T, T] truth values as words of 32 bits."""
    B, T, _ = m.shape
    out = torch.zeros((B, T, (T + 31) // 32), dtype=torch.int64)
    for j in range(T):
        out[:, :, j // 32] |= m[:, :, j].long() << (j % 32)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def tree_sees(start, m):
    def sees(b, n, total):
        out = torch.zeros((n, total), dtype=torch.bool)
        st = start[b]
        out[:, :max(0, st)] = True
        for j in range(n):
            if st + j >= 0:
                out[:, st + j] = m[b, :n, j]
        return out
    return sees


# page, Hq, Hkv, D, T, dtype, layout, starts, counts
TREES = [
    (16, 4, 4, 128, 1, "bf16", "heads", [0, 15, 127, 128, 1000], None),
    (64, 8, 4, 64, 7, "fp16", "tokens", [0, 60, 122, 127, 128, 700], [7, 7, 7, 1, 0, 5]),
    (32, 8, 2, 128, 4, "bf16", "pairs", [0, 125, 300, 2999], None),
    (128, 3, 1, 64, 40, "bf16", "heads", [0, 100, 127, 500], [40, 40, 33, 32]),
    (16, 32, 8, 128, 16, "bf16", "heads", [0, 120, 1500, 47], [16, 16, 3, 16]),
    (64, 14, 2, 128, 61, "fp16", "heads", [0, 70, 640, 3001], None),
    (32, 2, 2, 64, 200, "fp16", "tokens", [0, 56, 128, 1000], [200, 199, 65, 200]),
    (16, 4, 2, 64, 9, "fp16", "heads", [-4, 3, -20, 0], None),                           # tokens before the first position
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", TREES, ids=lambda c: "-".join(map(str, c)))
def test_tree(gpu, case):  # noqa: F811
    import scaled_dot_product_05_gb300 as lib
    page, Hq, Hkv, D, T, dt, layout, start, count = case
    cache, table, q = case_data(page, Hq, Hkv, D, T, dt, layout, start)
    parents = random_tree(len(start), T, 8)
    m = ancestors(parents)
    mask = lib.tree_mask(parents.to(DEV))
    assert torch.equal(mask.cpu(), pack(m))
    o, lse = outputs(q)
    lib.sdpa_fwd_paged_tree(q.to(DEV), cache, table.to(DEV), i32(start), mask, None if count is None else i32(count), o, lse)
    assert lib.sdpa_device_error() == 0
    check(cache, table, q, start, count, tree_sees(start, m), o, lse, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 33, 130])
def test_tree_any_mask(gpu, T):  # noqa: F811
    """Masks that are no trees: rows that see nothing new, later tokens, not themselves; with nothing before them too."""
    import scaled_dot_product_05_gb300 as lib
    start = [0, 130, 5]
    cache, table, q = case_data(16, 4, 2, 64, T, "fp16", "heads", start)
    m = torch.rand((3, T, T), generator=torch.Generator().manual_seed(1)) < 0.3
    m[:, T // 2] = False                                                # sequence 0: this row sees no key at all
    o, lse = outputs(q)
    lib.sdpa_fwd_paged_tree(q.to(DEV), cache, table.to(DEV), i32(start), pack(m).to(DEV), None, o, lse)
    check(cache, table, q, start, None, tree_sees(start, m), o, lse, "fp16")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 40])
def test_tree_nan_of_another_branch(gpu, T):  # noqa: F811
    """A NaN value reaches the rows that see it and no others."""
    import scaled_dot_product_05_gb300 as lib
    start = [100, 126]
    cache, table, q = case_data(16, 4, 2, 128, T, "bf16", "heads", start)
    m = ancestors(random_tree(2, T, 3))
    m[:, :, 1] = False
    m[:, 2, 1] = True

    def go():
        o, lse = outputs(q)
        lib.sdpa_fwd_paged_tree(q.to(DEV), cache, table.to(DEV), i32(start), pack(m).to(DEV), None, o, lse)
        return o, lse
    good = go()
    for b, s in enumerate(start):
        cache.v.view(torch.uint8)[table[b, (s + 1) // 16].long(), (s + 1) % 16, 0, 77] = 0x7F
    o, lse = go()
    want = torch.zeros_like(o, dtype=torch.bool)
    want[:, 2, :2, 77] = True
    assert torch.equal(o.isnan(), want) and torch.equal(o[~want], good[0][~want]) and torch.equal(lse, good[1])


@pytest.mark.gpu
def test_tree_of_one_branch_is_the_causal_pass(gpu):  # noqa: F811
    import scaled_dot_product_05_gb300 as lib
    for T in (3, 30):
        cache, table, q = case_data(32, 8, 2, 128, T, "bf16", "heads", [50, 777])
        mask = pack(torch.ones(2, T, T, dtype=torch.bool).tril())
        o, lse = outputs(q)
        lib.sdpa_fwd_paged_tree(q.to(DEV), cache, table.to(DEV), i32([50, 777]), mask.to(DEV), None, o, lse)
        o2, lse2 = outputs(q)
        lib.sdpa_fwd_paged(q.to(DEV), cache, table.to(DEV), i32([50, 777]), None, o2, lse2)
        assert (o.float() - o2.float()).abs().max() <= 2 * HALF["bf16"] * o2.float().abs().max()
        assert (lse - lse2).abs().max() <= 1e-4


@pytest.mark.gpu
def test_refusals(gpu):  # noqa: F811
    import scaled_dot_product_05_gb300 as lib
    cache, table, q = case_data(16, 4, 2, 64, 3, "bf16", "heads", [5])
    args = (q.to(DEV), cache, table.to(DEV), i32([5]))
    for window, sinks in ((0, 0), (5, -1)):
        with pytest.raises(lib.SdpaError):
            lib.sdpa_fwd_paged_window(*args, window=window, sinks=sinks)
    for bad in (torch.zeros((1, 3, 2), dtype=torch.int32, device=DEV), torch.zeros((1, 3, 1), dtype=torch.int64, device=DEV),
                torch.zeros((1, 3, 1), dtype=torch.int32)):
        with pytest.raises(ValueError):
            lib.sdpa_fwd_paged_tree(*args, bad)


# ------------------------------------------- 17 to 64 rows, and calls with none --

@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", [
    (16, 17, 1, 128, 1, "bf16", "heads"), (64, 8, 2, 64, 5, "fp16", "tokens"), (32, 32, 2, 128, 4, "bf16", "pairs"),
    (128, 4, 4, 64, 33, "bf16", "heads"), (16, 12, 4, 128, 21, "fp16", "heads")], ids=str)
def test_plain_attention_of_some_rows(gpu, case, causal):  # noqa: F811
    """The attention without a mask of its own, where its rows stand in the lanes twice."""
    from tests.test_paged_cache import check as check_plain, launch, read_case
    page, Hq, Hkv, D, Sq, dt, layout = case
    start, count = [0, 126, 1000, 3, 64, 2500], [Sq, Sq, max(1, Sq - 1), 1, 0, Sq]
    full = (page, Hq, Hkv, D, Sq, dt, layout, causal, start, count, None)
    cache, table, q = read_case(full)
    o, lse = launch(full, cache, table, q)
    check_plain(full, cache, table, q, o, lse, fill=7.0)
    # a NaN value of the last token stays out of the rows that do not see it
    if causal and Sq > 1:
        for b in (1, 5):
            pos = start[b] + Sq - 1
            cache.v.view(torch.uint8)[table[b, pos // page].long(), pos % page, 0, 5] = 0x7F
        o2, lse2 = launch(full, cache, table, q)
        want = torch.zeros_like(o, dtype=torch.bool)
        for b in (1, 5):
            want[b, Sq - 1, :Hq // Hkv, 5] = True
        assert torch.equal(o2.isnan(), want) and torch.equal(o2[~want], o[~want]) and torch.equal(lse2, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [1, 4, 12, 40])
def test_no_rows_at_all(gpu, Sq):  # noqa: F811
    """Counts of zero everywhere: nothing is written."""
    import scaled_dot_product_05_gb300 as lib
    cache, table, q = case_data(16, 8, 2, 64, Sq, "bf16", "heads", [30, 0, 500])
    o, lse = outputs(q)
    args = (q.to(DEV), cache, table.to(DEV), i32([30, 0, 500]))
    none = i32([0, 0, 0])
    lib.sdpa_fwd_paged_window(*args, none, o, lse, window=20, sinks=1)
    lib.sdpa_fwd_paged_tree(*args, torch.zeros((3, Sq, (Sq + 31) // 32), dtype=torch.int32, device=DEV), none, o, lse)
    out = torch.full((3, 2, table.shape[1] * 16), FILL, device=DEV)
    lib.sdpa_cache_weights(*args, none, lse, None, out)
    assert lib.sdpa_device_error() == 0
    assert (o == FILL).all() and (lse == FILL).all() and (out == FILL).all()
