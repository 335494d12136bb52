"""The attention that cached keys draw (sdpa_cache_weights) and the eviction of
those that draw the least (sdpa_cache_evict), alone and in a serving loop.

Tolerances.  A weight exp(s - LSE) has the error of its score (sums of D exact
products in 32 bits: 2^-17 of the sum of their magnitudes for D = 128, 1e-6 for
the exponent's and the LSE's own roundings) and of an exponential (2^-21); the sum
over R rows rounds by R 2^-24 of itself at most.  An eviction picks and moves: its
numbers, scores, codes and scales have to match bit for bit."""
import math

import pytest
import torch

from tests.test_paged_cache import DEV, DT, PlainCache, e4m3, gpu, i32, make_cache, pow2_scale, tables  # noqa: F401


# ------------------------------------------------------------------- weights --

def weights64(q, k, lse, seen, scale):
    """(sum over rows and heads of a group of the weights of each key, its error bound), [Hkv, n]."""
    Hkv = k.shape[1]
    G = q.shape[1] // Hkv
    kk = k.repeat_interleave(G, 1)
    s = torch.einsum("shd,nhd->hsn", q, kk) * scale
    mag = torch.einsum("shd,nhd->hsn", q.abs(), kk.abs()) * scale
    live = seen & (lse > -math.inf)[..., None]
    p = torch.where(live, (s - torch.where(lse.isinf(), 0.0, lse)[..., None]).exp(), torch.zeros_like(s))
    err = p * (2.0 ** -17 * mag + 2e-6)
    total = p.unflatten(0, (Hkv, G)).sum((1, 2))
    return total, err.unflatten(0, (Hkv, G)).sum((1, 2)) + q.shape[0] * G * 2.0 ** -24 * total


# page, Hq, Hkv, D, Sq, dtype, layout, causal, starts, counts, old sums
WEIGHTS = [
    (16, 4, 1, 128, 1, "bf16", "heads", True, [0, 15, 16, 127, 128, 1000], None, True),
    (64, 8, 2, 128, 1, "fp16", "tokens", True, [0, 63, 64, 2047, 5000, 129], None, False),
    (128, 3, 3, 64, 1, "bf16", "pairs", False, [0, 127, 128, 3000, 1, 255], None, True),
    (32, 10, 2, 64, 3, "fp16", "heads", True, [0, 29, 30, 126, 127, 700], [3, 3, 2, 3, 1, 0], True),
    (32, 8, 2, 64, 2, "bf16", "heads", False, [0, 29, 30, 126, 127, 700], [2, 1, 2, 2, 1, 0], True),
    (64, 32, 1, 128, 5, "bf16", "heads", True, [0, 250, 123, 4000, 60, 1], [5, 5, 4, 5, 1, 5], True),
    (16, 14, 2, 128, 40, "bf16", "tokens", True, [0, 100, 88, 7, 1, 500], [40, 17, 40, 1, 40, 40], True),
    (128, 6, 2, 64, 200, "fp16", "heads", True, [0, 56, 700, 57, 128, 1], [200, 200, 143, 1, 200, 64], False),
    (32, 4, 4, 128, 300, "fp16", "pairs", False, [0, 3, 126, 300, 0, 1], [300, 64, 300, 128, 1, 127], True),
    (16, 150, 1, 64, 2, "bf16", "heads", True, [0, 300], None, True),             # more heads than a tile has rows
    (16, 4, 2, 128, 20, "bf16", "heads", True, [-3, -30, 0, 5], None, True),      # tokens before the first position
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: "-".join(map(str, c)))
def test_weights(gpu, case):  # noqa: F811
    import scaled_dot_product_05_gb300 as lib
    page, Hq, Hkv, D, Sq, dt, layout, causal, start, count, old = case
    B, width = len(start), (max(start) + Sq) // page + 2
    cache = make_cache(B * width + 5, page, Hkv, D, layout, 3)
    table = tables(B * width + 5, B, width, 4)
    g = torch.Generator().manual_seed(5)
    q = torch.randn((B, Sq, Hq, D), generator=g).to(DT[dt])
    cnt = None if count is None else i32(count)
    lse = torch.full((B, Hq, Sq), math.nan, device=DEV)
    lib.sdpa_fwd_paged(q.to(DEV), cache, table.to(DEV), i32(start), cnt, None, lse, causal=causal)
    n_max = width * page
    score = torch.rand((B, Hkv, n_max), generator=g).to(DEV) if old else None
    out = torch.full((B, Hkv, n_max), 7.0, device=DEV)
    got = lib.sdpa_cache_weights(q.to(DEV), cache, table.to(DEV), i32(start), cnt, lse, score, out, causal=causal)
    assert got is out and lib.sdpa_device_error() == 0
    again = lib.sdpa_cache_weights(q.to(DEV), cache, table.to(DEV), i32(start), cnt, lse, score, torch.full_like(out, 7.0),
                                   causal=causal)
    assert torch.equal(out, again)
    if old:                                             # in place
        inplace = score.clone()
        lib.sdpa_cache_weights(q.to(DEV), cache, table.to(DEV), i32(start), cnt, lse, inplace, inplace, causal=causal)
    plain = PlainCache(cache)
    for b, st in enumerate(start):
        n = Sq if count is None else count[b]
        total = max(0, st + n) if n else 0
        assert (out[b, :, total:] == 7).all()
        if not total:
            continue
        k = plain.rows(0, table[b, :-(-total // page)].long(), total)
        i, j = st + torch.arange(n)[:, None], torch.arange(total)
        seen = (j <= i) if causal else torch.ones((n, total), dtype=torch.bool)
        want, tol = weights64(q[b, :n].double(), k, lse[b, :, :n].cpu().double(), seen, 1 / math.sqrt(D))
        if old:
            want[:, :max(0, st)] += score[b, :, :max(0, st)].cpu().double()
        tol += 2.0 ** -23 * want
        assert ((out[b, :, :total].cpu().double() - want).abs() <= tol).all(), b
        if old:
            assert torch.equal(inplace[b, :, :total], out[b, :, :total])
            assert torch.equal(inplace[b, :, total:], score[b, :, total:])
        # all weights of a call are one for each row that sees a key
        if not old:
            assert abs(out[b, :, :total].double().sum().item() - n * Hq) <= tol.sum().item()


@pytest.mark.gpu
def test_weights_bad_indexes_and_short_rows(gpu):  # noqa: F811
    import scaled_dot_product_05_gb300 as lib
    for Sq in (1, 40):
        cache = make_cache(20, 16, 2, 64, "heads", 3)
        q = torch.randn((1, Sq, 4, 64), device=DEV).bfloat16()
        table = i32([[0, 1, 99, 3, 4, 5, 6, 7, 8, 9, 10]])
        start = i32([120])
        lse = torch.zeros((1, 4, Sq), device=DEV)
        out = torch.full((1, 2, 176), 7.0, device=DEV)
        lib.sdpa_cache_weights(q, cache, table, start, None, lse, None, out)
        assert lib.sdpa_device_error() == 0x601
        assert (out[:, :, 32:48] == 7).all() and (out[:, :, :32] != 7).all() and (out[:, :, 48:120 + Sq] != 7).all()
        # rows of sums that end before the sequence, and a table that does
        table[0, 2] = 2
        buf = torch.full((1, 2, 100), 7.0, device=DEV)
        lib.sdpa_cache_weights(q, cache, table, start, None, lse, None, buf)
        assert lib.sdpa_device_error() == 0x602
        assert (buf != 7).all()
        out.fill_(7)
        lib.sdpa_cache_weights(q, cache, table[:, :6].contiguous(), start, None, lse, None, out)
        assert lib.sdpa_device_error() == 0x602
        assert (out[:, :, :96] != 7).all() and (out[:, :, 96:] == 7).all()


# ------------------------------------------------------------------ eviction --

def pick(score, n, budget, sinks, recent):
    """The tokens that stay, ascending."""
    if n <= budget:
        return list(range(n))
    middle = sorted(range(sinks, n - recent),
                    key=lambda j: (-math.inf if math.isnan(score[j]) else -score[j], not math.isnan(score[j]), j))
    return sorted(list(range(sinks)) + middle[:budget - sinks - recent] + list(range(n - recent, n)))


def check_evict(cache, before, table, new_table, length, score, kept, kept_score, budget, sinks, recent, fill):
    page, got = cache.page_size, PlainCache(cache)
    want = PlainCache.__new__(PlainCache)
    want.page, want.codes, want.scale = page, [c.clone() for c in before.codes], [s.clone() for s in before.scale]
    for b, n in enumerate(length):
        for h in range(cache.n_heads):
            stays = pick(score[b, h].tolist(), n, budget, sinks, recent)
            m = len(stays)
            assert kept[b, h, :m].tolist() == stays, (b, h)
            assert torch.equal(kept_score[b, h, :m].cpu().nan_to_num(-1.), score[b, h, stays].nan_to_num(-1.))
            assert (kept[b, h, m:] == fill).all() and (kept_score[b, h, m:] == fill).all()
            pos = torch.tensor(stays, dtype=torch.long)
            for which in (0, 1):
                src = table[b].long()[pos // page]
                x = before.codes[which][src, pos % page, h] * before.scale[which][src, h][:, None]
                for p in range(-(-m // page)):
                    rows, to = x[p * page:(p + 1) * page], int(new_table[b, p])
                    s = pow2_scale(rows.abs().max().item())
                    want.scale[which][to, h] = s
                    want.codes[which][to, :len(rows), h] = e4m3(rows / s)
    for which in (0, 1):
        assert torch.equal(got.scale[which], want.scale[which])
        assert torch.equal(got.codes[which], want.codes[which])


# page, Hkv, D, layout, lengths, budget, sinks, recent, scores
EVICTIONS = [
    (16, 2, 64, "heads", [0, 1, 15, 16, 17, 33, 100], 16, 2, 3, "normal"),
    (64, 3, 128, "tokens", [1000, 999, 64, 65, 2, 130], 64, 0, 0, "ties"),
    (32, 1, 128, "pairs", [500, 33, 32, 31], 32, 20, 12, "normal"),                  # no room between
    (128, 2, 64, "heads", [3000, 1025, 1024, 129], 1000, 4, 100, "zeros"),
    (16, 1, 64, "tokens", [70, 71, 5], 1, 0, 0, "normal"),
    (16, 2, 128, "heads", [70, 71, 5], 7, 0, 7, "special"),
    (64, 2, 128, "heads", [5000, 4097], 2500, 3, 0, "special"),
    (128, 1, 128, "heads", [40000, 33000, 20000], 3333, 4, 64, "ties"),               # two CTAs a row
]


def scores(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if kind == "ties":
        return torch.randint(0, 5, shape, generator=g).float() / 4
    if kind == "zeros":
        return torch.where(x > 1, x, torch.where(x > 0, 0.0, -0.0))
    if kind == "special":
        x[torch.rand(shape, generator=g) < 0.05] = math.inf
        x[torch.rand(shape, generator=g) < 0.05] = -math.inf
        x[torch.rand(shape, generator=g) < 0.002] = math.nan
        x[torch.rand(shape, generator=g) < 0.1] *= 1e-41
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("case", EVICTIONS, ids=lambda c: "-".join(map(str, c)))
def test_evict(gpu, case):  # noqa: F811
    import scaled_dot_product_05_gb300 as lib
    page, H, D, layout, length, budget, sinks, recent, kind = case
    B, width, more = len(length), max(length) // page + 1, (budget - 1) // page + 1
    total = B * (width + more) + 3
    cache = make_cache(total, page, H, D, layout, 2)
    ids = torch.randperm(total, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    table, new_table = ids[:B * width].reshape(B, width), ids[B * width:B * (width + more)].reshape(B, more)
    # pages of unlike scales, NaN codes, a page of zeros
    f = 2.0 ** torch.randint(-12, 3, (total, H), generator=torch.Generator().manual_seed(4)).float().to(DEV)
    cache.k_scale.mul_(f)
    cache.v.view(torch.uint8)[table[0, 0].long(), 0, 0, 3] = 0
    cache.k.view(torch.uint8)[table[-1, 0].long()] = 0
    score = scores(kind, (B, H, width * page), 5)
    before = PlainCache(cache)
    kept = torch.full((B, H, budget), -9, dtype=torch.int32, device=DEV)
    kept_score = torch.full((B, H, budget), -9.0, device=DEV)
    out = lib.sdpa_cache_evict(cache, table.to(DEV), i32(length), score.to(DEV), new_table.to(DEV), budget=budget, sinks=sinks,
                               recent=recent, kept=kept, kept_score=kept_score)
    assert out[0] is kept and out[1] is kept_score and lib.sdpa_device_error() == 0
    check_evict(cache, before, table, new_table, length, score, kept, kept_score, budget, sinks, recent, -9)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [401, 402, 403])
def test_evict_rows_of_any_length(gpu, n):  # noqa: F811
    """Rows of scores that begin on any multiple of four bytes."""
    import scaled_dot_product_05_gb300 as lib
    length, budget = [n, n - 1, 77], 100
    cache = make_cache(3 * 26 + 3 * 7, 16, 3, 64, "heads", 2)
    ids = torch.randperm(cache.n_pages, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    table, new_table = ids[:78].reshape(3, 26), ids[78:].reshape(3, 7)
    score = scores("ties", (3, 3, n), 5)
    before = PlainCache(cache)
    kept = torch.full((3, 3, budget), -9, dtype=torch.int32, device=DEV)
    kept_score = torch.full((3, 3, budget), -9.0, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (cache, table.to(DEV), i32(length), score.to(DEV), new_table.to(DEV))
    torch.cuda.synchronize()
    lib.sdpa_cache_evict(*args, budget=budget, sinks=1, recent=2, kept=kept, kept_score=kept_score, stream=s)
    s.synchronize()
    check_evict(cache, before, table, new_table, length, score, kept, kept_score, budget, 1, 2, -9)


@pytest.mark.gpu
def test_evict_more_than_shared_memory_holds(gpu):  # noqa: F811
    """Scores of 300 000 tokens (eight CTAs hold 262 144)."""
    import scaled_dot_product_05_gb300 as lib
    n, page, budget = 300000, 128, 1000
    width, more = n // page + 1, 8
    cache = make_cache(width + more, page, 1, 64, "heads", 2)
    table = torch.arange(width, dtype=torch.int32)[None]
    new_table = torch.arange(width, width + more, dtype=torch.int32)[None]
    score = scores("ties", (1, 1, width * page), 5)
    score[0, 0, ::701] += 3
    before = PlainCache(cache)
    kept, kept_score = lib.sdpa_cache_evict(cache, table.to(DEV), i32([n]), score.to(DEV), new_table.to(DEV), budget=budget,
                                            sinks=4, recent=10)
    check_evict(cache, before, table, new_table, [n], score, kept, kept_score, budget, 4, 10, -9)


@pytest.mark.gpu
def test_evict_nan_codes_odd_scales_and_bad_pages(gpu):  # noqa: F811
    import scaled_dot_product_05_gb300 as lib
    cache = make_cache(12, 16, 1, 64, "heads", 2)
    cache.k_scale.fill_(0.3)
    raw = cache.v.view(torch.uint8)
    raw[1, 5, 0, 7] = 0xFF
    before = PlainCache(cache)
    score = torch.arange(48, dtype=torch.float32).reshape(1, 1, 48).to(DEV)
    lib.sdpa_cache_evict(cache, i32([[0, 1, 2]]), i32([48]), score, i32([[8, 9]]), budget=32)
    got = PlainCache(cache)
    assert got.codes[1][8, 5, 0, 7].isnan() and got.codes[1][8].isnan().sum() == 1
    # a scale that is no power of two: values rounded to 32 bits, then to a code
    x = (before.codes[0][[1, 2]].float() * torch.tensor(0.3)).reshape(2, 16, 1, 64)
    for p in range(2):
        s = pow2_scale(x[p].abs().max().item())
        assert got.scale[0][8 + p, 0] == s and torch.equal(got.codes[0][8 + p], e4m3(x[p].double() / s))
    assert lib.sdpa_device_error() == 0
    # an old page outside the pool: zeros; a new one: nothing is written
    raw_before = cache.k.view(torch.uint8).clone()
    lib.sdpa_cache_evict(cache, i32([[0, 99, 2]]), i32([48]), score, i32([[10, -1]]), budget=32)
    assert lib.sdpa_device_error() == 0x601
    assert (cache.k.view(torch.uint8)[10] == 0).all()
    raw_before[10] = 0
    assert torch.equal(cache.k.view(torch.uint8), raw_before)
    # longer than the table
    kept, _ = lib.sdpa_cache_evict(cache, i32([[0, 1, 2]]), i32([4000]), score, i32([[10, 11]]), budget=32)
    assert lib.sdpa_device_error() == 0x602
    assert kept.flatten().tolist() == list(range(16, 48))


@pytest.mark.gpu
def test_refusals(gpu):  # noqa: F811
    import scaled_dot_product_05_gb300 as lib
    cache = make_cache(12, 16, 1, 64, "heads", 2)
    score = torch.zeros((1, 1, 48), device=DEV)
    args = (cache, i32([[0, 1, 2]]), i32([48]), score, i32([[8, 9]]))
    for kw in (dict(budget=33), dict(budget=0), dict(budget=8, sinks=5, recent=4), dict(budget=8, sinks=-1), dict(budget=8, recent=-1)):
        with pytest.raises((lib.SdpaError, ValueError)):
            lib.sdpa_cache_evict(*args, **kw)
    with pytest.raises(ValueError):
        lib.sdpa_cache_evict(cache, args[1], args[2], score[:, :, ::2], args[4], budget=8)
    q = torch.zeros((1, 1, 2, 64), device=DEV).bfloat16()
    with pytest.raises(ValueError):
        lib.sdpa_cache_weights(q, *args[:2], i32([5]), None, None)
    lse, buf = torch.zeros((1, 2, 1), device=DEV), torch.zeros((1, 1, 48), device=DEV)
    for kw in (dict(scale=-1.0), dict(scale=math.inf)):
        with pytest.raises(lib.SdpaError):
            lib.sdpa_cache_weights(q, *args[:2], i32([5]), None, lse, buf, buf, **kw)
    with pytest.raises(ValueError):                     # rows of unlike lengths
        lib.sdpa_cache_weights(q, *args[:2], i32([5]), None, lse, buf, torch.zeros((1, 1, 60), device=DEV))
    with pytest.raises(lib.SdpaError):                  # sums that overlap the old ones
        both = torch.zeros(60, device=DEV)
        lib.sdpa_cache_weights(q, *args[:2], i32([5]), None, lse, both[:48].view(1, 1, 48), both[12:].view(1, 1, 48))


# -------------------------------------------------------------- serving loop --

@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(gpu, graph):  # noqa: F811
    """Prompts are appended, their weights summed, the cache is brought down, and decoding goes on over what stayed,
    the last steps with a window: each step against the plain definition on the cache's own values."""
    import scaled_dot_product_05_gb300 as lib
    from tests.test_paged_masks import attention64
    B, Hq, Hkv, D, page, S, budget = 2, 8, 2, 64, 16, 100, 48
    cache = lib.PagedCache.empty(40, page, Hkv, D, device=DEV)
    table = torch.arange(14, dtype=torch.int32).reshape(2, 7)
    table2 = torch.arange(14, 14 + 8, dtype=torch.int32).reshape(2, 4)
    g = torch.Generator().manual_seed(0)
    x = {n: torch.randn((B, S + 3, h, D), generator=g).bfloat16().to(DEV) for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    zero, count = i32([0, 0]), i32([S, S - 31])
    lse = torch.full((B, Hq, S), math.nan, device=DEV)
    score = torch.zeros((B, Hkv, 7 * page), device=DEV)
    kept = torch.zeros((B, Hkv, budget), dtype=torch.int32, device=DEV)
    kept_score = torch.zeros((B, Hkv, 4 * page), device=DEV)
    small = torch.zeros((B, Hkv, budget), device=DEV)
    o = [torch.zeros((B, 1, Hq, D), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    lse1 = [torch.zeros((B, Hq, 1), device=DEV) for _ in range(3)]
    t, t2 = table.to(DEV), table2.to(DEV)
    prompt = {n: v[:, :S].contiguous() for n, v in x.items()}
    step = [{n: v[:, S + i:S + i + 1].contiguous() for n, v in x.items()} for i in range(3)]
    at = [torch.minimum(count, i32([budget])) + i for i in range(3)]
    ones = i32([1, 1])

    def run():
        lib.sdpa_cache_append(prompt["k"], prompt["v"], cache, t, zero, count)
        lib.sdpa_fwd_paged(prompt["q"], cache, t, zero, count, None, lse)
        lib.sdpa_cache_weights(prompt["q"], cache, t, zero, count, lse, None, score)
        lib.sdpa_cache_evict(cache, t, count, score, t2, budget=budget, sinks=2, recent=8, kept=kept, kept_score=small)
        kept_score[:, :, :budget] = small
        for i in range(3):
            lib.sdpa_cache_append(step[i]["k"], step[i]["v"], cache, t2, at[i], ones)
            if i < 2:
                lib.sdpa_fwd_paged(step[i]["q"], cache, t2, at[i], ones, o[i], lse1[i])
                lib.sdpa_cache_weights(step[i]["q"], cache, t2, at[i], ones, lse1[i], kept_score, kept_score)
            else:
                lib.sdpa_fwd_paged_window(step[i]["q"], cache, t2, at[i], ones, o[i], lse1[i], window=20, sinks=2)
    if graph:
        run()
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            run()
        for v in (lse, score, kept, kept_score, *o, *lse1):
            v.zero_()
        cg.replay()
        cg.replay()
    else:
        run()
    assert lib.sdpa_device_error() == 0
    plain = PlainCache(cache)
    sums = score.cpu().double()
    for b, n in enumerate(count.tolist()):
        k = plain.rows(0, table[b].long(), n)
        seen = torch.ones(n, n, dtype=torch.bool).tril()
        want, tol = weights64(prompt["q"][b, :n].cpu().double(), k, lse[b, :, :n].cpu().double(), seen, D ** -0.5)
        assert ((sums[b, :, :n] - want).abs() <= tol).all()
        m = min(n, budget)
        total = torch.zeros((Hkv, m + 3), dtype=torch.float64)
        for h in range(Hkv):
            stays = pick(score[b, h].tolist(), n, budget, 2, 8)
            assert kept[b, h, :m].tolist() == stays
            total[h, :m] = score[b, h, stays].cpu().double()
            for which in (0, 1):        # the values that stay are those of the old pages, to half a step of E4M3
                old = plain.rows(which, table[b].long(), n)[stays, h]
                new = plain.rows(which, table2[b].long(), m)[:, h]
                assert ((old - new).abs() <= 2.0 ** -4 * old.abs() + 2.0 ** -10 * 2 ** -4).all()
        tol_sum = torch.zeros_like(total)
        for i in range(3):
            e = m + i + 1
            # (pages' scales may have grown since: what they hold now is what the last step read)
            k, v = (plain.rows(w, table2[b].long(), e) for w in (0, 1))
            j = torch.arange(e)
            seen = (torch.ones(1, e, dtype=torch.bool) if i < 2 else ((j > e - 1 - 20) | (j < 2))[None])
            q = step[i]["q"][b].cpu().double()
            ref, z, spread, mag, _ = attention64(q, k, v, seen, D ** -0.5)
            if i == 2:
                ds = 2.0 ** -17 * mag + 1e-6
                tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * ds.T[..., None]) * spread + 2.0 ** -25
                assert ((o[i][b].cpu().double() - ref).abs() <= tol).all()
                assert ((lse1[i][b].cpu().double() - z).abs() <= ds + 2.0 ** -22 * z.abs()).all()
            else:
                w, t_ = weights64(q, k, lse1[i][b].cpu().double(), seen, D ** -0.5)
                total[:, :e] += w
                tol_sum[:, :e] += t_ + 2.0 ** -22 * total[:, :e] + 2.0 ** -4 * w    # (a scale that grew since: half a step)
        assert ((kept_score[b, :, :m + 2].cpu().double() - total[:, :m + 2]).abs() <= tol_sum[:, :m + 2] + 1e-6).all()
