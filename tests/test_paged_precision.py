"""How exactly sdpa_fwd_paged holds its weights and queries, and the kernel
instances of the attention and of the append that tests/test_paged_cache.py
does not reach.

Tolerances.  A weight exp(s - m) v_scale is rounded to f16 once: half a step,
2^-11 of itself, or half of the smallest step 2^-24 where it is subnormal, with the row's
largest weight at 2^11 at least (16 rows of a KV head or fewer) or 2^7 (more).
The products are summed in fp32: 32 keys a step, n / 32 steps of 2^-23, and
2^-16 for the sum of the weights and the exponential.  A score is off by 2^-17
of its summed magnitudes (fp32, D = 128); the output rounds once."""
import math

import pytest
import torch

from tests.test_paged_cache import (DEV, DT, HALF, PlainCache, attention64, gpu, i32, launch, make_cache,  # noqa: F401
                                    tables)
from tests.test_paged_cache import test_append as append_case

WEIGHT = 2.0 ** -11


def floor_of(rows):
    """Half of f16's smallest step over the largest weight, by the rows of a KV head."""
    return 2.0 ** -36 if rows <= 16 else 2.0 ** -32


# Sq with 4 query heads a KV head: 4, 16 and 32 rows
@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0.0, 0.5])
@pytest.mark.parametrize("depth", [9, 12, 14, 15, 17])
@pytest.mark.parametrize("dt,D,Sq", [("bf16", 128, 1), ("bf16", 64, 4), ("bf16", 128, 4), ("bf16", 128, 8),
                                     ("fp16", 128, 1), ("fp16", 64, 1), ("fp16", 128, 4), ("fp16", 64, 8)])
def test_small_weights_below_a_sink_without_a_value(gpu, dt, D, Sq, depth, spread):
    """One token far above the others whose value is zero: the output is the others' alone, however small their weights.
    All values are positive, so the bound is one relative to the output.  More items than CTAs, so that one CTA holds
    the sink and thousands of the others under one maximum (they share their pages, as requests with a common prefix)."""
    B, Hkv, G, page, n = 40, 8, 4, 64, 8192
    n_pages = n // page
    cache = make_cache(n_pages, page, Hkv, D, "heads", filled=False)
    g = torch.Generator().manual_seed(depth)
    for codes, scale, positive in ((cache.k, cache.k_scale, False), (cache.v, cache.v_scale, True)):
        x = torch.randn((n_pages, page, Hkv, D), generator=g)
        x = x.abs() if positive else x
        x[:, :, :, 0] *= 0 if not positive else 1
        c = (x * 64).clamp(-448, 448)
        if positive:
            c[0, 5] = 0
        else:
            c[0, 5] = 0
            c[0, 5, :, 0] = 448                         # the sink's key
        codes.view(torch.uint8).copy_(c.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV))
        scale.fill_(2.0 ** -6)
    q = (spread * torch.randn((B, Sq, G * Hkv, D), generator=g)).to(DT[dt])
    q[..., 0] = depth * math.sqrt(D) / 7                # times 448 / 64: its score is `depth`, the others' about 0
    table = torch.arange(n_pages, dtype=torch.int32).expand(B, -1).contiguous()
    case = (page, G * Hkv, Hkv, D, Sq, dt, "heads", True, [n - Sq] * B, None, None)
    o, lse = launch(case, cache, table, q)
    plain = PlainCache(cache)
    k, v = plain.rows(0, table[0].long(), n), plain.rows(1, table[0].long(), n)
    for b in (0, 17, 39):
        ref, z, total, mag, floor = attention64(q[b].double(), k, v, n - Sq, True, n, 1 / math.sqrt(D))
        ds = 2.0 ** -17 * mag + 1e-6
        steps = n / 32 * 2.0 ** -23 + 2.0 ** -16
        tol = (HALF[dt] + WEIGHT + steps + 2 * ds.T[..., None]) * ref + floor_of(G * Sq) * floor + 2.0 ** -25
        err = (o[b].cpu().double() - ref).abs()
        assert (err <= tol).all(), (b, (err / ref).max().item())
        assert ((lse[b].cpu().double() - z).abs() <= ds + 2.0 ** -22 * z.abs()).all()


# page, Hq, Hkv, D, Sq, dtype, layout, causal, starts, counts, scale
READS = [
    (64, 8, 2, 128, 1, "fp16", "tokens", True, [0, 63, 64, 2047, 5000, 129], None, None),
    (16, 4, 1, 128, 1, "bf16", "heads", True, [0, 15, 16, 127, 128, 1000], None, None),
    # 1 to 8 rows, D = 64
    (128, 16, 16, 64, 1, "fp16", "heads", True, [0, 127, 128, 4000], None, None),
    (16, 4, 2, 64, 4, "fp16", "pairs", True, [0, 13, 124, 700, 2], [4, 4, 3, 4, 0], 0.2),
    (64, 8, 1, 64, 1, "bf16", "tokens", False, [0, 63, 300, 1025], None, None),
    # 9 to 16 rows
    (64, 16, 4, 128, 4, "bf16", "heads", True, [0, 60, 125, 2047, 5], [4, 4, 4, 3, 0], None),
    (32, 16, 1, 128, 1, "fp16", "tokens", True, [0, 31, 127, 128, 3000], None, None),
    (16, 6, 2, 128, 3, "fp16", "pairs", True, [0, 14, 126, 513], [3, 3, 2, 3], 0.11),
    (16, 9, 1, 128, 1, "bf16", "heads", False, [0, 77, 400], None, None),
    (32, 12, 4, 64, 4, "bf16", "heads", True, [0, 30, 124, 1500], [4, 1, 4, 4], None),
    (128, 10, 2, 64, 3, "fp16", "tokens", False, [0, 126, 2000], None, None),
    # 17 rows and more
    (64, 17, 1, 64, 1, "bf16", "heads", True, [0, 63, 128, 900], None, None),
    (32, 32, 1, 128, 1, "fp16", "heads", True, [0, 31, 1000, 127], None, None),
    (64, 16, 2, 128, 16, "fp16", "tokens", True, [0, 120, 2000], [16, 16, 9], None),
    (64, 8, 2, 128, 33, "bf16", "pairs", False, [0, 200, 95], [33, 32, 1], None),
    (128, 6, 2, 64, 200, "fp16", "heads", True, [0, 56, 700, 57, 128, 1], [200, 200, 143, 1, 200, 64], None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", READS, ids=lambda c: "-".join(map(str, c[:8])))
def test_weights_of_eleven_bits(gpu, case):
    """Every instance of the kernels, with the bound of f16 weights for both types."""
    page, Hq, Hkv, D, Sq, dt, layout, causal, start, count, scale = case
    B, width = len(start), (max(start) + Sq) // page + 2
    cache = make_cache(B * width + 5, page, Hkv, D, layout, 19)
    table = tables(B * width + 5, B, width, 20)
    q = torch.randn((B, Sq, Hq, D), generator=torch.Generator().manual_seed(21)).to(DT[dt])
    o, lse = launch(case, cache, table, q)
    plain = PlainCache(cache)
    apart = (plain.scale[1].max() / plain.scale[1].min()).item()       # v_scale is part of a weight
    for b in range(B):
        n = Sq if count is None else count[b]
        total = start[b] + n
        if n:
            pages = table[b, :-(-total // page)].long()
            ref, z, spread, mag, floor = attention64(q[b, :n].double(), plain.rows(0, pages, total),
                                                     plain.rows(1, pages, total), start[b], causal, total,
                                                     scale or 1 / math.sqrt(D))
            ds = 2.0 ** -17 * mag + 1e-6
            steps = total / 32 * 2.0 ** -23 + 2.0 ** -16
            tol = (HALF[dt] * ref.abs() + (WEIGHT + steps + 2 * ds.T[..., None]) * spread +
                   floor_of(Sq * (Hq // Hkv)) * apart * floor + 2.0 ** -25)
            err = (o[b, :n].cpu().double() - ref).abs()
            assert (err <= tol).all(), (b, (err / tol).max().item())
            assert ((lse[b, :, :n].cpu().double() - z).abs() <= ds + 2.0 ** -22 * z.abs()).all(), b
        assert (o[b, n:] == 7).all() and (lse[b, :, n:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [1, 4, 40])
@pytest.mark.parametrize("shift", [70, 100, -70, -90])
def test_large_and_small_queries(gpu, Sq, shift):
    """bf16 reaches to 2^127: queries times a power of two and the scale by its inverse is the same attention, bit for
    bit."""
    case = (16, 8, 2, 128, Sq, "bf16", "heads", True, [0, 100, 700], None, 0.1)
    cache = make_cache(150, 16, 2, 128, "heads", 3)
    table = tables(150, 3, 50, 2)
    q = torch.randn((3, Sq, 8, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    ref = launch(case, cache, table, q)
    far = q * 2.0 ** shift
    assert torch.equal(far * 2.0 ** -shift, q)
    o, lse = launch(case[:10] + (0.1 * 2.0 ** -shift,), cache, table, far)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("Sq", [1, 4, 40])
def test_queries_with_one_large_channel(gpu, dt, Sq):
    """A channel 2^8 above the others, at which the keys are zero: the scores are the others' alone.  A query's element
    is held exactly, or within 2^-14 where its row's largest is above 224: 2^-21 of the largest.  Non-causal and one key each, so
    that the log-sum-exp is the score."""
    B, Hq, Hkv, D, page = 48, 8, 2, 128, 16
    cache = make_cache(B, page, Hkv, D, "heads", 3)
    cache.k.view(torch.uint8)[..., 7] = 0
    q = torch.randn((B, Sq, Hq, D), generator=torch.Generator().manual_seed(5))
    q[..., 7] = 768
    q = q.to(DT[dt])
    table = torch.arange(B, dtype=torch.int32)[:, None]
    # positions 1 - Sq .. 0: keys 0 .. 0
    case = (page, Hq, Hkv, D, Sq, dt, "heads", False, [1 - Sq] * B, None, None)
    o, lse = launch(case, cache, table, q)
    k = PlainCache(cache).rows(0, torch.arange(B), B * page).reshape(B, page, Hkv, D)[:, 0].repeat_interleave(Hq // Hkv, 1)
    s = torch.einsum("bihd,bhd->bhi", q.double(), k) / math.sqrt(D)
    mag = torch.einsum("bihd,bhd->bhi", q.double().abs(), k.abs()) / math.sqrt(D)
    tol = 2.0 ** -17 * mag + 2.0 ** -21.8 * 768 * k.abs().sum(-1)[..., None] / math.sqrt(D) + 1e-6
    err = (lse.cpu().double() - s).abs()
    assert (err <= tol).all(), (err / tol).max().item()


# page, Hkv, D, S, rot, interleaved, dtype, layout, starts, counts: four rows a lane group and unit
@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    (64, 2, 128, 200, 128, False, "bf16", "heads", [0, 5, 63, 64, 100], [200, 199, 65, 1, 0]),
    (64, 2, 128, 200, 64, True, "fp16", "tokens", [0, 5, 63, 64, 100], [200, 199, 65, 1, 2]),
    (64, 1, 128, 130, 128, False, "fp16", "pairs", [0, 1], None),
    (64, 1, 128, 130, 128, True, "bf16", "heads", [3, 63], None),
    (128, 2, 64, 300, 64, True, "bf16", "pairs", [0, 127, 129, 1], [300, 129, 127, 4]),
    (128, 2, 64, 300, 64, False, "fp16", "heads", [0, 127, 129, 1], [300, 129, 127, 4]),
    (32, 2, 128, 70, 0, False, "fp16", "heads", [0, 31, 17], None),
], ids=lambda c: "-".join(map(str, c[:8])))
def test_append_instances(gpu, case):
    append_case(gpu, case)
