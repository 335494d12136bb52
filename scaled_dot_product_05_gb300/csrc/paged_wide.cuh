// paged_wide.cuh -- attention over a paged 8-bit cache for many rows: chunks
// of prompts, drafts under many query heads a KV head (see paged_attn.cuh
// for the definition, and for the few rows of a decoding step).
//
// Here the rows (token, query head) of one KV head are the M side, 128 at a
// time, and a softmax thread has one row:
//     S[128 rows][128 keys] = Q K8^T          FP8, q in two or three 8-bit parts
//     O[128 rows][D] += W V                   f16, W = exp(s - m) v_scale
// The weights keep 11 bits: they are rounded to f16 (weight 1 as 2^7, the
// smallest step 2^-31 of that) and stay in tensor memory, and V's codes are
// turned into f16, which holds them exactly, by two warps of their own.  The
// two softmax warpgroups take alternate key tiles of the same rows, each with
// its own maxima, sums and accumulator, joined when the item is done, and
// issue their own W V; the
// scores of both go through one region of tensor memory, which is free for
// the next tile's as soon as they are read.  Bound by the tensor cores (128 x
// 128 x D FP8 products for each part of q and the f16 product: 1056 cycles a
// tile at D = 128 and bf16) and the exponentials (1024 cycles); measured 2000
// cycles a tile, the tensor pipe 33% busy: 2 chunks of 512 tokens behind up to
// 8192 keys (32 query heads on 8 of 128) 104 us and 13.5 us for the join.  What
// is between is the warpgroups' own chain (scores, maximum, weights, the wait
// for the product to be taken) and some 15 000 cycles for each change of piece.
#pragma once

#include "paged_attn.cuh"

namespace sdpa {
namespace paged {

constexpr int kWideRows = 128;
constexpr float kWideLag = 8.0f;           // a weight may reach 2^8 before the maximum moves
constexpr float kWideLog2W = 7.0f;         // weight 1 is held as 2^7: 2^15 at most

template <int D, bool kBF16>
struct WideLayout {
    static constexpr int kParts = kBF16 ? 2 : 3;
    static constexpr int kThreads = 384;   // 8 softmax warps; TMA producer, S issuer, 2 converters
    static constexpr int kTileBytes = kTileKeys * D;            // 8-bit K or V tile, a part of Q
    static constexpr int kV16Bytes = kTileKeys * D * 2;
    static constexpr int kStagesK = D == 64 ? 4 : 3;
    static constexpr int kStagesV = D == 64 ? 4 : 2;
    static constexpr int kPageBufs = 4;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kParts * kTileBytes;
    static constexpr int kOffV8 = kOffK + kStagesK * kTileBytes;
    static constexpr int kOffV16 = kOffV8 + kStagesV * kTileBytes;
    static constexpr int kOffPages = kOffV16 + 2 * kV16Bytes;   // [kPageBufs][8] float4: scales of 16 keys each
    static constexpr int kOffRows = kOffPages + kPageBufs * 8 * 16;     // [2][128] maxima and [2][128] sums; [D] NaN; any NaN
    static constexpr int kOffBar = kOffRows + 4 * (4 * kWideRows + D + 4);
    static constexpr int kBarBytes = 640;
    static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory budget");
    static constexpr uint32_t kTmemCols = 512;                  // S at 0; of warpgroup g: W at 128 + 64 g, O at 256 + 128 g
};

template <int NK, int NV>
struct WideBarriers {
    uint64_t k_full[NK], k_empty[NK], v_full[NV], v_empty[NV];
    uint64_t v16_full[2], v16_empty[2];    // converted V tile written / multiplied
    uint64_t pages_full[4], pages_free[4]; // a tile's scales written / read
    uint64_t s_full[2], s_free[2], w_full[2], pv_done[2];
    uint64_t q_full, drain[3];             // drain: one for each issuing thread
    uint32_t tmem_base;
    int abort;
    long long total, x, x_first;
    long long warp_sums[12];
    // the piece at hand, kept here while the softmax threads' registers hold
    // their scores
    Piece piece;
    Item item;
};

template <int D, bool kBF16>
__global__ void __launch_bounds__(384, 1)
paged_wide_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p)
{
    using L = WideLayout<D, kBF16>;
    constexpr int NK = L::kStagesK, NV = L::kStagesV, QP = L::kParts, NR = kWideRows;
    constexpr uint32_t kBarSoftmax = 1;
    using Bars = WideBarriers<NK, NV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    auto* bars = reinterpret_cast<Bars*>(smem + L::kOffBar);
    static_assert(sizeof(Bars) <= L::kBarBytes, "barrier block");
    volatile int* abort = &bars->abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint32_t sQ = smem_u32(smem + L::kOffQ), sK = smem_u32(smem + L::kOffK);
    const uint32_t sV8 = smem_u32(smem + L::kOffV8), sV16 = smem_u32(smem + L::kOffV16);
    float4* pages = reinterpret_cast<float4*>(smem + L::kOffPages);
    float* row_max = reinterpret_cast<float*>(smem + L::kOffRows);          // [2][128]
    float* row_sum = row_max + 2 * NR;                                      // [2][128]
    int* nan_at = reinterpret_cast<int*>(row_sum + 2 * NR);                 // [D]: first masked key with a NaN there
    int* any_nan = nan_at + D;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(smem_u32(&bars->k_full[i]), 1);
            mbar_init(smem_u32(&bars->k_empty[i]), 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(smem_u32(&bars->v_full[i]), 1);
            mbar_init(smem_u32(&bars->v_empty[i]), 64);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars->v16_full[i]), 64);
            mbar_init(smem_u32(&bars->v16_empty[i]), 1);
            mbar_init(smem_u32(&bars->s_full[i]), 1);
            mbar_init(smem_u32(&bars->s_free[i]), 128);
            mbar_init(smem_u32(&bars->w_full[i]), 128);
            mbar_init(smem_u32(&bars->pv_done[i]), 1);
        }
        for (int i = 0; i < L::kPageBufs; ++i) {
            mbar_init(smem_u32(&bars->pages_full[i]), 8);
            mbar_init(smem_u32(&bars->pages_free[i]), 128 + 64);
        }
        mbar_init(smem_u32(&bars->q_full), 256);
        for (int i = 0; i < 3; ++i)
            mbar_init(smem_u32(&bars->drain[i]), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(&bars->tmem_base), L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;
    grid_dependency_wait();
    grid_launch_dependents();
    find_share<NR, L::kThreads>(p, blockIdx.x, bars);

    Piece w;
    bool more = first_piece<NR>(p, bars, w);
    if (warp >= 8) {
        regs_release<104>();
        if (warp == 8) {
            // ========================= TMA producer =========================
            // as in paged_attn_kernel: lane i brings page i of a tile; and lane
            // i < 8 lays out the scales of the tile's keys 16 i .. 16 i + 15
            if (lane == 0 && blockIdx.x > 0)
                p.joins[blockIdx.x] = more ? join_of<NR>(p, bars->total, w) : make_int4(0, 0, 0, 0);
            const int ppt = kTileKeys >> p.page_shift;
            uint32_t n = 0;
            bool ok = true;
            for (; ok && more; more = next_piece<NR>(p, w)) {
                const Item it = item_of<NR>(p, w);
                auto entry_of = [&](int tile) -> int {
                    const int ord = tile * ppt + lane;
                    return lane < ppt && tile < w.end && ord << p.page_shift < it.keys
                               ? p.table[(long long)it.b * p.max_pages + ord]
                               : -1;
                };
                int ahead0 = entry_of(w.begin), ahead1 = entry_of(w.begin + 1);
                // a part's table entry two tiles ahead, its scales one ahead
                auto part_of = [&](int tile) -> int {
                    const int pos = tile * kTileKeys + lane * 16;
                    return lane < 8 && tile < w.end && pos < it.keys ? p.table[(long long)it.b * p.max_pages + (pos >> p.page_shift)]
                                                                     : INT_MIN;
                };
                auto scales_of = [&](int entry, float& a, float& b) -> bool {
                    a = b = 1.f;
                    const bool in = (unsigned)entry < (unsigned)p.n_pages;
                    if (in) {
                        a = p.k.scale[(long long)entry * p.Hkv + w.h];
                        b = p.v.scale[(long long)entry * p.Hkv + w.h];
                    } else if (entry != INT_MIN) {
                        atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrPage);
                    }
                    return in;
                };
                int entry = part_of(w.begin), entry_next = part_of(w.begin + 1);
                float k_scale, v_scale;
                bool valid_next = scales_of(entry, k_scale, v_scale);
                for (int j = w.begin; ok && j < w.end; ++j, ++n) {
                    const bool valid = valid_next;
                    const float k_now = k_scale;
                    const float v_now = fminf(fmaxf(v_scale, 8.673617379884035e-19f), 1.152921504606847e18f);   // 2^-60 .. 2^60
                    entry = entry_next;
                    entry_next = part_of(j + 2);
                    valid_next = scales_of(entry, k_scale, v_scale);
                    const int id = (unsigned)ahead0 < (unsigned)p.n_pages ? ahead0 : -1;
                    ahead0 = ahead1;
                    ahead1 = entry_of(j + 2);
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * p.page * D;
                    const uint32_t ks = n % NK, vs = n % NV;
                    if (n >= NK)
                        ok = wait_bar(smem_u32(&bars->k_empty[ks]), (n / NK - 1) & 1, abort, kErrPagedLoad);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)
                        break;
                    if (lane == 0)
                        mbar_arrive_expect_tx(smem_u32(&bars->k_full[ks]), bytes);
                    __syncwarp();
                    if (id >= 0)
                        tma_load_4d(sK + ks * L::kTileBytes + lane * p.page * D, &tm_k, smem_u32(&bars->k_full[ks]), 0, w.h, 0, id);
                    const uint32_t pb = n % L::kPageBufs;
                    if (n >= L::kPageBufs)
                        ok = wait_bar(smem_u32(&bars->pages_free[pb]), (n / L::kPageBufs - 1) & 1, abort, kErrPagedLoad + 2);
                    const bool some = __any_sync(0xffffffffu, lane < 8 && !valid);
                    if (ok && lane < 8) {
                        pages[pb * 8 + lane] = make_float4(k_now * p.scale_log2, valid ? __log2f(v_now) : -INFINITY,
                                                           __fdividef(1.f, v_now), some ? 1.f : 0.f);
                        mbar_arrive(smem_u32(&bars->pages_full[pb]));
                    }
                    if (n >= NV)
                        ok = ok && wait_bar(smem_u32(&bars->v_empty[vs]), (n / NV - 1) & 1, abort, kErrPagedLoad + 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)
                        break;
                    if (lane == 0)
                        mbar_arrive_expect_tx(smem_u32(&bars->v_full[vs]), bytes);
                    __syncwarp();
                    if (id >= 0)
                        tma_load_4d(sV8 + vs * L::kTileBytes + lane * p.page * D, &tm_v, smem_u32(&bars->v_full[vs]), 0, w.h, 0, id);
                }
            }
            if (lane == 0) {
                for (uint32_t i = n > NK ? n - NK : 0; i < n; ++i)
                    drain_wait(smem_u32(&bars->k_full[i % NK]), (i / NK) & 1);
                if (!ok)
                    drain_wait(smem_u32(&bars->k_full[n % NK]), (n / NK) & 1);
                for (uint32_t i = n > NV ? n - NV : 0; i < n; ++i)
                    drain_wait(smem_u32(&bars->v_full[i % NV]), (i / NV) & 1);
            }
            __syncwarp();
        } else if (warp == 9) {
            // =========================== S issuer ===========================
            // S of tile j + 1 as soon as the scores of tile j have been read
            if (lane == 0) {
                constexpr uint32_t kSwzCode = D == 128 ? 2u : 4u;
                constexpr uint32_t idesc_s = idesc_make(0u, NR, kTileKeys, false);
                const uint32_t hi = (uint32_t)(smem_desc(0, 16, 8 * D, kSwzCode) >> 32);
                uint32_t ns = 0, pieces = 0, f0 = 0, f1 = 0;       // S issued: all, for each warpgroup
                int prev = -1;                                     // warpgroup of the last S
                bool ok = true;
                for (; ok && more; more = next_piece<NR>(p, w), ++pieces) {
                    ok = wait_bar(smem_u32(&bars->q_full), pieces & 1, abort, kErrPagedMma + 2);
                    for (int j = 0; ok && j < w.end - w.begin; ++j, ++ns) {
                        const int g = j & 1;
                        const uint32_t ks = ns % NK;
                        ok = wait_bar(smem_u32(&bars->k_full[ks]), (ns / NK) & 1, abort, kErrPagedMma) &&
                             (prev < 0 ||
                              wait_bar(smem_u32(&bars->s_free[prev]), ((prev ? f1 : f0) - 1) & 1, abort, kErrPagedMma + 1));
                        if (!ok)
                            break;
                        tc_fence_after_sync();
                        const uint32_t k_lo = ((sK + ks * L::kTileBytes) >> 4) | (1u << 16);
#pragma unroll
                        for (int q = 0; q < QP; ++q) {
                            const uint32_t q_lo = ((sQ + q * L::kTileBytes) >> 4) | (1u << 16);
                            const uint32_t idesc = idesc_s | (q + 1 == QP ? 1u << 7 : 0u);      // q (A): E5M2 in the end
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk)
                                mma_f8_ss(tmem, desc_join(hi, q_lo + 2 * kk), desc_join(hi, k_lo + 2 * kk), idesc,
                                          q > 0 || kk > 0);
                        }
                        mma_commit(smem_u32(&bars->s_full[g]));
                        mma_commit(smem_u32(&bars->k_empty[ks]));
                        f0 += g ? 0 : 1;
                        f1 += g ? 1 : 0;
                        prev = g;
                    }
                }
                mma_commit(smem_u32(&bars->drain[0]));
                drain_wait(smem_u32(&bars->drain[0]), 0);
            }
            __syncwarp();
        } else {
            // ========================== converters ==========================
            // V's codes to f16, 16 at a time, into the layout of a 16-bit tile
            // (64 channels a chunk, 128-byte rows); rows that no row of the item
            // sees are zero, a NaN that only some see is taken out and kept in
            // mind
            const int tid = threadIdx.x - 320;                              // 0 .. 63
            uint32_t n = 0, pieces = 0;
            bool ok = true;
            for (; ok && more; more = next_piece<NR>(p, w), ++pieces) {
                const Item it = item_of<NR>(p, w);
                // the piece before has been read out and its NaN forgotten
                ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->q_full), pieces & 1, abort, kErrPagedSoftmax + 8));
                const long long row0 = p.causal ? it.start + it.r0 / p.group : it.start + it.count - 1;
                const int full = row0 < 0 ? 0 : (int)(row0 + 1 < it.keys ? row0 + 1 : it.keys);
                for (int j = w.begin; ok && j < w.end; ++j, ++n) {
                    const uint32_t b = n & 1, ring = n % NV, pb = n % L::kPageBufs;
                    ok = wait_bar(smem_u32(&bars->pages_full[pb]), (n / L::kPageBufs) & 1, abort, kErrPagedSoftmax + 6);
                    uint32_t valid_parts = 0xffu;
                    if (pages[pb * 8].w != 0.f) {
                        valid_parts = 0;
                        for (int i = 0; i < 8; ++i)
                            valid_parts |= pages[pb * 8 + i].y == -INFINITY ? 0u : 1u << i;
                    }
                    if (n >= 2)
                        ok = ok && wait_bar(smem_u32(&bars->v16_empty[b]), (n / 2 - 1) & 1, abort, kErrPagedSoftmax + 5);
                    ok = ok && wait_bar(smem_u32(&bars->v_full[ring]), (n / NV) & 1, abort, kErrPagedSoftmax + 7);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)
                        break;
                    // this thread's 16 channels c of keys key0, key0 + kStep, ..:
                    // a multiple of 8 apart, so all at one swizzled place
                    constexpr int kPer = D / 16, kStep = 64 / kPer, kTurns = kTileKeys / kStep;
                    const int key0 = tid / kPer, c = tid % kPer;
                    const int at = D == 128 ? c ^ (key0 & 7) : c ^ ((key0 >> 1) & 3);
                    uint8_t* src = smem + L::kOffV8 + ring * L::kTileBytes + key0 * D + at * 16;
                    const uint32_t row = sV16 + b * L::kV16Bytes + (c / 4) * (kTileKeys * 128) + key0 * 128;
                    const uint32_t dst0 = row + (((c % 4) * 2) ^ (key0 & 7)) * 16, dst1 = row + (((c % 4) * 2 + 1) ^ (key0 & 7)) * 16;
                    if ((j + 1) * kTileKeys > full || valid_parts != 0xffu) {
#pragma unroll 4
                        for (int i = 0; i < kTurns; ++i) {
                            const int key = key0 + i * kStep, pos = j * kTileKeys + key;
                            uint4* u = reinterpret_cast<uint4*>(src + i * kStep * D);
                            if (pos >= it.keys || !(valid_parts >> (key / 16) & 1)) {
                                *u = make_uint4(0, 0, 0, 0);
                            } else if (pos >= full) {
                                const uint4 q = *u;
                                auto nans = [](uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };    // 0x7F, 0xFF
                                if (nans(q.x) | nans(q.y) | nans(q.z) | nans(q.w)) {
                                    *any_nan = 1;
                                    for (int e = 0; e < 16; ++e) {
                                        uint8_t* byte = src + i * kStep * D + e;
                                        if ((*byte & 0x7f) == 0x7f) {
                                            atomicMin(&nan_at[16 * c + e], pos);
                                            *byte = 0;
                                        }
                                    }
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int i0 = 0; i0 < kTurns; i0 += 8) {
                        uint4 u[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            u[i] = *reinterpret_cast<const uint4*>(src + (i0 + i) * kStep * D);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t off = (uint32_t)((i0 + i) * kStep * 128);
                            st_shared_v4(dst0 + off, e4m3x2_to_f16x2((uint16_t)u[i].x), e4m3x2_to_f16x2((uint16_t)(u[i].x >> 16)),
                                         e4m3x2_to_f16x2((uint16_t)u[i].y), e4m3x2_to_f16x2((uint16_t)(u[i].y >> 16)));
                            st_shared_v4(dst1 + off, e4m3x2_to_f16x2((uint16_t)u[i].z), e4m3x2_to_f16x2((uint16_t)(u[i].z >> 16)),
                                         e4m3x2_to_f16x2((uint16_t)u[i].w), e4m3x2_to_f16x2((uint16_t)(u[i].w >> 16)));
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(smem_u32(&bars->pages_free[pb]));
                    mbar_arrive(smem_u32(&bars->v_empty[ring]));
                    mbar_arrive(smem_u32(&bars->v16_full[b]));
                }
            }
        }
    } else {
        regs_acquire<192>();
        // ======================== softmax warpgroups ========================
        const int g = warp >> 2;
        const int row = threadIdx.x & 127;                                  // of the tile; TMEM lane
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        constexpr uint32_t idesc_o = idesc_make(0u, NR, D, true);
        const uint32_t hi_v = (uint32_t)(smem_desc(0, 16, 1024, 2u) >> 32);
        constexpr uint32_t kLboV = (uint32_t)((kTileKeys * 128) >> 4) << 16;            // next 64 channels
        const uint32_t t_s = tmem + lanes, t_w = t_s + 128 + 64 * g, t_o = t_s + 256 + 128 * g;
        uint32_t ns = 0;                                                    // tiles of this warpgroup so far
        uint32_t nv = 0;                                                    // tiles of the CTA before this piece
        bool ok = true;
        for (; more; nv += w.end - w.begin, more = next_piece<NR>(p, w)) {
            Item it = item_of<NR>(p, w);
            // ---- q into 8-bit parts: two threads a row, half of its channels each
            float scale;                                                    // of this thread's row in the loop below
            {
                const int r = threadIdx.x >> 1, half = threadIdx.x & 1;
                const bool live = r < it.rows;
                const int i = (it.r0 + r) / p.group, hh = (it.r0 + r) % p.group;
                const uint4* q = reinterpret_cast<const uint4*>(
                    reinterpret_cast<const uint16_t*>(p.Q) + (long long)it.b * p.q_sb + (long long)i * p.q_ss +
                    (long long)(w.h * p.group + hh) * p.q_sh + half * (D / 2));
                uint32_t top = 0;
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint4 u = live ? q[s] : make_uint4(0, 0, 0, 0);
                    float v[8];
                    rope::unpack4<kBF16>(make_uint2(u.x, u.y), v);
                    rope::unpack4<kBF16>(make_uint2(u.z, u.w), v + 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                const float qs = query_scale(top), inv = 1.f / qs;
#pragma unroll 1
                for (int s = 0; s < D / 32; ++s) {         // (rolled: code that runs once an item is fetched anew each time)
                    float v[16];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint4 u = live ? q[2 * s + c] : make_uint4(0, 0, 0, 0);
                        rope::unpack4<kBF16>(make_uint2(u.x, u.y), &v[8 * c]);
                        rope::unpack4<kBF16>(make_uint2(u.z, u.w), &v[8 * c + 4]);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] *= inv;
                    const int seg = half * (D / 32) + s;
                    const int chunk = D == 128 ? seg ^ (r & 7) : seg ^ ((r >> 1) & 3);
#pragma unroll
                    for (int part = 0; part < QP; ++part) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            o[e / 4] = query_part(&v[e], part + 1 == QP);
                        st_shared_v4(sQ + part * L::kTileBytes + r * D + chunk * 16, o[0], o[1], o[2], o[3]);
                    }
                }
                if (half == 0)
                    row_max[r] = top < 0x7f800000u ? qs : NAN;              // handed to the row's own threads
                if (threadIdx.x < D)
                    nan_at[threadIdx.x] = INT_MAX;
                if (threadIdx.x == 0) {
                    bars->piece = w;
                    bars->item = it;
                    *any_nan = 0;
                    if (it.start + it.count > (long long)p.max_pages * p.page)
                        atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrTable);
                }
                fence_proxy_async_smem();
                named_bar_sync(kBarSoftmax, 256);
                scale = row_max[row];
                mbar_arrive(smem_u32(&bars->q_full));
            }
            const int q_row = (it.r0 + row) / p.group;
            const long long last_pos = p.causal ? it.start + q_row : it.start + it.count - 1;
            const int last = row >= it.rows || last_pos < 0 ? -1 : (int)(last_pos < it.keys ? last_pos : it.keys - 1);
            const long long row0 = p.causal ? it.start + it.r0 / p.group : it.start + it.count - 1;
            const int full = row0 < 0 ? 0 : (int)(row0 + 1 < it.keys ? row0 + 1 : it.keys);
            float nmax = kWideLog2W;                                        // 7 - maximum
            float l = 0.f;                                                  // sum of exp2(s - maximum + 7)
            bool seen = false;
            // j counts the piece's tiles
            const int tiles = w.end - w.begin, ahead = full - w.begin * kTileKeys, seen_end = last - w.begin * kTileKeys;
            for (int j = g; j < tiles; j += 2, ++ns) {
                const uint32_t vn = nv + (uint32_t)j, buf = vn % L::kPageBufs;
                ok = ok && wait_bar(smem_u32(&bars->s_full[g]), ns & 1, abort, kErrPagedSoftmax);
                ok = ok && wait_bar(smem_u32(&bars->pages_full[buf]), (vn / L::kPageBufs) & 1, abort, kErrPagedSoftmax + 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after_sync();
                uint32_t r[128];
                tmem_ld128_wait(t_s, t_s + 32, t_s + 64, t_s + 96, r);
                tc_fence_before_sync();
                mbar_arrive(smem_u32(&bars->s_free[g]));
                const bool edge = (j + 1) * kTileKeys > ahead;
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 pg = pages[buf * 8 + c];
                    const float a = scale * pg.x, b = pg.y + nmax;
                    const uint64_t a2 = f32x2(a, a), b2 = f32x2(b, b);
#pragma unroll
                    for (int e = 16 * c; e < 16 * c + 16; e += 2) {
                        float y0, y1;
                        f32x2_split(fma_f32x2(f32x2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), a2, b2), y0, y1);
                        r[e] = __float_as_uint(y0);
                        r[e + 1] = __float_as_uint(y1);
                    }
                }
                // keys that the row does not see, or whose page is none (.w: the
                // tile has such a page), whatever was there
                if (__builtin_expect(edge || pages[buf * 8].w != 0.f, 0)) {
                    const int seen_keys = seen_end - j * kTileKeys;             // of the tile, less one
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int end = pages[buf * 8 + c].y == -INFINITY ? -1 : seen_keys;
#pragma unroll
                        for (int e = 16 * c; e < 16 * c + 16; ++e)
                            r[e] = e > end ? 0xff800000u : r[e];
                    }
                }
                float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
                for (int e = 0; e < 128; e += 8) {
                    m0 = fmax3(m0, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                    m1 = fmax3(m1, __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
                    m2 = fmax3(m2, __uint_as_float(r[e + 4]), __uint_as_float(r[e + 5]));
                    m3 = fmax3(m3, __uint_as_float(r[e + 6]), __uint_as_float(r[e + 7]));
                }
                mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) - kWideLog2W;
                float shift = 0.f, factor = 1.f;
                if (!seen) {
                    if (mx > -INFINITY) {
                        shift = mx;                                         // nothing to rescale before the first key
                        seen = true;
                    }
                } else if (mx > kWideLag) {
                    shift = mx;
                    factor = ex2_approx(-shift);
                }
                if (__builtin_expect(__any_sync(0xffffffffu, shift != 0.f), 0)) {
                    nmax -= shift;
                    l *= factor;
                    const uint64_t s2 = f32x2(-shift, -shift);
#pragma unroll
                    for (int e = 0; e < 128; e += 2) {
                        float y0, y1;
                        f32x2_split(add_f32x2(f32x2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), s2), y0, y1);
                        r[e] = __float_as_uint(y0);
                        r[e + 1] = __float_as_uint(y1);
                    }
                }
                uint32_t pk[64];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint64_t acc = 0;
#pragma unroll
                    for (int e = 16 * c; e < 16 * c + 16; e += 2) {
                        const float y0 = ex2_approx(__uint_as_float(r[e])), y1 = ex2_approx(__uint_as_float(r[e + 1]));
                        acc = add_f32x2(acc, f32x2(y0, y1));
                        pk[e / 2] = f32x2_to_f16x2(y0, y1);
                    }
                    float s0, s1;
                    f32x2_split(acc, s0, s1);
                    l = fmaf(s0 + s1, pages[buf * 8 + c].z, l);
                }
                mbar_arrive(smem_u32(&bars->pages_free[buf]));
                // the product before has updated O
                if (ns > 0)
                    ok = wait_bar(smem_u32(&bars->pv_done[g]), (ns - 1) & 1, abort, kErrPagedSoftmax + 2);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after_sync();
                if (__builtin_expect(j > g && __any_sync(0xffffffffu, factor != 1.f), 0)) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32_wait(t_o + c, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
                        tmem_st32(t_o + c, o);
                    }
                }
                tmem_st32(t_w, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
                tmem_st32(t_w + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
                tmem_st_wait();
                tc_fence_before_sync();
                mbar_arrive(smem_u32(&bars->w_full[g]));
                // O (+)= W V: the warpgroup's first thread issues it when all
                // weights and the tile's V are there
                if (row == 0) {
                    const uint32_t vb = vn & 1;
                    ok = wait_bar(smem_u32(&bars->w_full[g]), ns & 1, abort, kErrPagedMma + 4) &&
                         wait_bar(smem_u32(&bars->v16_full[vb]), (vn / 2) & 1, abort, kErrPagedMma + 3);
                    if (ok) {
                        tc_fence_after_sync();
                        const uint32_t v_lo = ((sV16 + vb * L::kV16Bytes) >> 4) | kLboV;
#pragma unroll
                        for (int kk = 0; kk < kTileKeys / 16; ++kk)
                            mma_f16_ts(tmem + 256 + 128 * g, tmem + 128 + 64 * g + kk * 8,
                                       desc_join(hi_v, v_lo + (uint32_t)((kk * 16 * 128) >> 4)), idesc_o, j > g || kk > 0);
                        mma_commit(smem_u32(&bars->pv_done[g]));
                        mma_commit(smem_u32(&bars->v16_empty[vb]));
                    }
                }
                __syncwarp();
            }
            // ---- the piece's result: both warpgroups' accumulators, a half of the channels each
            w = bars->piece;
            it = bars->item;
            if (ok && g < w.end - w.begin)
                ok = wait_bar(smem_u32(&bars->pv_done[g]), (ns - 1) & 1, abort, kErrPagedSoftmax + 3);
            row_max[g * NR + row] = kWideLog2W - nmax;
            row_sum[g * NR + row] = l;
            ok = named_bar_all(kBarSoftmax, 256, ok);
            if (!ok)
                break;
            tc_fence_after_sync();
            const float l0 = row_sum[row], l1 = row_sum[NR + row];
            const float m0 = l0 == 0.f ? -INFINITY : row_max[row], m1 = l1 == 0.f ? -INFINITY : row_max[NR + row];
            const float m = fmaxf(m0, m1);
            const float f0 = l0 == 0.f ? 0.f : exp2f(m0 - m), f1 = l1 == 0.f ? 0.f : exp2f(m1 - m);
            const float sum = fmaf(l0, f0, l1 * f1);
            const float w0 = sum == 0.f ? 0.f : f0 / sum, w1 = sum == 0.f ? 0.f : f1 / sum;
            const bool whole = w.begin == 0 && w.end == w.n;
            const bool both = w.end - w.begin > 1;                          // warpgroup 1 had a tile
            const long long slot = (long long)blockIdx.x * 2 + (w.begin > 0 ? 0 : 1);
            const long long head = (long long)w.h * p.group + (it.r0 + row) % p.group;
            const int i = (it.r0 + row) / p.group;
            const bool live = row < it.rows;
            if (live && g == 0) {
                const float lse2 = sum == 0.f ? -INFINITY : m + (log2f(sum) - kWideLog2W);
                if (!whole)
                    p.part_lse[slot * NR + row] = lse2;
                else if (p.lse)
                    p.lse[((long long)it.b * p.Hq + head) * p.Sq + i] = lse2 * kLn2;
            }
            const bool nans = *any_nan != 0;
            const long long last_at = p.causal ? it.start + i : it.start + it.count - 1;
            const int last_key = last_at < it.keys ? (int)last_at : it.keys - 1;    // (a negative one is below any)
            uint16_t* out = reinterpret_cast<uint16_t*>(p.O) + (long long)it.b * p.o_sb + (long long)i * p.o_ss + head * p.o_sh;
#pragma unroll 1
            for (int c = g * (D / 2); c < (g + 1) * (D / 2); c += 32) {
                uint32_t a[32], b[32];
                tmem_ld32_wait(t_s + 256 + c, a);
                if (both)
                    tmem_ld32_wait(t_s + 384 + c, b);
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    // (an accumulator that no tile went to is not looked at)
                    o[e] = __uint_as_float(a[e]) * w0;
                    if (both)
                        o[e] = fmaf(__uint_as_float(b[e]), w1, o[e]);
                }
                if (nans) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (last_key >= nan_at[c + e])
                            o[e] = NAN;
                }
                if (live && !whole) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + (slot * NR + row) * D + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                } else if (live) {
                    uint4* dst = reinterpret_cast<uint4*>(out + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[e] = make_uint4(pack2<kBF16>(o[8 * e], o[8 * e + 1]), pack2<kBF16>(o[8 * e + 2], o[8 * e + 3]),
                                            pack2<kBF16>(o[8 * e + 4], o[8 * e + 5]), pack2<kBF16>(o[8 * e + 6], o[8 * e + 7]));
                }
            }
            tc_fence_before_sync();
            named_bar_sync(kBarSoftmax, 256);                  // the rows' numbers and O are read
            tc_fence_after_sync();
        }
        if (row == 0) {                                        // every product that this thread issued has completed
            mma_commit(smem_u32(&bars->drain[1 + g]));
            drain_wait(smem_u32(&bars->drain[1 + g]), 0);
        }
        __syncwarp();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

}  // namespace paged
}  // namespace sdpa
