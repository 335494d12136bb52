// cache_evict.cuh -- brings the sequences of a paged 8-bit cache down to a
// budget: of each sequence and KV head the first `sinks` tokens stay, the last
// `recent`, and of those between the ones with the largest scores (of equal
// ones the earlier), in their order, in pages of their own.
//
// Two kernels.  The first finds the tokens: a CTA (or a cluster, for long
// sequences) has the scores of one sequence and KV head in registers, as keys
// that order like integers, and finds the key of the last token that stays bit
// by bit, counting the keys that reach a candidate: 32 rounds of compares and
// one barrier each, without atomics.  Then the warps, each with consecutive
// positions, number their tokens.  The second moves the codes, a page of the
// new ones a unit: a token's 16-byte pieces wait in registers for the page's
// largest value, then are written under the smallest power of two that holds
// it (the append's rule).  A power of two moves a code exactly, but for those
// that become subnormal.
// Bound by reading and writing the codes that stay.
#pragma once

#include <cooperative_groups.h>

#include "cache_append.cuh"

namespace sdpa {
namespace evict {

struct EvictParams {
    cache::Pool pool[2];
    const int* table;                // [B][max_pages]
    const int* new_table;            // [B][new_max_pages]
    const int* length;               // [B]
    const float* score;              // [B][Hkv][stride]
    int* kept;                       // [B][Hkv][budget]
    float* kept_score;               // the same, or null
    long long stride;
    int B, Hkv, page, page_shift, n_pages, max_pages, new_max_pages;
    int sinks, recent, budget;
    int n_ord;                       // pages that the budget takes
};

// Tokens of sequence b (within its table and its row of scores).
__device__ __forceinline__ int tokens_of(const EvictParams& p, int b)
{
    const long long cap = min((long long)p.max_pages << p.page_shift, p.stride);
    return (int)max(0ll, min((long long)p.length[b], cap));
}

// ------------------------------------------------------------------- select --

constexpr int kSelectThreads = 1024;
constexpr int kSelectKeys = 32;      // keys a thread holds; what is more is read again in every round

// Larger scores have larger keys; both zeros the same one, NaN the largest.  None is 0.
__device__ __forceinline__ uint32_t key_of(float s)
{
    const uint32_t u = __float_as_uint(s + 0.f);
    return s != s ? ~0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads, 1) select_kernel(const EvictParams p)
{
    namespace cg = cooperative_groups;
    constexpr int kWarps = kSelectThreads / 32;
    __shared__ uint32_t warp_count[2][kWarps], cta_count[3], tie_count[kWarps], above_count[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = blockIdx.x / ranks;                // sequence and KV head: the cluster's
    const int b = row / p.Hkv;
    const int n = tokens_of(p, b);
    if (rank == 0 && threadIdx.x == 0 && p.length[b] > n)
        atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrTable);
    const float* score = p.score + (long long)row * p.stride;
    int* kept = p.kept + (long long)row * p.budget;
    float* kept_score = p.kept_score ? p.kept_score + (long long)row * p.budget : nullptr;
    if (n <= p.budget) {                               // (the whole cluster)
        for (int i = rank * kSelectThreads + threadIdx.x; i < n; i += ranks * kSelectThreads) {
            kept[i] = i;
            if (kept_score)
                kept_score[i] = score[i];
        }
        return;
    }
    const int first = p.sinks, last = n - p.recent;    // candidates: first .. last - 1
    const uint32_t room = p.budget - p.sinks - p.recent;       // of which so many stay (fewer than there are)
    // a warp has `turns` times 32 consecutive positions
    const int turns = (n + ranks * kWarps * 32 - 1) / (ranks * kWarps * 32);
    const int pos0 = (rank * kWarps + warp) * turns * 32 + lane;
    auto key_at = [&](int i) -> uint32_t {             // of turn i (0: no candidate)
        const int pos = pos0 + i * 32;
        return pos >= first && pos < last ? key_of(score[pos]) : 0u;
    };
    uint32_t key[kSelectKeys];
#pragma unroll
    for (int i = 0; i < kSelectKeys; ++i)
        key[i] = i < turns ? key_at(i) : 0u;
    // Counts over the cluster, the same in every thread: warps, then CTAs.
    int phase = 0;
    auto total = [&](uint32_t c) -> uint32_t {
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0)
            warp_count[phase & 1][warp] = c;
        __syncthreads();
        c = __reduce_add_sync(0xffffffffu, warp_count[phase & 1][lane]);
        if (ranks > 1) {
            if (threadIdx.x == 0)
                cta_count[phase % 3] = c;
            cluster.sync();
            c = lane < ranks ? *cluster.map_shared_rank(&cta_count[phase % 3], lane) : 0u;
            c = __reduce_add_sync(0xffffffffu, c);
        }
        ++phase;
        return c;
    };
    auto count_from = [&](uint32_t t) -> uint32_t {    // this thread's keys that reach t
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < kSelectKeys; ++i)
            c += key[i] >= t ? 1u : 0u;
        for (int i = kSelectKeys; i < turns; ++i)
            c += key_at(i) >= t ? 1u : 0u;
        return c;
    };
    // the largest key that `room` candidates reach
    uint32_t limit = 0;
    if (room > 0) {
#pragma unroll 1
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t t = limit | 1u << bit;
            if (total(count_from(t)) >= room)
                limit = t;
        }
    }
    const uint32_t above = room == 0 || limit == ~0u ? 0u : total(count_from(limit + 1));
    const uint32_t ties = room - above;                // so many of the keys that are the limit, from the first on
    // ---- tokens before each warp's: those that stay whatever the ties, and ties
    uint32_t mine_above = 0, mine_ties = 0;
    auto sort_out = [&](int i, uint32_t k, bool& stays, bool& tie) {
        const int pos = pos0 + i * 32;
        stays = pos < n && (pos < first || pos >= last || (room > 0 && k > limit));
        tie = room > 0 && k == limit;                  // (limit is a candidate's key, so not 0)
    };
#pragma unroll
    for (int i = 0; i < kSelectKeys; ++i) {
        bool stays, tie;
        sort_out(i, key[i], stays, tie);
        mine_above += stays && i < turns;
        mine_ties += tie;
    }
    for (int i = kSelectKeys; i < turns; ++i) {
        bool stays, tie;
        sort_out(i, key_at(i), stays, tie);
        mine_above += stays;
        mine_ties += tie;
    }
    mine_above = __reduce_add_sync(0xffffffffu, mine_above);
    mine_ties = __reduce_add_sync(0xffffffffu, mine_ties);
    if (lane == 0) {
        above_count[warp] = mine_above;
        tie_count[warp] = mine_ties;
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();
    uint32_t a = 0, t = 0;
    for (int r = 0; r <= rank; ++r) {
        const uint32_t ca = cluster.map_shared_rank(above_count, r)[lane], ct = cluster.map_shared_rank(tie_count, r)[lane];
        const bool before = r < rank || lane < warp;
        a += __reduce_add_sync(0xffffffffu, before ? ca : 0u);
        t += __reduce_add_sync(0xffffffffu, before ? ct : 0u);
    }
    // ---- the tokens, numbered
    auto write = [&](int i, uint32_t k) {
        const int pos = pos0 + i * 32;
        bool stays, tie;
        sort_out(i, k, stays, tie);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t m_ties = __ballot_sync(0xffffffffu, tie), m_stays = __ballot_sync(0xffffffffu, stays);
        const uint32_t tie_rank = t + __popc(m_ties & below);
        if (stays || (tie && tie_rank < ties)) {
            const uint32_t at = a + __popc(m_stays & below) + min(tie_rank, ties);
            kept[at] = pos;
            if (kept_score)
                kept_score[at] = score[pos];
        }
        a += __popc(m_stays);
        t += __popc(m_ties);
    };
#pragma unroll
    for (int i = 0; i < kSelectKeys; ++i)
        if (i < turns)
            write(i, key[i]);
    for (int i = kSelectKeys; i < turns; ++i)
        write(i, key_at(i));
    if (ranks > 1)
        cluster.sync();                                // (no CTA leaves while another reads its counts)
}

// --------------------------------------------------------------------- move --

constexpr int kMoveThreads = 256;

// kUnit threads a unit, kPasses 16-byte pieces a thread.
template <int D, int kUnit, int kPasses>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p)
{
    constexpr int kPieces = D / 16;                    // of a token
    constexpr int kUnits = kMoveThreads / kUnit;
    __shared__ float warp_max[kMoveThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    // unit -> (KV head fastest, K or V, new page, sequence)
    const int tid = threadIdx.x % kUnit;
    const uint32_t unit = blockIdx.x * kUnits + threadIdx.x / kUnit;
    uint32_t rest = unit / (uint32_t)p.Hkv;
    const int h = (int)(unit - rest * p.Hkv);
    const int kv = (int)(rest & 1);
    rest >>= 1;
    const int b = (int)(rest / (uint32_t)p.n_ord);
    const int ord = (int)(rest - b * p.n_ord);
    int rows = 0, to = -1;                             // tokens of the page, and the page
    if (b < p.B) {
        rows = max(0, min(p.page, min(tokens_of(p, b), p.budget) - (ord << p.page_shift)));
        if (rows > 0) {
            to = p.new_table[(long long)b * p.new_max_pages + ord];
            if ((unsigned)to >= (unsigned)p.n_pages) {
                if (tid == 0)
                    atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrPage);
                rows = 0;
            }
        }
    }
    const cache::Pool pool = p.pool[kv];
    uint4 u[kPasses];
    float scale[kPasses];
    float amax = 0.f;
    const int* kept = p.kept + ((long long)b * p.Hkv + h) * p.budget + ((long long)ord << p.page_shift);
    int from[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = (tid + i * kUnit) / kPieces;
        from[i] = r < rows ? kept[r] : -1;
    }
    int entry[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
        entry[i] = from[i] >= 0 ? p.table[(long long)b * p.max_pages + (from[i] >> p.page_shift)] : 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        u[i] = make_uint4(0, 0, 0, 0);
        scale[i] = 1.f;
        if (from[i] >= 0) {
            if ((unsigned)entry[i] < (unsigned)p.n_pages) {
                scale[i] = pool.scale[(long long)entry[i] * p.Hkv + h];
                u[i] = *reinterpret_cast<const uint4*>(pool.codes + (long long)entry[i] * pool.sp +
                                                       (long long)(from[i] & (p.page - 1)) * pool.ss + (long long)h * pool.sh +
                                                       (tid + i * kUnit) % kPieces * 16);
            } else {                                   // a token whose page is none is zero
                atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrPage);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        // the largest code: magnitudes order like integers, NaN (0x7F) left out
        uint32_t m = 0;
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t v = w[k] & 0x7f7f7f7fu;
            m = __vmaxu4(m, v & ~__vcmpeq4(v, 0x7f7f7f7fu));
        }
        m = max(max(m & 0xff, m >> 8 & 0xff), max(m >> 16 & 0xff, m >> 24));
        amax = fmaxf(amax, f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)m)).x * scale[i]);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    if constexpr (kUnit > 32) {
        if ((threadIdx.x & 31) == 0)
            warp_max[threadIdx.x >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kUnit / 32; ++i)
            amax = fmaxf(amax, warp_max[threadIdx.x / kUnit * (kUnit / 32) + i]);
    }
    if (rows == 0)
        return;
    const float fresh = cache::pow2_scale(amax), inv = 1.f / fresh;
    if (tid == 0)
        pool.scale[(long long)to * p.Hkv + h] = fresh;
    uint8_t* dst = pool.codes + (long long)to * pool.sp + (long long)h * pool.sh;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int at = tid + i * kUnit;
        if (from[i] < 0)
            continue;
        const float f = scale[i] * inv;                // (exact: inv is a power of two)
        if (f != 1.f) {
            uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)w[k]));
                const float2 y = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[k] >> 16)));
                w[k] = (uint32_t)f32x2_to_e4m3x2(x.x * f, x.y * f) | ((uint32_t)f32x2_to_e4m3x2(y.x * f, y.y * f) << 16);
            }
            u[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4*>(dst + (long long)(at / kPieces) * pool.ss + at % kPieces * 16) = u[i];
    }
}

}  // namespace evict
}  // namespace sdpa
