// paged_attn.cuh -- attention over a paged 8-bit cache.
//
// Token i of sequence b (i < count[b]) stands at position start[b] + i, the
// position at which the append put its key and value, and sees keys
// 0 .. start[b] + i (causal) or 0 .. start[b] + count[b] - 1.  A cached value
// is code * scale[page][KV head]:
//     s_j = scale * k_scale(page of j) * (q . k8_j),
//     O = sum_j exp(s_j - m) v_scale(page of j) v8_j / sum_j exp(s_j - m).
// A row that sees no key gives O = 0 and LSE = -inf.  Rows i >= count[b] are
// not written.  Keys whose page index is outside the pool, or whose position
// is outside the page table, are left out and reported in the device error
// word; no address is formed from such an index.
//
// The codes go to the FP8 tensor cores as they lie in the cache, and the
// 16-bit operands are split instead: q, scaled by a power of two, into E4M3
// parts that add up to it (two hold the 8 bits of bf16, three the 11 of fp16),
// and the weight w_j = exp(s_j - m) v_scale_j into two, the second 16 times as
// large as it counts so that small weights keep their bits (error 2^-8 of a
// weight at most, as rounding it to bf16 would give).  Products of E4M3 values are
// exact in the fp32 accumulator.  Nothing is dequantised, and K and V are
// read once as bytes.
//
// The rows (token, query head) of one KV head are the N side of the products,
// the keys of a tile the M side:
//     S^T[128 keys][rows] = K8 Q^T,   O^T[D][rows] += V8^T W^T,
// so a decoding step's few rows cost few columns and every thread of the
// softmax warpgroup has one key of the tile: its scales, its mask and its
// weights for all rows.
#pragma once

#include "cache_append.cuh"

namespace sdpa {
namespace paged {

struct Params {
    const void* Q;
    void* O;
    float* lse;                      // [B][Hq][Sq], or null
    long long q_sb, q_ss, q_sh, o_sb, o_ss, o_sh;
    cache::Pool k, v;
    const int* table;                // [B][max_pages]
    const int* start;                // [B]
    const int* count;                // [B], or null: Sq
    int B, Sq, Hq, Hkv, group;
    int page, n_pages, max_pages;
    int causal;
    float scale_log2;                // scale * log2(e)
    int row_tiles;                   // tiles of NR rows that Sq * group rows need
    int ctas;                        // CTAs that share the key tiles
    float* part_o;                   // [ctas][2][NR][D]: normalised results of pieces
    float* part_lse;                 // [ctas][2][NR]: their LSE in log2 units
};

enum : unsigned int { kErrPagedLoad = 0x801, kErrPagedMma = 0x811, kErrPagedSoftmax = 0x821 };

constexpr int kTileKeys = 128;
// The running maximum is let behind by up to 2^2 before everything is rescaled
// to a new one, so weights reach 4; times 112 they reach 448, the largest
// E4M3 value.
constexpr float kLag = 2.0f;
constexpr float kLog2W = 6.807354922057604f;   // log2(112)

// Shared memory and TMEM of one CTA: NR rows, QP parts of q.
template <int D, int NR, int QP>
struct PagedLayout {
    static_assert(D == 64 || D == 128, "head dimension");
    static_assert(NR == 16 || NR == 32 || NR == 64, "rows of a tile");
    static constexpr int kThreads = 192;   // 4 softmax warps, TMA producer, MMA issuer
    static constexpr int kTileBytes = kTileKeys * D;            // a K or V tile
    // depth of the rings and of the weights' buffers: what two CTAs fit into an SM
    static constexpr int kStagesK = D == 64 ? 4 : NR == 16 ? 3 : 2;
    static constexpr int kStagesV = D == 64 ? 4 : NR == 64 ? 2 : 3;
    static constexpr int kBufsW = NR == 64 ? 1 : 2;
    static constexpr int kQPartBytes = NR * D;
    static constexpr int kWRow = 2 * NR;                        // bytes of a key's weights: two parts
    static constexpr int kWBytes = kTileKeys * kWRow;
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kStagesK * kTileBytes;
    static constexpr int kOffW = kOffV + kStagesV * kTileBytes;  // at D = 64 also what the unused half of the last
    static constexpr int kOffQ = kOffW + kBufsW * kWBytes;       // V tile's operand reads
    static constexpr int kOffRows = kOffQ + QP * kQPartBytes;    // per-row numbers, see Rows
    static constexpr int kRowsBytes = 4 * (4 * NR + 4 * NR + D); // scale, max, last key, factor; 4 x exchange; NaN
    static constexpr int kOffBar = (kOffRows + kRowsBytes + 15) / 16 * 16;
    static constexpr int kSmemBytes = kOffBar + 512 + 1024;      // barriers, alignment
    static_assert(kOffQ % 1024 == 0 && kOffW % 1024 == 0, "swizzle atoms");
    static_assert(D == 128 || kBufsW * kWBytes + QP * kQPartBytes >= kTileBytes, "operand of the unused half");
    static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
    static constexpr uint32_t kTmemCols = 4 * NR;                // S twice, O (two parts)
    __host__ __device__ static constexpr uint32_t tmem_s(int i) { return i * NR; }
    static constexpr uint32_t kTmemO = 2 * NR;
};

template <int NK, int NV>
struct PagedBarriers {
    uint64_t k_full[NK], k_empty[NK], v_full[NV], v_empty[NV];
    uint64_t s_full[2], s_free[2];         // S^T computed / read out
    uint64_t w_full[2], pv_done[2];        // weights written / multiplied
    uint64_t q_full;                       // q's parts written
    uint64_t o_free;                       // O^T read out
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    // where the CTA's share of the tiles begins
    long long total, x, x_first;
    long long warp_sums[16];
};

// Number of key tiles of entry x = (sequence, row tile): 0 without rows, else
// at least 1.
template <int NR>
__device__ __forceinline__ int entry_tiles(const Params& p, long long x)
{
    const int b = (int)(x / p.row_tiles);
    const long long r0 = (x - (long long)b * p.row_tiles) * NR;
    const int count = p.count ? max(0, min(p.Sq, p.count[b])) : p.Sq;
    const long long rows = (long long)count * p.group;
    if (r0 >= rows)
        return 0;
    const long long last = (rows < r0 + NR ? rows : r0 + NR) - 1;
    const long long cap = (long long)p.max_pages * p.page;
    long long len = (long long)p.start[b] + (p.causal ? last / p.group + 1 : count);
    len = len < cap ? len : cap;
    return len < 1 ? 1 : (int)((len + kTileKeys - 1) / kTileKeys);
}

// First tile of CTA c's share of `total` tiles.  With fewer tiles than CTAs
// the first `total` CTAs have one each, so no share between two others is
// empty.
__device__ __forceinline__ long long share_begin(long long total, int c, int ctas)
{
    if (total < ctas)
        return c < total ? c : total;
    return total / ctas * c + total % ctas * c / ctas;
}

// Whole-block: counts the tiles of all entries (times Hkv each) and finds the
// entry that holds tile share_begin(c).  Entries are taken in order: the
// tiles of entry x are those of KV head 0, then 1, ...
template <int NR, int kThreads, typename Bars>
__device__ __forceinline__ void find_share(const Params& p, int c, Bars* bars)
{
    const long long entries = (long long)p.B * p.row_tiles;
    const long long per = (entries + kThreads - 1) / kThreads;
    const long long x0 = (long long)threadIdx.x * per;
    const long long x1 = x0 + per < entries ? x0 + per : entries;
    long long sum = 0;
    for (long long x = x0; x < x1; ++x)
        sum += (long long)entry_tiles<NR>(p, x) * p.Hkv;
    long long incl = sum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, m);
        if ((threadIdx.x & 31) >= m)
            incl += o;
    }
    if ((threadIdx.x & 31) == 31)
        bars->warp_sums[threadIdx.x >> 5] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long s = bars->warp_sums[w];
        before += w < (int)(threadIdx.x >> 5) ? s : 0;
        total += s;
    }
    long long first = before + incl - sum;
    const long long target = share_begin(total, c, p.ctas);
    if (threadIdx.x == 0)
        bars->total = total;
    if (target >= first && target < first + sum) {
        long long x = x0;
        for (;; ++x) {
            const long long n = (long long)entry_tiles<NR>(p, x) * p.Hkv;
            if (target < first + n)
                break;
            first += n;
        }
        bars->x = x;
        bars->x_first = first;
    }
    __syncthreads();
}

// A CTA's share of the tiles, as pieces: consecutive key tiles of one item
// (entry, KV head).
struct Piece {
    long long x;
    int h, n;                       // n: key tiles of the item
    int begin, end;                 // this piece
    long long left;                 // tiles of the share, this piece included
};

template <int NR, typename Bars>
__device__ __forceinline__ bool first_piece(const Params& p, const Bars* bars, Piece& w)
{
    const int c = blockIdx.x;
    const long long t0 = share_begin(bars->total, c, p.ctas);
    w.left = share_begin(bars->total, c + 1, p.ctas) - t0;
    if (w.left <= 0)
        return false;
    w.x = bars->x;
    w.n = entry_tiles<NR>(p, w.x);
    const long long off = t0 - bars->x_first;
    w.h = (int)(off / w.n);
    w.begin = (int)(off - (long long)w.h * w.n);
    w.end = (int)(w.n - w.begin < w.left ? w.n : w.begin + w.left);
    return true;
}

template <int NR>
__device__ __forceinline__ bool next_piece(const Params& p, Piece& w)
{
    w.left -= w.end - w.begin;
    if (w.left <= 0)
        return false;
    if (++w.h == p.Hkv) {
        w.h = 0;
        do {
            ++w.x;
            w.n = entry_tiles<NR>(p, w.x);
        } while (w.n == 0);
    }
    w.begin = 0;
    w.end = (int)(w.n < w.left ? w.n : w.left);
    return true;
}

// What a piece's item is about.
struct Item {
    int b, count;
    int r0, rows;                   // first row of the tile, valid rows in it
    long long start;
    int keys;                       // keys that some row of the item sees (within the table)
};

template <int NR>
__device__ __forceinline__ Item item_of(const Params& p, const Piece& w)
{
    Item t;
    t.b = (int)(w.x / p.row_tiles);
    t.r0 = (int)(w.x - (long long)t.b * p.row_tiles) * NR;
    t.count = p.count ? max(0, min(p.Sq, p.count[t.b])) : p.Sq;
    t.rows = min(NR, t.count * p.group - t.r0);
    t.start = p.start[t.b];
    const long long cap = (long long)p.max_pages * p.page;
    long long len = t.start + (p.causal ? (t.r0 + t.rows - 1) / p.group + 1 : t.count);
    len = len < 0 ? 0 : len;
    t.keys = (int)(len < cap ? len : cap);
    return t;
}

template <int D, bool kBF16, int NR, int QP>
__global__ void __launch_bounds__(192, 2)
paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p)
{
    using L = PagedLayout<D, NR, QP>;
    constexpr int NK = L::kStagesK, NV = L::kStagesV, NW = L::kBufsW;
    constexpr int kSoftmax = 128;
    constexpr uint32_t kBarSoftmax = 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    auto* bars = reinterpret_cast<PagedBarriers<NK, NV>*>(smem + L::kOffBar);
    static_assert(sizeof(PagedBarriers<NK, NV>) <= 512, "barrier block");
    volatile int* abort = &bars->abort;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t sK = smem_u32(smem + L::kOffK), sV = smem_u32(smem + L::kOffV);
    const uint32_t sW = smem_u32(smem + L::kOffW), sQ = smem_u32(smem + L::kOffQ);

    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(smem_u32(&bars->k_full[i]), 1);
            mbar_init(smem_u32(&bars->k_empty[i]), 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(smem_u32(&bars->v_full[i]), 1);
            mbar_init(smem_u32(&bars->v_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars->s_full[i]), 1);
            mbar_init(smem_u32(&bars->s_free[i]), kSoftmax);
            mbar_init(smem_u32(&bars->w_full[i]), kSoftmax);
            mbar_init(smem_u32(&bars->pv_done[i]), 1);
        }
        mbar_init(smem_u32(&bars->q_full), kSoftmax);
        mbar_init(smem_u32(&bars->o_free), kSoftmax);
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 4 && lane == 0) {
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    if (warp == 5) {
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
    if (warp == 4) {
        // =========================== TMA producer ===========================
        // lane i brings page i of a tile; pages that no row sees, or whose
        // index is outside the pool, are not loaded (their keys are masked)
        const int ppt = kTileKeys / p.page;
        uint32_t n = 0;                                    // tiles issued (ring position)
        bool ok = true;
        for (; ok && more; more = next_piece<NR>(p, w)) {
            const Item it = item_of<NR>(p, w);
            auto page_of = [&](int tile) -> int {
                const int ord = tile * ppt + lane;
                if (lane >= ppt || ord >= p.max_pages || (long long)ord * p.page >= it.keys)
                    return -1;
                const int id = p.table[(long long)it.b * p.max_pages + ord];
                return (unsigned)id < (unsigned)p.n_pages ? id : -1;
            };
            int next = page_of(w.begin);
            for (int j = w.begin; ok && j < w.end; ++j, ++n) {
                const int id = next;
                if (j + 1 < w.end)
                    next = page_of(j + 1);
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
                if (n >= NV)
                    ok = wait_bar(smem_u32(&bars->v_empty[vs]), (n / NV - 1) & 1, abort, kErrPagedLoad + 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                if (lane == 0)
                    mbar_arrive_expect_tx(smem_u32(&bars->v_full[vs]), bytes);
                __syncwarp();
                if (id >= 0)
                    tma_load_4d(sV + vs * L::kTileBytes + lane * p.page * D, &tm_v, smem_u32(&bars->v_full[vs]), 0, w.h, 0, id);
            }
        }
        // never leave with copies in flight (after an abort the last V tile
        // may not have been issued: its wait then runs out)
        if (lane == 0) {
            for (uint32_t i = n > NK ? n - NK : 0; i < n; ++i)
                drain_wait(smem_u32(&bars->k_full[i % NK]), (i / NK) & 1);
            if (!ok)
                drain_wait(smem_u32(&bars->k_full[n % NK]), (n / NK) & 1);
            for (uint32_t i = n > NV ? n - NV : 0; i < n; ++i)
                drain_wait(smem_u32(&bars->v_full[i % NV]), (i / NV) & 1);
        }
        __syncwarp();
    } else if (warp == 5) {
        // ============================ MMA issuer ============================
        if (lane == 0) {
            constexpr int kSwz = D;                        // bytes of a K / V row = swizzle span
            constexpr uint32_t kSwzCode = D == 128 ? 2u : 4u;
            constexpr uint32_t kWCode = NR == 16 ? 6u : NR == 32 ? 4u : 2u;
            constexpr uint32_t idesc_s = idesc_make(0u, kTileKeys, NR, false);
            // V^T: 128 rows of which D are the tile's; at D = 64 the others are
            // whatever lies behind the tile, and their results are not read
            constexpr uint32_t idesc_o = idesc_make_amn(0u, 128, 2 * NR, true);
            const uint32_t hi = (uint32_t)(smem_desc(0, 16, 8 * kSwz, kSwzCode) >> 32);
            const uint32_t hi_w = (uint32_t)(smem_desc(0, 16, 8 * L::kWRow, kWCode) >> 32);
            const uint32_t lbo_v = (uint32_t)(L::kTileBytes >> 4) << 16;
            uint32_t ns = 0, nv = 0, pieces = 0;           // S^T and O^T products issued, pieces begun
            bool ok = true;
            for (; ok && more; more = next_piece<NR>(p, w), ++pieces) {
                const int n = w.end - w.begin;
                auto issue_s = [&]() -> bool {
                    const uint32_t ks = ns % NK, buf = ns & 1;
                    if (!wait_bar(smem_u32(&bars->k_full[ks]), (ns / NK) & 1, abort, kErrPagedMma) ||
                        (ns >= 2 && !wait_bar(smem_u32(&bars->s_free[buf]), (ns / 2 - 1) & 1, abort, kErrPagedMma + 1)))
                        return false;
                    tc_fence_after_sync();
                    const uint32_t k_lo = ((sK + ks * L::kTileBytes) >> 4) | (1u << 16);
#pragma unroll
                    for (int q = 0; q < QP; ++q) {
                        const uint32_t q_lo = ((sQ + q * L::kQPartBytes) >> 4) | (1u << 16);
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk)
                            mma_f8_ss(tmem + L::tmem_s(buf), desc_join(hi, k_lo + 2 * kk), desc_join(hi, q_lo + 2 * kk),
                                      idesc_s, q > 0 || kk > 0);
                    }
                    mma_commit(smem_u32(&bars->s_full[buf]));
                    mma_commit(smem_u32(&bars->k_empty[ks]));
                    ++ns;
                    return true;
                };
                ok = wait_bar(smem_u32(&bars->q_full), pieces & 1, abort, kErrPagedMma + 2) && issue_s();
                for (int j = 0; ok && j < n; ++j, ++nv) {
                    if (j + 1 < n && !(ok = issue_s()))
                        break;
                    const uint32_t vs = nv % NV, buf = nv % NW;
                    ok = wait_bar(smem_u32(&bars->v_full[vs]), (nv / NV) & 1, abort, kErrPagedMma + 3) &&
                         wait_bar(smem_u32(&bars->w_full[buf]), (nv / NW) & 1, abort, kErrPagedMma + 4) &&
                         (j > 0 || pieces == 0 ||
                          wait_bar(smem_u32(&bars->o_free), (pieces - 1) & 1, abort, kErrPagedMma + 5));
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    const uint32_t v_lo = ((sV + vs * L::kTileBytes) >> 4) | lbo_v;
                    const uint32_t w_lo = ((sW + buf * L::kWBytes) >> 4) | (1u << 16);
#pragma unroll
                    for (int kk = 0; kk < kTileKeys / 32; ++kk)
                        mma_f8_ss(tmem + L::kTmemO, desc_join(hi, v_lo + (uint32_t)((kk * 32 * kSwz) >> 4)),
                                  desc_join(hi_w, w_lo + (uint32_t)((kk * 32 * L::kWRow) >> 4)), idesc_o, j > 0 || kk > 0);
                    mma_commit(smem_u32(&bars->pv_done[buf]));
                    mma_commit(smem_u32(&bars->v_empty[vs]));
                }
            }
            mma_commit(smem_u32(&bars->drain));
            drain_wait(smem_u32(&bars->drain), 0);
        }
        __syncwarp();
    } else {
        // ========================= softmax warpgroup ========================
        float* row_scale = reinterpret_cast<float*>(smem + L::kOffRows);    // q's power of two * scale * log2 e
        float* row_max = row_scale + NR;
        int* row_last = reinterpret_cast<int*>(row_max + NR);               // last key that a row sees
        float* row_factor = row_max + 2 * NR;                               // rescale, or 1 / l
        float* exch = row_max + 3 * NR;                                     // [4][NR]
        int* nan_at = reinterpret_cast<int*>(exch + 4 * NR);                // [D]: first masked key with a NaN there
        const int key = threadIdx.x;                                        // of the tile; TMEM lane
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        uint32_t ns = 0;                                                    // tiles so far
        bool ok = true;
        for (; more; more = next_piece<NR>(p, w)) {
            const Item it = item_of<NR>(p, w);
            // ---- q into E4M3 parts, and each row's numbers
            {
                constexpr int kPer = kSoftmax / NR;                         // threads of a row
                constexpr int kSegs = (D / 16 + kPer - 1) / kPer;           // 16-element runs of a thread
                const int r = threadIdx.x / kPer, sub = threadIdx.x % kPer;
                const bool live = r < it.rows;
                const int i = (it.r0 + r) / p.group, hh = (it.r0 + r) % p.group;
                const uint16_t* q = reinterpret_cast<const uint16_t*>(p.Q) + (long long)it.b * p.q_sb + (long long)i * p.q_ss +
                                    (long long)(w.h * p.group + hh) * p.q_sh;
                float v[kSegs][16];
                float amax = 0.f;
                bool finite = true;
#pragma unroll
                for (int s = 0; s < kSegs; ++s) {
                    const int seg = sub + kPer * s;
                    uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                    if (live && seg < D / 16) {
                        u[0] = reinterpret_cast<const uint4*>(q)[2 * seg];
                        u[1] = reinterpret_cast<const uint4*>(q)[2 * seg + 1];
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        rope::unpack4<kBF16>(make_uint2(u[c].x, u[c].y), &v[s][8 * c]);
                        rope::unpack4<kBF16>(make_uint2(u[c].z, u[c].w), &v[s][8 * c + 4]);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        finite = finite && fabsf(v[s][e]) < INFINITY;
                        amax = fmaxf(amax, fabsf(v[s][e]));
                    }
                }
#pragma unroll
                for (int m = 1; m < kPer; m <<= 1) {
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
                    finite = __shfl_xor_sync(0xffffffffu, (int)finite, m) && finite;
                }
                const float qs = cache::pow2_scale(amax), inv = 1.f / qs;
#pragma unroll
                for (int s = 0; s < kSegs; ++s) {
                    const int seg = sub + kPer * s;
                    if (seg >= D / 16)
                        continue;
                    const int chunk = D == 128 ? seg ^ (r & 7) : seg ^ ((r >> 1) & 3);
#pragma unroll
                    for (int part = 0; part < QP; ++part) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            if (part == 0) {
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    v[s][e + c] *= inv;
                            }
                            const uint16_t lo = f32x2_to_e4m3x2(v[s][e], v[s][e + 1]);
                            const uint16_t up = f32x2_to_e4m3x2(v[s][e + 2], v[s][e + 3]);
                            const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2(lo)), b = f16x2_to_f32x2(e4m3x2_to_f16x2(up));
                            v[s][e] -= a.x;
                            v[s][e + 1] -= a.y;
                            v[s][e + 2] -= b.x;
                            v[s][e + 3] -= b.y;
                            o[e / 4] = (uint32_t)lo | ((uint32_t)up << 16);
                        }
                        st_shared_v4(sQ + part * L::kQPartBytes + r * D + chunk * 16, o[0], o[1], o[2], o[3]);
                    }
                }
                if (sub == 0) {
                    const long long last = p.causal ? it.start + i : it.start + it.count - 1;
                    row_scale[r] = finite ? qs * p.scale_log2 : NAN;
                    row_max[r] = live ? 0.f : INFINITY;                     // rows that are none get no weight
                    row_last[r] = !live || last < 0 ? -1 : (int)(last < it.keys ? last : it.keys - 1);
                }
                for (int d = threadIdx.x; d < D; d += kSoftmax)
                    nan_at[d] = INT_MAX;
                if (threadIdx.x == 0 && it.start + it.count > (long long)p.max_pages * p.page)
                    atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrTable);
                fence_proxy_async_smem();
                named_bar_sync(kBarSoftmax, kSoftmax);
                mbar_arrive(smem_u32(&bars->q_full));
            }
            // every row of the item sees keys 0 .. full - 1
            const int full = row_last[0] + 1;
            float l[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r)
                l[r] = 0.f;
            bool seen = false;                                              // row threadIdx.x has a maximum
            bool force = true;                                              // some row has none yet
            // this thread's page, one and two tiles ahead, and its scales
            auto page_of = [&](int tile) -> int {
                const int pos = tile * kTileKeys + key;
                if (pos >= it.keys)
                    return -1;
                const int id = p.table[(long long)it.b * p.max_pages + pos / p.page];
                if ((unsigned)id < (unsigned)p.n_pages)
                    return id;
                atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrPage);
                return -1;
            };
            auto scales_of = [&](int id, float& a, float& b) {
                a = b = 1.f;
                if (id >= 0) {
                    a = p.k.scale[(long long)id * p.Hkv + w.h];
                    b = p.v.scale[(long long)id * p.Hkv + w.h];
                }
            };
            int id = page_of(w.begin);
            int id_next = w.begin + 1 < w.end ? page_of(w.begin + 1) : -1;
            float k_scale, v_scale;
            scales_of(id, k_scale, v_scale);
            for (int j = w.begin; j < w.end; ++j, ++ns) {
                const bool valid = id >= 0;
                const float ks = k_scale;
                const float vs = fminf(fmaxf(v_scale, 8.673617379884035e-19f), 1.152921504606847e18f);   // 2^-60 .. 2^60
                const float lvs = log2f(vs) , rvs = 1.f / vs;
                id = id_next;
                scales_of(id, k_scale, v_scale);
                id_next = j + 2 < w.end ? page_of(j + 2) : -1;
                const uint32_t sbuf = ns & 1, wbuf = ns % NW;
                const int pos = j * kTileKeys + key;
                const bool edge = (j + 1) * kTileKeys > full;
                ok = ok && wait_bar(smem_u32(&bars->s_full[sbuf]), (ns / 2) & 1, abort, kErrPagedSoftmax);
                tc_fence_after_sync();
                // t = s + log2(v_scale): the logarithm of a weight but for the maximum; x = t - max
                float x[NR];
                bool high = false;
#pragma unroll
                for (int c = 0; c < NR; c += 16) {
                    uint32_t s[16];
                    __syncwarp();
                    tmem_ld16_wait(tmem + lanes + L::tmem_s(sbuf) + c, s);
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        const float4 sc = *reinterpret_cast<const float4*>(row_scale + c + r);
                        const float4 mx = *reinterpret_cast<const float4*>(row_max + c + r);
                        const float scv[4] = {sc.x, sc.y, sc.z, sc.w}, mxv[4] = {mx.x, mx.y, mx.z, mx.w};
                        int last[4] = {INT_MAX, INT_MAX, INT_MAX, INT_MAX};
                        if (edge) {
                            const int4 la = *reinterpret_cast<const int4*>(row_last + c + r);
                            last[0] = la.x, last[1] = la.y, last[2] = la.z, last[3] = la.w;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float t = fmaf(__uint_as_float(s[r + e]) * scv[e], ks, lvs);
                            x[c + r + e] = valid && pos <= last[e] ? t - mxv[e] : -INFINITY;
                            high = high || x[c + r + e] > kLag;
                        }
                    }
                }
                tc_fence_before_sync();
                mbar_arrive(smem_u32(&bars->s_free[sbuf]));
                if (named_bar_any(kBarSoftmax, kSoftmax, high || force || !ok)) {
                    // ---- a weight above 2^kLag: everything to the rows' new maxima
                    if (ok && j > w.begin)
                        ok = wait_bar(smem_u32(&bars->pv_done[(ns - 1) % NW]), ((ns - 1) / NW) & 1, abort, kErrPagedSoftmax + 1);
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        float m = x[r];
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        if (lane == (r & 31))
                            exch[warp * NR + r] = m;
                    }
                    ok = named_bar_all(kBarSoftmax, kSoftmax, ok);
                    if (!ok)
                        break;
                    bool waits = false;                                     // this row may see its first key later
                    if (threadIdx.x < NR) {
                        const int r = threadIdx.x;
                        const float top = fmaxf(fmaxf(exch[r], exch[NR + r]), fmaxf(exch[2 * NR + r], exch[3 * NR + r]));
                        const float up = seen ? fmaxf(top, 0.f) : top > -INFINITY ? top : 0.f;
                        row_factor[r] = up;
                        exch[r] = seen ? ex2_approx(-up) : 1.f;             // nothing to rescale before the first key
                        row_max[r] += up;
                        seen = seen || top > -INFINITY;
                        waits = !seen && row_last[r] >= (j + 1) * kTileKeys;
                    }
                    force = named_bar_any(kBarSoftmax, kSoftmax, waits);
                    tc_fence_after_sync();
#pragma unroll
                    for (int c = 0; c < NR; c += 16) {
                        float f[16];
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            x[c + r] -= row_factor[c + r];
                            f[r] = exch[c + r];
                            l[c + r] *= f[r];
                        }
                        if (j > w.begin) {
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                uint32_t o[16];
                                const uint32_t at = tmem + lanes + L::kTmemO + part * NR + c;
                                tmem_ld16_wait(at, o);
#pragma unroll
                                for (int r = 0; r < 16; ++r)
                                    o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r]);
                                tmem_st16(at, o);
                            }
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before_sync();
                }
                // ---- V rows that no row of the item sees are zero; a NaN that only some see is taken out and kept
                // in mind
                if (edge || __any_sync(0xffffffffu, !valid)) {
                    ok = ok && wait_bar(smem_u32(&bars->v_full[ns % NV]), (ns / NV) & 1, abort, kErrPagedSoftmax + 2);
                    const uint32_t row = sV + (ns % NV) * L::kTileBytes + key * D;
                    if (ok && !valid) {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c)
                            st_shared_v4(row + c * 16, 0u, 0u, 0u, 0u);
                    } else if (ok && pos >= full) {
                        for (int c = 0; c < D / 4; ++c) {
                            // 16-byte chunk c / 4 of the row lies at its swizzled place
                            const int chunk = D == 128 ? (c / 4) ^ (key & 7) : (c / 4) ^ ((key >> 1) & 3);
                            uint32_t* at = reinterpret_cast<uint32_t*>(smem + L::kOffV + (ns % NV) * L::kTileBytes + key * D +
                                                                       chunk * 16 + (c & 3) * 4);
                            uint32_t u = *at;
                            const uint32_t mag = u & 0x7f7f7f7fu;
                            const uint32_t hit = (mag + 0x01010101u) & 0x80808080u;      // bytes 0x7F and 0xFF
                            if (hit) {
                                for (int e = 0; e < 4; ++e)
                                    if (hit >> (8 * e + 7) & 1) {
                                        atomicMin(&nan_at[4 * c + e], pos);
                                        u &= ~(0xffu << (8 * e));
                                    }
                                *at = u;
                            }
                        }
                    }
                }
                // ---- weights into two E4M3 parts
                if (ok && ns >= (uint32_t)NW)
                    ok = wait_bar(smem_u32(&bars->pv_done[wbuf]), (ns / NW - 1) & 1, abort, kErrPagedSoftmax + 3);
                const uint32_t w_row = sW + wbuf * L::kWBytes + key * L::kWRow;
                constexpr int kChunks = L::kWRow / 16;
                const int swz = kChunks == 2 ? (key >> 2) & 1 : kChunks == 4 ? (key >> 1) & 3 : key & 7;
#pragma unroll
                for (int c = 0; c < NR; c += 16) {
                    uint32_t up[4], lo[4];
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        float y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            y[e] = ex2_approx(x[c + r + e] + kLog2W);
                            l[c + r + e] = fmaf(y[e], rvs, l[c + r + e]);
                        }
                        const uint16_t a = f32x2_to_e4m3x2(y[0], y[1]), b = f32x2_to_e4m3x2(y[2], y[3]);
                        const float2 fa = f16x2_to_f32x2(e4m3x2_to_f16x2(a)), fb = f16x2_to_f32x2(e4m3x2_to_f16x2(b));
                        up[r / 4] = (uint32_t)a | ((uint32_t)b << 16);
                        lo[r / 4] = (uint32_t)f32x2_to_e4m3x2((y[0] - fa.x) * 16.f, (y[1] - fa.y) * 16.f) |
                                    ((uint32_t)f32x2_to_e4m3x2((y[2] - fb.x) * 16.f, (y[3] - fb.y) * 16.f) << 16);
                    }
                    if (ok) {
                        st_shared_v4(w_row + (uint32_t)(((c / 16) ^ swz) * 16), up[0], up[1], up[2], up[3]);
                        st_shared_v4(w_row + (uint32_t)(((c / 16 + kChunks / 2) ^ swz) * 16), lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                fence_proxy_async_smem();
                if (ok)
                    mbar_arrive(smem_u32(&bars->w_full[wbuf]));
            }
            // ---- the piece's result
            if (ok)
                ok = wait_bar(smem_u32(&bars->pv_done[(ns - 1) % NW]), ((ns - 1) / NW) & 1, abort, kErrPagedSoftmax + 4);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float s = rope::group_sum<32>(l[r]);
                if (lane == (r & 31))
                    exch[warp * NR + r] = s;
            }
            ok = named_bar_all(kBarSoftmax, kSoftmax, ok);
            if (!ok)
                break;
            tc_fence_after_sync();
            const bool whole = w.begin == 0 && w.end == w.n;
            const long long slot = (long long)blockIdx.x * 2 + (w.begin > 0 ? 0 : 1);
            if (threadIdx.x < NR) {
                const int r = threadIdx.x;
                const float s = (exch[r] + exch[NR + r]) + (exch[2 * NR + r] + exch[3 * NR + r]);
                row_factor[r] = s == 0.f ? 0.f : 1.f / s;
                // sum of exp2(s - max) = s / 112; -inf for a row that has seen no key
                const float lse2 = s == 0.f ? -INFINITY : row_max[r] + (log2f(s) - kLog2W);
                if (r < it.rows) {
                    if (!whole) {
                        p.part_lse[slot * NR + r] = lse2;
                    } else if (p.lse) {
                        const int i = (it.r0 + r) / p.group, hh = (it.r0 + r) % p.group;
                        p.lse[((long long)it.b * p.Hq + w.h * p.group + hh) * p.Sq + i] = lse2 * kLn2;
                    }
                }
            }
            named_bar_sync(kBarSoftmax, kSoftmax);
            const int d = threadIdx.x;
            const int nan_from = d < D ? nan_at[d] : INT_MAX;
#pragma unroll
            for (int c = 0; c < NR; c += 16) {
                uint32_t a[16], b[16];
                __syncwarp();
                tmem_ld16_wait(tmem + lanes + L::kTmemO + c, a);
                tmem_ld16_wait(tmem + lanes + L::kTmemO + NR + c, b);
                if (c + 16 == NR) {
                    tc_fence_before_sync();
                    mbar_arrive(smem_u32(&bars->o_free));
                }
                if (d < D) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        if (c + r >= it.rows)
                            break;
                        float o = fmaf(__uint_as_float(b[r]), 1.f / 16.f, __uint_as_float(a[r])) * row_factor[c + r];
                        if (row_last[c + r] >= nan_from)
                            o = NAN;
                        if (!whole) {
                            p.part_o[(slot * NR + c + r) * D + d] = o;
                        } else {
                            const int i = (it.r0 + c + r) / p.group, hh = (it.r0 + c + r) % p.group;
                            reinterpret_cast<uint16_t*>(p.O)[(long long)it.b * p.o_sb + (long long)i * p.o_ss +
                                                             (long long)(w.h * p.group + hh) * p.o_sh + d] =
                                (uint16_t)(pack2<kBF16>(o, 0.f) & 0xffffu);
                        }
                    }
                }
            }
            named_bar_sync(kBarSoftmax, kSoftmax);             // the rows' numbers are read
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Joins the pieces of the items that several CTAs share.  Block (c, r): if
// the item that holds the first tile of CTA c's share began in CTA c - 1's, its
// row r is the sum over the CTAs c - 1 .. of
//     O = sum_k exp2(lse_k - LSE) O_k,   LSE = log2 sum_k exp2(lse_k).
constexpr int kJoinThreads = 256;

struct JoinShared {
    long long total, x, x_first;
    long long warp_sums[16];
    float o[kJoinThreads];
    float w[kJoinThreads];
};

template <int D, bool kBF16, int NR>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const Params p)
{
    constexpr int kSlices = kJoinThreads / D;
    __shared__ JoinShared sh;
    grid_dependency_wait();
    grid_launch_dependents();
    const int c = blockIdx.x + 1, r = blockIdx.y;
    find_share<NR, kJoinThreads>(p, c, &sh);
    const long long total = sh.total;
    const long long t = share_begin(total, c, p.ctas);
    if (t >= total)
        return;
    Piece w;
    w.x = sh.x;
    w.n = entry_tiles<NR>(p, w.x);
    w.h = (int)((t - sh.x_first) / w.n);
    const long long first = sh.x_first + (long long)w.h * w.n;       // the item's first tile
    if (first == t || first < share_begin(total, c - 1, p.ctas))
        return;
    const Item it = item_of<NR>(p, w);
    if (r >= it.rows)
        return;
    // last CTA: the one that holds tile first + n - 1
    int last = c;
    {
        int hi = p.ctas - 1;                               // shares are in order: bisection
        while (last < hi) {
            const int mid = (last + hi + 1) >> 1;
            if (share_begin(total, mid, p.ctas) <= first + w.n - 1)
                last = mid;
            else
                hi = mid - 1;
        }
    }
    const int n = last - c + 2;                            // pieces: slot 1 of CTA c - 1, slot 0 of c .. last
    auto slot_of = [&](int k) -> long long { return k == 0 ? (long long)(c - 1) * 2 + 1 : (long long)(c - 1 + k) * 2; };
    float m = -INFINITY;
    for (int k = threadIdx.x; k < n; k += kJoinThreads)
        m = fmaxf(m, p.part_lse[slot_of(k) * NR + r]);
    sh.w[threadIdx.x] = m;
    __syncthreads();
    for (int s = kJoinThreads / 2; s > 0; s >>= 1) {
        if (threadIdx.x < s)
            sh.w[threadIdx.x] = fmaxf(sh.w[threadIdx.x], sh.w[threadIdx.x + s]);
        __syncthreads();
    }
    m = sh.w[0];
    __syncthreads();
    const int d = threadIdx.x % D, slice = threadIdx.x / D;
    float o = 0.f, den = 0.f;
#pragma unroll 4
    for (int k = slice; k < n; k += kSlices) {
        const long long slot = slot_of(k) * NR + r;
        const float z = p.part_lse[slot];
        const float f = z == -INFINITY ? 0.f : exp2f(z - m);   // a NaN stays one
        den += f;
        o = fmaf(f, p.part_o[slot * D + d], o);
    }
    sh.o[threadIdx.x] = o;
    sh.w[threadIdx.x] = den;
    __syncthreads();
    if (slice == 0) {
        for (int s = 1; s < kSlices; ++s) {
            o += sh.o[s * D + d];
            den += sh.w[s * D + d];
        }
        const int i = (it.r0 + r) / p.group, hh = (it.r0 + r) % p.group;
        const long long head = (long long)w.h * p.group + hh;
        o = den == 0.f ? 0.f : o / den;
        reinterpret_cast<uint16_t*>(p.O)[(long long)it.b * p.o_sb + (long long)i * p.o_ss + head * p.o_sh + d] =
            (uint16_t)(pack2<kBF16>(o, 0.f) & 0xffffu);
        if (p.lse && d == 0)
            p.lse[((long long)it.b * p.Hq + head) * p.Sq + i] = den == 0.f ? -INFINITY : (m + log2f(den)) * kLn2;
    }
}

}  // namespace paged
}  // namespace sdpa
