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
// 16-bit operands are split instead into 8-bit parts that add up to them; the
// products of 8-bit values are exact in the fp32 accumulator.  q, divided by a
// power of two that puts its row's largest element into (224, 448], becomes one
// (bf16) or two (fp16) E4M3 parts and a last one in E5M2: what rounding to
// E4M3 leaves of 8 bits, or of 11 the second time, are three bits and a sign, and
// E5M2 has the finer steps.  Elements down to 2^-13 (bf16) or 2^-10 (fp16) of
// the row's largest are held exactly, smaller ones within 2^-21 of it (2^-17,
// from 2^-9 and 2^-6 on, with E4M3 alone, in the same time).
//
// A weight w_j = exp(s_j - m) v_scale_j is rounded to f16, the only rounding
// that it sees (attention over fp16 keys and values rounds its weights so),
// and cut into four E5M2 parts: each is the upper byte of what the parts
// before it have left (3 bits of it), held 8 times as large as the one before,
// in columns of its own.  The parts are the f16 number exactly, subnormal ones
// included.  A row's largest weight is held as 2^11 to 2^15: weights down to
// e^-17 of it have 11 bits, and the smallest step is 2^-35 of it (the many
// small weights of a long cache are the whole output where a token with most
// of the weight has a value near zero).  Cutting costs no more than rounding
// into two E4M3 parts did, which lost what was below e^-14 (8 sequences of
// 32768 keys 91.3 us against 91.0).  Nothing is dequantised, and K and V are
// read once as bytes.
//
// The rows (token, query head) of one KV head are the N side of the products,
// the keys of a tile the M side:
//     S^T[128 keys][rows] = K8 Q^T,   O^T[D][rows] += V8^T W^T,
// so a decoding step's few rows cost few columns and every thread of the
// softmax warpgroup has one key of the tile: its scales, its mask and its
// weights for all rows.  Two warpgroups take turns, each with maxima, sums and
// an accumulator of its own, joined when the item is done: one alone leaves
// the schedulers waiting on its latencies.
//
// The key tiles of the whole call are shared out evenly over two CTAs an SM,
// wherever that cuts a sequence, so that ragged batches and single long
// sequences fill the machine alike; cut items are joined by a second kernel.
//
// Bound by HBM for long caches, by a chain of latencies below.  Measured (D =
// 128, 32 query heads on 8, bf16): 8 sequences of 32768 keys 88 - 92 us (537 MB:
// 5.8 - 6.1 TB/s), 64 of up to 8192 114 - 124 us (684 MB), one of 500 keys 8.6 us;
// without any loads the first of these takes 63 us, one tile of a CTA 0.9 us.
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
    int page_shift;                  // log2(page)
    int row_tiles;                   // tiles of NR rows that Sq * group rows need
    int ctas;                        // CTAs that share the key tiles
    unsigned long long ctas_inverse; // 2^64 / ctas, rounded up
    float* part_o;                   // [ctas][2][NR][D]: normalised results of pieces
    float* part_lse;                 // [ctas][2][NR]: their LSE in log2 units
    int4* joins;                     // [ctas]: entry, KV head, rows, pieces of an item to join (join_of)
};

enum : unsigned int { kErrPagedLoad = 0x801, kErrPagedMma = 0x811, kErrPagedSoftmax = 0x821 };

constexpr int kTileKeys = 128;

// The power of two that a row of q is divided by: all of bf16's range, but that
// it stops at 2^-118, for its inverse to be finite (a row whose largest is
// below 2^-110 keeps fewer bits).
__device__ __forceinline__ float query_scale(uint32_t top_bits)
{
    return cache::pow2_scale(__uint_as_float(top_bits), -118, 120);
}

// The next 8-bit part of four elements of a divided row, which it takes off them
// (exactly); `last`: what is left, as E5M2.
__device__ __forceinline__ uint32_t query_part(float* v, bool last)
{
    if (last)
        return (uint32_t)f32x2_to_e5m2x2(v[0], v[1]) | ((uint32_t)f32x2_to_e5m2x2(v[2], v[3]) << 16);
    const uint16_t lo = f32x2_to_e4m3x2(v[0], v[1]), up = f32x2_to_e4m3x2(v[2], v[3]);
    const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2(lo)), b = f16x2_to_f32x2(e4m3x2_to_f16x2(up));
    v[0] -= a.x;
    v[1] -= a.y;
    v[2] -= b.x;
    v[3] -= b.y;
    return (uint32_t)lo | ((uint32_t)up << 16);
}

// The running maximum is let behind by up to 2^4 before everything is rescaled
// to a new one, and weight 1 is held as 2^11: no weight passes 2^15, which the
// parts need (with 2^2 and 2^13: 64 sequences, 16 rows of 64, 73.6 us against 71.8).
constexpr float kLag = 4.0f;
constexpr float kLog2W = 11.0f;

// Shared memory and TMEM of one CTA: NR rows, q in kParts 8-bit parts, weights
// in kWParts E5M2 parts.
template <int D, bool kBF16, int NR>
struct PagedLayout {
    static_assert(D == 64 || D == 128, "head dimension");
    static_assert(NR == 8 || NR == 16, "rows of a tile");
    static constexpr int kParts = kBF16 ? 2 : 3;
    static constexpr int kWParts = 4;
    static constexpr int kGroups = 2;                           // softmax warpgroups
    static constexpr int kSoftmax = 128 * kGroups;              // warps 0 ..
    static constexpr int kThreads = kSoftmax + 64;              // then TMA producer, MMA issuer
    static constexpr int kTileBytes = kTileKeys * D;            // a K or V tile
    // depth of the rings: what two CTAs fit into an SM
    // (64 sequences of up to 8192 keys, 16 rows of 128: 154 us with 2 + 3 and 196 us with 3 + 2, as V waits longer;
    // one weight tile for both warpgroups leaves room for 3 + 3: 157 us)
    static constexpr int kStagesK = D == 64 ? 5 : NR == 16 ? 2 : 3;
    static constexpr int kStagesV = D == 64 ? 5 : 3;
    static constexpr int kQRows = 16;                           // columns of S^T: 16 at least
    static constexpr int kQPartBytes = kQRows * D;
    static constexpr int kWRow = kWParts * NR;                  // bytes of a key's weights: 32 or 64
    static constexpr int kWBytes = kTileKeys * kWRow;
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kStagesK * kTileBytes;
    static constexpr int kOffW = kOffV + kStagesV * kTileBytes;  // at D = 64 also what the unused half of the last
    static constexpr int kOffQ = kOffW + kGroups * kWBytes;      // V tile's operand reads
    static constexpr int kOffRows = kOffQ + kParts * kQPartBytes;
    // per row: q's scale, last key; per warpgroup: negative maximum, shift, factor, 4 x exchange; per channel: NaN
    static constexpr int kRowsBytes = 4 * (2 * NR + 7 * NR * kGroups + D);
    static constexpr int kOffBar = (kOffRows + kRowsBytes + 15) / 16 * 16;
    static constexpr int kBarBytes = 448;
    static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;                // + alignment
    static_assert(kOffQ % 1024 == 0 && kOffW % 1024 == 0, "swizzle atoms");
    static_assert(D == 128 || kGroups * kWBytes + kParts * kQPartBytes >= kTileBytes, "operand of the unused half");
    static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
    // a warpgroup's columns: S^T, then the parts of O^T
    static constexpr int kOCols = kWParts * NR;
    static constexpr int kGroupCols = kQRows + kOCols;
    static constexpr uint32_t kTmemCols = kGroups * kGroupCols <= 128 ? 128 : 256;
    static_assert(kGroups * kGroupCols <= 256, "two CTAs per SM");
};

template <int NK, int NV, int kGroups>
struct PagedBarriers {
    uint64_t k_full[NK], k_empty[NK], v_full[NV], v_empty[NV];
    // of each warpgroup: S^T computed / read out, weights written / multiplied
    uint64_t s_full[kGroups], s_free[kGroups], w_full[kGroups], pv_done[kGroups];
    uint64_t q_full;                       // q's parts written
    uint64_t o_free;                       // O^T read out
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    // where the CTA's share of the tiles begins
    long long total, x, x_first;
    long long warp_sums[12];
};

// Number of key tiles of entry x = (sequence, row tile): 0 without rows, else
// at least 1.  (In 32 bits the kernel of many rows comes out 12% slower.)
template <int NR>
__device__ __forceinline__ int entry_tiles(const Params& p, long long x)
{
    if constexpr (NR <= 16) {                          // one row tile holds a sequence's rows
        const int b = (int)x;
        const int count = p.count ? max(0, min(p.Sq, p.count[b])) : p.Sq;
        const long long len = min((long long)p.start[b] + count, (long long)p.max_pages << p.page_shift);
        return count == 0 ? 0 : len < 1 ? 1 : (int)((len + kTileKeys - 1) / kTileKeys);
    }
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

// First tile of CTA c's share of `total` tiles, c * total / ctas: the product
// with ctas' reciprocal is exact for totals below 2^64 / ctas^2.  With fewer
// tiles than CTAs the first `total` CTAs have one each, so no share between
// two others is empty.
__device__ __forceinline__ long long share_begin(const Params& p, long long total, int c)
{
    if (c >= p.ctas || total < p.ctas)
        return c < total && c < p.ctas ? c : total;
    return (long long)__umul64hi((unsigned long long)total, p.ctas_inverse * (unsigned)c);
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
    const long long target = share_begin(p, total, c);
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
    const long long t0 = share_begin(p, bars->total, c);
    w.left = share_begin(p, bars->total, c + 1) - t0;
    if (w.left <= 0)
        return false;
    w.x = bars->x;
    w.n = entry_tiles<NR>(p, w.x);
    const long long off = t0 - bars->x_first;
    w.h = off >> 32 ? (int)(off / w.n) : (int)((uint32_t)off / (uint32_t)w.n);
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
    t.b = NR <= 16 ? (int)w.x : (int)(w.x / p.row_tiles);
    t.r0 = NR <= 16 ? 0 : (int)(w.x - (long long)t.b * p.row_tiles) * NR;
    t.count = p.count ? max(0, min(p.Sq, p.count[t.b])) : p.Sq;
    t.rows = min(NR, t.count * p.group - t.r0);
    t.start = p.start[t.b];
    const long long cap = (long long)p.max_pages << p.page_shift;
    long long len = t.start + (NR > 16 && p.causal ? (t.r0 + t.rows - 1) / p.group + 1 : t.count);
    len = len < 0 ? 0 : len;
    t.keys = (int)(len < cap ? len : cap);
    return t;
}

// Sums over the warp of N values a lane: lanes r 32 / N .. get that of s[r].
// Each step hands half of the values to the lane across and adds the other
// half of its, then what is left goes round.
template <int N>
__device__ __forceinline__ float warp_sums(float (&s)[N], int lane)
{
#pragma unroll
    for (int h = N / 2; h > 0; h >>= 1) {
        const bool up = lane & (32 / N * h);
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float give = up ? s[i] : s[i + h];
            const float keep = up ? s[i + h] : s[i];
            s[i] = keep + __shfl_xor_sync(0xffffffffu, give, 32 / N * h);
        }
    }
    float v = s[0];
#pragma unroll
    for (int m = 32 / N / 2; m > 0; m >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// An item whose pieces several CTAs have is joined by the block of the second
// of them, c: joins[c].w is the number of pieces (0: nothing to join there).
template <int NR>
__device__ __forceinline__ int4 join_of(const Params& p, long long total, const Piece& w)
{
    const int c = blockIdx.x;
    const long long first = share_begin(p, total, c) - w.begin;          // the item's first tile
    if (w.begin == 0 || first < share_begin(p, total, c - 1))
        return make_int4(0, 0, 0, 0);
    int last = c, hi = p.ctas - 1;                     // the CTA that has the item's last tile: bisection
    while (last < hi) {
        const int mid = (last + hi + 1) >> 1;
        if (share_begin(p, total, mid) <= first + w.n - 1)
            last = mid;
        else
            hi = mid - 1;
    }
    return make_int4((int)w.x, w.h, item_of<NR>(p, w).rows, last - c + 2);
}

template <int D, bool kBF16, int NR>
__global__ void __launch_bounds__(PagedLayout<D, kBF16, NR>::kThreads, 2)
paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Params p)
{
    using L = PagedLayout<D, kBF16, NR>;
    constexpr int NK = L::kStagesK, NV = L::kStagesV, G = L::kGroups, QP = L::kParts, WP = L::kWParts;
    constexpr int kProducer = L::kSoftmax / 32, kIssuer = kProducer + 1;      // warps
    constexpr uint32_t kBarAll = 1;                    // named barriers: all softmax threads, 2 + g one warpgroup
    using Bars = PagedBarriers<NK, NV, G>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    auto* bars = reinterpret_cast<Bars*>(smem + L::kOffBar);
    static_assert(sizeof(Bars) <= L::kBarBytes, "barrier block");
    volatile int* abort = &bars->abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // known to be the same in the warp
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
        for (int i = 0; i < G; ++i) {
            mbar_init(smem_u32(&bars->s_full[i]), 1);
            mbar_init(smem_u32(&bars->s_free[i]), 128);
            mbar_init(smem_u32(&bars->w_full[i]), 128);
            mbar_init(smem_u32(&bars->pv_done[i]), 1);
        }
        mbar_init(smem_u32(&bars->q_full), L::kSoftmax);
        mbar_init(smem_u32(&bars->o_free), L::kSoftmax);
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == kProducer && lane == 0) {
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    if (warp == kIssuer) {
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
    if (warp == kProducer) {
        // =========================== TMA producer ===========================
        // lane i brings page i of a tile; pages that no row sees, or whose
        // index is outside the pool, are not loaded (their keys are masked)
        const int ppt = kTileKeys >> p.page_shift;
        uint32_t n = 0;                                    // tiles issued (ring position)
        bool ok = true;
        for (; ok && more; more = next_piece<NR>(p, w)) {
            const Item it = item_of<NR>(p, w);
            // table entries are read three tiles ahead and looked at when their
            // tile comes, so that no tile waits for one
            auto entry_of = [&](int tile) -> int {
                const int ord = tile * ppt + lane;
                return lane < ppt && tile < w.end && ord << p.page_shift < it.keys
                           ? p.table[(long long)it.b * p.max_pages + ord]
                           : -1;
            };
            int ahead[3] = {entry_of(w.begin), entry_of(w.begin + 1), entry_of(w.begin + 2)};
            for (int j = w.begin; ok && j < w.end; ++j, ++n) {
                const int id = (unsigned)ahead[0] < (unsigned)p.n_pages ? ahead[0] : -1;
                ahead[0] = ahead[1];
                ahead[1] = ahead[2];
                ahead[2] = entry_of(j + 3);
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
        if (lane == 0 && blockIdx.x > 0) {                 // (after the loads, which nothing should keep waiting)
            Piece first;
            p.joins[blockIdx.x] = first_piece<NR>(p, bars, first) ? join_of<NR>(p, bars->total, first) : make_int4(0, 0, 0, 0);
        }
        // never leave with copies in flight (after an abort the last K tile
        // may or may not have been issued: at worst its wait runs out)
        if (lane == 0) {
            for (uint32_t i = n > NK ? n - NK : 0; i < n; ++i)
                drain_wait(smem_u32(&bars->k_full[i % NK]), (i / NK) & 1);
            if (!ok)
                drain_wait(smem_u32(&bars->k_full[n % NK]), (n / NK) & 1);
            for (uint32_t i = n > NV ? n - NV : 0; i < n; ++i)
                drain_wait(smem_u32(&bars->v_full[i % NV]), (i / NV) & 1);
        }
        __syncwarp();
    } else if (warp == kIssuer) {
        // ============================ MMA issuer ============================
        if (lane == 0) {
            constexpr int kSwz = D;                        // bytes of a K / V row = swizzle span
            constexpr uint32_t kSwzCode = D == 128 ? 2u : 4u;
            constexpr uint32_t kWCode = L::kWRow == 32 ? 6u : 4u;
            constexpr uint32_t idesc_s = idesc_make(0u, kTileKeys, L::kQRows, false);
            // V^T: 128 rows of which D are the tile's; at D = 64 the others are
            // whatever lies behind the tile, and their results are not read
            // (B, the weights, is E5M2)
            constexpr uint32_t idesc_o = idesc_make_amn(0u, 128, L::kOCols, true) | (1u << 10);
            const uint32_t hi = (uint32_t)(smem_desc(0, 16, 8 * kSwz, kSwzCode) >> 32);
            const uint32_t hi_w = (uint32_t)(smem_desc(0, 16, 8 * L::kWRow, kWCode) >> 32);
            const uint32_t lbo_v = (uint32_t)(L::kTileBytes >> 4) << 16;
            uint32_t ks_n = 0, vs_n = 0, pieces = 0;       // S^T and O^T products issued, pieces begun
            uint32_t ns0 = 0, ns1 = 0, nv0 = 0, nv1 = 0;   // the same, of each warpgroup
            bool ok = true;
            for (; ok && more; more = next_piece<NR>(p, w), ++pieces) {
                const int n = w.end - w.begin;
                auto issue_s = [&](int g) -> bool {
                    const uint32_t ks = ks_n % NK, done = g ? ns1 : ns0;
                    if (!wait_bar(smem_u32(&bars->k_full[ks]), (ks_n / NK) & 1, abort, kErrPagedMma) ||
                        (done > 0 && !wait_bar(smem_u32(&bars->s_free[g]), (done - 1) & 1, abort, kErrPagedMma + 1)))
                        return false;
                    tc_fence_after_sync();
                    const uint32_t k_lo = ((sK + ks * L::kTileBytes) >> 4) | (1u << 16);
#pragma unroll
                    for (int q = 0; q < QP; ++q) {
                        const uint32_t q_lo = ((sQ + q * L::kQPartBytes) >> 4) | (1u << 16);
                        const uint32_t idesc = idesc_s | (q + 1 == QP ? 1u << 10 : 0u);         // q (B): E5M2 in the end
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk)
                            mma_f8_ss(tmem + g * L::kGroupCols, desc_join(hi, k_lo + 2 * kk), desc_join(hi, q_lo + 2 * kk),
                                      idesc, q > 0 || kk > 0);
                    }
                    mma_commit(smem_u32(&bars->s_full[g]));
                    mma_commit(smem_u32(&bars->k_empty[ks]));
                    ns0 += g ? 0 : 1;
                    ns1 += g ? 1 : 0;
                    ++ks_n;
                    return true;
                };
                ok = wait_bar(smem_u32(&bars->q_full), pieces & 1, abort, kErrPagedMma + 2) && issue_s(0);
                if (G > 1 && n > 1)
                    ok = ok && issue_s(1);
                for (int j = 0; ok && j < n; ++j, ++vs_n) {
                    const int g = G > 1 ? j & 1 : 0;
                    if (j + G < n && !(ok = issue_s(g)))
                        break;
                    const uint32_t vs = vs_n % NV;
                    ok = wait_bar(smem_u32(&bars->v_full[vs]), (vs_n / NV) & 1, abort, kErrPagedMma + 3) &&
                         wait_bar(smem_u32(&bars->w_full[g]), (g ? nv1 : nv0) & 1, abort, kErrPagedMma + 4) &&
                         (j > 0 || pieces == 0 ||
                          wait_bar(smem_u32(&bars->o_free), (pieces - 1) & 1, abort, kErrPagedMma + 5));
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    const uint32_t v_lo = ((sV + vs * L::kTileBytes) >> 4) | lbo_v;
                    const uint32_t w_lo = ((sW + g * L::kWBytes) >> 4) | (1u << 16);
#pragma unroll
                    for (int kk = 0; kk < kTileKeys / 32; ++kk)
                        mma_f8_ss(tmem + g * L::kGroupCols + L::kQRows, desc_join(hi, v_lo + (uint32_t)((kk * 32 * kSwz) >> 4)),
                                  desc_join(hi_w, w_lo + (uint32_t)((kk * 32 * L::kWRow) >> 4)), idesc_o, j >= G || kk > 0);
                    mma_commit(smem_u32(&bars->pv_done[g]));
                    mma_commit(smem_u32(&bars->v_empty[vs]));
                    nv0 += g ? 0 : 1;
                    nv1 += g ? 1 : 0;
                }
            }
            mma_commit(smem_u32(&bars->drain));
            drain_wait(smem_u32(&bars->drain), 0);
        }
        __syncwarp();
    } else {
        // ======================== softmax warpgroups ========================
        const int g = G > 1 ? warp >> 2 : 0;
        const uint32_t bar_group = 2 + g;
        const int tid = threadIdx.x & 127;                                  // key of the tile; TMEM lane
        float* row_scale = reinterpret_cast<float*>(smem + L::kOffRows);    // q's power of two * scale * log2 e
        int* row_last = reinterpret_cast<int*>(row_scale + NR);             // last key that a row sees
        float* group_rows = row_scale + 2 * NR;                             // 7 NR numbers of each warpgroup
        float* row_nmax = group_rows + 7 * NR * g;                          // kLog2W - maximum
        float* row_shift = row_nmax + NR;                                   // by how much the maximum grows
        float* row_factor = row_nmax + 2 * NR;                              // rescale; in the end the weight of O^T
        float* exch = row_nmax + 3 * NR;                                    // [4][NR]
        int* nan_at = reinterpret_cast<int*>(group_rows + 7 * NR * G);      // [D]: first masked key with a NaN there
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + g * L::kGroupCols, t_o = t_s + L::kQRows;
        uint32_t ns = 0;                                                    // tiles of this warpgroup so far
        uint32_t nv = 0;                                                    // tiles of the CTA before this piece
        bool ok = true;
        for (; more; nv += w.end - w.begin, more = next_piece<NR>(p, w)) {
            const Item it = item_of<NR>(p, w);
            // ---- q into 8-bit parts, and each row's numbers
            {
                constexpr int kPer = L::kSoftmax / L::kQRows;               // threads of a row
                static_assert(kPer >= D / 16, "a 16-element run a thread");
                const int r = threadIdx.x / kPer, seg = threadIdx.x % kPer;
                const bool live = r < it.rows;
                const int i = (it.r0 + r) / p.group, hh = (it.r0 + r) % p.group;
                const uint16_t* q = reinterpret_cast<const uint16_t*>(p.Q) + (long long)it.b * p.q_sb + (long long)i * p.q_ss +
                                    (long long)(w.h * p.group + hh) * p.q_sh;
                float v[16];
                uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (live && seg < D / 16) {
                    u[0] = reinterpret_cast<const uint4*>(q)[2 * seg];
                    u[1] = reinterpret_cast<const uint4*>(q)[2 * seg + 1];
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    rope::unpack4<kBF16>(make_uint2(u[c].x, u[c].y), &v[8 * c]);
                    rope::unpack4<kBF16>(make_uint2(u[c].z, u[c].w), &v[8 * c + 4]);
                }
                // the largest magnitude; infinities and NaN have the largest bits
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
                for (int m = 1; m < kPer; m <<= 1)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
                const bool finite = top < 0x7f800000u;
                const float qs = query_scale(top), inv = 1.f / qs;
                const int chunk = D == 128 ? seg ^ (r & 7) : seg ^ ((r >> 1) & 3);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    v[e] *= inv;
                if (seg < D / 16) {
#pragma unroll
                    for (int part = 0; part < QP; ++part) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            o[e / 4] = query_part(&v[e], part + 1 == QP);
                        st_shared_v4(sQ + part * L::kQPartBytes + r * D + chunk * 16, o[0], o[1], o[2], o[3]);
                    }
                }
                if (seg == 0 && r < NR) {
                    const long long last = p.causal ? it.start + i : it.start + it.count - 1;
                    row_scale[r] = finite ? qs * p.scale_log2 : NAN;
                    row_last[r] = !live || last < 0 ? -1 : (int)(last < it.keys ? last : it.keys - 1);
#pragma unroll
                    for (int k = 0; k < G; ++k)                             // rows that are none get no weight
                        group_rows[7 * NR * k + r] = live ? kLog2W : -INFINITY;
                }
                if (threadIdx.x < D)
                    nan_at[threadIdx.x] = INT_MAX;
                if (threadIdx.x == 0 && it.start + it.count > (long long)p.max_pages * p.page)
                    atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrTable);
                fence_proxy_async_smem();
                named_bar_sync(kBarAll, L::kSoftmax);
                mbar_arrive(smem_u32(&bars->q_full));
            }
            // every row of the item sees keys 0 .. full - 1
            const int full = row_last[0] + 1;
            uint64_t l[NR / 2];                                             // pairs of rows
#pragma unroll
            for (int r = 0; r < NR / 2; ++r)
                l[r] = 0;
            bool seen = false;                                              // row tid has a maximum
            bool force = true;                                              // some row has none yet
            // this thread's table entry two tiles of the warpgroup ahead, its
            // scales one ahead: each is looked at when the next is on its way
            const int* table = p.table + (long long)it.b * p.max_pages;
            auto entry_of = [&](int tile) -> int {
                const int pos = tile * kTileKeys + tid;
                return tile < w.end && pos < it.keys ? table[pos >> p.page_shift] : INT_MIN;
            };
            auto scales_of = [&](int entry, float& a, float& b) -> bool {
                a = b = 1.f;
                const bool ok = (unsigned)entry < (unsigned)p.n_pages;
                if (ok) {
                    a = p.k.scale[(long long)entry * p.Hkv + w.h];
                    b = p.v.scale[(long long)entry * p.Hkv + w.h];
                } else if (entry != INT_MIN) {
                    atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrPage);
                }
                return ok;
            };
            int entry = entry_of(w.begin + g);
            int entry_next = entry_of(w.begin + g + G);
            float k_scale, v_scale;
            bool valid_next = scales_of(entry, k_scale, v_scale);
            const int first = w.begin + g;                                  // this warpgroup's first tile
            for (int j = first; j < w.end; j += G, ++ns) {
                const bool valid = valid_next;
                const float ks = k_scale;
                const float vs = fminf(fmaxf(v_scale, 8.673617379884035e-19f), 1.152921504606847e18f);   // 2^-60 .. 2^60
                const float lvs = __log2f(vs), rvs = __fdividef(1.f, vs);
                entry = entry_next;
                entry_next = entry_of(j + 2 * G);
                valid_next = scales_of(entry, k_scale, v_scale);
                const uint32_t vn = nv + (uint32_t)(j - w.begin);           // V ring position
                const int pos = j * kTileKeys + tid;
                // tiles in which some row does not see some key, by the item's rows or by a page that is none
                const bool edge = (j + 1) * kTileKeys > full || __any_sync(0xffffffffu, !valid);
                ok = ok && wait_bar(smem_u32(&bars->s_full[g]), ns & 1, abort, kErrPagedSoftmax);
                tc_fence_after_sync();
                // s + log2(v_scale): the logarithm of a weight but for the maximum, which comes off with kLog2W on top
                const uint64_t ks2 = f32x2(ks, ks), lvs2 = f32x2(lvs, lvs);
                uint64_t x[NR / 2];
                float top;
                {
                    uint32_t s[NR];
                    if constexpr (NR == 8)
                        tmem_ld8_wait(t_s, s);
                    else
                        tmem_ld16_wait(t_s, s);
                    tc_fence_before_sync();
                    mbar_arrive(smem_u32(&bars->s_free[g]));
#pragma unroll
                    for (int r = 0; r < NR; r += 4) {
                        const ulonglong2 sc = *reinterpret_cast<const ulonglong2*>(row_scale + r);
                        const ulonglong2 nm = *reinterpret_cast<const ulonglong2*>(row_nmax + r);
                        x[r / 2] = fma_f32x2(f32x2(__uint_as_float(s[r]), __uint_as_float(s[r + 1])), mul_f32x2(sc.x, ks2),
                                             add_f32x2(nm.x, lvs2));
                        x[r / 2 + 1] = fma_f32x2(f32x2(__uint_as_float(s[r + 2]), __uint_as_float(s[r + 3])),
                                                 mul_f32x2(sc.y, ks2), add_f32x2(nm.y, lvs2));
                    }
                    if (edge) {
#pragma unroll
                        for (int r = 0; r < NR; r += 2) {
                            float a, b;
                            f32x2_split(x[r / 2], a, b);
                            x[r / 2] = f32x2(valid && pos <= row_last[r] ? a : -INFINITY,
                                             valid && pos <= row_last[r + 1] ? b : -INFINITY);
                        }
                    }
                    float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                    for (int r = 0; r < NR / 2; r += 2) {
                        float a, b;
                        f32x2_split(x[r], a, b);
                        m0 = fmax3(m0, a, b);
                        f32x2_split(x[r + 1], a, b);
                        m1 = fmax3(m1, a, b);
                    }
                    top = fmaxf(m0, m1);
                }
                if (named_bar_any(bar_group, 128, top > kLag + kLog2W || force || !ok)) {
                    // ---- a weight above 2^kLag, or a row's first key: everything to the rows' new maxima
                    if (ok && j > first)
                        ok = wait_bar(smem_u32(&bars->pv_done[g]), (ns - 1) & 1, abort, kErrPagedSoftmax + 1);
                    float mine = 0.f;                                       // lane r: the warp's maximum of row r
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        float a, b;
                        f32x2_split(x[r / 2], a, b);
                        const float m = warp_max(r & 1 ? b : a);
                        mine = lane == r ? m : mine;
                    }
                    if (lane < NR)
                        exch[(warp & 3) * NR + lane] = mine;
                    ok = named_bar_all(bar_group, 128, ok);
                    if (!ok)
                        break;
                    bool waits = false;                                     // this row may see its first key later
                    if (tid < NR) {
                        const float m = fmaxf(fmaxf(exch[tid], exch[NR + tid]), fmaxf(exch[2 * NR + tid], exch[3 * NR + tid])) - kLog2W;
                        const float up = seen ? fmaxf(m, 0.f) : m > -INFINITY ? m : 0.f;
                        row_shift[tid] = up;
                        row_factor[tid] = seen ? ex2_approx(-up) : 1.f;     // nothing to rescale before the first key
                        row_nmax[tid] -= up;
                        seen = seen || m > -INFINITY;
                        waits = !seen && row_last[tid] >= (j + G) * kTileKeys;
                    }
                    force = named_bar_any(bar_group, 128, waits);
                    tc_fence_after_sync();
                    float f[NR];
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        f[r] = row_factor[r];
#pragma unroll
                    for (int r = 0; r < NR / 2; ++r) {
                        l[r] = mul_f32x2(l[r], f32x2(f[2 * r], f[2 * r + 1]));
                        x[r] = add_f32x2(x[r], f32x2(-row_shift[2 * r], -row_shift[2 * r + 1]));
                    }
                    if (j > first) {
#pragma unroll 1
                        for (int part = 0; part < WP; ++part) {
                            uint32_t o[NR];
                            if constexpr (NR == 8)
                                tmem_ld8_wait(t_o + part * NR, o);
                            else
                                tmem_ld16_wait(t_o + part * NR, o);
#pragma unroll
                            for (int r = 0; r < NR; ++r)
                                o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r]);
                            if constexpr (NR == 8)
                                tmem_st8(t_o + part * NR, o);
                            else
                                tmem_st16(t_o + part * NR, o);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before_sync();
                }
                // ---- V rows that no row of the item sees are zero; a NaN that only some see is taken out and kept
                // in mind
                if (edge) {
                    ok = ok && wait_bar(smem_u32(&bars->v_full[vn % NV]), (vn / NV) & 1, abort, kErrPagedSoftmax + 2);
                    const uint32_t row = sV + (vn % NV) * L::kTileBytes + tid * D;
                    if (ok && !valid) {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c)
                            st_shared_v4(row + c * 16, 0u, 0u, 0u, 0u);
                    } else if (ok && pos >= full) {
                        for (int c = 0; c < D / 4; ++c) {
                            // 16-byte chunk c / 4 of the row lies at its swizzled place
                            const int chunk = D == 128 ? (c / 4) ^ (tid & 7) : (c / 4) ^ ((tid >> 1) & 3);
                            uint32_t* at = reinterpret_cast<uint32_t*>(smem + L::kOffV + (vn % NV) * L::kTileBytes + tid * D +
                                                                       chunk * 16 + (c & 3) * 4);
                            uint32_t u = *at;
                            const uint32_t hit = ((u & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;    // bytes 0x7F, 0xFF
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
                // ---- weights to f16 (11 bits) and into E5M2 parts
                if (ok && ns > 0)
                    ok = wait_bar(smem_u32(&bars->pv_done[g]), (ns - 1) & 1, abort, kErrPagedSoftmax + 3);
                const uint32_t w_row = sW + g * L::kWBytes + tid * L::kWRow;
                const int swz = L::kWRow == 32 ? (tid >> 2) & 1 : (tid >> 1) & 3;
                const uint64_t rvs2 = f32x2(rvs, rvs);
                constexpr int kWords = NR / 4;                              // 32-bit words of a part
                uint32_t words[WP * kWords];
#pragma unroll
                for (int r = 0; r < NR / 2; r += 2) {
                    uint32_t rest[2];                                       // four rows
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float a, b;
                        f32x2_split(x[r + i], a, b);
                        a = ex2_approx(a);
                        b = ex2_approx(b);
                        l[r + i] = fma_f32x2(f32x2(a, b), rvs2, l[r + i]);
                        rest[i] = f32x2_to_f16x2(a, b);
                    }
#pragma unroll
                    for (int k = 0; k < WP; ++k) {
                        words[k * kWords + r / 2] = __byte_perm(rest[0], rest[1], 0x7531);      // the upper bytes
                        if (k + 1 < WP)                                     // 8 (rest - part), both exact
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                rest[i] = mul_f16x2(add_f16x2(rest[i], (rest[i] & 0xff00ff00u) ^ 0x80008000u), 0x48004800u);
                    }
                }
                if (ok) {
#pragma unroll
                    for (int i = 0; i < WP * kWords / 4; ++i)
                        st_shared_v4(w_row + (uint32_t)((i ^ swz) * 16), words[4 * i], words[4 * i + 1], words[4 * i + 2],
                                     words[4 * i + 3]);
                }
                fence_proxy_async_smem();
                if (ok)
                    mbar_arrive(smem_u32(&bars->w_full[g]));
            }
            // ---- the piece's result
            const bool took = first < w.end;                               // this warpgroup had a tile
            if (ok && took)
                ok = wait_bar(smem_u32(&bars->pv_done[g]), (ns - 1) & 1, abort, kErrPagedSoftmax + 4);
            {
                float s[NR];
#pragma unroll
                for (int r = 0; r < NR / 2; ++r)
                    f32x2_split(l[r], s[2 * r], s[2 * r + 1]);
                const float sum = warp_sums<NR>(s, lane);
                if (lane % (32 / NR) == 0)
                    exch[(warp & 3) * NR + lane / (32 / NR)] = sum;
            }
            ok = named_bar_all(kBarAll, L::kSoftmax, ok);
            if (!ok)
                break;
            tc_fence_after_sync();
            const bool whole = w.begin == 0 && w.end == w.n;
            const long long slot = (long long)blockIdx.x * 2 + (w.begin > 0 ? 0 : 1);
            if (threadIdx.x < NR) {
                // join the warpgroups: sums s_g of exp2(logit - max_g + kLog2W), weights of their O^T
                const int r = threadIdx.x;
                float s[G], nm[G], m = -INFINITY, sum = 0.f;
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    const float* e = group_rows + 7 * NR * k + 3 * NR + r;
                    s[k] = (e[0] + e[NR]) + (e[2 * NR] + e[3 * NR]);
                    nm[k] = group_rows[7 * NR * k + r];
                    m = s[k] == 0.f ? m : fmaxf(m, kLog2W - nm[k]);
                }
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    nm[k] = s[k] == 0.f ? 0.f : exp2f(kLog2W - nm[k] - m);
                    sum = fmaf(s[k], nm[k], sum);
                }
#pragma unroll
                for (int k = 0; k < G; ++k)
                    group_rows[7 * NR * k + 2 * NR + r] = sum == 0.f ? 0.f : nm[k] / sum;
                const float lse2 = sum == 0.f ? -INFINITY : m + (log2f(sum) - kLog2W);
                if (r < it.rows) {
                    if (!whole) {
                        p.part_lse[slot * NR + r] = lse2;
                    } else if (p.lse) {
                        const int i = (it.r0 + r) / p.group, hh = (it.r0 + r) % p.group;
                        p.lse[((long long)it.b * p.Hq + w.h * p.group + hh) * p.Sq + i] = lse2 * kLn2;
                    }
                }
            }
            named_bar_sync(kBarAll, L::kSoftmax);
            // channel tid of every row, from both warpgroups' accumulators
            if (g == 0) {
                const int groups = w.end - w.begin < G ? w.end - w.begin : G;
                const int nan_from = tid < D ? nan_at[tid] : INT_MAX;
                float o[NR];
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    o[r] = 0.f;
#pragma unroll 1
                for (int k = 0; k < groups; ++k) {
                    float unit = 1.f;
#pragma unroll 1
                    for (int part = 0; part < WP; ++part, unit *= 1.f / 8.f) {
                        uint32_t a[NR];
                        const uint32_t at = tmem + lanes + k * L::kGroupCols + L::kQRows + part * NR;
                        if constexpr (NR == 8)
                            tmem_ld8_wait(at, a);
                        else
                            tmem_ld16_wait(at, a);
#pragma unroll
                        for (int r = 0; r < NR; ++r)
                            o[r] = fmaf(__uint_as_float(a[r]), unit * group_rows[7 * NR * k + 2 * NR + r], o[r]);
                    }
                }
                if (tid < D) {
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        if (r >= it.rows)
                            break;
                        const float v = row_last[r] >= nan_from ? NAN : o[r];
                        if (!whole) {
                            p.part_o[(slot * NR + r) * D + tid] = v;
                        } else {
                            const int i = (it.r0 + r) / p.group, hh = (it.r0 + r) % p.group;
                            reinterpret_cast<uint16_t*>(p.O)[(long long)it.b * p.o_sb + (long long)i * p.o_ss +
                                                             (long long)(w.h * p.group + hh) * p.o_sh + tid] =
                                (uint16_t)(pack2<kBF16>(v, 0.f) & 0xffffu);
                        }
                    }
                }
            }
            tc_fence_before_sync();
            mbar_arrive(smem_u32(&bars->o_free));
            named_bar_sync(kBarAll, L::kSoftmax);              // the rows' numbers are read
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kIssuer) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Joins the pieces of the items that several CTAs share.  Block (c, y): if
// joins[c] names an item, its rows y kRows .. are sums over its pieces, slot 1 of CTA c - 1
// and slot 0 of CTAs c .. :
//     O = sum_k exp2(lse_k - LSE) O_k,   LSE = log2 sum_k exp2(lse_k).
// Few rows have a block each, whose threads share the pieces out (there may be
// hundreds); many rows go eight to a block, a warp each where the pieces are
// few (measured on 1024 rows of 3 pieces: 25 us by blocks, 13.5 by warps).
constexpr int kJoinThreads = 256;

template <int D, bool kBF16, int NR>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const Params p)
{
    constexpr int kSlices = kJoinThreads / D;
    constexpr int kRows = NR <= 16 ? 1 : 8;
    __shared__ float sh_o[kJoinThreads], sh_w[kJoinThreads], sh_m[kJoinThreads];
    grid_dependency_wait();
    grid_launch_dependents();
    const int c = blockIdx.x + 1;
    const int4 join = p.joins[c];
    const int n = join.w;
    if (n == 0)
        return;
    struct { int b, r0, rows; } it = {NR <= 16 ? join.x : join.x / p.row_tiles, 0, join.z};
    it.r0 = NR <= 16 ? 0 : (join.x - it.b * p.row_tiles) * NR;
    const int kv_head = join.y;
    auto slot_of = [&](int k) -> long long { return k == 0 ? (long long)(c - 1) * 2 + 1 : (long long)(c - 1 + k) * 2; };
    auto store = [&](int r, int d, float o) {
        const int i = (it.r0 + r) / p.group;
        const long long head = (long long)kv_head * p.group + (it.r0 + r) % p.group;
        reinterpret_cast<uint16_t*>(p.O)[(long long)it.b * p.o_sb + (long long)i * p.o_ss + head * p.o_sh + d] =
            (uint16_t)(pack2<kBF16>(o, 0.f) & 0xffffu);
    };
    auto store_lse = [&](int r, float m, float den) {
        const int i = (it.r0 + r) / p.group;
        const long long head = (long long)kv_head * p.group + (it.r0 + r) % p.group;
        if (p.lse)
            p.lse[((long long)it.b * p.Hq + head) * p.Sq + i] = den == 0.f ? -INFINITY : (m + log2f(den)) * kLn2;
    };
    if (kRows > 1 && n <= 32) {
        // lane k has piece k's LSE; the channels go over the lanes
        const int r = blockIdx.y * kRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
        if (r >= it.rows)
            return;
        const float z = lane < n ? p.part_lse[slot_of(lane) * NR + r] : -INFINITY;
        float m = z;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
        const float f = z == -INFINITY ? 0.f : exp2f(z - m);       // a NaN stays one
        float den = f;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1)
            den += __shfl_xor_sync(0xffffffffu, den, s);
        float o[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            o[c] = 0.f;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                o[c] = fmaf(fk, p.part_o[(slot_of(k) * NR + r) * D + 32 * c + lane], o[c]);
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            store(r, 32 * c + lane, den == 0.f ? 0.f : o[c] / den);
        if (lane == 0)
            store_lse(r, m, den);
        return;
    }
    // one pass, eight pieces of a slice at a time, each batch under the largest LSE so far
    for (int r = blockIdx.y * kRows; r < min(it.rows, (int)(blockIdx.y + 1) * kRows); ++r) {
        const int d = threadIdx.x % D, slice = threadIdx.x / D;
        float m = -INFINITY, o = 0.f, den = 0.f;
        auto scaled = [](float z, float top) { return z == -INFINITY ? 0.f : exp2f(z - top); };   // a NaN stays one
        for (int k0 = slice; k0 < n; k0 += 8 * kSlices) {
            float z[8], v[8], top = m;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = k0 + i * kSlices;
                const long long slot = slot_of(k) * NR + r;
                z[i] = k < n ? p.part_lse[slot] : -INFINITY;
                v[i] = k < n ? p.part_o[slot * D + d] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = fmaxf(top, z[i]);
            const float c = scaled(m, top);
            o *= c;
            den *= c;
            m = top;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = scaled(z[i], m);
                den += f;
                o = fmaf(f, v[i], o);
            }
        }
        sh_o[threadIdx.x] = o;
        sh_w[threadIdx.x] = den;
        sh_m[threadIdx.x] = m;
        __syncthreads();
        if (slice == 0) {
            float top = m;
#pragma unroll
            for (int s = 1; s < kSlices; ++s)
                top = fmaxf(top, sh_m[s * D + d]);
            const float c = scaled(m, top);
            o *= c;
            den *= c;
#pragma unroll
            for (int s = 1; s < kSlices; ++s) {
                const float f = scaled(sh_m[s * D + d], top);
                o = fmaf(f, sh_o[s * D + d], o);
                den = fmaf(f, sh_w[s * D + d], den);
            }
            store(r, d, den == 0.f ? 0.f : o / den);
            if (d == 0)
                store_lse(r, top, den);
        }
        __syncthreads();
    }
}

}  // namespace paged
}  // namespace sdpa
