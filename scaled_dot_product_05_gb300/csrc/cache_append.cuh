// cache_append.cuh -- new keys and values into a paged 8-bit cache, the keys
// rotated on the way.
//
// The cache holds E4M3 codes and one fp32 scale for each page and KV head;
// a value is code * scale.  The scale is a power of two, the smallest with
// max|x| <= 448 scale over the page's tokens: E4M3 is a floating type, so a
// scale finer than that would not make its rounding (at most 2^-4 relative)
// smaller, while a power of two makes the division exact and lets the scale of
// a page that is filled over several calls grow without a second rounding of
// what it holds already (but for values that become subnormal).  A call that
// goes on in a page keeps at least the page's scale; a call that begins a page
// ignores what its scale was.
//
// One unit is a (sequence, page, KV head, K or V).  Two instances: eight warps
// a unit for prompts, one warp a unit (eight units a block) for the few tokens
// of a decoding step.  The rows wait in registers between the maximum and the
// rounding, so each is read once.  Measured (4 prompts of up to 2000 tokens, 8
// KV heads of 128, rotated): 13.6 us for 37 MB, bound by its latencies (table,
// page, rows, scale one after the other in one and a half waves of blocks) and
// by issue slots, of which two thirds are taken; 128 single tokens: 2.8 us,
// latency.
//
// A rotated key is off by an ulp or two of fp32, enough to send one key in a
// million to the code on the other side of a border.  Rows with an element
// that close to one are computed again without rounding (7% of the time of a
// prompt's append, most of it the test).
// (The border test looks at normal codes under a power-of-two scale, before the
// scale is known; the maximum behind the scale is fp32's.)
#pragma once

#include "rope.cuh"

namespace sdpa {
namespace cache {

enum : unsigned int {
    kErrPage = 0x601,            // a page index outside the pool
    kErrTable = 0x602,           // a position outside the page table
};

// A paged cache: page p, slot t, KV head h at p * sp + t * ss + h * sh (elements = bytes).
struct Pool {
    uint8_t* codes;
    float* scale;                // [n_pages][Hkv]
    long long sp, ss, sh;
};

struct AppendParams {
    const void* x[2];            // keys, values: [B][S][Hkv][D]
    long long x_sb[2], x_ss[2], x_sh[2];
    Pool pool[2];
    const int* table;            // [B][max_pages]
    const int* start;            // [B]
    const int* count;            // [B], or null: S
    const float* rope;           // [n_pos][rot / 2][2]
    int B, S, Hkv, page, page_shift, n_pages, max_pages;
    int n_pos, rot;
    int n_ord;                   // pages that S tokens can touch
};

constexpr int kAppendThreads = 256;

// Smallest e in [lo, hi] with amax <= 448 * 2^e (448 = 1.75 * 2^8), as 2^e.
__device__ __forceinline__ float pow2_scale(float amax, int lo = -60, int hi = 60)
{
    const uint32_t bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(lo, min(hi, e));
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// True for a value next to the middle between two codes (its 20 bits behind
// E4M3's mantissa within 16 of 2^19): there the roundings of a rotation in fp32
// decide which code it gets.
// border_at is the distance from 16 below it, in the upper 20 bits.
constexpr uint32_t kNear = 33u << 12;
__device__ __forceinline__ uint32_t border_at(float x)
{
    return (__float_as_uint(x) - (0x80000u - 16u)) << 12;
}

// a b + c d rounded to odd: the exact sum as hi + lo (error-free products and
// sum), the last bit set where something was rounded off, so that a second
// rounding to fewer bits is that of the exact sum.
__device__ __forceinline__ float dot2_to_odd(float a, float b, float c, float d)
{
    const float p = __fmul_rn(a, b), e = __fmaf_rn(a, b, -p);
    const float q = __fmul_rn(c, d), f = __fmaf_rn(c, d, -q);
    const float hi = __fadd_rn(p, q), t = __fsub_rn(hi, p);
    const float err = __fadd_rn(__fsub_rn(p, __fsub_rn(hi, t)), __fsub_rn(q, t));
    const float lo = __fadd_rn(__fadd_rn(e, f), err);
    const float z = __fadd_rn(hi, lo), rest = __fsub_rn(lo, __fsub_rn(z, hi));
    if (rest == 0.f)
        return z;
    return __uint_as_float((__float_as_uint(z) - ((rest < 0.f) != (z < 0.f) ? 1u : 0u)) | 1u);
}

// True if one of a lane's 8 elements is next to a border.
__device__ __forceinline__ bool any_near(const float* x)
{
    uint32_t nearest = border_at(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i)
        nearest = min(nearest, border_at(x[i]));
    return nearest < kNear;
}

// Rotates a lane's 8 elements, those next to a border by the exact product, so
// that they get its codes (but where its two terms cancel to less than an
// eighth, and for subnormal codes).
template <bool kInter>
__device__ __forceinline__ void rotate_for_codes(float* x, const float* cs, const float* sn)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = kInter ? 2 * i : i, q = kInter ? 2 * i + 1 : i + 4;
        const float u = x[p], v = x[q];
        x[p] = u * cs[i] - v * sn[i];
        x[q] = u * sn[i] + v * cs[i];
        if (border_at(x[p]) < kNear)
            x[p] = dot2_to_odd(u, cs[i], v, -sn[i]);
        if (border_at(x[q]) < kNear)
            x[q] = dot2_to_odd(u, sn[i], v, cs[i]);
    }
}

// kWarps warps a unit (1 or 8), kPasses rows at most for each lane group.
template <int D, bool kBF16, bool kInter, int kWarps, int kPasses>
__global__ void __launch_bounds__(kAppendThreads, kWarps > 1 && kPasses <= 4 ? 4 : 2) append_kernel(const AppendParams p)
{
    constexpr int kLanes = D / 8;
    constexpr int kUnitThreads = 32 * kWarps;
    constexpr int kRows = kUnitThreads / kLanes;       // rows of a pass
    __shared__ float warp_max[kAppendThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x % kUnitThreads;
    const uint32_t unit = blockIdx.x * (kAppendThreads / kUnitThreads) + threadIdx.x / kUnitThreads;
    const int lane = tid % kLanes;
    const int group = tid / kLanes;
    // unit -> (KV head fastest, K or V, page of the sequence's new tokens,
    // sequence); units fit into 31 bits, the host refuses more
    uint32_t rest = unit / (uint32_t)p.Hkv;
    const int h = (int)(unit - rest * p.Hkv);
    const int kv = (int)(rest & 1);
    rest >>= 1;
    const int b = (int)(rest / (uint32_t)p.n_ord);
    const int ord = (int)(rest - b * p.n_ord);
    if (b >= p.B)
        return;                                        // whole units: their warps leave together
    const long long start = p.start[b];
    const int count = p.count ? max(0, min(p.S, p.count[b])) : p.S;
    if (start < 0) {
        if (tid == 0 && count > 0)
            atomicCAS(&g_sdpa_error, 0u, (unsigned)kErrTable);
        return;
    }
    const long long ord_page = (start >> p.page_shift) + ord;      // ordinal of the page in its sequence
    const long long p0 = ord_page * p.page;            // position of its first slot
    const int lo = (int)(start > p0 ? start - p0 : 0);
    const long long end = start + count - p0;
    const int hi = (int)(end < p.page ? end : p.page);
    if (hi <= lo)
        return;
    if (ord_page >= p.max_pages) {
        if (tid == 0)
            atomicCAS(&g_sdpa_error, 0u, (unsigned)kErrTable);
        return;
    }
    const int id = p.table[(long long)b * p.max_pages + ord_page];     // (looked at when the rows are on their way)
    const int rot = kv ? 0 : p.rot;                    // only the keys are rotated
    int a, c;
    rope::lane_channels<kInter>(lane, rot, a, c);
    const int i0 = (int)(p0 + lo - start);             // first new token of the page
    const uint16_t* x = reinterpret_cast<const uint16_t*>(p.x[kv]) + b * p.x_sb[kv] + h * p.x_sh[kv];
    float v[kPasses][8];
    uint2 ra[kPasses], rb[kPasses];
    float cs[kPasses][4], sn[kPasses][4];
    uint32_t ok = 0;                                   // rows that are written
#pragma unroll
    for (int n = 0; n < kPasses; ++n) {
        const int r = n * kRows + group;               // row among the page's new ones
        ra[n] = rb[n] = make_uint2(0, 0);
        if (r < hi - lo) {
            const uint16_t* row = x + (i0 + r) * p.x_ss[kv];
            ra[n] = *reinterpret_cast<const uint2*>(row + a);
            rb[n] = *reinterpret_cast<const uint2*>(row + c);
            ok |= 1u << n;
            const long long pos = p0 + lo + r;
            if (rot && pos >= p.n_pos) {
                atomicCAS(&g_sdpa_error, 0u, (unsigned)rope::kErrPosition);
                ok &= ~(1u << n);
            } else if (rot) {
                rope::lane_angles(p.rope, (int)pos, rot, lane, cs[n], sn[n]);
            }
        }
    }
    if ((unsigned)id >= (unsigned)p.n_pages) {         // the whole unit
        if (tid == 0)
            atomicCAS(&g_sdpa_error, 0u, (unsigned)kErrPage);
        return;
    }
    const Pool pool = p.pool[kv];
    float* scale_at = pool.scale + (long long)id * p.Hkv + h;
    const float old = *scale_at;                       // before the barrier: written after it
    float amax = 0.f;
    uint32_t again = 0;                                // rows with elements next to a border
#pragma unroll
    for (int n = 0; n < kPasses; ++n) {
        if (!(ok >> n & 1))
            continue;
        rope::unpack4<kBF16>(ra[n], v[n]);
        rope::unpack4<kBF16>(rb[n], v[n] + 4);
        if (rot)
            rope::rotate<kInter>(v[n], cs[n], sn[n]);
        again |= rot && any_near(v[n]) ? 1u << n : 0u;
        // infinities (they saturate) and NaN stay out of the scale
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = fabsf(v[n][i]);
            amax = t < INFINITY ? fmaxf(amax, t) : amax;
        }
    }
    // (one row of a warp in a hundred; read again, so that nothing waits in
    // registers for it)
#pragma unroll 1
    for (int n = 0; again >> n; ++n) {
        if (!(again >> n & 1))
            continue;
        const int r = n * kRows + group;
        const uint16_t* row = x + (i0 + r) * p.x_ss[kv];
        float u[8], co[4], si[4];
        rope::unpack4<kBF16>(*reinterpret_cast<const uint2*>(row + a), u);
        rope::unpack4<kBF16>(*reinterpret_cast<const uint2*>(row + c), u + 4);
        rope::lane_angles(p.rope, (int)(p0 + lo + r), rot, lane, co, si);
        rotate_for_codes<kInter>(u, co, si);
#pragma unroll
        for (int m = 0; m < kPasses; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[m][i] = m == n ? u[i] : v[m][i];
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    if constexpr (kWarps > 1) {
        if ((threadIdx.x & 31) == 0)
            warp_max[threadIdx.x >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
            amax = fmaxf(amax, warp_max[i]);
    } else {
        __syncwarp();
    }
    float scale = pow2_scale(amax);
    uint8_t* page = pool.codes + (long long)id * pool.sp + h * pool.sh;
    bool exact = true;                                 // the scale is a power of two
    if (lo > 0) {
        if (old >= scale) {
            scale = old;
            exact = (__float_as_uint(old) & 0x7fffffu) == 0 && old < 1e37f;
        } else {
            // the page's earlier tokens, rounded to the scale that it has now
            const float f = old / scale;
            for (int i = tid; i < lo * (D / 4); i += kUnitThreads) {
                uint32_t* at = reinterpret_cast<uint32_t*>(page + (long long)(i / (D / 4)) * pool.ss + 4 * (i % (D / 4)));
                const uint32_t w = *at;
                const float2 s = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)w));
                const float2 t = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w >> 16)));
                *at = (uint32_t)f32x2_to_e4m3x2(s.x * f, s.y * f) | ((uint32_t)f32x2_to_e4m3x2(t.x * f, t.y * f) << 16);
            }
        }
    }
    if (tid == 0)
        *scale_at = scale;
    auto write = [&](auto quotient) {
#pragma unroll
        for (int n = 0; n < kPasses; ++n) {
            if (!(ok >> n & 1))
                continue;
            uint8_t* row = page + (long long)(lo + n * kRows + group) * pool.ss;
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = quotient(v[n][i]);
            *reinterpret_cast<uint32_t*>(row + a) =
                (uint32_t)f32x2_to_e4m3x2(q[0], q[1]) | ((uint32_t)f32x2_to_e4m3x2(q[2], q[3]) << 16);
            *reinterpret_cast<uint32_t*>(row + c) =
                (uint32_t)f32x2_to_e4m3x2(q[4], q[5]) | ((uint32_t)f32x2_to_e4m3x2(q[6], q[7]) << 16);
        }
    };
    // the product with the reciprocal is the quotient for a power of two
    const float inv = 1.f / scale;
    if (exact)
        write([&](float x) { return x * inv; });
    else
        write([&](float x) { return x / scale; });
}

}  // namespace cache
}  // namespace sdpa
