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
};

// One warp for each (sequence, token, query head), keys in order.
template <int D, bool kBF16>
__global__ void __launch_bounds__(128) paged_rows_kernel(const Params p)
{
    constexpr int kPer = D / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (long long)p.B * p.Sq * p.Hq)
        return;
    const int hq = (int)(row % p.Hq);
    const int i = (int)(row / p.Hq % p.Sq);
    const int b = (int)(row / p.Hq / p.Sq);
    const int h = hq / p.group;
    const int count = p.count ? max(0, min(p.Sq, p.count[b])) : p.Sq;
    if (i >= count)
        return;
    const long long last = (long long)p.start[b] + (p.causal ? i : count - 1);
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p.Q) + b * p.q_sb + i * p.q_ss + hq * p.q_sh + lane * kPer;
    float qv[kPer], acc[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
        qv[c] = kBF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(q)[c])
                      : __half2float(reinterpret_cast<const __half*>(q)[c]);
        acc[c] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    int id = 0;
    float sk = 0.f, sv = 0.f;
    for (long long j = 0; j <= last; ++j) {
        const int slot = (int)(j % p.page);
        if (slot == 0) {
            const long long ord = j / p.page;
            if (ord >= p.max_pages) {
                if (lane == 0)
                    atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrTable);
                break;
            }
            id = p.table[(long long)b * p.max_pages + ord];
            if ((unsigned)id >= (unsigned)p.n_pages) {
                if (lane == 0)
                    atomicCAS(&g_sdpa_error, 0u, (unsigned)cache::kErrPage);
                j += p.page - 1;
                continue;
            }
            sk = p.k.scale[(long long)id * p.Hkv + h] * p.scale_log2;
            sv = p.v.scale[(long long)id * p.Hkv + h];
        }
        const uint8_t* kp = p.k.codes + id * p.k.sp + slot * p.k.ss + h * p.k.sh + lane * kPer;
        const uint8_t* vp = p.v.codes + id * p.v.sp + slot * p.v.ss + h * p.v.sh + lane * kPer;
        float dot = 0.f;
        float vv[kPer];
#pragma unroll
        for (int c = 0; c < kPer; c += 2) {
            const float2 kk = f16x2_to_f32x2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kp + c)));
            const float2 v2 = f16x2_to_f32x2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(vp + c)));
            dot = fmaf(qv[c], kk.x, fmaf(qv[c + 1], kk.y, dot));
            vv[c] = v2.x;
            vv[c + 1] = v2.y;
        }
        const float s = rope::group_sum<32>(dot) * sk;
        // a NaN score stays one: the maximum leaves it out, the weight does not
        const float mn = fmaxf(m, s);
        const float alpha = mn == -INFINITY ? 1.f : exp2f(m - mn), w = exp2f(s - mn);
        m = mn;
        l = l * alpha + w;
#pragma unroll
        for (int c = 0; c < kPer; ++c)
            acc[c] = acc[c] * alpha + w * sv * vv[c];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* o = reinterpret_cast<uint16_t*>(p.O) + b * p.o_sb + i * p.o_ss + hq * p.o_sh + lane * kPer;
#pragma unroll
    for (int c = 0; c < kPer; c += 2)
        *reinterpret_cast<uint32_t*>(o + c) = pack2<kBF16>(acc[c] * inv, acc[c + 1] * inv);
    if (p.lse && lane == 0)
        p.lse[((long long)b * p.Hq + hq) * p.Sq + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace paged
}  // namespace sdpa
