// qk_norm_rope.cuh -- norm of queries and keys for each head and the position
// rotation in one pass, and its gradient.
//
// Forward, for every row x (D channels of one head of one token):
//     n = x * r * w,  r = 1 / sqrt(mean(x^2) + eps)      (left out without norm)
//     y = R(position) n                                  (rope.cuh)
// all in fp32, rounded once to the 16-bit output.  Backward, for the upstream
// gradient g of y:
//     h = R^T g,  dw += h * x r,  u = h * w,
//     dx = r (u - x r mean(u * x r))
// with r computed again from x (reading a stored r would save nothing: x is
// needed anyway).  Both are streams bound by HBM: 2 D bytes read and written
// per row forward, 4 D read and 2 D written backward.
#pragma once

#include "rope.cuh"

namespace sdpa {
namespace rope {

// One of the two tensors (queries, keys) of a call.
struct Side {
    const void* x;               // [B][S][H][D]
    const void* g;               // backward: upstream gradient
    void* y;                     // forward: result; backward: dx
    const void* w;               // weights of the norm, or null for ones
    long long x_sb, x_ss, x_sh;  // strides in elements
    long long g_sb, g_ss, g_sh;
    long long y_sb, y_ss, y_sh;
    int H;
    int chunks;                  // items of a token: ceil(H / kHeads)
};

struct NormRopeParams {
    Side side[2];                // queries, keys (H = 0: absent)
    const float* table;          // [n_pos][rot / 2][2]: cos, sin
    const int* positions;        // [B][S], or null: position s
    int S, n_pos, rot;
    uint32_t tokens;             // B * S
    int norm, w16;               // w16: weights are 16-bit like x, else fp32
    float eps;
    float* part;                 // backward: dw partial sums [blocks][D]
    int blocks[2];               // backward: blocks of each side
    float* dw[2];
};

// Measured (B = 2, S = 4096, 40 heads of 128): 128 threads a block 30.6 us, 256
// 33.2 us.
constexpr int kNormThreads = 128;

template <bool kBF16>
__device__ __forceinline__ float weight_at(const void* w, int w16, int c)
{
    if (!w)
        return 1.f;
    if (!w16)
        return reinterpret_cast<const float*>(w)[c];
    if constexpr (kBF16)
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[c]);
    else
        return __half2float(reinterpret_cast<const __half*>(w)[c]);
}

// One item: kHeads consecutive heads of one token, by a group of D / 8 lanes.
// More heads share a token's angles and have more loads in flight, but leave a
// decoding step with fewer groups (measured at 2, 4 and 8 heads: 39, 31 and 29
// us for the training batch, 2.2, 2.3 and 3.1 us for 64 tokens).
constexpr int kHeads = 4;

template <int D, bool kBF16, bool kInter>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const NormRopeParams p)
{
    constexpr int kLanes = D / 8;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % kLanes;
    // (items fit into 31 bits: the host refuses more)
    const uint32_t per_token = p.side[0].chunks + p.side[1].chunks;
    const uint32_t item = blockIdx.x * (kNormThreads / kLanes) + threadIdx.x / kLanes;
    const uint32_t token = item / per_token;
    const bool live = token < p.tokens;
    int chunk = (int)(item - token * per_token);
    const int k = chunk >= p.side[0].chunks;
    const Side& sd = p.side[k];
    chunk -= k ? p.side[0].chunks : 0;
    const int b = live ? (int)(token / (uint32_t)p.S) : 0;
    const int s = live ? (int)token - b * p.S : 0;
    int n_heads = live ? min(kHeads, sd.H - chunk * kHeads) : 0;
    int a, c;
    lane_channels<kInter>(lane, p.rot, a, c);
    float cs[4], sn[4];
    int pos = 0;
    if (p.rot) {
        pos = p.positions && live ? p.positions[token] : s;
        if ((unsigned)pos >= (unsigned)p.n_pos) {
            if (live)
                atomicCAS(&g_sdpa_error, 0u, (unsigned)kErrPosition);
            n_heads = 0;
            pos = 0;
        }
    }
    const uint16_t* x = reinterpret_cast<const uint16_t*>(sd.x) + b * sd.x_sb + s * sd.x_ss +
                        (long long)chunk * kHeads * sd.x_sh;
    uint2 va[kHeads], vb[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        va[h] = vb[h] = make_uint2(0, 0);
        if (h < n_heads) {
            va[h] = *reinterpret_cast<const uint2*>(x + h * sd.x_sh + a);
            vb[h] = *reinterpret_cast<const uint2*>(x + h * sd.x_sh + c);
        }
    }
    lane_angles(p.table, pos, p.rot, lane, cs, sn);
    float w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = p.norm ? weight_at<kBF16>(sd.w, p.w16, a + i) : 1.f;
        w[4 + i] = p.norm ? weight_at<kBF16>(sd.w, p.w16, c + i) : 1.f;
    }
    uint16_t* y = reinterpret_cast<uint16_t*>(sd.y) + b * sd.y_sb + s * sd.y_ss + (long long)chunk * kHeads * sd.y_sh;
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        float v[8];
        unpack4<kBF16>(va[h], v);
        unpack4<kBF16>(vb[h], v + 4);
        if (p.norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss = fmaf(v[i], v[i], ss);
            const float r = rsqrtf(group_sum<kLanes>(ss) * (1.f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] *= r * w[i];
        }
        rotate<kInter>(v, cs, sn);
        if (h < n_heads) {
            *reinterpret_cast<uint2*>(y + h * sd.y_sh + a) = pack4<kBF16>(v);
            *reinterpret_cast<uint2*>(y + h * sd.y_sh + c) = pack4<kBF16>(v + 4);
        }
    }
}

// Blocks of the backward pass (both sides together at most): each walks many
// items, so that dw is summed in registers and leaves as one row of partial
// sums a block.  All blocks are resident at once, five on each of 152 SMs
// (measured, training batch of 8192 tokens x 40 heads of 128 / 3996 x 32 of 64,
// the sum kernel included: 52 / 13.2 us; 4 blocks of 256 threads and 2 heads an
// item 53 / 14.3 us; a second item's loads ahead of the first's arithmetic cost
// more in occupancy than they hid, 62 us).
constexpr int kBwdThreads = 128;
constexpr int kBwdBlocks = 760;
constexpr int kBwdHeads = 4;

// Instructions count here as much as bytes (some 110 a lane and row): all
// arithmetic is on packed pairs, of a run's neighbouring channels with the
// halves order, of a rotated pair's two channels with the interleaved one.
template <int D, bool kBF16, bool kInter>
__global__ void __launch_bounds__(kBwdThreads, 5) norm_rope_bwd_kernel(const NormRopeParams p)
{
    constexpr int kLanes = D / 8;
    constexpr int kGroups = kBwdThreads / kLanes;
    __shared__ float sums[kGroups][D];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % kLanes;
    const int group = threadIdx.x / kLanes;
    const int k = (int)blockIdx.x >= p.blocks[0];
    const Side& sd = p.side[k];
    const int block = blockIdx.x - (k ? p.blocks[0] : 0);
    int a, c;
    lane_channels<kInter>(lane, p.rot, a, c);
    uint64_t w[4], dw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = i < 2 ? a + 2 * i : c + 2 * (i - 2);
        w[i] = p.norm ? f32x2(weight_at<kBF16>(sd.w, p.w16, at), weight_at<kBF16>(sd.w, p.w16, at + 1)) : f32x2(1.f, 1.f);
        dw[i] = 0;
    }
    // (items fit into 31 bits: the host refuses more)
    const uint32_t items = p.tokens * sd.chunks;
    const uint32_t stride = p.blocks[k] * kGroups;
    // every group of a warp runs the same number of turns: the sums shuffle
    for (uint32_t first = block * kGroups; first < items; first += stride) {
        const uint32_t item = first + group;
        const bool live = item < items;
        const uint32_t token = live ? item / (uint32_t)sd.chunks : 0;
        const int chunk = live ? (int)(item - token * sd.chunks) : 0;
        const int b = (int)(token / (uint32_t)p.S);
        const int s = (int)token - b * p.S;
        int n_heads = live ? min(kBwdHeads, sd.H - chunk * kBwdHeads) : 0;
        int pos = 0;
        if (p.rot) {
            pos = p.positions ? p.positions[token] : s;
            if ((unsigned)pos >= (unsigned)p.n_pos) {
                if (live)
                    atomicCAS(&g_sdpa_error, 0u, (unsigned)kErrPosition);
                n_heads = 0;
                pos = 0;
            }
        }
        const long long h0 = (long long)chunk * kBwdHeads;
        const uint16_t* x = reinterpret_cast<const uint16_t*>(sd.x) + b * sd.x_sb + s * sd.x_ss + h0 * sd.x_sh;
        const uint16_t* g = reinterpret_cast<const uint16_t*>(sd.g) + b * sd.g_sb + s * sd.g_ss + h0 * sd.g_sh;
        uint2 xa[kBwdHeads], xb[kBwdHeads], ga[kBwdHeads], gb[kBwdHeads];
#pragma unroll
        for (int h = 0; h < kBwdHeads; ++h) {
            xa[h] = xb[h] = ga[h] = gb[h] = make_uint2(0, 0);
            if (h < n_heads) {
                ga[h] = *reinterpret_cast<const uint2*>(g + h * sd.g_sh + a);
                gb[h] = *reinterpret_cast<const uint2*>(g + h * sd.g_sh + c);
                if (p.norm) {
                    xa[h] = *reinterpret_cast<const uint2*>(x + h * sd.x_sh + a);
                    xb[h] = *reinterpret_cast<const uint2*>(x + h * sd.x_sh + c);
                }
            }
        }
        float cs[4], sn[4];
        lane_angles(p.table, pos, p.rot, lane, cs, sn);
        uint16_t* y = reinterpret_cast<uint16_t*>(sd.y) + b * sd.y_sb + s * sd.y_ss + h0 * sd.y_sh;
#pragma unroll
        for (int h = 0; h < kBwdHeads; ++h) {
            uint64_t u[4];
            unpack_pairs<kBF16>(ga[h], u);
            unpack_pairs<kBF16>(gb[h], u + 2);
            // the inverse rotation
            if constexpr (kInter) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {                  // (x cos + y sin, y cos - x sin)
                    float e, f;
                    f32x2_split(u[i], e, f);
                    u[i] = fma_f32x2(f32x2(f, e), f32x2(sn[i], -sn[i]), mul_f32x2(u[i], f32x2(cs[i], cs[i])));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint64_t co = f32x2(cs[2 * i], cs[2 * i + 1]);
                    const uint64_t si = f32x2(sn[2 * i], sn[2 * i + 1]), ni = f32x2(-sn[2 * i], -sn[2 * i + 1]);
                    const uint64_t e = u[i], f = u[2 + i];
                    u[i] = fma_f32x2(f, si, mul_f32x2(e, co));
                    u[2 + i] = fma_f32x2(e, ni, mul_f32x2(f, co));
                }
            }
            if (p.norm) {
                uint64_t v[4];
                unpack_pairs<kBF16>(xa[h], v);
                unpack_pairs<kBF16>(xb[h], v + 2);
                const float ss = sum_pairs(fma_f32x2(v[0], v[0], mul_f32x2(v[1], v[1])), fma_f32x2(v[2], v[2], mul_f32x2(v[3], v[3])));
                const float r = rsqrtf(group_sum<kLanes>(ss) * (1.f / D) + p.eps);
                const uint64_t r2 = f32x2(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = mul_f32x2(v[i], r2);
                    if (h < n_heads)
                        dw[i] = fma_f32x2(u[i], v[i], dw[i]);
                    u[i] = mul_f32x2(u[i], w[i]);
                }
                float along = sum_pairs(fma_f32x2(u[0], v[0], mul_f32x2(u[1], v[1])), fma_f32x2(u[2], v[2], mul_f32x2(u[3], v[3])));
                along = group_sum<kLanes>(along) * (-1.f / D);
                const uint64_t al = f32x2(along, along);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    u[i] = mul_f32x2(r2, fma_f32x2(v[i], al, u[i]));
            }
            if (h < n_heads) {
                *reinterpret_cast<uint2*>(y + h * sd.y_sh + a) = pack_pairs<kBF16>(u);
                *reinterpret_cast<uint2*>(y + h * sd.y_sh + c) = pack_pairs<kBF16>(u + 2);
            }
        }
    }
    if (!p.part)
        return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float e, f;
        f32x2_split(dw[i], e, f);
        const int at = i < 2 ? a + 2 * i : c + 2 * (i - 2);
        sums[group][at] = e;
        sums[group][at + 1] = f;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kBwdThreads) {
        float t = 0.f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            t += sums[g][d];
        p.part[(long long)blockIdx.x * D + d] = t;
    }
}

// dw of each side: the sum of its blocks' rows, 16 columns a block, in an
// order that the sizes alone fix.
constexpr int kDwCols = 16;
constexpr int kDwThreads = 512;

__global__ void __launch_bounds__(kDwThreads) norm_dw_kernel(const NormRopeParams p, int D)
{
    constexpr int kSlices = kDwThreads / kDwCols;
    __shared__ float sums[kSlices][kDwCols];
    grid_dependency_wait();
    grid_launch_dependents();
    const int k = blockIdx.y;
    const int col = threadIdx.x % kDwCols;
    const int slice = threadIdx.x / kDwCols;
    const int d = blockIdx.x * kDwCols + col;
    const float* part = p.part + (long long)(k ? p.blocks[0] : 0) * D;
    float t = 0.f;
    for (int i = slice; i < p.blocks[k]; i += kSlices)
        t += part[(long long)i * D + d];
    sums[slice][col] = t;
    __syncthreads();
    if (slice == 0 && p.dw[k]) {
        for (int i = 1; i < kSlices; ++i)
            t += sums[i][col];
        p.dw[k][d] = t;
    }
}

}  // namespace rope
}  // namespace sdpa
