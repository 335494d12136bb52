// rope.cuh -- rows of one head as the rotation kernels hold them.
//
// A row of D 16-bit elements is held by a group of D / 8 lanes, 8 elements
// each: two runs of four, `a` and `b`.  The rotation turns pairs of channels,
// of the first `rot` of the row:
//     (x, y) -> (x cos - y sin, x sin + y cos),
// pair i by the angle of table entry [position][i], in one of two orders:
//   halves       pair i is channels (i, i + rot / 2); lane l < rot / 8 holds
//                a = channels 4 l .. 4 l + 3 and b = the same + rot / 2
//   interleaved  pair i is channels (2 i, 2 i + 1); lane l holds 8 l .. 8 l + 7
// In both orders lane l needs pairs 4 l .. 4 l + 3: 32 consecutive bytes of
// the (cos, sin) table.  Lanes l >= rot / 8 hold the channels 8 l .. 8 l + 7
// behind the rotated ones, which stay as they are (cos = 1, sin = 0), so
// rot % 8 == 0 keeps every pair inside one lane and no exchange is needed.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sdpa_kernel.cuh"

namespace sdpa {
namespace rope {

// Error codes of the device error word.
enum : unsigned int { kErrPosition = 0x701 };      // a position outside the rotation table

// First channels of a lane's two runs.
template <bool kInter>
__device__ __forceinline__ void lane_channels(int lane, int rot, int& a, int& b)
{
    if (kInter || 8 * lane >= rot) {
        a = 8 * lane;
        b = 8 * lane + 4;
    } else {
        a = 4 * lane;
        b = 4 * lane + rot / 2;
    }
}

template <bool kBF16>
__device__ __forceinline__ void unpack4(uint2 v, float* x)
{
    if constexpr (kBF16) {
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
        const float2 p = f16x2_to_f32x2(v.x), q = f16x2_to_f32x2(v.y);
        x[0] = p.x;
        x[1] = p.y;
        x[2] = q.x;
        x[3] = q.y;
    }
}

template <bool kBF16>
__device__ __forceinline__ uint2 pack4(const float* x)
{
    return make_uint2(pack2<kBF16>(x[0], x[1]), pack2<kBF16>(x[2], x[3]));
}

// The same as packed pairs of neighbours.
template <bool kBF16>
__device__ __forceinline__ void unpack_pairs(uint2 v, uint64_t* x)
{
    float f[4];
    unpack4<kBF16>(v, f);
    x[0] = f32x2(f[0], f[1]);
    x[1] = f32x2(f[2], f[3]);
}

template <bool kBF16>
__device__ __forceinline__ uint2 pack_pairs(const uint64_t* x)
{
    float f[4];
    f32x2_split(x[0], f[0], f[1]);
    f32x2_split(x[1], f[2], f[3]);
    return pack4<kBF16>(f);
}

__device__ __forceinline__ float sum_pairs(uint64_t a, uint64_t b)
{
    float e, f;
    f32x2_split(add_f32x2(a, b), e, f);
    return e + f;
}

// cos and sin of a lane's four pairs (1 and 0 for lanes behind `rot`).
__device__ __forceinline__ void lane_angles(const float* table, int pos, int rot, int lane, float* cs, float* sn)
{
    if (8 * lane < rot) {
        const float4* t = reinterpret_cast<const float4*>(table + (int64_t)pos * rot + 8 * lane);
        const float4 u = __ldg(t), v = __ldg(t + 1);
        cs[0] = u.x; sn[0] = u.y; cs[1] = u.z; sn[1] = u.w;
        cs[2] = v.x; sn[2] = v.y; cs[3] = v.z; sn[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cs[i] = 1.f;
            sn[i] = 0.f;
        }
    }
}

// Rotates a lane's 8 elements x = {a run, b run} in place.
template <bool kInter>
__device__ __forceinline__ void rotate(float* x, const float* cs, const float* sn)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = kInter ? 2 * i : i, q = kInter ? 2 * i + 1 : i + 4;
        const float u = x[p], v = x[q];
        x[p] = u * cs[i] - v * sn[i];
        x[q] = u * sn[i] + v * cs[i];
    }
}

// Sum over the kLanes lanes of a row's group (every lane gets it; the order
// of the additions is fixed).
template <int kLanes>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

}  // namespace rope
}  // namespace sdpa
