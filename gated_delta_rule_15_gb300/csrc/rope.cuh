// rope.cuh -- device helpers of the kernels that normalise and rotate rows: 8 storage elements of a
// row a lane, their angles and their pairs' other values.  `Args` has the rotation as members
// rot, table (dr_rope_table) and scale.
#pragma once

#include "common.cuh"

namespace dr {

template <typename T> struct Vec8;   // 8 storage elements
template <> struct Vec8<float> { float4 a, b; };
template <> struct Vec8<__nv_bfloat16> { uint4 a; };

__device__ __forceinline__ Vec8<float> ld8(const float *p) {
    return {*reinterpret_cast<const float4 *>(p), *reinterpret_cast<const float4 *>(p + 4)};
}
__device__ __forceinline__ Vec8<__nv_bfloat16> ld8(const __nv_bfloat16 *p) { return {*reinterpret_cast<const uint4 *>(p)}; }
__device__ __forceinline__ void unpack(const Vec8<float> &v, float (&f)[8]) {
    f[0] = v.a.x; f[1] = v.a.y; f[2] = v.a.z; f[3] = v.a.w;
    f[4] = v.b.x; f[5] = v.b.y; f[6] = v.b.z; f[7] = v.b.w;
}
__device__ __forceinline__ void unpack(const Vec8<__nv_bfloat16> &v, float (&f)[8]) {
    const uint32_t u[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // bf16 is the upper half of fp32
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ Vec8<float> shfl8(const Vec8<float> &v, int src) {
    Vec8<float> o;
    o.a.x = __shfl_sync(0xffffffffu, v.a.x, src); o.a.y = __shfl_sync(0xffffffffu, v.a.y, src);
    o.a.z = __shfl_sync(0xffffffffu, v.a.z, src); o.a.w = __shfl_sync(0xffffffffu, v.a.w, src);
    o.b.x = __shfl_sync(0xffffffffu, v.b.x, src); o.b.y = __shfl_sync(0xffffffffu, v.b.y, src);
    o.b.z = __shfl_sync(0xffffffffu, v.b.z, src); o.b.w = __shfl_sync(0xffffffffu, v.b.w, src);
    return o;
}
__device__ __forceinline__ Vec8<__nv_bfloat16> shfl8(const Vec8<__nv_bfloat16> &v, int src) {
    Vec8<__nv_bfloat16> o;
    o.a.x = __shfl_sync(0xffffffffu, v.a.x, src); o.a.y = __shfl_sync(0xffffffffu, v.a.y, src);
    o.a.z = __shfl_sync(0xffffffffu, v.a.z, src); o.a.w = __shfl_sync(0xffffffffu, v.a.w, src);
    return o;
}
__device__ __forceinline__ void st8(float *p, const float (&f)[8]) {
    store4(p, make_float4(f[0], f[1], f[2], f[3]));
    store4(p + 4, make_float4(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ void st8(__nv_bfloat16 *p, const float (&f)[8]) {
    uint4 u;
    uint32_t *w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = u;
}

// Of this lane's 8 values: the cosine (times c) of each one's pair and the signed sine (times c) its
// pair's other value enters with, for a rotation forwards or back; 1 and 0 behind the rotated part.
template <bool HALF, class Args>
__device__ __forceinline__ void angles(const Args &a, int64_t pos, int l, bool back, float (&co)[8], float (&si)[8]) {
    constexpr int NP = HALF ? 8 : 4;
    const int hr = a.rot / 2, i0 = HALF ? (8 * l < hr ? 8 * l : 8 * l - hr) : 4 * l;
    if (8 * l >= a.rot) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            co[e] = 1.f;
            si[e] = 0.f;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < NP; ++e) {
        const uint64_t turn = (uint64_t)pos * __ldg(a.table + i0 + e);
        // signed upper half: [-1/2, 1/2) turns, i.e. that many times 2 pi
        const float half_turns = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;   // 2^-31
        float s, c;
        sincospif(half_turns, &s, &c);
        c *= a.scale;
        s *= back ? -a.scale : a.scale;
        if (HALF) {
            co[e] = c;
            si[e] = 8 * l < hr ? -s : s;
        } else {
            co[2 * e] = co[2 * e + 1] = c;
            si[2 * e] = -s;
            si[2 * e + 1] = s;
        }
    }
}

// The lane that holds the other values of this lane's pairs (half layout).
template <bool HALF, class Args>
__device__ __forceinline__ int partner(const Args &a, int lane, int l) {
    return HALF && 8 * l < a.rot ? (16 * l < a.rot ? lane + a.rot / 16 : lane - a.rot / 16) : lane;
}
// Each value's pair's other one.
template <bool HALF, typename T>
__device__ __forceinline__ void others(const Vec8<T> &raw, const float (&x)[8], int src, float (&o)[8]) {
    if (HALF) {
        const Vec8<T> v = shfl8(raw, src);
        unpack(v, o);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = x[e ^ 1];
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

}  // namespace dr
