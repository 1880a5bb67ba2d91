// Vectors of 64 to 512 elements spread over D / 16 lanes, 16 consecutive elements
// each: loads, the Hadamard transform and 4-bit groups, as the kernels that write
// pages or prepare queries take them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "codes.h"

namespace hr {
namespace {

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}

// the value of lane ^ X (X = 1, 2, 4, 8 inside 16 lanes, 16 inside 32)
template <int X>
__device__ __forceinline__ float lane_xor(float v) {
    if constexpr (X == 1) return dpp<0xB1>(v);         // quad_perm [1,0,3,2]
    if constexpr (X == 2) return dpp<0x4E>(v);         // quad_perm [2,3,0,1]
    if constexpr (X == 4) return dpp<0x141>(dpp<0x1B>(v));  // quad_perm [3,2,1,0], then the row's half mirrored: ^ 3 ^ 7
    if constexpr (X == 8) return dpp<0x128>(v);         // row_ror 8
    return __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));   // lane ^ 16
}

template <int LANES, class F>
__device__ __forceinline__ float over_lanes(float v, F f) {
    if constexpr (LANES >= 2) v = f(v, lane_xor<1>(v));
    if constexpr (LANES >= 4) v = f(v, lane_xor<2>(v));
    if constexpr (LANES >= 8) v = f(v, lane_xor<4>(v));
    if constexpr (LANES >= 16) v = f(v, lane_xor<8>(v));
    if constexpr (LANES >= 32) v = f(v, lane_xor<16>(v));
    return v;
}

// (a product with 1 or -1 is exact, and costs less than a selection; the move
// between lanes is part of the addition)
template <int X>
__device__ __forceinline__ void lane_stage(float (&v)[16], int lane) {
#pragma clang fp contract(off)
    const float sign = (lane & X) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = lane_xor<X>(v[i]) + v[i] * sign;
}

template <int D>
__device__ __forceinline__ void hadamard(float (&v)[16], int lane, float norm) {
#pragma unroll
    for (int s = 1; s < 16; s *= 2)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (!(i & s)) {
                const float x = v[i], y = v[i + s];
                v[i] = x + y;
                v[i + s] = x - y;
            }
    lane_stage<1>(v, lane);
    lane_stage<2>(v, lane);
    if constexpr (D >= 128) lane_stage<4>(v, lane);
    if constexpr (D >= 256) lane_stage<8>(v, lane);
    if constexpr (D >= 512) lane_stage<16>(v, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= norm;
}

template <class T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4v x = reinterpret_cast<const uint4v*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __uint_as_float(x[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4v x = reinterpret_cast<const uint4v*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = __uint_as_float(x[j]);
        }
    }
}

// The codes of 16 elements y: quotient(y) is y / s, rounded to an integer.
// Codes are packed as float32, four of them to an integer below 2^16; symmetric
// ones with 8 added, which an XOR takes back.
template <bool SYM, class Q>
__device__ __forceinline__ uint2v pack_codes(const float (&v)[16], float z, Q quotient) {
#pragma clang fp contract(off)
    uint2v w;
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
        uint32_t half[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                const float q = quotient(v[i + 4 * j + k]);
                const float c = __builtin_amdgcn_fmed3f(q + z, 0.0f, 15.0f);   // (NaN: 0)
                sum = k == 3 ? c : __builtin_fmaf(sum, 16.0f, c);
            }
            half[j] = static_cast<uint32_t>(sum);
        }
        w[i / 8] = (half[1] << 16 | half[0]) ^ (SYM ? 0x88888888u : 0u);
    }
    return w;
}

// Quantizes the lane's 16 elements: scale s = range / steps of the group,
// stored (f32 or nearest-even bf16), codes from the stored scale.  A group with
// a NaN has a NaN scale, so that whoever reads it sees one.  y / s is the
// correctly rounded quotient: one division gives r = 1 / s, and with t = y r the
// remainder fma(-t, s, y) is exact, so fma(remainder, r, t) rounds to y / s (P.
// Markstein, IBM J. Res. Dev. 34, 1990).  That keeps every code equal to the
// definition's, ties included, at two more instructions than a product with the
// reciprocal.  Where r or the remainder could leave the normal numbers, and for
// scales that are not finite, each element is divided.
template <int LANES, bool SYM>
__device__ __forceinline__ uint2v quantize(const float (&v)[16], bool sf32, uint32_t* scale, uint32_t* zero) {
#pragma clang fp contract(off)
    float s, z = 0.0f;
    bool nan;
    if constexpr (SYM) {
        float top = fabsf(v[0]);
#pragma unroll
        for (int i = 1; i < 16; ++i) top = __builtin_elementwise_maximum(top, fabsf(v[i]));   // (keeps a NaN)
        nan = top != top;
        top = over_lanes<LANES>(top, [](float a, float b) { return fmaxf(a, b); });
        s = top / 7.0f;
    } else {
        float lo = fminf(v[0], 0.0f), hi = __builtin_elementwise_maximum(v[0], 0.0f);
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            lo = fminf(lo, v[i]);
            hi = __builtin_elementwise_maximum(hi, v[i]);
        }
        nan = hi != hi;
        lo = over_lanes<LANES>(lo, [](float a, float b) { return fminf(a, b); });
        hi = over_lanes<LANES>(hi, [](float a, float b) { return fmaxf(a, b); });
        s = (hi - lo) / 15.0f;
        z = lo;
    }
    if (s == 0.0f) s = 1.0f;
    const bool odd = __any(nan || !(s >= 0x1p-64f && s <= 0x1p64f));
    if (odd && over_lanes<LANES>(nan ? 1.0f : 0.0f, [](float a, float b) { return fmaxf(a, b); }) != 0.0f)
        s = __uint_as_float(0x7FC00000u);
    if (sf32) {
        *scale = __float_as_uint(s);
    } else {
        *scale = f2bf(s);
        s = bf2f(*scale);
    }
    if constexpr (SYM) {
        z = 8.0f;
    } else {
        z = fminf(fmaxf(rintf(-z / s), 0.0f), 15.0f);
        *zero = static_cast<uint32_t>(static_cast<int>(z));
    }
    if (odd) return pack_codes<SYM>(v, z, [s](float y) { return rintf(y / s); });
    const float r = 1.0f / s;
    return pack_codes<SYM>(v, z, [s, r](float y) {
        const float t = y * r;
        return rintf(__builtin_fmaf(__builtin_fmaf(-t, s, y), r, t));
    });
}

}  // namespace
}  // namespace hr
