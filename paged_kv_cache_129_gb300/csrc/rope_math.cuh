// Rotary angles and the chunks of a head row that the rotary kernels work on.
//
// Angles of far positions: p * inv_freq in float32 is off by p * 2^-24 radians, useless at p = 10^6.  A turn is
// therefore a 64-bit fixed-point fraction: u = frac(inv_freq / 2 pi) * 2^64, rounded to half a unit (a double alone would be off
// by 2^-54 of the quotient, 2^-25 turns at p = 2^31), and p * u modulo 2^64 is the angle in turns without whole ones, off by
// p * 2^-65.  Its distance from the nearest quarter turn, at most an eighth, goes to sincospi in
// float32, off by 2^-28 turns at most, and the quarters swap and negate (the whole angle in float32 would be off by 2^-26: rotated
// float32 rows 4.0e-8 from the exact ones instead of 2.8e-8).  One integer product per angle.
#pragma once

#include <cstdint>

#include "pa_common.cuh"

namespace pa {

// u of an angle per position (of magnitude below 2^30).  1 / 2 pi is the sum of two doubles, and an fma gives what the first's product
// was rounded by.
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
    const double x = fabs(inv_freq), high = x * 0.15915494309189535;
    const double low = fma(x, -9.839338337591243e-18, fma(x, 0.15915494309189535, -high));
    const double units = (high - floor(high)) * 18446744073709551616.0;  // * 2^64, below it
    const double whole = floor(units);
    const uint64_t u = __double2ull_rz(whole) + (uint64_t)__double2ll_rn(fma(low, 18446744073709551616.0, units - whole));
    return inv_freq < 0.0 ? 0 - u : u;
}

__device__ __forceinline__ float2 turn(uint64_t step, int pos, float factor) {
    const uint64_t a = step * (uint64_t)(int64_t)pos;
    const unsigned quarters = (unsigned)((a + (1ull << 61)) >> 62);
    const int rest = (int)((int64_t)(a - ((uint64_t)quarters << 62) + 0x80000000ull) >> 32);
    float s, c;
    sincospif((float)rest * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    if (quarters & 1) {
        const float x = c;
        c = -s;
        s = x;
    }
    if (quarters & 2) {
        c = -c;
        s = -s;
    }
    return make_float2(c * factor, s * factor);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 x);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float2 x) {
    const __half2 h = __float22half2_rn(x);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 x) {
    const __nv_bfloat162 h = __float22bfloat162_rn(x);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// VB bytes = V elements of type T, taken two at a time where there are two: elements of 16 bits one at a time would occupy a
// register each.
template <typename T, int VB>
struct Chunk {
    static constexpr int V = VB / (int)sizeof(T), W = VB < 4 ? 1 : VB / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VB == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else if constexpr (VB == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (VB == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (VB == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
        else *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
    // elements 2i and 2i + 1
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return unpack2<T>(w[i]);
    }
    __device__ __forceinline__ void put(int i, float2 x) {
        if constexpr (sizeof(T) == 4) w[2 * i] = __float_as_uint(x.x), w[2 * i + 1] = __float_as_uint(x.y);
        else w[i] = pack2<T>(x);
    }
    // the element of a chunk of one
    __device__ __forceinline__ float one() const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[0]);
        else return unpack2<T>(w[0]).x;
    }
    __device__ __forceinline__ void put_one(float x) {
        if constexpr (sizeof(T) == 4) w[0] = __float_as_uint(x);
        else w[0] = pack2<T>(make_float2(x, 0.f));
    }
};

}  // namespace pa
