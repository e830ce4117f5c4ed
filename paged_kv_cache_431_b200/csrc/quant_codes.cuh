// quant_codes.cuh -- the codes of quantized pools: rounding a value to a code, re-rounding a code
// to a larger scale, and packing.  IEEE fp32 with explicit round-to-nearest operations
// throughout, shared by every kernel that writes codes.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace pkv {

// The largest code of storage dtype DT: a tile's scale is its largest |x| over this.
template <int DT>
__device__ __forceinline__ constexpr float quant_limit()
{
    return DT == PKV_INT8 ? 127.f : DT == PKV_INT4 ? 7.f : 448.f;
}

// Code of x / s for storage dtype DT, IEEE fp32 round-to-nearest throughout.
template <int DT>
__device__ __forceinline__ uint32_t quant_code(float x, float s)
{
    if (s == 0.f) return 0u;
    const float r = __fdiv_rn(x, s);
    if constexpr (DT == PKV_FP8E4M3) {
        return (uint32_t)__nv_cvt_float_to_fp8(r, __NV_SATFINITE, __NV_E4M3);
    } else {
        constexpr float Q = DT == PKV_INT8 ? 127.f : 7.f;
        const float c = fminf(fmaxf(rintf(r), -Q), Q);
        return (uint32_t)(int)c & (DT == PKV_INT8 ? 0xffu : 0xfu);
    }
}

template <int DT>
__device__ __forceinline__ float code_value(uint32_t c)
{
    if constexpr (DT == PKV_FP8E4M3) {
        return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
    } else if constexpr (DT == PKV_INT8) {
        return (float)(int)(int8_t)c;
    } else {
        return (float)(((int)c ^ 8) - 8);   // 4-bit two's complement
    }
}

template <int DT>
__device__ __forceinline__ uint32_t requant_code(uint32_t c, float s_old, float s)
{
    const float r = __fdiv_rn(__fmul_rn(code_value<DT>(c), s_old), s);
    if constexpr (DT == PKV_FP8E4M3) {
        return (uint32_t)__nv_cvt_float_to_fp8(r, __NV_SATFINITE, __NV_E4M3);
    } else {
        constexpr float Q = DT == PKV_INT8 ? 127.f : 7.f;
        const float q = fminf(fmaxf(rintf(r), -Q), Q);
        return (uint32_t)(int)q & (DT == PKV_INT8 ? 0xffu : 0xfu);
    }
}

// Four codes of neighbouring elements, little-endian: a 32-bit word of bytes, or (int4) 16 bits
// of nibbles, the first element lowest.
template <int DT>
__device__ __forceinline__ uint32_t pack_codes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    constexpr int S = DT == PKV_INT4 ? 4 : 8;
    return a | (b << S) | (c << (2 * S)) | (d << (3 * S));
}

template <int DT>
__device__ __forceinline__ uint32_t code_at(uint32_t w, int i)
{
    return DT == PKV_INT4 ? (w >> (4 * i)) & 0xfu : (w >> (8 * i)) & 0xffu;
}

// The packed codes of elements d .. d + 3 (d a multiple of 4) of a row.
template <int DT>
__device__ __forceinline__ uint32_t load_codes4(const uint8_t* row, int d)
{
    if constexpr (DT == PKV_INT4) return *reinterpret_cast<const uint16_t*>(row + d / 2);
    else return *reinterpret_cast<const uint32_t*>(row + d);
}

template <int DT>
__device__ __forceinline__ void store_codes4(uint8_t* row, int d, uint32_t w)
{
    if constexpr (DT == PKV_INT4) *reinterpret_cast<uint16_t*>(row + d / 2) = (uint16_t)w;
    else *reinterpret_cast<uint32_t*>(row + d) = w;
}

// The packed codes of four elements over a scale s that they share, without four divisions.  With
// inv = fl(1 / s), r = fl(x inv) is off the rounded quotient fl(x / s) by less than 2^-22 of it (three
// roundings of 2^-24), and the code is a monotonic function of the quotient: so where the codes of
// r (1 - 2^-22) and r (1 + 2^-22) agree, that is the code; where one of the four does not (a quotient
// next to a border, a NaN), the divisions decide.  inv must be finite, and |x| <= s * the limit for
// finite x, so that no clamp is needed.
template <int DT>
__device__ __forceinline__ uint32_t quant_codes4(const float (&x)[4], float s, float inv)
{
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __fmul_rn(x[i], inv);
    constexpr float LO = 1.f - 0x1p-22f, HI = 1.f + 0x1p-22f;
    uint32_t w;
    bool same;
    if constexpr (DT == PKV_FP8E4M3) {
        auto pair = [](float a, float b) -> uint32_t {
            return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        };
        w = pair(r[0] * LO, r[1] * LO) | (pair(r[2] * LO, r[3] * LO) << 16);
        same = w == (pair(r[0] * HI, r[1] * HI) | (pair(r[2] * HI, r[3] * HI) << 16));
    } else {
        // the nearest integer in the low bits of r + 1.5 x 2^23
        constexpr float M = 12582912.f;
        uint32_t n[4];
        same = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = __fmaf_rn(r[i], LO, M), hi = __fmaf_rn(r[i], HI, M);
            same = same && lo == hi;
            n[i] = __float_as_uint(lo) & (DT == PKV_INT8 ? 0xffu : 0xfu);
        }
        w = pack_codes<DT>(n[0], n[1], n[2], n[3]);
    }
    if (same) return w;
    return pack_codes<DT>(quant_code<DT>(x[0], s), quant_code<DT>(x[1], s), quant_code<DT>(x[2], s), quant_code<DT>(x[3], s));
}

}  // namespace pkv
