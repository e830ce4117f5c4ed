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

}  // namespace pkv
