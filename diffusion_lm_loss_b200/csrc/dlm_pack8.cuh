// dlm_pack8.cuh -- the 8-bit form of an activation: blocks of
// DLM_PACK_BLOCK = 128 columns of a row share one fp32 factor.
//
// With a = max |x| over the block and top = 127 (int8) or 448 (e4m3):
//   inv = fl(top / a), code = rint(fl(x * inv)) or e4m3(fl(x * inv)),
//   scale = fl(a / top), value = code * scale.
// The divisions and the product are IEEE fp32 operations, so the code of an
// element is defined bit for bit.  a < 2^-100 (where top / a would leave
// fp32's range) is held as zeros, scale 0.  A block with an infinity or a NaN
// gets scale NaN and codes 0: all of it reads back as NaN, so that a failed
// step stays visible.
#pragma once

#include <cuda_fp8.h>

#include "dlm_device.cuh"

namespace dlm {

struct PackFactors { float inv, scale; };

__device__ __forceinline__ PackFactors pack_factors(float amax, int format) {
    const float top = format == DLM_PACK_INT8 ? 127.f : 448.f;
    PackFactors f;
    if (!(amax < __int_as_float(0x7f800000))) { f.inv = 0.f; f.scale = __int_as_float(0x7fc00000); }
    else if (amax < 0x1p-100f) { f.inv = 0.f; f.scale = 0.f; }
    else { f.inv = __fdiv_rn(top, amax); f.scale = __fdiv_rn(amax, top); }
    return f;
}

// Code of one element.  inv = 0 (a block held as zeros or NaN) gives code 0
// whatever x is: the caller passes 0 for x there.
__device__ __forceinline__ uint32_t pack_code(float x, float inv, int format) {
    const float u = __fmul_rn(x, inv);
    if (format == DLM_PACK_INT8) return uint32_t(__float2int_rn(u)) & 0xffu;
    return uint32_t(__nv_cvt_float_to_fp8(u, __NV_SATFINITE, __NV_E4M3));
}

// Four codes (as consecutive bytes) back to fp32, before the scale.
__device__ __forceinline__ void unpack_codes(uint32_t w, int format, float (&v)[4]) {
    if (format == DLM_PACK_INT8) {
        #pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = float(int(w << (24 - 8 * k)) >> 24);
    } else {
        #pragma unroll
        for (int k = 0; k < 2; ++k) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> (16 * k)), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            v[2 * k] = f.x; v[2 * k + 1] = f.y;
        }
    }
}

__device__ __forceinline__ float unpack_code(uint8_t c, int format) {
    if (format == DLM_PACK_INT8) return float(int8_t(c));
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(c), __NV_E4M3)));
}

// max |.| of 8 bf16 as fp32; a NaN among them comes back as NaN.
__device__ __forceinline__ float absmax8(uint4 r) {
    auto b = [](uint32_t w) { w &= 0x7fff7fffu; return *reinterpret_cast<__nv_bfloat162*>(&w); };
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(b(r.x), b(r.y)), __hmax2_nan(b(r.z), b(r.w)));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&m) & 0x7fff7fffu;
    // non-negative patterns order like their values, NaN above infinity
    return __uint_as_float(max(w << 16, w & 0xffff0000u));
}

// max of non-negative floats (or NaN) over groups of 16 lanes
__device__ __forceinline__ float absmax_half_warp(float a) {
    uint32_t u = __float_as_uint(a);
    #pragma unroll
    for (int o = 8; o; o >>= 1) u = max(u, __shfl_xor_sync(~0u, u, o));
    return __uint_as_float(u);
}

// Codes of 8 bf16 with the block's factors: 8 bytes.
__device__ __forceinline__ uint2 pack8_codes(uint4 r, PackFactors f, int format) {
    const uint32_t x[4] = {r.x, r.y, r.z, r.w};
    uint32_t c[4];
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float lo = f.inv != 0.f ? bf16lo(x[k]) : 0.f, hi = f.inv != 0.f ? bf16hi(x[k]) : 0.f;
        c[k] = pack_code(lo, f.inv, format) | pack_code(hi, f.inv, format) << 8;
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

}  // namespace dlm
