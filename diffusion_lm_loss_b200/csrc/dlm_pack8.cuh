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

__device__ __forceinline__ float unpack_code(uint8_t c, int format) {
    if (format == DLM_PACK_INT8) return float(int8_t(c));
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(c), __NV_E4M3)));
}

// Four codes (consecutive bytes) back to two fp32 pairs, before the scale.
// An integer code c goes into the fraction of 2^23 as c + 128: one byte
// permutation per code and one packed subtraction per pair, where int -> float
// conversions run at a quarter of that rate.
__device__ __forceinline__ void unpack_codes(uint32_t w, int format, uint64_t& lo, uint64_t& hi) {
    if (format == DLM_PACK_INT8) {
        w ^= 0x80808080u;
        auto at = [&](uint32_t sel) { return __uint_as_float(__byte_perm(w, 0x4b000000u, sel)); };
        const uint64_t off = f2pack(-8388736.f, -8388736.f);      // -(2^23 + 128)
        lo = f2add(f2pack(at(0x7440), at(0x7441)), off);
        hi = f2add(f2pack(at(0x7442), at(0x7443)), off);
    } else {
        const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w), __NV_E4M3)));
        const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> 16), __NV_E4M3)));
        lo = f2pack(a.x, a.y);
        hi = f2pack(b.x, b.y);
    }
}

// max |.| of 8 bf16 as two halves of a word (even and odd elements), by their
// patterns: non-negative bf16 order like 16-bit integers, NaN above infinity.
__device__ __forceinline__ uint32_t absmax8(uint4 r) {
    const uint32_t m = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(r.x & m, r.y & m), __vmaxu2(r.z & m, r.w & m));
}

// Packs M pieces of 8 bf16, each of 16 neighbouring lanes' m-th piece making a
// block: out[m] gets the lane's 8 codes; put(m, scale) is called by some
// lane of the 16 for each m.  The M maxima share their exchanges (each halving of
// the lanes also halves the blocks a lane carries on), and every lane divides
// for one block only.
template <int M, typename Put>
__device__ __forceinline__ void pack_pieces(const uint4 (&r)[M], int format, uint2 (&out)[M], Put&& put) {
    static_assert(M == 1 || M == 2 || M == 4, "pieces");
    const int lane = threadIdx.x & 31;
    const uint64_t zero = f2negative_zero(format);
    uint32_t a[M];
    #pragma unroll
    for (int m = 0; m < M; ++m) a[m] = absmax8(r[m]);
    int mine = 0, bit = 8;
    #pragma unroll
    for (int h = M / 2; h; h >>= 1, bit >>= 1) {
        const bool up = lane & bit;
        #pragma unroll
        for (int k = 0; k < h; ++k) {
            const uint32_t keep = up ? a[k + h] : a[k], send = up ? a[k] : a[k + h];
            a[k] = __vmaxu2(keep, __shfl_xor_sync(~0u, send, bit));
        }
        mine = 2 * mine + up;
    }
    #pragma unroll
    for (; bit; bit >>= 1) a[0] = __vmaxu2(a[0], __shfl_xor_sync(~0u, a[0], bit));
    const PackFactors f = pack_factors(__uint_as_float(max(a[0] << 16, a[0] & 0xffff0000u)), format);
    if ((lane & (16 / M - 1)) == 0) put(mine, f.scale);
    #pragma unroll
    for (int m = 0; m < M; ++m) {
        const float inv = M == 1 ? f.inv : __shfl_sync(~0u, f.inv, (lane & 16) | m * (16 / M));
        const uint64_t inv2 = f2pack(inv, inv);
        const uint32_t x[4] = {r[m].x, r[m].y, r[m].z, r[m].w};
        uint32_t c[4];
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint64_t u = f2mul_rounded(f2pack(bf16lo(x[k]), bf16hi(x[k])), inv2, zero);
            float lo, hi;
            if (format == DLM_PACK_INT8) {
                // adding 1.5 * 2^23 rounds to an integer, ties to even, and leaves it in the low bits
                u = f2add(u, f2pack(12582912.f, 12582912.f));
                f2unpack(u, lo, hi);
                c[k] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);
            } else {
                f2unpack(u, lo, hi);
                c[k] = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
            }
        }
        const bool none = inv == 0.f;               // zeros, or a block that is not finite
        out[m] = make_uint2(none ? 0u : __byte_perm(c[0], c[1], 0x5410), none ? 0u : __byte_perm(c[2], c[3], 0x5410));
    }
}

}  // namespace dlm
