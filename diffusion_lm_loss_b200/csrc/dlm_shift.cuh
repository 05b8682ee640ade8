// dlm_shift.cuh -- rows that start anywhere, by 16-byte accesses.
//
// A warp takes M stretches of 256 consecutive elements of a row, lane l the
// pieces of 8 elements from column c + 256 m on (c = its column in the first
// stretch, c - 8 l a multiple of 256 M).  In memory the pieces lie `sh`
// elements behind a border; sh is the same for all of them.  Loads take the
// aligned chunks, of which a piece needs its own and the next lane's (one
// shuffle per word), and move them by sh; stores put the end of the lane
// before and the lane's own start into one aligned chunk.  Only the chunks at
// the two ends of the stretches and of the row go by element.  By single
// elements throughout, packing 8,192 rows of 5,001 took 2.5 times as long.
#pragma once

#include "dlm_device.cuh"

namespace dlm {

// elements sh .. sh + 7 of the 16 in a, b (sh in 1..7)
__device__ __forceinline__ uint4 funnel16(uint4 a, uint4 b, int sh) {
    uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
    if (sh & 4) { w[0] = w[2]; w[1] = w[3]; w[2] = w[4]; w[3] = w[5]; w[4] = w[6]; w[5] = b.w; }
    if (sh & 2) { w[0] = w[1]; w[1] = w[2]; w[2] = w[3]; w[3] = w[4]; w[4] = w[5]; }
    const uint32_t sel = sh & 1 ? 0x5432u : 0x3210u;
    return make_uint4(__byte_perm(w[0], w[1], sel), __byte_perm(w[1], w[2], sel), __byte_perm(w[2], w[3], sel),
                      __byte_perm(w[3], w[4], sel));
}
// bytes sh .. sh + 7 of the 16 in a, b (sh in 1..7)
__device__ __forceinline__ uint2 funnel8(uint2 a, uint2 b, int sh) {
    uint32_t w[3] = {a.x, a.y, b.x};
    if (sh & 4) { w[0] = w[1]; w[1] = w[2]; w[2] = b.y; }
    return make_uint2(__funnelshift_r(w[0], w[1], 8 * (sh & 3)), __funnelshift_r(w[1], w[2], 8 * (sh & 3)));
}

__device__ __forceinline__ uint4 shfl(uint4 v, int src) {
    return make_uint4(__shfl_sync(~0u, v.x, src), __shfl_sync(~0u, v.y, src), __shfl_sync(~0u, v.z, src),
                      __shfl_sync(~0u, v.w, src));
}
__device__ __forceinline__ uint2 shfl(uint2 v, int src) {
    return make_uint2(__shfl_sync(~0u, v.x, src), __shfl_sync(~0u, v.y, src));
}
__device__ __forceinline__ uint4 funnel(uint4 a, uint4 b, int sh) { return funnel16(a, b, sh); }
__device__ __forceinline__ uint2 funnel(uint2 a, uint2 b, int sh) { return funnel8(a, b, sh); }

// element e of a piece
__device__ __forceinline__ uint16_t piece_at(uint4 v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return uint16_t(w >> (16 * (e & 1)));
}
__device__ __forceinline__ uint8_t piece_at(uint2 v, int e) { return uint8_t((e < 4 ? v.x : v.y) >> (8 * (e & 3))); }

// The element type E (16-bit or 8-bit) and the type P of 8 of them.
template <typename E> struct Piece;
template <> struct Piece<uint16_t> { using type = uint4; };
template <> struct Piece<uint8_t> { using type = uint2; };

// An aligned chunk; of a chunk that is not wholly inside [begin, end), the
// elements that are, and zeros.
template <typename E>
__device__ __forceinline__ typename Piece<E>::type load_chunk(const E* p, const E* begin, const E* end) {
    using P = typename Piece<E>::type;
    if (p >= begin && p + 8 <= end) return __ldg(reinterpret_cast<const P*>(p));
    uint32_t w[4] = {0, 0, 0, 0};
    constexpr int kPer = 4 / int(sizeof(E)), kBits = 8 * int(sizeof(E));
    #pragma unroll
    for (int e = 0; e < 8; ++e)
        if (p + e >= begin && p + e < end) w[e / kPer] |= uint32_t(__ldg(p + e)) << (kBits * (e % kPer));
    P v;
    if constexpr (sizeof(E) == 2) v = make_uint4(w[0], w[1], w[2], w[3]);
    else v = make_uint2(w[0], w[1]);
    return v;
}

// v[m] = elements p[256 m .. 256 m + 7]; what lies behind column d - 1 is
// anything.  begin, end: the tensor.
template <int M, typename E>
__device__ __forceinline__ void load_pieces(const E* p, int c, int d, const E* begin, const E* end,
                                            typename Piece<E>::type (&v)[M]) {
    using P = typename Piece<E>::type;
    const int lane = threadIdx.x & 31;
    const int sh = int((reinterpret_cast<uintptr_t>(p) & (sizeof(P) - 1)) / sizeof(E));
    #pragma unroll
    for (int m = 0; m < M; ++m)
        v[m] = c + 256 * m - sh < d ? load_chunk(p + 256 * m - sh, begin, end) : P{};
    if (sh == 0) return;
    P last = {};                             // the chunk behind the last lane's
    if (lane == 31 && c + 256 * (M - 1) + 8 - sh < d) last = load_chunk(p + 256 * (M - 1) + 8 - sh, begin, end);
    #pragma unroll
    for (int m = 0; m < M; ++m) {
        P next = shfl(lane == 0 && m + 1 < M ? v[m + 1 < M ? m + 1 : m] : v[m], (lane + 1) & 31);
        if (m + 1 == M && lane == 31) next = last;
        v[m] = funnel(v[m], next, sh);
    }
}

// p[256 m .. 256 m + 7] = v[m], up to column d - 1.
template <int M, typename E>
__device__ __forceinline__ void store_pieces(E* p, int c, int d, const typename Piece<E>::type (&v)[M]) {
    using P = typename Piece<E>::type;
    const int lane = threadIdx.x & 31, first = c - 8 * lane;
    const int sh = int((reinterpret_cast<uintptr_t>(p) & (sizeof(P) - 1)) / sizeof(E));
    #pragma unroll
    for (int m = 0; m < M; ++m) {
        P w = v[m];
        if (sh) {
            const P before = shfl(lane == 31 && m > 0 ? v[m > 0 ? m - 1 : 0] : v[m], (lane + 31) & 31);
            w = funnel(before, v[m], 8 - sh);
        }
        const int c0 = c + 256 * m - sh;
        E* at = p + 256 * m - sh;
        if (c0 >= first && c0 + 8 <= d) {
            *reinterpret_cast<P*>(at) = w;
        } else {
            #pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c0 + e >= first && c0 + e < d) at[e] = piece_at(w, e);
        }
    }
    if (sh && lane == 31) {                  // the end of the last lane's piece
        const int c0 = c + 256 * (M - 1);
        #pragma unroll
        for (int e = 1; e < 8; ++e)
            if (e >= 8 - sh && c0 + e < d) p[256 * (M - 1) + e] = piece_at(v[M - 1], e);
    }
}

// zeros from column d on
__device__ __forceinline__ uint4 clip_piece(uint4 v, int c, int d) {
    if (c + 8 <= d) return v;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] &= (c + 2 * k < d ? 0xffffu : 0u) | (c + 2 * k + 1 < d ? 0xffff0000u : 0u);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace dlm
