// dlm_act8.cu -- activations in 8 bits (dlm_pack8.cuh has the format):
// packing in the forward pass, unpacking in the backward pass.
//
// Both are one pass over memory: 2 bytes read and 1 written per element, or
// the reverse, and 4 bytes per 128 elements for the block's factor.  A warp
// takes slabs of 1,024 columns of a row, four pieces of 8 elements a lane;
// rows that do not start on 16-byte borders go through dlm_shift.cuh.  Bound by
// HBM: 16,384 x 4,096 packed and unpacked in 62.5 us, 0.99 of the copy rate
// (98 us with one load a lane in flight and conversions for the codes).
#include "dlm_host.h"
#include "dlm_pack8.cuh"
#include "dlm_shift.cuh"

namespace dlm {

constexpr int kActThreads = 256;

constexpr int kSlab = 1024;            // columns of a row that a warp takes at a time

// kAligned: rows of x on 16-byte and of q on 8-byte borders.
template <bool kAligned>
__global__ void __launch_bounds__(kActThreads) k_pack8(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                       int64_t ld, int format, uint8_t* __restrict__ q,
                                                       float* __restrict__ scale) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int nb = (cols + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK, slabs = (cols + kSlab - 1) / kSlab;
    const int64_t items = rows * slabs, step = int64_t(gridDim.x) * (kActThreads / 32);
    for (int64_t i = int64_t(blockIdx.x) * (kActThreads / 32) + threadIdx.x / 32; i < items; i += step) {
        const int64_t r = i / slabs;
        const int c = int(i - r * slabs) * kSlab + lane * 8;
        const uint16_t* src = x + r * ld + c;
        uint4 v[4];
        if constexpr (kAligned) {
            #pragma unroll
            for (int m = 0; m < 4; ++m)
                v[m] = c + 256 * m < cols ? __ldg(reinterpret_cast<const uint4*>(src + 256 * m)) : make_uint4(0, 0, 0, 0);
        } else {
            load_pieces<4>(src, c, cols, x, x + (rows - 1) * ld + cols, v);
            #pragma unroll
            for (int m = 0; m < 4; ++m) v[m] = clip_piece(v[m], c + 256 * m, cols);
        }
        uint2 code[4];
        float* s = scale + r * nb;
        pack_pieces<4>(v, format, code, [&](int m, float f) {
            const int b = (c - (lane & 15) * 8 + 256 * m) / DLM_PACK_BLOCK;
            if (b < nb) s[b] = f;
        });
        if constexpr (kAligned) {
            #pragma unroll
            for (int m = 0; m < 4; ++m)
                if (c + 256 * m < cols) *reinterpret_cast<uint2*>(q + r * cols + c + 256 * m) = code[m];
        } else {
            store_pieces<4>(q + r * cols + c, c, cols, code);
        }
    }
}

template <bool kAligned>
__global__ void __launch_bounds__(kActThreads) k_unpack8(const uint8_t* __restrict__ q,
                                                         const float* __restrict__ scale, int64_t rows, int cols,
                                                         int format, uint16_t* __restrict__ out, int64_t ld) {
    constexpr int kU = 4;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int nb = (cols + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK, slabs = (cols + kSlab - 1) / kSlab;
    const int64_t items = rows * slabs, step = int64_t(gridDim.x) * (kActThreads / 32);
    for (int64_t i = int64_t(blockIdx.x) * (kActThreads / 32) + threadIdx.x / 32; i < items; i += step) {
        const int64_t r = i / slabs;
        const int c = int(i - r * slabs) * kSlab + lane * 8;
        const uint8_t* src = q + r * cols + c;
        uint2 v[kU];
        float s[kU];
        #pragma unroll
        for (int m = 0; m < kU; ++m) {
            const bool in = c + 256 * m < cols;
            if constexpr (kAligned) v[m] = in ? __ldg(reinterpret_cast<const uint2*>(src + 256 * m)) : make_uint2(0, 0);
            s[m] = in ? __ldg(scale + r * nb + (c + 256 * m) / DLM_PACK_BLOCK) : 0.f;
        }
        if constexpr (!kAligned) load_pieces<kU>(src, c, cols, q, q + rows * cols, v);
        uint4 o[kU];
        #pragma unroll
        for (int m = 0; m < kU; ++m) {
            uint64_t p[4];
            unpack_codes(v[m].x, format, p[0], p[1]);
            unpack_codes(v[m].y, format, p[2], p[3]);
            uint32_t w[4];
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo, hi;
                f2unpack(f2mul(p[k], f2pack(s[m], s[m])), lo, hi);
                w[k] = pack_bf16x2(lo, hi);
            }
            o[m] = make_uint4(w[0], w[1], w[2], w[3]);
            if (kAligned && c + 256 * m < cols) *reinterpret_cast<uint4*>(out + r * ld + c + 256 * m) = o[m];
        }
        if constexpr (!kAligned) store_pieces<kU>(out + r * ld + c, c, cols, o);
    }
}

static bool pack_format_ok(int format) { return format == DLM_PACK_INT8 || format == DLM_PACK_E4M3; }

// CTAs for a warp per slab
static unsigned act_blocks(int64_t rows, int cols) {
    const int64_t b = (rows * ((cols + kSlab - 1) / kSlab) + kActThreads / 32 - 1) / (kActThreads / 32);
    return unsigned(b < (1 << 20) ? b : 1 << 20);
}

}  // namespace dlm

using namespace dlm;

extern "C" dlm_status_t dlm_pack8(const uint16_t* x, int64_t rows, int32_t cols, int64_t ld, int32_t format,
                                  uint8_t* q, float* scale, dlm_stream_t stream) {
    DLM_NVTX("dlm_pack8");
    if (rows < 0 || cols < 0 || cols > INT32_MAX - kSlab || ld < cols || !pack_format_ok(format))
        return DLM_ERR_INVALID_ARGUMENT;
    if (rows == 0 || cols == 0) return DLM_OK;
    if (!x || !q || !scale) return DLM_ERR_INVALID_ARGUMENT;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    const bool vec = cols % 8 == 0 && ld % 8 == 0 && aligned16(x) && (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    return launch_pdl(vec ? k_pack8<true> : k_pack8<false>, dim3(act_blocks(rows, cols)), dim3(kActThreads), 0,
                      (cudaStream_t)stream, "k_pack8 launch", x, rows, cols, ld, format, q, scale);
}

extern "C" dlm_status_t dlm_unpack8(const uint8_t* q, const float* scale, int64_t rows, int32_t cols, int32_t format,
                                    uint16_t* out, int64_t ld, dlm_stream_t stream) {
    DLM_NVTX("dlm_unpack8");
    if (rows < 0 || cols < 0 || cols > INT32_MAX - kSlab || ld < cols || !pack_format_ok(format))
        return DLM_ERR_INVALID_ARGUMENT;
    if (rows == 0 || cols == 0) return DLM_OK;
    if (!q || !scale || !out) return DLM_ERR_INVALID_ARGUMENT;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    const bool vec = cols % 8 == 0 && ld % 8 == 0 && aligned16(out) && (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    return launch_pdl(vec ? k_unpack8<true> : k_unpack8<false>, dim3(act_blocks(rows, cols)), dim3(kActThreads), 0,
                      (cudaStream_t)stream, "k_unpack8 launch", q, scale, rows, cols, format, out, ld);
}
