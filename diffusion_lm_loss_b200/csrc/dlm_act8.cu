// dlm_act8.cu -- activations in 8 bits (dlm_pack8.cuh has the format):
// packing in the forward pass, unpacking in the backward pass.
//
// Both are one pass over memory: 2 bytes read and 1 written per element, or
// the reverse, and 4 bytes per 128 elements for the block's factor.  Rows
// that start on 16-byte borders go 8 elements a lane, 16 lanes a block;
// others one element a lane and load, a warp per block.
#include "dlm_host.h"
#include "dlm_pack8.cuh"

namespace dlm {

constexpr int kActThreads = 256;

__global__ void __launch_bounds__(kActThreads) k_pack8(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                       int64_t ld, int format, uint8_t* __restrict__ q,
                                                       float* __restrict__ scale) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    const int nb = (cols + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK;
    const int64_t blocks = rows * nb;
    const int64_t step = int64_t(gridDim.x) * (kActThreads / 32) * 2;
    for (int64_t b0 = (int64_t(blockIdx.x) * (kActThreads / 32) + threadIdx.x / 32) * 2; b0 < blocks; b0 += step) {
        const int64_t b = b0 + half;
        const int64_t r = b / nb;
        const int col = int(b - r * nb) * DLM_PACK_BLOCK + l * 8;
        const bool in = b < blocks && col < cols;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in) v = __ldg(reinterpret_cast<const uint4*>(x + r * ld + col));
        const PackFactors f = pack_factors(absmax_half_warp(absmax8(v)), format);
        if (in) *reinterpret_cast<uint2*>(q + r * cols + col) = pack8_codes(v, f, format);
        if (b < blocks && l == 0) scale[b] = f.scale;
    }
}

__global__ void __launch_bounds__(kActThreads) k_pack8_any(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                           int64_t ld, int format, uint8_t* __restrict__ q,
                                                           float* __restrict__ scale) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int nb = (cols + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK;
    const int64_t blocks = rows * nb;
    const int64_t step = int64_t(gridDim.x) * (kActThreads / 32);
    for (int64_t b = int64_t(blockIdx.x) * (kActThreads / 32) + threadIdx.x / 32; b < blocks; b += step) {
        const int64_t r = b / nb;
        const int c0 = int(b - r * nb) * DLM_PACK_BLOCK + lane;
        uint16_t v[4];
        uint32_t m = 0;
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = c0 + 32 * k < cols ? __ldg(x + r * ld + c0 + 32 * k) : uint16_t(0);
            m = max(m, uint32_t(v[k] & 0x7fffu));
        }
        m = __reduce_max_sync(~0u, m);
        const PackFactors f = pack_factors(__uint_as_float(m << 16), format);
        #pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c0 + 32 * k < cols)
                q[r * cols + c0 + 32 * k] =
                    uint8_t(pack_code(f.inv != 0.f ? bf16_bits_to_float(v[k]) : 0.f, f.inv, format));
        if (lane == 0) scale[b] = f.scale;
    }
}

__global__ void __launch_bounds__(kActThreads) k_unpack8(const uint8_t* __restrict__ q,
                                                         const float* __restrict__ scale, int64_t rows, int cols,
                                                         int format, uint16_t* __restrict__ out, int64_t ld,
                                                         int vec) {
    pdl_wait();
    pdl_launch_dependents();
    const int nb = (cols + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK;
    const int64_t step = int64_t(gridDim.x) * kActThreads;
    const int per = vec ? cols / 8 : cols;
    const int64_t n = rows * per;
    for (int64_t i = int64_t(blockIdx.x) * kActThreads + threadIdx.x; i < n; i += step) {
        const int64_t r = i / per;
        const int c = int(i - r * per) * (vec ? 8 : 1);
        const float s = __ldg(scale + r * nb + c / DLM_PACK_BLOCK);
        if (vec) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(q + r * cols + c));
            float a[4], b[4];
            unpack_codes(w.x, format, a);
            unpack_codes(w.y, format, b);
            *reinterpret_cast<uint4*>(out + r * ld + c) =
                make_uint4(pack_bf16x2(a[0] * s, a[1] * s), pack_bf16x2(a[2] * s, a[3] * s),
                           pack_bf16x2(b[0] * s, b[1] * s), pack_bf16x2(b[2] * s, b[3] * s));
        } else {
            out[r * ld + c] = __bfloat16_as_ushort(__float2bfloat16_rn(unpack_code(q[r * cols + c], format) * s));
        }
    }
}

static bool pack_format_ok(int format) { return format == DLM_PACK_INT8 || format == DLM_PACK_E4M3; }

static unsigned act_blocks(int64_t items, int per_cta) {
    const int64_t b = (items + per_cta - 1) / per_cta;
    return unsigned(b < 148 * 16 ? b : 148 * 16);
}

}  // namespace dlm

using namespace dlm;

extern "C" dlm_status_t dlm_pack8(const uint16_t* x, int64_t rows, int32_t cols, int64_t ld, int32_t format,
                                  uint8_t* q, float* scale, dlm_stream_t stream) {
    DLM_NVTX("dlm_pack8");
    if (rows < 0 || cols < 0 || cols > INT32_MAX - DLM_PACK_BLOCK || ld < cols || !pack_format_ok(format))
        return DLM_ERR_INVALID_ARGUMENT;
    if (rows == 0 || cols == 0) return DLM_OK;
    if (!x || !q || !scale) return DLM_ERR_INVALID_ARGUMENT;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    const int64_t blocks = rows * ((cols + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK);
    const bool vec = cols % 8 == 0 && ld % 8 == 0 && aligned16(x) && (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    return launch_pdl(vec ? k_pack8 : k_pack8_any,
                      dim3(act_blocks(blocks, (kActThreads / 32) * (vec ? 2 : 1))), dim3(kActThreads), 0,
                      (cudaStream_t)stream, "k_pack8 launch", x, rows, cols, ld, format, q, scale);
}

extern "C" dlm_status_t dlm_unpack8(const uint8_t* q, const float* scale, int64_t rows, int32_t cols, int32_t format,
                                    uint16_t* out, int64_t ld, dlm_stream_t stream) {
    DLM_NVTX("dlm_unpack8");
    if (rows < 0 || cols < 0 || cols > INT32_MAX - DLM_PACK_BLOCK || ld < cols || !pack_format_ok(format))
        return DLM_ERR_INVALID_ARGUMENT;
    if (rows == 0 || cols == 0) return DLM_OK;
    if (!q || !scale || !out) return DLM_ERR_INVALID_ARGUMENT;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    const bool vec = cols % 8 == 0 && ld % 8 == 0 && aligned16(out) && (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    return launch_pdl(k_unpack8, dim3(act_blocks(rows * (vec ? cols / 8 : cols), kActThreads)), dim3(kActThreads), 0,
                      (cudaStream_t)stream, "k_unpack8 launch", q, scale, rows, cols, format, out, ld, int(vec));
}
