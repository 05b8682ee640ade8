// dlm_norm.cu -- layer norm and RMS norm, forward and backward.
//
//   mean = (1/d) sum x              (RMS: 0)
//   rstd = (mean((x - mean)^2) + eps)^(-1/2)
//   xh = (x - mean) rstd,  y = xh (w + offset) + b
//   g = dy (w + offset)
//   dx = rstd (g - mean(g) - xh mean(g xh))     (RMS: without mean(g))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both passes read and write each row once (4 and 6 bytes an element) and
// should be bound by HBM.  What has to be kept small beside that is the
// instructions per element (packed fp32 pairs, parameters in registers) and
// the exchanges per row.  Measured at 16,384 x 4,096 with weight and bias:
// forward 46 us (0.89 of the copy rate; one warp group per row without a ring
// 52, per row of one warp 105), backward 71 us (0.86; one row per CTA of 16
// warps with plain loads 194), forward that also writes the checkpoint 65 us
// (0.79, issue-bound: the codes double the instructions), backward from it 76
// (0.68, bound by its instructions' latency at 16 warps an SM).
//
// Many rows on 16-byte borders (k_norm_fwd_ring, k_norm_bwd_ring): one CTA of
// up to 16 warps per SM, split into groups that each hold a whole row; a group
// walks over its rows while asynchronous copies fill a ring of the next ones
// in shared memory, each thread copying just the pieces that it will read
// itself, so that the loads need no barrier of their own and no wait but the
// copy group's.  A row stays in registers between its sums and its output.  Where
// the width leaves room for one group only, nothing works while it exchanges its
// sums: there the forward pass takes three pieces a lane (two groups again), the
// backward pass two rows at a time (k_norm_bwd_two).
// Backward: the columns' dw and db stay in fp32 registers over all rows of a
// group; a CTA leaves one partial row, and k_norm_join adds the partial rows
// in a fixed order.  x comes as bf16 or from its 8-bit checkpoint.
// Few rows, or a checkpoint to write: one row per group of warps
// (k_norm_fwd_vec).  Rows that are not on 16-byte borders, but in step with one
// another (all tensors contiguous, an odd width): the rings again, by aligned
// chunks (kShift).  Rows out of step: rings read by element (k_norm_*_any).
// Rows too wide for a group: k_norm_*_wide.
#include "dlm_host.h"
#include "dlm_pack8.cuh"

namespace dlm {

struct NormFwdArgs {
    const uint16_t* x;
    int64_t rows, ld_x;
    int d;
    const void* w;
    const void* b;
    int param_f32, rms;
    float eps, offset;
    uint16_t* y;
    int64_t ld_y;
    float* mean;
    float* rstd;
    int format;            // 0: no checkpoint
    uint8_t* q;
    float* q_scale;
};

struct NormBwdArgs {
    const uint16_t* dy;
    int64_t ld_dy;
    const uint16_t* x;     // NULL: from q, q_scale
    int64_t ld_x;
    int format;
    const uint8_t* q;
    const float* q_scale;
    const float* mean;
    const float* rstd;
    const void* w;
    int param_f32, rms;
    float offset;
    int64_t rows;
    int d;
    uint16_t* dx;
    int64_t ld_dx;
    float* part;           // [partial rows][2][pitch]: dw, db
    int pitch;
    void* d_weight;        // NULL: not wanted
    void* d_bias;
    int grad_f32, accumulate;
};

__device__ __forceinline__ float param_at(const void* p, int f32, int c) {
    return f32 ? __ldg(static_cast<const float*>(p) + c) : bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(p) + c));
}

// 8 consecutive parameters from column c on, on a 16-byte border; `none` where
// there is no array
__device__ __forceinline__ void load_params(const void* p, int f32, int c, float none, float (&o)[8]) {
    if (!p) {
        #pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = none;
    } else if (f32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c));
        const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c) + 1);
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w; o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
    } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + c));
        const uint32_t t[4] = {v.x, v.y, v.z, v.w};
        #pragma unroll
        for (int k = 0; k < 4; ++k) { o[2 * k] = bf16lo(t[k]); o[2 * k + 1] = bf16hi(t[k]); }
    }
}

// One element of a parameter's gradient (out NULL: not wanted)
__device__ __forceinline__ void put_grad(void* out, int c, float v, int f32, int accumulate) {
    if (!out) return;
    if (f32) {
        float* o = static_cast<float*>(out) + c;
        *o = accumulate ? *o + v : v;
    } else {
        uint16_t* o = static_cast<uint16_t*>(out) + c;
        *o = __bfloat16_as_ushort(__float2bfloat16_rn(accumulate ? bf16_bits_to_float(*o) + v : v));
    }
}

__device__ __forceinline__ float warp_sum(float v) {
    #pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Sum over the kNW warps of a row's group; `slot`: a place in shared memory of
// kNW floats per group that no earlier exchange still reads.
template <int kNW>
__device__ __forceinline__ float group_sum(float v, float* slot, int warp_in_group) {
    v = warp_sum(v);
    if constexpr (kNW > 1) {
        if ((threadIdx.x & 31) == 0) slot[warp_in_group] = v;
        __syncthreads();
        v = 0.f;
        #pragma unroll
        for (int w = 0; w < kNW; ++w) v += slot[w];
    }
    return v;
}

__device__ __forceinline__ uint64_t f2splat(float v) { return f2pack(v, v); }
__device__ __forceinline__ uint64_t f2bf16(uint32_t w) { return f2pack(bf16lo(w), bf16hi(w)); }

__device__ __forceinline__ uint32_t f2to_bf16(uint64_t v) {
    float lo, hi;
    f2unpack(v, lo, hi);
    return pack_bf16x2(lo, hi);
}

// Groups of kNW warps per CTA: 4 warps with 1 or 2 a group, from 3 on one group.
constexpr int groups_per_cta(int nw) { return nw >= 4 ? 1 : 4 / nw; }

// ---------------------------------------------------------------------------
// forward, one row per group: in the registers of kNW warps, kN pieces of 8
// elements a lane
// ---------------------------------------------------------------------------
template <int kN, int kNW>
__global__ void __launch_bounds__(kNW * groups_per_cta(kNW) * 32) k_norm_fwd_vec(NormFwdArgs a) {
    constexpr int kG = groups_per_cta(kNW);
    __shared__ float s_x[2][kG][kNW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = warp / kNW, wg = warp % kNW;
    const int t = wg * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t want = int64_t(blockIdx.x) * kG + g;
    const bool live = want < a.rows;
    const int64_t row = live ? want : a.rows - 1;       // a group without a row follows the barriers
    const uint16_t* x = a.x + row * a.ld_x;
    uint4 raw[kN];
    #pragma unroll
    for (int j = 0; j < kN; ++j) {
        const int c = (j * kNW * 32 + t) * 8;
        raw[j] = c < a.d ? __ldg(reinterpret_cast<const uint4*>(x + c)) : make_uint4(0, 0, 0, 0);
    }
    if (a.format) {
        uint2 code[kN];
        pack_pieces<kN>(raw, a.format, code, [&](int m, float f) {
            const int c = (m * kNW * 32 + (t & ~15)) * 8, nb = (a.d + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK;
            if (live && c < a.d) a.q_scale[row * nb + c / DLM_PACK_BLOCK] = f;
        });
        #pragma unroll
        for (int j = 0; j < kN; ++j) {
            const int c = (j * kNW * 32 + t) * 8;
            if (live && c < a.d) *reinterpret_cast<uint2*>(a.q + row * a.d + c) = code[j];
        }
    }
    const float inv_d = 1.0f / float(a.d);
    float lo, hi, mean = 0.f;
    if (!a.rms) {
        uint64_t sum = 0;
        #pragma unroll
        for (int j = 0; j < kN; ++j) {
            const uint32_t u[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            #pragma unroll
            for (int k = 0; k < 4; ++k) sum = f2add(sum, f2bf16(u[k]));
        }
        f2unpack(sum, lo, hi);
        mean = group_sum<kNW>(lo + hi, s_x[0][g], wg) * inv_d;
    }
    uint64_t sq = 0;
    #pragma unroll
    for (int j = 0; j < kN; ++j) {
        const uint64_t nm = f2splat((j * kNW * 32 + t) * 8 < a.d ? -mean : 0.f);
        const uint32_t u[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t v = f2add(f2bf16(u[k]), nm);
            sq = f2fma(v, v, sq);
        }
    }
    f2unpack(sq, lo, hi);
    const float rstd = rsqrtf(group_sum<kNW>(lo + hi, s_x[1][g], wg) * inv_d + a.eps);
    if (live && t == 0) {
        if (!a.rms) a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
    uint16_t* y = a.y + row * a.ld_y;
    const float offset = a.w ? a.offset : 0.f;
    const uint64_t nm = f2splat(-mean), r2 = f2splat(rstd);
    #pragma unroll
    for (int j = 0; j < kN; ++j) {
        const int c = (j * kNW * 32 + t) * 8;
        const bool in = live && c < a.d;
        if (in) {
            float w[8], b[8];
            load_params(a.w, a.param_f32, c, 1.f, w);
            load_params(a.b, a.param_f32, c, 0.f, b);
            const uint32_t u[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            uint32_t o[4];
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint64_t xh = f2mul(f2add(f2bf16(u[k]), nm), r2);
                o[k] = f2to_bf16(f2fma(xh, f2pack(w[2 * k] + offset, w[2 * k + 1] + offset), f2pack(b[2 * k], b[2 * k + 1])));
            }
            *reinterpret_cast<uint4*>(y + c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// rings of rows
// ---------------------------------------------------------------------------
constexpr int kRingThreads = 512;

// How a width is split: `nw` warps hold a row at kN pieces of 8 elements a
// lane, `groups` of them make a CTA.
struct RingShape { int nw, groups; };

// The sums of s1 and s2 over a group, in every lane.  Lanes 0..15 carry s1,
// 16..31 s2.  slot: [nw] float2 that no earlier exchange still reads; `bar`:
// the group's barrier.  kAdd: every lane adds up to 8 warps' sums itself in
// place of four more shuffles (forward, 16,384 x 4,096: 47.4 -> 46.1 us; the
// backward pass, short of registers, gets slower: 70.5 -> 72.0).
template <bool kAdd>
__device__ __forceinline__ void group_sum2(float& s1, float& s2, float2* slot, int wg, const RingShape sh, int bar) {
    const int lane = threadIdx.x & 31;
    float v = lane < 16 ? s1 : s2;
    v += __shfl_xor_sync(~0u, lane < 16 ? s2 : s1, 16);
    #pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if (sh.nw > 1) {
        if ((lane & 15) == 0) reinterpret_cast<float*>(slot + wg)[lane >> 4] = v;
        named_barrier_sync(bar, sh.nw * 32);
        if (kAdd && sh.nw <= 8) {
            uint64_t p[8];
            #pragma unroll
            for (int w = 0; w < 8; ++w) p[w] = w < sh.nw ? *reinterpret_cast<const uint64_t*>(slot + w) : 0;
            #pragma unroll
            for (int o = 4; o; o >>= 1)
                #pragma unroll
                for (int w = 0; w < o; ++w) p[w] = f2add(p[w], p[w + o]);
            f2unpack(p[0], s1, s2);
            return;
        }
        v = (lane & 15) < sh.nw ? reinterpret_cast<const float*>(slot + (lane & 15))[lane >> 4] : 0.f;
        #pragma unroll
        for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    }
    const float other = __shfl_xor_sync(~0u, v, 16);
    s1 = lane < 16 ? v : other;
    s2 = lane < 16 ? other : v;
}

// The same for two rows in one exchange: lanes 8 q .. 8 q + 7 carry sum q of
// s1[0], s1[1], s2[0], s2[1].  slot: [nw] float4.
__device__ __forceinline__ void group_sum4(float (&s1)[2], float (&s2)[2], float4* slot, int wg, const RingShape sh,
                                           int bar) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, odd = lane & 8;
    const float a0 = (up ? s2[0] : s1[0]) + __shfl_xor_sync(~0u, up ? s1[0] : s2[0], 16);
    const float a1 = (up ? s2[1] : s1[1]) + __shfl_xor_sync(~0u, up ? s1[1] : s2[1], 16);
    float v = (odd ? a1 : a0) + __shfl_xor_sync(~0u, odd ? a0 : a1, 8);
    #pragma unroll
    for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((lane & 7) == 0) reinterpret_cast<float*>(slot + wg)[lane >> 3] = v;
    named_barrier_sync(bar, sh.nw * 32);
    const float* from = reinterpret_cast<const float*>(slot + (lane & 7)) + (lane >> 3);
    v = ((lane & 7) < sh.nw ? from[0] : 0.f) + ((lane & 7) + 8 < sh.nw ? from[32] : 0.f);
    #pragma unroll
    for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    s1[0] = __shfl_sync(~0u, v, 0);
    s1[1] = __shfl_sync(~0u, v, 8);
    s2[0] = __shfl_sync(~0u, v, 16);
    s2[1] = __shfl_sync(~0u, v, 24);
}

__device__ __forceinline__ float group_sum1(float v, float* slot, int wg, const RingShape sh, int bar) {
    const int lane = threadIdx.x & 31;
    v = warp_sum(v);
    if (sh.nw > 1) {
        if (lane == 0) slot[wg] = v;
        named_barrier_sync(bar, sh.nw * 32);
        v = (lane & 15) < sh.nw ? slot[lane & 15] : 0.f;
        #pragma unroll
        for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    }
    return v;
}

// 8 parameters as 4 pairs
__device__ __forceinline__ void param_pairs(const void* p, int f32, int c, float none, float add, uint64_t (&o)[4]) {
    float v[8];
    if (!p || (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        load_params(p, f32, c, none, v);
    } else {
        #pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = param_at(p, f32, c + k);
    }
    #pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = f2pack(v[2 * k] + add, v[2 * k + 1] + add);
}

// Stages of the rings, with kN pieces a lane: 80 to 196 KB (forward), 164 or 197
// KB (backward) of shared memory, all but one stage of it in flight.
template <int kN>
constexpr int fwd_stages() { return kN == 3 ? 4 : 5; }
template <int kN>
constexpr int bwd_stages() { return kN == 1 ? 10 : 6; }

// A thread's slots of the ring, [stages][pieces] of 16 bytes, the threads side
// by side.  Pieces that lie outside the row are never copied and stay zero.
template <int kS, int kPieces>
struct Ring {
    uint32_t base, pitch, put, get;
    __device__ __forceinline__ explicit Ring(uint4* smem) {
        base = smem_addr(smem + threadIdx.x);
        pitch = blockDim.x * 16u;
        put = get = base;
    }
    // zeros for good in one piece's slots
    __device__ __forceinline__ void clear(uint4* smem, int piece) const {
        for (int k = piece; k < kS * kPieces; k += kPieces) smem[threadIdx.x + k * blockDim.x] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void step(uint32_t& at) const {
        at += kPieces * pitch;
        if (at == base + uint32_t(kS * kPieces) * pitch) at = base;
    }
};

__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}

// Where a thread's pieces lie.  With kShift the rows are not on 16-byte borders:
// a piece is an aligned 16-byte chunk of memory all the same, and holds the
// columns 8 p - phase .. 8 p - phase + 7, phase = (row x stride) mod 8.  All rows
// of a group have one phase (their distance is a multiple of 8), so a thread
// keeps its columns, whose parameters and sums stay in its registers.  The
// first piece may begin with the end of the row before (masked after the load),
// the last one may end behind the row (not read); both are stored by element.
template <int kN, bool kShift>
struct Pieces {
    int c[kN];             // first column
    bool in[kN], edge[kN];
    __device__ __forceinline__ Pieces(int t, int gt, int d, int phase) {
        #pragma unroll
        for (int j = 0; j < kN; ++j) {
            c[j] = (j * gt + t) * 8 - (kShift ? phase : 0);
            in[j] = c[j] < d;
            edge[j] = kShift && in[j] && (c[j] < 0 || c[j] + 8 > d);
        }
    }
    // bytes of the piece that are read: all but those behind the row
    template <typename E>
    __device__ __forceinline__ int bytes(int j, int d) const {
        return int(sizeof(E)) * min(8, d - c[j]);
    }
    // zero outside the row
    __device__ __forceinline__ void clip(int j, int d, uint64_t (&f)[4]) const {
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo, hi;
            f2unpack(f[k], lo, hi);
            const int e = c[j] + 2 * k;
            f[k] = f2pack(e >= 0 && e < d ? lo : 0.f, e + 1 >= 0 && e + 1 < d ? hi : 0.f);
        }
    }
    __device__ __forceinline__ void params(int j, int d, const void* p, int f32, float none, float add,
                                           uint64_t (&o)[4]) const {
        if (!kShift) {
            param_pairs(p, f32, in[j] ? c[j] : 0, none, add, o);
        } else {
            float v[8];
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int e = c[j] + k;
                v[k] = p && e >= 0 && e < d ? param_at(p, f32, e) + add : none;
            }
            #pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = f2pack(v[2 * k], v[2 * k + 1]);
        }
    }
    // stores the piece at `at`, its aligned place in the row
    __device__ __forceinline__ void store(int j, int d, uint16_t* at, const uint64_t (&v)[4]) const {
        uint32_t o[4];
        #pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = f2to_bf16(v[k]);
        if (kShift && edge[j]) {
            #pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c[j] + k >= 0 && c[j] + k < d) at[k] = uint16_t(o[k / 2] >> (16 * (k & 1)));
        } else if (in[j]) {
            *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
};

// kMean: what is subtracted is known to be the mean (kSubtract) or nothing
// (kNothing), or is asked for (kAsk, nothing being subtracted as zero).  On
// 16-byte borders RMS norm runs faster as kAsk, however odd (13,107 x 5,120: 44 us
// against 46, 8,192 x 8,192: 43, 47); off them the work that kNothing saves
// counts (13,419 x 5,001: 72, 64).  Layer norm as kAsk: 46.7 against 46.1.
enum Mean { kSubtract, kNothing, kAsk };
template <int kN, bool kShift, Mean kMean>
__global__ void __launch_bounds__(kRingThreads, 1) k_norm_fwd_ring(NormFwdArgs a, RingShape sh) {
    constexpr int kS = fwd_stages<kN>(), kR = 2;                // two rows at a time: their exchanges share barriers
    extern __shared__ uint4 ring_mem[];
    __shared__ float2 s_x[2][2][kRingThreads / 32];       // [turn parity][sum][warp]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = warp / sh.nw, wg = warp - g * sh.nw;
    const int t = wg * 32 + lane, gt = sh.nw * 32;
    const int64_t first = int64_t(g) * gridDim.x + blockIdx.x, step = int64_t(sh.groups) * gridDim.x;
    const int phase = kShift ? int((first * a.ld_x) & 7) : 0;
    const Pieces<kN, kShift> pc(t, gt, a.d, phase);
    Ring<kS, kR * kN> ring(ring_mem);
    #pragma unroll
    for (int j = 0; j < kR * kN; ++j)
        if (!pc.in[j % kN]) ring.clear(ring_mem, j);
    pdl_wait();
    pdl_launch_dependents();
    int n = first < a.rows ? int((a.rows - first + step - 1) / step) : 0;
    const int64_t dx = step * a.ld_x, dy = step * a.ld_y;
    const uint16_t* px = a.x + first * a.ld_x + t * 8 - phase;
    int left = n;
    auto issue = [&]() {
        #pragma unroll
        for (int r = 0; r < kR; ++r) {
            if (left > 0) {
                #pragma unroll
                for (int j = 0; j < kN; ++j) {
                    const uint32_t dst = ring.put + (r * kN + j) * ring.pitch;
                    if (!pc.in[j]) continue;
                    if constexpr (kShift) cp_async16_part(dst, px + j * gt * 8, pc.template bytes<uint16_t>(j, a.d));
                    else cp_async16(dst, px + j * gt * 8);
                }
                px += dx;
                --left;
            }
        }
        cp_async_commit();
        ring.step(ring.put);
    };
    #pragma unroll 1
    for (int s = 0; s < kS - 1; ++s) issue();
    uint64_t w[kN][4], b[kN][4];
    #pragma unroll
    for (int j = 0; j < kN; ++j) {
        pc.params(j, a.d, a.w, a.param_f32, 1.f, a.w ? a.offset : 0.f, w[j]);
        pc.params(j, a.d, a.b, a.param_f32, 0.f, 0.f, b[j]);
    }
    const float inv_d = 1.0f / float(a.d);
    uint16_t* py = a.y + first * a.ld_y + t * 8 - phase;
    int par = 0;
    int64_t row = first;
    for (; n > 0; n -= kR, par ^= 1, row += kR * step, py += kR * dy) {
        cp_async_wait<kS - 2>();
        uint64_t f[kR][kN][4];
        float s1[kR], s2[kR], lo, hi;
        #pragma unroll
        for (int r = 0; r < kR; ++r) {
            uint64_t sum = 0;
            #pragma unroll
            for (int j = 0; j < kN; ++j) {
                const uint4 raw = lds16(ring.get + (r * kN + j) * ring.pitch);
                const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
                #pragma unroll
                for (int k = 0; k < 4; ++k) f[r][j][k] = f2bf16(u[k]);
                if (kShift && pc.edge[j]) pc.clip(j, a.d, f[r][j]);
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (kMean != kNothing) sum = f2add(sum, f[r][j][k]);
            }
            f2unpack(sum, lo, hi);
            s1[r] = lo + hi;
        }
        ring.step(ring.get);
        issue();
        if (kMean == kNothing || (kMean == kAsk && a.rms)) s1[0] = s1[1] = 0.f;
        else group_sum2<!kShift>(s1[0], s1[1], &s_x[par][0][g * sh.nw], wg, sh, 1 + g);
        #pragma unroll
        for (int r = 0; r < kR; ++r) {
            s1[r] *= inv_d;                               // the mean
            uint64_t sq = 0;
            #pragma unroll
            for (int j = 0; j < kN; ++j) {
                const uint64_t nm = f2splat(pc.in[j] ? -s1[r] : 0.f);
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (kMean != kNothing) f[r][j][k] = f2add(f[r][j][k], nm);
                if (kMean != kNothing && kShift && pc.edge[j]) pc.clip(j, a.d, f[r][j]);
                #pragma unroll
                for (int k = 0; k < 4; ++k) sq = f2fma(f[r][j][k], f[r][j][k], sq);
            }
            f2unpack(sq, lo, hi);
            s2[r] = lo + hi;
        }
        group_sum2<!kShift>(s2[0], s2[1], &s_x[par][1][g * sh.nw], wg, sh, 1 + g);
        #pragma unroll
        for (int r = 0; r < kR; ++r) {
            if (n <= r) break;
            const float rstd = rsqrtf(s2[r] * inv_d + a.eps);
            if (t == 0) {
                if (kMean == kSubtract || (kMean == kAsk && !a.rms)) a.mean[row + r * step] = s1[r];
                a.rstd[row + r * step] = rstd;
            }
            const uint64_t r2 = f2splat(rstd);
            #pragma unroll
            for (int j = 0; j < kN; ++j) {
                uint64_t o[4];
                #pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = f2fma(f2mul(f[r][j][k], r2), w[j][k], b[j][k]);
                pc.store(j, a.d, py + r * dy + j * gt * 8, o);
            }
        }
    }
    cp_async_wait<0>();
}

// kFormat: DLM_PACK_NONE (x itself) or the format of its checkpoint.  kLean: RMS
// norm whose bias gradient is not wanted: three packed operations a pair less
// (16,384 x 4,096: 69.3 -> 68.3 us, from 8 bits 75.5 -> 65.9; 13,419 x 5,001: 114 -> 88).
template <int kN, int kFormat, bool kShift, bool kLean>
__global__ void __launch_bounds__(kRingThreads, 1) k_norm_bwd_ring(NormBwdArgs a, RingShape sh) {
    constexpr int kS = bwd_stages<kN>();
    constexpr bool kHeld8 = kFormat != DLM_PACK_NONE;
    // when a row's place in the ring is filled again: with little to compute, after the exchange (kLean, 13,107 x
    // 5,120: 85.4 us before it, 80.6 after; from 8 bits 80.7, 82.4; not kLean, 26,214 x 2,560: 70.0, 71.6)
    constexpr bool kLate = kLean && !kShift && !kHeld8;
    extern __shared__ uint4 ring_mem[];                   // ring of dy, x pieces; at the end the groups' sums
    __shared__ float2 s_x[2][16];                         // [row parity][warp]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = warp / sh.nw, wg = warp - g * sh.nw;
    const int t = wg * 32 + lane, gt = sh.nw * 32;
    uint64_t w[kN][4], dw[kN][4], db[kLean ? 1 : kN][4];
    const int64_t first = int64_t(g) * gridDim.x + blockIdx.x, step = int64_t(sh.groups) * gridDim.x;
    const int phase = kShift ? int((first * a.ld_dy) & 7) : 0;
    const Pieces<kN, kShift> pc(t, gt, a.d, phase);
    Ring<kS, 2 * kN> ring(ring_mem);
    #pragma unroll
    for (int j = 0; j < 2 * kN; ++j)
        if (!pc.in[j / 2]) ring.clear(ring_mem, j);
    pdl_wait();
    pdl_launch_dependents();
    int n = first < a.rows ? int((a.rows - first + step - 1) / step) : 0;
    const int nb = (a.d + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK;
    const uint16_t* pdy = a.dy + first * a.ld_dy + t * 8 - phase;
    const uint16_t* px = kHeld8 ? nullptr : a.x + first * a.ld_x + t * 8 - phase;
    const uint8_t* pq = kHeld8 ? a.q + first * a.d + t * 8 - phase : nullptr;
    int left = n;
    auto issue = [&]() {
        if (left > 0) {
            #pragma unroll
            for (int j = 0; j < kN; ++j) {
                if (!pc.in[j]) continue;
                const uint32_t dst = ring.put + 2 * j * ring.pitch;
                if constexpr (kShift) {
                    const int nb16 = pc.template bytes<uint16_t>(j, a.d);
                    cp_async16_part(dst, pdy + j * gt * 8, nb16);
                    if constexpr (kHeld8) cp_async8_part(dst + ring.pitch, pq + j * gt * 8, nb16 / 2);
                    else cp_async16_part(dst + ring.pitch, px + j * gt * 8, nb16);
                } else {
                    cp_async16(dst, pdy + j * gt * 8);
                    if constexpr (kHeld8) cp_async8(dst + ring.pitch, pq + j * gt * 8);
                    else cp_async16(dst + ring.pitch, px + j * gt * 8);
                }
            }
            pdy += step * a.ld_dy;
            if constexpr (kHeld8) pq += step * a.d;
            else px += step * a.ld_x;
            --left;
        }
        cp_async_commit();
        ring.step(ring.put);
    };
    // statistics and block factors of the row after the one in work
    const float* pmean = a.mean + first;
    const float* prstd = a.rstd + first;
    const float* pqs = kHeld8 ? a.q_scale + first * nb : nullptr;
    float mean_n = 0.f, rstd_n = 0.f, qs_n[kN], qs2_n[kN];   // qs2: of the second block in a piece that holds two
    int two[kN];                                             // elements of the first one there, 8 if there is one only
    #pragma unroll
    for (int j = 0; j < kN; ++j)
        two[j] = kShift && pc.in[j] && (pc.c[j] & 127) > 120 && (pc.c[j] | 127) + 1 < a.d ? 128 - (pc.c[j] & 127) : 8;
    auto next_stats = [&](bool more) {
        if (!more) return;
        if (!kLean && !a.rms) mean_n = __ldg(pmean);
        rstd_n = __ldg(prstd);
        pmean += step;
        prstd += step;
        if constexpr (kHeld8) {
            #pragma unroll
            for (int j = 0; j < kN; ++j) {
                const int b0 = max(pc.c[j], 0) / DLM_PACK_BLOCK;
                qs_n[j] = pc.in[j] ? __ldg(pqs + b0) : 0.f;
                if (kShift) qs2_n[j] = two[j] < 8 ? __ldg(pqs + (pc.c[j] + 8) / DLM_PACK_BLOCK) : 0.f;
            }
            pqs += step * nb;
        }
    };
    #pragma unroll 1
    for (int s = 0; s < kS - 1; ++s) issue();
    next_stats(n > 0);
    #pragma unroll
    for (int j = 0; j < kN; ++j) {
        pc.params(j, a.d, a.w, a.param_f32, 1.f, a.w ? a.offset : 0.f, w[j]);
        #pragma unroll
        for (int k = 0; k < 4; ++k) dw[j][k] = db[kLean ? 0 : j][k] = 0;
    }
    const float inv_d = 1.0f / float(a.d);
    uint16_t* pdx = a.dx + first * a.ld_dx + t * 8 - phase;
    int par = 0;
    for (; n > 0; --n, par ^= 1, pdx += step * a.ld_dx) {
        const float rstd = rstd_n;
        const uint64_t nm = f2splat(-mean_n), r2 = f2splat(rstd);
        float qs[kN], qs2[kN];
        if constexpr (kHeld8) {
            #pragma unroll
            for (int j = 0; j < kN; ++j) { qs[j] = qs_n[j]; qs2[j] = kShift ? qs2_n[j] : 0.f; }
        }
        next_stats(n > 1);
        cp_async_wait<kS - 2>();
        uint64_t xh[kN][4], gr[kN][4], s1 = 0, s2 = 0;
        #pragma unroll
        for (int j = 0; j < kN; ++j) {
            const uint4 y4 = lds16(ring.get + 2 * j * ring.pitch);
            const uint32_t yw[4] = {y4.x, y4.y, y4.z, y4.w};
            if constexpr (kHeld8) {
                const uint2 q2 = lds8(ring.get + (2 * j + 1) * ring.pitch);
                unpack_codes(q2.x, kFormat, xh[j][0], xh[j][1]);
                unpack_codes(q2.y, kFormat, xh[j][2], xh[j][3]);
                // code * scale - mean in one FMA: the held value is not rounded (kLean: the code times
                // scale * rstd)
                const float f1 = kLean ? qs[j] * rstd : qs[j], f2 = kLean ? qs2[j] * rstd : qs2[j];
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint64_t s = f2splat(f1);
                    if (kShift && two[j] < 8) s = f2pack(2 * k < two[j] ? f1 : f2, 2 * k + 1 < two[j] ? f1 : f2);
                    xh[j][k] = kLean ? f2mul(xh[j][k], s) : f2fma(xh[j][k], s, nm);
                }
            } else {
                const uint4 x4 = lds16(ring.get + (2 * j + 1) * ring.pitch);
                const uint32_t xw[4] = {x4.x, x4.y, x4.z, x4.w};
                #pragma unroll
                for (int k = 0; k < 4; ++k) xh[j][k] = kLean ? f2mul(f2bf16(xw[k]), r2) : f2add(f2bf16(xw[k]), nm);
            }
            uint64_t dy4[4];
            #pragma unroll
            for (int k = 0; k < 4; ++k) dy4[k] = f2bf16(yw[k]);
            if (kShift && pc.edge[j]) {                   // the end of the row before
                pc.clip(j, a.d, xh[j]);
                pc.clip(j, a.d, dy4);
            }
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint64_t dy = dy4[k];
                if (!kLean) xh[j][k] = f2mul(xh[j][k], r2);
                gr[j][k] = f2mul(dy, w[j][k]);
                s2 = f2fma(gr[j][k], xh[j][k], s2);
                dw[j][k] = f2fma(dy, xh[j][k], dw[j][k]);
                if constexpr (!kLean) {
                    s1 = f2add(s1, gr[j][k]);
                    db[j][k] = f2add(db[j][k], dy);
                }
            }
        }
        ring.step(ring.get);
        if (!kLate) issue();
        float lo, hi, v1, v2;
        f2unpack(s1, lo, hi);
        v1 = lo + hi;
        f2unpack(s2, lo, hi);
        v2 = lo + hi;
        if constexpr (kLean) v2 = group_sum1(v2, reinterpret_cast<float*>(&s_x[par][g * sh.nw]), wg, sh, 1 + g);
        else group_sum2<false>(v1, v2, &s_x[par][g * sh.nw], wg, sh, 1 + g);
        if (kLate) issue();
        const float by = -rstd * inv_d;
        const uint64_t n1 = f2splat(a.rms ? 0.f : v1 * by), n2 = f2splat(v2 * by);
        #pragma unroll
        for (int j = 0; j < kN; ++j) {
            uint64_t o[4];
            #pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] = f2fma(gr[j][k], r2, kLean ? f2mul(xh[j][k], n2) : f2fma(xh[j][k], n2, n1));
            pc.store(j, a.d, pdx + j * gt * 8, o);
        }
    }
    // the groups' sums, side by side in shared memory, then added column by
    // column in the order of the groups
    cp_async_wait<0>();
    __syncthreads();
    float* acc = reinterpret_cast<float*>(ring_mem);      // [group][dw, db][kN gt 8]
    const int wide = kN * gt * 8;
    #pragma unroll
    for (int j = 0; j < kN; ++j) {
        #pragma unroll
        for (int h = 0; h < (kLean ? 1 : 2); ++h) {
            uint64_t* p = reinterpret_cast<uint64_t*>(acc + (2 * g + h) * wide + (j * gt + t) * 8);
            #pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = h ? db[kLean ? 0 : j][i] : dw[j][i];
        }
    }
    __syncthreads();
    float* part = a.part + int64_t(blockIdx.x) * 2 * a.pitch;
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        float sw = 0.f, sb = 0.f;
        for (int k = 0; k < sh.groups; ++k) {
            const int at = 2 * k * wide + c + (kShift ? int(((int64_t(k) * gridDim.x + blockIdx.x) * a.ld_dy) & 7) : 0);
            sw += acc[at];
            if (!kLean) sb += acc[at + wide];
        }
        if (gridDim.x == 1) {                             // the whole sum: no k_norm_join
            put_grad(a.d_weight, c, sw, a.grad_f32, a.accumulate);
            put_grad(a.d_bias, c, sb, a.grad_f32, a.accumulate);
        } else {
            if (a.d_weight) part[c] = sw;
            if (a.d_bias) part[a.pitch + c] = sb;
        }
    }
}

// The same for rows on 16-byte borders that leave room for one group of 9 to 12
// warps on an SM: no other group works while it exchanges its sums, so it takes
// two rows at a time, which its warps have the registers for (168 a lane).
// 13,107 x 5,120: 86 -> 73 us, RMS 81 -> 66, RMS from 8 bits 81 -> 67.  (Layer
// norm from 8 bits got slower, 98 -> 114, and stays with one row.  Two groups with
// two rows each, the weight in shared memory and dy read again for want of
// registers: 16,384 x 4,096 95 us instead of 71.)
constexpr int kTwoThreads = 384, kTwoStages = 8;

template <int kFormat, bool kLean>
__global__ void __launch_bounds__(kTwoThreads, 1) k_norm_bwd_two(NormBwdArgs a, RingShape sh) {
    constexpr int kN = 2, kS = kTwoStages, kR = 2;
    constexpr bool kHeld8 = kFormat != DLM_PACK_NONE;
    extern __shared__ uint4 ring_mem[];
    __shared__ float4 s_x[2][kTwoThreads / 32];
    const int t = threadIdx.x, wg = t >> 5, gt = sh.nw * 32;
    const int64_t first = blockIdx.x, step = gridDim.x;
    const Pieces<kN, false> pc(t, gt, a.d, 0);
    Ring<kS, 2 * kN> ring(ring_mem);
    #pragma unroll
    for (int j = 0; j < 2 * kN; ++j)
        if (!pc.in[j / 2]) ring.clear(ring_mem, j);
    pdl_wait();
    pdl_launch_dependents();
    int n = first < a.rows ? int((a.rows - first + step - 1) / step) : 0;
    const int nb = (a.d + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK;
    const uint16_t* pdy = a.dy + first * a.ld_dy + t * 8;
    const uint16_t* px = kHeld8 ? nullptr : a.x + first * a.ld_x + t * 8;
    const uint8_t* pq = kHeld8 ? a.q + first * a.d + t * 8 : nullptr;
    int left = n;
    auto issue = [&]() {
        if (left > 0) {
            #pragma unroll
            for (int j = 0; j < kN; ++j) {
                if (!pc.in[j]) continue;
                const uint32_t dst = ring.put + 2 * j * ring.pitch;
                cp_async16(dst, pdy + j * gt * 8);
                if constexpr (kHeld8) cp_async8(dst + ring.pitch, pq + j * gt * 8);
                else cp_async16(dst + ring.pitch, px + j * gt * 8);
            }
            pdy += step * a.ld_dy;
            if constexpr (kHeld8) pq += step * a.d;
            else px += step * a.ld_x;
            --left;
        }
        cp_async_commit();
        ring.step(ring.put);
    };
    // statistics and block factors of the rows after those in work
    const float* pmean = a.mean + first;
    const float* prstd = a.rstd + first;
    const float* pqs = kHeld8 ? a.q_scale + first * nb : nullptr;
    float mean_n[kR] = {}, rstd_n[kR], qs_n[kR][kN];
    auto next_stats = [&](int rows) {
        #pragma unroll
        for (int r = 0; r < kR; ++r) {
            if (r >= rows) break;
            if (!kLean && !a.rms) mean_n[r] = __ldg(pmean);
            rstd_n[r] = __ldg(prstd);
            pmean += step;
            prstd += step;
            if constexpr (kHeld8) {
                #pragma unroll
                for (int j = 0; j < kN; ++j) qs_n[r][j] = pc.in[j] ? __ldg(pqs + pc.c[j] / DLM_PACK_BLOCK) : 0.f;
                pqs += step * nb;
            }
        }
    };
    #pragma unroll 1
    for (int s = 0; s < kS - 1; ++s) issue();
    next_stats(n);
    uint64_t w[kN][4], dw[kN][4], db[kLean ? 1 : kN][4];
    #pragma unroll
    for (int j = 0; j < kN; ++j) {
        pc.params(j, a.d, a.w, a.param_f32, 1.f, a.w ? a.offset : 0.f, w[j]);
        #pragma unroll
        for (int k = 0; k < 4; ++k) dw[j][k] = db[kLean ? 0 : j][k] = 0;
    }
    const float inv_d = 1.0f / float(a.d);
    uint16_t* pdx = a.dx + first * a.ld_dx + t * 8;
    int par = 0;
    for (; n > 0; n -= kR, par ^= 1) {
        float rstd[kR], mean[kR], qs[kR][kN];
        #pragma unroll
        for (int r = 0; r < kR; ++r) {
            rstd[r] = rstd_n[r];
            mean[r] = mean_n[r];
            #pragma unroll
            for (int j = 0; j < kN; ++j) qs[r][j] = kHeld8 ? qs_n[r][j] : 0.f;
        }
        next_stats(n - kR);
        cp_async_wait<kS - 1 - kR>();
        uint64_t xh[kR][kN][4], gr[kR][kN][4];
        float v1[kR], v2[kR];
        #pragma unroll
        for (int r = 0; r < kR; ++r) {
            v1[r] = v2[r] = 0.f;
            if (r >= n) break;
            const uint64_t nm = f2splat(-mean[r]), r2 = f2splat(rstd[r]);
            uint64_t s1 = 0, s2 = 0;
            #pragma unroll
            for (int j = 0; j < kN; ++j) {
                const uint4 y4 = lds16(ring.get + 2 * j * ring.pitch);
                const uint32_t yw[4] = {y4.x, y4.y, y4.z, y4.w};
                if constexpr (kHeld8) {
                    const uint2 q2 = lds8(ring.get + (2 * j + 1) * ring.pitch);
                    unpack_codes(q2.x, kFormat, xh[r][j][0], xh[r][j][1]);
                    unpack_codes(q2.y, kFormat, xh[r][j][2], xh[r][j][3]);
                    const uint64_t s = f2splat(kLean ? qs[r][j] * rstd[r] : qs[r][j]);
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) xh[r][j][k] = kLean ? f2mul(xh[r][j][k], s) : f2fma(xh[r][j][k], s, nm);
                } else {
                    const uint4 x4 = lds16(ring.get + (2 * j + 1) * ring.pitch);
                    const uint32_t xw[4] = {x4.x, x4.y, x4.z, x4.w};
                    #pragma unroll
                    for (int k = 0; k < 4; ++k)
                        xh[r][j][k] = kLean ? f2mul(f2bf16(xw[k]), r2) : f2add(f2bf16(xw[k]), nm);
                }
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t dy = f2bf16(yw[k]);
                    if (!kLean) xh[r][j][k] = f2mul(xh[r][j][k], r2);
                    gr[r][j][k] = f2mul(dy, w[j][k]);
                    s2 = f2fma(gr[r][j][k], xh[r][j][k], s2);
                    dw[j][k] = f2fma(dy, xh[r][j][k], dw[j][k]);
                    if constexpr (!kLean) {
                        s1 = f2add(s1, gr[r][j][k]);
                        db[j][k] = f2add(db[j][k], dy);
                    }
                }
            }
            ring.step(ring.get);
            float lo, hi;
            f2unpack(s1, lo, hi);
            v1[r] = lo + hi;
            f2unpack(s2, lo, hi);
            v2[r] = lo + hi;
        }
        issue();
        group_sum4(v1, v2, s_x[par], wg, sh, 1);
        issue();                                              // (into a slot whose pieces the sums have used)
        #pragma unroll
        for (int r = 0; r < kR; ++r) {
            if (r >= n) break;
            const float by = -rstd[r] * inv_d;
            const uint64_t r2 = f2splat(rstd[r]), n1 = f2splat(a.rms ? 0.f : v1[r] * by), n2 = f2splat(v2[r] * by);
            #pragma unroll
            for (int j = 0; j < kN; ++j) {
                uint64_t o[4];
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = f2fma(gr[r][j][k], r2, kLean ? f2mul(xh[r][j][k], n2) : f2fma(xh[r][j][k], n2, n1));
                pc.store(j, a.d, pdx + j * gt * 8, o);
            }
            pdx += step * a.ld_dx;
        }
    }
    cp_async_wait<0>();
    // one group: a thread's columns are its own
    float* part = a.part + int64_t(blockIdx.x) * 2 * a.pitch;
    #pragma unroll
    for (int j = 0; j < kN; ++j) {
        if (!pc.in[j]) continue;
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = pc.c[j] + 2 * k;
            float w0, w1, b0, b1;
            f2unpack(dw[j][k], w0, w1);
            f2unpack(db[kLean ? 0 : j][k], b0, b1);
            if (gridDim.x == 1) {                             // the whole sum: no k_norm_join
                put_grad(a.d_weight, c, w0, a.grad_f32, a.accumulate);
                put_grad(a.d_weight, c + 1, w1, a.grad_f32, a.accumulate);
                put_grad(a.d_bias, c, b0, a.grad_f32, a.accumulate);
                put_grad(a.d_bias, c + 1, b1, a.grad_f32, a.accumulate);
            } else {
                if (a.d_weight) *reinterpret_cast<float2*>(part + c) = make_float2(w0, w1);
                if (a.d_bias) *reinterpret_cast<float2*>(part + a.pitch + c) = make_float2(b0, b1);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// rows that are not on 16-byte borders
// ---------------------------------------------------------------------------
// A row is copied to shared memory by the aligned 16-byte chunks that cover it
// (what a chunk holds besides the row is the tensor's own memory; the chunks
// that would leave the tensor, at its first row's start and its last row's
// end, are copied by element), and every thread then reads the elements
// k * gt + t of it.  Two-byte loads from global memory would keep too few bytes
// in flight: 13 % of the bandwidth at 8,192 rows of 5,001.
constexpr int kAnyE = 16;             // elements a lane
constexpr int kAnyStages = 6;

// Starts the copy of `bytes` bytes at src to dst (16-byte aligned; the row
// begins at dst + (src mod 16)); [begin, end): the tensor.
template <typename E>
__device__ __forceinline__ void stage_row(uint8_t* dst, const E* src, int n, const E* begin, const E* end, int t,
                                          int gt) {
    const uintptr_t s = reinterpret_cast<uintptr_t>(src), lo = s & ~uintptr_t(15);
    const int chunks = int((s + size_t(n) * sizeof(E) - lo + 15) / 16);
    for (int k = t; k < chunks; k += gt) {
        const uintptr_t at = lo + 16u * unsigned(k);
        if (at >= reinterpret_cast<uintptr_t>(begin) && at + 16 <= reinterpret_cast<uintptr_t>(end)) {
            cp_async16(smem_addr(dst + 16 * k), reinterpret_cast<const void*>(at));
        } else {
            #pragma unroll 1
            for (int e = 0; e < int(16 / sizeof(E)); ++e) {
                const E* p = reinterpret_cast<const E*>(at) + e;
                if (p >= src && p < src + n) reinterpret_cast<E*>(dst + 16 * k)[e] = *p;
            }
        }
    }
}

template <typename E>
__device__ __forceinline__ const E* staged(const uint8_t* dst, const E* src) {
    return reinterpret_cast<const E*>(dst + (reinterpret_cast<uintptr_t>(src) & 15));
}

__device__ __forceinline__ void group_barrier(const RingShape sh, int bar) {
    if (sh.nw > 1) named_barrier_sync(bar, sh.nw * 32);
    else __syncwarp();
}

__global__ void __launch_bounds__(kRingThreads, 1) k_norm_fwd_any(NormFwdArgs a, RingShape sh, int slot) {
    extern __shared__ uint4 ring_mem[];                   // [group][kAnyStages][slot bytes]
    __shared__ float s_x[2][2][kRingThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = warp / sh.nw, wg = warp - g * sh.nw;
    const int t = wg * 32 + lane, gt = sh.nw * 32;
    uint8_t* ring = reinterpret_cast<uint8_t*>(ring_mem) + size_t(g) * kAnyStages * slot;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t first = int64_t(g) * gridDim.x + blockIdx.x, step = int64_t(sh.groups) * gridDim.x;
    const uint16_t* end = a.x + (a.rows - 1) * a.ld_x + a.d;
    int put = 0, get = 0, par = 0;
    auto issue = [&](int64_t row) {
        if (row < a.rows) stage_row(ring + put * slot, a.x + row * a.ld_x, a.d, a.x, end, t, gt);
        cp_async_commit();
        put = put + 1 == kAnyStages ? 0 : put + 1;
    };
    #pragma unroll 1
    for (int s = 0; s < kAnyStages - 1; ++s) issue(first + s * step);
    float w[kAnyE], b[kAnyE];
    #pragma unroll
    for (int k = 0; k < kAnyE; ++k) {
        const int c = k * gt + t;
        w[k] = a.w && c < a.d ? param_at(a.w, a.param_f32, c) + a.offset : 1.f;
        b[k] = a.b && c < a.d ? param_at(a.b, a.param_f32, c) : 0.f;
    }
    const float inv_d = 1.0f / float(a.d);
    for (int64_t row = first; row < a.rows; row += step, par ^= 1) {
        cp_async_wait<kAnyStages - 2>();
        group_barrier(sh, 1 + g);                         // the other threads' chunks, too
        const uint16_t* x = staged(ring + get * slot, a.x + row * a.ld_x);
        get = get + 1 == kAnyStages ? 0 : get + 1;
        float f[kAnyE], sum = 0.f, sq = 0.f, mean = 0.f;
        #pragma unroll
        for (int k = 0; k < kAnyE; ++k) f[k] = k * gt + t < a.d ? bf16_bits_to_float(x[k * gt + t]) : 0.f;
        issue(row + (kAnyStages - 1) * step);             // into the slot of the row before: all have read it
        #pragma unroll
        for (int k = 0; k < kAnyE; ++k) sum += f[k];
        if (!a.rms) mean = group_sum1(sum, &s_x[par][0][g * sh.nw], wg, sh, 1 + g) * inv_d;
        #pragma unroll
        for (int k = 0; k < kAnyE; ++k) {
            f[k] = k * gt + t < a.d ? f[k] - mean : 0.f;
            sq += f[k] * f[k];
        }
        const float rstd = rsqrtf(group_sum1(sq, &s_x[par][1][g * sh.nw], wg, sh, 1 + g) * inv_d + a.eps);
        if (t == 0) {
            if (!a.rms) a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        uint16_t* y = a.y + row * a.ld_y;
        #pragma unroll
        for (int k = 0; k < kAnyE; ++k)
            if (k * gt + t < a.d)
                y[k * gt + t] = __bfloat16_as_ushort(__float2bfloat16_rn(f[k] * rstd * w[k] + b[k]));
    }
    cp_async_wait<0>();
}

template <int kFormat>
__global__ void __launch_bounds__(kRingThreads, 1) k_norm_bwd_any(NormBwdArgs a, RingShape sh, int slot) {
    constexpr bool kHeld8 = kFormat != DLM_PACK_NONE;
    extern __shared__ uint4 ring_mem[];                   // [group][kAnyStages][dy, x: slot bytes each]; then [2][d] floats
    __shared__ float2 s_x[2][kRingThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = warp / sh.nw, wg = warp - g * sh.nw;
    const int t = wg * 32 + lane, gt = sh.nw * 32;
    uint8_t* ring = reinterpret_cast<uint8_t*>(ring_mem) + size_t(g) * kAnyStages * 2 * slot;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t first = int64_t(g) * gridDim.x + blockIdx.x, step = int64_t(sh.groups) * gridDim.x;
    const int nb = (a.d + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK;
    const uint16_t* end_dy = a.dy + (a.rows - 1) * a.ld_dy + a.d;
    const uint16_t* end_x = kHeld8 ? nullptr : a.x + (a.rows - 1) * a.ld_x + a.d;
    const uint8_t* end_q = kHeld8 ? a.q + a.rows * a.d : nullptr;
    int put = 0, get = 0, par = 0;
    auto issue = [&](int64_t row) {
        if (row < a.rows) {
            uint8_t* at = ring + put * 2 * slot;
            stage_row(at, a.dy + row * a.ld_dy, a.d, a.dy, end_dy, t, gt);
            if constexpr (kHeld8) stage_row(at + slot, a.q + row * a.d, a.d, a.q, end_q, t, gt);
            else stage_row(at + slot, a.x + row * a.ld_x, a.d, a.x, end_x, t, gt);
        }
        cp_async_commit();
        put = put + 1 == kAnyStages ? 0 : put + 1;
    };
    #pragma unroll 1
    for (int s = 0; s < kAnyStages - 1; ++s) issue(first + s * step);
    float w[kAnyE], dw[kAnyE], db[kAnyE];
    #pragma unroll
    for (int k = 0; k < kAnyE; ++k) {
        const int c = k * gt + t;
        w[k] = a.w && c < a.d ? param_at(a.w, a.param_f32, c) + a.offset : 1.f;
        dw[k] = db[k] = 0.f;
    }
    const float inv_d = 1.0f / float(a.d);
    for (int64_t row = first; row < a.rows; row += step, par ^= 1) {
        const float mean = a.rms ? 0.f : __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
        cp_async_wait<kAnyStages - 2>();
        group_barrier(sh, 1 + g);
        const uint8_t* at = ring + get * 2 * slot;
        const uint16_t* y = staged(at, a.dy + row * a.ld_dy);
        get = get + 1 == kAnyStages ? 0 : get + 1;
        float xh[kAnyE], dy[kAnyE], s1 = 0.f, s2 = 0.f;
        #pragma unroll
        for (int k = 0; k < kAnyE; ++k) {
            const int c = k * gt + t;
            xh[k] = dy[k] = 0.f;
            if (c < a.d) {
                dy[k] = bf16_bits_to_float(y[c]);
                float x;
                if constexpr (kHeld8)
                    x = fmaf(unpack_code(staged(at + slot, a.q + row * a.d)[c], kFormat),
                             __ldg(a.q_scale + row * nb + c / DLM_PACK_BLOCK), -mean);
                else
                    x = bf16_bits_to_float(staged(at + slot, a.x + row * a.ld_x)[c]) - mean;
                xh[k] = x * rstd;
            }
        }
        issue(row + (kAnyStages - 1) * step);
        #pragma unroll
        for (int k = 0; k < kAnyE; ++k) {
            const float gk = dy[k] * w[k];
            s1 += gk;
            s2 += gk * xh[k];
            dw[k] += dy[k] * xh[k];
            db[k] += dy[k];
        }
        group_sum2<false>(s1, s2, &s_x[par][g * sh.nw], wg, sh, 1 + g);
        const float m1 = a.rms ? 0.f : s1 * inv_d, m2 = s2 * inv_d;
        uint16_t* dx = a.dx + row * a.ld_dx;
        #pragma unroll
        for (int k = 0; k < kAnyE; ++k)
            if (k * gt + t < a.d)
                dx[k * gt + t] = __bfloat16_as_ushort(__float2bfloat16_rn((dy[k] * w[k] - m1 - xh[k] * m2) * rstd));
    }
    // the groups' sums, added in the order of the groups
    cp_async_wait<0>();
    float* acc = reinterpret_cast<float*>(ring_mem);
    for (int i = 0; i < sh.groups; ++i) {
        __syncthreads();
        if (g != i) continue;
        #pragma unroll
        for (int k = 0; k < kAnyE; ++k) {
            const int c = k * gt + t;
            if (c < a.d) {
                acc[c] = i ? acc[c] + dw[k] : dw[k];
                acc[a.d + c] = i ? acc[a.d + c] + db[k] : db[k];
            }
        }
    }
    __syncthreads();
    float* part = a.part + int64_t(blockIdx.x) * 2 * a.pitch;
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        if (a.d_weight) part[c] = acc[c];
        if (a.d_bias) part[a.pitch + c] = acc[a.d + c];
    }
}

// Any width and alignment: a CTA per row, which it reads up to three times
// (from L2 after the first).  Two-byte loads: 7,455 x 9,001 in 149 us, 0.28 of
// the copy rate.
constexpr int kWideThreads = 512;

__device__ __forceinline__ float cta_sum(float v, float* s) {
    v = warp_sum(v);
    __syncthreads();                  // earlier readers of s are done
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < kWideThreads / 32; ++w) v += s[w];
    return v;
}

__global__ void __launch_bounds__(kWideThreads) k_norm_fwd_wide(NormFwdArgs a) {
    __shared__ float s[kWideThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const float inv_d = 1.0f / float(a.d);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const uint16_t* x = a.x + row * a.ld_x;
        float mean = 0.f, v = 0.f;
        if (!a.rms) {
            for (int c = threadIdx.x; c < a.d; c += kWideThreads) v += bf16_bits_to_float(__ldg(x + c));
            mean = cta_sum(v, s) * inv_d;
        }
        v = 0.f;
        for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
            const float u = bf16_bits_to_float(__ldg(x + c)) - mean;
            v += u * u;
        }
        const float rstd = rsqrtf(cta_sum(v, s) * inv_d + a.eps);
        if (threadIdx.x == 0) {
            if (!a.rms) a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
            const float w = a.w ? param_at(a.w, a.param_f32, c) + a.offset : 1.f;
            const float b = a.b ? param_at(a.b, a.param_f32, c) : 0.f;
            a.y[row * a.ld_y + c] = __bfloat16_as_ushort(
                __float2bfloat16_rn((bf16_bits_to_float(__ldg(x + c)) - mean) * rstd * w + b));
        }
    }
}

// Any width and alignment: a CTA walks over its rows twice each and keeps its
// partial row in the workspace, which only it touches.  Plain, not fast: two-byte
// loads, and 16 bytes an element for the partial row beside the pass's 6 (5,461 x
// 12,288: 1,188 us, 0.05 of the copy rate; 7,455 x 9,001: 1,064).
__global__ void __launch_bounds__(kWideThreads) k_norm_bwd_wide(NormBwdArgs a) {
    __shared__ float s[kWideThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const float inv_d = 1.0f / float(a.d);
    const int nb = (a.d + DLM_PACK_BLOCK - 1) / DLM_PACK_BLOCK;
    float* part = a.part + int64_t(blockIdx.x) * 2 * a.pitch;
    bool first = true;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false) {
        const float mean = a.rms ? 0.f : a.mean[row], rstd = a.rstd[row];
        auto xh_at = [&](int c) {
            const float x = a.x ? bf16_bits_to_float(__ldg(a.x + row * a.ld_x + c)) - mean
                                : fmaf(unpack_code(__ldg(a.q + row * a.d + c), a.format),
                                       __ldg(a.q_scale + row * nb + c / DLM_PACK_BLOCK), -mean);
            return x * rstd;
        };
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
            const float xh = xh_at(c), dy = bf16_bits_to_float(__ldg(a.dy + row * a.ld_dy + c));
            const float g = dy * (a.w ? param_at(a.w, a.param_f32, c) + a.offset : 1.f);
            s1 += g;
            s2 += g * xh;
            if (a.d_weight) part[c] = (first ? 0.f : part[c]) + dy * xh;
            if (a.d_bias) part[a.pitch + c] = (first ? 0.f : part[a.pitch + c]) + dy;
        }
        s1 = cta_sum(s1, s);
        s2 = cta_sum(s2, s);
        const float m1 = a.rms ? 0.f : s1 * inv_d, m2 = s2 * inv_d;
        for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
            const float dy = bf16_bits_to_float(__ldg(a.dy + row * a.ld_dy + c));
            const float g = dy * (a.w ? param_at(a.w, a.param_f32, c) + a.offset : 1.f);
            a.dx[row * a.ld_dx + c] = __bfloat16_as_ushort(__float2bfloat16_rn((g - m1 - xh_at(c) * m2) * rstd));
        }
    }
}

// dw (blockIdx.y = 0) and db (1) from the partial rows: a lane per column, the
// warps take consecutive parts of the rows.
constexpr int kNormJoinWarps = 16;

__global__ void __launch_bounds__(kNormJoinWarps * 32) k_norm_join(const float* __restrict__ part, int n_part,
                                                                   int pitch, int d, int grad_f32, int accumulate,
                                                                   void* __restrict__ d_weight,
                                                                   void* __restrict__ d_bias) {
    __shared__ float s[kNormJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    void* out = blockIdx.y ? d_bias : d_weight;
    pdl_wait();
    if (!out) return;
    const int per = (n_part + kNormJoinWarps - 1) / kNormJoinWarps;
    const int k0 = min(n_part, warp * per), k1 = min(n_part, k0 + per);
    float acc = 0.f;
    if (c < d) {
        const float* p = part + blockIdx.y * pitch + c;
        constexpr int kU = 10;         // loads in flight: 148 partial rows are one batch for each warp
        for (int k = k0; k < k1; k += kU) {
            float v[kU];
            #pragma unroll
            for (int u = 0; u < kU; ++u) v[u] = k + u < k1 ? p[int64_t(k + u) * 2 * pitch] : 0.f;
            #pragma unroll
            for (int u = 0; u < kU; ++u) acc += v[u];
        }
    }
    s[warp][lane] = acc;
    __syncthreads();
    if (warp || c >= d) return;
    acc = 0.f;
    #pragma unroll
    for (int w = 0; w < kNormJoinWarps; ++w) acc += s[w][lane];
    put_grad(out, c, acc, grad_f32, accumulate);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static bool finite_f(float v) { return v - v == 0.0f; }

static bool param_aligned(const void* p) { return !p || aligned16(p); }

template <int kNW>
static dlm_status_t launch_fwd(void (*kern)(NormFwdArgs), const NormFwdArgs& a, cudaStream_t s) {
    constexpr int kG = groups_per_cta(kNW);
    return launch_pdl(kern, dim3(unsigned((a.rows + kG - 1) / kG)), dim3(kNW * kG * 32), 0, s, "k_norm_fwd launch", a);
}

// Which forward kernel, by the call's 16-byte pieces (rows x d / 8).  The fewer,
// the more warps share a row, so that one row's time, not the bandwidth,
// counts less; the ring pays once its start is spread over enough rows.
// Measured (us), d = 4,096, one / two / four pieces a lane / ring:
//   148 rows 2.5 / 2.9 / 3.6 / 4.4   600 rows 4.8 / 3.8 / 4.5 / 5.0
//   1,000 rows 6.5 / 5.7 / 4.7 / 5.6   16,384 rows - / - / 52.0 / 46.2
// and at d = 1,024: 1,000 rows 2.9 / 3.0 / 3.7, 6,144 rows - / - / 7.3 / 6.8.
// With the checkpoint written too the ring is not faster (67.2 against 65.4 at
// 16,384 x 4,096) and is not built.
constexpr int64_t kOnePiece = 148 * 1024, kTwoPieces = 148 * 2560, kRingPieces = 148 * 4608;

// warps that a row of `pieces` pieces takes at `per` pieces a lane: a power of
// two up to 32, with four a lane any number up to 8; 0 if they do not hold it.
// (With the checkpoint, 13,107 x 5,120: 91.1 us with 8 warps, 69.0 with 5.)
static int warps_for(int64_t pieces, int per) {
    for (int nw = 1; nw <= 32; nw = per == 4 && nw < 8 ? nw + 1 : 2 * nw)
        if (pieces <= int64_t(nw) * 32 * per) return nw;
    return 0;
}

template <int kN>
static dlm_status_t launch_fwd_vec(const NormFwdArgs& a, cudaStream_t s) {
    switch (warps_for(a.d / 8, kN)) {
        case 1: return launch_fwd<1>(k_norm_fwd_vec<kN, 1>, a, s);
        case 2: return launch_fwd<2>(k_norm_fwd_vec<kN, 2>, a, s);
        case 4: return launch_fwd<4>(k_norm_fwd_vec<kN, 4>, a, s);
        case 8: return launch_fwd<8>(k_norm_fwd_vec<kN, 8>, a, s);
        case 16: return launch_fwd<16>(k_norm_fwd_vec<kN, 16>, a, s);
        default: break;
    }
    if constexpr (kN == 4) {
        switch (warps_for(a.d / 8, kN)) {
            case 3: return launch_fwd<3>(k_norm_fwd_vec<kN, 3>, a, s);
            case 5: return launch_fwd<5>(k_norm_fwd_vec<kN, 5>, a, s);
            case 6: return launch_fwd<6>(k_norm_fwd_vec<kN, 6>, a, s);
            case 7: return launch_fwd<7>(k_norm_fwd_vec<kN, 7>, a, s);
            default: break;
        }
    }
    return launch_fwd<32>(k_norm_fwd_vec<kN, 32>, a, s);
}

// Ring kernels: one piece a lane up to 256 columns, two beyond, as long as 16
// warps hold a row; nw = 0: they do not.  `three`: three pieces where that makes
// two groups out of one, whose exchanges then hide each other (forward, 13,107 x
// 5,120: 59.6 us with two, 52.6 with three; 10,923 x 6,144: 53.9, 50.6).  The
// backward pass would spill registers (86.9, 146.9).
static RingShape ring_shape(int32_t d, bool shift, bool three, int* pieces) {
    const int nv = (d + 7) / 8 + (shift ? 1 : 0);        // a row may reach into one chunk more
    constexpr int warps = kRingThreads / 32;
    *pieces = nv <= 32 ? 1 : 2;
    RingShape sh = {(nv + 32 * *pieces - 1) / (32 * *pieces), 0};
    if (three && sh.nw > warps / 2 && nv <= warps / 2 * 96) {
        *pieces = 3;
        sh.nw = (nv + 95) / 96;
    }
    if (sh.nw > warps) sh.nw = 0;
    else sh.groups = warps / sh.nw < 15 || sh.nw == 1 ? warps / sh.nw : 15;   // a barrier for each
    return sh;
}

// kSlots: a thread's 16-byte slots in shared memory; kThreads: the kernel's bound
template <auto kKern, int kSlots, int kThreads, typename Args>
static dlm_status_t launch_ring(const Args& a, RingShape sh, unsigned grid, cudaStream_t s, const char* what) {
    const unsigned threads = unsigned(sh.nw * sh.groups * 32);
    dlm_status_t st = allow_smem<kKern, kSlots * kThreads * 16>(what);
    if (st != DLM_OK) return st;
    return launch_pdl(kKern, dim3(grid), dim3(threads), size_t(kSlots) * threads * 16, s, what, a, sh);
}

template <int kN, bool kShift>
static dlm_status_t launch_fwd_ring(const NormFwdArgs& a, RingShape sh, unsigned grid, cudaStream_t s) {
    const char* what = "k_norm_fwd launch";
    constexpr int kSlots = 2 * kN * fwd_stages<kN>();
    return a.rms ? launch_ring<k_norm_fwd_ring<kN, kShift, kShift ? kNothing : kAsk>, kSlots, kRingThreads>(a, sh, grid, s, what)
                 : launch_ring<k_norm_fwd_ring<kN, kShift, kSubtract>, kSlots, kRingThreads>(a, sh, grid, s, what);
}

template <bool kShift>
static dlm_status_t launch_fwd_ring(int pieces, const NormFwdArgs& a, RingShape sh, unsigned grid, cudaStream_t s) {
    return pieces == 1 ? launch_fwd_ring<1, kShift>(a, sh, grid, s)
         : pieces == 2 ? launch_fwd_ring<2, kShift>(a, sh, grid, s) : launch_fwd_ring<3, kShift>(a, sh, grid, s);
}

template <int kN, int kFormat, bool kShift, bool kLean>
static dlm_status_t launch_bwd_ring(const NormBwdArgs& a, RingShape sh, unsigned grid, cudaStream_t s) {
    const char* what = "k_norm_bwd launch";
    if constexpr (kN == 2 && !kShift && (kLean || kFormat == DLM_PACK_NONE))
        if (sh.groups == 1 && sh.nw * 32 <= kTwoThreads)
            return launch_ring<k_norm_bwd_two<kFormat, kLean>, 4 * kTwoStages, kTwoThreads>(a, sh, grid, s, what);
    return launch_ring<k_norm_bwd_ring<kN, kFormat, kShift, kLean>, 2 * kN * bwd_stages<kN>(), kRingThreads>(a, sh, grid,
                                                                                                             s, what);
}

template <int kFormat, bool kShift>
static dlm_status_t launch_bwd_ring(int pieces, const NormBwdArgs& a, RingShape sh, unsigned grid, cudaStream_t s) {
    if (a.rms && !a.d_bias)
        return pieces == 1 ? launch_bwd_ring<1, kFormat, kShift, true>(a, sh, grid, s)
                           : launch_bwd_ring<2, kFormat, kShift, true>(a, sh, grid, s);
    return pieces == 1 ? launch_bwd_ring<1, kFormat, kShift, false>(a, sh, grid, s)
                       : launch_bwd_ring<2, kFormat, kShift, false>(a, sh, grid, s);
}

template <bool kShift>
static dlm_status_t launch_bwd_ring(int pieces, const NormBwdArgs& a, RingShape sh, unsigned grid, cudaStream_t s) {
    return a.format == DLM_PACK_NONE ? launch_bwd_ring<DLM_PACK_NONE, kShift>(pieces, a, sh, grid, s)
         : a.format == DLM_PACK_INT8 ? launch_bwd_ring<DLM_PACK_INT8, kShift>(pieces, a, sh, grid, s)
                                     : launch_bwd_ring<DLM_PACK_E4M3, kShift>(pieces, a, sh, grid, s);
}

static unsigned ring_grid(int64_t rows) { return unsigned(rows < 148 ? rows : 148); }

// CTAs for rows that are not on 16-byte borders: the rows of a group are a
// multiple of 8 apart.
static unsigned shift_grid(int64_t rows, RingShape sh) {
    unsigned grid = ring_grid(rows);
    if (rows > grid)
        while (grid * unsigned(sh.groups) % 8) --grid;
    return grid;
}

// Kernels for any alignment: 16 elements a lane, as long as 16 warps hold a row.
static RingShape any_shape(int32_t d) {
    RingShape sh = {(d + 32 * kAnyE - 1) / (32 * kAnyE), 0};
    if (sh.nw > 16) sh.nw = 0;
    else sh.groups = kRingThreads / 32 / sh.nw < 15 || sh.nw == 1 ? kRingThreads / 32 / sh.nw : 15;
    return sh;
}

// A slot holds a row's chunks.  16 warps x 512 elements bound what a CTA's
// groups hold together: 12 slots a group (backward: two tensors) of 2 d + 45
// bytes at most are 12 x (16 KB + 16 x 45 B); the sums at the end, 8 d, are less.
constexpr int kAnySmem = 12 * (16 * 1024 + 16 * 45);

template <auto kKern, typename Args>
static dlm_status_t launch_any(const Args& a, RingShape sh, int tensors, cudaStream_t s, const char* what) {
    const int slot = int(align_up(size_t(a.d) * 2 + 30, 16));
    size_t smem = size_t(sh.groups) * kAnyStages * tensors * slot;
    if (smem < size_t(a.d) * 8) smem = size_t(a.d) * 8;
    dlm_status_t st = allow_smem<kKern, kAnySmem>(what);
    if (st != DLM_OK) return st;
    return launch_pdl(kKern, dim3(ring_grid(a.rows)), dim3(unsigned(sh.nw * sh.groups * 32)), smem, s, what, a, sh, slot);
}

// The backward pass leaves one partial row per CTA, of which there is at most
// one per SM, whatever the kernel.
// Up to so many rows a group, one CTA takes them all and writes the gradients
// itself, without a second launch (d = 4,096, GPU time alone: 2 rows 5.9 us in
// one launch, 5 rows 6.4 in two; 4 rows a group took 9.0 against 6.4).
constexpr int kAloneRows = 2;

struct NormBwdPlan { unsigned grid; int pitch; size_t bytes; };

static bool norm_bwd_plan(int64_t rows, int32_t d, NormBwdPlan* p) {
    if (rows < 0 || rows > INT32_MAX || d < 1 || d > INT32_MAX - 1024) return false;
    p->grid = ring_grid(rows);
    p->pitch = int(align_up(size_t(d), 32));
    p->bytes = align_up((size_t(p->grid) * 2 + 1) * size_t(p->pitch) * 4, kWsAlign);
    return true;
}

}  // namespace dlm

using namespace dlm;

extern "C" dlm_status_t dlm_norm_fwd(const uint16_t* x, int64_t rows, int32_t d_model, int64_t ld_x,
                                     const void* weight, const void* bias, int32_t param_dtype, int32_t kind,
                                     float eps, float weight_offset, uint16_t* y, int64_t ld_y, float* mean,
                                     float* rstd, int32_t pack_format, uint8_t* q, float* q_scale,
                                     dlm_stream_t stream) {
    DLM_NVTX("dlm_norm_fwd");
    if (rows < 0 || rows > INT32_MAX || d_model < 1 || d_model > INT32_MAX - 1024 || ld_x < d_model || ld_y < d_model)
        return DLM_ERR_INVALID_ARGUMENT;
    if (kind != DLM_NORM_LAYER && kind != DLM_NORM_RMS) return DLM_ERR_INVALID_ARGUMENT;
    if (param_dtype != DLM_BF16 && param_dtype != DLM_F32) return DLM_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0.0f) || !finite_f(eps) || !finite_f(weight_offset)) return DLM_ERR_INVALID_ARGUMENT;
    if (pack_format != DLM_PACK_NONE && pack_format != DLM_PACK_INT8 && pack_format != DLM_PACK_E4M3)
        return DLM_ERR_INVALID_ARGUMENT;
    if (rows == 0) return DLM_OK;
    if (!x || !y || !rstd || (kind == DLM_NORM_LAYER && !mean)) return DLM_ERR_INVALID_ARGUMENT;
    if (pack_format != DLM_PACK_NONE && (!q || !q_scale)) return DLM_ERR_INVALID_ARGUMENT;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    NormFwdArgs a = {x, rows, ld_x, d_model, weight, bias, param_dtype == DLM_F32, kind == DLM_NORM_RMS, eps,
                     weight_offset, y, ld_y, mean, rstd, pack_format, q, q_scale};
    const bool vec = d_model % 8 == 0 && ld_x % 8 == 0 && ld_y % 8 == 0 && aligned16(x) && aligned16(y) &&
                     param_aligned(weight) && param_aligned(bias) && (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    int pieces = 0;
    RingShape sh = ring_shape(d_model, false, true, &pieces);
    if (vec) {
        const int nv = d_model / 8;
        const int64_t all = rows * nv;                   // 16-byte pieces of the call
        if (sh.nw && all >= kRingPieces && pack_format == DLM_PACK_NONE)
            return launch_fwd_ring<false>(pieces, a, sh, ring_grid(rows), s);
        // (rows of up to 256 or 512 columns fill a warp by one or two pieces a lane: 262,147 x 256 with the
        // checkpoint 92 us, with four pieces 165)
        if ((all <= kOnePiece || nv <= 32) && warps_for(nv, 1)) return launch_fwd_vec<1>(a, s);
        if ((all <= kTwoPieces || nv <= 64) && warps_for(nv, 2)) return launch_fwd_vec<2>(a, s);
        if (warps_for(nv, 4)) return launch_fwd_vec<4>(a, s);
    }
    // rows of x and y in step with one another, if not with the 16-byte borders
    const bool shift = aligned16(x) && aligned16(y) && (ld_x - ld_y) % 8 == 0;
    sh = ring_shape(d_model, true, true, &pieces);
    const RingShape any = any_shape(d_model);
    if (shift && sh.nw)
        st = launch_fwd_ring<true>(pieces, a, sh, shift_grid(rows, sh), s);
    else if (any.nw) st = launch_any<k_norm_fwd_any>(a, any, 1, s, "k_norm_fwd launch");
    else st = launch_pdl(k_norm_fwd_wide, dim3(unsigned(rows < 148 * 4 ? rows : 148 * 4)), dim3(kWideThreads), 0, s,
                         "k_norm_fwd_wide launch", a);
    if (st != DLM_OK || pack_format == DLM_PACK_NONE) return st;
    return dlm_pack8(x, rows, d_model, ld_x, pack_format, q, q_scale, stream);
}

extern "C" size_t dlm_norm_bwd_workspace_size(int64_t rows, int32_t d_model) {
    NormBwdPlan p;
    return norm_bwd_plan(rows, d_model, &p) ? p.bytes : 0;
}

extern "C" dlm_status_t dlm_norm_bwd(const uint16_t* d_y, int64_t ld_dy, const uint16_t* x, int64_t ld_x,
                                     int32_t pack_format, const uint8_t* q, const float* q_scale, const float* mean,
                                     const float* rstd, const void* weight, int32_t param_dtype, int32_t kind,
                                     float weight_offset, int64_t rows, int32_t d_model, uint16_t* d_x,
                                     int64_t ld_dx, int32_t grad_dtype, int32_t accumulate, void* d_weight,
                                     void* d_bias, void* workspace, size_t workspace_bytes, dlm_stream_t stream) {
    DLM_NVTX("dlm_norm_bwd");
    NormBwdPlan p;
    if (!norm_bwd_plan(rows, d_model, &p)) return DLM_ERR_INVALID_ARGUMENT;
    if (ld_dy < d_model || ld_dx < d_model) return DLM_ERR_INVALID_ARGUMENT;
    if (kind != DLM_NORM_LAYER && kind != DLM_NORM_RMS) return DLM_ERR_INVALID_ARGUMENT;
    if ((param_dtype != DLM_BF16 && param_dtype != DLM_F32) || (grad_dtype != DLM_BF16 && grad_dtype != DLM_F32))
        return DLM_ERR_INVALID_ARGUMENT;
    if ((accumulate != 0 && accumulate != 1) || !finite_f(weight_offset)) return DLM_ERR_INVALID_ARGUMENT;
    if (pack_format == DLM_PACK_NONE) {
        if (ld_x < d_model || (rows > 0 && !x)) return DLM_ERR_INVALID_ARGUMENT;
    } else if ((pack_format != DLM_PACK_INT8 && pack_format != DLM_PACK_E4M3) || (rows > 0 && (!q || !q_scale))) {
        return DLM_ERR_INVALID_ARGUMENT;
    }
    if (rows > 0 && (!d_y || !d_x || !rstd || (kind == DLM_NORM_LAYER && !mean))) return DLM_ERR_INVALID_ARGUMENT;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kWsAlign) return DLM_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < p.bytes) return DLM_ERR_WORKSPACE_TOO_SMALL;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    NormBwdArgs a = {d_y, ld_dy, pack_format == DLM_PACK_NONE ? x : nullptr, ld_x, pack_format, q, q_scale, mean,
                     rstd, weight, param_dtype == DLM_F32, kind == DLM_NORM_RMS, weight_offset, rows, d_model, d_x,
                     ld_dx, static_cast<float*>(workspace), p.pitch,
                     d_weight, d_bias, grad_dtype == DLM_F32, accumulate};
    bool alone = false;      // one CTA, which writes the gradients itself
    if (rows > 0) {
        const bool vec = d_model % 8 == 0 && ld_dy % 8 == 0 && ld_dx % 8 == 0 && aligned16(d_y) && aligned16(d_x) &&
                         (a.x ? ld_x % 8 == 0 && aligned16(x) : (reinterpret_cast<uintptr_t>(q) & 7) == 0);
        // rows in step with one another, if not with the 16-byte borders
        const bool shift = aligned16(d_y) && aligned16(d_x) && (ld_dy - ld_dx) % 8 == 0 &&
                           (a.x ? aligned16(x) && (ld_dy - ld_x) % 8 == 0
                                : (reinterpret_cast<uintptr_t>(q) & 7) == 0 && (ld_dy - d_model) % 8 == 0);
        int pieces = 0;
        const RingShape sh = ring_shape(d_model, !vec, false, &pieces), any = any_shape(d_model);
        const bool ring = (vec || shift) && sh.nw;
        // (a group's rows are `groups` apart then: in step only if that is a multiple of 8)
        if (ring && rows <= (vec || sh.groups % 8 == 0 ? int64_t(kAloneRows) * sh.groups : sh.groups)) {
            p.grid = 1;
            alone = true;
        }
        if (vec && sh.nw) {
            st = launch_bwd_ring<false>(pieces, a, sh, p.grid, s);
        } else if (shift && sh.nw) {
            if (!alone) p.grid = shift_grid(rows, sh);
            st = launch_bwd_ring<true>(pieces, a, sh, p.grid, s);
        } else if (any.nw) {
            const char* what = "k_norm_bwd launch";
            st = pack_format == DLM_PACK_NONE ? launch_any<k_norm_bwd_any<DLM_PACK_NONE>>(a, any, 2, s, what)
               : pack_format == DLM_PACK_INT8 ? launch_any<k_norm_bwd_any<DLM_PACK_INT8>>(a, any, 2, s, what)
                                              : launch_any<k_norm_bwd_any<DLM_PACK_E4M3>>(a, any, 2, s, what);
        } else {
            st = launch_pdl(k_norm_bwd_wide, dim3(p.grid), dim3(kWideThreads), 0, s, "k_norm_bwd_wide launch", a);
        }
        if (st != DLM_OK) return st;
    }
    if ((!d_weight && !d_bias) || alone || (rows == 0 && accumulate)) return DLM_OK;
    return launch_pdl(k_norm_join, dim3(unsigned((d_model + 31) / 32), 2), dim3(kNormJoinWarps * 32), 0, s,
                      "k_norm_join launch", (const float*)a.part, int(p.grid), p.pitch, d_model,
                      int(grad_dtype == DLM_F32), accumulate, d_weight, d_bias);
}
