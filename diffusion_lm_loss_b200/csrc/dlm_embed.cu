// dlm_embed.cu -- token embedding with a scale, and its gradient.
//
// Forward: out[i, :] = bf16(scale * W[id_i, :]), a warp per 1,024 columns of a
// token's row; bound by HBM (16,384 tokens of 4,096 columns: 33 us, 0.92 of the
// copy rate).
//
// Gradient: dW[v, :] = scale * sum over the tokens i with id_i = v of
// dOut[i, :].  Absorbing noise makes one id (the mask) carry about half of
// the tokens while most other ids have none or one, so the work is split by
// sorted token positions, not by vocabulary rows:
//   k_embed_sort   one CTA per range of vocabulary rows reads all ids, counts
//                  those of its range per warp and row, and writes the range's
//                  tokens in row order at the right place (the ids below the
//                  range, counted in the same pass, give the offset): no
//                  communication between CTAs, and an order that depends on
//                  the ids and pads, not on timing.
//   k_embed_grad   one CTA per 8 to 32 sorted positions and column tile adds
//                  rows in that order, in fp32 registers; a row that begins
//                  and ends inside the chunk is written at once, a row that
//                  crosses a chunk's border leaves one fp32 partial per chunk.
//   k_embed_join   adds the partials of the crossing rows, in chunk order.
// The rows that no token has are written by more CTAs of the last two launches.
// Nothing is added atomically: results are bitwise reproducible.  The table's
// gradient has to be written once and every token's row read once: 16,384
// tokens, half of them masked, on a table of 1 GB take 184 us, 0.97 of the copy
// rate; about 8 us of that is the sort, which nothing hides (zeroing part of the
// table beside it gained nothing: the memory is still writing what came before).
// Added to another gradient they take 60 us, 0.67.
#include <type_traits>

#include "dlm_device.cuh"
#include "dlm_host.h"
#include "dlm_shift.cuh"

namespace dlm {

constexpr int kEmbThreads = 256;
// Sorted positions per CTA (at most one per lane): 32, or fewer until the call
// has 16 warps per SM -- with few warps the chunks' rows, read one batch after
// the other, set the time (256 tokens of 2,048 columns: 23 us with 32, 19 with
// 8; adding 300 tokens to a large table 20 and 13).
constexpr int kMaxChunk = 32, kMinChunk = 8;
// Vocabulary rows per sorting CTA: one CTA per SM up to 265,216 rows.  A
// counter for each row and warp: 32 warps with up to 896 rows, 16 with more
// (112 KB either way).
constexpr int kMaxRange = 1792;
constexpr size_t kSortSmem = 16 * kMaxRange * 4;
constexpr int kGradThreads = 128;
constexpr int kJoinWarps = 16;

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <bool kAligned>
__global__ void __launch_bounds__(kEmbThreads) k_embed_fwd(const int32_t* __restrict__ ids,
                                                           const uint8_t* __restrict__ pad, int64_t n_tokens,
                                                           const uint16_t* __restrict__ w, int64_t ld_w, int vocab,
                                                           int d, float scale, uint16_t* __restrict__ out,
                                                           int64_t ld_out, uint32_t* __restrict__ status) {
    constexpr int kU = 4;              // pieces of 8 columns a lane, 256 apart
    pdl_wait();                        // ids come from the corruption kernel
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int slabs = (d + 256 * kU - 1) / (256 * kU);
    const int64_t items = n_tokens * slabs;
    const int64_t step = int64_t(gridDim.x) * (kEmbThreads / 32);
    for (int64_t it = int64_t(blockIdx.x) * (kEmbThreads / 32) + threadIdx.x / 32; it < items; it += step) {
        const int64_t i = it / slabs;
        const int s = int(it - i * slabs);
        const bool is_pad = pad && pad[i];
        const int id = is_pad ? -1 : ids[i];
        const bool ok = uint32_t(id) < uint32_t(vocab);
        if (!ok && !is_pad && s == 0 && lane == 0 && status) atomicOr(status, DLM_DEV_BAD_TOKEN_ID);
        const int c = s * 256 * kU + lane * 8;
        const uint16_t* src = w + int64_t(ok ? id : 0) * ld_w + c;
        uint16_t* dst = out + i * ld_out + c;
        uint4 r[kU];
        if constexpr (kAligned) {
            #pragma unroll
            for (int u = 0; u < kU; ++u)
                r[u] = c + 256 * u < d ? __ldg(reinterpret_cast<const uint4*>(src + 256 * u)) : make_uint4(0, 0, 0, 0);
        } else {
            load_pieces<kU>(src, c, d, w, w + (vocab - 1) * ld_w + d, r);
        }
        #pragma unroll
        for (int u = 0; u < kU; ++u) {
            uint32_t x[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
            #pragma unroll
            for (int k = 0; k < 4; ++k)
                x[k] = ok ? pack_bf16x2(bf16lo(x[k]) * scale, bf16hi(x[k]) * scale) : 0u;
            r[u] = make_uint4(x[0], x[1], x[2], x[3]);
            if (kAligned && c + 256 * u < d) *reinterpret_cast<uint4*>(dst + 256 * u) = r[u];
        }
        if constexpr (!kAligned) store_pieces<kU>(dst, c, d, r);
    }
}

// ---------------------------------------------------------------------------
// gradient: the sort
// ---------------------------------------------------------------------------
struct EmbHeader {
    uint32_t status;      // DLM_DEV_* bits of this call
};

// Calls f(token, ids) for the tokens of one warp's section, 128 at a time, four
// consecutive ones a lane, with kDeep times as many loaded ahead; every lane
// takes part in every call.  Pads and places without a token come as id -1.
// bad: becomes true where a token that is no pad has an id outside [0, vocab);
// NULL: not looked for.
template <int kDeep, typename F>
__device__ __forceinline__ void for_section(const int32_t* __restrict__ ids, const uint8_t* __restrict__ pad,
                                            int64_t beg, int64_t end, bool wide, int vocab, bool* bad, F&& f) {
    const int lane = threadIdx.x & 31;
    #pragma unroll 1
    for (int64_t i = beg; i < end; i += 128 * kDeep) {
        int id[kDeep][4];
        #pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int64_t at = i + 128 * k + lane * 4;
            if (wide && at + 4 <= end) {
                const int4 q = __ldg(reinterpret_cast<const int4*>(ids + at));
                id[k][0] = q.x; id[k][1] = q.y; id[k][2] = q.z; id[k][3] = q.w;
            } else {
                #pragma unroll
                for (int e = 0; e < 4; ++e) id[k][e] = at + e < end ? __ldg(ids + at + e) : -1;
            }
        }
        uint32_t pads = 0;                 // bit 4 k + e: a pad, or no token
        if (pad || i + 128 * kDeep > end) {
            #pragma unroll
            for (int k = 0; k < kDeep; ++k)
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t at = i + 128 * k + lane * 4 + e;
                    if (at >= end || (pad && pad[at])) pads |= 1u << (4 * k + e);
                }
        }
        if (bad) {
            #pragma unroll
            for (int k = 0; k < kDeep; ++k)
                #pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (uint32_t(id[k][e]) >= uint32_t(vocab) && !(pads >> (4 * k + e) & 1)) *bad = true;
        }
        #pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            if (i + 128 * k >= end) break;
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (pads >> (4 * k + e) & 1) id[k][e] = -1;
            f(int(i + 128 * k) + lane * 4, id[k]);
        }
    }
}

// How many of a section's tokens each of the rows v0 .. v0 + n - 1 has: added to
// mine, which is this warp's.
__device__ __forceinline__ void count_rows(const int (&id)[4], int v0, int n, int* mine) {
    #pragma unroll
    for (int e = 0; e < 4; ++e)
        if (uint32_t(id[e]) - uint32_t(v0) < uint32_t(n)) atomicAdd(&mine[id[e] - v0], 1);
}

// Calls put(place, token, row) for the tokens of these rows; mine: each row's
// next place, advanced.  The order within 128 tokens is that of (token mod 4, token).
template <typename Put>
__device__ __forceinline__ void place_rows(int token, const int (&id)[4], int v0, int n, int* mine, Put&& put) {
    const int lane = threadIdx.x & 31;
    bool any = false;
    #pragma unroll
    for (int e = 0; e < 4; ++e) any |= uint32_t(id[e]) - uint32_t(v0) < uint32_t(n);
    if (!__ballot_sync(~0u, any)) return;
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int r = int(uint32_t(id[e]) - uint32_t(v0));
        const bool in = uint32_t(r) < uint32_t(n);
        const uint32_t m = __ballot_sync(~0u, in);
        if (m == 0) continue;
        if (in) {
            const uint32_t peers = __match_any_sync(m, r);
            const int first = mine[r], rank = __popc(peers & ((1u << lane) - 1u));
            put(first + rank, token + e, r);
            __syncwarp(m);
            if (rank == 0) mine[r] = first + __popc(peers);
        }
        __syncwarp();
    }
}

__global__ void __launch_bounds__(1024) k_embed_sort(const int32_t* __restrict__ ids,
                                                             const uint8_t* __restrict__ pad, int64_t n_tokens,
                                                             int vocab, int range, EmbHeader* __restrict__ hdr,
                                                             int32_t* __restrict__ row_start,
                                                             int32_t* __restrict__ order, int32_t* __restrict__ sid,
                                                             int wide) {
    extern __shared__ int cnt[];       // [warps][range]: counts, then next places
    __shared__ int s_warp[32];
    __shared__ int s_below;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    const int v0 = blockIdx.x * range;
    const int n = min(range, vocab - v0);
    for (int k = tid; k < warps * range / 4; k += threads) reinterpret_cast<int4*>(cnt)[k] = make_int4(0, 0, 0, 0);
    if (tid == 0) s_below = 0;
    __syncthreads();
    pdl_wait();
    const int64_t per = ((n_tokens + warps - 1) / warps + 127) / 128 * 128;
    const int64_t beg = warp * per < n_tokens ? warp * per : n_tokens;
    const int64_t end = beg + per < n_tokens ? beg + per : n_tokens;
    int* mine = cnt + warp * range;

    int below = 0;
    bool bad = false;
    for_section<4>(ids, pad, beg, end, wide, vocab, blockIdx.x == 0 ? &bad : nullptr, [&](int, const int (&id)[4]) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) below += uint32_t(id[e]) < uint32_t(v0);
        count_rows(id, v0, n, mine);
    });
    below = __reduce_add_sync(~0u, below);
    if (lane == 0 && below) atomicAdd(&s_below, below);
    const int any_bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && tid == 0) hdr->status = any_bad ? DLM_DEV_BAD_TOKEN_ID : 0u;

    // exclusive scan over the range's rows, a row per thread and round
    int carry = s_below;
    for (int r0 = 0; r0 < n; r0 += threads) {
        const int r = r0 + tid;
        int tot = 0;
        if (r < n) {
            #pragma unroll 16
            for (int w = 0; w < warps; ++w) tot += cnt[w * range + r];
        }
        int at = tot;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(~0u, at, o);
            if (lane >= o) at += t;
        }
        if (lane == 31) s_warp[warp] = at;
        __syncthreads();
        const int mine_before = lane < warp ? s_warp[lane] : 0, all = lane < warps ? s_warp[lane] : 0;
        at += carry + __reduce_add_sync(~0u, mine_before) - tot;
        carry += __reduce_add_sync(~0u, all);
        if (r < n) {
            row_start[v0 + r] = at;
            #pragma unroll 16
            for (int w = 0; w < warps; ++w) {
                const int c = cnt[w * range + r];
                cnt[w * range + r] = at;
                at += c;
            }
            if (v0 + r == vocab - 1) row_start[vocab] = at;
        }
        __syncthreads();
    }

    for_section<4>(ids, pad, beg, end, wide, vocab, nullptr, [&](int token, const int (&id)[4]) {
        place_rows(token, id, v0, n, mine, [&](int at, int i, int r) {
            order[at] = i;
            sid[at] = v0 + r;
        });
    });
}

// ---------------------------------------------------------------------------
// gradient: sums over sorted positions, zero rows
// ---------------------------------------------------------------------------
__device__ __forceinline__ float grad_value(float v) { return v; }
__device__ __forceinline__ float grad_value(uint16_t v) { return bf16_bits_to_float(v); }
__device__ __forceinline__ void put_grad_value(float* dst, float v) { *dst = v; }
__device__ __forceinline__ void put_grad_value(uint16_t* dst, float v) {
    *dst = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// What 8 elements of a gradient on a 16-byte border held (zeros where it is not
// added to), and the same with scale * acc added, stored.
template <typename GT> constexpr int kOldWords = sizeof(GT) / 2;      // of 16 bytes
template <typename GT>
__device__ __forceinline__ void load_old(const GT* src, bool there, uint4 (&old)[kOldWords<GT>]) {
    #pragma unroll
    for (int h = 0; h < kOldWords<GT>; ++h) {
        old[h] = make_uint4(0, 0, 0, 0);
        if (there)
            asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(old[h].x), "=r"(old[h].y), "=r"(old[h].z), "=r"(old[h].w)
                         : "l"(reinterpret_cast<const uint4*>(src) + h) : "memory");
    }
}
__device__ __forceinline__ void put8(float* dst, const float (&acc)[8], float scale, const uint4 (&old)[2]) {
    #pragma unroll
    for (int h = 0; h < 2; ++h)
        reinterpret_cast<float4*>(dst)[h] =
            make_float4(__uint_as_float(old[h].x) + scale * acc[4 * h], __uint_as_float(old[h].y) + scale * acc[4 * h + 1],
                        __uint_as_float(old[h].z) + scale * acc[4 * h + 2], __uint_as_float(old[h].w) + scale * acc[4 * h + 3]);
}
__device__ __forceinline__ void put8(uint16_t* dst, const float (&acc)[8], float scale, const uint4 (&old)[1]) {
    uint32_t x[4] = {old[0].x, old[0].y, old[0].z, old[0].w};
    #pragma unroll
    for (int k = 0; k < 4; ++k)
        x[k] = pack_bf16x2(bf16lo(x[k]) + scale * acc[2 * k], bf16hi(x[k]) + scale * acc[2 * k + 1]);
    *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
}

template <int kVec, typename GT>
__device__ __forceinline__ void put_row(GT* __restrict__ dst, const float (&acc)[kVec], float scale, bool accumulate) {
    if constexpr (kVec == 8) {
        uint4 old[kOldWords<GT>];
        load_old(dst, accumulate, old);
        put8(dst, acc, scale, old);
    } else {
        put_grad_value(dst, (accumulate ? grad_value(*dst) : 0.f) + scale * acc[0]);
    }
}

// Loads a piece of a row, whatever becomes of it (volatile: the compiler would
// move it down to its use, and with it the wait).
template <int kVec>
__device__ __forceinline__ uint4 load_piece(const uint16_t* p) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if constexpr (kVec == 8) {
        asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p));
    } else {
        uint16_t v;
        asm volatile("ld.global.nc.b16 %0, [%1];" : "=h"(v) : "l"(p));
        q.x = uint32_t(v) << 16;
    }
    return q;
}

// Adds a piece of a row: 8 bf16, or the fp32 pattern of one in x.
template <int kVec>
__device__ __forceinline__ void add_piece(uint4 q, float (&acc)[kVec]) {
    if constexpr (kVec == 8) {
        const uint32_t x[4] = {q.x, q.y, q.z, q.w};
        #pragma unroll
        for (int k = 0; k < 4; ++k) { acc[2 * k] += bf16lo(x[k]); acc[2 * k + 1] += bf16hi(x[k]); }
    } else {
        acc[0] += __uint_as_float(q.x);
    }
}

struct EmbGradArgs {
    const uint16_t* d_out;
    int64_t ld;
    int vocab, d;
    float scale;
    int accumulate;
    void* d_weight;
    int64_t ld_dw;
    const int32_t* row_start;
    const int32_t* order;
    const int32_t* sid;
    float* part;          // [chunks][2][pitch]: 0 = rows begun before the chunk, 1 = the row that goes on behind it
    int pitch;
    int chunk;            // sorted positions per CTA of k_embed_grad
    int tiles;            // column tiles of a row in k_embed_grad
    int64_t n_tokens;
    int64_t chunk_ctas;   // k_embed_grad's CTAs that add up; those behind them write zeros
    int64_t join_ctas;    // the same for k_embed_join: groups of 32 chunks x join_tiles
    int join_tiles;
    int zero_rows;        // rows of a zero-writing warp
    int zero_split;       // rows below it are zeroed in k_embed_grad, the others in k_embed_join
};

// Zeros for the rows without a token, by CTA `cta` of those that write them;
// rows [first, last).  A warp takes kZeroBytes of the table, up to 32 rows,
// with 16-byte stores between a row's first and last 16-byte border and single
// elements outside.  (Many short CTAs that sweep over the table: one persistent
// CTA per SM wrote 1 GB in 170 us instead of 139, by plain and by bulk stores.)
constexpr int kZeroBytes = 16384;

template <typename GT>
__device__ __forceinline__ void zero_rows(const EmbGradArgs& a, int64_t cta, int first, int last) {
    constexpr int kPer = 16 / int(sizeof(GT));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t r0 = first + (cta * warps + warp) * a.zero_rows, r = r0 + lane;
    const bool empty = lane < a.zero_rows && r < last && a.row_start[r] == a.row_start[r + 1];
    uint32_t m = __ballot_sync(~0u, empty);
    while (m) {
        // neighbouring rows without a gap between them are one stretch
        const int s = __ffs(m) - 1, run = a.ld_dw == a.d ? __ffs(~(m >> s)) - 1 : 1;
        const int len = run < 0 ? 32 : run;             // all 32 rows
        m &= ~((len == 32 ? ~0u : (1u << len) - 1u) << s);
        GT* dst = static_cast<GT*>(a.d_weight) + (r0 + s) * a.ld_dw;
        const int n = len * a.d;
        const int head = min(n, int(((16u - unsigned(reinterpret_cast<uintptr_t>(dst) & 15u)) & 15u) / sizeof(GT)));
        const int nv = (n - head) / kPer, rest = n - head - nv * kPer;
        uint4* mid = reinterpret_cast<uint4*>(dst + head);
        #pragma unroll 8
        for (int v = lane; v < nv; v += 32) mid[v] = make_uint4(0, 0, 0, 0);
        if (lane < head + rest) dst[lane < head ? lane : n - rest + (lane - head)] = GT(0);
    }
}

// kAligned: rows of d_out and d_weight on 16-byte borders.  Otherwise d_out is
// read as dlm_shift.cuh does, and a finished row is written by single elements
// side by side, through a warp's 1 KB of shared memory.
// kAdd: added to what d_weight holds, which is read ahead with the rows
// (16,384 x 4,096, half of them masked: 65 -> 60 us; with 8 rows in flight
// instead of 4, on 112 registers instead of 72, again 65).
template <bool kAligned, bool kAdd, typename GT>
__global__ void __launch_bounds__(kGradThreads) k_embed_grad(EmbGradArgs a) {
    constexpr int kU = kAligned && !kAdd ? 8 : 4;       // rows in flight
    extern __shared__ float s_rows[];          // not kAligned: [warp][256]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    if (int64_t(blockIdx.x) >= a.chunk_ctas) {
        zero_rows<GT>(a, int64_t(blockIdx.x) - a.chunk_ctas, 0, a.zero_split);
        return;
    }
    GT* dw = static_cast<GT*>(a.d_weight);
    const int64_t c = blockIdx.x / a.tiles;
    const int col = (int(blockIdx.x - c * a.tiles) * blockDim.x + threadIdx.x) * 8;
    const bool active = col < a.d;
    const int64_t p0 = c * a.chunk;
    const int64_t total = a.row_start[a.vocab];
    const int n = int(min(int64_t(a.chunk), total - p0));
    if (n <= 0) return;
    const int tok = lane < n ? a.order[p0 + lane] : 0;
    const int row = lane < n ? a.sid[p0 + lane] : -1;
    const int before = p0 > 0 ? a.sid[p0 - 1] : -1;
    const int after = p0 + n < total ? a.sid[p0 + n] : -1;
    bool open = before == __shfl_sync(~0u, row, 0);      // the current row began before this chunk
    float acc[8];
    #pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    float* part = a.part + (c * 2) * int64_t(a.pitch) + col;
    const uint16_t* column = a.d_out + (kAligned && !active ? 0 : col);
    const uint16_t* end = a.d_out + (a.n_tokens - 1) * a.ld + a.d;
    for (int p = 0; p < n; p += kU) {
        uint4 q[kU], more[kU];                 // more: the chunk behind the last lane's
        uint4 old[kAligned && kAdd ? kU : 1][kOldWords<GT>];
        int sh[kU];
        #pragma unroll
        for (int u = 0; u < kU; ++u) {
            const uint16_t* at = column + __shfl_sync(~0u, tok, min(p + u, n - 1)) * a.ld;
            if constexpr (kAligned) {
                q[u] = load_piece<8>(at);
                if constexpr (kAdd) {          // a row that ends here and is written by this thread
                    const int id = __shfl_sync(~0u, row, (p + u) & 31), nx = __shfl_sync(~0u, row, (p + u + 1) & 31);
                    const bool ends = p + u < n && id != (p + u + 1 == n ? after : nx) && id != before;
                    load_old(dw + int64_t(ends ? id : 0) * a.ld_dw + col, ends && active, old[u]);
                }
            } else {
                sh[u] = int(reinterpret_cast<uintptr_t>(at) & 15) / 2;
                q[u] = col - sh[u] < a.d ? load_chunk(at - sh[u], a.d_out, end) : make_uint4(0, 0, 0, 0);
                more[u] = make_uint4(0, 0, 0, 0);
                if (lane == 31 && sh[u] && col + 8 - sh[u] < a.d) more[u] = load_chunk(at + 8 - sh[u], a.d_out, end);
            }
        }
        #pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (p + u >= n) break;
            if (!kAligned && sh[u]) {
                const uint4 next = shfl(q[u], (lane + 1) & 31);
                q[u] = funnel16(q[u], lane == 31 ? more[u] : next, sh[u]);
            }
            add_piece<8>(q[u], acc);
            const int id = __shfl_sync(~0u, row, p + u);
            const int nx = __shfl_sync(~0u, row, (p + u + 1) & 31);
            const bool last = p + u + 1 == n;
            const int next = last ? after : nx;
            if (id != next || last) {
                if (open || id == next) {                // crosses a border: fp32 partial
                    float* dst = part + (open ? 0 : a.pitch);
                    #pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (kAligned ? active : col + k < a.d) dst[k] = acc[k];
                } else if constexpr (kAligned) {
                    GT* dst = dw + int64_t(id) * a.ld_dw + col;
                    if constexpr (kAdd) {
                        if (active) put8(dst, acc, a.scale, old[u]);
                    } else {
                        if (active) put_row<8, GT>(dst, acc, a.scale, false);
                    }
                } else {
                    __syncwarp();
                    #pragma unroll
                    for (int k = 0; k < 8; ++k) s_rows[warp * 256 + lane * 8 + k] = acc[k];
                    __syncwarp();
                    GT* dst = dw + int64_t(id) * a.ld_dw + col - lane * 8;
                    const int left = a.d - (col - lane * 8);
                    float o[8];
                    #pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[k] = kAdd && lane + 32 * k < left ? grad_value(dst[lane + 32 * k]) : 0.f;
                    #pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (lane + 32 * k < left)
                            put_grad_value(dst + lane + 32 * k, o[k] + a.scale * s_rows[warp * 256 + lane + 32 * k]);
                }
                open = false;
                #pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = 0.f;
            }
        }
    }
}

// Adds up the rows that cross chunk borders: a CTA looks at 32 chunks (one
// per lane) for rows that begin in them and end behind them, 128 columns at a
// time.  A row of up to kFewChunks chunks is a single warp's; of a longer one the
// warps take consecutive parts of its chunks, whose sums are added in that order.
// (All rows the second way, one after the other: 4,096 tokens drawn as words are,
// the r-th most frequent with a share of 1 / r, 43 us instead of 28.)
constexpr int kJoinCols = 128;
constexpr int kFewChunks = 8;

template <typename GT>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) k_embed_join(EmbGradArgs a) {
    __shared__ float4 s[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    if (int64_t(blockIdx.x) >= a.join_ctas) {
        zero_rows<GT>(a, int64_t(blockIdx.x) - a.join_ctas, a.zero_split, a.vocab);
        return;
    }
    GT* dw = static_cast<GT*>(a.d_weight);
    const int64_t c0 = int64_t(blockIdx.x) / a.join_tiles * 32, n_tokens = a.n_tokens;
    const int tile = int(blockIdx.x % a.join_tiles), col = tile * kJoinCols + lane * 4;
    const int64_t total = a.row_start[a.vocab];
    {
        int last = 0, row = -1;
        const int64_t behind = (c0 + lane + 1) * a.chunk;
        if (behind < n_tokens) {
            // read before `total` is known; meaningless behind it, and then not used as an index
            const int v = a.sid[behind - 1], w = a.sid[behind];
            if (behind < total && v == w && a.row_start[v] >= behind - a.chunk) {
                row = v;
                last = (a.row_start[v + 1] - 1) / a.chunk;
            }
        }
        // a row of few chunks is a warp's alone
        const uint32_t few = __ballot_sync(~0u, row >= 0 && last - (c0 + lane) < kFewChunks);
        int turn = 0;
        for (uint32_t q = few; q; q &= q - 1, ++turn) {
            if (turn % kJoinWarps != warp) continue;
            const int src = __ffs(q) - 1;
            const int v = __shfl_sync(~0u, row, src);
            const int64_t f = c0 + src;
            const int cnt = int(__shfl_sync(~0u, last, src) - f) + 1;
            if (col >= a.pitch) continue;
            float4 x[kFewChunks];
            #pragma unroll
            for (int k = 0; k < kFewChunks; ++k)
                x[k] = k < cnt ? *reinterpret_cast<const float4*>(a.part + ((f + k) * 2 + (k == 0)) * int64_t(a.pitch) + col)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            #pragma unroll
            for (int k = 0; k < kFewChunks; ++k) { t[0] += x[k].x; t[1] += x[k].y; t[2] += x[k].z; t[3] += x[k].w; }
            GT* dst = dw + int64_t(v) * a.ld_dw + col;
            float old[4] = {0.f, 0.f, 0.f, 0.f};
            if (a.accumulate) {
                #pragma unroll
                for (int e = 0; e < 4; ++e) old[e] = col + e < a.d ? grad_value(dst[e]) : 0.f;
            }
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < a.d) put_grad_value(dst + e, old[e] + a.scale * t[e]);
        }
        uint32_t m = __ballot_sync(~0u, row >= 0) & ~few;
        while (m) {
            const int src = __ffs(m) - 1;
            m &= m - 1;
            const int v = __shfl_sync(~0u, row, src);
            const int64_t f = c0 + src;
            const int cnt = int(__shfl_sync(~0u, last, src) - f) + 1;
            const int per = (cnt + kJoinWarps - 1) / kJoinWarps;
            const int k0 = min(cnt, warp * per), k1 = min(cnt, k0 + per);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (col < a.pitch) {
                constexpr int kU = 8;      // loads in flight
                for (int k = k0; k < k1; k += kU) {
                    float4 x[kU];
                    #pragma unroll
                    for (int u = 0; u < kU; ++u)
                        x[u] = k + u < k1 ? *reinterpret_cast<const float4*>(
                                                a.part + ((f + k + u) * 2 + (k + u == 0)) * int64_t(a.pitch) + col)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                    #pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        acc.x += x[u].x; acc.y += x[u].y; acc.z += x[u].z; acc.w += x[u].w;
                    }
                }
            }
            s[warp][lane] = acc;
            __syncthreads();
            const int c = tile * kJoinCols + threadIdx.x;
            if (threadIdx.x < kJoinCols && c < a.d) {
                float t[1] = {0.f};
                #pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) t[0] += reinterpret_cast<const float*>(s[w])[threadIdx.x];
                put_row<1, GT>(dw + int64_t(v) * a.ld_dw + c, t, a.scale, a.accumulate);
            }
            __syncthreads();
        }
    }
}

// Few tokens (at most kSmallTokens): one launch.  A CTA owns 32 rows of the
// table and 256 columns.  It zeroes them, reads all ids, sorts those of its
// rows in shared memory as k_embed_sort does, and its warps add up equal parts
// of that list; the rows that cross from one warp's part into the next are
// joined through shared memory.
//
// Measured (us), this kernel / the three above: 128 tokens on a table of 0.5 MB
// 4.7 / 12.2, 512 on 1 MB 7.4 / 13.1; 512 on 65 MB 28.2 / 20.8, 64 on 1 GB
// 182 / 161: its many small CTAs write a large table more slowly.
constexpr int kSmallTokens = 1024;
constexpr int64_t kSmallBytes = 16 << 20;
constexpr int kSmallWarps = 8;

struct EmbSmallArgs {
    const int32_t* ids;
    const uint8_t* pad;
    int n_tokens;
    const uint16_t* d_out;
    int64_t ld;
    int vocab, d;
    float scale;
    int accumulate;
    void* d_weight;
    int64_t ld_dw;
    EmbHeader* hdr;
    int tiles;            // column tiles of a row
    int wide;             // ids on a 16-byte border
};

template <int kVec, typename GT>
__global__ void __launch_bounds__(kSmallWarps * 32) k_embed_small(EmbSmallArgs a) {
    constexpr int kU = 8;              // rows of d_out in flight
    constexpr int kCols = 8 / kVec;    // pieces of kVec columns a lane, 32 * kVec apart
    __shared__ int s_place[kSmallWarps][32];             // tokens of a warp's section and a row; then their places
    __shared__ int s_count;
    __shared__ uint16_t s_tok[kSmallTokens];
    __shared__ int8_t s_row[kSmallTokens];
    __shared__ float s_part[kSmallWarps][2][256];
    __shared__ int s_edge[kSmallWarps][2];               // the row of each part, or -1
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = int64_t(blockIdx.x) / a.tiles * 32;
    const int tile0 = int(blockIdx.x % unsigned(a.tiles)) * 256, c0 = tile0 + lane * kVec;
    const int v0 = int(r0), n = min(32, a.vocab - v0);
    s_place[warp][lane] = 0;
    if (lane < 2) s_edge[warp][lane] = -1;
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();
    GT* dw = static_cast<GT*>(a.d_weight) + r0 * a.ld_dw + c0;
    if (!a.accumulate) {
        const float none[kVec] = {};
        for (int r = warp; r < n; r += kSmallWarps)
            #pragma unroll
            for (int k = 0; k < kCols; ++k)
                if (c0 + 32 * kVec * k < a.d) put_row<kVec, GT>(dw + r * a.ld_dw + 32 * kVec * k, none, 0.f, false);
    }
    const int per = ((a.n_tokens + kSmallWarps - 1) / kSmallWarps + 127) / 128 * 128;
    const int beg = min(a.n_tokens, warp * per), end = min(a.n_tokens, beg + per);
    int* mine = s_place[warp];
    bool bad = false, any = false;
    for_section<1>(a.ids, a.pad, beg, end, a.wide, a.vocab, blockIdx.x == 0 ? &bad : nullptr,
                   [&](int, const int (&id)[4]) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) any |= uint32_t(id[e]) - uint32_t(v0) < uint32_t(n);
        count_rows(id, v0, n, mine);
    });
    any = __any_sync(~0u, any);
    if (blockIdx.x == 0) {
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) a.hdr->status = bad ? DLM_DEV_BAD_TOKEN_ID : 0u;
    }
    if (!__syncthreads_or(any)) return;
    if (warp == 0) {
        int tot = 0;
        #pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) tot += s_place[w][lane];
        int at = tot;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(~0u, at, o);
            if (lane >= o) at += t;
        }
        if (lane == 31) s_count = at;
        at -= tot;
        #pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) {
            const int c = s_place[w][lane];
            s_place[w][lane] = at;
            at += c;
        }
    }
    __syncthreads();
    if (any)
        for_section<1>(a.ids, a.pad, beg, end, a.wide, a.vocab, nullptr, [&](int token, const int (&id)[4]) {
            place_rows(token, id, v0, n, mine, [&](int at, int i, int r) {
                s_tok[at] = uint16_t(i);
                s_row[at] = int8_t(r);
            });
        });
    __syncthreads();
    const int count = s_count, part = (count + kSmallWarps - 1) / kSmallWarps;
    const int p0 = min(count, warp * part), p1 = min(count, p0 + part);
    bool open = p0 > 0 && p0 < p1 && s_row[p0 - 1] == s_row[p0];
    float acc[kCols][kVec];
    #pragma unroll
    for (int k = 0; k < kCols; ++k)
        #pragma unroll
        for (int e = 0; e < kVec; ++e) acc[k][e] = 0.f;
    for (int p = p0; p < p1; p += kU) {
        uint4 q[kU][kCols];
        #pragma unroll
        for (int u = 0; u < kU; ++u) {
            const uint16_t* src = a.d_out + int64_t(s_tok[min(p + u, p1 - 1)]) * a.ld;
            #pragma unroll
            for (int k = 0; k < kCols; ++k)
                q[u][k] = load_piece<kVec>(src + (c0 + 32 * kVec * k < a.d ? c0 + 32 * kVec * k : 0));
        }
        #pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (p + u >= p1) break;
            const int r = s_row[p + u], next = p + u + 1 < count ? s_row[p + u + 1] : -1;
            #pragma unroll
            for (int k = 0; k < kCols; ++k) add_piece<kVec>(q[u][k], acc[k]);
            const bool last = p + u + 1 == p1;
            if (r != next || last) {
                if (open || r == next) {
                    #pragma unroll
                    for (int k = 0; k < kCols; ++k)
                        #pragma unroll
                        for (int e = 0; e < kVec; ++e)
                            s_part[warp][open ? 0 : 1][lane * kVec + 32 * kVec * k + e] = acc[k][e];
                    if (lane == 0) s_edge[warp][open ? 0 : 1] = r;
                } else {
                    #pragma unroll
                    for (int k = 0; k < kCols; ++k)
                        if (c0 + 32 * kVec * k < a.d)
                            put_row<kVec, GT>(dw + r * a.ld_dw + 32 * kVec * k, acc[k], a.scale, a.accumulate);
                }
                #pragma unroll
                for (int k = 0; k < kCols; ++k)
                    #pragma unroll
                    for (int e = 0; e < kVec; ++e) acc[k][e] = 0.f;
                open = false;
            }
        }
    }
    __syncthreads();
    const int c = threadIdx.x;
    if (tile0 + c >= a.d) return;
    for (int w = 0; w < kSmallWarps; ++w) {
        const int r = s_edge[w][1];
        if (r < 0) continue;
        float sum[1] = {s_part[w][1][c]};
        for (int v = w + 1; v < kSmallWarps && s_edge[v][0] == r; ++v) sum[0] += s_part[v][0][c];
        put_row<1, GT>(static_cast<GT*>(a.d_weight) + (r0 + r) * a.ld_dw + tile0 + c, sum, a.scale, a.accumulate);
    }
}

// Workspace of the gradient: header, row_start [vocab + 1], order and sid
// [n_tokens], partials; and the CTAs of its launches, but for those that write zeros.
struct EmbPlan {
    int chunk;
    int64_t chunks;
    int pitch;
    size_t off_start, off_order, off_sid, off_part, bytes;
    unsigned threads;     // of a CTA of k_embed_grad
    int tiles, join_tiles, zero_split;
    int64_t join_ctas, small_ctas;
};

// The CTAs that write zeros, by the bytes of a row of the gradient.
struct EmbZeros { int rows; int64_t grad, join; };

static EmbZeros embed_zeros(const EmbPlan& p, int32_t vocab, int64_t row_bytes) {
    EmbZeros z;
    z.rows = row_bytes >= kZeroBytes ? 1 : row_bytes * 32 <= kZeroBytes ? 32 : int(kZeroBytes / row_bytes);
    const int64_t per_grad = z.rows * int64_t(p.threads / 32), per_join = z.rows * int64_t(kJoinWarps);
    z.grad = (p.zero_split + per_grad - 1) / per_grad;
    z.join = (vocab - p.zero_split + per_join - 1) / per_join;
    return z;
}

static bool embed_plan(const dlm_layout_t* L, int32_t vocab, int32_t d, EmbPlan* p) {
    if (!layout_ok(L) || vocab < 1 || d < 1 || vocab == INT32_MAX || d > INT32_MAX - 1024) return false;
    p->chunk = kMaxChunk;
    while (p->chunk > kMinChunk && L->n_tokens / p->chunk * ((int64_t(d) + 255) / 256) < 148 * 16) p->chunk /= 2;
    p->chunks = (L->n_tokens + p->chunk - 1) / p->chunk;
    p->pitch = int(align_up(size_t(d), 32));
    p->off_start = kWsAlign;
    p->off_order = align_up(p->off_start + (size_t(vocab) + 1) * 4, kWsAlign);
    p->off_sid = align_up(p->off_order + size_t(L->n_tokens) * 4, kWsAlign);
    p->off_part = align_up(p->off_sid + size_t(L->n_tokens) * 4, kWsAlign);
    p->bytes = align_up(p->off_part + size_t(p->chunks) * 2 * size_t(p->pitch) * 4, kWsAlign);
    const int nv = (d + 7) / 8;
    p->threads = nv >= kGradThreads ? kGradThreads : unsigned(align_up(size_t(nv), 32));
    p->tiles = int((unsigned(nv) + p->threads - 1) / p->threads);
    p->join_tiles = (d + kJoinCols - 1) / kJoinCols;
    p->join_ctas = p->chunks > 1 ? (p->chunks + 31) / 32 * p->join_tiles : 0;
    p->small_ctas = (int64_t(vocab) + 31) / 32 * ((d + 255) / 256);
    // half of the table's zeros are written beside the sums, half beside the joins:
    // both wait on memory more than they use it
    p->zero_split = p->join_ctas == 0 ? vocab : vocab / 2;
    // blocks that a launch can have, with the zeros of the wider type
    const EmbZeros z = embed_zeros(*p, vocab, int64_t(d) * 4);
    return p->chunks * p->tiles + z.grad <= INT32_MAX && p->join_ctas + z.join <= INT32_MAX && p->small_ctas <= INT32_MAX;
}

}  // namespace dlm

using namespace dlm;

extern "C" dlm_status_t dlm_embed_fwd(const dlm_layout_t* layout, const int32_t* ids, const uint16_t* weight,
                                      int64_t ld_weight, int32_t vocab, int32_t d_model, float scale, uint16_t* out,
                                      int64_t ld_out, uint32_t* dev_status, dlm_stream_t stream) {
    DLM_NVTX("dlm_embed_fwd");
    if (!layout_ok(layout) || vocab < 1 || d_model < 1 || d_model > INT32_MAX - 1024 || ld_weight < d_model || ld_out < d_model)
        return DLM_ERR_INVALID_ARGUMENT;
    if (!(scale - scale == 0.0f)) return DLM_ERR_INVALID_ARGUMENT;       // inf or NaN
    if (layout->n_tokens == 0) return DLM_OK;
    if (!ids || !weight || !out) return DLM_ERR_INVALID_ARGUMENT;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    const bool vec = d_model % 8 == 0 && ld_weight % 8 == 0 && ld_out % 8 == 0 && aligned16(weight) && aligned16(out);
    const int64_t items = layout->n_tokens * ((d_model + 1023) / 1024);
    int64_t blocks = (items + kEmbThreads / 32 - 1) / (kEmbThreads / 32);
    if (blocks > (1 << 20)) blocks = 1 << 20;
    return launch_pdl(vec ? k_embed_fwd<true> : k_embed_fwd<false>, dim3(unsigned(blocks)), dim3(kEmbThreads), 0,
                      (cudaStream_t)stream, "k_embed_fwd launch", ids, layout->pad_mask, layout->n_tokens, weight,
                      ld_weight, vocab, d_model, scale, out, ld_out, dev_status);
}

extern "C" size_t dlm_embed_bwd_workspace_size(const dlm_layout_t* layout, int32_t d_model, int32_t vocab) {
    EmbPlan p;
    return embed_plan(layout, vocab, d_model, &p) ? p.bytes : 0;
}

extern "C" dlm_status_t dlm_embed_bwd(const dlm_layout_t* layout, const int32_t* ids, const uint16_t* d_out,
                                      int64_t ld, int32_t vocab, int32_t d_model, float scale, int32_t grad_dtype,
                                      int32_t accumulate, void* d_weight, int64_t ld_dw, void* workspace,
                                      size_t workspace_bytes, dlm_stream_t stream) {
    DLM_NVTX("dlm_embed_bwd");
    EmbPlan p;
    if (!embed_plan(layout, vocab, d_model, &p)) return DLM_ERR_INVALID_ARGUMENT;
    if (ld < d_model || ld_dw < d_model || !(scale - scale == 0.0f)) return DLM_ERR_INVALID_ARGUMENT;
    if ((grad_dtype != DLM_BF16 && grad_dtype != DLM_F32) || (accumulate != 0 && accumulate != 1))
        return DLM_ERR_INVALID_ARGUMENT;
    if (layout->n_tokens > 0 && (!ids || !d_out)) return DLM_ERR_INVALID_ARGUMENT;
    if (!d_weight || !workspace || reinterpret_cast<uintptr_t>(workspace) % kWsAlign) return DLM_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < p.bytes) return DLM_ERR_WORKSPACE_TOO_SMALL;
    const bool f32 = grad_dtype == DLM_F32;
    const bool vec = d_model % 8 == 0 && ld % 8 == 0 && ld_dw % 8 == 0 && aligned16(d_out) && aligned16(d_weight);
    const EmbZeros zeros = embed_zeros(p, vocab, int64_t(d_model) * (f32 ? 4 : 2));
    const int64_t zero_grad = accumulate ? 0 : zeros.grad, zero_join = accumulate ? 0 : zeros.join;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    EmbHeader* hdr = reinterpret_cast<EmbHeader*>(ws);
    int32_t* row_start = reinterpret_cast<int32_t*>(ws + p.off_start);
    int32_t* order = reinterpret_cast<int32_t*>(ws + p.off_order);
    int32_t* sid = reinterpret_cast<int32_t*>(ws + p.off_sid);

    if (layout->n_tokens <= kSmallTokens && int64_t(vocab) * d_model * (f32 ? 4 : 2) <= kSmallBytes) {
        EmbSmallArgs b = {ids, layout->pad_mask, int(layout->n_tokens), d_out, ld, vocab, d_model, scale, accumulate,
                          d_weight, ld_dw, hdr, (d_model + 255) / 256, int(aligned16(ids))};
        auto kern = f32 ? (vec ? k_embed_small<8, float> : k_embed_small<1, float>)
                        : (vec ? k_embed_small<8, uint16_t> : k_embed_small<1, uint16_t>);
        return launch_pdl(kern, dim3(unsigned(p.small_ctas)), dim3(kSmallWarps * 32), 0, s, "k_embed_small launch", b);
    }
    // a range of vocabulary rows per SM, as far as the counters fit
    int range = int(align_up((size_t(vocab) + 147) / 148, 32));
    if (range > kMaxRange) range = kMaxRange;
    const int warps = range <= kMaxRange / 2 ? 32 : 16;
    if ((st = allow_smem<k_embed_sort, int(kSortSmem)>("k_embed_sort attributes")) != DLM_OK) return st;
    st = launch_pdl(k_embed_sort, dim3(unsigned((int64_t(vocab) + range - 1) / range)), dim3(unsigned(warps * 32)),
                    size_t(warps) * range * 4, s, "k_embed_sort launch", ids, layout->pad_mask, layout->n_tokens, vocab,
                    range, hdr, row_start, order, sid, int(aligned16(ids)));
    if (st != DLM_OK) return st;

    EmbGradArgs a;
    a.d_out = d_out; a.ld = ld; a.vocab = vocab; a.d = d_model; a.scale = scale; a.accumulate = accumulate;
    a.d_weight = d_weight; a.ld_dw = ld_dw; a.row_start = row_start; a.order = order; a.sid = sid;
    a.part = reinterpret_cast<float*>(ws + p.off_part);
    a.pitch = p.pitch; a.chunk = p.chunk; a.tiles = p.tiles; a.n_tokens = layout->n_tokens; a.chunk_ctas = p.chunks * p.tiles;
    a.join_ctas = p.join_ctas; a.join_tiles = p.join_tiles; a.zero_rows = zeros.rows; a.zero_split = p.zero_split;
    if (a.chunk_ctas + zero_grad > 0) {
        auto kern = f32 ? (vec ? (accumulate ? k_embed_grad<true, true, float> : k_embed_grad<true, false, float>)
                               : (accumulate ? k_embed_grad<false, true, float> : k_embed_grad<false, false, float>))
                        : (vec ? (accumulate ? k_embed_grad<true, true, uint16_t> : k_embed_grad<true, false, uint16_t>)
                               : (accumulate ? k_embed_grad<false, true, uint16_t> : k_embed_grad<false, false, uint16_t>));
        st = launch_pdl(kern, dim3(unsigned(a.chunk_ctas + zero_grad)), dim3(p.threads), vec ? 0 : p.threads * 8 * sizeof(float),
                        s, "k_embed_grad launch", a);
        if (st != DLM_OK) return st;
    }
    if (p.join_ctas == 0) return DLM_OK;
    return launch_pdl(f32 ? k_embed_join<float> : k_embed_join<uint16_t>, dim3(unsigned(p.join_ctas + zero_join)),
                      dim3(kJoinWarps * 32), 0, s, "k_embed_join launch", a);
}
