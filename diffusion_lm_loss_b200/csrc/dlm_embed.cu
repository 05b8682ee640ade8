// dlm_embed.cu -- token embedding with a scale, and its gradient.
//
// Forward: out[i, :] = bf16(scale * W[id_i, :]), one warp per 128 vectors of
// a token's row.
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
//                  the ids alone.
//   k_embed_grad   one CTA per kChunk sorted positions and column tile adds
//                  rows in that order, in fp32 registers; a row that begins
//                  and ends inside the chunk is written at once, a row that
//                  crosses a chunk's border leaves one fp32 partial per chunk.
//                  More CTAs of the same launch write the zero rows.
//   k_embed_join   adds the partials of the crossing rows, in chunk order.
// Nothing is added atomically: results are bitwise reproducible.
#include <type_traits>

#include "dlm_device.cuh"
#include "dlm_host.h"

namespace dlm {

constexpr int kEmbThreads = 256;
constexpr int kChunk = 32;             // sorted positions per CTA: one per lane
constexpr int kSortWarps = 16;
constexpr int kSortThreads = kSortWarps * 32;
constexpr int kMaxRange = 1792;        // vocabulary rows per sorting CTA: 16 x 1,792 counters fill 112 KB
constexpr int kZeroRows = 32;          // vocabulary rows per zero-writing CTA: one per lane
constexpr int kGradThreads = 128;
constexpr int kJoinWarps = 8;

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <int kVec>
__global__ void __launch_bounds__(kEmbThreads) k_embed_fwd(const int32_t* __restrict__ ids,
                                                           const uint8_t* __restrict__ pad, int64_t n_tokens,
                                                           const uint16_t* __restrict__ w, int64_t ld_w, int vocab,
                                                           int d, float scale, uint16_t* __restrict__ out,
                                                           int64_t ld_out, uint32_t* __restrict__ status) {
    constexpr int kU = 4;              // loads in flight per lane
    pdl_wait();                        // ids come from the corruption kernel
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int nv = d / kVec;
    const int slabs = (nv + 32 * kU - 1) / (32 * kU);
    const int64_t items = n_tokens * slabs;
    const int64_t step = int64_t(gridDim.x) * (kEmbThreads / 32);
    for (int64_t it = int64_t(blockIdx.x) * (kEmbThreads / 32) + threadIdx.x / 32; it < items; it += step) {
        const int64_t i = it / slabs;
        const int s = int(it - i * slabs);
        const bool is_pad = pad && pad[i];
        const int id = is_pad ? -1 : ids[i];
        const bool ok = uint32_t(id) < uint32_t(vocab);
        if (!ok && !is_pad && s == 0 && lane == 0 && status) atomicOr(status, DLM_DEV_BAD_TOKEN_ID);
        const uint16_t* src = w + int64_t(ok ? id : 0) * ld_w;
        uint16_t* dst = out + i * ld_out;
        const int v0 = s * 32 * kU + lane;
        if constexpr (kVec == 8) {
            uint4 r[kU];
            #pragma unroll
            for (int u = 0; u < kU; ++u)
                r[u] = (ok && v0 + 32 * u < nv) ? __ldg(reinterpret_cast<const uint4*>(src) + v0 + 32 * u)
                                                : make_uint4(0, 0, 0, 0);
            #pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (v0 + 32 * u >= nv) break;
                uint32_t x[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
                #pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = pack_bf16x2(bf16lo(x[k]) * scale, bf16hi(x[k]) * scale);
                reinterpret_cast<uint4*>(dst)[v0 + 32 * u] = make_uint4(x[0], x[1], x[2], x[3]);
            }
        } else {
            float r[kU];
            #pragma unroll
            for (int u = 0; u < kU; ++u)
                r[u] = (ok && v0 + 32 * u < nv) ? bf16_bits_to_float(__ldg(src + v0 + 32 * u)) : 0.f;
            #pragma unroll
            for (int u = 0; u < kU; ++u)
                if (v0 + 32 * u < nv)
                    dst[v0 + 32 * u] = __bfloat16_as_ushort(__float2bfloat16_rn(r[u] * scale));
        }
    }
}

// ---------------------------------------------------------------------------
// gradient: the sort
// ---------------------------------------------------------------------------
struct EmbHeader {
    uint32_t status;      // DLM_DEV_* bits of this call
};

// Calls f(token, id, valid) for the tokens of one warp's section, 128 at a
// time; every lane takes part in every call.
template <typename F>
__device__ __forceinline__ void for_section(const int32_t* __restrict__ ids, const uint8_t* __restrict__ pad,
                                            int64_t beg, int64_t end, bool wide, F&& f) {
    const int lane = threadIdx.x & 31;
    for (int64_t i = beg; i < end; i += 128) {
        const int64_t at = i + lane * 4;
        int id[4];
        if (wide && at + 4 <= end) {
            const int4 q = __ldg(reinterpret_cast<const int4*>(ids + at));
            id[0] = q.x; id[1] = q.y; id[2] = q.z; id[3] = q.w;
        } else {
            #pragma unroll
            for (int e = 0; e < 4; ++e) id[e] = at + e < end ? __ldg(ids + at + e) : 0;
        }
        #pragma unroll
        for (int e = 0; e < 4; ++e) f(int(at + e), id[e], at + e < end && !(pad && pad[at + e]));
    }
}

__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const int32_t* __restrict__ ids,
                                                             const uint8_t* __restrict__ pad, int64_t n_tokens,
                                                             int vocab, int range, EmbHeader* __restrict__ hdr,
                                                             int32_t* __restrict__ row_start,
                                                             int32_t* __restrict__ order, int32_t* __restrict__ sid,
                                                             int wide) {
    extern __shared__ int cnt[];       // [kSortWarps][range]: counts, then next places
    __shared__ int s_warp[kSortWarps];
    __shared__ int s_below;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v0 = blockIdx.x * range;
    const int n = min(range, vocab - v0);
    for (int k = tid; k < kSortWarps * range; k += kSortThreads) cnt[k] = 0;
    if (tid == 0) s_below = 0;
    __syncthreads();
    pdl_wait();
    const int64_t per = ((n_tokens + kSortWarps - 1) / kSortWarps + 127) / 128 * 128;
    const int64_t beg = warp * per < n_tokens ? warp * per : n_tokens;
    const int64_t end = beg + per < n_tokens ? beg + per : n_tokens;
    int* mine = cnt + warp * range;

    int below = 0;
    bool bad = false;
    for_section(ids, pad, beg, end, wide, [&](int, int id, bool valid) {
        bad |= valid && uint32_t(id) >= uint32_t(vocab);
        below += valid && id >= 0 && id < v0;
        const int r = id - v0;
        const bool in = valid && uint32_t(r) < uint32_t(n);
        const uint32_t m = __ballot_sync(~0u, in);
        if (m == 0) return;
        if (in) {
            const uint32_t peers = __match_any_sync(m, r);
            if (lane == __ffs(peers) - 1) mine[r] += __popc(peers);
        }
        __syncwarp();
    });
    below = __reduce_add_sync(~0u, below);
    if (lane == 0 && below) atomicAdd(&s_below, below);
    const int any_bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && tid == 0) hdr->status = any_bad ? DLM_DEV_BAD_TOKEN_ID : 0u;

    // exclusive scan over the range's rows: kRowsPer consecutive rows a thread
    constexpr int kRowsPer = (kMaxRange + kSortThreads - 1) / kSortThreads;
    int tot[kRowsPer], sum = 0;
    #pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
        const int r = tid * kRowsPer + k;
        tot[k] = 0;
        if (r < n) {
            #pragma unroll
            for (int w = 0; w < kSortWarps; ++w) tot[k] += cnt[w * range + r];
        }
        sum += tot[k];
    }
    int inc = sum;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int at = s_below + inc - sum;
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    #pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
        const int r = tid * kRowsPer + k;
        if (r < n) {
            row_start[v0 + r] = at;
            int place = at;
            #pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = cnt[w * range + r];
                cnt[w * range + r] = place;
                place += c;
            }
            if (v0 + r == vocab - 1) row_start[vocab] = place;
        }
        at += tot[k];
    }
    __syncthreads();

    for_section(ids, pad, beg, end, wide, [&](int i, int id, bool valid) {
        const int r = id - v0;
        const bool in = valid && uint32_t(r) < uint32_t(n);
        const uint32_t m = __ballot_sync(~0u, in);
        if (m == 0) return;
        if (in) {
            const uint32_t peers = __match_any_sync(m, r);
            const int first = mine[r];
            const int rank = __popc(peers & ((1u << lane) - 1u));
            order[first + rank] = i;
            sid[first + rank] = id;
            __syncwarp(m);
            if (rank == 0) mine[r] = first + __popc(peers);
        }
        __syncwarp();
    });
}

// ---------------------------------------------------------------------------
// gradient: sums over sorted positions, zero rows
// ---------------------------------------------------------------------------
template <int kVec, typename GT>
__device__ __forceinline__ void put_row(GT* __restrict__ dst, const float (&acc)[kVec], float scale, bool accumulate) {
    if constexpr (kVec == 8 && std::is_same<GT, float>::value) {
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 o = accumulate ? reinterpret_cast<const float4*>(dst)[h] : make_float4(0.f, 0.f, 0.f, 0.f);
            o.x += scale * acc[4 * h]; o.y += scale * acc[4 * h + 1];
            o.z += scale * acc[4 * h + 2]; o.w += scale * acc[4 * h + 3];
            reinterpret_cast<float4*>(dst)[h] = o;
        }
    } else if constexpr (kVec == 8) {
        const uint4 o = accumulate ? *reinterpret_cast<const uint4*>(dst) : make_uint4(0, 0, 0, 0);
        uint32_t x[4] = {o.x, o.y, o.z, o.w};
        #pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = pack_bf16x2(bf16lo(x[k]) + scale * acc[2 * k], bf16hi(x[k]) + scale * acc[2 * k + 1]);
        *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
    } else if constexpr (std::is_same<GT, float>::value) {
        *dst = (accumulate ? *dst : 0.f) + scale * acc[0];
    } else {
        *dst = __bfloat16_as_ushort(
            __float2bfloat16_rn((accumulate ? bf16_bits_to_float(*dst) : 0.f) + scale * acc[0]));
    }
}

// One row of zeros by the whole CTA: 16-byte stores between the first and the
// last 16-byte border, single elements outside.
template <typename GT>
__device__ __forceinline__ void zero_row(GT* __restrict__ dst, int d) {
    constexpr int kPer = 16 / int(sizeof(GT));
    const int head = min(d, int(((16u - unsigned(reinterpret_cast<uintptr_t>(dst) & 15u)) & 15u) / sizeof(GT)));
    const int nv = (d - head) / kPer;
    uint4* mid = reinterpret_cast<uint4*>(dst + head);
    for (int v = threadIdx.x; v < nv; v += blockDim.x) mid[v] = make_uint4(0, 0, 0, 0);
    const int rest = d - head - nv * kPer;
    for (int k = threadIdx.x; k < head + rest; k += blockDim.x) dst[k < head ? k : d - rest + (k - head)] = GT(0);
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
    int tiles;            // column tiles of a row
    int64_t chunk_ctas;   // chunks x tiles; the CTAs behind them write zero rows
};

template <int kVec, typename GT>
__global__ void __launch_bounds__(kGradThreads) k_embed_grad(EmbGradArgs a) {
    constexpr int kU = 8;              // rows in flight
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    GT* dw = static_cast<GT*>(a.d_weight);
    if (int64_t(blockIdx.x) >= a.chunk_ctas) {
        const int64_t r0 = (int64_t(blockIdx.x) - a.chunk_ctas) * kZeroRows;
        const int64_t r = r0 + lane;
        const bool empty = r < a.vocab && a.row_start[r] == a.row_start[r + 1];
        uint32_t m = __ballot_sync(~0u, empty);
        while (m) {
            zero_row(dw + (r0 + __ffs(m) - 1) * a.ld_dw, a.d);
            m &= m - 1;
        }
        return;
    }
    const int64_t c = blockIdx.x / a.tiles;
    const int col = (int(blockIdx.x - c * a.tiles) * blockDim.x + threadIdx.x) * kVec;
    const bool active = col < a.d;
    const int64_t p0 = c * kChunk;
    const int64_t total = a.row_start[a.vocab];
    const int n = int(min(int64_t(kChunk), total - p0));
    if (n <= 0) return;
    const int tok = lane < n ? a.order[p0 + lane] : 0;
    const int row = lane < n ? a.sid[p0 + lane] : -1;
    const int before = p0 > 0 ? a.sid[p0 - 1] : -1;
    const int after = p0 + n < total ? a.sid[p0 + n] : -1;
    bool open = before == __shfl_sync(~0u, row, 0);      // the current row began before this chunk
    float acc[kVec];
    #pragma unroll
    for (int k = 0; k < kVec; ++k) acc[k] = 0.f;
    float* part = a.part + (c * 2) * int64_t(a.pitch) + col;
    for (int p = 0; p < n; p += kU) {
        uint4 q[kU];
        #pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int t = __shfl_sync(~0u, tok, (p + u) & 31);
            q[u] = make_uint4(0, 0, 0, 0);
            if (active && p + u < n) {
                const uint16_t* src = a.d_out + t * a.ld + col;
                if constexpr (kVec == 8) q[u] = __ldg(reinterpret_cast<const uint4*>(src));
                else q[u].x = uint32_t(__ldg(src)) << 16;
            }
        }
        #pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (p + u >= n) break;
            if constexpr (kVec == 8) {
                const uint32_t x[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                #pragma unroll
                for (int k = 0; k < 4; ++k) { acc[2 * k] += bf16lo(x[k]); acc[2 * k + 1] += bf16hi(x[k]); }
            } else {
                acc[0] += __uint_as_float(q[u].x);
            }
            const int id = __shfl_sync(~0u, row, p + u);
            const int nx = __shfl_sync(~0u, row, (p + u + 1) & 31);
            const bool last = p + u + 1 == n;
            const int next = last ? after : nx;
            if (id != next || last) {
                if (active) {
                    if (open || id == next) {            // crosses a border: fp32 partial
                        float* dst = part + (open ? 0 : a.pitch);
                        #pragma unroll
                        for (int k = 0; k < kVec; ++k) dst[k] = acc[k];
                    } else {
                        put_row<kVec, GT>(dw + int64_t(id) * a.ld_dw + col, acc, a.scale, a.accumulate);
                    }
                }
                open = false;
                #pragma unroll
                for (int k = 0; k < kVec; ++k) acc[k] = 0.f;
            }
        }
    }
}

// Adds up the rows that cross chunk borders: a CTA looks at 32 chunks (one
// per lane) for rows that begin in them and end behind them, 32 columns at a
// time; its warps take consecutive parts of the row's chunks and their sums
// are added in that order.
template <typename GT>
__global__ void __launch_bounds__(kJoinWarps * 32) k_embed_join(EmbGradArgs a) {
    __shared__ float s[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    pdl_wait();
    const int64_t total = a.row_start[a.vocab];
    GT* dw = static_cast<GT*>(a.d_weight);
    for (int64_t c0 = int64_t(blockIdx.y) * 32; (c0 + 1) * kChunk < total; c0 += int64_t(gridDim.y) * 32) {
        int first = 0, last = 0, row = -1;
        const int64_t behind = (c0 + lane + 1) * kChunk;
        if (behind < total) {
            const int v = a.sid[behind - 1];
            if (v == a.sid[behind] && a.row_start[v] >= behind - kChunk) {
                row = v;
                first = int(c0) + lane;
                last = (a.row_start[v + 1] - 1) / kChunk;
            }
        }
        uint32_t m = __ballot_sync(~0u, row >= 0);
        while (m) {
            const int src = __ffs(m) - 1;
            m &= m - 1;
            const int v = __shfl_sync(~0u, row, src);
            const int64_t f = __shfl_sync(~0u, first, src);
            const int cnt = __shfl_sync(~0u, last, src) - int(f) + 1;
            const int per = (cnt + kJoinWarps - 1) / kJoinWarps;
            const int k0 = min(cnt, warp * per), k1 = min(cnt, k0 + per);
            float acc = 0.f;
            if (col < a.d) {
                constexpr int kU = 8;      // loads in flight
                for (int k = k0; k < k1; k += kU) {
                    float x[kU];
                    #pragma unroll
                    for (int u = 0; u < kU; ++u)
                        x[u] = k + u < k1 ? a.part[((f + k + u) * 2 + (k + u == 0)) * int64_t(a.pitch) + col] : 0.f;
                    #pragma unroll
                    for (int u = 0; u < kU; ++u) acc += x[u];
                }
            }
            s[warp][lane] = acc;
            __syncthreads();
            if (warp == 0 && col < a.d) {
                float t[1] = {0.f};
                #pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) t[0] += s[w][lane];
                put_row<1, GT>(dw + int64_t(v) * a.ld_dw + col, t, a.scale, a.accumulate);
            }
            __syncthreads();
        }
    }
}

// Workspace of the gradient: header, row_start [vocab + 1], order and sid
// [n_tokens], partials.
struct EmbPlan {
    int64_t chunks;
    int pitch;
    size_t off_start, off_order, off_sid, off_part, bytes;
};

static bool embed_plan(const dlm_layout_t* L, int32_t vocab, int32_t d, EmbPlan* p) {
    if (!layout_ok(L) || vocab < 1 || d < 1 || vocab == INT32_MAX || d > INT32_MAX - 64) return false;
    p->chunks = (L->n_tokens + kChunk - 1) / kChunk;
    p->pitch = int(align_up(size_t(d), 32));
    p->off_start = kWsAlign;
    p->off_order = align_up(p->off_start + (size_t(vocab) + 1) * 4, kWsAlign);
    p->off_sid = align_up(p->off_order + size_t(L->n_tokens) * 4, kWsAlign);
    p->off_part = align_up(p->off_sid + size_t(L->n_tokens) * 4, kWsAlign);
    p->bytes = align_up(p->off_part + size_t(p->chunks) * 2 * size_t(p->pitch) * 4, kWsAlign);
    return true;
}

template <int kVec, typename GT>
static dlm_status_t launch_grad(const EmbGradArgs& a, unsigned grid, unsigned threads, cudaStream_t s) {
    return launch_pdl(k_embed_grad<kVec, GT>, dim3(grid), dim3(threads), 0, s, "k_embed_grad launch", a);
}

}  // namespace dlm

using namespace dlm;

extern "C" dlm_status_t dlm_embed_fwd(const dlm_layout_t* layout, const int32_t* ids, const uint16_t* weight,
                                      int64_t ld_weight, int32_t vocab, int32_t d_model, float scale, uint16_t* out,
                                      int64_t ld_out, uint32_t* dev_status, dlm_stream_t stream) {
    DLM_NVTX("dlm_embed_fwd");
    if (!layout_ok(layout) || vocab < 1 || d_model < 1 || ld_weight < d_model || ld_out < d_model)
        return DLM_ERR_INVALID_ARGUMENT;
    if (!(scale - scale == 0.0f)) return DLM_ERR_INVALID_ARGUMENT;       // inf or NaN
    if (layout->n_tokens == 0) return DLM_OK;
    if (!ids || !weight || !out) return DLM_ERR_INVALID_ARGUMENT;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    const bool vec = d_model % 8 == 0 && ld_weight % 8 == 0 && ld_out % 8 == 0 && aligned16(weight) && aligned16(out);
    const int64_t nv = vec ? d_model / 8 : d_model;
    const int64_t items = layout->n_tokens * ((nv + 127) / 128);
    int64_t blocks = (items + kEmbThreads / 32 - 1) / (kEmbThreads / 32);
    if (blocks > (1 << 20)) blocks = 1 << 20;
    return launch_pdl(vec ? k_embed_fwd<8> : k_embed_fwd<1>, dim3(unsigned(blocks)), dim3(kEmbThreads), 0,
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
    const int nv = vec ? d_model / 8 : d_model;
    const unsigned threads = nv >= kGradThreads ? kGradThreads : unsigned(align_up(size_t(nv), 32));
    const int tiles = int((unsigned(nv) + threads - 1) / threads);
    const int64_t grid = p.chunks * tiles + (accumulate ? 0 : (int64_t(vocab) + kZeroRows - 1) / kZeroRows);
    if (grid > INT32_MAX) return DLM_ERR_INVALID_ARGUMENT;
    dlm_status_t st = check_device();
    if (st != DLM_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    EmbHeader* hdr = reinterpret_cast<EmbHeader*>(ws);
    int32_t* row_start = reinterpret_cast<int32_t*>(ws + p.off_start);
    int32_t* order = reinterpret_cast<int32_t*>(ws + p.off_order);
    int32_t* sid = reinterpret_cast<int32_t*>(ws + p.off_sid);

    // a range of vocabulary rows per SM, as far as the counters fit
    int range = int(align_up(size_t((vocab + 147) / 148), 32));
    if (range > kMaxRange) range = kMaxRange;
    const size_t smem = size_t(kSortWarps) * range * 4;
    cudaError_t e = cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSortWarps * kMaxRange * 4);
    if (e != cudaSuccess) { cudaGetLastError(); return cuda_status(e, "k_embed_sort attributes"); }
    st = launch_pdl(k_embed_sort, dim3(unsigned((int64_t(vocab) + range - 1) / range)), dim3(kSortThreads), smem, s,
                    "k_embed_sort launch", ids, layout->pad_mask, layout->n_tokens, vocab, range, hdr, row_start,
                    order, sid, int(aligned16(ids)));
    if (st != DLM_OK) return st;

    if (grid == 0) return DLM_OK;
    EmbGradArgs a;
    a.d_out = d_out; a.ld = ld; a.vocab = vocab; a.d = d_model; a.scale = scale; a.accumulate = accumulate;
    a.d_weight = d_weight; a.ld_dw = ld_dw; a.row_start = row_start; a.order = order; a.sid = sid;
    a.part = reinterpret_cast<float*>(ws + p.off_part);
    a.pitch = p.pitch; a.tiles = tiles; a.chunk_ctas = p.chunks * tiles;
    if (f32) st = vec ? launch_grad<8, float>(a, unsigned(grid), threads, s)
                      : launch_grad<1, float>(a, unsigned(grid), threads, s);
    else st = vec ? launch_grad<8, uint16_t>(a, unsigned(grid), threads, s)
                  : launch_grad<1, uint16_t>(a, unsigned(grid), threads, s);
    if (st != DLM_OK || p.chunks < 2) return st;
    const int64_t groups = (p.chunks + 31) / 32;
    const dim3 jgrid(unsigned((d_model + 31) / 32), unsigned(groups < 65535 ? groups : 65535));
    return launch_pdl(f32 ? k_embed_join<float> : k_embed_join<uint16_t>, jgrid, dim3(kJoinWarps * 32), 0, s,
                      "k_embed_join launch", a);
}
