// bsa_chunk.cuh -- what the kernels of the attention of new tokens share: the
// sequences, which tiles of slots they see, and how the parts of a row that
// several CTAs worked on are handed to the merge.
#pragma once

#include <limits.h>
#include <math.h>

#include "bsa_internal.h"
#include "bsa_ptx.cuh"

namespace bsa {

constexpr int kTile = 128;            // key slots of a step
constexpr int kChunkMaxCtas = 160;    // parts are sized for this many
constexpr int kShortRows = 16;        // query rows of a key head up to which a sequence is "short"

struct ChunkCommon {
    const int32_t *ctx, *q_ptr, *table;
    const uint8_t *ks, *vs;           // 8-bit pools: the rows' scales
    int32_t B, tokens, Hq, Hkv, G, page, P, n_pages;
    int32_t window, sinks;
    void* out;
    float* lse;
    int32_t* err;
    float scale_log2;
    unsigned long long wait_limit_ns;
};

// The item that a CTA's range of steps starts inside of (start < 0: none): its
// first step and the one behind its last, the steps of a range, its rows.
struct PartMeta {
    int start, end, per;
    int row0, n;   // first token (row of q) and tokens
    int h;
    int pad[2];
};

struct Seq {
    int row0, n, ctx;
};

// New tokens of sequence b; none where q_ptr makes no sense or positions leave an int.
__device__ __forceinline__ Seq sequence(const ChunkCommon& p, int b, bool report) {
    Seq s{b, 1, max(p.ctx[b], 0)};
    if (p.q_ptr) {
        const int lo = p.q_ptr[b], hi = p.q_ptr[b + 1];
        if (lo < 0 || hi < lo || hi > p.tokens) {
            if (report) atomicOr(p.err, ERR_BAD_ROW);
            return Seq{0, 0, 0};
        }
        s.row0 = lo;
        s.n = hi - lo;
    }
    if (s.n > 0 && s.ctx > INT_MAX - 1024 - s.n) {
        if (report) atomicOr(p.err, ERR_BAD_PAGE);
        s.n = 0;
    }
    if (report && s.n > 0 && s.ctx + s.n > p.P * p.page) atomicOr(p.err, ERR_BAD_PAGE);
    return s;
}

// Tiles of slots that the tokens in slots first .. end - 1 see: the sinks' and,
// from lo_tile on, those of their windows.
struct Span {
    int sink_tiles, lo_tile, steps;
    __device__ __forceinline__ int tile(int step) const {
        return step < sink_tiles ? step : lo_tile + step - sink_tiles;
    }
};
__device__ __forceinline__ int first_slot(const ChunkCommon& p, int first) {
    return p.window > 0 ? max(0, first - p.window + 1) : 0;
}
__device__ __forceinline__ Span visible_span(const ChunkCommon& p, int first, int end) {
    end = min(end, p.P * p.page);
    Span s;
    s.lo_tile = first_slot(p, first) / kTile;
    const int tiles = (int)(((unsigned)end + kTile - 1) / kTile);
    s.sink_tiles = p.window > 0 ? min((int)(((unsigned)min(p.sinks, end) + kTile - 1) / kTile), s.lo_tile) : 0;
    // at least one, so that rows which see nothing pass through and write their zeros
    s.steps = max(1, s.sink_tiles + max(0, tiles - s.lo_tile));
    return s;
}

// Slots u that a token in slot pos sees among base .. base + 63, as bits; none where
// they lie in no page (have 0).
__device__ __forceinline__ unsigned long long below(int n) {  // bits 0 .. n - 1
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ unsigned long long seen_slots(const ChunkCommon& p, int base, int pos, int have) {
    unsigned long long m = below(pos + 1 - base);
    if (p.window > 0) m &= ~below(max(pos - p.window + 1, 0) - base) | below(p.sinks - base);
    return have ? m : 0ull;
}

// Page j of sequence b for tokens that see from slot lo to slot end - 1 (and the
// sinks): its first row in the pools, or -1 where nothing of it is seen or it is
// not there (reported).
__device__ __forceinline__ int page_row(const ChunkCommon& p, int b, int h, int j, int lo, int end) {
    const unsigned s0 = (unsigned)j * p.page;
    if (j >= p.P || s0 >= (unsigned)end) return -1;
    if (s0 + p.page <= (unsigned)lo && !(p.window > 0 && s0 < (unsigned)p.sinks)) return -1;
    const int pg = p.table[(int64_t)b * p.P + j];
    if ((unsigned)pg >= (unsigned)p.n_pages) {
        atomicOr(p.err, ERR_BAD_PAGE);
        return -1;
    }
    return (pg * p.Hkv + h) * p.page;
}

// Natural-log LSE of a row from its reference (log2) and sum.
__device__ __forceinline__ float lse_of(float m, float sum) {
    return sum == 0.f ? -INFINITY : (m + __log2f(sum)) * 0.69314718055994531f;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile WaitFlag* wf) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, wf));
}

// Whole warp: until the counter (which only grows) is at `want`.  A barrier's
// parity tells a phase from its neighbours only, so who does not wait for every
// phase of a barrier first makes sure that the phase it wants is the current one
// or the one before: a tile's load was issued, so its slot's last use is over.
__device__ __forceinline__ bool reached(volatile uint32_t* count, uint32_t want, volatile WaitFlag* wf) {
    if (__any_sync(0xffffffffu, *count >= want)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (__any_sync(0xffffffffu, *count >= want)) return true;
        if ((it & 31u) == 0) {
            const bool late = globaltimer_ns() - t0 > wf->limit_ns;
            if (late) wf->abort = 1;
            if (__any_sync(0xffffffffu, late || wf->abort)) return false;
        }
    }
}

// Untiled bulk copy global -> shared (16-byte aligned, bytes % 16 == 0), counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

struct ShortLaunch {
    ChunkCommon c;
    const void *k, *v, *q;
    int32_t D, sms;
    PartMeta* meta;
    float* part_o;
    float2* part_ml;
    bool merge;            // else the caller joins the parts (of the last launch, if there are several)
};
// Sequences whose new tokens make at most kShortRows rows of a key head (csrc/bsa_decode.cu).
int launch_short(const ShortLaunch& L, cudaStream_t s);
// Rows of a key head that its sequences can have, at most.
inline int short_rows(const ChunkCommon& c) {
    return c.G <= 8 && (!c.q_ptr || (int64_t)c.tokens * c.G <= 8) ? 8 : kShortRows;
}

// Joins the parts of items that range boundaries cut, in range order: with parts i,
// m = max m_i, w_i = 2^(m_i - m), O = sum w_i O_i / sum w_i l_i.  Chunks: a CTA to 32
// rows, a lane to each, a warp to an eighth of the columns, which is how their parts lie
// in memory: whole lines both written and read (with rows behind one another a part of
// 128-wide rows took its CTA 5.3 us, now 2.0).  Short sequences, which can have a part from every CTA: eight warps to a row,
// every eighth part each.  Bound by dependent reads from the L2.
struct PartSet {
    const PartMeta* meta;
    const float* o;       // short sequences: [2 * ctas][16][D]; chunks: [2 * ctas][D / 4][256][4]
    const float2* ml;     // [2 * ctas][rows]
};
// The item that the boundary in front of range x + 1 is the first to cut: its
// parts are those of ranges x .. last.
struct CutItem {
    PartMeta mt;
    int first, last;
    __device__ __forceinline__ bool find(const PartMeta* meta, int x) {
        mt = meta[x + 1];
        first = x;
        if (mt.start < 0 || mt.start < x * mt.per) return false;  // not cut here, or by an earlier boundary too
        last = (mt.end - 1) / mt.per;
        return true;
    }
    __device__ __forceinline__ int slot(int k) const { return 2 * k + (k == first && mt.start > first * mt.per ? 1 : 0); }
};

template <int D>
__device__ __forceinline__ void store_row(const ChunkCommon& p, int64_t orow, int lane, const float* acc, float m, float l) {
    constexpr int C = D / 32;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (lane == 0) p.lse[orow] = lse_of(m, l);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + orow * D;
    if (C == 4)
        reinterpret_cast<uint2*>(out)[lane] =
            make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[C - 2] * inv, acc[C - 1] * inv));
    else
        reinterpret_cast<uint32_t*>(out)[lane] = pack_bf16x2(acc[0] * inv, acc[1] * inv);
}
template <int D>
__device__ __forceinline__ void add_part(float* acc, const float* src, float w) {
    constexpr int C = D / 32;
    if (C == 4) {
        const float4 o = *reinterpret_cast<const float4*>(src);
        acc[0] += w * o.x;
        acc[1] += w * o.y;
        acc[C - 2] += w * o.z;
        acc[C - 1] += w * o.w;
    } else {
        const float2 o = *reinterpret_cast<const float2*>(src);
        acc[0] += w * o.x;
        acc[1] += w * o.y;
    }
}

// blockIdx.y < rows_short: row blockIdx.y of a short sequence's item; behind those, 32
// rows of a chunk's item (256 rows, two tiles of tq tokens).
template <int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkCommon p, const PartSet few, const PartSet many,
                                                          int rows_short, int tq) {
    constexpr int C = D / 32;
    __shared__ float red[8][D + 1];
    __shared__ uint2 rows[32][D / 4 + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    CutItem it;
    if ((int)blockIdx.y < rows_short) {
        if (!it.find(few.meta, blockIdx.x)) return;
        const int r = blockIdx.y;
        if (r >= it.mt.n * p.G) return;
        float m = -INFINITY, l = 0.f, acc[C];
#pragma unroll
        for (int x = 0; x < C; ++x) acc[x] = 0.f;
        for (int k = it.first + lane; k <= it.last; k += 32) m = fmaxf(m, few.ml[(int64_t)it.slot(k) * kShortRows + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m > -INFINITY ? m : 0.f;
#pragma unroll 4
        for (int k = it.first + warp; k <= it.last; k += 8) {
            const int64_t pr = (int64_t)it.slot(k) * kShortRows + r;
            const float2 ml = few.ml[pr];
            const float w = ex2_approx(ml.x - ref);  // 0 for a part that saw nothing
            l += w * ml.y;
            add_part<D>(acc, few.o + pr * D + lane * C, w);
        }
#pragma unroll
        for (int x = 0; x < C; ++x) red[warp][lane * C + x] = acc[x];
        if (lane == 0) red[warp][D] = l;
        __syncthreads();
        if (warp > 0) return;
        for (int w = 1; w < 8; ++w) {
#pragma unroll
            for (int x = 0; x < C; ++x) acc[x] += red[w][lane * C + x];
            l += red[w][D];
        }
        store_row<D>(p, (int64_t)(it.mt.row0 + r / p.G) * p.Hq + it.mt.h * p.G + r % p.G, lane, acc, m, l);
        return;
    }
    if (!it.find(many.meta, blockIdx.x)) return;
    const int r0 = ((int)blockIdx.y - rows_short) * 32;
    // row of q that row r of the item is, times Hq, plus its head; < 0: none
    auto place = [&](int r) -> int64_t {
        const int i = r & 127, t = (r >> 7) * tq + i / p.G;  // row in its tile, token
        return i < tq * p.G && t < it.mt.n ? (int64_t)(it.mt.row0 + t) * p.Hq + it.mt.h * p.G + i % p.G : -1;
    };
    const int64_t mine = place(r0 + lane);
    if (!__any_sync(0xffffffffu, mine >= 0)) return;  // the same in every warp
    float m = -INFINITY, l = 0.f, acc[C][4];
#pragma unroll
    for (int q = 0; q < C; ++q)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[q][x] = 0.f;
    if (mine >= 0) {
#pragma unroll 4
        for (int k = it.first; k <= it.last; ++k) m = fmaxf(m, many.ml[(int64_t)it.slot(k) * 256 + r0 + lane].x);
        const float ref = m > -INFINITY ? m : 0.f;
#pragma unroll 2
        for (int k = it.first; k <= it.last; ++k) {
            const int64_t part = it.slot(k);
            const float2 ml = many.ml[part * 256 + r0 + lane];
            const float w = ex2_approx(ml.x - ref);  // 0 for a part that saw nothing
            l += w * ml.y;
            const float4* src = reinterpret_cast<const float4*>(many.o) + (part * (D / 4) + warp) * 256 + r0 + lane;
#pragma unroll
            for (int q = 0; q < C; ++q) {
                const float4 o = src[q * 8 * 256];
                acc[q][0] += w * o.x;
                acc[q][1] += w * o.y;
                acc[q][2] += w * o.z;
                acc[q][3] += w * o.w;
            }
        }
        if (warp == 0) p.lse[mine] = lse_of(m, l);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int q = 0; q < C; ++q)
        rows[lane][warp + 8 * q] = make_uint2(pack_bf16x2(acc[q][0] * inv, acc[q][1] * inv), pack_bf16x2(acc[q][2] * inv, acc[q][3] * inv));
    __syncthreads();
#pragma unroll
    for (int x = threadIdx.x; x < 32 * (D / 4); x += 256) {
        const int64_t at = place(r0 + x / (D / 4));
        if (at >= 0) reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at * D)[x % (D / 4)] = rows[x / (D / 4)][x % (D / 4)];
    }
}

}  // namespace bsa
