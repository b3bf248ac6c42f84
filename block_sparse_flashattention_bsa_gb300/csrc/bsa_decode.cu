// bsa_decode.cu -- attention over a paged cache for sequences whose new tokens
// make at most 16 query rows of a key head (one token of up to 16 grouped heads,
// or a few tokens): the serving form of the chunk attention.
//
// Mathematics: O = softmax(q K^T scale) V over the slots a row sees, in one pass.
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that the
// keys and the head's values fill the 16-row side of mma.sync and the few query
// rows the 8-column side.
//
// What bounds it: every K and V row is read once, 2 D bytes (8-bit) or 4 D bytes
// a slot, for 4 D flops a row: memory.  An SM's share of the copy rate is ~24
// bytes a cycle.  tcgen05 would take 128 rows and operands in shared memory: of
// 8-bit rows 96 bytes of shared-memory traffic for every 32 loaded (the converted
// tile written and read, Q read for every step), 1,700 cycles a step against
// 1,400 for its bytes.  Here a warp reads its 16 keys from shared memory once,
// converts them in registers and multiplies: 2 bytes of traffic per byte.
//
// Work: a step is 256 slots (128 with more than 8 rows, or few steps); an item the steps of one key head of one sequence;
// the steps of the batch, cut into equal ranges, one per CTA.  An item that a
// range boundary cuts leaves unnormalised fp32 parts that the merge joins in range
// order: no atomics, results do not depend on timing.
//
// One CTA per SM: a producer warp walks the range, resolves pages and TMA-loads K
// and V tiles into a ring, and an item's queries; ten consumer warps take units of 16
// keys (of both tiles of a step) in turn, each with a running maximum, sum and
// accumulator of its own, so steps need no exchange; what they have at an item's end
// one more warp joins while they go on.
// bf16 rows: P is multiplied as two bf16 parts, high and low, so that its rounding
// (2^-16) does not add to the result's.  8-bit rows: fp16 products, since a
// code is an fp16 number (one conversion instruction for two; to bf16 it takes
// four and a product) and P rounds at 2^-11 in it.

#include <cuda_fp16.h>

#include <algorithm>

#include "bsa.h"
#include "bsa_chunk.cuh"
#include "bsa_q8.cuh"

namespace bsa {
namespace {

constexpr int kShortUnits = 1024;   // sequences of a launch (their prefix sums sit in shared memory)
constexpr int kShortSmem = 232448;
constexpr int kShortCtrl = 7168;
constexpr int kShortMaxSlots = 16;
constexpr int kShortInfos = 4;      // step descriptions ahead
constexpr int kWarps = 10;          // consumer warps
constexpr int kJoiner = kWarps, kProducer = kWarps + 1;
constexpr int kShortItems = 2;      // items ahead
constexpr int kThreads = (kWarps + 2) * 32;

enum : int { kMask = 1, kOne = 2 };  // of a step: some row sees a part of it only; it is one tile
constexpr int kHaveBit = 2;

struct ShortInfo {      // a step
    int flags;          // and from kHaveBit on, per tile, the halves that lie in a page
    int base[2];        // first slot of each tile
    uint32_t tile;      // number of its first K tile in the order of loads
};
struct ShortItem {
    int step0, steps;   // its steps of this CTA; steps < 0: no more items
    int row0, rows, h;  // first token, query rows, key head
    int ctx, end;       // slot of the first new token, slot behind the last one
    int part;           // -1: write the output, else the partial slot
};

struct ShortCtrl {
    uint64_t t_full[kShortMaxSlots], t_empty[kShortMaxSlots];
    uint64_t i_full[kShortInfos], i_empty[kShortInfos];
    uint64_t it_full[kShortItems], it_empty[kShortItems];
    uint64_t x_full, x_empty;  // all consumers posted their part of an item; it has been read
    ShortInfo info[kShortInfos];
    ShortItem item[kShortItems];
    float2 stats[kWarps][16];  // [warp][row]
    int red[kThreads / 32];
    WaitFlag wf;
    volatile uint32_t loaded;  // tiles whose load was issued
    int prefix[kShortUnits + 1];
};
static_assert(sizeof(ShortCtrl) <= kShortCtrl, "control block too large");

struct ShortParams {
    ChunkCommon c;
    const __nv_bfloat16* q;
    int32_t unit0, units, n_slots;
    PartMeta* meta;
    float* part_o;     // [2 * grid][16][D]
    float2* part_ml;   // [2 * grid][16]
};

template <int D, bool Q8, int NT>
struct ShortCfg {
    static constexpr int SUB = NT == 1 ? 2 : 1;       // tiles of a step, at most
    static constexpr int ROWB = Q8 ? D : 128;         // bytes of a row of a box
    static constexpr int NBOX = Q8 ? 1 : D / 64;
    static constexpr int BOX = kTile * ROWB;
    static constexpr int TILE = NBOX * BOX;
    static constexpr int PITCH = D + 4;               // floats of an exchanged row
    static constexpr int XCH = kWarps * 8 * NT * PITCH * 4;
    static constexpr int QROWS = 8 * NT, QBUF = kShortItems * QROWS * D * 2;  // items' queries
    static constexpr int FIXED = XCH + QBUF + kShortCtrl + (Q8 ? kShortMaxSlots * kTile : 0);
    static constexpr int FIT = (kShortSmem - FIXED) / TILE;
    static constexpr int SLOTS = FIT > kShortMaxSlots ? kShortMaxSlots : FIT;
    static constexpr int SMEM = SLOTS * TILE + FIXED;
    // A step is announced when all of its loads were issued, unless the ring is too short
    // for that; then who waits for a tile looks for its load first (reached()).
    static constexpr bool LATE = SLOTS >= 4 * SUB;
    static_assert(SLOTS >= 2 * SUB, "ring too small");
};

// Steps (of `sub` tiles) of a short sequence's item; 0: it has no new tokens or is not short.
__device__ __forceinline__ int short_steps(const ChunkCommon& p, int b, int sub, bool report) {
    const Seq s = sequence(p, b, report);
    if (s.n == 0 || s.n * (int64_t)p.G > kShortRows) return 0;
    return (visible_span(p, s.ctx, s.ctx + s.n).steps + sub - 1) / sub;
}

// ---------------------------------------------------------------- producer
template <int D, bool Q8, int NT>
__device__ void short_producer(const CUtensorMap* tk, const CUtensorMap* tv, const ShortParams& p, uint8_t* sT,
                               uint8_t* sS, __nv_bfloat16* sQ, ShortCtrl* c, int lo, int hi, int per, int sub,
                               volatile WaitFlag* wf) {
    using C = ShortCfg<D, Q8, NT>;
    const ChunkCommon& cc = p.c;
    const int lane = threadIdx.x & 31, Hkv = cc.Hkv, ppt = kTile / cc.page, pps = sub * ppt;
    const bool leader = elect_one();
    constexpr uint32_t infos = kShortInfos;
    uint32_t slot = 0, phase = 0, nload = 0, g = 0, ni = 0;
    bool ok = true;
    PartMeta mt{-1, 0, per, 0, 0, 0, {0, 0}};
    // the next item's description and queries, as soon as there is room
    auto announce = [&](const ShortItem& it) -> bool {
        const uint32_t x = ni % kShortItems;
        if (ni >= kShortItems && !warp_wait(&c->it_empty[x], ((ni / kShortItems) & 1) ^ 1, wf)) return false;
        if (leader) {
            c->item[x] = it;
            if (it.steps > 0) {
                const int n = it.rows / cc.G;  // a token's heads are neighbours
                mbar_arrive_expect_tx(&c->it_full[x], (uint32_t)(it.rows * D * 2));
                for (int t = 0; t < n; ++t)
                    bulk_load(sQ + (x * C::QROWS + t * cc.G) * D,
                              p.q + ((int64_t)(it.row0 + t) * cc.Hq + it.h * cc.G) * D, (uint32_t)(cc.G * D * 2),
                              &c->it_full[x]);
            } else {
                mbar_arrive(&c->it_full[x]);
            }
        }
        __syncwarp();
        ++ni;
        return true;
    };
    if (lo < hi) {
        int u = 0;  // the sequence that holds step lo: last one whose first step is not behind it
        for (int span = p.units; span > 1;) {
            const int stride = (span + 31) >> 5, off = lane * stride;
            const bool le = off < span && c->prefix[u + off] * Hkv <= lo;
            u += (__popc(__ballot_sync(0xffffffffu, le)) - 1) * stride;
            span = min(stride, p.units - u);
        }
        int base = c->prefix[u], per_item = c->prefix[u + 1] - base;
        int h = (lo - base * Hkv) / per_item;
        int pos = lo;
        while (ok && pos < hi) {
            const int b = p.unit0 + u;
            const Seq sq = sequence(cc, b, false);
            const int seq_end = sq.ctx + sq.n, vis0 = first_slot(cc, sq.ctx);
            const Span sp = visible_span(cc, sq.ctx, seq_end);
            const int start = base * Hkv + h * per_item, end = start + per_item;
            const int s0 = pos - start, s1 = min(end, hi) - start;
            const bool whole = s0 == 0 && start + s1 == end;
            const int part = whole ? -1 : 2 * (int)blockIdx.x + (pos == lo ? 0 : 1);
            if (start < lo) mt = PartMeta{start, end, per, sq.row0, sq.n, h, {0, 0}};
            if (!announce(ShortItem{(int)g, s1 - s0, sq.row0, sq.n * cc.G, h, sq.ctx, seq_end, part})) {
                ok = false;
                break;
            }
            for (int e0 = s0 * pps; e0 < s1 * pps && ok; e0 += 32) {
                // 32 pages resolved at a time
                const int e = e0 + lane, tl = e / ppt;
                const int j = sp.tile(tl) * ppt + e % ppt;
                const int y = e < s1 * pps && tl < sp.steps ? page_row(cc, b, h, j, vis0, seq_end) : -1;
                const int cnt = min(32, s1 * pps - e0);
                for (int q = 0; q < cnt && ok; q += pps) {
                    const int st = (e0 + q) / pps;
                    int y0[C::SUB], y1[C::SUB];  // rows of each tile's halves
#pragma unroll
                    for (int x = 0; x < C::SUB; ++x) {
                        y0[x] = __shfl_sync(0xffffffffu, y, q + x * ppt);
                        y1[x] = __shfl_sync(0xffffffffu, y, q + x * ppt + ppt - 1);
                    }
                    const int nx = min(sub, max(1, sp.steps - st * sub));  // its tiles
                    const uint32_t is = g % infos;
                    if (g >= infos && !warp_wait(&c->i_empty[is], ((g / infos) & 1) ^ 1, wf)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        ShortInfo& f = c->info[is];
                        bool plain = true;
                        int have = 0;
#pragma unroll
                        for (int x = 0; x < C::SUB; ++x) {
                            if (x >= nx) continue;
                            const int first = sp.tile(st * sub + x) * kTile;
                            const int hv = ppt == 1 ? (y0[x] >= 0 ? 3 : 0) : (y0[x] >= 0 ? 1 : 0) | (y1[x] >= 0 ? 2 : 0);
                            // every row sees all of it: up to the first token, inside the last one's window
                            plain &= hv == 3 && first + kTile <= sq.ctx + 1 &&
                                     (cc.window <= 0 || first > seq_end - 1 - cc.window || first + kTile <= cc.sinks);
                            have |= hv << (2 * x);
                            f.base[x] = first;
                        }
                        f.flags = (plain ? 0 : kMask) | (nx == 1 ? kOne : 0) | have << kHaveBit;
                        f.tile = nload;
                        if (!C::LATE) mbar_arrive(&c->i_full[is]);
                    }
                    __syncwarp();
                    ++g;
#pragma unroll
                    for (int kv = 0; kv < 2 * C::SUB; ++kv) {  // K tiles, then V tiles
                        const bool val = kv >= C::SUB;
                        const int r0 = y0[kv % C::SUB], r1 = y1[kv % C::SUB];
                        if (kv % C::SUB >= nx) continue;
                        if (nload >= (uint32_t)p.n_slots && !warp_wait(&c->t_empty[slot], phase ^ 1, wf)) {
                            ok = false;
                            break;
                        }
                        if (leader) {
                            uint64_t* bar = &c->t_full[slot];
                            const uint8_t* sc = val ? cc.vs : cc.ks;
                            uint32_t bytes = C::TILE;
                            if (Q8) bytes += (r0 >= 0 ? cc.page : 0) + (ppt == 2 && r1 >= 0 ? cc.page : 0);
                            mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
                            for (int x = 0; x < C::NBOX; ++x) {
                                uint8_t* dst = sT + slot * C::TILE + x * C::BOX;
                                tma_load_2d(dst, val ? tv : tk, bar, x * 64, r0 >= 0 ? r0 : -cc.page);
                                if (ppt == 2)
                                    tma_load_2d(dst + 64 * C::ROWB, val ? tv : tk, bar, x * 64, r1 >= 0 ? r1 : -cc.page);
                            }
                            if (Q8) {
                                if (r0 >= 0) bulk_load(sS + slot * kTile, sc + r0, cc.page, bar);
                                if (ppt == 2 && r1 >= 0) bulk_load(sS + slot * kTile + 64, sc + r1, cc.page, bar);
                            }
                        }
                        ++nload;
                        if (!C::LATE && leader) c->loaded = nload;
                        if (++slot == (uint32_t)p.n_slots) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
                    if (C::LATE && ok && leader) mbar_arrive(&c->i_full[is]);
                }
            }
            pos = start + s1;
            if (++h == Hkv && pos < hi) {
                h = 0;
                do {
                    ++u;
                    base = c->prefix[u];
                    per_item = c->prefix[u + 1] - base;
                } while (per_item == 0);
            }
        }
    }
    if (ok) announce(ShortItem{0, -1, 0, 0, 0, 0, 0, 0});
    if (lane == 0) p.meta[blockIdx.x] = mt;
    __syncwarp();
    if (leader) {
        // copies still in flight must land before the CTA exits
        const uint32_t ns = (uint32_t)p.n_slots;
        for (uint32_t n = nload > ns ? nload - ns : 0; n < nload; ++n)
            mbar_wait_drain(&c->t_full[n % ns], (n / ns) & 1);
        for (uint32_t n = ni > kShortItems ? ni - kShortItems : 0; n < ni; ++n)
            mbar_wait_drain(&c->it_full[n % kShortItems], (n / kShortItems) & 1);
    }
}

// ---------------------------------------------------------------- consumers
// F16: fp16 operands, else bf16.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// 16-byte chunk `ch` of row `row` of a swizzled box.
template <int ROWB>
__device__ __forceinline__ const uint8_t* chunk_at(const uint8_t* box, int row, int ch) {
    return box + row * ROWB + ((ch ^ (ROWB == 64 ? (row >> 1) & 3 : row & 7)) << 4);
}

// A lane (g = lane / 4, c = lane % 4) holds, of keys g and g + 8, the values
// that S^T's k-steps ask for; which values those are is free as long as Q has
// the same order.  8-bit rows: bytes 32 c .. (128-wide; 64-wide 16 c ..), k-step
// j the word 4 j ..: bytes 0, 2 and bytes 1, 3.  bf16 rows: chunks 2 c and 2 c + 1
// of each box, k-step 2 q + i the words 2 i and 2 i + 1 of chunk q.
template <int D, bool Q8>
__device__ __forceinline__ int q_chunk(int c, int q) {  // first value of the lane's q-th 8 values
    return Q8 ? (D / 4) * c + 8 * q : 64 * (q >> 1) + 8 * (2 * c + (q & 1));
}
// First value of the lane's 4 values in accumulator tiles 2 i and 2 i + 1 of O^T.
template <int D, bool Q8>
__device__ __forceinline__ int o_value(int g, int i) {
    return Q8 ? (D / 8) * g + 4 * i : 64 * (i >> 1) + 8 * g + 4 * (i & 1);
}

template <int D, bool Q8, int NT>
__device__ void short_consumer(const ShortParams& p, const uint8_t* sT, const uint8_t* sS, const __nv_bfloat16* sQ,
                               float* xch, ShortCtrl* c, volatile WaitFlag* wf) {
    using C = ShortCfg<D, Q8, NT>;
    constexpr int KS = D / 16, SUB = C::SUB;
    const ChunkCommon& cc = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, cq = lane & 3;
    uint32_t qf[KS][NT][2];
    float o[KS][NT][4];
    float m[NT][2], l[NT][2], sl[NT][2];
    float rv[NT][2];  // 8-bit: what the rows' weights times V's scales are multiplied with, a power of two
    float lv[NT][2];  // 8-bit: the product that rv was set for, times rv, against the present maximum
    for (uint32_t items = 0;; ++items) {
        const uint32_t ii = items % kShortItems;
        if (!warp_wait(&c->it_full[ii], (items / kShortItems) & 1, wf)) return;
        const int step0 = c->item[ii].step0, steps = c->item[ii].steps, rows = c->item[ii].rows;
        const int ctx = c->item[ii].ctx, end = c->item[ii].end;
        if (steps < 0) return;
        // Eight units of 16 keys (of each of its tiles) to a step; the warps take them in turn.
        const uint32_t u0 = (uint32_t)step0 * 8, u1 = u0 + (uint32_t)steps * 8;
        const uint32_t mine = u0 + (warp + kWarps - u0 % kWarps) % kWarps;
        if (mine < u1) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = 8 * nt + g;
                const bool on = r < rows;
                const __nv_bfloat16* src = sQ + (ii * C::QROWS + r) * D;
                uint4 v[KS / 2];
#pragma unroll
                for (int q = 0; q < KS / 2; ++q) {
                    v[q] = make_uint4(0, 0, 0, 0);
                    if (on) v[q] = *reinterpret_cast<const uint4*>(src + q_chunk<D, Q8>(cq, q));
                }
                int up = 0;
                if (Q8) {
                    // fp16 with the row's largest magnitude at 2^14: no bf16 value of the
                    // row above 2^-29 of it is rounded
                    float top = 0.f;
#pragma unroll
                    for (int q = 0; q < KS / 2; ++q)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            top = fmax3(top, fabsf(__uint_as_float(word(v[q], i) << 16)),
                                        fabsf(__uint_as_float(word(v[q], i) & 0xffff0000u)));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    up = min(14 + 127 - (int)(__float_as_uint(top) >> 23), 126);
                }
                const float qs = exp2_int(up);
#pragma unroll
                for (int q = 0; q < KS / 2; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = word(v[q], i);
                        qf[2 * q + (i >> 1)][nt][i & 1] =
                            Q8 ? pack_f16x2(__uint_as_float(w << 16) * qs, __uint_as_float(w & 0xffff0000u) * qs) : w;
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i)  // the lane's columns of S^T are rows 2 cq and 2 cq + 1
                    sl[nt][i] = cc.scale_log2 * exp2_int(-__shfl_sync(0xffffffffu, up, (2 * cq + i) * 4));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    m[nt][i] = -INFINITY;
                    l[nt][i] = 0.f;
                    rv[nt][i] = exp2_int(120);
                    lv[nt][i] = 0.f;
                }
#pragma unroll
                for (int t = 0; t < KS; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][nt][i] = 0.f;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->it_empty[ii]);
        for (uint32_t unit = mine; unit < u1; unit += kWarps) {
            const uint32_t gs = unit >> 3, is = gs % kShortInfos;
            const int slab = (int)(unit & 7) * 16;
            if (!warp_wait(&c->i_full[is], (gs / kShortInfos) & 1, wf)) return;
            const int flags = c->info[is].flags;
            int base[SUB];
#pragma unroll
            for (int x = 0; x < SUB; ++x) base[x] = c->info[is].base[x];
            uint32_t tile = c->info[is].tile;
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->i_empty[is]);
            const int nx = flags & kOne ? 1 : SUB;
            uint32_t ts[2 * SUB], tn[2 * SUB];  // slots and numbers of the K and V tiles
#pragma unroll
            for (int x = 0; x < 2 * SUB; ++x) {
                // one that is not there: what the one before it holds is read and not used
                tn[x] = x % SUB >= nx ? tn[x - 1] : tile++;
                ts[x] = tn[x] % C::SLOTS;
            }
            // mostly all of the step's loads were issued by now
            const bool issued = C::LATE || __any_sync(0xffffffffu, c->loaded >= tile);
            auto landed = [&](int x) -> bool {
                return (issued || reached(&c->loaded, tn[x] + 1, wf)) &&
                       warp_wait(&c->t_full[ts[x]], (tn[x] / C::SLOTS) & 1, wf);
            };
            float s[SUB][NT][4];
            uint32_t kb[SUB][2];  // 8-bit: the scale bytes of keys g and g + 8
#pragma unroll
            for (int x = 0; x < SUB; ++x) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[x][nt][i] = 0.f;
                if (x < nx && !landed(x)) return;
            }
            if (Q8) {
                uint4 kr[SUB][2][D / 64];
#pragma unroll
                for (int x = 0; x < SUB; ++x)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        kb[x][r] = sS[ts[x] * kTile + slab + g + 8 * r];
#pragma unroll
                        for (int i = 0; i < D / 64; ++i)
                            kr[x][r][i] = *reinterpret_cast<const uint4*>(
                                chunk_at<C::ROWB>(sT + ts[x] * C::TILE, slab + g + 8 * r, (D / 64) * cq + i));
                    }
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int x = 0; x < SUB; ++x) {
                        const uint32_t w0 = word(kr[x][0][j / 4], j % 4), w1 = word(kr[x][1][j / 4], j % 4);
                        const uint32_t a[4] = {codes_f16(w0, 0), codes_f16(w1, 0), codes_f16(w0, 1), codes_f16(w1, 1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816<true>(s[x][nt], a, qf[j][nt][0], qf[j][nt][1]);
                    }
            } else {
#pragma unroll
                for (int q = 0; q < KS / 2; ++q)
#pragma unroll
                    for (int x = 0; x < SUB; ++x) {
                        uint4 kr[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            kr[r] = *reinterpret_cast<const uint4*>(chunk_at<128>(
                                sT + ts[x] * C::TILE + (q >> 1) * C::BOX, slab + g + 8 * r, 2 * cq + (q & 1)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t a[4] = {word(kr[0], 2 * i), word(kr[1], 2 * i), word(kr[0], 2 * i + 1),
                                                   word(kr[1], 2 * i + 1)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<false>(s[x][nt], a, qf[2 * q + i][nt][0], qf[2 * q + i][nt][1]);
                        }
                    }
            }
            __syncwarp();
            if (lane == 0) {
#pragma unroll
                for (int x = 0; x < SUB; ++x)
                    if (x < nx) mbar_arrive(&c->t_empty[ts[x]]);
            }
            // s[x][nt]: key g rows 2 cq, 2 cq + 1; key g + 8 the same rows
            bool grow = false;
#pragma unroll
            for (int x = 0; x < SUB; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // 2^e (a byte of an unwritten slot is hidden below, whatever comes of it)
                    const float ke = Q8 ? __uint_as_float(kb[x][i >> 1] << 23) : 1.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) s[x][nt][i] *= Q8 ? sl[nt][i & 1] * ke : sl[nt][i & 1];
                }
            if (flags & kMask) {
#pragma unroll
                for (int x = 0; x < SUB; ++x)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * nt + 2 * cq + (i & 1), key = slab + g + 8 * (i >> 1), u = base[x] + key;
                            const int pos = ctx + r / cc.G;
                            const bool see = r < rows && ((flags >> (kHaveBit + 2 * x + (key >> 6))) & 1) && u <= pos &&
                                             (cc.window <= 0 || u > pos - cc.window || u < cc.sinks);
                            if (!see) s[x][nt][i] = -INFINITY;
                        }
            }
            if (nx < SUB) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[SUB - 1][nt][i] = -INFINITY;
            }
#pragma unroll
            for (int x = 0; x < SUB; ++x)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) grow |= s[x][nt][i] > m[nt][i & 1] + 8.f;
            // the reference follows the maximum only where it grows by more than 2^8
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float top = m[nt][i];
#pragma unroll
                        for (int x = 0; x < SUB; ++x) top = fmax3(top, s[x][nt][i], s[x][nt][i + 2]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        float w = top == -INFINITY ? 1.f : ex2_approx(m[nt][i] - top);
                        m[nt][i] = top;
                        l[nt][i] *= w;
                        if (Q8) {
                            // The products met so far shrink by w too, and rv rises with that (to 2^120 at
                            // most), or what follows would be rounded against weights that are none any more.
                            lv[nt][i] *= w;
                            if (lv[nt][i] < 64.f) {
                                const int at = (int)(__float_as_uint(rv[nt][i]) >> 23) - 127, room = 120 - at;
                                const int k = lv[nt][i] > 0.f
                                                  ? min(127 + 6 - (int)(__float_as_uint(lv[nt][i]) >> 23), room)
                                                  : room;  // nothing was met yet, or nothing is left of it (w is 0)
                                const float up = exp2_int(min(k, 126));
                                w *= up;
                                lv[nt][i] *= up;
                                rv[nt][i] = exp2_int(at + k);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < KS; ++t) {
                            o[t][nt][i] *= w;
                            o[t][nt][i + 2] *= w;
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float ref = m[nt][i & 1] == -INFINITY ? 0.f : m[nt][i & 1];
#pragma unroll
                    for (int x = 0; x < SUB; ++x) {
                        s[x][nt][i] = ex2_approx(s[x][nt][i] - ref);
                        l[nt][i & 1] += s[x][nt][i];
                    }
                }
#pragma unroll
            for (int x = 0; x < SUB; ++x)
                if (x < nx && !landed(SUB + x)) return;
            if (Q8) {
                // Values are fp16 codes; their scales go into the weights: p 2^e, times a power of
                // two of the row's that keeps it below 2^15 and puts the largest one met, measured
                // against the present maximum, at 2^6 or more.  Down to 2^-20 of that one they are
                // normal numbers, rounded at 2^-11.
                float big[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) big[nt][0] = big[nt][1] = 0.f;
#pragma unroll
                for (int x = 0; x < SUB; ++x)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int key = slab + g + 8 * k;
                        uint32_t vb = sS[ts[SUB + x] * kTile + key];
                        if ((flags & kMask) &&
                            !(((flags >> (kHaveBit + 2 * x + (key >> 6))) & 1) && base[x] + key < end))
                            vb = 0;
                        const float ve = __uint_as_float((x < nx ? vb : 0u) << 23);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                s[x][nt][2 * k + i] *= ve;
                                big[nt][i] = fmaxf(big[nt][i], s[x][nt][2 * k + i]);
                            }
                    }
                bool over = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) over |= big[nt][i] * rv[nt][i] > 32768.f;
                if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float top = big[nt][i];
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                            if (!(top * rv[nt][i] > 32768.f)) continue;
                            // exponents: top's at 6 and above
                            const int was = 127 - (int)(__float_as_uint(rv[nt][i]) >> 23);
                            const int to = (int)(__float_as_uint(top) >> 23) - 127 - 6;
                            const float w = exp2_int(max(was - to, -126));
                            rv[nt][i] = exp2_int(-to);
                            lv[nt][i] = top * rv[nt][i];
#pragma unroll
                            for (int t = 0; t < KS; ++t) {
                                o[t][nt][i] *= w;
                                o[t][nt][i + 2] *= w;
                            }
                        }
                }
#pragma unroll
                for (int x = 0; x < SUB; ++x)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[x][nt][i] *= rv[nt][i & 1];
            }
            uint32_t hi[SUB][NT][2], lo[SUB][NT][2];
#pragma unroll
            for (int x = 0; x < SUB; ++x)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float a = s[x][nt][2 * k], b = s[x][nt][2 * k + 1];
                        if (Q8) {
                            hi[x][nt][k] = transpose8x8(pack_f16x2(a, b));
                        } else {
                            const uint32_t h2 = pack_bf16x2(a, b);
                            hi[x][nt][k] = transpose8x8(h2);
                            lo[x][nt][k] = transpose8x8(
                                pack_bf16x2(a - __uint_as_float(h2 << 16), b - __uint_as_float(h2 & 0xffff0000u)));
                        }
                    }
            // keys 2 cq, 2 cq + 1 and 2 cq + 8, 2 cq + 9
#pragma unroll
            for (int x = 0; x < SUB; ++x) {
                if (x >= nx) continue;
                const uint8_t* vt = sT + ts[SUB + x] * C::TILE;
                if (Q8) {
                    constexpr int W = D / 32;  // words of the lane's values in a key's row
                    uint32_t vw[4][W];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = slab + 2 * cq + 8 * (k >> 1) + (k & 1);
                        if (D == 128) {
                            const uint4 v = *reinterpret_cast<const uint4*>(chunk_at<C::ROWB>(vt, row, g));
#pragma unroll
                            for (int i = 0; i < W; ++i) vw[k][i] = word(v, i);
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(chunk_at<C::ROWB>(vt, row, g >> 1) + 8 * (g & 1));
                            vw[k][0] = v.x;
                            vw[k][1] = v.y;
                        }
                        // codes behind the last token may be NaN, and 0 * NaN is none of the sum
                        if ((flags & kMask) && base[x] + row >= end) {
#pragma unroll
                            for (int i = 0; i < W; ++i) vw[k][i] = 0;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < W; ++i)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {  // tile 2 i + t: bytes 2 t and 2 t + 1 of the word, key by key
                            uint32_t a[4];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t w = __byte_perm(vw[2 * k][i], vw[2 * k + 1][i], t ? 0x7362 : 0x5140);
                                a[2 * k] = codes_f16(w, 0);
                                a[2 * k + 1] = codes_f16(w, 1);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816<true>(o[2 * i + t][nt], a, hi[x][nt][0], hi[x][nt][1]);
                        }
                } else {
                    uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
                    if (flags & kMask) {
                        // rows behind the last token may hold NaN, and 0 * NaN is none of the sum
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int u = base[x] + slab + 2 * cq + 8 * k;
                            keep[k] = (u < end ? 0xffffu : 0u) | (u + 1 < end ? 0xffff0000u : 0u);
                        }
                    }
#pragma unroll
                    for (int bx = 0; bx < D / 64; ++bx) {
                        uint4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = *reinterpret_cast<const uint4*>(
                                chunk_at<128>(vt + bx * C::BOX, slab + 2 * cq + 8 * (k >> 1) + (k & 1), g));
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            uint32_t a[4];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t va = word(v[2 * k], t), vb = word(v[2 * k + 1], t);
                                a[2 * k] = __byte_perm(va, vb, 0x5410) & keep[k];
                                a[2 * k + 1] = __byte_perm(va, vb, 0x7632) & keep[k];
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816<false>(o[4 * bx + t][nt], a, hi[x][nt][0], hi[x][nt][1]);
                                mma16816<false>(o[4 * bx + t][nt], a, lo[x][nt][0], lo[x][nt][1]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->t_empty[ts[SUB + x]]);
            }
        }
        // The item's end: the warp's sums and accumulator go to the joining warp.
        if (!warp_wait(&c->x_empty, (items & 1) ^ 1, wf)) return;
        if (mine < u1) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
                    const int r = 8 * nt + 2 * cq + i;
                    if (g == 0) c->stats[warp][r] = make_float2(m[nt][i], l[nt][i]);
                    const float w = Q8 ? __uint_as_float((254u << 23) - __float_as_uint(rv[nt][i])) : 1.f;  // 1 / rv
                    float* dst = xch + (warp * 8 * NT + r) * C::PITCH;
#pragma unroll
                    for (int t = 0; t < KS / 2; ++t)
                        *reinterpret_cast<float4*>(dst + o_value<D, Q8>(g, t)) =
                            make_float4(w * o[2 * t][nt][i], w * o[2 * t][nt][i + 2], w * o[2 * t + 1][nt][i],
                                        w * o[2 * t + 1][nt][i + 2]);
                }
        } else if (lane < 8 * NT) {
            c->stats[warp][lane] = make_float2(-INFINITY, 0.f);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->x_full);
    }
}

// ---------------------------------------------------------------- joining warp
// One warp adds an item's parts up and writes it out, while the others are at the
// next item (all of them at it, between two barriers, and Q loaded by each warp: 96
// ragged sequences up to 8,192 slots, 8 key heads of 128, 8-bit rows 160 us; 148 so).
template <int D, bool Q8, int NT>
__device__ void short_joiner(const ShortParams& p, const float* xch, ShortCtrl* c, volatile WaitFlag* wf) {
    using C = ShortCfg<D, Q8, NT>;
    constexpr int LPR = D / 4;  // lanes of a row
    const ChunkCommon& cc = p.c;
    const int lane = threadIdx.x & 31, d = lane % LPR * 4;
    for (uint32_t items = 0;; ++items) {
        const uint32_t ii = items % kShortItems;
        if (!warp_wait(&c->it_full[ii], (items / kShortItems) & 1, wf)) return;
        const ShortItem it = c->item[ii];
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->it_empty[ii]);
        if (it.steps < 0) return;
        if (!warp_wait(&c->x_full, items & 1, wf)) return;
        for (int r = lane / LPR; r < it.rows; r += 32 / LPR) {
            float2 ml[kWarps];
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = c->stats[w][r];
                top = fmaxf(top, ml[w].x);
            }
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (ml[w].x == -INFINITY) continue;  // saw nothing of the row
                const float f = ex2_approx(ml[w].x - top);
                sum += f * ml[w].y;
                const float4 a = *reinterpret_cast<const float4*>(xch + (w * 8 * NT + r) * C::PITCH + d);
                v.x += f * a.x;
                v.y += f * a.y;
                v.z += f * a.z;
                v.w += f * a.w;
            }
            if (it.part < 0) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int64_t orow = (int64_t)(it.row0 + r / cc.G) * cc.Hq + it.h * cc.G + r % cc.G;
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(cc.out) + orow * D + d) =
                    make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                if (d == 0) cc.lse[orow] = lse_of(top, sum);
            } else {
                const int64_t prow = (int64_t)it.part * kShortRows + r;
                *reinterpret_cast<float4*>(p.part_o + prow * D + d) = v;
                if (d == 0) p.part_ml[prow] = make_float2(top, sum);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->x_empty);
    }
}

// ---------------------------------------------------------------- kernel
template <int D, bool Q8, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    short_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const ShortParams p) {
    using C = ShortCfg<D, Q8, NT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {
        griddep_wait();
        if (threadIdx.x == 0) {
            p.meta[blockIdx.x].start = -1;
            atomicOr(p.c.err, ERR_LAUNCH);
        }
        return;
    }
    uint8_t* sT = smem;
    float* xch = reinterpret_cast<float*>(sT + C::SLOTS * C::TILE);
    uint8_t* sS = reinterpret_cast<uint8_t*>(xch) + C::XCH;
    __nv_bfloat16* sQ = reinterpret_cast<__nv_bfloat16*>(sS + (Q8 ? kShortMaxSlots * kTile : 0));
    ShortCtrl* c = reinterpret_cast<ShortCtrl*>(reinterpret_cast<uint8_t*>(sQ) + C::QBUF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    {
        const int x = threadIdx.x;
        if (x < kShortMaxSlots) {
            mbar_init(&c->t_full[x], 1);
            mbar_init(&c->t_empty[x], 8);  // a warp for each of its units
        } else if (x < kShortMaxSlots + kShortInfos) {
            mbar_init(&c->i_full[x - kShortMaxSlots], 1);
            mbar_init(&c->i_empty[x - kShortMaxSlots], 8);
        } else if (x < kShortMaxSlots + kShortInfos + kShortItems) {
            mbar_init(&c->it_full[x - kShortMaxSlots - kShortInfos], 1);
            mbar_init(&c->it_empty[x - kShortMaxSlots - kShortInfos], kWarps + 1);  // and the joining warp
        } else if (x == 32) {
            mbar_init(&c->x_full, kWarps);
            mbar_init(&c->x_empty, 1);
            c->wf.abort = 0;
            c->wf.limit_ns = p.c.wait_limit_ns;
            c->loaded = 0;
            c->prefix[0] = 0;
        }
        fence_mbar_init();
    }
    if (warp == kProducer && lane == 0) {
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    // Nothing before this line reads or writes global memory.
    griddep_wait();
    // prefix sums of the sequences' steps per item: every thread a run of them, then a scan
    const int run = (p.units + kThreads - 1) / kThreads;
    const int u0 = min(p.units, (int)threadIdx.x * run), u1 = min(p.units, u0 + run);
    auto sums = [&](int sub, bool report) {
        int sum = 0;
        for (int u = u0; u < u1; ++u) {
            sum += short_steps(p.c, p.unit0 + u, sub, report);
            c->prefix[u + 1] = sum;
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) c->red[warp] = incl;
        __syncthreads();
        const int before = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? c->red[lane] : 0);
        for (int u = u0; u < u1; ++u) c->prefix[u + 1] += before;
        __syncthreads();
    };
    int sub = C::SUB;
    sums(sub, blockIdx.x == 0);
    if (C::SUB > 1 && 2 * (int64_t)c->prefix[p.units] * p.c.Hkv <= (int)gridDim.x) {
        // fewer steps than half of the SMs: single tiles
        __syncthreads();
        sub = 1;
        sums(sub, false);
    }
    const int total = c->prefix[p.units] * p.c.Hkv;
    const int per = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    const int lo = min(total, (int)blockIdx.x * per), hi = min(total, lo + per);
    volatile WaitFlag* wf = &c->wf;
    if (warp == kProducer)
        short_producer<D, Q8, NT>(&tk, &tv, p, sT, sS, sQ, c, lo, hi, per, sub, wf);
    else if (warp == kJoiner)
        short_joiner<D, Q8, NT>(p, xch, c, wf);
    else
        short_consumer<D, Q8, NT>(p, sT, sS, sQ, xch, c, wf);
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && c->wf.abort) atomicOr(p.c.err, ERR_TIMEOUT);
}

template <int D, bool Q8, int NT>
int go(const ShortLaunch& L, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    using C = ShortCfg<D, Q8, NT>;
    static std::atomic<uint64_t> raised{0};
    if (raise_smem_limit(reinterpret_cast<const void*>(short_kernel<D, Q8, NT>), C::SMEM, &raised) != cudaSuccess)
        return BSA_ERR_CUDA;
    ShortParams p{};
    p.c = L.c;
    p.q = static_cast<const __nv_bfloat16*>(L.q);
    p.n_slots = C::SLOTS;
    p.meta = L.meta;
    p.part_o = L.part_o;
    p.part_ml = L.part_ml;
    // the steps of one launch stay below 2^30 (sums and range ends fit an int)
    const int64_t most = (((int64_t)L.c.P * L.c.page + kTile - 1) / kTile) * L.c.Hkv;
    const int chunk = (int)std::min<int64_t>(kShortUnits, std::max<int64_t>(1, (1 << 30) / most));
    const int ctas = std::min(L.sms, kChunkMaxCtas);
    for (int u0 = 0; u0 < L.c.B; u0 += chunk) {
        p.unit0 = u0;
        p.units = std::min(chunk, L.c.B - u0);
        cudaError_t e = launch_after(short_kernel<D, Q8, NT>, dim3((unsigned)ctas), kThreads, C::SMEM, s, tk, tv, p);
        if (e != cudaSuccess) return BSA_ERR_CUDA;
        if (ctas < 2 || (!L.merge && u0 + chunk >= L.c.B)) continue;
        const PartSet few{p.meta, p.part_o, p.part_ml};
        e = launch_after(chunk_merge_kernel<D>, dim3((unsigned)ctas - 1, (unsigned)(8 * NT)), 256, 0, s, p.c, few,
                         PartSet{}, 8 * NT, 0);
        if (e != cudaSuccess) return BSA_ERR_CUDA;
    }
    return BSA_OK;
}

}  // namespace

int launch_short(const ShortLaunch& L, cudaStream_t s) {
    const bool q8 = L.c.ks != nullptr;
    const uint64_t krows = (uint64_t)L.c.n_pages * L.c.Hkv * L.c.page;
    auto encode = q8 ? encode_rows_e4m3 : encode_rows_bf16;
    CUtensorMap tk, tv;
    int st;
    if ((st = encode(&tk, L.k, krows, L.D, L.c.page)) != BSA_OK) return st;
    if ((st = encode(&tv, L.v, krows, L.D, L.c.page)) != BSA_OK) return st;
    const bool one = short_rows(L.c) == 8;  // one 8-column tile of query rows
    if (L.D == 128)
        return one ? (q8 ? go<128, true, 1>(L, tk, tv, s) : go<128, false, 1>(L, tk, tv, s))
                   : (q8 ? go<128, true, 2>(L, tk, tv, s) : go<128, false, 2>(L, tk, tv, s));
    return one ? (q8 ? go<64, true, 1>(L, tk, tv, s) : go<64, false, 1>(L, tk, tv, s))
               : (q8 ? go<64, true, 2>(L, tk, tv, s) : go<64, false, 2>(L, tk, tv, s));
}

}  // namespace bsa
