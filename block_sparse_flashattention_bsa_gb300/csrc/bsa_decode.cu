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
// Work: a step is 128 slots; an item the steps of one key head of one sequence;
// the steps of the batch, cut into equal ranges, one per CTA.  An item that a
// range boundary cuts leaves unnormalised fp32 parts that the merge joins in range
// order: no atomics, results do not depend on timing.
//
// One CTA per SM: a producer warp walks the range, resolves pages and TMA-loads K
// and V tiles into a ring; NW consumer warps, each with 16 keys of a step, a
// running maximum, sum and accumulator of its own (so steps need no exchange), and
// with 16 warps two steps at a time.  At an item's end the warps meet in shared
// memory.  P is multiplied as two bf16 parts, high and low, so that its rounding
// (2^-17) does not add to the result's.

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

enum : int { kFirst = 1, kLast = 2, kMask = 4, kEnd = 8 };

struct ShortInfo {
    int flags, step;    // step of the item
    int base, have;     // first slot; halves that lie in a page
    int row0, rows, h;  // first token, query rows, key head
    int ctx, end;       // slot of the first new token, slot behind the last one
    int part;           // -1: write the output, else the partial slot
};

struct ShortCtrl {
    uint64_t t_full[kShortMaxSlots], t_empty[kShortMaxSlots];
    uint64_t i_empty[kShortMaxSlots / 2];
    uint64_t st_full, x_full;  // all consumers posted their sums, their parts of O
    ShortInfo info[kShortMaxSlots / 2];
    float2 stats[16][16];      // [warp][row]; 8 warps x 16 rows or 16 x 8 are used
    int red[18];
    WaitFlag wf;
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
    static constexpr int NW = NT == 1 ? 16 : 8;       // consumer warps
    static constexpr int THREADS = (NW + 1) * 32;
    static constexpr int ROWB = Q8 ? D : 128;         // bytes of a row of a box
    static constexpr int NBOX = Q8 ? 1 : D / 64;
    static constexpr int BOX = kTile * ROWB;
    static constexpr int TILE = NBOX * BOX;
    static constexpr int PITCH = D + 4;               // floats of an exchanged row
    static constexpr int XCH = NW * 8 * NT * PITCH * 4;
    static constexpr int FIXED = XCH + kShortCtrl + (Q8 ? kShortMaxSlots * kTile : 0);
    static constexpr int FIT = (kShortSmem - FIXED) / TILE;
    static constexpr int SLOTS = FIT > kShortMaxSlots ? kShortMaxSlots : FIT;
    static constexpr int SMEM = SLOTS * TILE + FIXED;
    static_assert(SLOTS >= 4, "ring too small");
};

// Steps of a short sequence's item; 0: it has no new tokens or is not short.
__device__ __forceinline__ int short_steps(const ChunkCommon& p, int b, bool report) {
    const Seq s = sequence(p, b, report);
    if (s.n == 0 || s.n * (int64_t)p.G > kShortRows) return 0;
    return visible_span(p, s.ctx, s.ctx + s.n).steps;
}

// ---------------------------------------------------------------- producer
template <int D, bool Q8, int NT>
__device__ void short_producer(const CUtensorMap* tk, const CUtensorMap* tv, const ShortParams& p, uint8_t* sT,
                               uint8_t* sS, ShortCtrl* c, int lo, int hi, int per, volatile WaitFlag* wf) {
    using C = ShortCfg<D, Q8, NT>;
    const ChunkCommon& cc = p.c;
    const int lane = threadIdx.x & 31, Hkv = cc.Hkv, ppt = kTile / cc.page;
    const bool leader = elect_one();
    const uint32_t infos = (uint32_t)p.n_slots / 2;
    uint32_t slot = 0, phase = 0, nload = 0, g = 0;
    bool ok = true, ended = false;
    PartMeta mt{-1, 0, per, 0, 0, 0, {0, 0}};
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
            for (int e0 = s0 * ppt; e0 < s1 * ppt && ok; e0 += 32) {
                // 32 pages resolved at a time
                const int e = e0 + lane, est = e / ppt;
                const int j = sp.tile(est) * ppt + e % ppt;
                const int y = est < s1 ? page_row(cc, b, h, j, vis0, seq_end) : -1;
                const int cnt = min(32, s1 * ppt - e0);
                for (int q = 0; q < cnt && ok; q += ppt) {
                    const int st = (e0 + q) / ppt;
                    const int y0 = __shfl_sync(0xffffffffu, y, q), y1 = __shfl_sync(0xffffffffu, y, q + ppt - 1);
                    const uint32_t is = g % infos;
                    if (g >= infos && !warp_wait(&c->i_empty[is], ((g / infos) & 1) ^ 1, wf)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        ShortInfo& f = c->info[is];
                        const int first = sp.tile(st) * kTile;
                        const int have = ppt == 1 ? (y0 >= 0 ? 3 : 0) : (y0 >= 0 ? 1 : 0) | (y1 >= 0 ? 2 : 0);
                        // every row sees all of it: up to the first token, inside the last one's window
                        const bool plain = have == 3 && first + kTile <= sq.ctx + 1 &&
                                           (cc.window <= 0 || first > seq_end - 1 - cc.window ||
                                            first + kTile <= cc.sinks);
                        f.flags = (st == s0 ? kFirst : 0) | (st + 1 == s1 ? kLast : 0) | (plain ? 0 : kMask);
                        f.step = st - s0;
                        f.base = first;
                        f.have = have;
                        f.row0 = sq.row0;
                        f.rows = sq.n * cc.G;
                        f.h = h;
                        f.ctx = sq.ctx;
                        f.end = seq_end;
                        f.part = part;
                    }
                    __syncwarp();
                    ++g;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (nload >= (uint32_t)p.n_slots && !warp_wait(&c->t_empty[slot], phase ^ 1, wf)) {
                            ok = false;
                            break;
                        }
                        if (leader) {
                            uint64_t* bar = &c->t_full[slot];
                            const uint8_t* sc = kv ? cc.vs : cc.ks;
                            uint32_t bytes = C::TILE;
                            if (Q8) bytes += (y0 >= 0 ? cc.page : 0) + (ppt == 2 && y1 >= 0 ? cc.page : 0);
                            mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
                            for (int x = 0; x < C::NBOX; ++x) {
                                uint8_t* dst = sT + slot * C::TILE + x * C::BOX;
                                tma_load_2d(dst, kv ? tv : tk, bar, x * 64, y0 >= 0 ? y0 : -cc.page);
                                if (ppt == 2)
                                    tma_load_2d(dst + 64 * C::ROWB, kv ? tv : tk, bar, x * 64, y1 >= 0 ? y1 : -cc.page);
                            }
                            if (Q8) {
                                if (y0 >= 0) bulk_load(sS + slot * kTile, sc + y0, cc.page, bar);
                                if (ppt == 2 && y1 >= 0) bulk_load(sS + slot * kTile + 64, sc + y1, cc.page, bar);
                            }
                        }
                        ++nload;
                        if (++slot == (uint32_t)p.n_slots) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
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
    if (ok) {
        // the end mark, with a slot's barrier
        const uint32_t is = g % infos;
        if ((g < infos || warp_wait(&c->i_empty[is], ((g / infos) & 1) ^ 1, wf)) &&
            (nload < (uint32_t)p.n_slots || warp_wait(&c->t_empty[slot], phase ^ 1, wf)) && leader) {
            c->info[is].flags = kEnd;
            mbar_arrive(&c->t_full[slot]);
            ended = true;
        }
    }
    if (lane == 0) p.meta[blockIdx.x] = mt;
    __syncwarp();
    if (leader) {
        // copies still in flight must land before the CTA exits (the end mark used
        // the slot of the oldest one, which was consumed before)
        const uint32_t ns = (uint32_t)p.n_slots;
        const uint32_t from = nload > ns ? nload - ns : 0;
        for (uint32_t n = from; n < nload; ++n) {
            if (ended && n % ns == nload % ns) continue;
            mbar_wait_drain(&c->t_full[n % ns], (n / ns) & 1);
        }
    }
}

// ---------------------------------------------------------------- consumers
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ void short_consumer(const ShortParams& p, const uint8_t* sT, const uint8_t* sS, float* xch, ShortCtrl* c,
                               volatile WaitFlag* wf) {
    using C = ShortCfg<D, Q8, NT>;
    constexpr int KS = D / 16;
    const ChunkCommon& cc = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, cq = lane & 3;
    const int slab = (warp & 7) * 16, group = warp >> 3;
    const uint32_t infos = (uint32_t)p.n_slots / 2;
    uint32_t qf[KS][NT][2];
    float o[KS][NT][4];
    float m[NT][2], l[NT][2];
    uint32_t slot = 0, phase = 0, items = 0;
    auto next = [&](uint32_t& s, uint32_t& ph) {
        if (++s == (uint32_t)p.n_slots) {
            s = 0;
            ph ^= 1;
        }
    };
    for (uint32_t gs = 0;; ++gs) {
        if (!warp_wait(&c->t_full[slot], phase, wf)) return;
        const uint32_t is = gs % infos;
        const ShortInfo f = c->info[is];
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->i_empty[is]);
        if (f.flags & kEnd) return;
        const uint32_t kslot = slot;
        next(slot, phase);
        const uint32_t vslot = slot, vphase = phase;
        next(slot, phase);
        if (f.flags & kFirst) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = 8 * nt + g;
                const bool on = r < f.rows;
                const __nv_bfloat16* src =
                    p.q + ((int64_t)(f.row0 + (on ? r / cc.G : 0)) * cc.Hq + f.h * cc.G + (on ? r % cc.G : 0)) * D;
#pragma unroll
                for (int q = 0; q < KS / 2; ++q) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (on) v = *reinterpret_cast<const uint4*>(src + q_chunk<D, Q8>(cq, q));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a = word(v, 2 * i), b = word(v, 2 * i + 1);
                        qf[2 * q + i][nt][0] = Q8 ? __byte_perm(a, b, 0x5410) : a;
                        qf[2 * q + i][nt][1] = Q8 ? __byte_perm(a, b, 0x7632) : b;
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    m[nt][i] = -INFINITY;
                    l[nt][i] = 0.f;
                }
#pragma unroll
                for (int t = 0; t < KS; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][nt][i] = 0.f;
            }
        }
        if (C::NW == 8 || (f.step & 1) == group) {
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
            const uint8_t* kt = sT + kslot * C::TILE;
            if (Q8) {
                uint32_t f1[2], f2_[2];
                bool two = false;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t e = sS[kslot * kTile + slab + g + 8 * r];
                    f1[r] = scale_first(e) * 0x10001u;
                    f2_[r] = scale_rest(e) * 0x10001u;
                    two |= e > kOneStep;
                }
                two = __any_sync(0xffffffffu, two);
                uint4 kr[2][D / 64];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        kr[r][x] = *reinterpret_cast<const uint4*>(
                            chunk_at<C::ROWB>(kt, slab + g + 8 * r, (D / 64) * cq + x));
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    uint32_t a[4];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t w = word(kr[r][j / 4], j % 4);
                        a[r] = mul_bf16x2(spread_even(w), f1[r]);
                        a[2 + r] = mul_bf16x2(spread_odd(w), f1[r]);
                        if (two) {
                            a[r] = mul_bf16x2(a[r], f2_[r]);
                            a[2 + r] = mul_bf16x2(a[2 + r], f2_[r]);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a, qf[j][nt][0], qf[j][nt][1]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < KS / 2; ++q) {
                    uint4 kr[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        kr[r] = *reinterpret_cast<const uint4*>(
                            chunk_at<128>(kt + (q >> 1) * C::BOX, slab + g + 8 * r, 2 * cq + (q & 1)));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a[4] = {word(kr[0], 2 * i), word(kr[1], 2 * i), word(kr[0], 2 * i + 1),
                                               word(kr[1], 2 * i + 1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a, qf[2 * q + i][nt][0], qf[2 * q + i][nt][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->t_empty[kslot]);
            // s[nt]: key g rows 2 cq, 2 cq + 1; key g + 8 the same rows
            uint32_t hi[NT][2], lo[NT][2];
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[nt][i] *= cc.scale_log2;
                    if (f.flags & kMask) {
                        const int r = 8 * nt + 2 * cq + (i & 1), key = slab + g + 8 * (i >> 1), u = f.base + key;
                        const int pos = f.ctx + r / cc.G;
                        const bool see = r < f.rows && ((f.have >> (key >> 6)) & 1) && u <= pos &&
                                         (cc.window <= 0 || u > pos - cc.window || u < cc.sinks);
                        if (!see) s[nt][i] = -INFINITY;
                    }
                    grow |= s[nt][i] > m[nt][i & 1] + 8.f;
                }
            // the reference follows the maximum only where it grows by more than 2^8
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = fmaxf(s[nt][i], s[nt][i + 2]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        x = fmaxf(x, m[nt][i]);
                        const float w = x == -INFINITY ? 1.f : ex2_approx(m[nt][i] - x);
                        m[nt][i] = x;
                        l[nt][i] *= w;
#pragma unroll
                        for (int t = 0; t < KS; ++t) {
                            o[t][nt][i] *= w;
                            o[t][nt][i + 2] *= w;
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float ref = m[nt][i & 1] == -INFINITY ? 0.f : m[nt][i & 1];
                    e[i] = ex2_approx(s[nt][i] - ref);
                    l[nt][i & 1] += e[i];
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t h2 = pack_bf16x2(e[2 * k], e[2 * k + 1]);
                    const uint32_t l2 = pack_bf16x2(e[2 * k] - __uint_as_float(h2 << 16),
                                                    e[2 * k + 1] - __uint_as_float(h2 & 0xffff0000u));
                    hi[nt][k] = transpose8x8(h2);
                    lo[nt][k] = transpose8x8(l2);
                }
            }
            if (!warp_wait(&c->t_full[vslot], vphase, wf)) return;
            const uint8_t* vt = sT + vslot * C::TILE;
            // keys 2 cq, 2 cq + 1 and 2 cq + 8, 2 cq + 9
            if (Q8) {
                constexpr int W = D / 32;  // words of the lane's values in a key's row
                uint32_t f1[2], f2_[2];
                bool two = false;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t ea = sS[vslot * kTile + slab + 2 * cq + 8 * k];
                    const uint32_t eb = sS[vslot * kTile + slab + 2 * cq + 8 * k + 1];
                    f1[k] = scale_first(ea) | scale_first(eb) << 16;
                    f2_[k] = scale_rest(ea) | scale_rest(eb) << 16;
                    two |= ea > kOneStep || eb > kOneStep;
                }
                two = __any_sync(0xffffffffu, two);
                uint32_t vw[4][W];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = slab + 2 * cq + 8 * (k >> 1) + (k & 1);
                    if (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4*>(chunk_at<C::ROWB>(vt, row, g));
#pragma unroll
                        for (int x = 0; x < W; ++x) vw[k][x] = word(v, x);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(chunk_at<C::ROWB>(vt, row, g >> 1) + 8 * (g & 1));
                        vw[k][0] = v.x;
                        vw[k][1] = v.y;
                    }
                }
#pragma unroll
                for (int x = 0; x < W; ++x)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {  // tile 2 x + t: bytes 2 t and 2 t + 1 of the word
                        uint32_t a[4];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int by = 2 * t + r;
                                const uint32_t two_keys =
                                    __byte_perm(vw[2 * k][x], vw[2 * k + 1][x], (4 + by) << 12 | by << 4);
                                uint32_t v = mul_bf16x2(spread_odd(two_keys), f1[k]);
                                if (two) v = mul_bf16x2(v, f2_[k]);
                                a[r + 2 * k] = v;
                            }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816(o[2 * x + t][nt], a, hi[nt][0], hi[nt][1]);
                            mma16816(o[2 * x + t][nt], a, lo[nt][0], lo[nt][1]);
                        }
                    }
            } else {
                uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
                if (f.flags & kMask) {
                    // rows behind the last token may hold NaN, and 0 * NaN is none of the sum
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int u = f.base + slab + 2 * cq + 8 * k;
                        keep[k] = (u < f.end ? 0xffffu : 0u) | (u + 1 < f.end ? 0xffff0000u : 0u);
                    }
                }
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    uint4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[k] = *reinterpret_cast<const uint4*>(
                            chunk_at<128>(vt + x * C::BOX, slab + 2 * cq + 8 * (k >> 1) + (k & 1), g));
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
                            mma16816(o[4 * x + t][nt], a, hi[nt][0], hi[nt][1]);
                            mma16816(o[4 * x + t][nt], a, lo[nt][0], lo[nt][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->t_empty[vslot]);
        }
        if (!(f.flags & kLast)) continue;
        // The item's end: all warps' sums and accumulators meet.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
                if (g == 0) c->stats[warp][8 * nt + 2 * cq + i] = make_float2(m[nt][i], l[nt][i]);
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->st_full);
        if (!warp_wait(&c->st_full, items & 1, wf)) return;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * nt + 2 * cq + i;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < C::NW; ++w) top = fmaxf(top, c->stats[w][r].x);
                const float w = top == -INFINITY ? 0.f : ex2_approx(m[nt][i] - top);
                float* dst = xch + (warp * 8 * NT + r) * C::PITCH;
#pragma unroll
                for (int t = 0; t < KS / 2; ++t)
                    *reinterpret_cast<float4*>(dst + o_value<D, Q8>(g, t)) =
                        make_float4(w * o[2 * t][nt][i], w * o[2 * t][nt][i + 2], w * o[2 * t + 1][nt][i],
                                    w * o[2 * t + 1][nt][i + 2]);
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->x_full);
        if (!warp_wait(&c->x_full, items & 1, wf)) return;
        ++items;
        for (int x = threadIdx.x; x < f.rows * (D / 4); x += C::NW * 32) {
            const int r = x / (D / 4), d = x % (D / 4) * 4;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < C::NW; ++w) top = fmaxf(top, c->stats[w][r].x);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < C::NW; ++w) {
                const float2 ml = c->stats[w][r];
                if (top > -INFINITY) sum += ex2_approx(ml.x - top) * ml.y;
                const float4 a = *reinterpret_cast<const float4*>(xch + (w * 8 * NT + r) * C::PITCH + d);
                v.x += a.x;
                v.y += a.y;
                v.z += a.z;
                v.w += a.w;
            }
            if (f.part < 0) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int64_t orow = (int64_t)(f.row0 + r / cc.G) * cc.Hq + f.h * cc.G + r % cc.G;
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(cc.out) + orow * D + d) =
                    make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                if (d == 0) cc.lse[orow] = lse_of(top, sum);
            } else {
                const int64_t prow = (int64_t)f.part * kShortRows + r;
                *reinterpret_cast<float4*>(p.part_o + prow * D + d) = v;
                if (d == 0) p.part_ml[prow] = make_float2(top, sum);
            }
        }
    }
}

// ---------------------------------------------------------------- kernel
template <int D, bool Q8, int NT>
__global__ void __launch_bounds__(ShortCfg<D, Q8, NT>::THREADS, 1)
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
    ShortCtrl* c = reinterpret_cast<ShortCtrl*>(sS + (Q8 ? kShortMaxSlots * kTile : 0));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    {
        const int x = threadIdx.x;
        if (x < kShortMaxSlots) {
            mbar_init(&c->t_full[x], 1);
            mbar_init(&c->t_empty[x], 8);  // the eight warps whose step it is
        } else if (x < kShortMaxSlots + kShortMaxSlots / 2) {
            mbar_init(&c->i_empty[x - kShortMaxSlots], C::NW);
        } else if (x == 32) {
            mbar_init(&c->st_full, C::NW);
            mbar_init(&c->x_full, C::NW);
            c->wf.abort = 0;
            c->wf.limit_ns = p.c.wait_limit_ns;
            c->prefix[0] = 0;
        }
        fence_mbar_init();
    }
    if (warp == C::NW && lane == 0) {
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    // Nothing before this line reads or writes global memory.
    griddep_wait();
    // prefix sums of the sequences' steps per item: every thread a run of them, then a scan
    const int run = (p.units + C::THREADS - 1) / C::THREADS;
    const int u0 = min(p.units, (int)threadIdx.x * run), u1 = min(p.units, u0 + run);
    int sum = 0;
    for (int u = u0; u < u1; ++u) {
        sum += short_steps(p.c, p.unit0 + u, blockIdx.x == 0);
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
    const int total = c->prefix[p.units] * p.c.Hkv;
    const int per = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    const int lo = min(total, (int)blockIdx.x * per), hi = min(total, lo + per);
    volatile WaitFlag* wf = &c->wf;
    if (warp == C::NW)
        short_producer<D, Q8, NT>(&tk, &tv, p, sT, sS, c, lo, hi, per, wf);
    else
        short_consumer<D, Q8, NT>(p, sT, sS, xch, c, wf);
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
        cudaError_t e = launch_after(short_kernel<D, Q8, NT>, dim3((unsigned)ctas), C::THREADS, C::SMEM, s, tk, tv, p);
        if (e != cudaSuccess) return BSA_ERR_CUDA;
        if (ctas < 2) continue;
        e = launch_after(chunk_merge_kernel<D, kShortRows, 1>, dim3((unsigned)ctas - 1, (unsigned)(8 * NT)), 256, 0, s,
                         p.c, p.meta, p.part_o, p.part_ml, 128);
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
    // one 8-column tile of query rows where no short sequence can have more
    const bool one = L.c.G <= 8 && (!L.c.q_ptr || (int64_t)L.c.tokens * L.c.G <= 8);
    if (L.D == 128)
        return one ? (q8 ? go<128, true, 1>(L, tk, tv, s) : go<128, false, 1>(L, tk, tv, s))
                   : (q8 ? go<128, true, 2>(L, tk, tv, s) : go<128, false, 2>(L, tk, tv, s));
    return one ? (q8 ? go<64, true, 1>(L, tk, tv, s) : go<64, false, 1>(L, tk, tv, s))
               : (q8 ? go<64, true, 2>(L, tk, tv, s) : go<64, false, 2>(L, tk, tv, s));
}

}  // namespace bsa
