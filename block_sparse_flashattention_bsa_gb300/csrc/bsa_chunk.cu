// bsa_chunk.cu -- attention of chunks of new tokens over a paged cache (a prompt
// behind a cached prefix, ragged batches), over all slots or a sliding window with
// sinks, bf16 or 8-bit pools.
//
// Mathematics: O = softmax(q K^T scale) V over the slots u <= s a token in slot s
// sees (with a window w: u > s - w or u < sinks), in one pass over the slots with
// the running maximum and sum of the softmax.  The G query heads of a key head are
// rows of the same tile: row t * G + g is head g of the tile's token t.
//
// What it cannot do without: 4 D flops for every (row, slot) pair on the tensor cores,
// beside them an exponential a pair and, for 8-bit rows, the conversions.  None of these
// fills a step (two tiles of 128 rows, 128 slots): it takes 3,060 cycles with 128-wide bf16
// rows (tensor pipe 65 %, exponentials 33 %) and 2,700 with 64-wide ones (26 %, 26 %, issue
// slots 49 %); what it waits for has not been found.
//
// Work: an item is two tiles of 128 rows of one key head of one sequence (both
// tiles use every K / V tile that is loaded); a step 128 slots.  The steps of the
// whole batch are cut into equal ranges, one per CTA, so that one long chunk loads
// the SMs as evenly as many short ones.  Items that a range boundary cuts leave unnormalised fp32
// parts, which the merge joins in range order: results do not depend on timing.
//
// One CTA per SM:
//   warps 0-3, 4-7  softmax of tile A, B: thread = row (TMEM lane).  S in
//              registers, P back over it in bf16.  O is rescaled in TMEM only when
//              the maximum grows by more than 2^8.
//   warp 8     producer: walks the range, resolves pages, TMA-loads K / V tiles;
//              bf16: zeroes V rows behind the last token (they may hold NaN)
//   warps 9, 10  MMA of tile A, B: S = Q K^T and O += P V on tcgen05, 64 slots at a
//              time, two S buffers to a tile: a tile's scores are two halves of a step
//              ahead of its product
//   warp 11    loads an item's Q tiles as soon as the item before has used its own
//   warps 12-19  8-bit: convert tiles to bf16 (code * 2^e, exact)

#include <algorithm>
#include <cmath>

#include "bsa.h"
#include "bsa_chunk.cuh"
#include "bsa_q8.cuh"

namespace bsa {
namespace {

constexpr int kSmem = 232448;
constexpr int kCtrl = 2560;
constexpr int kInfos = 4;
constexpr int kQAhead = 4;
constexpr int kMaxTiles = 16;
constexpr int kHalf = 64;     // key slots of a tile: half of a step
constexpr int kProducer = 8, kMma = 9, kQLoader = 11, kConverter = 12;
constexpr int kRows = 256;  // rows of an item

enum : int { kFirst = 1, kLast = 2, kMask = 4, kEnd = 8, kFix = 16 };

struct StepInfo {
    int flags;
    int base, have;      // first slot; halves that lie in a page
    int row0, n, h;      // first token (row of q), tokens, key head of the item
    int pos0, end;       // slot of its first token, slot behind the sequence's last one
    int part;            // -1: write the output, else the partial slot
};

// Tiles of 64 slots are loaded in the order in which the products take them, x
// counting halves of steps: K(0) K(1) V(0) K(2) V(1) K(3) ..., so that a V tile takes
// no room long before its turn (K and V of whole steps left 64 KB of loads in
// flight, a step of 3,100 cycles whatever the products and the softmax took).
__device__ __forceinline__ uint32_t v_tile(uint32_t x) { return 2 * x + 2; }  // their numbers in that order
__device__ __forceinline__ uint32_t k_tile(uint32_t x) { return x < 2 ? x : 2 * x - 1; }

struct Place {
    int b, h, i;          // sequence, key head, group
    int head, cum;        // steps of one of its key heads; of the head's groups before this one
    int start;            // first step of the item
};

struct Ctrl {
    uint64_t t_full[kMaxTiles], t_empty[kMaxTiles];   // bf16 tiles
    uint64_t r_full[kMaxTiles], r_empty[kMaxTiles];   // 8-bit tiles
    uint64_t q_full[2], q_empty[2];
    uint64_t qi_full[kQAhead], qi_empty[kQAhead];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [tile][half of a step]
    uint64_t o_full[2];
    uint64_t i_full[kInfos], i_empty[kInfos];
    uint64_t fix_full[kInfos][2], drain[2];  // fix_full: a half's V rows behind the last token are zeros
    volatile uint32_t issued;        // steps the producer has issued
    volatile uint32_t first[2];      // 8-bit: halves of K(0) that are converted
    int2 qitem[kQAhead];             // first query head and token of an item; x < 0: no more
    StepInfo info[kInfos];
    uint32_t tmem_base;
    WaitFlag wf;
    Place place;                     // where the CTA's range starts
    long long sums[32];
};
static_assert(sizeof(Ctrl) <= kCtrl, "control block too large");

struct ChunkParams {
    ChunkCommon c;
    int32_t tq;                // tokens of a tile
    int32_t least;             // sequences of fewer query rows of a key head are not worked on
    PartMeta* meta;
    float* part_o;             // [2 * grid][D / 4][256][4]
    float2* part_ml;           // [2 * grid][256]
};

template <int D, bool Q8>
struct Cfg {
    static constexpr int THREADS = Q8 ? 640 : 512;
    static constexpr int CONV = 2;                     // converting warps of a tile
    static constexpr int NBOX = D / 64;
    static constexpr int QBOX = 128 * 128, QTILE = NBOX * QBOX;
    static constexpr int BOX = kHalf * 128, TILE = NBOX * BOX;
    static constexpr int RAW = kHalf * D;              // an 8-bit tile
    static constexpr int FREE = kSmem - kCtrl - 2 * QTILE;
    // 8-bit: eight bf16 tiles, the rest holds what is in flight; both in fours, so that
    // a slot's tiles are all converted by the same two warps
    static constexpr int RAWFIT = (FREE - 8 * TILE) / (RAW + kHalf) / 4 * 4;
    static constexpr int NRAW = !Q8 ? 0 : RAWFIT > kMaxTiles ? kMaxTiles : RAWFIT;
    static constexpr int NT = Q8 ? 8 : FREE / TILE > kMaxTiles ? kMaxTiles : FREE / TILE;
    // Finished rows on their way out, 128 bytes of each of a warp's 32 rows, for stores of whole
    // lines: an item's end 1.1 us, straight from the lanes 1.5.  Rows of 128 values leave no
    // room for it.
    static constexpr int STAGE = D == 64 ? 8 * 32 * 128 : 0;
    static constexpr int SMEM = 2 * QTILE + NT * TILE + NRAW * (RAW + kHalf) + STAGE + kCtrl;
    static constexpr int O_COL = 2 * kTile;
    static_assert(SMEM <= kSmem && NT >= 6 && (!Q8 || NRAW >= 4), "shared memory");
};

// ---------------------------------------------------------------- plan
// An item's place in the order of all steps: sequences, their key heads, their
// groups of two tiles of tokens.  Every CTA works out for itself where its range
// starts (a kernel that listed the items for all: 5 us in front of this one).

// Groups of sequence s; 0: it is not worked on here.
__device__ __forceinline__ int group_count(const ChunkParams& p, const Seq& s) {
    return s.n * (int64_t)p.c.G < p.least ? 0 : (s.n + 2 * p.tq - 1) / (2 * p.tq);
}
// Steps of group i, and one for its end, which takes about as long (with windows of ten
// steps to an item the last CTA was 6 % behind the others without it).
__device__ __forceinline__ int group_steps(const ChunkParams& p, const Seq& s, int i) {
    const int t0 = i * 2 * p.tq;
    return visible_span(p.c, s.ctx + t0, s.ctx + min(s.n, t0 + 2 * p.tq)).steps + 1;
}
// Steps of one key head of sequences b0 + lane (0 from b1 on), a lane each; the
// whole warp takes those of many groups.
__device__ int head_steps(const ChunkParams& p, int b0, int b1, bool report) {
    const int lane = threadIdx.x & 31;
    Seq s{0, 0, 0};
    if (b0 + lane < b1) s = sequence(p.c, b0 + lane, report);
    const int n = group_count(p, s);
    int sum = 0;
    if (n <= 4)
        for (int i = 0; i < n; ++i) sum += group_steps(p, s, i);
    for (unsigned m = __ballot_sync(0xffffffffu, n > 4); m; m &= m - 1) {
        const int from = __ffs(m) - 1;
        Seq w;
        w.row0 = 0;
        w.n = __shfl_sync(0xffffffffu, s.n, from);
        w.ctx = __shfl_sync(0xffffffffu, s.ctx, from);
        const int cnt = __shfl_sync(0xffffffffu, n, from);
        int x = 0;
        for (int i = lane; i < cnt; i += 32) x += group_steps(p, w, i);
        x = __reduce_add_sync(0xffffffffu, x);
        if (lane == from) sum = x;
    }
    return sum;
}
__device__ __forceinline__ int inclusive_sum(int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)(threadIdx.x & 31) >= o) v += x;
    }
    return v;
}

// ---------------------------------------------------------------- producer
template <int D, bool Q8>
__device__ void producer(const CUtensorMap* tk, const CUtensorMap* tv, const ChunkParams& p, uint8_t* sT, uint8_t* sS,
                         Ctrl* c, int lo, int hi, int per, volatile WaitFlag* wf) {
    using C = Cfg<D, Q8>;
    constexpr uint32_t NS = Q8 ? C::NRAW : C::NT;
    constexpr int ROWB = Q8 ? D : 128, NBOX = Q8 ? 1 : C::NBOX, BOX = kHalf * ROWB, TILE = NBOX * BOX;
    const ChunkCommon& cc = p.c;
    uint64_t* full = Q8 ? c->r_full : c->t_full;
    uint64_t* empty = Q8 ? c->r_empty : c->t_empty;
    const int lane = threadIdx.x & 31, ppt = kTile / cc.page;
    const bool leader = elect_one();
    uint32_t slot = 0, phase = 0, nload = 0, g = 0, nq = 0;
    bool ok = true;
    PartMeta mt{-1, 0, per, 0, 0, 0, {0, 0}};
    int v0 = -1, v1 = -1;  // rows of the V tiles still to load, of the step before
    // the next tile, from row y on (-1: nothing is there, zeros)
    auto load = [&](bool val, int y) -> bool {
        if (nload >= NS && !warp_wait(&empty[slot], phase ^ 1, wf)) return false;
        if (leader) {
            const bool sc = Q8 && y >= 0;
            mbar_arrive_expect_tx(&full[slot], TILE + (sc ? kHalf : 0));
#pragma unroll
            for (int x = 0; x < NBOX; ++x)
                tma_load_2d(sT + slot * TILE + x * BOX, val ? tv : tk, &full[slot], x * 64, y >= 0 ? y : -kHalf);
            if (sc) bulk_load(sS + slot * kHalf, (val ? cc.vs : cc.ks) + y, kHalf, &full[slot]);
        }
        ++nload;
        if (++slot == NS) {
            slot = 0;
            phase ^= 1;
        }
        return true;
    };
    // V of half hf of the step before (number g - 1): its load, and what its last rows need
    int v_held = kTile;  // its slots up to the last token
    auto load_v = [&](int hf, int y, uint32_t g) -> bool {
        const uint32_t s = slot, ph = phase;
        if (!load(true, y)) return false;
        if (Q8) return true;
        const int from = max(v_held - hf * kHalf, 0);
        if (from < kHalf) {
            // rows behind the last token may hold NaN, and 0 * NaN is none of the sum
            if (!warp_wait(&full[s], ph, wf)) return false;
#pragma unroll
            for (int x = 0; x < NBOX; ++x)
                for (int i = from * 8 + lane; i < kHalf * 8; i += 32)
                    reinterpret_cast<uint4*>(sT + s * TILE + x * BOX)[i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
        }
        __syncwarp();
        if (leader) mbar_arrive(&c->fix_full[(g - 1) % kInfos][hf]);  // at every step: its phase goes with the step
        return true;
    };
    if (lo < hi) {
        // c->place: the sequence that step lo lies in, and its first step; then the head, and
        // the group: the last one whose first step is not behind it
        Place at = c->place;
        Seq sq = sequence(cc, at.b, false);
        int n_groups = group_count(p, sq);
        at.h = (lo - at.start) / at.head;
        const int in = lo - at.start - at.h * at.head;
        at.i = at.cum = 0;
        for (int i0 = 0, before = 0; i0 < n_groups; i0 += 32) {
            const int st = i0 + lane < n_groups ? group_steps(p, sq, i0 + lane) : 0;
            const int incl = before + inclusive_sum(st), cum = incl - st;
            const unsigned le = __ballot_sync(0xffffffffu, i0 + lane < n_groups && cum <= in);
            if (le) {
                const int x = 31 - __clz(le);
                at.i = i0 + x;
                at.cum = __shfl_sync(0xffffffffu, cum, x);
            }
            before = __shfl_sync(0xffffffffu, incl, 31);
            if (before > in) break;
        }
        at.start += at.h * at.head + at.cum;
        int pos = lo;
        while (ok && pos < hi) {
            const int b = at.b, h = at.h, t0 = at.i * 2 * p.tq;
            const int n = min(sq.n - t0, 2 * p.tq), first = sq.ctx + t0, last = first + n;
            const int vis0 = first_slot(cc, first);
            const Span sp = visible_span(cc, first, last);
            const int start = at.start, end = start + sp.steps;  // then the step of its end
            const int s0 = pos - start, s1 = min(end, hi) - start;
            const bool whole = s0 == 0 && start + s1 == end;
            const int part = whole ? -1 : 2 * (int)blockIdx.x + (pos == lo ? 0 : 1);
            if (start < lo && lo < end) mt = PartMeta{start, end, per, sq.row0 + t0, n, h, {0, 0}};
            // the Q loader's turn, as soon as its buffers are free
            if (s0 < s1 && nq >= kQAhead && !warp_wait(&c->qi_empty[nq % kQAhead], ((nq / kQAhead) & 1) ^ 1, wf)) {
                ok = false;
                break;
            }
            if (s0 < s1) {
                if (leader) {
                    c->qitem[nq % kQAhead] = make_int2(h * cc.G, sq.row0 + t0);
                    mbar_arrive(&c->qi_full[nq % kQAhead]);
                }
                ++nq;
            }
            for (int e0 = s0 * ppt; e0 < s1 * ppt && ok; e0 += 32) {
                const int e = e0 + lane, est = e / ppt;  // 32 pages resolved at a time
                const int j = sp.tile(est) * ppt + e % ppt;
                const int y = est < s1 ? page_row(cc, b, h, j, vis0, last) : -1;
                const int cnt = min(32, s1 * ppt - e0);
                for (int q = 0; q < cnt && ok; q += ppt) {
                    const int st = (e0 + q) / ppt;
                    const int y0 = __shfl_sync(0xffffffffu, y, q), y1 = __shfl_sync(0xffffffffu, y, q + ppt - 1);
                    const uint32_t is = g % kInfos;
                    if (g >= kInfos && !warp_wait(&c->i_empty[is], ((g / kInfos) & 1) ^ 1, wf)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        StepInfo& f = c->info[is];
                        const int base = sp.tile(st) * kTile;
                        const int have = ppt == 1 ? (y0 >= 0 ? 3 : 0) : (y0 >= 0 ? 1 : 0) | (y1 >= 0 ? 2 : 0);
                        // every row sees all of it: up to the first token, inside the last one's window
                        const bool plain = have == 3 && base + kTile <= first + 1 &&
                                           (cc.window <= 0 || base > last - 1 - cc.window || base + kTile <= cc.sinks);
                        f.flags = (st == s0 ? kFirst : 0) | (st + 1 == s1 ? kLast : 0) | (plain ? 0 : kMask) |
                                  (base + kTile > sq.ctx + sq.n ? kFix : 0);
                        f.base = base;
                        f.have = have;
                        f.row0 = sq.row0 + t0;
                        f.n = n;
                        f.h = h;
                        f.pos0 = first;
                        f.end = sq.ctx + sq.n;
                        f.part = part;
                        mbar_arrive(&c->i_full[is]);
                    }
                    __syncwarp();
                    const int k1 = ppt == 2 ? y1 : y0 >= 0 ? y0 + kHalf : -1;
                    if (g > 0) ok = load_v(0, v0, g);
                    ok = ok && load(false, y0);
                    if (g > 0) ok = ok && load_v(1, v1, g);
                    ok = ok && load(false, k1);
                    v0 = y0;
                    v1 = k1;
                    const int base = sp.tile(st) * kTile;
                    v_held = base + kTile > sq.ctx + sq.n ? sq.ctx + sq.n - base : kTile;
                    ++g;
                    if (leader) c->issued = g;
                }
            }
            pos = at.start = end + 1;
            if (++at.i == n_groups && pos < hi) {
                at.i = 0;
                if (++at.h == cc.Hkv) {
                    at.h = 0;
                    do {
                        sq = sequence(cc, ++at.b, false);
                        n_groups = group_count(p, sq);
                    } while (n_groups == 0);
                }
            }
        }
    }
    if (ok) {
        // the end mark in the place of the next K tile; the converters and the MMA lanes pass it on
        const uint32_t is = g % kInfos;
        if (g > 0) ok = load_v(0, v0, g);
        ok = ok && (g < kInfos || warp_wait(&c->i_empty[is], ((g / kInfos) & 1) ^ 1, wf));
        ok = ok && (nload < NS || warp_wait(&empty[slot], phase ^ 1, wf));
        if (ok) {
            if (leader) {
                c->info[is].flags = kEnd;
                mbar_arrive(&c->i_full[is]);
                mbar_arrive(&full[slot]);
            }
            __syncwarp();
            ++nload;
            if (++slot == NS) {
                slot = 0;
                phase ^= 1;
            }
            if (g > 0) load_v(1, v1, g);
        }
        if ((nq < kQAhead || warp_wait(&c->qi_empty[nq % kQAhead], ((nq / kQAhead) & 1) ^ 1, wf)) && leader) {
            c->qitem[nq % kQAhead] = make_int2(-1, 0);
            mbar_arrive(&c->qi_full[nq % kQAhead]);
        }
    }
    if (lane == 0) p.meta[blockIdx.x] = mt;
    __syncwarp();
    if (leader) {
        // copies still in flight must land before the CTA exits
        for (uint32_t x = nload > NS ? nload - NS : 0; x < nload; ++x) mbar_wait_drain(&full[x % NS], (x / NS) & 1);
    }
}

// ---------------------------------------------------------------- Q loader
// One lane.  Tile B's queries follow tile A's; rows behind a tile's tokens * G
// stay the zeros of the start (or another tile's queries: they are not stored).
template <int D>
__device__ void q_loader(const CUtensorMap* tq, const ChunkParams& p, uint8_t* sQ, Ctrl* c, volatile WaitFlag* wf) {
    constexpr int NBOX = D / 64, QBOX = 128 * 128;
    if (elect_one()) {
        uint32_t n = 0;  // items
        uint32_t loads[2] = {0, 0};
        for (;; ++n) {
            const uint32_t qi = n % kQAhead;
            // the next item is announced when this one's loads are through, which may take
            // longer than a wait: the limit counts from the last step issued
            bool there;
            uint32_t seen;
            do {
                seen = c->issued;
                const unsigned long long t0 = globaltimer_ns();
                there = false;
                for (uint32_t it = 1; !there; ++it) {
                    there = mbar_try_wait(&c->qi_full[qi], (n / kQAhead) & 1);
                    if ((it & 31u) == 0 && (wf->abort || globaltimer_ns() - t0 > wf->limit_ns)) break;
                }
            } while (!there && !wf->abort && c->issued != seen);
            if (!there) {
                wf->abort = 1;
                break;
            }
            const int2 it = c->qitem[qi];
            mbar_arrive(&c->qi_empty[qi]);
            if (it.x < 0) break;
            bool ok = true;
            for (int t = 0; t < 2 && ok; ++t) {
                ok = mbar_wait(&c->q_empty[t], (n & 1) ^ 1, wf);
                if (!ok) break;
                mbar_arrive_expect_tx(&c->q_full[t], (uint32_t)(p.tq * p.c.G * 128 * NBOX));
                ++loads[t];
#pragma unroll
                for (int x = 0; x < NBOX; ++x)
                    tma_load_3d(sQ + (t * NBOX + x) * QBOX, tq, &c->q_full[t], x * 64, it.x, it.y + t * p.tq);
            }
            if (!ok) break;
        }
        // a copy still in flight must land before the CTA exits
        for (int t = 0; t < 2; ++t)
            if (loads[t] > 0) mbar_wait_drain(&c->q_full[t], (loads[t] - 1) & 1);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- MMA
// One lane for each tile: issuing takes a lane as long as half of the products do.
//   ... PV(x-2) QK(x) PV(x-1) QK(x+1) ...
// A tile's scores are two halves of a step ahead of its product, so that its
// softmax never waits for the product of the half before.
template <int D, bool Q8>
__device__ void mma_lane(int t, uint8_t* sQ, uint8_t* sT, Ctrl* c, uint32_t tmem, volatile WaitFlag* wf) {
    using C = Cfg<D, Q8>;
    constexpr uint64_t KDESC = sdesc_sw128_base(16, 1024), VDESC = sdesc_sw128_base(C::BOX, 1024);
    constexpr uint64_t QDESC = KDESC;
    constexpr uint32_t IQK = idesc_bf16_f32(128, kHalf, false), IPV = idesc_bf16_f32(128, D, true);
    if (elect_one()) {
        uint32_t slot = 0, phase = 0, items = 0;
        int flags = 0, pflags = 0;  // of this step and of the one before
        const uint64_t qd = QDESC + (smem_u32(sQ + t * C::QTILE) >> 4);
        const uint32_t t_o = tmem + C::O_COL + t * D;
        auto next = [&]() {
            if (++slot == (uint32_t)C::NT) {
                slot = 0;
                phase ^= 1;
            }
        };
        // O += P V of half y, whose V tile is the next one; its step's flags are pf
        auto pv = [&](uint32_t y, int pf) -> bool {
            const uint32_t hf = y & 1, g = y >> 1;
            if (!mbar_wait(&c->t_full[slot], phase, wf)) return false;
            if (!Q8 && (pf & kFix) && !mbar_wait(&c->fix_full[g % kInfos][hf], (g / kInfos) & 1, wf)) return false;
            if (!mbar_wait(&c->p_full[t][hf], g & 1, wf)) return false;
            tc_fence_after();
            const uint64_t vd = VDESC + (smem_u32(sT + slot * C::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ts(t_o, tmem + t * kTile + hf * kHalf + kk * 8, vd + (uint64_t)((kk * 16 * 128) >> 4), IPV,
                       ((pf & kFirst) && hf == 0 && kk == 0) ? 0u : 1u);
            mma_commit(&c->pv_done[t][hf]);
            mma_commit(&c->t_empty[slot]);
            if (hf == 1 && (pf & kLast)) mma_commit(&c->o_full[t]);
            next();
            return true;
        };
        for (uint32_t x = 0;; ++x) {
            const uint32_t hf = x & 1;
            if (x >= 2 && !pv(x - 2, pflags)) break;
            if (!mbar_wait(&c->t_full[slot], phase, wf)) break;
            if (hf == 0) {
                flags = c->info[(x >> 1) % kInfos].flags;
                if (flags & kEnd) {
                    next();
                    if (x >= 2 && !pv(x - 1, pflags)) break;
                    mbar_arrive(&c->s_full[t][0]);
                    mbar_arrive(&c->s_full[t][0]);
                    break;
                }
                if ((flags & kFirst) && !mbar_wait(&c->q_full[t], items & 1, wf)) break;
            }
            tc_fence_after();
            // S of the half's 64 slots, into the half's buffer
            const uint64_t kd = KDESC + (smem_u32(sT + slot * C::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(tmem + t * kTile + hf * kHalf, qd + (uint64_t)(((kk >> 2) * C::QBOX + (kk & 3) * 32) >> 4),
                       kd + (uint64_t)(((kk >> 2) * C::BOX + (kk & 3) * 32) >> 4), IQK, kk > 0);
            mma_commit(&c->s_full[t][hf]);
            mbar_arrive(&c->s_full[t][hf]);
            mma_commit(&c->t_empty[slot]);
            next();
            if (hf == 1) {
                if (flags & kLast) {
                    mma_commit(&c->q_empty[t]);
                    ++items;
                }
                pflags = flags;
            }
        }
        mma_commit(&c->drain[t]);
        mbar_wait_drain(&c->drain[t], 0);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- converters
// Eight warps, two to each tile of a step (K and V of either half), so that four
// tiles are under way at a time: codes times 2^e, in bf16, into the tile that the
// products read; 16-byte pieces, both sides in their copy's swizzle.  They share the
// schedulers with two softmax warps each and take as long as those do: 8,192 tokens
// behind as many slots, 32 heads of 128, 1,325 us (1.25 PFLOP/s; bf16 pools 1.37 PFLOP/s;
// a warp to a tile 1,545, two for all four 1,747).
template <int D>
__device__ void converter(const uint8_t* sR, const uint8_t* sS, uint8_t* sT, Ctrl* c, volatile WaitFlag* wf) {
    using C = Cfg<D, true>;
    constexpr int LPR = D / 16, RPP = 32 / LPR;  // lanes of a row (a 16-byte piece each), rows at a time
    const int lane = threadIdx.x & 31, id = (threadIdx.x >> 5) - kConverter, hf = id & 1, piece = lane % LPR;
    const bool val = id & 2;
    const int from = (id >> 2) * (kHalf / C::CONV);  // this warp's rows
    for (uint32_t g = 0;; ++g) {
        const uint32_t is = g % kInfos, x = 2 * g + hf, n = val ? v_tile(x) : k_tile(x);
        if (!warp_wait(&c->i_full[is], (g / kInfos) & 1, wf)) return;
        const int flags = c->info[is].flags, left = c->info[is].end - c->info[is].base - hf * kHalf;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->i_empty[is]);
        const bool end = flags & kEnd;
        if (end && (id & 3)) return;  // the end mark stands in the place of the next K tile
        const uint32_t rs = n % C::NRAW, ts = n % C::NT;
        // A barrier's parity tells a phase from its neighbours only: who skips phases may
        // take one for another.  These warps see every phase of their slots' barriers, but
        // for K(0), which stands where V(-1) would: it has landed once it is converted.
        if (g == 0 && id % 4 == 3 && (!reached(&c->first[0], 1, wf) || !reached(&c->first[1], 1, wf))) return;
        if (!warp_wait(&c->r_full[rs], (n / C::NRAW) & 1, wf)) return;
        if (!warp_wait(&c->t_empty[ts], ((n / C::NT) & 1) ^ 1, wf)) return;
        if (!end) {
            // V rows behind the last token may be NaN, and 0 * NaN is none of the sum
            const int keep = val && (flags & kFix) ? left : kHalf;
#pragma unroll 4
            for (int r0 = from; r0 < from + kHalf / C::CONV; r0 += RPP) {
                const int row = r0 + lane / LPR;
                const int rx = D == 64 ? (row >> 1) & 3 : row & 7, wx = row & 7;
                uint4 v = *reinterpret_cast<const uint4*>(sR + rs * C::RAW + row * D + ((piece ^ rx) << 4));
                // 2^e (bytes that are never written: any finite factor)
                const uint32_t e = sS[rs * kHalf + row];
                const float f = __uint_as_float((uint32_t)min(max((int)e, 127 + kMinExp), 127 + kMaxExp) << 23);
                if (row >= keep) v = make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t o[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const f2 y = mul2(codes_f32(w[k >> 1], k & 1), {f, f});
                    o[k] = pack_bf16x2(y.x, y.y);
                }
                uint8_t* dst = sT + ts * C::TILE + (piece >> 2) * C::BOX + row * 128;
                const int ch = (piece & 3) * 2;
                *reinterpret_cast<uint4*>(dst + ((ch ^ wx) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(dst + (((ch + 1) ^ wx) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&c->r_empty[rs]);
            mbar_arrive(&c->t_full[ts]);
            if (n == 0) c->first[id >> 2] = 1;
        }
        if (end) return;
    }
}

// ---------------------------------------------------------------- softmax
template <int D, bool Q8>
__device__ void softmax(const ChunkParams& p, uint8_t* stage, Ctrl* c, uint32_t tmem, volatile WaitFlag* wf) {
    using C = Cfg<D, Q8>;
    const ChunkCommon& cc = p.c;
    const int t = threadIdx.x >> 7, row = threadIdx.x & 127, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(row & 96) << 16;
    const uint32_t t_s = tmem + lanes + t * kTile, t_o = tmem + lanes + C::O_COL + t * D;
    const int tok = t * p.tq + row / cc.G, hd = row % cc.G;  // the row's token of the item, head of the group
    const bool in_tile = row < p.tq * cc.G;
    float m = -INFINITY, l = 0.f;
    uint32_t items = 0;
    const f2 sl2 = {cc.scale_log2, cc.scale_log2};
    // x counts halves of steps, 64 slots each
    for (uint32_t x = 0;; ++x) {
        const uint32_t g = x >> 1, hf = x & 1, is = g % kInfos;
        if (!warp_wait(&c->s_full[t][hf], g & 1, wf)) return;
        tc_fence_after();
        const StepInfo& f = c->info[is];
        const int flags = f.flags;
        if (flags & kEnd) return;
        const bool first = hf == 0 && (flags & kFirst);
        if (first) {
            m = -INFINITY;
            l = 0.f;
        }
        const uint32_t t_x = t_s + hf * 64;
        uint32_t s[2][32];
        tmem_ld32(t_x, s[0]);
        tmem_ld32(t_x + 32, s[1]);
        tmem_wait_ld();
        reg_fence(s[0]);
        reg_fence(s[1]);
        if (flags & kMask) {
            const unsigned long long vis =
                seen_slots(cc, f.base + 64 * (int)hf, in_tile && tok < f.n ? f.pos0 + tok : -1, (f.have >> hf) & 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t v = (uint32_t)(vis >> (32 * i));
                if (__all_sync(0xffffffffu, v == 0xffffffffu)) continue;
#pragma unroll
                for (int q = 0; q < 32; ++q)
                    if (!((v >> q) & 1u)) s[i][q] = __float_as_uint(-INFINITY);
            }
        }
        float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 32; q += 2)
                a[(q >> 1) & 3] = fmax3(a[(q >> 1) & 3], __uint_as_float(s[i][q]), __uint_as_float(s[i][q + 1]));
        const float top = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * cc.scale_log2;
        // The reference follows the maximum only where it grows by more than 2^8
        // (exact after the final division).
        if (__any_sync(0xffffffffu, top > m + 8.f)) {
            const float up = fmaxf(m, top);
            const float w = up == -INFINITY ? 1.f : ex2_approx(m - up);
            if (!first) {
                // O is at rest once the half before has been added; nothing follows before p_full
                const uint32_t y = x - 1;
                if (!warp_wait(&c->pv_done[t][y & 1], (y >> 1) & 1, wf)) return;
                tc_fence_after();
                const f2 w2 = {w, w};
#pragma unroll 1
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t o[32];
                    tmem_ld32(t_o + i * 32, o);
                    tmem_wait_ld();
                    reg_fence(o);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const f2 v = mul2({__uint_as_float(o[2 * q]), __uint_as_float(o[2 * q + 1])}, w2);
                        o[2 * q] = __float_as_uint(v.x);
                        o[2 * q + 1] = __float_as_uint(v.y);
                    }
                    tmem_st32(t_o + i * 32, o);
                }
            }
            l *= w;
            m = up;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const f2 nm2 = {-ref, -ref};
        f2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const f2 v = fma2({__uint_as_float(s[i][2 * q]), __uint_as_float(s[i][2 * q + 1])}, sl2, nm2);
                const f2 e = {ex2_approx(v.x), ex2_approx(v.y)};
                sum[q & 1] = add2(sum[q & 1], e);
                pk[q] = pack_bf16x2(e.x, e.y);
            }
            tmem_st16(t_x + i * 16, pk);
        }
        const f2 both = add2(sum[0], sum[1]);
        l += both.x + both.y;
        const int n = f.n, part = f.part, h = f.h;
        const int64_t row0 = f.row0;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&c->p_full[t][hf]);
            if (hf) mbar_arrive(&c->i_empty[is]);
        }
        if (!hf || !(flags & kLast)) continue;
        // The item's end: its row, normalised, or a part of it.
        if (!warp_wait(&c->o_full[t], items & 1, wf)) return;
        tc_fence_after();
        ++items;
        const bool live = in_tile && tok < n;
        const float w = part >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;
        const int64_t orow = (row0 + tok) * cc.Hq + h * cc.G + hd;
        const int64_t prow = (int64_t)part * kRows + threadIdx.x;
        if (live) {
            if (part < 0)
                cc.lse[orow] = lse_of(m, l);
            else
                p.part_ml[prow] = make_float2(m, l);
        }
#pragma unroll 1
        for (int y = 0; y < D / 32; ++y) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(t_o + y * 32, o);
            tmem_wait_ld();
            reg_fence(o);
            if (part >= 0) {
                if (!live) continue;
                uint4* dst = reinterpret_cast<uint4*>(p.part_o) + ((int64_t)part * (D / 4) + y * 8) * kRows + threadIdx.x;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    dst[q * kRows] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                continue;
            }
            uint4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * q]) * w, __uint_as_float(o[8 * q + 1]) * w),
                                  pack_bf16x2(__uint_as_float(o[8 * q + 2]) * w, __uint_as_float(o[8 * q + 3]) * w),
                                  pack_bf16x2(__uint_as_float(o[8 * q + 4]) * w, __uint_as_float(o[8 * q + 5]) * w),
                                  pack_bf16x2(__uint_as_float(o[8 * q + 6]) * w, __uint_as_float(o[8 * q + 7]) * w));
            if (C::STAGE == 0) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cc.out) + orow * D + y * 32);
                if (live)
#pragma unroll
                    for (int q = 0; q < 4; ++q) dst[q] = v[q];
                continue;
            }
            // 16-byte pieces of the lane's row, in a swizzle; two turns fill a line
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(stage + lane * 128 + ((((y & 1) * 4 + q) ^ (lane & 7)) << 4)) = v[q];
            if (!(y & 1)) continue;
            __syncwarp();
            char* dst = static_cast<char*>(cc.out) + (y >> 1) * 128 + (lane & 7) * 16;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = 4 * k + (lane >> 3);
                const long long at = __shfl_sync(0xffffffffu, live ? (long long)orow : -1ll, r);
                const uint4 x = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane ^ r) & 7) << 4));
                if (at >= 0) *reinterpret_cast<uint4*>(dst + at * (D * 2)) = x;
            }
        }
        __syncwarp();
        tc_fence_before();
    }
}

// ---------------------------------------------------------------- kernel
template <int D, bool Q8>
__global__ void __launch_bounds__(Cfg<D, Q8>::THREADS, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const ChunkParams p) {
    using C = Cfg<D, Q8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {
        griddep_wait();
        if (threadIdx.x == 0) {
            p.meta[blockIdx.x].start = -1;
            atomicOr(p.c.err, ERR_LAUNCH);
        }
        return;
    }
    uint8_t* sQ = smem;
    uint8_t* sT = sQ + 2 * C::QTILE;
    uint8_t* sR = sT + C::NT * C::TILE;
    uint8_t* sS = sR + C::NRAW * C::RAW;
    Ctrl* c = reinterpret_cast<Ctrl*>(sS + C::NRAW * kHalf + C::STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    {
        const int x = threadIdx.x;
        if (x < kMaxTiles) {
            mbar_init(&c->t_full[x], Q8 ? C::CONV : 1);  // its converters, or the copy
            mbar_init(&c->t_empty[x], 2);  // both tiles' products
            mbar_init(&c->r_full[x], 1);
            mbar_init(&c->r_empty[x], C::CONV);
        } else if (x >= 32 && x < 32 + kInfos) {
            mbar_init(&c->i_full[x - 32], 1);
            mbar_init(&c->i_empty[x - 32], 8 + (Q8 ? 4 * C::CONV : 0));  // the softmax warps and the converters
            mbar_init(&c->fix_full[x - 32][0], 1);
            mbar_init(&c->fix_full[x - 32][1], 1);
        } else if (x >= 64 && x < 66) {
            mbar_init(&c->q_full[x - 64], 1);
            mbar_init(&c->q_empty[x - 64], 1);
            for (int hf = 0; hf < 2; ++hf) {
                mbar_init(&c->s_full[x - 64][hf], 2);  // the scores' commit and the MMA lane itself
                mbar_init(&c->p_full[x - 64][hf], 4);
                mbar_init(&c->pv_done[x - 64][hf], 1);
            }
            mbar_init(&c->o_full[x - 64], 1);
        } else if (x >= 96 && x < 96 + kQAhead) {
            mbar_init(&c->qi_full[x - 96], 1);
            mbar_init(&c->qi_empty[x - 96], 1);
        } else if (x == 128) {
            mbar_init(&c->drain[0], 1);
            mbar_init(&c->drain[1], 1);
            c->wf.abort = 0;
            c->wf.limit_ns = p.c.wait_limit_ns;
            c->issued = 0;
            c->first[0] = c->first[1] = 0;
        }
        fence_mbar_init();
        for (int z = x; z < 2 * C::QTILE / 16; z += C::THREADS)
            reinterpret_cast<uint4*>(sQ)[z] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == kProducer && lane == 0) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    // Nothing before this line reads or writes global memory or takes tensor memory.
    griddep_wait();
    if (warp == kMma) {
        tmem_alloc(&c->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem_base;
    volatile WaitFlag* wf = &c->wf;
    // steps of all sequences, a run of 32 after another to a warp; then the range's start
    constexpr int NW = C::THREADS / 32;
    const int each = (p.c.B + 32 * NW - 1) / (32 * NW) * 32;  // sequences of a warp
    const int b0 = min(p.c.B, warp * each), b1 = min(p.c.B, b0 + each);
    long long mine = 0;
    int some = 0;
    for (int b = b0; b < b1; b += 32) mine += some = head_steps(p, b, b1, blockIdx.x == 0);  // this lane's
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) c->sums[warp] = mine;
    __syncthreads();
    long long ahead = lane < NW ? c->sums[lane] : 0;  // inclusive sums over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, ahead, o);
        if (lane >= o) ahead += x;
    }
    long long all = __shfl_sync(0xffffffffu, ahead, 31);
    ahead = __shfl_sync(0xffffffffu, ahead, warp) - mine;
    if (all * p.c.Hkv > 1 << 30) {  // only where sequences overlap: their rows make no sense
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.c.err, ERR_BAD_ROW);
        all = 0;
    }
    const int total = (int)all * p.c.Hkv;
    const int per = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    const int lo = min(total, (int)blockIdx.x * per), hi = min(total, lo + per);
    if (lo < hi && ahead * p.c.Hkv <= lo && lo < (ahead + mine) * p.c.Hkv) {
        int before = (int)ahead * p.c.Hkv;
        for (int b = b0; b < b1; b += 32) {
            const int st = each == 32 ? some : head_steps(p, b, b1, false), incl = inclusive_sum(st);
            const int first = before + (incl - st) * p.c.Hkv;
            if (first <= lo && lo < first + st * p.c.Hkv) c->place = Place{b + lane, 0, 0, st, 0, first};
            before += __shfl_sync(0xffffffffu, incl, 31) * p.c.Hkv;
        }
    }
    __syncthreads();
    // A split of the launch's registers: bf16 512 x 128 = 256 x 184 + 256 x 72, 8-bit
    // 640 x 96 = 256 x 144 + 384 x 64.
    if (warp < 8) {
        if (Q8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        softmax<D, Q8>(p, sS + C::NRAW * kHalf + warp * (C::STAGE / 8), c, tmem, wf);
    } else {
        if (Q8)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kProducer)
            producer<D, Q8>(&tk, &tv, p, Q8 ? sR : sT, sS, c, lo, hi, per, wf);
        else if (warp == kMma || warp == kMma + 1)
            mma_lane<D, Q8>(warp - kMma, sQ, sT, c, tmem, wf);
        else if (warp == kQLoader)
            q_loader<D>(&tq, p, sQ, c, wf);
        else if (Q8)
            converter<D>(sR, sS, sT, c, wf);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && c->wf.abort) atomicOr(p.c.err, ERR_TIMEOUT);
}

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int tile_tokens(int G) { return 128 / G; }

// The workspace: both kernels' part descriptions and the parts.
struct Layout {
    int64_t short_meta, short_o, short_ml, meta, o, ml, bytes;
};
int64_t up(int64_t x) { return (x + 255) / 256 * 256; }
Layout layout(int64_t B, int64_t tokens, int G, int D) {
    Layout w{};
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t x = at;
        at = up(at + n);
        return x;
    };
    const int64_t parts = 2 * kChunkMaxCtas;
    w.short_meta = take(kChunkMaxCtas * (int64_t)sizeof(PartMeta));
    w.short_o = take(parts * kShortRows * D * 4);
    w.short_ml = take(parts * kShortRows * 8);
    if (tokens * G > kShortRows) {
        w.meta = take(kChunkMaxCtas * (int64_t)sizeof(PartMeta));
        w.o = take(parts * kRows * D * 4);
        w.ml = take(parts * kRows * 8);
    }
    w.bytes = at;
    return w;
}

template <int D, bool Q8>
int go(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& p, const PartSet& few,
       int few_rows, int ctas, cudaStream_t s) {
    using C = Cfg<D, Q8>;
    static std::atomic<uint64_t> raised{0};
    if (raise_smem_limit(reinterpret_cast<const void*>(chunk_kernel<D, Q8>), C::SMEM, &raised) != cudaSuccess)
        return BSA_ERR_CUDA;
    {
        // the register split takes all of what 512 threads of 128 are given: with less it would wait forever
        static std::atomic<int> regs{0};
        if (regs.load() == 0) {
            cudaFuncAttributes at;
            if (cudaFuncGetAttributes(&at, chunk_kernel<D, Q8>) != cudaSuccess) return BSA_ERR_CUDA;
            regs.store(at.numRegs);
        }
        if (regs.load() < (Q8 ? 96 : 128)) return BSA_ERR_UNSUPPORTED;
    }
    cudaError_t e = launch_after(chunk_kernel<D, Q8>, dim3((unsigned)ctas), C::THREADS, C::SMEM, s, tq, tk, tv, p);
    if (e == cudaSuccess && ctas > 1)
        e = launch_after(chunk_merge_kernel<D>, dim3((unsigned)ctas - 1, (unsigned)(few_rows + kRows / 32)), 256, 0, s, p.c,
                         few, PartSet{p.meta, p.part_o, p.part_ml}, few_rows, p.tq);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace
}  // namespace bsa

extern "C" {

int64_t bsa_chunk_attention_workspace(int32_t B, int32_t tokens, int32_t Hq, int32_t Hkv, int32_t D) {
    if (B <= 0 || tokens <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv || Hq / Hkv > 128) return 0;
    return bsa::layout(B, tokens, Hq / Hkv, D).bytes;
}

int bsa_chunk_attention(const bsa_chunk_args* a, const bsa_page_cache* c, const bsa_page_scales* scales,
                        void* workspace, int64_t workspace_bytes, bsa_stream_t stream) {
    using namespace bsa;
    if (!a) return BSA_ERR_INVALID_ARG;
    int st = check_page_cache(c);
    if (st != BSA_OK) return st;
    if (scales && (st = check_page_scales(c, scales)) != BSA_OK) return st;
    if (a->B < 0 || a->tokens < 0 || a->Hq <= 0 || a->Hq % c->Hkv || c->layers != 1 || c->n_seqs != a->B)
        return BSA_ERR_INVALID_ARG;
    if (!a->q_ptr && a->tokens != a->B) return BSA_ERR_INVALID_ARG;
    if (a->window < 0 || a->sinks < 0 || a->max_context < 0 || !(a->scale > 0.f) || !std::isfinite(a->scale)) return BSA_ERR_INVALID_ARG;
    if (!al(a->q, 16) || !al(a->out, 16) || !al(a->lse, 4) || !al(a->context_len, 4) || !al(a->q_ptr, 4))
        return BSA_ERR_INVALID_ARG;
    if (a->Hq / c->Hkv > 128) return BSA_ERR_UNSUPPORTED;
    if (a->B > 0 && a->tokens > 0 && (!a->q || !a->context_len || !a->out || !a->lse || !c->page_table))
        return BSA_ERR_INVALID_ARG;
    if (a->B == 0 || a->tokens == 0) return BSA_OK;
    const int G = a->Hq / c->Hkv;
    const Layout w = layout(a->B, a->tokens, G, c->D);
    // the steps of the chunks stay below 2^30 (sums and range ends fit an int): a sequence has
    // its tokens over 2 tq, rounded up, groups (the kernel refuses sequences that overlap so far)
    const int64_t most = ((int64_t)c->max_pages * c->page + kTile - 1) / kTile;
    const double groups = (double)a->tokens / (2 * tile_tokens(G)) + a->B;
    if (c->Hkv * most > 1 << 30 || groups * (most + 1) * c->Hkv > (double)(1 << 30)) return BSA_ERR_INVALID_ARG;
    if (!workspace || !al(workspace, 256)) return BSA_ERR_INVALID_ARG;
    if (workspace_bytes < w.bytes) return BSA_ERR_CAPACITY;
    ChunkCommon p{};
    int sms;
    if ((st = device_context(&p.err, &sms)) != BSA_OK) return st;
    p.ctx = a->context_len;
    p.q_ptr = a->q_ptr;
    p.table = c->page_table;
    p.ks = scales ? static_cast<const uint8_t*>(scales->k) : nullptr;
    p.vs = scales ? static_cast<const uint8_t*>(scales->v) : nullptr;
    p.B = a->B;
    p.tokens = a->tokens;
    p.Hq = a->Hq;
    p.Hkv = c->Hkv;
    p.G = G;
    p.page = c->page;
    p.P = c->max_pages;
    p.n_pages = c->n_pages;
    p.window = a->window;
    p.sinks = a->sinks;
    p.out = a->out;
    p.lse = a->lse;
    p.scale_log2 = a->scale * 1.4426950408889634f;
    p.wait_limit_ns = wait_limit_ns();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    // Short sequences have a kernel of their own where that pays: a row of a chunk's tile
    // costs them nothing but time, a launch and the wait for it do.  Counted in steps of
    // single sequences per SM, at most (as long as the longest may be), batches of which a
    // tenth are chunks of 60 to 500 tokens, us with and without that kernel:
    //   bf16   8: 57, 39   34: 90, 74   70: 163, 157   105: 182, 196   190: 345, 383
    //   8-bit  8: 54, 42   34: 77, 96   70: 139, 204   (a chunk's step takes 2.5 times as long)
    // These hold where max_context, or else the table's width, is the longest context; under
    // a table for 131,072 slots and without max_context 8 sequences of up to 1,000 slots take
    // 31 us instead of 20 (bf16) and 35 instead of 23 (8-bit).  A window bounds the steps too:
    // 8 sequences of up to 32,000 slots under one of 1,024, four steps per SM, 39 and 29 (bf16),
    // 42 and 33 (8-bit); 24, 13 steps, 74 and 59, 70 and 69; 48, 25 steps, 109 and 99, 109 and 118.
    // Single tokens of more heads than its rows are chunks too.
    const bool all_short = !a->q_ptr || (int64_t)a->tokens * G <= kShortRows;  // if their heads allow
    auto tiles = [](int64_t slots) { return (slots + kTile - 1) / kTile; };
    int64_t longest = a->max_context > 0 ? std::min(most, tiles(a->max_context)) : most;
    if (a->window > 0) longest = std::min(longest, tiles(a->window) + 1 + tiles(a->sinks));
    const bool some_short =
        G <= kShortRows && (all_short || (a->B > 1 && a->B * longest * c->Hkv > (scales ? 16ll : 64ll) * sms));
    PartSet few{};
    int few_rows = 0;
    if (some_short) {
        ShortLaunch L{};
        L.c = p;
        L.k = c->k;
        L.v = c->v;
        L.q = a->q;
        L.D = c->D;
        L.sms = sms;
        L.meta = reinterpret_cast<PartMeta*>(ws + w.short_meta);
        L.part_o = reinterpret_cast<float*>(ws + w.short_o);
        L.part_ml = reinterpret_cast<float2*>(ws + w.short_ml);
        L.merge = all_short;
        if ((st = launch_short(L, s)) != BSA_OK) return st;
        if (all_short) return BSA_OK;
        few = PartSet{L.meta, L.part_o, L.part_ml};
        few_rows = short_rows(p);
    }
    ChunkParams cp{};
    cp.c = p;
    cp.tq = tile_tokens(G);
    cp.least = some_short ? kShortRows + 1 : 1;
    cp.meta = reinterpret_cast<PartMeta*>(ws + w.meta);
    cp.part_o = reinterpret_cast<float*>(ws + w.o);
    cp.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    CUtensorMap tq, tk, tv;
    const uint64_t krows = (uint64_t)c->n_pages * c->Hkv * c->page;
    auto encode = scales ? encode_rows_e4m3 : encode_rows_bf16;
    if ((st = encode_token_rows_bf16(&tq, a->q, (uint64_t)a->tokens, a->Hq, c->D, G, cp.tq)) != BSA_OK) return st;
    if ((st = encode(&tk, c->k, krows, c->D, kHalf)) != BSA_OK) return st;
    if ((st = encode(&tv, c->v, krows, c->D, kHalf)) != BSA_OK) return st;
    const int ctas = std::min(sms, kChunkMaxCtas);
    auto launch = c->D == 128 ? (scales ? go<128, true> : go<128, false>) : (scales ? go<64, true> : go<64, false>);
    return launch(tq, tk, tv, cp, few, few_rows, ctas, s);
}

}  // extern "C"
