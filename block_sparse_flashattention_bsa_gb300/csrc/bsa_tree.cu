// bsa_tree.cu -- attention of drafted tokens over a paged cache (one token per
// sequence: decoding; a tree of up to 64: verification), for sm_103a.
//
// Mathematics: for the T * G query rows of a sequence that read one key head
// (G query heads per key head), O = softmax(q K^T scale) V over the visible
// slots in one pass, with the running maximum and sum of the softmax.  A slot
// is visible when it is committed, or a draft whose bit is set in the row's
// tree mask; with block lists, only inside listed pages.
//
// What bounds it: every K and V row is read once, 4 D bytes a slot, and used
// for 4 D T G flops; below ~280 flops per byte (T G <= 128) memory is the limit,
// so the kernel is built to keep loads in flight and everything else behind
// them.  With more rows the exponentials are (2,400 cycles for a step of 128).
//
// Work: a step is 128 key slots (one page of 128 or two of 64); an item the
// steps of one key head of one sequence.  All steps of the batch form one
// sequence of (unit, item, step), cut into equal ranges, one per CTA: ragged
// lengths, long contexts with few rows and large batches all load every SM
// alike.  Several row tiles: as many CTAs to a range, which read its pages at
// about the same time, all but one of them from the L2 (ranges over (item, tile)
// read them from DRAM once per tile: 40 drafts over 4 contexts of 128K, 160 rows
// a head, 617 us against 551; 64 drafts, 1,024 rows, 635 against 515).  An item
// that lies in one range is written out directly; one that a range boundary cuts
// leaves an unnormalised fp32 part (with its maximum and sum) per range in the
// workspace, and merge_kernel joins the parts in range order -- no atomics, so
// results do not depend on timing.
//
// Measured: 4 contexts of 131,000 slots, 16 drafts, 32 query heads over 8 key
// heads of 128 (2.15 GB of cache): 311 to 321 us, 6.7 to 6.9 TB/s, the rate of
// a plain copy; 96 ragged sequences up to 8,192 slots, one token each (1.8 GB):
// 270 to 285 us; one sequence of 1,500 slots: 8.1 us.  Long contexts are bound
// by DRAM (a step of 64 KB per SM every 1.4 us, 7 TB/s); ragged batches lose 5 %
// to SMs that get less of it; short sequences are bound by the chain of an item
// (first page, scores, weights, product, result: 3 us a time for two steps).
//
// One CTA per SM, 11 warps:
//   warps 0-7  softmax, thread = query row (TMEM lane): warpgroup h takes
//              columns 64 h .. 64 h + 63 of every step, with an O accumulator,
//              a running maximum and a sum of its own, so that the two need not
//              meet before an item's end (where both write half of the joined
//              row) and a step's softmax takes half as long.  64-wide heads with
//              at most 32 rows: four splits of 32 columns, one to each of warps
//              0-3, on copies of the rows.  The maximum is
//              raised only when it grows by more than 2^8.  P goes back over S
//              as two bf16 parts, high and low, so that its rounding (2^-17)
//              does not add to the result's; the second product costs tensor
//              time that is not the limit.
//   warp 8     producer: walks the CTA's range, resolves pages and TMA-loads the
//              K / V tiles (a ring); publishes one description per step.
//   warp 10    loads an item's Q as soon as the item before has used its own.
//   warp 9     MMA: S = Q K^T and O += P V on tcgen05, M = 128 rows whatever
//              T G is (the rows behind it are zeros and are never stored).

#include <algorithm>
#include <cmath>

#include "bsa.h"
#include "bsa_internal.h"
#include "bsa_ptx.cuh"

namespace bsa {
namespace {

constexpr int kTreeThreads = 352;
constexpr int kProducer = 8, kMma = 9, kQLoader = 10;
constexpr int kMaxUnits = 2048;   // units of one launch (their prefix sums sit in shared memory)
constexpr int kMaxCtas = 160;     // partial slots are sized for this many
constexpr int kMaxSlots = 12;     // K / V ring
constexpr int kInfos = 8;         // step descriptions ahead (more than the ring's kMaxSlots / 2 steps)
static_assert(2 * kInfos > kMaxSlots + 2, "a description could be overwritten before its MMA");
constexpr int kTreeSmem = 232448;
constexpr int kCtrlBytes = 14336;
constexpr int kStep = 128;        // key slots per step
constexpr int kQBox = 128 * 128;  // one 64-column box of Q: 128 rows, those behind the item's zero
constexpr int kQAhead = 4;        // items announced to the Q loader
// Where the splits hand over their accumulators (floats of a row), in bytes.
__host__ __device__ constexpr int exchange_bytes(int D, int NS, int dup) {
    return (NS == 4 ? 4 * 32 : dup) * D * 4;
}

enum : int { kFirst = 1, kLast = 2, kMask = 4, kEnd = 8 };  // kFirst, kLast: of an item

struct StepInfo {
    int flags;
    int slot0[2];  // first slot of each sub-block (64-slot pages: two)
    int nv[2];     // its slots that hold something
    int b, h, t0;  // sequence, key head, first drafted token of the row tile
    int ctx, dl;
    int part;      // -1: write the output, else the partial slot
    int vslot;     // ring slot of the V tile, bit 31: its phase
};

struct Meta {  // one per CTA: the item its range starts inside of
    int start, end, per;  // start < 0: none
    int b, h, t0, dl;
    int pad;
};

struct TreeCtrl {
    uint64_t t_full[kMaxSlots], t_empty[kMaxSlots];
    uint64_t q_full, q_empty;
    uint64_t qi_full[kQAhead], qi_empty[kQAhead];
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t i_empty[kInfos];
    uint64_t st_full[4], x_full[4];  // per group of warps with the same rows: all posted their sums, their parts of O
    uint64_t drain;
    volatile uint32_t issued;        // steps the producer has issued
    int2 qitem[kQAhead];             // first query head and token of an item's row tile; x < 0: no more
    StepInfo info[kInfos];
    float2 stats[2][256];            // [item parity][split][row]: maximum and sum posted at an item's end
    int red[kTreeThreads / 32];
    uint32_t tmem_base;
    WaitFlag wf;
    int prefix[kMaxUnits + 1];       // sums of the units' steps per item
};

struct TreeParams {
    const int32_t *ctx, *dl, *row_ptr, *col_idx, *table;
    const unsigned long long* mask;
    int64_t col_cap;
    int32_t B, T, Hq, Hkv, G, page, P, n_pages;
    int32_t unit0, units;      // units of this launch
    int32_t tq, RT;            // drafted tokens per row tile, row tiles
    int32_t n_slots;           // ring slots
    int32_t dup;               // TMEM lanes between a row and its copies for the other splits' warps (0: none)
    int32_t ranges;            // the grid is (RT, ranges)
    void* out;
    float* lse;
    float* part_o;             // [2 * grid][rows][D]
    float2* part_ml;           // [2 * grid][rows]
    Meta* meta;
    int32_t* err;
    float scale_log2;
    unsigned long long wait_limit_ns;
};

__device__ __forceinline__ bool twait(uint64_t* bar, uint32_t parity, volatile WaitFlag* wf) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, wf));
}

// Sequence lengths as they are used: nothing negative, drafts at most T.
__device__ __forceinline__ int seq_ctx(const TreeParams& p, int b) { return max(p.ctx[b], 0); }
__device__ __forceinline__ int seq_dl(const TreeParams& p, int b) {
    return p.dl ? min(max(p.dl[b], 0), p.T) : p.T;
}

// Page sizes are 64 and 128: shifts, not divisions, on the way to the first load.
__device__ __forceinline__ int page_shift(const TreeParams& p) { return p.page == 64 ? 6 : 7; }
// Pages to steps (128 slots each), rounded up.
__device__ __forceinline__ int pages_to_steps(const TreeParams& p, int n) { return p.page == 64 ? (n + 1) >> 1 : n; }

// Pages a unit's row visits: listed entries, or the sequence's pages.
__device__ int unit_pages(const TreeParams& p, int u, bool report) {
    if (p.row_ptr) {
        const int64_t beg = p.row_ptr[u], end = min((int64_t)p.row_ptr[u + 1], p.col_cap);
        if (beg < 0 || end < beg || end - beg > p.P) {
            if (report) atomicOr(p.err, ERR_BAD_ROW);
            return 0;
        }
        return (int)(end - beg);
    }
    const uint32_t len = (uint32_t)seq_ctx(p, u) + seq_dl(p, u);
    const uint32_t n = (len + p.page - 1) >> page_shift(p);
    if (n > (uint32_t)p.P && report) atomicOr(p.err, ERR_BAD_PAGE);
    return (int)min(n, (uint32_t)p.P);
}

// Steps of one item of unit u; at least one, so that a row without any key
// still passes through the pipeline and writes its zeros.
__device__ __forceinline__ int unit_steps(const TreeParams& p, int u, bool report) {
    return max(1, pages_to_steps(p, unit_pages(p, u, report)));
}

// Bit k: slot base + k is visible to a row with these draft bits.
__device__ __forceinline__ unsigned long long visible64(int base, int ctx, unsigned long long bits) {
    const int d = ctx - base;
    if (d >= 64) return ~0ull;
    if (d > 0) return ((1ull << d) - 1) | (bits << d);
    return d > -64 ? bits >> -d : 0ull;
}

// ---------------------------------------------------------------- producer
template <int D>
__device__ void tree_producer(const CUtensorMap* tk, const CUtensorMap* tv, const TreeParams& p, uint8_t* sT,
                              TreeCtrl* c, int lo, int hi, int per, int t0, volatile WaitFlag* wf) {
    constexpr int NBOX = D / 64, T_BOX = kStep * 128, T_BYTES = NBOX * T_BOX;
    const int lane = threadIdx.x & 31;
    const bool leader = elect_one();
    const int ppt = p.page == 64 ? 2 : 1, shift = page_shift(p);
    const int mult = p.row_ptr ? 1 : p.Hkv, cta = blockIdx.y * p.RT + blockIdx.x;
    uint32_t slot = 0, phase = 0, nload = 0, g = 0, nq = 0;
    bool ok = true, ended = false;
    Meta mt{-1, 0, per, 0, 0, 0, 0, 0};
    if (lo < hi) {
        // the unit that holds step lo: last u whose first step is not behind it
        int u = 0;
        for (int span = p.units; span > 1;) {
            const int stride = (span + 31) >> 5, off = lane * stride;
            const bool le = off < span && c->prefix[u + off] * mult <= lo;
            u += (__popc(__ballot_sync(0xffffffffu, le)) - 1) * stride;
            span = min(stride, p.units - u);
        }
        int base = c->prefix[u], per_item = c->prefix[u + 1] - base;
        int k = lo == base * mult ? 0 : (lo - base * mult) / per_item;  // item of the unit
        int pos = lo;
        while (ok && pos < hi) {
            const int gu = p.unit0 + u;  // unit of the whole call
            const int b = p.row_ptr ? gu / p.Hkv : gu;
            const int ctx = seq_ctx(p, b), dl = seq_dl(p, b);
            const uint32_t len = (uint32_t)ctx + dl;
            const int start = base * mult + k * per_item, end = start + per_item;
            const int s0 = pos - start, s1 = min(end, hi) - start;
            // the first pages are looked up before the item's length is known:
            // list entries, or without a list the table's
            const int64_t beg = p.row_ptr ? p.row_ptr[gu] : 0;
            int pre = 0;
            if (!p.row_ptr) {
                pre = p.table[(int64_t)b * p.P + min(s0 * ppt + lane, p.P - 1)];
            } else {
                const int64_t at = min(beg + s0 * ppt + lane, p.col_cap - 1);
                if (at >= 0) pre = p.col_idx[at];
            }
            const int n = unit_pages(p, gu, false);
            const int h = p.row_ptr ? gu - b * p.Hkv : k;
            const bool whole = s0 == 0 && start + s1 == end;
            const int part = whole ? -1 : 2 * cta + (pos == lo ? 0 : 1);
            if (start < lo) mt = Meta{start, end, per, b, h, t0, dl, 0};
            // the Q loader's turn, as soon as its buffer is free
            if (nq >= kQAhead && !twait(&c->qi_empty[nq % kQAhead], ((nq / kQAhead) & 1) ^ 1, wf)) {
                ok = false;
                break;
            }
            if (leader) {
                c->qitem[nq % kQAhead] = make_int2(h * p.G, b * p.T + t0);
                mbar_arrive(&c->qi_full[nq % kQAhead]);
            }
            ++nq;
            // steps, 32 pages resolved at a time
            for (int e0 = s0 * ppt; e0 < s1 * ppt && ok; e0 += 32) {
                const int e = e0 + lane;
                int nv = 0, j = 0, y = -p.page;
                if (e < n && e < s1 * ppt) {
                    j = !p.row_ptr ? e : e0 > s0 * ppt ? p.col_idx[beg + e] : pre;
                    if ((unsigned)j >= (unsigned)p.P) {
                        atomicOr(p.err, ERR_BAD_COL);
                        j = 0;
                    } else {
                        const uint32_t first = (uint32_t)j << shift;
                        nv = len > first ? (int)min(len - first, (uint32_t)p.page) : 0;
                        if (nv > 0) {
                            const int pg = p.row_ptr || e0 > s0 * ppt ? p.table[(int64_t)b * p.P + j] : pre;
                            if ((unsigned)pg < (unsigned)p.n_pages) {
                                y = (pg * p.Hkv + h) * p.page;
                            } else {
                                atomicOr(p.err, ERR_BAD_PAGE);
                                nv = 0;
                            }
                        }
                    }
                }
                const int cnt = min(32, s1 * ppt - e0);
                for (int q = 0; q < cnt && ok; q += ppt) {
                    const int sl0 = __shfl_sync(0xffffffffu, j, q) << shift, nv0 = __shfl_sync(0xffffffffu, nv, q);
                    const int y0 = __shfl_sync(0xffffffffu, y, q);
                    const int q1 = q + ppt - 1;  // the step's second page, if it has two
                    const int sl1 = __shfl_sync(0xffffffffu, j, q1) << shift, nv1 = __shfl_sync(0xffffffffu, nv, q1);
                    const int y1 = __shfl_sync(0xffffffffu, y, q1);
                    const int st = (e0 + q) >> (ppt - 1);
                    const uint32_t is = g % kInfos;
                    if (g >= kInfos && !twait(&c->i_empty[is], ((g / kInfos) & 1) ^ 1, wf)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        StepInfo& f = c->info[is];
                        // written before the K tile's barrier is armed, by the same lane
                        const bool plain = nv0 == p.page && sl0 + p.page <= ctx &&
                                           (ppt == 1 || (nv1 == p.page && sl1 + p.page <= ctx));
                        f.flags = (st == s0 ? kFirst : 0) | (st + 1 == s1 ? kLast : 0) | (plain ? 0 : kMask);
                        f.slot0[0] = sl0;
                        f.slot0[1] = ppt == 2 ? sl1 : sl0 + 64;
                        f.nv[0] = nv0;
                        f.nv[1] = ppt == 2 ? nv1 : nv0;
                        f.b = b;
                        f.h = h;
                        f.t0 = t0;
                        f.ctx = ctx;
                        f.dl = dl;
                        f.part = part;
                        const bool wrap = slot + 1 == (uint32_t)p.n_slots;
                        f.vslot = (wrap ? 0 : slot + 1) | ((phase ^ (wrap ? 1u : 0u)) << 31);
                    }
                    __syncwarp();
                    ++g;
                    if (leader) c->issued = g;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (nload >= (uint32_t)p.n_slots && !twait(&c->t_empty[slot], phase ^ 1, wf)) {
                            ok = false;
                            break;
                        }
                        if (leader) {
                            mbar_arrive_expect_tx(&c->t_full[slot], T_BYTES);
#pragma unroll
                            for (int x = 0; x < NBOX; ++x) {
                                uint8_t* dst = sT + slot * T_BYTES + x * T_BOX;
                                tma_load_2d(dst, kv ? tv : tk, &c->t_full[slot], x * 64, y0);
                                if (ppt == 2) tma_load_2d(dst + 64 * 128, kv ? tv : tk, &c->t_full[slot], x * 64, y1);
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
            if (++k == mult && pos < hi) {
                k = 0;
                ++u;
                base = c->prefix[u];
                per_item = c->prefix[u + 1] - base;
            }
        }
    }
    if (ok) {
        // the end mark, with a slot's barrier; the MMA lane passes it on
        const uint32_t is = g % kInfos;
        if (twait(&c->i_empty[is], ((g / kInfos) & 1) ^ 1, wf) && twait(&c->t_empty[slot], phase ^ 1, wf) &&
            leader) {
            c->info[is].flags = kEnd;
            mbar_arrive(&c->t_full[slot]);
            ended = true;
        }
        if (twait(&c->qi_empty[nq % kQAhead], ((nq / kQAhead) & 1) ^ 1, wf) && leader) {
            c->qitem[nq % kQAhead] = make_int2(-1, 0);
            mbar_arrive(&c->qi_full[nq % kQAhead]);
        }
    }
    if (lane == 0) p.meta[cta] = mt;
    __syncwarp();
    if (leader) {
        // copies still in flight must land before the CTA exits (the end mark
        // used the slot of the oldest one, which was consumed before)
        const uint32_t ns = (uint32_t)p.n_slots;
        for (uint32_t n = nload > ns ? nload - ns + (ended ? 1 : 0) : (ended && nload == ns ? 1 : 0); n < nload; ++n)
            mbar_wait_drain(&c->t_full[n % ns], (n / ns) & 1);
    }
}

// mbar_wait that leaves it to the caller what a wait beyond the limit means.
__device__ bool mbar_wait_quiet(uint64_t* bar, uint32_t parity, volatile WaitFlag* wf) {
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 31u) == 0 && (wf->abort || globaltimer_ns() - t0 > wf->limit_ns)) return false;
    }
}

// ---------------------------------------------------------------- Q loader
// One lane.  An item's queries go to rows 0 .. of a 128-row tile (and, with
// copies, to rows dup ..); the other rows stay the zeros of the start: the
// tensor cores work on 128 rows whatever there is, and zeros cost less power
// than leftovers do (128K trees, 3,000 calls on end, where the power limit
// lowers the clock: 319 -> 313 us).  A warp of its own, so that waiting for the
// one buffer holds up no K / V tile.
template <int D, int NS>
__device__ void tree_q_loader(const CUtensorMap* tq, const TreeParams& p, uint8_t* sQ, TreeCtrl* c,
                              volatile WaitFlag* wf) {
    constexpr int NBOX = D / 64;
    const int copies = p.dup ? NS : 1;
    if (elect_one()) {
        uint32_t n = 0;
        for (;; ++n) {
            const uint32_t qi = n % kQAhead;
            // the next item is announced when this one's loads are through, which
            // may take longer than a wait: the limit counts from the last step issued
            bool there;
            uint32_t seen;
            do {
                seen = c->issued;
                there = mbar_wait_quiet(&c->qi_full[qi], (n / kQAhead) & 1, wf);
            } while (!there && !wf->abort && c->issued != seen);
            if (!there) {
                wf->abort = 1;
                break;
            }
            const int2 it = c->qitem[qi];
            mbar_arrive(&c->qi_empty[qi]);
            if (it.x < 0 || !mbar_wait(&c->q_empty, (n & 1) ^ 1, wf)) break;
            mbar_arrive_expect_tx(&c->q_full, (uint32_t)(p.tq * p.G * 128 * NBOX * copies));
#pragma unroll
            for (int x = 0; x < NBOX; ++x)
                for (int y = 0; y < copies; ++y)
                    tma_load_3d(sQ + x * kQBox + y * p.dup * 128, tq, &c->q_full, x * 64, it.x, it.y);
        }
        // a copy still in flight must land before the CTA exits
        if (n > 0) mbar_wait_drain(&c->q_full, (n - 1) & 1);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- MMA
// One lane does everything: a wait of the whole warp (vote included) costs
// ~130 cycles even when its barrier is ready, and four of them per step left
// the tensor pipe idle half the time (4 contexts of 128K slots, 16 drafts, 8
// key heads of 64: 232 us; 200 us since).  Step descriptions come with the K
// tile's barrier: the producer writes them before it arms it, and does not
// come round to them again before the ring has (kInfos is more than the ring's
// steps).  The lane passes them on with its own arrival on the scores'
// barrier, so the softmax has one wait per step.
template <int D, int NS>
__device__ void tree_mma(const TreeParams& p, uint8_t* sQ, uint8_t* sT, TreeCtrl* c, uint32_t tmem,
                         volatile WaitFlag* wf) {
    constexpr int NBOX = D / 64, T_BOX = kStep * 128, T_BYTES = NBOX * T_BOX;
    constexpr uint64_t KDESC = sdesc_sw128_base(16, 1024), VDESC = sdesc_sw128_base(T_BOX, 1024);
    constexpr uint32_t IQK = idesc_bf16_f32(128, kStep, false), IPV = idesc_bf16_f32(128, D, true);
    constexpr int O_COL = 2 * kStep;
    if (elect_one()) {
        uint32_t slot = 0, phase = 0, nq = 0, pslot = 0, pphase = 0;
        bool pend = false, pfirst = false;
        auto issue_pv = [&](uint32_t pg) -> bool {
            const uint32_t sb = pg & 1;
            if (!mbar_wait(&c->t_full[pslot], pphase, wf) || !mbar_wait(&c->p_full[sb], (pg >> 1) & 1, wf)) return false;
            tc_fence_after();
            const uint64_t vdesc = VDESC + (smem_u32(sT + pslot * T_BYTES) >> 4);
#pragma unroll
            for (int kk = 0; kk < 2 * kStep / 16; ++kk) {
                // 16 keys, high parts of P, then the same keys' low parts;
                // an accumulator for every split's keys
                const int k16 = kk >> 1, h = k16 / (8 / NS);
                mma_ts(tmem + O_COL + h * D, tmem + sb * kStep + (k16 >> 1) * 32 + (kk & 1) * 16 + (k16 & 1) * 8,
                       vdesc + (uint64_t)((k16 * 16 * 128) >> 4), IPV, (pfirst && kk % (16 / NS) == 0) ? 0u : 1u);
            }
            mma_commit(&c->pv_done[sb]);
            mma_commit(&c->t_empty[pslot]);
            return true;
        };
        for (uint32_t g = 0;; ++g) {
            if (!mbar_wait(&c->t_full[slot], phase, wf)) break;
            const int flags = c->info[g % kInfos].flags;
            if (flags & kEnd) {
                if (pend && !issue_pv(g - 1)) break;
                mbar_arrive(&c->s_full[g & 1]);
                mbar_arrive(&c->s_full[g & 1]);
                break;
            }
            const uint32_t sb = g & 1;
            if ((flags & kFirst) && !mbar_wait(&c->q_full, nq & 1, wf)) break;
            tc_fence_after();
            const uint64_t kdesc = KDESC + (smem_u32(sT + slot * T_BYTES) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t qd = KDESC + (smem_u32(sQ + (kk >> 2) * kQBox + (kk & 3) * 32) >> 4);
                mma_ss(tmem + sb * kStep, qd, kdesc + (uint64_t)(((kk >> 2) * T_BOX + (kk & 3) * 32) >> 4), IQK,
                       kk > 0 ? 1u : 0u);
            }
            mma_commit(&c->s_full[sb]);
            mbar_arrive(&c->s_full[sb]);  // what this lane has seen (the step's description) the softmax sees
            mma_commit(&c->t_empty[slot]);
            if (flags & kLast) {
                mma_commit(&c->q_empty);
                ++nq;
            }
            if (pend && !issue_pv(g - 1)) break;
            pend = true;
            pfirst = flags & kFirst;
            // the V tile follows in the ring
            if (++slot == (uint32_t)p.n_slots) {
                slot = 0;
                phase ^= 1;
            }
            pslot = slot;
            pphase = phase;
            if (++slot == (uint32_t)p.n_slots) {
                slot = 0;
                phase ^= 1;
            }
        }
        mma_commit(&c->drain);
        mbar_wait_drain(&c->drain, 0);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- softmax
// Natural-log LSE of a row from its reference (log2) and sum: -infinity where
// nothing was visible, NaN where the row's scores are not numbers.
__device__ __forceinline__ float row_lse(float m, float sum) {
    return sum == 0.f ? -INFINITY : (m + __log2f(sum)) * 0.69314718055994531f;
}

// Columns whose bit is 0 score -infinity (whatever stood there, NaN included).
__device__ __forceinline__ void hide(uint32_t (&s)[32], uint32_t vis) {
#pragma unroll
    for (int q = 0; q < 32; ++q)
        if (!((vis >> q) & 1u)) s[q] = __float_as_uint(-INFINITY);
}

// p = 2^(s * sl2 - m) of 32 NG columns as bf16 high and low parts; their sum.
// m = -infinity: nothing was visible yet (0 stands in, every p is 0).
template <int NG>
__device__ __forceinline__ f2 weights(const uint32_t (&s)[NG][32], f2 sl2, float m, uint32_t (&hi)[NG][16],
                                      uint32_t (&lo)[NG][16]) {
    const float ref = m == -INFINITY ? 0.f : m;
    const f2 nm2 = {-ref, -ref};
    f2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int x = 0; x < NG; ++x)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const f2 a = fma2({__uint_as_float(s[x][2 * q]), __uint_as_float(s[x][2 * q + 1])}, sl2, nm2);
            const f2 e = {ex2_approx(a.x), ex2_approx(a.y)};
            sum[q & 1] = add2(sum[q & 1], e);
            hi[x][q] = pack_bf16x2(e.x, e.y);
            const f2 n = {-__uint_as_float(hi[x][q] << 16), -__uint_as_float(hi[x][q] & 0xffff0000u)};
            const f2 r = add2(e, n);
            lo[x][q] = pack_bf16x2(r.x, r.y);
        }
    return add2(sum[0], sum[1]);
}

// Warpgroup wh (threads 128 wh ..): columns 64 wh .. of every step.
template <int D, int NS>
__device__ void tree_softmax(const TreeParams& p, uint8_t* sT, float4* xo, TreeCtrl* c, uint32_t tmem,
                             volatile WaitFlag* wf) {
    constexpr int O_COL = 2 * kStep;
    constexpr int NG = 4 / NS;  // 32-column groups of a split
    const int wg = threadIdx.x >> 7, tl = threadIdx.x & 127, lane = threadIdx.x & 31;
    const int wh = NS == 4 ? tl >> 5 : wg;  // split
    const uint32_t lanes = (uint32_t)(tl & 96) << 16;
    const uint32_t t_o = tmem + lanes + O_COL + wh * D;
    // query row of this TMEM lane (the other splits work on the copies, if there are any)
    const int rows = p.tq * p.G, row = NS == 4 ? lane : (tl - wh * p.dup) & 127, group = row >> 5;
    const int rt = row / p.G, rg = row - rt * p.G;  // its drafted token (in the tile) and query head
    // the whole warp lies behind the tile's rows, or its warpgroup is not needed
    const bool idle = NS == 4 ? wg == 1 : (row & 96) >= rows;
    // V's rows are zeroed by the idle warps, if there are any, else by all: this
    // thread's number among them (below 0: none), their number
    const int busy = rows > 96 ? 0 : (rows + 31) & ~31;
    const int zi = NS == 4 ? (wg ? tl : -1) : row - busy, zn = NS == 4 ? 128 : 128 - busy;
    constexpr int SR = NS == 4 ? 32 : 128;  // rows of a split's sums
    float m = -INFINITY, l = 0.f;
    const f2 sl2 = {p.scale_log2, p.scale_log2};
    uint32_t items = 0;
    // The item whose last product is still to come.  Its result is written after
    // the next item's first weights are taken, which takes as long as that
    // product does, and before those are handed over, since the next product
    // starts O anew (96 sequences up to 600 slots: 51 -> 43 us).
    bool pending = false;
    int b = 0, h = 0, t = 0, dl = 0, part = 0;
    for (uint32_t g = 0;; ++g) {
        const uint32_t is = g % kInfos, sb = g & 1;
        const StepInfo& f = c->info[is];
        if (!twait(&c->s_full[sb], (g >> 1) & 1, wf)) break;
        tc_fence_after();
        const int flags = f.flags;
        if (!(flags & kEnd)) {
            uint32_t vis[2] = {~0u, ~0u};  // visible slots among this split's
            if (flags & kMask) {
                const int half = wh * NG / 2, tok = f.t0 + rt, n = f.dl, nv = f.nv[half];
                unsigned long long bits = 0;
                if (tok < n) {
                    bits = p.mask ? p.mask[(int64_t)f.b * p.T + tok] : (2ull << tok) - 1;
                    if (n < 64) bits &= (1ull << n) - 1;
                }
                const unsigned long long v = nv > 0 ? visible64(f.slot0[half], f.ctx, bits) : 0ull;
                vis[0] = (uint32_t)(NS == 4 && (wh & 1) ? v >> 32 : v);
                vis[1] = (uint32_t)(v >> 32);
                // The V rows of a page's unused slots are zeroed (this half's
                // keys): their weights are 0, but 0 * NaN would reach O.  A page
                // that holds nothing was not loaded, its rows are zeros already.
                if (zi >= 0) {
                    const int h0 = NS == 4 ? 0 : wh, h1 = NS == 4 ? 2 : wh + 1;
                    const uint32_t vslot = (uint32_t)f.vslot;
                    bool landed = false;
                    for (int hh = h0; hh < h1; ++hh) {
                        const int used = p.page == 64 ? f.nv[hh] : min(max(f.nv[hh] - hh * 64, 0), 64);
                        if (f.nv[hh] <= 0 || used >= 64) continue;
                        if (!landed) landed = twait(&c->t_full[vslot & 0x7fffffffu], vslot >> 31, wf);
                        if (!landed) break;
                        uint8_t* tile = sT + (vslot & 0x7fffffffu) * (D / 64 * kStep * 128) + (hh * 64 + used) * 128;
                        for (int x = zi; x < (64 - used) * 8 * (D / 64); x += zn) {
                            const int r = x / (D / 8), q = x % (D / 8);
                            *reinterpret_cast<uint4*>(tile + (q >> 3) * (kStep * 128) + r * 128 + (q & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                    }
                    if (landed) fence_proxy_async_smem();
                }
            }
            if (flags & kFirst) {
                m = -INFINITY;
                l = 0.f;
            }
            if (!idle) {
                const uint32_t t_s = tmem + lanes + sb * kStep + wh * NG * 32;
                uint32_t s[NG][32], hi[NG][16], lo[NG][16];
#pragma unroll
                for (int x = 0; x < NG; ++x) tmem_ld32(t_s + x * 32, s[x]);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < NG; ++x) {
                    reg_fence(s[x]);
                    if (flags & kMask) hide(s[x], vis[x]);
                }
                float mx[2 * NG];
#pragma unroll
                for (int x = 0; x < 2 * NG; ++x) {
                    const uint32_t* v = s[x >> 1] + (x & 1) * 16;
                    mx[x] = __uint_as_float(v[0]);
#pragma unroll
                    for (int q = 1; q < 15; q += 2)
                        mx[x] = fmax3(mx[x], __uint_as_float(v[q]), __uint_as_float(v[q + 1]));
                    mx[x] = fmaxf(mx[x], __uint_as_float(v[15]));
                }
                float top = fmaxf(mx[0], mx[1]);
                if (NG == 2) top = fmax3(top, mx[2 * NG - 2], mx[2 * NG - 1]);
                top *= p.scale_log2;
                // raise the reference when it would grow by more than 2^8 (exact
                // after the division by the sum, which uses the same reference).
                // Taking the weights before the maximum is known, and again where
                // a score has outgrown the reference, was slower (128K trees of
                // 64-wide heads 200 -> 238 us).
                const bool grow = top > m + 8.f || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, grow)) {
                    const float alpha = grow ? ex2_approx(m - top) : 1.f;
                    if (grow) {
                        m = top;
                        l *= alpha;
                    }
                    if (!(flags & kFirst)) {
                        // O must hold every earlier step's product before it is scaled
                        if (!twait(&c->pv_done[sb ^ 1], ((g - 1) >> 1) & 1, wf)) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < D / 32; ++x) {
                            uint32_t o[32];
                            tmem_ld32(t_o + x * 32, o);
                            tmem_wait_ld();
                            reg_fence(o);
#pragma unroll
                            for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
                            tmem_st32(t_o + x * 32, o);
                        }
                    }
                }
                const f2 all = weights(s, sl2, m, hi, lo);
                __syncwarp();
                l += all.x + all.y;
                // 32 columns of P in the columns of their S: 16 of high parts, 16 of low
#pragma unroll
                for (int x = 0; x < NG; ++x) {
                    tmem_st16(t_s + x * 32, hi[x]);
                    tmem_st16(t_s + x * 32 + 16, lo[x]);
                }
                tmem_wait_st();
            }
        }
        if (pending && !idle) {
            // the item's (or its part's) result: every split's sums and accumulators
            if (!twait(&c->st_full[group], items & 1, wf)) break;
            const bool live = row < rows && t < dl;
            const float2* st = c->stats[items & 1] + row;
            float mm = st[0].x, sum = 0.f, w0 = 0.f, w1 = 0.f;  // w1: of the other half
#pragma unroll
            for (int x = 1; x < NS; ++x) mm = fmaxf(mm, st[x * SR].x);
#pragma unroll
            for (int x = 0; x < NS; ++x) {
                const float2 ml = st[x * SR];
                const float w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mm);
                sum += ml.y * w;  // the same in every split
                if (x == wh) w0 = w;
                else w1 = w;
            }
            const int64_t orow = ((int64_t)b * p.T + t) * p.Hq + h * p.G + rg;
            const int64_t prow = (int64_t)part * rows + row;
            if (part < 0) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
                w0 *= inv;
                w1 *= inv;
                if (live && wh == 0) p.lse[orow] = row_lse(mm, sum);
            } else if (live && wh == 0) {
                p.part_ml[prow] = make_float2(mm, sum);
            }
            if (!twait(&c->pv_done[sb ^ 1], ((g - 1) >> 1) & 1, wf)) break;
            tc_fence_after();
            if constexpr (NS == 4) {
                // every split lays its weighted accumulator down, [split][column / 4][row],
                // and adds up and writes a quarter of the row's columns
#pragma unroll 1
                for (int x = 0; x < D / 32; ++x) {
                    uint32_t o[32];
                    tmem_ld32(t_o + x * 32, o);
                    tmem_wait_ld();
                    reg_fence(o);
                    float4* dst = xo + (wh * (D / 4) + x * 8) * 32 + row;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        dst[q * 32] = make_float4(__uint_as_float(o[4 * q]) * w0, __uint_as_float(o[4 * q + 1]) * w0,
                                                  __uint_as_float(o[4 * q + 2]) * w0,
                                                  __uint_as_float(o[4 * q + 3]) * w0);
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&c->x_full[group]);
                if (!twait(&c->x_full[group], items & 1, wf)) break;
                if (live) {
                    const int64_t col = wh * (D / 4);
                    float4 v[D / 16];
#pragma unroll
                    for (int q = 0; q < D / 16; ++q) {
                        const float4* src = xo + (wh * (D / 16) + q) * 32 + row;
                        v[q] = src[0];
#pragma unroll
                        for (int y = 1; y < NS; ++y) {
                            const float4 o = src[y * (D / 4) * 32];
                            v[q] = make_float4(v[q].x + o.x, v[q].y + o.y, v[q].z + o.z, v[q].w + o.w);
                        }
                    }
                    if (part < 0) {
                        uint2* dst = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * D + col);
#pragma unroll
                        for (int q = 0; q < D / 16; ++q)
                            dst[q] = make_uint2(pack_bf16x2(v[q].x, v[q].y), pack_bf16x2(v[q].z, v[q].w));
                    } else {
                        float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + col);
#pragma unroll
                        for (int q = 0; q < D / 16; ++q) dst[q] = v[q];
                    }
                }
            } else {
                const f2 w02 = {w0, w0}, w12 = {p.dup ? 1.f : w1, p.dup ? 1.f : w1};
                // This half writes columns wh * D/2 .. of the row.  With copies the
                // other accumulator lies in other lanes: each half hands over its
                // (weighted) part of the other's columns, [column / 4][row].
                const uint32_t t_a = t_o + wh * (D / 2), t_b = tmem + lanes + O_COL + (wh ^ 1) * D + wh * (D / 2);
                if (p.dup) {
#pragma unroll 1
                    for (int x = 0; x < D / 64; ++x) {
                        uint32_t o[32];
                        tmem_ld32(t_o + (wh ^ 1) * (D / 2) + x * 32, o);
                        tmem_wait_ld();
                        reg_fence(o);
                        float4* dst = xo + (wh * (D / 8) + x * 8) * p.dup + row;
                        if (row < p.dup) {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                dst[q * p.dup] = make_float4(
                                    __uint_as_float(o[4 * q]) * w0, __uint_as_float(o[4 * q + 1]) * w0,
                                    __uint_as_float(o[4 * q + 2]) * w0, __uint_as_float(o[4 * q + 3]) * w0);
                        }
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(&c->x_full[group]);
                    if (!twait(&c->x_full[group], items & 1, wf)) break;
                }
#pragma unroll 1
                for (int x = 0; x < D / 64; ++x) {
                    uint32_t o[32], o1[32];
                    __syncwarp();
                    tmem_ld32(t_a + x * 32, o);
                    if (p.dup) {
                        const float4* src = xo + ((wh ^ 1) * (D / 8) + x * 8) * p.dup + (row & (p.dup - 1));
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float4 f4 = src[q * p.dup];
                            o1[4 * q] = __float_as_uint(f4.x);
                            o1[4 * q + 1] = __float_as_uint(f4.y);
                            o1[4 * q + 2] = __float_as_uint(f4.z);
                            o1[4 * q + 3] = __float_as_uint(f4.w);
                        }
                    } else {
                        tmem_ld32(t_b + x * 32, o1);
                    }
                    tmem_wait_ld();
                    reg_fence(o);
                    reg_fence(o1);
                    if (!live) continue;
                    f2 v[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        v[q] = fma2({__uint_as_float(o1[2 * q]), __uint_as_float(o1[2 * q + 1])}, w12,
                                    mul2({__uint_as_float(o[2 * q]), __uint_as_float(o[2 * q + 1])}, w02));
                    const int64_t col = wh * (D / 2) + x * 32;
                    if (part < 0) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * D + col);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            dst[q] = make_uint4(pack_bf16x2(v[4 * q].x, v[4 * q].y),
                                                pack_bf16x2(v[4 * q + 1].x, v[4 * q + 1].y),
                                                pack_bf16x2(v[4 * q + 2].x, v[4 * q + 2].y),
                                                pack_bf16x2(v[4 * q + 3].x, v[4 * q + 3].y));
                    } else {
                        float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + col);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dst[q] = make_float4(v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y);
                    }
                }
            }
        }
        if (flags & kEnd) break;
        if (flags & kFirst) {
            items += pending;
            pending = false;
        }
        if (flags & kLast) {
            // two buffers: the other splits may still be at the item before
            if (!idle) c->stats[items & 1][wh * SR + row] = make_float2(m, l);
            pending = true;
            b = f.b;
            h = f.h;
            t = f.t0 + rt;
            dl = f.dl;
            part = f.part;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&c->i_empty[is]);
            mbar_arrive(&c->p_full[sb]);
            if ((flags & kLast) && !idle) mbar_arrive(&c->st_full[group]);
        }
    }
}

// ---------------------------------------------------------------- kernel
template <int D, int NS>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const TreeParams p) {
    constexpr int NBOX = D / 64, T_BYTES = NBOX * kStep * 128;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {
        griddep_wait();
        if (threadIdx.x == 0) {
            p.meta[blockIdx.y * p.RT + blockIdx.x].start = -1;  // nothing to join
            atomicOr(p.err, ERR_LAUNCH);
        }
        return;
    }
    uint8_t* sQ = smem;
    uint8_t* sT = sQ + NBOX * kQBox;
    float4* xo = reinterpret_cast<float4*>(sT + p.n_slots * T_BYTES);
    TreeCtrl* c = reinterpret_cast<TreeCtrl*>(sT + p.n_slots * T_BYTES + exchange_bytes(D, NS, p.dup));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    {
        const int x = threadIdx.x;
        if (x < kMaxSlots) {
            mbar_init(&c->t_full[x], 1);
            mbar_init(&c->t_empty[x], 1);
        } else if (x >= 32 && x < 32 + kInfos) {
            mbar_init(&c->i_empty[x - 32], 8);  // the softmax warps
        } else if (x >= 64 && x < 66) {
            mbar_init(&c->s_full[x - 64], 2);  // the scores' commit and the MMA lane itself
            mbar_init(&c->p_full[x - 64], 8);
            mbar_init(&c->pv_done[x - 64], 1);
        } else if (x >= 96 && x < 100) {
            mbar_init(&c->st_full[x - 96], NS);
            mbar_init(&c->x_full[x - 96], NS);
            mbar_init(&c->qi_full[x - 96], 1);
            mbar_init(&c->qi_empty[x - 96], 1);
        } else if (x == 128) {
            mbar_init(&c->drain, 1);
            mbar_init(&c->q_full, 1);
            mbar_init(&c->q_empty, 1);
            c->wf.abort = 0;
            c->issued = 0;
            c->wf.limit_ns = p.wait_limit_ns;
            c->prefix[0] = 0;
        }
        fence_mbar_init();
        for (int z = x; z < NBOX * kQBox / 16; z += kTreeThreads)
            reinterpret_cast<uint4*>(sQ)[z] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == kProducer && lane == 0) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    // Nothing before this line reads or writes global memory or takes tensor
    // memory (which a kernel before this one may still want): only what is
    // this CTA's own is set up while that one ends.
    griddep_wait();
    if (warp == kMma) {
        tmem_alloc(&c->tmem_base, 512);
        tmem_relinquish();
    }
    // prefix sums of the units' steps: every thread a run of units, then a scan
    const int mult = p.row_ptr ? 1 : p.Hkv;
    const int run = (p.units + kTreeThreads - 1) / kTreeThreads;
    const int u0 = min(p.units, (int)threadIdx.x * run), u1 = min(p.units, u0 + run);
    int sum = 0;
    for (int u = u0; u < u1; ++u) {
        sum += unit_steps(p, p.unit0 + u, blockIdx.x + blockIdx.y == 0);
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem_base;
    volatile WaitFlag* wf = &c->wf;
    const int total = c->prefix[p.units] * mult;
    const int range = blockIdx.y;
    const int per = (total + p.ranges - 1) / p.ranges;
    const int lo = min(total, range * per), hi = min(total, lo + per);
    const int t0 = (int)blockIdx.x * p.tq;  // first drafted token of the CTA's rows
    if (warp == kProducer)
        tree_producer<D>(&tk, &tv, p, sT, c, lo, hi, per, t0, wf);
    else if (warp == kMma)
        tree_mma<D, NS>(p, sQ, sT, c, tmem, wf);
    else if (warp == kQLoader)
        tree_q_loader<D, NS>(&tq, p, sQ, c, wf);
    else
        tree_softmax<D, NS>(p, sT, xo, c, tmem, wf);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && c->wf.abort) atomicOr(p.err, ERR_TIMEOUT);
}

// ---------------------------------------------------------------- merge
// Block (x, tile) joins the item that the boundary in front of range x + 1 is
// the first to cut, RB query rows of it, 8 / RB warps to a row (each takes every
// (8 / RB)-th part; their sums meet in shared memory).  With parts i in range
// order: m = max m_i, w_i = 2^(m_i - m), O = sum w_i O_i / sum w_i l_i.
// Bound by three dependent reads from the L2 (~2 us, and ~1 us after the last
// CTA of the main kernel); one row over 147 ranges: 27 us for the whole call
// with eight warps to the row, 42 with one.
template <int D, int RB>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams p) {
    constexpr int WPR = 8 / RB, C = D / 32;
    __shared__ float red[WPR > 1 ? WPR : 1][D + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int tile = blockIdx.z, c = blockIdx.x + 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Meta mt = p.meta[c * p.RT + tile];
    if (mt.start < 0) return;
    const int rows = p.tq * p.G, per = mt.per, first = c - 1;
    if (mt.start < first * per) return;  // an earlier boundary cuts it too
    const int last = (mt.end - 1) / per;
    const int r = blockIdx.y * RB + warp / WPR, part = warp % WPR;
    const int t = mt.t0 + r / p.G;
    const bool on = r < rows && t < mt.dl;
    if (WPR == 1 && !on) return;
    auto slot_of = [&](int k) { return 2 * (k * p.RT + tile) + (k == first && mt.start > first * per ? 1 : 0); };
    float m = -INFINITY, l = 0.f, acc[C];
#pragma unroll
    for (int x = 0; x < C; ++x) acc[x] = 0.f;
    if (on) {
        for (int k = first + lane; k <= last; k += 32) m = fmaxf(m, p.part_ml[(int64_t)slot_of(k) * rows + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m > -INFINITY ? m : 0.f;
#pragma unroll 4
        for (int k = first + part; k <= last; k += WPR) {
            const int64_t pr = (int64_t)slot_of(k) * rows + r;
            const float2 ml = p.part_ml[pr];
            const float w = ex2_approx(ml.x - ref);  // 0 for a part that saw nothing
            l += w * ml.y;
            if (C == 4) {
                const float4 o = reinterpret_cast<const float4*>(p.part_o + pr * D)[lane];
                acc[0] += w * o.x;
                acc[1] += w * o.y;
                acc[C - 2] += w * o.z;
                acc[C - 1] += w * o.w;
            } else {
                const float2 o = reinterpret_cast<const float2*>(p.part_o + pr * D)[lane];
                acc[0] += w * o.x;
                acc[1] += w * o.y;
            }
        }
    }
    if (WPR > 1) {
#pragma unroll
        for (int x = 0; x < C; ++x) red[part][lane * C + x] = acc[x];
        if (lane == 0) red[part][D] = l;
        __syncthreads();
        if (part > 0 || !on) return;
        for (int w = 1; w < WPR; ++w) {
#pragma unroll
            for (int x = 0; x < C; ++x) acc[x] += red[w][lane * C + x];
            l += red[w][D];
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t orow = ((int64_t)mt.b * p.T + t) * p.Hq + mt.h * p.G + r % p.G;
    if (lane == 0) p.lse[orow] = row_lse(m, l);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + orow * D;
    if (C == 4)
        reinterpret_cast<uint2*>(out)[lane] =
            make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[C - 2] * inv, acc[C - 1] * inv));
    else
        reinterpret_cast<uint32_t*>(out)[lane] = pack_bf16x2(acc[0] * inv, acc[1] * inv);
}

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// TMEM lanes between the query rows and their copies, 0 for none; 32: four
// splits of a step's columns, else two.  TMEM ties a
// warp to a quarter of the lanes, and a quarter to one of the SM's four
// schedulers: with few rows both halves' warps share one, and its exponentials
// are what a step of 64-wide heads waits for.  A second copy of Q in lanes of
// its own puts the second half's warps on other schedulers: 4 contexts of 128K
// slots, 64 rows: 200 -> 177 us; 96 ragged sequences up to 8K, 4 rows: 197 ->
// 173 us.  Up to 32 rows there is room for four copies, a quarter of the columns
// each (155.6 -> 153.6 us, listed trees 44.7 -> 43.8).  At 128-wide heads a step has twice the bytes to hide the same
// softmax, and the ring slot that the copies cost is worth more (4 rows: 290
// us without, 293 with them).
int row_copies(int rows, int D) {
    if (D != 64 || rows > 64) return 0;
    return rows <= 32 ? 32 : 64;
}

// Drafted tokens of a row tile: as many as fit 128 rows.
int tile_tokens(int T, int G) { return std::min(T, 128 / G); }

int64_t ws_part_offset() { return (kMaxCtas * (int64_t)sizeof(Meta) + 255) / 256 * 256; }

template <int D, int NS>
int launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, TreeParams p, int units,
                int chunk, size_t smem, cudaStream_t s) {
    static_assert(sizeof(TreeCtrl) <= kCtrlBytes, "control block too large");
    static std::atomic<uint64_t> raised{0};
    if (raise_smem_limit(reinterpret_cast<const void*>(tree_kernel<D, NS>), kTreeSmem, &raised) != cudaSuccess)
        return BSA_ERR_CUDA;
    for (int u0 = 0; u0 < units; u0 += chunk) {
        p.unit0 = u0;
        p.units = std::min(chunk, units - u0);
        cudaError_t e = launch_after(tree_kernel<D, NS>, dim3((unsigned)p.RT, (unsigned)p.ranges), kTreeThreads, smem,
                                     s, tq, tk, tv, p);
        if (e != cudaSuccess) return BSA_ERR_CUDA;
        if (p.ranges < 2) continue;
        // few rows: their parts are dealt over eight warps; many: a warp each
        const int rows = p.tq * p.G, rb = rows <= 16 ? 1 : 8;
        e = launch_after(rb == 1 ? tree_merge_kernel<D, 1> : tree_merge_kernel<D, 8>,
                         dim3((unsigned)p.ranges - 1, (unsigned)((rows + rb - 1) / rb), (unsigned)p.RT), 256, 0, s, p);
        if (e != cudaSuccess) return BSA_ERR_CUDA;
    }
    return BSA_OK;
}

}  // namespace
}  // namespace bsa

extern "C" {

int64_t bsa_tree_attention_workspace(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D) {
    if (B <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv || Hq / Hkv > 128) return 0;
    const int64_t rows = (int64_t)bsa::tile_tokens(T, Hq / Hkv) * (Hq / Hkv);
    return bsa::ws_part_offset() + 2ll * bsa::kMaxCtas * rows * (D + 2) * (int64_t)sizeof(float);
}

int bsa_tree_attention(const bsa_tree_args* a, const bsa_page_cache* c, void* workspace, int64_t workspace_bytes,
                       bsa_stream_t stream) {
    if (!a) return BSA_ERR_INVALID_ARG;
    int st = bsa::check_page_cache(c);
    if (st != BSA_OK) return st;
    if (a->B < 0 || a->T <= 0 || a->Hq <= 0 || a->Hq % c->Hkv || c->layers != 1 || c->n_seqs != a->B)
        return BSA_ERR_INVALID_ARG;
    if (a->B > 0 && (!a->q || !a->context_len || !a->out || !a->lse || !c->page_table)) return BSA_ERR_INVALID_ARG;
    if (!bsa::al(a->q, 16) || !bsa::al(a->out, 16) || !bsa::al(a->lse, 4) || !bsa::al(a->context_len, 4) ||
        !bsa::al(a->draft_len, 4) || !bsa::al(a->tree_mask, 8) || !bsa::al(a->row_ptr, 4) || !bsa::al(a->col_idx, 4))
        return BSA_ERR_INVALID_ARG;
    if ((a->row_ptr != nullptr) != (a->col_idx != nullptr) || a->col_capacity < 0) return BSA_ERR_INVALID_ARG;
    if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return BSA_ERR_INVALID_ARG;
    if (a->T > BSA_MAX_DRAFT || a->Hq / c->Hkv > 128) return BSA_ERR_UNSUPPORTED;
    if (a->B == 0) return BSA_OK;
    if (!workspace || !bsa::al(workspace, 256)) return BSA_ERR_INVALID_ARG;
    if (workspace_bytes < bsa_tree_attention_workspace(a->B, a->T, a->Hq, c->Hkv, c->D)) return BSA_ERR_CAPACITY;
    bsa::TreeParams p{};
    p.G = a->Hq / c->Hkv;
    p.tq = bsa::tile_tokens(a->T, p.G);
    p.RT = (a->T + p.tq - 1) / p.tq;
    // the steps of one launch stay below 2^30 (sums and range ends fit an int)
    const int64_t mult = a->row_ptr ? 1 : c->Hkv;
    const int64_t most = ((int64_t)c->max_pages * c->page + bsa::kStep - 1) / bsa::kStep;
    const int64_t units = a->row_ptr ? (int64_t)a->B * c->Hkv : a->B;
    if ((int64_t)a->B * a->T > INT32_MAX || units >= INT32_MAX || mult * most > 1 << 30) return BSA_ERR_INVALID_ARG;
    const int chunk = (int)std::min<int64_t>(bsa::kMaxUnits, (1 << 30) / (mult * most));
    int sms;
    if ((st = bsa::device_context(&p.err, &sms)) != BSA_OK) return st;
    const int rows = p.tq * p.G, nbox = c->D / 64;
    p.dup = bsa::row_copies(rows, c->D);
    const int tile = nbox * bsa::kStep * 128;
    const int splits = p.dup == 32 ? 4 : 2;
    const int fixed = bsa::kCtrlBytes + nbox * bsa::kQBox + bsa::exchange_bytes(c->D, splits, p.dup);
    p.n_slots = std::min(bsa::kMaxSlots, (bsa::kTreeSmem - fixed) / tile);
    const size_t smem = (size_t)p.n_slots * tile + fixed;
    CUtensorMap tq, tk, tv;
    const uint64_t krows = (uint64_t)c->n_pages * c->Hkv * c->page;
    if ((st = bsa::encode_token_rows_bf16(&tq, a->q, (uint64_t)a->B * a->T, a->Hq, c->D, p.G, p.tq)) != BSA_OK) return st;
    if ((st = bsa::encode_rows_bf16(&tk, c->k, krows, c->D, c->page)) != BSA_OK) return st;
    if ((st = bsa::encode_rows_bf16(&tv, c->v, krows, c->D, c->page)) != BSA_OK) return st;
    p.ctx = a->context_len;
    p.dl = a->draft_len;
    p.row_ptr = a->row_ptr;
    p.col_idx = a->col_idx;
    p.table = c->page_table;
    p.mask = reinterpret_cast<const unsigned long long*>(a->tree_mask);
    p.col_cap = a->col_capacity;
    p.B = a->B;
    p.T = a->T;
    p.Hq = a->Hq;
    p.Hkv = c->Hkv;
    p.page = c->page;
    p.P = c->max_pages;
    p.n_pages = c->n_pages;
    p.ranges = std::max(1, std::min(sms, bsa::kMaxCtas) / p.RT);  // RT <= 64
    p.out = a->out;
    p.lse = a->lse;
    p.meta = static_cast<bsa::Meta*>(workspace);
    p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + bsa::ws_part_offset());
    p.part_ml = reinterpret_cast<float2*>(p.part_o + 2ll * bsa::kMaxCtas * rows * c->D);
    p.scale_log2 = a->scale * 1.4426950408889634f;
    p.wait_limit_ns = bsa::wait_limit_ns();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto launch = c->D == 128  ? bsa::launch_tree<128, 2>
                  : splits == 4 ? bsa::launch_tree<64, 4>
                                : bsa::launch_tree<64, 2>;
    return launch(tq, tk, tv, p, (int)units, chunk, smem, s);
}

}  // extern "C"
