// bsa_cache.cu -- the pages of a key/value cache: requests for pages (resize,
// fork), defragmentation (compact) and the compaction of accepted drafts
// within a sequence (accept).  No arithmetic: integer bookkeeping on the
// device, so a serving loop never waits for it, and copies at the rate of
// device memory.
//
// A request runs as three launches, few requests as two (check and plan in one
// CTA).  Check: one warp per request walks its table row, finds whether it can
// be served and how many pages it takes, and snapshots page_ref.  Plan: one CTA settles repeated sequences, adds up the
// needs in request order and lists that many free pages, lowest first.
// Apply: table and counts (a warp per request) and, in the other CTAs, the
// rows of part-filled pages.  Every decision is taken on the snapshot and the
// free list holds only pages that were free in it, so requests that share
// pages do not see each other's changes, a copy never reads a page that the
// same call writes, and the result does not depend on the order of the warps.
//
// Bound by DRAM where rows move (983 pages of 512 KB in each of two pools: 150
// us, 6.9 TB/s), else by the launches: 8.5 us for a call that moves nothing.

#include <algorithm>

#include "bsa.h"
#include "bsa_internal.h"
#include "bsa_ptx.cuh"

namespace bsa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kHeader = 64;  // ints in front of the workspace's arrays

struct PageWs {
    int32_t* head;      // [0]: moved pages (compact)
    int32_t* need;      // [n] pages the request takes, -1: cannot be served
    int32_t* offset;    // [n] first of them in the free list
    int32_t* src;       // [n] page whose rows are copied
    int32_t* rows;      // [n] rows of it (0: none)
    int32_t* claim;     // [n_seqs] first request of a sequence
    int32_t* free_list; // [n_pages]; compact: holes
    int32_t* ref0;      // [n_pages] snapshot of page_ref; compact: movers
};

int64_t ws_ints(int64_t n, int64_t n_seqs, int64_t n_pages) { return kHeader + 4 * n + n_seqs + 2 * n_pages; }

PageWs split_ws(void* ws, int64_t n, int64_t n_seqs, int64_t n_pages) {
    PageWs w;
    w.head = static_cast<int32_t*>(ws);
    w.need = w.head + kHeader;
    w.offset = w.need + n;
    w.src = w.offset + n;
    w.rows = w.src + n;
    w.claim = w.rows + n;
    w.free_list = w.claim + n_seqs;
    w.ref0 = w.free_list + n_pages;
    return w;
}

struct PageReq {
    int32_t* table;
    int32_t* ref;
    int32_t n_seqs, max_pages, n_pages, page;
    int32_t n;
    const int32_t *a, *b, *c;  // resize: seqs, keep, capacity; fork: dst, src, len
    int32_t* granted;
    int32_t* err;
    PageWs w;
    // copies
    uint4 *k, *v;
    uint8_t *ks, *vs;            // 8-bit pools: a scale byte per row (else null)
    int32_t layers, Hkv, row16;  // row16: 16-byte chunks of a row
};

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Entries of a table row before its first -1 (whole warp).
__device__ int row_held(const int32_t* row, int max_pages) {
    const int lane = threadIdx.x & 31;
    for (int j0 = 0; j0 < max_pages; j0 += 128) {
        int e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + u * 32 + lane;
            e[u] = j < max_pages ? row[j] : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const unsigned m = __ballot_sync(0xffffffffu, e[u] < 0);
            if (m) return min(max_pages, j0 + u * 32 + __ffs(m) - 1);
        }
    }
    return max_pages;
}

// Check, one warp per request: thread t of nt (whole warps).
template <bool FORK>
__device__ void check_requests(const PageReq& p, int64_t t, int64_t nt, int32_t* needs) {
    const int lane = threadIdx.x & 31;
    for (int64_t i = t >> 5; i < p.n; i += nt >> 5) {
        int need = -1, src = -1, rows = 0;
        const int seq = p.a[i];
        if ((unsigned)seq < (unsigned)p.n_seqs) {
            const int32_t* row = p.table + (int64_t)seq * p.max_pages;
            const int most = p.max_pages * p.page;
            if (FORK) {
                const int from = p.b[i], len = p.c[i];
                if ((unsigned)from < (unsigned)p.n_seqs && len >= 0 && len <= most && row[0] < 0) {
                    const int32_t* srow = p.table + (int64_t)from * p.max_pages;
                    const int full = len / p.page, part = len % p.page, all = full + (part > 0);
                    int bad = 0;
#pragma unroll 4
                    for (int j = lane; j < all; j += 32) {
                        const int e = srow[j];
                        bad |= (unsigned)e >= (unsigned)p.n_pages || p.ref[e] <= 0;
                    }
                    if (!__any_sync(0xffffffffu, bad)) {
                        need = part > 0;
                        rows = part;
                        if (part) src = srow[full];
                    }
                }
            } else {
                const int keep = p.b[i], cap = p.c[i];
                if (keep >= 0 && keep <= cap && cap <= most) {
                    const int held = row_held(row, p.max_pages);
                    const int full = keep / p.page, part = keep % p.page, first = full + (part > 0);
                    const int want = (int)(((int64_t)cap + p.page - 1) / p.page);
                    int bad = first > held, cnt = 0, cow = 0;
                    for (int j = lane; j < held; j += 32) {
                        const int e = row[j];
                        const int r = (unsigned)e < (unsigned)p.n_pages ? p.ref[e] : 0;
                        bad |= r <= 0;
                        if (j >= first && j < want && r != 1) ++cnt;
                        if (j == full && part && r > 1) {
                            cow = 1;
                            src = e;
                        }
                    }
                    for (int j = max(held, first) + lane; j < want; j += 32) ++cnt;
                    const int any_cow = __any_sync(0xffffffffu, cow);
                    cnt = warp_sum(cnt);
                    src = __reduce_max_sync(0xffffffffu, src);
                    if (!__any_sync(0xffffffffu, bad)) {
                        need = cnt + any_cow;
                        rows = any_cow ? part : 0;
                    }
                }
            }
        }
        if (lane == 0) {
            needs[i] = need;
            p.w.src[i] = src;
            p.w.rows[i] = rows;
        }
    }
}

template <bool FORK>
__global__ void __launch_bounds__(256) pages_check_kernel(const PageReq p) {
    griddep_launch_dependents();
    griddep_wait();
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, nt = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = t; i < p.n_pages; i += nt) p.w.ref0[i] = p.ref[i];
    for (int64_t i = t; i < p.n_seqs; i += nt) p.w.claim[i] = 0x7fffffff;
    check_requests<FORK>(p, t, nt, p.w.need);
}

// Inclusive sum of v over the CTA's threads in order; *total for everyone.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* total, T* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    __syncthreads();
    if (lane == 31) red[warp] = v;
    __syncthreads();
    T w = red[lane];  // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T x = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += x;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const T before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return v + (warp ? before : 0);
}

// Requests in order: the later ones of a repeated sequence drop out, the needs
// are added up, the first free pages listed and the answers given.  needs and
// claims may lie in shared or global memory (barriers between the phases, and
// fences for global memory, are the caller's).
struct Plan {
    const PageReq& p;
    int32_t *needs, *claims, *offsets;

    __device__ void claim() const {
        for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
            const int seq = p.a[i];
            if ((unsigned)seq < (unsigned)p.n_seqs) atomicMin(&claims[seq], i);
        }
    }
    // Sum of the needs (passes 31 bits where requests ask for far more than there is).
    __device__ long long add_up(long long* red64) const {
        long long sum = 0;
        for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
            const int i = i0 + threadIdx.x;
            int need = -1;
            if (i < p.n) {
                need = needs[i];
                if (need >= 0 && static_cast<volatile int32_t*>(claims)[p.a[i]] != i) need = -1;
                needs[i] = need;
            }
            long long total;
            const long long v = max(need, 0);
            const long long before = sum + block_scan(v, &total, red64) - v;
            if (i < p.n) p.w.offset[i] = offsets[i] = (int)min(before, 0x7fffffffll);
            sum += total;
        }
        return sum;
    }
    __device__ void answer(int have) const {
        for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
            const int need = needs[i];
            const bool ok = need == 0 || (need > 0 && (int64_t)offsets[i] + need <= have);
            p.granted[i] = ok;
            if (!ok) {
                p.w.rows[i] = 0;
                atomicOr(p.err, ERR_PAGES);
            }
        }
    }
};

// Plan after the check kernel.
__global__ void __launch_bounds__(kPlanThreads) pages_plan_kernel(const PageReq p) {
    __shared__ int red[32];
    __shared__ long long red64[32];
    const int tid = threadIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    const Plan plan{p, p.w.need, p.w.claim, p.w.offset};
    plan.claim();
    __threadfence();
    __syncthreads();
    const long long sum = plan.add_up(red64);
    // the free pages, ascending, as many as are asked for
    int have = 0;
    for (int i0 = 0; i0 < p.n_pages && have < sum; i0 += 4 * kPlanThreads) {
        int fr[4], cnt = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 4 * tid + u;
            fr[u] = i < p.n_pages && p.w.ref0[i] == 0;
            cnt += fr[u];
        }
        int total;
        int at = have + block_scan(cnt, &total, red) - cnt;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (fr[u]) p.w.free_list[at++] = i0 + 4 * tid + u;
        have += total;
    }
    plan.answer(have);
}

// Check and plan of few requests in one CTA, with what the phases hand on in
// shared memory (free pages as bits).  32 requests of 16 pages in a pool of
// 3,000: 10.1 to 12.4 us for the two kernels, 7.4 to 9.2 in one CTA over global
// memory, 1.2 less in shared memory.  For many requests, long rows or a large
// pool the check is worth the whole GPU.
constexpr int kSmallRequests = 2048, kSmallSeqs = 4096, kSmallPages = 32 * kPlanThreads / 2;
template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) pages_small_kernel(const PageReq p) {
    __shared__ int red[32];
    __shared__ long long red64[32];
    __shared__ int32_t needs[kSmallRequests], offsets[kSmallRequests], claims[kSmallSeqs];
    __shared__ unsigned free_bits[kSmallPages / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    for (int i = tid; i < p.n_seqs; i += kPlanThreads) claims[i] = 0x7fffffff;
    for (int i0 = tid - lane; i0 < p.n_pages; i0 += kPlanThreads) {
        const int r = i0 + lane < p.n_pages ? p.ref[i0 + lane] : 1;
        if (i0 + lane < p.n_pages) p.w.ref0[i0 + lane] = r;
        const unsigned m = __ballot_sync(0xffffffffu, r == 0);
        if (lane == 0) free_bits[i0 >> 5] = m;
    }
    check_requests<FORK>(p, tid, kPlanThreads, needs);
    __syncthreads();
    const Plan plan{p, needs, claims, offsets};
    plan.claim();
    __syncthreads();
    const long long sum = plan.add_up(red64);
    // a word of free pages per thread
    unsigned m = tid < (p.n_pages + 31) / 32 ? free_bits[tid] : 0;
    int have;
    const int cnt = __popc(m);
    for (int at = block_scan(cnt, &have, red) - cnt; m && at < sum; ++at, m &= m - 1)
        p.w.free_list[at] = tid * 32 + __ffs(m) - 1;
    plan.answer(have);
}

// Copies `chunks` 16-byte pieces, the whole CTA, eight in flight per thread.
__device__ __forceinline__ void copy_rows(const uint4* src, uint4* dst, int chunks) {
    for (int c0 = threadIdx.x; c0 < chunks; c0 += 8 * kCopyThreads) {
        uint4 t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = c0 + u * kCopyThreads;
            if (c < chunks) t[u] = __ldcs(src + c);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = c0 + u * kCopyThreads;
            if (c < chunks) __stcs(dst + c, t[u]);
        }
    }
}

// First row of (copy, layer, K or V, head) number `unit` of a list of page copies.
__device__ __forceinline__ int64_t unit_row(const PageReq& p, int64_t sub, int pg, bool* is_v) {
    const int h = (int)(sub % p.Hkv);
    const int64_t lk = sub / p.Hkv;
    *is_v = lk & 1;
    return (((lk >> 1) * p.n_pages + pg) * p.Hkv + h) * (int64_t)p.page;
}

// `rows` rows from row s to row d of a pool, with their scales (a page has at most 128).
__device__ __forceinline__ void copy_page_rows(const PageReq& p, int64_t s, int64_t d, int rows, bool is_v) {
    uint4* pool = is_v ? p.v : p.k;
    uint8_t* scale = is_v ? p.vs : p.ks;
    if (scale && (int)threadIdx.x < rows) scale[d + threadIdx.x] = scale[s + threadIdx.x];
    copy_rows(pool + s * p.row16, pool + d * p.row16, rows * p.row16);
}

template <bool FORK>
__global__ void __launch_bounds__(kCopyThreads) pages_apply_kernel(const PageReq p, int table_ctas) {
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    if ((int)blockIdx.x < table_ctas) {
        const int wpc = kCopyThreads / 32;
        for (int64_t i = (int64_t)blockIdx.x * wpc + (threadIdx.x >> 5); i < p.n; i += (int64_t)table_ctas * wpc) {
            if (!p.granted[i]) continue;
            int32_t* row = p.table + (int64_t)p.a[i] * p.max_pages;
            const int32_t* fresh = p.w.free_list + p.w.offset[i];
            if (FORK) {
                const int32_t* srow = p.table + (int64_t)p.b[i] * p.max_pages;
                const int full = p.c[i] / p.page, part = p.c[i] % p.page;
#pragma unroll 4
                for (int j = lane; j < full; j += 32) {
                    const int e = srow[j];
                    row[j] = e;
                    atomicAdd(&p.ref[e], 1);
                }
                if (part && lane == 0) {
                    row[full] = fresh[0];
                    p.ref[fresh[0]] = 1;
                }
            } else {
                const int keep = p.b[i], cap = p.c[i];
                const int full = keep / p.page, part = keep % p.page, first = full + (part > 0);
                const int want = (int)(((int64_t)cap + p.page - 1) / p.page);
                const int held = row_held(row, p.max_pages);
                int at = 0;
                if (p.w.rows[i]) {
                    if (lane == 0) {
                        row[full] = fresh[0];
                        p.ref[fresh[0]] = 1;
                        atomicSub(&p.ref[p.w.src[i]], 1);
                    }
                    at = 1;
                }
                for (int j0 = first; j0 < max(held, want); j0 += 32) {
                    const int j = j0 + lane;
                    const int e = j < held ? row[j] : -1;
                    const bool stay = j < held && j < want && p.w.ref0[e] == 1;
                    const bool take = j < want && !stay;
                    const unsigned m = __ballot_sync(0xffffffffu, take);
                    if (j < held && !stay) atomicSub(&p.ref[e], 1);
                    if (take) {
                        const int np = fresh[at + __popc(m & ((1u << lane) - 1u))];
                        row[j] = np;
                        p.ref[np] = 1;
                    } else if (j < held && !stay) {
                        row[j] = -1;
                    }
                    at += __popc(m);
                }
            }
        }
        return;
    }
    const int64_t per = (int64_t)p.layers * 2 * p.Hkv;
    for (int64_t x = blockIdx.x - table_ctas; x < p.n * per; x += gridDim.x - table_ctas) {
        const int i = (int)(x / per);
        const int rows = p.w.rows[i];
        if (!rows) continue;
        bool is_v;
        const int64_t s = unit_row(p, x - i * per, p.w.src[i], &is_v);
        const int64_t d = unit_row(p, x - i * per, p.w.free_list[p.w.offset[i]], &is_v);
        copy_page_rows(p, s, d, rows, is_v);
    }
}

// One CTA: which live page moves into which hole (header[0]: how many).
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PageReq p, int32_t* new_page) {
    __shared__ int red[32];
    __shared__ int below;  // live pages among the first n_live
    const int tid = threadIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    int n_live = 0;
    for (int i0 = 0; i0 < p.n_pages; i0 += 4 * kPlanThreads) {
        int cnt = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 4 * tid + u;
            cnt += i < p.n_pages && p.ref[i] > 0;
        }
        int total;
        block_scan(cnt, &total, red);
        n_live += total;
    }
    if (tid == 0) below = n_live;  // the pool is full
    __syncthreads();
    int before = 0;  // live pages before this chunk
    for (int pass = 0; pass < 2; ++pass) {
        before = 0;
        for (int i0 = 0; i0 < p.n_pages; i0 += 4 * kPlanThreads) {
            int lv[4], cnt = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 4 * tid + u;
                lv[u] = i < p.n_pages && p.ref[i] > 0;
                cnt += lv[u];
            }
            int total;
            int at = before + block_scan(cnt, &total, red) - cnt;
            before += total;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 4 * tid + u;
                if (i < p.n_pages) {
                    if (pass == 0) {
                        // holes below n_live, and the live count at n_live
                        if (i == n_live) below = at;
                        if (!lv[u] && i < n_live) p.w.free_list[i - at] = i;
                    } else {
                        int to = lv[u] ? i : -1;
                        if (lv[u] && i >= n_live) {
                            to = p.w.free_list[at - below];
                            p.w.ref0[at - below] = i;
                        }
                        new_page[i] = to;
                    }
                }
                at += lv[u];
            }
        }
        __threadfence_block();
        __syncthreads();
    }
    if (tid == 0) p.w.head[0] = n_live - below;
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const PageReq p, const int32_t* new_page,
                                                                     int table_ctas) {
    griddep_launch_dependents();
    griddep_wait();
    const int moved = p.w.head[0];
    const int32_t *holes = p.w.free_list, *movers = p.w.ref0;
    if ((int)blockIdx.x < table_ctas) {
        const int64_t t = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x, nt = (int64_t)table_ctas * kCopyThreads;
        for (int64_t i = t; i < moved; i += nt) {
            p.ref[holes[i]] = p.ref[movers[i]];
            p.ref[movers[i]] = 0;
        }
        for (int64_t i = t; i < (int64_t)p.n_seqs * p.max_pages; i += nt) {
            const int e = p.table[i];
            if ((unsigned)e >= (unsigned)p.n_pages) continue;
            const int to = new_page[e];
            if (to < 0) atomicOr(p.err, ERR_BAD_PAGE);
            if (to != e) p.table[i] = to;
        }
        return;
    }
    const int64_t per = (int64_t)p.layers * 2 * p.Hkv;
    for (int64_t x = blockIdx.x - table_ctas; x < moved * per; x += gridDim.x - table_ctas) {
        const int i = (int)(x / per);
        bool is_v;
        const int64_t s = unit_row(p, x - i * per, movers[i], &is_v);
        const int64_t d = unit_row(p, x - i * per, holes[i], &is_v);
        copy_page_rows(p, s, d, p.page, is_v);
    }
}

// One CTA per (sequence, K or V, layer), so that the chain of dependent reads
// (length, list, table) is walked once for all heads.  Heads go in groups of
// at most 2048 16-byte pieces; of a group every accepted row is loaded before
// the first one is written, since a row's new place may hold one that still
// has to move.  256 sequences, 8 drafts, 8 heads of 128, one layer: ~5 us
// (10.9 with a CTA per head, which walks the chain once each).
constexpr int kAcceptThreads = 256;
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const PageReq p, const int32_t* ctx_len,
                                                                const int32_t* accepted, const int32_t* n_acc, int T,
                                                                int32_t* new_len) {
    __shared__ int64_t from[64], to[64];  // of head 0, in 16-byte pieces
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x, is_v = blockIdx.y & 1, layer = blockIdx.y >> 1;
    const int ctx = ctx_len[b], na = n_acc[b], tid = threadIdx.x;
    bool ok = ctx >= 0 && na >= 0 && na <= T && ctx <= p.max_pages * p.page;
    if (ok && tid < na) {
        const int u = accepted[(int64_t)b * T + tid], prev = tid ? accepted[(int64_t)b * T + tid - 1] : -1;
        ok = u > prev && u < T;
        const int64_t s[2] = {(int64_t)ctx + u, (int64_t)ctx + tid};
        if (ok) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int64_t j = s[k] / p.page;
                const int e = j < p.max_pages ? p.table[(int64_t)b * p.max_pages + j] : -1;
                if ((unsigned)e >= (unsigned)p.n_pages) ok = false;
                else (k ? to : from)[tid] = ((int64_t)e * p.Hkv * p.page + s[k] % p.page) * p.row16;
            }
        }
    }
    ok = __syncthreads_and(ok);
    if (tid == 0 && blockIdx.y == 0) {
        new_len[b] = ok ? ctx + na : ctx;
        if (!ok) atomicOr(p.err, ERR_BAD_PAGE);
    }
    if (!ok || na == 0) return;
    const int64_t head = (int64_t)p.page * p.row16;
    uint4* pool = (is_v ? p.v : p.k) + (int64_t)layer * p.n_pages * p.Hkv * head;
    const int per = na * p.row16, group = max(1, 8 * kAcceptThreads / per);  // per <= 1024
    for (int h0 = 0; h0 < p.Hkv; h0 += group) {
        const int chunks = min(group, p.Hkv - h0) * per;
        uint4 t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = u * kAcceptThreads + tid;
            if (c < chunks) {
                const int h = c / per, i = (c - h * per) / p.row16, q = c - h * per - i * p.row16;
                if (from[i] != to[i]) t[u] = pool[(h0 + h) * head + from[i] + q];
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = u * kAcceptThreads + tid;
            if (c < chunks) {
                const int h = c / per, i = (c - h * per) / p.row16, q = c - h * per - i * p.row16;
                if (from[i] != to[i]) pool[(h0 + h) * head + to[i] + q] = t[u];
            }
        }
    }
    // the rows' scales, whole heads at a time: all of a head's are read before one is written
    uint8_t* scale = is_v ? p.vs : p.ks;
    if (!scale) return;
    scale += (int64_t)layer * p.n_pages * p.Hkv * p.page;
    const int heads = kAcceptThreads / na, i = tid % na;
    for (int h0 = 0; h0 < p.Hkv; h0 += heads) {
        const int h = h0 + tid / na;
        const bool on = tid < heads * na && h < p.Hkv;
        uint8_t e = 0;
        if (on) e = scale[(int64_t)h * p.page + from[i] / p.row16];
        __syncthreads();
        if (on) scale[(int64_t)h * p.page + to[i] / p.row16] = e;
    }
}

// What the page calls share: sizes, pools, workspace.
int fill_req(const bsa_page_cache* c, const bsa_page_scales* scales, PageReq* p) {
    int st = check_page_cache(c);
    if (st != BSA_OK) return st;
    if (scales && (st = check_page_scales(c, scales)) != BSA_OK) return st;
    if (!c->page_table && c->n_seqs > 0) return BSA_ERR_INVALID_ARG;
    *p = PageReq{};
    p->table = c->page_table;
    p->n_seqs = c->n_seqs;
    p->max_pages = c->max_pages;
    p->n_pages = c->n_pages;
    p->page = c->page;
    p->k = static_cast<uint4*>(c->k);
    p->v = static_cast<uint4*>(c->v);
    p->layers = c->layers;
    p->Hkv = c->Hkv;
    p->row16 = scales ? c->D / 16 : c->D / 8;
    if (scales) {
        p->ks = static_cast<uint8_t*>(scales->k);
        p->vs = static_cast<uint8_t*>(scales->v);
    }
    return BSA_OK;
}

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether two int32 vectors share a byte.
bool meet(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + 4 * (uint64_t)nb && y < x + 4 * (uint64_t)na;
}

int run_request(bool fork, const bsa_page_cache* c, const bsa_page_scales* scales, int32_t* page_ref, int32_t n,
                const int32_t* a, const int32_t* b, const int32_t* len, int32_t* granted, void* ws, int64_t ws_bytes,
                cudaStream_t s) {
    PageReq p;
    int sms;
    int st = fill_req(c, scales, &p);
    if (st != BSA_OK) return st;
    if (n < 0) return BSA_ERR_INVALID_ARG;
    if (n == 0) return BSA_OK;
    if (c->n_seqs == 0) return BSA_ERR_INVALID_ARG;
    if (!page_ref || !a || !b || !len || !granted) return BSA_ERR_INVALID_ARG;
    for (const void* x : {(const void*)page_ref, (const void*)a, (const void*)b, (const void*)len, (const void*)granted})
        if (!al(x, 4)) return BSA_ERR_INVALID_ARG;
    if (!ws || !al(ws, 256)) return BSA_ERR_INVALID_ARG;
    if (ws_bytes < bsa_cache_pages_workspace(n, c->n_seqs, c->n_pages)) return BSA_ERR_CAPACITY;
    // the requests are read again once they are answered
    for (const int32_t* x : {a, b, len})
        if (meet(granted, n, x, n)) return BSA_ERR_INVALID_ARG;
    if (meet(granted, n, page_ref, c->n_pages) || meet(granted, n, c->page_table, (int64_t)c->n_seqs * c->max_pages))
        return BSA_ERR_INVALID_ARG;
    if ((st = device_context(&p.err, &sms)) != BSA_OK) return st;
    p.ref = page_ref;
    p.n = n;
    p.a = a;
    p.b = b;
    p.c = len;
    p.granted = granted;
    p.w = split_ws(ws, n, c->n_seqs, c->n_pages);
    const int64_t work = std::max<int64_t>(std::max<int64_t>((int64_t)n * 32, c->n_pages), c->n_seqs);
    const unsigned grid = (unsigned)std::min<int64_t>((work + 255) / 256, 4ll * sms);
    const int table_ctas = (int)std::min<int64_t>((n + 7) / 8, sms);
    const int64_t units = (int64_t)n * c->layers * 2 * c->Hkv;
    const unsigned copy_ctas = (unsigned)std::min<int64_t>(units, 8ll * sms);
    const bool small = (int64_t)n * c->max_pages <= 16384 && n <= kSmallRequests && c->n_pages <= kSmallPages &&
                       c->n_seqs <= kSmallSeqs;
    cudaError_t e;
    if (small) {
        e = launch_after(fork ? pages_small_kernel<true> : pages_small_kernel<false>, dim3(1), kPlanThreads, 0, s, p);
    } else {
        e = launch_after(fork ? pages_check_kernel<true> : pages_check_kernel<false>, dim3(grid), 256, 0, s, p);
        if (e == cudaSuccess) e = launch_after(pages_plan_kernel, dim3(1), kPlanThreads, 0, s, p);
    }
    if (e == cudaSuccess)
        e = launch_after(fork ? pages_apply_kernel<true> : pages_apply_kernel<false>, dim3(table_ctas + copy_ctas),
                         kCopyThreads, 0, s, p, table_ctas);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

int run_compact(const bsa_page_cache* c, const bsa_page_scales* scales, int32_t* page_ref, int32_t* new_page,
                void* workspace, int64_t workspace_bytes, cudaStream_t s) {
    PageReq p;
    int sms;
    int st = fill_req(c, scales, &p);
    if (st != BSA_OK) return st;
    if (c->n_seqs == 0) return BSA_ERR_INVALID_ARG;  // the table is what says where the pages go
    if (!page_ref || !new_page || !al(page_ref, 4) || !al(new_page, 4)) return BSA_ERR_INVALID_ARG;
    if (!workspace || !al(workspace, 256)) return BSA_ERR_INVALID_ARG;
    if (workspace_bytes < bsa_cache_pages_workspace(0, c->n_seqs, c->n_pages)) return BSA_ERR_CAPACITY;
    if (meet(new_page, c->n_pages, page_ref, c->n_pages) ||
        meet(new_page, c->n_pages, c->page_table, (int64_t)c->n_seqs * c->max_pages))
        return BSA_ERR_INVALID_ARG;
    if ((st = device_context(&p.err, &sms)) != BSA_OK) return st;
    p.ref = page_ref;
    p.w = split_ws(workspace, 0, c->n_seqs, c->n_pages);
    cudaError_t e = launch_after(compact_plan_kernel, dim3(1), kPlanThreads, 0, s, p, new_page);
    if (e != cudaSuccess) return BSA_ERR_CUDA;
    const int64_t entries = (int64_t)c->n_seqs * c->max_pages;
    const int table_ctas = (int)std::min<int64_t>((entries + 1023) / 1024, sms);
    const int64_t units = (int64_t)c->n_pages * c->layers * 2 * c->Hkv;
    const unsigned copy_ctas = (unsigned)std::min<int64_t>(units, 8ll * sms);
    e = launch_after(compact_apply_kernel, dim3(table_ctas + copy_ctas), kCopyThreads, 0, s, p, new_page, table_ctas);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

int run_accept(const bsa_page_cache* c, const bsa_page_scales* scales, const int32_t* context_len,
               const int32_t* accepted, const int32_t* n_accepted, int32_t T, int32_t* new_len, cudaStream_t s) {
    PageReq p;
    int sms;
    int st = fill_req(c, scales, &p);
    if (st != BSA_OK) return st;
    if (T < 1 || T > BSA_MAX_DRAFT) return BSA_ERR_INVALID_ARG;
    if (2ll * c->layers > 65535) return BSA_ERR_UNSUPPORTED;
    if (c->n_seqs == 0) return BSA_OK;
    if (!context_len || !accepted || !n_accepted || !new_len) return BSA_ERR_INVALID_ARG;
    for (const void* x : {(const void*)context_len, (const void*)accepted, (const void*)n_accepted, (const void*)new_len})
        if (!al(x, 4)) return BSA_ERR_INVALID_ARG;
    // every CTA of a sequence reads these, one of them writes the new length
    const int64_t S = c->n_seqs;
    if (meet(new_len, S, context_len, S) || meet(new_len, S, n_accepted, S) ||
        meet(new_len, S, accepted, S * T) || meet(new_len, S, c->page_table, S * c->max_pages))
        return BSA_ERR_INVALID_ARG;
    if ((st = device_context(&p.err, &sms)) != BSA_OK) return st;
    const dim3 grid((unsigned)c->n_seqs, (unsigned)(2 * c->layers));
    const cudaError_t e =
        launch_after(accept_kernel, grid, kAcceptThreads, 0, s, p, context_len, accepted, n_accepted, T, new_len);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace
}  // namespace bsa

extern "C" {

int64_t bsa_cache_pages_workspace(int32_t n, int32_t n_seqs, int32_t n_pages) {
    if (n < 0 || n_seqs < 0 || n_pages < 0) return 0;
    return bsa::ws_ints(n, n_seqs, n_pages) * (int64_t)sizeof(int32_t);
}

int bsa_cache_resize(const bsa_page_cache* c, int32_t* page_ref, int32_t n, const int32_t* seqs, const int32_t* keep,
                     const int32_t* capacity, int32_t* granted, void* workspace, int64_t workspace_bytes,
                     bsa_stream_t stream) {
    return bsa::run_request(false, c, nullptr, page_ref, n, seqs, keep, capacity, granted, workspace, workspace_bytes,
                            reinterpret_cast<cudaStream_t>(stream));
}

int bsa_cache_fork(const bsa_page_cache* c, int32_t* page_ref, int32_t n, const int32_t* src, const int32_t* dst,
                   const int32_t* len, int32_t* granted, void* workspace, int64_t workspace_bytes,
                   bsa_stream_t stream) {
    return bsa::run_request(true, c, nullptr, page_ref, n, dst, src, len, granted, workspace, workspace_bytes,
                            reinterpret_cast<cudaStream_t>(stream));
}

int bsa_cache_compact(const bsa_page_cache* c, int32_t* page_ref, int32_t* new_page, void* workspace,
                      int64_t workspace_bytes, bsa_stream_t stream) {
    return bsa::run_compact(c, nullptr, page_ref, new_page, workspace, workspace_bytes,
                            reinterpret_cast<cudaStream_t>(stream));
}

int bsa_cache_accept(const bsa_page_cache* c, const int32_t* context_len, const int32_t* accepted,
                     const int32_t* n_accepted, int32_t T, int32_t* new_len, bsa_stream_t stream) {
    return bsa::run_accept(c, nullptr, context_len, accepted, n_accepted, T, new_len,
                           reinterpret_cast<cudaStream_t>(stream));
}

int bsa_cache_resize_fp8(const bsa_page_cache* c, const bsa_page_scales* scales, int32_t* page_ref, int32_t n,
                         const int32_t* seqs, const int32_t* keep, const int32_t* capacity, int32_t* granted,
                         void* workspace, int64_t workspace_bytes, bsa_stream_t stream) {
    if (!scales) return BSA_ERR_INVALID_ARG;
    return bsa::run_request(false, c, scales, page_ref, n, seqs, keep, capacity, granted, workspace, workspace_bytes,
                            reinterpret_cast<cudaStream_t>(stream));
}

int bsa_cache_fork_fp8(const bsa_page_cache* c, const bsa_page_scales* scales, int32_t* page_ref, int32_t n,
                       const int32_t* src, const int32_t* dst, const int32_t* len, int32_t* granted, void* workspace,
                       int64_t workspace_bytes, bsa_stream_t stream) {
    if (!scales) return BSA_ERR_INVALID_ARG;
    return bsa::run_request(true, c, scales, page_ref, n, dst, src, len, granted, workspace, workspace_bytes,
                            reinterpret_cast<cudaStream_t>(stream));
}

int bsa_cache_compact_fp8(const bsa_page_cache* c, const bsa_page_scales* scales, int32_t* page_ref,
                          int32_t* new_page, void* workspace, int64_t workspace_bytes, bsa_stream_t stream) {
    if (!scales) return BSA_ERR_INVALID_ARG;
    return bsa::run_compact(c, scales, page_ref, new_page, workspace, workspace_bytes,
                            reinterpret_cast<cudaStream_t>(stream));
}

int bsa_cache_accept_fp8(const bsa_page_cache* c, const bsa_page_scales* scales, const int32_t* context_len,
                         const int32_t* accepted, const int32_t* n_accepted, int32_t T, int32_t* new_len,
                         bsa_stream_t stream) {
    if (!scales) return BSA_ERR_INVALID_ARG;
    return bsa::run_accept(c, scales, context_len, accepted, n_accepted, T, new_len,
                           reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
