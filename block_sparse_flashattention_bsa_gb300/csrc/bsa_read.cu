// bsa_read.cu -- rows of a paged cache back as the contiguous head-major K and V
// that the forward takes, key heads repeated, rows behind a sequence's end zero.
//
// No arithmetic but code * 2^e (exact in bf16) for 8-bit pools.  Bound by device
// memory: every row is read once and written kv_repeat times.  A CTA takes 64
// rows of one head, K and V, all of its loads before its first store; a thread
// holds 16 bytes of an output row (8 bytes of codes), so a warp's stores cover
// whole rows.

#include <cuda_fp16.h>

#include <algorithm>

#include "bsa.h"
#include "bsa_internal.h"
#include "bsa_ptx.cuh"
#include "bsa_q8.cuh"

namespace bsa {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadRows = 64;  // rows of a task

struct ReadParams {
    const void *k, *v;
    const uint8_t *ks, *vs;
    const int32_t *table, *seq_ids, *first, *len;
    uint4 *ok, *ov;
    int32_t R, n, rep, Hkv, page, n_pages, n_seqs, max_pages;
    int32_t* err;
};

// Value of an e8m0 byte (255: NaN).
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}

// Two codes times a scale, as bf16.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t two, float s) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf16x2(f.x * s, f.y * s);
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadParams p) {
    constexpr int LPR = D / 8, TB = kReadThreads / LPR, U = kReadRows / TB;
    griddep_launch_dependents();
    griddep_wait();
    const int c = threadIdx.x % LPR;
    const int tiles = (p.n + kReadRows - 1) / kReadRows;
    const int64_t tasks = (int64_t)p.R * p.Hkv * tiles;
    for (int64_t x = blockIdx.x; x < tasks; x += gridDim.x) {
        const int h = (int)(x % p.Hkv);
        const int64_t y = x / p.Hkv;
        const int tile = (int)(y % tiles), r = (int)(y / tiles);
        const int seq = p.seq_ids[r], first = p.first ? p.first[r] : 0;
        int len = p.len ? p.len[r] : p.n;
        bool bad = false;
        if (seq < 0) {
            len = 0;
        } else if (seq >= p.n_seqs || len < 0 || len > p.n || first < 0) {
            bad = true;
            len = 0;
        }
        uint4 val[2][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tile * kReadRows + u * TB + threadIdx.x / LPR;
            val[0][u] = val[1][u] = make_uint4(0, 0, 0, 0);
            if (i >= len) continue;
            const int64_t slot = (int64_t)first + i, j = slot / p.page;
            const int pg = j < p.max_pages ? p.table[(int64_t)seq * p.max_pages + j] : -1;
            if ((unsigned)pg >= (unsigned)p.n_pages) {
                bad = true;
                continue;
            }
            // Ordinary loads: this kernel may have started before the one that writes these rows
            // ended, and the read-only path is for memory that nobody writes meanwhile.
            const int64_t row = ((int64_t)pg * p.Hkv + h) * p.page + slot % p.page;
            if (Q8) {
                const uint2 a = reinterpret_cast<const uint2*>(p.k)[row * LPR + c];
                const uint2 b = reinterpret_cast<const uint2*>(p.v)[row * LPR + c];
                val[0][u] = make_uint4(a.x, a.y, p.ks[row], 0);
                val[1][u] = make_uint4(b.x, b.y, p.vs[row], 0);
            } else {
                val[0][u] = reinterpret_cast<const uint4*>(p.k)[row * LPR + c];
                val[1][u] = reinterpret_cast<const uint4*>(p.v)[row * LPR + c];
            }
        }
        if (bad) atomicOr(p.err, ERR_BAD_PAGE);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tile * kReadRows + u * TB + threadIdx.x / LPR;
            if (i >= p.n) continue;
            const int64_t at = (((int64_t)r * p.Hkv + h) * p.rep * p.n + i) * LPR + c;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                uint4 o = val[kv][u];
                if (Q8) {
                    const float s = e8m0_value(o.z);
                    o = make_uint4(scaled_pair(o.x & 0xffffu, s), scaled_pair(o.x >> 16, s),
                                   scaled_pair(o.y & 0xffffu, s), scaled_pair(o.y >> 16, s));
                }
                uint4* dst = (kv ? p.ov : p.ok) + at;
                for (int k = 0; k < p.rep; ++k) dst[(int64_t)k * p.n * LPR] = o;
            }
        }
    }
}

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace bsa

extern "C" {

int bsa_cache_read(const bsa_read_args* a, const bsa_page_cache* c, const bsa_page_scales* scales,
                   bsa_stream_t stream) {
    if (!a) return BSA_ERR_INVALID_ARG;
    int st = bsa::check_page_cache(c);
    if (st != BSA_OK) return st;
    if (scales && (st = bsa::check_page_scales(c, scales)) != BSA_OK) return st;
    if (a->R < 0 || a->n < 0 || a->kv_repeat <= 0 || c->layers != 1) return BSA_ERR_INVALID_ARG;
    if ((int64_t)c->Hkv * a->kv_repeat > INT32_MAX) return BSA_ERR_INVALID_ARG;
    // a head's rows are at most n * D elements from one another: products of three sizes fit 64 bits
    if ((double)a->R * c->Hkv * a->kv_repeat * a->n * c->D >= 9e18) return BSA_ERR_INVALID_ARG;
    for (const int32_t* x : {a->seq_ids, a->first, a->len})
        if (!bsa::al(x, 4)) return BSA_ERR_INVALID_ARG;
    if (!bsa::al(a->k, 16) || !bsa::al(a->v, 16)) return BSA_ERR_INVALID_ARG;
    if (a->R == 0 || a->n == 0) return BSA_OK;
    if (c->n_seqs == 0 || !c->page_table || !a->seq_ids || !a->k || !a->v) return BSA_ERR_INVALID_ARG;
    bsa::ReadParams p{};
    int sms;
    if ((st = bsa::device_context(&p.err, &sms)) != BSA_OK) return st;
    p.k = c->k;
    p.v = c->v;
    p.ks = scales ? static_cast<const uint8_t*>(scales->k) : nullptr;
    p.vs = scales ? static_cast<const uint8_t*>(scales->v) : nullptr;
    p.table = c->page_table;
    p.seq_ids = a->seq_ids;
    p.first = a->first;
    p.len = a->len;
    p.ok = static_cast<uint4*>(a->k);
    p.ov = static_cast<uint4*>(a->v);
    p.R = a->R;
    p.n = a->n;
    p.rep = a->kv_repeat;
    p.Hkv = c->Hkv;
    p.page = c->page;
    p.n_pages = c->n_pages;
    p.n_seqs = c->n_seqs;
    p.max_pages = c->max_pages;
    const int64_t tasks = ((int64_t)a->n + bsa::kReadRows - 1) / bsa::kReadRows * a->R * c->Hkv;
    const unsigned grid = (unsigned)std::min<int64_t>(tasks, 64ll * sms);
    auto kern = c->D == 128 ? (scales ? bsa::read_kernel<128, true> : bsa::read_kernel<128, false>)
                            : (scales ? bsa::read_kernel<64, true> : bsa::read_kernel<64, false>);
    const cudaError_t e = bsa::launch_after(kern, dim3(grid), bsa::kReadThreads, 0,
                                            reinterpret_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"
