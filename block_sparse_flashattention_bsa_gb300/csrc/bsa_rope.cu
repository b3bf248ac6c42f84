// bsa_rope.cu -- what stands between a projection and the attention: the RMS
// norm of every query and key head and the position rotation in one pass,
// token-major rows in, head-major rows (or rows of a paged cache) out, and
// the gradients of the head-major form.
//
// Mathematics, for a head row x of D values at position t:
//   y = x * r * w,  r = 1 / sqrt(mean(x^2) + eps)          (no weight: y = x)
//   a pair (y_a, y_b) of the first rotary_dim values, with its frequency f:
//   z_a = gain * (y_a cos(t f) - y_b sin(t f)),  z_b = gain * (y_b cos(t f) + y_a sin(t f))
// The angle is kept in turns: f / (2 pi) as a 64-bit fixed-point fraction,
// multiplied by the position modulo 2^64 (integer arithmetic, so no range
// reduction and no loss at far positions: the product is exact and the
// fraction is good to 2^-53 of a turn per position); its top 32 bits give the
// angle in [-pi, pi), where sin.approx / cos.approx are within 2^-20 of the
// true values.  That is 2^11 times finer than the bf16 rounding of the result.
// Keys that are written as 8-bit codes take them to fp32's precision.
//
// Gradients, with dy the rotated-back gradient (by -t f, times gain), g = dy * w:
//   dx = r g - x r^3 mean(g x),   dw = sum over rows of dy * x * r
// (a repeated key or value head first sums the gradients of its copies, fp32).

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "bsa.h"
#include "bsa_internal.h"
#include "bsa_ptx.cuh"
#include "bsa_q8.cuh"

namespace bsa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 64;  // rotary_dim / 2 <= 64
constexpr int kFwdRows = 4;    // rows of a lane group's task (forward, large calls)
constexpr int kAppendRows = 2; // the same of appending
constexpr int kFwdWaves = 8;   // forward CTAs per SM (two resident)
constexpr int kBwdResident = 2;  // the gradients' CTAs per SM
constexpr int kBwdStages = 3;  // rows in a lane's ring
constexpr int kBwdSmem = kBwdStages * 4 * kRopeThreads * 16;

// Rows of one kind (q, k or v): token-major side and its head-major side.
struct RopeSide {
    const void* x;              // token-major rows
    int64_t sb, sn, sh;         // its strides in elements
    void* out;                  // forward: head-major rows (append: q only, token-major rows)
    const void* dz;             // backward: head-major gradients
    void* dx;                   // backward: token-major gradients
    int64_t gb, gn, gh;         // strides of dx
    const float* w;             // norm weight or null
    float* partial;             // backward: per-CTA sums of the weight's gradient
    int32_t H;                  // token-major heads
    int32_t rep;                // head-major copies of each
    int32_t ctas;               // CTAs working on this kind
    int32_t rotate;             // 0 for values
    // backward: heads side by side in a CTA, tokens side by side, runs of such
    // heads per task, tasks per token block, tasks in all
    int32_t hs, toks, runs, splits, tasks;
    int64_t z_copy, z_step, x_step, dx_step;  // bytes to the next copy; from the last copy's end, and on the token side, to the next row
};

struct RopeParams {
    RopeSide side[3];
    const double* inv_freq;
    const int32_t* pos;
    int64_t pos_sb;
    int64_t tokens;  // B * N
    int32_t N, rd;
    float eps, gain;
    // append: rows of k and v go to pages
    void *k_cache, *v_cache;
    uint8_t *k_scale, *v_scale;  // 8-bit pools: a scale per row
    const int32_t *page_table, *seq_ids, *slots;
    int32_t n_seqs, max_pages, page, n_pages;
    int32_t* err;
};

// Fraction of a turn per position, in units of 2^-64.
__device__ __forceinline__ unsigned long long to_turns(double f) {
    const double t = f * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ void unpack8(const uint4& v, f2* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = {__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)};
}
__device__ __forceinline__ uint4 pack8(const f2* f) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}

// A head row is spread over LPR = D / 16 lanes, 16 values (two 16-byte
// chunks) each, placed so that both members of every pair sit in one lane and
// neighbouring lanes own neighbouring chunks (32-byte sectors used whole: with
// chunks 2s and 2s + 1 in lane s the 16K gradients took 132 us instead of 86):
//   interleaved (2i, 2i + 1): chunks s and s + LPR; pairs 4s .. and 4 (s + LPR) ..
//   halves (i, i + rd/2), nr = rd/16 lanes: chunks s and s + nr, pairs 8s .. 8s + 7;
//   the other lanes own the values that are not rotated.
template <int D, bool IL>
struct Lane {
    static constexpr int LPR = D / 16;
    int s, ca, cb;
    bool ra, rb;  // chunk a / b is rotated
    __device__ Lane(int rd) {
        s = threadIdx.x % LPR;
        const int nr = rd / 16;
        if (IL) {
            ca = s;
            cb = s + LPR;
            ra = ca < 2 * nr;
            rb = cb < 2 * nr;
        } else {
            ra = rb = s < nr;
            ca = ra ? s : s + nr;
            cb = ra ? s + nr : s + LPR;
        }
    }
};

// Sum over the LPR lanes of a row (every lane gets it).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// cos and sin of this lane's 8 pairs at position pos, times gain.  FINE: to fp32's
// precision (2^-20 is far below a bf16 rounding, but moves one in 10^5 values that
// go straight to an 8-bit code to the next one).
template <int LPR, bool IL, bool FINE = false>
__device__ __forceinline__ void lane_angles(const unsigned long long* turns, int s, int pos, float gain, float* cs,
                                            float* sn) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = IL ? 4 * s + e + (e < 4 ? 0 : 4 * LPR - 4) : 8 * s + e;
        const unsigned long long t = turns[i] * (unsigned long long)(long long)pos;
        if (FINE) {
            // Whole quarter turns apart; the rest, a = within pi / 4, by its power series:
            // the first terms left out are a^11 / 11! < 2^-28 a and a^12 / 12! < 2^-33
            const uint32_t u = (uint32_t)(t >> 32), q = (u + (1u << 29)) >> 30;
            const float a = (float)(int)(u - (q << 30)) * 1.46291807926715968e-9f, x = a * a;
            const float s0 = fmaf(a * x, fmaf(x, fmaf(x, fmaf(x, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), a);
            const float c0 = fmaf(
                x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
            const float c1 = q & 1 ? s0 : c0, s1 = q & 1 ? c0 : s0;
            cs[e] = (q + 1) & 2 ? -gain * c1 : gain * c1;
            sn[e] = q & 2 ? -gain * s1 : gain * s1;
            continue;
        }
        const float a = (float)(int)(unsigned)(t >> 32) * 1.46291807926715968e-9f;  // 2 pi / 2^32
        cs[e] = __cosf(a) * gain;
        sn[e] = __sinf(a) * gain;
    }
}

// The lane's pairs rotated: f[0..3] chunk a, f[4..7] chunk b, two values each;
// cs and sn hold pairs 2e and 2e + 1 in element e.
template <bool IL>
__device__ __forceinline__ void rotate16(f2* f, const f2* cs, const f2* sn, bool ra, bool rb) {
    if (IL) {
        if (ra) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float c = e & 1 ? cs[e / 2].y : cs[e / 2].x, s = e & 1 ? sn[e / 2].y : sn[e / 2].x;
                f[e] = {f[e].x * c - f[e].y * s, f[e].y * c + f[e].x * s};
            }
        }
        if (rb) {
#pragma unroll
            for (int e = 4; e < 8; ++e) {
                const float c = e & 1 ? cs[e / 2].y : cs[e / 2].x, s = e & 1 ? sn[e / 2].y : sn[e / 2].x;
                f[e] = {f[e].x * c - f[e].y * s, f[e].y * c + f[e].x * s};
            }
        }
    } else if (ra) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f2 a = f[e], b = f[e + 4], ns = {-sn[e].x, -sn[e].y};
            f[e] = fma2(a, cs[e], mul2(b, ns));
            f[e + 4] = fma2(b, cs[e], mul2(a, sn[e]));
        }
    }
}

// Which kind this CTA works on, and its index and count among that kind's CTAs.
__device__ __forceinline__ int cta_side(const RopeParams& p, int* idx) {
    int b = blockIdx.x, k = 0;
    while (k < 2 && b >= p.side[k].ctas) b -= p.side[k++].ctas;
    *idx = b;
    return k;
}

// The lane's two chunks of a row, normed and rotated, in fp32.
template <int D, bool IL>
__device__ __forceinline__ void norm_rotate_f32(const uint4& a, const uint4& b, f2 (&f)[8], bool norm, const f2* w,
                                                float eps, bool turn, const f2* cs, const f2* sn,
                                                const Lane<D, IL>& ln) {
    unpack8(a, f);
    unpack8(b, f + 4);
    if (norm) {
        f2 ss = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fma2(f[e], f[e], ss);
        const float r = rsqrtf(row_sum<D / 16>(ss.x + ss.y) * (1.f / D) + eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = mul2(f[e], mul2({r, r}, w[e]));
    }
    if (turn) rotate16<IL>(f, cs, sn, ln.ra, ln.rb);
}

// The same in place, rounded to bf16.
template <int D, bool IL>
__device__ __forceinline__ void norm_rotate(uint4& a, uint4& b, bool norm, const f2* w, float eps, bool turn,
                                            const f2* cs, const f2* sn, const Lane<D, IL>& ln) {
    f2 f[8];
    norm_rotate_f32<D, IL>(a, b, f, norm, w, eps, turn, cs, sn, ln);
    a = pack8(f);
    b = pack8(f + 4);
}

// Scale exponent of the row whose 16 values each of LPR lanes hold, and the
// lane's codes, eight bytes for each chunk: one rounding from the fp32 values.
template <int LPR>
__device__ __forceinline__ int quantise16(const f2 (&f)[8], uint2& a, uint2& b) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmax3(m, fabsf(f[e].x), fabsf(f[e].y));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int ex = row_exponent(m);
    const float inv = exp2_int(-ex);
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = e4m3x2(f[e].x * inv, f[e].y * inv);
    a = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    b = make_uint2(h[4] | h[5] << 16, h[6] | h[7] << 16);
    return ex;
}

// One CTA item: TB = 256 / LPR consecutive tokens times U heads.  A lane
// group takes one token and loads its U rows at once (32 bytes a lane and
// row), so the angles are computed once for U rows; neighbouring
// lane groups take neighbouring tokens, so the head-major stores of a head
// run over TB consecutive rows.
template <int D, int U, bool IL>
__global__ void __launch_bounds__(kRopeThreads, U == 1 ? 3 : 2) norm_rope_kernel(const RopeParams p) {
    constexpr int LPR = D / 16, TB = kRopeThreads / LPR;
    __shared__ unsigned long long turns[kMaxPairs];
    int idx;
    const int kind = cta_side(p, &idx);
    const RopeSide& sd = p.side[kind];
    const Lane<D, IL> ln(p.rd);
    griddep_launch_dependents();
    griddep_wait();
    // the first rows are requested before the frequencies are waited for
    const double freq = sd.rotate && threadIdx.x < p.rd / 2 ? p.inv_freq[threadIdx.x] : 0.0;
    bool first = true;
    f2 w[8];
    const bool norm = sd.w != nullptr;
    if (norm) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float* we = sd.w + (e < 4 ? ln.ca : ln.cb) * 8 + (2 * e & 7);
            w[e] = {we[0], we[1]};
        }
    }
    const int hgroups = (sd.H + U - 1) / U;
    const int64_t items = (p.tokens + TB - 1) / TB * hgroups;
    for (int64_t it = idx; it < items; it += sd.ctas) {
        const int hg = (int)(it % hgroups);
        const int64_t tok = it / hgroups * TB + threadIdx.x / LPR;
        const bool live = tok < p.tokens;
        const int64_t b = live ? (int)tok / p.N : 0, n = live ? tok - b * p.N : 0;
        const int h0 = hg * U;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(sd.x) + b * sd.sb +
                                                          n * sd.sn + h0 * sd.sh);
        const int64_t sh8 = sd.sh / 8;
        uint4 ra[U], rb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = live && h0 + u < sd.H;
            ra[u] = on ? src[u * sh8 + ln.ca] : make_uint4(0, 0, 0, 0);
            rb[u] = on ? src[u * sh8 + ln.cb] : make_uint4(0, 0, 0, 0);
        }
        const int pos = !live ? 0 : p.pos ? p.pos[b * p.pos_sb + n] : (int)n;
        // where the row goes: head 0, distance between heads, in 16-byte chunks
        uint4* dst = nullptr;
        int64_t dh = 0;
        if (live) {
            dst = reinterpret_cast<uint4*>(sd.out) + (b * sd.H * sd.rep * (int64_t)p.N + n) * (D / 8);
            dh = (int64_t)p.N * (D / 8);
        }
        if (first) {
            first = false;
            if (threadIdx.x < p.rd / 2) turns[threadIdx.x] = to_turns(freq);
            __syncthreads();
        }
        f2 cs[4], sn[4];
        const bool turn = sd.rotate && (ln.ra || ln.rb);
        if (turn && live) {
            float c[8], s[8];
            lane_angles<LPR, IL>(turns, ln.s, pos, p.gain, c, s);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[e] = {c[2 * e], c[2 * e + 1]};
                sn[e] = {s[2 * e], s[2 * e + 1]};
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint4 oa = ra[u], ob = rb[u];
            if (sd.rotate) norm_rotate<D, IL>(oa, ob, norm, w, p.eps, turn, cs, sn, ln);
            if (dst && h0 + u < sd.H) {
                const int copies = sd.rep;
                uint4* d = dst + (int64_t)(h0 + u) * copies * dh;
                for (int c = 0; c < copies; ++c) {
                    d[c * dh + ln.ca] = oa;
                    d[c * dh + ln.cb] = ob;
                }
            }
        }
    }
}

// Appending.  A CTA's items are neighbours, heads first, so that a token's
// angles and its page are looked up once for its heads, and the next item's
// rows are on their way while this one's are worked on.  Queries stay
// token-major; what the forward gains from neighbouring CTAs at neighbouring
// tokens (runs of a head's rows) there is not, and reading is half of the
// traffic, not a fifth: 32K tokens of 48 heads of 128 (805 MB) 159 us with the
// forward's loop, 132 with this one, 6.1 TB/s (the forward 130 with its own, 151
// with this one); 2,048 tokens 14.0 and 12.9, one token 2.8 and 2.4.
template <int D, int U, bool IL, bool Q8>
__global__ void __launch_bounds__(kRopeThreads, 2) norm_rope_append_kernel(const RopeParams p) {
    constexpr int LPR = D / 16, TB = kRopeThreads / LPR;
    __shared__ unsigned long long turns[kMaxPairs];
    int idx;
    const int kind = cta_side(p, &idx);
    const RopeSide& sd = p.side[kind];
    const Lane<D, IL> ln(p.rd);
    griddep_launch_dependents();
    griddep_wait();
    const double freq = sd.rotate && threadIdx.x < p.rd / 2 ? p.inv_freq[threadIdx.x] : 0.0;
    f2 w[8];
    const bool norm = sd.w != nullptr;
    if (norm) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float* we = sd.w + (e < 4 ? ln.ca : ln.cb) * 8 + (2 * e & 7);
            w[e] = {we[0], we[1]};
        }
    }
    const int hgroups = (sd.H + U - 1) / U;
    const int64_t items = (p.tokens + TB - 1) / TB * hgroups;
    const int64_t lo = items * idx / sd.ctas, hi = items * (idx + 1) / sd.ctas;
    // A lane group's token: what it reads is requested by open(), where its rows
    // go and its angles follow in place() when the token's turn has come.
    struct Token {
        const uint4* src;
        int64_t tok;
        int seq, slot, pos;
        bool live;
    };
    auto open = [&](int64_t tb) {
        Token t;
        t.tok = tb * TB + threadIdx.x / LPR;
        t.live = t.tok < p.tokens;
        t.seq = t.live ? p.seq_ids[t.tok] : -1;
        t.slot = t.live ? p.slots[t.tok] : 0;
        t.pos = t.live && p.pos ? p.pos[t.tok] : t.slot;
        t.src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(sd.x) + (t.live ? t.tok * sd.sn : 0));
        return t;
    };
    const int64_t sh8 = sd.sh / 8;
    auto load = [&](const Token& t, int hg, uint4 (&a)[U], uint4 (&b)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = t.live && hg * U + u < sd.H;
            const uint4* src = t.src + (hg * U + u) * sh8;
            a[u] = on ? src[ln.ca] : make_uint4(0, 0, 0, 0);
            b[u] = on ? src[ln.cb] : make_uint4(0, 0, 0, 0);
        }
    };
    // where the row goes: base of head 0 and distance between heads, in chunks
    // (16 bytes; rows of an 8-bit pool: 8)
    uint4* dst = nullptr;
    uint8_t* dscale = nullptr;  // 8-bit pools: the scale of head 0
    int64_t dh = 0;
    f2 cs[4], sn[4];
    const bool turn = sd.rotate && (ln.ra || ln.rb);
    auto place = [&](const Token& t) {
        dst = nullptr;
        if (t.seq < 0) return;  // padding: read, not written
        if (kind == 0) {
            dst = reinterpret_cast<uint4*>(sd.out) + t.tok * sd.H * (D / 8);
            dh = D / 8;
        } else {
            // a token outside the table, or a slot without a page, is reported and not written
            int pg = -1;
            if (t.seq < p.n_seqs && t.slot >= 0 && t.slot / p.page < p.max_pages)
                pg = p.page_table[(int64_t)t.seq * p.max_pages + t.slot / p.page];
            if ((unsigned)pg < (unsigned)p.n_pages) {
                const int64_t row = (int64_t)pg * sd.H * p.page + t.slot % p.page;
                dh = (int64_t)p.page * (D / 8);
                if (Q8) {
                    dst = reinterpret_cast<uint4*>(reinterpret_cast<uint2*>(kind == 1 ? p.k_cache : p.v_cache) +
                                                   row * (D / 8));
                    dscale = (kind == 1 ? p.k_scale : p.v_scale) + row;
                } else {
                    dst = reinterpret_cast<uint4*>(kind == 1 ? p.k_cache : p.v_cache) + row * (D / 8);
                }
            } else if (ln.s == 0) {
                atomicOr(p.err, ERR_BAD_PAGE);
            }
        }
        if (turn) {
            float c[8], s[8];
            if (Q8 && kind == 1)
                lane_angles<LPR, IL, true>(turns, ln.s, t.pos, p.gain, c, s);
            else
                lane_angles<LPR, IL>(turns, ln.s, t.pos, p.gain, c, s);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[e] = {c[2 * e], c[2 * e + 1]};
                sn[e] = {s[2 * e], s[2 * e + 1]};
            }
        }
    };
    int64_t tb = lo / hgroups;
    int hg = (int)(lo - tb * hgroups);
    Token t;
    uint4 ra[U], rb[U];
    if (lo < hi) {
        t = open(tb);
        load(t, hg, ra, rb);
    }
    if (threadIdx.x < p.rd / 2) turns[threadIdx.x] = to_turns(freq);
    __syncthreads();
    if (lo < hi) place(t);
    for (int64_t it = lo; it < hi; ++it) {
        // the next item's rows are requested before this one's are worked on
        uint4 na[U], nb[U];
        const bool over = hg + 1 == hgroups, more = it + 1 < hi;
        if (more) {
            if (over) t = open(++tb);
            load(t, over ? 0 : hg + 1, na, nb);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint4 oa = ra[u], ob = rb[u];
            if (Q8 && kind > 0) {
                f2 f[8];
                if (sd.rotate) {
                    norm_rotate_f32<D, IL>(oa, ob, f, norm, w, p.eps, turn, cs, sn, ln);
                } else {
                    unpack8(oa, f);
                    unpack8(ob, f + 4);
                }
                uint2 qa, qb;
                const int ex = quantise16<LPR>(f, qa, qb);
                if (dst && hg * U + u < sd.H) {
                    uint2* d = reinterpret_cast<uint2*>(dst) + (hg * U + u) * dh;
                    d[ln.ca] = qa;
                    d[ln.cb] = qb;
                    if (ln.s == 0) dscale[(int64_t)(hg * U + u) * p.page] = (uint8_t)(ex + 127);
                }
                continue;
            }
            if (sd.rotate) norm_rotate<D, IL>(oa, ob, norm, w, p.eps, turn, cs, sn, ln);
            if (dst && hg * U + u < sd.H) {
                uint4* d = dst + (hg * U + u) * dh;
                d[ln.ca] = oa;
                d[ln.cb] = ob;
            }
        }
        if (!more) break;
        if (over) place(t);
        hg = over ? 0 : hg + 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ra[u] = na[u];
            rb[u] = nb[u];
        }
    }
}

// The gradients.  A CTA works on `hs` heads (two where H is even, else one) of
// `toks` consecutive tokens at a time, one row per lane group, so that both
// sides are touched in runs: hs * D values of a token, toks * D of a head.  A
// task is a block of tokens times `runs` such head groups, one after the
// other, so a token's angles are computed once for them.  What a lane reads
// of a row -- two chunks of dz and two of x, or two of another copy's dz -- goes
// through a ring of its own in shared memory (cp.async, across task
// boundaries): registers hold one row only, and the loads of the next two are
// in flight behind the arithmetic.  No lane reads
// another's slots, so the ring needs no barrier.
// The weight's gradient is summed per lane over all of the CTA's rows, then
// over the CTA's lanes, into one row of `partial` per CTA, which
// reduce_weight_kernel adds in a fixed order.
// Bound by DRAM: 16K tokens of 16 + 16 heads of 128 (537 MB): 87 us, 6.2 TB/s
// (102 us with two rows per lane loaded into registers at a time).
template <int D, bool NORM, bool REP>
struct RowIter {
    static constexpr int LPR = D / 16;
    int task, left, c;  // task, rows left in it, copy of the row
    bool live;          // the lane group has a token
    const char *z, *x;
    char* dst;

    __device__ __forceinline__ void start(const RopeParams& p, const RopeSide& sd, int t, int* tok_out) {
        task = t;
        c = 0;
        if (t >= sd.tasks) return;
        const int tb = t / sd.splits, lg = threadIdx.x / LPR, sub = lg / sd.hs;
        const int run0 = (t - tb * sd.splits) * sd.runs;
        const int h = run0 * sd.hs + (lg - sub * sd.hs);
        left = min(sd.runs, sd.H / sd.hs - run0);
        const int64_t tok = (int64_t)tb * sd.toks + sub;
        live = sub < sd.toks && tok < p.tokens;
        const int64_t b = live ? (int)tok / p.N : 0, n = live ? tok - b * p.N : 0;
        *tok_out = (int)(b * p.N + n);
        x = static_cast<const char*>(sd.x) + 2 * (b * sd.sb + n * sd.sn + h * sd.sh);
        dst = static_cast<char*>(sd.dx) + 2 * (b * sd.gb + n * sd.gn + h * sd.gh);
        z = static_cast<const char*>(sd.dz) + ((b * sd.H + h) * sd.rep * (int64_t)p.N + n) * (D * 2);
    }
    // Copies of the row that this step takes: with x one, else two where there are two left.
    __device__ __forceinline__ int copies(const RopeSide& sd) const {
        return REP && !(NORM && c == 0) && c + 1 < sd.rep ? 2 : 1;
    }
    // The next copies of the row, or the next row; true at the end of the task.
    __device__ __forceinline__ bool next(const RopeSide& sd) {
        if (REP) {
            const int n = copies(sd);
            z += n * sd.z_copy;
            if ((c += n) < sd.rep) return false;
            c = 0;
        }
        z += sd.z_step;
        x += sd.x_step;
        dst += sd.dx_step;
        return --left == 0;
    }
};

__device__ __forceinline__ void cp_async16(uint4* dst, const char* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes)
                 : "memory");
}

// The rows of one kind that this CTA takes; acc: this lane's share of the
// weight's gradient.  NORM: the kind has a weight; REP: its rows have copies.
template <int D, bool IL, bool NORM, bool REP>
__device__ __forceinline__ void bwd_rows(const RopeParams& p, const RopeSide& sd, int idx, uint4* ring,
                                         const unsigned long long* turns, const float* wsh, f2* acc) {
    constexpr int LPR = D / 16, C4 = kRopeThreads;
    const Lane<D, IL> ln(p.rd);
    RowIter<D, NORM, REP> pre, cur;
    int tok = 0, pre_tok;
    pre.start(p, sd, idx, &pre_tok);
    cur.start(p, sd, idx, &tok);
    uint4* mine = ring + threadIdx.x;
    const int oa = ln.ca * 16, ob = ln.cb * 16;
    auto fetch = [&](int stage) {
        if (pre.task < sd.tasks) {
            uint4* r = mine + stage * 4 * C4;
            const int bytes = pre.live ? 16 : 0;
            cp_async16(r, pre.z + oa, bytes);
            cp_async16(r + C4, pre.z + ob, bytes);
            if (NORM && (!REP || pre.c == 0)) {
                cp_async16(r + 2 * C4, pre.x + oa, bytes);
                cp_async16(r + 3 * C4, pre.x + ob, bytes);
            } else if (REP && pre.copies(sd) == 2) {
                cp_async16(r + 2 * C4, pre.z + sd.z_copy + oa, bytes);
                cp_async16(r + 3 * C4, pre.z + sd.z_copy + ob, bytes);
            }
            if (pre.next(sd)) pre.start(p, sd, pre.task + sd.ctas, &pre_tok);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kBwdStages - 1; ++s) fetch(s);
    __syncthreads();  // turns and weights
    f2 cs[4], sn[4], g[8], x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = x[e] = {0.f, 0.f};
    const bool turn = sd.rotate && (ln.ra || ln.rb);
    bool fresh = true;
    int stage = 0;
    while (cur.task < sd.tasks) {
        if (fresh && turn) {
            fresh = false;
            float c[8], s[8];
            lane_angles<LPR, IL>(turns, ln.s, p.pos ? p.pos[tok / p.N * p.pos_sb + tok % p.N] : tok % p.N, p.gain, c, s);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[e] = {c[2 * e], c[2 * e + 1]};
                sn[e] = {-s[2 * e], -s[2 * e + 1]};
            }
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kBwdStages - 2) : "memory");
        const uint4* r = mine + stage * 4 * C4;
        if (!REP || cur.c == 0) {
            unpack8(r[0], g);
            unpack8(r[C4], g + 4);
            if (NORM) {
                unpack8(r[2 * C4], x);
                unpack8(r[3 * C4], x + 4);
            }
        } else {
            f2 t[8];
            unpack8(r[0], t);
            unpack8(r[C4], t + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = add2(g[e], t[e]);
        }
        if (REP && cur.copies(sd) == 2) {
            f2 t[8];
            unpack8(r[2 * C4], t);
            unpack8(r[3 * C4], t + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = add2(g[e], t[e]);
        }
        // the slot read in the step before is free
        fetch(stage == 0 ? kBwdStages - 1 : stage - 1);
        stage = stage + 1 == kBwdStages ? 0 : stage + 1;
        char* dst = cur.dst;
        const bool live = cur.live, more = REP && cur.c + cur.copies(sd) < sd.rep;
        if (cur.next(sd)) {
            cur.start(p, sd, cur.task + sd.ctas, &tok);
            fresh = true;
        }
        if (more) continue;
        if (turn) rotate16<IL>(g, cs, sn, ln.ra, ln.rb);
        if (NORM) {
            f2 ss = {0.f, 0.f}, sg = {0.f, 0.f}, gw[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 w4 = *reinterpret_cast<const float4*>(wsh + (q < 2 ? ln.ca : ln.cb) * 8 + (q & 1) * 4);
                gw[2 * q] = mul2(g[2 * q], {w4.x, w4.y});
                gw[2 * q + 1] = mul2(g[2 * q + 1], {w4.z, w4.w});
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fma2(x[e], x[e], ss);
                sg = fma2(gw[e], x[e], sg);
            }
            const float rr = rsqrtf(row_sum<LPR>(ss.x + ss.y) * (1.f / D) + p.eps);
            const float c = row_sum<LPR>(sg.x + sg.y) * (-1.f / D) * rr * rr * rr;
            const float ra = live ? rr : 0.f;  // lanes without a token add nothing
            const f2 r2 = {rr, rr}, c2 = {c, c}, a2 = {ra, ra};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[e] = fma2(g[e], mul2(x[e], a2), acc[e]);
                g[e] = fma2(x[e], c2, mul2(gw[e], r2));
            }
        }
        if (live) {
            *reinterpret_cast<uint4*>(dst + oa) = pack8(g);
            *reinterpret_cast<uint4*>(dst + ob) = pack8(g + 4);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads, kBwdResident) norm_rope_bwd_kernel(const RopeParams p) {
    constexpr int LPR = D / 16;
    extern __shared__ uint4 ring[];  // [stage][dz a, dz b, x a, x b][thread]
    __shared__ unsigned long long turns[kMaxPairs];
    __shared__ float red[kRopeThreads / 32][D];
    __shared__ __align__(16) float wsh[D];
    int idx;
    const RopeSide& sd = p.side[cta_side(p, &idx)];
    griddep_launch_dependents();
    griddep_wait();
    if (sd.w)
        for (int d = threadIdx.x; d < D; d += kRopeThreads) wsh[d] = sd.w[d];
    if (sd.rotate)
        for (int i = threadIdx.x; i < p.rd / 2; i += kRopeThreads) turns[i] = to_turns(p.inv_freq[i]);
    f2 acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = {0.f, 0.f};
    if (!sd.w) {
        if (sd.rep == 1)
            bwd_rows<D, IL, false, false>(p, sd, idx, ring, turns, wsh, acc);
        else
            bwd_rows<D, IL, false, true>(p, sd, idx, ring, turns, wsh, acc);
        return;
    }
    if (sd.rep == 1)
        bwd_rows<D, IL, true, false>(p, sd, idx, ring, turns, wsh, acc);
    else
        bwd_rows<D, IL, true, true>(p, sd, idx, ring, turns, wsh, acc);
    const Lane<D, IL> ln(p.rd);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float a = e & 1 ? acc[e / 2].y : acc[e / 2].x;
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if ((threadIdx.x & 31) < LPR) red[threadIdx.x / 32][(e < 8 ? ln.ca : ln.cb) * 8 + (e & 7)] = a;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kRopeThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kRopeThreads / 32; ++k) s += red[k][d];
        sd.partial[(int64_t)idx * D + d] = s;
    }
}

// dw[d] = sum of rows[0 .. n) [d]; block 0: q, block 1: k.  Four columns a
// thread, the rows dealt over the block, then one tree over shared memory.
struct ReduceParams {
    const float* rows[2];
    float* out[2];
    int32_t n[2];
};
template <int D>
__global__ void __launch_bounds__(1024) reduce_weight_kernel(const ReduceParams p) {
    constexpr int C4 = D / 4, G = 1024 / C4;
    __shared__ float4 red[G][C4];
    const int k = blockIdx.x, c = threadIdx.x % C4, g = threadIdx.x / C4;
    griddep_launch_dependents();
    griddep_wait();
    if (!p.out[k]) return;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = g; i < p.n[k]; i += G) {
        const float4 v = reinterpret_cast<const float4*>(p.rows[k])[(int64_t)i * C4 + c];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
    }
    red[g][c] = a;
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (g < o) {
            const float4 v = red[g + o][c];
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
            red[g][c] = a;
        }
    }
    if (g == 0) reinterpret_cast<float4*>(p.out[k])[c] = a;
}

// CTAs of each kind, in proportion to the bytes it moves, none without an item.
// Several times what is resident: kinds and rows of unequal cost then even out
// over the SMs (128K tokens, 48 heads, 4.83 GB: 920 us with two CTAs per SM in
// all, 750 with eight; 16K tokens of 24 heads: 38.9 with eight, 40.7 with 16).
void deal_ctas(RopeParams* p, int D, int U, int ctas, const double* bytes) {
    const int TB = kRopeThreads / (D / 16);
    // a group of fewer than U heads takes as long as a whole one (32K tokens of
    // 64 + 1 heads, forward: 236 us by bytes alone, 184)
    double cost[3], all = 0;
    for (int k = 0; k < 3; ++k) {
        const int H = p->side[k].H;
        cost[k] = H > 0 ? bytes[k] * ((H + U - 1) / U * U) / H : 0;
        all += cost[k];
    }
    for (int k = 0; k < 3; ++k) {
        RopeSide& sd = p->side[k];
        const int64_t items = sd.H > 0 ? (p->tokens + TB - 1) / TB * ((sd.H + U - 1) / U) : 0;
        const int64_t share = std::max<int64_t>(1, (int64_t)std::lround(ctas * cost[k] / all));
        sd.ctas = (int32_t)std::min(items, share);
    }
}

constexpr int kRopeMaxCtas = 1024;  // the gradients' CTAs are held to this: rows of the workspace a kind has

template <bool APPEND, bool Q8 = false>
cudaError_t launch_fwd(const RopeParams& p, int D, int U, bool il, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.side[0].ctas + p.side[1].ctas + p.side[2].ctas);
    auto go = [&](auto kern) { return launch_after(kern, dim3(grid), kRopeThreads, 0, s, p); };
    auto pick = [&](auto d, auto u) {
        if constexpr (APPEND)
            return il ? go(norm_rope_append_kernel<d.value, u.value, true, Q8>)
                      : go(norm_rope_append_kernel<d.value, u.value, false, Q8>);
        else
            return il ? go(norm_rope_kernel<d.value, u.value, true>) : go(norm_rope_kernel<d.value, u.value, false>);
    };
    constexpr std::integral_constant<int, APPEND ? kAppendRows : kFwdRows> many;
    constexpr std::integral_constant<int, 1> one;
    constexpr std::integral_constant<int, 128> d128;
    constexpr std::integral_constant<int, 64> d64;
    if (D == 128) return U > 1 ? pick(d128, many) : pick(d128, one);
    return U > 1 ? pick(d64, many) : pick(d64, one);
}

// The gradients' tasks and CTAs of each kind: all heads of a token block in
// one task unless that leaves the SMs short of tasks.
void deal_tasks(RopeParams* p, int D, int sm_count, const double* bytes) {
    const int groups = kRopeThreads / (D / 16);
    const double all = bytes[0] + bytes[1] + bytes[2];
    // Four CTAs per SM even out kinds of unequal cost, two save the start of
    // the second pair: four from 400 KB each on (537 MB: 86.1 us with four,
    // 89.1 with two; 121 MB: 30.9 and 27.9; 134 MB: 30.0 and 28.3; nothing was
    // measured between 134 and 537 MB, where the turn is).
    const double moved = all * p->tokens * D * 2;
    const int waves = moved >= 4.0 * sm_count * 400e3 ? 4 : kBwdResident;
    const int ctas = std::min(waves * sm_count, kRopeMaxCtas);
    for (int k = 0; k < 3; ++k) {
        RopeSide& sd = p->side[k];
        if (sd.H == 0) continue;
        sd.hs = sd.H % 2 == 0 ? 2 : 1;  // 8 side by side: 98 us for the 537 MB above
        sd.toks = groups / sd.hs;
        const int64_t blocks = (p->tokens + sd.toks - 1) / sd.toks;
        const int64_t share = std::max<int64_t>(1, (int64_t)std::lround(ctas * bytes[k] / all));
        const int32_t all_runs = sd.H / sd.hs;
        // at least 8 tasks for each of the kind's CTAs, or single runs
        const int64_t want = std::max<int64_t>(1, std::min<int64_t>(all_runs, 8 * share / std::max<int64_t>(1, blocks)));
        sd.runs = (int32_t)((all_runs + want - 1) / want);
        sd.splits = (all_runs + sd.runs - 1) / sd.runs;
        sd.tasks = (int32_t)(blocks * sd.splits);
        sd.ctas = (int32_t)std::min<int64_t>(sd.tasks, share);
        // from a row (of rep copies) to the one hs heads on; next() has moved past its copies already
        sd.z_copy = sd.rep > 1 ? (int64_t)p->N * D * 2 : 0;
        sd.z_step = (int64_t)sd.hs * sd.rep * p->N * D * 2 - sd.rep * sd.z_copy;
        sd.x_step = 2 * sd.hs * sd.sh;
        sd.dx_step = 2 * sd.hs * sd.gh;
    }
}

cudaError_t launch_bwd(const RopeParams& p, int D, bool il, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.side[0].ctas + p.side[1].ctas + p.side[2].ctas);
    static std::atomic<uint64_t> raised[4];  // [D == 128][interleaved]
    auto go = [&](auto kern) {
        const cudaError_t e =
            raise_smem_limit(reinterpret_cast<const void*>(kern), kBwdSmem, &raised[(D == 128) * 2 + il]);
        if (e != cudaSuccess) return e;
        return launch_after(kern, dim3(grid), kRopeThreads, kBwdSmem, s, p);
    };
    if (D == 128) return il ? go(norm_rope_bwd_kernel<128, true>) : go(norm_rope_bwd_kernel<128, false>);
    return il ? go(norm_rope_bwd_kernel<64, true>) : go(norm_rope_bwd_kernel<64, false>);
}

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Token-major strides: rows start on 16 bytes, one element after another.
bool strides_ok(const int64_t* st) {
    for (int i = 0; i < 3; ++i)
        if (st[i] < 0 || st[i] % 8) return false;
    return true;
}

// Heads of a lane group's task: `rows` share one computation of the angles and
// are read at once; single heads spread a small call over more CTAs.  Several
// from half an item per SM on (with four, 2,048 tokens of 48 heads appended, then
// accepted: 18.9 us, 23.8 with single heads; 512 tokens: 8.2 and 9.7).
int pick_heads(int64_t tokens, int D, int Hq, int Hkv, int rows, int sm_count) {
    const int TB = kRopeThreads / (D / 16);
    const int64_t items = (tokens + TB - 1) / TB * ((Hq + rows - 1) / rows + 2 * ((Hkv + rows - 1) / rows));
    return 2 * items >= sm_count ? rows : 1;
}

// Appending: CTAs per SM.  Four start fewer times, six even out what the
// kinds' items cost (2,048 tokens of 32 + 8 heads, 2.5 items a CTA of four: 12.9
// us, with six 13.7; 32K of 32 + 32, 80 items: 300 and 255; the turn lies
// somewhere between).
int append_waves(int64_t tokens, int D, int Hq, int Hkv, int U, int sm_count) {
    const int TB = kRopeThreads / (D / 16);
    const int64_t items = (tokens + TB - 1) / TB * ((Hq + U - 1) / U + 2 * ((Hkv + U - 1) / U));
    return items >= 64ll * sm_count ? 6 : 4;
}

int fill(const bsa_norm_rope_args* a, RopeParams* p) {
    if (!a || a->B < 0 || a->N < 0 || a->Hq <= 0 || a->Hkv <= 0 || a->D <= 0) return BSA_ERR_INVALID_ARG;
    if (a->kv_repeat <= 0 || (int64_t)a->Hkv * a->kv_repeat > INT32_MAX) return BSA_ERR_INVALID_ARG;
    if (a->rotary_dim < 0 || a->rotary_dim > a->D || a->rotary_dim % 16) return BSA_ERR_INVALID_ARG;
    if (a->interleaved != 0 && a->interleaved != 1) return BSA_ERR_INVALID_ARG;
    if (!(a->eps >= 0.f) || !std::isfinite(a->eps) || !std::isfinite(a->gain)) return BSA_ERR_INVALID_ARG;
    if (a->rotary_dim > 0 && (!a->inv_freq || !al(a->inv_freq, 8))) return BSA_ERR_INVALID_ARG;
    if (!strides_ok(a->q_stride) || !strides_ok(a->k_stride) || (a->v && !strides_ok(a->v_stride)))
        return BSA_ERR_INVALID_ARG;
    if (!al(a->q, 16) || !al(a->k, 16) || !al(a->v, 16) || !al(a->positions, 4) || !al(a->q_weight, 4) ||
        !al(a->k_weight, 4) || a->position_stride < 0)
        return BSA_ERR_INVALID_ARG;
    if (a->D != 64 && a->D != 128) return BSA_ERR_UNSUPPORTED;
    p->tokens = (int64_t)a->B * a->N;
    // a kind's tasks, of at least one head of 4 tokens, are counted in an int
    if (p->tokens > INT32_MAX || (p->tokens / 4 + 1) * std::max(a->Hq, a->Hkv) > INT32_MAX - (1 << 16))
        return BSA_ERR_INVALID_ARG;
    const void* x[3] = {a->q, a->k, a->v};
    const int64_t* st[3] = {a->q_stride, a->k_stride, a->v_stride};
    for (int k = 0; k < 3; ++k) {
        RopeSide& sd = p->side[k];
        sd = RopeSide{};
        sd.x = x[k];
        sd.sb = st[k][0];
        sd.sn = st[k][1];
        sd.sh = st[k][2];
        sd.H = k == 0 ? a->Hq : (k == 2 && !a->v ? 0 : a->Hkv);
        sd.rep = k == 0 ? 1 : a->kv_repeat;
        sd.rotate = k < 2;
        sd.w = k == 0 ? a->q_weight : k == 1 ? a->k_weight : nullptr;
    }
    p->inv_freq = a->inv_freq;
    p->pos = a->positions;
    p->pos_sb = a->position_stride;
    p->N = std::max(a->N, 1);
    p->rd = a->rotary_dim;
    p->eps = a->eps;
    p->gain = a->gain;
    return BSA_OK;
}

// Appending to bf16 pools, or (scales) 8-bit ones.
int append(const bsa_norm_rope_args* a, const bsa_page_cache* c, const bsa_page_scales* scales, const int32_t* seq_ids,
           const int32_t* slots, void* q_out, cudaStream_t stream) {
    RopeParams p{};
    int st = fill(a, &p);
    if (st != BSA_OK) return st;
    if ((st = check_page_cache(c)) != BSA_OK) return st;
    if (scales && (st = check_page_scales(c, scales)) != BSA_OK) return st;
    if (a->B != 1 || a->kv_repeat != 1 || c->layers != 1 || c->Hkv != a->Hkv || c->D != a->D)
        return BSA_ERR_INVALID_ARG;
    if (p.tokens == 0) return BSA_OK;
    if (c->n_seqs == 0) return BSA_ERR_INVALID_ARG;  // tokens of no sequence
    if (!a->q || !a->k || !a->v || !q_out || !seq_ids || !slots || !c->page_table) return BSA_ERR_INVALID_ARG;
    if (!al(q_out, 16) || !al(seq_ids, 4) || !al(slots, 4)) return BSA_ERR_INVALID_ARG;
    int sms;
    if ((st = device_context(&p.err, &sms)) != BSA_OK) return st;
    p.side[0].out = q_out;
    p.k_cache = c->k;
    p.v_cache = c->v;
    if (scales) {
        p.k_scale = static_cast<uint8_t*>(scales->k);
        p.v_scale = static_cast<uint8_t*>(scales->v);
    }
    p.page_table = c->page_table;
    p.seq_ids = seq_ids;
    p.slots = slots;
    p.n_seqs = c->n_seqs;
    p.max_pages = c->max_pages;
    p.page = c->page;
    p.n_pages = c->n_pages;
    // K and V: 1.2 for their pages' look-up (32K tokens of 64 + 1 heads 203 -> 192 us, of 32 + 8 133 -> 131)
    const double bytes[3] = {(double)a->Hq, 1.2 * a->Hkv, 1.2 * a->Hkv};
    const int U = pick_heads(p.tokens, a->D, a->Hq, a->Hkv, kAppendRows, sms);
    const int waves = append_waves(p.tokens, a->D, a->Hq, a->Hkv, U, sms);
    deal_ctas(&p, a->D, U, waves * sms, bytes);
    const cudaError_t e = scales ? launch_fwd<true, true>(p, a->D, U, a->interleaved != 0, stream)
                                 : launch_fwd<true>(p, a->D, U, a->interleaved != 0, stream);
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace
}  // namespace bsa

extern "C" {

int bsa_rope_inv_freq(const bsa_rope_spec* s, double* inv_freq) {
    if (!s || !inv_freq) return BSA_ERR_INVALID_ARG;
    if (s->rotary_dim <= 0 || s->rotary_dim % 2) return BSA_ERR_INVALID_ARG;
    if (!(s->base > 0.0) || !std::isfinite(s->base) || !(s->factor > 0.0) || !std::isfinite(s->factor))
        return BSA_ERR_INVALID_ARG;
    if (s->scaling < BSA_ROPE_PLAIN || s->scaling > BSA_ROPE_BY_PARTS) return BSA_ERR_INVALID_ARG;
    if (s->scaling == BSA_ROPE_BASE && s->rotary_dim <= 2) return BSA_ERR_INVALID_ARG;
    if (s->scaling == BSA_ROPE_BY_PARTS &&
        (!(s->original_length > 0.0) || !std::isfinite(s->original_length) || !std::isfinite(s->low) ||
         !std::isfinite(s->high) || !(s->high > s->low)))
        return BSA_ERR_INVALID_ARG;
    const int n = s->rotary_dim / 2;
    double base = s->base;
    if (s->scaling == BSA_ROPE_BASE)
        base *= std::pow(s->factor, (double)s->rotary_dim / (double)(s->rotary_dim - 2));
    for (int i = 0; i < n; ++i) {
        double f = std::pow(base, -2.0 * i / (double)s->rotary_dim);
        if (s->scaling == BSA_ROPE_LINEAR) f /= s->factor;
        if (s->scaling == BSA_ROPE_BY_PARTS) {
            const double turns = s->original_length * f / 6.283185307179586476925;
            const double ramp = std::min(1.0, std::max(0.0, (turns - s->low) / (s->high - s->low)));
            f *= ramp + (1.0 - ramp) / s->factor;
        }
        inv_freq[i] = f;
    }
    return BSA_OK;
}

int bsa_qk_norm_rope(const bsa_norm_rope_args* a, void* q_out, void* k_out, void* v_out, bsa_stream_t stream) {
    bsa::RopeParams p{};
    int st = bsa::fill(a, &p);
    if (st != BSA_OK) return st;
    if (p.tokens == 0) return BSA_OK;
    if (!a->q || !a->k || !q_out || !k_out || (a->v != nullptr) != (v_out != nullptr)) return BSA_ERR_INVALID_ARG;
    if (!bsa::al(q_out, 16) || !bsa::al(k_out, 16) || !bsa::al(v_out, 16)) return BSA_ERR_INVALID_ARG;
    int32_t* err;
    int sms;
    if ((st = bsa::device_context(&err, &sms)) != BSA_OK) return st;
    void* out[3] = {q_out, k_out, v_out};
    double bytes[3];
    for (int k = 0; k < 3; ++k) {
        p.side[k].out = out[k];
        bytes[k] = (double)p.side[k].H * (1 + p.side[k].rep);
    }
    const int U = bsa::pick_heads(p.tokens, a->D, a->Hq, a->Hkv, bsa::kFwdRows, sms);
    bsa::deal_ctas(&p, a->D, U, bsa::kFwdWaves * sms, bytes);
    const cudaError_t e =
        bsa::launch_fwd<false>(p, a->D, U, a->interleaved != 0, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

int bsa_cache_append(const bsa_norm_rope_args* a, const bsa_page_cache* c, const int32_t* seq_ids,
                     const int32_t* slots, void* q_out, bsa_stream_t stream) {
    return bsa::append(a, c, nullptr, seq_ids, slots, q_out, reinterpret_cast<cudaStream_t>(stream));
}

int bsa_cache_append_fp8(const bsa_norm_rope_args* a, const bsa_page_cache* c, const bsa_page_scales* scales,
                         const int32_t* seq_ids, const int32_t* slots, void* q_out, bsa_stream_t stream) {
    if (!scales) return BSA_ERR_INVALID_ARG;
    return bsa::append(a, c, scales, seq_ids, slots, q_out, reinterpret_cast<cudaStream_t>(stream));
}

int64_t bsa_qk_norm_rope_backward_workspace(int32_t D) {
    return D > 0 ? 2ll * bsa::kRopeMaxCtas * D * (int64_t)sizeof(float) : 0;
}

int bsa_qk_norm_rope_backward(const bsa_norm_rope_args* a, const bsa_norm_rope_grads* g, void* workspace,
                              int64_t workspace_bytes, bsa_stream_t stream) {
    bsa::RopeParams p{};
    int st = bsa::fill(a, &p);
    if (st != BSA_OK) return st;
    if (!g) return BSA_ERR_INVALID_ARG;
    const bool dw = a->q_weight || a->k_weight;
    if ((a->q_weight != nullptr) != (g->q_weight != nullptr) || (a->k_weight != nullptr) != (g->k_weight != nullptr))
        return BSA_ERR_INVALID_ARG;
    if (!bsa::al(g->q_weight, 16) || !bsa::al(g->k_weight, 16) || !bsa::al(workspace, 16)) return BSA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const void* dz[3] = {g->dq, g->dk, g->dv};
    void* dx[3] = {g->q, g->k, g->v};
    const int64_t* gs[3] = {g->q_stride, g->k_stride, g->v_stride};
    if ((g->dv != nullptr) != (g->v != nullptr)) return BSA_ERR_INVALID_ARG;
    p.side[2].H = g->dv ? a->Hkv : 0;
    for (int k = 0; k < 3; ++k) {
        if (k == 2 && !g->dv) continue;
        const int32_t ext[3] = {a->B, a->N, k == 0 ? a->Hq : a->Hkv};
        for (int i = 0; i < 3; ++i)  // written rows must not coincide
            if (ext[i] > 1 && gs[k][i] == 0) return BSA_ERR_INVALID_ARG;
        if (!bsa::strides_ok(gs[k]) || !bsa::al(dz[k], 16) || !bsa::al(dx[k], 16)) return BSA_ERR_INVALID_ARG;
        if (p.tokens > 0 && (!dz[k] || !dx[k])) return BSA_ERR_INVALID_ARG;
    }
    if (p.tokens > 0 && ((a->q_weight && !a->q) || (a->k_weight && !a->k))) return BSA_ERR_INVALID_ARG;
    if (dw && (!workspace || workspace_bytes < bsa_qk_norm_rope_backward_workspace(a->D))) return BSA_ERR_CAPACITY;
    int32_t* err;
    int sms;
    if ((st = bsa::device_context(&err, &sms)) != BSA_OK) return st;
    if (p.tokens == 0) {
        for (float* o : {g->q_weight, g->k_weight})
            if (o && cudaMemsetAsync(o, 0, (size_t)a->D * sizeof(float), s) != cudaSuccess) return BSA_ERR_CUDA;
        return BSA_OK;
    }
    double bytes[3];
    for (int k = 0; k < 3; ++k) {
        bsa::RopeSide& sd = p.side[k];
        sd.dz = dz[k];
        sd.dx = dx[k];
        sd.gb = gs[k][0];
        sd.gn = gs[k][1];
        sd.gh = gs[k][2];
        sd.partial = static_cast<float*>(workspace) + (int64_t)k * bsa::kRopeMaxCtas * a->D;
        bytes[k] = (double)sd.H * (1 + sd.rep + (sd.w ? 1 : 0));
    }
    p.side[2].partial = nullptr;
    bsa::deal_tasks(&p, a->D, sms, bytes);
    cudaError_t e = bsa::launch_bwd(p, a->D, a->interleaved != 0, s);
    if (e == cudaSuccess && dw) {
        bsa::ReduceParams r{{p.side[0].partial, p.side[1].partial},
                            {g->q_weight, g->k_weight},
                            {p.side[0].ctas, p.side[1].ctas}};
        e = bsa::launch_after(a->D == 128 ? bsa::reduce_weight_kernel<128> : bsa::reduce_weight_kernel<64>, dim3(2), 1024,
                              0, s, r);
    }
    return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"
