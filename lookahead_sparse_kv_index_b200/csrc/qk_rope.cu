// A step's query and key heads (lsa_qk_norm_rope): for each token and head
//     y = x * w / sqrt(mean(x^2) + eps),   pairs (a, b) turned by phi = pos * freq:
//     a' = m (a cos phi - b sin phi),  b' = m (a sin phi + b cos phi),
// written to q_out / k_out and, with the values, to the slots of a paged cache.
//
// One pass: a row is read once and written once, so the call is bound by HBM for many tokens (16384 tokens of 48 bf16
// heads of 128: 70 us, 5.7 TB/s, 89% of the copy rate) and by its latency for few.  A warp does rows of one token after
// the other, LPR lanes a row, and the device's warps share all rows evenly, whatever the number of tokens.  A lane owns
// units of VP pairs of the row, i.e. VP elements of the rotated part's first half and the VP that pair with them (or whole
// pairs of either half of the row where pairs are interleaved), so rotating needs no exchange between lanes, and both
// accesses are as wide as the sizes allow (16 bytes at VP = 8 bf16 or 4 fp32) with neighbouring lanes side by side.  As a
// lane's pairs are the same in every row, the products of its weights with cos and sin stay in registers while the token's
// heads pass (its rows come through a ring of cp.async copies in shared memory, which each lane reads back itself), and a
// rotation is four products a pair:
//     a' = f (x_a (m w_a cos) - x_b (m w_b sin)),  b' = f (x_a (m w_a sin) + x_b (m w_b cos)),  f = 1 / sqrt(mean + eps).
// The warp computes the token's angles once, reduced to a fraction of a turn in fp64 (pos * freq reaches millions of
// radians, where fp32 keeps no fraction); only the fraction goes to the fp32 sincospi, and its rounding is made good after.
// (Before that a CTA held the angles of four tokens in shared memory and each row read them and its weights again: 380
// instructions for four rows of 128, and 99 us for 16384 tokens of 48 heads, bound by instruction issue.)
#include <math.h>

#include "paged.cuh"

namespace lsa {
namespace {

using paged::CacheView;

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kAhead = 4;            // rounds of a warp in its ring: three on their way while one is computed

struct QkArgs {
    const uint8_t *q, *k, *v;
    uint8_t *q_out, *k_out;
    int64_t q_stride, q_out_stride, k_stride, k_out_stride, v_stride;   // bytes between tokens
    int32_t row_bytes;           // of a head of q, k, v
    int32_t Hq, Hkv, D, rot;
    float sign, mscale, eps, inv_d;
    const uint8_t *wq, *wk;
    const int32_t *pos;
    const double *freq;
    CacheView cache;
    int32_t append;              // 0: no cache, 1: rows of the inputs' type, 2: e4m3 rows
    const int32_t *table, *seq, *at;
    int64_t table_stride;
    int32_t n_rows;
    int64_t reach;
    int32_t *err;
    int32_t lpr;                 // lanes of a row, a power of two
    int32_t nq, nk, nv;          // rounds of a token's queries, keys, values: 32 / lpr rows each
    int64_t share, spare;        // rounds of a warp; the first `spare` warps have one more
    int64_t warps;
};
// What chooses the kernel besides.
struct QkForm {
    bool interleaved;
    bool mixed;                  // parts hold whole pairs, some of which may turn
};

// N consecutive elements as they lie in memory, and in fp32.
template <typename T, int N>
struct Raw {
    static constexpr int kBytes = N * int(sizeof(T)), kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const uint8_t *p) {
        if constexpr (kBytes == 16) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(p);
        }
    }
    // Global to shared memory, asynchronously where the size allows it.
    static __device__ __forceinline__ void copy(uint8_t *to, const uint8_t *from) {
        const uint32_t at = uint32_t(__cvta_generic_to_shared(to));
        if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
        else if constexpr (kBytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(from) : "memory");
        else if constexpr (kBytes == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(from) : "memory");
        else *reinterpret_cast<uint16_t *>(to) = *reinterpret_cast<const uint16_t *>(from);
    }
    __device__ __forceinline__ void get(float (&x)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
            else x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
    }
};

template <typename T, int N>
__device__ __forceinline__ void store_n(uint8_t *p, const float (&x)[N]) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (N == 4) {
            *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) reinterpret_cast<float *>(p)[i] = x[i];
        }
    } else {
        if constexpr (N == 1) {
            *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(x[0]);
        } else {
            uint32_t w[N / 2];
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            if constexpr (N == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            else if constexpr (N == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t *>(p) = w[0];
        }
    }
}

// x / scale: one step of correction by the remainder makes the product with the rounded reciprocal `inv` the rounded
// quotient (P. Markstein, IBM J. Res. Dev. 34, 1990).  Without it what lies on the middle between two codes goes either
// way: 4 codes in 10000 of bf16 values.  (16384 tokens of 48 bf16 heads into e4m3 rows take 81 us, without the correction
// 77, with a division an element 90.)  Remainders have to be normal numbers: the caller passes x and scale times a power
// of two where scale is tiny.
__device__ __forceinline__ float quotient(float x, float scale, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, scale, x), inv, q);
}

// x / scale as e4m3 codes.
template <int N>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&x)[N], float up, float scale, float inv) {
    if constexpr (N == 1) {
        *p = uint8_t(__nv_cvt_float_to_fp8(quotient(x[0] * up, scale, inv), __NV_SATFINITE, __NV_E4M3));
    } else {
        uint16_t c[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            c[i] = uint16_t(__nv_cvt_float2_to_fp8x2(make_float2(quotient(x[2 * i] * up, scale, inv),
                                                                 quotient(x[2 * i + 1] * up, scale, inv)),
                                                     __NV_SATFINITE, __NV_E4M3));
        if constexpr (N == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(c[0] | uint32_t(c[1]) << 16, c[2] | uint32_t(c[3]) << 16);
        else if constexpr (N == 4) *reinterpret_cast<uint32_t *>(p) = c[0] | uint32_t(c[1]) << 16;
        else *reinterpret_cast<uint16_t *>(p) = c[0];
    }
}

// T: element type of q, k, v; VP: pairs of a unit; MU: units of a lane; LPR: lanes of a row (0: a.lpr); IL: interleaved
// pairs; MIX: a part of a unit may hold pairs that turn and pairs that do not (whole pairs alone).
template <typename T, int VP, int MU, int LPR, bool IL, bool MIX>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope(QkArgs a) {
    constexpr int E = int(sizeof(T));
    constexpr int kPart = VP * E, kSlot = 32 * 2 * MU * kPart;
    extern __shared__ __align__(16) uint8_t smem[];   // [warps] rings of kAhead rounds, then the angles [warps][rot / 2]
    const int lpr = LPR ? LPR : a.lpr, half = a.rot / 2, U = a.D / 2 / VP, rest = (a.D - a.rot) / 2;
    const int wl = threadIdx.x & 31, lane = wl & (lpr - 1), group = wl / lpr, groups = 32 / lpr;
    const int64_t self = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int rounds = a.nq + a.nk + a.nv;
    int64_t left = self < a.warps ? a.share + (self < a.spare) : 0;       // rounds still to compute
    const int64_t start = self * a.share + (self < a.spare ? self : a.spare);
    int64_t tok = paged::div_units(start, rounds);
    int rd = int(start - tok * rounds);

    // A unit's two parts of VP elements: byte offsets, and its first pair (of each part, where the parts hold whole pairs;
    // `turns`: whether they turn).  Lanes are neighbours in both parts, so that their accesses fill whole sectors.
    static_assert(!IL || VP * E == 16, "interleaved pairs always go by whole 16 bytes");
    static_assert(IL || !MIX, "parts of halves of pairs turn as one");
    int ia[MU], ib[MU], pa[MU], pb[MU];
    bool mine[MU], turns[MU][MIX ? VP : 2];
#pragma unroll
    for (int m = 0; m < MU; ++m) {
        const int u = lane + lpr * m, p = u * VP;
        mine[m] = u < U;
        if (IL) {
            ia[m] = p * E;
            ib[m] = (p + a.D / 2) * E;
            pa[m] = p / 2;
            pb[m] = (p + a.D / 2) / 2;
        } else {
            ia[m] = (p < half ? p : a.rot + (p - half)) * E;
            ib[m] = (p < half ? p + half : a.rot + rest + (p - half)) * E;
            pa[m] = pb[m] = p;
        }
        if constexpr (MIX) {
#pragma unroll
            for (int e = 0; e < VP; ++e) turns[m][e] = (e < VP / 2 ? pa[m] + e : pb[m] + e - VP / 2) < half;
        } else {
            turns[m][0] = pa[m] < half;
            turns[m][1] = pb[m] < half;
        }
    }
    pdl_launch_dependents();
    pdl_wait();
    if (left == 0) return;
    // the token's rounds are its queries' (kind 0), keys' and values', `groups` rows each; the next rounds' elements are on
    // their way while one is computed (a lane without a unit keeps zeros in the ring, a row that is not there what was there
    // before, and neither is stored)
    uint8_t *ring = smem + (threadIdx.x >> 5) * (kAhead * kSlot) + wl * kPart;
#pragma unroll
    for (int m = 0; m < MU; ++m) {
        if (!mine[m]) {
            for (int s = 0; s < kAhead; ++s)
                for (int i = 0; i < kPart; i += 2) {
                    *reinterpret_cast<uint16_t *>(ring + s * kSlot + 2 * m * 32 * kPart + i) = 0;
                    *reinterpret_cast<uint16_t *>(ring + s * kSlot + (2 * m + 1) * 32 * kPart + i) = 0;
                }
        }
    }
    auto source = [&](int64_t tok, int kind, int h) {
        return (kind == 0 ? a.q + tok * a.q_stride : kind == 1 ? a.k + tok * a.k_stride : a.v + tok * a.v_stride) +
               int64_t(h) * a.row_bytes;
    };
    const int step = groups * a.row_bytes;
    int kind = rd < a.nq ? 0 : rd < a.nq + a.nk ? 1 : 2;
    int first = kind == 0 ? 0 : kind == 1 ? a.nq : a.nq + a.nk;            // the kind's first round
    int h = (rd - first) * groups + group;
    // the fetching side's place, and what a token needs besides its rows, asked for a token ahead
    int64_t f_tok = tok, f_left = left;
    int f_rd = rd, f_kind = kind, f_h = h, f_last = first + (kind == 0 ? a.nq : kind == 1 ? a.nk : a.nv);
    const uint8_t *src = source(tok, kind, h);
    int32_t n_pos = 0, n_row = 0, n_at = -1;
    auto meet = [&](int64_t t) {
        if (half) n_pos = a.pos[t];
        if (a.append) {
            n_row = a.seq ? a.seq[t] : int32_t(t);
            n_at = a.at[t];
        }
    };
    auto fetch = [&](int slot) {
        if (f_left > 0) {
            if (f_h < (f_kind == 0 ? a.Hq : a.Hkv)) {
#pragma unroll
                for (int m = 0; m < MU; ++m) {
                    if (mine[m]) {
                        Raw<T, VP>::copy(ring + slot * kSlot + 2 * m * 32 * kPart, src + ia[m]);
                        Raw<T, VP>::copy(ring + slot * kSlot + (2 * m + 1) * 32 * kPart, src + ib[m]);
                    }
                }
            }
            f_h += groups;
            src += step;
            --f_left;
            if (++f_rd == f_last && f_left > 0) {
                f_h = group;
                if (f_rd == rounds) {
                    f_rd = 0;
                    f_kind = 0;
                    f_last = a.nq;
                    ++f_tok;
                } else {
                    ++f_kind;
                    f_last += f_kind == 1 ? a.nk : a.nv;
                }
                src = source(f_tok, f_kind, group);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    meet(tok);
    for (int s = 0; s < kAhead - 1; ++s) fetch(s);
    int now = 0;
    float2 *cs = reinterpret_cast<float2 *>(smem + kWarps * kAhead * kSlot) + (threadIdx.x >> 5) * half;

    while (left > 0) {
        // ---- a token: where it goes in the cache (every lane finds it), and its angles
        const int32_t pos = n_pos;
        const int end = int(left < rounds - rd ? rd + left : rounds), begun = rd;
        int64_t off = -1, slot = 0;
        if (a.append && end > a.nq && n_row >= 0 && n_at >= 0) {
            int64_t page = -1;
            const uint32_t size = a.cache.page_size, p = uint32_t(n_at) / size, s = uint32_t(n_at) - p * size;
            if (n_row < a.n_rows && n_at < a.reach) page = a.table[n_row * a.table_stride + p];
            if (page >= 0 && page < a.cache.n_pages) {
                off = page * a.cache.page_stride + int64_t(s) * a.cache.slot_stride;
                slot = page * size + s;
            } else if (wl == 0) {
                raise_err(a.err, LSA_ERR_INVALID);
            }
        }
        if (left > end - rd) meet(tok + 1);      // (used when the next token's turn comes)
        if (rd < a.nq + a.nk) {
            __syncwarp();           // (the token before has read its angles)
            for (int i = wl; i < half; i += 32) {
                const double turn = double(pos) * a.freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
                // half turns; what rounding them to fp32 left turns the sine and cosine by as much (they would be off by
                // up to pi 2^-25 else, more than by their own rounding)
                const double h = 2.0 * (turn - rint(turn));
                const float f = float(h), d = float(h - double(f)) * 3.14159265f;
                float s, c;
                sincospif(f, &s, &c);
                cs[i] = make_float2(a.mscale * fmaf(-s, d, c), a.mscale * a.sign * fmaf(c, d, s));
            }
            __syncwarp();
        }

        float ac[MU][VP], as[MU][VP], bc[MU][VP], bs[MU][VP];   // weights times cos and sin, of a unit's two parts
        while (rd < end) {
            const int heads = kind == 0 ? a.Hq : a.Hkv;
            const int last = min(end, first + (kind == 0 ? a.nq : kind == 1 ? a.nk : a.nv));
            const uint8_t *w = kind == 0 ? a.wq : kind == 1 ? a.wk : nullptr;
            uint8_t *out = kind == 0 ? a.q_out + tok * a.q_out_stride
                                     : kind == 1 && a.k_out ? a.k_out + tok * a.k_out_stride : nullptr;
            if (out) out += int64_t(h) * a.row_bytes;
            uint8_t *cache = kind != 0 && off >= 0 ? (kind == 1 ? a.cache.k : a.cache.v) + off + h * a.cache.head_stride : nullptr;
            if (kind != 2) {
#pragma unroll
                for (int m = 0; m < MU; ++m) {
                    float wt[2 * VP];        // of the unit's elements, in the order of the row where pairs are neighbours
                    if (w && mine[m]) {
                        float y[VP];
                        Raw<T, VP> x;
                        x.load(w + ia[m]);
                        x.get(y);
#pragma unroll
                        for (int e = 0; e < VP; ++e) wt[e] = y[e];
                        x.load(w + ib[m]);
                        x.get(y);
#pragma unroll
                        for (int e = 0; e < VP; ++e) wt[VP + e] = y[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < 2 * VP; ++e) wt[e] = 1.f;
                    }
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        const int second = IL && e >= VP / 2;
                        const float2 c = turns[m][MIX ? e : second] ? cs[second ? pb[m] + e - VP / 2 : pa[m] + e] : make_float2(1.f, 0.f);
                        const float u = IL ? wt[2 * e] : wt[e], v = IL ? wt[2 * e + 1] : wt[VP + e];
                        ac[m][e] = u * c.x;
                        as[m][e] = u * c.y;
                        bc[m][e] = v * c.x;
                        bs[m][e] = v * c.y;
                    }
                }
            }
#pragma unroll 1
            for (; rd < last; ++rd, h += groups) {
                const bool on = h < heads;
                float x[MU][2 * VP];         // the unit's first part, then its second
                float sum = 0.f;
                asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
                const uint8_t *at = ring + now * kSlot;
#pragma unroll
                for (int m = 0; m < MU; ++m) {
                    float y[VP];
                    Raw<T, VP> r;
                    r.load(at + 2 * m * 32 * kPart);
                    r.get(y);
#pragma unroll
                    for (int e = 0; e < VP; ++e) x[m][e] = y[e];
                    r.load(at + (2 * m + 1) * 32 * kPart);
                    r.get(y);
#pragma unroll
                    for (int e = 0; e < VP; ++e) x[m][VP + e] = y[e];
                }
                fetch((now + kAhead - 1) % kAhead);
                now = (now + 1) % kAhead;
                if (w) {
#pragma unroll
                    for (int m = 0; m < MU; ++m)
#pragma unroll
                        for (int e = 0; e < 2 * VP; ++e) sum = fmaf(x[m][e], x[m][e], sum);
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1)
                        if (d < lpr) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                }
                if (kind != 2) {
                    const float f = w ? rsqrtf(fmaf(sum, a.inv_d, a.eps)) : 1.f;
#pragma unroll
                    for (int m = 0; m < MU; ++m) {
#pragma unroll
                        for (int e = 0; e < VP; ++e) {
                            float &x0 = x[m][IL ? 2 * e : e], &x1 = x[m][IL ? 2 * e + 1 : VP + e];
                            float p = x0 * ac[m][e], q = x1 * bc[m][e];
                            if (turns[m][MIX ? e : IL && e >= VP / 2]) {       // (an element that does not turn never meets its partner)
                                p = fmaf(-x1, bs[m][e], p);
                                q = fmaf(x0, as[m][e], q);
                            }
                            x0 = p * f;
                            x1 = q * f;
                        }
                    }
                }
                float ya[MU][VP], yb[MU][VP];
#pragma unroll
                for (int m = 0; m < MU; ++m)
#pragma unroll
                    for (int e = 0; e < VP; ++e) ya[m][e] = x[m][e], yb[m][e] = x[m][VP + e];
                if (out) {
                    if (on) {
#pragma unroll
                        for (int m = 0; m < MU; ++m) {
                            if (mine[m]) {
                                store_n<T, VP>(out + ia[m], ya[m]);
                                store_n<T, VP>(out + ib[m], yb[m]);
                            }
                        }
                    }
                    out += step;
                }
                if (cache) {
                    if (a.append == 1) {
                        if (on) {
#pragma unroll
                            for (int m = 0; m < MU; ++m) {
                                if (mine[m]) {
                                    store_n<T, VP>(cache + ia[m], ya[m]);
                                    store_n<T, VP>(cache + ib[m], yb[m]);
                                }
                            }
                        }
                    } else {
                        float amax = 0.f;
#pragma unroll
                        for (int m = 0; m < MU; ++m)
#pragma unroll
                            for (int e = 0; e < 2 * VP; ++e) amax = fmaxf(amax, fabsf(x[m][e]));
#pragma unroll
                        for (int d = 16; d > 0; d >>= 1)
                            if (d < lpr) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                        // (a row of tiny values keeps a normal scale, so that 0 / scale is 0)
                        const float scale = amax > 0.f ? fmaxf(amax / 448.f, 1.17549435e-38f) : 1.f;
                        const float up = scale < 0x1p-60f ? 0x1p64f : 1.f, su = scale * up, inv = 1.f / su;
                        if (on) {
#pragma unroll
                            for (int m = 0; m < MU; ++m) {
                                if (mine[m]) {
                                    store_e4m3<VP>(cache + ia[m] / E, ya[m], up, su, inv);
                                    store_e4m3<VP>(cache + ib[m] / E, yb[m], up, su, inv);
                                }
                            }
                            if (lane == 0) (kind == 1 ? a.cache.ks : a.cache.vs)[slot * a.cache.Hkv + h] = scale;
                        }
                    }
                    cache += int64_t(groups) * a.cache.head_stride;
                }
            }
            first = last;
            ++kind;
            h = group;
        }
        // ---- the next token
        left -= end - begun;
        ++tok;
        rd = first = kind = 0;
        h = group;
    }
}

template <typename T, int VP, int MU, int LPR, bool IL, bool MIX = false>
lsa_status launch_as(const QkArgs &a, unsigned grid, cudaStream_t st) {
    const size_t smem = size_t(kWarps) * (size_t(kAhead) * 32 * 2 * MU * VP * sizeof(T) + size_t(a.rot / 2) * 8);
    auto *kernel = qk_norm_rope<T, VP, MU, LPR, IL, MIX>;
    LSA_CUDA(ensure_smem(kernel, smem));
    LSA_CUDA(launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, st, a));
    LSA_LAUNCHED("qk_norm_rope");
    return LSA_OK;
}
// Units of 16-byte parts: the usual head dims have the lanes of a row at compile time (64, 128 and 256 elements).
template <typename T, bool IL>
lsa_status launch_wide(const QkArgs &a, bool mixed, unsigned grid, cudaStream_t st) {
    constexpr int VP = 16 / int(sizeof(T)), kRow = 128 / 2 / VP, kMost = 8 / VP;    // units of a lane: 2 (fp32) or 1
    const int units = (a.D / 2 / VP + a.lpr - 1) / a.lpr;
    if constexpr (IL) {
        if constexpr (kMost > 1)
            if (mixed && units > 1) return launch_as<T, VP, kMost, 0, IL, true>(a, grid, st);
        if (mixed) return launch_as<T, VP, 1, 0, IL, true>(a, grid, st);
    }
    if constexpr (kMost > 1)
        if (units > 1) return launch_as<T, VP, kMost, 0, IL>(a, grid, st);
    if (a.lpr == kRow / 2) return launch_as<T, VP, 1, kRow / 2, IL>(a, grid, st);
    if (a.lpr == kRow) return launch_as<T, VP, 1, kRow, IL>(a, grid, st);
    if (a.lpr == 2 * kRow) return launch_as<T, VP, 1, 2 * kRow, IL>(a, grid, st);
    return launch_as<T, VP, 1, 0, IL>(a, grid, st);
}
// Narrower ones, of halves of pairs alone.
template <typename T, int VP>
lsa_status launch_vp(const QkArgs &a, unsigned grid, cudaStream_t st) {
    const int units = (a.D / 2 / VP + a.lpr - 1) / a.lpr;    // of a lane: at most 8 / VP
    if (units == 1) return launch_as<T, VP, 1, 0, false>(a, grid, st);
    if constexpr (VP <= 1)
        if (units > 4) return launch_as<T, VP, 8, 0, false>(a, grid, st);
    if constexpr (VP <= 2)
        if (units > 2) return launch_as<T, VP, 4, 0, false>(a, grid, st);
    return launch_as<T, VP, 2, 0, false>(a, grid, st);
}
lsa_status launch_form(const QkArgs &a, const QkForm &f, int vp, unsigned grid, cudaStream_t st, bool bf16) {
    if (bf16) {
        switch (vp) {
        case 8:
            return f.interleaved ? launch_wide<uint16_t, true>(a, f.mixed, grid, st)
                                 : launch_wide<uint16_t, false>(a, false, grid, st);
        case 4: return launch_vp<uint16_t, 4>(a, grid, st);
        case 2: return launch_vp<uint16_t, 2>(a, grid, st);
        default: return launch_vp<uint16_t, 1>(a, grid, st);
        }
    }
    switch (vp) {
    case 4:
        return f.interleaved ? launch_wide<float, true>(a, f.mixed, grid, st)
                             : launch_wide<float, false>(a, false, grid, st);
    case 2: return launch_vp<float, 2>(a, grid, st);
    default: return launch_vp<float, 1>(a, grid, st);
    }
}

// Whether two arrays of T rows share bytes (rows `as` and `bs` bytes apart, `aw` and `bw` wide).  Of arrays with different
// strides, whose rows might still pass each other, it is enough that the ranges meet.
bool overlap(const void *a, int64_t as, int64_t aw, const void *b, int64_t bs, int64_t bw, int64_t T) {
    if (!a || !b) return false;
    const int64_t x = int64_t(reinterpret_cast<uintptr_t>(a)), y = int64_t(reinterpret_cast<uintptr_t>(b));
    if (x + (T - 1) * as + aw <= y || y + (T - 1) * bs + bw <= x) return false;
    if (as != bs) return true;
    const int64_t d = ((y - x) % as + as) % as;      // of a's row to the next of b's
    return d < aw || d + bw > as;
}

}  // namespace
}  // namespace lsa

using namespace lsa;

extern "C" lsa_status lsa_qk_norm_rope(const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride,
                                       const void *k, int64_t k_stride, void *k_out, int64_t k_out_stride,
                                       const void *v, int64_t v_stride, lsa_dtype dtype, int64_t T, int32_t Hq,
                                       int32_t Hkv, int32_t D, const void *q_weight, const void *k_weight, float eps,
                                       const int32_t *pos, const lsa_rope *rope, const lsa_page_cache *cache,
                                       const int32_t *table, int64_t table_stride, int32_t n_rows, int32_t max_pages,
                                       const int32_t *seq, const int32_t *at, int32_t *err, void *stream) {
    clear_error();
    LSA_CHECK_SUPPORTED(dtype == LSA_F32 || dtype == LSA_BF16, "lsa_qk_norm_rope: dtype must be F32 or BF16");
    LSA_CHECK_ARG(T >= 0 && T < (int64_t(1) << 31), "lsa_qk_norm_rope: T=%lld", (long long)T);
    if (T == 0) return LSA_OK;   // (a tensor without tokens has no address)
    LSA_CHECK_ARG(q && q_out, "lsa_qk_norm_rope: q and q_out are required");
    LSA_CHECK_ARG(D >= 1 && Hq >= 1 && Hq <= 65535 && (k ? Hkv >= 1 && Hkv <= 65535 : Hkv >= 0),
                  "lsa_qk_norm_rope: Hq=%d Hkv=%d D=%d", Hq, Hkv, D);
    LSA_CHECK_SUPPORTED(D % 16 == 0 && D <= 512, "lsa_qk_norm_rope: D=%d is not a multiple of 16 up to 512", D);
    const int64_t e = int64_t(elem_size(dtype));
    const struct {
        const void *p;
        int64_t stride;
        int32_t heads;
        const char *name;
    } in[5] = {{q, q_stride, Hq, "q"}, {q_out, q_out_stride, Hq, "q_out"}, {k, k_stride, Hkv, "k"},
               {k_out, k_out_stride, Hkv, "k_out"}, {v, v_stride, Hkv, "v"}};
    for (const auto &x : in) {
        if (!x.p) continue;
        LSA_CHECK_ARG(x.stride >= int64_t(x.heads) * D && x.stride < (int64_t(1) << 28) && x.stride * e % 16 == 0 &&
                          aligned16(x.p),
                      "lsa_qk_norm_rope: %s: token stride %lld is less than heads * D, or pointer or stride is no "
                      "multiple of 16 bytes", x.name, (long long)x.stride);
    }
    LSA_CHECK_ARG(k || (!k_out && !v && !cache && !k_weight),
                  "lsa_qk_norm_rope: k_out, v, k_weight and a cache go with k");
    LSA_CHECK_ARG(!k || k_out || cache, "lsa_qk_norm_rope: k needs k_out or a cache");
    // an output may be its own input, each of whose rows is read by the warp that writes it; any other overlap is a race
    for (int o = 1; o < 5; o += 2)
        for (int x = 0; x < 5; ++x) {
            const bool own = x == o - 1 && in[x].p == in[o].p && in[x].stride == in[o].stride;
            LSA_CHECK_ARG(x == o || own || !overlap(in[o].p, in[o].stride * e, in[o].heads * D * e, in[x].p,
                                                    in[x].stride * e, in[x].heads * D * e, T),
                          "lsa_qk_norm_rope: %s overlaps %s (an output in place of its input has the same strides)",
                          in[o].name, in[x].name);
        }
    LSA_CHECK_ARG((!q_weight || aligned16(q_weight)) && (!k_weight || aligned16(k_weight)),
                  "lsa_qk_norm_rope: weights must be 16-byte aligned");
    LSA_CHECK_ARG(eps >= 0.f && eps < 1e30f, "lsa_qk_norm_rope: eps must be finite and not negative");
    const int rot = rope ? rope->rot_dim : 0;
    LSA_CHECK_ARG(rot >= 0 && rot % 2 == 0 && rot <= D, "lsa_qk_norm_rope: rot_dim=%d is not even in [0, D]", rot);
    LSA_CHECK_ARG(rot == 0 || (pos && rope->freq), "lsa_qk_norm_rope: a rotation needs pos and freq");
    LSA_CHECK_ARG(!rope || (rope->mscale >= 0.f && rope->mscale < 1e30f),
                  "lsa_qk_norm_rope: mscale must be finite and not negative");
    QkArgs a = {};
    if (cache) {
        const lsa_status s = paged::check_cache(cache, "lsa_qk_norm_rope");
        if (s != LSA_OK) return s;
        LSA_CHECK_SUPPORTED(cache->dtype == dtype || cache->dtype == LSA_E4M3,
                            "lsa_qk_norm_rope: the cache's rows are of dtype, or E4M3");
        LSA_CHECK_ARG(cache->Hkv == Hkv && cache->D == D, "lsa_qk_norm_rope: the cache has Hkv=%d D=%d, not %d and %d",
                      cache->Hkv, cache->D, Hkv, D);
        LSA_CHECK_ARG((cache->v == cache->k) == (v == nullptr), "lsa_qk_norm_rope: v is required, unless the cache is latent");
        LSA_CHECK_ARG(table && at, "lsa_qk_norm_rope: a cache needs table and at");
        LSA_CHECK_ARG(n_rows >= 1 && max_pages >= 1 && table_stride >= max_pages && table_stride < (int64_t(1) << 40) &&
                          int64_t(max_pages) * cache->page_size < (int64_t(1) << 31),
                      "lsa_qk_norm_rope: n_rows=%d max_pages=%d table_stride=%lld", n_rows, max_pages,
                      (long long)table_stride);
        a.cache = paged::view_of(*cache);
        a.append = cache->dtype == dtype ? 1 : 2;
        a.reach = int64_t(max_pages) * cache->page_size;
    } else {
        LSA_CHECK_ARG(!v, "lsa_qk_norm_rope: v goes to a cache");
    }
    // nor may an output lie over what else the call reads or writes: it is enough that the ranges meet
    const paged::Span rest[] = {
        {q_weight, D * e, "q_weight"},
        {k_weight, D * e, "k_weight"},
        {rot ? pos : nullptr, T * 4, "pos"},
        {rot ? rope->freq : nullptr, rot / 2 * 8, "freq"},
        {cache ? cache->k : nullptr, cache ? paged::row_span(*cache) : 0, "the cache's keys"},
        {cache ? cache->v : nullptr, cache ? paged::row_span(*cache) : 0, "the cache's values"},
        {cache ? cache->k_scale : nullptr, cache ? paged::scale_span(*cache) : 0, "k_scale"},
        {cache ? cache->v_scale : nullptr, cache ? paged::scale_span(*cache) : 0, "v_scale"},
        {cache ? table : nullptr, cache ? paged::table_span(n_rows, table_stride, max_pages) : 0, "table"},
        {cache ? seq : nullptr, T * 4, "seq"},
        {cache ? at : nullptr, T * 4, "at"},
        {err, 4, "err"}};
    for (int o = 1; o < 5; o += 2)
        for (const auto &x : rest)
            LSA_CHECK_ARG(!paged::meet({in[o].p, ((T - 1) * in[o].stride + int64_t(in[o].heads) * D) * e, in[o].name}, x),
                          "lsa_qk_norm_rope: %s overlaps %s", in[o].name, x.name);

    a.q = static_cast<const uint8_t *>(q);
    a.k = static_cast<const uint8_t *>(k);
    a.v = static_cast<const uint8_t *>(v);
    a.q_out = static_cast<uint8_t *>(q_out);
    a.k_out = static_cast<uint8_t *>(k_out);
    a.q_stride = q_stride * e;
    a.q_out_stride = q_out_stride * e;
    a.k_stride = k_stride * e;
    a.k_out_stride = k_out_stride * e;
    a.v_stride = v_stride * e;
    a.Hq = Hq;
    a.Hkv = k ? Hkv : 0;
    a.D = D;
    a.rot = rot;
    QkForm form = {};
    form.interleaved = rot == 0 || rope->interleaved;   // without a rotation, the layout with the wider accesses
    a.sign = rope && rope->inverse ? -1.f : 1.f;
    a.mscale = rope && rope->mscale != 0.f ? rope->mscale : 1.f;
    a.eps = eps;
    a.inv_d = 1.f / float(D);
    a.wq = static_cast<const uint8_t *>(q_weight);
    a.wk = static_cast<const uint8_t *>(k_weight);
    a.pos = pos;
    a.freq = rot ? rope->freq : nullptr;
    a.table = table;
    a.seq = seq;
    a.at = at;
    a.table_stride = table_stride;
    a.n_rows = n_rows;
    a.err = err;
    a.row_bytes = int32_t(D * e);
    // The widest unit that the sizes allow, of parts whose pairs all turn or all stay.  Where pairs are interleaved the
    // widest always does, with a flag for each pair (8319 tokens of 24 bf16 heads of 256 with 38 turning: 39 us, and 103 with
    // units of one pair): a kernel of its own, since the flags cost a few instructions.
    int vp = dtype == LSA_BF16 ? 8 : 4;
    auto fits = [&](int n) { return rot / 2 % n == 0 && (D - rot) / 2 % n == 0; };
    form.mixed = form.interleaved && !fits(vp);
    while (!form.mixed && !fits(vp)) vp /= 2;
    a.lpr = 1;
    while (a.lpr < 32 && a.lpr * vp < D / 2) a.lpr *= 2;
    const int groups = 32 / a.lpr;
    a.nq = (Hq + groups - 1) / groups;
    a.nk = (a.Hkv + groups - 1) / groups;
    a.nv = v ? a.nk : 0;
    // every warp takes the same number of rounds, through the ends of tokens: 16 warps an SM, all resident at once
    const int rounds = a.nq + a.nk + a.nv;
    const int64_t total = T * rounds, most = int64_t(sm_count()) * 16;
    a.warps = total < most ? total : most;
    a.share = total / a.warps;
    a.spare = total - a.share * a.warps;
    const unsigned grid = unsigned((a.warps + kWarps - 1) / kWarps);
    cudaStream_t st = as_stream(stream);
    return launch_form(a, form, vp, grid, st, dtype == LSA_BF16);
}

extern "C" lsa_status lsa_rope_frequencies(lsa_rope_kind kind, int32_t rot_dim, double base, double factor,
                                           int64_t orig_len, double beta_fast, double beta_slow, double *freq_host,
                                           float *mscale_host) {
    clear_error();
    LSA_CHECK_ARG(freq_host && mscale_host, "lsa_rope_frequencies: freq_host and mscale_host are required");
    LSA_CHECK_ARG(kind >= LSA_ROPE_PLAIN && kind <= LSA_ROPE_YARN, "lsa_rope_frequencies: kind=%d", int(kind));
    LSA_CHECK_ARG(rot_dim >= 2 && rot_dim % 2 == 0, "lsa_rope_frequencies: rot_dim=%d is not even and positive",
                  rot_dim);
    LSA_CHECK_ARG(base > 1.0 && base < 1e300, "lsa_rope_frequencies: base must be above 1");
    LSA_CHECK_ARG(kind == LSA_ROPE_PLAIN || (factor >= 1.0 && factor < 1e300),
                  "lsa_rope_frequencies: factor must be at least 1");
    LSA_CHECK_ARG(kind != LSA_ROPE_NTK || rot_dim >= 4, "lsa_rope_frequencies: NTK needs rot_dim >= 4");
    LSA_CHECK_ARG(kind != LSA_ROPE_YARN || (orig_len >= 1 && beta_slow > 0.0 && beta_fast > beta_slow),
                  "lsa_rope_frequencies: YARN needs orig_len >= 1 and 0 < beta_slow < beta_fast");
    const double r = rot_dim;
    if (kind == LSA_ROPE_NTK) base *= pow(factor, r / (r - 2.0));
    // the pair that turns `beta` times over orig_len positions
    auto pair_of = [&](double beta) {
        return r * log(double(orig_len) / (beta * 6.283185307179586477)) / (2.0 * log(base));
    };
    double low = 0.0, high = 0.0;
    if (kind == LSA_ROPE_YARN) {
        low = fmax(floor(pair_of(beta_fast)), 0.0);
        high = fmin(ceil(pair_of(beta_slow)), r - 1.0);
        if (high <= low) high = low + 0.001;
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double theta = pow(base, -2.0 * i / r);
        double f = theta;
        if (kind == LSA_ROPE_LINEAR) f = theta / factor;
        if (kind == LSA_ROPE_YARN) {
            const double g = fmin(fmax((i - low) / (high - low), 0.0), 1.0);
            f = theta * (1.0 - g) + theta / factor * g;
        }
        freq_host[i] = f;
    }
    *mscale_host = kind == LSA_ROPE_YARN ? float(0.1 * log(factor) + 1.0) : 1.f;
    return LSA_OK;
}
