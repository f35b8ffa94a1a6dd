// A step's query and key heads (lsa_qk_norm_rope): for each token and head
//     y = x * w / sqrt(mean(x^2) + eps),   pairs (a, b) turned by phi = pos * freq:
//     a' = m (a cos phi - b sin phi),  b' = m (a sin phi + b cos phi),
// written to q_out / k_out and, with the values, to the slots of a paged cache.
//
// One pass: a row is read once and written once, so the call is bound by HBM for many tokens and by its latency for
// few.  A group of LPR lanes owns a row; a lane owns units of VP pairs, i.e. VP elements of the row's first half and
// the VP that pair with them (or 2 VP neighbours where pairs are interleaved), so rotating needs no exchange between
// lanes and both accesses are as wide as the sizes allow (16 bytes at VP = 8 bf16 or 4 fp32).  The angles are shared by
// a token's heads: each CTA first computes the cos and sin of its tokens' pairs into shared memory.  The angle is
// reduced to a fraction of a turn in fp64 (pos * freq reaches millions of radians, where fp32 keeps no fraction), and
// only the fraction goes to the fp32 sincospi.
#include <math.h>

#include "paged.cuh"

namespace lsa {
namespace {

using paged::CacheView;

constexpr int kThreads = 256;

struct QkArgs {
    const uint8_t *q, *k, *v;
    uint8_t *q_out, *k_out;
    int64_t q_stride, q_out_stride, k_stride, k_out_stride, v_stride;   // bytes between tokens
    int64_t T;
    int32_t Hq, Hkv, D, rot, interleaved;
    float sign, mscale, eps;
    const uint8_t *wq, *wk;
    const int32_t *pos;
    const double *freq;
    CacheView cache;
    int32_t append;              // 0: no cache, 1: rows of the inputs' type, 2: e4m3 rows
    int32_t latent;
    const int32_t *table, *seq, *at;
    int64_t table_stride;
    int32_t n_rows;
    int64_t reach;
    int32_t *err;
    int32_t tt;                  // tokens of a CTA
    int32_t rows;                // rows of a token: Hq + Hkv (+ Hkv)
    int32_t lpr;                 // lanes of a row, a power of two
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

template <int N>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&x)[N], float scale) {
    uint8_t c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = uint8_t(__nv_cvt_float_to_fp8(x[i] / scale, __NV_SATFINITE, __NV_E4M3));
    if constexpr (N == 8) {
        uint2 w;
        memcpy(&w, c, 8);
        *reinterpret_cast<uint2 *>(p) = w;
    } else if constexpr (N == 4) {
        uint32_t w;
        memcpy(&w, c, 4);
        *reinterpret_cast<uint32_t *>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = c[i];
    }
}

// T: element type of q, k, v; VP: pairs of a unit; MU: units of a lane (VP * MU = 8: D <= 512 on 32 lanes).
template <typename T, int VP>
__global__ void __launch_bounds__(kThreads) qk_norm_rope(QkArgs a) {
    constexpr int MU = 8 / VP;
    constexpr int E = int(sizeof(T));
    extern __shared__ float2 cs[];                    // [tt][rot / 2]
    int64_t *dst = reinterpret_cast<int64_t *>(cs + a.tt * (a.rot / 2));   // [tt][2]: byte offset, flat slot
    const int64_t t0 = int64_t(blockIdx.x) * a.tt;
    const int nt = int(a.T - t0 < a.tt ? a.T - t0 : a.tt), half = a.rot / 2;
    const int groups = kThreads / a.lpr;              // of this CTA
    const int lane = threadIdx.x & (a.lpr - 1), group = threadIdx.x / a.lpr;

    // an item is a row: token t, row r of its queries, keys, values.  A group's items are `step` apart; the next one's
    // elements are on their way while one is computed, the first one's while the angles are
    const int U = a.D / 2 / VP, rest = (a.D - a.rot) / 2;
    const int items = nt * a.rows, step = groups * gridDim.y, step_t = step / a.rows, step_r = step - step_t * a.rows;
    int ia[MU], ib[MU];      // element index of a unit's first and second part
#pragma unroll
    for (int m = 0; m < MU; ++m) {
        const int p = (lane + a.lpr * m) * VP;
        if (a.interleaved) {
            ia[m] = 2 * p;
            ib[m] = 2 * p + VP;
        } else {
            ia[m] = p < half ? p : a.rot + (p - half);
            ib[m] = p < half ? p + half : a.rot + rest + (p - half);
        }
    }
    Raw<T, VP> ra[MU], rb[MU];
    auto fetch = [&](int t, int r) {
        const int64_t tok = t0 + t;
        const uint8_t *src = r < a.Hq ? a.q + tok * a.q_stride + int64_t(r) * a.D * E
                             : r < a.Hq + a.Hkv ? a.k + tok * a.k_stride + int64_t(r - a.Hq) * a.D * E
                                                : a.v + tok * a.v_stride + int64_t(r - a.Hq - a.Hkv) * a.D * E;
#pragma unroll
        for (int m = 0; m < MU; ++m) {
            if (lane + a.lpr * m < U) {
                ra[m].load(src + ia[m] * E);
                rb[m].load(src + ib[m] * E);
            }
        }
    };
    const int i_first = blockIdx.y * groups + group;
    int t = i_first / a.rows, r = i_first - t * a.rows;

    pdl_launch_dependents();
    pdl_wait();
    if (i_first < items) fetch(t, r);
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int tt = i / half, p = i - tt * half;
        const double turns = double(a.pos[t0 + tt]) * a.freq[p] * 0.15915494309189533577;   // 1 / (2 pi)
        float s, c;
        sincospif(float(2.0 * (turns - rint(turns))), &s, &c);
        cs[i] = make_float2(a.mscale * c, a.mscale * a.sign * s);
    }
    if (a.append && threadIdx.x < nt) {
        const int64_t t = t0 + threadIdx.x;
        const int64_t row = a.seq ? a.seq[t] : t, at = a.at[t];
        int64_t off = -1, slot = 0;
        if (row >= 0 && at >= 0) {
            int64_t page = -1;
            if (row < a.n_rows && at < a.reach) page = a.table[row * a.table_stride + at / a.cache.page_size];
            if (page >= 0 && page < a.cache.n_pages) {
                const int s = int(at % a.cache.page_size);
                off = page * a.cache.page_stride + s * a.cache.slot_stride;
                slot = page * a.cache.page_size + s;
            } else {
                raise_err(a.err, LSA_ERR_INVALID);
            }
        }
        dst[2 * threadIdx.x] = off;
        dst[2 * threadIdx.x + 1] = slot;
    }
    __syncthreads();

    // every lane of a warp makes the same number of rounds, as the reductions below need all of them
    for (int i0 = blockIdx.y * groups; i0 < items; i0 += step) {
        const bool on = i0 + group < items;
        const int kind = r < a.Hq ? 0 : r < a.Hq + a.Hkv ? 1 : 2;        // query, key, value
        const int h = kind == 0 ? r : kind == 1 ? r - a.Hq : r - a.Hq - a.Hkv;
        const int tn = on ? t : 0;                                       // (past the last item t has no angles)
        const int64_t tok = t0 + t;
        float xa[MU][VP], xb[MU][VP];
        float sum = 0.f;
#pragma unroll
        for (int m = 0; m < MU; ++m) {
            if (on && lane + a.lpr * m < U) {
                ra[m].get(xa[m]);
                rb[m].get(xb[m]);
#pragma unroll
                for (int e = 0; e < VP; ++e) sum = fmaf(xa[m][e], xa[m][e], fmaf(xb[m][e], xb[m][e], sum));
            } else {
#pragma unroll
                for (int e = 0; e < VP; ++e) xa[m][e] = xb[m][e] = 0.f;
            }
        }
        t += step_t;
        r += step_r;
        if (r >= a.rows) {
            r -= a.rows;
            ++t;
        }
        if (i0 + step + group < items) fetch(t, r);
        const uint8_t *w = kind == 0 ? a.wq : kind == 1 ? a.wk : nullptr;
        if (a.wq || a.wk)
            for (int x = a.lpr / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if (w) {
            const float f = 1.f / sqrtf(sum / float(a.D) + a.eps);
#pragma unroll
            for (int m = 0; m < MU; ++m) {
                if (lane + a.lpr * m < U) {
                    float wa[VP], wb[VP];
                    Raw<T, VP> x;
                    x.load(w + ia[m] * E);
                    x.get(wa);
                    x.load(w + ib[m] * E);
                    x.get(wb);
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        xa[m][e] = xa[m][e] * f * wa[e];
                        xb[m][e] = xb[m][e] * f * wb[e];
                    }
                }
            }
        }
        if (kind != 2 && half) {
#pragma unroll
            for (int m = 0; m < MU; ++m) {
                const int p = (lane + a.lpr * m) * VP;
                const float2 *c = cs + tn * half + p;
                if (a.interleaved) {
                    float y[2 * VP];
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        y[e] = xa[m][e];
                        y[VP + e] = xb[m][e];
                    }
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        if (p + e < half) {
                            const float x0 = y[2 * e], x1 = y[2 * e + 1];
                            y[2 * e] = x0 * c[e].x - x1 * c[e].y;
                            y[2 * e + 1] = x0 * c[e].y + x1 * c[e].x;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        xa[m][e] = y[e];
                        xb[m][e] = y[VP + e];
                    }
                } else if (p < half) {
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        const float x0 = xa[m][e], x1 = xb[m][e];
                        xa[m][e] = x0 * c[e].x - x1 * c[e].y;
                        xb[m][e] = x0 * c[e].y + x1 * c[e].x;
                    }
                }
            }
        }
        uint8_t *out = kind == 0 ? a.q_out + tok * a.q_out_stride
                                 : kind == 1 && a.k_out ? a.k_out + tok * a.k_out_stride : nullptr;
        if (on && out) {
            out += int64_t(h) * a.D * E;
#pragma unroll
            for (int m = 0; m < MU; ++m) {
                if (lane + a.lpr * m < U) {
                    store_n<T, VP>(out + ia[m] * E, xa[m]);
                    store_n<T, VP>(out + ib[m] * E, xb[m]);
                }
            }
        }
        if (a.append) {
            float amax = 0.f;
            if (a.append == 2) {
#pragma unroll
                for (int m = 0; m < MU; ++m)
#pragma unroll
                    for (int e = 0; e < VP; ++e) amax = fmaxf(amax, fmaxf(fabsf(xa[m][e]), fabsf(xb[m][e])));
                for (int x = a.lpr / 2; x > 0; x >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, x));
            }
            if (on && kind != 0 && dst[2 * tn] >= 0) {
                uint8_t *row = (kind == 1 ? a.cache.k : a.cache.v) + dst[2 * tn] + h * a.cache.head_stride;
                if (a.append == 1) {
#pragma unroll
                    for (int m = 0; m < MU; ++m) {
                        if (lane + a.lpr * m < U) {
                            store_n<T, VP>(row + ia[m] * E, xa[m]);
                            store_n<T, VP>(row + ib[m] * E, xb[m]);
                        }
                    }
                } else {
                    // (a row of tiny values keeps a normal scale, so that 0 / scale is 0)
                    const float scale = amax > 0.f ? fmaxf(amax / 448.f, 1.17549435e-38f) : 1.f;
#pragma unroll
                    for (int m = 0; m < MU; ++m) {
                        if (lane + a.lpr * m < U) {
                            store_e4m3<VP>(row + ia[m], xa[m], scale);
                            store_e4m3<VP>(row + ib[m], xb[m], scale);
                        }
                    }
                    if (lane == 0)
                        (kind == 1 ? a.cache.ks : a.cache.vs)[dst[2 * tn + 1] * a.cache.Hkv + h] = scale;
                }
            }
        }
    }
}

template <typename T, int VP>
lsa_status launch_vp(const QkArgs &a, dim3 grid, size_t smem, cudaStream_t st) {
    LSA_CUDA(ensure_smem(qk_norm_rope<T, VP>, smem));
    LSA_CUDA(launch_pdl(qk_norm_rope<T, VP>, grid, dim3(kThreads), smem, st, a));
    LSA_LAUNCHED("qk_norm_rope");
    return LSA_OK;
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
    LSA_CHECK_ARG((q_out != q || q_out_stride == q_stride) && (!k_out || k_out != k || k_out_stride == k_stride),
                  "lsa_qk_norm_rope: an output in place of its input has the same stride");
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
        a.latent = cache->v == cache->k;
        LSA_CHECK_ARG(a.latent == (v == nullptr), "lsa_qk_norm_rope: v is required, unless the cache is latent");
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
    a.T = T;
    a.Hq = Hq;
    a.Hkv = k ? Hkv : 0;
    a.D = D;
    a.rot = rot;
    a.interleaved = rot == 0 || rope->interleaved;   // without a rotation, the layout with the wider accesses
    a.sign = rope && rope->inverse ? -1.f : 1.f;
    a.mscale = rope && rope->mscale != 0.f ? rope->mscale : 1.f;
    a.eps = eps;
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
    a.rows = Hq + a.Hkv + (v ? Hkv : 0);
    // the widest unit that the sizes allow
    int vp = dtype == LSA_BF16 ? 8 : 4;
    auto fits = [&](int n) { return a.interleaved ? D / 2 % n == 0 : rot / 2 % n == 0 && (D - rot) / 2 % n == 0; };
    while (!fits(vp)) vp /= 2;
    a.lpr = 1;
    while (a.lpr < 32 && a.lpr * vp < D / 2) a.lpr *= 2;
    const int groups = kThreads / a.lpr;
    // tokens of a CTA: enough CTAs to fill the device, else one token, and then its rows over several
    const int64_t per = (int64_t(a.rows) + groups - 1) / groups;
    a.tt = 1;
    while (a.tt < 4 && T / (2 * a.tt) >= int64_t(sm_count()) * 8) a.tt *= 2;
    int gy = 1;
    if (a.tt == 1)
        while (gy < per && T * gy < int64_t(sm_count()) * 4) ++gy;
    const dim3 grid(unsigned((T + a.tt - 1) / a.tt), gy);
    const size_t smem = size_t(a.tt) * (rot / 2) * 8 + size_t(a.tt) * 16;
    cudaStream_t st = as_stream(stream);
    if (dtype == LSA_BF16) {
        switch (vp) {
        case 8: return launch_vp<uint16_t, 8>(a, grid, smem, st);
        case 4: return launch_vp<uint16_t, 4>(a, grid, smem, st);
        case 2: return launch_vp<uint16_t, 2>(a, grid, smem, st);
        default: return launch_vp<uint16_t, 1>(a, grid, smem, st);
        }
    }
    switch (vp) {
    case 4: return launch_vp<float, 4>(a, grid, smem, st);
    case 2: return launch_vp<float, 2>(a, grid, smem, st);
    default: return launch_vp<float, 1>(a, grid, smem, st);
    }
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
