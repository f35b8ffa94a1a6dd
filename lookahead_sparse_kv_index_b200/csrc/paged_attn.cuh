// Attention of one new token over a paged cache: what its two kernels and the combine share.
//
// The work is cut into units.  A segment is one sequence's one group of up to `HS` query heads of a kv head; it has
// `lead` units for what starting and ending it costs, then one for each `tile` entries.  Units are numbered sequence
// by sequence, head group by head group, and CTA c of the grid, which fills the device once, owns the `share`
// consecutive units from c * share on, so every SM gets the same work whatever the sequences' lengths are (without the
// leading units a CTA that met many short sequences took twice as long as the others: a batch of 64 sequences of 0 to
// 16384 entries took 198 us; with 2 leading units it takes 88, as with 3, with 6 it takes 90 and with 14 101).  A segment whose entries lie in one CTA's share is finished
// there; of the others each CTA writes a partial (unnormalised o, and the running max m and sum l of its softmax, both
// for 2^x), and the combine kernel joins a segment's partials in unit order:
//     M = max m_c,  L = sum l_c 2^(m_c - M),  o = sum o_c 2^(m_c - M) / L,  lse = (M + log2 L) ln 2.
// Where the heads divide the grid well enough, the CTAs are split among them first: CTA c does head group c % heads of
// the units (of sequences alone, then) of run c / heads, so that neighbours read neighbouring heads of the same entries
// at the same time and HBM sees whole lines of the cache rather than one head's 128 bytes of each (e4m3 heads of 64: 98 us
// before, 79 after; bf16 heads of 32: 193 before, 105 after; heads of 128 gain 1 to 4%).
// A CTA has at most two partials: slot 2c for the piece that continues a segment, 2c + 1 for one that begins it; where
// it begins one, it records which, and the record's combine CTAs join it.  There is a record for each CTA, or for each
// segment where these are fewer.
#pragma once

#include "paged.cuh"

namespace lsa {
namespace paged {

// A segment that CTA `first` begins and the CTAs up to `last` continue (b < 0: none).
struct alignas(16) Record {
    int32_t b, hseg, first, last;
};

struct AttnArgs {
    CacheView cache;
    const void *q;
    int64_t q_stride;            // bytes
    const int32_t *table;
    int64_t table_stride;
    int64_t reach;               // max_pages * page_size
    const int32_t *seq_len;
    int32_t B, Hq, G;            // G = Hq / Hkv query heads of a kv head
    int32_t HG, HS;              // head groups of a kv head, query heads of a group
    int32_t window;
    float scale;
    void *out;
    float *lse;
    float *part_o, *part_ml;     // [2 * grid][HS][D], [2 * grid][HS][2]
    Record *records;             // [grid], or [segments]
    int32_t by_segment;
    int32_t lanes;               // head groups that the CTAs are split among (1: units run through them)
    int32_t *err;
    int32_t tile, lead;
    int32_t whole;               // 1: CTA c does segment c and no partials are written
    int32_t q_f32;
};

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

// Entries [lo, hi) of sequence b that are attended.
struct Seen {
    int32_t lo, hi;
};
__device__ __forceinline__ Seen seen_of(const AttnArgs &a, int b) {
    int64_t n = a.seq_len[b];
    n = n < 0 ? 0 : n > a.reach ? a.reach : n;
    Seen s;
    s.hi = int32_t(n);
    s.lo = a.window > 0 && n > a.window ? int32_t(n - a.window) : 0;
    return s;
}
__device__ __forceinline__ int32_t tiles_of(const AttnArgs &a, int b) {
    const Seen s = seen_of(a, b);
    return (s.hi - s.lo + a.tile - 1) / a.tile;
}

__device__ __forceinline__ int32_t units_of(const AttnArgs &a, int b) {
    const int32_t n = tiles_of(a, b);
    return n ? n + a.lead : 0;
}

// Where a unit lies: sequence b, whose first unit is `base`.
struct Where {
    int64_t total, share;   // units of the call, units of a CTA
    int64_t base;
    int32_t b;              // -1: past the last unit
};

// Finds where the first unit of CTA `cta` of `ctas` lies (whole block; `scratch`: 40 int64 of shared memory).
__device__ inline Where find_start(const AttnArgs &a, int64_t cta, int64_t ctas, int heads_of_unit, int64_t *scratch) {
    const int threads = blockDim.x, warps = threads >> 5;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int per = (a.B + threads - 1) / threads;
    const int b0 = min(a.B, t * per), b1 = min(a.B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += units_of(a, b);
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) scratch[warp] = inc;
    if (t == 0) scratch[34] = -1;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    const int64_t heads = heads_of_unit;
    Where r;
    r.total = total * heads;
    r.share = div_units(r.total + ctas - 1, ctas);
    const int64_t start = cta * r.share;
    int64_t pre = before + inc - mine;
    if (start >= pre * heads && start < (pre + mine) * heads) {
        for (int b = b0; b < b1; ++b) {
            const int64_t n = units_of(a, b);
            if (start < (pre + n) * heads) {
                scratch[34] = b;
                scratch[35] = pre * heads;
                break;
            }
            pre += n;
        }
    }
    __syncthreads();
    r.b = int32_t(scratch[34]);
    r.base = scratch[35];
    __syncthreads();
    return r;
}

// Where an entry lies: the byte offset of its rows in K and V (head 0), negative where the table names no page of the
// pool, and the flat index of its slot (page * page_size + slot).
struct Entry {
    int64_t off, slot;
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// log sum_t exp(a_t) from a softmax's reference m and sum L, both for 2^x.  lg2.approx is within 2^-22 of a value near 0
// and of a part of 2^-22 of the others, below an fp32 lse's own step.
__device__ __forceinline__ float lse_of(float m, float L) { return L == 0.f ? -INFINITY : (m + log2_approx(L)) * kLn2; }

// Four consecutive elements of the output.
__device__ __forceinline__ void store_out4(const AttnArgs &a, int64_t i, const float4 &v) {
    if (a.q_f32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + i) = v;
    } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + i) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
}
__device__ __forceinline__ void store_out(const AttnArgs &a, int64_t i, float v) {
    if (a.q_f32) static_cast<float *>(a.out)[i] = v;
    else static_cast<__nv_bfloat16 *>(a.out)[i] = __float2bfloat16_rn(v);
}

// The pieces of CTA `cta` of `ctas` (a cluster counts as one), in unit order: f(b, hseg, lo, hi, slot) for entries
// [lo, hi) of sequence b and segment hseg (kv head hseg / HG, head group hseg % HG); slot: where the piece's partial goes,
// -1 where the piece is a whole segment.
template <typename F>
__device__ __forceinline__ void for_pieces(const AttnArgs &a, int cta, int ctas, int64_t *scratch, F f) {
    const int heads = a.cache.Hkv * a.HG;
    if (a.whole) {
        const int b = cta / heads;
        const Seen s = seen_of(a, b);
        f(b, cta - b * heads, s.lo, s.hi, -1);
        return;
    }
    if (threadIdx.x == 0 && !a.by_segment) a.records[cta] = Record{-1, 0, 0, 0};
    // sequences without entries have no units
    for (int e = cta; e < a.B; e += ctas) {
        if (tiles_of(a, e) != 0) continue;
        if (a.by_segment)
            for (int i = threadIdx.x; i < heads; i += blockDim.x) a.records[e * heads + i] = Record{-1, 0, 0, 0};
        for (int64_t i = threadIdx.x; i < int64_t(a.Hq) * a.cache.D; i += blockDim.x)
            store_out(a, int64_t(e) * a.Hq * a.cache.D + i, 0.f);
        if (a.lse)
            for (int i = threadIdx.x; i < a.Hq; i += blockDim.x) a.lse[int64_t(e) * a.Hq + i] = -INFINITY;
    }
    const int run = cta / a.lanes, own = cta - run * a.lanes, through = heads / a.lanes;   // (lanes is 1 or heads)
    const Where w = find_start(a, run, ctas / a.lanes, through, scratch);
    if (w.b < 0) return;
    int b = w.b;
    int64_t base = w.base, u = run * w.share;
    const int64_t end = u + w.share < w.total ? u + w.share : w.total;
    while (u < end) {
        const Seen s = seen_of(a, b);
        const int n = (s.hi - s.lo + a.tile - 1) / a.tile, units = n ? n + a.lead : 0;
        if (u - base >= int64_t(units) * through) {   // past this sequence
            base += int64_t(units) * through;
            ++b;
            continue;
        }
        const int pass = int(div_units(u - base, units)), at = int((u - base) - int64_t(pass) * units);
        const int hseg = own + pass;
        const int take = int(end - u < units - at ? end - u : units - at);
        const int t0 = max(at - a.lead, 0), t1 = max(at + take - a.lead, 0);
        if (t1 > t0) {
            const int lo = s.lo + t0 * a.tile, hi = t1 == n ? s.hi : s.lo + t1 * a.tile;
            if (t0 == 0 && threadIdx.x == 0 && (t1 < n || a.by_segment))
                a.records[a.by_segment ? b * heads + hseg : cta] =
                    Record{t1 < n ? b : -1, hseg, cta, int32_t(div_units(u - at + units - 1, w.share)) * a.lanes + own};
            f(b, hseg, lo, hi, t0 == 0 && t1 == n ? -1 : 2 * cta + (t0 == 0));
        }
        u += take;
    }
}

// Ends a piece (whole block): joins the `n` parts that its warps left in shared memory, o [n][HS][D], ml [n][HS][2],
// and writes the segment's output or the piece's partial.
__device__ __forceinline__ void finish_piece(const AttnArgs &a, int b, int hseg, int slot, int n, const float *o,
                                             const float *ml) {
    const int quads = a.cache.D / 4, HS = a.HS;
    const int first = (hseg % a.HG) * HS, heads = min(HS, a.G - first);
    const int64_t hq = int64_t(b) * a.Hq + (hseg / a.HG) * a.G + first;
    for (int i = threadIdx.x; i < heads * quads; i += blockDim.x) {
        const int h = i / quads, d = i - h * quads;
        float M = -INFINITY;
        for (int p = 0; p < n; ++p) M = fmaxf(M, ml[(p * HS + h) * 2]);
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int p = 0; p < n; ++p) {
            const float w = exp2_approx(ml[(p * HS + h) * 2] - ref);
            const float4 x = reinterpret_cast<const float4 *>(o)[(p * HS + h) * quads + d];
            L = fmaf(w, ml[(p * HS + h) * 2 + 1], L);
            v.x = fmaf(w, x.x, v.x);
            v.y = fmaf(w, x.y, v.y);
            v.z = fmaf(w, x.z, v.z);
            v.w = fmaf(w, x.w, v.w);
        }
        if (slot < 0) {
            const float r = L == 0.f ? 0.f : 1.f / L;
            store_out4(a, ((hq + h) * quads + d) * 4, make_float4(v.x * r, v.y * r, v.z * r, v.w * r));
            if (d == 0 && a.lse) a.lse[hq + h] = lse_of(M, L);
        } else {
            reinterpret_cast<float4 *>(a.part_o)[(int64_t(slot) * HS + h) * quads + d] = v;
            if (d == 0) reinterpret_cast<float2 *>(a.part_ml)[int64_t(slot) * HS + h] = make_float2(M, L);
        }
    }
}

// Host side.  How a call is cut: query heads of a group, units, CTAs (a function of the cache's shape and the device
// alone, so that the workspace's size does not depend on the call's lengths).
struct AttnPlan {
    int32_t HG, HS, tile, lead, grid, threads, stages;
    size_t smem;
};
// fp32 rows (paged_attn_f32.cu).
AttnPlan plan_f32(const lsa_page_cache &c, int Hq);
lsa_status launch_f32(const AttnArgs &a, const AttnPlan &p, int grid, cudaStream_t st);
// bf16 and e4m3 rows: the tensor-core kernel (paged_attn_mma.cu).
AttnPlan plan_mma(const lsa_page_cache &c, int Hq);
lsa_status launch_mma(const lsa_page_cache &c, const AttnArgs &a, const AttnPlan &p, int grid, cudaStream_t st);
// A latent bf16 head of 512 under more than 8 query heads: the tcgen05 kernel (paged_attn_latent.cu).
bool latent_supported(const lsa_page_cache &c, int Hq);
AttnPlan plan_latent(const lsa_page_cache &c, int Hq);
lsa_status launch_latent(const AttnArgs &a, int grid, cudaStream_t st);
lsa_status paged_combine(const AttnArgs &a, int grid, cudaStream_t st);

}  // namespace paged
}  // namespace lsa
