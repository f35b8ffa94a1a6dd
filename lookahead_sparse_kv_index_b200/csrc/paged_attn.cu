// Attention of one new token per sequence over a paged key-value cache (lsa_paged_attn):
//     a_t = scale q . K_t,   out = sum_t softmax(a)_t V_t,   lse = log sum_t exp(a_t).
//
// This file holds the entry point and the combine; the kernels are paged_attn_mma.cu's (bf16 and e4m3 rows),
// paged_attn_latent.cu's (a bf16 latent head of 512 under more than 8 query heads) and paged_attn_f32.cu's.
// paged_attn.cuh says how the work is cut.
#include "paged_attn.cuh"

namespace lsa {
namespace paged {
namespace {

// Joins a segment's partials (paged_attn.cuh): CTA (r, i) those of record r, for head i of the group.  A group of
// D / 4 threads adds 16-byte pieces of every kGroups-th partial; its first loads are on their way while the weights are
// made.  Its bytes are few (two partials a CTA of the kernel before); what it costs is a launch and three dependent trips
// to memory, about 3 us of a call.
constexpr int kCombineThreads = 256, kAhead = 4;
__global__ void __launch_bounds__(kCombineThreads) paged_attn_combine(AttnArgs a) {
    __shared__ float red[2][kCombineThreads / 32];
    __shared__ float4 sums[kCombineThreads];
    extern __shared__ float wgt[];   // [grid]
    const int h = blockIdx.y, D = a.cache.D, HS = a.HS;
    pdl_launch_dependents();
    pdl_wait();
    const Record rec = a.records[blockIdx.x];
    const int in = (rec.hseg % a.HG) * HS + h;
    if (rec.b < 0 || in >= a.G) return;
    const int c = rec.first, P = (rec.last - c) / a.lanes + 1;
    auto slot = [&](int p) { return int64_t(p == 0 ? 2 * c + 1 : 2 * (c + p * a.lanes)) * HS + h; };
    const int lanes = D / 4, groups = kCombineThreads / lanes, lane4 = threadIdx.x % lanes, grp = threadIdx.x / lanes;
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int p = grp + i * groups;
        if (grp < groups && p < P) ahead[i] = reinterpret_cast<const float4 *>(a.part_o + slot(p) * D)[lane4];
    }

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto ml = [&](int p) { return reinterpret_cast<const float2 *>(a.part_ml)[slot(p)]; };
    // (m, l) of the thread's first partial stays in registers; few segments have more than 256
    const float2 mine = threadIdx.x < P ? ml(threadIdx.x) : make_float2(-INFINITY, 0.f);
    float M = mine.x;
    for (int p = threadIdx.x + kCombineThreads; p < P; p += kCombineThreads) M = fmaxf(M, ml(p).x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kCombineThreads / 32; ++w) M = fmaxf(M, red[0][w]);
    const float ref = M == -INFINITY ? 0.f : M, f0 = exp2_approx(mine.x - ref);
    float L = f0 * mine.y;
    if (threadIdx.x < P) wgt[threadIdx.x] = f0;
    for (int p = threadIdx.x + kCombineThreads; p < P; p += kCombineThreads) {
        const float2 x = ml(p);
        const float f = exp2_approx(x.x - ref);
        wgt[p] = f;
        L = fmaf(f, x.y, L);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
    if (lane == 0) red[1][warp] = L;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kCombineThreads / 32; ++w) L += red[1][w];

    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float f, const float4 &x) {
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
    };
    if (grp < groups) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (grp + i * groups < P) add(wgt[grp + i * groups], ahead[i]);
#pragma unroll 4
        for (int p = grp + kAhead * groups; p < P; p += groups)
            add(wgt[p], reinterpret_cast<const float4 *>(a.part_o + slot(p) * D)[lane4]);
        sums[threadIdx.x] = v;
    }
    __syncthreads();
    const int64_t hq = int64_t(rec.b) * a.Hq + (rec.hseg / a.HG) * a.G + in;
    if (threadIdx.x < lanes) {
        for (int i = 1; i < groups; ++i) add(1.f, sums[i * lanes + lane4]);
        const float r = L == 0.f ? 0.f : 1.f / L;
        store_out4(a, hq * D + 4 * lane4, make_float4(v.x * r, v.y * r, v.z * r, v.w * r));
    }
    if (threadIdx.x == 0 && a.lse) a.lse[hq] = lse_of(M, L);
}

AttnPlan plan_of(const lsa_page_cache &c, int Hq) {
    if (c.dtype == LSA_F32) return plan_f32(c, Hq);
    return latent_supported(c, Hq) ? plan_latent(c, Hq) : plan_mma(c, Hq);
}

// Where no segment has more than this many tiles, each is done by one CTA, without partials and a second launch: up to 5
// tiles always, up to 8 where the segments are a sixth of the grid's CTAs or more.  Whole against split: bf16, 8 kv heads
// of 128, one sequence of 5 tiles 7.1 us against 9.1, of 8 tiles 9.6 against 9.1, 16 sequences of 8 tiles 12.5 against 15.2;
// latent, 128 heads, one sequence of 5 tiles 18.5 against 18.6, of 8 tiles 23.5 against 18.8, 32 of 8 tiles 24.9 against
// 41.7; fp32, 8 kv heads, one of 4 tiles 9.1 against 10.1, of 8 tiles 15.0 against 10.2, 32 of 8 tiles 20.6 against 29.7.
// At 16 tiles the split wins (bf16: one sequence 16.8 against 9.1, 75 of up to 16 tiles 25.8 against 24.6).
constexpr int kWholeFew = 5, kWholeMany = 8;

}  // namespace

lsa_status check_cache(const lsa_page_cache *c, const char *who) {
    LSA_CHECK_ARG(c, "%s: a cache is required", who);
    LSA_CHECK_ARG(c->k && c->v, "%s: the cache's k and v are required", who);
    LSA_CHECK_ARG(valid_dtype(c->dtype), "%s: unknown cache dtype", who);
    LSA_CHECK_ARG(c->page_size >= 1 && c->Hkv >= 1 && c->D >= 1 && c->n_pages >= 1,
                  "%s: the cache's page_size=%d Hkv=%d D=%d n_pages=%lld must be positive", who, c->page_size, c->Hkv,
                  c->D, (long long)c->n_pages);
    LSA_CHECK_SUPPORTED(c->D % 16 == 0 && c->D <= 512, "%s: D=%d is not a multiple of 16 up to 512", who, c->D);
    LSA_CHECK_SUPPORTED(c->Hkv <= 65535, "%s: Hkv=%d > 65535", who, c->Hkv);
    LSA_CHECK_ARG(c->n_pages < (int64_t(1) << 31) && c->n_pages * c->page_size < (int64_t(1) << 31),
                  "%s: the cache has 2^31 entries or more", who);
    const bool scaled = c->dtype == LSA_E4M3;
    LSA_CHECK_ARG(scaled == (c->k_scale != nullptr) && scaled == (c->v_scale != nullptr),
                  "%s: k_scale and v_scale are required for E4M3 rows and only for them", who);
    LSA_CHECK_ARG(c->v != c->k || c->v_scale == c->k_scale, "%s: a latent cache (v == k) has v_scale == k_scale", who);
    const int64_t e = int64_t(elem_size(c->dtype)), lim = int64_t(1) << 56;
    const struct {
        int64_t stride, extent;
        const char *name;
    } dims[3] = {{c->page_stride, c->n_pages, "page_stride"}, {c->slot_stride, c->page_size, "slot_stride"},
                 {c->head_stride, c->Hkv, "head_stride"}};
    for (const auto &d : dims) {
        LSA_CHECK_ARG(d.stride >= (d.extent > 1 ? c->D : 0) && d.stride < lim / (e * d.extent),
                      "%s: %s=%lld", who, d.name, (long long)d.stride);
        LSA_CHECK_ARG(d.stride * e % 16 == 0, "%s: %s=%lld elements is not a multiple of 16 bytes", who, d.name,
                      (long long)d.stride);
    }
    LSA_CHECK_ARG(aligned16(c->k) && aligned16(c->v), "%s: k and v must be 16-byte aligned", who);
    return LSA_OK;
}

lsa_status paged_combine(const AttnArgs &a, int grid, cudaStream_t st) {
    const int heads = a.HS < a.G ? a.HS : a.G;
    const int records = a.by_segment ? a.B * a.cache.Hkv * a.HG : grid;
    LSA_CUDA(launch_pdl(paged_attn_combine, dim3(records, heads), dim3(kCombineThreads), size_t(grid) * 4, st, a));
    LSA_LAUNCHED("paged_attn_combine");
    return LSA_OK;
}

}  // namespace paged
}  // namespace lsa

using namespace lsa;
using namespace lsa::paged;

// partial outputs, their (m, l), and the records (D is a multiple of 16: every part is 16-byte aligned)
static size_t workspace_bytes(const AttnPlan &p, int D) {
    return size_t(p.grid) * 2 * p.HS * (D + 2) * 4 + size_t(p.grid) * sizeof(Record);
}

static lsa_status check_heads(const lsa_page_cache *cache, int32_t Hq, const char *who) {
    LSA_CHECK_ARG(Hq >= 1 && Hq % cache->Hkv == 0, "%s: Hq=%d is not a positive multiple of Hkv=%d", who, Hq,
                  cache->Hkv);
    LSA_CHECK_SUPPORTED(Hq <= 65535, "%s: Hq=%d > 65535", who, Hq);
    return LSA_OK;
}

extern "C" size_t lsa_paged_attn_workspace_size(const lsa_page_cache *cache, int32_t B, int32_t Hq) {
    clear_error();
    if (check_cache(cache, "lsa_paged_attn_workspace_size") != LSA_OK || B < 1 ||
        check_heads(cache, Hq, "lsa_paged_attn_workspace_size") != LSA_OK)
        return 0;
    return workspace_bytes(plan_of(*cache, Hq), cache->D);
}

extern "C" lsa_status lsa_paged_attn(const void *Q, lsa_dtype q_dtype, int64_t q_stride, const lsa_page_cache *cache,
                                     const int32_t *table, int64_t table_stride, int32_t max_pages,
                                     const int32_t *seq_len, int32_t B, int32_t Hq, int32_t window, float scale,
                                     void *out, float *lse, void *workspace, size_t ws_bytes, int32_t *err,
                                     void *stream) {
    clear_error();
    LSA_CHECK_ARG(Q && table && seq_len && out && workspace,
                  "lsa_paged_attn: Q, table, seq_len, out and workspace are required");
    lsa_status s = check_cache(cache, "lsa_paged_attn");
    if (s != LSA_OK) return s;
    LSA_CHECK_ARG(B >= 1, "lsa_paged_attn: B=%d", B);
    s = check_heads(cache, Hq, "lsa_paged_attn");
    if (s != LSA_OK) return s;
    LSA_CHECK_ARG(valid_dtype(q_dtype), "lsa_paged_attn: unknown q_dtype");
    LSA_CHECK_SUPPORTED(q_dtype == (cache->dtype == LSA_F32 ? LSA_F32 : LSA_BF16),
                        "lsa_paged_attn: Q must be F32 with an F32 cache and BF16 with a BF16 or E4M3 one");
    const int64_t e = int64_t(elem_size(q_dtype));
    LSA_CHECK_ARG(q_stride >= int64_t(Hq) * cache->D && q_stride < (int64_t(1) << 40) && q_stride * e % 16 == 0,
                  "lsa_paged_attn: q_stride=%lld is less than Hq * D or no multiple of 16 bytes", (long long)q_stride);
    LSA_CHECK_ARG(aligned16(Q) && aligned16(out), "lsa_paged_attn: Q and out must be 16-byte aligned");
    LSA_CHECK_ARG(max_pages >= 1 && table_stride >= max_pages && table_stride < (int64_t(1) << 40),
                  "lsa_paged_attn: max_pages=%d table_stride=%lld", max_pages, (long long)table_stride);
    // (places of entries are int32 in the kernels, which step past a sequence's end by up to a tile of every warp)
    LSA_CHECK_ARG(int64_t(max_pages) * cache->page_size <= (int64_t(1) << 30),
                  "lsa_paged_attn: a table row reaches more than 2^30 entries");
    LSA_CHECK_ARG(window >= 0, "lsa_paged_attn: window=%d", window);
    LSA_CHECK_ARG(scale > 0.0f && scale < 1e30f, "lsa_paged_attn: scale must be positive and finite");
    const AttnPlan p = plan_of(*cache, Hq);
    LSA_CHECK_ARG(ws_bytes >= workspace_bytes(p, cache->D) && aligned16(workspace),
                  "lsa_paged_attn: workspace of %zu bytes < %zu", ws_bytes, workspace_bytes(p, cache->D));

    // what a call writes lies apart from all else of it, but for an output in place of the queries: each head's is written
    // when no one reads its query any more
    const int64_t heads_bytes = int64_t(Hq) * cache->D * e;
    const Span read[] = {{Q, (B - 1) * q_stride * e + heads_bytes, "Q"},
                         {cache->k, row_span(*cache), "the cache's keys"},
                         {cache->v, row_span(*cache), "the cache's values"},
                         {cache->k_scale, scale_span(*cache), "k_scale"},
                         {cache->v_scale, scale_span(*cache), "v_scale"},
                         {table, table_span(B, table_stride, max_pages), "table"},
                         {seq_len, int64_t(B) * 4, "seq_len"}};
    const Span written[] = {{out, B * heads_bytes, "out"},
                            {lse, int64_t(B) * Hq * 4, "lse"},
                            {workspace, int64_t(workspace_bytes(p, cache->D)), "the workspace"},
                            {err, 4, "err"}};
    for (int w = 0; w < 4; ++w) {
        for (const Span &x : read) {
            const bool in_place = w == 0 && x.p == Q && out == Q && (B == 1 || q_stride == int64_t(Hq) * cache->D);
            LSA_CHECK_ARG(in_place || !meet(written[w], x), "lsa_paged_attn: %s overlaps %s", written[w].name, x.name);
        }
        for (int i = 0; i < w; ++i)
            LSA_CHECK_ARG(!meet(written[w], written[i]), "lsa_paged_attn: %s overlaps %s", written[w].name,
                          written[i].name);
    }

    AttnArgs a = {};
    a.cache = view_of(*cache);
    a.q = Q;
    a.q_stride = q_stride * e;
    a.table = table;
    a.table_stride = table_stride;
    a.reach = int64_t(max_pages) * cache->page_size;
    a.seq_len = seq_len;
    a.B = B;
    a.Hq = Hq;
    a.G = Hq / cache->Hkv;
    a.HG = p.HG;
    a.HS = p.HS;
    a.window = window;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = a.part_o + int64_t(p.grid) * 2 * p.HS * cache->D;
    a.records = reinterpret_cast<Record *>(a.part_ml + int64_t(p.grid) * 2 * p.HS * 2);
    a.err = err;
    a.tile = p.tile;
    a.lead = p.lead;
    a.q_f32 = q_dtype == LSA_F32;
    const int64_t most = window > 0 && window < a.reach ? window : a.reach;
    const int64_t segments = int64_t(B) * cache->Hkv * p.HG;
    a.whole = most <= int64_t(segments * 6 >= p.grid ? kWholeMany : kWholeFew) * p.tile && segments < (int64_t(1) << 30);
    const int grid = a.whole ? int(segments) : p.grid;
    a.by_segment = segments <= grid;
    const int heads = cache->Hkv * p.HG;
    a.lanes = heads <= grid && grid % heads * 16 <= grid ? heads : 1;      // at most a sixteenth of the CTAs stays idle
    cudaStream_t st = as_stream(stream);
    s = cache->dtype == LSA_F32 ? launch_f32(a, p, grid, st)
        : latent_supported(*cache, Hq) ? launch_latent(a, grid, st) : launch_mma(*cache, a, p, grid, st);
    if (s != LSA_OK || a.whole) return s;
    return paged_combine(a, grid, st);
}
