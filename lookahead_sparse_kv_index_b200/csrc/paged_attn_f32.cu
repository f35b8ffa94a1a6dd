// Attention of one new token over a paged cache of fp32 rows, on the CUDA cores (the tensor cores have no fp32 product;
// paged_attn.cuh says how the work is cut).
//
// HBM bounds it as long as no row is read for more than one group of heads, so o of all of a group's NH query heads is
// kept in registers: LT lanes share an entry, each with KC 16-byte pieces of its row, and NH * KC * 4 <= 64.  LT is the
// least that this allows, since an entry's shuffles and exponentials are shared by its lanes (heads of 32 elements: 87 us
// with 4 lanes an entry, 104 with 8; of 64 elements 70 and 75).  Eight heads take twice the lanes an entry of four, which
// costs shuffles, not bytes (sixteen on 32 lanes were slower than two groups of eight: 463 us against 2 x 186 for 537 MB of
// rows).  As in the tensor-core kernel every warp is a pipeline of its own, here with stages of 8 KB of K and V rows
// (cp.async); a lane works on two entries of a step at a time, and every group of LT lanes runs its own online softmax,
// with a reference that moves only when a score passes it by 2^8.  The groups and warps meet at the end of a piece.
//
// Measured: 537 MB of rows under 1 to 4 query heads a kv head 116 us (4.6 TB/s, 71% of the copy rate), under 8 heads 185
// us (45%).  No unit is full at 8 heads: the schedulers issue in 48% of the cycles, the fp32 pipe is busy in 27%, shared
// memory in 45%; with 255 registers there are two warps a scheduler, which wait for shared memory and shuffles (0.7 of
// 2.1 waiting cycles an instruction), for results (0.9) and for instructions (0.5), so the chain of an entry (its rows and
// q from shared memory, products, shuffles, exponentials, products) is what the time goes to.  Heads of 64 elements: 121
// us under 4 heads (69%), 183 under 8; of 32 elements 150 (56%) and 195, by the work an entry costs whatever its length.  A
// batch of 17 MB with a window takes 13 us, of which 9 are the two launches' own latencies.
#include <limits.h>

#include "paged_attn.cuh"

namespace lsa {
namespace paged {
namespace {

constexpr int kMaxWarps = 4, kMaxStages = 4;
constexpr float kLag = 8.f;

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait(int left) {
    if (left <= 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// LT: lanes of an entry; KC: 16-byte pieces of a lane (D <= 4 LT KC); NH: query heads; ST: entries of a stage.
template <int LT, int KC, int NH>
struct Shape {
    static constexpr int kMaxD = 4 * LT * KC;
    static constexpr int kStep = 2 * 32 / LT;                       // entries that a warp works on at a time
    static constexpr int kStage = kMaxD <= 32 ? 32 : kMaxD <= 64 ? 16 : kMaxD <= 128 ? 8 : kMaxD <= 256 ? 4 : 2;
    static constexpr int kCopyLanes = kStage >= 4 ? 8 : 16;         // that copy a row
    static_assert(kStage % kStep == 0 && kStage * kCopyLanes % 32 == 0, "a stage is whole steps and whole copies");
    // bytes between staged rows: where two groups of lanes read neighbouring rows at once, an odd number of 64
    static __host__ __device__ int pitch(int D) { return D * 4 + (LT == 4 && D % 32 == 0 ? 64 : 0); }
    static __host__ __device__ int stage(int D, bool latent) { return kStage * pitch(D) * (latent ? 1 : 2) + 16; }
};

template <int LT, int KC, int NH>
__global__ void __launch_bounds__(kMaxWarps * 32) paged_attn_f32(AttnArgs a, int stages) {
    using C = Shape<LT, KC, NH>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scratch[40];
    const int D = a.cache.D, nch = D / 4, row_bytes = D * 4;
    const bool latent = a.cache.v == a.cache.k;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane / LT, dl = lane % LT;
    const int pitch = C::pitch(D), stage_bytes = C::stage(D, latent), rows = C::kStage * pitch, v_at = latent ? 0 : rows;
    float *qs = reinterpret_cast<float *>(smem);                       // [NH][D]
    uint8_t *ring = smem + NH * row_bytes + size_t(warp) * stages * stage_bytes;
    // where the parts of a piece meet, over the stages
    float *po = reinterpret_cast<float *>(smem + NH * row_bytes), *pml = po + size_t(warps) * NH * D;
    const float scale2 = a.scale * kLog2e;

    pdl_launch_dependents();
    pdl_wait();
    for_pieces(a, blockIdx.x, gridDim.x, scratch, [&](int b, int hseg, int lo, int hi, int slot) {
        const int kvh = hseg / a.HG, first = (hseg % a.HG) * NH;
        const int32_t *row = a.table + int64_t(b) * a.table_stride;
        const int steps = (hi - lo + C::kStage - 1) / C::kStage;
        const int n = steps > warp ? (steps - warp + warps - 1) / warps : 0;   // of this warp: warp, warp + warps, ...

        // lane r places row r of the warp's stages: entry t, slot s of the sequence's page p
        int t = lo + warp * C::kStage + lane, p = t / a.cache.page_size, s = t - p * a.cache.page_size;
        const int hop = warps * C::kStage, hop_p = hop / a.cache.page_size, hop_s = hop - hop_p * a.cache.page_size;
        if (lane >= C::kStage) t = INT_MAX - (1 << 24);     // (past every end; never reaches it)
        auto locate = [&]() {                               // of the next stage
            int64_t off = -1;
            if (t < hi) {
                const int64_t page = row[p];
                if (page >= 0 && page < a.cache.n_pages)
                    off = page * a.cache.page_stride + s * a.cache.slot_stride;
                else
                    raise_err(a.err, LSA_ERR_INVALID);
                t += hop;
                p += hop_p;
                s += hop_s;
                if (s >= a.cache.page_size) {
                    s -= a.cache.page_size;
                    ++p;
                }
            }
            return off;
        };
        const int cr = lane / C::kCopyLanes, cp = lane % C::kCopyLanes;
        const uint8_t *ksrc = a.cache.k + kvh * a.cache.head_stride, *vsrc = a.cache.v + kvh * a.cache.head_stride;
        auto issue = [&](int j, int stage, int64_t off) {
            if (j < n) {
                uint8_t *st = ring + stage * stage_bytes;
#pragma unroll
                for (int k = 0; k < C::kStage * C::kCopyLanes / 32; ++k) {
                    const int r = cr + 32 / C::kCopyLanes * k;
                    const int64_t o = __shfl_sync(0xffffffffu, off, r);
                    const bool ok = o >= 0;
                    const uint8_t *kf = ksrc + (ok ? o : 0), *vf = vsrc + (ok ? o : 0);
                    const uint32_t to = smem_addr(st) + r * pitch;
                    for (int i = cp; i < nch; i += C::kCopyLanes) {
                        cp_async16(to + i * 16, kf + i * 16, ok);
                        if (!latent) cp_async16(to + v_at + i * 16, vf + i * 16, ok);
                    }
                }
                const uint32_t mask = __ballot_sync(0xffffffffu, off >= 0);
                if (lane == 0) *reinterpret_cast<uint32_t *>(st + v_at + rows) = mask;
            }
            cp_commit();
        };

        // the loads that the first stages wait for are all on their way before any is waited for: q, then the pages
        const float *q = reinterpret_cast<const float *>(static_cast<const uint8_t *>(a.q) + int64_t(b) * a.q_stride) +
                         (int64_t(kvh) * a.G + first) * D;
        for (int i = threadIdx.x; i < NH * nch; i += blockDim.x)
            cp_async16(smem_addr(qs) + i * 16, q + i * 4, first + i / nch < a.G);
        int64_t early[kMaxStages - 1];
#pragma unroll
        for (int j = 0; j < kMaxStages - 1; ++j)
            if (j < stages - 1) early[j] = locate();
        int64_t ahead = locate();
#pragma unroll
        for (int j = 0; j < kMaxStages - 1; ++j)
            if (j < stages - 1) issue(j, j, early[j]);      // (q is in the first group)
        // (a warp's first wait does not cover the q of other warps)
        cp_wait(stages - 2);
        __syncthreads();

        float m[NH], l[NH], o[NH][KC][4];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[h][c][e] = 0.f;
        }
        for (int j = 0, now = 0, next = stages - 1; j < n; ++j) {
            cp_wait(stages - 2);
            __syncwarp();
            issue(j + stages - 1, next, ahead);
            ahead = locate();
            const uint8_t *sk = ring + now * stage_bytes, *sv = sk + v_at;
            const uint32_t mask = *reinterpret_cast<const uint32_t *>(sv + rows);
            now = now + 1 == stages ? 0 : now + 1;
            next = next + 1 == stages ? 0 : next + 1;
#pragma unroll
            for (int i = 0; i < C::kStage / C::kStep; ++i) {
                // entries t0 and t1 of the stage
                const int t0 = i * C::kStep + grp, t1 = t0 + C::kStep / 2;
                float s0[NH], s1[NH];
#pragma unroll
                for (int h = 0; h < NH; ++h) s0[h] = s1[h] = 0.f;
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const int ch = c * LT + dl;
                    if (ch < nch) {
                        const float4 x = *reinterpret_cast<const float4 *>(sk + t0 * pitch + ch * 16);
                        const float4 y = *reinterpret_cast<const float4 *>(sk + t1 * pitch + ch * 16);
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            const float4 w = *reinterpret_cast<const float4 *>(qs + h * D + ch * 4);
                            s0[h] = fmaf(w.x, x.x, fmaf(w.y, x.y, fmaf(w.z, x.z, fmaf(w.w, x.w, s0[h]))));
                            s1[h] = fmaf(w.x, y.x, fmaf(w.y, y.y, fmaf(w.z, y.z, fmaf(w.w, y.w, s1[h]))));
                        }
                    }
                }
                const bool ok0 = (mask >> t0) & 1u, ok1 = (mask >> t1) & 1u;
                bool moved = false;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
#pragma unroll
                    for (int x = 1; x < LT; x <<= 1) {
                        s0[h] += __shfl_xor_sync(0xffffffffu, s0[h], x);
                        s1[h] += __shfl_xor_sync(0xffffffffu, s1[h], x);
                    }
                    s0[h] = ok0 ? s0[h] * scale2 : -INFINITY;
                    s1[h] = ok1 ? s1[h] * scale2 : -INFINITY;
                    moved |= fmaxf(s0[h], s1[h]) > m[h] + kLag;
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        const float mn = fmaxf(m[h], fmaxf(s0[h], s1[h]));
                        const float f = exp2_approx(m[h] - (mn == -INFINITY ? 0.f : mn));
                        m[h] = mn;
                        l[h] *= f;
#pragma unroll
                        for (int c = 0; c < KC; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[h][c][e] *= f;
                    }
                }
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float ref = m[h] == -INFINITY ? 0.f : m[h];
                    s0[h] = exp2_approx(s0[h] - ref);
                    s1[h] = exp2_approx(s1[h] - ref);
                    l[h] += s0[h] + s1[h];
                }
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const int ch = c * LT + dl;
                    if (ch < nch) {
                        const float4 x = *reinterpret_cast<const float4 *>(sv + t0 * pitch + ch * 16);
                        const float4 y = *reinterpret_cast<const float4 *>(sv + t1 * pitch + ch * 16);
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            o[h][c][0] = fmaf(s0[h], x.x, fmaf(s1[h], y.x, o[h][c][0]));
                            o[h][c][1] = fmaf(s0[h], x.y, fmaf(s1[h], y.y, o[h][c][1]));
                            o[h][c][2] = fmaf(s0[h], x.z, fmaf(s1[h], y.z, o[h][c][2]));
                            o[h][c][3] = fmaf(s0[h], x.w, fmaf(s1[h], y.w, o[h][c][3]));
                        }
                    }
                }
            }
        }
        cp_wait(0);
        __syncthreads();      // the parts overlay every warp's stages
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            float M = m[h];
#pragma unroll
            for (int x = LT; x < 32; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
            const float f = exp2_approx(m[h] - (M == -INFINITY ? 0.f : M));
            float L = l[h] * f;
#pragma unroll
            for (int x = LT; x < 32; x <<= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = o[h][c][e] * f;
#pragma unroll
                    for (int x = LT; x < 32; x <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], x);
                }
                const int ch = c * LT + dl;
                if (grp == 0 && ch < nch)
                    *reinterpret_cast<float4 *>(po + (size_t(warp) * NH + h) * D + ch * 4) =
                        make_float4(v[0], v[1], v[2], v[3]);
            }
            if (lane == 0) {
                pml[(warp * NH + h) * 2] = M;
                pml[(warp * NH + h) * 2 + 1] = L;
            }
        }
        __syncthreads();
        finish_piece(a, b, hseg, slot, warps, po, pml);
        __syncthreads();
    });
    if (blockIdx.x == 0 && a.err)
        for (int b = threadIdx.x; b < a.B; b += blockDim.x)
            if (a.seq_len[b] > a.reach) raise_err(a.err, LSA_ERR_CAPACITY);
}

template <int LT, int KC, int NH>
struct Run {
    static void plan(bool latent, int D, int G, AttnPlan &p) {
        using C = Shape<LT, KC, NH>;
        const int stage = C::stage(D, latent), q = NH * D * 4;
        p.HS = NH;
        p.HG = (G + NH - 1) / NH;
        // two CTAs of four warps on an SM: up to three stages a warp
        int stages = (112 * 1024 - q) / (kMaxWarps * stage);
        p.stages = stages > kMaxStages ? kMaxStages : stages < 2 ? 2 : stages;
        p.threads = kMaxWarps * 32;
        p.tile = C::kStage * kMaxWarps;
        p.lead = 3;
        p.grid = sm_count() * 2;
        const size_t ring = size_t(p.stages) * kMaxWarps * stage, join = size_t(kMaxWarps) * NH * (D + 2) * 4;
        p.smem = q + (ring > join ? ring : join);
    }
    static lsa_status launch(const AttnArgs &a, const AttnPlan &p, int grid, cudaStream_t st) {
        LSA_CUDA(ensure_smem(paged_attn_f32<LT, KC, NH>, p.smem));
        LSA_CUDA(launch_pdl(paged_attn_f32<LT, KC, NH>, dim3(grid), dim3(p.threads), p.smem, st, a, int(p.stages)));
        LSA_LAUNCHED("paged_attn_f32");
        return LSA_OK;
    }
};

// Calls f with the kernel's shape for a head dim and a group's query heads.
template <typename F>
auto with_shape(int D, int G, F f) {
    const bool few = G <= 4;
    if (D <= 16) return few ? f(Run<4, 1, 4>()) : f(Run<4, 1, 8>());
    if (D <= 32) return few ? f(Run<4, 2, 4>()) : f(Run<4, 2, 8>());
    if (D <= 64) return few ? f(Run<4, 4, 4>()) : f(Run<8, 2, 8>());
    if (D <= 96 && few) return f(Run<8, 3, 4>());
    if (D <= 128) return few ? f(Run<8, 4, 4>()) : f(Run<16, 2, 8>());
    if (D <= 192 && few) return f(Run<16, 3, 4>());
    if (D <= 256) return few ? f(Run<16, 4, 4>()) : f(Run<32, 2, 8>());
    return f(Run<32, 4, 4>());
}

}  // namespace

AttnPlan plan_f32(const lsa_page_cache &c, int Hq) {
    AttnPlan p = {};
    const int G = Hq / c.Hkv;
    with_shape(c.D, G, [&](auto run) { run.plan(c.v == c.k, c.D, G, p); });
    return p;
}

lsa_status launch_f32(const AttnArgs &a, const AttnPlan &p, int grid, cudaStream_t st) {
    return with_shape(a.cache.D, a.G, [&](auto run) { return run.launch(a, p, grid, st); });
}

}  // namespace paged
}  // namespace lsa
