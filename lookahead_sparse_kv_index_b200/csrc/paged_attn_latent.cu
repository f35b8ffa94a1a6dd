// Attention of one new token over a paged cache with one latent head of 512 under many query heads (K = V, bf16), on
// tcgen05 (paged_attn.cuh says how the work is cut).
//
// 128 query heads on one row make 256 flops a byte: tensor and HBM time are about equal, so both have to run all the
// time.  O for 128 heads x 512 elements fills the tensor memory, and Q with two tiles of rows does not fit in shared
// memory, so two CTAs (a cluster) share a piece and split the 512 columns:
//   * CTA r holds Q's and the rows' columns 256 r .. 256 r + 255: it multiplies S_r = Q_r K_r^T (M = 128 heads, N = 64
//     entries, K = 256) and, from the same staged rows read MN-major, O_r += P V_r (N = 256, K = 64).  No row is read
//     twice and no product is made twice;
//   * S = S_0 + S_1: each CTA writes its S_r to the other's shared memory (32 KB a tile) and adds what it gets, so both
//     hold the same scores and make the same weights;
//   * P enters as two bf16 numbers (a weight and what its rounding left), as in paged_attn_mma.cu.
// Eleven warps: 0-7 softmax (thread = head, half of the tile's entries), 8 issues the MMAs, 9-10 copy rows (cp.async,
// 64 rows x 512 B a tile, three tiles in the ring).  S of tile i + 1 is issued before P V of tile i, so the softmax of a
// tile runs beside P V of the one before and S of the one after; S has two buffers in tensor memory (columns 256 .. 383),
// O has columns 0 .. 255.  The running max is a reference that moves, and O is rescaled, only when a score passes it by
// 2^8.  Every wait is bounded; the two CTAs leave together.
#include <cuda.h>

#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace lsa {
namespace paged {
namespace {

using namespace ptx;

constexpr int kHeads = 128, kD = 512, kCols = 256, kTile = 64, kStages = 3;
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kLoadWarps = 2;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kQSlice = kHeads * 128;            // 64 columns of Q: 16 KB
constexpr int kQBytes = 4 * kQSlice;
constexpr int kBlock = kTile * 128;              // 64 columns of a tile: 8 KB
constexpr int kStageBytes = 4 * kBlock;
constexpr int kPBytes = kHeads * 128;            // weights of a tile: 16 KB (and as much for what their rounding left)
constexpr int kRecvBytes = kHeads * kTile * 4;   // the other CTA's S of a tile
constexpr size_t kSmem = 1024 + kQBytes + kStages * size_t(kStageBytes) + 2 * kPBytes + kRecvBytes;
// the S buffer is not reused: the other CTA may already send the next piece's
static_assert(kSoftWarps * 32 * 32 * 4 <= 2 * kPBytes, "a warp's 32 x 32 output block is staged over the weights");
static_assert(kLoadWarps * 32 == kTile, "a load warp's lanes place one row each");
constexpr float kLag = 8.f;

struct Bars {
    uint64_t q_full, kv_full[kStages], kv_free[kStages], mask_full[kStages], s_full[2], p_full, s_recv, send_ok, drain;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Shared-memory descriptor of an MN-major operand with the 128-byte swizzle: 64-element blocks along MN `lbo` bytes
// apart, 8-row groups along K 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t addr, uint32_t lbo) {
    uint64_t d = 0;
    d |= uint64_t((addr >> 4) & 0x3FFFu);
    d |= uint64_t((lbo >> 4) & 0x3FFFu) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address of a shared-memory variable of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// mbar_wait whose success also acquires what the cluster's other CTA released.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const uint64_t t0 = global_timer_ns();
    while (true) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (done) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
            "r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
paged_attn_latent(const __grid_constant__ CUtensorMap qmap, AttnArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qs = smem, *kvs = qs + kQBytes, *ps = kvs + kStages * kStageBytes, *recv = ps + 2 * kPBytes;
    __shared__ Bars bars;
    __shared__ int64_t scratch[40];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ uint32_t s_mask[kStages][kLoadWarps];     // bit r of word w: row 32 w + r of the tile is there
    __shared__ float s_max[2][kHeads];                   // and the piece's sums, once its last weights are made
    volatile int *abort_v = &abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
    const int cta = blockIdx.x >> 1, ctas = gridDim.x >> 1;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(&bars.q_full, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.kv_full[s], 32 * kLoadWarps);
            mbar_init(&bars.kv_free[s], 1);
            mbar_init(&bars.mask_full[s], kLoadWarps);
        }
        mbar_init(&bars.s_full[0], 1);
        mbar_init(&bars.s_full[1], 1);
        mbar_init(&bars.p_full, kSoftWarps);
        mbar_init(&bars.s_recv, kSoftWarps);
        mbar_init(&bars.send_ok, kSoftWarps);
        mbar_init(&bars.drain, 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    cluster_sync();      // the other CTA's barriers are set up too
    const uint32_t tmem = tmem_slot;
    pdl_wait();

    uint32_t tiles = 0, pieces = 0;    // done by this CTA: the phases of its barriers go on from piece to piece
    bool gave_up = false;
    for_pieces(a, cta, ctas, scratch, [&](int b, int hseg, int lo, int hi, int slot) {
        if (gave_up) return;
        const int kvh = hseg / a.HG, first = (hseg % a.HG) * kHeads;
        const int n = (hi - lo + kTile - 1) / kTile;
        if (warp >= kLoadWarp) {
            // ---- rows: lane l of warp w places row 32 w + l; the warp then copies its 32 rows, one a pass
            const int w = warp - kLoadWarp;
            const int32_t *row = a.table + int64_t(b) * a.table_stride;
            const uint8_t *base = a.cache.k + kvh * a.cache.head_stride + rank * (kCols * 2) + lane * 16;
            int64_t ahead = -1;
            auto locate = [&](int j) {
                const int t = lo + j * kTile + 32 * w + lane;
                return j < n && t < hi ? entry_at(a, row, t).off : int64_t(-1);
            };
            ahead = locate(0);
            for (int j = 0; j < n; ++j) {
                const uint32_t g = tiles + j, s = g % kStages;
                if (g >= kStages && !mbar_wait(&bars.kv_free[s], (g / kStages - 1) & 1, abort_v, kWaitLimitNs)) break;
                const uint32_t mask = __ballot_sync(0xffffffffu, ahead >= 0);
                const uint32_t dst = smem_u32(kvs) + s * kStageBytes;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    // lane l copies piece l of the half row: piece l % 8 of column block l / 8
                    const int r = 32 * w + i;
                    const int64_t off = __shfl_sync(0xffffffffu, ahead, i);
                    cp_async_16(dst + (lane >> 3) * kBlock + r * 128 + (((lane & 7) ^ (r & 7)) << 4),
                                base + (off >= 0 ? off : 0), off >= 0 ? 16u : 0u);
                }
                cp_async_arrive_noinc(&bars.kv_full[s]);
                if (lane == 0) {
                    s_mask[s][w] = mask;
                    mbar_arrive(&bars.mask_full[s]);
                }
                ahead = locate(j + 1);
            }
        } else if (warp == kMmaWarp) {
            // ---- MMAs
            if (lane == 0 && n > 0) {
                constexpr uint32_t kIdescS = idesc_bf16(kHeads, kTile);
                constexpr uint32_t kIdescO = idesc_bf16(kHeads, kCols) | (1u << 16);   // B (V) is MN-major
                mbar_arrive_expect_tx(&bars.q_full, kQBytes);
                for (int i = 0; i < 4; ++i)
                    tma_load_3d(qs + i * kQSlice, &qmap, &bars.q_full, int(rank) * kCols + i * 64, kvh * a.G + first, b);
                bool ok = mbar_wait(&bars.q_full, pieces & 1, abort_v, kWaitLimitNs);
                auto s_tile = [&](int j) {
                    const uint32_t g = tiles + j, s = g % kStages;
                    if (!mbar_wait(&bars.kv_full[s], (g / kStages) & 1, abort_v, kWaitLimitNs)) return false;
                    fence_proxy_async_smem();    // the rows were written by cp.async
                    tc_fence_after();
                    const uint32_t q = smem_u32(qs), kv = smem_u32(kvs) + s * kStageBytes;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        mma_f16(tmem + kCols + (g & 1) * kTile, desc_sw128(q + (i >> 2) * kQSlice + (i & 3) * 32),
                                desc_sw128(kv + (i >> 2) * kBlock + (i & 3) * 32), kIdescS, i != 0);
                    mma_commit(&bars.s_full[g & 1]);
                    return true;
                };
                ok = ok && s_tile(0);
                for (int j = 0; j < n && ok; ++j) {
                    if (j + 1 < n) ok = s_tile(j + 1);
                    const uint32_t g = tiles + j, s = g % kStages;
                    ok = ok && mbar_wait(&bars.p_full, g & 1, abort_v, kWaitLimitNs);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t p = smem_u32(ps), kv = smem_u32(kvs) + s * kStageBytes;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_f16(tmem, desc_sw128(p + x * kPBytes + i * 32), desc_sw128_mn(kv + i * 2048, kBlock),
                                    kIdescO, j != 0 || x != 0 || i != 0);
                    mma_commit(&bars.kv_free[s]);
                }
                if (!ok) {
                    // what was issued still reads shared memory: let it end before the CTA does
                    volatile int none = 0;
                    mma_commit(&bars.drain);
                    mbar_wait(&bars.drain, 0, &none, kWaitLimitNs);
                }
            }
        } else {
            // ---- softmax: thread = head 32 * quarter + lane, entries 32 * half .. of each tile
            const int quarter = warp & 3, half = warp >> 2, head = 32 * quarter + lane;
            const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
            const float scale2 = a.scale * kLog2e;
            const uint32_t slot_at = smem_u32(recv) + (half * 8 * kHeads + head) * 16;
            const uint32_t peer_slot = in_cta(slot_at, peer);
            const uint32_t peer_recv = in_cta(smem_u32(&bars.s_recv), peer), peer_ok = in_cta(smem_u32(&bars.send_ok), peer);
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < n; ++j) {
                const uint32_t g = tiles + j, s = g % kStages;
                ok = mbar_wait(&bars.s_full[g & 1], (g >> 1) & 1, abort_v, kWaitLimitNs);
                ok = ok && (g == 0 || wait_cluster(&bars.send_ok, (g - 1) & 1, abort_v));
                if (!named_barrier_and(1, 32 * kSoftWarps, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t sv[32];
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    tmem_ld_32x32b_x16(lanes + kCols + (g & 1) * kTile + half * 32 + c * 16,
                                       *reinterpret_cast<uint32_t(*)[16]>(&sv[c * 16]));
                tmem_ld_wait();
                tc_fence_before();
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    st_cluster(peer_slot + c * kHeads * 16, sv[4 * c], sv[4 * c + 1], sv[4 * c + 2], sv[4 * c + 3]);
                fence_cluster();
                __syncwarp();
                if (lane == 0) arrive_cluster(peer_recv);
                ok = wait_cluster(&bars.s_recv, g & 1, abort_v) &&
                     mbar_wait(&bars.mask_full[s], (g / kStages) & 1, abort_v, kWaitLimitNs);
                const uint32_t mask = s_mask[s][half];
                float v[32], top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 o = *reinterpret_cast<const float4 *>(recv + (half * 8 + c) * kHeads * 16 + head * 16);
                    v[4 * c] = __uint_as_float(sv[4 * c]) + o.x;
                    v[4 * c + 1] = __uint_as_float(sv[4 * c + 1]) + o.y;
                    v[4 * c + 2] = __uint_as_float(sv[4 * c + 2]) + o.z;
                    v[4 * c + 3] = __uint_as_float(sv[4 * c + 3]) + o.w;
                }
                __syncwarp();
                if (lane == 0) arrive_cluster(peer_ok);
                if (mask == 0xffffffffu) {
#pragma unroll
                    for (int u = 0; u < 32; ++u) v[u] *= scale2;
                } else {
#pragma unroll
                    for (int u = 0; u < 32; ++u) v[u] = (mask >> u) & 1u ? v[u] * scale2 : -INFINITY;
                }
#pragma unroll
                for (int u = 0; u < 32; ++u) top = fmaxf(top, v[u]);
                s_max[half][head] = top;
                // P V of the tile before is done with the weights' buffer and with O
                if (j > 0) ok = ok && mbar_wait(&bars.kv_free[(g - 1) % kStages], ((g - 1) / kStages) & 1, abort_v, kWaitLimitNs);
                if (!named_barrier_and(1, 32 * kSoftWarps, ok)) {
                    ok = false;
                    break;
                }
                top = fmaxf(s_max[0][head], s_max[1][head]);
                const bool move = top > m + kLag;
                if (__any_sync(0xffffffffu, move)) {
                    const float mn = fmaxf(m, top);
                    const float f = exp2_approx(m - (mn == -INFINITY ? 0.f : mn));
                    m = mn;
                    l *= f;
                    if (j > 0) {
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(lanes + half * 128 + c * 16, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                            tmem_st_32x32b_x16(lanes + half * 128 + c * 16, o);
                        }
                        tmem_st_wait();
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const uint32_t p = smem_u32(ps) + head * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t hi4[4], lo4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p0 = exp2_approx(v[8 * c + 2 * e] - ref), p1 = exp2_approx(v[8 * c + 2 * e + 1] - ref);
                        l += p0 + p1;
                        const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
                        const float2 f = __bfloat1622float2(h);
                        const __nv_bfloat162 r = __floats2bfloat162_rn(p0 - f.x, p1 - f.y);
                        hi4[e] = *reinterpret_cast<const uint32_t *>(&h);
                        lo4[e] = *reinterpret_cast<const uint32_t *>(&r);
                    }
                    const uint32_t at = p + (((4 * half + c) ^ (head & 7)) << 4);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(hi4[0]), "r"(hi4[1]),
                                 "r"(hi4[2]), "r"(hi4[3])
                                 : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + kPBytes), "r"(lo4[0]), "r"(lo4[1]),
                                 "r"(lo4[2]), "r"(lo4[3])
                                 : "memory");
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full);
            }
            // ---- the piece's output: this CTA's 256 columns, 32 heads x 32 columns a warp at a time through shared memory
            const uint32_t last = tiles + n - 1;
            if (n > 0) ok = ok && mbar_wait(&bars.kv_free[last % kStages], (last / kStages) & 1, abort_v, kWaitLimitNs);
            s_max[half][head] = l;
            if (named_barrier_and(1, 32 * kSoftWarps, ok)) {
                tc_fence_after();
                const float L = s_max[0][head] + s_max[1][head];
                const int heads = min(kHeads, a.G - first);
                const int64_t hq = int64_t(b) * a.Hq + kvh * a.G + first;
                const float f = slot < 0 ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
                float *stage = reinterpret_cast<float *>(ps) + warp * 32 * 32;   // 16-byte piece p of row r at p ^ (r % 8)
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        tmem_ld_32x32b_x16(lanes + half * 128 + c * 32 + x * 16, *reinterpret_cast<uint32_t(*)[16]>(&o[x * 16]));
                    tmem_ld_wait();
#pragma unroll
                    for (int u = 0; u < 32; u += 4)
                        *reinterpret_cast<float4 *>(stage + lane * 32 + (((u >> 2) ^ (lane & 7)) << 2)) =
                            n == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                   : make_float4(__uint_as_float(o[u]) * f, __uint_as_float(o[u + 1]) * f,
                                                 __uint_as_float(o[u + 2]) * f, __uint_as_float(o[u + 3]) * f);
                    __syncwarp();
                    // eight lanes a row: 16 bytes each
                    const int col = int(rank) * kCols + half * 128 + c * 32 + (lane & 7) * 4;
#pragma unroll
                    for (int r0 = 0; r0 < 32; r0 += 4) {
                        const int r = r0 + (lane >> 3), h = 32 * quarter + r;
                        const float4 x = *reinterpret_cast<const float4 *>(stage + r * 32 + (((lane & 7) ^ (r & 7)) << 2));
                        if (h < heads) {
                            if (slot >= 0) {
                                *reinterpret_cast<float4 *>(a.part_o + (int64_t(slot) * kHeads + h) * kD + col) = x;
                            } else {
                                const __nv_bfloat162 lo2 = __floats2bfloat162_rn(x.x, x.y), hi2 = __floats2bfloat162_rn(x.z, x.w);
                                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + (hq + h) * kD + col) =
                                    make_uint2(*reinterpret_cast<const uint32_t *>(&lo2), *reinterpret_cast<const uint32_t *>(&hi2));
                            }
                        }
                    }
                    __syncwarp();
                }
                if (rank == 0 && half == 0 && head < heads) {
                    if (slot >= 0) {
                        a.part_ml[(int64_t(slot) * kHeads + head) * 2] = m;
                        a.part_ml[(int64_t(slot) * kHeads + head) * 2 + 1] = L;
                    } else if (a.lse) {
                        a.lse[hq + head] = L == 0.f ? -INFINITY : (m + log2f(L)) * kLn2;
                    }
                }
            }
            tc_fence_before();
        }
        tiles += n;
        pieces += n > 0;
        __syncwarp();
        __syncthreads();      // O, Q and the weights' buffer are free again
        tc_fence_after();
        gave_up = *abort_v != 0;
    });
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    __syncthreads();
    cluster_sync();           // nothing of the other CTA is on its way here any more
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0) {
        if (*abort_v) raise_err(a.err, LSA_ERR_TIMEOUT);
    }
    if (blockIdx.x == 0 && a.err)
        for (int b = threadIdx.x; b < a.B; b += blockDim.x)
            if (a.seq_len[b] > a.reach) raise_err(a.err, LSA_ERR_CAPACITY);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

}  // namespace

bool latent_supported(const lsa_page_cache &c, int Hq) {
    return c.dtype == LSA_BF16 && c.v == c.k && c.D == kD && Hq / c.Hkv > 8;
}

AttnPlan plan_latent(const lsa_page_cache &c, int Hq) {
    AttnPlan p = {};
    p.HS = kHeads;
    p.HG = (Hq / c.Hkv + kHeads - 1) / kHeads;
    p.tile = kTile;
    p.lead = 5;
    p.grid = sm_count() / 2;      // clusters of two CTAs
    return p;
}

lsa_status launch_latent(const lsa_page_cache &c, const AttnArgs &a, int grid, cudaStream_t st) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) {
        set_error("lsa_paged_attn: cuTensorMapEncodeTiled is unavailable");
        return LSA_ERR_CUDA;
    }
    CUtensorMap qmap;
    const cuuint32_t estr[3] = {1, 1, 1};
    const cuuint64_t dims[3] = {cuuint64_t(kD), cuuint64_t(a.Hq), cuuint64_t(a.B)};
    const cuuint64_t strides[2] = {cuuint64_t(kD) * 2, cuuint64_t(a.q_stride)};
    const cuuint32_t box[3] = {64, kHeads, 1};
    const CUresult r = enc(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("lsa_paged_attn: cuTensorMapEncodeTiled failed (%d)", int(r));
        return LSA_ERR_CUDA;
    }
    LSA_CUDA(ensure_smem(paged_attn_latent, kSmem));
    LSA_CUDA(launch_pdl(paged_attn_latent, dim3(2 * grid), dim3(kThreads), kSmem, st, qmap, a));
    LSA_LAUNCHED("paged_attn_latent");
    return LSA_OK;
}

}  // namespace paged
}  // namespace lsa
