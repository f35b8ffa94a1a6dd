// Attention of one new token over a paged cache with one latent head of 512 under many query heads (K = V, bf16), on
// tcgen05 (paged_attn.cuh says how the work is cut).
//
// 128 query heads on one row make 256 flops a byte: tensor and HBM time are about equal, so both have to run all the
// time.  O for 128 heads x 512 elements would fill the tensor memory, so two CTAs (a cluster) share a piece and split the
// 512 columns:
//   * CTA r holds the rows' columns 256 r .. 256 r + 255: it multiplies S_r = Q_r K_r^T (M = 128 heads, N = 64 entries,
//     K = 256) and, from the same staged rows read MN-major, O_r += P V_r (N = 256, K = 64).  No row is read twice and
//     no product is made twice;
//   * S = S_0 + S_1: each CTA stores its S_r into the other's shared memory (32 KB a tile, st.async, which counts its
//     bytes on the other's barrier) and adds what it gets, so both hold the same scores and make the same weights;
//   * P enters as two bf16 numbers (a weight and what its rounding left), as in paged_attn_mma.cu.
// Tensor memory: O in columns 0 .. 255, two buffers of S in 256 .. 383, Q_r (bf16, the MMA's A operand) in 384 .. 511;
// Q there leaves shared memory to four tiles of rows (32 KB each), P (2 x 16 KB) and two buffers of the other's S.
// Sixteen warps: 0-7 softmax (thread = head, half of the tile's entries), 8-11 send S_r, 12 issues the MMAs, 13-14 load
// rows (TMA or cp.async), 15 tells the other CTA what was read of its scores.  Sending and telling have warps of their own
// because they are slow and nothing depends on them at once: the 32 KB of a tile cross in about 1300 cycles, and a
// release at cluster scope takes 350.
// A tile passes load, S, exchange, softmax, P V; what counts is that these overlap.  S of tile i + 2 is issued as soon as
// the scores of tile i are in registers, before P V of tile i, so neither the exchange nor a product is waited for (with
// S of tile i + 1 issued after P V of tile i - 1 the softmax and the tensor pipe took turns: 423 us for 128 heads over
// 4 x 131072 entries).  The running max is a reference that moves, and O is rescaled, only when a score passes it by 2^8;
// a barrier that every tile needs anyway tells whether one did.  Every wait is bounded; the two CTAs leave together.
//
// Measured: 128 heads over 4 x 131072 entries, 537 MB, 216 to 222 us at 1965 MHz, and 262 us called back to back for
// seconds, where the board's power limit (1000 W) holds the clock at 1640 MHz.  A tile takes about 3800 cycles.  In these
// the MMAs need 1540 at the nominal rate (two thirds of them P V, whose second piece costs a third of all), the exchange
// 1700 (20 bytes a clock each way, measured alone), shared memory 2050 (256 KB at 128 bytes a clock), and the softmax
// warps' own chain 2900: no resource is full, the dependences between them take the rest.  Two sets of softmax warps
// that take turns (240 us) and weights in tensor memory in place of shared memory (224 us) were no faster; sixteen warps on
// one tile took 226 us.
// Under 8 heads or fewer a kv head the mma.sync kernel is faster (64 x 4096 entries: 84 us against 121), from 9 on, where
// it would read the rows twice, this one (16 heads: 123 us against 133; 4 x 32768 entries 69 against 80).  Between 9 and 64
// heads HBM would allow 41 us there (64 x 4096) and 21 (4 x 32768): a tile costs what 128 heads cost, most rows of it empty.
#include <cuda.h>

#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace lsa {
namespace paged {
namespace {

using namespace ptx;

constexpr int kHeads = 128, kD = 512, kCols = 256, kTile = 64, kStages = 4;
constexpr int kSoftWarps = 8, kSendWarp = 8, kSendWarps = 4, kMmaWarp = 12, kLoadWarp = 13, kLoadWarps = 2, kAckWarp = 15;
constexpr int kThreads = 32 * (kAckWarp + 1);
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kTmemS = kCols, kTmemQ = kCols + 2 * kTile;
constexpr int kBlock = kTile * 128;              // 64 columns of a tile: 8 KB
constexpr int kStageBytes = 4 * kBlock;
constexpr int kPBytes = kHeads * 128;            // weights of a tile: 16 KB (and as much for what their rounding left)
constexpr int kRecvBytes = kHeads * kTile * 4;   // the other CTA's S of a tile
constexpr size_t kSmem = 1024 + kStages * size_t(kStageBytes) + 2 * kPBytes + 2 * kRecvBytes;
// the S buffer is not reused: the other CTA may already send the next piece's
static_assert(kSoftWarps * 32 * 32 * 4 <= 2 * kPBytes, "a warp stages 32 x 32 outputs over the weights");
static_assert(kLoadWarps * 32 == kTile, "a load warp's lanes place one row each");
constexpr float kLag = 8.f;

struct Bars {
    uint64_t q_full, kv_full[kStages], kv_free[kStages], mask_full[kStages], s_full[2], s_free[2], s_recv[2], send_ok[2], p_full,
        drain;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Low word of a shared-memory descriptor: start address and leading byte offset in 16-byte units.  K-major operands (P,
// K) have 128-byte rows, whose leading offset is not used; V^T, the same rows read MN-major, has 64-element blocks along
// its elements `lead` bytes apart.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
    return ((addr >> 4) & 0x3FFFu) | ((lead >> 4) & 0x3FFFu) << 16;
}
// High word: groups of 8 rows 1024 bytes apart, descriptor version for tcgen05, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r;
}
// D[tmem] (+)= A * B[smem]^T by the lane with `lead`, bf16 inputs, f32 accumulate: A in shared memory or in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}\n"
        ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}\n"
        ::"r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
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
// Stores 16 bytes in the other CTA and counts them on a barrier of its.
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::
                     "r"(addr), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// mbar_try_wait and mbar_wait that also acquire what the cluster's other CTA released.
__device__ __forceinline__ bool try_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (try_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (try_cluster(bar, parity)) return true;
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
// 4-D tiled TMA load into shared memory of this CTA, completion counted on `bar`.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// rows_map: the cache as [page][slot][head][element]; box: rows of a TMA load, 0 for none.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
paged_attn_latent(const __grid_constant__ CUtensorMap rows_map, AttnArgs a, int box) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *kvs = smem, *ps = kvs + kStages * kStageBytes, *recv = ps + 2 * kPBytes;
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
        mbar_init(&bars.q_full, kSoftWarps);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.kv_full[s], 32 * kLoadWarps);
            mbar_init(&bars.kv_free[s], 1);
            mbar_init(&bars.mask_full[s], kLoadWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars.s_full[s], 1);
            mbar_init(&bars.s_recv[s], 1);
            mbar_init(&bars.s_free[s], kSoftWarps + kSendWarps);
            mbar_init(&bars.send_ok[s], 1);
        }
        mbar_init(&bars.p_full, kSoftWarps);
        mbar_init(&bars.drain, 1);
        fence_mbar_init();
        // a tile's scores from the other CTA: a buffer's next tile is announced when one has come
        mbar_arrive_expect_tx(&bars.s_recv[0], kRecvBytes);
        mbar_arrive_expect_tx(&bars.s_recv[1], kRecvBytes);
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
        if (warp == kAckWarp) {
            // ---- the scores of tile j have been read: the other CTA may send tile j + 2
            if (lane == 0) {
                const uint32_t peer_ok = in_cta(smem_u32(&bars.send_ok[0]), peer);
                for (int j = 0; j < n; ++j) {
                    const uint32_t g = tiles + j, x = g & 1;
                    if (!mbar_wait(&bars.s_free[x], (g >> 1) & 1, abort_v, kWaitLimitNs)) break;
                    arrive_cluster(peer_ok + x * 8);
                }
            }
        } else if (warp >= kLoadWarp) {
            // ---- rows: lane l of warp w places row 32 w + l (entry t, slot s of the sequence's page p; the page's index is
            // read a tile ahead).  Where `box` rows of the tile always lie side by side in a page, one lane of each `box`
            // loads them by TMA, a 64-column block a time (a box of a page that is not there loads zeros: its index is
            // past the cache's end).  Else, and in a piece's last tile, whose entries may end inside a box, eight lanes
            // copy a row, 16 bytes each of its four 128-byte blocks.
            const bool boxes = box > 0 && lo % box == 0;
            const int w = warp - kLoadWarp, lr = lane >> 3, lp = lane & 7;
            const int32_t *row = a.table + int64_t(b) * a.table_stride;
            const uint8_t *base = a.cache.k + kvh * a.cache.head_stride + rank * (kCols * 2) + lp * 16;
            const int hop_p = kTile / a.cache.page_size, hop_s = kTile - hop_p * a.cache.page_size;
            int t = lo + 32 * w + lane, p = t / a.cache.page_size, s_in = t - p * a.cache.page_size;
            int64_t page = t < hi ? row[p] : -1;
            for (int j = 0; j < n; ++j) {
                const uint32_t g = tiles + j, s = g % kStages;
                int64_t off = -1;
                if (t < hi) {
                    if (page >= 0 && page < a.cache.n_pages)
                        off = page * a.cache.page_stride + s_in * a.cache.slot_stride;
                    else
                        raise_err(a.err, LSA_ERR_INVALID);
                }
                const int64_t now_page = page;
                const int now_slot = s_in;
                t += kTile;
                p += hop_p;
                s_in += hop_s;
                if (s_in >= a.cache.page_size) {
                    s_in -= a.cache.page_size;
                    ++p;
                }
                page = t < hi ? row[p] : -1;
                const bool waited = g < kStages || mbar_wait(&bars.kv_free[s], (g / kStages - 1) & 1, abort_v, kWaitLimitNs);
                if (!__all_sync(0xffffffffu, waited)) break;
                const uint32_t mask = __ballot_sync(0xffffffffu, off >= 0);
                const uint32_t dst = smem_u32(kvs) + s * kStageBytes;
                if (boxes && lo + (j + 1) * kTile <= hi) {
                    if (lane == 0) mbar_arrive_expect_tx(&bars.kv_full[s], kStageBytes / kLoadWarps);
                    else mbar_arrive(&bars.kv_full[s]);
                    if (lane % box == 0) {
                        const int pg = off >= 0 ? int(now_page) : int(a.cache.n_pages);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            tma_load_4d(dst + c * kBlock + (32 * w + lane) * 128, &rows_map, &bars.kv_full[s],
                                        int(rank) * kCols + c * 64, kvh, now_slot, pg);
                    }
                    __syncwarp();
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 32 * w + 4 * i + lr;
                        const int64_t from = __shfl_sync(0xffffffffu, off, 4 * i + lr);
                        const uint32_t bytes = from >= 0 ? 16u : 0u;
                        const uint8_t *src = base + (from >= 0 ? from : 0);
                        const uint32_t to = dst + r * 128 + ((lp ^ (r & 7)) << 4);
#pragma unroll
                        for (int c = 0; c < 4; ++c) cp_async_16(to + c * kBlock, src + c * 128, bytes);
                    }
                    cp_async_arrive_noinc(&bars.kv_full[s]);
                }
                if (lane == 0) {
                    s_mask[s][w] = mask;
                    mbar_arrive(&bars.mask_full[s]);
                }
            }
        } else if (warp == kMmaWarp) {
            // ---- MMAs.  The whole warp runs this, so that addresses are the same in all its lanes and stay in uniform
            // registers, and one lane issues: from a branch of one lane each MMA took 85 cycles to issue
            if (n > 0) {
                constexpr uint32_t kIdescS = idesc_bf16(kHeads, kTile);
                constexpr uint32_t kIdescO = idesc_bf16(kHeads, kCols) | (1u << 16);   // B (V) is MN-major
                const uint32_t lead = elect_one();
                const uint32_t kv_lo = desc_lo(smem_u32(kvs), 16), vt_lo = desc_lo(smem_u32(kvs), kBlock);
                const uint32_t p_lo = desc_lo(smem_u32(ps), 16);
                bool ok = mbar_wait(&bars.q_full, pieces & 1, abort_v, kWaitLimitNs);
                auto s_tile = [&](int j) {
                    const uint32_t g = tiles + j, s = g % kStages;
                    if (!mbar_wait(&bars.kv_full[s], (g / kStages) & 1, abort_v, kWaitLimitNs)) return false;
                    if (g >= 2 && !mbar_wait(&bars.s_free[g & 1], ((g >> 1) - 1) & 1, abort_v, kWaitLimitNs)) return false;
                    fence_proxy_async_smem();    // the rows were written by cp.async
                    tc_fence_after();
                    const uint32_t kv = kv_lo + s * (kStageBytes >> 4), d = tmem + kTmemS + (g & 1) * kTile;
#pragma unroll
                    for (int i = 0; i < 16; ++i)      // 16 elements of K: 8 columns of Q
                        mma_ts(lead, d, tmem + kTmemQ + i * 8, kv + (i >> 2) * (kBlock >> 4) + (i & 3) * 2, kIdescS, i != 0);
                    commit_if(lead, &bars.s_full[g & 1]);
                    return true;
                };
                ok = __all_sync(0xffffffffu, ok && s_tile(0) && (n < 2 || s_tile(1)));
                for (int j = 0; j < n && ok; ++j) {
                    if (j + 2 < n) ok = s_tile(j + 2);
                    const uint32_t g = tiles + j, s = g % kStages;
                    ok = __all_sync(0xffffffffu, ok && mbar_wait(&bars.p_full, g & 1, abort_v, kWaitLimitNs));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t vt = vt_lo + s * (kStageBytes >> 4);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_ss(lead, tmem, p_lo + x * (kPBytes >> 4) + i * 2, vt + i * (2048 >> 4), kIdescO,
                                   x != 0 || i != 0 ? 1u : uint32_t(j != 0));
                    commit_if(lead, &bars.kv_free[s]);
                }
                if (!ok) {
                    // what was issued still reads shared memory: let it end before the CTA does
                    volatile int none = 0;
                    commit_if(lead, &bars.drain);
                    mbar_wait(&bars.drain, 0, &none, kWaitLimitNs);
                }
            }
        } else if (warp >= kSendWarp) {
            // ---- S_r of each tile to the other CTA: thread = head, 16 pieces of four entries
            const int quarter = warp & 3, head = 32 * quarter + lane;
            const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
            const uint32_t peer_slot = in_cta(smem_u32(recv) + head * 16, peer);
            const uint32_t peer_recv = in_cta(smem_u32(&bars.s_recv[0]), peer);
            for (int j = 0; j < n; ++j) {
                const uint32_t g = tiles + j, x = g & 1;
                bool ok = mbar_wait(&bars.s_full[x], (g >> 1) & 1, abort_v, kWaitLimitNs);
                // the other CTA has read tile g - 2, which lay there
                ok = ok && (g < 2 || wait_cluster(&bars.send_ok[x], ((g >> 1) - 1) & 1, abort_v));
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after();
                uint32_t sv[64];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld_32x32b_x16(lanes + kTmemS + x * kTile + c * 16, *reinterpret_cast<uint32_t(*)[16]>(&sv[c * 16]));
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.s_free[x]);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    st_async(peer_slot + x * kRecvBytes + c * kHeads * 16, sv[4 * c], sv[4 * c + 1], sv[4 * c + 2],
                             sv[4 * c + 3], peer_recv + x * 8);
            }
        } else {
            // ---- softmax: thread = head 32 * quarter + lane, entries 32 * half .. of each tile
            const int quarter = warp & 3, half = warp >> 2, head = 32 * quarter + lane;
            const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
            const float scale2 = a.scale * kLog2e;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            if (n > 0) {
                // Q_r: this thread's head, 128 of the 256 columns, two to a column of tensor memory
                const int heads = min(kHeads, a.G - first);
                const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.q) + int64_t(b) * a.q_stride +
                                                                 (int64_t(kvh) * a.G + first + head) * (kD * 2) +
                                                                 rank * (kCols * 2) + half * 256);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint4 x = head < heads ? q[4 * c + y] : make_uint4(0, 0, 0, 0);
                        w[4 * y] = x.x;
                        w[4 * y + 1] = x.y;
                        w[4 * y + 2] = x.z;
                        w[4 * y + 3] = x.w;
                    }
                    tmem_st_32x32b_x16(lanes + kTmemQ + half * 64 + c * 16, w);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.q_full);
            }
            for (int j = 0; j < n; ++j) {
                const uint32_t g = tiles + j, s = g % kStages, x = g & 1;
                // three waits, tried together (each takes a hundred cycles even when there is nothing to wait for): S_r, the
                // other CTA's scores, and which rows are there
                const bool t0 = mbar_try_wait(&bars.s_full[x], (g >> 1) & 1);
                const bool t1 = mbar_try_wait(&bars.mask_full[s], (g / kStages) & 1);
                const bool t2 = try_cluster(&bars.s_recv[x], (g >> 1) & 1);
                ok = ok && (t0 || mbar_wait(&bars.s_full[x], (g >> 1) & 1, abort_v, kWaitLimitNs)) &&
                     (t1 || mbar_wait(&bars.mask_full[s], (g / kStages) & 1, abort_v, kWaitLimitNs)) &&
                     (t2 || wait_cluster(&bars.s_recv[x], (g >> 1) & 1, abort_v));
                ok = __all_sync(0xffffffffu, ok);
                if (ok) tc_fence_after();
                if (ok && threadIdx.x == 0) mbar_arrive_expect_tx(&bars.s_recv[x], kRecvBytes);
                // P V of the tile before: when it is done, the weights' buffer is free and O is whole
                auto before_done = [&]() {
                    return j == 0 || mbar_wait(&bars.kv_free[(g + kStages - 1) % kStages], ((g - 1) / kStages) & 1, abort_v,
                                               kWaitLimitNs);
                };
                float v[32], top = -INFINITY;
                if (ok) {
                    const uint32_t mask = s_mask[s][half];
                    uint32_t sv[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tmem_ld_32x32b_x16(lanes + kTmemS + x * kTile + half * 32 + c * 16,
                                           *reinterpret_cast<uint32_t(*)[16]>(&sv[c * 16]));
                    const uint8_t *came = recv + x * kRecvBytes + (half * 8 * kHeads + head) * 16;
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float4 o = *reinterpret_cast<const float4 *>(came + c * kHeads * 16);
                        v[4 * c] = (__uint_as_float(sv[4 * c]) + o.x) * scale2;
                        v[4 * c + 1] = (__uint_as_float(sv[4 * c + 1]) + o.y) * scale2;
                        v[4 * c + 2] = (__uint_as_float(sv[4 * c + 2]) + o.z) * scale2;
                        v[4 * c + 3] = (__uint_as_float(sv[4 * c + 3]) + o.w) * scale2;
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.s_free[x]);
                    if (mask != 0xffffffffu) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) v[u] = (mask >> u) & 1u ? v[u] : -INFINITY;
                    }
                    float t4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int u = 4; u < 32; ++u) t4[u & 3] = fmaxf(t4[u & 3], v[u]);
                    top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                }
                if (!named_barrier_and(1, 32 * kSoftWarps, ok && !(top > m + kLag))) {
                    // a wait gave up, or a reference has to move
                    s_max[half][head] = top;
                    ok = ok && before_done();
                    if (!named_barrier_and(1, 32 * kSoftWarps, ok)) {
                        ok = false;
                        break;
                    }
                    top = fmaxf(s_max[0][head], s_max[1][head]);
                    const float mn = fmaxf(m, top);
                    const float f = exp2_approx(m - (mn == -INFINITY ? 0.f : mn));
                    m = mn;
                    l *= f;
                    if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
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
                    // the two halves of a head have both read s_max before either writes it again
                    named_barrier(2 + quarter, 64);
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const uint32_t p = smem_u32(ps) + head * 128;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t near[16], rest[16];      // the weights, and what their rounding left
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float p0 = exp2_approx(v[2 * e] - ref), p1 = exp2_approx(v[2 * e + 1] - ref);
                    sum[e & 3] += p0 + p1;
                    const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
                    const float2 f = __bfloat1622float2(h);
                    const __nv_bfloat162 r = __floats2bfloat162_rn(p0 - f.x, p1 - f.y);
                    near[e] = *reinterpret_cast<const uint32_t *>(&h);
                    rest[e] = *reinterpret_cast<const uint32_t *>(&r);
                }
                // (a wait that gives up here shows at the next tile's barrier, or at the piece's end)
                ok = before_done();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t at = p + (((4 * half + c) ^ (head & 7)) << 4);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(near[4 * c]), "r"(near[4 * c + 1]),
                                 "r"(near[4 * c + 2]), "r"(near[4 * c + 3])
                                 : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + kPBytes), "r"(rest[4 * c]),
                                 "r"(rest[4 * c + 1]), "r"(rest[4 * c + 2]), "r"(rest[4 * c + 3])
                                 : "memory");
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
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
                        a.lse[hq + head] = lse_of(m, L);
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
    if (*abort_v) {
        // scores and rows that are on their way and were not waited for land well within this time
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000) {}
        __syncwarp();
    }
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

lsa_status launch_latent(const AttnArgs &a, int grid, cudaStream_t st) {
    // rows side by side in a page from any multiple of `box` entries on, at least the 8 of a swizzle atom
    const int size = a.cache.page_size;
    int box = size % 32 == 0 ? 32 : size % 16 == 0 ? 16 : size % 8 == 0 ? 8 : 0;
    CUtensorMap rows_map = {};
    if (box) {
        EncodeTiledFn enc = encode_fn();
        if (!enc) {
            set_error("lsa_paged_attn: cuTensorMapEncodeTiled is unavailable");
            return LSA_ERR_CUDA;
        }
        const cuuint32_t unit[4] = {1, 1, 1, 1}, extent[4] = {64, 1, cuuint32_t(box), 1};
        const cuuint64_t dims[4] = {cuuint64_t(kD), cuuint64_t(a.cache.Hkv), cuuint64_t(size), cuuint64_t(a.cache.n_pages)};
        const cuuint64_t row = kD * 2;
        const cuuint64_t strides[3] = {a.cache.Hkv > 1 ? cuuint64_t(a.cache.head_stride) : row,
                                       cuuint64_t(a.cache.slot_stride),
                                       a.cache.n_pages > 1 ? cuuint64_t(a.cache.page_stride) : row};
        const CUresult r = enc(&rows_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.cache.k, dims, strides, extent, unit,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) box = 0;      // strides that a map cannot hold (2^40 bytes or more): the rows are copied
    }
    LSA_CUDA(ensure_smem(paged_attn_latent, kSmem));
    LSA_CUDA(launch_pdl(paged_attn_latent, dim3(2 * grid), dim3(kThreads), kSmem, st, rows_map, a, box));
    LSA_LAUNCHED("paged_attn_latent");
    return LSA_OK;
}

}  // namespace paged
}  // namespace lsa
