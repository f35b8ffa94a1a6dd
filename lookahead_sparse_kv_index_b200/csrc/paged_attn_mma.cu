// Attention of one new token over a paged cache, on the tensor cores (bf16 and e4m3 rows; paged_attn.cuh says how the
// work is cut).
//
// One new token per sequence makes S = q K^T a product with as few rows as query heads share a kv head (1 .. 32), so
// the entries take the 16-row side of mma.m16n8k16 and the heads its 8-column side: S^T = K q^T, then O^T = V^T P^T.
// Nothing of it is near the tensor rate; what bounds the kernel is HBM, and the layout serves that:
//   * every warp is a pipeline of its own: it copies steps of 16 or 32 entries (8 KB of K and V rows at a head dim of
//     128 bf16) through `stages` cp.async stages and never waits for another warp before the end of a piece;
//   * K is read from shared memory 16 bytes a lane, straight into A fragments: which 8 (16 for e4m3) elements of a head
//     dim are a fragment's k index is a free choice as long as q's fragment makes the same one;
//   * V^T needs pairs of entries side by side for one element: bf16 rows are transposed as they are loaded (ldmatrix),
//     of e4m3 rows a lane reads 16 bytes of four entries and byte permutes pair them; the entry of each fragment index is
//     chosen (entry_of) so that no read has bank conflicts;
//   * the running max is a reference that lags: it moves (and o is rescaled) only when a score passes it by 2^8, so most
//     steps need neither the max over the step's entries nor a shuffle;
//   * P^T leaves the accumulators with entries along its rows and has to enter with entries along k: one 8 x 8
//     movmatrix transpose a tile.
// Types.  bf16 rows are multiplied as they are.  e4m3 rows become f16 (exactly); q becomes f16 times a power of two of
// its own head, which is exact for elements down to 2^-28 of the head's largest and off by less than 2^-38 of it below;
// the scales of K multiply the fp32 scores, those of V the weights before they are rounded.
// Weights.  A bf16 weight's rounding (2^-8) is as large as the output's own, and with one such number a weight the error
// of the result is 1.4 times that of rounding it once; so what the rounding left is rounded too and multiplied as well
// (2^-16 then).  An f16 weight's rounding (2^-11) is an eighth of the output's: one number does while it is a normal f16.
// The range that leaves is kept around what counts: with p a row's softmax weight and s its V scale, p s enters times
// 2^(9 - r), where 2^r is the power of two at or below a head's largest p s so far, less what the running max has moved
// since.  It moves up (and o is rescaled) only when a product would pass 2^15, so products down to 2^-23 of the head's
// largest are normal, and smaller ones off by at most 2^-34 of that.  Rows of zeros do not count as the largest: their
// scale says nothing of a value.  (A reference that follows the scales alone, whatever the rows' weights, is lost to one
// row of zeros at scale 1 among values of 1e-4.)
//
// Measured: 2 x 65536 entries of 8 bf16 heads of 128 under 64 query heads, 537 MB, 96 us, 5.6 TB/s (86% of the copy rate);
// 64 sequences of up to 16384 entries, 479 MB, 89 us (83%).  The same bytes of e4m3 rows, 118 us (72%): twice the elements
// a byte, each converted, permuted and multiplied; 322 MB of ragged e4m3 contexts 75 us (66%).  More heads a kv head
// cost e4m3 rows more work on the same bytes: 277 MB (2 x 65536 entries of 8 heads of 128) take 67 us under 8 heads a kv
// head, 84 under 16 and 154 under 32, where the loop spills 480 bytes.  Keeping the products' range is two products and a
// maximum a weight: 2 to 6% of the time under up to 8 heads, 9% under 16, 18% under 32.  Where 5% of the rows are zeros at
// scale 1 among values of 0.01, most steps move a reference: 72 us in place of 66.
#include <limits.h>

#include "paged_attn.cuh"

namespace lsa {
namespace paged {
namespace {

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait(int left) {
    if (left <= 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ float lds_f(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// Four 8 x 8 tiles of 16-bit elements, each transposed.
__device__ __forceinline__ void ldmatrix_trans(uint32_t at, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(at));
}
// Two e4m3 values (low 16 bits; high 16 bits) to two f16.
__device__ __forceinline__ void e4m3_to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two weights as bf16 numbers, and what their rounding left as two more.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Staged row of fragment index r (0 .. 15), chosen so that no read of shared memory has bank conflicts while rows are an
// odd number of 16-byte pieces apart, or have their pieces permuted by the row's low bits.  A K read's phase is eight
// lanes with the rows of indices (2j, 2j + 1) and four pieces: these rows lie 4 apart.  V^T of bf16 comes by transposing
// 8 x 8 loads, whose eight rows are any eight neighbours; V of e4m3 by phases of the rows of (0, 2, 4, 6), (1, 3, 5, 7)
// and so on and two pieces: rows 2 apart.
template <bool E4M3>
__device__ __forceinline__ int entry_of(int r) {
    const int j = (r >> 1) & 3, hi = r >> 3;
    if (E4M3) return r & 1 ? 8 + ((2 * j + 4) & 7) + hi : 2 * j + hi;
    return 8 * hi + 4 * (r & 1) + j;
}

// A shape of the kernel.  KB: 64-byte blocks of a row; NT: groups of 8 query heads.
template <bool E4M3, int KB, int NT>
struct Shape {
    static constexpr int kPieces = KB * 4;                              // 16-byte pieces of a staged row
    static constexpr bool kSwizzle = kPieces % 8 == 0;
    static constexpr int kPitch = (kSwizzle ? kPieces : kPieces + 1) * 16;
    static constexpr int kM = KB <= 2 ? 2 : 1;                          // 16-entry tiles of a step
    static constexpr int kStep = 16 * kM;
    static constexpr int kElems = E4M3 ? 16 : 8;                        // elements of a piece
    static constexpr int kPass = (kPieces + 7) / 8;                     // e4m3: 8-piece passes over a V row
    static constexpr int kTiles = E4M3 ? 8 * kPass : kPieces / 2;       // O^T tiles of 16 elements
    static constexpr int kQPer = E4M3 ? 2 : 1;                          // 16-byte q fragments of a block and head group
    static constexpr bool kQInRegs = KB * NT * kQPer * 4 <= 32;
    static constexpr int kQBytes = KB * NT * kQPer * 512;
    static constexpr int kLanes = kSwizzle ? 8 : 4;                     // lanes that copy a row, piece by piece
    static constexpr int kRows = kStep * kPitch;                        // bytes of a stage's K (or V) rows
    static constexpr int kTail = 16 + (E4M3 ? kStep * 8 : 0);           // entry mask, scales
    static constexpr int kHeads = 8 * NT;
    __host__ __device__ static constexpr int stage(bool latent) { return kRows * (latent ? 1 : 2) + kTail; }
};

constexpr int kMaxWarps = 4, kMaxStages = 4;
constexpr float kLag = 8.f;
constexpr uint32_t kMostFactor = 127 + 9 + 100;     // of e4m3 weights, as a biased exponent
constexpr float kMostWeight = 32768.f;              // (f16 ends at 65504)

template <bool E4M3, int KB, int NT>
__global__ void __launch_bounds__(kMaxWarps * 32) paged_attn_mma(AttnArgs a, int stages) {
    using C = Shape<E4M3, KB, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scratch[40];
    __shared__ float q_scale[C::kHeads];
    const int D = a.cache.D, nch = D / C::kElems;
    const bool latent = a.cache.v == a.cache.k;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int stage_bytes = C::stage(latent), v_at = latent ? 0 : C::kRows;
    const uint32_t mine = smem_addr(smem) + C::kQBytes + warp * stages * stage_bytes;
    const uint32_t qf = smem_addr(smem);
    // where the parts of a piece meet, over the stages
    float *po = reinterpret_cast<float *>(smem + C::kQBytes);
    float *pml = po + size_t(warps) * C::kHeads * D;
    const float scale2 = a.scale * kLog2e;

    auto piece_at = [](int row, int p) { return row * C::kPitch + ((C::kSwizzle ? p ^ (row & 7) : p) << 4); };

    pdl_launch_dependents();
    pdl_wait();
    auto do_piece = [&](int b, int hseg, int lo, int hi, int slot) {
        const int kvh = hseg / a.HG, first = (hseg % a.HG) * C::kHeads;
        const int32_t *row = a.table + int64_t(b) * a.table_stride;
        const uint8_t *kbase = a.cache.k + kvh * a.cache.head_stride, *vbase = a.cache.v + kvh * a.cache.head_stride;
        const int steps = (hi - lo + C::kStep - 1) / C::kStep;
        const int n = steps > warp ? (steps - warp + warps - 1) / warps : 0;   // of this warp: warp, warp + warps, ...

        // lane r places row r of the warp's steps: entry t, slot s of the sequence's page p
        int t = lo + warp * C::kStep + lane, p = t / a.cache.page_size, s = t - p * a.cache.page_size;
        const int hop = warps * C::kStep, hop_p = hop / a.cache.page_size, hop_s = hop - hop_p * a.cache.page_size;
        if (lane >= C::kStep) t = INT_MAX - (1 << 24);     // (past every end; never reaches it)
        auto locate = [&]() {                              // of the next step
            Entry e{-1, 0};
            if (t < hi) {
                const int64_t page = row[p];
                if (page >= 0 && page < a.cache.n_pages) {
                    e.off = page * a.cache.page_stride + s * a.cache.slot_stride;
                    e.slot = page * a.cache.page_size + s;
                } else {
                    raise_err(a.err, LSA_ERR_INVALID);
                }
                t += hop;
                p += hop_p;
                s += hop_s;
                if (s >= a.cache.page_size) {
                    s -= a.cache.page_size;
                    ++p;
                }
            }
            return e;
        };
        const int lr = lane / C::kLanes, lp = lane % C::kLanes;
        const uint8_t *ksrc = kbase + lp * 16, *vsrc = vbase + lp * 16;
        auto issue = [&](int j, int stage, const Entry &e) {
            if (j < n) {
                const uint32_t st = mine + stage * stage_bytes;
#pragma unroll
                for (int k = 0; k < C::kStep * C::kLanes / 32; ++k) {
                    const int r = lr + 32 / C::kLanes * k;
                    const int64_t off = __shfl_sync(0xffffffffu, e.off, r);
                    const bool there = off >= 0;
                    const int64_t from = there ? off : 0;
                    const uint32_t to = st + piece_at(r, lp);
#pragma unroll
                    for (int i = 0; i < C::kPieces / C::kLanes; ++i) {
                        const bool ok = there && lp + i * C::kLanes < nch;
                        cp_async16(to + i * C::kLanes * 16, ksrc + from + i * C::kLanes * 16, ok);
                        if (!latent) cp_async16(to + v_at + i * C::kLanes * 16, vsrc + from + i * C::kLanes * 16, ok);
                    }
                }
                const uint32_t tail = st + v_at + C::kRows;
                const uint32_t mask = __ballot_sync(0xffffffffu, e.off >= 0);
                if (lane == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(tail), "r"(mask) : "memory");
                if (E4M3 && lane < C::kStep) {
                    const bool ok = e.off >= 0;
                    const int64_t at = ok ? e.slot * a.cache.Hkv + kvh : 0;
                    cp_async4(tail + 16 + lane * 4, a.cache.ks + at, ok);
                    cp_async4(tail + 16 + (C::kStep + lane) * 4, a.cache.vs + at, ok);
                }
            }
            cp_commit();
        };

        // the pages of the first stages are all on their way before any is waited for
        Entry early[kMaxStages - 1];
#pragma unroll
        for (int j = 0; j < kMaxStages - 1; ++j)
            if (j < stages - 1) early[j] = locate();
        Entry ahead = locate();

        // q fragments of the piece's heads: lane (g, c) of block kb and head group nt holds head 8 nt + g, piece 4 kb + c
        {
            const uint16_t *q = reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(a.q) +
                                                                   int64_t(b) * a.q_stride) +
                                (int64_t(kvh) * a.G + first) * D;
            if constexpr (E4M3) {
                for (int h = warp; h < C::kHeads; h += warps) {
                    float m = 0.f;
                    if (first + h < a.G)
                        for (int d = lane; d < D; d += 32) m = fmaxf(m, fabsf(bf16_to_f32(q[int64_t(h) * D + d])));
#pragma unroll
                    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                    // 2^(13 - exponent): the largest element comes to lie in [2^13, 2^14)
                    int e = int(__float_as_uint(m) >> 23) - 127;
                    e = m == 0.f || e == 128 ? 13 : e < -110 ? -110 : e;
                    if (lane == 0) q_scale[h] = __uint_as_float(uint32_t(127 + 13 - e) << 23);
                }
                __syncthreads();
            }
            for (int i = threadIdx.x; i < KB * NT * 32; i += blockDim.x) {
                const int l = i & 31, nt = (i >> 5) % NT, kb = (i >> 5) / NT;
                const int h = nt * 8 + (l >> 2), p = kb * 4 + (l & 3);
                const bool ok = first + h < a.G && p < nch;
                const uint16_t *from = q + int64_t(h) * D + p * C::kElems;
                const uint32_t to = qf + ((kb * NT + nt) * C::kQPer) * 512 + l * 16;
                if constexpr (!E4M3) {
                    cp_async16(to, from, ok);
                } else {
                    const float f = q_scale[h];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint4 v = ok ? reinterpret_cast<const uint4 *>(from)[x] : make_uint4(0, 0, 0, 0);
                        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const __half2 t = __floats2half2_rn(__uint_as_float(w[y] << 16) * f,
                                                                __uint_as_float(w[y] & 0xffff0000u) * f);
                            w[y] = *reinterpret_cast<const uint32_t *>(&t);
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + x * 512), "r"(w[0]), "r"(w[1]),
                                     "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kMaxStages - 1; ++j)
            if (j < stages - 1) issue(j, j, early[j]);      // (q is in the first group)
        // (a warp's first wait does not cover the q of other warps)
        if constexpr (!E4M3) cp_wait(stages - 2);
        __syncthreads();
        uint4 qr[C::kQInRegs ? KB * NT * C::kQPer : 1];
        if constexpr (C::kQInRegs) {
#pragma unroll
            for (int i = 0; i < KB * NT * C::kQPer; ++i) qr[i] = lds16(qf + i * 512 + lane * 16);
        }
        float sf[NT][2];      // score factor of heads 8 nt + 2c, + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) sf[nt][x] = E4M3 ? scale2 / q_scale[nt * 8 + 2 * c + x] : scale2;

        float m[NT][2], l[NT][2], o[C::kTiles][NT][4];
        uint32_t ge[NT][2];   // e4m3: biased exponent of 2^(9 - r), the factor of a head's weights (r >= -100)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
            ge[nt][0] = ge[nt][1] = kMostFactor;
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
        }
        auto rescale = [&](int nt, float f0, float f1) {
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) {
                o[t][nt][0] *= f0;
                o[t][nt][1] *= f1;
                o[t][nt][2] *= f0;
                o[t][nt][3] *= f1;
            }
        };

        for (int j = 0, now = 0, next = stages - 1; j < n; ++j) {
            cp_wait(stages - 2);
            __syncwarp();
            issue(j + stages - 1, next, ahead);
            ahead = locate();
            const uint32_t st = mine + now * stage_bytes, sv = st + v_at, tail = sv + C::kRows;
            now = now + 1 == stages ? 0 : now + 1;
            next = next + 1 == stages ? 0 : next + 1;
            uint32_t mask;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(mask) : "r"(tail));

            float s[C::kM][NT][4];
#pragma unroll
            for (int tm = 0; tm < C::kM; ++tm)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[tm][nt][e] = 0.f;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                uint4 q[NT][C::kQPer];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < C::kQPer; ++x)
                        q[nt][x] = C::kQInRegs ? qr[C::kQInRegs ? (kb * NT + nt) * C::kQPer + x : 0]
                                               : lds16(qf + ((kb * NT + nt) * C::kQPer + x) * 512 + lane * 16);
#pragma unroll
                for (int tm = 0; tm < C::kM; ++tm) {
                    const uint4 k0 = lds16(st + piece_at(tm * 16 + entry_of<E4M3>(g), kb * 4 + c));
                    const uint4 k1 = lds16(st + piece_at(tm * 16 + entry_of<E4M3>(g + 8), kb * 4 + c));
                    if constexpr (E4M3) {
                        const uint32_t u0[4] = {k0.x, k0.y, k0.z, k0.w}, u1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t a0, a1, a2, a3;
                            e4m3_to_f16(u0[i], a0, a2);
                            e4m3_to_f16(u1[i], a1, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint4 qq = q[nt][i >> 1];
                                mma<true>(s[tm][nt], a0, a1, a2, a3, i & 1 ? qq.z : qq.x, i & 1 ? qq.w : qq.y);
                            }
                        }
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma<false>(s[tm][nt], k0.x, k1.x, k0.y, k1.y, q[nt][0].x, q[nt][0].y);
                            mma<false>(s[tm][nt], k0.z, k1.z, k0.w, k1.w, q[nt][0].z, q[nt][0].w);
                        }
                    }
                }
            }

            // scores in units of log2; entries that are not there get -infinity
            float vs[C::kM][2];
#pragma unroll
            for (int tm = 0; tm < C::kM; ++tm) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int r = tm * 16 + entry_of<E4M3>(g + 8 * y);
                    const bool ok = (mask >> r) & 1u;
                    const float ks = E4M3 ? lds_f(tail + 16 + r * 4) : 1.f;
                    vs[tm][y] = E4M3 ? lds_f(tail + 16 + (C::kStep + r) * 4) : 1.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float &v = s[tm][nt][2 * y + x];
                            v = ok ? v * (E4M3 ? ks * sf[nt][x] : sf[nt][x]) : -INFINITY;
                        }
                }
            }
            bool moved = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int tm = 0; tm < C::kM; ++tm)
                        moved |= fmaxf(s[tm][nt][x], s[tm][nt][2 + x]) > m[nt][x] + kLag;
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float alpha[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float v = m[nt][x];
#pragma unroll
                        for (int tm = 0; tm < C::kM; ++tm) v = fmaxf(v, fmaxf(s[tm][nt][x], s[tm][nt][2 + x]));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        const float fall = m[nt][x] - (v == -INFINITY ? 0.f : v);
                        alpha[x] = exp2_approx(fall);
                        m[nt][x] = v;
                        l[nt][x] *= alpha[x];
                        if constexpr (E4M3) {       // the reference of the products falls with the weights so far
                            const uint32_t to = min(ge[nt][x] + uint32_t(fminf(ceilf(-fall), 256.f)), kMostFactor);
                            alpha[x] = exp2_approx(fall + float(to - ge[nt][x]));
                            ge[nt][x] = to;
                        }
                    }
                    rescale(nt, alpha[0], alpha[1]);
                }
            }
            float ref[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) ref[nt][x] = m[nt][x] == -INFINITY ? 0.f : m[nt][x];
            uint32_t ph[C::kM][NT][2], pl[C::kM][NT][2];    // (pl: bf16 rows alone)
#pragma unroll
            for (int tm = 0; tm < C::kM; ++tm)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float p0 = exp2_approx(s[tm][nt][2 * y] - ref[nt][0]);
                        const float p1 = exp2_approx(s[tm][nt][2 * y + 1] - ref[nt][1]);
                        l[nt][0] += p0;
                        l[nt][1] += p1;
                        if constexpr (E4M3) {
                            s[tm][nt][2 * y] = p0 * vs[tm][y];
                            s[tm][nt][2 * y + 1] = p1 * vs[tm][y];
                        } else {
                            uint32_t h, r;
                            split_bf16(p0, p1, h, r);
                            ph[tm][nt][y] = movmatrix(h);
                            pl[tm][nt][y] = movmatrix(r);
                        }
                    }
            if constexpr (E4M3) {
                auto largest = [&](int nt, int x) {
                    float v = 0.f;
#pragma unroll
                    for (int tm = 0; tm < C::kM; ++tm) v = fmaxf(v, fmaxf(fabsf(s[tm][nt][x]), fabsf(s[tm][nt][2 + x])));
                    return v;
                };
                bool past = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) past |= largest(nt, x) * __uint_as_float(ge[nt][x] << 23) > kMostWeight;
                if (__any_sync(0xffffffffu, past)) {
                    // rows of zeros leave; of the others' products the largest is a head's new reference
                    uint32_t bits = 0;
#pragma unroll 1
                    for (int p = lane / C::kStep; p < nch; p += 32 / C::kStep) {
                        const uint4 v = lds16(sv + piece_at(lane % C::kStep, p));
                        bits |= (v.x | v.y) | (v.z | v.w);
                    }
                    uint32_t some = __ballot_sync(0xffffffffu, (bits & 0x7f7f7f7fu) != 0);
                    if (C::kStep == 16) some |= some >> 16;
#pragma unroll
                    for (int tm = 0; tm < C::kM; ++tm)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            if (!((some >> (tm * 16 + entry_of<E4M3>(g + 8 * y))) & 1u)) {
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) s[tm][nt][2 * y] = s[tm][nt][2 * y + 1] = 0.f;
                            }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float f[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float v = largest(nt, x);
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                            // 2^(9 - e) for a largest product of exponent e (e at most 127)
                            const uint32_t to = min(ge[nt][x], 127 + 9 + 127 - min(__float_as_uint(v) >> 23, 254u));
                            f[x] = __uint_as_float(uint32_t(max(127 - int(ge[nt][x] - to), 0)) << 23);
                            ge[nt][x] = to;
                        }
                        rescale(nt, f[0], f[1]);
                    }
                }
#pragma unroll
                for (int tm = 0; tm < C::kM; ++tm)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            ph[tm][nt][y] = movmatrix(pack_f16(s[tm][nt][2 * y] * __uint_as_float(ge[nt][0] << 23),
                                                               s[tm][nt][2 * y + 1] * __uint_as_float(ge[nt][1] << 23)));
            }
            if constexpr (E4M3) {
#pragma unroll
                for (int p = 0; p < C::kPass; ++p) {
#pragma unroll
                    for (int tm = 0; tm < C::kM; ++tm) {
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = tm * 16 + entry_of<E4M3>(2 * c + (i & 1) + 8 * (i >> 1));
                            v[i] = p * 8 + 7 < C::kPieces || p * 8 + g < C::kPieces ? lds16(sv + piece_at(r, p * 8 + g))
                                                                                 : make_uint4(0, 0, 0, 0);
                        }
                        const uint32_t v0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, v1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
                        const uint32_t v8[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, v9[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // bytes (e, e') of two entries: elements 4i, 4i + 1, then 4i + 2, 4i + 3
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t sel = y ? 0x7362 : 0x5140;
                                uint32_t a0, a1, a2, a3;
                                e4m3_to_f16(prmt(v0[i], v1[i], sel), a0, a1);
                                e4m3_to_f16(prmt(v8[i], v9[i], sel), a2, a3);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float(&d)[4] = o[p * 8 + 2 * i + y][nt];
                                    mma<true>(d, a0, a1, a2, a3, ph[tm][nt][0], ph[tm][nt][1]);
                                }
                            }
                        }
                    }
                }
            } else {
                // lane l gives the address of matrix l / 8's row l % 8: pieces 2t, 2t + 1 of entries 0 .. 7, then 8 .. 15
                const int r = entry_of<E4M3>((lane & 7) + 8 * (lane >> 4));
#pragma unroll
                for (int tm = 0; tm < C::kM; ++tm)
#pragma unroll
                    for (int t = 0; t < C::kTiles; ++t) {
                        uint32_t a0, a1, a2, a3;
                        ldmatrix_trans(sv + piece_at(tm * 16 + r, 2 * t + ((lane >> 3) & 1)), a0, a1, a2, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma<false>(o[t][nt], a0, a1, a2, a3, ph[tm][nt][0], ph[tm][nt][1]);
                            mma<false>(o[t][nt], a0, a1, a2, a3, pl[tm][nt][0], pl[tm][nt][1]);
                        }
                    }
            }
        }
        cp_wait(0);
        __syncthreads();      // the parts overlay every warp's stages
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int h = nt * 8 + 2 * c + x;
                float L = l[nt][x];
                L += __shfl_xor_sync(0xffffffffu, L, 4);
                L += __shfl_xor_sync(0xffffffffu, L, 8);
                L += __shfl_xor_sync(0xffffffffu, L, 16);
                if (g == 0) {
                    pml[(warp * C::kHeads + h) * 2] = m[nt][x];
                    pml[(warp * C::kHeads + h) * 2 + 1] = L;
                }
                float *part = po + (size_t(warp) * C::kHeads + h) * D;
                const float back = E4M3 ? __uint_as_float((254u - ge[nt][x]) << 23) : 1.f;      // 2^(r - 9)
#pragma unroll
                for (int t = 0; t < C::kTiles; ++t) {
                    if constexpr (E4M3) {
                        const int d = (t / 8 * 8 + g) * 16 + 2 * (t % 8);
                        if (d < D)
                            *reinterpret_cast<float2 *>(part + d) = make_float2(o[t][nt][x] * back, o[t][nt][2 + x] * back);
                    } else {
                        if (16 * t + g < D) part[16 * t + g] = o[t][nt][x];
                        if (16 * t + 8 + g < D) part[16 * t + 8 + g] = o[t][nt][2 + x];
                    }
                }
            }
        __syncthreads();
        finish_piece(a, b, hseg, slot, warps, po, pml);
        __syncthreads();
    };
    for_pieces(a, blockIdx.x, gridDim.x, scratch, do_piece);
    if (blockIdx.x == 0 && a.err)
        for (int b = threadIdx.x; b < a.B; b += blockDim.x)
            if (a.seq_len[b] > a.reach) raise_err(a.err, LSA_ERR_CAPACITY);
}

int blocks_of(const lsa_page_cache &c) {
    const int need = int((size_t(c.D) * elem_size(c.dtype) + 63) / 64);
    for (int k : {1, 2, 3, 4, 6, 8})
        if (need <= k) return k;
    return 16;
}

template <bool E4M3, int KB, int NT>
struct Run {
    static void plan(bool latent, int D, AttnPlan &p) {
        using C = Shape<E4M3, KB, NT>;
        const int stage = C::stage(latent);
        // two CTAs of four warps on an SM while three stages fit; else one, then one of two warps
        int warps = 4, ctas = 2;
        auto fit = [&](int budget) { return (budget - C::kQBytes) / (warps * stage); };
        int stages = fit(112 * 1024);
        if (stages < 3) {
            ctas = 1;
            stages = fit(222 * 1024);
            if (stages < 2) {
                warps = 2;
                stages = fit(222 * 1024);
            }
        }
        p.stages = stages > kMaxStages ? kMaxStages : stages;
        p.threads = warps * 32;
        p.tile = C::kStep * warps;
        p.lead = 3;
        p.grid = sm_count() * ctas;
        const size_t ring = size_t(p.stages) * warps * stage, join = size_t(warps) * C::kHeads * (D + 2) * 4;
        p.smem = C::kQBytes + (ring > join ? ring : join);
    }
    static lsa_status launch(const AttnArgs &a, const AttnPlan &p, int grid, cudaStream_t st) {
        LSA_CUDA(ensure_smem(paged_attn_mma<E4M3, KB, NT>, p.smem));
        LSA_CUDA(launch_pdl(paged_attn_mma<E4M3, KB, NT>, dim3(grid), dim3(p.threads), p.smem, st, a, int(p.stages)));
        LSA_LAUNCHED(E4M3 ? "paged_attn_mma e4m3" : "paged_attn_mma bf16");
        return LSA_OK;
    }
};

// Calls f with the kernel's shape: Run<type, blocks of a row, head groups>.
template <bool E4M3, int KB, typename F>
auto with_heads(int nt, F f) {
    constexpr int kMost = (E4M3 ? KB * 64 : KB * 32) <= 128 ? 4 : (E4M3 ? KB * 64 : KB * 32) <= 256 ? 2 : 1;
    if constexpr (kMost >= 4)
        if (nt > 2) return f(Run<E4M3, KB, 4>());
    if constexpr (kMost >= 2)
        if (nt > 1) return f(Run<E4M3, KB, 2>());
    return f(Run<E4M3, KB, 1>());
}
template <bool E4M3, typename F>
auto with_shape(int kb, int nt, F f) {
    switch (kb) {
    case 1: return with_heads<E4M3, 1>(nt, f);
    case 2: return with_heads<E4M3, 2>(nt, f);
    case 3: return with_heads<E4M3, 3>(nt, f);
    case 4: return with_heads<E4M3, 4>(nt, f);
    case 6: return with_heads<E4M3, 6>(nt, f);
    case 8: return with_heads<E4M3, 8>(nt, f);
    default:
        // (e4m3 rows end at 8 blocks)
        return with_heads<E4M3, E4M3 ? 8 : 16>(nt, f);
    }
}

}  // namespace

AttnPlan plan_mma(const lsa_page_cache &c, int Hq) {
    AttnPlan p = {};
    const int G = Hq / c.Hkv, kb = blocks_of(c), width = kb * (c.dtype == LSA_E4M3 ? 64 : 32);
    const int most = width <= 128 ? 32 : width <= 256 ? 16 : 8;   // query heads whose o fits in registers
    p.HG = (G + most - 1) / most;
    const int per = (G + p.HG - 1) / p.HG, nt = per <= 8 ? 1 : per <= 16 ? 2 : 4;
    p.HS = 8 * nt;
    p.HG = (G + p.HS - 1) / p.HS;
    const bool latent = c.v == c.k;
    auto f = [&](auto run) { run.plan(latent, c.D, p); };
    if (c.dtype == LSA_E4M3) with_shape<true>(kb, nt, f);
    else with_shape<false>(kb, nt, f);
    return p;
}

lsa_status launch_mma(const lsa_page_cache &c, const AttnArgs &a, const AttnPlan &p, int grid, cudaStream_t st) {
    const int kb = blocks_of(c), nt = p.HS / 8;
    auto f = [&](auto run) { return run.launch(a, p, grid, st); };
    return c.dtype == LSA_E4M3 ? with_shape<true>(kb, nt, f) : with_shape<false>(kb, nt, f);
}

}  // namespace paged
}  // namespace lsa
